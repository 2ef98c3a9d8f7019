// The adapter term of a 16-row MFMA epilogue: acc += h . B[l]^T for the rows of
// each adapter l, in the accumulators of a projection kernel, before its one
// rounding (lora.hip states the operation and forms h).
#pragma once

#include <cfloat>
#include <utility>

#include "common.hpp"

namespace w4a16 {

constexpr int kLoraMaxRank = 128;

struct LoraArgs {
  const uint16_t* h;    // [2, M, R] bf16: h as its rounding and the rounding of what is left
  const uint16_t* b;    // [L, N, R] bf16
  const int32_t* ids;   // [M], outside [0, L): no adapter
  int M, N, L, R;
};

// f(0) ... f(N - 1) with constant indices, whatever the size of the body (the
// compiler left the loop over the row tiles rolled in some instances, their
// accumulators indexed at run time)
template <class F, int... I>
__device__ __forceinline__ void static_for_each(std::integer_sequence<int, I...>, F f) {
  (f(std::integral_constant<int, I>{}), ...);
}
template <int N, class F>
__device__ __forceinline__ void static_for(F f) {
  static_for_each(std::make_integer_sequence<int, N>{}, f);
}

// The adapters of the rows of a 16 MS-row tile, one after another: id[q] is the
// adapter of row 64 q + lane (-1: none).
template <int MS>
struct LoraRows {
  static constexpr int Q = (16 * MS + 63) / 64;
  uint64_t todo[Q];
  int turn;
  __device__ __forceinline__ void reset(const int (&id)[Q]) {
#pragma unroll
    for (int q = 0; q < Q; ++q) todo[q] = __ballot(id[q] >= 0);
    turn = 0;
  }
  // The next adapter (in the order of their first row) whose turn is `part` of
  // `nparts`: its id, or -1 when none is left, and its rows.
  __device__ __forceinline__ int next(const int (&id)[Q], uint64_t (&rows)[Q], int part, int nparts) {
    for (;;) {
      int l = -1;
#pragma unroll
      for (int q = Q - 1; q >= 0; --q)
        if (todo[q] != 0) l = __builtin_amdgcn_readlane(id[q], __builtin_ctzll(todo[q]));
      if (l < 0) return -1;
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        rows[q] = __ballot(id[q] == l);
        todo[q] &= ~rows[q];
      }
      const bool own = turn == part;
      turn = turn + 1 == nparts ? 0 : turn + 1;
      if (own) return l;
    }
  }
};

// B fragments of adapter l: column n0 + 16 ns + lane % 16, ranks 32 st + 8
// (lane / 16) + 0..7; zeros past N and past R.
template <int SN, int NS>
__device__ __forceinline__ void lora_load_b(bf16x8 (&bf)[NS][SN], const LoraArgs& la, int l, int n0, int lane) {
  const int m16 = lane & 15, kb = lane >> 4;
  const __amdgpu_buffer_rsrc_t rbuf =
      make_rsrc(la.b + (size_t)l * la.N * la.R, (uint32_t)la.N * (uint32_t)la.R * 2u);
#pragma unroll
  for (int st = 0; st < NS; ++st)
#pragma unroll
    for (int ns = 0; ns < SN; ++ns) {
      const int n = n0 + 16 * ns + m16, r = 32 * st + 8 * kb;
      const uint32_t off = r < la.R && n < la.N ? ((uint32_t)n * (uint32_t)la.R + (uint32_t)r) * 2u : 0xFFFFFFF0u;
      bf[st][ns] = __builtin_bit_cast(bf16x8, ld128(rbuf, off));
    }
}

// acc += h . B^T for the rows `mine` (bit 4 (lane / 16) + i: the lane's row i).
// The product is formed apart and selected by row, so that another adapter's
// infinities or NaN reach no row. The second parts of h come first: an infinite
// element of B makes their sum NaN or infinite (0 * infinity, or a sign that is
// not the first part's), where the first parts alone give what is right; so
// that sum is brought to a finite value by v_med3, which leaves finite ones as
// they are (any value: the first parts' sum is infinite or NaN then; where the
// second parts overflow by themselves, a product of the first, at least 2^8
// times as large, does too). Up to 2 % of a call: 1000 x 5120 x 5120, rank 128,
// 8 adapters mixed 116.8 -> 119.0 us, one after the other 92.4 -> 94.1, 1322 x
// 19456 x 2560, rank 64, 4 mixed 185.1 -> 187.0, one after the other and small
// batches within 0.3 us (a compare and a select in its place 190.0 for the 4
// mixed; a test of each adapter's B for infinities and a clear only then 121.3
// for the 8).
template <int SN, int NS>
__device__ __forceinline__ void lora_mac(f32x4 (&acc)[SN], const u32x4 (&hi)[NS], const u32x4 (&lo)[NS],
                                         const bf16x8 (&bf)[NS][SN], uint32_t mine, int kb) {
  f32x4 d[SN];
#pragma unroll
  for (int ns = 0; ns < SN; ++ns) d[ns] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int st = 0; st < NS; ++st)
#pragma unroll
    for (int ns = 0; ns < SN; ++ns)
      d[ns] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, lo[st]), bf[st][ns], d[ns], 0, 0, 0);
#pragma unroll
  for (int ns = 0; ns < SN; ++ns)
#pragma unroll
    for (int i = 0; i < 4; ++i) d[ns][i] = __builtin_amdgcn_fmed3f(d[ns][i], -FLT_MAX, FLT_MAX);
#pragma unroll
  for (int st = 0; st < NS; ++st)
#pragma unroll
    for (int ns = 0; ns < SN; ++ns)
      d[ns] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, hi[st]), bf[st][ns], d[ns], 0, 0, 0);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const bool own = (mine >> (4 * kb + i)) & 1;
#pragma unroll
    for (int ns = 0; ns < SN; ++ns) acc[ns][i] += own ? d[ns][i] : 0.0f;
  }
}

// ---- tile kernels: h of the tile's rows in LDS, read by every wave. The two
// parts lie in two of the pipeline's stages, which are free while the last
// group is computed; the DMA that fills them is issued ahead of that group, so
// that its flight is covered (h staged through registers behind the last
// barrier: three tile rounds of 1322 x 19456 x 2560, rank 64, 2-3 us longer).
// Row r holds the ranks up to 32 NS (zeros past R) in 16-byte chunks, chunk c
// in slot c ^ lora_swz(r): the 16 rows of a fragment read (chunks 4 st + 0..3)
// then cover all banks evenly.
__device__ __forceinline__ int lora_swz(int r, int lg) {   // NS = 1 << lg
  return lg == 0 ? 0 : lg == 1 ? 4 * ((r >> 1) & 1) : 4 * (r & 3);
}
__device__ __forceinline__ int lora_lg(int R) { return R <= 32 ? 0 : R <= 64 ? 1 : 2; }
// a part of h, then (behind the first part) the rows' adapters
constexpr int lora_plane_bytes(int rows) { return rows * 2 * kLoraMaxRank + (rows + 63) / 64 * 256; }

// 1 KiB DMA instructions, dealt out over NW waves; rows past `live` and ranks
// past R are zeros (past the extent).
template <int MS, int NW>
__device__ __forceinline__ void lora_tile_fetch(uint8_t* hi, uint8_t* lo, const LoraArgs& la, int row0, int live,
                                                int lane, int wv) {
  const int lg = lora_lg(la.R);
  const uint32_t plane = (uint32_t)la.M * (uint32_t)la.R * 2u;
  const __amdgpu_buffer_rsrc_t rh = make_rsrc(la.h, 2u * plane);
  for (int q = wv; q < MS << lg; q += NW) {
    const int i = 64 * q + lane, r = i >> (2 + lg), c = (i & ((4 << lg) - 1)) ^ lora_swz(r, lg);
    const bool ok = r < live && 8 * c < la.R;
    const uint32_t off = ((uint32_t)(row0 + r) * (uint32_t)la.R + 8u * (uint32_t)c) * 2u;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rh, (__attribute__((address_space(3))) void*)(hi + 1024 * q), 16,
                                             ok ? off : 0xFFFFFFF0u, 0, 0, 0);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rh, (__attribute__((address_space(3))) void*)(lo + 1024 * q), 16,
                                             ok ? plane + off : 0xFFFFFFF0u, 0, 0, 0);
  }
  // rows past M: zeros, which lora_tile_add does not look at
  if (wv < LoraRows<MS>::Q)
    __builtin_amdgcn_raw_ptr_buffer_load_lds(make_rsrc(la.ids, (uint32_t)la.M * 4u),
                                             (__attribute__((address_space(3))) void*)(hi + 4096 * MS + 256 * wv), 4,
                                             4u * (uint32_t)(row0 + 64 * wv + lane), 0, 0, 0);
}

template <int MS, int SN, int NS>
__device__ __forceinline__ void lora_tile_ns(f32x4 (&acc)[MS][SN], const uint8_t* hi, const uint8_t* lo,
                                             const int (&id)[LoraRows<MS>::Q], const LoraArgs& la, int n0, int lane,
                                             int part, int nparts) {
  // adapters whose B fragments are in flight at once: 4 fragment steps of them
  // (with 2 and 8: 200 x 4096 x 4096, rank 32, an adapter each 52.0, 50.7, 50.4
  // us, rank 128, an adapter each 107.1, 106.1, 108.4; 1322 x 19456 x 2560, rank
  // 64, 4 mixed 179.1, 181.3, 186.6)
  constexpr int NB = 4 / NS, Q = LoraRows<MS>::Q, LG = NS == 1 ? 0 : NS == 2 ? 1 : 2;
  const int m16 = lane & 15, kb = lane >> 4;
  LoraRows<MS> adapters;
  adapters.reset(id);
  // rows 16 ms + m16 share m16's swizzle: chunk 4 st + kb of row tile ms is
  // 64 NS * 16 ms + 64 (st ^ swizzle / 4) behind the lane's row
  uint32_t at[NS];
#pragma unroll
  for (int st = 0; st < NS; ++st)
    at[st] = (uint32_t)m16 * (64u * NS) + 16u * (uint32_t)((4 * st + kb) ^ lora_swz(m16, LG));
  for (;;) {
    int l[NB];
    uint64_t rows[NB][Q];
    bf16x8 bf[NB][NS][SN];
#pragma unroll
    for (int k = 0; k < NB; ++k) {
      l[k] = (k == 0 || l[k > 0 ? k - 1 : 0] >= 0) ? adapters.next(id, rows[k], part, nparts) : -1;
      if (l[k] >= 0) lora_load_b<SN, NS>(bf[k], la, l[k], n0, lane);
    }
#pragma unroll
    for (int k = 0; k < NB; ++k) {
      if (l[k] < 0) return;
      static_for<MS>([&](auto i) {
        constexpr int ms = decltype(i)::value;
        const uint32_t mine = (uint32_t)(rows[k][ms / 4] >> (16 * (ms % 4))) & 0xFFFFu;
        if (mine != 0) {
          u32x4 h[NS], g[NS];
#pragma unroll
          for (int st = 0; st < NS; ++st) g[st] = *reinterpret_cast<const u32x4*>(lo + at[st] + 1024 * NS * ms);
#pragma unroll
          for (int st = 0; st < NS; ++st) h[st] = *reinterpret_cast<const u32x4*>(hi + at[st] + 1024 * NS * ms);
          lora_mac<SN, NS>(acc[ms], h, g, bf[k], mine, kb);
        }
      });
    }
  }
}

// behind a wait for the DMA and a barrier; part = K slice of nparts, so that
// the slices share the adapters
template <int MS, int SN>
__device__ __forceinline__ void lora_tile_add(f32x4 (&acc)[MS][SN], const uint8_t* hi, const uint8_t* lo,
                                              const LoraArgs& la, int live, int n0, int lane, int part, int nparts) {
  int id[LoraRows<MS>::Q];
#pragma unroll
  for (int q = 0; q < LoraRows<MS>::Q; ++q) {
    const int i = reinterpret_cast<const int*>(hi + 4096 * MS)[64 * q + lane];
    id[q] = 64 * q + lane < live && (uint32_t)i < (uint32_t)la.L ? i : -1;
  }
  if (la.R <= 32) lora_tile_ns<MS, SN, 1>(acc, hi, lo, id, la, n0, lane, part, nparts);
  else if (la.R <= 64) lora_tile_ns<MS, SN, 2>(acc, hi, lo, id, la, n0, lane, part, nparts);
  else lora_tile_ns<MS, SN, 4>(acc, hi, lo, id, la, n0, lane, part, nparts);
}

// ---- small batch (M <= 16 MS rows): h read straight into the fragments by the
// waves that hold an adapter, `part` of `nparts`; 4 / NS adapters' B fragments
// are in flight at once, together with h of their rows (with half as many, and
// twice: 5 x 17408 x 5120, rank 16, an adapter each 24.9, 21.4, 21.5 us, 24 x
// 17408 x 5120 46.0, 43.4, 44.8, 16 x 8192 x 8192, rank 64 23.4, 22.5, 22.4).
// begin() requests them; add() uses them, and goes on with the adapters that
// are left.

// the adapter of row `lane`: a load at the kernel's start, used at its end
__device__ __forceinline__ int lora_id(const LoraArgs& la, int lane) { return lane < la.M ? la.ids[lane] : -1; }

template <int MS, int SN, int NS>
struct LoraSmall {
  static_assert(MS <= 4, "one row per lane");
  static constexpr int NB = 4 / NS;
  int id[1];
  LoraRows<MS> adapters;   // from begin() on
  int l[NB];
  uint64_t rows[NB][1];
  bf16x8 bf[NB][NS][SN];
  u32x4 hi[MS][NS], lo[MS][NS];

  // (here row_id is waited for)
  __device__ __forceinline__ void begin(const LoraArgs& la, int row_id, int n0, int lane, int part, int nparts) {
    id[0] = lane < 16 * MS && (uint32_t)row_id < (uint32_t)la.L ? row_id : -1;
    adapters.reset(id);
    start(la, n0, lane, part, nparts);
  }

  // the next adapters' B, and h of their rows (the other rows' loads go past
  // the extent and move nothing)
  __device__ __forceinline__ void start(const LoraArgs& la, int n0, int lane, int part, int nparts) {
    uint64_t own = 0;
#pragma unroll
    for (int k = 0; k < NB; ++k) {
      l[k] = (k == 0 || l[k > 0 ? k - 1 : 0] >= 0) ? adapters.next(id, rows[k], part, nparts) : -1;
      if (l[k] >= 0) {
        lora_load_b<SN, NS>(bf[k], la, l[k], n0, lane);
        own |= rows[k][0];
      }
    }
    if (l[0] < 0) return;
    const int m16 = lane & 15, kb = lane >> 4;
    const uint32_t plane = (uint32_t)la.M * (uint32_t)la.R * 2u;
    const __amdgpu_buffer_rsrc_t rh = make_rsrc(la.h, 2u * plane);
#pragma unroll
    for (int ms = 0; ms < MS; ++ms)
#pragma unroll
      for (int st = 0; st < NS; ++st) {
        const int r = 32 * st + 8 * kb, m = 16 * ms + m16;
        const bool ok = ((own >> m) & 1) && r < la.R;
        const uint32_t off = ((uint32_t)m * (uint32_t)la.R + (uint32_t)r) * 2u;
        hi[ms][st] = ld128(rh, ok ? off : 0xFFFFFFF0u);
        lo[ms][st] = ld128(rh, ok ? plane + off : 0xFFFFFFF0u);
      }
  }

  __device__ __forceinline__ void add(f32x4 (&acc)[MS][SN], const LoraArgs& la, int n0, int lane, int part,
                                      int nparts) {
    while (l[0] >= 0) {
#pragma unroll
      for (int k = 0; k < NB; ++k) {
        if (l[k] < 0) return;
        static_for<MS>([&](auto i) {
          constexpr int ms = decltype(i)::value;
          const uint32_t mine = (uint32_t)(rows[k][0] >> (16 * ms)) & 0xFFFFu;
          if (mine != 0) lora_mac<SN, NS>(acc[ms], hi[ms], lo[ms], bf[k], mine, lane >> 4);
        });
      }
      start(la, n0, lane, part, nparts);
    }
  }
};

// fragment steps of a rank
inline int lora_steps(int R) { return R <= 32 ? 1 : R <= 64 ? 2 : 4; }

}  // namespace w4a16
