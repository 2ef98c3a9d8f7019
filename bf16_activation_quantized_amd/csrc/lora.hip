// Low-rank adapters of many requests beside the shared W4A16 projection:
//
//   h[m, r] = sc[l] * sum_k x[m, k] A[l, r, k],  l = ids[m]
//   y[m, n] = bf16(base[m, n] + sum_r h[m, r] B[l, n, r])
//
// The kernels here form h, the first product; the second joins the fp32
// accumulators of the projection's own kernels (lora.hpp), so y is written
// once and rounded once. There h enters the matrix core as two bf16 values
// (its rounding and the rounding of what is left: 16 of its bits). Rows whose
// id is outside [0, L) get the projection alone.
#include <algorithm>

#include "common.hpp"
#include "launch.hpp"
#include "lora.hpp"
#include "rowsum.hpp"

namespace w4a16 {

namespace {

__device__ __forceinline__ bf16x8 frag(u32x4 v) { return __builtin_bit_cast(bf16x8, v); }

constexpr int kWaves = 8;   // per workgroup, in every kernel here

constexpr uint32_t kOutside = 0xFFFFFFF0u;   // a buffer offset past every extent: the load returns zeros

// An element of h as its rounding to bf16 and the rounding of what is left. A
// finite element that rounds to infinity (past the largest bf16, 255 * 2^120)
// is that largest value and what is left of it, cut off so that the two do not
// add up to infinity either (off by less than 2^112, 2^-16 of it); the second
// part of an infinite one is 0, where infinity - infinity would be NaN.
__device__ __forceinline__ void store_h(uint16_t* h, size_t plane, size_t e, float v) {
  uint16_t hi = to_bf16(v);
  const bool past = (hi & 0x7FFFu) == 0x7F80u, finite = fabsf(v) < __builtin_inff();
  if (past && finite) hi -= 1;
  const float left = v - bf16f(hi);
  h[e] = hi;
  h[plane + e] = !past ? to_bf16(left) : finite ? (uint16_t)(__float_as_uint(left) >> 16) : (uint16_t)0;
}

}  // namespace

// ---------------------------------------------------------------- few rows
// Workgroup (row, RP ranks): dot products on the VALU. The 8 waves take 512-k
// pieces in turn (one contiguous 1 KiB run of x and of each rank's row of A
// per wave instruction), two pieces in flight, and are summed through LDS in
// wave order.
constexpr int kRowWaves = kWaves;

template <int RP>
__device__ __forceinline__ void shrink_row(const uint16_t* __restrict__ x, const uint16_t* __restrict__ a,
                                           const int32_t* __restrict__ ids, const float* __restrict__ scaling,
                                           uint16_t* __restrict__ h, int M, int K, int L, int R, int block) {
  __shared__ float red[kRowWaves][RP];
  const int lane = threadIdx.x & 63;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int per_row = R / RP, m = block / per_row, r0 = (block - m * per_row) * RP;
  const int l = __builtin_amdgcn_readfirstlane(ids[m]);
  if ((uint32_t)l >= (uint32_t)L) return;
  const uint32_t KB = (uint32_t)K * 2u;
  const __amdgpu_buffer_rsrc_t rx = make_rsrc(x + (size_t)m * K, KB);
  const __amdgpu_buffer_rsrc_t ra = make_rsrc(a + ((size_t)l * R + r0) * K, (uint32_t)RP * KB);
  float acc[RP];
#pragma unroll
  for (int r = 0; r < RP; ++r) acc[r] = 0.0f;
  u32x4 xv[2], av[2][RP];
  const int pieces = (K + 511) / 512;
  auto issue = [&](int u, int c) {
    const uint32_t o = 1024u * (uint32_t)c + 16u * (uint32_t)lane;
    const bool ok = c < pieces && o < KB;   // past the row: zeros
    xv[u] = ld128(rx, ok ? o : kOutside);
#pragma unroll
    for (int r = 0; r < RP; ++r) av[u][r] = ld128(ra, ok ? o + (uint32_t)r * KB : kOutside);
    __builtin_amdgcn_sched_barrier(0);   // one piece's loads together: waits are exact counts
  };
  auto add = [&](int u) {
    const u32x4 v = xv[u];
#pragma unroll
    for (int r = 0; r < RP; ++r) {
      const u32x4 w = av[u][r];
      acc[r] = __builtin_amdgcn_fdot2_f32_bf16(as_bf16x2(v.x), as_bf16x2(w.x), acc[r], false);
      acc[r] = __builtin_amdgcn_fdot2_f32_bf16(as_bf16x2(v.y), as_bf16x2(w.y), acc[r], false);
      acc[r] = __builtin_amdgcn_fdot2_f32_bf16(as_bf16x2(v.z), as_bf16x2(w.z), acc[r], false);
      acc[r] = __builtin_amdgcn_fdot2_f32_bf16(as_bf16x2(v.w), as_bf16x2(w.w), acc[r], false);
    }
  };
  issue(0, wv);
  for (int c = wv; c < pieces; c += 2 * kRowWaves) {
    issue(1, c + kRowWaves);
    add(0);
    issue(0, c + 2 * kRowWaves);
    add(1);
  }
#pragma unroll
  for (int r = 0; r < RP; ++r) {
    const float s = wave64_sum(acc[r]);
    if (lane == 63) red[wv][r] = s;
  }
  __syncthreads();
  if (threadIdx.x < RP) {
    float s = red[0][threadIdx.x];
#pragma unroll
    for (int q = 1; q < kRowWaves; ++q) s += red[q][threadIdx.x];
    if (scaling != nullptr) s *= scaling[l];
    store_h(h, (size_t)M * R, (size_t)m * R + r0 + threadIdx.x, s);
  }
}

// ---------------------------------------------------------------- many rows
// Workgroup (turn, block of 64 rows, rank tile of 16): MFMA 16x16x32 over the
// whole K range, for every turns-th unit of the block. A unit is up to 16 rows
// of one adapter, wherever they lie in the block, in the order of their first
// rows; so the rows of a request, one after another, are units of 16, and A is
// read once per block for an adapter whose rows are strewn over it (against
// 16-row tiles, this kernel: 2048 x 5120 x 5120, rank 64, 16 adapters mixed 54
// -> 45 us, 512 x 8192 x 8192, rank 64, 8 mixed 26.5 -> 14.7; one after the
// other 12.2 -> 9.6). Bound by its round trips where units are few (1322 rows,
// rank 64, with the row sums: 9.8 us), by reading x and A again from the
// caches where they are many (11 TB/s at 4096 rows, rank 128). The 8 waves take the 128-k groups in turn; a group of x
// and of A is fetched in whole lines (4 rows x 256 bytes per instruction) and
// turned into fragments through the wave's own LDS tile, two fetches ahead.
// The waves are summed through LDS in wave order.
constexpr int kTileWaves = kWaves;
constexpr int kUnitBlock = 64;   // rows: one per lane

__device__ __forceinline__ void shrink_tile(const uint16_t* __restrict__ x, const uint16_t* __restrict__ a,
                                            const int32_t* __restrict__ ids, const float* __restrict__ scaling,
                                            uint16_t* __restrict__ h, int M, int K, int L, int R, int block,
                                            int turns, int bits) {
  __shared__ u32x4 tile[kTileWaves][16 * 16];   // [row][piece p of a group in slot p ^ row]
  __shared__ f32x4 red[2][kTileWaves][64];
  const int lane = threadIdx.x & 63;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int m16 = lane & 15, kb = lane >> 4;
  const int rt = (R + 15) / 16, mt = (M + kUnitBlock - 1) / kUnitBlock;
  // the rank tiles of a unit follow one another on one XCD (workgroups go
  // round the 8 of them), whose L2 then holds its rows of x
  const int at = block / (8 * rt) * 8 + block % 8;
  const int r0 = block % (8 * rt) / 8 * 16, m0 = at % mt * kUnitBlock, me = at / mt;
  if (me >= turns) return;   // the grid's last workgroups
  const int Gk = K / kGroup;
  const uint32_t KB = (uint32_t)K * 2u;
  int id = m0 + lane < M ? ids[m0 + lane] : -1;
  id = (uint32_t)id < (uint32_t)L ? id : -1;

  // the rows of the lane's adapter, the lane's place among them, and the units' first rows
  uint64_t same = __ballot(id >= 0);
  for (int b = 0; b < bits; ++b) {
    const bool one = (id >> b) & 1;
    const uint64_t v = __ballot(one);
    same &= one ? v : ~v;
  }
  const int place = (int)__popcll(same & ((1ull << lane) - 1));
  uint64_t todo = __ballot(id >= 0 && place % 16 == 0);
  for (int i = 0; i < me; ++i) todo &= todo - 1;   // (0 stays 0)

  const __amdgpu_buffer_rsrc_t rx =
      make_rsrc(x + (size_t)m0 * K, (uint32_t)min(kUnitBlock, M - m0) * KB);
  const uint32_t piece = 16u * (uint32_t)m16;   // of a group
  u32x4* tw = tile[wv];
  // lane (m16, kb) of step j: row m16, piece 4 kb + j (k = 32 kb + 8 j + 0..7, the same in both operands)
  auto turned = [&](const u32x4 (&v)[4], u32x4 (&f)[4]) {
    wave_lds_exchange();
#pragma unroll
    for (int j = 0; j < 4; ++j) tw[16 * (4 * j + kb) + (m16 ^ (4 * j + kb))] = v[j];
    wave_lds_exchange();
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = tw[16 * m16 + ((4 * kb + j) ^ m16)];
  };

  for (int parity = 0; todo != 0; parity ^= 1) {   // the same in every wave
    const int first = __builtin_ctzll(todo);
    const int l = __builtin_amdgcn_readlane(id, first);
    const int from = __builtin_amdgcn_readlane(place, first);
    const bool own = id == l && place >= from && place < from + 16;
    const int count = (int)__popcll(__ballot(own));
    // lane i < count: the unit's row i (the others are sent to lanes past the 16th)
    const int row = __builtin_amdgcn_ds_permute(4 * (own ? place - from : 16 + (lane & 31)), lane);
    // row (rank) 4 j + kb, 16-byte piece m16 of a group; zeros past the unit's rows and past R
    uint32_t xo[4], ao[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int r = __shfl(row, 4 * j + kb);
      xo[j] = 4 * j + kb < count ? (uint32_t)r * KB + piece : kOutside;
      ao[j] = r0 + 4 * j + kb < R ? (uint32_t)(4 * j + kb) * KB + piece : kOutside;
    }
    const __amdgpu_buffer_rsrc_t ra = make_rsrc(a + ((size_t)l * R + r0) * K, (uint32_t)min(16, R - r0) * KB);
    struct Item {
      u32x4 xv[4], av[4];
    };
    auto fetch = [&](Item& t, int g) {
      const uint32_t o = g < Gk ? (uint32_t)g * 256u : kOutside;   // past K: zeros
#pragma unroll
      for (int j = 0; j < 4; ++j) t.av[j] = ld128(ra, __builtin_elementwise_add_sat(ao[j], o));
#pragma unroll
      for (int j = 0; j < 4; ++j) t.xv[j] = ld128(rx, __builtin_elementwise_add_sat(xo[j], o));
      __builtin_amdgcn_sched_barrier(0);   // one fetch's loads stay together
    };
    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
    auto use = [&](const Item& t) {
      u32x4 xf[4], af[4];
      turned(t.xv, xf);
      turned(t.av, af);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(frag(xf[j]), frag(af[j]), acc, 0, 0, 0);
    };
    Item t0, t1;
    fetch(t0, wv);
    fetch(t1, wv + kTileWaves);
    for (int g = wv; g < Gk; g += 2 * kTileWaves) {
      use(t0);
      fetch(t0, g + 2 * kTileWaves);
      use(t1);
      fetch(t1, g + 3 * kTileWaves);
    }
    red[parity][wv][lane] = acc;
    __syncthreads();   // (the other half is written while wave 0 reads this one)
    if (wv == 0) {
      f32x4 v = red[parity][0][lane];
#pragma unroll
      for (int q = 1; q < kTileWaves; ++q) {
        const f32x4 p = red[parity][q][lane];
        v.x += p.x;
        v.y += p.y;
        v.z += p.z;
        v.w += p.w;
      }
      const float sc = scaling != nullptr ? scaling[l] : 1.0f;
      // lane: rows 4 kb + i, rank r0 + m16 (every lane is active where their places are read)
      const float f[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int m = m0 + __shfl(row, 4 * kb + i);
        if (4 * kb + i < count && r0 + m16 < R) store_h(h, (size_t)M * R, (size_t)m * R + r0 + m16, sc * f[i]);
      }
    }
    for (int i = 0; i < turns; ++i) todo &= todo - 1;
  }
}

// ---------------------------------------------------------------- launch
// The first workgroups form the tile kernel's row sums of X where it wants
// them from ahead (8 rows each; GS = 0: none): both passes read x and neither
// waits for the other (two launches cost about 4 us more).
struct ShrinkArgs {
  const uint16_t* x;
  const uint16_t* a;
  const int32_t* ids;
  const float* scaling;
  uint16_t* h;
  float* rowsums;
  int M, K, L, R, ld, rowsum_blocks, turns, bits;
};

template <int GS>
__device__ __forceinline__ bool rowsum_block(const ShrinkArgs& p) {
  if constexpr (GS != 0) {
    if ((int)blockIdx.x < p.rowsum_blocks) {
      rowsum_neg136_row<GS>(p.x, p.rowsums, blockIdx.x * kWaves + (threadIdx.x >> 6), p.M, p.K, p.ld,
                            threadIdx.x & 63);
      return true;
    }
  }
  return false;
}

template <int RP, int GS>
__global__ __launch_bounds__(64 * kWaves) void lora_shrink_row_kernel(const ShrinkArgs p) {
  if (rowsum_block<GS>(p)) return;
  shrink_row<RP>(p.x, p.a, p.ids, p.scaling, p.h, p.M, p.K, p.L, p.R, (int)blockIdx.x - p.rowsum_blocks);
}

template <int GS>
__global__ __launch_bounds__(64 * kWaves, 4) void lora_shrink_tile_kernel(const ShrinkArgs p) {
  if (rowsum_block<GS>(p)) return;
  shrink_tile(p.x, p.a, p.ids, p.scaling, p.h, p.M, p.K, p.L, p.R, (int)blockIdx.x - p.rowsum_blocks, p.turns,
              p.bits);
}

// Few rows one by one, more in units: the row kernel reads A once per row,
// the tile kernel once per unit of 16, but through fewer workgroups and in
// shorter runs. The whole call, row against tile kernel: 64 x 8192 x
// 8192, rank 16, an adapter each 36.9 / 40.3 us, 4 adapters one after the other
// 28.5 / 32.4; rank 64, 64 adapters 50.0 / 53.6, 4 adapters 30.9 / 32.9; 100 x
// 8192 x 4096, rank 64, 8 adapters, mixed 33.1 / 30.8, one after the other 31.9
// / 29.9; 333 x 2560 x 9728, group 32, rank 24, 5 adapters, mixed 54.9 / 50.3;
// 1000 x 5120 x 5120, rank 8, 8 mixed 91.7 / 88.0. Past the border the row
// kernel still wins where every row has an adapter of its own (64 x 4096 x
// 9728, rank 128: 63.7 / 68.1; 4 adapters 36.1 / 34.2), which the host does not
// know.
// Turns: as many as a block can have units, up to about a thousand workgroups,
// but four at least; a workgroup that finds no unit left to it ends at once.
template <int GS>
static hipError_t launch_shrink_gs(ShrinkArgs p, hipStream_t stream) {
  p.rowsum_blocks = GS != 0 ? (p.M + kWaves - 1) / kWaves : 0;
  p.turns = 1;
  const int64_t MR = (int64_t)p.M * p.R;
  const dim3 threads(64 * kWaves);
  if (MR <= 4096) {
#define W4A16_ROW(RP) \
  hipLaunchKernelGGL((lora_shrink_row_kernel<RP, GS>), dim3(p.rowsum_blocks + p.M * (p.R / RP)), threads, 0, stream, p)
    // Ranks per workgroup: x is read once for all of them, against the number of
    // workgroups. The whole call with 1, 2, 4 (and 8) ranks: 16 x 4096 x 4096,
    // rank 16, an adapter each 12.7, 12.8, 13.2 (13.8) us, 1 x 17408 x 5120,
    // rank 16 12.9, 13.0, 13.2 (13.9); 64 x 8192 x 8192, rank 64, an adapter
    // each 52.4, 50.6, 51.8 (53.4), 4 adapters one after the other 33.2, 30.9,
    // 30.7 (31.6); 120 x 2560 x 9728, group 32, rank 32, 5 mixed 40.0, 37.7,
    // 39.0 (four wins by 2 % at most, where it does).
    if (MR >= 512) W4A16_ROW(2);
    else W4A16_ROW(1);
#undef W4A16_ROW
    return hipGetLastError();
  }
  const int64_t mt = (p.M + kUnitBlock - 1) / kUnitBlock, rt = (p.R + 15) / 16;
  // units of a block: at most 64, and 64 / 16 + 15 / 16 for each adapter
  const int64_t units = std::min(kUnitBlock, 4 + std::min(p.L, kUnitBlock) * 15 / 16);
  p.turns = (int)std::min(units, std::max<int64_t>(4, 1024 / (mt * rt)));
  p.bits = 1;
  while (p.bits < 31 && (1 << p.bits) < p.L) ++p.bits;
  const int64_t blocks = p.rowsum_blocks + rt * ((mt * p.turns + 7) / 8 * 8);
  hipLaunchKernelGGL((lora_shrink_tile_kernel<GS>), dim3((unsigned)blocks), threads, 0, stream, p);
  return hipGetLastError();
}

hipError_t launch_lora_shrink(const uint16_t* x, const uint16_t* a, const int32_t* ids, const float* scaling,
                              uint16_t* h, int M, int K, int L, int R, float* rowsums, int ld, int gsize,
                              hipStream_t stream) {
  const ShrinkArgs p = {x, a, ids, scaling, h, rowsums, M, K, L, R, ld, 0, 1, 0};
  if (rowsums == nullptr) return launch_shrink_gs<0>(p, stream);
  if (gsize == 128) return launch_shrink_gs<128>(p, stream);
  if (gsize == 32) return launch_shrink_gs<32>(p, stream);
  return hipErrorInvalidValue;
}

}  // namespace w4a16
