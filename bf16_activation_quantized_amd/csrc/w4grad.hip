// Input gradient of the 4-bit products, for gfx950:
//
//   dX[m, k] = sum_n dY[m, n] s[n, k / g] (q[n, k] - 8)
//
// The scale varies along the contraction, so it has to enter the matrix
// core's operand. s (q - 8) has 8 + 3 significant bits: it is exact in fp16
// and would be rounded in bf16. Both operands are therefore brought into fp16
// by powers of two, each row of dY by its own and each column group of scales
// by its own, and the accumulator is brought back by their product:
//  * a row of dY has its largest finite magnitude in [2^14, 2^15): values down
//    to 2^-31 of it are exact (8 bits from 2^-17 on, the last one 2^-24, the step of
//    fp16's subnormals), smaller ones are off by half a step, 2^-39 of it at most;
//  * a group of scales (one k group, all n) has its largest finite magnitude in
//    [2^10, 2^11): products with q - 8 are exact for scales down to 2^-27 of
//    it, smaller scales are off by 2^-35 of it at most.
// A prepass writes dY in fp16, the scales transposed to [k group, n] and their
// largest magnitudes per 128 n; both are ordered (0 4 1 5 2 6 3 7) within 8 n,
// the order in which a word of 8 nibbles unpacks into pairs.
#include <algorithm>
#include <type_traits>

#include "common.hpp"
#include "launch.hpp"
#include "loadorder.hpp"
#include "tilemap.hpp"
#include "tilestore.hpp"

namespace w4a16 {

namespace {

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

constexpr int kNW = 8;
constexpr int kBN = 256;       // output columns (k) per tile
constexpr int kSt = 64;        // contraction elements (n) per stage

template <int VM>
__device__ __forceinline__ void wait_vm_barrier() {
  static_assert(VM >= 0 && VM < 64, "vmcnt range");
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(VM) : "memory");
}
typedef __attribute__((address_space(3))) void* lds_ptr;
__device__ __forceinline__ void dma16(__amdgpu_buffer_rsrc_t r, uint8_t* lds_dst, uint32_t voff, uint32_t soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_ptr)lds_dst, 16, voff, soff, 0, 0);
}

// the power of two that brings the largest finite magnitude (bf16 bits) to
// [2^to, 2^(to + 1)); subnormal maxima count as 2^-126
__device__ __forceinline__ int up_by(uint32_t top16, int to) { return to + 127 - (int)max(top16 >> 7, 1u); }

__device__ __forceinline__ uint32_t f16_pair(float a, float b, int e) {
  const f16x2 h = {(_Float16)ldexpf(a, e), (_Float16)ldexpf(b, e)};
  return __builtin_bit_cast(uint32_t, h);
}

}  // namespace

// ---------------------------------------------------------------- prepass
struct GradPrep {
  const uint16_t* dy;   // [M, N]
  const uint16_t* s;    // [G, N, Kg]
  uint16_t* h;          // [M, Np] fp16, zero past N
  int* up;              // [M] the power of two of each row
  uint16_t* st;         // [G, Kg, Np] bf16 scales, zero past N
  uint16_t* tops;       // [G, Np / 128, Kg] bf16 bits of the largest finite magnitudes
  int M, N, Np, Kg, G;
  int sblocks;          // workgroups per 128 n of the scales
  int stotal;           // workgroups of all scales, the grid's first
  int per_row;          // threads per row of dY
};

// The first workgroups take 128 n of the scales of one expert each: up to
// kPrepWide groups they are one run of memory, read in 16-byte pieces, past that 64
// groups at a time are read by rows. The others take rows of dY, 64 to 512 threads
// each, which hold the row in registers between its largest magnitude and its
// conversion up to kPrepRegs x 8 elements per thread (read again past that).
__global__ __launch_bounds__(kPrepThreads) void grad_prep_kernel(const GradPrep a) {
  __shared__ __attribute__((aligned(16))) uint16_t tile[128 * (kPrepWide + 1)];   // [n][k group], odd pitch
  const int t = threadIdx.x;
  if ((int)blockIdx.x >= a.stotal) {
    uint32_t* part = reinterpret_cast<uint32_t*>(tile);
    const int T = a.per_row, lt = t & (T - 1);
    const int m = ((int)blockIdx.x - a.stotal) * (kPrepThreads / T) + t / T;
    const int n8 = m < a.M ? a.N / 8 : 0, p8 = m < a.M ? a.Np / 8 : 0;
    const u32x4* src = reinterpret_cast<const u32x4*>(a.dy + (size_t)m * a.N);
    uint32_t top = 0;
    auto take = [&](u32x4 v) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t lo = v[i] & 0x7FFFu, hi = (v[i] >> 16) & 0x7FFFu;
        top = max(top, max(lo < 0x7F80u ? lo : 0u, hi < 0x7F80u ? hi : 0u));
      }
    };
    u32x4 held[kPrepRegs];
#pragma unroll
    for (int i = 0; i < kPrepRegs; ++i) {
      const int at = lt + T * i;
      held[i] = at < n8 ? src[at] : u32x4{0u, 0u, 0u, 0u};
    }
#pragma unroll
    for (int i = 0; i < kPrepRegs; ++i) take(held[i]);
    for (int at = lt + T * kPrepRegs; at < n8; at += T) take(src[at]);
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) top = max(top, (uint32_t)__shfl_xor((int)top, d));
    if (T > 64) {
      if ((t & 63) == 0) part[t >> 6] = top;
      __syncthreads();
      for (int i = 0; i < T / 64; ++i) top = max(top, part[t / T * (T / 64) + i]);
    }
    const int e = up_by(top, 14);
    u32x4* dst = reinterpret_cast<u32x4*>(a.h + (size_t)m * a.Np);
    auto put = [&](int at, u32x4 v) {
      dst[at] = u32x4{f16_pair(bf16lo(v.x), bf16lo(v.z), e), f16_pair(bf16hi(v.x), bf16hi(v.z), e),
                      f16_pair(bf16lo(v.y), bf16lo(v.w), e), f16_pair(bf16hi(v.y), bf16hi(v.w), e)};
    };
#pragma unroll
    for (int i = 0; i < kPrepRegs; ++i) {
      const int at = lt + T * i;
      if (at < p8) put(at, held[i]);
    }
    for (int at = lt + T * kPrepRegs; at < p8; at += T) put(at, at < n8 ? src[at] : u32x4{0u, 0u, 0u, 0u});
    if (lt == 0 && m < a.M) a.up[m] = e;
    return;
  }
  int b = blockIdx.x;
  const int kc = b % a.sblocks;
  b /= a.sblocks;
  const int chunks = a.Np / 128;
  const int nc = b % chunks, g = b / chunks;
  const int n0 = 128 * nc, rows = min(128, a.N - n0);
  const bool wide = a.Kg <= kPrepWide;
  const int k0 = wide ? 0 : 64 * kc, kn = wide ? a.Kg : min(64, a.Kg - k0);   // groups of this workgroup
  // the 16 threads of a group read rows 8 apart: with an odd pitch from different banks
  const int pitch = kn | 1;
  const uint16_t* src = a.s + ((size_t)g * a.N + n0) * a.Kg + k0;
  if (wide) {
    // (rows is a multiple of 8, so the run is one of 16 bytes and 16-byte aligned)
    for (int i = t; i < rows * kn / 8; i += kPrepThreads) {
      const u32x4 v = reinterpret_cast<const u32x4*>(src)[i];
      int n = 8 * i / kn, k = 8 * i - n * kn;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        tile[n * pitch + k] = (uint16_t)(v[j >> 1] >> (16 * (j & 1)));
        if (++k == kn) {
          k = 0;
          ++n;
        }
      }
    }
  } else {
    for (int i = t; i < rows * 64; i += kPrepThreads)
      if ((i & 63) < kn) tile[(i >> 6) * pitch + (i & 63)] = src[(size_t)(i >> 6) * a.Kg + (i & 63)];
  }
  __syncthreads();
  for (int i = t; i < kn * 16; i += kPrepThreads) {   // 8 n of one group each; the group's 16 threads are neighbours
    const int kk = i >> 4, n = 8 * (i & 15);
    uint32_t o[4] = {0u, 0u, 0u, 0u}, top = 0;
    if (n < rows) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t lo = tile[(n + j) * pitch + kk], hi = tile[(n + j + 4) * pitch + kk];
        o[j] = lo | (hi << 16);
        const uint32_t ml = lo & 0x7FFFu, mh = hi & 0x7FFFu;
        top = max(top, max(ml < 0x7F80u ? ml : 0u, mh < 0x7F80u ? mh : 0u));
      }
    }
    *reinterpret_cast<u32x4*>(a.st + ((size_t)g * a.Kg + k0 + kk) * a.Np + n0 + n) = u32x4{o[0], o[1], o[2], o[3]};
#pragma unroll
    for (int d = 1; d < 16; d <<= 1) top = max(top, (uint32_t)__shfl_xor((int)top, d));
    if ((i & 15) == 0) a.tops[((size_t)g * chunks + nc) * a.Kg + k0 + kk] = (uint16_t)top;
  }
}

// ---------------------------------------------------------------- tile kernel
// One workgroup of 8 waves (WM x WN) per BM x 256 tile of dX; a stage is 64 n:
// dY in fp16 [BM rows, 128 B], the packed weights [64 rows, 128 B], which a
// transposing LDS read turns into 16 n of one column per lane, and the tile's
// NG groups of scales, s and -24 s in fp16 (a nibble reads as 16 + q: (16 + q) s
// - 24 s = s (q - 8), one exact packed FMA for two weights).
// Bound by the products in fp16 (the bf16 library product of 8192^3 reaches 1620
// TFLOP/s, 1380 with this one's operand order) at the clock that the power limit
// leaves, which keep the matrix core busy for 54 % of the time (1322 x 19456 x 2560, 2.0
// GHz), by the unpacking, which every tile repeats, and by waits for stages: at most
// heights the ring runs empty every second or fourth stage (below). Hence tall tiles
// (1322 x 19456 x 2560 146 us with 224 rows and four slices, 183 with 64 rows), waves
// side by side so that each unpacks its own columns only, and the next stage's
// unpacking between the products of this one.
// 8192^3 900 us (1220 TFLOP/s); 1322 x 19456 x 2560 146 us with its prepass and the
// reduce; 2048 rows of 8 experts of 2048 x 4096, group 32, 51 us.
struct GradArgs {
  const uint16_t* h;       // [M, Np] fp16
  const int* up;           // [M]
  const uint8_t* w;        // [G, N, K / 2]
  const uint16_t* st;      // [G, Kg, Np]
  const uint16_t* tops;    // [G, Np / 128, Kg]
  uint16_t* dx;            // [M, K]
  float* part;             // [SK, M, K] or nullptr
  const int32_t* m_sizes;
  int M, N, Np, K, G;
  int sps;                 // stages per slice
  int mtiles, otiles;
};

template <int BM, int GS>
struct GradStage {
  static constexpr int NG = kBN / GS;               // scale groups of a tile
  static constexpr int kA = BM * 2 * kSt;
  static constexpr int kW = kSt * kBN / 2;
  static constexpr int kS = NG * kSt * 2;           // s, and as many bytes for -24 s
  static constexpr int kBytes = kA + kW + 2 * kS;
};

template <int BM, int WM, int NS, int GS>
__global__ __launch_bounds__(64 * kNW) void w4_grad_kernel(const GradArgs a) {
  using ST = GradStage<BM, GS>;
  constexpr int WN = kNW / WM;
  constexpr int TM = BM / WM, TN = kBN / WN;
  constexpr int MS = TM / 16, SN = TN / 16;
  constexpr int NG = ST::NG;
  constexpr int NQA = BM / 8, QA = (NQA + kNW - 1) / kNW;
  constexpr int SPT = NG * kSt / 2;               // scale pairs per stage
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  __shared__ int gup[NG];                         // the power of two of each scale group

  const int tid = threadIdx.x, lane = tid & 63;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wv / WN, wn = wv % WN;
  const int r16 = lane & 15, q4 = lane >> 4;

  int mt, ot;
  TileRows tr;
  if (a.m_sizes != nullptr) {
    const GroupScan gs(a.m_sizes, a.G, a.M, BM);
    const int nblocks = gs.tiles * a.otiles;
    if ((int)blockIdx.x >= nblocks) return;
    tile_coords(blockIdx.x, nblocks, gs.tiles, a.otiles, &mt, &ot);
    tr = gs.find(mt);
  } else {
    tile_coords(blockIdx.x, (int)gridDim.x, a.mtiles, a.otiles, &mt, &ot);
    tr = TileRows{0, mt * BM, min(BM, a.M - mt * BM)};
  }
  if (tr.rows <= 0) return;

  const int K = a.K, Kg = K / GS, Np = a.Np, chunks = Np / 128;
  const uint32_t K2 = (uint32_t)K / 2u;
  const int o0 = ot * kBN, g0 = o0 / GS;
  const int s0 = blockIdx.y * a.sps;
  const int ns_ = min(Np / kSt, s0 + a.sps) - s0;   // stages

  const __amdgpu_buffer_rsrc_t ra = make_rsrc(a.h + (size_t)tr.row0 * Np, (uint32_t)tr.rows * (uint32_t)Np * 2u);
  const __amdgpu_buffer_rsrc_t rw =
      make_rsrc(a.w + (size_t)tr.wg * a.N * K2 + (uint32_t)o0 / 2u, (uint32_t)a.N * K2 - (uint32_t)o0 / 2u);
  // groups past the last column read zeros
  const __amdgpu_buffer_rsrc_t rs =
      make_rsrc(a.st + ((size_t)tr.wg * Kg + g0) * Np, (uint32_t)(Kg - g0) * (uint32_t)Np * 2u);

  // Part i of the loads of stage s: QA of dY, one of the weights. Wave wv's load i
  // fills the 1 KiB block wv + 8 i of dY (8 rows each) and block wv of the weights
  // (8 n each); the opaque copies keep the sums from being held in registers.
  // 16-byte chunks lie in the slots of pair_swz (dY) and of the row pair (weights).
  constexpr int kParts = QA + 1;
  const uint32_t AB = (uint32_t)Np * 2u;
  uint32_t ab = (uint32_t)(8 * wv + (lane >> 3)) * AB +
                16u * ((uint32_t)(lane & 7) ^ pair_swz((4 * (wv & 1)) | (lane >> 4)));
  uint32_t wb = (uint32_t)(8 * wv + (lane >> 3)) * K2 +
                16u * ((uint32_t)(lane & 7) ^ (uint32_t)((4 * (wv & 1)) | (lane >> 4)));
  auto issue = [&](int s, int stage, int i) {
    uint8_t* base = lds + stage * ST::kBytes;
    if (i < QA) {
      if (NQA % kNW == 0 || wv + kNW * i < NQA) {
        asm volatile("" : "+v"(ab));
        dma16(ra, base + 1024 * (wv + kNW * i), ab + (uint32_t)(64 * i) * AB,
              __builtin_amdgcn_readfirstlane((uint32_t)s * (2u * kSt)));
      }
    } else {
      asm volatile("" : "+v"(wb));
      // (rows past N end past the extent, which checks the vector offset only)
      dma16(rw, base + ST::kA + 1024 * wv, wb + __builtin_amdgcn_readfirstlane((uint32_t)s * kSt * K2), 0u);
    }
  };
  // Scales: pair p of a stage is n pair p % 32 of group p / 32; every thread takes
  // pair tid % SPT (the same words several times rather than a branch).
  const int sp = tid % SPT;
  const uint32_t sb = ((uint32_t)(sp >> 5) * (uint32_t)Np + 2u * (uint32_t)(sp & 31)) * 2u;
  auto scale_word = [&](int s) { return ld32(rs, sb, __builtin_amdgcn_readfirstlane((uint32_t)s * (2u * kSt))); };
  auto put_scales = [&](int stage, uint32_t v, int e) {
    uint8_t* p = lds + stage * ST::kBytes + ST::kA + ST::kW + 4 * sp;
    const uint32_t h = f16_pair(bf16lo(v), bf16hi(v), e);
    const f16x2 m24 = {(_Float16)-24.0f, (_Float16)-24.0f};
    const f16x2 c = __builtin_bit_cast(f16x2, h) * m24;
    *reinterpret_cast<uint32_t*>(p) = h;
    *reinterpret_cast<uint32_t*>(p + ST::kS) = __builtin_bit_cast(uint32_t, c);
  };

  // largest scale of each of the tile's groups over all n
  for (int g = wv; g < NG; g += kNW) {
    uint32_t top = 0;
    if (g0 + g < Kg)
      for (int c = lane; c < chunks; c += 64)
        top = max(top, (uint32_t)a.tops[((size_t)tr.wg * chunks + c) * Kg + g0 + g]);
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) top = max(top, (uint32_t)__shfl_xor((int)top, d));
    if (lane == 0) gup[g] = up_by(top, 10);
  }
  __syncthreads();
  const int sup = gup[sp >> 5];

  f32x4 acc[MS][SN];
#pragma unroll
  for (int ms = 0; ms < MS; ++ms)
#pragma unroll
    for (int ns = 0; ns < SN; ++ns) acc[ms][ns] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

  // ---- LDS operand offsets within a stage
  // dY: row TM wm + 16 ms + r16, chunk 2 q4 + st
  const uint32_t ao = (uint32_t)(TM * wm + r16) * (2 * kSt) + 16u * ((uint32_t)(2 * q4) ^ pair_swz(r16 >> 1));
  // weights: lane r of a group of 16 points at 8 bytes (16 columns) of row 16 q4 +
  // r and receives column r's 16 n
  const uint32_t wo = ST::kA + (uint32_t)(16 * q4 + r16) * (kBN / 2);
  // scales of n 16 q4 + 8 st .. + 7
  const uint32_t so = ST::kA + ST::kW + 32u * (uint32_t)q4;

  const uint32_t magic = vgpr_const(0x4C004C00u);   // a pair of 16
  const uint32_t mask = __builtin_amdgcn_readfirstlane(vgpr_const(0x03C003C0u));
  constexpr int NF = 2 * SN;    // weight fragments of a stage: st = f / SN, ns = f % SN
  f16x8 wf[2][NF];              // of this stage and the next
  u32x2 raw[SN];
  u32x4 sc, cc;
  f16x8 xf[2][2];
  auto read_x = [&](int stage, int ms) {
    const uint8_t* p = lds + stage * ST::kBytes + 16 * 2 * kSt * ms;
    xf[ms & 1][0] = *reinterpret_cast<const f16x8*>(p + ao);
    xf[ms & 1][1] = *reinterpret_cast<const f16x8*>(p + (ao ^ 16u));
  };
  auto read_raw = [&](int stage) {
    static_assert(SN == 2 || SN == 4, "column tiles are read by twos");
    constexpr int kPairs = SN / 2;
    const uint32_t at = lds_offset(lds) + (uint32_t)(stage * ST::kBytes) + wo;
    // 16-byte chunk TN wn / 32 + i of the row, slot chunk ^ (row pair)
    const uint32_t slot = 16u * ((uint32_t)(TN * wn / 32) ^ (uint32_t)(r16 >> 1));
    if constexpr (kPairs == 2) lds_tr4_pairs(at + slot, at + (slot ^ 16u), raw[0], raw[1], raw[2], raw[3]);
    else lds_tr4_pair(at + slot, raw[0], raw[1]);
  };
  // fragment f of the raw weights: nibbles j and j + 4 of a word go to mantissa
  // bits 6 .. 9 of the two halves of 16 + q
  auto unpack = [&](int stage, int f, f16x8& out) {
    const int st = f / SN, ns = f % SN;
    if ((16 * ns) % GS == 0) {
      const uint8_t* p = lds + stage * ST::kBytes + so + (TN * wn + 16 * ns) / GS * (2 * kSt) + 16 * st;
      sc = *reinterpret_cast<const u32x4*>(p);
      cc = *reinterpret_cast<const u32x4*>(p + ST::kS);
    }
    const uint32_t v = st == 0 ? raw[ns].x : raw[ns].y;
    u32x4 o;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t u = and_or_sv(j == 0 ? v << 6 : j == 1 ? v << 2 : j == 2 ? v >> 2 : v >> 6, mask, magic);
      const uint32_t s = sc[j], c = cc[j];
      const f16x2 r = __builtin_elementwise_fma(__builtin_bit_cast(f16x2, u), __builtin_bit_cast(f16x2, s),
                                                __builtin_bit_cast(f16x2, c));
      o[j] = __builtin_bit_cast(uint32_t, r);
    }
    out = __builtin_bit_cast(f16x8, o);
  };

  // One stage j: its products, from weights that are in registers, while stage j +
  // 1's weights are unpacked, a fragment at each row tile, and stage j + NS - 1 is
  // loaded, a few loads at each row tile. Its scales were requested kAhead stages
  // earlier (waiting for a load waits for all that was issued before it). As built,
  // the first of every kAhead steps waits for more: the loop may end after any step,
  // the compiler sees ways from each end back to its head, on which the scales that
  // the first step puts away were requested a moment ago, and waits for all but the
  // last one to three loads (at all heights but 192 and 256 rows): the ring runs empty
  // there. Past the last stage the last one's loads are repeated, unused: one form of
  // the loop keeps the registers where they are.
  constexpr int kPer = NQA / kNW + 2;   // loads issued per stage, by any wave at least
  // (kAhead stages are unrolled: a register with a load in flight cannot be moved)
  constexpr int kAhead = NS > 5 ? 4 : 2;
  static_assert(kAhead < NS, "a scale word behind each of the last stages ahead of the loop");
  // Loads in flight that leave stages 0 and 1 landed ahead of the loop, and stage j + 2
  // at the end of step j. (The first steps' waits count stages 3 .. NS - 2, requested
  // ahead of the loop, as steps: with one load less each, stage j + 2 might be missing.)
  constexpr int kStart = (NS - 3) * (kPer - 1) + (kAhead < NS - 3 ? kAhead : NS - 3);
  constexpr int kStep = (NS - 3) * kPer;
  uint32_t sv[kAhead];                  // the scales of stages j + NS - 1 .. j + NS + kAhead - 2
  auto body = [&](auto P, int stage, int after, int next, int word, int nstage) {
    constexpr int p = P.value & 1;
    read_x(stage, 0);
#pragma unroll
    for (int ms = 0; ms < MS; ++ms) {
      if (ms + 1 < MS) read_x(stage, ms + 1);
#pragma unroll
      for (int i = ms * kParts / MS; i < (ms + 1) * kParts / MS; ++i) issue(next, nstage, i);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int st = 0; st < 2; ++st)
#pragma unroll
        for (int ns = 0; ns < SN; ++ns)
          acc[ms][ns] =
              __builtin_amdgcn_mfma_f32_16x16x32_f16(wf[p][st * SN + ns], xf[ms & 1][st], acc[ms][ns], 0, 0, 0);
      if (ms == 0) read_raw(after);   // (it waits, behind the first products)
      // (a chain of conversions and a write to LDS: between the products rather than
      // ahead of the barrier, 957 -> 935 us at 8192^3 and 128 rows, 933 -> 927 at 192;
      // at 256 rows, with few registers left, 918 ahead of the barrier and 946 here)
      if (ms == (BM < 256 ? MS / 2 : MS - 1)) {
        put_scales(nstage, sv[P.value], sup);
        sv[P.value] = scale_word(word);
      }
#pragma unroll
      for (int f = ms * NF / MS; f < (ms + 1) * NF / MS; ++f) unpack(after, f, wf[1 - p][f]);
    }
    wait_vm_barrier<kStep>();   // stage j + 2 has landed
  };

  static_assert(NS >= 3, "stages j, j + 1 (whose weights are unpacked) and j + 2 (being loaded)");
  if (ns_ > 0) {
    auto at = [&](int j) { return s0 + min(j, ns_ - 1); };
    uint32_t first[NS - 1];
#pragma unroll
    for (int s = 0; s < NS - 1; ++s) first[s] = scale_word(at(s));
    // The stages ahead of the loop: the last kAhead of them with a scale word behind
    // each, as in the steps. (The empty asm keeps the loads in this order, which the
    // waits count on.)
    asm volatile("" ::: "memory");
#pragma unroll
    for (int s = 0; s < NS - 1; ++s) {
#pragma unroll
      for (int i = 0; i < kParts; ++i) issue(at(s), s, i);
      asm volatile("" ::: "memory");
      const int i = s - (NS - 1 - kAhead);
      if (i >= 0) sv[i] = scale_word(at(NS - 1 + i));
      asm volatile("" ::: "memory");
    }
#pragma unroll
    for (int s = 0; s < NS - 1; ++s) put_scales(s, first[s], sup);
    static_assert(ring_waits_hold(NS, kPer - 1, NS - 1 - kAhead, kStart, kStep), "waits of the ring");
    wait_vm_barrier<kStart>();   // stages 0 and 1 have landed
    read_raw(0);
#pragma unroll
    for (int f = 0; f < NF; ++f) unpack(0, f, wf[0][f]);
    auto inc = [](int s, int by) { return s + by >= NS ? s + by - NS : s + by; };
    int st = 0, j = 0;   // st = j % NS
    auto step = [&](auto P) {
      body(P, st, inc(st, 1), at(j + NS - 1), at(j + NS - 1 + kAhead), inc(st, NS - 1));
      st = inc(st, 1);
      return ++j >= ns_;
    };
    for (;;) {
      if (step(std::integral_constant<int, 0>{})) break;
      if (step(std::integral_constant<int, 1>{})) break;
      if constexpr (kAhead == 4) {
        if (step(std::integral_constant<int, 2>{})) break;
        if (step(std::integral_constant<int, 3>{})) break;
      }
    }
    wait_vm_barrier<0>();   // the repeated loads: LDS is used again below
  }

  // ---- epilogue: lane holds row 16 ms + r16 of the wave's, columns 16 ns + 4 q4 .. + 3
  const int ow = o0 + TN * wn;
#pragma unroll
  for (int ms = 0; ms < MS; ++ms) {
    const int row = TM * wm + 16 * ms + r16;
    const int down = row < tr.rows ? -a.up[tr.row0 + row] : 0;
#pragma unroll
    for (int ns = 0; ns < SN; ++ns) {
      const int e = down - gup[(TN * wn + 16 * ns) / GS];
      acc[ms][ns] = f32x4{ldexpf(acc[ms][ns].x, e), ldexpf(acc[ms][ns].y, e), ldexpf(acc[ms][ns].z, e),
                          ldexpf(acc[ms][ns].w, e)};
    }
  }
  if (a.part == nullptr) {
    __syncthreads();
    const __amdgpu_buffer_rsrc_t ry = make_rsrc(a.dx + (size_t)tr.row0 * K, (uint32_t)tr.rows * (uint32_t)K * 2u);
    store_tile_bf16<TM, TN>(lds + wv * (TM * TN * 2), acc, [&](int ns) { return 16 * ns + 4 * q4; }, ry, TM * wm, ow, K,
                            lane);
    return;
  }
  const size_t part0 = ((size_t)blockIdx.y * a.M + tr.row0) * K;
#pragma unroll
  for (int ms = 0; ms < MS; ++ms) {
    const int row = TM * wm + 16 * ms + r16;
    if (row >= tr.rows) continue;
#pragma unroll
    for (int ns = 0; ns < SN; ++ns) {
      const int c = ow + 16 * ns + 4 * q4;
      if (c < K) *reinterpret_cast<f32x4*>(a.part + part0 + (size_t)row * K + c) = acc[ms][ns];
    }
  }
}

template <int BM, int WM, int NS, int GS>
static hipError_t launch_w4_grad_t(GradArgs a, int sk, hipStream_t stream) {
  // the stages, afterwards the outputs
  constexpr int lds_bytes = std::max(NS * GradStage<BM, GS>::kBytes, BM * kBN * 2);
  static_assert(lds_bytes <= 159 * 1024, "LDS");
  static std::atomic<uint64_t> lds_set{0};
  const hipError_t ea =
      ensure_dyn_lds(reinterpret_cast<const void*>(&w4_grad_kernel<BM, WM, NS, GS>), lds_bytes, lds_set);
  if (ea != hipSuccess) return ea;
  a.mtiles = a.m_sizes != nullptr ? group_tiles_bound(a.M, BM, a.G) : (a.M + BM - 1) / BM;
  a.otiles = (a.K + kBN - 1) / kBN;
  const long long blocks = (long long)a.mtiles * a.otiles;
  if (blocks > kMaxBlocks) return hipErrorInvalidValue;
  hipLaunchKernelGGL((w4_grad_kernel<BM, WM, NS, GS>), dim3((unsigned)blocks, sk), dim3(64 * kNW), lds_bytes, stream,
                     a);
  return hipGetLastError();
}

// Stages: as many as LDS takes, up to 8. One row of waves (each unpacks the
// weights of its own 32 columns only) against two: 128 rows 986 against 1090 us at
// 8192^3, 192 rows 970 against 997; at 256 rows, where each wave then reads every
// row of dY, 946 against 924 (at group 32, where two rows of waves leave registers
// short, 956 against 959). (Both sides before the last steps; now 965, 956 and 935.)
template <int GS>
static hipError_t launch_w4_grad_gs(const GradArgs& a, int sk, int bm, hipStream_t stream) {
  switch (bm) {
    case 256: return launch_w4_grad_t<256, GS == 128 ? 2 : 1, 3, GS>(a, sk, stream);
    case 224: return launch_w4_grad_t<224, 1, 4, GS>(a, sk, stream);
    case 192: return launch_w4_grad_t<192, 1, 4, GS>(a, sk, stream);
    case 160: return launch_w4_grad_t<160, 1, 5, GS>(a, sk, stream);
    case 128: return launch_w4_grad_t<128, 1, 6, GS>(a, sk, stream);
    case 96: return launch_w4_grad_t<96, 1, 6, GS>(a, sk, stream);
    case 64: return launch_w4_grad_t<64, 1, 8, GS>(a, sk, stream);
    case 32: return launch_w4_grad_t<32, 1, 8, GS>(a, sk, stream);
    case 16: return launch_w4_grad_t<16, 1, 8, GS>(a, sk, stream);
    default: return hipErrorInvalidValue;
  }
}

hipError_t launch_w4_grad(const uint16_t* dy, const uint8_t* w, const uint16_t* s, uint16_t* dx, const int32_t* m_sizes,
                          int M, int N, int K, int G, int gsize, const W4GradPlan& p, uint8_t* ws, hipStream_t stream) {
  const int Np = (int)w4_grad_padded(N), Kg = K / gsize;
  GradPrep pr;
  pr.dy = dy; pr.s = s;
  pr.h = reinterpret_cast<uint16_t*>(ws + p.h);
  pr.up = reinterpret_cast<int*>(ws + p.up);
  pr.st = reinterpret_cast<uint16_t*>(ws + p.st);
  pr.tops = reinterpret_cast<uint16_t*>(ws + p.tops);
  pr.M = M; pr.N = N; pr.Np = Np; pr.Kg = Kg; pr.G = G;
  pr.sblocks = w4_grad_scale_blocks(Kg);
  pr.per_row = w4_grad_row_threads(N);
  const int64_t blocks = w4_grad_prep_blocks(G, M, N, Kg);
  if (blocks > kMaxBlocks) return hipErrorInvalidValue;
  pr.stotal = (int)((int64_t)G * (Np / 128) * pr.sblocks);
  hipLaunchKernelGGL(grad_prep_kernel, dim3((unsigned)blocks), dim3(kPrepThreads), 0, stream, pr);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  GradArgs a;
  a.h = pr.h; a.up = pr.up; a.w = w; a.st = pr.st; a.tops = pr.tops; a.dx = dx;
  a.part = p.sk > 1 ? reinterpret_cast<float*>(ws + p.part) : nullptr;
  a.m_sizes = m_sizes; a.M = M; a.N = N; a.Np = Np; a.K = K; a.G = G;
  a.sps = (Np / kSt + p.sk - 1) / p.sk;
  a.mtiles = a.otiles = 0;
  const hipError_t el = gsize == 32 ? launch_w4_grad_gs<32>(a, p.sk, p.bm, stream)
                                    : launch_w4_grad_gs<128>(a, p.sk, p.bm, stream);
  if (el != hipSuccess || p.sk == 1) return el;
  if (m_sizes != nullptr) return launch_splitk_reduce_rows(a.part, dx, m_sizes, G, M, K, p.sk, stream);
  return launch_splitk_reduce(a.part, dx, (uint64_t)M * (uint64_t)K, p.sk, stream);
}

}  // namespace w4a16
