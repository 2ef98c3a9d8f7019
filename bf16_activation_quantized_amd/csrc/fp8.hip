// 8-bit products with a scale for each block of 128, for gfx950.
//
//   Y[m, n] = sum_b sx[m, b] sw[n / 128, b] sum_{k in block b} X[m, k] W[n, k]
//
// and the input gradient, whose contraction runs over n instead of k. X and W
// are e4m3 (OCP); an inner sum is one v_mfma_f32_16x16x128_f8f6f4, which aligns
// the exact products of each 8 contraction elements to the largest of them, keeps
// 13 bits below its leading one (65536 + 8 is kept, 65536 + 4 is not), and adds
// everything else in fp32. Each inner sum is scaled by the fp32 product of its two
// scales and added to the fp32 accumulator, and the result is rounded once to bf16.
//
// The weights are the MFMA's A operand (its rows are output columns) and the
// activations its B operand, so a lane holds one row m and four consecutive
// output columns of each tile: one product of scales per row tile and block
// serves all of a wave's column tiles, and the outputs of a lane are
// contiguous.
#include <algorithm>
#include <type_traits>

#include "common.hpp"
#include "launch.hpp"
#include "tilemap.hpp"
#include "tilestore.hpp"

namespace w4a16 {

namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef int i32x2 __attribute__((ext_vector_type(2)));

constexpr int kNW = 8;        // waves per workgroup
constexpr int kBlk = 128;     // contraction elements per scale block (one MFMA)

template <int VM>
__device__ __forceinline__ void wait_vm_barrier() {
  static_assert(VM >= 0 && VM < 64, "vmcnt range");
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(VM) : "memory");
}

typedef __attribute__((address_space(3))) void* lds_ptr;
__device__ __forceinline__ void dma16(__amdgpu_buffer_rsrc_t r, uint8_t* lds_dst, uint32_t voff, uint32_t soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_ptr)lds_dst, 16, voff, soff, 0, 0);
}
__device__ __forceinline__ void dma4(__amdgpu_buffer_rsrc_t r, uint8_t* lds_dst, uint32_t voff, uint32_t soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_ptr)lds_dst, 4, voff, soff, 0, 0);
}

__device__ __forceinline__ i32x8 frag(u32x4 a, u32x4 b) {
  return i32x8{(int)a.x, (int)a.y, (int)a.z, (int)a.w, (int)b.x, (int)b.y, (int)b.z, (int)b.w};
}

// one 16 x 16 tile's product over a block of 128, from zero
__device__ __forceinline__ f32x4 block_product(i32x8 w, i32x8 x) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, f32x4{0.0f, 0.0f, 0.0f, 0.0f}, 0, 0, 0, 0, 0, 0);
}

__device__ __forceinline__ void add_scaled(f32x4& acc, float s, f32x4 t) {
  acc.x = fmaf(s, t.x, acc.x);
  acc.y = fmaf(s, t.y, acc.y);
  acc.z = fmaf(s, t.z, acc.z);
  acc.w = fmaf(s, t.w, acc.w);
}

}  // namespace

// ---------------------------------------------------------------- quantise
// s = max(amax, 2^-100) / 448 and q = e4m3(x * (448 / max(amax, 2^-100))), both
// in fp32, rounded to nearest even; a block with an infinity or a NaN: s = NaN,
// q = 0. The largest magnitude of a block is taken on the bf16 bit patterns
// (their order is that of the magnitudes, and infinities and NaN come last).
constexpr float kE4m3Max = 448.0f;
constexpr float kMinTop = 0x1p-100f;

__device__ __forceinline__ uint32_t pk_max_u16(uint32_t a, uint32_t b) {
  typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
  const u16x2 r = __builtin_elementwise_max(__builtin_bit_cast(u16x2, a), __builtin_bit_cast(u16x2, b));
  return __builtin_bit_cast(uint32_t, r);
}

// packed maxima of the magnitudes of 8 bf16
__device__ __forceinline__ uint32_t top_of(u32x4 v) {
  constexpr uint32_t m = 0x7FFF7FFFu;
  return pk_max_u16(pk_max_u16(v.x & m, v.y & m), pk_max_u16(v.z & m, v.w & m));
}

struct BlockScale {
  float s, r;   // the scale, and the factor that the values are multiplied by
  bool fine;
};
__device__ __forceinline__ BlockScale block_scale(uint32_t top16) {
  BlockScale b;
  b.fine = top16 < 0x7F80u;
  const float top = fmaxf(bf16f((uint16_t)top16), kMinTop);
  b.s = b.fine ? top / kE4m3Max : __uint_as_float(0x7FC00000u);
  b.r = kE4m3Max / top;
  return b;
}

__device__ __forceinline__ uint32_t e4m3x4(uint32_t lo, uint32_t hi, float r) {
  int o = __builtin_amdgcn_cvt_pk_fp8_f32(bf16lo(lo) * r, bf16hi(lo) * r, 0, false);
  o = __builtin_amdgcn_cvt_pk_fp8_f32(bf16lo(hi) * r, bf16hi(hi) * r, o, true);
  return (uint32_t)o;
}
__device__ __forceinline__ u32x4 e4m3x16(u32x4 a, u32x4 b, const BlockScale& s) {
  if (!s.fine) return u32x4{0u, 0u, 0u, 0u};
  return u32x4{e4m3x4(a.x, a.y, s.r), e4m3x4(a.z, a.w, s.r), e4m3x4(b.x, b.y, s.r), e4m3x4(b.z, b.w, s.r)};
}

// Bound by memory: 2 bytes read and 1 written per element, one pass. Blocks of 1 x
// 128: with K a multiple of 128 they are consecutive runs of 128 elements, 8 lanes
// each with two 16-byte loads (16384 x 8192: 70 us, 5.8 TB/s; a 2 GiB copy 5.2).
__global__ __launch_bounds__(256) void fp8_quantize_rows_kernel(const uint16_t* __restrict__ x,
                                                                uint8_t* __restrict__ q, float* __restrict__ scales,
                                                                int64_t blocks) {
  const int64_t b = (int64_t)blockIdx.x * 32 + (threadIdx.x >> 3);
  if (b >= blocks) return;   // whole groups of 8 lanes
  const int l = threadIdx.x & 7;
  const u32x4* src = reinterpret_cast<const u32x4*>(x + b * kBlk + 16 * l);
  const u32x4 v0 = src[0], v1 = src[1];
  uint32_t t = pk_max_u16(top_of(v0), top_of(v1));
  t = max(t & 0xFFFFu, t >> 16);
  t = max(t, (uint32_t)__shfl_xor((int)t, 1));
  t = max(t, (uint32_t)__shfl_xor((int)t, 2));
  t = max(t, (uint32_t)__shfl_xor((int)t, 4));
  const BlockScale s = block_scale(t);
  *reinterpret_cast<u32x4*>(q + b * kBlk + 16 * l) = e4m3x16(v0, v1, s);
  if (l == 0) scales[b] = s.s;
}

// Blocks of 128 x 128 (the last rows' may be shorter): one workgroup each, which
// holds its block in registers between the maximum and the conversion (8192 x 8192: 37.6
// us, 5.4 TB/s; in blocks of 1 x 128 35.7).
__global__ __launch_bounds__(256) void fp8_quantize_blocks_kernel(const uint16_t* __restrict__ x,
                                                                  uint8_t* __restrict__ q,
                                                                  float* __restrict__ scales, int64_t M, int K,
                                                                  int kblocks) {
  __shared__ uint32_t tops[4];
  const int64_t rb = blockIdx.x / kblocks;
  const int cb = blockIdx.x % kblocks;
  const int l = threadIdx.x & 7;
  u32x4 v[4][2];
  uint32_t t = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t row = rb * kBlk + 32 * i + (threadIdx.x >> 3);
    v[i][0] = v[i][1] = u32x4{0u, 0u, 0u, 0u};
    if (row < M) {
      const u32x4* src = reinterpret_cast<const u32x4*>(x + row * K + cb * kBlk + 16 * l);
      v[i][0] = src[0];
      v[i][1] = src[1];
    }
    t = pk_max_u16(t, pk_max_u16(top_of(v[i][0]), top_of(v[i][1])));
  }
  t = max(t & 0xFFFFu, t >> 16);
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) t = max(t, (uint32_t)__shfl_xor((int)t, d));
  if ((threadIdx.x & 63) == 0) tops[threadIdx.x >> 6] = t;
  __syncthreads();
  const BlockScale s = block_scale(max(max(tops[0], tops[1]), max(tops[2], tops[3])));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t row = rb * kBlk + 32 * i + (threadIdx.x >> 3);
    if (row < M) *reinterpret_cast<u32x4*>(q + row * K + cb * kBlk + 16 * l) = e4m3x16(v[i][0], v[i][1], s);
  }
  if (threadIdx.x == 0) scales[rb * kblocks + cb] = s.s;
}

hipError_t launch_fp8_quantize(const uint16_t* x, uint8_t* q, float* scales, int64_t M, int K, int block_rows,
                               hipStream_t stream) {
  // (a launch takes fewer than 2^32 threads)
  const int kblocks = K / kBlk;
  if (block_rows == 1) {
    const int64_t blocks = M * kblocks, most = (int64_t)1 << 28;   // 2^23 workgroups
    for (int64_t b = 0; b < blocks; b += most) {
      const int64_t n = std::min(blocks - b, most);
      hipLaunchKernelGGL(fp8_quantize_rows_kernel, dim3((unsigned)((n + 31) / 32)), dim3(256), 0, stream,
                         x + b * kBlk, q + b * kBlk, scales + b, n);
    }
  } else {
    // (M K < 2^37: fewer than 2^23 + K / 128 blocks, and than 2^24 where M <= 128)
    const int64_t grid = (M + kBlk - 1) / kBlk * kblocks;
    if (grid >= (int64_t)1 << 24) return hipErrorInvalidValue;
    hipLaunchKernelGGL(fp8_quantize_blocks_kernel, dim3((unsigned)grid), dim3(256), 0, stream, x, q, scales, M, K,
                       kblocks);
  }
  return hipGetLastError();
}

// ---------------------------------------------------------------- tile kernel
// One workgroup of 8 waves (WM x WN) per BM x 256 output tile; a stage is one
// contraction block: X [BM rows, 128 B], W [256 columns, 128 B] (gradient: [128
// rows, 256 B], transposed as it is read) and the BM row scales, filled by
// buffer loads that write LDS directly, NS stages in a ring.
// Work per block of 128 at 256 rows: 256 products of 16 x 16 and, per lane, as many
// times four scaled additions. The products alone run at 4944 TFLOP/s on this card,
// with the additions (on the VALU, beside them) at 4000: two thirds of the largest
// cases' time at the clock that the power limit leaves them (2.04 GHz of 2.4 at 8192^3,
// the matrix core busy for 55 % of it). The rest is waits: at 192 rows and more, with
// two stages, the last loads of a block go out 8 products ahead of the wait for them.
//  * 8 waves of 128 x 64 (2 x 4), so that a lane's scale product serves 4 tiles and
//    the two operands' LDS reads (24 KiB per wave and block) stay below the products.
//  * The loads of a stage are issued between the row tiles: all at the stage's start
//    they filled the memory pipeline's queue and held the waves up (1322 x 19456 x
//    2560 115 us, spread 79).
//  * One product of scales per lane and row tile: the activations are the B operand.
// 8192^3 470 us (2340 TFLOP/s); 1322 x 19456 x 2560 72 us; 16384 rows of 32 experts of
// 2048 x 4096 186 us; gradient of 777 x 9728 x 2560 37 us (50 tiles of 160 rows, split
// five ways over the contraction), of 4096 rows of 8 experts 52 us.
struct Fp8Args {
  const uint8_t* x;        // [M, C] e4m3: C = K, gradient: N
  const float* xs;         // [M, C / 128]
  const uint8_t* w;        // [G, N, K] e4m3
  const float* ws;         // [G, ceil(N / 128), K / 128]
  uint16_t* y;             // [M, O] bf16: O = N, gradient: K
  float* part;             // [SK, M, O] fp32 partials, or nullptr
  const int32_t* m_sizes;  // [G] on the device, or nullptr
  int M, N, K, G;
  int cps;                 // contraction blocks per slice
  int mtiles, otiles;
};

constexpr int kBN = 256;      // output columns per tile

template <int BM>
constexpr int fp8_stage_bytes() { return BM * kBlk + kBN * kBlk + ((BM + 63) / 64 + 1) * 256; }

template <int BM, int WM, int NS, bool GRAD>
__global__ __launch_bounds__(64 * kNW) void fp8_tile_kernel(const Fp8Args a) {
  constexpr int WN = kNW / WM;
  constexpr int TM = BM / WM, TN = kBN / WN;   // rows and columns per wave
  constexpr int MS = TM / 16, SN = TN / 16;
  constexpr int kX = BM * kBlk, kW = kBN * kBlk, kStage = fp8_stage_bytes<BM>();
  constexpr int NQX = BM / 8;                  // 1 KiB loads of X per stage
  constexpr int kSX = (BM + 63) / 64;          // waves that load row scales
  constexpr int QX = (NQX + kNW - 1) / kNW;
  constexpr int QW = kBN / 8 / kNW;            // of W per wave
  static_assert(kSX < kNW && TN <= kBlk && MS >= 1 && SN >= 1, "a wave's columns lie in one block");
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];

  const int lane = threadIdx.x & 63;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
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

  const int C = GRAD ? a.N : a.K, O = GRAD ? a.K : a.N;
  const int Cb = C / kBlk, KB = a.K / kBlk, NB = (a.N + kBlk - 1) / kBlk;
  const int o0 = ot * kBN;
  const __amdgpu_buffer_rsrc_t rx = make_rsrc(a.x + (size_t)tr.row0 * C, (uint32_t)tr.rows * (uint32_t)C);
  const uint32_t wk = (uint32_t)a.K;
  const uint8_t* wg = a.w + (size_t)tr.wg * a.N * a.K;
  const __amdgpu_buffer_rsrc_t rw = GRAD ? make_rsrc(wg + o0, (uint32_t)a.N * wk - (uint32_t)o0)
                                         : make_rsrc(wg + (size_t)o0 * a.K, (uint32_t)min(kBN, O - o0) * wk);
  const int cb0 = blockIdx.y * a.cps;
  const int nc = min(Cb, cb0 + a.cps) - cb0;

  // Part i of the loads of block cb: QX of X, then QW of W. Wave wv's load i fills
  // the 1 KiB block wv + 8 i of X (8 rows each) and of W (8 columns; gradient: 4
  // rows): the lane offsets are those of i = 0 plus whole rows, added at each load
  // (the opaque copies keep the sums from being held in registers). The 16-byte
  // chunks of an LDS row lie in slots by pair_swz of the row pair that a fragment
  // read sees (W: rows 4 SN (r >> 2) + (r & 3) are one read's).
  constexpr int kParts = QX + QW;
  uint32_t xb = (uint32_t)(8 * wv + (lane >> 3)) * (uint32_t)C +
                16u * ((uint32_t)(lane & 7) ^ pair_swz((4 * (wv & 1)) | (lane >> 4)));
  uint32_t wb, wb2 = 0;
  if constexpr (GRAD) {
    // slot of chunk c of row r: c ^ (r & 7 | (r & 32) / 4)
    const uint32_t row = (uint32_t)(4 * wv + (lane >> 4)), c = (uint32_t)(lane & 15) ^ (row & 7u);
    wb = row * wk + 16u * c;
    wb2 = row * wk + 16u * (c ^ 8u);   // odd i: r & 32 set
  } else {
    const int row = 8 * wv + (lane >> 3);
    wb = (uint32_t)row * wk +
         16u * ((uint32_t)(lane & 7) ^ pair_swz(((row >> 1) & 1) | ((row / (4 * SN)) & 3) << 1));
  }
  static_assert(GRAD || (64 / (4 * SN)) % 4 == 0, "the slots of a wave's columns repeat every 64");
  auto issue = [&](int cb, int stage, int i) {
    uint8_t* base = lds + stage * kStage;
    const uint32_t so = __builtin_amdgcn_readfirstlane((uint32_t)cb * kBlk);
    if (i < QX) {
      if (NQX % kNW == 0 || wv + kNW * i < NQX) {
        asm volatile("" : "+v"(xb));
        dma16(rx, base + 1024 * (wv + kNW * i), xb + (uint32_t)(64 * i) * (uint32_t)C, so);
      }
    } else {
      const int k = i - QX;
      uint8_t* dst = base + kX + 1024 * (wv + kNW * k);
      if constexpr (GRAD) {
        uint32_t& o = k & 1 ? wb2 : wb;
        asm volatile("" : "+v"(o));
        // (the whole offset is checked against the extent: the last row's end)
        dma16(rw, dst, o + __builtin_amdgcn_readfirstlane(((uint32_t)cb * kBlk + 32u * (uint32_t)k) * wk), 0u);
      } else {
        asm volatile("" : "+v"(wb));
        dma16(rw, dst, wb + (uint32_t)(64 * k) * wk, so);
      }
    }
  };
  // The scales: one dword per lane and wave. Waves below BM / 64 (at least one)
  // take the row scales, the others all the same two column scales (lanes 0 and
  // 1; an offset past every extent reads zero).
  const bool sxw = wv < kSX;
  const __amdgpu_buffer_rsrc_t rsc =
      make_rsrc(sxw ? a.xs + (size_t)tr.row0 * Cb : a.ws + (size_t)tr.wg * NB * KB,
                sxw ? (uint32_t)tr.rows * (uint32_t)Cb * 4u : (uint32_t)NB * (uint32_t)KB * 4u);
  const int ob = o0 / kBlk + lane;
  const bool colw = lane < kBN / kBlk && ob < (GRAD ? KB : NB);
  const uint32_t sv = sxw ? (uint32_t)(64 * wv + lane) * (uint32_t)Cb * 4u
                          : colw ? (uint32_t)ob * (GRAD ? 4u : (uint32_t)KB * 4u) : 0xFFFFFFF0u;
  const uint32_t sstep = GRAD && !sxw ? (uint32_t)KB * 4u : 4u;
  const uint32_t sdst = kX + kW + 256u * (uint32_t)min(wv, kSX);
  auto issue_scales = [&](int cb, int stage) {
    dma4(rsc, lds + stage * kStage + sdst, sv, __builtin_amdgcn_readfirstlane((uint32_t)cb * sstep));
  };

  f32x4 acc[MS][SN];
#pragma unroll
  for (int ms = 0; ms < MS; ++ms)
#pragma unroll
    for (int ns = 0; ns < SN; ++ns) acc[ms][ns] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

  // ---- LDS operand offsets within a stage
  // X: row TM wm + 16 ms + r16, chunks 2 q4 and 2 q4 + 1
  const uint32_t xo = (uint32_t)(TM * wm + r16) * kBlk + 16u * ((uint32_t)(2 * q4) ^ pair_swz(r16 >> 1));
  // W: MFMA row r of column tile ns is column 4 SN (r >> 2) + 4 ns + (r & 3) of the
  // wave's, so that a lane's outputs are 4 SN consecutive columns
  const uint32_t wo = kX + (uint32_t)(TN * wn + 4 * SN * (r16 >> 2) + (r16 & 3)) * kBlk +
                      16u * ((uint32_t)(2 * q4) ^ pair_swz(r16 >> 1));
  // gradient: 8 rows x 16 columns are transposed by each group of 16 lanes: lanes
  // 2 j and 2 j + 1 point at row j's two 8-byte halves, lane c receives column c
  const uint32_t go = kX + (uint32_t)(32 * q4 + (r16 >> 1)) * kBN + 8u * (uint32_t)(r16 & 1) +
                      16u * (uint32_t)((TN * wn / 16) ^ ((r16 >> 1) | (q4 & 1) << 3));
  const uint32_t so_x = kX + kW + 4u * (uint32_t)(TM * wm + r16);
  const uint32_t so_w = kX + kW + 256u * kSX + 4u * (uint32_t)(TN * wn / kBlk);

  i32x8 wf[SN], xf[2];
  float sx[2], sc = 0.0f;
  auto read_x = [&](int stage, int ms) {
    const uint8_t* base = lds + stage * kStage;
    const uint8_t* p = base + 16 * kBlk * ms;
    xf[ms & 1] = frag(*reinterpret_cast<const u32x4*>(p + xo), *reinterpret_cast<const u32x4*>(p + (xo ^ 16u)));
    sx[ms & 1] = *reinterpret_cast<const float*>(base + so_x + 64 * ms);
  };
  auto read_w = [&](int stage) {
    const uint8_t* base = lds + stage * kStage;
    if constexpr (GRAD) {
      static_assert(!GRAD || SN % 2 == 0, "column tiles are read by twos");
#pragma unroll
      for (int ns = 0; ns < SN; ns += 2) {
        u32x2 d[2][4];
        lds_tr8_rows(lds_offset(base) + (go ^ (16u * ns)), lds_offset(base) + (go ^ (16u * ns + 16u)), d[0], d[1]);
#pragma unroll
        for (int i = 0; i < 2; ++i)
          wf[ns + i] = i32x8{(int)d[i][0].x, (int)d[i][0].y, (int)d[i][1].x, (int)d[i][1].y,
                             (int)d[i][2].x, (int)d[i][2].y, (int)d[i][3].x, (int)d[i][3].y};
      }
    } else {
#pragma unroll
      for (int ns = 0; ns < SN; ++ns) {
        const uint8_t* p = base + 4 * kBlk * ns;
        wf[ns] = frag(*reinterpret_cast<const u32x4*>(p + wo), *reinterpret_cast<const u32x4*>(p + (wo ^ 16u)));
      }
    }
  };

  // One block. Row tile ms + 1 is read and row tile ms - 1 scaled and added while
  // the products of row tile ms are formed. With AHEAD, block next is loaded into
  // stage nstage, a few loads at each row tile: all of them at once would hold the
  // waves up in the memory pipeline's queue before their first product.
  constexpr int kPer = QW + NQX / kNW + 1;  // loads of a stage, by any wave at least
  auto body = [&](auto AHEAD, int stage, int next, int nstage) {
    f32x4 t[2][SN];
    float sp = 0.0f;
    if constexpr (AHEAD.value) issue_scales(next, nstage);
    sc = *reinterpret_cast<const float*>(lds + stage * kStage + so_w);
    read_x(stage, 0);
    read_w(stage);
#pragma unroll
    for (int ms = 0; ms < MS; ++ms) {
      if (ms + 1 < MS) read_x(stage, ms + 1);
      if constexpr (AHEAD.value) {
#pragma unroll
        for (int i = ms * kParts / MS; i < (ms + 1) * kParts / MS; ++i) issue(next, nstage, i);
      }
      __builtin_amdgcn_sched_barrier(0);
      const float s = sc * sx[ms & 1];
#pragma unroll
      for (int ns = 0; ns < SN; ++ns) t[ms & 1][ns] = block_product(wf[ns], xf[ms & 1]);
      if (ms > 0) {
#pragma unroll
        for (int ns = 0; ns < SN; ++ns) add_scaled(acc[ms - 1][ns], sp, t[(ms - 1) & 1][ns]);
      }
      sp = s;
    }
#pragma unroll
    for (int ns = 0; ns < SN; ++ns) add_scaled(acc[MS - 1][ns], sp, t[(MS - 1) & 1][ns]);
  };

#pragma unroll
  for (int s = 0; s < NS - 1; ++s)
    if (s < nc) {
#pragma unroll
      for (int i = 0; i < kParts; ++i) issue(cb0 + s, s, i);
      issue_scales(cb0 + s, s);
    }
  int j = 0;
  if (TM * wm < tr.rows) {
    for (; j < nc - (NS - 1); ++j) {
      wait_vm_barrier<(NS - 2) * kPer>();
      body(std::true_type{}, j % NS, cb0 + j + NS - 1, (j + NS - 1) % NS);
    }
    for (; j < nc; ++j) {
      wait_vm_barrier<0>();
      body(std::false_type{}, j % NS, 0, 0);
    }
  } else {
    // a wave whose rows are all past the tile's last only loads (1322 x 19456 x
    // 2560, 42 rows in the last tile of 256: 77.7 -> 73 us)
    for (; j < nc - (NS - 1); ++j) {
      wait_vm_barrier<(NS - 2) * kPer>();
      issue_scales(cb0 + j + NS - 1, (j + NS - 1) % NS);
#pragma unroll
      for (int i = 0; i < kParts; ++i) issue(cb0 + j + NS - 1, (j + NS - 1) % NS, i);
    }
    for (; j < nc; ++j) wait_vm_barrier<0>();
  }

  // ---- epilogue: lane holds row 16 ms + r16 of the wave's, columns col(ns) .. + 3
  auto col = [&](int ns) { return GRAD ? 16 * ns + 4 * q4 : 4 * SN * q4 + 4 * ns; };
  const int ow = o0 + TN * wn;   // the wave's first column
  if (a.part == nullptr) {
    static_assert(kNW * TM * TN * 2 <= NS * kStage, "the outputs fit the stages");
    __syncthreads();
    uint8_t* reg = lds + wv * (TM * TN * 2);
    uint16_t* y = a.y + (size_t)tr.row0 * O;
    // (four columns per lane stored one by one: 1322 x 19457 x 2560 143 us, 74 so)
    if (GRAD || O % 8 == 0)
      store_tile_bf16<TM, TN>(reg, acc, col, make_rsrc(y, (uint32_t)tr.rows * (uint32_t)O * 2u), TM * wm, ow, O, lane);
    else
      store_tile_bf16_odd<TM, TN>(reg, acc, col, y, tr.rows, TM * wm, ow, O, lane);
    return;
  }
  typedef float f32x4_a4 __attribute__((ext_vector_type(4), aligned(4)));
  float* part = a.part + ((size_t)blockIdx.y * a.M + tr.row0) * O;
#pragma unroll
  for (int ms = 0; ms < MS; ++ms) {
    const int row = TM * wm + 16 * ms + r16;
    if (row >= tr.rows) continue;
#pragma unroll
    for (int ns = 0; ns < SN; ++ns) {
      const int c = ow + col(ns);
      float* p = part + (size_t)row * O + c;
      if (c + 4 <= O) {
        *reinterpret_cast<f32x4_a4*>(p) = acc[ms][ns];
      } else {
#pragma unroll
        for (int i = 0; i < 3; ++i)
          if (c + i < O) p[i] = acc[ms][ns][i];
      }
    }
  }
}

// ---------------------------------------------------------------- few rows
// Up to 16 rows: the weights stream from memory straight into the MFMA's operand
// registers, each once; the 8 waves of a workgroup take every eighth contraction
// block of the same 16 NT columns and add their sums through LDS, in wave order. A
// workgroup takes column tiles gridDim.x apart, and each wave's blocks of all of
// them are one sequence, with U blocks in flight throughout. XR > 0: the rows, XR
// (8 or 16) of them, lie in LDS: from L2 they would cost as much traffic as the
// weights (16 rows of 17408 x 5120: 32 us against 18.5). A wave reads its own blocks
// of them only, so it loads them itself, each with the weights of the first tile that
// it multiplies, and waits for no one (16 x 8192 x 8192 13.3 us; 16.6 with all rows
// loaded first, by all waves).
// Bound by the weights' stream: 1 x 17408 x 5120 16.9 us (5.3 TB/s), 16 x 8192 x 8192
// 13.3 us (5.0 TB/s), 96 rows of 64 experts of 2048 x 4096 77 us (4.7 TB/s: 43 or 44
// experts have rows).
template <int NT>
constexpr int kRowsSums = 2 * kNW * NT * 256 * 4;   // bytes of the sums, two buffers

template <int NT, int U, bool GROUPED, int XR>
__global__ __launch_bounds__(64 * kNW) void fp8_rows_kernel(const Fp8Args a) {
  constexpr int TC = 16 * NT;
  constexpr int kSum = NT * 256;
  constexpr int XB = XR * kBlk;   // bytes of a block of the rows
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  float* const sums = reinterpret_cast<float*>(lds);                       // [2][kNW][kSum]
  uint8_t* const xl = lds + kRowsSums<NT>;                                 // [KB + 1][XR][128 B]
  const int lane = threadIdx.x & 63;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, q4 = lane >> 4;

  TileRows tr{0, 16 * (int)blockIdx.y, min(16, a.M - 16 * (int)blockIdx.y)};
  int first = blockIdx.x, step = gridDim.x, end = a.otiles;
  if constexpr (GROUPED) {
    const GroupScan gs(a.m_sizes, a.G, a.M, 16);
    const int nblocks = gs.tiles * a.otiles;
    if ((int)blockIdx.x >= nblocks) return;
    int mt, ot;
    tile_coords(blockIdx.x, nblocks, gs.tiles, a.otiles, &mt, &ot);
    tr = gs.find(mt);
    if (tr.rows <= 0) return;
    first = ot;
    step = a.otiles;   // one tile
  }
  const int K = a.K, KB = K / kBlk, NB = (a.N + kBlk - 1) / kBlk;
  const uint8_t* wg = a.w + (size_t)tr.wg * a.N * K;
  const __amdgpu_buffer_rsrc_t rxs = make_rsrc(a.xs + (size_t)tr.row0 * KB, (uint32_t)tr.rows * (uint32_t)KB * 4u);
  const __amdgpu_buffer_rsrc_t rws = make_rsrc(a.ws + (size_t)tr.wg * NB * KB, (uint32_t)NB * (uint32_t)KB * 4u);
  const uint32_t roff = (uint32_t)r16 * (uint32_t)K + 32u * (uint32_t)q4;

  const int nb = (KB + kNW - 1) / kNW;                      // blocks of a wave and tile
  const int tiles = first < end ? (end - first + step - 1) / step : 0;
  const int total = tiles * nb;

  // row scales in LDS, [KB][XR]: on their way while the first blocks are requested
  float* const sl = reinterpret_cast<float*>(xl + (KB + 1) * XB);
  constexpr int kSl = XR > 0 ? (int)((kRowsLds / kBlk + 64 * kNW - 1) / (64 * kNW)) : 1;   // XR KB XB <= kRowsLds
  uint32_t rs[kSl];
  if constexpr (XR > 0) {
#pragma unroll
    for (int j = 0; j < kSl; ++j) {
      const int i = (int)threadIdx.x + 64 * kNW * j;   // (rows past the last: zero)
      rs[j] = ld32(rxs, i < XR * KB ? (uint32_t)((i % XR) * KB + i / XR) * 4u : 0xFFFFFFF0u);
    }
  }

  // row r of a block: 16-byte chunk c in slot c ^ pair_swz(r / 2)
  uint32_t xoff[2];
#pragma unroll
  for (int d = 0; d < 2; ++d)
    xoff[d] = (uint32_t)(8 * d + (lane >> 3)) * (uint32_t)K +
              16u * ((uint32_t)(lane & 7) ^ pair_swz(4 * d + (lane >> 4)));

  u32x4 wr[U][NT][2], xr[XR > 0 ? 1 : U][2];
  uint32_t sx[XR > 0 ? 1 : U], sc[U];
  // the next block to load: tile lt, block lu of it
  int lt = first, lu = 0;
  auto load = [&](int u) {
    const int b = wv + kNW * lu;
    // a wave's last block may be past the end: extents of zero, so that nothing is
    // read and the products are zero
    const bool in = b < KB && lt < end;
    const int o0 = lt * TC;
    const uint32_t so = (uint32_t)b * kBlk;
    if constexpr (XR > 0) {
      // (past the first tile zeros, to a block that is not read)
      const bool xin = b < KB && lt == first;
      const __amdgpu_buffer_rsrc_t rx =
          make_rsrc(a.x + (size_t)tr.row0 * K, xin ? (uint32_t)tr.rows * (uint32_t)K : 0u);
      uint8_t* dst = xl + (xin ? b : KB) * XB;
#pragma unroll
      for (int d = 0; d < XR / 8; ++d) dma16(rx, dst + 1024 * d, xoff[d], so);
      // ahead of the weights: once those are there, so are the rows (compute())
      asm volatile("" ::: "memory");
    }
    const __amdgpu_buffer_rsrc_t rw =
        make_rsrc(wg + (size_t)o0 * K, in ? (uint32_t)min(TC, a.N - o0) * (uint32_t)K : 0u);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      wr[u][t][0] = ld128(rw, roff + (uint32_t)(16 * t) * (uint32_t)K, so);
      wr[u][t][1] = ld128(rw, roff + (uint32_t)(16 * t) * (uint32_t)K + 16u, so);
    }
    if constexpr (XR == 0) {
      const __amdgpu_buffer_rsrc_t rx =
          make_rsrc(a.x + (size_t)tr.row0 * K, in ? (uint32_t)tr.rows * (uint32_t)K : 0u);
      xr[u][0] = ld128(rx, roff, so);
      xr[u][1] = ld128(rx, roff + 16u, so);
      sx[u] = ld32(rxs, (uint32_t)r16 * (uint32_t)KB * 4u, (uint32_t)min(b, KB - 1) * 4u);
    }
    // TC divides 128: the tile's columns lie in one block. (The whole offset is a
    // vector offset, which the extent checks: past the last tile it lies outside.)
    sc[u] = ld32(rws, ((uint32_t)(o0 / kBlk) * (uint32_t)KB + (uint32_t)b) * 4u);
    if constexpr (XR > 0) asm volatile("" ::: "memory");   // the blocks' loads stay apart: one block's are waited for
    if (++lu == nb) {
      lu = 0;
      lt += step;
    }
  };

  f32x4 acc[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) acc[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int u = 0; u < U; ++u) {
    load(u);
  }
  if constexpr (XR > 0) {
#pragma unroll
    for (int j = 0; j < kSl; ++j) {
      const int i = (int)threadIdx.x + 64 * kNW * j;
      if (i < XR * KB) sl[i] = __uint_as_float(rs[j]);
    }
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
  }
  const int xrow = XR == 8 ? r16 & 7 : r16;   // (rows past the last are not stored)
  const uint32_t xo = (uint32_t)xrow * kBlk + 16u * ((uint32_t)(2 * q4) ^ pair_swz(xrow >> 1));
  int ct = first, cu = 0, buf = 0;   // the block to compute
  auto compute = [&](auto NEXT, int u) {   // NEXT: another block is requested in its place
    const int b = wv + kNW * cu;
    i32x8 xf;
    float f;
    if constexpr (XR > 0) {
      // the rows of this block were requested ahead of its weights: here once those are
      asm volatile("" : "+v"(wr[u][0][0]) : : "memory");
      const int bx = min(b, KB - 1);
      const uint8_t* p = xl + bx * XB;
      xf = frag(*reinterpret_cast<const u32x4*>(p + xo), *reinterpret_cast<const u32x4*>(p + (xo ^ 16u)));
      f = sl[bx * XR + xrow];
    } else {
      xf = frag(xr[u][0], xr[u][1]);
      f = __uint_as_float(sx[u]);
    }
    f *= __uint_as_float(sc[u]);
    if constexpr (XR > 0) asm volatile("" : "+v"(f));   // (not in the branches below, which would hold the reads back)
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const f32x4 p = block_product(frag(wr[u][t][0], wr[u][t][1]), xf);
      if (b < KB) add_scaled(acc[t], f, p);
    }
    if constexpr (NEXT.value) load(u);
    if (++cu == nb) {
      // ---- the tile's sums
      float* sm = sums + buf * kNW * kSum;
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        *reinterpret_cast<f32x4*>(sm + wv * kSum + t * 256 + r16 * 16 + 4 * q4) = acc[t];
        acc[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      }
      // (the loads in flight are not waited for; the other buffer's readers are
      // past this barrier before it is written again)
      asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
      const int o0 = ct * TC;
      for (int e = threadIdx.x; e < kSum; e += 64 * kNW) {
        const int row = e / TC, c = e % TC;
        const int at = (c >> 4) * 256 + row * 16 + (c & 15);
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < kNW; ++w) v += sm[w * kSum + at];
        if (row < tr.rows && o0 + c < a.N) a.y[(size_t)(tr.row0 + row) * a.N + o0 + c] = to_bf16(v);
      }
      buf ^= 1;
      cu = 0;
      ct += step;
    }
  };
  int s = 0;
  if constexpr (XR == 0) {
    for (; s < total; s += U) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (s + u >= total) break;
        compute(std::true_type{}, u);
      }
    }
  } else {
    // Whole rounds of U, then the rest: with an exit within the loop the compiler
    // sees ways round it on which a block was requested last, and waits as if it were
    // (16 x 8192 x 8192: 13.8 us against 13.3).
    for (; s + U <= total; s += U) {
#pragma unroll
      for (int u = 0; u < U; ++u) compute(std::true_type{}, u);
    }
#pragma unroll
    for (int u = 0; u < U - 1; ++u)
      if (s + u < total) compute(std::false_type{}, u);
  }
}

// ---------------------------------------------------------------- launches
template <int BM, int WM, int NS, bool GRAD>
static hipError_t launch_fp8_tile_t(Fp8Args a, int sk, hipStream_t stream) {
  constexpr int lds_bytes = NS * fp8_stage_bytes<BM>();
  static_assert(lds_bytes <= 160 * 1024, "LDS");
  static std::atomic<uint64_t> lds_set{0};
  const hipError_t ea =
      ensure_dyn_lds(reinterpret_cast<const void*>(&fp8_tile_kernel<BM, WM, NS, GRAD>), lds_bytes, lds_set);
  if (ea != hipSuccess) return ea;
  a.mtiles = a.m_sizes != nullptr ? group_tiles_bound(a.M, BM, a.G) : (a.M + BM - 1) / BM;
  a.otiles = ((GRAD ? a.K : a.N) + kBN - 1) / kBN;
  const long long blocks = (long long)a.mtiles * a.otiles;
  if (blocks > kMaxBlocks) return hipErrorInvalidValue;
  hipLaunchKernelGGL((fp8_tile_kernel<BM, WM, NS, GRAD>), dim3((unsigned)blocks, sk), dim3(64 * kNW), lds_bytes,
                     stream, a);
  return hipGetLastError();
}

template <int XR>
static hipError_t launch_fp8_rows_t(Fp8Args a, int grid, hipStream_t stream) {
  static std::atomic<uint64_t> lds_set{0};
  const hipError_t ea =
      ensure_dyn_lds(reinterpret_cast<const void*>(&fp8_rows_kernel<1, 4, false, XR>), kRowsLds, lds_set);
  if (ea != hipSuccess) return ea;
  a.otiles = (a.N + 15) / 16;
  const dim3 blocks((unsigned)min(grid, a.otiles), (unsigned)((a.M + 15) / 16));
  hipLaunchKernelGGL((fp8_rows_kernel<1, 4, false, XR>), blocks, dim3(64 * kNW), (unsigned)fp8_rows_lds(a.M, a.K),
                     stream, a);
  return hipGetLastError();
}

template <int NT, int U>
static hipError_t launch_fp8_rows_grouped_t(Fp8Args a, hipStream_t stream) {
  a.otiles = (a.N + 16 * NT - 1) / (16 * NT);
  const long long blocks = (long long)group_tiles_bound(a.M, 16, a.G) * a.otiles;
  if (blocks > kMaxBlocks) return hipErrorInvalidValue;
  hipLaunchKernelGGL((fp8_rows_kernel<NT, U, true, 0>), dim3((unsigned)blocks), dim3(64 * kNW), kRowsSums<NT>, stream,
                     a);
  return hipGetLastError();
}

// Plain: 16 columns at a time by workgroups that stay, two per compute unit where
// their LDS allows it. By expert: a workgroup per tile (fp8_rows_tiles).
static hipError_t launch_fp8_rows(const Fp8Args& a, int cus, hipStream_t stream) {
  if (a.m_sizes != nullptr) {
    const int nt = fp8_rows_tiles(a.M, a.N, a.G, cus);
    return nt == 4 ? launch_fp8_rows_grouped_t<4, 2>(a, stream)
           : nt == 2 ? launch_fp8_rows_grouped_t<2, 4>(a, stream) : launch_fp8_rows_grouped_t<1, 4>(a, stream);
  }
  const int grid = 2 * fp8_rows_lds(a.M, a.K) <= kRowsLds ? 2 * cus : cus;
  return a.M <= 8 ? launch_fp8_rows_t<8>(a, grid, stream) : launch_fp8_rows_t<16>(a, grid, stream);
}

// stages: as many as fit LDS
template <bool GRAD>
static hipError_t launch_fp8_tile_bm(const Fp8Args& a, int sk, int bm, hipStream_t stream) {
  switch (bm) {
    case 256: return launch_fp8_tile_t<256, 2, 2, GRAD>(a, sk, stream);
    case 224: return launch_fp8_tile_t<224, 2, 2, GRAD>(a, sk, stream);
    case 192: return launch_fp8_tile_t<192, 2, 2, GRAD>(a, sk, stream);
    case 160: return launch_fp8_tile_t<160, 2, 3, GRAD>(a, sk, stream);
    case 128: return launch_fp8_tile_t<128, 2, 3, GRAD>(a, sk, stream);
    case 96: return launch_fp8_tile_t<96, 2, 3, GRAD>(a, sk, stream);
    case 64: return launch_fp8_tile_t<64, 1, 3, GRAD>(a, sk, stream);
    case 32: return launch_fp8_tile_t<32, 1, 4, GRAD>(a, sk, stream);
    default: return hipErrorInvalidValue;
  }
}

hipError_t launch_fp8_gemm(const uint8_t* x, const float* xs, const uint8_t* w, const float* ws, uint16_t* y,
                           float* part, const int32_t* m_sizes, int M, int N, int K, int G, bool grad, int cps, int sk,
                           int bm, int cus, hipStream_t stream) {
  const Fp8Args a = {x, xs, w, ws, y, part, m_sizes, M, N, K, G, cps, 0, 0};
  if (bm == 16) return grad || sk != 1 ? hipErrorInvalidValue : launch_fp8_rows(a, cus, stream);
  return grad ? launch_fp8_tile_bm<true>(a, sk, bm, stream) : launch_fp8_tile_bm<false>(a, sk, bm, stream);
}

}  // namespace w4a16
