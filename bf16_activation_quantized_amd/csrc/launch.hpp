// Host-side launchers of the device kernels (internal to the library).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>

namespace w4a16 {

struct LoraArgs;   // lora.hpp: per-row adapters, which the projection's kernels add to their sums

// Raises a kernel's dynamic-LDS limit to `bytes` on the current device, once
// per device: `done` is the caller's per-kernel set of devices already set
// (bit d = device d; a device index past 63 sets it on every call).
inline hipError_t ensure_dyn_lds(const void* fn, int bytes, std::atomic<uint64_t>& done) {
  int dev = -1;
  if (hipGetDevice(&dev) != hipSuccess) dev = -1;
  const uint64_t bit = (dev >= 0 && dev < 64) ? (uint64_t{1} << dev) : 0;
  if (bit != 0 && (done.load(std::memory_order_acquire) & bit) != 0) return hipSuccess;
  const hipError_t e = hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == hipSuccess && bit != 0) done.fetch_or(bit, std::memory_order_release);
  return e;
}

hipError_t launch_pack_int4(const uint8_t* q, uint8_t* out, uint64_t total_in, hipStream_t stream);
hipError_t launch_splitk_reduce(const float* ws, uint16_t* y, uint64_t mn, int sk, hipStream_t stream);

// M = 1 decode GEMV; gps = 128-groups per split-K slice (<= 64), sk slices;
// ws == nullptr writes bf16 y, else fp32 partials ws[s, 0, :]. The MFMA layout
// where the slice length has a tiling of 16 (row, group) pairs per
// instruction, otherwise (or when forced) the half-wave layout. la: the row's
// adapter (MFMA layout only).
hipError_t launch_gemv_m1(const uint16_t* x, const uint8_t* w, const uint16_t* s, uint16_t* y, float* ws,
                          int N, int K, int gps, int sk, bool force_halfwave, hipStream_t stream,
                          const LoraArgs* la = nullptr);
bool gemv_mfma_fits(int gps);   // the MFMA layout takes slices of gps groups

// 1 <= M <= kSkinnyMaxRows decode on MFMA 16x16x32; nt column tiles of 16 per
// wave (1 or 2), 8 waves per workgroup (past 32 rows only nt = 1).
hipError_t launch_skinny(const uint16_t* x, const uint8_t* w, const uint16_t* s, uint16_t* y, float* ws,
                         int M, int N, int K, int gps, int sk, int nt, int waves, hipStream_t stream,
                         const LoraArgs* la = nullptr);

// 1 <= M <= 16 decode with X and the weights staged in LDS by DMA (skinny_lds.hip)
bool skinny_lds_fits(int M, int gps);
hipError_t launch_skinny_lds(const uint16_t* x, const uint8_t* w, const uint16_t* s, uint16_t* y, float* ws, int M,
                             int N, int K, int gps, int sk, int geometry, hipStream_t stream,
                             const LoraArgs* la = nullptr);

// slices of at most this many groups stage their scales in LDS (16 NT x gps x 2
// bytes, at most 32 KiB)
constexpr int kSkinnyMaxScaleGroups = 256;
// rows of the small-batch kernel: 16 per row tile, two or three row tiles
// with 8 waves of 1 or 2 column tiles
constexpr int kSkinnyMaxRows = 48;

// out[g * ld + m] = -136 * sum_{k in group g} x[m, k], groups of gsize = 128 or 32 k
hipError_t launch_rowsum_neg136(const uint16_t* x, float* out, int M, int K, int ld, int gsize,
                                hipStream_t stream);

// LDS-DMA tile GEMM with bm x 256 output tiles (bm = 48 .. 144 rows in steps
// of 16; scale groups of gsize = 128 or 32 k, see tile_rows_ok): plain
// (m_sizes == nullptr, m_uniform == 0, G == 1), grouped (rows per weight group
// in m_sizes on the device) or batched (G weight groups of m_uniform rows
// each). With ws != nullptr (plain and batched) slice s of gridDim.y = sk
// writes fp32 partials ws[s, :, :]. la (plain): per-row adapters, dealt
// out over the slices. sxn: the -136 * row sums [K/gsize, ld] of
// launch_rowsum_neg136, or nullptr for the kernel to form them itself.
hipError_t launch_tile(const uint16_t* x, const uint8_t* w, const uint16_t* s, const float* sxn, int ld, uint16_t* y,
                       float* ws, const int32_t* m_sizes, int m_uniform, int M_total, int N, int K, int G, int gps,
                       int sk, int bm, int gsize, hipStream_t stream, const LoraArgs* la = nullptr);
// whether the tile kernel is built for bm-row tiles at scale group gsize
bool tile_rows_ok(int bm, int gsize);
constexpr int kTileCols = 256;

// ---- low-rank adapters beside the projection (lora.hip)
// h = sc * x . A^T as two bf16 parts [2, M, R] (rows with an adapter only);
// with rowsums != nullptr launch_rowsum_neg136's work too
hipError_t launch_lora_shrink(const uint16_t* x, const uint16_t* a, const int32_t* ids, const float* scaling,
                              uint16_t* h, int M, int K, int L, int R, float* rowsums, int ld, int gsize,
                              hipStream_t stream);

// ---- rows of a mixture of experts (experts.hip)
constexpr int kExpertMaxGroups = 4096;
int expert_sort_blocks(int64_t S, int G);   // past one: a row of G + 1 counts of workspace for each, and one more
hipError_t launch_expert_sort(const int32_t* ids, int32_t* order, int32_t* pos, int32_t* m_sizes, int64_t S, int G,
                              int32_t* ws, hipStream_t stream);
hipError_t launch_expert_gather(const uint16_t* x, const int32_t* pos, uint16_t* xs, int64_t T, int k, int64_t rows,
                                int width, hipStream_t stream);
// w == nullptr: all weights 1
hipError_t launch_expert_combine(const uint16_t* z, const int32_t* pos, const float* w, uint16_t* y, int64_t T, int k,
                                 int64_t rows, int width, hipStream_t stream);
hipError_t launch_expert_combine_grad(const uint16_t* dy, const uint16_t* z, const int32_t* pos, const float* w,
                                      uint16_t* dz, float* dw, int64_t T, int k, int64_t rows, int width,
                                      hipStream_t stream);

// Workgroups of 512 threads in one launch: fewer than 2^32 threads, past which a grid
// is cut short without an error.
constexpr int64_t kMaxBlocks = ((int64_t)1 << 23) - 1;

// Row tiles of height bm that M rows in G groups take at most: each of the groups
// that have rows (at most min(G, M)) ends in a tile that may hold a single row.
inline int group_tiles_bound(int M, int bm, int G) {
  return (int)(((long long)M + (long long)(bm - 1) * (G < M ? G : M)) / bm);
}

// ---- 8-bit products with a scale for each block of 128 (fp8.hip)
// scales of blocks of block_rows (1 or 128) x 128
hipError_t launch_fp8_quantize(const uint16_t* x, uint8_t* q, float* scales, int64_t M, int K, int block_rows,
                               hipStream_t stream);
// LDS of the kernel for few rows: the sums of 16 columns, the rows (8 or 16, one
// block of them spare) and their scales. It takes rows that fit (kRowsLds).
constexpr int64_t kRowsLds = 160 * 1024;
constexpr int64_t fp8_rows_lds(int64_t M, int64_t K) {
  const int64_t kb = K / 128, r = M <= 8 ? 8 : 16;
  return 2 * 8 * 256 * 4 + (kb + 1) * r * 128 + kb * r * 4;
}
// The same by expert: column tiles of 16 per workgroup. A workgroup per tile, of 64
// columns while that leaves two tiles per compute unit, else of 32 or 16 (96 rows of 64
// experts, 2048 x 4096: 77.4 us with 64 columns, 88.7 with 32, 118 with 16).
inline int fp8_rows_tiles(int M, int N, int G, int cus) {
  const long long tiles = G < M ? G : M;   // at least so many with rows, if rows are spread
  return tiles * ((N + 63) / 64) >= 2 * cus ? 4 : tiles * ((N + 31) / 32) >= 2 * cus ? 2 : 1;
}
// grad: the input gradient (x: dY, contraction over N). bm: rows per tile (16:
// the kernel for few rows, whole contractions of the products only). With
// part != nullptr slice s of sk, cps contraction blocks, writes fp32
// partials part[s, :, :]. cus: compute units of the device.
hipError_t launch_fp8_gemm(const uint8_t* x, const float* xs, const uint8_t* w, const float* ws, uint16_t* y,
                           float* part, const int32_t* m_sizes, int M, int N, int K, int G, bool grad, int cps, int sk,
                           int bm, int cus, hipStream_t stream);

// The split-K reduce of the rows that m_sizes names: those behind the last group's
// are left as they were. K a multiple of 8.
hipError_t launch_splitk_reduce_rows(const float* ws, uint16_t* y, const int32_t* m_sizes, int G, int M, int K, int sk,
                                     hipStream_t stream);

// ---- input gradient of the 4-bit products (w4grad.hip)
constexpr int64_t w4_grad_padded(int64_t N) { return (N + 127) / 128 * 128; }
// Prepass: threads per row of dY, as few as hold it in registers (a row is a chain of a
// load, a reduction and a store: 2048 rows of 2048 15.5 us with 512 threads each, 8 with
// 64); workgroups per 128 n of an expert's Kg groups of scales; all workgroups.
constexpr int kPrepThreads = 512;
constexpr int kPrepRegs = 5;     // times 8 elements per thread
constexpr int kPrepWide = 128;   // groups of scales read as one run
constexpr int w4_grad_row_threads(int N) {
  int t = 64;
  while (t < kPrepThreads && N > t * 8 * kPrepRegs) t *= 2;
  return t;
}
constexpr int w4_grad_scale_blocks(int Kg) { return Kg <= kPrepWide ? 1 : (Kg + 63) / 64; }
constexpr int64_t w4_grad_prep_blocks(int64_t G, int64_t M, int N, int Kg) {
  const int rows = kPrepThreads / w4_grad_row_threads(N);
  return G * (w4_grad_padded(N) / 128) * w4_grad_scale_blocks(Kg) + (M + rows - 1) / rows;
}
struct W4GradPlan {
  int bm, sk;                       // rows per tile, slices of the contraction
  uint64_t h, up, st, tops, part;   // byte offsets into the workspace
  uint64_t bytes;
};
hipError_t launch_w4_grad(const uint16_t* dy, const uint8_t* w, const uint16_t* s, uint16_t* dx, const int32_t* m_sizes,
                          int M, int N, int K, int G, int gsize, const W4GradPlan& p, uint8_t* ws, hipStream_t stream);

}  // namespace w4a16
