// Low-rank adapters of many requests beside the shared W4A16 projection:
//
//   h[m, r] = sc[l] * sum_k x[m, k] A[l, r, k],  l = ids[m]
//   y[m, n] = bf16(base[m, n] + sum_r h[m, r] B[l, n, r])
//
// The kernels here form h, the first product; the second joins the fp32
// accumulators of the projection's own kernels (lora.hpp), so y is written
// once and rounded once. There h enters the matrix core as two bf16 values
// (its rounding and the rounding of what is left: 16 of its bits). Rows whose id is outside [0, L) get the
// projection alone.
#include "common.hpp"
#include "launch.hpp"
#include "lora.hpp"
#include "rowsum.hpp"

namespace w4a16 {

namespace {

__device__ __forceinline__ bf16x8 frag(u32x4 v) { return __builtin_bit_cast(bf16x8, v); }

constexpr int kWaves = 8;   // per workgroup, in every kernel here

constexpr uint32_t kOutside = 0xFFFFFFF0u;   // a buffer offset past every extent: the load returns zeros

__device__ __forceinline__ void store_h(uint16_t* h, size_t plane, size_t e, float v) {
  const uint16_t hi = to_bf16(v);
  h[e] = hi;
  h[plane + e] = to_bf16(v - bf16f(hi));
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
// Workgroup (turn, row tile of 16, rank tile of 16): MFMA 16x16x32 over the
// whole K range, for every turns-th adapter of the row tile in the order
// of their first row (one, where the rows of a request lie together). The 8
// waves take the 128-k groups in turn; a group of x (only the rows of the
// turn's adapters) and of A is fetched in whole lines (4 rows x 256 bytes per
// instruction) and turned into fragments through the wave's own LDS tile, two
// fetches ahead. x stays in registers while the turn's adapters follow one
// another, and each product is added to the rows of its adapter only (one
// accumulator: a row has one adapter). The waves are summed through LDS in
// wave order.
constexpr int kTileWaves = kWaves;

__device__ __forceinline__ void shrink_tile(const uint16_t* __restrict__ x, const uint16_t* __restrict__ a,
                                            const int32_t* __restrict__ ids, const float* __restrict__ scaling,
                                            uint16_t* __restrict__ h, int M, int K, int L, int R, int block,
                                            int turns) {
  __shared__ u32x4 tile[kTileWaves][16 * 16];   // [row][piece p of a group in slot p ^ row]
  __shared__ f32x4 red[kTileWaves][64];
  const int lane = threadIdx.x & 63;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int m16 = lane & 15, kb = lane >> 4;
  const int rt = (R + 15) / 16, mt = (M + 15) / 16;
  const int r0 = block % rt * 16, m0 = block / rt % mt * 16, me = block / rt / mt;
  const int Gk = K / kGroup;
  const uint32_t KB = (uint32_t)K * 2u;
  int id = m0 + m16 < M ? ids[m0 + m16] : -1;
  id = (uint32_t)id < (uint32_t)L ? id : -1;

  // this turn's adapters (bits: the first row of each) and their rows
  uint32_t lead = 0, own = 0;
  {
    uint32_t todo = (uint32_t)__ballot(id >= 0) & 0xFFFFu;
    for (int turn = 0; todo != 0; turn = turn + 1 == turns ? 0 : turn + 1) {
      const int first = __builtin_ctz(todo);
      const uint32_t rows = (uint32_t)__ballot(id == __builtin_amdgcn_readlane(id, first)) & 0xFFFFu;
      if (turn == me) {
        lead |= 1u << first;
        own |= rows;
      }
      todo &= ~rows;
    }
  }
  if (lead == 0) return;   // the same in every wave

  const __amdgpu_buffer_rsrc_t rx = make_rsrc(x + (size_t)m0 * K, (uint32_t)min(16, M - m0) * KB);
  // row 4 j + kb, 16-byte piece m16 of a group
  const uint32_t off = (uint32_t)kb * KB + 16u * (uint32_t)m16;
  uint32_t xo[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) xo[j] = (own >> (4 * j + kb)) & 1 ? off + (uint32_t)(4 * j) * KB : kOutside;
  struct Item {
    u32x4 xv[4], av[4];
    uint32_t rows;
    bool fresh, live;
  };
  // the sequence of (group, adapter) of this wave
  uint32_t todo = lead;
  int g = wv;
  auto fetch = [&](Item& t) {
    t.live = g < Gk;
    if (!t.live) return;
    t.fresh = todo == lead;
    const int first = __builtin_ctz(todo);
    const int l = __builtin_amdgcn_readlane(id, first);
    t.rows = (uint32_t)__ballot(id == l) & 0xFFFFu;
    const __amdgpu_buffer_rsrc_t ra =   // ranks past R read zeros
        make_rsrc(a + ((size_t)l * R + r0) * K, (uint32_t)min(16, R - r0) * KB);
#pragma unroll
    for (int j = 0; j < 4; ++j) t.av[j] = ld128(ra, off + (uint32_t)(4 * j) * KB + (uint32_t)g * 256u);
    if (t.fresh) {
#pragma unroll
      for (int j = 0; j < 4; ++j) t.xv[j] = ld128(rx, __builtin_elementwise_add_sat(xo[j], (uint32_t)g * 256u));
    }
    todo &= todo - 1;
    if (todo == 0) {
      todo = lead;
      g += kTileWaves;
    }
    __builtin_amdgcn_sched_barrier(0);   // one fetch's loads stay together
  };
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
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  u32x4 xf[4];
  auto use = [&](const Item& t) {
    u32x4 af[4];
    if (t.fresh) turned(t.xv, xf);
    turned(t.av, af);
    f32x4 d = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < 4; ++j) d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(frag(xf[j]), frag(af[j]), d, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] += (t.rows >> (4 * kb + i)) & 1 ? d[i] : 0.0f;
  };
  Item t0, t1;
  fetch(t0);
  fetch(t1);
  while (t0.live) {
    use(t0);
    fetch(t0);
    if (!t1.live) break;
    use(t1);
    fetch(t1);
  }
  red[wv][lane] = acc;
  // the lane's rows' scales, with every lane active (a lane of a rank past R
  // may hold the id)
  float sc[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int l = __shfl(id, 4 * kb + i);
    sc[i] = scaling != nullptr && l >= 0 ? scaling[l] : 1.0f;
  }
  __syncthreads();
  if (wv == 0 && r0 + m16 < R) {
    f32x4 v = red[0][lane];
#pragma unroll
    for (int q = 1; q < kTileWaves; ++q) {
      const f32x4 p = red[q][lane];
      v.x += p.x;
      v.y += p.y;
      v.z += p.z;
      v.w += p.w;
    }
    // lane: rows 4 kb + i, rank r0 + m16
    const float f[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 4 * kb + i;
      if ((own >> r) & 1) store_h(h, (size_t)M * R, (size_t)(m0 + r) * R + r0 + m16, sc[i] * f[i]);
    }
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
  int M, K, L, R, ld, rowsum_blocks, turns;
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
  shrink_tile(p.x, p.a, p.ids, p.scaling, p.h, p.M, p.K, p.L, p.R, (int)blockIdx.x - p.rowsum_blocks, p.turns);
}

// Few rows one by one, more in row tiles: the row kernel reads A once per row,
// the tile kernel once per adapter of 16 rows, but through fewer workgroups
// and in shorter runs. The whole call, row against tile kernel: 64 x 8192 x
// 8192, rank 16, an adapter each 36.9 / 39.9 us, 4 adapters one after the other
// 28.5 / 32.9; 100 x 8192 x 4096, rank 64, 8 adapters, mixed 32.4 / 30.6, one
// after the other 31.4 / 29.4; 333 x 2560 x 9728, group 32, rank 24, 5
// adapters, mixed 54.5 / 54.6, one after the other 53.2 / 49.3. Turns: as many
// as there are adapters, up to 16 and about a thousand workgroups, for row
// tiles of several adapters (the 333 rows mixed: 54.6 us with 4 turns, 50.7
// with 8); a workgroup that finds no adapter left to it ends at once.
template <int GS>
static hipError_t launch_shrink_gs(ShrinkArgs p, hipStream_t stream) {
  p.rowsum_blocks = GS != 0 ? (p.M + kWaves - 1) / kWaves : 0;
  p.turns = 1;
  const int64_t MR = (int64_t)p.M * p.R;
  const dim3 threads(64 * kWaves);
  if (MR <= 4096) {
#define W4A16_ROW(RP) \
  hipLaunchKernelGGL((lora_shrink_row_kernel<RP, GS>), dim3(p.rowsum_blocks + p.M * (p.R / RP)), threads, 0, stream, p)
    // ranks per workgroup: x is read once for all of them, but a few hundred
    // workgroups should be there
    if (MR >= 2048) W4A16_ROW(8);
    else if (MR >= 1024) W4A16_ROW(4);
    else if (MR >= 512) W4A16_ROW(2);
    else W4A16_ROW(1);
#undef W4A16_ROW
    return hipGetLastError();
  }
  const int64_t tiles = (int64_t)((p.M + 15) / 16) * ((p.R + 15) / 16);
  while (p.turns < 16 && p.turns < p.L && tiles * 2 * p.turns <= 1024) p.turns *= 2;
  hipLaunchKernelGGL((lora_shrink_tile_kernel<GS>), dim3((unsigned)(p.rowsum_blocks + tiles * p.turns)), threads, 0,
                     stream, p);
  return hipGetLastError();
}

hipError_t launch_lora_shrink(const uint16_t* x, const uint16_t* a, const int32_t* ids, const float* scaling,
                              uint16_t* h, int M, int K, int L, int R, float* rowsums, int ld, int gsize,
                              hipStream_t stream) {
  const ShrinkArgs p = {x, a, ids, scaling, h, rowsums, M, K, L, R, ld, 0, 1};
  if (rowsums == nullptr) return launch_shrink_gs<0>(p, stream);
  if (gsize == 128) return launch_shrink_gs<128>(p, stream);
  if (gsize == 32) return launch_shrink_gs<32>(p, stream);
  return hipErrorInvalidValue;
}

}  // namespace w4a16
