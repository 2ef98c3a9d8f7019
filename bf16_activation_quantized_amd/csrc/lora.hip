// Low-rank adapters of many requests beside the shared W4A16 projection:
//
//   h[m, r] = sc[l] * sum_k x[m, k] A[l, r, k],  l = ids[m]
//   y[m, n] = bf16(base[m, n] + sum_r h[m, r] B[l, n, r])
//
// The kernels here form h, the first product; the second joins the fp32
// accumulators of the projection's own kernels (lora.hpp), so y is written
// once and rounded once. h is kept as two bf16 values (its rounding and the
// rounding of what is left: 16 of its bits), the operands of the second
// product on the matrix core. Rows whose id is outside [0, L) get the
// projection alone.
#include "common.hpp"
#include "launch.hpp"
#include "lora.hpp"

namespace w4a16 {

namespace {

__device__ __forceinline__ bf16x8 frag(u32x4 v) { return __builtin_bit_cast(bf16x8, v); }

constexpr uint32_t kOutside = 0xFFFFFFF0u;   // a buffer offset past every extent: the load returns zeros

__device__ __forceinline__ void store_h(uint16_t* h, size_t plane, size_t e, float v) {
  const uint16_t hi = to_bf16(v);
  h[e] = hi;
  h[plane + e] = to_bf16(v - bf16f(hi));
}

}  // namespace

// ---------------------------------------------------------------- few rows
// Block (row, RP ranks): dot products on the VALU. The 8 waves take 512-k
// pieces in turn (one contiguous 1 KiB run of x and of each rank's row of A
// per wave instruction), two pieces in flight, and are summed through LDS in
// wave order.
constexpr int kRowWaves = 8;

template <int RP>
__global__ __launch_bounds__(64 * kRowWaves) void lora_shrink_row_kernel(const uint16_t* __restrict__ x,
                                                                         const uint16_t* __restrict__ a,
                                                                         const int32_t* __restrict__ ids,
                                                                         const float* __restrict__ scaling,
                                                                         uint16_t* __restrict__ h, int M, int K, int L,
                                                                         int R) {
  __shared__ float red[kRowWaves][RP];
  const int lane = threadIdx.x & 63;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int m = blockIdx.x, r0 = blockIdx.y * RP;
  const int l = __builtin_amdgcn_readfirstlane(ids[m]);
  if ((uint32_t)l >= (uint32_t)L) return;
  const uint32_t KB = (uint32_t)K * 2u;
  const __amdgpu_buffer_rsrc_t rx = make_rsrc(x + (size_t)m * K, KB);
  const __amdgpu_buffer_rsrc_t ra = make_rsrc(a + ((size_t)l * R + r0) * K, (uint32_t)RP * KB);
  float acc[RP];
#pragma unroll
  for (int r = 0; r < RP; ++r) acc[r] = 0.0f;
  u32x4 xv[2], av[2][RP];
  auto issue = [&](int u, uint32_t c) {
    const uint32_t o = 1024u * c + 16u * (uint32_t)lane;
    const bool ok = o < KB;   // pieces past the row read zeros
    xv[u] = ld128(rx, ok ? o : kOutside);
#pragma unroll
    for (int r = 0; r < RP; ++r) av[u][r] = ld128(ra, ok ? o + (uint32_t)r * KB : kOutside);
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
  const int pieces = (K + 511) / 512;
  issue(0, (uint32_t)wv);
  for (int c = wv; c < pieces; c += 2 * kRowWaves) {
    issue(1, (uint32_t)(c + kRowWaves));
    add(0);
    issue(0, (uint32_t)(c + 2 * kRowWaves));
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
// Block (row tile of 16, rank tile of 16): MFMA 16x16x32 over the whole K
// range. The 8 waves take the 128-k groups in turn; a group of x and of A is
// fetched in whole lines (4 rows x 256 bytes per instruction) and turned into
// fragments through the wave's own LDS tile. Where the row tile holds several
// adapters, x stays in registers while they follow one another, and each
// product is added to the rows of its adapter only (one accumulator: a row has
// one adapter). The next group (or adapter) is in flight meanwhile. The waves
// are summed through LDS in wave order.
constexpr int kTileWaves = 8;

__global__ __launch_bounds__(64 * kTileWaves) void lora_shrink_tile_kernel(
    const uint16_t* __restrict__ x, const uint16_t* __restrict__ a, const int32_t* __restrict__ ids,
    const float* __restrict__ scaling, uint16_t* __restrict__ h, int M, int K, int L, int R) {
  __shared__ u32x4 tile[kTileWaves][16 * 16];   // [row][piece p of the group in slot p ^ row]
  __shared__ f32x4 red[kTileWaves][64];
  const int lane = threadIdx.x & 63;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int m16 = lane & 15, kb = lane >> 4;
  const int m0 = blockIdx.x * 16, r0 = blockIdx.y * 16;
  const int Gk = K / kGroup;
  const int row = m0 + m16;
  const int id = row < M ? ids[row] : -1;
  const uint64_t all = __ballot((uint32_t)id < (uint32_t)L) & 0xFFFFull;
  if (all == 0) return;
  const uint32_t KB = (uint32_t)K * 2u;
  const __amdgpu_buffer_rsrc_t rx = make_rsrc(x + (size_t)m0 * K, (uint32_t)min(16, M - m0) * KB);
  // row 4 j + kb, 16-byte piece m16 of a group
  const uint32_t off = (uint32_t)kb * KB + 16u * (uint32_t)m16;
  auto load = [&](u32x4 (&v)[4], __amdgpu_buffer_rsrc_t rs, int g) {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = ld128(rs, off + (uint32_t)(4 * j) * KB + (uint32_t)g * 256u);
  };
  u32x4* tw = tile[wv];
  // lane (m16, kb) of step j: row m16, piece 4 kb + j (k = 32 kb + 8 j + 0..7, the same in both operands)
  auto turn = [&](const u32x4 (&v)[4], u32x4 (&f)[4]) {
    wave_lds_exchange();
#pragma unroll
    for (int j = 0; j < 4; ++j) tw[16 * (4 * j + kb) + (m16 ^ (4 * j + kb))] = v[j];
    wave_lds_exchange();
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = tw[16 * m16 + ((4 * kb + j) ^ m16)];
  };
  // the sequence of (group, adapter) of this wave
  uint64_t todo = all;
  int g = wv;
  auto adapter = [&](uint64_t& mine) {
    const int l = __builtin_amdgcn_readlane(id, __builtin_ctzll(todo));
    mine = __ballot(id == l) & 0xFFFFull;
    return l;
  };
  auto ranks = [&](int l) {   // ranks past R read zeros
    return make_rsrc(a + ((size_t)l * R + r0) * K, (uint32_t)min(16, R - r0) * KB);
  };
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  if (g < Gk) {
    u32x4 xn[4], an[4], xf[4], af[4];
    uint64_t mine;
    load(an, ranks(adapter(mine)), g);
    load(xn, rx, g);
    bool fresh = true;
    for (;;) {
      if (fresh) turn(xn, xf);
      turn(an, af);
      const uint64_t cur = mine;
      todo &= ~mine;
      fresh = todo == 0;
      if (fresh) {
        todo = all;
        g += kTileWaves;
      }
      const bool more = g < Gk;
      if (more) {
        load(an, ranks(adapter(mine)), g);
        if (fresh) load(xn, rx, g);
      }
      f32x4 d = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int j = 0; j < 4; ++j)
        d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(frag(xf[j]), frag(af[j]), d, 0, 0, 0);
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] += (cur >> (4 * kb + i)) & 1 ? d[i] : 0.0f;
      if (!more) break;
    }
  }
  red[wv][lane] = acc;
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
      const int m = m0 + 4 * kb + i;
      const int l = __shfl(id, 4 * kb + i);
      if ((all >> (4 * kb + i)) & 1)
        store_h(h, (size_t)M * R, (size_t)m * R + r0 + m16, scaling != nullptr ? scaling[l] * f[i] : f[i]);
    }
  }
}

hipError_t launch_lora_shrink(const uint16_t* x, const uint16_t* a, const int32_t* ids, const float* scaling,
                              uint16_t* h, int M, int K, int L, int R, hipStream_t stream) {
  if (M <= kSkinnyMaxRows) {
#define W4A16_ROW(RP)                                                                                      \
  hipLaunchKernelGGL(lora_shrink_row_kernel<RP>, dim3(M, R / RP), dim3(64 * kRowWaves), 0, stream, x, a, ids, \
                     scaling, h, M, K, L, R)
    if (M * R >= 2048) W4A16_ROW(8);
    else if (M * R >= 1024) W4A16_ROW(4);
    else if (M * R >= 512) W4A16_ROW(2);
    else W4A16_ROW(1);
#undef W4A16_ROW
  } else {
    hipLaunchKernelGGL(lora_shrink_tile_kernel, dim3((M + 15) / 16, (R + 15) / 16), dim3(64 * kTileWaves), 0, stream,
                       x, a, ids, scaling, h, M, K, L, R);
  }
  return hipGetLastError();
}

}  // namespace w4a16
