// Low-rank adapters of many requests beside the shared W4A16 projection:
//
//   h[m, r] = sc[l] * sum_k x[m, k] A[l, r, k],  l = ids[m]
//   y[m, n] = bf16(base[m, n] + sum_r h[m, r] B[l, n, r])
//
// base is the projection's fp32 sum (split-K slices included), so y is rounded
// once. Rows whose id is outside [0, L) get the projection alone; an adapter's
// values never reach a row of another adapter (per-adapter products are
// selected by row, not masked by zeros, so infinities and NaN stay where they
// are).
#include "common.hpp"
#include "launch.hpp"

namespace w4a16 {

namespace {

__device__ __forceinline__ f32x4 mfma32(bf16x8 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ bf16x8 frag(u32x4 v) { return __builtin_bit_cast(bf16x8, v); }

constexpr uint32_t kOutside = 0xFFFFFFF0u;   // a buffer offset past every extent: the load returns zeros

}  // namespace

// ---------------------------------------------------------------- x . A^T
// Block (row tile of 16, K slice): hp[slice][m][r] = sc * the slice's part of
// the sum, for the rows that have an adapter. The 4 waves take the slice's
// 128-k blocks in turn and are summed through LDS in wave order.
template <int RT>   // rank tiles of 16
__global__ __launch_bounds__(256) void lora_shrink_kernel(const uint16_t* __restrict__ x,
                                                          const uint16_t* __restrict__ a,
                                                          const int32_t* __restrict__ ids,
                                                          const float* __restrict__ scaling, float* __restrict__ hp,
                                                          int M, int K, int L, int R, int gps) {
  __shared__ f32x4 red[4][RT][64];
  const int lane = threadIdx.x & 63;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int m16 = lane & 15, kb = lane >> 4;
  const int m0 = blockIdx.x * 16;
  const int Gk = K / kGroup;
  const int gb = blockIdx.y * gps, ge = min(Gk, gb + gps);
  const int row = m0 + m16;
  const int id = row < M ? ids[row] : -1;
  uint64_t todo = __ballot((uint32_t)id < (uint32_t)L) & 0xFFFFull;
  const __amdgpu_buffer_rsrc_t rx = make_rsrc(x + (size_t)m0 * K, (uint32_t)min(16, M - m0) * (uint32_t)K * 2u);
  while (todo != 0) {
    const int l = __builtin_amdgcn_readlane(id, __builtin_ctzll(todo));
    const uint64_t mine = __ballot(id == l) & 0xFFFFull;
    todo &= ~mine;
    const __amdgpu_buffer_rsrc_t ra = make_rsrc(a + (size_t)l * R * K, (uint32_t)R * (uint32_t)K * 2u);
    f32x4 acc[RT];
#pragma unroll
    for (int t = 0; t < RT; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int g = gb + wv; g < ge; g += 4) {
#pragma unroll
      for (int st = 0; st < 4; ++st) {
        const uint32_t ko = ((uint32_t)g * 128u + 32u * st + 8u * (uint32_t)kb) * 2u;
        const bf16x8 xa = frag(ld128(rx, (uint32_t)m16 * (uint32_t)K * 2u + ko));
#pragma unroll
        for (int t = 0; t < RT; ++t)
          acc[t] = mfma32(xa, frag(ld128(ra, (uint32_t)(16 * t + m16) * (uint32_t)K * 2u + ko)), acc[t]);
      }
    }
    __syncthreads();
#pragma unroll
    for (int t = 0; t < RT; ++t) red[wv][t][lane] = acc[t];
    __syncthreads();
    const float sc = scaling != nullptr ? scaling[l] : 1.0f;
    for (int t = wv; t < RT; t += 4) {
      f32x4 v = red[0][t][lane];
      for (int q = 1; q < 4; ++q) {
        const f32x4 p = red[q][t][lane];
        v.x += p.x;
        v.y += p.y;
        v.z += p.z;
        v.w += p.w;
      }
      // lane: rows 4 kb + i, rank 16 t + m16
      const float f[4] = {v.x, v.y, v.z, v.w};
      if (16 * t + m16 < R)
        for (int i = 0; i < 4; ++i)
          if ((mine >> (4 * kb + i)) & 1)
            hp[((size_t)blockIdx.y * M + m0 + 4 * kb + i) * R + 16 * t + m16] = sc * f[i];
    }
  }
}

// ---------------------------------------------------------------- + h . B^T
// Block (row tile of 16, 256 columns): the sum of the projection's fp32 slices
// plus each adapter's product for its rows. h enters the matrix core as two
// bf16 parts (its rounding and the rounding of what is left), which keeps 16
// of its bits.
__global__ __launch_bounds__(256) void lora_expand_kernel(const float* __restrict__ ws, const float* __restrict__ hp,
                                                          const uint16_t* __restrict__ b,
                                                          const int32_t* __restrict__ ids, uint16_t* __restrict__ y,
                                                          int M, int N, int L, int R, int sk, int ks) {
  const int lane = threadIdx.x & 63;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int m16 = lane & 15, kb = lane >> 4;
  const int nt = (N + 255) / 256;
  const int m0 = (int)(blockIdx.x / nt) * 16, n0 = (int)(blockIdx.x % nt) * 256 + 64 * wv;
  const int row = m0 + m16;
  const int id = row < M ? ids[row] : -1;
  f32x4 acc[4];
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int n = n0 + 16 * t + m16;
    for (int s = 0; s < sk; ++s)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int m = m0 + 4 * kb + i;
        if (m < M && n < N) acc[t][i] += ws[((size_t)s * M + m) * N + n];
      }
  }
  uint64_t todo = __ballot((uint32_t)id < (uint32_t)L) & 0xFFFFull;
  while (todo != 0) {
    const int l = __builtin_amdgcn_readlane(id, __builtin_ctzll(todo));
    const uint64_t mine = __ballot(id == l) & 0xFFFFull;
    todo &= ~mine;
    const __amdgpu_buffer_rsrc_t rb = make_rsrc(b + (size_t)l * N * R, (uint32_t)N * (uint32_t)R * 2u);
    f32x4 d[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) d[t] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int r0 = 0; r0 < R; r0 += 32) {
      const int r = r0 + 8 * kb;
      float h[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) h[i] = 0.0f;
      if (r < R && ((mine >> m16) & 1)) {
        for (int s = 0; s < ks; ++s)
#pragma unroll
          for (int i = 0; i < 8; ++i) h[i] += hp[((size_t)s * M + row) * R + r + i];
      }
      u32x4 hi, lo;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        hi[i] = pack_bf16x2(h[2 * i], h[2 * i + 1]);
        lo[i] = pack_bf16x2(h[2 * i] - bf16lo(hi[i]), h[2 * i + 1] - bf16hi(hi[i]));
      }
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const int n = n0 + 16 * t + m16;
        const bf16x8 bv = frag(ld128(rb, r < R && n < N ? ((uint32_t)n * (uint32_t)R + (uint32_t)r) * 2u : kOutside));
        d[t] = mfma32(frag(hi), bv, d[t]);
        d[t] = mfma32(frag(lo), bv, d[t]);
      }
    }
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[t][i] = ((mine >> (4 * kb + i)) & 1) ? acc[t][i] + d[t][i] : acc[t][i];
  }
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    const int n = n0 + 16 * t + m16;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int m = m0 + 4 * kb + i;
      if (m < M && n < N) y[(size_t)m * N + n] = to_bf16(acc[t][i]);
    }
  }
}

hipError_t launch_lora_shrink(const uint16_t* x, const uint16_t* a, const int32_t* ids, const float* scaling,
                              float* hp, int M, int K, int L, int R, int gps, int ks, hipStream_t stream) {
  const dim3 grid((M + 15) / 16, ks);
#define W4A16_SHRINK(RT)                                                                                     \
  hipLaunchKernelGGL(lora_shrink_kernel<RT>, grid, dim3(256), 0, stream, x, a, ids, scaling, hp, M, K, L, R, gps)
  if (R <= 16) W4A16_SHRINK(1);
  else if (R <= 32) W4A16_SHRINK(2);
  else if (R <= 64) W4A16_SHRINK(4);
  else W4A16_SHRINK(8);
#undef W4A16_SHRINK
  return hipGetLastError();
}

hipError_t launch_lora_expand(const float* ws, const float* hp, const uint16_t* b, const int32_t* ids, uint16_t* y,
                              int M, int N, int L, int R, int sk, int ks, hipStream_t stream) {
  const dim3 grid((unsigned)((N + 255) / 256) * (unsigned)((M + 15) / 16));
  hipLaunchKernelGGL(lora_expand_kernel, grid, dim3(256), 0, stream, ws, hp, b, ids, y, M, N, L, R, sk, ks);
  return hipGetLastError();
}

}  // namespace w4a16
