// Row sums of X for the tile kernel, formed ahead of it.
#pragma once

#include "common.hpp"

namespace w4a16 {

// out[g * ld + m] = -136 * sum_{k in group g} x[m, k], fp32, for groups of GS
// = 128 or 32 k: the initial accumulators of the tile kernel's group chains
// when they come from a separate pass (the tile kernel forms them itself
// otherwise). One wave per row; a wave instruction covers 512 consecutive k
// and up to 8 of them are in flight before any is reduced; a group's lanes
// (16 for 128 k, 4 for 32 k) are summed with DPP. Loads past the row read
// zeros (exact buffer extent).
template <int GS>
__device__ __forceinline__ void rowsum_neg136_row(const uint16_t* __restrict__ x, float* __restrict__ out, int m, int M,
                                                  int K, int ld, int lane) {
  constexpr int U = 8;
  constexpr int LPG = GS / 8;   // lanes per group
  if (m >= M) return;
  const __amdgpu_buffer_rsrc_t rx = make_rsrc(x + (size_t)m * K, (uint32_t)K * 2u);
  for (int base = 0; base < K; base += 512 * U) {
    u32x4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) v[u] = ld128(rx, (uint32_t)(base + 512 * u + 8 * lane) * 2u);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = base + 512 * u + 8 * lane;
      float p = (bf16lo(v[u].x) + bf16hi(v[u].x)) + (bf16lo(v[u].y) + bf16hi(v[u].y)) +
                (bf16lo(v[u].z) + bf16hi(v[u].z)) + (bf16lo(v[u].w) + bf16hi(v[u].w));
      if constexpr (LPG == 16) {
        p = row16_sum(p);
      } else {
        p += dpp_f<0xB1>(p);   // quad_perm [1,0,3,2]
        p += dpp_f<0x4E>(p);   // quad_perm [2,3,0,1]
      }
      if ((lane & (LPG - 1)) == 0 && k < K) out[(size_t)(k / GS) * ld + m] = -136.0f * p;
    }
  }
}

}  // namespace w4a16
