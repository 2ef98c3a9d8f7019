// Outputs of the tile kernels whose accumulators hold one row and four
// consecutive columns per lane and 16 x 16 tile.
#pragma once

#include "common.hpp"

namespace w4a16 {

// A wave's TM x TN tile, rounded to bf16, through its TM TN 2 bytes of LDS at
// `reg` (not read by anyone else any more), so that whole runs of the output's
// rows are stored, 16 bytes per lane. acc[ms][ns] of lane (r, q) is row 16 ms + r,
// columns col(ns) .. + 3 (multiples of 4) of the tile; the tile's first row is row
// row0 and its first column column c0 of the output at ry (O columns, a multiple
// of 8); rows past ry's extent are dropped. 16-byte chunk c of an LDS row lies in
// slot c ^ (row & mask).
template <int TM, int TN, int MS, int SN, class COL>
__device__ __forceinline__ void store_tile_bf16(uint8_t* reg, const f32x4 (&acc)[MS][SN], COL col,
                                                __amdgpu_buffer_rsrc_t ry, int row0, int c0, int O, int lane) {
  static_assert(TM == 16 * MS && TN == 16 * SN, "the tile of the accumulators");
  constexpr int RB = TN * 2, NCH = RB / 16;   // bytes and chunks of a row
  constexpr int RI = 64 / NCH;                // rows per store
  const int r16 = lane & 15;
#pragma unroll
  for (int ms = 0; ms < MS; ++ms)
#pragma unroll
    for (int ns = 0; ns < SN; ++ns) {
      const int b = 2 * col(ns);
      *reinterpret_cast<u32x2*>(reg + (16 * ms + r16) * RB + 16 * ((b >> 4) ^ (r16 & (NCH - 1))) + (b & 8)) =
          u32x2{pack_bf16x2(acc[ms][ns].x, acc[ms][ns].y), pack_bf16x2(acc[ms][ns].z, acc[ms][ns].w)};
    }
  wave_lds_exchange();   // the rows below were written by other lanes
  const int rr = lane / NCH, cc = lane % NCH;
  if (c0 + 8 * cc >= O) return;
#pragma unroll
  for (int i = 0; i < (TM + RI - 1) / RI; ++i) {
    const int row = RI * i + rr;
    if (TM % RI != 0 && row >= TM) break;
    const u32x4 v = *reinterpret_cast<const u32x4*>(reg + row * RB + 16 * (cc ^ (row & (NCH - 1))));
    st128(v, ry, ((uint32_t)(row0 + row) * (uint32_t)O + (uint32_t)(c0 + 8 * cc)) * 2u);
  }
}

}  // namespace w4a16
