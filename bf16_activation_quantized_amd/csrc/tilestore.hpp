// Outputs of the tile kernels whose accumulators hold one row and four
// consecutive columns per lane and 16 x 16 tile.
#pragma once

#include "common.hpp"

namespace w4a16 {

// A wave's TM x TN tile, rounded to bf16, through its TM TN 2 bytes of LDS at
// `reg` (not read by anyone else any more), so that whole runs of the output's
// rows are stored, 16 bytes per lane: put(row, c, v) with columns c .. c + 7 of
// the tile's row. acc[ms][ns] of lane (r, q) is row 16 ms + r, columns col(ns) ..
// + 3 (multiples of 4). 16-byte chunk c of an LDS row lies in slot c ^ (row & mask).
template <int TM, int TN, int MS, int SN, class COL, class PUT>
__device__ __forceinline__ void tile_rows_bf16(uint8_t* reg, const f32x4 (&acc)[MS][SN], COL col, int lane, PUT put) {
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
#pragma unroll
  for (int i = 0; i < (TM + RI - 1) / RI; ++i) {
    const int row = RI * i + rr;
    if (TM % RI != 0 && row >= TM) break;
    put(row, 8 * cc, *reinterpret_cast<const u32x4*>(reg + row * RB + 16 * (cc ^ (row & (NCH - 1)))));
  }
}

// The tile's first row is row row0 and its first column column c0 of the output
// at ry (O columns, a multiple of 8); rows past ry's extent are dropped, as long as
// the offsets of all the workgroup's rows fit 32 bits (the caller's plan sees to it).
template <int TM, int TN, int MS, int SN, class COL>
__device__ __forceinline__ void store_tile_bf16(uint8_t* reg, const f32x4 (&acc)[MS][SN], COL col,
                                                __amdgpu_buffer_rsrc_t ry, int row0, int c0, int O, int lane) {
  tile_rows_bf16<TM, TN>(reg, acc, col, lane, [&](int row, int c, u32x4 v) {
    if (c0 + c < O) st128(v, ry, ((uint32_t)(row0 + row) * (uint32_t)O + (uint32_t)(c0 + c)) * 2u);
  });
}

// The same for any O: 16-byte stores at 2-byte alignment, the last columns one by
// one. y: the output's row 0; rows past `rows` are dropped.
template <int TM, int TN, int MS, int SN, class COL>
__device__ __forceinline__ void store_tile_bf16_odd(uint8_t* reg, const f32x4 (&acc)[MS][SN], COL col, uint16_t* y,
                                                    int rows, int row0, int c0, int O, int lane) {
  typedef uint32_t u32x4_a2 __attribute__((ext_vector_type(4), aligned(2)));
  tile_rows_bf16<TM, TN>(reg, acc, col, lane, [&](int row, int c, u32x4 v) {
    if (row0 + row >= rows) return;
    uint16_t* p = y + (size_t)(row0 + row) * O + c0 + c;
    if (c0 + c + 8 <= O) {
      *reinterpret_cast<u32x4_a2*>(p) = v;
    } else {
#pragma unroll
      for (int i = 0; i < 7; ++i)
        if (c0 + c + i < O) p[i] = (uint16_t)(v[i >> 1] >> (16 * (i & 1)));
    }
  });
}

}  // namespace w4a16
