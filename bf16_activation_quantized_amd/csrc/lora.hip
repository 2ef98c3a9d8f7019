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
// Units of up to 16 rows of one adapter, whatever their order in the batch:
// rows are grouped within blocks of kBlockRows rows, and every workgroup finds
// its unit by itself: it counts the block's rows per adapter in LDS, takes the
// unit-th run of 16 in adapter order, and picks the unit's rows by their rank
// among the adapter's rows (about 1 us, against a launch of its own for a
// sort). Past kTableAdapters adapters the counts do not fit, and a unit is 16
// consecutive rows, whose adapters follow one another.
//
// Workgroup (unit, rank tile of 16, K slice): MFMA 16x16x32. The 8 waves take
// the slice's 128-k groups in turn; a group of x and of A is fetched in whole
// lines (4 rows x 256 bytes per instruction) and turned into fragments through
// the wave's own LDS tile; the next group is in flight meanwhile. The waves
// are summed through LDS in wave order; the slices of K (fp32) by the reader.
constexpr int kTileWaves = 8, kTileThreads = 64 * kTileWaves;
constexpr int kBlockRows = 4096, kTableAdapters = 8192;

// exclusive sum over the workgroup's threads; `total` gets the whole sum
__device__ __forceinline__ int block_scan(int v, int* s, int tid, int* total) {
  const int lane = tid & 63, wv = tid >> 6;
  int in = v;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(in, d);
    if (lane >= d) in += o;
  }
  __syncthreads();
  if (lane == 63) s[wv] = in;
  __syncthreads();
  int below = 0, all = 0;
#pragma unroll
  for (int q = 0; q < kTileWaves; ++q) {
    below += q < wv ? s[q] : 0;
    all += s[q];
  }
  *total = all;
  return below + in - v;
}

struct ShrinkLds {
  union {
    u32x4 tile[kTileWaves][16 * 16];   // [row][piece p of a group in slot p ^ row]
    int count[kTableAdapters];
  };
  f32x4 red[kTileWaves][64];
  int scan[kTileWaves];
  int rows[16];
  int adapter, chunk;
};

// The unit's adapter, or -1 when there is no such unit; its rows in s.rows (-1
// past the last).
__device__ __forceinline__ int find_unit(ShrinkLds& s, const int32_t* ids, int b0, int bn, int L, int unit, int tid) {
  const int per_l = (L + kTileThreads - 1) / kTileThreads, per_m = (bn + kTileThreads - 1) / kTileThreads;
  for (int l = tid; l < L; l += kTileThreads) s.count[l] = 0;
  if (tid < 16) s.rows[tid] = -1;
  if (tid == 0) s.adapter = -1;
  __syncthreads();
  for (int m = tid; m < bn; m += kTileThreads) {
    const int id = ids[b0 + m];
    if ((uint32_t)id < (uint32_t)L) atomicAdd(&s.count[id], 1);
  }
  __syncthreads();
  const int l0 = min(L, tid * per_l), l1 = min(L, l0 + per_l);
  int units = 0, total = 0;
  for (int l = l0; l < l1; ++l) units += (s.count[l] + 15) >> 4;
  int at = block_scan(units, s.scan, tid, &total);
  if (unit >= total) return -1;   // the same in every thread
  for (int l = l0; l < l1; ++l) {
    const int n = (s.count[l] + 15) >> 4;
    if (unit >= at && unit < at + n) {
      s.adapter = l;
      s.chunk = unit - at;
    }
    at += n;
  }
  __syncthreads();
  const int l = __builtin_amdgcn_readfirstlane(s.adapter), first = 16 * s.chunk;
  const int m0 = min(bn, tid * per_m), m1 = min(bn, m0 + per_m);
  int mine = 0;
  for (int m = m0; m < m1; ++m) mine += ids[b0 + m] == l ? 1 : 0;
  int k = block_scan(mine, s.scan, tid, &total) - first;
  if (mine > 0 && k < 16 && k + mine > 0)
    for (int m = m0; m < m1; ++m)
      if (ids[b0 + m] == l) {
        if (k >= 0 && k < 16) s.rows[k] = b0 + m;
        ++k;
      }
  __syncthreads();
  return l;
}

template <bool TABLE>
__global__ __launch_bounds__(kTileThreads) void lora_shrink_unit_kernel(
    const uint16_t* __restrict__ x, const uint16_t* __restrict__ a, const int32_t* __restrict__ ids,
    const float* __restrict__ scaling, float* __restrict__ hp, int M, int K, int L, int R, int gps,
    int units_per_block) {
  __shared__ ShrinkLds s;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int m16 = lane & 15, kb = lane >> 4;
  const int r0 = blockIdx.y * 16;
  const int gb = blockIdx.z * gps, ge = min(K / kGroup, gb + gps);
  const uint32_t KB = (uint32_t)K * 2u;

  int id;                 // adapter of row m16 of the unit, -1 past its rows
  uint32_t xo[4];         // offset of the lane's piece of row 4 j + kb
  int row_out[4];         // row 4 kb + i
  if constexpr (TABLE) {
    const int blk = blockIdx.x / units_per_block, b0 = blk * kBlockRows;
    const int l = find_unit(s, ids, b0, min(kBlockRows, M - b0), L, (int)blockIdx.x - blk * units_per_block, tid);
    if (l < 0) return;
    id = s.rows[m16] >= 0 ? l : -1;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int r = s.rows[4 * j + kb];
      xo[j] = r >= 0 ? (uint32_t)r * KB + 16u * (uint32_t)m16 : kOutside;
      row_out[j] = s.rows[4 * kb + j];
    }
  } else {
    const int m0 = blockIdx.x * 16;
    id = m0 + m16 < M ? ids[m0 + m16] : -1;
    id = (uint32_t)id < (uint32_t)L ? id : -1;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int r = m0 + 4 * j + kb;
      xo[j] = r < M ? (uint32_t)r * KB + 16u * (uint32_t)m16 : kOutside;
      row_out[j] = m0 + 4 * kb + j;
    }
  }
  const uint64_t all = __ballot(id >= 0) & 0xFFFFull;
  if (all == 0) return;
  if constexpr (TABLE) __syncthreads();   // the counts' LDS becomes the waves' tiles

  const __amdgpu_buffer_rsrc_t rx = make_rsrc(x, (uint32_t)M * KB);
  auto load_x = [&](u32x4 (&v)[4], int g) {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = ld128(rx, __builtin_elementwise_add_sat(xo[j], (uint32_t)g * 256u));
  };
  const uint32_t ao = (uint32_t)kb * KB + 16u * (uint32_t)m16;
  auto load_a = [&](u32x4 (&v)[4], int l, int g) {   // ranks past R read zeros
    const __amdgpu_buffer_rsrc_t ra = make_rsrc(a + ((size_t)l * R + r0) * K, (uint32_t)min(16, R - r0) * KB);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = ld128(ra, ao + (uint32_t)(4 * j) * KB + (uint32_t)g * 256u);
  };
  u32x4* tw = s.tile[wv];
  // lane (m16, kb) of step j: row m16, piece 4 kb + j (k = 32 kb + 8 j + 0..7, the same in both operands)
  auto turn = [&](const u32x4 (&v)[4], u32x4 (&f)[4]) {
    wave_lds_exchange();
#pragma unroll
    for (int j = 0; j < 4; ++j) tw[16 * (4 * j + kb) + (m16 ^ (4 * j + kb))] = v[j];
    wave_lds_exchange();
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = tw[16 * m16 + ((4 * kb + j) ^ m16)];
  };
  // the sequence of (group, adapter) of this wave: one adapter with TABLE; else
  // x stays in registers while the adapters follow one another, and a product
  // is added to the rows of its adapter only
  uint64_t todo = all;
  int g = gb + wv;
  auto adapter = [&](uint64_t& mine) {
    const int l = __builtin_amdgcn_readlane(id, __builtin_ctzll(todo));
    mine = TABLE ? all : __ballot(id == l) & 0xFFFFull;
    return l;
  };
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  if (g < ge) {
    u32x4 xn[4], an[4], xf[4], af[4];
    uint64_t mine;
    load_a(an, adapter(mine), g);
    load_x(xn, g);
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
      const bool more = g < ge;
      if (more) {
        load_a(an, adapter(mine), g);
        if (fresh) load_x(xn, g);
      }
      if constexpr (TABLE) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(frag(xf[j]), frag(af[j]), acc, 0, 0, 0);
      } else {
        f32x4 d = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < 4; ++j)
          d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(frag(xf[j]), frag(af[j]), d, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] += (cur >> (4 * kb + i)) & 1 ? d[i] : 0.0f;
      }
      if (!more) break;
    }
  }
  s.red[wv][lane] = acc;
  __syncthreads();
  if (wv == 0 && r0 + m16 < R) {
    f32x4 v = s.red[0][lane];
#pragma unroll
    for (int q = 1; q < kTileWaves; ++q) {
      const f32x4 p = s.red[q][lane];
      v.x += p.x;
      v.y += p.y;
      v.z += p.z;
      v.w += p.w;
    }
    // lane: rows 4 kb + i, rank r0 + m16
    const float f[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int l = __shfl(id, 4 * kb + i);
      if ((all >> (4 * kb + i)) & 1)
        hp[((size_t)blockIdx.z * M + row_out[i]) * R + r0 + m16] = scaling != nullptr ? scaling[l] * f[i] : f[i];
    }
  }
}

// K slices: enough workgroups for the compute units (about three each), at
// least one group per wave (the tile kernel adds the slices up, in every
// column tile).
int lora_shrink_slices(int M, int K, int L, int R) {
  const int64_t units = L <= kTableAdapters ? M / 16 + (L < M ? L : M) / 2 + 1 : (M + 15) / 16;
  const int64_t wgs = units * ((R + 15) / 16), most = (K / kGroup + kTileWaves - 1) / kTileWaves;
  int64_t ks = 768 / wgs;
  if (ks > most) ks = most;
  return (int)(ks < 1 ? 1 : ks > kLoraMaxSlices ? kLoraMaxSlices : ks);
}

hipError_t launch_lora_shrink_rows(const uint16_t* x, const uint16_t* a, const int32_t* ids, const float* scaling,
                                   uint16_t* h, int M, int K, int L, int R, hipStream_t stream) {
#define W4A16_ROW(RP)                                                                                         \
  hipLaunchKernelGGL(lora_shrink_row_kernel<RP>, dim3(M, R / RP), dim3(64 * kRowWaves), 0, stream, x, a, ids, \
                     scaling, h, M, K, L, R)
  if (M * R >= 2048) W4A16_ROW(8);
  else if (M * R >= 1024) W4A16_ROW(4);
  else if (M * R >= 512) W4A16_ROW(2);
  else W4A16_ROW(1);
#undef W4A16_ROW
  return hipGetLastError();
}

hipError_t launch_lora_shrink_units(const uint16_t* x, const uint16_t* a, const int32_t* ids, const float* scaling,
                                    float* hp, int M, int K, int L, int R, int ks, hipStream_t stream) {
  const int gps = (K / kGroup + ks - 1) / ks;
  if (L <= kTableAdapters) {
    const int bn = M < kBlockRows ? M : kBlockRows, upb = bn / 16 + (L < bn ? L : bn);
    const dim3 grid((unsigned)((M + kBlockRows - 1) / kBlockRows) * (unsigned)upb, (R + 15) / 16, ks);
    hipLaunchKernelGGL(lora_shrink_unit_kernel<true>, grid, dim3(kTileThreads), 0, stream, x, a, ids, scaling, hp, M,
                       K, L, R, gps, upb);
  } else {
    const dim3 grid((M + 15) / 16, (R + 15) / 16, ks);
    hipLaunchKernelGGL(lora_shrink_unit_kernel<false>, grid, dim3(kTileThreads), 0, stream, x, a, ids, scaling, hp, M,
                       K, L, R, gps, 0);
  }
  return hipGetLastError();
}

}  // namespace w4a16
