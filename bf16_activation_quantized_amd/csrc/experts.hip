// Rows of a mixture of experts around the grouped GEMM: slots sorted by
// expert, token rows gathered into that order, expert rows combined back with
// weights, and the gradients of both.
//
//   slots s = t k + j, expert e = ids[s] (dropped when outside [0, G))
//   sort:         m_sizes[g] = #{s : e = g}; pos[s] = the slot's row in
//                 (expert, slot) order, -1 when dropped; order = its inverse,
//                 dropped slots behind the others
//   gather:       xs[pos[t, j]] = x[t]
//   combine:      y[t] = bf16(sum_j w[t, j] z[pos[t, j]]), j ascending in fp32
//   combine_grad: dz[pos[t, j]] = bf16(w[t, j] dy[t]),
//                 dw[t, j] = sum_n dy[t, n] z[pos[t, j], n] in fp32
// The gradient of gather is combine without weights. No atomics on results:
// every result is bitwise reproducible.
#include "common.hpp"
#include "launch.hpp"

namespace w4a16 {

namespace {

// 16 bytes of a row whose start is only 2-byte aligned (odd widths)
typedef uint32_t u32x4_a2 __attribute__((ext_vector_type(4), aligned(2)));

template <bool ALIGNED>
__device__ __forceinline__ u32x4 load8(const uint16_t* p) {
  if constexpr (ALIGNED) return *reinterpret_cast<const u32x4*>(p);
  else return *reinterpret_cast<const u32x4_a2*>(p);
}
template <bool ALIGNED>
__device__ __forceinline__ void store8(uint16_t* p, u32x4 v) {
  if constexpr (ALIGNED) *reinterpret_cast<u32x4*>(p) = v;
  else *reinterpret_cast<u32x4_a2*>(p) = v;
}

__device__ __forceinline__ void fma8(float (&a)[8], float w, u32x4 v) {
  a[0] = fmaf(w, bf16lo(v.x), a[0]);
  a[1] = fmaf(w, bf16hi(v.x), a[1]);
  a[2] = fmaf(w, bf16lo(v.y), a[2]);
  a[3] = fmaf(w, bf16hi(v.y), a[3]);
  a[4] = fmaf(w, bf16lo(v.z), a[4]);
  a[5] = fmaf(w, bf16hi(v.z), a[5]);
  a[6] = fmaf(w, bf16lo(v.w), a[6]);
  a[7] = fmaf(w, bf16hi(v.w), a[7]);
}
__device__ __forceinline__ u32x4 pack8f(const float (&a)[8]) {
  return u32x4{pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3]), pack_bf16x2(a[4], a[5]), pack_bf16x2(a[6], a[7])};
}

constexpr int kSortThreads = 256;
constexpr int kSortWaves = kSortThreads / 64;

__device__ __forceinline__ int bin_of(const int32_t* ids, int64_t s, int G) {
  const int e = ids[s];
  return (uint32_t)e < (uint32_t)G ? e : G;   // bin G: dropped
}

}  // namespace

// ---------------------------------------------------------------- sort
// Pass 1: block b counts the bins of its chunk of slots, hist[b][0 .. G].
__global__ __launch_bounds__(kSortThreads) void expert_hist_kernel(const int32_t* __restrict__ ids,
                                                                   int32_t* __restrict__ hist, int S, int G,
                                                                   int chunk) {
  extern __shared__ __attribute__((aligned(16))) int32_t cnt[];
  for (int g = threadIdx.x; g <= G; g += kSortThreads) cnt[g] = 0;
  __syncthreads();
  const int64_t lo = (int64_t)blockIdx.x * chunk;
  const int64_t hi = min((int64_t)S, lo + chunk);
  for (int64_t s = lo + threadIdx.x; s < hi; s += kSortThreads) atomicAdd(&cnt[bin_of(ids, s, G)], 1);
  __syncthreads();
  for (int g = threadIdx.x; g <= G; g += kSortThreads) hist[(int64_t)blockIdx.x * (G + 1) + g] = cnt[g];
}

// Pass 2: every block forms the start of each bin for its own chunk (all bins
// before it, plus the same bin in the chunks before it), splits it over its
// waves' sub-chunks, and each wave ranks its slots 64 at a time: the lanes of
// equal bin are found with one ballot per bin bit, a lane's rank is the number
// of equal lanes below it, and the last lane of a bin moves the bin's running
// count on. Slots keep their order, so the sort is stable.
__global__ __launch_bounds__(kSortThreads) void expert_scatter_kernel(
    const int32_t* __restrict__ ids, const int32_t* __restrict__ hist, int32_t* __restrict__ order,
    int32_t* __restrict__ pos, int32_t* __restrict__ m_sizes, int S, int G, int chunk, int blocks, int bits) {
  extern __shared__ __attribute__((aligned(16))) int32_t lds[];
  const int nb = G + 1;
  int32_t* start = lds;              // [nb] start of each bin for this chunk
  int32_t* run = lds + nb;           // [waves][nb] counts, then running starts of each wave's sub-chunk
  __shared__ int32_t part[kSortThreads];
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;

  // bins of this thread: a contiguous run, so that the scan over bins is one
  // scan over the threads
  const int per = (nb + kSortThreads - 1) / kSortThreads;
  const int g0 = min(nb, tid * per), g1 = min(nb, g0 + per);
  int mine = 0;
  for (int g = g0; g < g1; ++g) {
    int tot = 0, before = 0;
    for (int b = 0; b < blocks; ++b) {
      const int v = hist[(int64_t)b * nb + g];
      tot += v;
      before += b < (int)blockIdx.x ? v : 0;
    }
    if (blockIdx.x == 0 && g < G) m_sizes[g] = tot;
    start[g] = mine + before;
    mine += tot;
  }
  part[tid] = mine;
  for (int i = tid; i < kSortWaves * nb; i += kSortThreads) run[i] = 0;
  __syncthreads();
  int below = 0;
  for (int t = 0; t < tid; ++t) below += part[t];
  for (int g = g0; g < g1; ++g) start[g] += below;

  const int sub = chunk / kSortWaves;
  const int64_t lo = min((int64_t)S, (int64_t)blockIdx.x * chunk + (int64_t)wv * sub);
  const int64_t hi = min((int64_t)S, lo + sub);
  for (int64_t s = lo + lane; s < hi; s += 64) atomicAdd(&run[wv * nb + bin_of(ids, s, G)], 1);
  __syncthreads();
  for (int g = tid; g < nb; g += kSortThreads) {
    int at = start[g];
    for (int w = 0; w < kSortWaves; ++w) {
      const int c = run[w * nb + g];
      run[w * nb + g] = at;
      at += c;
    }
  }
  __syncthreads();
  int32_t* r = run + wv * nb;
  for (int64_t s0 = lo; s0 < hi; s0 += 64) {
    const int64_t s = s0 + lane;
    const bool live = s < hi;
    const int e = live ? bin_of(ids, s, G) : G;
    uint64_t same = __ballot(live);
    for (int b = 0; b < bits; ++b) {
      const uint64_t v = __ballot((e >> b) & 1);
      same &= ((e >> b) & 1) ? v : ~v;
    }
    const int rank = __popcll(same & ((1ull << lane) - 1));
    wave_lds_exchange();   // after the last step's writes
    const int p = r[e] + rank;
    wave_lds_exchange();   // every lane has read before the counts move on
    if (live && (same >> lane) == 1ull) r[e] = p + 1;
    if (live) {
      order[p] = (int32_t)s;
      pos[s] = e < G ? p : -1;
    }
  }
}

__global__ void expert_zero_kernel(int32_t* __restrict__ m_sizes, int G) {
  for (int g = threadIdx.x; g < G; g += blockDim.x) m_sizes[g] = 0;
}

// ---------------------------------------------------------------- gather
template <bool ALIGNED>
__global__ __launch_bounds__(256) void expert_gather_kernel(const uint16_t* __restrict__ x,
                                                            const int32_t* __restrict__ pos,
                                                            uint16_t* __restrict__ xs, int64_t T, int k, int64_t rows,
                                                            int width) {
  for (int64_t t = blockIdx.x; t < T; t += gridDim.x) {
    const uint16_t* src = x + t * width;
    for (int c = 8 * threadIdx.x; c < width; c += 8 * 256) {
      const bool full = c + 8 <= width;
      u32x4 v;
      if (full) v = load8<ALIGNED>(src + c);
      for (int j = 0; j < k; ++j) {
        const int64_t p = pos[t * k + j];
        if (p < 0 || p >= rows) continue;
        uint16_t* dst = xs + p * width + c;
        if (full) store8<ALIGNED>(dst, v);
        else
          for (int i = 0; c + i < width; ++i) dst[i] = src[c + i];
      }
    }
  }
}

// ---------------------------------------------------------------- combine
// w == nullptr: all weights 1 (the gradient of gather)
template <bool ALIGNED>
__global__ __launch_bounds__(256) void expert_combine_kernel(const uint16_t* __restrict__ z,
                                                             const int32_t* __restrict__ pos,
                                                             const float* __restrict__ w, uint16_t* __restrict__ y,
                                                             int64_t T, int k, int64_t rows, int width) {
  for (int64_t t = blockIdx.x; t < T; t += gridDim.x) {
    for (int c = 8 * threadIdx.x; c < width; c += 8 * 256) {
      const int n = min(8, width - c);
      float a[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      for (int j = 0; j < k; ++j) {
        const int64_t p = pos[t * k + j];
        if (p < 0 || p >= rows) continue;
        const float wj = w != nullptr ? w[t * k + j] : 1.0f;
        const uint16_t* src = z + p * width + c;
        if (n == 8) fma8(a, wj, load8<ALIGNED>(src));
        else
          for (int i = 0; i < n; ++i) a[i] = fmaf(wj, bf16f(src[i]), a[i]);
      }
      uint16_t* dst = y + t * width + c;
      if (n == 8) store8<ALIGNED>(dst, pack8f(a));
      else
        for (int i = 0; i < n; ++i) dst[i] = to_bf16(a[i]);
    }
  }
}

// ---------------------------------------------------------------- combine's gradient
template <bool ALIGNED>
__global__ __launch_bounds__(256) void expert_combine_grad_kernel(const uint16_t* __restrict__ dy,
                                                                  const uint16_t* __restrict__ z,
                                                                  const int32_t* __restrict__ pos,
                                                                  const float* __restrict__ w,
                                                                  uint16_t* __restrict__ dz, float* __restrict__ dw,
                                                                  int64_t T, int k, int64_t rows, int width) {
  __shared__ float red[4];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  for (int64_t t = blockIdx.x; t < T; t += gridDim.x) {
    for (int j = 0; j < k; ++j) {
      const int64_t p = pos[t * k + j];
      if (p < 0 || p >= rows) {
        if (threadIdx.x == 0) dw[t * k + j] = 0.0f;
        continue;
      }
      const float wj = w[t * k + j];
      float dot = 0.0f;
      for (int c = 8 * threadIdx.x; c < width; c += 8 * 256) {
        const int n = min(8, width - c);
        const uint16_t* d = dy + t * width + c;
        const uint16_t* zr = z + p * width + c;
        uint16_t* o = dz + p * width + c;
        if (n == 8) {
          const u32x4 dv = load8<ALIGNED>(d), zv = load8<ALIGNED>(zr);
          float a[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
          fma8(a, wj, dv);
          store8<ALIGNED>(o, pack8f(a));
          const uint32_t dd[4] = {dv.x, dv.y, dv.z, dv.w}, zz[4] = {zv.x, zv.y, zv.z, zv.w};
          for (int i = 0; i < 4; ++i) {
            dot = fmaf(bf16lo(dd[i]), bf16lo(zz[i]), dot);
            dot = fmaf(bf16hi(dd[i]), bf16hi(zz[i]), dot);
          }
        } else {
          for (int i = 0; i < n; ++i) {
            o[i] = to_bf16(wj * bf16f(d[i]));
            dot = fmaf(bf16f(d[i]), bf16f(zr[i]), dot);
          }
        }
      }
      dot = wave64_sum(dot);
      if (lane == 63) red[wv] = dot;
      __syncthreads();
      if (threadIdx.x == 0) dw[t * k + j] = (red[0] + red[1]) + (red[2] + red[3]);
      __syncthreads();
    }
  }
}

// ---------------------------------------------------------------- launchers
// Slots per block of the sort: whole sub-chunks of 64 slots per wave, at most
// about 256 blocks.
int expert_sort_chunk(int64_t S) {
  const int64_t per = (S + 255) / 256;
  const int64_t c = (per + kSortThreads - 1) / kSortThreads * kSortThreads;
  return (int)(c < 1024 ? 1024 : c);
}
int expert_sort_blocks(int64_t S) {
  const int c = expert_sort_chunk(S);
  return (int)((S + c - 1) / c);
}

hipError_t launch_expert_sort(const int32_t* ids, int32_t* order, int32_t* pos, int32_t* m_sizes, int64_t S, int G,
                              int32_t* ws, hipStream_t stream) {
  if (S == 0) {
    hipLaunchKernelGGL(expert_zero_kernel, dim3(1), dim3(256), 0, stream, m_sizes, G);
    return hipGetLastError();
  }
  const int chunk = expert_sort_chunk(S), blocks = expert_sort_blocks(S);
  int bits = 1;
  while ((1 << bits) <= G) ++bits;
  const size_t lds1 = (size_t)(G + 1) * 4, lds2 = (size_t)(G + 1) * 4 * (1 + kSortWaves);
  static std::atomic<uint64_t> lds_set{0};
  const hipError_t ea = ensure_dyn_lds(reinterpret_cast<const void*>(&expert_scatter_kernel),
                                       (kExpertMaxGroups + 1) * 4 * (1 + kSortWaves), lds_set);
  if (ea != hipSuccess) return ea;
  hipLaunchKernelGGL(expert_hist_kernel, dim3(blocks), dim3(kSortThreads), lds1, stream, ids, ws, (int)S, G, chunk);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(expert_scatter_kernel, dim3(blocks), dim3(kSortThreads), lds2, stream, ids, ws, order, pos,
                     m_sizes, (int)S, G, chunk, blocks, bits);
  return hipGetLastError();
}

static unsigned row_grid(int64_t T) { return (unsigned)(T < (1 << 20) ? T : (1 << 20)); }

hipError_t launch_expert_gather(const uint16_t* x, const int32_t* pos, uint16_t* xs, int64_t T, int k, int64_t rows,
                                int width, hipStream_t stream) {
  if (width % 8 == 0)
    hipLaunchKernelGGL(expert_gather_kernel<true>, dim3(row_grid(T)), dim3(256), 0, stream, x, pos, xs, T, k, rows,
                       width);
  else
    hipLaunchKernelGGL(expert_gather_kernel<false>, dim3(row_grid(T)), dim3(256), 0, stream, x, pos, xs, T, k, rows,
                       width);
  return hipGetLastError();
}

hipError_t launch_expert_combine(const uint16_t* z, const int32_t* pos, const float* w, uint16_t* y, int64_t T, int k,
                                 int64_t rows, int width, hipStream_t stream) {
  if (width % 8 == 0)
    hipLaunchKernelGGL(expert_combine_kernel<true>, dim3(row_grid(T)), dim3(256), 0, stream, z, pos, w, y, T, k, rows,
                       width);
  else
    hipLaunchKernelGGL(expert_combine_kernel<false>, dim3(row_grid(T)), dim3(256), 0, stream, z, pos, w, y, T, k,
                       rows, width);
  return hipGetLastError();
}

hipError_t launch_expert_combine_grad(const uint16_t* dy, const uint16_t* z, const int32_t* pos, const float* w,
                                      uint16_t* dz, float* dw, int64_t T, int k, int64_t rows, int width,
                                      hipStream_t stream) {
  if (width % 8 == 0)
    hipLaunchKernelGGL(expert_combine_grad_kernel<true>, dim3(row_grid(T)), dim3(256), 0, stream, dy, z, pos, w, dz,
                       dw, T, k, rows, width);
  else
    hipLaunchKernelGGL(expert_combine_grad_kernel<false>, dim3(row_grid(T)), dim3(256), 0, stream, dy, z, pos, w, dz,
                       dw, T, k, rows, width);
  return hipGetLastError();
}

}  // namespace w4a16
