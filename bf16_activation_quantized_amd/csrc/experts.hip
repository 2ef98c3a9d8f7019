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
#include <algorithm>
#include <type_traits>

#include "common.hpp"
#include "launch.hpp"

namespace w4a16 {

namespace {

// 16 bytes of a row whose start is only 2-byte aligned (odd widths)
typedef uint32_t u32x4_a2 __attribute__((ext_vector_type(4), aligned(2)));

template <bool ALIGNED, bool NT = false>
__device__ __forceinline__ u32x4 load8(const uint16_t* p) {
  if constexpr (ALIGNED && NT) return __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p));
  else if constexpr (ALIGNED) return *reinterpret_cast<const u32x4*>(p);
  else if constexpr (NT) return __builtin_nontemporal_load(reinterpret_cast<const u32x4_a2*>(p));
  else return *reinterpret_cast<const u32x4_a2*>(p);
}
template <bool ALIGNED, bool NT>
__device__ __forceinline__ void store8(uint16_t* p, u32x4 v) {
  if constexpr (ALIGNED && NT) __builtin_nontemporal_store(v, reinterpret_cast<u32x4*>(p));
  else if constexpr (ALIGNED) *reinterpret_cast<u32x4*>(p) = v;
  else if constexpr (NT) __builtin_nontemporal_store(v, reinterpret_cast<u32x4_a2*>(p));
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

__device__ __forceinline__ float dot8(u32x4 a, u32x4 b, float c) {
  c = fmaf(bf16lo(a.x), bf16lo(b.x), c);
  c = fmaf(bf16hi(a.x), bf16hi(b.x), c);
  c = fmaf(bf16lo(a.y), bf16lo(b.y), c);
  c = fmaf(bf16hi(a.y), bf16hi(b.y), c);
  c = fmaf(bf16lo(a.z), bf16lo(b.z), c);
  c = fmaf(bf16hi(a.z), bf16hi(b.z), c);
  c = fmaf(bf16lo(a.w), bf16lo(b.w), c);
  return fmaf(bf16hi(a.w), bf16hi(b.w), c);
}

constexpr int kBatch = 4;   // slots of a token whose rows are in flight together

// Sort: a block of W waves takes tiles of PER slots per lane in turn.
constexpr int kSortMaxBlocks = 256;
// Slots that one block takes alone, in up to two tiles, ahead of two launches
// (one block against several, us: 1500 slots of 8 experts 5.6 / 6.9, 2048 slots
// of 8 6.0 / 7.1, of 128 7.0 / 7.3; but 4096 slots of 8 9.7 / 7.2, of 128 11.8 /
// 7.7).
constexpr int kSortSingle = 2048;

__device__ __forceinline__ int bin_of(int e, int G) {
  return (uint32_t)e < (uint32_t)G ? e : G;   // bin G: dropped
}

// inclusive sum over the wave's lanes
__device__ __forceinline__ int wave_scan(int v, int lane) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(v, d);
    if (lane >= d) v += o;
  }
  return v;
}

// Counts the bins of slots [lo, hi) into cnt (LDS, zeroed). The lanes that
// share the first lane's bin are counted at once (a popular expert would
// otherwise be up to 64 additions to one address), the others one by one.
template <int PER>
__device__ __forceinline__ void count_bins(int32_t* cnt, const int32_t* ids, int64_t lo, int64_t hi, int G, int tid,
                                           int nthr) {
  for (int64_t s0 = lo; s0 < hi; s0 += PER * nthr) {
    int e[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int64_t s = s0 + (int64_t)i * nthr + tid;
      e[i] = s < hi ? bin_of(ids[s], G) : -1;
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const uint64_t live = __ballot(e[i] >= 0);
      if (live == 0) continue;
      const int first = __builtin_ctzll(live);
      const uint64_t same = __ballot(e[i] == __builtin_amdgcn_readlane(e[i], first));
      if ((tid & 63) == first) atomicAdd(&cnt[e[i]], (int)__popcll(same));
      else if (e[i] >= 0 && !((same >> (tid & 63)) & 1)) atomicAdd(&cnt[e[i]], 1);
    }
  }
}

}  // namespace

// ---------------------------------------------------------------- sort
// Pass 1 (more than one block): block b counts the bins of its slots,
// hist[b][0 .. G].
template <int W, int PER>
__global__ __launch_bounds__(64 * W) void expert_hist_kernel(const int32_t* __restrict__ ids,
                                                             int32_t* __restrict__ hist, int64_t S, int G,
                                                             int64_t chunk) {
  extern __shared__ __attribute__((aligned(16))) int32_t cnt[];
  for (int g = threadIdx.x; g <= G; g += 64 * W) cnt[g] = 0;
  __syncthreads();
  const int64_t lo = (int64_t)blockIdx.x * chunk, hi = lo + chunk < S ? lo + chunk : S;
  count_bins<PER>(cnt, ids, lo, hi, G, threadIdx.x, 64 * W);
  __syncthreads();
  for (int g = threadIdx.x; g <= G; g += 64 * W) hist[(int64_t)blockIdx.x * (G + 1) + g] = cnt[g];
}

// Between them, where the blocks' counts are many: each becomes the sum of the
// blocks before it, and row `blocks` the sum of all. A workgroup takes 64 bins,
// its 16 waves consecutive runs of blocks.
__global__ __launch_bounds__(1024) void expert_prefix_kernel(int32_t* __restrict__ hist, int nb, int blocks) {
  __shared__ int32_t sum[16][64];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int g = 64 * (int)blockIdx.x + lane;
  constexpr int kRun = kSortMaxBlocks / 16;
  const int run = (blocks + 15) / 16;   // <= kRun
  const int b0 = wv * run, b1 = min(blocks, b0 + run);
  int v[kRun], mine = 0;
#pragma unroll
  for (int u = 0; u < kRun; ++u) {
    v[u] = g < nb && b0 + u < b1 ? hist[(b0 + u) * nb + g] : 0;
  }
#pragma unroll
  for (int u = 0; u < kRun; ++u) mine += v[u];
  sum[wv][lane] = mine;
  __syncthreads();
  int at = 0;
  for (int w = 0; w < wv; ++w) at += sum[w][lane];
#pragma unroll
  for (int u = 0; u < kRun; ++u) {
    if (g < nb && b0 + u < b1) hist[(b0 + u) * nb + g] = at;
    at += v[u];
  }
  if (wv == 15 && g < nb) hist[blocks * nb + g] = at;
}

// Pass 2: the start of each bin for the block's slots (all bins before it,
// plus the same bin in the blocks before), then tile by tile: each wave ranks
// its slots 64 at a time (the lanes of equal bin are found with one ballot per
// bin bit; the last of them moves the wave's count of the bin on), the waves'
// counts become their starts, and every slot is written. Slots keep their
// order within a bin: the sort is stable, and exact whatever the scheduling.
template <int W, int PER>
__global__ __launch_bounds__(64 * W) void expert_scatter_kernel(
    const int32_t* __restrict__ ids, const int32_t* __restrict__ hist, int32_t* __restrict__ order,
    int32_t* __restrict__ pos, int32_t* __restrict__ m_sizes, int64_t S, int G, int64_t chunk, int blocks, int bits,
    bool summed) {
  constexpr int NTHR = 64 * W;
  extern __shared__ __attribute__((aligned(16))) int32_t lds[];
  const int nb = G + 1;
  int32_t* at = lds;             // [nb] where the block's next slot of each bin goes
  int32_t* total = lds + nb;     // [nb] slots of each bin: aliased by the waves' counts below
  int32_t* run = lds + nb;       // [W][nb]
  int32_t* shift = run + W * nb;   // [nb]
  int2* place = reinterpret_cast<int2*>(lds + ((W + 2) * nb + 1) / 2 * 2);   // [tile]
  __shared__ int32_t wave_sum[W];
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
  const int64_t lo = (int64_t)blockIdx.x * chunk, hi = lo + chunk < S ? lo + chunk : S;

  for (int g = tid; g < 2 * nb; g += NTHR) lds[g] = 0;
  __syncthreads();
  if (blocks == 1) {
    count_bins<PER>(total, ids, lo, hi, G, tid, NTHR);
  } else if (summed) {
    for (int g = tid; g < nb; g += NTHR) {
      total[g] = hist[blocks * nb + g];
      at[g] = hist[(int)blockIdx.x * nb + g];
    }
  } else {
    // thread (q, g): bin g of every parts-th block, 16 blocks in flight (a
    // thread takes bins in turn where there are more of them than threads);
    // counts past the last block's read as zeros
    const int parts = nb < NTHR ? NTHR / nb : 1;
    const int q = nb < NTHR ? tid / nb : 0;
    const uint32_t row = 4u * (uint32_t)nb, before_me = blockIdx.x * row, step = (uint32_t)parts * row;
    const __amdgpu_buffer_rsrc_t rh = make_rsrc(hist, (uint32_t)blocks * row);   // blocks <= 256, nb <= 4097
    for (int g = tid - q * nb; g < nb && q < parts; g += NTHR) {
      uint32_t o = (uint32_t)q * row + 4u * (uint32_t)g;
      int all = 0, before = 0;
      for (int b0 = 0; b0 < blocks; b0 += 16 * parts) {
        int v[16];
#pragma unroll
        for (int u = 0; u < 16; ++u) v[u] = (int)ld32(rh, o + (uint32_t)u * step);
#pragma unroll
        for (int u = 0; u < 16; ++u) {
          all += v[u];
          before += o + (uint32_t)u * step < before_me ? v[u] : 0;
        }
        o += 16u * step;
      }
      atomicAdd(&total[g], all);
      atomicAdd(&at[g], before);
    }
  }
  __syncthreads();
  // exclusive sum over the bins: a contiguous run of bins per thread
  const int per = (nb + NTHR - 1) / NTHR;
  const int g0 = min(nb, tid * per), g1 = min(nb, g0 + per);
  int mine = 0;
  for (int g = g0; g < g1; ++g) mine += total[g];
  const int in = wave_scan(mine, lane);
  if (lane == 63) wave_sum[wv] = in;
  __syncthreads();
  int below = in - mine;
#pragma unroll
  for (int w = 0; w < W; ++w) below += w < wv ? wave_sum[w] : 0;
  for (int g = g0; g < g1; ++g) {
    const int n = total[g];
    if (blockIdx.x == 0 && g < G) m_sizes[g] = n;
    at[g] += below;
    below += n;
  }

  int32_t* r = run + wv * nb;
  for (int64_t t0 = lo; t0 < hi; t0 += PER * NTHR) {
    const int64_t s0 = t0 + (int64_t)wv * (64 * PER) + lane;
    int e[PER], rank[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) e[i] = s0 + 64 * i < hi ? bin_of(ids[s0 + 64 * i], G) : -1;
    __syncthreads();   // the tile before (or the totals) is done with the counts
    for (int i = tid; i < W * nb; i += NTHR) run[i] = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      uint64_t same = __ballot(e[i] >= 0);
      if (same == 0) break;   // the waves past the last slot
      for (int b = 0; b < bits; ++b) {
        const bool one = (e[i] >> b) & 1;
        const uint64_t v = __ballot(one);
        same &= one ? v : ~v;
      }
      wave_lds_exchange();   // after the last step's counts
      if (e[i] >= 0) rank[i] = r[e[i]] + (int)__popcll(same & ((1ull << lane) - 1));
      wave_lds_exchange();   // every lane has read before the counts move on
      if (e[i] >= 0 && (same >> lane) == 1ull) r[e[i]] = rank[i] + 1;
    }
    __syncthreads();
    // the waves' counts become their starts
    int own = 0;
    for (int g = g0; g < g1; ++g) {
      int a = at[g];
      shift[g] = a;
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const int c = run[w * nb + g];
        run[w * nb + g] = a;
        a += c;
      }
      own += a - shift[g];
      at[g] = a;
    }
    if (blocks > 1) {
      // the bins' starts within the tile: shift = global row minus place in the tile
      const int sum = wave_scan(own, lane);
      if (lane == 63) wave_sum[wv] = sum;
      __syncthreads();
      int first = sum - own;
#pragma unroll
      for (int w = 0; w < W; ++w) first += w < wv ? wave_sum[w] : 0;
      for (int g = g0; g < g1; ++g) {
        const int n = at[g] - shift[g];
        shift[g] -= first;
        first += n;
      }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      if (e[i] >= 0) {
        const int p = r[e[i]] + rank[i];
        const int s = (int)(s0 + 64 * i);
        pos[s] = e[i] < G ? p : -1;
        if (blocks > 1) place[p - shift[e[i]]] = make_int2(p, s);
        else order[p] = s;
      }
    }
    if (blocks > 1) {
      // order goes through LDS in bin order, so that a bin's slots of the tile
      // leave as one run (65536 x 8 slots, 128 experts: 12.1 -> 11.1 us for
      // this kernel in tiles of 4096; one block's few slots are 0.7 us faster without)
      __syncthreads();
      const int n = hi - t0 < PER * NTHR ? (int)(hi - t0) : PER * NTHR;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int q = i * NTHR + tid;
        if (q < n) order[place[q].x] = place[q].y;
      }
    }
  }
}

__global__ void expert_zero_kernel(int32_t* __restrict__ m_sizes, int G) {
  for (int g = threadIdx.x; g < G; g += blockDim.x) m_sizes[g] = 0;
}

// ---------------------------------------------------------------- rows
// TPT threads (32 to 256) hold a token, 8 columns each, so that narrow rows
// leave no lanes idle (30000 x 4 x 256 gradient: 65 us with a workgroup per
// token). From 64 on the token is the same in a whole wave, and saying so
// keeps its positions and weights in scalar registers.
template <int TPT>
__device__ __forceinline__ int token_in_block() {
  const int s = (int)threadIdx.x / TPT;
  return TPT >= 64 ? __builtin_amdgcn_readfirstlane(s) : s;
}

// ---------------------------------------------------------------- gather
template <bool ALIGNED, int TPT, bool NT>
__global__ __launch_bounds__(256) void expert_gather_kernel(const uint16_t* __restrict__ x,
                                                            const int32_t* __restrict__ pos,
                                                            uint16_t* __restrict__ xs, int64_t T, int k, int64_t rows,
                                                            int width) {
  constexpr int TOK = 256 / TPT;
  const int in = (int)threadIdx.x % TPT;
  for (int64_t t = (int64_t)blockIdx.x * TOK + token_in_block<TPT>(); t < T; t += (int64_t)gridDim.x * TOK) {
    const uint16_t* src = x + t * width;
    const int32_t* pt = pos + t * k;
    for (int64_t c = 8 * ((int64_t)blockIdx.y * TPT + in); c < width; c += 8 * (int64_t)gridDim.y * TPT) {
      if (c + 8 <= width) {
        const u32x4 v = load8<ALIGNED>(src + c);
        for (int j = 0; j < k; ++j) {
          const int64_t p = pt[j];
          if (p >= 0 && p < rows) store8<ALIGNED, NT>(xs + p * width + c, v);
        }
      } else {
        for (int j = 0; j < k; ++j) {
          const int64_t p = pt[j];
          if (p >= 0 && p < rows)
            for (int64_t i = c; i < width; ++i) xs[p * width + i] = src[i];
        }
      }
    }
  }
}

// ---------------------------------------------------------------- combine
// w == nullptr: all weights 1 (the gradient of gather)
template <bool ALIGNED, int TPT, bool NT>
__global__ __launch_bounds__(256) void expert_combine_kernel(const uint16_t* __restrict__ z,
                                                             const int32_t* __restrict__ pos,
                                                             const float* __restrict__ w, uint16_t* __restrict__ y,
                                                             int64_t T, int k, int64_t rows, int width) {
  constexpr int TOK = 256 / TPT;
  const int in = (int)threadIdx.x % TPT;
  for (int64_t t = (int64_t)blockIdx.x * TOK + token_in_block<TPT>(); t < T; t += (int64_t)gridDim.x * TOK) {
    for (int64_t c = 8 * ((int64_t)blockIdx.y * TPT + in); c < width; c += 8 * (int64_t)gridDim.y * TPT) {
      const int n = width - c < 8 ? (int)(width - c) : 8;
      float a[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      for (int j0 = 0; j0 < k; j0 += kBatch) {
        int64_t p[kBatch];
        float wj[kBatch];
        u32x4 v[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          p[u] = j0 + u < k ? pos[t * k + j0 + u] : -1;
          if (p[u] >= rows) p[u] = -1;
          wj[u] = p[u] >= 0 && w != nullptr ? w[t * k + j0 + u] : 1.0f;
        }
        if (n == 8) {
#pragma unroll
          for (int u = 0; u < kBatch; ++u)
            if (p[u] >= 0) v[u] = load8<ALIGNED, NT>(z + p[u] * width + c);
#pragma unroll
          for (int u = 0; u < kBatch; ++u)
            if (p[u] >= 0) fma8(a, wj[u], v[u]);
        } else {
#pragma unroll
          for (int u = 0; u < kBatch; ++u)
            if (p[u] >= 0)
#pragma unroll
              for (int i = 0; i < 7; ++i)
                if (i < n) a[i] = fmaf(wj[u], bf16f(z[p[u] * width + c + i]), a[i]);
        }
      }
      uint16_t* dst = y + t * width + c;
      if (n == 8) {
        store8<ALIGNED, NT>(dst, pack8f(a));
      } else {
#pragma unroll
        for (int i = 0; i < 7; ++i)
          if (i < n) dst[i] = to_bf16(a[i]);
      }
    }
  }
}

// ---------------------------------------------------------------- combine's gradient
// A token's dots need its whole width in one workgroup: its threads go over the
// columns in turn, kBatch slots at a time (dy is read again from the caches
// for every further batch), and are summed over the wave's lanes, then over
// the token's waves through LDS. Each element of z is read by the thread that
// writes that element of dz, before it does: dz may be z.
template <bool ALIGNED, int TPT, bool NT>
__global__ __launch_bounds__(256) void expert_combine_grad_kernel(const uint16_t* __restrict__ dy,
                                                                  const uint16_t* z,
                                                                  const int32_t* __restrict__ pos,
                                                                  const float* __restrict__ w, uint16_t* dz,
                                                                  float* __restrict__ dw, int64_t T, int k,
                                                                  int64_t rows, int width) {
  constexpr int TOK = 256 / TPT, WPT = TPT >= 64 ? TPT / 64 : 1;
  __shared__ float red[2][4][kBatch];
  const int in = (int)threadIdx.x % TPT, lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int sub = token_in_block<TPT>();
  int turn = 0;
  // (every thread of a workgroup makes the same trips: the barriers are met by all)
  for (int64_t t0 = (int64_t)blockIdx.x * TOK; t0 < T; t0 += (int64_t)gridDim.x * TOK) {
    const int64_t t = t0 + sub;
    const bool live = t < T;
    for (int j0 = 0; j0 < k; j0 += kBatch) {
      int64_t p[kBatch];
      float wj[kBatch], dot[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        p[u] = live && j0 + u < k ? pos[t * k + j0 + u] : -1;
        if (p[u] >= rows) p[u] = -1;
        wj[u] = p[u] >= 0 ? w[t * k + j0 + u] : 0.0f;
        dot[u] = 0.0f;
      }
      for (int64_t c = 8 * in; c < width && live; c += 8 * TPT) {
        const int n = width - c < 8 ? (int)(width - c) : 8;
        const uint16_t* d = dy + t * width + c;
        if (n == 8) {
          const u32x4 dv = load8<ALIGNED>(d);
          u32x4 zv[kBatch];
#pragma unroll
          for (int u = 0; u < kBatch; ++u)
            if (p[u] >= 0) zv[u] = load8<ALIGNED, NT>(z + p[u] * width + c);
#pragma unroll
          for (int u = 0; u < kBatch; ++u)
            if (p[u] >= 0) {
              float a[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
              fma8(a, wj[u], dv);
              store8<ALIGNED, NT>(dz + p[u] * width + c, pack8f(a));
              dot[u] = dot8(dv, zv[u], dot[u]);
            }
        } else {
#pragma unroll
          for (int u = 0; u < kBatch; ++u)
            if (p[u] >= 0)
              for (int i = 0; i < n; ++i) {
                const float di = bf16f(d[i]);
                dot[u] = fmaf(di, bf16f(z[p[u] * width + c + i]), dot[u]);
                dz[p[u] * width + c + i] = to_bf16(wj[u] * di);
              }
        }
      }
      if constexpr (TPT <= 64) {
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          const float s = TPT == 64 ? wave64_sum(dot[u]) : half32_sum(dot[u]);
          if (in == TPT - 1 && live && j0 + u < k) dw[t * k + j0 + u] = s;
        }
      } else {
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          const float s = wave64_sum(dot[u]);
          if (lane == 63) red[turn][wv][u] = s;
        }
        __syncthreads();
        if (in < kBatch && live && j0 + in < k) {
          float s = red[turn][sub * WPT][in];
#pragma unroll
          for (int q = 1; q < WPT; ++q) s += red[turn][sub * WPT + q][in];
          dw[t * k + j0 + in] = s;
        }
        turn ^= 1;   // the next sums go elsewhere: one barrier per batch
      }
    }
  }
}

// ---------------------------------------------------------------- launchers
// Shape of a sort: one block up to kSortSingle slots (one launch), else whole
// tiles per block, at most kSortMaxBlocks blocks. Smaller tiles spread fewer
// slots over more blocks, larger ones keep the blocks' counts few (pairs of
// waves and slots per lane, us, 128 experts: 32768 slots 8.0 with 8 x 2, 9.3
// with 16 x 2, 11.5 with 16 x 4; 524288 slots 15.0, 12.0, 12.9; 2097152 slots
// 34.5, 24.8, 22.5); past 1024 bins the waves' counts take the LDS.
struct SortShape {
  int waves, per, blocks;
  int64_t chunk;   // slots of a block
};
static SortShape sort_shape(int64_t S, int G) {
  SortShape h;
  h.waves = G > 2048 ? 4 : G > 1024 || S <= (1 << 17) ? 8 : 16;
  h.per = G > 2048 ? 8 : G > 1024 || S > (1 << 19) ? 4 : 2;
  const int64_t tile = 64 * h.per * h.waves, tiles = (S + tile - 1) / tile;
  h.chunk = S <= kSortSingle ? kSortSingle : (tiles + kSortMaxBlocks - 1) / kSortMaxBlocks * tile;
  h.blocks = (int)((S + h.chunk - 1) / h.chunk);
  return h;
}
int expert_sort_blocks(int64_t S, int G) { return sort_shape(S, G).blocks; }

template <int W, int PER>
static hipError_t launch_sort_w(const int32_t* ids, int32_t* order, int32_t* pos, int32_t* m_sizes, int64_t S, int G,
                                int32_t* ws, const SortShape& h, hipStream_t stream) {
  const int64_t chunk = h.chunk;
  const int blocks = h.blocks;
  int bits = 1;
  while ((1 << bits) <= G) ++bits;
  const int lds1 = (G + 1) * 4;
  // starts, waves' counts, shifts; then the tile's (row, slot) pairs
  const int lds2 = ((G + 1) * (2 + W) + 1) / 2 * 8 + 64 * W * PER * 8;
  static std::atomic<uint64_t> set{0};
  const hipError_t ea = ensure_dyn_lds(reinterpret_cast<const void*>(&expert_scatter_kernel<W, PER>),
                                       160 * 1024 - 512, set);
  if (ea != hipSuccess) return ea;
  // Up to 64 counts per thread every block adds the others' up itself; past
  // that a third launch does (524288 slots: 128 experts 12.1 us without it, 14.7
  // with it; 256 experts 14.5 and 14.6; 512 experts 19.8 and 16.1; 65536 x 8
  // slots of 4096 experts 124 and 37).
  const bool summed = blocks > 1 && blocks * (G + 1) > 64 * 64 * W;
  if (blocks > 1) {
    hipLaunchKernelGGL((expert_hist_kernel<W, PER>), dim3(blocks), dim3(64 * W), lds1, stream, ids, ws, S, G, chunk);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (summed) {
    hipLaunchKernelGGL(expert_prefix_kernel, dim3((G + 64) / 64), dim3(1024), 0, stream, ws, G + 1, blocks);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL((expert_scatter_kernel<W, PER>), dim3(blocks), dim3(64 * W), lds2, stream, ids, ws, order, pos,
                     m_sizes, S, G, chunk, blocks, bits, summed);
  return hipGetLastError();
}

hipError_t launch_expert_sort(const int32_t* ids, int32_t* order, int32_t* pos, int32_t* m_sizes, int64_t S, int G,
                              int32_t* ws, hipStream_t stream) {
  if (S == 0) {
    hipLaunchKernelGGL(expert_zero_kernel, dim3(1), dim3(256), 0, stream, m_sizes, G);
    return hipGetLastError();
  }
  const SortShape h = sort_shape(S, G);
  if (h.waves == 4) return launch_sort_w<4, 8>(ids, order, pos, m_sizes, S, G, ws, h, stream);
  if (h.waves == 8 && h.per == 4) return launch_sort_w<8, 4>(ids, order, pos, m_sizes, S, G, ws, h, stream);
  if (h.waves == 8) return launch_sort_w<8, 2>(ids, order, pos, m_sizes, S, G, ws, h, stream);
  if (h.per == 2) return launch_sort_w<16, 2>(ids, order, pos, m_sizes, S, G, ws, h, stream);
  return launch_sort_w<16, 4>(ids, order, pos, m_sizes, S, G, ws, h, stream);
}

// The variant by the rows: threads per token, the power of two that holds the
// row, 32 to 256; and the non-temporal hint on the expert rows where they are
// larger than the last-level cache (256 MB), so that their reader or writer
// could not meet them there anyway: combine at 16384 x 8 x 4096 (1.1 GB) 237.7
// -> 206.8 us, its gradient at 8192 x 8 x 4096 229.6 -> 210.1, gather at 16384
// x 4 x 5120 159.3 -> 155.8; but gather, grouped GEMM and combine of 1024 x 2
// tokens, K 4096, N 2048 (25 MB) one after the other 72.8 -> 76.5 us with it.
template <class F>
static hipError_t by_rows(int64_t rows, int width, F launch) {
  const int chunks = width / 8 + (width % 8 != 0 ? 1 : 0);
  const auto go = [&](auto aligned, auto nt) {
    if (chunks <= 32) launch(aligned, std::integral_constant<int, 32>{}, nt);
    else if (chunks <= 64) launch(aligned, std::integral_constant<int, 64>{}, nt);
    else if (chunks <= 128) launch(aligned, std::integral_constant<int, 128>{}, nt);
    else launch(aligned, std::integral_constant<int, 256>{}, nt);
  };
  const bool nt = rows * width > ((int64_t)128 << 20);   // values of 2 bytes
  if (width % 8 == 0 && nt) go(std::true_type{}, std::true_type{});
  else if (width % 8 == 0) go(std::true_type{}, std::false_type{});
  else if (nt) go(std::false_type{}, std::true_type{});
  else go(std::false_type{}, std::false_type{});
  return hipGetLastError();
}

// x: tokens, 256 / tpt per workgroup; y: 8 tpt columns each where `split` (the
// kernels stride over what is beyond the grid, which has at most 2^23
// workgroups: a launch takes fewer than 2^32 threads)
static dim3 row_grid(int64_t T, int width, int tpt, bool split) {
  const int64_t most = (int64_t)1 << 20;
  const int64_t x = std::min((T + 256 / tpt - 1) / (256 / tpt), most);
  const int64_t y = split ? ((int64_t)width + 8 * tpt - 1) / (8 * tpt) : 1;
  return dim3((unsigned)x, (unsigned)std::min(y, std::min<int64_t>(65535, 8 * most / x)));
}

hipError_t launch_expert_gather(const uint16_t* x, const int32_t* pos, uint16_t* xs, int64_t T, int k, int64_t rows,
                                int width, hipStream_t stream) {
  return by_rows(rows, width, [&](auto al, auto tpt, auto nt) {
    hipLaunchKernelGGL((expert_gather_kernel<decltype(al)::value, decltype(tpt)::value, decltype(nt)::value>),
                       row_grid(T, width, decltype(tpt)::value, true), dim3(256), 0, stream, x, pos, xs, T, k, rows,
                       width);
  });
}

hipError_t launch_expert_combine(const uint16_t* z, const int32_t* pos, const float* w, uint16_t* y, int64_t T, int k,
                                 int64_t rows, int width, hipStream_t stream) {
  return by_rows(rows, width, [&](auto al, auto tpt, auto nt) {
    hipLaunchKernelGGL((expert_combine_kernel<decltype(al)::value, decltype(tpt)::value, decltype(nt)::value>),
                       row_grid(T, width, decltype(tpt)::value, true), dim3(256), 0, stream, z, pos, w, y, T, k, rows,
                       width);
  });
}

hipError_t launch_expert_combine_grad(const uint16_t* dy, const uint16_t* z, const int32_t* pos, const float* w,
                                      uint16_t* dz, float* dw, int64_t T, int k, int64_t rows, int width,
                                      hipStream_t stream) {
  return by_rows(rows, width, [&](auto al, auto tpt, auto nt) {
    hipLaunchKernelGGL((expert_combine_grad_kernel<decltype(al)::value, decltype(tpt)::value, decltype(nt)::value>),
                       row_grid(T, width, decltype(tpt)::value, false), dim3(256), 0, stream, dy, z, pos, w, dz, dw, T,
                       k, rows, width);
  });
}

}  // namespace w4a16
