// C-ABI entry points: argument validation on the host (before anything is
// enqueued), path and split-K selection, workspace layout and launches.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <mutex>

#include <stddef.h>
#include <stdint.h>

#include "../../include/w4a16.h"
#include "launch.hpp"
#include "lora.hpp"
#include "w4a16_internal.h"

namespace {

constexpr int64_t kGroup = 128;       // k per pipeline stage (and the default scale group)
constexpr int32_t kGroupSmall = 32;   // the other scale group size (tile path only)
constexpr int64_t kMaxDim = 0x7FFFFFFFLL;
constexpr uint64_t kMaxBytes = 0xFFFFFFFFULL;   // one buffer resource extent

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
uint64_t round_up(uint64_t v, uint64_t a) { return (v + a - 1) / a * a; }

bool valid_split(int32_t sk) { return sk == 0 || sk == 1 || sk == 2 || sk == 4 || sk == 8 || sk == 16; }

// Which kernel family runs a plain GEMM at this shape.
enum Path { kPathAuto = 0, kPathGemv = 1, kPathSkinny = 2, kPathTile = 3 };

int32_t pow2_at_least(int64_t v) {
  int32_t p = 1;
  while (p < v && p < 16) p <<= 1;
  return p;
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Compute units of the current device (cached per device; safe to call from
// several host threads).
int device_cus() {
  static std::atomic<int> cache[64];
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return 256;
  int v = cache[dev].load(std::memory_order_relaxed);
  if (v == 0) {
    if (hipDeviceGetAttribute(&v, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || v <= 0) v = 256;
    cache[dev].store(v, std::memory_order_relaxed);
  }
  return v;
}

// Small batch: the register-streaming kernel with one column tile of 16 per
// wave up to 8 rows and past 32, two between (8 waves per workgroup; at
// 17408 x 5120 and 8192 x 8192: M = 2-4 7-10 % faster with one tile, M >= 9
// 4-12 % faster with two; past 32 rows the three row tiles leave registers
// for one only). At 9-16 rows the LDS-staged kernel (variant 6: stages of 4
// groups, 4 in flight) instead: over N x K = 8192 x 8192, 17408 x 5120,
// 7168 x 8192, 4096 x 4096, 2560 x 9728, 2048 x 5120 and 896 x 5120 it ran
// 2-18 % faster at M = 16; at M = 8 it lost at four of the seven, at M <= 4
// at five, by up to 33 % (its X stage is read in full whatever M is).
int skinny_default_tiles(int64_t M) {
  if (M > 8 && M <= 16) return 6;
  return M <= 8 || M > 32 ? 1 : 2;
}
constexpr int kSkinnyWaves = 8;

Path auto_path(int64_t M, int64_t N, int64_t K, int32_t sk) {
  const int64_t Gk = K / kGroup;
  if (M == 1) {
    // the GEMV keeps a lane's x in registers: at most 64 groups per slice
    const int64_t s = sk > 0 ? sk : 16;
    return ceil_div(Gk, s) <= 64 ? kPathGemv : kPathSkinny;
  }
  if (M <= 16) return kPathSkinny;
  // two row tiles of 16 (one 8-wave workgroup per compute unit per round):
  // at 17 <= M <= 32 the small-batch kernel ran 6-33 % faster than the tile
  // kernel at 17408 x 5120, 8192 x 8192 and 2560 x 9728 (at most 2.1 rounds
  // of workgroups), 4-12 % slower at 28672 x 8192 (3.5 rounds)
  if (M <= 32 && ceil_div(N, 32) <= 3 * (int64_t)device_cus()) return kPathSkinny;
  // three row tiles (8 waves of one column tile): only while one round of
  // workgroups covers N (4096 x 4096 and 2560 x 9728 at 33-48 rows: 8-35 %
  // faster than the tile kernel; 8192 x 8192, two rounds: 15-30 % slower)
  if (M <= w4a16::kSkinnyMaxRows && ceil_div(N, 16) <= (int64_t)device_cus()) return kPathSkinny;
  return kPathTile;
}

// Cost model of the tile path, in units of one row x one 128-group of work on
// one compute unit at the 128-row tile's rate (≈0.0162 us on MI355X: the
// 144-row tile runs 20 groups in 48.7 us). One workgroup per compute unit:
// a launch takes ceil(tiles x SK / CUs) rounds of (rows / rate) x groups per
// slice. A split adds its fp32 partials, written by the tile kernel and read
// by the reduce (8 x SK x M x N bytes at ≈4 TB/s), the reduce launch (≈1 us)
// and ≈1.5 us per 8 slices (the reduce has the loads of up to 8 slices in
// flight before it adds them, so every 8 slices are one more round trip).
// Splits only where tiles x SK fit one round (a second, mostly idle round of
// slices never pays: at M = 96..384, N x K = 17408 x 5120 doubling past it
// cost 24-52 %). The three split costs and the rates of the 48- to 80-row
// tiles below were fitted to every explicit choice timed at 42 shapes (M
// 64..4096; N x K 896..17408 x 2560..8192): the automatic choice is within
// 1 % of the fastest at 41 of them and 5.6 % at the last (with the partials
// at 5 TB/s, a 2 us launch and no per-8-slices term: 1.7 % on average, 10 %
// at worst, by choosing SK 16 where 8 was faster), and the deep prefill,
// grouped and batched workloads keep their choices.
constexpr double kUnitUs = 0.0162, kReduceBytesPerUs = 4.0e6, kReduceLaunchUs = 1.0, kReduceBatchUs = 1.5;

double tile_cost(int64_t M, int64_t N, int64_t Gk, int64_t tiles, int bm, double rate, int64_t sk, int64_t cus) {
  double c = (double)ceil_div(tiles * sk, cus) * bm / rate * (double)ceil_div(Gk, sk);
  if (sk > 1)
    c += (8.0 * (double)sk * (double)M * (double)N / kReduceBytesPerUs + kReduceLaunchUs +
          (double)ceil_div(sk, 8) * kReduceBatchUs) /
         kUnitUs;
  return c;
}

// The split of least cost for `tiles` tiles of bm rows (rate: per-row rate of
// the height): 1, or a power of two up to 16 (and the group count) whose
// slices fit one round.
int32_t tile_split_rate(int64_t M, int64_t N, int64_t Gk, int64_t tiles, int bm, double rate) {
  const int64_t cus = device_cus();
  int32_t best = 1;
  double best_cost = tile_cost(M, N, Gk, tiles, bm, rate, 1, cus);
  for (int32_t sk = 2; sk <= 16 && sk <= Gk && tiles * sk <= cus; sk <<= 1) {
    const double c = tile_cost(M, N, Gk, tiles, bm, rate, sk, cus);
    if (c < best_cost * (1.0 - 1e-9)) {
      best = sk;
      best_cost = c;
    }
  }
  return best;
}

// Per-row rates of the tile heights, relative to the 128-row tile (shorter
// tiles amortise the per-group dequantisation and barrier over fewer rows;
// at 1322 x 19456 x 2560 on one box: 4 rounds of 128 rows 166 us, 4 of 112
// rows 161 us, 3 of 144 rows 146 us, 5 of 96 rows 176 us; the 80-, 64- and
// 48-row rates fitted with the split costs above).
struct TileCand { int bm; double rate; };
constexpr TileCand kTileCands[] = {{128, 1.0}, {144, 0.96}, {112, 0.91}, {96, 0.907},
                                   {80, 0.80}, {64, 0.66},  {48, 0.58}};

double tile_rate(int bm) {
  for (const TileCand& c : kTileCands)
    if (c.bm == bm) return c.rate;
  return 0.9;
}

int32_t tile_split(int64_t M, int64_t N, int64_t Gk, int64_t tiles, int bm) {
  return tile_split_rate(M, N, Gk, tiles, bm, tile_rate(bm));
}

// Tile height of the least estimated cost, with its own best split when
// split_k is automatic (`split` < 0) or the given one. `tiles(bm)` counts the
// output tiles of a height. Only heights built for the scale group size gs
// are candidates.
template <class T>
int pick_tile_rows(int64_t M, int64_t N, int64_t Gk, T tiles, int64_t split, int32_t gs) {
  const int64_t cus = device_cus();
  int best = 128;
  double best_cost = 0.0;
  for (const TileCand& c : kTileCands) {
    if (!w4a16::tile_rows_ok(c.bm, gs)) continue;
    const int64_t t = tiles(c.bm);
    const int64_t sk = split > 0 ? split : tile_split_rate(M, N, Gk, t, c.bm, c.rate);
    const double cost = tile_cost(M, N, Gk, t, c.bm, c.rate, sk, cus);
    if (best_cost == 0.0 || cost < best_cost * (1.0 - 1e-9)) {
      best = c.bm;
      best_cost = cost;
    }
  }
  return best;
}

int64_t tile_cols(int64_t N) { return ceil_div(N, w4a16::kTileCols); }

// split_k = 0: automatic, chosen with the height; otherwise fixed
int default_tile_rows(int64_t M, int64_t N, int64_t K, int32_t split_k, int32_t gs) {
  const int64_t nt = tile_cols(N), Gk = K / kGroup;
  return pick_tile_rows(
      M, N, Gk, [&](int bm) { return ceil_div(std::max<int64_t>(M, 1), bm) * nt; }, split_k > 0 ? split_k : -1,
      gs);
}

// grouped (no split-K): M_sizes stays on the device, so the tile count is
// estimated as ceil(M_total / bm) + G / 2 per column (each group's partial
// last tile adds half a tile on average; the kernel maps only the real tiles)
int default_grouped_tile_rows(int64_t G, int64_t M_total, int64_t N, int64_t K, int32_t gs) {
  const int64_t nt = tile_cols(N);
  return pick_tile_rows(
      M_total, N, K / kGroup,
      [&](int bm) { return (ceil_div(std::max<int64_t>(M_total, 1), bm) + G / 2) * nt; }, 1, gs);
}

int32_t auto_split(Path path, int64_t M, int64_t N, int64_t K, int bm, int nt) {
  const int64_t Gk = K / kGroup;
  int32_t sk = 1;
  switch (path) {
    case kPathGemv:
      // only what the register budget for x needs (at most 64 groups per
      // slice): a split adds the reduce kernel, and over N x K from 1024 x
      // 8192 to 28672 x 8192 one slice was fastest wherever it fits
      sk = pow2_at_least(ceil_div(Gk, 64));
      break;
    case kPathSkinny: {
      // split only when fewer than half of the compute units have a
      // workgroup, and then as far as one round of workgroups goes: the
      // reduce kernel and the partials cost more than the shorter slices save
      // once the grid is half full (4096 x 4096, 128 workgroups: SK 1 8-16 %
      // faster than 2), while a grid a quarter full or less gains from
      // filling the GPU (M = 16 at 2048 x 5120, 64 workgroups: SK 4 9.3 us,
      // SK 2 10.3; at 896 x 5120, 28 workgroups: SK 8 8.7, SK 4 9.1;
      // 2560 x 9728, 80 workgroups: SK 2 20 % faster than 4)
      const int64_t wgs = ceil_div(N, 16 * (int64_t)nt), cus = device_cus();
      if (2 * wgs < cus)
        while (sk < 16 && 2 * sk <= Gk && wgs * sk * 2 <= cus) sk <<= 1;
      break;
    }
    case kPathTile:
      sk = tile_split(M, N, Gk, ceil_div(M, bm) * tile_cols(N), bm);
      break;
    default:
      break;
  }
  return sk;
}

// Row sums of X on the tile path: the tile kernel forms -136 * sum_k x per
// (row, scale group) itself, on the matrix core, in every column tile; a
// separate pre-pass forms them once, into the workspace. The kernel's own
// sums cost more once many column tiles repeat them (1322 x 19456 x 2560,
// 76 column tiles: 157 against 150.5 us with the pre-pass; N = 2048 and
// 4096 at 1322 rows, 8 and 16 tiles: 1-3 us faster than the pre-pass; at
// group 32 the in-kernel sums take four MFMAs per stage instead of one chain
// and the crossover is lower), so the pre-pass is used from 32 column tiles
// at group 128 and 8 at group 32, when the caller gives the workspace room.
bool tile_prepass(int64_t N, int32_t gs) { return tile_cols(N) * (kGroup / gs) >= 32; }

// bytes of the [K / gs, ld] fp32 row sums of the pre-pass
uint64_t rowsum_bytes(int64_t M, int64_t K, int32_t gs) {
  return (uint64_t)(K / gs) * round_up((uint64_t)M, 4) * 4u;
}

struct Plan {
  Path path;
  int32_t sk;         // effective split-K
  int32_t gps;        // 128-groups per slice
  int variant;        // GEMV: 1 = half-wave layout; small batch: column tiles per wave; tile: rows per tile
  uint64_t ws_split;  // bytes of the [SK, M, N] fp32 partials
  uint64_t ws_sx;     // bytes of the pre-pass row sums (tile path with a wide N), else 0
};

// Group size 32 runs on the tile path only (the GEMV and small-batch kernels
// take one scale per 128 k), whatever M is.
w4a16_status make_plan(int64_t M, int64_t N, int64_t K, int32_t split_k, const w4a16_config* cfg, int32_t gs,
                       Plan* p) {
  const int64_t Gk = K / kGroup;
  Path path = gs == kGroup ? auto_path(M, N, K, split_k) : kPathTile;
  int variant = -1;
  if (cfg != nullptr) {
    if (cfg->path < 0 || cfg->path > 3) return W4A16_ERR_SHAPE;
    if (cfg->path != 0) path = (Path)cfg->path;
    variant = cfg->variant;
  }
  if (path == kPathGemv && M != 1) return W4A16_ERR_SHAPE;
  if (path == kPathSkinny && M > w4a16::kSkinnyMaxRows) return W4A16_ERR_SHAPE;
  if (path != kPathTile && gs != kGroup) return W4A16_ERR_GROUP_SIZE;
  switch (path) {
    case kPathGemv:
      if (variant > 1) return W4A16_ERR_SHAPE;
      if (variant < 0) variant = 0;   // the MFMA layout where it applies
      break;
    case kPathSkinny:
      if (variant <= 0) variant = skinny_default_tiles(M);
      // past 32 rows (three row tiles) one column tile per wave only; variants
      // 3..6: the LDS-staged kernel (M <= 16), stage geometries 0..3
      if (variant > 6 || (M > 32 && variant != 1) || (variant >= 3 && M > 16)) return W4A16_ERR_SHAPE;
      break;
    case kPathTile:
      if (variant <= 0) variant = default_tile_rows(M, N, K, split_k, gs);
      if (!w4a16::tile_rows_ok(variant, kGroup) && !w4a16::tile_rows_ok(variant, kGroupSmall))
        return W4A16_ERR_SHAPE;
      if (!w4a16::tile_rows_ok(variant, gs)) return W4A16_ERR_GROUP_SIZE;
      break;
    default:
      return W4A16_ERR_SHAPE;
  }
  int32_t sk = split_k > 0 ? split_k : auto_split(path, M, N, K, variant, variant >= 3 ? 2 : variant);
  if (sk > Gk && split_k == 0) sk = 1;
  if (path == kPathGemv && ceil_div(Gk, sk) > 64) {
    if (split_k != 0) return W4A16_ERR_SPLIT_K;   // explicit split too small for the GEMV path
    sk = pow2_at_least(ceil_div(Gk, 64));
  }
  p->path = path;
  p->sk = sk;
  p->gps = (int32_t)ceil_div(Gk, sk);
  p->variant = variant;
  p->ws_split = sk > 1 ? (uint64_t)sk * (uint64_t)M * (uint64_t)N * 4u : 0u;
  p->ws_sx = path == kPathTile && tile_prepass(N, gs) ? rowsum_bytes(M, K, gs) : 0u;
  return W4A16_OK;
}

uint64_t plan_bytes(const Plan& p) { return round_up(p.ws_split, 256) + p.ws_sx; }

w4a16_status check_dims(int64_t M, int64_t N, int64_t K, int32_t group_size) {
  if (M < 0 || N < 1 || K < 1 || M > kMaxDim || N > kMaxDim || K > kMaxDim) return W4A16_ERR_SHAPE;
  if ((group_size != kGroup && group_size != kGroupSmall) || K % kGroup != 0) return W4A16_ERR_GROUP_SIZE;
  // buffer extents of one resource
  if ((uint64_t)N * (uint64_t)K / 2u > kMaxBytes) return W4A16_ERR_SHAPE;
  if ((uint64_t)M * (uint64_t)K * 2u > kMaxBytes) return W4A16_ERR_SHAPE;
  if ((uint64_t)M * (uint64_t)N * 4u > kMaxBytes) return W4A16_ERR_SHAPE;
  return W4A16_OK;
}

w4a16_status check_batched(int32_t B, int64_t M, int64_t N, int64_t K, int32_t group_size) {
  if (B < 1 || M < 0) return W4A16_ERR_SHAPE;
  if ((uint64_t)B * (uint64_t)M > (uint64_t)kMaxDim) return W4A16_ERR_SHAPE;
  w4a16_status st = check_dims((int64_t)B * M, N, K, group_size);
  if (st != W4A16_OK) return st;
  // one buffer resource covers the scales of all problems
  if ((uint64_t)B * (uint64_t)N * (uint64_t)(K / group_size) * 2u > kMaxBytes) return W4A16_ERR_SHAPE;
  return W4A16_OK;
}

w4a16_status launched(hipError_t e) { return e == hipSuccess ? W4A16_OK : W4A16_ERR_LAUNCH; }

// Validated plan of a plain GEMM: status, or W4A16_OK with *p filled and
// *empty set when M == 0 (nothing to enqueue).
w4a16_status plan_gemm(const uint16_t* x, const uint8_t* w, const uint16_t* s, uint16_t* y, int64_t M, int64_t N,
                       int64_t K, int32_t group_size, int32_t split_k, const w4a16_config* cfg, Plan* p,
                       bool* empty) {
  *empty = false;
  if (!valid_split(split_k)) return W4A16_ERR_SPLIT_K;
  w4a16_status st = check_dims(M, N, K, group_size);
  if (st != W4A16_OK) return st;
  if (M == 0) {   // empty problem: nothing to read or write
    *empty = true;
    return W4A16_OK;
  }
  if (x == nullptr || w == nullptr || s == nullptr || y == nullptr) return W4A16_ERR_NULL;
  if (!aligned16(x) || !aligned16(w) || !aligned16(s) || !aligned16(y)) return W4A16_ERR_ALIGN;
  st = make_plan(M, N, K, split_k, cfg, group_size, p);
  if (st != W4A16_OK) return st;
  if (p->ws_split > kMaxBytes) return W4A16_ERR_SHAPE;
  return W4A16_OK;
}

// Enqueues a planned GEMM; `partials` holds the [SK, M, N] fp32 slices when
// p.sk > 1 (unused otherwise); `rowsums` (tile path, may be nullptr) the
// pre-pass row sums; `la` per-row adapters (the row sums are there already).
w4a16_status launch_plan(const Plan& p, const uint16_t* x, const uint8_t* w, const uint16_t* s, uint16_t* y,
                         int64_t M, int64_t N, int64_t K, int32_t group_size, float* partials, float* rowsums,
                         hipStream_t strm, const w4a16::LoraArgs* la = nullptr) {
  float* ws_split = p.sk > 1 ? partials : nullptr;
  const int iM = (int)M, iN = (int)N, iK = (int)K;
  hipError_t e = hipSuccess;
  switch (p.path) {
    case kPathGemv:
      e = w4a16::launch_gemv_m1(x, w, s, y, ws_split, iN, iK, p.gps, p.sk, p.variant == 1, strm, la);
      break;
    case kPathSkinny:
      if (p.variant >= 3 && w4a16::skinny_lds_fits(iM, p.gps))
        e = w4a16::launch_skinny_lds(x, w, s, y, ws_split, iM, iN, iK, p.gps, p.sk, p.variant - 3, strm, la);
      else
        e = w4a16::launch_skinny(x, w, s, y, ws_split, iM, iN, iK, p.gps, p.sk, p.variant >= 3 ? 1 : p.variant,
                                 kSkinnyWaves, strm, la);
      break;
    case kPathTile: {
      const int ld = (int)round_up((uint64_t)M, 4);
      // with adapters they came with x . A^T
      if (rowsums != nullptr && la == nullptr)
        e = w4a16::launch_rowsum_neg136(x, rowsums, iM, iK, ld, group_size, strm);
      if (e == hipSuccess)
        e = w4a16::launch_tile(x, w, s, rowsums, ld, y, ws_split, nullptr, 0, iM, iN, iK, 1, p.gps, p.sk, p.variant,
                               group_size, strm, la);
      break;
    }
    default:
      return W4A16_ERR_SHAPE;
  }
  if (e != hipSuccess) return W4A16_ERR_LAUNCH;
  if (p.sk > 1) return launched(w4a16::launch_splitk_reduce(ws_split, y, (uint64_t)M * (uint64_t)N, p.sk, strm));
  return W4A16_OK;
}

w4a16_status run_gemm(const uint16_t* x, const uint8_t* w, const uint16_t* s, uint16_t* y, int64_t M, int64_t N,
                      int64_t K, int32_t group_size, int32_t split_k, float* workspace, size_t workspace_bytes,
                      void* stream, const w4a16_config* cfg) {
  Plan p;
  bool empty = false;
  w4a16_status st = plan_gemm(x, w, s, y, M, N, K, group_size, split_k, cfg, &p, &empty);
  if (st != W4A16_OK || empty) return st;
  if (p.ws_split > 0) {
    if (workspace == nullptr) return W4A16_ERR_WORKSPACE;
    if (!aligned16(workspace)) return W4A16_ERR_ALIGN;
    if (workspace_bytes < round_up(p.ws_split, 256)) return W4A16_ERR_WORKSPACE;
  }
  // the pre-pass row sums only where the workspace has room for them too
  float* rowsums = nullptr;
  if (p.ws_sx > 0 && workspace != nullptr && aligned16(workspace) && workspace_bytes >= plan_bytes(p))
    rowsums = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(workspace) + round_up(p.ws_split, 256));
  return launch_plan(p, x, w, s, y, M, N, K, group_size, workspace, rowsums, reinterpret_cast<hipStream_t>(stream));
}

size_t gemm_workspace_bytes(int64_t M, int64_t N, int64_t K, int32_t group_size, int32_t split_k,
                            const w4a16_config* cfg) {
  if (!valid_split(split_k) || check_dims(M, N, K, group_size) != W4A16_OK || M == 0) return 0;
  Plan p;
  if (make_plan(M, N, K, split_k, cfg, group_size, &p) != W4A16_OK) return 0;
  return (size_t)plan_bytes(p);
}

// Batched: B problems of M rows on the tile kernel (weight group b = problem
// b, its M rows at b * M), tile height and split-K as for one problem of B x
// ceil(M / h) row tiles per column. (M <= 16 problems run the tile kernel too:
// the per-problem scale tensors are not 16-byte aligned in general, which the
// decode kernels require.)
struct BatchedPlan {
  int bm;
  int32_t sk, gps;
  uint64_t ws_split, ws_sx;
};

w4a16_status make_batched_plan(int32_t B, int64_t M, int64_t N, int64_t K, int32_t split_k, const w4a16_config* cfg,
                               int32_t gs, BatchedPlan* p) {
  const int64_t Gk = K / kGroup, nt = tile_cols(N), Mt = (int64_t)B * M;
  int bm = -1;
  if (cfg != nullptr) {
    if (cfg->path != 0 && cfg->path != kPathTile) return W4A16_ERR_SHAPE;
    bm = cfg->variant;
  }
  if (bm <= 0)
    bm = pick_tile_rows(
        Mt, N, Gk, [&](int h) { return (int64_t)B * ceil_div(M, h) * nt; }, split_k > 0 ? split_k : -1, gs);
  if (!w4a16::tile_rows_ok(bm, kGroup) && !w4a16::tile_rows_ok(bm, kGroupSmall)) return W4A16_ERR_SHAPE;
  if (!w4a16::tile_rows_ok(bm, gs)) return W4A16_ERR_GROUP_SIZE;
  const int64_t tiles = (int64_t)B * ceil_div(M, bm) * nt;
  int32_t sk = split_k > 0 ? split_k : tile_split(Mt, N, Gk, tiles, bm);
  if (sk > Gk && split_k == 0) sk = 1;
  p->bm = bm;
  p->sk = sk;
  p->gps = (int32_t)ceil_div(Gk, sk);
  p->ws_split = sk > 1 ? (uint64_t)sk * (uint64_t)Mt * (uint64_t)N * 4u : 0u;
  p->ws_sx = tile_prepass(N, gs) ? rowsum_bytes(Mt, K, gs) : 0u;
  return W4A16_OK;
}

size_t batched_workspace_bytes(int32_t B, int64_t M, int64_t N, int64_t K, int32_t group_size, int32_t split_k,
                               const w4a16_config* cfg) {
  if (!valid_split(split_k) || check_batched(B, M, N, K, group_size) != W4A16_OK || M == 0) return 0;
  BatchedPlan p;
  if (make_batched_plan(B, M, N, K, split_k, cfg, group_size, &p) != W4A16_OK) return 0;
  return (size_t)(round_up(p.ws_split, 256) + p.ws_sx);
}

// ---------------------------------------------------------------- scratch of the no-allocation entry point
// Device scratch for w4a16_gemm_noalloc: the split-K partials and the
// pre-pass row sums live here instead of in a caller's workspace. Each GPU
// holds its own copy (allocated with the library's code object) until the
// process ends. In host code `scratch` names a host-side stand-in, so its
// device address comes from hipGetSymbolAddress, once per device.
constexpr size_t kScratchBytes = (size_t)W4A16_NOALLOC_SCRATCH_BYTES;
__device__ __align__(256) uint8_t scratch[kScratchBytes];

constexpr int kMaxDevices = 64;
std::mutex g_scratch_mu;
void* g_scratch_ptr[kMaxDevices] = {};

// The device address of this GPU's scratch (nullptr on failure): looked up
// with the device current, on the first call per device, and kept.
void* scratch_ptr() {
  int dev = -1;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) return nullptr;
  std::lock_guard<std::mutex> lock(g_scratch_mu);
  if (g_scratch_ptr[dev] == nullptr) {
    void* p = nullptr;
    if (hipGetSymbolAddress(&p, HIP_SYMBOL(scratch)) != hipSuccess) return nullptr;
    g_scratch_ptr[dev] = p;
  }
  return g_scratch_ptr[dev];
}

// ---------------------------------------------------------------- low-rank adapters
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

struct LoraPlan {
  Plan base;       // the projection
  uint64_t ws_h;   // bytes of the [2, M, R] bf16 parts of x . A^T, ahead of the projection's workspace
};

w4a16_status make_lora_plan(int64_t M, int64_t N, int64_t K, int32_t group_size, int32_t L, int32_t R,
                            int32_t split_k, LoraPlan* p) {
  if (!valid_split(split_k)) return W4A16_ERR_SPLIT_K;
  w4a16_status st = check_dims(M, N, K, group_size);
  if (st != W4A16_OK) return st;
  if (L < 1 || R < 8 || R > w4a16::kLoraMaxRank || R % 8 != 0) return W4A16_ERR_SHAPE;
  if ((uint64_t)N * (uint64_t)R * 2u > kMaxBytes || (uint64_t)K * (uint64_t)R * 2u > kMaxBytes ||
      (uint64_t)M * (uint64_t)R * 4u > kMaxBytes)
    return W4A16_ERR_SHAPE;
  if (M == 0) return W4A16_OK;
  st = make_plan(M, N, K, split_k, nullptr, group_size, &p->base);
  if (st != W4A16_OK) return st;
  if (p->base.path == kPathGemv && !w4a16::gemv_mfma_fits(p->base.gps)) {
    // a slice length of the half-wave GEMV, which takes no adapters
    const w4a16_config cfg = {kPathSkinny, -1};
    st = make_plan(M, N, K, split_k, &cfg, group_size, &p->base);
    if (st != W4A16_OK) return st;
  }
  if (p->base.ws_split > kMaxBytes) return W4A16_ERR_SHAPE;
  p->ws_h = round_up((uint64_t)M * (uint64_t)R * 4u, 256);
  return W4A16_OK;
}

uint64_t lora_bytes(const LoraPlan& p) { return p.ws_h + plan_bytes(p.base); }

// ---------------------------------------------------------------- rows of a mixture of experts
bool expert_slots_ok(int64_t T, int32_t k) { return T >= 0 && k >= 1 && T <= kMaxDim / k; }

uint64_t expert_sort_bytes(int64_t T, int32_t k, int32_t G) {
  const int blocks = w4a16::expert_sort_blocks(T * k, G);
  return blocks > 1 ? round_up((uint64_t)(blocks + 1) * (uint64_t)(G + 1) * 4u, 256) : 0u;
}

// Checks of the calls on rows; *empty: nothing to enqueue.
w4a16_status check_expert_rows(int64_t T, int32_t k, int64_t rows, int64_t width, const int32_t* pos, bool* empty) {
  *empty = false;
  if (!expert_slots_ok(T, k) || rows < 0 || rows > kMaxDim || width < 1 || width > kMaxDim) return W4A16_ERR_SHAPE;
  if (T == 0) {
    *empty = true;
    return W4A16_OK;
  }
  if (pos == nullptr) return W4A16_ERR_NULL;
  if (!aligned4(pos)) return W4A16_ERR_ALIGN;
  return W4A16_OK;
}

w4a16_status run_expert_combine(const uint16_t* z, const int32_t* pos, const float* weights, uint16_t* y, int64_t T,
                                int32_t k, int64_t rows, int64_t width, void* stream) {
  bool empty = false;
  const w4a16_status st = check_expert_rows(T, k, rows, width, pos, &empty);
  if (st != W4A16_OK || empty) return st;
  if (y == nullptr || (z == nullptr && rows > 0)) return W4A16_ERR_NULL;
  if (!aligned16(y) || !aligned16(z) || !aligned4(weights)) return W4A16_ERR_ALIGN;
  return launched(w4a16::launch_expert_combine(z, pos, weights, y, T, k, rows, (int)width,
                                               reinterpret_cast<hipStream_t>(stream)));
}

// ---------------------------------------------------------------- 8-bit products and input gradients
struct RowsPlan {
  int bm;       // rows per tile
  int32_t sk;   // slices of the contraction
};

// Estimated time of the tile kernels in us: `tiles` workgroups (one per compute
// unit at a time) of `steps` contraction steps of `step_us`, and what a workgroup
// costs besides (first loads, outputs). Past one round the last, partly filled
// one counts in part: workgroups do not end together (1322 x 19456 x 2560: 2.08
// rounds of 192 rows run like 2.4, 3.3 of 128 like 3.5).
double rounds_us(double tiles, double steps, double step_us, double extra_us, double cus) {
  const double r = tiles / cus;
  const double eff = r <= 1.0 ? 1.0 : 0.4 * r + 0.6 * std::ceil(r);
  return eff * (extra_us + steps * step_us);
}

// Partial sums of a split contraction, written and read, and the launch of the
// reduce (777 x 9728 x 2560: 8, 10, 13 us for 2, 3, 4 slices of 8 MB).
double split_us(int32_t sk, double outputs) { return sk > 1 ? 2.5 + 8.0 * sk * outputs / 6.0e6 : 0.0; }

struct TileTime {
  int bm;
  double us;   // of one contraction step
};

// Row tiles of height bm of G groups with M rows together, if their sizes spread like
// an exponential distribution; 2 % fewer, so that barely more than a round counts as
// one. (By M / bm + G / 2, which short groups exceed, 4096 rows of 32 experts of 2048 x
// 4096 took 122 us, 87 to 92 so.)
double expected_tiles(int64_t G, int64_t M, int bm) {
  const double groups = (double)std::max<int64_t>(std::min(G, M), 1), rows = (double)std::max<int64_t>(M, 1);
  return 0.98 * groups / (1.0 - std::exp(-(double)bm * groups / rows));
}

// Least estimated time over the tile heights and (unless `split` is false) the
// splits whose workgroups, as many as there may be, fit one round (by expert, by the
// expected number instead: 200 rows of 8 experts of 4096 x 4096 44 -> 56 us); `forced`
// > 0 fixes the height. half_from > 0: from this height on, past one round, a plain
// problem's last row tile counts as a half if it has at most half the height's rows
// (two rows of waves, of which those without rows only load). weight_bytes (0: not
// regarded): no choice takes less than reading them, at a copy's rate (80 x 8192 x
// 8192: 8 slices of 128 rows 30.8 us, 4 of 64 28.8); least_step: nor a step less than
// this. row_bytes: the longest row that a tile addresses. Its offsets within a tile are
// 32 bits, those of the rows past the last one too (they would wrap into the rows that
// are there), so that only heights are taken whose rows fit one extent, and whose
// workgroups one launch; bm = 0: none.
template <size_t NT>
RowsPlan plan_tiles(const TileTime (&cands)[NT], double extra_us, int64_t G, int64_t M, int64_t O, int64_t steps,
                    int forced, int64_t min_steps, int half_from, bool split, double weight_bytes, double least_step,
                    uint64_t row_bytes) {
  RowsPlan best = {0, 1};
  double least = -1.0;
  const int64_t ot = ceil_div(O, 256);
  const double cus = device_cus();
  for (const TileTime& c : cands) {
    if ((forced > 0 && c.bm != forced) || (uint64_t)c.bm * row_bytes > kMaxBytes) continue;
    const double mt = G > 0 ? expected_tiles(G, M, c.bm) : (double)ceil_div(std::max<int64_t>(M, 1), c.bm);
    const double tiles = mt * (double)ot;
    const double most = G > 0 ? (double)(ot * w4a16::group_tiles_bound((int)M, c.bm, (int)G)) : tiles;
    if (most > (double)w4a16::kMaxBlocks) continue;
    const bool half = half_from > 0 && c.bm >= half_from && G == 0 && tiles > cus && M % c.bm != 0 &&
                      M % c.bm <= c.bm / 2;
    for (const int32_t sk : {1, 2, 3, 4, 5, 6, 8, 10, 12, 16}) {
      const int64_t part = sk == 1 ? steps : ceil_div(steps, sk);
      if (sk > 1 && (!split || most * sk > cus || part < min_steps)) break;
      const double wgs = half ? tiles - 0.5 * (double)ot : tiles * sk;
      const double step = std::max(c.us, least_step);
      const double us = std::max(rounds_us(wgs, (double)part, step, extra_us, cus), 1.0 + weight_bytes / 5.2e6) +
                        split_us(sk, (double)M * (double)O);
      if (least < 0.0 || us < least * (1.0 - 1e-9)) {
        least = us;
        best = {c.bm, sk};
      }
    }
  }
  return best;
}

// One block of 128 of the 8-bit tile kernel by height, between what it takes
// alone and with every compute unit busy (lower clocks): at 777 x 9728 x 2560 and
// 8192^3 256 rows 1.42 and 1.78 us, 128 rows 0.93 and 1.04, 64 rows 0.70 and 0.63
// (with the weights from memory 0.81); 32 rows serve experts with few (300 rows of 8
// experts of 2048 x 4096 22.7 -> 17.7 us, gradient of 1000 rows of 64 139 -> 116).
constexpr TileTime kFp8Times[] = {{256, 1.65}, {224, 1.60}, {192, 1.37}, {160, 1.15},
                                  {128, 0.99}, {96, 0.82},  {64, 0.72},  {32, 0.50}};
constexpr double kFp8ExtraUs = 6.0;

// The kernel for few rows holds those of a plain product in LDS (its grid has 16 rows
// per y); by expert it takes up to 64 output columns at a time, whose offsets are 32
// bits, a workgroup for each row tile and columns.
bool fp8_rows_built(bool grad, int64_t G, int64_t M, int64_t O, int64_t cb) {
  if (grad) return false;
  if (G == 0) return w4a16::fp8_rows_lds(M, cb * kGroup) <= w4a16::kRowsLds && M <= 16 * 65535;
  const int64_t cols = 16 * w4a16::fp8_rows_tiles((int)M, (int)O, (int)G, device_cus());
  return 64 * (uint64_t)(cb * kGroup) <= kMaxBytes &&
         w4a16::group_tiles_bound((int)M, 16, (int)G) * ceil_div(O, cols) <= w4a16::kMaxBlocks;
}

// M rows of G groups (0: plain), O output columns, cb contraction blocks; bm = 0: no
// tile can address the rows (or, in the products, 256 output columns' weights), or all
// heights have more workgroups than a launch takes
RowsPlan fp8_plan(bool grad, int64_t G, int64_t M, int64_t O, int64_t cb, int forced) {
  const int64_t per = G > 0 ? ceil_div(M, G) : M;
  if (forced == 16 || (forced == 0 && per <= 16 && fp8_rows_built(grad, G, M, O, cb))) return {16, 1};
  const double bytes = G > 0 ? 0.0 : (double)O * (double)cb * kGroup;
  // (plain: a stage of weights from memory; 17 x 17408 x 5120 at 32 rows: 3 slices 24.3
  // us, 2 slices, as 0.50 would have it, 27.3)
  const double least_step = G > 0 ? 0.0 : 0.68;
  const uint64_t C = (uint64_t)cb * kGroup;
  if (!grad && 256 * C > kMaxBytes) return {0, 1};
  return plan_tiles(kFp8Times, kFp8ExtraUs, G, M, O, cb, forced, 4, 96, G == 0, bytes, least_step,
                    std::max(C, 2 * (uint64_t)O));
}

// Rows of one call: the row tiles of all experts are found with 32-bit sums of 64
// sizes. The kernels take their buffers' extents tile by tile, so that the arrays
// may pass 4 GiB, 256 rows of them not (nor, where there are fewer, the rows of the
// tiles that the plan takes).
constexpr int64_t kMaxRows = 1 << 24;
uint64_t tile_rows_of(int64_t M) { return (uint64_t)std::min<int64_t>(M, 256); }

w4a16_status check_fp8(bool grad, bool grouped, int32_t G, int64_t M, int64_t N, int64_t K) {
  if (G < 1 || (!grouped && G != 1)) return W4A16_ERR_SHAPE;
  if (M < 0 || N < 1 || K < 1 || M > kMaxRows || N > kMaxDim || K > kMaxDim) return W4A16_ERR_SHAPE;
  if (K % kGroup != 0 || (grad && N % kGroup != 0)) return W4A16_ERR_SHAPE;
  const uint64_t m = tile_rows_of(M), n = (uint64_t)N, k = (uint64_t)K;
  if (n * k > kMaxBytes || m * k * 2u > kMaxBytes || m * n * 2u > kMaxBytes) return W4A16_ERR_SHAPE;
  if (n * k * (uint64_t)G > (uint64_t)INT64_MAX / 2) return W4A16_ERR_SHAPE;
  return W4A16_OK;
}

// The plan with the forced choices; partial sums in *bytes.
w4a16_status make_fp8_plan(bool grad, int64_t G, int64_t M, int64_t N, int64_t K, int32_t bm, int32_t sk, RowsPlan* p,
                           uint64_t* bytes) {
  const int64_t O = grad ? K : N, cb = (grad ? N : K) / kGroup;
  if (bm != 0) {
    bool built = bm == 16 && fp8_rows_built(grad, G, M, O, cb);
    for (const TileTime& c : kFp8Times) built = built || c.bm == bm;
    if (!built) return W4A16_ERR_SHAPE;
  }
  *p = fp8_plan(grad, G, M, O, cb, bm);
  if (p->bm == 0) return W4A16_ERR_SHAPE;
  if (sk != 0) {
    if (sk < 1 || sk > 16 || (sk > 1 && (G > 0 || p->bm == 16))) return W4A16_ERR_SPLIT_K;
    p->sk = sk;
  }
  *bytes = p->sk > 1 ? (uint64_t)p->sk * (uint64_t)M * (uint64_t)O * 4u : 0u;
  return *bytes > kMaxBytes ? W4A16_ERR_SHAPE : W4A16_OK;
}

size_t fp8_workspace_bytes(bool grad, int64_t M, int64_t N, int64_t K, int32_t bm, int32_t sk) {
  RowsPlan p;
  uint64_t bytes = 0;
  if (check_fp8(grad, false, 1, M, N, K) != W4A16_OK || M == 0) return 0;
  if (make_fp8_plan(grad, 0, M, N, K, bm, sk, &p, &bytes) != W4A16_OK) return 0;
  return (size_t)round_up(bytes, 256);
}

w4a16_status run_fp8(bool grad, const uint8_t* x, const float* xs, const uint8_t* w, const float* ws,
                     const int32_t* m_sizes, uint16_t* y, int32_t G, int64_t M, int64_t N, int64_t K, int32_t bm,
                     int32_t sk, float* workspace, size_t workspace_bytes, void* stream) {
  RowsPlan p;
  uint64_t bytes = 0;
  w4a16_status st = check_fp8(grad, m_sizes != nullptr, G, M, N, K);
  if (st != W4A16_OK || M == 0) return st;
  if (x == nullptr || xs == nullptr || w == nullptr || ws == nullptr || y == nullptr) return W4A16_ERR_NULL;
  if (!aligned16(x) || !aligned16(w) || !aligned16(y) || !aligned4(xs) || !aligned4(ws) || !aligned4(m_sizes))
    return W4A16_ERR_ALIGN;
  st = make_fp8_plan(grad, m_sizes != nullptr ? G : 0, M, N, K, bm, sk, &p, &bytes);
  if (st != W4A16_OK) return st;
  if (bytes > 0) {
    if (workspace == nullptr || workspace_bytes < bytes) return W4A16_ERR_WORKSPACE;
    if (!aligned16(workspace)) return W4A16_ERR_ALIGN;
  }
  const int64_t O = grad ? K : N, cb = (grad ? N : K) / kGroup;
  hipStream_t strm = reinterpret_cast<hipStream_t>(stream);
  const hipError_t e =
      w4a16::launch_fp8_gemm(x, xs, w, ws, y, p.sk > 1 ? workspace : nullptr, m_sizes, (int)M, (int)N, (int)K, G,
                             grad, (int)ceil_div(cb, p.sk), p.sk, p.bm, device_cus(), strm);
  if (e != hipSuccess || p.sk == 1) return launched(e);
  return launched(w4a16::launch_splitk_reduce(workspace, y, (uint64_t)M * (uint64_t)O, p.sk, strm));
}

// ---- input gradient of the 4-bit products
// One stage of 64 n by height, as for the 8-bit tiles (at 8192^3: 256 rows 1.77
// us, 224 rows 1.40, 192 rows 1.24, 128 rows 0.88, 64 rows 0.56; below that each
// stage's chain of LDS reads and its barrier).
constexpr TileTime kW4GradTimes[] = {{256, 1.75}, {224, 1.42}, {192, 1.22}, {160, 1.05}, {128, 0.86},
                                     {96, 0.70},  {64, 0.55},  {32, 0.50},  {16, 0.46}};
constexpr double kW4GradExtraUs = 6.0;

w4a16_status check_w4_grad(bool grouped, int32_t G, int64_t M, int64_t N, int64_t K, int32_t group_size) {
  if (G < 1 || (!grouped && G != 1)) return W4A16_ERR_SHAPE;
  if (M < 0 || N < 1 || K < 1 || M > kMaxRows || N > kMaxDim || K > kMaxDim) return W4A16_ERR_SHAPE;
  if ((group_size != kGroup && group_size != kGroupSmall) || K % kGroup != 0) return W4A16_ERR_GROUP_SIZE;
  if (N % 8 != 0 || (uint64_t)N * (uint64_t)K / 2u > kMaxBytes) return W4A16_ERR_SHAPE;
  const uint64_t np = (uint64_t)w4a16::w4_grad_padded(N), m = tile_rows_of(M);
  if (m * np * 2u > kMaxBytes || m * (uint64_t)K * 2u > kMaxBytes) return W4A16_ERR_SHAPE;
  if (np * (uint64_t)(K / group_size) * 2u > kMaxBytes) return W4A16_ERR_SHAPE;
  if ((uint64_t)N * (uint64_t)K / 2u * (uint64_t)G > (uint64_t)INT64_MAX / 2) return W4A16_ERR_SHAPE;
  return W4A16_OK;
}

w4a16_status make_w4_grad_plan(int32_t G, int64_t M, int64_t N, int64_t K, int32_t group_size, int32_t bm, int32_t sk,
                               w4a16::W4GradPlan* p) {
  const uint64_t np = (uint64_t)w4a16::w4_grad_padded(N), kg = (uint64_t)(K / group_size);
  if (bm != 0) {
    bool built = false;
    for (const TileTime& c : kW4GradTimes) built = built || c.bm == bm;
    if (!built) return W4A16_ERR_SHAPE;
  }
  const RowsPlan r =
      plan_tiles(kW4GradTimes, kW4GradExtraUs, G > 1 ? G : 0, M, K, (int64_t)np / 64, bm, 8, 0, true,
                 G > 1 ? 0.0 : 0.5 * (double)N * (double)K, 0.0, 2 * std::max(np, (uint64_t)K));
  if (r.bm == 0 || w4a16::w4_grad_prep_blocks(G, M, (int)N, (int)kg) > w4a16::kMaxBlocks) return W4A16_ERR_SHAPE;
  p->bm = r.bm;
  p->sk = r.sk;
  if (sk != 0) {
    if (sk < 1 || sk > 16) return W4A16_ERR_SPLIT_K;
    p->sk = sk;
  }
  p->h = 0;
  p->up = round_up((uint64_t)M * np * 2u, 256);
  p->st = p->up + round_up((uint64_t)M * 4u, 256);
  p->tops = p->st + round_up((uint64_t)G * kg * np * 2u, 256);
  p->part = p->tops + round_up((uint64_t)G * (np / 128) * kg * 2u, 256);
  const uint64_t part = p->sk > 1 ? (uint64_t)p->sk * (uint64_t)M * (uint64_t)K * 4u : 0u;
  p->bytes = p->part + round_up(part, 256);
  return part > kMaxBytes ? W4A16_ERR_SHAPE : W4A16_OK;
}

w4a16_status run_w4_grad(const uint16_t* dy, const uint8_t* w, const uint16_t* s, const int32_t* m_sizes, uint16_t* dx,
                         int32_t G, int64_t M, int64_t N, int64_t K, int32_t group_size, int32_t bm, int32_t sk,
                         void* workspace, size_t workspace_bytes, void* stream) {
  w4a16::W4GradPlan p;
  w4a16_status st = check_w4_grad(m_sizes != nullptr, G, M, N, K, group_size);
  if (st != W4A16_OK || M == 0) return st;
  if (dy == nullptr || w == nullptr || s == nullptr || dx == nullptr) return W4A16_ERR_NULL;
  if (!aligned16(dy) || !aligned16(w) || !aligned16(s) || !aligned16(dx) || !aligned4(m_sizes)) return W4A16_ERR_ALIGN;
  st = make_w4_grad_plan(G, M, N, K, group_size, bm, sk, &p);
  if (st != W4A16_OK) return st;
  if (workspace == nullptr || workspace_bytes < p.bytes) return W4A16_ERR_WORKSPACE;
  if (!aligned16(workspace)) return W4A16_ERR_ALIGN;
  return launched(w4a16::launch_w4_grad(dy, w, s, dx, m_sizes, (int)M, (int)N, (int)K, G, group_size, p,
                                        reinterpret_cast<uint8_t*>(workspace), reinterpret_cast<hipStream_t>(stream)));
}

}  // namespace

extern "C" {

const char* w4a16_status_string(int status) {
  switch (status) {
    case W4A16_OK: return "W4A16_OK";
    case W4A16_ERR_NULL: return "W4A16_ERR_NULL: a required pointer is NULL";
    case W4A16_ERR_SHAPE: return "W4A16_ERR_SHAPE: invalid dimension or size limit exceeded";
    case W4A16_ERR_GROUP_SIZE:
      return "W4A16_ERR_GROUP_SIZE: group_size must be 128 or 32 (32: tile path only) and K a multiple of 128";
    case W4A16_ERR_SPLIT_K: return "W4A16_ERR_SPLIT_K: split_k must be 0, 1, 2, 4, 8 or 16";
    case W4A16_ERR_WORKSPACE: return "W4A16_ERR_WORKSPACE: workspace missing or too small";
    case W4A16_ERR_ALIGN: return "W4A16_ERR_ALIGN: pointers must be 16-byte aligned";
    case W4A16_ERR_LAUNCH: return "W4A16_ERR_LAUNCH: kernel launch failed";
    default: return "W4A16: unknown status";
  }
}

w4a16_status w4a16_pack_int4(const uint8_t* q, uint8_t* w_packed, int64_t rows, int64_t K, void* stream) {
  if (rows < 0 || K < 2 || K % 2 != 0) return W4A16_ERR_SHAPE;
  if (q == nullptr || w_packed == nullptr) return W4A16_ERR_NULL;
  if (!aligned16(q) || !aligned16(w_packed)) return W4A16_ERR_ALIGN;
  if (rows == 0) return W4A16_OK;
  if ((uint64_t)rows > (uint64_t)INT64_MAX / (uint64_t)K) return W4A16_ERR_SHAPE;
  return launched(
      w4a16::launch_pack_int4(q, w_packed, (uint64_t)rows * (uint64_t)K, reinterpret_cast<hipStream_t>(stream)));
}

int32_t w4a16_gemm_auto_split_k(int64_t M, int64_t N, int64_t K, int32_t group_size) {
  if (check_dims(M, N, K, group_size) != W4A16_OK || M == 0) return 0;
  Plan p;
  if (make_plan(M, N, K, 0, nullptr, group_size, &p) != W4A16_OK) return 0;
  return p.sk;
}

w4a16_status w4a16_gemm_auto_config(int64_t M, int64_t N, int64_t K, int32_t group_size, w4a16_config* cfg_out,
                                    int32_t* split_k_out) {
  if (cfg_out == nullptr || split_k_out == nullptr) return W4A16_ERR_NULL;
  cfg_out->path = 0;
  cfg_out->variant = -1;
  *split_k_out = 0;
  const w4a16_status st = check_dims(M, N, K, group_size);
  if (st != W4A16_OK || M == 0) return st;
  Plan p;
  const w4a16_status sp = make_plan(M, N, K, 0, nullptr, group_size, &p);
  if (sp != W4A16_OK) return sp;
  cfg_out->path = (int32_t)p.path;
  cfg_out->variant = p.variant;
  *split_k_out = p.sk;
  return W4A16_OK;
}

size_t w4a16_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K, int32_t split_k) {
  return gemm_workspace_bytes(M, N, K, kGroup, split_k, nullptr);
}

size_t w4a16_gemm_workspace_bytes_gs(int64_t M, int64_t N, int64_t K, int32_t group_size, int32_t split_k) {
  return gemm_workspace_bytes(M, N, K, group_size, split_k, nullptr);
}

size_t w4a16_gemm_workspace_bytes_ex(int64_t M, int64_t N, int64_t K, int32_t group_size, int32_t split_k,
                                     const w4a16_config* cfg) {
  return gemm_workspace_bytes(M, N, K, group_size, split_k, cfg);
}

w4a16_status w4a16_gemm(const uint16_t* x, const uint8_t* w_packed, const uint16_t* scales, uint16_t* y, int64_t M,
                        int64_t N, int64_t K, int32_t group_size, int32_t split_k, float* workspace,
                        size_t workspace_bytes, void* stream) {
  return run_gemm(x, w_packed, scales, y, M, N, K, group_size, split_k, workspace, workspace_bytes, stream, nullptr);
}

w4a16_status w4a16_gemm_noalloc(const uint16_t* x, const uint8_t* w_packed, const uint16_t* scales, uint16_t* y,
                                int64_t M, int64_t N, int64_t K, int32_t group_size, int32_t split_k, void* stream) {
  Plan p;
  bool empty = false;
  w4a16_status st = plan_gemm(x, w_packed, scales, y, M, N, K, group_size, split_k, nullptr, &p, &empty);
  if (st != W4A16_OK || empty) return st;
  // the partials must fit the scratch; the row sums only where they fit too
  // (otherwise the tile kernel forms them), as with a caller's workspace
  if (round_up(p.ws_split, 256) > kScratchBytes) return W4A16_ERR_WORKSPACE;
  float* ws = nullptr;
  if (p.ws_split > 0 || p.ws_sx > 0) {
    ws = reinterpret_cast<float*>(scratch_ptr());
    if (ws == nullptr) return W4A16_ERR_LAUNCH;
  }
  float* rowsums = nullptr;
  if (p.ws_sx > 0 && plan_bytes(p) <= kScratchBytes)
    rowsums = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(ws) + round_up(p.ws_split, 256));
  return launch_plan(p, x, w_packed, scales, y, M, N, K, group_size, ws, rowsums,
                     reinterpret_cast<hipStream_t>(stream));
}

w4a16_status w4a16_gemm_ex(const uint16_t* x, const uint8_t* w_packed, const uint16_t* scales, uint16_t* y,
                           int64_t M, int64_t N, int64_t K, int32_t group_size, int32_t split_k, float* workspace,
                           size_t workspace_bytes, void* stream, const w4a16_config* cfg) {
  return run_gemm(x, w_packed, scales, y, M, N, K, group_size, split_k, workspace, workspace_bytes, stream, cfg);
}

w4a16_status w4a16_gemm_grouped(const uint16_t* x, const uint8_t* w_packed, const uint16_t* scales,
                                const int32_t* m_sizes, uint16_t* y, int32_t G, int64_t M_total, int64_t N, int64_t K,
                                int32_t group_size, void* stream) {
  return w4a16_gemm_grouped_ex(x, w_packed, scales, m_sizes, y, G, M_total, N, K, group_size, stream, nullptr);
}

w4a16_status w4a16_gemm_grouped_ex(const uint16_t* x, const uint8_t* w_packed, const uint16_t* scales,
                                   const int32_t* m_sizes, uint16_t* y, int32_t G, int64_t M_total, int64_t N,
                                   int64_t K, int32_t group_size, void* stream, const w4a16_config* cfg) {
  if (G < 1 || M_total < 0) return W4A16_ERR_SHAPE;
  w4a16_status st = check_dims(M_total, N, K, group_size);
  if (st != W4A16_OK) return st;
  if ((uint64_t)N * (uint64_t)K / 2u * (uint64_t)G > (uint64_t)INT64_MAX / 2) return W4A16_ERR_SHAPE;
  // one buffer resource covers the scales of all groups
  if ((uint64_t)G * (uint64_t)N * (uint64_t)(K / group_size) * 2u > kMaxBytes) return W4A16_ERR_SHAPE;
  if (M_total == 0) return W4A16_OK;   // empty problem: nothing to read or write
  if (x == nullptr || w_packed == nullptr || scales == nullptr || m_sizes == nullptr || y == nullptr)
    return W4A16_ERR_NULL;
  if (!aligned16(x) || !aligned16(w_packed) || !aligned16(scales) || !aligned16(y)) return W4A16_ERR_ALIGN;
  if (((uintptr_t)m_sizes & 3u) != 0) return W4A16_ERR_ALIGN;
  int bm = -1;
  if (cfg != nullptr) {
    if (cfg->path != 0 && cfg->path != kPathTile) return W4A16_ERR_SHAPE;
    bm = cfg->variant;
  }
  if (bm <= 0) bm = default_grouped_tile_rows(G, M_total, N, K, group_size);
  if (!w4a16::tile_rows_ok(bm, kGroup) && !w4a16::tile_rows_ok(bm, kGroupSmall)) return W4A16_ERR_SHAPE;
  if (!w4a16::tile_rows_ok(bm, group_size)) return W4A16_ERR_GROUP_SIZE;
  const int Gk = (int)(K / kGroup);
  // row sums formed in the kernel: the call takes no workspace
  return launched(w4a16::launch_tile(x, w_packed, scales, nullptr, 0, y, nullptr, m_sizes, 0, (int)M_total, (int)N,
                                     (int)K, G, Gk, 1, bm, group_size, reinterpret_cast<hipStream_t>(stream)));
}

size_t w4a16_gemm_batched_workspace_bytes(int32_t B, int64_t M, int64_t N, int64_t K, int32_t group_size,
                                          int32_t split_k) {
  return batched_workspace_bytes(B, M, N, K, group_size, split_k, nullptr);
}

size_t w4a16_gemm_batched_workspace_bytes_ex(int32_t B, int64_t M, int64_t N, int64_t K, int32_t group_size,
                                             int32_t split_k, const w4a16_config* cfg) {
  return batched_workspace_bytes(B, M, N, K, group_size, split_k, cfg);
}

w4a16_status w4a16_gemm_batched_ex(const uint16_t* x, const uint8_t* w_packed, const uint16_t* scales, uint16_t* y,
                                   int32_t B, int64_t M, int64_t N, int64_t K, int32_t group_size, int32_t split_k,
                                   float* workspace, size_t workspace_bytes, void* stream, const w4a16_config* cfg) {
  if (!valid_split(split_k)) return W4A16_ERR_SPLIT_K;
  w4a16_status st = check_batched(B, M, N, K, group_size);
  if (st != W4A16_OK) return st;
  if (M == 0) return W4A16_OK;   // empty problems: nothing to read or write
  if (x == nullptr || w_packed == nullptr || scales == nullptr || y == nullptr) return W4A16_ERR_NULL;
  if (!aligned16(x) || !aligned16(w_packed) || !aligned16(scales) || !aligned16(y)) return W4A16_ERR_ALIGN;
  BatchedPlan p;
  st = make_batched_plan(B, M, N, K, split_k, cfg, group_size, &p);
  if (st != W4A16_OK) return st;
  if (p.ws_split > kMaxBytes) return W4A16_ERR_SHAPE;
  if (p.ws_split > 0) {
    if (workspace == nullptr) return W4A16_ERR_WORKSPACE;
    if (!aligned16(workspace)) return W4A16_ERR_ALIGN;
    if (workspace_bytes < round_up(p.ws_split, 256)) return W4A16_ERR_WORKSPACE;
  }
  hipStream_t strm = reinterpret_cast<hipStream_t>(stream);
  float* ws_split = p.sk > 1 ? workspace : nullptr;
  const int Mt = (int)((int64_t)B * M);
  const int ld = (int)round_up((uint64_t)Mt, 4);
  float* rowsums = nullptr;
  if (p.ws_sx > 0 && workspace != nullptr && aligned16(workspace) &&
      workspace_bytes >= round_up(p.ws_split, 256) + p.ws_sx)
    rowsums = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(workspace) + round_up(p.ws_split, 256));
  hipError_t e = hipSuccess;
  if (rowsums != nullptr) e = w4a16::launch_rowsum_neg136(x, rowsums, Mt, (int)K, ld, group_size, strm);
  if (e == hipSuccess)
    e = w4a16::launch_tile(x, w_packed, scales, rowsums, ld, y, ws_split, nullptr, (int)M, Mt, (int)N, (int)K, B,
                           p.gps, p.sk, p.bm, group_size, strm);
  if (e != hipSuccess) return W4A16_ERR_LAUNCH;
  if (p.sk > 1) return launched(w4a16::launch_splitk_reduce(ws_split, y, (uint64_t)Mt * (uint64_t)N, p.sk, strm));
  return W4A16_OK;
}

w4a16_status w4a16_gemm_batched(const uint16_t* x, const uint8_t* w_packed, const uint16_t* scales, uint16_t* y,
                                int32_t B, int64_t M, int64_t N, int64_t K, int32_t group_size, int32_t split_k,
                                float* workspace, size_t workspace_bytes, void* stream) {
  return w4a16_gemm_batched_ex(x, w_packed, scales, y, B, M, N, K, group_size, split_k, workspace, workspace_bytes,
                               stream, nullptr);
}

w4a16_status w4a16_splitk_reduce(const float* workspace, uint16_t* y, int32_t split_k, int64_t M, int64_t N,
                                 void* stream) {
  if (split_k < 1 || split_k > 64 || M < 0 || N < 0) return W4A16_ERR_SHAPE;
  if (M == 0 || N == 0) return W4A16_OK;
  if (workspace == nullptr || y == nullptr) return W4A16_ERR_NULL;
  if (!aligned16(workspace) || !aligned16(y)) return W4A16_ERR_ALIGN;
  if ((uint64_t)M > (uint64_t)INT64_MAX / (uint64_t)N / 64u) return W4A16_ERR_SHAPE;
  return launched(w4a16::launch_splitk_reduce(workspace, y, (uint64_t)M * (uint64_t)N, split_k,
                                              reinterpret_cast<hipStream_t>(stream)));
}

size_t w4a16_gemm_lora_workspace_bytes(int64_t M, int64_t N, int64_t K, int32_t group_size, int32_t L, int32_t R,
                                       int32_t split_k) {
  LoraPlan p;
  if (make_lora_plan(M, N, K, group_size, L, R, split_k, &p) != W4A16_OK || M == 0) return 0;
  return (size_t)lora_bytes(p);
}

w4a16_status w4a16_gemm_lora(const uint16_t* x, const uint8_t* w_packed, const uint16_t* scales, const uint16_t* a,
                             const uint16_t* b, const int32_t* adapter_ids, const float* scaling, uint16_t* y,
                             int64_t M, int64_t N, int64_t K, int32_t group_size, int32_t L, int32_t R,
                             int32_t split_k, float* workspace, size_t workspace_bytes, void* stream) {
  LoraPlan p;
  const w4a16_status st = make_lora_plan(M, N, K, group_size, L, R, split_k, &p);
  if (st != W4A16_OK || M == 0) return st;
  if (x == nullptr || w_packed == nullptr || scales == nullptr || a == nullptr || b == nullptr ||
      adapter_ids == nullptr || y == nullptr)
    return W4A16_ERR_NULL;
  if (!aligned16(x) || !aligned16(w_packed) || !aligned16(scales) || !aligned16(a) || !aligned16(b) || !aligned16(y))
    return W4A16_ERR_ALIGN;
  if (!aligned4(adapter_ids) || !aligned4(scaling)) return W4A16_ERR_ALIGN;
  if (workspace == nullptr || workspace_bytes < lora_bytes(p)) return W4A16_ERR_WORKSPACE;
  if (!aligned16(workspace)) return W4A16_ERR_ALIGN;
  hipStream_t strm = reinterpret_cast<hipStream_t>(stream);
  uint8_t* ws = reinterpret_cast<uint8_t*>(workspace);
  float* partials = reinterpret_cast<float*>(ws + p.ws_h);
  float* rowsums =
      p.base.ws_sx > 0 ? reinterpret_cast<float*>(ws + p.ws_h + round_up(p.base.ws_split, 256)) : nullptr;
  uint16_t* h = reinterpret_cast<uint16_t*>(ws);
  const hipError_t e = w4a16::launch_lora_shrink(x, a, adapter_ids, scaling, h, (int)M, (int)K, L, R,
                                                 rowsums, (int)round_up((uint64_t)M, 4), group_size, strm);
  if (e != hipSuccess) return W4A16_ERR_LAUNCH;
  const w4a16::LoraArgs la = {h, b, adapter_ids, (int)M, (int)N, L, R};
  return launch_plan(p.base, x, w_packed, scales, y, M, N, K, group_size, partials, rowsums, strm, &la);
}

size_t w4a16_expert_sort_workspace_bytes(int64_t T, int32_t k, int32_t G) {
  if (!expert_slots_ok(T, k) || G < 1 || G > w4a16::kExpertMaxGroups || T == 0) return 0;
  return (size_t)expert_sort_bytes(T, k, G);
}

w4a16_status w4a16_expert_sort(const int32_t* ids, int32_t* order, int32_t* pos, int32_t* m_sizes, int64_t T,
                               int32_t k, int32_t G, void* workspace, size_t workspace_bytes, void* stream) {
  if (!expert_slots_ok(T, k) || G < 1 || G > w4a16::kExpertMaxGroups) return W4A16_ERR_SHAPE;
  if (m_sizes == nullptr) return W4A16_ERR_NULL;
  if (T > 0 && (ids == nullptr || order == nullptr || pos == nullptr)) return W4A16_ERR_NULL;
  if (!aligned4(ids) || !aligned4(order) || !aligned4(pos) || !aligned4(m_sizes)) return W4A16_ERR_ALIGN;
  if (T > 0 && expert_sort_bytes(T, k, G) > 0) {
    if (workspace == nullptr || workspace_bytes < expert_sort_bytes(T, k, G)) return W4A16_ERR_WORKSPACE;
    if (!aligned16(workspace)) return W4A16_ERR_ALIGN;
  }
  return launched(w4a16::launch_expert_sort(ids, order, pos, m_sizes, T * k, G, reinterpret_cast<int32_t*>(workspace),
                                            reinterpret_cast<hipStream_t>(stream)));
}

w4a16_status w4a16_expert_gather(const uint16_t* x, const int32_t* pos, uint16_t* xs, int64_t T, int32_t k,
                                 int64_t rows, int64_t width, void* stream) {
  bool empty = false;
  const w4a16_status st = check_expert_rows(T, k, rows, width, pos, &empty);
  if (st != W4A16_OK || empty || rows == 0) return st;
  if (x == nullptr || xs == nullptr) return W4A16_ERR_NULL;
  if (!aligned16(x) || !aligned16(xs)) return W4A16_ERR_ALIGN;
  return launched(w4a16::launch_expert_gather(x, pos, xs, T, k, rows, (int)width,
                                              reinterpret_cast<hipStream_t>(stream)));
}

w4a16_status w4a16_expert_gather_grad(const uint16_t* dxs, const int32_t* pos, uint16_t* dx, int64_t T, int32_t k,
                                      int64_t rows, int64_t width, void* stream) {
  return run_expert_combine(dxs, pos, nullptr, dx, T, k, rows, width, stream);
}

w4a16_status w4a16_expert_combine(const uint16_t* z, const int32_t* pos, const float* weights, uint16_t* y, int64_t T,
                                  int32_t k, int64_t rows, int64_t width, void* stream) {
  return run_expert_combine(z, pos, weights, y, T, k, rows, width, stream);
}

w4a16_status w4a16_expert_combine_grad(const uint16_t* dy, const uint16_t* z, const int32_t* pos,
                                       const float* weights, uint16_t* dz, float* dweights, int64_t T, int32_t k,
                                       int64_t rows, int64_t width, void* stream) {
  bool empty = false;
  const w4a16_status st = check_expert_rows(T, k, rows, width, pos, &empty);
  if (st != W4A16_OK || empty) return st;
  if (dy == nullptr || weights == nullptr || dweights == nullptr) return W4A16_ERR_NULL;
  if (rows > 0 && (z == nullptr || dz == nullptr)) return W4A16_ERR_NULL;
  if (!aligned16(dy) || !aligned16(z) || !aligned16(dz) || !aligned4(weights) || !aligned4(dweights))
    return W4A16_ERR_ALIGN;
  return launched(w4a16::launch_expert_combine_grad(dy, z, pos, weights, dz, dweights, T, k, rows, (int)width,
                                                    reinterpret_cast<hipStream_t>(stream)));
}

w4a16_status w4a16_fp8_quantize(const uint16_t* x, uint8_t* q, float* scales, int64_t M, int64_t K,
                                int32_t block_rows, void* stream) {
  if (M < 0 || K < 1 || M > kMaxDim || K > kMaxDim || K % kGroup != 0) return W4A16_ERR_SHAPE;
  if (block_rows != 1 && block_rows != kGroup) return W4A16_ERR_SHAPE;
  if ((uint64_t)M * (uint64_t)K >= (uint64_t{1} << 37)) return W4A16_ERR_SHAPE;
  if (M == 0) return W4A16_OK;
  if (x == nullptr || q == nullptr || scales == nullptr) return W4A16_ERR_NULL;
  if (!aligned16(x) || !aligned16(q) || !aligned4(scales)) return W4A16_ERR_ALIGN;
  return launched(
      w4a16::launch_fp8_quantize(x, q, scales, M, (int)K, block_rows, reinterpret_cast<hipStream_t>(stream)));
}

size_t w4a16_fp8_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  return fp8_workspace_bytes(false, M, N, K, 0, 0);
}

size_t w4a16_fp8_gemm_grad_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  return fp8_workspace_bytes(true, M, N, K, 0, 0);
}

size_t w4a16_fp8_gemm_workspace_bytes_ex(int32_t grad, int64_t M, int64_t N, int64_t K, int32_t bm, int32_t sk) {
  return fp8_workspace_bytes(grad != 0, M, N, K, bm, sk);
}

w4a16_status w4a16_fp8_gemm(const uint8_t* x, const float* x_scales, const uint8_t* w, const float* w_scales,
                            uint16_t* y, int64_t M, int64_t N, int64_t K, float* workspace, size_t workspace_bytes,
                            void* stream) {
  return run_fp8(false, x, x_scales, w, w_scales, nullptr, y, 1, M, N, K, 0, 0, workspace, workspace_bytes, stream);
}

w4a16_status w4a16_fp8_gemm_grouped(const uint8_t* x, const float* x_scales, const uint8_t* w, const float* w_scales,
                                    const int32_t* m_sizes, uint16_t* y, int32_t G, int64_t M_total, int64_t N,
                                    int64_t K, void* stream) {
  const w4a16_status st = check_fp8(false, true, G, M_total, N, K);
  if (st != W4A16_OK || M_total == 0) return st;
  if (m_sizes == nullptr) return W4A16_ERR_NULL;
  return run_fp8(false, x, x_scales, w, w_scales, m_sizes, y, G, M_total, N, K, 0, 0, nullptr, 0, stream);
}

w4a16_status w4a16_fp8_gemm_grad(const uint8_t* dy, const float* dy_scales, const uint8_t* w, const float* w_scales,
                                 const int32_t* m_sizes, uint16_t* dx, int32_t G, int64_t M, int64_t N, int64_t K,
                                 float* workspace, size_t workspace_bytes, void* stream) {
  return run_fp8(true, dy, dy_scales, w, w_scales, m_sizes, dx, G, M, N, K, 0, 0, workspace, workspace_bytes, stream);
}

w4a16_status w4a16_fp8_gemm_ex(int32_t grad, const uint8_t* x, const float* x_scales, const uint8_t* w,
                               const float* w_scales, const int32_t* m_sizes, uint16_t* y, int32_t G, int64_t M,
                               int64_t N, int64_t K, int32_t bm, int32_t sk, float* workspace,
                               size_t workspace_bytes, void* stream) {
  return run_fp8(grad != 0, x, x_scales, w, w_scales, m_sizes, y, G, M, N, K, bm, sk, workspace, workspace_bytes,
                 stream);
}

w4a16_status w4a16_fp8_gemm_auto(int32_t grad, int32_t grouped, int32_t G, int64_t M, int64_t N, int64_t K,
                                 int32_t* bm_out, int32_t* sk_out) {
  if (bm_out == nullptr || sk_out == nullptr) return W4A16_ERR_NULL;
  const w4a16_status st = check_fp8(grad != 0, grouped != 0, G, M, N, K);
  if (st != W4A16_OK) return st;
  RowsPlan p;
  uint64_t bytes = 0;
  const w4a16_status sp = make_fp8_plan(grad != 0, grouped != 0 ? G : 0, M, N, K, 0, 0, &p, &bytes);
  *bm_out = p.bm;
  *sk_out = p.sk;
  return sp;
}

size_t w4a16_gemm_grad_workspace_bytes_ex(int32_t G, int64_t M, int64_t N, int64_t K, int32_t group_size, int32_t bm,
                                          int32_t sk) {
  w4a16::W4GradPlan p;
  if (check_w4_grad(true, G, M, N, K, group_size) != W4A16_OK || M == 0) return 0;
  if (make_w4_grad_plan(G, M, N, K, group_size, bm, sk, &p) != W4A16_OK) return 0;
  return (size_t)p.bytes;
}

size_t w4a16_gemm_grad_workspace_bytes(int32_t G, int64_t M, int64_t N, int64_t K, int32_t group_size) {
  return w4a16_gemm_grad_workspace_bytes_ex(G, M, N, K, group_size, 0, 0);
}

w4a16_status w4a16_gemm_grad(const uint16_t* dy, const uint8_t* w_packed, const uint16_t* scales,
                             const int32_t* m_sizes, uint16_t* dx, int32_t G, int64_t M, int64_t N, int64_t K,
                             int32_t group_size, void* workspace, size_t workspace_bytes, void* stream) {
  return run_w4_grad(dy, w_packed, scales, m_sizes, dx, G, M, N, K, group_size, 0, 0, workspace, workspace_bytes,
                     stream);
}

w4a16_status w4a16_gemm_grad_ex(const uint16_t* dy, const uint8_t* w_packed, const uint16_t* scales,
                                const int32_t* m_sizes, uint16_t* dx, int32_t G, int64_t M, int64_t N, int64_t K,
                                int32_t group_size, int32_t bm, int32_t sk, void* workspace, size_t workspace_bytes,
                                void* stream) {
  return run_w4_grad(dy, w_packed, scales, m_sizes, dx, G, M, N, K, group_size, bm, sk, workspace, workspace_bytes,
                     stream);
}

w4a16_status w4a16_gemm_grad_auto(int32_t grouped, int32_t G, int64_t M, int64_t N, int64_t K, int32_t group_size,
                                  int32_t* bm_out, int32_t* sk_out) {
  if (bm_out == nullptr || sk_out == nullptr) return W4A16_ERR_NULL;
  const w4a16_status st = check_w4_grad(grouped != 0, G, M, N, K, group_size);
  if (st != W4A16_OK) return st;
  w4a16::W4GradPlan p;
  const w4a16_status sp = make_w4_grad_plan(G, M, N, K, group_size, 0, 0, &p);
  if (sp != W4A16_OK) return sp;
  *bm_out = p.bm;
  *sk_out = p.sk;
  return W4A16_OK;
}

}  // extern "C"
