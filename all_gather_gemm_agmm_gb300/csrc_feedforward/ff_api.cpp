// ff_api.cpp -- the C ABI of include/agmm_feedforward.h: argument checks, plans,
// tile schedules and launches of the feed-forward operators.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <climits>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstdlib>
#include <mutex>
#include <new>

#include <cudaTypedefs.h>

#include "agmm_feedforward.h"
#include "ff_params.h"

namespace agmm {
agmm_status_t set_last_error(agmm_status_t status, const char* message);
}

using namespace agmm;
using namespace agmm::ff;

struct ProductPlan {
  int64_t k, n;
  int act;
  bool transpose, f16;  // weights stored [n, k]; fp16
  bool saved_f32;       // what the forward pass saves is float32
  int device, sms;
  int pairs;                  // CTA pairs that run at once
  int clusters[kMaxSplit + 1];  // clusters of that many CTAs that do
  int joined[kMaxPairs + 1];    // clusters of that many pairs that do
  int path, bn, cut, split, merge;  // overrides for tests and experiments; -1: by the rules
  uint64_t wait_limit_cycles;
  int test_drop;
};
struct agmm_gated_s : ProductPlan {};
struct agmm_linear_s : ProductPlan {};
struct agmm_layer_norm_s {
  int columns, device, sms;
  float eps;
  bool f16;
};

namespace {

// Row tiles that sweep the columns together: as many as hold this much of the rows' operand, 8 to
// 16 of them, which then stays in L2.  (8192 rows of 4096 values by 14336 columns: 497 us in bands
// of 8, 489 us of 16, 500 us of 24; 16384 of 7168 by 8192: 995, 1009 and 1025 us.)
constexpr int64_t kBandBytes = 34 << 20;
constexpr int64_t kMostRows = INT_MAX - 1024;  // coordinates of tiles behind the last row fit 32 bits
constexpr int64_t kMostTiles = 1 << 30;
constexpr int64_t kMostWidth = 1 << 20;
constexpr int64_t kMostStride = 1 << 29;  // the bytes of a row fit 32 bits

agmm_status_t fail(agmm_status_t s, const char* fmt, ...) {
  char text[256];
  va_list ap;
  va_start(ap, fmt);
  std::vsnprintf(text, sizeof text, fmt, ap);
  va_end(ap);
  return set_last_error(s, text);
}

#define AGMM_TRY(expr)                        \
  do {                                        \
    const agmm_status_t st_ = (expr);         \
    if (st_ != AGMM_OK) return st_;           \
  } while (0)

agmm_status_t check_cuda(cudaError_t e, const char* what) {
  return e == cudaSuccess ? AGMM_OK : fail(AGMM_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

agmm_status_t check_device(int* device, int* sms) {
  int major = 0, minor = 0;
  cudaError_t e = cudaGetDevice(device);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, *device);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, *device);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, *device);
  AGMM_TRY(check_cuda(e, "device query"));
  if (major != 10 || minor != 3)
    return fail(AGMM_ERR_UNSUPPORTED, "this library is built for sm_103a only; device is sm_%d%d", major, minor);
  return AGMM_OK;
}

agmm_status_t check_plan_device(int device) {
  int now = -1;
  AGMM_TRY(check_cuda(cudaGetDevice(&now), "cudaGetDevice"));
  if (now != device) return fail(AGMM_ERR_INVALID_ARG, "the plan belongs to device %d, the current device is %d", device, now);
  return AGMM_OK;
}

agmm_status_t check_width(const char* name, int64_t v, int64_t most) {
  if (v < 8 || v > most || v % 8)
    return fail(AGMM_ERR_INVALID_ARG, "%s must be a multiple of 8 in [8, %lld]: %lld", name, (long long)most, (long long)v);
  return AGMM_OK;
}

agmm_status_t check_dtype(int dtype) {
  if (dtype != AGMM_BF16 && dtype != AGMM_F16)
    return fail(AGMM_ERR_INVALID_ARG, "dtype must be AGMM_BF16 or AGMM_F16: %d", dtype);
  return AGMM_OK;
}

agmm_status_t check_pointer(const char* name, const void* p, size_t align) {
  if (!p) return fail(AGMM_ERR_INVALID_ARG, "%s is NULL", name);
  if (reinterpret_cast<uintptr_t>(p) % align) return fail(AGMM_ERR_ALIGNMENT, "%s is not %zu-byte aligned", name, align);
  return AGMM_OK;
}

// A matrix: there, 16-byte aligned, its rows whole and a multiple of 16 bytes apart.
// One row has no stride to speak of.
agmm_status_t check_matrix(const char* name, const void* p, int64_t* stride, int64_t rows, int64_t cols) {
  AGMM_TRY(check_pointer(name, p, 16));
  if (rows <= 1) {
    *stride = cols;
    return AGMM_OK;
  }
  if (*stride < cols || *stride > kMostStride)
    return fail(AGMM_ERR_INVALID_ARG, "%s: the row stride (%lld) must be at least the row's %lld values, and at most 2^29", name,
                (long long)*stride, (long long)cols);
  if (*stride % 8) return fail(AGMM_ERR_ALIGNMENT, "%s: the row stride (%lld) must be a multiple of 8", name, (long long)*stride);
  return AGMM_OK;
}

// Whether two 16-bit matrices of as many rows may share memory: their ranges meet.
bool may_overlap(const void* a, int64_t a_stride, const void* b, int64_t b_stride, int64_t rows) {
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
  return a0 < b0 + (uintptr_t)(rows * b_stride * 2) && b0 < a0 + (uintptr_t)(rows * a_stride * 2);
}

// The device's peak clock.  Asked once per device: CUDA takes most of a
// millisecond to answer.
int peak_clock_khz(int device) {
  static std::atomic<int> known[64];
  const bool cached = device >= 0 && device < 64;
  int khz = cached ? known[device].load(std::memory_order_relaxed) : 0;
  if (khz > 0) return khz;
  if (cudaDeviceGetAttribute(&khz, cudaDevAttrClockRate, device) != cudaSuccess || khz <= 0) {
    (void)cudaGetLastError();
    khz = 2100000;  // above the part's 2.07 GHz peak
  }
  if (cached) known[device].store(khz, std::memory_order_relaxed);
  return khz;
}

// ------------------------------------------------------------------ workspace
// status words, counters of cut tiles | partial results.  Fewer than two tiles to a cluster
// are cut, with a counter for each CTA's epilogue warps.
constexpr int kMostSms = (AGMM_FEEDFORWARD_HEAD_BYTES - kStatusBytes) / (2 * kEpiWarps * (int)sizeof(int));
size_t partial_bytes(const ProductPlan* pl) { return (size_t)pl->sms * kSlots * kSlotBytes; }
size_t workspace_bytes(const ProductPlan* pl) { return AGMM_FEEDFORWARD_HEAD_BYTES + partial_bytes(pl); }

// -------------------------------------------------------------- tensor maps
struct TensorMapCalls {
  PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
  PFN_cuTensorMapReplaceAddress_v12000 replace = nullptr;
};
const TensorMapCalls& tensor_map_calls() {
  static TensorMapCalls calls;
  static std::once_flag once;
  std::call_once(once, [] {
    const auto find = [](const char* name) {
      void* f = nullptr;
      cudaDriverEntryPointQueryResult q;
      return cudaGetDriverEntryPointByVersion(name, &f, 12000, cudaEnableDefault, &q) == cudaSuccess && q == cudaDriverEntryPointSuccess
                 ? f
                 : nullptr;
    };
    calls.encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(find("cuTensorMapEncodeTiled"));
    calls.replace = reinterpret_cast<PFN_cuTensorMapReplaceAddress_v12000>(find("cuTensorMapReplaceAddress"));
  });
  return calls;
}

// A matrix of 16-bit values: rows of `inner` values, `stride` apart, in segments.
struct Matrix {
  const char* name;
  const void* ptr;
  int64_t inner, rows, segments, stride;
};

// A matrix as an operand that is contracted along its rows' values (K-major), or along its rows
// (MN-major); a tile has tile_rows of its rows or values.  128-byte swizzled, zeros outside: what lies
// behind a segment's last row is not its neighbour's.
//
// Encoding takes half a microsecond, and a training step has ten maps: a thread keeps
// those of its latest layouts (sizes and strides, whatever the memory) and puts the address in.
agmm_status_t encode_operand(CUtensorMap* map, OperandParams* o, const Matrix& m, bool mn_major, int tile_rows, bool f16) {
  const TensorMapCalls& calls = tensor_map_calls();
  if (!calls.encode || !calls.replace) return fail(AGMM_ERR_CUDA, "tensor maps are not available from the driver");
  o->mn_major = mn_major;
  o->blocked = mn_major && m.inner % 64 == 0;
  struct Layout {
    int64_t inner, rows, segments, stride, kind;
    bool operator==(const Layout& x) const {
      return inner == x.inner && rows == x.rows && segments == x.segments && stride == x.stride && kind == x.kind;
    }
  };
  struct Known {
    Layout layout = {};
    CUtensorMap map;
  };
  constexpr int kKnown = 64;
  thread_local Known known[kKnown];
  const Layout l = {m.inner, m.rows, m.segments, m.stride, (int64_t)tile_rows * 4 + (mn_major ? 2 : 0) + (f16 ? 1 : 0)};
  const uint64_t mix = ((uint64_t)l.inner * 0x9e3779b97f4a7c15ull) ^ ((uint64_t)l.rows * 0xc2b2ae3d27d4eb4full) ^
                       ((uint64_t)l.stride * 0x165667b19e3779f9ull) ^ ((uint64_t)(l.segments * 1024 + l.kind) * 0xd6e8feb86659fd93ull);
  Known& k = known[(mix >> 32) % kKnown];
  CUresult r = CUDA_SUCCESS;
  if (!(k.layout == l)) {
    const cuuint64_t inner = (cuuint64_t)m.inner, rows = (cuuint64_t)m.rows, step = (cuuint64_t)m.stride * 2;
    const cuuint64_t blocks = o->blocked ? inner / 64 : 1;
    const cuuint64_t dims[4] = {inner / blocks, rows, blocks, (cuuint64_t)m.segments};
    const cuuint64_t strides[3] = {step, o->blocked ? 128 : step, (m.segments > 1 ? rows : 1) * step};
    const cuuint32_t box[4] = {kTileK, (cuuint32_t)(mn_major ? 64 : tile_rows), (cuuint32_t)(o->blocked ? tile_rows / 64 : 1), 1};
    const cuuint32_t one[4] = {1, 1, 1, 1};
    k.layout = {};
    r = calls.encode(&k.map, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, mn_major ? 4 : 2,
                     const_cast<void*>(m.ptr), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r == CUDA_SUCCESS) k.layout = l;
  }
  if (r == CUDA_SUCCESS) {
    *map = k.map;
    r = calls.replace(map, const_cast<void*>(m.ptr));
  }
  if (r != CUDA_SUCCESS) return fail(AGMM_ERR_CUDA, "tensor map of %s: the driver gave %d", m.name, (int)r);
  return AGMM_OK;
}

// ---------------------------------------------------------------- schedules
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// The time that a schedule takes, in cycles, as far as it differs from others: clusters that each
// work through `blocks` k blocks.  The constants were measured on this GPU, kernel by kernel.
constexpr double kWideBlock = 512, kNarrowBlock = 340;    // a k block of a row tile's main loop (narrow: 306 to 367, few and all pairs at work)
constexpr double kWideTile = 4000, kNarrowTile = 2500;    // its results, beside the next tile's main loop
constexpr double kWideCut = 16000, kNarrowCut = 6500;     // the parts' way to L2 and back
constexpr double kWidePart = 3000, kNarrowPart = 1400;    // ... and each part that is added
constexpr double kJoinTile = 3500;                        // pairs' parts in distributed shared memory
constexpr double kLaunch = 7000;                          // a launch's start and last results
constexpr double kSwapByte = 0.019;                       // swapped tiles: a byte, for one CTA alone
constexpr double kMemoryByte = 2.84e-4;                   // ... and for each CTA that shares the device's memory
constexpr double kSplitTile = 1500;                       // ... the parts' way through distributed shared memory

// Whole tiles go round the clusters; or those of a ragged last wave, with the wave before it, are
// cut along k evenly over the clusters.
int cut_tiles(int tiles, int clusters) { return tiles < clusters ? tiles : tiles % clusters ? clusters + tiles % clusters : 0; }

// `parts`: clusters that share the cut tiles (0: none is cut).
void make_schedule(GemmParams* p, int clusters, int parts) {
  const int shared = parts ? cut_tiles(p->num_tiles, clusters) : 0;
  const int64_t units = (int64_t)shared * p->k_blocks;
  p->dp_tiles = p->num_tiles - shared;
  p->sk_clusters = (int)std::min<int64_t>(parts, units);
  if (p->sk_clusters) {
    p->sk_share = (int)(units / p->sk_clusters);
    p->sk_extra = (int)(units % p->sk_clusters);
  }
}

bool can_cut(int64_t tiles, int k_blocks, int clusters) {
  const int64_t shared = cut_tiles((int)tiles, clusters);
  return shared > 0 && k_blocks > 1 && shared * k_blocks <= INT_MAX;
}

// How the tokens' rows lie in tiles: boxes of rows that never leave their shard.
void chunk_rows(Product* p, int shards, int64_t rows, int box) {
  p->shards = shards;
  p->shard_rows = rows;
  p->box = box;
  p->shard_chunks = (int)ceil_div(rows, box);
  p->chunks = p->shard_chunks * shards;
}

// Row tiles of several shards: the box that makes the fewest tiles, the largest of those.
int row_box(int shards, int64_t rows) {
  int best = 128;
  if (shards == 1) return best;
  int64_t fewest = INT64_MAX;
  for (int box = 128; box >= 8; box /= 2) {
    const int64_t tiles = ceil_div(ceil_div(rows, box) * shards, 128 / box);
    if (tiles < fewest) {
      fewest = tiles;
      best = box;
    }
  }
  return best;
}

// Swapped tiles hold all tokens: their box, or 0 where they are too many.
int swap_box(int shards, int64_t rows) {
  if (rows > kMaxSwapRows) return 0;
  const int box = (int)ceil_div(rows, 8) * 8;
  return box * shards <= kMaxSwapRows ? box : 0;
}

void common_params(const ProductPlan* pl, GemmParams* p, void* workspace) {
  char* const ws = static_cast<char*>(workspace);
  p->status = reinterpret_cast<int*>(ws);
  p->counters = reinterpret_cast<int*>(ws + kStatusBytes);
  p->partial = reinterpret_cast<float*>(ws + AGMM_FEEDFORWARD_HEAD_BYTES);
  p->wait_limit_cycles = pl->wait_limit_cycles;
  p->test_drop = pl->test_drop;
  p->f16 = pl->f16;
  p->problems = 1;
  p->seg_blocks = p->k_blocks = 1;
  p->split = 1;
}

// Cut tiles of full waves are worked on at different places of k, and no longer share what they
// load while it is in L2: their operands have to fit there, more or less.  (8192 x 4096 by 14336
// values, 352 MB of operands: 499 us whole, 562 us cut; 2048 x 8192 by 7168, 147 MB: 139 and
// 134 us; 4096 x 2560 by 5120, 68 MB: 76 and 67 us.)
constexpr int64_t kCutBytes = 160 << 20;

// Row tiles: their width, and the clusters that share cut ones (0: none is cut), by the shortest
// estimate.
struct RowChoice {
  int bn, parts, split;  // split: pairs of a cluster that share a tile
  double time;
};
RowChoice choose_rows(const ProductPlan* pl, int64_t m_tiles, int64_t cols, int k_blocks, int problems, bool gated) {
  RowChoice best = {kWideN, 0, 1, 1e300};
  const int C = pl->pairs;
  for (int bn = kWideN; bn >= kNarrowN; bn -= kWideN - kNarrowN) {
    if (pl->bn >= 0 && pl->bn != bn) continue;
    const int64_t tiles = m_tiles * ceil_div(cols, gated ? bn / 2 : bn) * problems;
    if (tiles > kMostTiles) continue;
    const bool wide = bn == kWideN;
    const double block = wide ? kWideBlock : kNarrowBlock, tile = wide ? kWideTile : kNarrowTile;
    const double cut = wide ? kWideCut : kNarrowCut, part = wide ? kWidePart : kNarrowPart;
    const auto offer = [&](double time, int parts, int split) {
      if (time < best.time) best = {bn, parts, split, time};
    };
    bool joined = false;
    if (!wide && pl->cut != 1) {
      for (int n = 2; n <= kMaxPairs && n <= k_blocks && tiles <= pl->joined[n]; ++n) {
        if (pl->split >= 1 && n != pl->split) continue;
        joined = true;
        offer(ceil_div(k_blocks, n) * block + kJoinTile, 0, n);
      }
    }
    if (joined && pl->split > 1) continue;
    const int64_t bytes = (m_tiles * 2 * kTileM + cols) * problems * k_blocks * kTileK * 2;
    const bool can = can_cut(tiles, k_blocks, C) && (tiles < C || bytes <= kCutBytes) && pl->cut != 0;
    if (!can || pl->cut != 1) offer((double)ceil_div(tiles, C) * std::max(k_blocks * block, tile), 0, 1);
    if (!can) continue;
    if (tiles > C) {
      offer(std::max(k_blocks * block, tile) * tiles / C + cut + 2 * part, C, 1);
    } else {
      // every tile in `n` parts, or all clusters at work
      for (int64_t n = 2; n * tiles <= C && n <= k_blocks; ++n) offer(ceil_div(k_blocks, n) * block + cut + n * part, (int)(n * tiles), 1);
      offer(k_blocks * block * tiles / C + cut + (double)(ceil_div(C, tiles) + 1) * part, C, 1);
    }
  }
  return best;
}

// The tiles of a product; its rows' tiles are known.
agmm_status_t lay_tiles(Product* q, int64_t m_tiles) {
  const int64_t n_tiles = ceil_div(q->cols, q->b_tile_step);
  if (m_tiles * n_tiles * q->problems > kMostTiles) return fail(AGMM_ERR_UNSUPPORTED, "more than 2^30 tiles of results");
  q->m_tiles = (int)m_tiles;
  q->n_tiles = (int)n_tiles;
  q->tiles_per_problem = q->m_tiles * q->n_tiles;
  q->group_m = (int)std::min<int64_t>(16, std::max<int64_t>(8, kBandBytes / ((int64_t)2 * kTileM * q->k_blocks * kTileK * 2)));
  return AGMM_OK;
}

agmm_status_t run_rows(const ProductPlan* pl, GemmParams* p, int epi, RowChoice choice, int64_t m_tiles, cudaStream_t stream) {
  AGMM_TRY(lay_tiles(p, m_tiles));
  p->num_tiles = p->tiles_per_problem * p->problems;
  const size_t stage = kTileBytes + choice.bn * kTileK;
  p->split = choice.split;
  // a pair owns every split-th quarter of its rows, in two halves of the columns
  p->recv_bytes = choice.split > 1 ? (uint32_t)(ceil_div(4, choice.split) * 2 * choice.split * 32 * 64 * sizeof(float)) : 0;
  const size_t rest = 1024 + (size_t)kEpiWarps * kStageOutBytes + p->recv_bytes + kCtlBytes;
  p->stages = (int)std::min<size_t>(choice.bn == kWideN ? kWideStages : kNarrowStages, (kMaxSmem - rest) / stage);
  p->tmem_cols = 2 * choice.bn;
  make_schedule(p, pl->pairs, choice.parts);
  const int clusters = choice.split > 1 ? p->num_tiles : std::min(pl->pairs, std::max(p->dp_tiles, p->sk_clusters));
  return check_cuda(launch_gemm(select_gemm(choice.bn, epi, pl->f16, pl->saved_f32 && p->saved[0]), *p, clusters, 2 * choice.split, rest + p->stages * stage, stream),
                    "product launch");
}

// Swapped tiles: the CTAs of a cluster that share a tile's k, by the shortest estimate.
struct SwapChoice {
  int split;
  double time;
};
SwapChoice choose_swap(const ProductPlan* pl, int tiles, int k_blocks, size_t stage_bytes) {
  SwapChoice best = {1, 1e300};
  for (int split = 1; split <= kMaxSplit; ++split) {
    if (split > 1 && (split > k_blocks || tiles > pl->clusters[split])) break;
    if (pl->split >= 1 && split != std::min(pl->split, k_blocks)) continue;
    const int ctas = std::min(tiles * split, pl->clusters[1]);
    const double time = (double)k_blocks / split * stage_bytes * std::max(kSwapByte, kMemoryByte * ctas) + (split > 1 ? kSplitTile : 0);
    if (time < 1.02 * best.time) best = {split, time};  // of two alike the one with more copies in flight
  }
  return best;
}

size_t swap_stage_bytes(int accs, int token_columns) { return (size_t)accs * kTileBytes + (size_t)ceil_div(token_columns, 16) * 16 * 128; }

agmm_status_t run_swap(const ProductPlan* pl, GemmParams* p, int epi, int64_t features, cudaStream_t stream) {
  p->m_tiles = (int)ceil_div(features, kTileM);
  p->n_tiles = 1;
  p->tiles_per_problem = p->num_tiles = p->m_tiles;
  p->group_m = 1;
  p->mma_n = (int)ceil_div(p->chunks * p->box, 16) * 16;
  const int accs = epi == kEpiGated ? 2 : 1, tiles = p->num_tiles, groups = (int)ceil_div(p->chunks * p->box, 8);
  const size_t stage = swap_stage_bytes(accs, p->mma_n);
  p->split = choose_swap(pl, tiles, p->k_blocks, stage).split;
  p->recv_slots = (int)ceil_div(groups, p->split);
  p->recv_bytes = p->split > 1 ? (uint32_t)(p->split * p->recv_slots * accs * kTileM * 8 * sizeof(float)) : 0;
  p->stages = (int)std::min<size_t>(kMaxStages, (kMaxSmem - 1024 - kCtlBytes - p->recv_bytes) / stage);
  p->tmem_cols = 32;
  while ((int)p->tmem_cols < 2 * accs * p->mma_n) p->tmem_cols *= 2;
  make_schedule(p, pl->clusters[1], 0);
  const int clusters = p->split > 1 ? tiles : std::min(pl->clusters[1], tiles);
  const size_t smem = 1024 + p->stages * stage + p->recv_bytes + kCtlBytes;
  return check_cuda(launch_gemm(select_gemm(0, epi, pl->f16, pl->saved_f32 && p->saved[0]), *p, clusters, p->split, smem, stream), "product launch");
}

// X Wi for one weight or two (gated), with an epilogue.
agmm_status_t forward(const ProductPlan* pl, GemmParams* p, int epi, int shards, int64_t rows, const void* const* x, int64_t x_stride,
                      const void* const* w, int64_t w_stride, cudaStream_t stream) {
  const int weights = epi == kEpiGated ? 2 : 1;
  const int swap = pl->path == 0 ? 0 : swap_box(shards, rows);
  const int box = swap ? swap : row_box(shards, rows);
  chunk_rows(p, shards, rows, box);
  p->cols = pl->n;
  p->k_blocks = p->seg_blocks = (int)ceil_div(pl->k, kTileK);
  const int64_t m_tiles = ceil_div((int64_t)p->chunks * box, 2 * kTileM);
  const RowChoice choice = choose_rows(pl, m_tiles, pl->n, p->k_blocks, 1, epi == kEpiGated);
  const int w_rows = swap ? kTileM : choice.bn / 2;  // rows of a weight in a tile
  OperandParams &xo = swap ? p->b : p->a, &wo = swap ? p->a : p->b;
  CUtensorMap *xm = swap ? p->b_map : p->a_map, *wm = swap ? p->a_map : p->b_map;
  xo.maps = shards;
  xo.by_shard = 1;
  for (int s = 0; s < shards; ++s) AGMM_TRY(encode_operand(&xm[s], &xo, {"x", x[s], pl->k, rows, 1, x_stride}, false, box, pl->f16));
  wo.maps = weights;
  for (int i = 0; i < weights; ++i) {
    const Matrix m = pl->transpose ? Matrix{"a weight", w[i], pl->k, pl->n, 1, w_stride} : Matrix{"a weight", w[i], pl->n, pl->k, 1, w_stride};
    AGMM_TRY(encode_operand(&wm[i], &wo, m, !pl->transpose, w_rows, pl->f16));
  }
  if (swap) return run_swap(pl, p, epi, pl->n, stream);
  if (epi == kEpiGated) {
    wo.by_rank = 1;
    p->b_tile_step = choice.bn / 2;
  } else {
    p->b_tile_step = choice.bn;
    p->b_half_step = choice.bn / 2;
  }
  return run_rows(pl, p, epi, choice, m_tiles, stream);
}

// Backward passes of few tokens: both gradients may share a launch of row tiles, which read small
// weights as fast as swapped tiles do, but not large ones (16 tokens, 4096 x 4096: 24.1 us in one
// launch, 21.1 us in two; 64 tokens, 2048 x 2048: 10.7 and 13.0 us).
constexpr int64_t kFewTokenBytes = 16 << 20;

// What the products of a backward pass are made of.
struct Grads {
  int weights, shards;
  int64_t rows;  // of a shard
  const void* const* x;
  int64_t x_stride;
  const void* const* d;  // of each weight's product
  int64_t d_stride;
  const void* const* w;
  int64_t w_stride;
  void* dx;  // NULL: not wanted
  int64_t dx_stride;
  void* const* dw;  // NULL: not wanted
  int64_t dw_stride;
  bool f32;
};

// dx = sum over the weights of d_i Wi^T; tiles of bn columns, or swapped with a box of `swap` tokens.
agmm_status_t input_grad(const ProductPlan* pl, Product* p, const Grads& g, int swap, int bn) {
  const int64_t tokens = g.shards * g.rows;
  chunk_rows(p, 1, tokens, swap ? swap : kTileM);
  p->problems = 1;
  p->out[0] = g.dx;
  p->ldo = g.dx_stride;
  p->cols = pl->k;
  p->seg_blocks = (int)ceil_div(pl->n, kTileK);
  p->k_blocks = g.weights * p->seg_blocks;
  p->b_tile_step = bn;
  p->b_half_step = bn / 2;
  OperandParams &to = swap ? p->b : p->a, &wo = swap ? p->a : p->b;
  CUtensorMap *tm = swap ? p->b_map : p->a_map, *wm = swap ? p->a_map : p->b_map;
  to.maps = wo.maps = g.weights;
  to.by_segment = wo.by_segment = 1;
  for (int i = 0; i < g.weights; ++i) {
    AGMM_TRY(encode_operand(&tm[i], &to, {"a gradient", g.d[i], pl->n, tokens, 1, g.d_stride}, false, p->box, pl->f16));
    const Matrix m = pl->transpose ? Matrix{"a weight", g.w[i], pl->k, pl->n, 1, g.w_stride} : Matrix{"a weight", g.w[i], pl->n, pl->k, 1, g.w_stride};
    AGMM_TRY(encode_operand(&wm[i], &wo, m, pl->transpose, swap ? kTileM : bn / 2, pl->f16));
  }
  return AGMM_OK;
}

// dWi = X^T d_i, stored like the weight; the tokens of each shard are a segment of the sum.
agmm_status_t weight_grad(const ProductPlan* pl, Product* p, const Grads& g, int bn) {
  chunk_rows(p, 1, pl->transpose ? pl->n : pl->k, kTileM);
  p->problems = g.weights;
  for (int i = 0; i < g.weights; ++i) p->out[i] = g.dw[i];
  p->ldo = g.dw_stride;
  p->out_f32 = g.f32;
  p->cols = pl->transpose ? pl->k : pl->n;
  p->seg_blocks = (int)ceil_div(g.rows, kTileK);
  p->k_blocks = p->seg_blocks * g.shards;
  p->b_tile_step = bn;
  p->b_half_step = bn / 2;
  const int x_rows = pl->transpose ? bn / 2 : kTileM, d_rows = pl->transpose ? kTileM : bn / 2;
  OperandParams &xo = pl->transpose ? p->b : p->a, &go = pl->transpose ? p->a : p->b;
  CUtensorMap *xm = pl->transpose ? p->b_map : p->a_map, *gm = pl->transpose ? p->a_map : p->b_map;
  xo.maps = g.shards;
  go.maps = g.weights;
  xo.by_segment = 1;
  go.by_problem = 1;
  go.z_segment = 1;
  for (int s = 0; s < g.shards; ++s) AGMM_TRY(encode_operand(&xm[s], &xo, {"x", g.x[s], pl->k, g.rows, 1, g.x_stride}, true, x_rows, pl->f16));
  for (int i = 0; i < g.weights; ++i)
    AGMM_TRY(encode_operand(&gm[i], &go, {"a gradient", g.d[i], pl->n, g.rows, g.shards, g.d_stride}, true, d_rows, pl->f16));
  return AGMM_OK;
}

// Two products in one launch: how the second's tiles go round, and the estimate of its time.
struct TwoChoice {
  int bn, lead, ahead, each, rest;
  bool dx_first;
  double time;
};
TwoChoice choose_two(const ProductPlan* pl, int64_t dx_m_tiles, int dx_blocks, int64_t dw_m_tiles, int64_t dw_cols, int dw_blocks, int weights) {
  TwoChoice best = {};
  best.time = 1e300;
  const int64_t C = pl->pairs;
  for (int bn = kWideN; bn >= kNarrowN; bn -= kWideN - kNarrowN) {
    if (pl->bn >= 0 && pl->bn != bn) continue;
    const bool wide = bn == kWideN;
    const double block = wide ? kWideBlock : kNarrowBlock, tile = wide ? kWideTile : kNarrowTile;
    const int64_t dx_tiles = dx_m_tiles * ceil_div(pl->k, bn), dw_tiles = dw_m_tiles * ceil_div(dw_cols, bn) * weights;
    if (dx_tiles > kMostTiles || dw_tiles > kMostTiles) continue;
    const bool dx_first = dx_blocks >= dw_blocks;  // long tiles first
    const int64_t t0 = dx_first ? dx_tiles : dw_tiles, t1 = dx_first ? dw_tiles : dx_tiles;
    const double one0 = std::max((dx_first ? dx_blocks : dw_blocks) * block, tile), one1 = std::max((dx_first ? dw_blocks : dx_blocks) * block, tile);
    TwoChoice c = {};
    c.bn = bn;
    c.dx_first = dx_first;
    c.lead = (int)(t0 % C);
    const int64_t others = C - c.lead;
    c.ahead = c.lead ? (int)std::min<int64_t>((int64_t)(one0 / one1), t1 / others) : 0;
    c.each = (int)((t1 - c.ahead * others) / C);
    c.rest = (int)((t1 - c.ahead * others) % C);
    // the last of either kind of cluster; the others take the rest first
    const double others_end = (t0 / C) * one0 + (c.ahead + c.each + (c.rest > 0)) * one1;
    const double lead_end = c.lead ? (t0 / C + 1) * one0 + (c.each + (c.rest > others)) * one1 : 0;
    c.time = std::max(others_end, lead_end);
    if (c.time < best.time) best = c;
  }
  return best;
}

agmm_status_t run_two(const ProductPlan* pl, const Grads& g, const TwoChoice& c, int64_t dx_m_tiles, int64_t dw_m_tiles, void* workspace,
                      cudaStream_t stream) {
  TwoParams p = {};
  common_params(pl, &p, workspace);
  Product *dx = c.dx_first ? &p : &p.second, *dw = c.dx_first ? &p.second : &p;
  AGMM_TRY(input_grad(pl, dx, g, 0, c.bn));
  AGMM_TRY(weight_grad(pl, dw, g, c.bn));
  AGMM_TRY(lay_tiles(dx, dx_m_tiles));
  AGMM_TRY(lay_tiles(dw, dw_m_tiles));
  p.num_tiles = p.dp_tiles = p.tiles_per_problem * p.problems;
  p.lead = c.lead;
  p.ahead = c.ahead;
  p.each = c.each;
  p.rest = c.rest;
  p.stages = c.bn == kWideN ? kWideStages : kNarrowStages;
  p.tmem_cols = 2 * c.bn;
  const size_t smem = 1024 + p.stages * (size_t)(kTileBytes + c.bn * kTileK) + (size_t)kEpiWarps * kStageOutBytes + kCtlBytes;
  return check_cuda(launch_two(c.bn == kWideN ? wide_two(pl->f16) : narrow_two(pl->f16), p, pl->pairs, smem, stream), "products launch");
}

// The products of a backward pass: in one launch where that is estimated to be shorter.  It saves a
// launch and a ragged last wave, but cuts no tile along k.  (500 tokens, 2048 -> 512: 8.4 us in one
// launch, 13.5 in two; gated, 1003 tokens, 1288 -> 2056: 36 and 47 us; 4096 tokens, 2560 -> 5120: 115
// and 128 us; 4096 tokens, 4096 -> 14336: 495 and 524 us; 8192 tokens, 4096 -> 7168: 500 us either way.)
agmm_status_t run_grads(const ProductPlan* pl, const Grads& g, void* workspace, cudaStream_t stream) {
  const int64_t tokens = g.shards * g.rows, dw_rows = pl->transpose ? pl->n : pl->k, dw_cols = pl->transpose ? pl->k : pl->n;
  const int64_t dx_m_tiles = ceil_div(tokens, 2 * kTileM), dw_m_tiles = ceil_div(dw_rows, 2 * kTileM);
  const int64_t dw_blocks = ceil_div(g.rows, kTileK) * g.shards, dx_blocks = g.weights * ceil_div(pl->n, kTileK);
  if (dw_blocks > INT_MAX) return fail(AGMM_ERR_UNSUPPORTED, "too many rows");
  const int swap = g.dx && pl->path != 0 ? swap_box(1, tokens) : 0;
  RowChoice for_dx = {}, for_dw = {};
  if (g.dx && !swap) for_dx = choose_rows(pl, dx_m_tiles, pl->k, (int)dx_blocks, 1, false);
  if (g.dx && swap) for_dx.time = choose_swap(pl, (int)ceil_div(pl->k, kTileM), (int)dx_blocks, swap_stage_bytes(1, swap)).time;
  const bool may_merge = g.dx && g.dw && pl->merge != 0 && (!swap || g.weights * pl->k * pl->n * 2 <= kFewTokenBytes);
  if (g.dw) for_dw = choose_rows(pl, dw_m_tiles, dw_cols, (int)dw_blocks, g.weights, false);
  if (may_merge) {
    const TwoChoice two = choose_two(pl, dx_m_tiles, (int)dx_blocks, dw_m_tiles, dw_cols, (int)dw_blocks, g.weights);
    if (two.time < 1e300 && (pl->merge == 1 || two.time < for_dx.time + for_dw.time + kLaunch))
      return run_two(pl, g, two, dx_m_tiles, dw_m_tiles, workspace, stream);
  }
  if (g.dx) {
    GemmParams p = {};
    common_params(pl, &p, workspace);
    AGMM_TRY(input_grad(pl, &p, g, swap, for_dx.bn));
    AGMM_TRY(swap ? run_swap(pl, &p, kEpiPlain, pl->k, stream) : run_rows(pl, &p, kEpiPlain, for_dx, dx_m_tiles, stream));
  }
  if (g.dw) {
    GemmParams p = {};
    common_params(pl, &p, workspace);
    AGMM_TRY(weight_grad(pl, &p, g, for_dw.bn));
    AGMM_TRY(run_rows(pl, &p, kEpiPlain, for_dw, dw_m_tiles, stream));
  }
  return AGMM_OK;
}

agmm_status_t zero_rows(const char* name, void* p, int64_t stride, int64_t rows, int64_t cols, bool f32, cudaStream_t stream) {
  const size_t size = f32 ? 4 : 2;
  return check_cuda(cudaMemset2DAsync(p, (size_t)stride * size, 0, (size_t)cols * size, (size_t)rows, stream), name);
}

// Rows up to which the sums of columns are one launch with the activation's gradient, 64 columns to a
// block (gelu, 4096 columns, both ways: 37 rows 2.2 and 4.1 us, 384 rows 5.4 and 6.8, 512 rows 6.3 and
// 7.8; 1000 columns: 2.3 and 3.6, 5.3 and 5.3, 6.3 and 4.8 us).
constexpr int64_t kFewRows = 384;

// ---------------------------------------------------------------------- plans
// An environment override for tests and experiments, as agmm_plan reads them; -1: none in [lo, hi].
int env_int(const char* name, int lo, int hi) {
  const char* v = std::getenv(name);
  if (!v || !*v) return -1;
  const int i = std::atoi(v);
  return i >= lo && i <= hi ? i : -1;
}

// The kernels of an epilogue: their shared memory, and the clusters of them that run at once.
agmm_status_t prepare_kernels(ProductPlan* pl, int epi, bool save_f32) {
  int fit = 0;
  for (int bn : {kNarrowN, kWideN}) {
    AGMM_TRY(check_cuda(prepare_gemm(select_gemm(bn, epi, pl->f16, save_f32), 2, &fit), "kernel attributes"));
    pl->pairs = std::min(pl->pairs, fit);
  }
  for (int n = 2; n <= kMaxPairs; ++n) {
    AGMM_TRY(check_cuda(prepare_gemm(select_gemm(kNarrowN, epi, pl->f16, save_f32), 2 * n, &fit), "kernel attributes"));
    pl->joined[n] = std::min(pl->joined[n], fit);
  }
  for (int split = 1; split <= kMaxSplit; ++split) {
    AGMM_TRY(check_cuda(prepare_gemm(select_gemm(0, epi, pl->f16, save_f32), split, &fit), "kernel attributes"));
    pl->clusters[split] = std::min(pl->clusters[split], fit);
  }
  if (pl->pairs < 1 || pl->clusters[1] < 1) return fail(AGMM_ERR_UNSUPPORTED, "the kernels do not fit this device");
  return AGMM_OK;
}

agmm_status_t fill_plan(ProductPlan* pl, int64_t k, int64_t n, int act, int transpose, int dtype) {
  pl->k = k;
  pl->n = n;
  pl->act = act;
  pl->transpose = transpose != 0;
  pl->f16 = dtype == AGMM_F16;
  const int khz = peak_clock_khz(pl->device);
  const char* ms = std::getenv("AGMM_WAIT_LIMIT_MS");
  const int limit = ms && *ms ? std::atoi(ms) : 0;
  pl->wait_limit_cycles = (uint64_t)(limit > 0 ? limit : 2000) * (uint64_t)khz;
  const char* drop = std::getenv("AGMM_TEST_DROP_ARRIVE");
  pl->test_drop = drop && std::atoi(drop) != 0;
  if (pl->sms > kMostSms) return fail(AGMM_ERR_UNSUPPORTED, "more than %d SMs", kMostSms);
  pl->path = env_int("AGMM_PATH", 0, 1);
  pl->bn = env_int("AGMM_BN", kNarrowN, kWideN);
  if (pl->bn != kNarrowN && pl->bn != kWideN) pl->bn = -1;
  pl->cut = env_int("AGMM_STREAMK", 0, 1);
  pl->split = env_int("AGMM_SPLITK", 1, kMaxSplit);
  pl->merge = env_int("AGMM_MERGE", 0, 1);
  pl->pairs = pl->sms / 2;
  for (int split = 1; split <= kMaxSplit; ++split) pl->clusters[split] = pl->sms / split;
  for (int n = 2; n <= kMaxPairs; ++n) pl->joined[n] = pl->sms / (2 * n);
  int fit = 0;
  for (TwoFn fn : {wide_two(pl->f16), narrow_two(pl->f16)}) {
    AGMM_TRY(check_cuda(prepare_two(fn, &fit), "kernel attributes"));
    pl->pairs = std::min(pl->pairs, fit);
  }
  for (int epi = kEpiPlain; epi <= kEpiLinear; ++epi) AGMM_TRY(prepare_kernels(pl, epi, false));
  return AGMM_OK;
}

template <class Plan>
agmm_status_t product_plan(int64_t k, int64_t n, int act, bool none_ok, int transpose, int dtype, Plan** out) {
  AGMM_TRY(check_width("k", k, kMostWidth));
  AGMM_TRY(check_width("n", n, kMostWidth));
  AGMM_TRY(check_dtype(dtype));
  if (act < (none_ok ? kActNone : kActRelu) || act > kActGeluTanh) return fail(AGMM_ERR_INVALID_ARG, "unknown activation: %d", act);
  if (transpose != 0 && transpose != 1) return fail(AGMM_ERR_INVALID_ARG, "rhs_transpose must be 0 or 1: %d", transpose);
  int device = 0, sms = 0;
  AGMM_TRY(check_device(&device, &sms));
  Plan* pl = new (std::nothrow) Plan();
  if (!pl) return fail(AGMM_ERR_NOMEM, "plan allocation");
  pl->device = device;
  pl->sms = sms;
  const agmm_status_t st = fill_plan(pl, k, n, act, transpose, dtype);
  if (st != AGMM_OK) {
    delete pl;
    return st;
  }
  *out = pl;
  return AGMM_OK;
}

agmm_status_t save_float(ProductPlan* pl, int epi, int on) {
  if (!pl) return fail(AGMM_ERR_INVALID_ARG, "plan is NULL");
  if (on != 0 && on != 1) return fail(AGMM_ERR_INVALID_ARG, "on must be 0 or 1: %d", on);
  AGMM_TRY(check_plan_device(pl->device));
  if (on) AGMM_TRY(prepare_kernels(pl, epi, true));
  pl->saved_f32 = on != 0;
  return AGMM_OK;
}

agmm_status_t check_tokens(int64_t shards, int64_t rows) {
  if (shards < 1 || shards > kMaxShards) return fail(AGMM_ERR_INVALID_ARG, "shards must be in [1, 8]: %lld", (long long)shards);
  if (rows < 0 || rows > kMostRows / shards)
    return fail(AGMM_ERR_INVALID_ARG, "shards * rows must be in [0, 2^31 - 1024]: %lld * %lld", (long long)shards, (long long)rows);
  return AGMM_OK;
}

agmm_status_t check_x(const void* const* x, int64_t shards, int64_t* stride, int64_t rows, int64_t k) {
  for (int s = 0; s < shards; ++s) AGMM_TRY(check_matrix("x", x[s], stride, rows, k));
  return AGMM_OK;
}

}  // namespace

extern "C" {

// ----------------------------------------------------------------- layer_norm
agmm_status_t agmm_layer_norm_plan(const agmm_layer_norm_desc_t* d, agmm_layer_norm_t* out) {
  if (!out) return fail(AGMM_ERR_INVALID_ARG, "out_plan is NULL");
  *out = nullptr;
  if (!d) return fail(AGMM_ERR_INVALID_ARG, "desc is NULL");
  AGMM_TRY(check_width("columns", d->columns, kMaxNormColumns));
  AGMM_TRY(check_dtype(d->dtype));
  if (!(d->eps >= 0.0f) || !std::isfinite(d->eps)) return fail(AGMM_ERR_INVALID_ARG, "eps must be finite and not negative");
  int device = 0, sms = 0;
  AGMM_TRY(check_device(&device, &sms));
  AGMM_TRY(check_cuda(prepare_norm(d->dtype == AGMM_F16), "kernel attributes"));
  agmm_layer_norm_s* pl = new (std::nothrow) agmm_layer_norm_s();
  if (!pl) return fail(AGMM_ERR_NOMEM, "plan allocation");
  pl->columns = d->columns;
  pl->eps = d->eps;
  pl->f16 = d->dtype == AGMM_F16;
  pl->device = device;
  pl->sms = sms;
  *out = pl;
  return AGMM_OK;
}

void agmm_layer_norm_destroy(agmm_layer_norm_t plan) { delete plan; }

size_t agmm_layer_norm_workspace_bytes(agmm_layer_norm_t pl) {
  if (!pl) return 0;
  return AGMM_FEEDFORWARD_HEAD_BYTES + (size_t)norm_grad_blocks(INT_MAX, pl->columns, pl->sms) * 2 * pl->columns * sizeof(float);
}

agmm_status_t agmm_layer_norm_run(agmm_layer_norm_t pl, const agmm_layer_norm_args_t* a, void* stream) {
  if (!pl || !a) return fail(AGMM_ERR_INVALID_ARG, "plan or args is NULL");
  if (a->rows < 0 || a->rows > INT_MAX) return fail(AGMM_ERR_INVALID_ARG, "rows must be in [0, 2^31 - 1]: %lld", (long long)a->rows);
  if (a->rows == 0) return AGMM_OK;
  NormParams p = {};
  p.ldx = a->x_stride;
  p.ldo = a->out_stride;
  AGMM_TRY(check_matrix("x", a->x, &p.ldx, a->rows, pl->columns));
  AGMM_TRY(check_matrix("out", a->out, &p.ldo, a->rows, pl->columns));
  if (a->weight) AGMM_TRY(check_pointer("weight", a->weight, 16));
  if (a->bias) AGMM_TRY(check_pointer("bias", a->bias, 16));
  if (a->mean) AGMM_TRY(check_pointer("mean", a->mean, 4));
  if (a->rstd) AGMM_TRY(check_pointer("rstd", a->rstd, 4));
  AGMM_TRY(check_plan_device(pl->device));
  p.rows = a->rows;
  p.cols = pl->columns;
  p.eps = pl->eps;
  p.x = static_cast<const uint16_t*>(a->x);
  p.weight = static_cast<const uint16_t*>(a->weight);
  p.bias = static_cast<const uint16_t*>(a->bias);
  p.out = static_cast<uint16_t*>(a->out);
  p.mean = a->mean;
  p.rstd = a->rstd;
  return check_cuda(launch_norm(p, pl->f16, pl->sms, static_cast<cudaStream_t>(stream)), "layer_norm launch");
}

agmm_status_t agmm_layer_norm_backward(agmm_layer_norm_t pl, const agmm_layer_norm_grad_args_t* a, void* stream) {
  if (!pl || !a) return fail(AGMM_ERR_INVALID_ARG, "plan or args is NULL");
  if (a->rows < 0 || a->rows > INT_MAX) return fail(AGMM_ERR_INVALID_ARG, "rows must be in [0, 2^31 - 1]: %lld", (long long)a->rows);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool sums = a->d_weight || a->d_bias;
  if (a->d_weight) AGMM_TRY(check_pointer("d_weight", a->d_weight, 16));
  if (a->d_bias) AGMM_TRY(check_pointer("d_bias", a->d_bias, 16));
  if (a->rows == 0) {
    if (sums) AGMM_TRY(check_plan_device(pl->device));
    if (a->d_weight) AGMM_TRY(zero_rows("d_weight", a->d_weight, pl->columns, 1, pl->columns, a->f32_grads != 0, s));
    if (a->d_bias) AGMM_TRY(zero_rows("d_bias", a->d_bias, pl->columns, 1, pl->columns, a->f32_grads != 0, s));
    return AGMM_OK;
  }
  if (!a->dx && !sums) return AGMM_OK;
  NormGradParams p = {};
  p.ld_out = a->d_out_stride;
  p.ldx = a->x_stride;
  p.ld_add = a->add_stride;
  p.ld_dx = a->dx_stride;
  AGMM_TRY(check_matrix("d_out", a->d_out, &p.ld_out, a->rows, pl->columns));
  AGMM_TRY(check_matrix("x", a->x, &p.ldx, a->rows, pl->columns));
  AGMM_TRY(check_pointer("mean", a->mean, 4));
  AGMM_TRY(check_pointer("rstd", a->rstd, 4));
  if (a->weight) AGMM_TRY(check_pointer("weight", a->weight, 16));
  if (a->add && !a->dx) return fail(AGMM_ERR_INVALID_ARG, "add is given without dx");
  if (a->add) AGMM_TRY(check_matrix("add", a->add, &p.ld_add, a->rows, pl->columns));
  if (a->dx) AGMM_TRY(check_matrix("dx", a->dx, &p.ld_dx, a->rows, pl->columns));
  if (sums) AGMM_TRY(check_pointer("workspace", a->workspace, 256));
  AGMM_TRY(check_plan_device(pl->device));
  p.rows = a->rows;
  p.cols = pl->columns;
  p.d_out = static_cast<const uint16_t*>(a->d_out);
  p.x = static_cast<const uint16_t*>(a->x);
  p.weight = static_cast<const uint16_t*>(a->weight);
  p.add = static_cast<const uint16_t*>(a->add);
  p.mean = a->mean;
  p.rstd = a->rstd;
  p.dx = static_cast<uint16_t*>(a->dx);
  p.part = sums ? reinterpret_cast<float*>(static_cast<char*>(a->workspace) + AGMM_FEEDFORWARD_HEAD_BYTES) : nullptr;
  // One launch has other blocks for the rows than for the sums, which would find dx in the place of what they read.
  const bool over = sums && a->dx && (may_overlap(a->dx, p.ld_dx, a->d_out, p.ld_out, a->rows) || may_overlap(a->dx, p.ld_dx, a->x, p.ldx, a->rows));
  if (!over && few_norm_rows(a->rows, pl->columns)) {
    p.d_weight = a->d_weight;
    p.d_bias = a->d_bias;
    p.out_f32 = a->f32_grads != 0;
    return check_cuda(launch_norm_grad_few(p, pl->f16, s), "layer_norm backward launch");
  }
  const int blocks = norm_grad_blocks(a->rows, pl->columns, pl->sms);
  AGMM_TRY(check_cuda(launch_norm_grad(p, pl->f16, blocks, s), "layer_norm backward launch"));
  if (!sums) return AGMM_OK;
  SumPartsParams q = {};
  q.part = p.part;
  q.parts = blocks;
  q.sums = 2;
  q.cols = pl->columns;
  q.out[0] = a->d_weight;
  q.out[1] = a->d_bias;
  q.out_f32 = a->f32_grads != 0;
  return check_cuda(launch_sum_parts(q, pl->f16, s), "layer_norm sums launch");
}

// ---------------------------------------------------------------------- gated
agmm_status_t agmm_gated_plan(const agmm_gated_desc_t* d, agmm_gated_t* out) {
  if (!out) return fail(AGMM_ERR_INVALID_ARG, "out_plan is NULL");
  *out = nullptr;
  if (!d) return fail(AGMM_ERR_INVALID_ARG, "desc is NULL");
  return product_plan(d->k, d->n, d->activation, false, d->rhs_transpose, d->dtype, out);
}

void agmm_gated_destroy(agmm_gated_t plan) { delete plan; }

agmm_status_t agmm_gated_save_float(agmm_gated_t pl, int on) { return save_float(pl, kEpiGated, on); }

size_t agmm_gated_workspace_bytes(agmm_gated_t pl) { return pl ? workspace_bytes(pl) : 0; }

agmm_status_t agmm_gated_run(agmm_gated_t pl, const agmm_gated_args_t* a, void* stream) {
  if (!pl || !a) return fail(AGMM_ERR_INVALID_ARG, "plan or args is NULL");
  AGMM_TRY(check_tokens(a->shards, a->rows));
  if (a->rows == 0) return AGMM_OK;
  const int64_t tokens = a->shards * a->rows, w_rows = pl->transpose ? pl->n : pl->k, w_cols = pl->transpose ? pl->k : pl->n;
  int64_t x_stride = a->x_stride, w_stride = a->w_stride, out_stride = a->out_stride, saved_stride = a->saved_stride;
  AGMM_TRY(check_x(a->x, a->shards, &x_stride, a->rows, pl->k));
  AGMM_TRY(check_matrix("w_gate", a->w_gate, &w_stride, w_rows, w_cols));
  AGMM_TRY(check_matrix("w_up", a->w_up, &w_stride, w_rows, w_cols));
  AGMM_TRY(check_matrix("out", a->out, &out_stride, tokens, pl->n));
  if (!a->gate != !a->up) return fail(AGMM_ERR_INVALID_ARG, "gate and up are given together or not at all");
  if (a->gate) {
    AGMM_TRY(check_matrix("gate", a->gate, &saved_stride, tokens, pl->n));
    AGMM_TRY(check_matrix("up", a->up, &saved_stride, tokens, pl->n));
  }
  AGMM_TRY(check_pointer("workspace", a->workspace, 256));
  AGMM_TRY(check_plan_device(pl->device));
  GemmParams p = {};
  common_params(pl, &p, a->workspace);
  p.out[0] = a->out;
  p.ldo = out_stride;
  p.saved[0] = a->gate;
  p.saved[1] = a->up;
  p.lds = saved_stride;
  p.act = pl->act;
  const void* const w[2] = {a->w_gate, a->w_up};
  return forward(pl, &p, kEpiGated, (int)a->shards, a->rows, a->x, x_stride, w, w_stride, static_cast<cudaStream_t>(stream));
}

agmm_status_t agmm_gated_backward(agmm_gated_t pl, const agmm_gated_grad_args_t* a, void* stream) {
  if (!pl || !a) return fail(AGMM_ERR_INVALID_ARG, "plan or args is NULL");
  AGMM_TRY(check_tokens(a->shards, a->rows));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int64_t tokens = a->shards * a->rows, w_rows = pl->transpose ? pl->n : pl->k, w_cols = pl->transpose ? pl->k : pl->n;
  int64_t x_stride = a->x_stride, w_stride = a->w_stride, out_stride = a->d_out_stride, saved_stride = a->saved_stride,
          d_stride = a->d_stride, dx_stride = a->dx_stride, dw_stride = a->dw_stride;
  if (!a->dw_gate != !a->dw_up) return fail(AGMM_ERR_INVALID_ARG, "dw_gate and dw_up are given together or not at all");
  if (a->dw_gate) {
    AGMM_TRY(check_matrix("dw_gate", a->dw_gate, &dw_stride, w_rows, w_cols));
    AGMM_TRY(check_matrix("dw_up", a->dw_up, &dw_stride, w_rows, w_cols));
  }
  void* const dw[2] = {a->dw_gate, a->dw_up};
  if (a->rows == 0) {
    if (!a->dw_gate) return AGMM_OK;
    AGMM_TRY(check_plan_device(pl->device));
    AGMM_TRY(zero_rows("dw_gate", a->dw_gate, dw_stride, w_rows, w_cols, a->f32_grads != 0, s));
    return zero_rows("dw_up", a->dw_up, dw_stride, w_rows, w_cols, a->f32_grads != 0, s);
  }
  AGMM_TRY(check_matrix("d_out", a->d_out, &out_stride, tokens, pl->n));
  AGMM_TRY(check_matrix("gate", a->gate, &saved_stride, tokens, pl->n));
  AGMM_TRY(check_matrix("up", a->up, &saved_stride, tokens, pl->n));
  AGMM_TRY(check_matrix("d_gate", a->d_gate, &d_stride, tokens, pl->n));
  AGMM_TRY(check_matrix("d_up", a->d_up, &d_stride, tokens, pl->n));
  if (pl->saved_f32 && (a->d_gate == a->gate || a->d_gate == a->up || a->d_up == a->gate || a->d_up == a->up))
    return fail(AGMM_ERR_INVALID_ARG, "d_gate and d_up cannot lie over gate and up that are float32");
  if (a->dx) {
    AGMM_TRY(check_matrix("w_gate", a->w_gate, &w_stride, w_rows, w_cols));
    AGMM_TRY(check_matrix("w_up", a->w_up, &w_stride, w_rows, w_cols));
    AGMM_TRY(check_matrix("dx", a->dx, &dx_stride, tokens, pl->k));
  }
  if (a->dw_gate) AGMM_TRY(check_x(a->x, a->shards, &x_stride, a->rows, pl->k));
  AGMM_TRY(check_pointer("workspace", a->workspace, 256));
  AGMM_TRY(check_plan_device(pl->device));
  GatedGradParams g = {};
  g.rows = tokens;
  g.cols = pl->n;
  g.d_out = static_cast<const uint16_t*>(a->d_out);
  g.gate = a->gate;
  g.up = a->up;
  g.d_gate = static_cast<uint16_t*>(a->d_gate);
  g.d_up = static_cast<uint16_t*>(a->d_up);
  g.ld_out = out_stride;
  g.ld_saved = saved_stride;
  g.ld_grad = d_stride;
  g.act = pl->act;
  g.saved_f32 = pl->saved_f32;
  AGMM_TRY(check_cuda(launch_gated_grad(g, pl->f16, pl->sms, s), "gated backward launch"));
  const void* const d[2] = {a->d_gate, a->d_up};
  const void* const w[2] = {a->w_gate, a->w_up};
  const Grads products = {2, (int)a->shards, a->rows, a->x, x_stride, d, d_stride, w, w_stride, a->dx, dx_stride, a->dw_gate ? dw : nullptr,
                          dw_stride, a->f32_grads != 0};
  return run_grads(pl, products, a->workspace, s);
}

// --------------------------------------------------------------------- linear
agmm_status_t agmm_linear_plan(const agmm_linear_desc_t* d, agmm_linear_t* out) {
  if (!out) return fail(AGMM_ERR_INVALID_ARG, "out_plan is NULL");
  *out = nullptr;
  if (!d) return fail(AGMM_ERR_INVALID_ARG, "desc is NULL");
  return product_plan(d->k, d->n, d->activation, true, d->rhs_transpose, d->dtype, out);
}

void agmm_linear_destroy(agmm_linear_t plan) { delete plan; }

agmm_status_t agmm_linear_save_float(agmm_linear_t pl, int on) { return save_float(pl, kEpiLinear, on); }

size_t agmm_linear_workspace_bytes(agmm_linear_t pl) { return pl ? workspace_bytes(pl) : 0; }

agmm_status_t agmm_linear_run(agmm_linear_t pl, const agmm_linear_args_t* a, void* stream) {
  if (!pl || !a) return fail(AGMM_ERR_INVALID_ARG, "plan or args is NULL");
  AGMM_TRY(check_tokens(a->shards, a->rows));
  if (a->rows == 0) return AGMM_OK;
  const int64_t tokens = a->shards * a->rows, w_rows = pl->transpose ? pl->n : pl->k, w_cols = pl->transpose ? pl->k : pl->n;
  int64_t x_stride = a->x_stride, w_stride = a->w_stride, out_stride = a->out_stride, res_stride = a->residual_stride,
          pre_stride = a->pre_stride;
  AGMM_TRY(check_x(a->x, a->shards, &x_stride, a->rows, pl->k));
  AGMM_TRY(check_matrix("w", a->w, &w_stride, w_rows, w_cols));
  if (a->bias) AGMM_TRY(check_pointer("bias", a->bias, 16));
  if (a->residual) AGMM_TRY(check_matrix("residual", a->residual, &res_stride, tokens, pl->n));
  AGMM_TRY(check_matrix("out", a->out, &out_stride, tokens, pl->n));
  if (a->pre) AGMM_TRY(check_matrix("pre", a->pre, &pre_stride, tokens, pl->n));
  AGMM_TRY(check_pointer("workspace", a->workspace, 256));
  AGMM_TRY(check_plan_device(pl->device));
  GemmParams p = {};
  common_params(pl, &p, a->workspace);
  p.out[0] = a->out;
  p.ldo = out_stride;
  p.saved[0] = a->pre;
  p.lds = pre_stride;
  p.bias = a->bias;
  p.residual = a->residual;
  p.ldr = res_stride;
  p.act = pl->act;
  return forward(pl, &p, kEpiLinear, (int)a->shards, a->rows, a->x, x_stride, &a->w, w_stride, static_cast<cudaStream_t>(stream));
}

agmm_status_t agmm_linear_backward(agmm_linear_t pl, const agmm_linear_grad_args_t* a, void* stream) {
  if (!pl || !a) return fail(AGMM_ERR_INVALID_ARG, "plan or args is NULL");
  AGMM_TRY(check_tokens(a->shards, a->rows));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int64_t tokens = a->shards * a->rows, w_rows = pl->transpose ? pl->n : pl->k, w_cols = pl->transpose ? pl->k : pl->n;
  int64_t x_stride = a->x_stride, w_stride = a->w_stride, out_stride = a->d_out_stride, pre_stride = a->pre_stride,
          d_stride = a->d_pre_stride, dx_stride = a->dx_stride, dw_stride = a->dw_stride;
  const bool f32 = a->f32_grads != 0;
  if (a->dw) AGMM_TRY(check_matrix("dw", a->dw, &dw_stride, w_rows, w_cols));
  if (a->d_bias) AGMM_TRY(check_pointer("d_bias", a->d_bias, 16));
  if (a->rows == 0) {
    if (a->dw || a->d_bias) AGMM_TRY(check_plan_device(pl->device));
    if (a->dw) AGMM_TRY(zero_rows("dw", a->dw, dw_stride, w_rows, w_cols, f32, s));
    if (a->d_bias) AGMM_TRY(zero_rows("d_bias", a->d_bias, pl->n, 1, pl->n, f32, s));
    return AGMM_OK;
  }
  const bool acts = pl->act != kActNone;
  AGMM_TRY(check_matrix("d_out", a->d_out, &out_stride, tokens, pl->n));
  if (acts) {
    AGMM_TRY(check_matrix("pre", a->pre, &pre_stride, tokens, pl->n));
    AGMM_TRY(check_matrix("d_pre", a->d_pre, &d_stride, tokens, pl->n));
    if (pl->saved_f32 && a->d_pre == a->pre) return fail(AGMM_ERR_INVALID_ARG, "d_pre cannot lie over a pre that is float32");
  } else if (a->pre || a->d_pre) {
    return fail(AGMM_ERR_INVALID_ARG, "pre and d_pre belong to an activation, and the plan has none");
  }
  if (a->dx) {
    AGMM_TRY(check_matrix("w", a->w, &w_stride, w_rows, w_cols));
    AGMM_TRY(check_matrix("dx", a->dx, &dx_stride, tokens, pl->k));
  }
  if (a->dw) AGMM_TRY(check_x(a->x, a->shards, &x_stride, a->rows, pl->k));
  AGMM_TRY(check_pointer("workspace", a->workspace, 256));
  AGMM_TRY(check_plan_device(pl->device));
  if (acts || a->d_bias) {
    GemmParams where = {};
    common_params(pl, &where, a->workspace);
    ActGradParams g = {};
    g.rows = tokens;
    g.cols = pl->n;
    g.d_out = static_cast<const uint16_t*>(a->d_out);
    g.pre = a->pre;
    g.d_pre = static_cast<uint16_t*>(a->d_pre);
    g.ld_out = out_stride;
    g.ld_pre = pre_stride;
    g.ld_grad = d_stride;
    g.act = pl->act;
    g.saved_f32 = pl->saved_f32;
    const bool few = a->d_bias && tokens <= kFewRows;
    if (few) {
      g.d_bias = a->d_bias;
      g.out_f32 = f32;
    } else {
      g.part = a->d_bias ? where.partial : nullptr;
      g.row_blocks = act_grad_row_blocks(tokens, pl->n, pl->sms);
      const int64_t room = (int64_t)(partial_bytes(pl) / ((size_t)pl->n * sizeof(float)));
      if (a->d_bias) g.row_blocks = (int)std::min<int64_t>(g.row_blocks, room);
    }
    AGMM_TRY(check_cuda(launch_act_grad(g, pl->f16, s), "linear backward launch"));
    if (g.part) {
      SumPartsParams q = {};
      q.part = g.part;
      q.parts = g.row_blocks;
      q.sums = 1;
      q.cols = pl->n;
      q.out[0] = a->d_bias;
      q.out_f32 = f32;
      AGMM_TRY(check_cuda(launch_sum_parts(q, pl->f16, s), "linear backward sums launch"));
    }
  }
  const void* const d = acts ? a->d_pre : a->d_out;
  if (!acts) d_stride = out_stride;
  const Grads products = {1, (int)a->shards, a->rows, a->x, x_stride, &d, d_stride, &a->w, w_stride, a->dx, dx_stride,
                          a->dw ? &a->dw : nullptr, dw_stride, f32};
  return run_grads(pl, products, a->workspace, s);
}

}  // extern "C"
