// ff_gemm.cuh -- the matrix products of the feed-forward operators: a persistent
// warp-specialised tcgen05 kernel with the operators' epilogues.
//
//   gated   out = act(X Wg) * (X Wu)         both products' tiles in one accumulator
//   linear  out = act(X W + bias) + residual
//   plain   the products of the backward passes (gradients of X and of the weights)
//
// Warp 0 loads operand tiles by TMA, warp 1 issues the MMAs (float32 accumulators in
// tensor memory, two of them, so that a tile's epilogue runs beside the next tile's
// products), warps 2-9 are the epilogue.  Either operand may be stored along k or
// along its own rows or columns (the weights come in both layouts, and the gradients
// of the weights sum over tokens): that is a matter of the tensor maps' boxes and two
// bits of the MMA's descriptor, chosen at run time.
//
//   row tiles      a CTA pair multiplies 256 rows by 256 columns (cta_group::2), or by
//                  128 where that makes better use of the CTAs, each CTA holding its
//                  own rows and half of the columns' operand.  Gated: the leader's half
//                  is columns of the gate's weight, the follower's the same columns of
//                  the other, so both products of an output value land in one thread.
//                  Bound: the tensor cores, active in 91 to 97 % of the cycles: 8192 x 4096 x
//                  14336 490-496 us (1.94-1.96 PFLOP/s), its gradients 490 and 496 us, in bursts;
//                  in long runs the power limit.  A k block of wide tiles takes 512 to 520 cycles,
//                  512 of them products, and each SM reads 64 bytes a cycle from L2.  Narrow ones
//                  would read 96 at the products' 256 cycles; they read 80 with 4 pairs at work
//                  (306 cycles) and 67 with all 76 (367).  One CTA with 128 x 128 tiles would need
//                  128 bytes a cycle.
//   swapped tiles  for up to 64 tokens: 128 columns of the weights are the MMA's rows
//                  and all tokens its columns, so that each thread of the epilogue has
//                  one column of the weights and only the tokens that there are.
//                  Bound: the weights' bytes: one token of 4096 -> 2 x 7168 22 us (5.4 TB/s, 4 us
//                  of them start and end), 64 tokens 25 us; row tiles take 39 and 28 us.  Above
//                  64 tokens narrow row tiles win (128 tokens of 2048 -> 2 x 2048: 13 against 20 us).
//
// Work: cluster c takes whole tiles in turn.  Where few tiles leave SMs idle, k is shared: by
// the CTAs (narrow row tiles: two to four pairs) of a cluster, whose parts meet in distributed
// shared memory (1 us; through L2 it was 4 us: one token of 7168 -> 4096 13 and 16 us).  Row tiles
// of a ragged last wave, and the wave before it, are cut evenly over the clusters.  Every
// warp of a cut row tile's epilogue leaves its float32 partial results in the workspace and
// counts its k blocks; the warp that completes the count adds all parts and goes on to the
// results.  Nobody waits for another cluster, and parts are added in the order of k.  Both
// gradients of a layer may be one launch (kTwo): the second product's tiles, all whole, follow
// the first's, and clusters with one less of those take more of them.
//
// Every mbarrier wait is bounded; one that runs out records AGMM_ERR_TIMEOUT in the
// status words, all roles leave their loops, wait (bounded) for their own work in
// flight, and the CTA frees its tensor memory and returns.
#pragma once

#include <type_traits>

#include "ff_math.cuh"
#include "ptx_sm103.cuh"

namespace agmm {
namespace ff {
namespace {

constexpr int kStatusTimeout = 5;  // AGMM_ERR_TIMEOUT
enum Role : int { kRoleProducer = 1, kRoleMma = 2, kRoleEpilogue = 3, kRoleDrain = 4 };

// Control block: full[], empty[], acc_full[2], acc_empty[2], drain; then the abort flag,
// the TMEM address and the swapped tiles' table of output rows.
__device__ __forceinline__ uint32_t bar_full(uint32_t ctl, int s) { return ctl + 8u * s; }
__device__ __forceinline__ uint32_t bar_empty(uint32_t ctl, int s) { return ctl + 8u * (kMaxStages + s); }
__device__ __forceinline__ uint32_t bar_acc_full(uint32_t ctl, int a) { return ctl + 8u * (2 * kMaxStages + a); }
__device__ __forceinline__ uint32_t bar_acc_empty(uint32_t ctl, int a) { return ctl + 8u * (2 * kMaxStages + 2 + a); }
__device__ __forceinline__ uint32_t bar_drain(uint32_t ctl) { return ctl + 8u * (2 * kMaxStages + 4); }
constexpr int kAbortOffset = 8 * (2 * kMaxStages + 6);
constexpr int kTmemOffset = kAbortOffset + 8;
constexpr int kTableOffset = 256;  // int[kMaxSwapRows + 16]: groups of tokens may be read past the last
static_assert(kTmemOffset + 4 <= kTableOffset && kTableOffset + 4 * (kMaxSwapRows + 16) <= kCtlBytes, "control block");

enum WaitResult : int { kWaitOk = 1, kWaitTimeout = 0, kWaitAborted = -1 };
constexpr uint32_t kSleepHintNs = 20000;

template <bool kClusterScope>
__device__ __forceinline__ bool try_wait(uint32_t bar, uint32_t parity) {
  if constexpr (kClusterScope)
    return ptx::mbar_try_wait_cluster(bar, parity);
  else
    return ptx::mbar_try_wait(bar, parity);
}

template <bool kClusterScope = false>
__device__ __forceinline__ int wait_phase(uint32_t bar, uint32_t parity, volatile int* abort, uint64_t limit) {
  if (try_wait<kClusterScope>(bar, parity)) return kWaitOk;
  const uint64_t t0 = ptx::clock_cycles();
  for (;;) {
    bool done;
    if constexpr (kClusterScope)
      done = ptx::mbar_try_wait_cluster_sleep(bar, parity, kSleepHintNs);
    else
      done = ptx::mbar_try_wait_sleep(bar, parity, kSleepHintNs);
    if (done) return kWaitOk;
    if (*abort) return kWaitAborted;
    if (ptx::clock_cycles() - t0 > limit) return kWaitTimeout;
  }
}

// Waits for work in flight whatever the abort flag says.
__device__ __forceinline__ bool wait_drain(uint32_t bar, uint32_t parity, uint64_t limit) {
  if (ptx::mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = ptx::clock_cycles();
  for (;;) {
    if (ptx::mbar_try_wait_sleep(bar, parity, kSleepHintNs)) return true;
    if (ptx::clock_cycles() - t0 > limit) return false;
  }
}

__device__ __noinline__ void record_failure(const GemmParams& p, volatile int* abort, int result, int role, int stage, int tile) {
  *abort = 1;
  if (result == kWaitTimeout && atomicCAS(p.status, 0, kStatusTimeout) == 0) {
    p.status[1] = role;
    p.status[2] = stage;
    p.status[3] = tile;
  }
}

// A cluster's share of the work, one segment after another: its even share of the cut
// tiles' k blocks first, so that the parts are there early, then its whole tiles.
struct Segment {
  int tile, problem, mt, nt;  // tile: of its product
  bool second;
  int kb0, kb1;
  bool whole;
};

__device__ __forceinline__ int first_unit(const GemmParams& p, int cluster) {
  return cluster * p.sk_share + min(cluster, p.sk_extra);
}

template <bool kTwo>
using ParamsOf = std::conditional_t<kTwo, TwoParams, GemmParams>;

template <bool kTwo>
__device__ __forceinline__ const Product& product_of(const ParamsOf<kTwo>& p, const Segment& s) {
  if constexpr (kTwo)
    if (s.second) return p.second;
  return p;
}

template <bool kTwo>
struct SegmentIter {
  int u, hi, next_dp, clusters, part, split;
  int cluster, taken;  // of the second product's tiles

  __device__ __forceinline__ void init(const GemmParams& p, int cluster_id, int nclusters, int k_part, int splits) {
    cluster = cluster_id;
    taken = 0;
    clusters = nclusters;
    next_dp = cluster;
    part = k_part;
    split = splits;
    u = hi = 0;
    if (cluster < p.sk_clusters) {
      u = first_unit(p, cluster);
      hi = first_unit(p, cluster + 1);
    }
  }

  // The next tile of the second product; -1 behind the last.
  __device__ __forceinline__ int next_second(const TwoParams& p) {
    const int others = clusters - p.lead;
    int i = taken++;
    if (cluster >= p.lead) {
      if (i < p.ahead) return i * others + cluster - p.lead;
      i -= p.ahead;
    }
    const int base = others * p.ahead;
    if (i < p.each) return base + i * clusters + cluster;
    const int place = cluster >= p.lead ? cluster - p.lead : others + cluster;
    return i == p.each && place < p.rest ? base + p.each * clusters + place : -1;
  }

  __device__ __forceinline__ bool next(const ParamsOf<kTwo>& p, Segment& s) {
    s.second = false;
    if (u < hi) {
      const int t = u / p.k_blocks;
      s.tile = p.dp_tiles + t;
      s.kb0 = u - t * p.k_blocks;
      s.kb1 = min(p.k_blocks, s.kb0 + (hi - u));
      u += s.kb1 - s.kb0;
    } else if (next_dp < p.dp_tiles) {
      s.tile = next_dp;
      s.kb0 = split > 1 ? p.k_blocks * part / split : 0;
      s.kb1 = split > 1 ? p.k_blocks * (part + 1) / split : p.k_blocks;
      next_dp += clusters;
    } else {
      if constexpr (kTwo) {
        s.tile = next_second(p);
        s.second = true;
        s.kb0 = 0;
        s.kb1 = p.second.k_blocks;
        if (s.tile < 0) return false;
      } else {
        return false;
      }
    }
    const Product& w = product_of<kTwo>(p, s);
    s.whole = s.kb0 == 0 && s.kb1 == w.k_blocks;
    s.problem = s.tile >= w.tiles_per_problem;
    // bands of group_m row tiles sweep the columns together: their rows stay in L2
    const int t = s.tile - s.problem * w.tiles_per_problem;
    const int per_group = w.group_m * w.n_tiles;
    const int group = t / per_group, first = group * w.group_m;
    const int in_group = min(w.m_tiles - first, w.group_m), r = t - group * per_group;
    s.nt = r / in_group;
    s.mt = first + r - s.nt * in_group;
    return true;
  }
};

// Where the parts of a cut tile lie: clusters [first, last], the tile's k in their order.
// Each has its first tile's part in slot 0: this tile's, but for a first cluster that began before it.
struct Parts {
  int first, last, first_slot;
};
__device__ __forceinline__ int cluster_of(const GemmParams& p, int unit) {
  const int longer = p.sk_extra * (p.sk_share + 1);  // the units of the first sk_extra clusters
  return unit < longer ? unit / (p.sk_share + 1) : p.sk_extra + (unit - longer) / p.sk_share;
}
__device__ __forceinline__ Parts find_parts(const GemmParams& p, int tile) {
  const int u0 = (tile - p.dp_tiles) * p.k_blocks;
  Parts r;
  r.first = cluster_of(p, u0);
  r.last = cluster_of(p, u0 + p.k_blocks - 1);
  r.first_slot = first_unit(p, r.first) < u0 ? 1 : 0;
  return r;
}

// A warp's part of a cut tile.
__device__ __forceinline__ float4* part_slot(const GemmParams& p, int c, int ctas, int rank, int slot, int ewarp) {
  return reinterpret_cast<float4*>(reinterpret_cast<char*>(p.partial) + (((size_t)c * ctas + rank) * kSlots + slot) * kSlotBytes +
                                   (size_t)ewarp * (kSlotBytes / kEpiWarps));
}

// Counts this warp's k blocks of a cut tile, after its part was stored; true for the
// warp that completes the tile.
__device__ __forceinline__ bool complete_tile(const GemmParams& p, int* counter, int blocks, int lane) {
  __threadfence();
  __syncwarp();
  int last = 0;
  if (lane == 0) {
    last = atomicAdd(counter, blocks) + blocks == p.k_blocks;
    if (last) *counter = 0;  // ready for the next run
  }
  last = __shfl_sync(0xffffffffu, last, 0);
  __threadfence();
  __syncwarp();
  return last != 0;
}

// kCount values of this lane from column `col` on (of its warp's columns, in the order in which
// they are stored), of kArrays arrays `stride` columns apart, summed over the parts; the loads of
// kDepth parts are in flight together.
template <int kArrays, int kCount, int kDepth>
__device__ __forceinline__ void sum_parts(const GemmParams& p, const Parts& parts, int ctas, int rank, int ewarp, int col, int stride,
                                          int lane, uint32_t (&v)[kArrays][kCount]) {
  constexpr int kQuads = kCount / 4;
  float4 sum[kArrays][kQuads];
#pragma unroll
  for (int t = 0; t < kArrays; ++t)
#pragma unroll
    for (int i = 0; i < kQuads; ++i) sum[t][i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 1
  for (int c0 = parts.first; c0 <= parts.last; c0 += kDepth) {
    float4 x[kDepth][kArrays][kQuads];
#pragma unroll
    for (int d = 0; d < kDepth; ++d) {
      const float4* const src = part_slot(p, c0 + d, ctas, rank, c0 + d == parts.first ? parts.first_slot : 0, ewarp) + lane;
#pragma unroll
      for (int t = 0; t < kArrays; ++t)
#pragma unroll
        for (int i = 0; i < kQuads; ++i)
          x[d][t][i] = c0 + d <= parts.last ? __ldcg(src + ((col + t * stride) / 4 + i) * 32) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
#pragma unroll
    for (int d = 0; d < kDepth; ++d)
#pragma unroll
      for (int t = 0; t < kArrays; ++t)
#pragma unroll
        for (int i = 0; i < kQuads; ++i) {
          sum[t][i].x += x[d][t][i].x;
          sum[t][i].y += x[d][t][i].y;
          sum[t][i].z += x[d][t][i].z;
          sum[t][i].w += x[d][t][i].w;
        }
  }
#pragma unroll
  for (int t = 0; t < kArrays; ++t)
#pragma unroll
    for (int i = 0; i < kQuads; ++i) {
      v[t][4 * i] = __float_as_uint(sum[t][i].x);
      v[t][4 * i + 1] = __float_as_uint(sum[t][i].y);
      v[t][4 * i + 2] = __float_as_uint(sum[t][i].z);
      v[t][4 * i + 3] = __float_as_uint(sum[t][i].w);
    }
}

__device__ __forceinline__ void tmem_ld_x8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr)
               : "memory");
}

template <bool kPair>
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const void* map, uint32_t bar, int c0, int c1, int c2, int c3) {
  if constexpr (kPair)
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst), "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst), "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar)
        : "memory");
}

// How an operand's tile is copied: rows of 64 values of k each in one box, or (chunks) by the
// other lanes; or MN-major, 128 (or 64) values of 64 rows of k as blocks of 64 x 64, in one
// box where the map has the blocks as a dimension.
enum LayoutKind : int { kLayoutRows = 0, kLayoutChunks = 1, kLayoutBlocks = 2, kLayoutTwoBoxes = 3 };
template <int kLayout>
using Layout = std::integral_constant<int, kLayout>;

template <bool kPair>
__device__ __forceinline__ void load_rows_of(uint32_t dst, const CUtensorMap* map, uint32_t bar, int k, int row) {
  if constexpr (kPair)
    ptx::tma_load_2d_pair(dst, map, bar, k, row);
  else
    ptx::tma_load_2d(dst, map, bar, k, row);
}

template <bool kPair, int kLayout, int kRows>
__device__ __forceinline__ void load_operand(uint32_t dst, const CUtensorMap* map, uint32_t bar, int k, int row, int z) {
  if constexpr (kLayout == kLayoutRows) {
    load_rows_of<kPair>(dst, map, bar, k, row);
  } else if constexpr (kLayout == kLayoutBlocks) {
    tma_load_4d<kPair>(dst, map, bar, 0, k, row >> 6, z);
  } else if constexpr (kLayout == kLayoutTwoBoxes) {
    tma_load_4d<kPair>(dst, map, bar, row, k, 0, z);
    if constexpr (kRows > 64) tma_load_4d<kPair>(dst + 8192u, map, bar, row + 64, k, 0, z);
  }
}

template <class F>
__device__ __forceinline__ void with_layout(int mn_major, int blocked, bool chunks, F&& f) {
  if (!mn_major) {
    if (chunks)
      f(Layout<kLayoutChunks>());
    else
      f(Layout<kLayoutRows>());
  } else if (blocked) {
    f(Layout<kLayoutBlocks>());
  } else {
    f(Layout<kLayoutTwoBoxes>());
  }
}

__device__ __forceinline__ void st_cluster_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
constexpr uint32_t kPartBytes = kTileM * 8 * sizeof(float);  // swapped tiles: one product's part of 8 tokens

template <int kCount>
__device__ __forceinline__ void store_part(float4* slot, int col, int lane, const uint32_t (&v)[kCount]) {
#pragma unroll
  for (int i = 0; i < kCount / 4; ++i)
    __stcg(slot + (size_t)(col / 4 + i) * 32 + lane,
           make_float4(__uint_as_float(v[4 * i]), __uint_as_float(v[4 * i + 1]), __uint_as_float(v[4 * i + 2]),
                       __uint_as_float(v[4 * i + 3])));
}

constexpr uint32_t kRowPartBytes = 32 * 64 * sizeof(float);  // narrow row tiles: a warp's part, 32 rows of 64 columns

// kArrays x 32 values of this lane's row, from column `c` on, `stride` apart, summed over the pairs'
// parts in shared memory.
template <int kArrays>
__device__ __forceinline__ void sum_received(const uint8_t* parts, int split, int c, int stride, int lane, uint32_t (&v)[kArrays][32]) {
  float sum[kArrays][32];
#pragma unroll
  for (int t = 0; t < kArrays; ++t)
#pragma unroll
    for (int i = 0; i < 32; ++i) sum[t][i] = 0.0f;
#pragma unroll 1
  for (int r = 0; r < split; ++r) {
    const float4* const src = reinterpret_cast<const float4*>(parts + (uint32_t)r * kRowPartBytes) + lane;
#pragma unroll
    for (int t = 0; t < kArrays; ++t)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float4 x = src[((c + t * stride) / 4 + i) * 32];
        sum[t][4 * i] += x.x;
        sum[t][4 * i + 1] += x.y;
        sum[t][4 * i + 2] += x.z;
        sum[t][4 * i + 3] += x.w;
      }
  }
#pragma unroll
  for (int t = 0; t < kArrays; ++t)
#pragma unroll
    for (int i = 0; i < 32; ++i) v[t][i] = __float_as_uint(sum[t][i]);
}

// A warp's staging buffer: 32 rows of 128 bytes, 16-byte pieces swizzled by the row, so
// that both a lane's own row and four whole rows at a time are free of bank conflicts.
__device__ __forceinline__ uint4* staged(uint8_t* stage, int row, int piece) {
  return reinterpret_cast<uint4*>(stage + row * 128 + ((piece ^ (row & 7)) << 4));
}

// The rows of the results that a lane reads and writes in a block of 32 rows of kPieces 16-byte
// pieces, kPieces lanes to a row: of row `mine` of each lane (< 0: none).
template <int kPieces>
__device__ __forceinline__ void block_rows(int (&rows)[kPieces], int mine, int lane) {
#pragma unroll
  for (int i = 0; i < kPieces; ++i) rows[i] = __shfl_sync(0xffffffffu, mine, (32 / kPieces) * i + lane / kPieces);
}

__device__ __forceinline__ char* row_address(const void* base, int row, uint32_t row_bytes) {
  return const_cast<char*>(static_cast<const char*>(base)) + (uint64_t)(uint32_t)row * row_bytes;
}

// Writes a staged block to its rows of `out` (of which `base` is this lane's piece of row 0).
template <int kPieces>
__device__ __forceinline__ void write_staged(uint8_t* stage, void* base, uint32_t row_bytes, const int (&rows)[kPieces], bool inside, int lane) {
  __syncwarp();
  uint4 v[kPieces];
#pragma unroll
  for (int i = 0; i < kPieces; ++i) v[i] = *staged(stage, (32 / kPieces) * i + lane / kPieces, lane % kPieces);
#pragma unroll
  for (int i = 0; i < kPieces; ++i)
    if (rows[i] >= 0 && inside) *reinterpret_cast<uint4*>(row_address(base, rows[i], row_bytes)) = v[i];
  __syncwarp();
}

// The same block's rows of `in`, into the staging buffer, asynchronously; zeros where there are none.
__device__ __forceinline__ void stage_rows(uint8_t* stage, const void* base, uint32_t row_bytes, const int (&rows)[8], bool inside, int lane) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const bool there = rows[i] >= 0 && inside;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(ptx::smem_addr(staged(stage, 4 * i + (lane >> 3), lane & 7))),
                 "l"(there ? row_address(base, rows[i], row_bytes) : base), "r"(there ? 16 : 0)
                 : "memory");
  }
}

template <int kCount>
__device__ __forceinline__ Two pair_of(const uint32_t (&v)[kCount], int i) {
  return two(__uint_as_float(v[i]), __uint_as_float(v[i + 1]));
}
template <int kCount>
__device__ __forceinline__ void set_pair(uint32_t (&v)[kCount], int i, Two x) {
  const float2 f = halves(x);
  v[i] = __float_as_uint(f.x);
  v[i + 1] = __float_as_uint(f.y);
}

template <bool kF16>
__device__ __forceinline__ void pack32(const uint32_t (&v)[32], uint32_t (&w)[16]) {
#pragma unroll
  for (int i = 0; i < 16; ++i) w[i] = pack2<kF16>(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
}

// A lane's 64 packed values, as its row of the staging buffer.
__device__ __forceinline__ void stage_half(uint8_t* stage, int lane, int half, const uint32_t (&w)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) *staged(stage, lane, half * 4 + i) = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
}

// kBN: columns of a row tile (0: swapped tiles).  kTwo: two products in one launch.  kSaveF32: what is
// saved is float32 (kernels of their own: as a branch it cost the others 0.5 to 2 %).
template <int kBN, int kEpi, bool kF16, bool kTwo = false, bool kSaveF32 = false>
__global__ void __launch_bounds__(kThreads, 1) agmm_ff_gemm(const __grid_constant__ ParamsOf<kTwo> p) {
  constexpr bool kSwap = kBN == 0, kPair = !kSwap;
  constexpr int kHalf = kBN / 2;  // columns of the accumulator that a warp of the epilogue has
  constexpr int kCtas = kPair ? 2 : 1;
  constexpr int kAccs = kSwap && kEpi == kEpiGated ? 2 : 1;  // swapped tiles: products of a tile
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw = ptx::smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* const base_ptr = smem_raw + (base - raw);
  const int S = p.stages;
  constexpr uint32_t a_slot = (uint32_t)kAccs * kTileBytes;
  const uint32_t b_slot = (uint32_t)(kSwap ? p.mma_n : kHalf) * 128u;
  const uint32_t a0 = base, b0 = base + (uint32_t)S * a_slot;
  const uint32_t out0 = b0 + (uint32_t)S * b_slot;  // row tiles: staged results
  const uint32_t recv = out0 + (kSwap ? 0u : (uint32_t)(kEpiWarps * kStageOutBytes));  // other CTAs' parts
  const uint32_t ctl = recv + p.recv_bytes;
  uint8_t* const ctl_ptr = base_ptr + (ctl - base);
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(ctl_ptr + kAbortOffset);
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(ctl_ptr + kTmemOffset);
  int* const row_table = reinterpret_cast<int*>(ctl_ptr + kTableOffset);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint64_t limit = p.wait_limit_cycles;
  // The pairs (swapped tiles: CTAs) of a cluster share a tile's k, or the cluster is one of them.
  const int split = kBN == kWideN ? 1 : p.split;
  const int cluster = (int)blockIdx.x / (kCtas * split), clusters = (int)gridDim.x / (kCtas * split);
  const int place = (int)blockIdx.x - cluster * kCtas * split;  // in the cluster
  const int rank = place % kCtas, part = place / kCtas;
  const uint32_t leader_place = (uint32_t)(place - rank);
  const uint16_t pair_mask = (uint16_t)(3u << leader_place);

  // A CTA takes more than half of an SM's shared memory: the next kernel's cannot come before this
  // one's tensor memory is allocated.
  if (threadIdx.x == 0) ptx::griddep_launch_dependents();
  if (warp == 0) {
    if (lane < S) {
      ptx::mbar_init(bar_full(ctl, lane), kCtas);  // a pair: both producers count on the leader's
      ptx::mbar_init(bar_empty(ctl, lane), 1);
    } else if (lane < S + 2) {
      ptx::mbar_init(bar_acc_full(ctl, lane - S), 1);
      ptx::mbar_init(bar_acc_empty(ctl, lane - S), kEpiWarps * kCtas);
    } else if (lane == S + 2) {
      ptx::mbar_init(bar_drain(ctl), 1);
    }
    if (lane < p.a.maps) ptx::prefetch_tensormap(&p.a_map[lane]);
    if (lane < p.b.maps) ptx::prefetch_tensormap(&p.b_map[lane]);
    if constexpr (kTwo) {
      if (lane < p.second.a.maps) ptx::prefetch_tensormap(&p.second.a_map[lane]);
      if (lane < p.second.b.maps) ptx::prefetch_tensormap(&p.second.b_map[lane]);
    }
    if (lane == 0) *abort_flag = 0;
    ptx::fence_mbar_init();
  }
  if (kSwap && warp >= 2) {
    // the output row of each token column
    const int c = (warp - 2) * 32 + lane;
    if (c < p.mma_n) {
      const int chunk = c / p.box, r = c - chunk * p.box;
      const int shard = chunk / p.shard_chunks;
      const int64_t row = (int64_t)(chunk - shard * p.shard_chunks) * p.box + r;
      row_table[c] = chunk < p.chunks && row < p.shard_rows ? (int)(shard * p.shard_rows + row) : -1;
    }
  }
  if (warp == 1) {
    if constexpr (kPair) {
      ptx::tmem_alloc_pair(ptx::smem_addr(tmem_slot), p.tmem_cols);
      ptx::tmem_relinquish_pair();
    } else {
      ptx::tmem_alloc(ptx::smem_addr(tmem_slot), p.tmem_cols);
      ptx::tmem_relinquish();
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  if constexpr (kPair) {
    // both CTAs' barriers are there before either's loads and MMAs signal them
    ptx::cluster_arrive_relaxed();
    ptx::cluster_wait();
  } else if (split > 1) {
    ptx::cluster_arrive_relaxed();  // matched before the first store to another CTA
  }
  ptx::tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  if (warp == 0) {
    // ---------------------------------------------------------------- producer
    // One elected lane of the converged warp issues the copies.  What a copy needs is worked out
    // once for a tile and a segment of k, and the operands' layouts are compiled in: with both
    // inside the loop over k, the issue took 750 cycles a k block, and the MMAs take 512.
    const bool leader = ptx::elect_one();
    int stage = 0;
    uint32_t phase = 0, armed = 0, armed_parity = 0;
    bool ok = true, dropped = p.test_drop == 0;
    SegmentIter<kTwo> iter;
    iter.init(p, cluster, clusters, part, split);
    Segment sg;
    const int per_tile = kSwap ? p.chunks : kTileM / p.box;  // chunks of the tokens: at most 16
    const uint32_t bytes = a_slot + (uint32_t)(kSwap ? p.chunks * p.box : kHalf) * 128u;
    const uint32_t full0 = kPair ? ptx::map_shared_rank(bar_full(ctl, 0), leader_place) : bar_full(ctl, 0);
    // The loads of k blocks [kb0, kb1) of one segment, from value ko of it on.
    auto produce = [&](auto a_layout, auto b_layout, int kb0, int kb1, int ko, const CUtensorMap* a_map, int a_row, int a_z,
                       const CUtensorMap* b_map, int b_row, int b_z, const CUtensorMap* lane_map, int lane_row) {
      constexpr int kA = a_layout.value, kB = b_layout.value;
      constexpr bool kChunks = kA == kLayoutChunks || kB == kLayoutChunks;
      bool empty_ready = false;
#pragma unroll 1
      for (int kb = kb0; kb < kb1; ++kb, ko += kTileK) {
        if (!__all_sync(0xffffffffu, empty_ready)) {
          int res = wait_phase(bar_empty(ctl, stage), phase ^ 1u, abort_flag, limit);
          res = __shfl_sync(0xffffffffu, res, 0);
          if (res != kWaitOk) {
            if (leader) record_failure(p, abort_flag, res, kRoleProducer, stage, sg.tile);
            ok = false;
            return;
          }
        }
        const int next_stage = stage + 1 == S ? 0 : stage + 1;
        const uint32_t next_phase = stage + 1 == S ? phase ^ 1u : phase;
        // A look ahead at the next stage.  Lanes may get different answers; the vote on them, which
        // every lane takes, stands where they are used: by then the looks are done, and it costs
        // nothing (right behind the look it cost 0.5 of 10.4 us for one token).
        empty_ready = kb + 1 < kb1 && ptx::mbar_test_wait(bar_empty(ctl, next_stage), next_phase ^ 1u);
        if (dropped) {
          if (!kPair || rank == 0) {
            armed |= 1u << stage;
            armed_parity = (armed_parity & ~(1u << stage)) | (phase << stage);
          }
          const uint32_t full = full0 + 8u * stage;
          const uint32_t a_dst = a0 + (uint32_t)stage * a_slot, b_dst = b0 + (uint32_t)stage * b_slot;
          if (leader) {
            if (kPair && rank == 1)
              ptx::mbar_arrive_expect_tx_remote(full, bytes);
            else
              ptx::mbar_arrive_expect_tx(bar_full(ctl, stage), bytes);
          }
          if constexpr (kChunks) {
            __syncwarp();
            if (lane < per_tile) load_rows_of<kPair>((kSwap ? b_dst : a_dst) + (uint32_t)(lane * p.box) * 128u, lane_map, full, ko, lane_row);
          }
          if (leader) {
#pragma unroll
            for (int t = 0; t < kAccs; ++t)
              load_operand<kPair, kA, kTileM>(a_dst + (uint32_t)t * kTileBytes, a_map + t, full, ko, a_row, a_z);
            load_operand<kPair, kB, kHalf>(b_dst, b_map, full, ko, b_row, b_z);
          }
          if constexpr (kChunks) __syncwarp();
        }
        dropped = true;
        stage = next_stage;
        phase = next_phase;
      }
    };
    ptx::griddep_wait();  // no access to global memory and no bounded wait before this, in any role
    while (ok && iter.next(p, sg)) {
      const Product& w = product_of<kTwo>(p, sg);
      const int row_tile = kPair ? sg.mt * 2 + rank : sg.mt;
      // Chunks of the tokens in a stage.  One to a stage is the elected lane's, with operands
      // that are uniform over the warp; else lane j has chunk j's map and row.  A chunk behind
      // the last lies outside its map: zeros.
      const int chunk0 = kSwap ? 0 : row_tile * per_tile;
      const int shard0 = min(chunk0 / w.shard_chunks, w.shards - 1);
      const int row0 = (chunk0 - shard0 * w.shard_chunks) * w.box;
      const int chunk = chunk0 + lane, shard = min(chunk / w.shard_chunks, w.shards - 1);
      const int lane_row = (chunk - shard * w.shard_chunks) * w.box;
      const int b_row = kSwap ? row0 : sg.nt * w.b_tile_step + rank * w.b_half_step;
      const int a_row = kSwap || w.a.mn_major ? row_tile * kTileM : row0;
      int seg = sg.kb0 / w.seg_blocks;
      for (int kb = sg.kb0; ok && kb < sg.kb1; ++seg) {
        const int end = min(sg.kb1, (seg + 1) * w.seg_blocks);
        const int ko = (kb - seg * w.seg_blocks) * kTileK, a_z = seg * w.a.z_segment, b_z = seg * w.b.z_segment;
        const CUtensorMap* a_map = w.a_map + sg.problem * w.a.by_problem + seg * w.a.by_segment;
        const CUtensorMap* b_map = w.b_map + sg.problem * w.b.by_problem + seg * w.b.by_segment + rank * w.b.by_rank;
        const CUtensorMap* const lane_map = kSwap ? b_map + shard * w.b.by_shard : a_map + shard * w.a.by_shard;
        if (kSwap)
          b_map += shard0 * w.b.by_shard;
        else
          a_map += shard0 * w.a.by_shard;
        with_layout(w.a.mn_major, w.a.blocked, !kSwap && per_tile > 1, [&](auto a_layout) {
          // swapped tiles: the tokens' rows lie along k
          if constexpr (kSwap) {
            if (per_tile > 1)
              produce(a_layout, Layout<kLayoutChunks>(), kb, end, ko, a_map, a_row, a_z, b_map, b_row, b_z, lane_map, lane_row);
            else
              produce(a_layout, Layout<kLayoutRows>(), kb, end, ko, a_map, a_row, a_z, b_map, b_row, b_z, lane_map, lane_row);
          } else {
            with_layout(w.b.mn_major, w.b.blocked, false, [&](auto b_layout) {
              produce(a_layout, b_layout, kb, end, ko, a_map, a_row, a_z, b_map, b_row, b_z, lane_map, lane_row);
            });
          }
        });
        kb = end;
      }
    }
    // only after an abort can a load be unconsumed
    if (leader)
      for (int s = 0; s < S; ++s)
        if ((armed >> s) & 1u)
          if (!wait_drain(bar_full(ctl, s), (armed_parity >> s) & 1u, limit))
            record_failure(p, abort_flag, kWaitTimeout, kRoleDrain, s, -1);
    __syncwarp();
    if (split > 1) {
      if (kSwap) ptx::cluster_wait();
      ptx::cluster_sync_all();  // the parts of k meet
    }
  } else if (warp == 1) {
    // -------------------------------------------------------------- MMA issuer
    if (!kPair || rank == 0) {
      const bool issuer = ptx::elect_one();
      const int n = kSwap ? p.mma_n : kBN;
      int stage = 0, it = 0;
      uint32_t phase = 0;
      bool ok = true;
      SegmentIter<kTwo> iter;
      iter.init(p, cluster, clusters, part, split);
      Segment sg;
      ptx::griddep_wait();  // a wait's bound counts from here, and the status words are the kernel before's until now
      for (; ok && iter.next(p, sg); ++it) {
        const int acc = it & 1;
        int res = wait_phase<kPair>(bar_acc_empty(ctl, acc), (uint32_t)((it >> 1) & 1) ^ 1u, abort_flag, limit);
        res = __shfl_sync(0xffffffffu, res, 0);
        if (res != kWaitOk) {
          if (issuer) record_failure(p, abort_flag, res, kRoleMma, -1, sg.tile);
          break;
        }
        ptx::tc_fence_after();
        const Product& w = product_of<kTwo>(p, sg);
        const uint32_t idesc = ptx::idesc_f16kind_f32(kPair ? 2 * kTileM : kTileM, n, w.a.mn_major != 0, w.b.mn_major != 0, kF16);
        // a k step of 16 values: 32 bytes inside the swizzle row, or 16 rows of 128 bytes
        const uint64_t a_step = w.a.mn_major ? 2048u / 16u : 32u / 16u, b_step = w.b.mn_major ? 2048u / 16u : 32u / 16u;
        const uint32_t a_lbo = w.a.mn_major ? 8192u : 16u, b_lbo = w.b.mn_major ? 8192u : 16u;
        const uint32_t d = tmem_base + (uint32_t)(acc * kAccs * n);
        bool full_ready = false;
        for (int kb = sg.kb0; kb < sg.kb1; ++kb) {
          if (!__all_sync(0xffffffffu, full_ready)) {
            res = wait_phase(bar_full(ctl, stage), phase, abort_flag, limit);
            res = __shfl_sync(0xffffffffu, res, 0);
            if (res != kWaitOk) {
              if (issuer) record_failure(p, abort_flag, res, kRoleMma, stage, sg.tile);
              ok = false;
              break;
            }
          }
          ptx::tc_fence_after();
          const int next_stage = stage + 1 == S ? 0 : stage + 1;
          const uint32_t next_phase = stage + 1 == S ? phase ^ 1u : phase;
          full_ready = kb + 1 < sg.kb1 && ptx::mbar_test_wait(bar_full(ctl, next_stage), next_phase);
          const uint64_t b_desc = ptx::smem_desc_sw128(b0 + (uint32_t)stage * b_slot, b_lbo, 1024u);
          if (issuer) {
#pragma unroll
            for (int t = 0; t < kAccs; ++t) {
              const uint64_t a_desc = ptx::smem_desc_sw128(a0 + (uint32_t)stage * a_slot + (uint32_t)t * kTileBytes, a_lbo, 1024u);
#pragma unroll
              for (int kk = 0; kk < kTileK / 16; ++kk) {
                const uint32_t accumulate = kb > sg.kb0 || kk > 0 ? 1u : 0u;
                if constexpr (kPair)
                  ptx::mma_bf16_pair(d, a_desc + a_step * (uint64_t)kk, b_desc + b_step * (uint64_t)kk, idesc, accumulate);
                else
                  ptx::mma_bf16(d + (uint32_t)(t * n), a_desc + a_step * (uint64_t)kk, b_desc + b_step * (uint64_t)kk, idesc, accumulate);
              }
            }
            if constexpr (kPair)
              ptx::mma_commit_pair(bar_empty(ctl, stage), pair_mask);
            else
              ptx::mma_commit(bar_empty(ctl, stage));
          }
          stage = next_stage;
          phase = next_phase;
        }
        if (!ok) break;
        if (issuer) {
          if constexpr (kPair)
            ptx::mma_commit_pair(bar_acc_full(ctl, acc), pair_mask);
          else
            ptx::mma_commit(bar_acc_full(ctl, acc));
        }
      }
      if (issuer) {
        if constexpr (kPair)
          ptx::mma_commit_pair(bar_drain(ctl), pair_mask);
        else
          ptx::mma_commit(bar_drain(ctl));
        if (!wait_drain(bar_drain(ctl), 0, limit)) record_failure(p, abort_flag, kWaitTimeout, kRoleDrain, -1, -1);
      }
      __syncwarp();
    }
    if (split > 1) {
      if (kSwap) ptx::cluster_wait();
      ptx::cluster_sync_all();  // the parts of k meet
    }
  } else {
    // ---------------------------------------------------------------- epilogue
    const int q = warp & 3, ewarp = warp - 2, half = ewarp >> 2;
    const uint32_t lane_base = tmem_base + ((uint32_t)(q * 32) << 16);
    uint8_t* const stage_out = base_ptr + (out0 - base) + ewarp * kStageOutBytes;  // row tiles
    SegmentIter<kTwo> iter;
    iter.init(p, cluster, clusters, part, split);
    const int first_cut = p.dp_tiles + iter.u / p.k_blocks;  // the tile whose part lies in slot 0
    Segment sg;
    ptx::griddep_wait();
    if (kSwap && split > 1) ptx::cluster_wait();  // every CTA of the cluster is there
    // Swapped tiles: the results of 8 tokens, columns [c, c + 8), of this lane's column of the weights.
    auto finish = [&](uint32_t (&v)[kAccs][8], int c) {
      const int64_t f = (int64_t)sg.mt * kTileM + q * 32 + lane;
      const bool there = f < p.cols;
      int row[8];
#pragma unroll
      for (int i = 0; i < 8; i += 4) {
        const int4 r = *reinterpret_cast<const int4*>(row_table + c + i);
        row[i] = there ? r.x : -1;
        row[i + 1] = there ? r.y : -1;
        row[i + 2] = there ? r.z : -1;
        row[i + 3] = there ? r.w : -1;
      }
      float bias = 0.0f;
      uint16_t res16[8];
      if constexpr (kEpi == kEpiLinear) {
        if (p.bias && there) bias = unpack1<kF16>(static_cast<const uint16_t*>(p.bias)[f]);
        if (p.residual) {
          const uint16_t* const base = static_cast<const uint16_t*>(p.residual) + f;
#pragma unroll
          for (int i = 0; i < 8; ++i)
            res16[i] = row[i] >= 0 ? *reinterpret_cast<const uint16_t*>(row_address(base, row[i], (uint32_t)p.ldr * 2u)) : (uint16_t)0;
        }
      }
      // all values first, then the stores: no branches between them
      uint32_t pre[8];
      with_activation(p.act, [&](auto act) {
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          Two x = pair_of(v[0], i);
          if constexpr (kEpi == kEpiLinear) x = add2(x, both(bias));
          set_pair(pre, i, x);
          if constexpr (kEpi != kEpiPlain) x = activate<act.value>(x);
          if constexpr (kEpi == kEpiGated) x = mul2(x, pair_of(v[kAccs - 1], i));
          if constexpr (kEpi == kEpiLinear)
            if (p.residual) x = add2(x, two(unpack1<kF16>(res16[i]), unpack1<kF16>(res16[i + 1])));
          set_pair(v[0], i, x);
        }
      });
      auto store = [&](void* out, uint32_t ld, const uint32_t (&x)[8]) {
        uint16_t* const base = static_cast<uint16_t*>(out) + f;
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (row[i] >= 0) *reinterpret_cast<uint16_t*>(row_address(base, row[i], ld)) = pack1<kF16>(__uint_as_float(x[i]));
      };
      auto save = [&](void* out, const uint32_t (&x)[8]) {
        if constexpr (kSaveF32) {
          uint32_t* const base = static_cast<uint32_t*>(out) + f;
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (row[i] >= 0) *reinterpret_cast<uint32_t*>(row_address(base, row[i], (uint32_t)p.lds * 4u)) = x[i];
        } else {
          store(out, (uint32_t)p.lds * 2u, x);
        }
      };
      if (kEpi == kEpiGated && p.saved[0]) save(p.saved[1], v[kAccs - 1]);
      store(p.out[0], (uint32_t)p.ldo * 2u, v[0]);
      if (kEpi != kEpiPlain && p.saved[0]) save(p.saved[0], pre);
    };
    const int owner = q % split;  // row tiles: the pair that goes on with these 32 rows
    bool met = false;
    for (int it = 0; iter.next(p, sg); ++it) {
      const Product& w = product_of<kTwo>(p, sg);
      const int acc = it & 1;
      // Row tiles: this lane's row, those that it reads and writes, and this warp's half of the columns.
      int out_row = -1, rows[8];
      // gated: as many columns of each product, the second's a half of the accumulator on
      const int first_col = kEpi == kEpiGated ? half * (kHalf / 2) : half * kHalf;
      const int64_t tile_col = (int64_t)sg.nt * (kEpi == kEpiGated ? kHalf : kBN) + first_col;
      // columns [c, c + 64) of this warp's half, into its staging buffer
      auto fetch_residual = [&](int c) {
        if constexpr (!kSwap && kEpi == kEpiLinear) {
          const int64_t at = tile_col + c + 8 * (lane & 7);
          stage_rows(stage_out, static_cast<const uint16_t*>(p.residual) + (at < w.cols ? at : 0), (uint32_t)p.ldr * 2u, rows, at < w.cols, lane);
        }
      };
      const bool has_residual = kEpi == kEpiLinear && p.residual != nullptr;
      // (what is saved in float32 goes through the staging buffer before the residual does)
      const bool residual_ahead = has_residual && !kSaveF32;
      if constexpr (!kSwap) {
        const int trow = (sg.mt * 2 + rank) * kTileM + q * 32 + lane;
        const int chunk = trow / w.box, shard = chunk / w.shard_chunks;
        const int in_shard = trow - shard * w.shard_chunks * w.box;
        if (shard < w.shards && in_shard < w.shard_rows) out_row = (int)(shard * w.shard_rows) + in_shard;
        block_rows(rows, out_row, lane);
        if (residual_ahead && (sg.whole || (split > 1 && owner == part))) fetch_residual(0);  // while the products are made
      }
      int res = kWaitOk;
      if (lane == 0) res = wait_phase(bar_acc_full(ctl, acc), (uint32_t)(it >> 1) & 1u, abort_flag, limit);
      res = __shfl_sync(0xffffffffu, res, 0);
      if (res != kWaitOk) {
        if (lane == 0) record_failure(p, abort_flag, res, kRoleEpilogue, acc, sg.tile);
        if (has_residual) asm volatile("cp.async.wait_all;" ::: "memory");
        break;
      }
      ptx::tc_fence_after();
      // the accumulator may be refilled (a pair's leader refills both CTAs')
      auto release = [&]() {
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (kPair && rank == 1)
            ptx::mbar_arrive_remote(ptx::map_shared_rank(bar_acc_empty(ctl, acc), leader_place));
          else
            ptx::mbar_arrive(bar_acc_empty(ctl, acc));
        }
      };
      if constexpr (kSwap) {
        // This lane's column of the weights, and this warp's half of the tokens, 8 at a time.
        const int n = p.mma_n, end = min((half + 1) * (n / 2), w.chunks * w.box);
        const uint32_t t0 = lane_base + (uint32_t)(acc * kAccs * n);
        for (int c = half * (n / 2); c < end; c += 8) {
          uint32_t v[kAccs][8];
#pragma unroll
          for (int t = 0; t < kAccs; ++t) tmem_ld_x8(t0 + (uint32_t)(t * n + c), v[t]);
          ptx::tmem_ld_wait();
          if (split == 1) {
            finish(v, c);
          } else {
            // to the CTA that owns these tokens: group c / 8 is slot c / 8 / split of CTA c / 8 % split
            const int slot = c / 8 / split;
            const uint32_t at = ptx::map_shared_rank(recv, (uint32_t)(c / 8 - slot * split)) +
                                (uint32_t)((part * p.recv_slots + slot) * kAccs) * kPartBytes + (uint32_t)(q * 32 + lane) * 16u;
#pragma unroll
            for (int t = 0; t < kAccs; ++t) {
              st_cluster_v4(at + (uint32_t)t * kPartBytes, v[t][0], v[t][1], v[t][2], v[t][3]);
              st_cluster_v4(at + (uint32_t)t * kPartBytes + kPartBytes / 2, v[t][4], v[t][5], v[t][6], v[t][7]);
            }
          }
        }
        release();
      } else {
        const uint32_t t0 = lane_base + (uint32_t)(acc * kBN);
        Parts parts = {0, 0, 0};
        if (!sg.whole) {
          // to the workspace, or to the pair that owns these rows: 8 KiB for each half of each of its
          // quarters of the rows, from each pair
          float4* const slot = split > 1 ? nullptr : part_slot(p, cluster, kCtas, rank, sg.tile == first_cut ? 0 : 1, ewarp);
          const uint32_t there = ptx::map_shared_rank(recv, (uint32_t)(owner * kCtas + rank)) +
                                 (uint32_t)(((q / split) * 2 + half) * split + part) * kRowPartBytes + (uint32_t)lane * 16u;
#pragma unroll 1
          for (int c = 0; c < kHalf; c += 32) {
            uint32_t v[32];
            // gated: this warp's columns of the first product, then of the second
            const int col = kEpi == kEpiGated && c >= kHalf / 2 ? kHalf + first_col + c - kHalf / 2 : first_col + c;
            ptx::tmem_ld_32x32b_x32(t0 + (uint32_t)col, v);
            ptx::tmem_ld_wait();
            if (split > 1) {
#pragma unroll
              for (int i = 0; i < 8; ++i) st_cluster_v4(there + (uint32_t)(c / 4 + i) * 512u, v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
            } else {
              store_part<32>(slot, c, lane, v);
            }
          }
          release();
          if (split > 1) {
            ptx::cluster_sync_all();  // the parts of k meet
            met = true;
            if (owner != part) continue;
          } else {
            int* const counter = p.counters + ((size_t)(sg.tile - p.dp_tiles) * kCtas + rank) * kEpiWarps + ewarp;
            if (!complete_tile(p, counter, sg.kb1 - sg.kb0, lane)) continue;
            parts = find_parts(p, sg.tile);
            if (residual_ahead) fetch_residual(0);
          }
        }
        // the sums over the parts of `v`'s columns from `c` on
        auto join = [&](auto& v, int c, int stride) {
          constexpr int kArrays = sizeof(v) / sizeof(v[0]);
          if (split > 1)
            sum_received<kArrays>(base_ptr + (recv - base) + ((q / split) * 2 + half) * split * kRowPartBytes, split, c, stride, lane, v);
          else
            sum_parts<kArrays, 32, kArrays == 1 && kEpi == kEpiPlain ? 2 : 1>(p, parts, kCtas, rank, ewarp, c, stride, lane, v);
        };
        // 32 values of this lane's row in float32, columns [col, col + 32), to `out`
        auto write_f32 = [&](void* out, int64_t ld, int64_t col, const uint32_t (&v)[32], const int (&at_rows)[8]) {
#pragma unroll
          for (int i = 0; i < 8; ++i) *staged(stage_out, lane, i) = make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
          const int64_t at = col + 4 * (lane & 7);
          write_staged<8>(stage_out, static_cast<float*>(out) + at, (uint32_t)ld * 4u, at_rows, at < w.cols, lane);
        };
        if constexpr (kEpi == kEpiGated && kSaveF32) {
          // 32 columns at a time through the staging buffer: both products, then the results
#pragma unroll 1
          for (int h = 0; h < kHalf / 64; ++h) {
            uint32_t v[2][32], o16[16];
            if (sg.whole) {
              ptx::tmem_ld_32x32b_x32(t0 + (uint32_t)(first_col + 32 * h), v[0]);
              ptx::tmem_ld_32x32b_x32(t0 + (uint32_t)(kHalf + first_col + 32 * h), v[1]);
              ptx::tmem_ld_wait();
              if (h == kHalf / 64 - 1) release();
            } else {
              join(v, 32 * h, kHalf / 2);
            }
            write_f32(p.saved[0], p.lds, tile_col + 32 * h, v[0], rows);
            write_f32(p.saved[1], p.lds, tile_col + 32 * h, v[1], rows);
            with_activation(p.act, [&](auto act) {
#pragma unroll
              for (int i = 0; i < 32; i += 2) set_pair(v[0], i, mul2(activate<act.value>(pair_of(v[0], i)), pair_of(v[1], i)));
            });
            pack32<kF16>(v[0], o16);
            stage_half(stage_out, lane, 0, o16);
            int rows4[4];
            block_rows(rows4, out_row, lane);
            const int64_t at = tile_col + 32 * h + 8 * (lane % 4);
            write_staged<4>(stage_out, static_cast<uint16_t*>(w.out[0]) + at, (uint32_t)w.ldo * 2u, rows4, at < w.cols, lane);
          }
        } else if constexpr (kEpi == kEpiGated) {
          constexpr int kBlocks = kHalf / 64;  // of 32 columns of results
          constexpr int kPieces = 4 * kBlocks;
          const int64_t col = tile_col + 8 * (lane % kPieces);  // of this lane's piece
          const bool inside = col < w.cols;
          int rows[kPieces];
          block_rows(rows, out_row, lane);
          uint32_t g16[kBlocks][16], u16[kBlocks][16];
#pragma unroll
          for (int h = 0; h < kBlocks; ++h) {
            uint32_t v[2][32], o16[16];
            if (sg.whole) {
              ptx::tmem_ld_32x32b_x32(t0 + (uint32_t)(first_col + 32 * h), v[0]);
              ptx::tmem_ld_32x32b_x32(t0 + (uint32_t)(kHalf + first_col + 32 * h), v[1]);
              ptx::tmem_ld_wait();
              if (h == kBlocks - 1) release();
            } else {
              join(v, 32 * h, kHalf / 2);
            }
            if (p.saved[0]) {
              pack32<kF16>(v[0], g16[h]);
              pack32<kF16>(v[1], u16[h]);
            }
            with_activation(p.act, [&](auto act) {
#pragma unroll
              for (int i = 0; i < 32; i += 2) set_pair(v[0], i, mul2(activate<act.value>(pair_of(v[0], i)), pair_of(v[1], i)));
            });
            pack32<kF16>(v[0], o16);
            stage_half(stage_out, lane, h, o16);
          }
          write_staged<kPieces>(stage_out, static_cast<uint16_t*>(w.out[0]) + col, (uint32_t)w.ldo * 2u, rows, inside, lane);
          if (p.saved[0]) {
#pragma unroll
            for (int h = 0; h < kBlocks; ++h) stage_half(stage_out, lane, h, g16[h]);
            write_staged<kPieces>(stage_out, static_cast<uint16_t*>(p.saved[0]) + col, (uint32_t)p.lds * 2u, rows, inside, lane);
#pragma unroll
            for (int h = 0; h < kBlocks; ++h) stage_half(stage_out, lane, h, u16[h]);
            write_staged<kPieces>(stage_out, static_cast<uint16_t*>(p.saved[1]) + col, (uint32_t)p.lds * 2u, rows, inside, lane);
          }
        } else {
          if (kEpi == kEpiPlain && w.out_f32) {
#pragma unroll 1
            for (int c = 0; c < kHalf; c += 32) {
              uint32_t v[1][32];
              if (sg.whole) {
                ptx::tmem_ld_32x32b_x32(t0 + (uint32_t)(first_col + c), v[0]);
                ptx::tmem_ld_wait();
                if (c + 32 == kHalf) release();
              } else {
                join(v, c, 0);
              }
              write_f32(w.out[sg.problem], w.ldo, tile_col + c, v[0], rows);
            }
          } else {
#pragma unroll 1
            for (int c = 0; c < kHalf; c += 64) {
              const int64_t col = tile_col + c, at = col + 8 * (lane & 7);  // this lane's piece
              const bool inside = at < w.cols;
              if (residual_ahead && c > 0) fetch_residual(c);  // beside the loads and the activation below
              uint32_t z16[2][16];
              const bool has_saved = kEpi == kEpiLinear && p.saved[0] != nullptr && !kSaveF32;
              uint32_t x2[2][1][32];
              if (sg.whole) {
                ptx::tmem_ld_32x32b_x32(t0 + (uint32_t)(first_col + c), x2[0][0]);
                ptx::tmem_ld_32x32b_x32(t0 + (uint32_t)(first_col + c + 32), x2[1][0]);
                ptx::tmem_ld_wait();
                if (c + 64 == kHalf) release();
              } else {
                join(x2[0], c, 0);
                join(x2[1], c + 32, 0);
              }
              auto add_bias = [&](uint32_t (&v)[32], int h) {
                if (!p.bias) return;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  if (col + 32 * h + 8 * i < w.cols) {
                    Two b[4];
                    widen<kF16>(__ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.bias) + col + 32 * h + 8 * i)), b);
#pragma unroll
                    for (int e = 0; e < 4; ++e) set_pair(v, 8 * i + 2 * e, add2(pair_of(v, 8 * i + 2 * e), b[e]));
                  }
                }
              };
              if constexpr (kSaveF32) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  add_bias(x2[h][0], h);
                  write_f32(p.saved[0], p.lds, col + 32 * h, x2[h][0], rows);
                }
                if (has_residual) fetch_residual(c);
              }
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                uint32_t(&v)[32] = x2[h][0];
                if constexpr (kEpi == kEpiLinear) {
                  if (!kSaveF32) add_bias(v, h);
                  if (has_saved) pack32<kF16>(v, z16[h]);
                  with_activation(p.act, [&](auto act) {
#pragma unroll
                    for (int i = 0; i < 32; i += 2) set_pair(v, i, activate<act.value>(pair_of(v, i)));
                  });
                  if (has_residual) {
                    if (h == 0) {
                      asm volatile("cp.async.wait_all;" ::: "memory");
                      __syncwarp();
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                      Two r[4];
                      widen<kF16>(*staged(stage_out, lane, h * 4 + i), r);
#pragma unroll
                      for (int e = 0; e < 4; ++e) set_pair(v, 8 * i + 2 * e, add2(pair_of(v, 8 * i + 2 * e), r[e]));
                    }
                  }
                }
                uint32_t o16[16];
                pack32<kF16>(v, o16);
                stage_half(stage_out, lane, h, o16);
              }
              write_staged<8>(stage_out, static_cast<uint16_t*>(w.out[sg.problem]) + at, (uint32_t)w.ldo * 2u, rows, inside, lane);
              if (has_saved) {
                stage_half(stage_out, lane, 0, z16[0]);
                stage_half(stage_out, lane, 1, z16[1]);
                write_staged<8>(stage_out, static_cast<uint16_t*>(p.saved[0]) + at, (uint32_t)p.lds * 2u, rows, inside, lane);
              }
            }
          }
        }
      }
    }
    if (kPair && split > 1 && !met) {  // after an abort
      __syncwarp();
      ptx::cluster_sync_all();
    }
    if (kSwap && split > 1) {
      // The parts are all there: the owner adds them in the order of k.
      __syncwarp();
      ptx::cluster_sync_all();
      const uint4* const parts = reinterpret_cast<const uint4*>(base_ptr + (recv - base)) + q * 32 + lane;
      const int groups = (p.chunks * p.box + 7) / 8;
      for (int slot = half; slot * split + part < groups; slot += 2) {
        float sum[kAccs][8];
        uint32_t v[kAccs][8];
#pragma unroll
        for (int t = 0; t < kAccs; ++t)
#pragma unroll
          for (int i = 0; i < 8; ++i) sum[t][i] = 0.0f;
#pragma unroll 2
        for (int r = 0; r < split; ++r) {
#pragma unroll
          for (int t = 0; t < kAccs; ++t) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint4 x = parts[(((r * p.recv_slots + slot) * kAccs + t) * 2 + h) * kTileM];
              sum[t][4 * h] += __uint_as_float(x.x);
              sum[t][4 * h + 1] += __uint_as_float(x.y);
              sum[t][4 * h + 2] += __uint_as_float(x.z);
              sum[t][4 * h + 3] += __uint_as_float(x.w);
            }
          }
        }
#pragma unroll
        for (int t = 0; t < kAccs; ++t)
#pragma unroll
          for (int i = 0; i < 8; ++i) v[t][i] = __float_as_uint(sum[t][i]);
        finish(v, (slot * split + part) * 8);
      }
    }
  }

  if constexpr (kPair) {
    // the leader's MMAs read the follower's shared memory, and its commits arrive there
    __syncwarp();
    ptx::cluster_sync_all();
  }
  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    if constexpr (kPair)
      ptx::tmem_dealloc_pair(tmem_base, p.tmem_cols);
    else
      ptx::tmem_dealloc(tmem_base, p.tmem_cols);
  }
}

}  // namespace
}  // namespace ff
}  // namespace agmm
