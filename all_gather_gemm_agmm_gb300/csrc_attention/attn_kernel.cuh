// attn_kernel.cuh -- the attention kernel: packed prompts, and drafted tokens
// over a paged cache.
//
//   out_i = sum_j softmax_j(scale * q_i . k_j) v_j   over the keys j that row i sees
//
// in one pass over the keys: S = Q K^T for a tile of 128 rows and 128 keys, p =
// 2^(c s - c m + w) with a reference m for each row, O += P V, l += sum p, and O /
// l at the end.  m is the running maximum, but it follows only when it has grown by
// more than 2^8, so the rescaling of O, a round trip through tensor
// memory, is rare after the first keys.
//
// P is an operand of the tensor cores: the weights are rounded to the 16-bit type, and l
// sums them as they are rounded.  In bf16 that is a relative 2^-9 whatever their
// size, and w = 0.  fp16 ends at 65504 and begins at 2^-24, so w = 7: the largest weight
// is 2^(8 + 7), a weight keeps all its bits down to 2^-21 of the reference's, and is lost
// below 2^-32 of it (2^-25 with w = 0, which lost up to 0.39 % of the mass of one key
// and 131072 faint ones).  The factor 2^w is in O as in l and cancels.
//
// One persistent CTA per SM.  Two "streams" of 128 query rows each, so that
// the tensor cores work on one while the other's weights are computed:
//   warps 0-3, 4-7  the softmax of stream 0 and 1: a thread owns a row; S comes
//                   from tensor memory, P goes back there (over S, as 16-bit
//                   pairs) and is the second product's A operand;
//   warp 8          TMA loads of Q tiles and of a ring of K and V tiles;
//   warps 9, 11     issue tcgen05.mma for stream 0 and 1: P V of a tile, then
//                   Q K^T of the next;
//   warp 10         decides the work items.
// Tensor memory (512 columns): S of both streams, O of both.
//
// A work item is paired (the streams hold two row tiles and share every key
// tile) or, where there is one row tile only, alternating (the streams hold the
// same rows and take even and odd key tiles; their sums are joined at the end).
//
// Prompts: an item is up to 256 rows of a sequence for a head, or up to 128 rows
// for two heads of a group.  Trees: a tile packs the heads of a group (row = token *
// group + head), so that each key is read once for all of them.  The key tiles of all
// items are laid out in a line that the CTAs cut into equal parts (struct Line).
// A part that covers only some of an item's keys leaves O, m and l in device
// memory, and agmm_attn_join sums the parts in order.  Prompts that have many items for
// every CTA are not cut: the CTAs draw them from a counter (struct Draw).
//
// What a row does not see never reaches it: its scores are replaced, not
// added to; value rows past the end are cleared in shared memory; and a row whose
// result is not finite, in an item with a value that is not finite and that the row
// does not see, is computed again without it.
//
// Measured: a prompt of 8191 tokens, 32 heads of 128: 369 us back to back under the power
// cap, 1.49 PFLOP/s (341 to 378 us over boxes and builds); the tensor cores were active in 69%
// of the cycles of one launch.  A pair of tiles took 2671 cycles, its products
// need 2048; the likely bound is shared memory's bandwidth under Q K^T and TMA
// (calculated, not counted).  Two contexts of 100000 to 131000 keys, 5 tokens each: 153
// us, 6.2 TB/s: device memory.  Without turns of the two MMA warps the streams fell into
// step: 451 us against 356 us, in one build.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "attn_params.h"
#include "attn_ptx.cuh"

namespace agmm {
namespace {

constexpr int kItemSlots = 2;
constexpr int kDrawAhead = 3;  // key tiles still to be loaded when the next item is asked for
constexpr float kMaxGrowth = 8.0f;  // log2 of how far the weights may grow past the reference's

template <int kD>
struct Layout {
  static constexpr int kHalves = kD / 64;                      // 64-column (128-byte) pieces of a row
  static constexpr uint32_t kTileBytes = kRows * kD * 2;        // a Q, K or V tile
  static constexpr uint32_t kHalfBytes = kRows * 128;           // its 64-column piece
  static constexpr int kStages = kD == 128 ? 5 : 10;
  static constexpr uint32_t kRing = 2 * kTileBytes;
  static constexpr uint32_t kCtl = kRing + kStages * kTileBytes;
  // control block
  static constexpr uint32_t kBars = kCtl;
  static constexpr uint32_t kItems = kCtl + 384;                // kItemSlots x 96 bytes
  static constexpr uint32_t kFlags = kItems + kItemSlots * 96;  // abort, TMEM base, pulse
  static constexpr uint32_t kStats = kFlags + 16;               // [2 streams][128 rows][2] float
  static constexpr size_t kBytes = kStats + 2 * 128 * 2 * 4;
  static_assert(kBytes <= 232448, "more shared memory than a CTA can have");
};

struct Bars {
  uint32_t base;
  int stages;
  __device__ __forceinline__ uint32_t full(int s) const { return base + 8 * s; }
  __device__ __forceinline__ uint32_t empty(int s) const { return base + 8 * (10 + s); }
  __device__ __forceinline__ uint32_t q_full(int x) const { return base + 8 * (20 + x); }
  __device__ __forceinline__ uint32_t q_empty(int x) const { return base + 8 * (22 + x); }
  __device__ __forceinline__ uint32_t s_full(int s) const { return base + 8 * (24 + s); }
  __device__ __forceinline__ uint32_t p_ready(int s, int h) const { return base + 8 * (26 + 2 * s + h); }
  __device__ __forceinline__ uint32_t o_full(int s) const { return base + 8 * (30 + s); }
  __device__ __forceinline__ uint32_t o_free(int s) const { return base + 8 * (32 + s); }
  __device__ __forceinline__ uint32_t item_full(int i) const { return base + 8 * (34 + i); }
  __device__ __forceinline__ uint32_t item_empty(int i) const { return base + 8 * (36 + i); }
  __device__ __forceinline__ uint32_t stats() const { return base + 8 * 38; }
  __device__ __forceinline__ uint32_t drained(int s) const { return base + 8 * (39 + s); }
  // by parity of the stream's tile: the softmax warps wait for it before they
  // know that the tile before had its arrival
  __device__ __forceinline__ uint32_t v_there(int s, uint32_t tile) const { return base + 8 * (41 + 2 * s + (tile & 1u)); }
  __device__ __forceinline__ uint32_t turn(int s) const { return base + 8 * (45 + s); }
  __device__ __forceinline__ uint32_t next_item() const { return base + 8 * 47; }
};

// A work item, written by the scheduler warp.
struct __align__(8) Item {
  int valid;
  int alternate;    // the streams share the rows and take key tiles in turn
  int n[2];         // key tiles of each stream
  int tiles;        // key tiles loaded
  int kv_tile;      // first of them in the sequence
  int kv_len;       // keys of the sequence
  int kv_row;       // prompts: its first key row
  int seq;
  int kv_head, head;  // head: of the tile's first row
  int head_step;      // stream 1 has the head after: 1 (the streams' tokens are the same), else 0
  int q0, q_len;      // the sequence's first query row, and how many
  int off;            // row i sees keys below i + off + 1 (causal, chains); trees: the context
  int tok[2], cnt[2];  // each stream's first token in the sequence, and how many
  int slot;            // -1: the whole result; else where the partial one goes
  int masked_from;     // the first place that not all rows see
};
static_assert(sizeof(Item) <= 96, "item slot too small");

// Ring positions of an item's key and value tiles.  The tiles are loaded in the
// order in which the MMA warp first waits for them: keys run `lead` tiles ahead.
__device__ __forceinline__ int k_index(int t, int lead) { return t + max(0, t - lead); }
__device__ __forceinline__ int v_index(int t, int lead, int tiles) { return t + min(t + 1 + lead, tiles); }

__device__ __forceinline__ int ceil_div(int a, int b) { return (a + b - 1) / b; }

// ------------------------------------------------------------------ scheduler
struct Sequence {
  int q0, q_len, kv_row, kv_len, off;
};

template <bool kPaged>
__device__ __forceinline__ Sequence sequence_of(const AttnParams& p, int s) {
  Sequence x;
  const int64_t a = min(max((int64_t)__ldg(p.starts + s), (int64_t)0), p.tokens);
  const int64_t b = min(max((int64_t)__ldg(p.starts + s + 1), a), p.tokens);
  x.q0 = (int)a;
  x.q_len = (int)(b - a);
  if constexpr (kPaged) {
    const int64_t most = p.table_pages << p.page_shift;
    const int64_t ctx = max(__ldg(p.context_lens + s), 0);
    x.kv_row = 0;
    // nodes past max_nodes are not computed, but a mask may let those before them see them
    const int nodes = min(x.q_len, p.max_nodes);
    x.kv_len = (int)min(ctx + (p.mask ? x.q_len : nodes), most);
    x.q_len = nodes;
    x.off = (int)min(ctx, most);
  } else {
    const int64_t c = min(max((int64_t)__ldg(p.kv_starts + s), (int64_t)0), p.kv_tokens);
    const int64_t d = min(max((int64_t)__ldg(p.kv_starts + s + 1), c), p.kv_tokens);
    x.kv_row = (int)c;
    x.kv_len = (int)(d - c);
    x.off = x.kv_len - x.q_len;
  }
  return x;
}

// Prompts: the key tiles that the rows before token `end` need.
__device__ __forceinline__ int key_tiles(const AttnParams& p, const Sequence& x, int end) {
  return ceil_div(p.causal ? min(x.kv_len, max(end + x.off, 0)) : x.kv_len, kKeys);
}

// The work is laid out in a line: sequences, in each its sets of row tiles (one
// or two tiles), for each the heads, for each item its key tiles.  In front of
// its tiles an item has kItemCost places for what it takes besides them (32 decode
// steps over 150 to 8100 keys, in one build: 61.4 us with 1 place, 55.9 with 2, 53.6 with 4,
// 55.6 with 6; 56.3 us now, with 4).  The line is cut into a part for every CTA, equal but for cuts that would leave
// less than p.min_tiles of an item on one side: those move to the item's edge.
constexpr int kItemCost = 4;

struct Spot {
  int seq, set, head;  // head: among the set's items
  int len;             // key tiles of each (at least 1)
  int64_t start;       // the item's first place
};

template <bool kPaged>
struct Line {
  const AttnParams& p;
  int lane;
  int64_t total;
  int parts;  // CTAs that have work: no two cuts are the same place

  __device__ __forceinline__ int sets(const Sequence& x) const { return ceil_div(x.q_len, 2 * p.tile_tokens); }
  __device__ __forceinline__ bool single(const Sequence& x, int set) const {
    return x.q_len - set * 2 * p.tile_tokens <= p.tile_tokens;
  }
  // Items of a row set: a key head each (trees), or a query head each.
  __device__ __forceinline__ int heads() const { return kPaged ? p.kv_heads : p.q_heads; }
  __device__ __forceinline__ int length(const Sequence& x, int set) const {
    if (kPaged) return ceil_div(x.kv_len, kKeys);
    return max(1, key_tiles(p, x, min(x.q_len, (set + 1) * 2 * p.tile_tokens)));
  }
  __device__ __forceinline__ int64_t places(int seq) const {
    if (seq >= p.sequences) return 0;
    const Sequence x = sequence_of<kPaged>(p, seq);
    int64_t sum = 0;
    const int n = sets(x);
#pragma unroll 1
    for (int set = 0; set < n; ++set) sum += (int64_t)heads() * (length(x, set) + kItemCost);
    return sum;
  }
  __device__ __forceinline__ void init() {
    lane = threadIdx.x & 31;
    int64_t sum = 0;
#pragma unroll 1
    for (int s = lane; s < p.sequences; s += 32) sum += places(s);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    total = sum;
    parts = (int)min((int64_t)gridDim.x, total);
  }
  // The CTA whose part begins at or before place u, uncut by items.
  __device__ __forceinline__ int cta_of(int64_t u) const { return (int)(((u + 1) * parts - 1) / total); }

  // The item of place u (0 <= u < total).
  __device__ __noinline__ Spot find(int64_t u) const {
    Spot at = {};
    int64_t first = 0;  // first place of the sequence
#pragma unroll 1
    for (int s0 = 0; s0 < p.sequences; s0 += 32) {
      const int64_t mine = places(s0 + lane);
      int64_t run = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, run, o);
        if (lane >= o) run += y;
      }
      const uint32_t past = __ballot_sync(0xffffffffu, first + run > u);
      if (past) {
        const int j = __ffs(past) - 1;
        at.seq = s0 + j;
        first += __shfl_sync(0xffffffffu, run - mine, j);
        break;
      }
      first += __shfl_sync(0xffffffffu, run, 31);
    }
    const Sequence x = sequence_of<kPaged>(p, at.seq);
    for (;;) {
      at.len = length(x, at.set);
      const int each = at.len + kItemCost;
      if (u < first + (int64_t)heads() * each || at.set + 1 >= sets(x)) {
        at.head = (int)((u - first) / each);
        at.start = first + (int64_t)at.head * each;
        return at;
      }
      first += (int64_t)heads() * each;
      ++at.set;
    }
  }
  // Where the part of CTA c begins, and the item that lies there.
  __device__ __forceinline__ int64_t cut(int c, Spot& at) const {
    if (c >= parts) return total;
    const int64_t u = total * c / parts;
    at = find(u);
    const int t = (int)(u - at.start) - kItemCost;
    if (t < p.min_tiles) return at.start;
    if (at.len - t < p.min_tiles) return at.start + kItemCost + at.len;
    return u;
  }
};

// Prompts with many items for each CTA: whole items, drawn one at a time from a
// counter, those of the last row set of their sequence first (of one sequence they see
// the most keys), and of one such level the sets of two tiles first, then by sequence,
// then by head.  No result makes a round trip through memory, and what the line's cost
// model misses evens out.  Keys before the queries are not looked at: a short piece behind a
// long prefix is drawn among the last, and its items are one CTA's each.
struct Draw {
  const AttnParams& p;
  int lane;
  int level, base, pairs, singles;  // the level's items begin at `base`; sequences with a two-tile, a one-tile set there
  int items, next;

  // Row sets of a sequence; `single`: the last one is a tile that has two heads to an item.
  __device__ __forceinline__ int sets_of(int s, bool& single) const {
    single = false;
    if (s >= p.sequences) return 0;
    const int64_t a = min(max((int64_t)__ldg(p.starts + s), (int64_t)0), p.tokens);
    const int64_t b = min(max((int64_t)__ldg(p.starts + s + 1), a), p.tokens);
    const int n = (int)((b - a + 2 * kRows - 1) / (2 * kRows));
    single = p.pair_heads && n > 0 && b - a <= (int64_t)(2 * n - 1) * kRows;
    return n;
  }
  __device__ __forceinline__ int level_items() const { return pairs * p.q_heads + singles * (p.q_heads / 2); }
  __device__ __forceinline__ void init() {
    lane = threadIdx.x & 31;
    int most = 0;
    int64_t sum = 0;
#pragma unroll 1
    for (int s = lane; s < p.sequences; s += 32) {
      bool single;
      const int n = sets_of(s, single);
      most = max(most, n);
      sum += (int64_t)n * p.q_heads - (single ? p.q_heads - p.q_heads / 2 : 0);
    }
    // The host bounds the items of starts that do not fall.  Starts that fall can stand for
    // more rows than there are, and for more items than can be counted: none is done then.
    const int64_t total = ((int64_t)__reduce_add_sync(0xffffffffu, (unsigned)(sum >> 16 & 0x3ffffff)) << 16) +
                          __reduce_add_sync(0xffffffffu, (unsigned)(sum & 0xffff));
    const bool countable = !__any_sync(0xffffffffu, sum >> 42) && total < kMostItems;
    items = countable ? (int)total : 0;
    level = __reduce_max_sync(0xffffffffu, most);
    base = pairs = singles = 0;
    next = (int)blockIdx.x - (int)gridDim.x;  // the first item is this CTA's number
  }
  // The next item, of Spot's seq, set and head (among the set's); false: none.
  __device__ __noinline__ bool draw(Spot& at) {
    if (next < 0) {
      next += gridDim.x;
    } else {
      // the CTA that draws the last number puts the counter back to zero
      if (lane == 0) {
        next = atomicAdd(p.counter, 1);
        if (next == items - 1) atomicExch(p.counter, 0);
        next += gridDim.x;
      }
      next = __shfl_sync(0xffffffffu, next, 0);
    }
    if (next >= items) return false;
    while (next >= base + level_items()) {
      base += level_items();
      --level;
      int c = 0, d = 0;
#pragma unroll 1
      for (int s = lane; s < p.sequences; s += 32) {
        bool single;
        const int n = sets_of(s, single);
        const bool one = single && n == level + 1;
        c += n > level && !one;
        d += one;
      }
      pairs = __reduce_add_sync(0xffffffffu, c);
      singles = __reduce_add_sync(0xffffffffu, d);
    }
    at.set = level;
    int left = next - base;
    const bool want_single = left >= pairs * p.q_heads;
    if (want_single) left -= pairs * p.q_heads;
    const int heads = want_single ? p.q_heads / 2 : p.q_heads;
    int rank = left / heads;
    at.head = left - rank * heads;
#pragma unroll 1
    for (int s0 = 0; s0 < p.sequences; s0 += 32) {
      bool single;
      const int n = sets_of(s0 + lane, single);
      const bool mine = n > level && (single && n == level + 1) == want_single;
      const uint32_t has = __ballot_sync(0xffffffffu, mine);
      const uint32_t here = __ballot_sync(0xffffffffu, mine && __popc(has & ((1u << lane) - 1u)) == rank);
      if (here) {
        at.seq = s0 + __ffs(here) - 1;
        return true;
      }
      rank -= __popc(has);
    }
    return false;
  }
};

// Key tiles [t0, t1) of the item at a spot.
template <bool kPaged>
__device__ __noinline__ Item make_item(const AttnParams& p, const Line<kPaged>& line, const Sequence& x, const Spot& at, int t0,
                                       int t1) {
  Item it = {};
  it.valid = 1;
  it.slot = -1;
  it.seq = at.seq;
  it.q0 = x.q0;
  it.q_len = x.q_len;
  it.kv_len = x.kv_len;
  it.kv_row = x.kv_row;
  it.off = x.off;
  it.kv_tile = t0;
  const int tok = at.set * 2 * p.tile_tokens;
  const bool single = line.single(x, at.set);
  it.tok[0] = it.tok[1] = tok;
  it.cnt[0] = it.cnt[1] = min(p.tile_tokens, x.q_len - tok);
  if (!single) {
    it.tok[1] = tok + p.tile_tokens;
    it.cnt[1] = min(p.tile_tokens, x.q_len - it.tok[1]);
  }
  it.alternate = single;
  if (kPaged) {
    it.kv_head = at.head;
    it.head = at.head * p.group;
    it.n[0] = it.n[1] = t1 - t0;
    it.masked_from = p.mask ? min(x.off, x.kv_len) : min(x.kv_len, tok + x.off + 1);
  } else {
    if (single && p.pair_heads) {
      it.alternate = 0;
      it.head_step = 1;
    }
    it.head = at.head << it.head_step;
    it.kv_head = it.head / p.group;
    it.n[0] = max(0, min(key_tiles(p, x, it.tok[0] + it.cnt[0]), t1) - t0);
    it.n[1] = max(0, min(key_tiles(p, x, it.tok[1] + it.cnt[1]), t1) - t0);
    it.masked_from = p.causal ? min(x.kv_len, max(tok + x.off + 1, 0)) : x.kv_len;
  }
  it.tiles = max(it.n[0], it.n[1]);
  if (it.alternate) {  // stream 0 takes the even tiles
    it.n[0] = (it.tiles + 1) / 2;
    it.n[1] = it.tiles / 2;
  }
  return it;
}

template <bool kPaged>
__device__ __forceinline__ void scheduler(const AttnParams& p, const Bars& bars, Item* slots, const Waiter& wait) {
  Line<kPaged> line{p};
  Draw drawn{p};
  const int lane = threadIdx.x & 31;
  const bool by_draw = !kPaged && p.by_draw;
  int* const join = p.joins + (size_t)blockIdx.x * kJoinInts;
  if (lane == 0) join[0] = 0;
  int64_t u = 0, end = 0;
  Spot at = {};
  Sequence x = {};
  if (by_draw) {
    drawn.init();
  } else {
    line.init();
    if ((int)blockIdx.x < line.parts) {
      end = line.cut(blockIdx.x + 1, at);
      u = line.cut(blockIdx.x, at);
      x = sequence_of<kPaged>(p, at.seq);
    }
  }
  int k = 0;
  for (bool more = true; more;) {
    // An item is drawn when the last loads of the one before come up: a CTA that
    // drew further ahead would hold items from the others.
    if (k > 0 && !wait.compact(bars.next_item(), (uint32_t)(k - 1) & 1u, 100000 + k)) return;
    if (k >= kItemSlots && !wait.compact(bars.item_empty(k % kItemSlots), (uint32_t)(k / kItemSlots - 1) & 1u, k)) return;
    Item it = {};
    if (by_draw) {
      more = drawn.draw(at);
      if (more) {
        x = sequence_of<kPaged>(p, at.seq);
        it = make_item(p, line, x, at, 0, line.length(x, at.set));
      }
    } else {
      // the item at u, where it is not one that ends there
      while (u < end && u >= at.start + kItemCost + at.len) {
        at.start += kItemCost + at.len;
        if (++at.head < line.heads()) continue;
        at.head = 0;
        if (++at.set >= line.sets(x)) {
          at.set = 0;
          do
            x = sequence_of<kPaged>(p, ++at.seq);
          while (x.q_len == 0);  // the line goes on: there is one more
        }
        at.len = line.length(x, at.set);
      }
      more = u < end;
      if (more) {
        const int64_t tiles0 = at.start + kItemCost;
        const int t0 = u <= at.start ? 0 : (int)(u - tiles0);
        const int t1 = (int)min((int64_t)at.len, end - tiles0);
        const bool whole = t0 == 0 && t1 == at.len;
        u = tiles0 + t1;
        it = make_item(p, line, x, at, t0, t1);
        if (!whole) it.slot = 2 * (int)blockIdx.x + (t0 == 0);
        if (!whole && t0 == 0 && lane == 0) {
          // this CTA holds the first keys of an item that goes on: the record of its join
          join[1] = x.q0 + it.tok[0];
          join[2] = it.cnt[0] * p.pack;
          join[3] = it.head;
          join[4] = line.cta_of(tiles0 + at.len - p.min_tiles);  // the CTA of the item's last tiles
          join[5] = x.q0 + it.tok[1];
          join[6] = it.alternate ? 0 : it.cnt[1] * p.pack;
          join[7] = it.head + it.head_step;
          join[0] = 1;
        }
      }
    }
    if (lane == 0) {
      slots[k % kItemSlots] = it;
      ptx::mbar_arrive(bars.item_full(k % kItemSlots));
    }
    ++k;
  }
}

// ------------------------------------------------------------------- producer
template <int kD, bool kPaged>
__device__ __forceinline__ void producer(const AttnParams& p, const Bars& bars, const Item* slots, uint32_t smem,
                                         const Waiter& wait) {
  using L = Layout<kD>;
  const int lane = threadIdx.x & 31;
  uint32_t fills = 0;
  uint32_t q_uses[2] = {0, 0};
  bool drop = p.test_drop_first_load != 0;
  const int page_rows = kPaged ? min(1 << p.page_shift, kKeys) : kKeys;
  const int pages_per_tile = kKeys / page_rows;
  bool ok = true;
  for (int k = 0; ok; ++k) {
    const int slot = k % kItemSlots;
    if (!wait.compact(bars.item_full(slot), (uint32_t)(k / kItemSlots) & 1u, k)) break;
    const Item it = slots[slot];
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(bars.item_empty(slot));
    if (!it.valid) break;
    if (it.tiles <= kDrawAhead && lane == 0) ptx::mbar_arrive(bars.next_item());
    if (it.tiles == 0) continue;
    for (int s = 0; s < 2 && ok; ++s) {
      if (s == 1 && it.alternate) break;
      if (it.n[s] == 0) continue;
      ok = wait.compact(bars.q_empty(s), (q_uses[s] & 1u) ^ 1u, 1000 + s);
      if (!ok) break;
      ++q_uses[s];
      if (lane == 0) {
        const uint32_t bytes = (uint32_t)(p.tile_tokens * p.pack) * 128u;
        ptx::mbar_arrive_expect_tx(bars.q_full(s), bytes * L::kHalves);
#pragma unroll
        for (int h = 0; h < L::kHalves; ++h)
          ptx::tma_load_3d(smem + s * L::kTileBytes + h * L::kHalfBytes, &p.qmap, bars.q_full(s), h * 64,
                           it.head + s * it.head_step, it.q0 + it.tok[s]);
      }
      __syncwarp();
    }
    if (!ok) break;
    // loads in ring order: key tile t + lead, then value tile t
    const int lead = it.alternate ? 2 : 1;
#pragma unroll 1
    for (int f = -2 * lead; f < 2 * it.tiles && ok; ++f) {
      const bool value = f & 1;
      const int t = value ? f >> 1 : (f >> 1) + lead;
      if (t < 0 || t >= it.tiles) continue;
      if (value && t == it.tiles - 1 - kDrawAhead && lane == 0) ptx::mbar_arrive(bars.next_item());
      const CUtensorMap* const map = value ? &p.vmap : &p.kmap;
      const int st = (int)(fills % L::kStages);
      ok = wait.compact(bars.empty(st), ((fills / L::kStages) & 1u) ^ 1u, 2000 + st);
      if (!ok) break;
      ++fills;
      if (drop) {  // test hook
        drop = false;
        continue;
      }
      const uint32_t dst = smem + L::kRing + st * L::kTileBytes, bar = bars.full(st);
      const int place = (it.kv_tile + t) * kKeys;
      if constexpr (kPaged) {
        const int mine = place + lane * page_rows;
        const bool there = lane < pages_per_tile && mine < it.kv_len;
        const int n = __popc(__ballot_sync(0xffffffffu, there));
        int page = 0;
        if (there) page = __ldg(p.page_table + it.seq * p.table_stride + (mine >> p.page_shift));
        if (lane == 0) ptx::mbar_arrive_expect_tx(bar, (uint32_t)(n * page_rows) * 128u * L::kHalves);
        __syncwarp();
        if (there) {
#pragma unroll
          for (int h = 0; h < L::kHalves; ++h)
            ptx::tma_load_4d(dst + h * L::kHalfBytes + lane * page_rows * 128, map, bar, h * 64,
                             mine & ((1 << p.page_shift) - 1), it.kv_head, page);
        }
      } else if (lane == 0) {
        ptx::mbar_arrive_expect_tx(bar, L::kTileBytes);
#pragma unroll
        for (int h = 0; h < L::kHalves; ++h)
          ptx::tma_load_4d(dst + h * L::kHalfBytes, map, bar, h * 64, it.kv_row + place, it.kv_head, 0);
      }
      __syncwarp();
    }
  }
  if (*wait.abort) {
    // copies in flight end before the CTA does
    for (int st = 0; st < L::kStages; ++st) {
      if (p.test_drop_first_load && st == 0) continue;  // never filled
      if (fills > (uint32_t)st) {  // its last fill
        const uint32_t last = (fills - 1 - st) / L::kStages;
        wait.drain(bars.full(st), last & 1u);
      }
    }
    for (int s = 0; s < 2; ++s)
      if (q_uses[s]) wait.drain(bars.q_full(s), (q_uses[s] - 1) & 1u);
  }
}

// ------------------------------------------------------------------------ MMA
// A place in the ring: stage, and the parity of its full barrier's phase.
template <int kStages>
struct RingPos {
  int stage = 0;
  uint32_t parity = 0;
  __device__ __forceinline__ RingPos after(int n) const {
    RingPos x = *this;
    x.stage += n;
    if (x.stage >= kStages) {
      x.stage -= kStages;
      x.parity ^= 1u;
    }
    return x;
  }
};

// The products of stream kS.  Each stream has a warp of its own: a warp can run
// only a product or two ahead of the tensor cores, so what it spends on waits
// and commits is lost to them unless another warp's products run meanwhile.
//
// The two take turns, a tile each: left to themselves they fall into step, both
// streams' weights being computed while the tensor cores wait and the other way
// round.
//
// The warp runs converged and one elected lane issues; the operands of
// tcgen05.mma are uniform registers, so everything that they come from is
// uniform too: constants, the kernel's shared-memory address (the CTA has all of
// tensor memory, from address 0), and loop counters whose bounds are broadcast.
//
// Both warps see every fill of every stage, used or not, and a stage is free
// when both have let go of it: neither can take one fill for another.
template <int kD, bool kF16, int kS>
__device__ __forceinline__ void mma_issuer(const Bars& bars, const Item* slots, uint32_t smem, const Waiter& wait) {
  using L = Layout<kD>;
  using Pos = RingPos<L::kStages>;
  constexpr uint32_t kIdescS = ptx::idesc_f16kind_f32(kRows, kKeys, false, false, kF16);
  constexpr uint32_t kIdescO = ptx::idesc_f16kind_f32(kRows, kD, false, true, kF16);
  constexpr uint32_t kTmemS = kS * kKeys, kTmemO = 2 * kKeys + kS * kD;
  const bool leader = ptx::elect_one();
  Pos pos;  // of the next load in ring order
  uint32_t q_parity = 0, o_parity = 1;     // of the next phases (q: bit x of Q tile x)
  uint32_t steps = 0;                      // the stream's tiles so far
  uint32_t turn_parity = kS == 0 ? 1 : 0;             // stream 0 has the first turn
  bool ok = true;
  for (int k = 0; ok; ++k) {
    const int slot = k % kItemSlots;
    if (!wait.compact(bars.item_full(slot), (uint32_t)(k / kItemSlots) & 1u, k)) break;
    const Item& it = slots[slot];
    const int valid = __shfl_sync(0xffffffffu, it.valid, 0), alternate = __shfl_sync(0xffffffffu, it.alternate, 0);
    const int tiles = __shfl_sync(0xffffffffu, it.tiles, 0), mine = __shfl_sync(0xffffffffu, it.n[kS], 0);
    const uint32_t q_used = __shfl_sync(0xffffffffu, (it.n[0] > 0 ? 1u : 0u) | (!it.alternate && it.n[1] > 0 ? 2u : 0u), 0);
    if (leader) ptx::mbar_arrive(bars.item_empty(slot));
    if (!valid) break;
    if (tiles == 0) continue;
    const int x = alternate ? 0 : kS;  // this stream's Q tile
    for (int y = 0; y < 2 && ok; ++y)
      if (q_used >> y & 1u) {
        ok = wait.compact(bars.q_full(y), q_parity >> y & 1u, 1000 + y);
        if (ok && leader && (y != x || mine == 0)) ptx::mbar_arrive(bars.q_empty(y));  // not for this stream
      }
    q_parity ^= q_used;
    // At t the ring holds key tile t + lead, then value tile t.  This stream takes
    // the first `mine` tiles, or every second one.
    const int lead = alternate ? 2 : 1;
    int done_k = 0, done_v = 0;
#pragma unroll 1
    for (int t = -lead; t < tiles && ok; ++t) {
      const bool has_k = t + lead < tiles, has_v = t >= 0;
      const Pos at_k = pos, at_v = pos.after(has_k);
      pos = at_v.after(has_v);
      const bool own = alternate ? (t & 1) == kS : true;
      const bool with_k = has_k && own && done_k < mine, with_v = has_v && own && done_v < mine;
      if (has_v) {
        if (!(ok = wait.compact(bars.full(at_v.stage), at_v.parity, 3000 + at_v.stage))) break;
        if (!with_v && leader) ptx::mbar_arrive(bars.empty(at_v.stage));
      }
      if (has_k) {
        if (!(ok = wait.compact(bars.full(at_k.stage), at_k.parity, 2000 + at_k.stage))) break;
        if (!with_k && leader) ptx::mbar_arrive(bars.empty(at_k.stage));
      }
      if (with_v) {
        // O += P V, in halves of the keys as their weights come.  The softmax warps
        // learn here that the value tile is there.
        if (leader) ptx::mbar_arrive(bars.v_there(kS, steps));
        if (done_v == 0) {
          if (!(ok = wait.compact(bars.o_free(kS), o_parity, 4000 + kS))) break;
          o_parity ^= 1u;
        }
        const uint64_t b = ptx::smem_desc_sw128(smem + L::kRing + at_v.stage * L::kTileBytes, L::kHalfBytes, 1024u);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (!(ok = wait.compact(bars.p_ready(kS, h), steps & 1u, 5000 + 2 * kS + h))) break;
          if (h == 0 && !(ok = wait.compact(bars.turn(kS), turn_parity, 5500 + kS))) break;
          ptx::tc_fence_after();
          if (leader) {
#pragma unroll
            for (int kk = h * kKeys / 32; kk < (h + 1) * kKeys / 32; ++kk)
              ptx::mma_f16_ts(kTmemO, kTmemS + kk * 8, b + (uint64_t)(kk * 2048u >> 4), kIdescO, done_v > 0 || kk > 0);
          }
          __syncwarp();
        }
        if (!ok) break;
        ++steps;
        ++done_v;
        if (leader) {
          ptx::mma_commit(bars.empty(at_v.stage));
          if (done_v == mine) ptx::mma_commit(bars.o_full(kS));
        }
        __syncwarp();
      }
      if (own && has_v && !with_v && !(ok = wait.compact(bars.turn(kS), turn_parity, 5600 + kS))) break;
      if (with_k) {
        // S = Q K^T
        ptx::tc_fence_after();
        ++done_k;
        if (leader) {
          const uint64_t a = ptx::smem_desc_sw128(smem + x * L::kTileBytes, 16u, 1024u);
          const uint64_t b = ptx::smem_desc_sw128(smem + L::kRing + at_k.stage * L::kTileBytes, 16u, 1024u);
#pragma unroll
          for (int kk = 0; kk < kD / 16; ++kk) {
            // 16 columns further: 32 bytes in the 128-byte row, then the next 64-column piece
            const uint64_t step = (uint64_t)((kk / 4) * L::kHalfBytes + (kk % 4) * 32u) >> 4;
            ptx::mma_bf16(kTmemS, a + step, b + step, kIdescS, kk > 0);
          }
          // This barrier also says that the product before it, P V of the tile
          // before, has ended.
          ptx::mma_commit(bars.s_full(kS));
          ptx::mma_commit(bars.empty(at_k.stage));
          if (done_k == mine) ptx::mma_commit(bars.q_empty(x));
        }
        __syncwarp();
      }
      if (own && has_v) {
        turn_parity ^= 1u;
        if (leader) ptx::mbar_arrive(bars.turn(kS ^ 1));
      }
    }
    if (kS == 1 && alternate && (tiles & 1) && ok) {
      // stream 0 had a tile more: this turn is passed on
      ok = wait.compact(bars.turn(1), turn_parity, 5700);
      turn_parity ^= 1u;
      if (leader) ptx::mbar_arrive(bars.turn(0));
    }
  }
  // every product issued has ended before the CTA does
  if (leader) ptx::mma_commit(bars.drained(kS));
  __syncwarp();
  wait.drain(bars.drained(kS), 0);
}

// -------------------------------------------------------------------- softmax
template <bool kF16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (kF16) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}

// What is added to c s for the exponent of a weight.  A row that has seen nothing has no reference.
template <bool kF16>
__device__ __forceinline__ float weight_shift(float m, float c) {
  return (m == -INFINITY ? 0.0f : -m * c) + (kF16 ? 7.0f : 0.0f);
}

template <bool kF16>
__device__ __forceinline__ float value16(uint16_t b) {
  if constexpr (kF16)
    return __half2float(__ushort_as_half(b));
  else
    return __bfloat162float(__ushort_as_bfloat16(b));
}

// Bits [at, at + 32) of a row of mask words; at >= 0.
__device__ __forceinline__ uint32_t mask_window(const int64_t* row, int words, int at) {
  const int w = at >> 6, sh = at & 63;
  if (w >= words) return 0;
  uint64_t v = (uint64_t)__ldg(row + w) >> sh;
  if (sh > 32 && w + 1 < words) v |= (uint64_t)__ldg(row + w + 1) << (64 - sh);
  return (uint32_t)v;
}

__device__ __forceinline__ uint32_t low_bits(int n) { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u; }

// A thread's row of an item.
struct Row {
  bool there;          // one of the tile's tokens, not padding
  int token;           // in its sequence
  int limit;           // the first place that it does not see, without a mask
  const int64_t* mask;  // its mask words, or null
};

template <bool kPaged>
__device__ __forceinline__ Row row_of(const AttnParams& p, const Item& it, int s, int r) {
  Row x;
  x.there = r < it.cnt[s] * p.pack;
  x.token = it.tok[s] + (p.pack == 1 ? r : r / p.pack);
  x.limit = it.kv_len;
  x.mask = nullptr;
  if (kPaged && p.mask != nullptr) {
    if (x.there)
      x.mask = p.mask + (int64_t)(it.q0 + x.token) * p.mask_words;
    else
      x.limit = 0;
  } else if (p.causal) {
    x.limit = min(x.limit, max(x.token + it.off + 1, 0));
  }
  return x;
}

// Which of the places [place, place + 32) a row sees.
__device__ __forceinline__ uint32_t seen32(const Item& it, const Row& row, int words, int place) {
  if (row.mask == nullptr) return low_bits(row.limit - place);
  uint32_t bits = low_bits(it.off - place);
  const int node = place - it.off;
  if (node >= 0)
    bits = mask_window(row.mask, words, node);
  else if (node > -32)
    bits |= mask_window(row.mask, words, 0) << -node;
  return bits & low_bits(it.kv_len - place);
}

template <bool kF16>
__device__ __forceinline__ bool not_finite(uint16_t b) {
  constexpr uint16_t kExp = kF16 ? 0x7c00u : 0x7f80u;
  return (b & kExp) == kExp;
}

// Offset of (place, column 0) in keys (or values) with these strides; -1: a page
// outside the cache, which reads as zeros.
template <bool kPaged>
__device__ __forceinline__ int64_t row_offset(const AttnParams& p, const Item& it, int place, int64_t ts, int64_t hs, int64_t ps) {
  if constexpr (kPaged) {
    const int64_t page = __ldg(p.page_table + it.seq * p.table_stride + (place >> p.page_shift));
    if (page < 0 || page >= p.pages) return -1;
    return page * ps + (int64_t)(place & ((1 << p.page_shift) - 1)) * ts + it.kv_head * hs;
  } else {
    return ((int64_t)it.kv_row + place) * ts + it.kv_head * hs;
  }
}

// The exact results of rows whose products came out not finite (`rows`: lanes of
// this warp).  In a tile that a row does not see all of, a value that is not finite
// times a weight of zero is not zero.  Where there is such a value that the row
// does not see, its result is computed again, key by key, with the weights that it had
// (m, l); else it stands.  A warp takes a row at a time: a lane takes a key's
// score, then some columns of all 32 keys' values.  Slow and rare: 8191 tokens, 32 heads
// with one such value at key 127 take 2.1 ms, at key 8000 54 ms, and 0.35 ms without.
// Loads are 4 to 16 bytes, in the order that the sums need (2 bytes at a time: 7.6 and
// 146 ms).  Unrolled by 8 it took 48 ms (57 in that build), but prompts without such a value, which never
// come here, 348 us instead of 341.  Other warps may wait for this one longer than a wait
// lasts (2 s are reached at about 300 thousand keys): it shows them that it goes on.
template <int kD, bool kF16, bool kPaged>
__device__ __noinline__ void repair_rows(const AttnParams* p, const Item* it, const Waiter* wait, int s, uint32_t rows, float m,
                                         float l, int col0, int col1, uint16_t* out, float* part) {
  constexpr int kN = kD / 32;
  const int lane = threadIdx.x & 31;
  const int begin = it->kv_tile * kKeys, end = min(it->kv_len, (it->kv_tile + it->tiles) * kKeys);
#pragma unroll 1
  for (; rows; rows &= rows - 1) {
    const int from = __ffs(rows) - 1;
    const Row row = row_of<kPaged>(*p, *it, s, (threadIdx.x & 96) + from);
    bool found = false;
    wait->beat();
#pragma unroll 1
    for (int place = max(it->masked_from / kKeys * kKeys, begin) + lane; place < end; place += 32) {
      if (seen32(*it, row, p->mask_words, place) & 1u) continue;
      const int64_t at = row_offset<kPaged>(*p, *it, place, p->v_ts, p->v_hs, p->v_ps);
      if (at < 0) continue;
#pragma unroll 2
      for (int c = col0; c < col1; c += 8) {
        const uint4 x = *reinterpret_cast<const uint4*>(p->v + at + c);
        const uint32_t xw[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) found |= not_finite<kF16>((uint16_t)xw[e]) | not_finite<kF16>((uint16_t)(xw[e] >> 16));
      }
    }
    if (!__any_sync(0xffffffffu, found)) continue;
    const float row_m = __shfl_sync(0xffffffffu, m, from), row_l = __shfl_sync(0xffffffffu, l, from);
    const float shift = weight_shift<kF16>(row_m, p->scale_log2);
    const int head = it->head + s * (it->alternate ? 0 : it->head_step) +
                     (p->pack == 1 ? 0 : (threadIdx.x & 96) + from - (row.token - it->tok[s]) * p->pack);
    const uint16_t* const q = p->q + (int64_t)(it->q0 + row.token) * p->q_ts + head * p->q_hs;
    float o[kN];
#pragma unroll
    for (int e = 0; e < kN; ++e) o[e] = 0.0f;
#pragma unroll 1
    for (int place0 = begin; place0 < end; place0 += 32) {
      if (__any_sync(0xffffffffu, *wait->abort != 0)) return;
      wait->beat();
      float w = 0.0f;
      int64_t v_at = -1;
      if (place0 + lane < end && (seen32(*it, row, p->mask_words, place0 + lane) & 1u)) {
        const int64_t k_at = row_offset<kPaged>(*p, *it, place0 + lane, p->k_ts, p->k_hs, p->k_ps);
        v_at = row_offset<kPaged>(*p, *it, place0 + lane, p->v_ts, p->v_hs, p->v_ps);
        float dot = 0.0f;
        if (k_at >= 0) {
#pragma unroll 2
          for (int c = 0; c < kD; c += 8) {
            const uint4 a = *reinterpret_cast<const uint4*>(q + c), b = *reinterpret_cast<const uint4*>(p->k + k_at + c);
            const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              dot = fmaf(value16<kF16>((uint16_t)aw[e]), value16<kF16>((uint16_t)bw[e]), dot);
              dot = fmaf(value16<kF16>((uint16_t)(aw[e] >> 16)), value16<kF16>((uint16_t)(bw[e] >> 16)), dot);
            }
          }
        }
        w = value16<kF16>((uint16_t)pack2<kF16>(ptx::exp2_approx(fmaf(dot, p->scale_log2, shift)), 0.0f));
      }
#pragma unroll 1
      for (int j0 = 0; j0 < 32; j0 += 4) {
        uint32_t x[4][kN / 2];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int64_t at = __shfl_sync(0xffffffffu, v_at, j0 + j);
#pragma unroll
          for (int e = 0; e < kN / 2; ++e)
            x[j][e] = at < 0 ? 0u : *reinterpret_cast<const uint32_t*>(p->v + at + lane * kN + 2 * e);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const bool seen = __shfl_sync(0xffffffffu, v_at, j0 + j) >= 0;
          const float wj = __shfl_sync(0xffffffffu, w, j0 + j);
#pragma unroll
          for (int e = 0; e < kN / 2; ++e) {
            if (!seen) continue;
            o[2 * e] = fmaf(wj, value16<kF16>((uint16_t)x[j][e]), o[2 * e]);
            o[2 * e + 1] = fmaf(wj, value16<kF16>((uint16_t)(x[j][e] >> 16)), o[2 * e + 1]);
          }
        }
      }
    }
    uint16_t* const row_out = reinterpret_cast<uint16_t*>(__shfl_sync(0xffffffffu, reinterpret_cast<uintptr_t>(out), from));
    float* const row_part = reinterpret_cast<float*>(__shfl_sync(0xffffffffu, reinterpret_cast<uintptr_t>(part), from));
    if (lane * kN < col0 || lane * kN >= col1) continue;
#pragma unroll
    for (int e = 0; e < kN; ++e) {
      if (row_part)
        row_part[lane * kN + e] = o[e];
      else
        row_out[lane * kN + e] = (uint16_t)pack2<kF16>(row_l == 0.0f ? 0.0f : o[e] / row_l, 0.0f);
    }
  }
}

// The largest of 128 scores, in eight chains.
__device__ __forceinline__ float row_max(const uint32_t (&v)[4][32]) {
  float top[8];
#pragma unroll
  for (int w = 0; w < 8; ++w) top[w] = fmaxf(__uint_as_float(v[w & 3][w >> 2]), __uint_as_float(v[w & 3][2 + (w >> 2)]));
#pragma unroll
  for (int e = 4; e < 32; e += 4)
#pragma unroll
    for (int w = 0; w < 8; ++w)
      top[w] = ptx::max3(top[w], __uint_as_float(v[w & 3][e + (w >> 2)]), __uint_as_float(v[w & 3][e + 2 + (w >> 2)]));
  return ptx::max3(ptx::max3(top[0], top[1], top[2]), ptx::max3(top[3], top[4], top[5]), fmaxf(top[6], top[7]));
}

// The weights 2^(c s + shift) of 64 scores as 16-bit pairs, and their sums.  The
// sums are of the rounded weights, those that multiply V: a row with one weight
// that counts gives exactly its value.
template <bool kF16>
__device__ __forceinline__ void weights(const uint32_t (&a)[32], const uint32_t (&b)[32], float c, float shift, uint32_t (&pk)[32],
                                        float (&sum)[4]) {
  const uint64_t c2 = ptx::pair(c, c), shift2 = ptx::pair(shift, shift);
#pragma unroll
  for (int e = 0; e < 32; ++e) {
    const uint32_t (&v)[32] = e < 16 ? a : b;
    const float2 y = ptx::unpair(
        ptx::fma_pair(ptx::pair(__uint_as_float(v[2 * (e & 15)]), __uint_as_float(v[2 * (e & 15) + 1])), c2, shift2));
    pk[e] = ptx::round_pair<kF16>(ptx::exp2_approx(y.x), ptx::exp2_approx(y.y));
    ptx::add_halves<kF16>(sum[e & 1], sum[2 + (e & 1)], pk[e]);
  }
}

// The parts of a key tile's work that most tiles do not need are functions of
// their own, called when no scores are held in registers: the key loop stays
// short enough for the instruction cache and spills nothing.

// Clears the rows of a value tile that lie past the keys: they may hold anything, and
// a weight of zero does not make up for it.
template <int kD>
__device__ __noinline__ bool clear_past(const Waiter* wait, uint32_t value_bar, uint32_t parity, uint8_t* value_tile, int keys) {
  using L = Layout<kD>;
  const int r = threadIdx.x & 127;
  if (!(*wait)(value_bar, parity, 8000)) return false;
  if (r >= keys) {
#pragma unroll 1
    for (int c = 0; c < kD / 8; ++c)
      reinterpret_cast<uint4*>(value_tile + (c >> 3) * L::kHalfBytes + r * 128)[(c + r) & 7] = make_uint4(0, 0, 0, 0);
    ptx::fence_proxy_async_smem();
  }
  return true;
}

// Puts -inf over the scores, in tensor memory, of the keys of such a tile that
// this thread's row does not see, whatever they were.
template <bool kPaged>
__device__ __noinline__ void mask_scores(const AttnParams* p, const Item* it, uint32_t t_s, int s, int place) {
  const Row row = row_of<kPaged>(*p, *it, s, threadIdx.x & 127);
#pragma unroll 1
  for (int w = 0; w < 4; ++w) {
    const uint32_t bits = seen32(*it, row, p->mask_words, place + 32 * w);
    if (__all_sync(0xffffffffu, bits == 0xffffffffu)) continue;
    uint32_t v[32];
    if (__any_sync(0xffffffffu, bits)) {
      ptx::tmem_ld_32x32b_x32(t_s + w * 32, v);
      ptx::tmem_ld_wait();
    }
#pragma unroll
    for (int e = 0; e < 32; ++e)
      if (!(bits >> e & 1u)) v[e] = 0xff800000u;
    ptx::tmem_st_32x32b_x32(t_s + w * 32, v);
  }
  ptx::tmem_st_wait();
}

// The largest score of a row.
__device__ __noinline__ float tile_max(uint32_t t_s) {
  float top = -INFINITY;
#pragma unroll 1
  for (int w = 0; w < 4; w += 2) {
    uint32_t a[32], b[32];
    ptx::tmem_ld_32x32b_x32(t_s + w * 32, a);
    ptx::tmem_ld_32x32b_x32(t_s + w * 32 + 32, b);
    ptx::tmem_ld_wait();
    float t[4] = {top, top, top, top};
#pragma unroll
    for (int e = 0; e < 32; e += 4) {
      t[0] = ptx::max3(t[0], __uint_as_float(a[e]), __uint_as_float(a[e + 1]));
      t[1] = ptx::max3(t[1], __uint_as_float(a[e + 2]), __uint_as_float(a[e + 3]));
      t[2] = ptx::max3(t[2], __uint_as_float(b[e]), __uint_as_float(b[e + 1]));
      t[3] = ptx::max3(t[3], __uint_as_float(b[e + 2]), __uint_as_float(b[e + 3]));
    }
    top = ptx::max3(fmaxf(t[0], t[1]), t[2], t[3]);
  }
  return top;
}

// Stores kWords 32-bit words of each lane's row to `to`, the lane's own address.  Lane
// 4 g + j has piece i (16 bytes) of row 4 g + j in words 4 i ..; after two
// exchanges it has piece j of row 4 g + i.
template <int kWords, typename T>
__device__ __forceinline__ void store_rows(const uint32_t (&words)[kWords], int lane, uint32_t rows, T* to) {
#pragma unroll
  for (int w = 0; w < kWords; w += 16) {
    uint32_t x[4][4];
#pragma unroll
    for (int e = 0; e < 16; ++e) x[e / 4][e % 4] = words[w + e];
#pragma unroll
    for (int bit = 1; bit <= 2; bit <<= 1) {
      const bool upper = lane & bit;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (e & bit) continue;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          // the lower lane keeps the lower piece and sends the upper one
          const uint32_t keep = upper ? x[e | bit][q] : x[e][q];
          const uint32_t got = __shfl_xor_sync(0xffffffffu, upper ? x[e][q] : x[e | bit][q], bit);
          x[e][q] = upper ? got : keep;
          x[e | bit][q] = upper ? keep : got;
        }
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int from = (lane & ~3) + e;
      T* const at = reinterpret_cast<T*>(__shfl_sync(0xffffffffu, reinterpret_cast<uintptr_t>(to), from));
      if (rows >> from & 1u) reinterpret_cast<uint4*>(at)[w / 4 + (lane & 3)] = make_uint4(x[e][0], x[e][1], x[e][2], x[e][3]);
    }
  }
}

// O *= keep.  The last product into it has ended: the scores that showed the new
// maximum were issued after it.
template <int kD>
__device__ __noinline__ void rescale(uint32_t t_o, float keep) {
#pragma unroll 1
  for (int col = 0; col < kD; col += 32) {
    uint32_t o[32];
    ptx::tmem_ld_32x32b_x32(t_o + col, o);
    ptx::tmem_ld_wait();
#pragma unroll
    for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * keep);
    ptx::tmem_st_32x32b_x32(t_o + col, o);
  }
  ptx::tmem_st_wait();
}

__device__ __forceinline__ void load_scores(uint32_t t_s, uint32_t (&v)[4][32]) {
#pragma unroll
  for (int w = 0; w < 4; ++w) ptx::tmem_ld_32x32b_x32(t_s + w * 32, v[w]);
  ptx::tmem_ld_wait();
}

template <int kD, bool kF16, bool kPaged>
__device__ __forceinline__ void softmax(const AttnParams& p, const Bars& bars, const Item* slots, uint8_t* smem, uint32_t tmem,
                                        const Waiter& wait, int s, float* stats) {
  using L = Layout<kD>;
  const int lane = threadIdx.x & 31;
  const int r = threadIdx.x & 127;  // the row this thread owns
  const uint32_t lanes = (uint32_t)((threadIdx.x >> 5) & 3) << 21;  // its warp's quarter of the TMEM lanes
  const uint32_t t_s = tmem + lanes + s * kKeys;
  const uint32_t t_o = tmem + lanes + 2 * kKeys;
  const float c = p.scale_log2;
  uint32_t fills = 0, steps = 0, results = 0, results_other = 0;
  uint32_t joint = 0;  // alternating items so far
  bool ok = true;
  for (int k = 0; ok; ++k) {
    const int slot = k % kItemSlots;
    if (!wait(bars.item_full(slot), (uint32_t)(k / kItemSlots) & 1u, k)) break;
    // The item stays in shared memory until this warp has its results out: what
    // the key loop does not need on every tile takes no register there.
    const Item& it = slots[slot];
    if (!it.valid) break;
    const int n = it.n[s];
    const int stride = it.alternate ? 2 * kKeys : kKeys;
    const bool any = __any_sync(0xffffffffu, r < it.cnt[s] * p.pack);
    const int edge = it.masked_from;  // tiles that end before this place are seen by all rows
    int place = (it.kv_tile + (it.alternate ? s : 0)) * kKeys;
    float m = -INFINITY, l = 0.0f;
#pragma unroll 1
    for (int i = 0; i < n; ++i, place += stride) {
      const bool partly = place + kKeys > edge;
      if (place + kKeys > it.kv_len) {
        const uint32_t f = fills + (uint32_t)v_index(place / kKeys - it.kv_tile, it.alternate ? 2 : 1, it.tiles);
        ok = clear_past<kD>(&wait, bars.v_there(s, steps + i), (steps + i) >> 1 & 1u, smem + L::kRing + (f % L::kStages) * L::kTileBytes,
                            it.kv_len - place);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
      }
      ok = wait(bars.s_full(s), (steps + i) & 1u, 6000 + s);
      if (!ok) break;
      ptx::tc_fence_after();
      if (partly && any) mask_scores<kPaged>(&p, &it, t_s, s, place);
      // The weights, in halves of 64 keys, so that the first half's product runs
      // while the second half's weights are computed.
      if (any) {
        if (i == 0) m = tile_max(t_s);
        uint32_t v[4][32], pk[32];
        float sum[4];
        // The weights of the first half are computed with the reference there is,
        // and the tile's maximum on the way: only where a row's maximum has grown
        // too far, which is rare, they are computed again.
        for (;;) {
          load_scores(t_s, v);
          sum[0] = sum[1] = sum[2] = sum[3] = 0.0f;
          weights<kF16>(v[0], v[1], c, weight_shift<kF16>(m, c), pk, sum);
          const float top = row_max(v);
          const bool grows = (top - m) * c > kMaxGrowth;  // also from -inf to anything
          if (!__any_sync(0xffffffffu, grows)) break;
          const float keep = grows ? ptx::exp2_approx((m - top) * c) : 1.0f;
          if (grows) m = top;
          l *= keep;
          rescale<kD>(t_o + s * kD, keep);
        }
        ptx::tmem_st_32x32b_x32(t_s, pk);
        ptx::tmem_st_wait();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bars.p_ready(s, 0));
        weights<kF16>(v[2], v[3], c, weight_shift<kF16>(m, c), pk, sum);
        ptx::tmem_st_32x32b_x32(t_s + 32, pk);
        ptx::tmem_st_wait();
        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bars.p_ready(s, 1));
      } else if (lane == 0) {
        ptx::mbar_arrive(bars.p_ready(s, 0));
        ptx::mbar_arrive(bars.p_ready(s, 1));
      }
    }
    if (!ok) break;

    // ---- the item's result
    float scale0 = 0.0f, scale1 = 0.0f;  // of the streams' sums
    int col0 = 0, col1 = kD;             // columns this thread writes
    bool has0 = s == 0 && n > 0, has1 = s == 1 && n > 0;
    if (n > 0) ok = wait(bars.o_full(s), results & 1u, 7100 + s);
    if (!ok) break;
    if (it.alternate) {
      // The streams' maxima and sums change hands.  A stream that had keys has
      // just seen its product end, which waited for all warps to be done with the
      // item before: what it left here then has been read.
      if (n > 0) *reinterpret_cast<float2*>(stats + 256 * s + 2 * r) = make_float2(m, l);
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(bars.stats());
      ok = wait(bars.stats(), joint & 1u, 9000);
      if (!ok) break;
      ++joint;
      float2 other = make_float2(-INFINITY, 0.0f);
      if (it.n[s ^ 1] > 0) {
        other = *reinterpret_cast<const float2*>(stats + 256 * (s ^ 1) + 2 * r);
        ok = wait(bars.o_full(s ^ 1), results_other & 1u, 7200 + s);
        if (!ok) break;
      }
      const float both = fmaxf(m, other.x);
      const float mine_w = m == -INFINITY ? (l != l ? 1.0f : 0.0f) : ptx::exp2_approx((m - both) * c);
      const float other_w = other.x == -INFINITY ? (other.y != other.y ? 1.0f : 0.0f) : ptx::exp2_approx((other.x - both) * c);
      l = l * mine_w + other.y * other_w;
      m = both;
      scale0 = s == 0 ? mine_w : other_w;
      scale1 = s == 0 ? other_w : mine_w;
      has0 = it.n[0] > 0;
      has1 = it.n[1] > 0;
      col0 = s * (kD / 2);
      col1 = col0 + kD / 2;
    } else {
      scale0 = scale1 = 1.0f;
    }
    ptx::tc_fence_after();
    if (any) {
      const Row own = row_of<kPaged>(p, it, s, r);
      const bool whole = it.slot < 0;
      if (whole) {
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        scale0 *= inv;
        scale1 *= inv;
      }
      const int tile_row = (it.alternate ? 0 : s * p.tile_tokens * p.pack) + r;
      const int head = it.head + s * (it.alternate ? 0 : it.head_step) + (p.pack == 1 ? 0 : r - (own.token - it.tok[s]) * p.pack);
      uint16_t* const out = p.out + (int64_t)(it.q0 + own.token) * p.out_ts + head * p.out_hs;
      float* const part = whole ? nullptr : p.partial + ((size_t)it.slot * p.partial_rows + tile_row) * kD;
      // A row's results are in one lane.  Four lanes exchange theirs, so that each
      // stores 16 bytes of all four rows and together 64 consecutive bytes of one: a
      // store of 32 rows takes a cycle for each of 32 lines and more, 3400 cycles a tile
      // against 1300.
      const uint32_t rows_there = __ballot_sync(0xffffffffu, own.there);
      uint32_t top = 0;  // of the results' magnitudes, as 16-bit pairs
#pragma unroll 1
      for (int col = col0; col < col1; col += 32) {
        uint32_t o[32];
        if (has0 != has1) {
          ptx::tmem_ld_32x32b_x32(t_o + (has1 ? kD : 0) + col, o);
          ptx::tmem_ld_wait();
          const float scale = has1 ? scale1 : scale0;
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * scale);
        } else if (has0) {
          uint32_t a[32];
          ptx::tmem_ld_32x32b_x32(t_o + col, o);
          ptx::tmem_ld_32x32b_x32(t_o + kD + col, a);
          ptx::tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 32; ++e)
            o[e] = __float_as_uint(fmaf(__uint_as_float(a[e]), scale1, __uint_as_float(o[e]) * scale0));
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0;
        }
        uint32_t packed[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          packed[e] = pack2<kF16>(__uint_as_float(o[2 * e]), __uint_as_float(o[2 * e + 1]));
          // in bf16, whose range is float32's: the sums of a part may be past fp16's and finite
          top = __vmaxu2(top, (kF16 ? pack2<false>(__uint_as_float(o[2 * e]), __uint_as_float(o[2 * e + 1])) : packed[e]) & 0x7fff7fffu);
        }
        if (whole)
          store_rows(packed, lane, rows_there, out + col);
        else
          store_rows(o, lane, rows_there, part + col);
      }
      // (a weight sum that is NaN makes the row NaN, as it should be)
      const uint32_t bad = __ballot_sync(0xffffffffu, own.there && l == l && __vcmpgeu2(top, 0x7f807f80u) != 0);
      if (bad) {
        __syncwarp();  // the other lanes' stores come first
        repair_rows<kD, kF16, kPaged>(&p, &it, &wait, s, bad, m, l, col0, col1, out, part);
      }
      if (!whole && own.there && col0 == 0) {
        float* const ml =
            p.partial + (size_t)gridDim.x * 2 * p.partial_rows * kD + ((size_t)it.slot * p.partial_rows + tile_row) * 2;
        ml[0] = m;
        ml[1] = l;
      }
    }
    ptx::tc_fence_before();
    __syncwarp();
    if (lane == 0) {
      if (has0) ptx::mbar_arrive_n(bars.o_free(0), it.alternate ? 1 : 2);
      if (has1) ptx::mbar_arrive_n(bars.o_free(1), it.alternate ? 1 : 2);
    }
    fills += 2u * (uint32_t)it.tiles;
    steps += n;
    results += n > 0;
    results_other += it.n[s ^ 1] > 0;
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(bars.item_empty(slot));
  }
}

// --------------------------------------------------------------------- kernel
template <int kD, bool kF16, bool kPaged>
__global__ void __launch_bounds__(kAttnThreads, 1) agmm_attention(const __grid_constant__ AttnParams p) {
  using L = Layout<kD>;
  extern __shared__ __align__(1024) uint8_t raw[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t smem = ptx::smem_addr(raw);
  uint8_t* const base = raw;
  if (smem & 1023u) {  // the swizzled tiles need the alignment that `raw` asks for
    if (threadIdx.x == 0 && atomicCAS(p.status, 0, 4) == 0) p.status[1] = 0;
    return;
  }
  const Bars bars{smem + L::kBars, L::kStages};
  Item* const slots = reinterpret_cast<Item*>(base + L::kItems);
  int* const flags = reinterpret_cast<int*>(base + L::kFlags);  // [0] abort, [1] TMEM base, [2] pulse
  float* const stats = reinterpret_cast<float*>(base + L::kStats);

  if (warp == 9) {
    ptx::tmem_alloc(ptx::smem_addr(&flags[1]), 512);
    ptx::tmem_relinquish();
  }
  if (threadIdx.x == 0) {
    flags[0] = flags[2] = 0;
    for (int i = 0; i < L::kStages; ++i) {
      ptx::mbar_init(bars.full(i), 1);
      ptx::mbar_init(bars.empty(i), 2);  // both MMA warps
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(bars.q_full(i), 1);
      ptx::mbar_init(bars.q_empty(i), 2);
      ptx::mbar_init(bars.s_full(i), 1);
      ptx::mbar_init(bars.p_ready(i, 0), 4);
      ptx::mbar_init(bars.p_ready(i, 1), 4);
      ptx::mbar_init(bars.o_full(i), 1);
      ptx::mbar_init(bars.v_there(i, 0), 1);
      ptx::mbar_init(bars.v_there(i, 1), 1);
      ptx::mbar_init(bars.turn(i), 1);
      ptx::mbar_init(bars.o_free(i), 8);
    }
    for (int i = 0; i < kItemSlots; ++i) {
      ptx::mbar_init(bars.item_full(i), 1);
      ptx::mbar_init(bars.item_empty(i), 11);  // all warps but the scheduler's
    }
    ptx::mbar_init(bars.stats(), 8);
    ptx::mbar_init(bars.next_item(), 1);
    ptx::mbar_init(bars.drained(0), 1);
    ptx::mbar_init(bars.drained(1), 1);
    ptx::fence_mbar_init();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  // All 512 columns are this CTA's, so they begin at 0; the MMA warp counts on it.
  constexpr uint32_t tmem = 0;
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();

  Waiter wait{flags, p.wait_limit_cycles, p.status, 3};
  // Of the 168 registers a thread that 384 threads start with, the third
  // warpgroup gives up 96 and the softmax warps take 48 more each:
  // 2 x 216 + 72 = 504 = 3 x 168.
  if (warp < 8)
    ptx::more_registers<216>();
  else
    ptx::fewer_registers<72>();
  if (warp < 8) {
    softmax<kD, kF16, kPaged>(p, bars, slots, base, tmem, wait, warp >> 2, stats);
  } else if (warp == 8) {
    if (lane == 0) {
      ptx::prefetch_tensormap(&p.qmap);
      if (kPaged || p.kv_tokens > 0) {  // else there are no such maps
        ptx::prefetch_tensormap(&p.kmap);
        ptx::prefetch_tensormap(&p.vmap);
      }
    }
    wait.role = 1;
    producer<kD, kPaged>(p, bars, slots, smem, wait);
  } else if (warp == 9) {
    wait.role = 2;
    mma_issuer<kD, kF16, 0>(bars, slots, smem, wait);
  } else if (warp == 10) {
    wait.role = 4;
    scheduler<kPaged>(p, bars, slots, wait);
  } else {
    wait.role = 2;
    mma_issuer<kD, kF16, 1>(bars, slots, smem, wait);
  }
  __syncwarp();
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
}

}  // namespace
}  // namespace agmm

#define AGMM_ATTN_VARIANT(D, F16, PAGED) \
  AttnFn { &agmm_attention<D, F16, PAGED>, Layout<D>::kBytes }
