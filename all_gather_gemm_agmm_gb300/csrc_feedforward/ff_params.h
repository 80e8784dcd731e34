// ff_params.h -- parameter blocks shared by the host code (ff_api.cpp) and the
// kernels of the feed-forward operators.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace agmm {
namespace ff {

constexpr int kMaxShards = 8;
constexpr int kThreads = 320;     // warp 0: TMA producer, warp 1: MMA issuer, warps 2-9: epilogue
constexpr int kEpiWarps = 8;
constexpr int kTileM = 128;       // rows of the A operand of one CTA = TMEM lanes
constexpr int kWideN = 256, kNarrowN = 128;  // row tiles: columns of a CTA pair's tile
constexpr int kTileK = 64;        // one 128-byte swizzle row of 16-bit values
constexpr int kTileBytes = kTileM * kTileK * 2;  // 16 KiB
constexpr int kMaxStages = 12;
constexpr int kWideStages = 6, kNarrowStages = 8;  // 192 KiB of operands beside 32 KiB of staged results
constexpr int kMaxSplit = 8;      // CTAs of a cluster that share a swapped tile's k
constexpr int kMaxPairs = 4;      // pairs that share a narrow row tile's
constexpr int kMaxSwapRows = 64;  // swapped tiles: token columns of a tile, at most
constexpr int kStageOutBytes = 4096;  // row tiles: a warp's staging buffer, 32 rows x 128 bytes
constexpr int kCtlBytes = 1024;
constexpr size_t kMaxSmem = 232448;   // 227 KiB
constexpr int kStatusBytes = 256;     // status words at the start of the workspace
constexpr size_t kSlotBytes = (size_t)kTileM * kWideN * sizeof(float);  // one CTA's float32 partial results
constexpr int kSlots = 2;             // of each CTA: the first and the last tile of its share

enum Act : int { kActNone = 0, kActRelu = 1, kActSilu = 2, kActGelu = 3, kActGeluTanh = 4 };
enum Epi : int { kEpiPlain = 0, kEpiGated = 1, kEpiLinear = 2 };

// One operand's tensor maps, boxes of 64 values along the rows.  K-major: {k, rows}.
// MN-major: {64, k, blocks of 64 values, segments} where the rows are whole blocks, so that one
// box brings two of them, else {values, k, 1, segments}.  The map of a load: problem *
// by_problem + segment * by_segment + shard * by_shard (+ CTA rank * by_rank); its last
// coordinate, if MN-major: segment * z_segment.
struct OperandParams {
  int maps;      // how many there are
  int mn_major;  // rows run along the tile, not along k
  int blocked;   // ... and are whole blocks
  int by_problem, by_segment, by_shard, by_rank, z_segment;
};

// One matrix product (or two of one shape: the gradients of two weights).
struct __align__(128) Product {
  CUtensorMap a_map[kMaxShards];
  CUtensorMap b_map[kMaxShards];
  OperandParams a, b;
  // Row tiles: pair tiles of 256 x 256 or 128 (gated: half of them columns of each product).
  // Swapped tiles: 128 columns of the weights, all tokens.
  int problems, tiles_per_problem, m_tiles, n_tiles, group_m;
  int b_tile_step;         // row tiles: B rows from one tile to the next
  int b_half_step;         // row tiles: ... and from the leader's half to the follower's
  int k_blocks;            // of all segments
  int seg_blocks;          // of one segment
  // Tokens (row tiles: the rows of A; swapped tiles: the rows of B) in chunks of
  // box rows that lie in one shard.
  int shards, box, shard_chunks;  // shard_chunks: chunks of a shard
  int chunks;                     // of all shards
  int64_t shard_rows;
  void* out[2];            // by problem
  int64_t ldo;
  int out_f32;             // plain products: float32 results
  int64_t cols;            // columns of the results
};

struct __align__(128) GemmParams : Product {
  int num_tiles;
  int dp_tiles;            // tiles [0, dp_tiles) are worked on whole
  int sk_clusters;         // the k blocks of the others are dealt evenly to this many clusters:
  int sk_share, sk_extra;  // sk_share to each, and one more to the first sk_extra
  int mma_n;               // swapped tiles: token columns, a multiple of 16
  int recv_slots;          // ... groups of 8 tokens that each CTA of a cluster owns
  int split;               // CTAs, or pairs, of a cluster that share a tile's k
  uint32_t recv_bytes;     // their parts, in the shared memory of the owner
  int stages;
  uint32_t tmem_cols;
  void* saved[2];          // gated: the two products; linear: the sum before the activation
  int64_t lds;
  const void* bias;
  const void* residual;
  int64_t ldr;
  int act;
  int f16;
  // workspace
  int* status;
  int* counters;           // [shared tiles][CTAs of a cluster][kEpiWarps], zero between runs
  float* partial;          // [CTAs][kSlots][kSlotBytes]
  uint64_t wait_limit_cycles;
  int test_drop;           // test hook: the first arrival of a producer is dropped
};

// Two products in one launch (both gradients of a layer), all tiles whole: after the first's,
// `lead` clusters of which have one more than the others; those others take `ahead` tiles of the
// second meanwhile, then all take `each`, and `rest` of them one more.
struct __align__(128) TwoParams : GemmParams {
  Product second;
  int lead, ahead, each, rest;
};

using GemmFn = void (*)(GemmParams);
using TwoFn = void (*)(TwoParams);
// bn: columns of row tiles (0: swapped tiles); save_f32: what is saved is float32 (gated, linear)
GemmFn select_gemm(int bn, int epi, bool f16, bool save_f32);
TwoFn wide_two(bool f16);
TwoFn narrow_two(bool f16);
GemmFn wide_plain(bool f16);
GemmFn wide_gated(bool f16, bool save_f32);
GemmFn wide_linear(bool f16, bool save_f32);
GemmFn narrow_plain(bool f16);
GemmFn narrow_gated(bool f16, bool save_f32);
GemmFn narrow_linear(bool f16, bool save_f32);
GemmFn swap_plain(bool f16);
GemmFn swap_gated(bool f16, bool save_f32);
GemmFn swap_linear(bool f16, bool save_f32);

// Sets the shared-memory limit of a kernel and reports the clusters that fit.
cudaError_t prepare_gemm(GemmFn fn, int cluster, int* clusters);
cudaError_t prepare_two(TwoFn fn, int* clusters);
cudaError_t launch_gemm(GemmFn fn, const GemmParams& p, int clusters, int cluster, size_t smem, cudaStream_t stream);
cudaError_t launch_two(TwoFn fn, const TwoParams& p, int clusters, size_t smem, cudaStream_t stream);

// --------------------------------------------------------------- pointwise
// d_gate = d_out * up * act'(gate), d_up = d_out * act(gate)
struct GatedGradParams {
  int64_t rows, cols;
  const uint16_t* d_out;
  const void *gate, *up;  // as the outputs, or (saved_f32) in float32
  uint16_t *d_gate, *d_up;
  int64_t ld_out, ld_saved, ld_grad;
  int act, saved_f32;
};
cudaError_t launch_gated_grad(const GatedGradParams& p, bool f16, int sms, cudaStream_t stream);

// d_pre = d_out * act'(pre) (pre NULL: no activation, nothing is written), and the sums of
// its columns: in parts of [blocks][cols], or (few rows) the whole of them.
struct ActGradParams {
  int64_t rows, cols;
  const uint16_t* d_out;
  const void* pre;  // as d_out, or (saved_f32) in float32
  uint16_t* d_pre;
  int64_t ld_out, ld_pre, ld_grad;
  int act, saved_f32;
  float* part;  // NULL: no parts
  int row_blocks;
  void* d_bias;  // few rows: the sums; NULL: no sums, or parts
  int out_f32;
};
int act_grad_row_blocks(int64_t rows, int64_t cols, int sms);
cudaError_t launch_act_grad(const ActGradParams& p, bool f16, cudaStream_t stream);

// out[c] = sum over parts of part[i][c], for one or two sums of `cols` columns
struct SumPartsParams {
  const float* part;  // [parts][sums][cols]
  int parts, sums;
  int64_t cols;
  void* out[2];       // NULL: not wanted
  int out_f32;
};
cudaError_t launch_sum_parts(const SumPartsParams& p, bool f16, cudaStream_t stream);

// -------------------------------------------------------------- layer norm
constexpr int kMaxNormColumns = 16384;
struct NormParams {
  int64_t rows;
  int cols;
  float eps;
  const uint16_t* x;
  int64_t ldx;
  const uint16_t *weight, *bias;
  uint16_t* out;
  int64_t ldo;
  float *mean, *rstd;
};
cudaError_t prepare_norm(bool f16);  // shared-memory limits, once for a plan
cudaError_t launch_norm(const NormParams& p, bool f16, int sms, cudaStream_t stream);

struct NormGradParams {
  int64_t rows;
  int cols;
  const uint16_t *d_out, *x, *weight, *add;
  int64_t ld_out, ldx, ld_add;
  const float *mean, *rstd;
  uint16_t* dx;
  int64_t ld_dx;
  float* part;  // [blocks][2][cols]: the sums of d_out * xhat and of d_out; NULL: not wanted
  int stages;   // rows in flight, where they stream
  // few rows: the sums themselves (NULL: not wanted), and the blocks that have columns
  void *d_weight, *d_bias;
  int out_f32, column_blocks;
};
// Few rows: dx and the sums in one launch.  dx must not lie over d_out if sums are wanted.
bool few_norm_rows(int64_t rows, int cols);
cudaError_t launch_norm_grad_few(const NormGradParams& p, bool f16, cudaStream_t stream);
int norm_grad_blocks(int64_t rows, int cols, int sms);
cudaError_t launch_norm_grad(const NormGradParams& p, bool f16, int blocks, cudaStream_t stream);

}  // namespace ff
}  // namespace agmm
