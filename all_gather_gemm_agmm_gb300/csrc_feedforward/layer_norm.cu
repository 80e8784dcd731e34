// layer_norm.cu -- layer norm of rows and its backward pass.
//
//   y = (x - mean) * rstd * w + b,   rstd = 1 / sqrt(mean((x - mean)^2) + eps)
//   g = dy * w,  xhat = (x - mean) * rstd
//   dx = rstd * (g - mean(g) - xhat * mean(g * xhat)) (+ add)
//   dw = sum over rows of dy * xhat,  db = sum over rows of dy
//
// Bound: device memory; every value is read once and written once.  A team of threads (a
// warp for short rows, else the block) holds a row in registers, 8 values to a piece, so
// the variance is a sum of squares about the mean and not a difference of large numbers.
// The backward pass keeps a team on its columns: the sums for dw and db stay in
// registers while it walks over the rows, and each block leaves one part of them; few rows have their
// sums made by other blocks of the same launch.  Arithmetic is
// on pairs of values: with single ones both passes were bound by instructions (2.8 of 4 a cycle).
// Measured, 16384 x 8192: forward 88 us (6.1 TB/s), backward with a gradient to add 172 us (6.2 TB/s,
// 5 us of it the parts' sums), without one 154 us (5.2 TB/s).
#include "ff_math.cuh"
#include "ptx_sm103.cuh"

namespace agmm {
namespace ff {
namespace {

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The sum over the block, whose warps meet in `s`; it may be written again behind another barrier.
__device__ __forceinline__ float block_sum(float v, float* s) {
  v = warp_sum(v);
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
  __syncthreads();
  return warp_sum((threadIdx.x & 31) < (blockDim.x >> 5) ? s[threadIdx.x & 31] : 0.0f);
}

// The sum over a team: a warp, or the block.
template <bool kWarpRow>
__device__ __forceinline__ float team_sum(float v, float* s) {
  return kWarpRow ? warp_sum(v) : block_sum(v, s);
}

// Eight ones: a weight that is not there.
template <bool kF16>
__device__ __forceinline__ uint4 ones() {
  constexpr uint32_t w = kF16 ? 0x3c003c00u : 0x3f803f80u;
  return make_uint4(w, w, w, w);
}

// x * rstd * w + b of a piece
template <bool kF16>
__device__ __forceinline__ uint4 scaled(const Two (&x)[4], float rstd, const uint4& w16, const uint4& b16) {
  Two w[4], b[4], y[4];
  widen<kF16>(w16, w);
  widen<kF16>(b16, b);
#pragma unroll
  for (int e = 0; e < 4; ++e) y[e] = fma2(mul2(x[e], both(rstd)), w[e], b[e]);
  return narrow<kF16>(y);
}

// A piece of the backward pass: xhat, and g = d * w.
struct GradPiece {
  Two x[4], g[4];
};
template <bool kF16>
__device__ __forceinline__ GradPiece grad_piece(const uint4& x16, const uint4& d16, float mean, float rstd) {
  GradPiece q;
  widen<kF16>(x16, q.x);
  widen<kF16>(d16, q.g);
#pragma unroll
  for (int e = 0; e < 4; ++e) q.x[e] = mul2(add2(q.x[e], both(-mean)), both(rstd));
  return q;
}
template <bool kF16>
__device__ __forceinline__ void weigh(GradPiece& q, const uint4& w16) {
  Two w[4];
  widen<kF16>(w16, w);
#pragma unroll
  for (int e = 0; e < 4; ++e) q.g[e] = mul2(q.g[e], w[e]);
}
// rstd * (g - mg - xhat * mgx) + add
template <bool kF16>
__device__ __forceinline__ uint4 input_grad(const GradPiece& q, float rstd, float mg, float mgx, const uint4& a16) {
  Two a[4], y[4];
  widen<kF16>(a16, a);
#pragma unroll
  for (int e = 0; e < 4; ++e) y[e] = fma2(fma2(q.x[e], both(-mgx), add2(q.g[e], both(-mg))), both(rstd), a[e]);
  return narrow<kF16>(y);
}

constexpr int kWarpRowWarps = 4;

// The statistics of a row that a team holds, x less its mean on return.
template <bool kWarpRow, int kPieces>
__device__ __forceinline__ float2 row_stats(Two (&x)[kPieces][4], int t, int team, int cols, float eps, float (&s)[2][32]) {
  const float inv = 1.0f / (float)cols;
  Two sum = 0, squares = 0;
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    if ((t + i * team) * 8 < cols) {
#pragma unroll
      for (int e = 0; e < 4; ++e) sum = add2(sum, x[i][e]);
    }
  }
  const float mean = team_sum<kWarpRow>(sum2(sum), s[0]) * inv;
  const Two minus = both(-mean);
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    if ((t + i * team) * 8 < cols) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[i][e] = add2(x[i][e], minus);
        squares = fma2(x[i][e], x[i][e], squares);
      }
    }
  }
  return make_float2(mean, rsqrtf(team_sum<kWarpRow>(sum2(squares), s[1]) * inv + eps));
}

// One row to a team: short rows (a warp to each), few long ones, and the longest.
template <bool kF16, bool kWarpRow, int kPieces>
__global__ void __launch_bounds__(kWarpRow ? 32 * kWarpRowWarps : 1024) agmm_layer_norm(const __grid_constant__ NormParams p) {
  __shared__ float s[2][32];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int team = kWarpRow ? 32 : blockDim.x;
  const int t = kWarpRow ? threadIdx.x & 31 : threadIdx.x;
  const int64_t row = kWarpRow ? (int64_t)blockIdx.x * kWarpRowWarps + (threadIdx.x >> 5) : blockIdx.x;
  if (row >= p.rows) return;
  uint4 in[kPieces];
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const int c = (t + i * team) * 8;
    if (c < p.cols) in[i] = *reinterpret_cast<const uint4*>(p.x + row * p.ldx + c);
  }
  Two x[kPieces][4];
#pragma unroll
  for (int i = 0; i < kPieces; ++i)
    if ((t + i * team) * 8 < p.cols) widen<kF16>(in[i], x[i]);
  const float2 stats = row_stats<kWarpRow>(x, t, team, p.cols, p.eps, s);
  if (t == 0) {
    if (p.mean) p.mean[row] = stats.x;
    if (p.rstd) p.rstd[row] = stats.y;
  }
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const int c = (t + i * team) * 8;
    if (c < p.cols) {
      const uint4 w = p.weight ? __ldg(reinterpret_cast<const uint4*>(p.weight + c)) : ones<kF16>();
      const uint4 b = p.bias ? __ldg(reinterpret_cast<const uint4*>(p.bias + c)) : make_uint4(0, 0, 0, 0);
      *reinterpret_cast<uint4*>(p.out + row * p.ldo + c) = scaled<kF16>(x[i], stats.y, w, b);
    }
  }
}

// Weights are read again for every row (they stay in L1): held over the rows, their registers
// would be another block's.
__device__ __forceinline__ uint4 load_again(const uint16_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

// Many long rows: a block walks over rows, four pieces to a thread, and loads the next row
// beside this one's sums.  16384 x 8192: 88 us, 6.1 TB/s; a block to each row 93 us; rows through
// shared memory 114 us; two pieces to a thread 106 us.  (Rows of 16384 values need 512 threads and
// leave room for one block: 64 us so, 55 us with a block to each row.)
template <bool kF16>
__global__ void __launch_bounds__(256, 3) agmm_layer_norm_rows(const __grid_constant__ NormParams p) {
  constexpr int kPieces = 4;
  __shared__ float s[2][32];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int t = threadIdx.x, team = blockDim.x;
  const int64_t step = gridDim.x;
  uint4 in[kPieces];
  auto fetch = [&](int64_t row) {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int c = (t + i * team) * 8;
      if (c < p.cols) in[i] = __ldcs(reinterpret_cast<const uint4*>(p.x + row * p.ldx + c));
    }
  };
  fetch(blockIdx.x);
#pragma unroll 1
  for (int64_t row = blockIdx.x; row < p.rows; row += step) {
    Two x[kPieces][4];
#pragma unroll
    for (int i = 0; i < kPieces; ++i)
      if ((t + i * team) * 8 < p.cols) widen<kF16>(in[i], x[i]);
    if (row + step < p.rows) fetch(row + step);
    const float2 stats = row_stats<false>(x, t, team, p.cols, p.eps, s);
    if (t == 0) {
      if (p.mean) p.mean[row] = stats.x;
      if (p.rstd) p.rstd[row] = stats.y;
    }
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int c = (t + i * team) * 8;
      if (c < p.cols) {
        const uint4 w = p.weight ? load_again(p.weight + c) : ones<kF16>();
        const uint4 b = p.bias ? load_again(p.bias + c) : make_uint4(0, 0, 0, 0);
        *reinterpret_cast<uint4*>(p.out + row * p.ldo + c) = scaled<kF16>(x[i], stats.y, w, b);
      }
    }
  }
}

// Rows that stream through shared memory: a thread copies its own pieces of the next rows
// there (16 bytes at a time, asynchronously), a ring of `stages` rows ahead, and reads back
// only those, so that rows in flight need no barrier.
__device__ __forceinline__ void copy_async(uint4* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(ptx::smem_addr(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Waits until at most `left` of this thread's latest groups are in flight.
__device__ __forceinline__ void copy_wait(int left) {
  switch (left) {
    case 0: asm volatile("cp.async.wait_group 0;" ::: "memory"); break;
    case 1: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
    case 2: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
    case 3: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
    case 4: asm volatile("cp.async.wait_group 4;" ::: "memory"); break;
    case 5: asm volatile("cp.async.wait_group 5;" ::: "memory"); break;
    case 6: asm volatile("cp.async.wait_group 6;" ::: "memory"); break;
    default: asm volatile("cp.async.wait_group 7;" ::: "memory"); break;
  }
}
constexpr int kMostStages = 8;
constexpr int kSumBytes = 512;  // the warps' sums, at the start of shared memory

// Short rows: a warp to a row.
template <bool kF16, int kPieces>
__global__ void __launch_bounds__(32 * kWarpRowWarps) agmm_layer_norm_grad_short(const __grid_constant__ NormGradParams p) {
  extern __shared__ __align__(16) uint8_t shared_bytes[];
  float* const shared = reinterpret_cast<float*>(shared_bytes);  // a part of each warp
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int t = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t step = (int64_t)gridDim.x * kWarpRowWarps;
  const float inv = 1.0f / (float)p.cols;
  Two dw[kPieces][4], db[kPieces][4];
  uint4 w16[kPieces];
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const int c = (t + i * 32) * 8;
#pragma unroll
    for (int e = 0; e < 4; ++e) dw[i][e] = db[i][e] = 0;
    w16[i] = p.weight && c < p.cols ? __ldg(reinterpret_cast<const uint4*>(p.weight + c)) : ones<kF16>();
  }
#pragma unroll 1
  for (int64_t row = (int64_t)blockIdx.x * kWarpRowWarps + warp; row < p.rows; row += step) {
    uint4 x16[kPieces], d16[kPieces], a16[kPieces];
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int c = (t + i * 32) * 8;
      a16[i] = make_uint4(0, 0, 0, 0);
      if (c < p.cols) {
        x16[i] = *reinterpret_cast<const uint4*>(p.x + row * p.ldx + c);
        d16[i] = *reinterpret_cast<const uint4*>(p.d_out + row * p.ld_out + c);
        if (p.add) a16[i] = *reinterpret_cast<const uint4*>(p.add + row * p.ld_add + c);
      }
    }
    const float mean = __ldg(p.mean + row), r = __ldg(p.rstd + row);
    GradPiece q[kPieces];
    Two sum_g = 0, sum_gx = 0;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      if ((t + i * 32) * 8 < p.cols) {
        q[i] = grad_piece<kF16>(x16[i], d16[i], mean, r);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          dw[i][e] = fma2(q[i].g[e], q[i].x[e], dw[i][e]);
          db[i][e] = add2(db[i][e], q[i].g[e]);
        }
        weigh<kF16>(q[i], w16[i]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          sum_g = add2(sum_g, q[i].g[e]);
          sum_gx = fma2(q[i].g[e], q[i].x[e], sum_gx);
        }
      }
    }
    if (p.dx) {
      const float mg = warp_sum(sum2(sum_g)) * inv, mgx = warp_sum(sum2(sum_gx)) * inv;
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        const int c = (t + i * 32) * 8;
        if (c < p.cols) *reinterpret_cast<uint4*>(p.dx + row * p.ld_dx + c) = input_grad<kF16>(q[i], r, mg, mgx, a16[i]);
      }
    }
  }
  if (p.part == nullptr) return;
  // the warps' sums, in the order of the warps
  float* const part = p.part + (int64_t)blockIdx.x * 2 * p.cols;
  float* const mine = shared + (size_t)warp * 2 * p.cols;
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const int c = (t + i * 32) * 8;
    if (c < p.cols) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        *reinterpret_cast<Two*>(mine + c + 2 * e) = dw[i][e];
        *reinterpret_cast<Two*>(mine + p.cols + c + 2 * e) = db[i][e];
      }
    }
  }
  __syncthreads();
  for (int c = threadIdx.x; c < 2 * p.cols; c += blockDim.x) {
    float sum = shared[c];
#pragma unroll
    for (int k = 1; k < kWarpRowWarps; ++k) sum += shared[(size_t)k * 2 * p.cols + c];
    part[c] = sum;
  }
}

// Other rows: a block to kRows rows, the rows streaming through shared memory.  Two rows to a
// turn: their sums meet in one barrier, and the latency of one row's sums hides behind the other
// (16384 x 8192: 177 us with one row to a turn; 236 us with four pieces to a thread and two blocks to an SM).
template <bool kF16, int kPieces, int kRows>
__global__ void __launch_bounds__(512, 1) agmm_layer_norm_grad(const __grid_constant__ NormGradParams p) {
  extern __shared__ __align__(16) uint8_t shared[];
  uint4* const ring = reinterpret_cast<uint4*>(shared + kSumBytes);
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int t = threadIdx.x, warp = threadIdx.x >> 5, team = blockDim.x, stages = p.stages;
  const int inputs = p.add ? 3 : 2;
  const int64_t grid = gridDim.x, step = kRows * grid;
  const float inv = 1.0f / (float)p.cols;
  auto slot = [&](int stage, int k, int input, int i) { return ring + (((stage * kRows + k) * inputs + input) * kPieces + i) * team + t; };
  auto fetch = [&](int64_t first, int stage) {
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      const int64_t row = first + k * grid;
      if (row < p.rows) {
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
          const int c = (t + i * team) * 8;
          if (c < p.cols) {
            copy_async(slot(stage, k, 0, i), p.x + row * p.ldx + c);
            copy_async(slot(stage, k, 1, i), p.d_out + row * p.ld_out + c);
            if (p.add) copy_async(slot(stage, k, 2, i), p.add + row * p.ld_add + c);
          }
        }
      }
    }
    copy_commit();
  };
  Two dw[kPieces][4], db[kPieces][4];
  uint4 w16[kPieces];
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const int c = (t + i * team) * 8;
#pragma unroll
    for (int e = 0; e < 4; ++e) dw[i][e] = db[i][e] = 0;
    w16[i] = p.weight && c < p.cols ? __ldg(reinterpret_cast<const uint4*>(p.weight + c)) : ones<kF16>();
  }
  for (int k = 0; k < stages - 1; ++k) fetch(blockIdx.x + k * step, k);
  float next_mean[kRows], next_rstd[kRows];
  auto fetch_stats = [&](int64_t first) {
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      const int64_t row = first + k * grid;
      next_mean[k] = row < p.rows ? __ldg(p.mean + row) : 0.0f;
      next_rstd[k] = row < p.rows ? __ldg(p.rstd + row) : 0.0f;
    }
  };
  fetch_stats(blockIdx.x);
  int stage = 0, turn = 0;
#pragma unroll 1
  for (int64_t first = blockIdx.x; first < p.rows; first += step) {
    fetch(first + (stages - 1) * step, stage == 0 ? stages - 1 : stage - 1);
    float mean[kRows], r[kRows];
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      mean[k] = next_mean[k];
      r[k] = next_rstd[k];
    }
    fetch_stats(first + step);
    copy_wait(stages - 1);
    Two sum_g[kRows], sum_gx[kRows];
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      sum_g[k] = sum_gx[k] = 0;
      if (first + k * grid < p.rows) {
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
          if ((t + i * team) * 8 < p.cols) {
            GradPiece q = grad_piece<kF16>(*slot(stage, k, 0, i), *slot(stage, k, 1, i), mean[k], r[k]);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              dw[i][e] = fma2(q.g[e], q.x[e], dw[i][e]);
              db[i][e] = add2(db[i][e], q.g[e]);
            }
            weigh<kF16>(q, w16[i]);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              sum_g[k] = add2(sum_g[k], q.g[e]);
              sum_gx[k] = fma2(q.g[e], q.x[e], sum_gx[k]);
            }
          }
        }
      }
    }
    if (p.dx) {
      // two sets of sums in turn: one barrier
      float2* const s = reinterpret_cast<float2*>(shared) + 32 * turn;
      turn ^= 1;
      float2 v[kRows];
#pragma unroll
      for (int k = 0; k < kRows; ++k) v[k] = make_float2(warp_sum(sum2(sum_g[k])), warp_sum(sum2(sum_gx[k])));
      if ((t & 31) == 0) {
#pragma unroll
        for (int k = 0; k < kRows; ++k) s[k * 16 + warp] = v[k];
      }
      __syncthreads();
#pragma unroll
      for (int k = 0; k < kRows; ++k) {
        v[k] = (t & 31) < (int)(blockDim.x >> 5) ? s[k * 16 + (t & 31)] : make_float2(0.0f, 0.0f);
        v[k] = make_float2(warp_sum(v[k].x) * inv, warp_sum(v[k].y) * inv);
      }
#pragma unroll
      for (int k = 0; k < kRows; ++k) {
        const int64_t row = first + k * grid;
        if (row < p.rows) {
#pragma unroll
          for (int i = 0; i < kPieces; ++i) {
            const int c = (t + i * team) * 8;
            if (c < p.cols) {
              // read again rather than held: registers
              GradPiece q = grad_piece<kF16>(*slot(stage, k, 0, i), *slot(stage, k, 1, i), mean[k], r[k]);
              weigh<kF16>(q, w16[i]);
              const uint4 a16 = p.add ? *slot(stage, k, 2, i) : make_uint4(0, 0, 0, 0);
              *reinterpret_cast<uint4*>(p.dx + row * p.ld_dx + c) = input_grad<kF16>(q, r[k], v[k].x, v[k].y, a16);
            }
          }
        }
      }
    }
    stage = stage + 1 == stages ? 0 : stage + 1;
  }
  if (p.part == nullptr) return;
  float* const part = p.part + (int64_t)blockIdx.x * 2 * p.cols;
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const int c = (t + i * team) * 8;
    if (c < p.cols) {
#pragma unroll
      for (int e = 0; e < 4; e += 2) {
        *reinterpret_cast<ulonglong2*>(part + c + 2 * e) = make_ulonglong2(dw[i][e], dw[i][e + 1]);
        *reinterpret_cast<ulonglong2*>(part + p.cols + c + 2 * e) = make_ulonglong2(db[i][e], db[i][e + 1]);
      }
    }
  }
}

// Few rows: some blocks have rows, for dx (a warp or a block to a row), the others 64 columns each, for
// the sums over the rows.  Those read x and d_out again, out of L2, and need nothing of the former: the
// statistics are there.  No parts and no second launch.  Columns come first, as they take longer, and two
// blocks share an SM (59 registers): 512 x 4096 5.6 us; rows first 6.4, one block to an SM 7.9 us.
constexpr int kFewWarps = 16, kFewPieces = 8, kFewCols = kFewPieces * 8, kFewRowsAWarp = 32 / kFewPieces, kFewUnroll = 3;
static_assert(kFewWarps * 32 >= 2 * kFewCols, "a thread for each sum");

template <bool kF16, int kTeamWarps, int kPieces>
__device__ __forceinline__ void few_rows(const NormGradParams& p, int block, float2 (&s)[kFewWarps]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int team = kTeamWarps * 32, kRows = kFewWarps / kTeamWarps;
  const int t = threadIdx.x % team;
  const int64_t place = (int64_t)block * kRows + threadIdx.x / team;
  const bool there = place < p.rows;
  const int64_t row = there ? place : p.rows - 1;  // a team without a row meets the others all the same
  uint4 x16[kPieces], d16[kPieces], a16[kPieces], w16[kPieces];
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const int c = (t + i * team) * 8;
    a16[i] = make_uint4(0, 0, 0, 0);
    w16[i] = ones<kF16>();
    if (c < p.cols) {
      x16[i] = *reinterpret_cast<const uint4*>(p.x + row * p.ldx + c);
      d16[i] = *reinterpret_cast<const uint4*>(p.d_out + row * p.ld_out + c);
      if (p.add) a16[i] = *reinterpret_cast<const uint4*>(p.add + row * p.ld_add + c);
      if (p.weight) w16[i] = __ldg(reinterpret_cast<const uint4*>(p.weight + c));
    }
  }
  const float mean = __ldg(p.mean + row), r = __ldg(p.rstd + row), inv = 1.0f / (float)p.cols;
  Two sum_g = 0, sum_gx = 0;
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    if ((t + i * team) * 8 < p.cols) {
      GradPiece q = grad_piece<kF16>(x16[i], d16[i], mean, r);
      weigh<kF16>(q, w16[i]);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        sum_g = add2(sum_g, q.g[e]);
        sum_gx = fma2(q.g[e], q.x[e], sum_gx);
      }
    }
  }
  float2 v = make_float2(warp_sum(sum2(sum_g)), warp_sum(sum2(sum_gx)));
  if constexpr (kTeamWarps > 1) {
    if (lane == 0) s[warp] = v;
    __syncthreads();
    v = lane < kTeamWarps ? s[warp / kTeamWarps * kTeamWarps + lane] : make_float2(0.0f, 0.0f);
    v = make_float2(warp_sum(v.x), warp_sum(v.y));
  }
  if (!there) return;
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const int c = (t + i * team) * 8;
    if (c < p.cols) {
      GradPiece q = grad_piece<kF16>(x16[i], d16[i], mean, r);
      weigh<kF16>(q, w16[i]);
      *reinterpret_cast<uint4*>(p.dx + row * p.ld_dx + c) = input_grad<kF16>(q, r, v.x * inv, v.y * inv, a16[i]);
    }
  }
}

template <bool kF16>
__device__ __forceinline__ void few_columns(const NormGradParams& p, int block, float (&s)[2][kFewWarps][kFewCols]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, piece = lane % kFewPieces;
  const int64_t col = ((int64_t)block * kFewPieces + piece) * 8;
  constexpr int step = kFewWarps * kFewRowsAWarp;
  Two sum[2][4] = {};
  if (col < p.cols) {
    for (int64_t first = warp * kFewRowsAWarp + lane / kFewPieces; first < p.rows; first += step * kFewUnroll) {
      uint4 x16[kFewUnroll], d16[kFewUnroll];
      float mean[kFewUnroll], r[kFewUnroll];
#pragma unroll
      for (int i = 0; i < kFewUnroll; ++i) {
        const int64_t row = first + i * step;
        if (row < p.rows) {
          x16[i] = *reinterpret_cast<const uint4*>(p.x + row * p.ldx + col);
          d16[i] = *reinterpret_cast<const uint4*>(p.d_out + row * p.ld_out + col);
          mean[i] = __ldg(p.mean + row);
          r[i] = __ldg(p.rstd + row);
        }
      }
#pragma unroll
      for (int i = 0; i < kFewUnroll; ++i) {
        if (first + i * step < p.rows) {
          const GradPiece q = grad_piece<kF16>(x16[i], d16[i], mean[i], r[i]);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            sum[0][e] = fma2(q.g[e], q.x[e], sum[0][e]);
            sum[1][e] = add2(sum[1][e], q.g[e]);
          }
        }
      }
    }
  }
#pragma unroll
  for (int k = 0; k < 2; ++k) {
#pragma unroll
    for (int o = kFewPieces; o < 32; o *= 2)
#pragma unroll
      for (int e = 0; e < 4; ++e) sum[k][e] = add2(sum[k][e], __shfl_xor_sync(0xffffffffu, sum[k][e], o));
    if (lane < kFewPieces) {
      ulonglong2* const mine = reinterpret_cast<ulonglong2*>(&s[k][warp][piece * 8]);
      mine[0] = make_ulonglong2(sum[k][0], sum[k][1]);
      mine[1] = make_ulonglong2(sum[k][2], sum[k][3]);
    }
  }
  __syncthreads();
  const int k = threadIdx.x / kFewCols, c = threadIdx.x % kFewCols;
  const int64_t at = (int64_t)block * kFewCols + c;
  if (k >= 2 || at >= p.cols) return;
  void* const out = k == 0 ? p.d_weight : p.d_bias;
  if (out == nullptr) return;
  float total = s[k][0][c];
#pragma unroll
  for (int i = 1; i < kFewWarps; ++i) total += s[k][i][c];
  store_sum<kF16>(out, at, total, p.out_f32);
}

template <bool kF16, int kTeamWarps, int kPieces>
__global__ void __launch_bounds__(kFewWarps * 32, kPieces == 4 ? 1 : 2) agmm_layer_norm_grad_few(const __grid_constant__ NormGradParams p) {
  __shared__ __align__(16) float s[2][kFewWarps][kFewCols];
  __shared__ float2 team_sums[kFewWarps];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  if ((int)blockIdx.x < p.column_blocks)
    few_columns<kF16>(p, (int)blockIdx.x, s);
  else
    few_rows<kF16, kTeamWarps, kPieces>(p, (int)blockIdx.x - p.column_blocks, team_sums);
}

template <class P>
cudaError_t launch(void (*fn)(P), const P& p, unsigned blocks, int threads, size_t smem, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fn, p);
}

constexpr int kWarpRowPieces = 128;  // rows of up to 1024 values are one warp's

int round_warp(int threads) { return (threads + 31) / 32 * 32; }

// Blocks that stream: two pieces to a thread and two rows to a turn, for the widest rows four
// and one; 512 threads to an SM (their registers); and the turns' rows that each has in flight.
struct Stream {
  int pieces, rows, threads, blocks, stages;
  size_t smem;
};
Stream stream_of(int cols, int inputs) {
  Stream s;
  const int pieces = cols / 8;
  s.pieces = pieces <= 1024 ? 2 : 4;
  s.rows = pieces <= 1024 ? 2 : 1;
  s.threads = round_warp((pieces + s.pieces - 1) / s.pieces);
  s.blocks = 512 / s.threads;
  const size_t turn = (size_t)s.threads * s.pieces * 16 * inputs * s.rows;
  const size_t stages = (kMaxSmem / s.blocks - 1024 - kSumBytes) / turn;
  s.stages = (int)(stages > kMostStages ? kMostStages : stages);
  s.smem = kSumBytes + s.stages * turn;
  return s;
}

template <bool kF16>
cudaError_t launch_norm_t(const NormParams& p, int sms, cudaStream_t stream) {
  const int pieces = p.cols / 8;
  if (pieces <= kWarpRowPieces) {
    const unsigned blocks = (unsigned)((p.rows + kWarpRowWarps - 1) / kWarpRowWarps);
    void (*fn)(NormParams) = pieces <= 32   ? &agmm_layer_norm<kF16, true, 1>
                             : pieces <= 64 ? &agmm_layer_norm<kF16, true, 2>
                                            : &agmm_layer_norm<kF16, true, 4>;
    return launch(fn, p, blocks, 32 * kWarpRowWarps, 0, stream);
  }
  if (p.rows <= 2 * sms && pieces <= 1024)
    return launch(&agmm_layer_norm<kF16, false, 1>, p, (unsigned)p.rows, round_warp(pieces), 0, stream);
  const int threads = round_warp((pieces + 3) / 4);
  if (pieces > 1024) return launch(&agmm_layer_norm<kF16, false, 4>, p, (unsigned)p.rows, threads, 0, stream);
  // twelve blocks to an SM, more than it holds at once: they end apart
  const int64_t blocks = p.rows < (int64_t)sms * 12 ? p.rows : (int64_t)sms * 12;
  return launch(&agmm_layer_norm_rows<kF16>, p, (unsigned)blocks, threads, 0, stream);
}

template <bool kF16>
cudaError_t launch_norm_grad_t(NormGradParams p, int blocks, cudaStream_t stream) {
  const int pieces = p.cols / 8;
  if (pieces <= kWarpRowPieces) {
    void (*fn)(NormGradParams) = pieces <= 32   ? &agmm_layer_norm_grad_short<kF16, 1>
                                 : pieces <= 64 ? &agmm_layer_norm_grad_short<kF16, 2>
                                                : &agmm_layer_norm_grad_short<kF16, 4>;
    return launch(fn, p, (unsigned)blocks, 32 * kWarpRowWarps, (size_t)kWarpRowWarps * 2 * p.cols * sizeof(float), stream);
  }
  const Stream st = stream_of(p.cols, p.add ? 3 : 2);
  p.stages = st.stages;
  void (*fn)(NormGradParams) = st.pieces == 2 ? &agmm_layer_norm_grad<kF16, 2, 2> : &agmm_layer_norm_grad<kF16, 4, 1>;
  return launch(fn, p, (unsigned)blocks, st.threads, st.smem, stream);
}

template <bool kF16>
cudaError_t launch_norm_grad_few_t(NormGradParams p, cudaStream_t stream) {
  const int pieces = p.cols / 8;
  const bool sums = p.d_weight || p.d_bias;
  const int team = pieces <= 32 ? 1 : pieces <= 128 ? 4 : kFewWarps, rows = kFewWarps / team;  // warps to a row, rows to a block
  p.column_blocks = sums ? (p.cols + kFewCols - 1) / kFewCols : 0;  // first: they take longer
  const int blocks = p.column_blocks + (p.dx ? (int)((p.rows + rows - 1) / rows) : 0);
  void (*fn)(NormGradParams) = team == 1        ? &agmm_layer_norm_grad_few<kF16, 1, 1>
                               : team == 4      ? &agmm_layer_norm_grad_few<kF16, 4, 1>
                               : pieces <= 512  ? &agmm_layer_norm_grad_few<kF16, kFewWarps, 1>
                               : pieces <= 1024 ? &agmm_layer_norm_grad_few<kF16, kFewWarps, 2>
                                                : &agmm_layer_norm_grad_few<kF16, kFewWarps, 4>;
  return launch(fn, p, (unsigned)blocks, kFewWarps * 32, 0, stream);
}

}  // namespace

// Backward with a gradient to add and the sums, few rows' way and the other: 256 columns, 768 rows 4.7 and
// 5.0 us, 1024 rows 5.9 and 5.0; 1000 columns, 37 rows 2.1 and 4.6, 768 rows 6.2 and 7.1; 4096 columns,
// 37 rows 2.2 and 7.1, 1024 rows 9.2 and 12.8; 16384 columns, 1024 rows 42 and 47 us.  dx alone is alike.
bool few_norm_rows(int64_t rows, int cols) { return rows <= (cols > 1024 ? 1024 : 768); }

cudaError_t launch_norm_grad_few(const NormGradParams& p, bool f16, cudaStream_t stream) {
  return f16 ? launch_norm_grad_few_t<true>(p, stream) : launch_norm_grad_few_t<false>(p, stream);
}

cudaError_t prepare_norm(bool f16) {
  for (void (*fn)(NormGradParams) : {f16 ? &agmm_layer_norm_grad<true, 2, 2> : &agmm_layer_norm_grad<false, 2, 2>,
                                     f16 ? &agmm_layer_norm_grad<true, 4, 1> : &agmm_layer_norm_grad<false, 4, 1>}) {
    const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMaxSmem);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t launch_norm(const NormParams& p, bool f16, int sms, cudaStream_t stream) {
  return f16 ? launch_norm_t<true>(p, sms, stream) : launch_norm_t<false>(p, sms, stream);
}

int norm_grad_blocks(int64_t rows, int cols, int sms) {
  const int pieces = cols / 8;
  const int64_t teams = pieces <= kWarpRowPieces ? kWarpRowWarps : 1;
  const int64_t most = (rows + teams - 1) / teams;
  const int64_t want = (int64_t)sms * (pieces <= kWarpRowPieces ? 8 : stream_of(cols, 3).blocks);
  return (int)(most < want ? most : want);
}

cudaError_t launch_norm_grad(const NormGradParams& p, bool f16, int blocks, cudaStream_t stream) {
  return f16 ? launch_norm_grad_t<true>(p, blocks, stream) : launch_norm_grad_t<false>(p, blocks, stream);
}

}  // namespace ff
}  // namespace agmm
