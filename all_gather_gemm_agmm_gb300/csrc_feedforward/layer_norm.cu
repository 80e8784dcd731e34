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
// registers while it walks over the rows, and each block leaves one part of them.
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

// The sum over a team: a warp, or the whole block (`s` has room for a value of each warp).
template <bool kWarpRow>
__device__ __forceinline__ float team_sum(float v, float* s) {
  v = warp_sum(v);
  if constexpr (!kWarpRow) {
    const int warps = blockDim.x >> 5;
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
    __syncthreads();
    v = (int)(threadIdx.x & 31) < warps ? s[threadIdx.x & 31] : 0.0f;
    v = warp_sum(v);
  }
  return v;
}

constexpr int kWarpRowWarps = 4;

template <bool kF16, bool kWarpRow, int kPieces>
__global__ void __launch_bounds__(kWarpRow ? 32 * kWarpRowWarps : 512) agmm_layer_norm(const __grid_constant__ NormParams p) {
  __shared__ float s[32];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int team = kWarpRow ? 32 : blockDim.x;
  const int t = kWarpRow ? threadIdx.x & 31 : threadIdx.x;
  const int64_t row = kWarpRow ? (int64_t)blockIdx.x * kWarpRowWarps + (threadIdx.x >> 5) : blockIdx.x;
  if (row >= p.rows) return;
  uint4 in[kPieces];
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const int c = (t + i * team) * 8;
    if (c < p.cols) in[i] = *reinterpret_cast<const uint4*>(p.x + row * p.ldx + c);
  }
  float x[kPieces][8];
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    if ((t + i * team) * 8 < p.cols) {
      unpack8<kF16>(in[i], x[i]);
#pragma unroll
      for (int e = 0; e < 8; ++e) sum += x[i][e];
    }
  }
  const float inv = 1.0f / (float)p.cols;
  const float mean = team_sum<kWarpRow>(sum, s) * inv;
  float squares = 0.0f;
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    if ((t + i * team) * 8 < p.cols) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[i][e] -= mean;
        squares += x[i][e] * x[i][e];
      }
    }
  }
  const float rstd = rsqrtf(team_sum<kWarpRow>(squares, s) * inv + p.eps);
  if (t == 0) {
    if (p.mean) p.mean[row] = mean;
    if (p.rstd) p.rstd[row] = rstd;
  }
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const int c = (t + i * team) * 8;
    if (c < p.cols) {
      float w[8], b[8];
      if (p.weight) unpack8<kF16>(__ldg(reinterpret_cast<const uint4*>(p.weight + c)), w);
      if (p.bias) unpack8<kF16>(__ldg(reinterpret_cast<const uint4*>(p.bias + c)), b);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[i][e] *= rstd;
        if (p.weight) x[i][e] *= w[e];
        if (p.bias) x[i][e] += b[e];
      }
      *reinterpret_cast<uint4*>(p.out + row * p.ldo + c) = pack8<kF16>(x[i]);
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

template <bool kF16, int kPieces>
__global__ void __launch_bounds__(512, kPieces > 2 ? 1 : 2) agmm_layer_norm_stream(const __grid_constant__ NormParams p) {
  extern __shared__ __align__(16) uint8_t shared[];
  float* const s = reinterpret_cast<float*>(shared);
  uint4* const ring = reinterpret_cast<uint4*>(shared + kSumBytes);
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int t = threadIdx.x, team = blockDim.x, stages = p.stages;
  const int64_t step = gridDim.x;
  auto fetch = [&](int64_t row, int stage) {
    if (row < p.rows) {
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        const int c = (t + i * team) * 8;
        if (c < p.cols) copy_async(ring + (stage * kPieces + i) * team + t, p.x + row * p.ldx + c);
      }
    }
    copy_commit();
  };
  uint4 w16[kPieces], b16[kPieces];
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const int c = (t + i * team) * 8;
    if (p.weight && c < p.cols) w16[i] = __ldg(reinterpret_cast<const uint4*>(p.weight + c));
    if (p.bias && c < p.cols) b16[i] = __ldg(reinterpret_cast<const uint4*>(p.bias + c));
  }
  for (int k = 0; k < stages - 1; ++k) fetch(blockIdx.x + k * step, k);
  const float inv = 1.0f / (float)p.cols;
  int stage = 0;
  for (int64_t row = blockIdx.x; row < p.rows; row += step) {
    fetch(row + (stages - 1) * step, stage == 0 ? stages - 1 : stage - 1);
    copy_wait(stages - 1);
    float x[kPieces][8], sum = 0.0f, squares = 0.0f;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      if ((t + i * team) * 8 < p.cols) {
        unpack8<kF16>(ring[(stage * kPieces + i) * team + t], x[i]);
#pragma unroll
        for (int e = 0; e < 8; ++e) sum += x[i][e];
      }
    }
    const float mean = team_sum<false>(sum, s) * inv;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      if ((t + i * team) * 8 < p.cols) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          x[i][e] -= mean;
          squares += x[i][e] * x[i][e];
        }
      }
    }
    const float rstd = rsqrtf(team_sum<false>(squares, s + 32) * inv + p.eps);
    if (t == 0) {
      if (p.mean) p.mean[row] = mean;
      if (p.rstd) p.rstd[row] = rstd;
    }
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int c = (t + i * team) * 8;
      if (c < p.cols) {
        float w[8], b[8];
        if (p.weight) unpack8<kF16>(w16[i], w);
        if (p.bias) unpack8<kF16>(b16[i], b);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          x[i][e] *= rstd;
          if (p.weight) x[i][e] *= w[e];
          if (p.bias) x[i][e] += b[e];
        }
        *reinterpret_cast<uint4*>(p.out + row * p.ldo + c) = pack8<kF16>(x[i]);
      }
    }
    stage = stage + 1 == stages ? 0 : stage + 1;
  }
}

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
  float dw[kPieces][8], db[kPieces][8];
  uint4 w16[kPieces];
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const int c = (t + i * 32) * 8;
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[i][e] = db[i][e] = 0.0f;
    if (p.weight && c < p.cols) w16[i] = __ldg(reinterpret_cast<const uint4*>(p.weight + c));
  }
#pragma unroll 1
  for (int64_t row = (int64_t)blockIdx.x * kWarpRowWarps + warp; row < p.rows; row += step) {
    uint4 x16[kPieces], d16[kPieces], a16[kPieces];
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int c = (t + i * 32) * 8;
      if (c < p.cols) {
        x16[i] = *reinterpret_cast<const uint4*>(p.x + row * p.ldx + c);
        d16[i] = *reinterpret_cast<const uint4*>(p.d_out + row * p.ld_out + c);
        if (p.add) a16[i] = *reinterpret_cast<const uint4*>(p.add + row * p.ld_add + c);
      }
    }
    const float mean = __ldg(p.mean + row), r = __ldg(p.rstd + row);
    float x[kPieces][8], g[kPieces][8];
    float sum_g = 0.0f, sum_gx = 0.0f;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      if ((t + i * 32) * 8 < p.cols) {
        float w[8];
        unpack8<kF16>(x16[i], x[i]);
        unpack8<kF16>(d16[i], g[i]);
        if (p.weight) unpack8<kF16>(w16[i], w);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          x[i][e] = (x[i][e] - mean) * r;
          dw[i][e] += g[i][e] * x[i][e];
          db[i][e] += g[i][e];
          if (p.weight) g[i][e] *= w[e];
          sum_g += g[i][e];
          sum_gx += g[i][e] * x[i][e];
        }
      }
    }
    if (p.dx) {
      const float mg = warp_sum(sum_g) * inv, mgx = warp_sum(sum_gx) * inv;
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        const int c = (t + i * 32) * 8;
        if (c < p.cols) {
          float a[8];
          if (p.add) unpack8<kF16>(a16[i], a);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            g[i][e] = r * (g[i][e] - mg - x[i][e] * mgx);
            if (p.add) g[i][e] += a[e];
          }
          *reinterpret_cast<uint4*>(p.dx + row * p.ld_dx + c) = pack8<kF16>(g[i]);
        }
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
      for (int e = 0; e < 8; ++e) {
        mine[c + e] = dw[i][e];
        mine[p.cols + c + e] = db[i][e];
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

// Other rows: a block to a row, the rows streaming through shared memory.
template <bool kF16, int kPieces>
__global__ void __launch_bounds__(512, 1) agmm_layer_norm_grad(const __grid_constant__ NormGradParams p) {
  extern __shared__ __align__(16) uint8_t shared[];
  uint4* const ring = reinterpret_cast<uint4*>(shared + kSumBytes);
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int t = threadIdx.x, warp = threadIdx.x >> 5, team = blockDim.x, stages = p.stages;
  const int inputs = p.add ? 3 : 2;
  const int64_t step = gridDim.x;
  const float inv = 1.0f / (float)p.cols;
  auto slot = [&](int stage, int input, int i) { return ring + ((stage * inputs + input) * kPieces + i) * team + t; };
  auto fetch = [&](int64_t row, int stage) {
    if (row < p.rows) {
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        const int c = (t + i * team) * 8;
        if (c < p.cols) {
          copy_async(slot(stage, 0, i), p.x + row * p.ldx + c);
          copy_async(slot(stage, 1, i), p.d_out + row * p.ld_out + c);
          if (p.add) copy_async(slot(stage, 2, i), p.add + row * p.ld_add + c);
        }
      }
    }
    copy_commit();
  };
  float dw[kPieces][8], db[kPieces][8];
  uint4 w16[kPieces];
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const int c = (t + i * team) * 8;
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[i][e] = db[i][e] = 0.0f;
    if (p.weight && c < p.cols) w16[i] = __ldg(reinterpret_cast<const uint4*>(p.weight + c));
  }
  for (int k = 0; k < stages - 1; ++k) fetch(blockIdx.x + k * step, k);
  float next_mean = __ldg(p.mean + blockIdx.x), next_rstd = __ldg(p.rstd + blockIdx.x);
  int stage = 0, turn = 0;
#pragma unroll 1
  for (int64_t row = blockIdx.x; row < p.rows; row += step) {
    fetch(row + (stages - 1) * step, stage == 0 ? stages - 1 : stage - 1);
    const float mean = next_mean, r = next_rstd;
    if (row + step < p.rows) {
      next_mean = __ldg(p.mean + row + step);
      next_rstd = __ldg(p.rstd + row + step);
    }
    copy_wait(stages - 1);
    float sum_g = 0.0f, sum_gx = 0.0f;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      if ((t + i * team) * 8 < p.cols) {
        float x[8], g[8], w[8];
        unpack8<kF16>(*slot(stage, 0, i), x);
        unpack8<kF16>(*slot(stage, 1, i), g);
        if (p.weight) unpack8<kF16>(w16[i], w);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          x[e] = (x[e] - mean) * r;
          dw[i][e] += g[e] * x[e];
          db[i][e] += g[e];
          if (p.weight) g[e] *= w[e];
          sum_g += g[e];
          sum_gx += g[e] * x[e];
        }
      }
    }
    if (p.dx) {
      // two sets of sums in turn: one barrier a row
      float2* const s = reinterpret_cast<float2*>(shared) + 32 * turn;
      turn ^= 1;
      sum_g = warp_sum(sum_g);
      sum_gx = warp_sum(sum_gx);
      if ((t & 31) == 0) s[warp] = make_float2(sum_g, sum_gx);
      __syncthreads();
      const float2 v = (t & 31) < (int)(blockDim.x >> 5) ? s[t & 31] : make_float2(0.0f, 0.0f);
      const float mg = warp_sum(v.x) * inv, mgx = warp_sum(v.y) * inv;
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        const int c = (t + i * team) * 8;
        if (c < p.cols) {
          // read again rather than held: registers
          float x[8], g[8], w[8], a[8];
          unpack8<kF16>(*slot(stage, 0, i), x);
          unpack8<kF16>(*slot(stage, 1, i), g);
          if (p.weight) unpack8<kF16>(w16[i], w);
          if (p.add) unpack8<kF16>(*slot(stage, 2, i), a);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            x[e] = (x[e] - mean) * r;
            if (p.weight) g[e] *= w[e];
            g[e] = r * (g[e] - mg - x[e] * mgx);
            if (p.add) g[e] += a[e];
          }
          *reinterpret_cast<uint4*>(p.dx + row * p.ld_dx + c) = pack8<kF16>(g);
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
      for (int e = 0; e < 8; e += 4) {
        *reinterpret_cast<float4*>(part + c + e) = make_float4(dw[i][e], dw[i][e + 1], dw[i][e + 2], dw[i][e + 3]);
        *reinterpret_cast<float4*>(part + p.cols + c + e) = make_float4(db[i][e], db[i][e + 1], db[i][e + 2], db[i][e + 3]);
      }
    }
  }
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

// Blocks that stream: two or four pieces to a thread, at most 512 threads.
int stream_pieces(int pieces) { return pieces <= 1024 ? 2 : 4; }
int stream_threads(int pieces) { return round_warp((pieces + stream_pieces(pieces) - 1) / stream_pieces(pieces)); }

// Blocks of an SM, by their threads: 1024 threads at least (512 for the widest rows), and the
// rows that each has in flight.
int stream_blocks(int pieces, int most_threads) {
  const int blocks = most_threads / stream_threads(pieces);
  return blocks < 1 ? 1 : blocks > 8 ? 8 : blocks;
}
int stream_stages(int pieces, int blocks, int inputs) {
  const int bytes = stream_threads(pieces) * stream_pieces(pieces) * 16 * inputs;
  const int stages = ((int)kMaxSmem / blocks - 1024 - kSumBytes) / bytes;
  return stages > kMostStages ? kMostStages : stages;
}

template <bool kF16>
cudaError_t launch_norm_t(NormParams p, int sms, cudaStream_t stream) {
  const int pieces = p.cols / 8;
  if (pieces <= kWarpRowPieces) {
    const unsigned blocks = (unsigned)((p.rows + kWarpRowWarps - 1) / kWarpRowWarps);
    void (*fn)(NormParams) = pieces <= 32   ? &agmm_layer_norm<kF16, true, 1>
                             : pieces <= 64 ? &agmm_layer_norm<kF16, true, 2>
                                            : &agmm_layer_norm<kF16, true, 4>;
    return launch(fn, p, blocks, 32 * kWarpRowWarps, 0, stream);
  }
  const int per_sm = stream_blocks(pieces, pieces <= 1024 ? 1024 : 512);
  if (p.rows > (int64_t)sms * per_sm) {
    p.stages = stream_stages(pieces, per_sm, 1);
    const int threads = stream_threads(pieces);
    const size_t smem = kSumBytes + (size_t)p.stages * threads * stream_pieces(pieces) * 16;
    void (*fn)(NormParams) = pieces <= 1024 ? &agmm_layer_norm_stream<kF16, 2> : &agmm_layer_norm_stream<kF16, 4>;
    const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMaxSmem);
    if (e != cudaSuccess) return e;
    return launch(fn, p, (unsigned)(sms * per_sm), threads, smem, stream);
  }
  if (pieces <= 512) return launch(&agmm_layer_norm<kF16, false, 1>, p, (unsigned)p.rows, round_warp(pieces), 0, stream);
  return launch(&agmm_layer_norm<kF16, false, 4>, p, (unsigned)p.rows, round_warp((pieces + 3) / 4), 0, stream);
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
  const int threads = stream_threads(pieces), inputs = p.add ? 3 : 2;
  p.stages = stream_stages(pieces, stream_blocks(pieces, 512), inputs);
  const size_t smem = kSumBytes + (size_t)p.stages * threads * stream_pieces(pieces) * 16 * inputs;
  void (*fn)(NormGradParams) = pieces <= 1024 ? &agmm_layer_norm_grad<kF16, 2> : &agmm_layer_norm_grad<kF16, 4>;
  const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMaxSmem);
  if (e != cudaSuccess) return e;
  return launch(fn, p, (unsigned)blocks, threads, smem, stream);
}

}  // namespace

cudaError_t launch_norm(const NormParams& p, bool f16, int sms, cudaStream_t stream) {
  return f16 ? launch_norm_t<true>(p, sms, stream) : launch_norm_t<false>(p, sms, stream);
}

int norm_grad_blocks(int64_t rows, int cols, int sms) {
  const int pieces = cols / 8;
  const int64_t teams = pieces <= kWarpRowPieces ? kWarpRowWarps : 1;
  const int64_t most = (rows + teams - 1) / teams;
  const int64_t want = (int64_t)sms * (pieces <= kWarpRowPieces ? 8 : stream_blocks(pieces, 512));
  return (int)(most < want ? most : want);
}

cudaError_t launch_norm_grad(const NormGradParams& p, bool f16, int blocks, cudaStream_t stream) {
  return f16 ? launch_norm_grad_t<true>(p, blocks, stream) : launch_norm_grad_t<false>(p, blocks, stream);
}

}  // namespace ff
}  // namespace agmm
