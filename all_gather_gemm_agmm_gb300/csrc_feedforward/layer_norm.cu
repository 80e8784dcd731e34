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

template <bool kF16, bool kWarpRow, int kPieces>
__global__ void __launch_bounds__(kWarpRow ? 32 * kWarpRowWarps : 1024 / (kPieces > 1 ? 2 : 1))
    agmm_layer_norm_grad(const __grid_constant__ NormGradParams p) {
  extern __shared__ float shared[];  // 64 sums; short rows: a part of each warp
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int team = kWarpRow ? 32 : blockDim.x;
  const int t = kWarpRow ? threadIdx.x & 31 : threadIdx.x;
  const int teams = kWarpRow ? kWarpRowWarps : 1;
  const int warp = threadIdx.x >> 5;
  const int64_t first = (int64_t)blockIdx.x * teams + (kWarpRow ? warp : 0);
  const int64_t step = (int64_t)gridDim.x * teams;
  const float inv = 1.0f / (float)p.cols;
  float dw[kPieces][8], db[kPieces][8];
  uint4 w16[kPieces];
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const int c = (t + i * team) * 8;
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[i][e] = db[i][e] = 0.0f;
    if (p.weight && c < p.cols) w16[i] = __ldg(reinterpret_cast<const uint4*>(p.weight + c));
  }
  uint4 x16[kPieces], d16[kPieces];
  float mean = 0.0f, rstd = 0.0f;
  auto fetch = [&](int64_t row) {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int c = (t + i * team) * 8;
      if (c < p.cols) {
        x16[i] = __ldcs(reinterpret_cast<const uint4*>(p.x + row * p.ldx + c));
        d16[i] = __ldcs(reinterpret_cast<const uint4*>(p.d_out + row * p.ld_out + c));
      }
    }
    mean = __ldg(p.mean + row);
    rstd = __ldg(p.rstd + row);
  };
  if (first < p.rows) fetch(first);
  int turn = 0;
  for (int64_t row = first; row < p.rows; row += step) {
    float x[kPieces][8], g[kPieces][8];
    const float r = rstd;
    float sum_g = 0.0f, sum_gx = 0.0f;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      if ((t + i * team) * 8 < p.cols) {
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
    if (row + step < p.rows) fetch(row + step);  // in flight beside the sums and the stores
    sum_g = warp_sum(sum_g);
    sum_gx = warp_sum(sum_gx);
    if constexpr (!kWarpRow) {
      // two sets of sums in turn: one barrier a row
      float2* const s = reinterpret_cast<float2*>(shared) + 32 * turn;
      turn ^= 1;
      if ((threadIdx.x & 31) == 0) s[warp] = make_float2(sum_g, sum_gx);
      __syncthreads();
      const float2 v = (int)(threadIdx.x & 31) < (int)(blockDim.x >> 5) ? s[threadIdx.x & 31] : make_float2(0.0f, 0.0f);
      sum_g = warp_sum(v.x);
      sum_gx = warp_sum(v.y);
    }
    if (p.dx) {
      const float mg = sum_g * inv, mgx = sum_gx * inv;
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        const int c = (t + i * team) * 8;
        if (c < p.cols) {
          float a[8];
          if (p.add) unpack8<kF16>(*reinterpret_cast<const uint4*>(p.add + row * p.ld_add + c), a);
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
  float* const part = p.part + (int64_t)blockIdx.x * 2 * p.cols;
  if constexpr (kWarpRow) {
    // the warps' sums, in the order of the warps
    float* const mine = shared + (size_t)warp * 2 * p.cols;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int c = (t + i * team) * 8;
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
      for (int k = 1; k < teams; ++k) sum += shared[(size_t)k * 2 * p.cols + c];
      part[c] = sum;
    }
  } else {
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

template <bool kF16>
cudaError_t launch_norm_t(const NormParams& p, cudaStream_t stream) {
  const int pieces = p.cols / 8;
  if (pieces <= kWarpRowPieces) {
    const unsigned blocks = (unsigned)((p.rows + kWarpRowWarps - 1) / kWarpRowWarps);
    void (*fn)(NormParams) = pieces <= 32   ? &agmm_layer_norm<kF16, true, 1>
                             : pieces <= 64 ? &agmm_layer_norm<kF16, true, 2>
                                            : &agmm_layer_norm<kF16, true, 4>;
    return launch(fn, p, blocks, 32 * kWarpRowWarps, 0, stream);
  }
  if (pieces <= 512) return launch(&agmm_layer_norm<kF16, false, 2>, p, (unsigned)p.rows, round_warp((pieces + 1) / 2), 0, stream);
  return launch(&agmm_layer_norm<kF16, false, 4>, p, (unsigned)p.rows, round_warp((pieces + 3) / 4), 0, stream);
}

int grad_threads(int pieces) {
  if (pieces <= kWarpRowPieces) return 32 * kWarpRowWarps;
  return pieces <= 1024 ? round_warp(pieces) : 512;
}

template <bool kF16>
cudaError_t launch_norm_grad_t(const NormGradParams& p, int blocks, cudaStream_t stream) {
  const int pieces = p.cols / 8, threads = grad_threads(pieces);
  if (pieces <= kWarpRowPieces) {
    void (*fn)(NormGradParams) = pieces <= 32   ? &agmm_layer_norm_grad<kF16, true, 1>
                                 : pieces <= 64 ? &agmm_layer_norm_grad<kF16, true, 2>
                                                : &agmm_layer_norm_grad<kF16, true, 4>;
    return launch(fn, p, (unsigned)blocks, threads, (size_t)kWarpRowWarps * 2 * p.cols * sizeof(float), stream);
  }
  if (pieces <= 1024) return launch(&agmm_layer_norm_grad<kF16, false, 1>, p, (unsigned)blocks, threads, 64 * sizeof(float2), stream);
  return launch(&agmm_layer_norm_grad<kF16, false, 4>, p, (unsigned)blocks, threads, 64 * sizeof(float2), stream);
}

}  // namespace

cudaError_t launch_norm(const NormParams& p, bool f16, cudaStream_t stream) {
  return f16 ? launch_norm_t<true>(p, stream) : launch_norm_t<false>(p, stream);
}

int norm_grad_blocks(int64_t rows, int cols, int sms) {
  const int pieces = cols / 8, threads = grad_threads(pieces);
  const int64_t teams = pieces <= kWarpRowPieces ? kWarpRowWarps : 1;
  const int64_t most = (rows + teams - 1) / teams;
  const int64_t want = (int64_t)sms * (threads >= 512 ? 1 : 1024 / threads);
  return (int)(most < want ? most : want);
}

cudaError_t launch_norm_grad(const NormGradParams& p, bool f16, int blocks, cudaStream_t stream) {
  return f16 ? launch_norm_grad_t<true>(p, blocks, stream) : launch_norm_grad_t<false>(p, blocks, stream);
}

}  // namespace ff
}  // namespace agmm
