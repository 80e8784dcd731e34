// ff_pointwise.cu -- the elementwise steps of the feed-forward operators' backward
// passes, and the sums over tokens.
//
//   gated   d_gate = d_out * up * act'(gate),  d_up = d_out * act(gate)
//   linear  d_pre = d_out * act'(pre),  d_bias = sum over tokens of d_pre
//
// The results are rounded to the operands' 16-bit type: the tensor cores multiply them next.
// Bound: device memory.  A thread keeps its 8 columns and walks down the rows, so that
// sums of columns stay in its registers; the blocks' sums are added in a fixed order.
// Measured: gated silu, 8192 x 7168: 88 us, 6.7 TB/s (four blocks to an SM; with three, 98 us).
// Linear gelu with sums, 4096 x 5120: 28 us with the parts' 4 us, 4.5 TB/s (64 registers and one wave
// of blocks; with 80 and two waves 31 us): two exponentials to a value take 9 us of the
// special-function units, and the arithmetic 11 us.
#include "ff_math.cuh"
#include "ptx_sm103.cuh"

namespace agmm {
namespace ff {
namespace {

// 8 values that the forward pass saved, in 16 bits or in float32.
template <bool kSavedF32>
struct Saved {
  uint4 v[kSavedF32 ? 2 : 1];
  // plain loads: the gradients may lie over what was saved
  __device__ __forceinline__ void load(const void* p, int64_t at) {
    if constexpr (kSavedF32) {
      const uint4* const q = reinterpret_cast<const uint4*>(static_cast<const float*>(p) + at);
      v[0] = q[0];
      v[1] = q[1];
    } else {
      v[0] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + at);
    }
  }
  template <bool kF16>
  __device__ __forceinline__ void values(Two (&x)[4]) const {
    if constexpr (kSavedF32) {
      x[0] = two(__uint_as_float(v[0].x), __uint_as_float(v[0].y));
      x[1] = two(__uint_as_float(v[0].z), __uint_as_float(v[0].w));
      x[2] = two(__uint_as_float(v[1].x), __uint_as_float(v[1].y));
      x[3] = two(__uint_as_float(v[1].z), __uint_as_float(v[1].w));
    } else {
      widen<kF16>(v[0], x);
    }
  }
};

template <bool kF16, int kAct, bool kSavedF32>
__device__ __forceinline__ void gated_grad_piece(const uint4& d16, const Saved<kSavedF32>& gs, const Saved<kSavedF32>& us, uint4& dg, uint4& du) {
  Two d[4], g[4], u[4];
  widen<kF16>(d16, d);
  gs.template values<kF16>(g);
  us.template values<kF16>(u);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    Two a, slope;
    activate_with_slope<kAct>(g[i], a, slope);
    g[i] = mul2(mul2(d[i], u[i]), slope);
    u[i] = mul2(d[i], a);
  }
  dg = narrow<kF16>(g);
  du = narrow<kF16>(u);
}

constexpr int kUnroll = 2, kActUnroll = 4;  // rows whose loads are in flight together (float32: half as many)

template <bool kF16, bool kSavedF32>
__global__ void __launch_bounds__(256, 4) agmm_gated_grad(const __grid_constant__ GatedGradParams p) {
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int64_t col = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) * 8;
  if (col >= p.cols) return;
  constexpr int kRows = kSavedF32 ? kUnroll / 2 : kUnroll;
  with_activation(p.act, [&](auto act) {
    const int64_t step = gridDim.y;
    for (int64_t r = blockIdx.y; r < p.rows; r += step * kRows) {
      uint4 d[kRows];
      Saved<kSavedF32> g[kRows], u[kRows];
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const int64_t row = r + i * step;
        if (row < p.rows) {
          d[i] = *reinterpret_cast<const uint4*>(p.d_out + row * p.ld_out + col);
          g[i].load(p.gate, row * p.ld_saved + col);
          u[i].load(p.up, row * p.ld_saved + col);
        }
      }
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const int64_t row = r + i * step;
        if (row < p.rows) {
          uint4 dg, du;
          gated_grad_piece<kF16, act.value, kSavedF32>(d[i], g[i], u[i], dg, du);
          *reinterpret_cast<uint4*>(p.d_gate + row * p.ld_grad + col) = dg;
          *reinterpret_cast<uint4*>(p.d_up + row * p.ld_grad + col) = du;
        }
      }
    }
  });
}

// Rows first, first + step, ... of 8 columns, and their sums.
template <bool kF16, bool kSavedF32>
__device__ __forceinline__ void act_grad_rows(const ActGradParams& p, int64_t col, int64_t first, int64_t step, Two (&sum)[4]) {
  constexpr int kRows = kSavedF32 ? kActUnroll / 2 : kActUnroll;
  with_activation(p.act, [&](auto act) {
    for (int64_t r = first; r < p.rows; r += step * kRows) {
      uint4 d[kRows];
      Saved<kSavedF32> z[kRows];
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const int64_t row = r + i * step;
        if (row < p.rows) {
          d[i] = *reinterpret_cast<const uint4*>(p.d_out + row * p.ld_out + col);
          if constexpr (act.value != kActNone) z[i].load(p.pre, row * p.ld_pre + col);
        }
      }
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const int64_t row = r + i * step;
        if (row < p.rows) {
          Two dv[4];
          widen<kF16>(d[i], dv);
          if constexpr (act.value != kActNone) {
            Two zv[4];
            z[i].template values<kF16>(zv);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              Two a, slope;
              activate_with_slope<act.value>(zv[e], a, slope);
              dv[e] = mul2(dv[e], slope);
            }
            *reinterpret_cast<uint4*>(p.d_pre + row * p.ld_grad + col) = narrow<kF16>(dv);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) sum[e] = add2(sum[e], dv[e]);
        }
      }
    }
  });
}

template <bool kF16, bool kSavedF32>
__global__ void __launch_bounds__(256, 4) agmm_act_grad(const __grid_constant__ ActGradParams p) {
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int64_t col = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) * 8;
  if (col >= p.cols) return;
  Two sum[4] = {0, 0, 0, 0};
  act_grad_rows<kF16, kSavedF32>(p, col, blockIdx.y, gridDim.y, sum);
  if (p.part) {
    ulonglong2* const dst = reinterpret_cast<ulonglong2*>(p.part + (int64_t)blockIdx.y * p.cols + col);
    dst[0] = make_ulonglong2(sum[0], sum[1]);
    dst[1] = make_ulonglong2(sum[2], sum[3]);
  }
}

// Few rows, with their sums: 64 columns to a block, four rows to a warp, whose sums meet in shared
// memory.  No parts and no second launch.
constexpr int kFewWarps = 16, kFewPieces = 8, kFewCols = kFewPieces * 8, kFewRowsAWarp = 32 / kFewPieces;
static_assert(kFewWarps * 32 >= kFewCols, "a thread for each column's sum");

template <bool kF16, bool kSavedF32>
__global__ void __launch_bounds__(kFewWarps * 32) agmm_act_grad_few(const __grid_constant__ ActGradParams p) {
  __shared__ __align__(16) float s[kFewWarps][kFewCols];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, piece = lane % kFewPieces;
  const int64_t col = ((int64_t)blockIdx.x * kFewPieces + piece) * 8;
  Two sum[4] = {0, 0, 0, 0};
  if (col < p.cols) act_grad_rows<kF16, kSavedF32>(p, col, warp * kFewRowsAWarp + lane / kFewPieces, kFewWarps * kFewRowsAWarp, sum);
#pragma unroll
  for (int o = kFewPieces; o < 32; o *= 2)
#pragma unroll
    for (int e = 0; e < 4; ++e) sum[e] = add2(sum[e], __shfl_xor_sync(0xffffffffu, sum[e], o));
  if (lane < kFewPieces) {
    ulonglong2* const mine = reinterpret_cast<ulonglong2*>(&s[warp][piece * 8]);
    mine[0] = make_ulonglong2(sum[0], sum[1]);
    mine[1] = make_ulonglong2(sum[2], sum[3]);
  }
  __syncthreads();
  const int64_t c = (int64_t)blockIdx.x * kFewCols + threadIdx.x;
  if (threadIdx.x >= kFewCols || c >= p.cols) return;
  float total = s[0][threadIdx.x];
#pragma unroll
  for (int i = 1; i < kFewWarps; ++i) total += s[i][threadIdx.x];
  store_sum<kF16>(p.d_bias, c, total, p.out_f32);
}

// 32 columns to a block, their parts dealt to its 16 warps.
constexpr int kSumWarps = 16;

template <bool kF16>
__global__ void __launch_bounds__(kSumWarps * 32) agmm_sum_parts(const __grid_constant__ SumPartsParams p) {
  __shared__ float s[kSumWarps][32];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  if (p.out[blockIdx.y] == nullptr) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t col = (int64_t)blockIdx.x * 32 + lane;
  float sum = 0.0f;
  if (col < p.cols) {
    const float* const src = p.part + (int64_t)blockIdx.y * p.cols + col;
    const int64_t stride = (int64_t)p.sums * p.cols;
#pragma unroll 8
    for (int i = warp; i < p.parts; i += kSumWarps) sum += __ldcg(src + i * stride);
  }
  s[warp][lane] = sum;
  __syncthreads();
  if (warp == 0 && col < p.cols) {
#pragma unroll
    for (int i = 1; i < kSumWarps; ++i) sum += s[i][lane];
    store_sum<kF16>(p.out[blockIdx.y], col, sum, p.out_f32);
  }
}

template <class P>
cudaError_t launch(void (*fn)(P), const P& p, dim3 grid, int threads, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fn, p);
}

// Threads of a block: the fewest idle ones beside the last columns.
int threads_for(int64_t pieces) {
  const int64_t blocks = (pieces + 255) / 256;
  return (int)(((pieces + blocks - 1) / blocks + 31) / 32 * 32);
}

}  // namespace

cudaError_t launch_gated_grad(const GatedGradParams& p, bool f16, int sms, cudaStream_t stream) {
  const int64_t pieces = p.cols / 8;
  const int threads = threads_for(pieces);
  const int64_t x = (pieces + threads - 1) / threads;
  // enough blocks for 2048 threads on every SM twice over, and no more rows than there are
  int64_t y = (int64_t)sms * 2 * (2048 / threads) / x;
  y = y < 1 ? 1 : y;
  const int64_t most = (p.rows + kUnroll - 1) / kUnroll;
  if (y > most) y = most;
  if (y > 65535) y = 65535;
  const dim3 grid((unsigned)x, (unsigned)y);
  if (p.saved_f32) return launch(f16 ? &agmm_gated_grad<true, true> : &agmm_gated_grad<false, true>, p, grid, threads, stream);
  return launch(f16 ? &agmm_gated_grad<true, false> : &agmm_gated_grad<false, false>, p, grid, threads, stream);
}

int act_grad_row_blocks(int64_t rows, int64_t cols, int sms) {
  const int64_t pieces = cols / 8;
  const int threads = threads_for(pieces);
  const int64_t x = (pieces + threads - 1) / threads;
  int64_t y = (int64_t)sms * (1024 / threads) / x;  // one wave: 64 registers a thread
  y = y < 1 ? 1 : y;
  const int64_t most = (rows + kUnroll - 1) / kUnroll;
  if (y > most) y = most;
  return (int)(y > 1024 ? 1024 : y);
}

cudaError_t launch_act_grad(const ActGradParams& p, bool f16, cudaStream_t stream) {
  if (p.d_bias) {
    const dim3 few((unsigned)((p.cols + kFewCols - 1) / kFewCols));
    if (p.saved_f32) return launch(f16 ? &agmm_act_grad_few<true, true> : &agmm_act_grad_few<false, true>, p, few, kFewWarps * 32, stream);
    return launch(f16 ? &agmm_act_grad_few<true, false> : &agmm_act_grad_few<false, false>, p, few, kFewWarps * 32, stream);
  }
  const int64_t pieces = p.cols / 8;
  const int threads = threads_for(pieces);
  const dim3 grid((unsigned)((pieces + threads - 1) / threads), (unsigned)p.row_blocks);
  if (p.saved_f32) return launch(f16 ? &agmm_act_grad<true, true> : &agmm_act_grad<false, true>, p, grid, threads, stream);
  return launch(f16 ? &agmm_act_grad<true, false> : &agmm_act_grad<false, false>, p, grid, threads, stream);
}

cudaError_t launch_sum_parts(const SumPartsParams& p, bool f16, cudaStream_t stream) {
  const dim3 grid((unsigned)((p.cols + 31) / 32), (unsigned)p.sums);
  return launch(f16 ? &agmm_sum_parts<true> : &agmm_sum_parts<false>, p, grid, kSumWarps * 32, stream);
}

}  // namespace ff
}  // namespace agmm
