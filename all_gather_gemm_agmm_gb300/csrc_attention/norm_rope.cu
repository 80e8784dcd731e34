// norm_rope.cu -- RMS norm of every query and key head, the rotation by the
// token's position, and the writes of keys and values to cache slots, in one
// pass over the rows of a QKV product.
//
//   y = x * rsqrt(mean(x^2) + eps) * w,   (a, b) -> (a cos - b sin, b cos + a sin)
//
// Bound: device memory (each value is read once and written once per
// destination; about 8 flops per value).  One block per token: the token's
// angles are computed once, by one thread per pair, and shared by all its
// heads.  A head is held by head_dim / 16 lanes, each with two 16-byte pieces
// chosen so that both values of every pair sit in one lane: the rotation needs
// no exchange, and the norm one butterfly over those lanes.
//
// Angles: position * (inv_freq / 2 pi) in float64, reduced to a fraction of a
// turn there and rounded to float32 only then, so that the error of the angle
// does not grow with the position (a float32 product is off by up to
// position * 2^-24 radians).
//
// Measured: 16384 tokens of 80 heads of 128: 129 us, 5.5 TB/s.  In one build: 127 us; blocks
// of 256 threads 142 us; of 512: 226 us; of 64: 137 us at best.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "attn_params.h"

namespace agmm {
namespace {

constexpr int kThreads = 128;
constexpr int kInFlight = 3;  // heads a thread loads before it works on the first

template <bool kF16>
__device__ __forceinline__ void unpack8(const uint4& u, float (&x)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float2 f;
    if constexpr (kF16)
      f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    else
      f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]));
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}

template <bool kF16>
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (kF16) {
      const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    } else {
      const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <int kD, bool kF16>
__global__ void __launch_bounds__(kThreads, 8) agmm_norm_rope(const __grid_constant__ NormRopeParams p) {
  constexpr int kLanes = kD / 16;            // lanes per head
  constexpr int kGroups = kThreads / kLanes;  // heads in flight per block
  __shared__ float s_cos[kD / 2], s_sin[kD / 2];
  const int64_t t = blockIdx.x;
  const int lane = threadIdx.x % kLanes;
  const int group = threadIdx.x / kLanes;

  // This lane's two pieces, and the first of the 8 pairs they hold.
  const int rot_lanes = p.pairs / 8;  // lanes that rotate
  const bool rotates = lane < rot_lanes;
  const bool split = rotates && !p.adjacent;
  const int e0 = split ? lane * 8 : lane * 16;
  const int e1 = split ? lane * 8 + p.pairs : lane * 16 + 8;

  const int norm_heads = p.q_heads + p.kv_heads;
  const int heads = norm_heads + (p.v_cache ? p.kv_heads : 0);
  const uint16_t* const row = p.qkv + t * p.qkv_ts;

  uint4 in[kInFlight][2];
#pragma unroll
  for (int u = 0; u < kInFlight; ++u) {
    const int h = group + u * kGroups;
    if (h < heads) {
      const uint16_t* const x = row + h * p.qkv_hs;
      in[u][0] = *reinterpret_cast<const uint4*>(x + e0);
      in[u][1] = *reinterpret_cast<const uint4*>(x + e1);
    }
  }
  int64_t slot = -1;
  if (p.k_cache) slot = p.slots[t];

  static_assert(kD / 2 <= kThreads, "a thread for every pair");
  if ((int)threadIdx.x < p.pairs) {
    const int i = threadIdx.x;
    const int64_t at = (int64_t)p.axis[i] * p.position_axis_stride + t;
    const double pos = p.position64 ? (double)static_cast<const int64_t*>(p.positions)[at]
                                    : (double)static_cast<const int32_t*>(p.positions)[at];
    const double turns = pos * p.turns[i];
    float s, c;
    sincospif(2.0f * (float)(turns - rint(turns)), &s, &c);
    s_cos[i] = c;
    s_sin[i] = s;
  }
  __syncthreads();
  float cs[8], sn[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    cs[i] = rotates ? s_cos[lane * 8 + i] : 1.0f;
    sn[i] = rotates ? s_sin[lane * 8 + i] : 0.0f;
  }

  const bool cached = slot >= 0 && slot < p.num_slots;
  int64_t cache_at = 0;
  if (cached) {
    const int64_t page = p.page_shift >= 0 ? slot >> p.page_shift : slot / p.page_size;
    cache_at = page * p.cache_ps + (slot - page * p.page_size) * p.cache_ts;
  }

  for (int h0 = group; h0 < heads; h0 += kInFlight * kGroups) {
#pragma unroll
    for (int u = 0; u < kInFlight; ++u) {
      const int h = h0 + u * kGroups;
      if (h >= heads) break;  // the lanes of a head leave together
      const uint16_t* const x = row + h * p.qkv_hs;
      uint4 a = in[u][0], b = in[u][1];
      if (h0 != group) {
        a = *reinterpret_cast<const uint4*>(x + e0);
        b = *reinterpret_cast<const uint4*>(x + e1);
      }
      if (h >= norm_heads) {
        if (cached) {
          uint16_t* const dst = p.v_cache + cache_at + (h - norm_heads) * p.cache_hs;
          *reinterpret_cast<uint4*>(dst + e0) = a;
          *reinterpret_cast<uint4*>(dst + e1) = b;
        }
        continue;
      }
      float xa[8], xb[8];
      unpack8<kF16>(a, xa);
      unpack8<kF16>(b, xb);
      const bool is_q = h < p.q_heads;
      const uint16_t* const w = is_q ? p.q_weight : p.k_weight;
      if (w) {
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) sum += xa[i] * xa[i] + xb[i] * xb[i];
        const unsigned mask = (kLanes == 32 ? 0xffffffffu : ((1u << kLanes) - 1u) << ((threadIdx.x & 31) / kLanes * kLanes));
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(mask, sum, o);
        const float r = rsqrtf(sum * (1.0f / kD) + p.eps);
        float wa[8], wb[8];
        unpack8<kF16>(*reinterpret_cast<const uint4*>(w + e0), wa);
        unpack8<kF16>(*reinterpret_cast<const uint4*>(w + e1), wb);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          xa[i] *= r * wa[i];
          xb[i] *= r * wb[i];
        }
      }
      if (rotates) {
        if (p.adjacent) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float a0 = xa[2 * i], a1 = xa[2 * i + 1], b0 = xb[2 * i], b1 = xb[2 * i + 1];
            xa[2 * i] = a0 * cs[i] - a1 * sn[i];
            xa[2 * i + 1] = a1 * cs[i] + a0 * sn[i];
            xb[2 * i] = b0 * cs[4 + i] - b1 * sn[4 + i];
            xb[2 * i + 1] = b1 * cs[4 + i] + b0 * sn[4 + i];
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float a0 = xa[i], b0 = xb[i];
            xa[i] = a0 * cs[i] - b0 * sn[i];
            xb[i] = b0 * cs[i] + a0 * sn[i];
          }
        }
      }
      const uint4 ya = pack8<kF16>(xa), yb = pack8<kF16>(xb);
      if (is_q) {
        uint16_t* const dst = p.q + t * p.q_ts + h * p.q_hs;
        *reinterpret_cast<uint4*>(dst + e0) = ya;
        *reinterpret_cast<uint4*>(dst + e1) = yb;
      } else {
        const int hk = h - p.q_heads;
        if (p.k) {
          uint16_t* const dst = p.k + t * p.k_ts + hk * p.k_hs;
          *reinterpret_cast<uint4*>(dst + e0) = ya;
          *reinterpret_cast<uint4*>(dst + e1) = yb;
        }
        if (cached) {
          uint16_t* const dst = p.k_cache + cache_at + hk * p.cache_hs;
          *reinterpret_cast<uint4*>(dst + e0) = ya;
          *reinterpret_cast<uint4*>(dst + e1) = yb;
        }
      }
    }
  }
}

template <bool kF16>
void launch(const NormRopeParams& p, int head_dim, cudaStream_t stream) {
  const dim3 grid((unsigned)p.tokens);
  if (head_dim == 64)
    agmm_norm_rope<64, kF16><<<grid, kThreads, 0, stream>>>(p);
  else if (head_dim == 128)
    agmm_norm_rope<128, kF16><<<grid, kThreads, 0, stream>>>(p);
  else
    agmm_norm_rope<256, kF16><<<grid, kThreads, 0, stream>>>(p);
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeParams& p, int head_dim, bool f16, cudaStream_t stream) {
  if (f16)
    launch<true>(p, head_dim, stream);
  else
    launch<false>(p, head_dim, stream);
  return cudaGetLastError();
}

}  // namespace agmm
