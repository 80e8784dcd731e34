// attn_ptx.cuh -- the inline PTX that the attention kernels use beyond
// ptx_sm103.cuh, and their bounded waits.
#pragma once

#include "ptx_sm103.cuh"

namespace agmm {
namespace ptx {

// 4-D tiled load of one box; c0 is the innermost (contiguous) coordinate.
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const void* map, uint32_t bar, int c0, int c1, int c2, int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void mbar_arrive_n(uint32_t bar, uint32_t n) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(n) : "memory");
}

// D[tmem] (+)= A[tmem] * B[smem desc], A holding two 16-bit values per column.
__device__ __forceinline__ void mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void tmem_st_32x32b_x32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]),
      "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
      "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(taddr)
      : "memory");
}

__device__ __forceinline__ void tmem_st_32x32b_x16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(taddr)
      : "memory");
}

__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 2^x, the hardware's approximation (relative error about 2^-22); 2^-inf = 0.
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Registers of the warps of a warpgroup from here on (all its warps run it).
template <int kRegs>
__device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}

// Two float32 values in a 64-bit register, and arithmetic on both at once.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 unpair(uint64_t x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
  return r;
}
__device__ __forceinline__ uint64_t fma_pair(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// Two values rounded to 16 bits, the first in the low half.
template <bool kF16>
__device__ __forceinline__ uint32_t round_pair(float lo, float hi) {
  uint32_t w;
  if constexpr (kF16)
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
  return w;
}
// acc + each 16-bit half of w, in float32.
template <bool kF16>
__device__ __forceinline__ void add_halves(float& acc0, float& acc1, uint32_t w) {
  if constexpr (kF16)
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tadd.f32.f16 %0, l, %0;\n\tadd.f32.f16 %1, h, %1;\n\t}"
                 : "+f"(acc0), "+f"(acc1)
                 : "r"(w));
  else
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tadd.f32.bf16 %0, l, %0;\n\tadd.f32.bf16 %1, h, %1;\n\t}"
                 : "+f"(acc0), "+f"(acc1)
                 : "r"(w));
}

}  // namespace ptx

// Bounded waits.  A wait that runs out raises the CTA's abort flag and records
// AGMM_ERR_TIMEOUT (5) in the status words; every other wait of the CTA then
// ends too, and all roles leave their loops.
//
// Work whose length grows with the problem while other warps wait for it (rows that
// are computed again) leaves the time of its last step in the pulse: a wait runs out
// when it has lasted for its limit and no step came in as long a time.  That work ends
// by itself, and when the flag is raised.
struct Waiter {
  volatile int* abort;  // [0] the flag, [2] the pulse: cycles / 1024, odd; 0: no step yet
  uint64_t limit;
  int* status;
  int role;

  // Whether a wait that has lasted for its limit is given up; raises the flag.  A call of
  // its own: the softmax warps' key loop has to stay short (inlined, 256 became 279 us and 371
  // became 381 us for a piece of a prompt and a long one).
  __device__ __noinline__ bool expired(int where) const {
    const int last = abort[2];
    // the pulse may be one ahead of the clock
    const uint32_t since = (uint32_t)(ptx::clock_cycles() >> 10) + 1u - (uint32_t)last;
    if (__any_sync(0xffffffffu, last != 0 && since <= (uint32_t)(limit >> 10) + 2u)) return false;
    *abort = 1;
    if ((threadIdx.x & 31) == 0 && atomicCAS(status, 0, 5) == 0) {
      status[1] = role;
      status[2] = where;
      status[3] = (int)blockIdx.x;
    }
    __syncwarp();
    return true;
  }

  // A converged warp waits; every lane gets the same answer.
  __device__ __forceinline__ bool retry(uint32_t bar, uint32_t parity, int where) const {
    const uint64_t t0 = ptx::clock_cycles();
    for (;;) {
      if (__all_sync(0xffffffffu, ptx::mbar_try_wait_sleep(bar, parity, 20000))) return true;
      if (__any_sync(0xffffffffu, *abort != 0)) return false;
      if (__any_sync(0xffffffffu, ptx::clock_cycles() - t0 > limit) && expired(where)) return false;
    }
  }
  __device__ __forceinline__ bool operator()(uint32_t bar, uint32_t parity, int where) const {
    if (__all_sync(0xffffffffu, ptx::mbar_try_wait(bar, parity))) return true;
    return retry(bar, parity, where);
  }
  // The same with the retries as a call: for the warps with many waits, whose
  // code would crowd the instruction cache.
  __device__ __noinline__ bool retry_call(uint32_t bar, uint32_t parity, int where) const { return retry(bar, parity, where); }
  __device__ __forceinline__ bool compact(uint32_t bar, uint32_t parity, int where) const {
    if (__all_sync(0xffffffffu, ptx::mbar_try_wait(bar, parity))) return true;
    return retry_call(bar, parity, where);
  }
  // A converged warp has done a step of such work.
  __device__ __forceinline__ void beat() const {
    abort[2] = (int)(ptx::clock_cycles() >> 10) | 1;
  }
  // Waits for work in flight, whatever the abort flag says.
  __device__ __forceinline__ void drain(uint32_t bar, uint32_t parity) const {
    const uint64_t t0 = ptx::clock_cycles();
    while (!__all_sync(0xffffffffu, ptx::mbar_try_wait_sleep(bar, parity, 20000)))
      if (__any_sync(0xffffffffu, ptx::clock_cycles() - t0 > limit)) return;
  }
};

}  // namespace agmm
