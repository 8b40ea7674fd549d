// Device helpers shared by the kvc kernels: shared-memory addresses,
// programmatic dependent launch, exp2, a block scan and the status word.
#pragma once

#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <stdint.h>

namespace kvc {

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

// Programmatic dependent launch.  grid_dep_wait: block until the grid this
// one was launched behind has completed and its writes are visible (returns
// at once when there is none).  grid_dep_launch: let the next grid on the
// stream be scheduled as SMs free up; it still waits for this grid's
// completion before it reads anything this grid writes.
__device__ __forceinline__ void grid_dep_wait() { asm volatile("griddepcontrol.wait;\n" ::: "memory"); }
__device__ __forceinline__ void grid_dep_launch() { asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory"); }

// 2^x with the hardware approximation (relative error about 2^-22); 2^-inf = 0.
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}

// 1 / x with the hardware approximation (relative error about 2^-23).
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}

// log2 of a power of two: its exponent in the lowest bits of 2^23.
__device__ __forceinline__ float log2_of(float s) {
  return __uint_as_float(__float_as_uint(s) >> 23 | 0x4b000000u) - (8388608.f + 127.f);
}

// tanh(x), relative error below 1e-6.  Up to kTanhNear an odd polynomial (fitted to
// tanh(x) / x over x^2: 1.2e-7 off by itself, 2.2e-7 with fp32's roundings), where
// 1 - 2 / (1 + e^2x) would cancel; that form beyond.
constexpr float kTanhNear = 0.625f;
__device__ __forceinline__ float tanh_near(float x) {
  const float w = x * x;
  float p = fmaf(w, 0.015050944872200489f, -0.051821865141391754f);
  p = fmaf(w, p, 0.1330452561378479f);
  p = fmaf(w, p, -0.3333195447921753f);
  p = fmaf(w, p, 0.9999998807907104f);
  return x * p;
}
__device__ __forceinline__ float tanh_far(float x) {
  return fmaf(-2.f, rcp(1.f + ex2(x * 2.8853900817779268f)), 1.f);
}
__device__ __forceinline__ float tanh_of(float x) { return fabsf(x) <= kTanhNear ? tanh_near(x) : tanh_far(x); }

// Inclusive sum over a block of blockDim.x (multiple of 32, <= 1024) threads.
// `scratch` holds 32 ints.  Returns the inclusive prefix; *total gets the sum.
__device__ __forceinline__ int block_inclusive_scan(int v, int* scratch, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int nw = blockDim.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    int t = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += t;
  }
  if (lane == 31) scratch[warp] = v;
  __syncthreads();
  if (warp == 0) {
    int w = lane < nw ? scratch[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      int t = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += t;
    }
    scratch[lane] = w;
  }
  __syncthreads();
  int res = v + (warp > 0 ? scratch[warp - 1] : 0);
  *total = scratch[nw - 1];
  __syncthreads();
  return res;
}

__device__ __forceinline__ void record_status(int* status, int code) {
  if (status) atomicCAS(status, 0, code);
}

}  // namespace kvc
