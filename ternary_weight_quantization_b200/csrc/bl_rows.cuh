// Device and host helpers of the kernels that walk the rows of an activation:
// sums over a row's threads, asynchronous copies of a thread's own columns,
// parameters of either type.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "bl_act8.cuh"
#include "bl_device.cuh"

namespace bl {

// 8 consecutive parameters from column c, or the one at c.
__device__ __forceinline__ void load_params8(const void* p, int f32, int c, f32x2 (&v)[4]) {
  if (f32) {
    Raw8<float> r;
    r.load(static_cast<const float*>(p) + c);
    r.get(v);
  } else {
    Raw8<__nv_bfloat16> r;
    r.load(static_cast<const __nv_bfloat16*>(p) + c);
    r.get(v);
  }
}
__device__ __forceinline__ float load_param(const void* p, int f32, int c) {
  return f32 ? static_cast<const float*>(p)[c] : __bfloat162float(static_cast<const __nv_bfloat16*>(p)[c]);
}

__device__ __forceinline__ void group_barrier(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) v += __shfl_xor_sync(0xffffffffu, v, s);
  return v;
}

// Sums of kN values over the tpr threads of a row's group; every thread gets
// them, added in the same order. `buf`: kN floats per warp of the group. The
// caller alternates between two buffers, so that one barrier per call is enough.
template <int kN>
__device__ __forceinline__ void group_sum(float (&v)[kN], float* buf, int t, int tpr, int barrier) {
#pragma unroll
  for (int i = 0; i < kN; ++i) v[i] = warp_sum(v[i]);
  if (tpr == 32) return;
  if ((t & 31) == 0) {
#pragma unroll
    for (int i = 0; i < kN; ++i) buf[(t >> 5) * kN + i] = v[i];
  }
  group_barrier(barrier, tpr);
#pragma unroll
  for (int i = 0; i < kN; ++i) v[i] = 0.0f;
#pragma unroll 4
  for (int w = 0; w < (tpr >> 5); ++w) {
#pragma unroll
    for (int i = 0; i < kN; ++i) v[i] += buf[w * kN + i];
  }
}

// 1 / sqrt(v): the hardware's approximation and one Newton step
// r + r (1 - v r^2) / 2, within an ulp. 0 and infinity have no step to take.
__device__ __forceinline__ float rsqrt_of(float v) {
  const float r = rsqrtf(v);
  const float e = fmaf(-v * r, r, 1.0f);
  return v > 0.0f && v < __uint_as_float(0x7F800000u) ? fmaf(0.5f * r, e, r) : r;
}

// Asynchronous copies into the thread's own places of shared memory: what a
// thread copies only that thread reads, so no barrier is needed.
__device__ __forceinline__ void copy_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// Through L1: for neighbouring 16-byte halves of a sector taken by two copies.
__device__ __forceinline__ void copy_async16_l1(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_async8(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kPending>
__device__ __forceinline__ void copy_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kPending) : "memory");
}

// 8 values of a thread in shared memory: 16-byte pieces `stride` bytes apart.
__device__ __forceinline__ void issue8(uint32_t dst, uint32_t stride, const __nv_bfloat16* src) {
  copy_async16(dst, src);
}
__device__ __forceinline__ void issue8(uint32_t dst, uint32_t stride, const float* src) {
  copy_async16_l1(dst, src);
  copy_async16_l1(dst + stride, src + 4);
}
__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
// A thread's raw 8 values back from shared memory.
__device__ __forceinline__ void read_raw(uint32_t a, uint32_t stride, Raw8<__nv_bfloat16>& r) { r.a = lds16(a); }
__device__ __forceinline__ void read_raw(uint32_t a, uint32_t stride, Raw8<float>& r) {
  const uint4 x = lds16(a), y = lds16(a + stride);
  r.a = make_float4(__uint_as_float(x.x), __uint_as_float(x.y), __uint_as_float(x.z), __uint_as_float(x.w));
  r.b = make_float4(__uint_as_float(y.x), __uint_as_float(y.y), __uint_as_float(y.z), __uint_as_float(y.w));
}

// ---------------------------------------------------------------- host side
inline int round32(int n) { return (n + 31) / 32 * 32; }

// Lets `kernel` use `smem` bytes of dynamic shared memory (once per device;
// `done`: the caller's table, one entry per device).
template <typename K>
cudaError_t allow_smem(K kernel, size_t smem, bool (&done)[64]) {
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev >= 0 && dev < 64 && done[dev]) return cudaSuccess;
  const cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e == cudaSuccess && dev >= 0 && dev < 64) done[dev] = true;
  return e;
}

}  // namespace bl
