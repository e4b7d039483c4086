// The 8-bit form of an activation, shared by the kernels that write or read it:
// groups of 128 values of a row,
//
//   a = max(absmax, 1e-30);        inv = fp32(fp32(1 / a) * 127)
//   code = rint(fp32(x * inv));    scale = fp32(a * fp32(1 / 127))
//   saved value = fp32(code * scale)
//
// (one reciprocal and two products per group instead of two divisions; three
// half steps of fp32 cannot lift |x * inv| to 127.5, so codes end at 127).
//
// Two thread layouts. Vector (K % 8 == 0): 16 lanes hold 8 consecutive values
// each, one 16-byte load (two for fp32) and one 8-byte code access per lane,
// two groups to a warp. Scalar (any K: rows start at any element): 32 lanes
// hold values l, l + 32, l + 64, l + 96 of the group, so every access of the
// warp stays contiguous.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

namespace bl {

constexpr int kAct8Group = 128;
constexpr float kAct8Floor = 1e-30f;

template <bool kVec>
struct Act8Lane {
  static constexpr int N = kVec ? 8 : 4;    // values per lane
  static constexpr int W = kVec ? 16 : 32;  // lanes per group
};

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// {hi, lo} -> bf16x2, each rounded once to nearest even.
__device__ __forceinline__ uint32_t pack_bf16x2(float hi, float lo) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// 8 consecutive values at a 16-byte aligned address.
template <typename T>
struct Raw8;
template <>
struct Raw8<__nv_bfloat16> {
  uint4 a;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { a = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void clear() { a = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = bf16_lo(a.x), v[1] = bf16_hi(a.x), v[2] = bf16_lo(a.y), v[3] = bf16_hi(a.y);
    v[4] = bf16_lo(a.z), v[5] = bf16_hi(a.z), v[6] = bf16_lo(a.w), v[7] = bf16_hi(a.w);
  }
};
template <>
struct Raw8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ void clear() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
};

__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(v[1], v[0]), pack_bf16x2(v[3], v[2]),
                                            pack_bf16x2(v[5], v[4]), pack_bf16x2(v[7], v[6]));
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }
__device__ __forceinline__ void store1(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// Absmax of the group over its W lanes (every lane gets it), as bits: for
// non-negative fp32 the order of the bits is the order of the values, with
// infinity and NaN above all finite ones.
template <bool kVec>
__device__ __forceinline__ uint32_t act8_absmax_bits(const float (&v)[Act8Lane<kVec>::N]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < Act8Lane<kVec>::N; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
#pragma unroll
  for (int s = Act8Lane<kVec>::W / 2; s > 0; s >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, s));
  return m;
}

struct Act8Scale {
  float inv, scale;
};

__device__ __forceinline__ Act8Scale act8_scale(uint32_t absmax_bits) {
  if (absmax_bits >= 0x7F800000u) return {0.0f, __uint_as_float(0x7FC00000u)};
  const float a = fmaxf(__uint_as_float(absmax_bits), kAct8Floor);
  return {__fmul_rn(__frcp_rn(a), 127.0f), __fmul_rn(a, 1.0f / 127.0f)};
}

// The code in the low byte: |x * inv| rounds to at most 127, so adding
// 1.5 * 2^23 rounds the product to an integer (half to even) in the low bits
// of the sum. inv = 0 marks a group without finite codes: 0.
__device__ __forceinline__ uint32_t act8_code(float x, float inv) {
  const uint32_t t = __float_as_uint(__fadd_rn(__fmul_rn(x, inv), 12582912.0f));
  return inv == 0.0f ? 0u : t;
}

__device__ __forceinline__ uint2 act8_codes8(const float (&v)[8], float inv) {
  uint32_t t[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) t[i] = act8_code(v[i], inv);
  return make_uint2(__byte_perm(__byte_perm(t[0], t[1], 0x0040), __byte_perm(t[2], t[3], 0x0040), 0x5410),
                    __byte_perm(__byte_perm(t[4], t[5], 0x0040), __byte_perm(t[6], t[7], 0x0040), 0x5410));
}

// Saved values of 8 codes. fp32(code) through the 2^23 shifter: the bits
// 0x4B0000uu are 2^23 + u with u = code + 128.
__device__ __forceinline__ void act8_values8(const uint2& c, float scale, float (&v)[8]) {
  const uint32_t w[2] = {c.x ^ 0x80808080u, c.y ^ 0x80808080u};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    v[i] = __fmul_rn(__fsub_rn(__uint_as_float(__byte_perm(w[i >> 2], 0x4B000000u, 0x7440u | (i & 3))), 8388736.0f),
                     scale);
}

__device__ __forceinline__ float act8_value(int8_t code, float scale) {
  return __fmul_rn(static_cast<float>(code), scale);
}

}  // namespace bl
