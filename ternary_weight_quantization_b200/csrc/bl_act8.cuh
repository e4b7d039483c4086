// The 8-bit form of an activation, shared by the kernels that write or read it:
// groups of 128 values of a row,
//
//   a = max(absmax, 1e-30);        inv = fp32(fp32(1 / a) * 127)
//   code = rint(fp32(x * inv));    scale = fp32(a * fp32(1 / 127))
//   saved value = fp32(code * scale)
//
// (one reciprocal and two products per group instead of two divisions: A1 of
// 4096 x 6912 bf16 in 17.0 us for 17.7, of 1021 x 2565 fp32 in 5.0 for 5.3. The
// factors are within an fp32 step or two of 127 / a and a / 127, so a code is
// another one than rint(127 x / a) only next to a tie, and as near to x. Three
// half steps of fp32 cannot lift |x * inv| to 127.5, so codes end at 127.)
//
// The arithmetic on 8 consecutive values runs on pairs (packed fp32x2
// instructions, each half rounded like the scalar one): these kernels are
// bound by the instructions they issue as much as by HBM.
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

// ---- pairs of fp32 values
using f32x2 = uint64_t;

__device__ __forceinline__ f32x2 pair2(float lo, float hi) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ f32x2 both2(float v) { return pair2(v, v); }
__device__ __forceinline__ void split2(f32x2 v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ float sum2(f32x2 v) {
  float lo, hi;
  split2(v, lo, hi);
  return lo + hi;
}

// Maxima that keep a NaN.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ uint32_t max_nan_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// 8 consecutive values at a 16-byte aligned address, as loaded.
template <typename T>
struct Raw8;
template <>
struct Raw8<__nv_bfloat16> {
  uint4 a;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { a = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void clear() { a = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void get(f32x2 (&v)[4]) const {
    v[0] = pair2(bf16_lo(a.x), bf16_hi(a.x)), v[1] = pair2(bf16_lo(a.y), bf16_hi(a.y));
    v[2] = pair2(bf16_lo(a.z), bf16_hi(a.z)), v[3] = pair2(bf16_lo(a.w), bf16_hi(a.w));
  }
  // The largest |x|; a NaN if there is one.
  __device__ __forceinline__ float absmax() const {
    const uint32_t m = max_nan_bf16x2(max_nan_bf16x2(a.x & 0x7FFF7FFFu, a.y & 0x7FFF7FFFu),
                                      max_nan_bf16x2(a.z & 0x7FFF7FFFu, a.w & 0x7FFF7FFFu));
    return max_nan(bf16_lo(m), bf16_hi(m));
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
  __device__ __forceinline__ void get(f32x2 (&v)[4]) const {
    v[0] = pair2(a.x, a.y), v[1] = pair2(a.z, a.w), v[2] = pair2(b.x, b.y), v[3] = pair2(b.z, b.w);
  }
  __device__ __forceinline__ float absmax() const {
    return max_nan(max_nan(max_nan(fabsf(a.x), fabsf(a.y)), max_nan(fabsf(a.z), fabsf(a.w))),
                   max_nan(max_nan(fabsf(b.x), fabsf(b.y)), max_nan(fabsf(b.z), fabsf(b.w))));
  }
};

__device__ __forceinline__ uint32_t pack_bf16x2(f32x2 v) {
  float lo, hi;
  split2(v, lo, hi);
  return pack_bf16x2(hi, lo);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const f32x2 (&v)[4]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(v[0]), pack_bf16x2(v[1]), pack_bf16x2(v[2]), pack_bf16x2(v[3]));
}
__device__ __forceinline__ void store8(float* p, const f32x2 (&v)[4]) {
  float f[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) split2(v[i], f[2 * i], f[2 * i + 1]);
  reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
}

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }
__device__ __forceinline__ void store1(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// The group's absmax from its kLanes lanes' own (every lane gets it).
template <int kLanes>
__device__ __forceinline__ float act8_absmax(float m) {
#pragma unroll
  for (int s = kLanes / 2; s > 0; s >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, s));
  return m;
}

struct Act8Scale {
  float inv, scale;
};

__device__ __forceinline__ Act8Scale act8_scale(float absmax) {
  // infinity and NaN have the bits above all finite values'
  if (__float_as_uint(absmax) >= 0x7F800000u) return {0.0f, __uint_as_float(0x7FC00000u)};
  const float a = fmaxf(absmax, kAct8Floor);
  return {__fmul_rn(__frcp_rn(a), 127.0f), __fmul_rn(a, 1.0f / 127.0f)};
}

// The code in the low byte: |x * inv| rounds to at most 127, so adding
// 1.5 * 2^23 rounds the product to an integer (half to even) in the low bits
// of the sum. (In a group that holds an infinity or a NaN inv is 0; its codes
// do not matter, as its scale is NaN.)
__device__ __forceinline__ uint32_t act8_code(float x, float inv) {
  return __float_as_uint(__fadd_rn(__fmul_rn(x, inv), 12582912.0f));
}

__device__ __forceinline__ uint2 act8_codes8(const f32x2 (&v)[4], float inv) {
  const f32x2 inv2 = both2(inv);
  uint32_t t[4];  // two codes each
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // the product is rounded before the addition: a packed addition after the
    // packed product was measured to come out as one fused operation (codes
    // at ties differ), the scalar ones do not
    float lo, hi;
    split2(mul2(v[i], inv2), lo, hi);
    t[i] = __byte_perm(__float_as_uint(__fadd_rn(lo, 12582912.0f)), __float_as_uint(__fadd_rn(hi, 12582912.0f)), 0x0040);
  }
  return make_uint2(__byte_perm(t[0], t[1], 0x5410), __byte_perm(t[2], t[3], 0x5410));
}

// Saved values of 8 codes. fp32(code) through the 2^23 shifter: the bits
// 0x4B0000uu are 2^23 + u with u = code + 128. The product is an fma with 0, so
// that it is rounded: a packed product was measured to be fused with a packed
// addition that follows (the norm's x - mean), half an fp32 step of x away.
__device__ __forceinline__ void act8_values8(const uint2& c, float scale, f32x2 (&v)[4]) {
  const uint32_t w[2] = {c.x ^ 0x80808080u, c.y ^ 0x80808080u};
  const f32x2 shift2 = both2(-8388736.0f), scale2 = both2(scale);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t b = 2 * (i & 1);
    const uint32_t lo = __byte_perm(w[i >> 1], 0x4B000000u, 0x7440u | b);
    const uint32_t hi = __byte_perm(w[i >> 1], 0x4B000000u, 0x7440u | (b + 1));
    v[i] = fma2(add2((static_cast<uint64_t>(hi) << 32) | lo, shift2), scale2, 0);
  }
}

__device__ __forceinline__ float act8_value(int8_t code, float scale) {
  return __fmul_rn(static_cast<float>(code), scale);
}

}  // namespace bl
