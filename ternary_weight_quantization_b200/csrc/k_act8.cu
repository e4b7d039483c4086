// Activations kept in 8 bits until the backward, and the SwiGLU gate that
// saves its inputs that way.
//
//   A1 encode    x -> codes, one scale per 128 values of a row
//   A2 decode    codes, scales -> x
//   U1 forward   y = silu(gate) * up, and the 8-bit forms of gate and up in the
//                same pass
//   U2 backward  dgate = dy u s (1 + g (1 - s)), dup = dy g s with g and u the
//                saved values, s = 1 / (1 + exp(-g))
//
// All four are streams bound by HBM: per value (bf16) A1 moves 3 bytes, A2 3,
// U1 8 (6 without the 8-bit forms) and U2 8. A unit of work is one group of
// 128 values (half a warp of 8-value lanes where K % 8 == 0, else a warp, see
// bl_act8.cuh). A block takes consecutive units, kU per thread, and issues all
// of a thread's loads before it computes.
//
// Measured on B200 (back to back in a graph, over inputs that rotate past L2), 4096 x
// 6912 bf16: A1 + A2 28.7 us (0.91 of the copy rate), U1 with codes + U2 74.9 (0.94).
// 1021 x 2565 fp32 (scalar, 4-byte accesses): A1 + A2 11.3 (0.35).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "bl_act8.cuh"
#include "bl_device.cuh"
#include "bl_internal.h"

namespace bl {
namespace {

constexpr int kThreads = 256;

// A unit: its first element and its length.
struct Unit {
  int64_t off;
  int len;  // values of the group (0: no unit)
};

// The units of a block: kPer consecutive ones. With whole groups only
// (K % 128 == 0) unit u starts at element 128 u; else each row before it
// takes `pad` = 128 G - K off. The row of a unit is found once per block by a
// division and from there by a product: for n < 2^22, floor((n + 1/2) (1 / G))
// in fp32 is floor(n / G) (the product is off by less than 1 / (2 G)).
struct Units {
  int64_t first, count, row0;
  int g0, groups, pad, last;
  float inv;
  __device__ __forceinline__ Units(int64_t f, int64_t n, int g, int K) : first(f), count(n), groups(g) {
    pad = g * kAct8Group - K;
    last = kAct8Group - pad;
    if (pad) {
      row0 = n <= 0xFFFFFFFFll ? static_cast<int64_t>(static_cast<uint32_t>(f) / static_cast<uint32_t>(g)) : f / g;
      g0 = static_cast<int>(f - row0 * g);
      inv = 1.0f / static_cast<float>(g);
    }
  }
  __device__ __forceinline__ Unit at(int i) const {
    const int64_t u = first + i;
    if (u >= count) return {0, 0};
    if (!pad) return {u * kAct8Group, kAct8Group};
    // more groups than 2^21 to a row: the block's units cross one row end at most
    const int n = g0 + i;
    const int q = groups > (1 << 21) ? (n >= groups) : static_cast<int>((static_cast<float>(n) + 0.5f) * inv);
    return {u * kAct8Group - (row0 + q) * pad, n - q * groups == groups - 1 ? last : kAct8Group};
  }
};

// A lane's values of a unit, as loaded; n() of them come in `Val`s (pairs in
// the vector layout, single values in the scalar one).
template <typename T, bool kVec>
struct Loaded;
template <typename T>
struct Loaded<T, true> {
  Raw8<T> r;
  __device__ __forceinline__ void load(const T* p, const Unit& u, int l) {
    if (l * 8 < u.len) r.load(p + u.off + l * 8);
    else r.clear();
  }
  __device__ __forceinline__ void get(f32x2 (&v)[4]) const { r.get(v); }
  __device__ __forceinline__ float absmax() const { return act8_absmax<16>(r.absmax()); }
};
template <typename T>
struct Loaded<T, false> {
  float r[4];
  __device__ __forceinline__ void load(const T* p, const Unit& u, int l) {
#pragma unroll
    for (int j = 0; j < 4; ++j) r[j] = l + 32 * j < u.len ? to_f32(p[u.off + l + 32 * j]) : 0.0f;
  }
  __device__ __forceinline__ void get(float (&v)[4]) const {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = r[j];
  }
  __device__ __forceinline__ float absmax() const {
    return act8_absmax<32>(max_nan(max_nan(fabsf(r[0]), fabsf(r[1])), max_nan(fabsf(r[2]), fabsf(r[3]))));
  }
};

template <bool kVec>
struct LoadedCodes;
template <>
struct LoadedCodes<true> {
  uint2 c;
  __device__ __forceinline__ void load(const int8_t* p, const Unit& u, int l) {
    c = l * 8 < u.len ? *reinterpret_cast<const uint2*>(p + u.off + l * 8) : make_uint2(0u, 0u);
  }
  __device__ __forceinline__ void get(float scale, f32x2 (&v)[4]) const { act8_values8(c, scale, v); }
};
template <>
struct LoadedCodes<false> {
  int8_t c[4];
  __device__ __forceinline__ void load(const int8_t* p, const Unit& u, int l) {
#pragma unroll
    for (int j = 0; j < 4; ++j) c[j] = l + 32 * j < u.len ? p[u.off + l + 32 * j] : int8_t(0);
  }
  __device__ __forceinline__ void get(float scale, float (&v)[4]) const {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = act8_value(c[j], scale);
  }
};

template <typename T>
__device__ __forceinline__ void store_values(T* p, const Unit& u, int l, const f32x2 (&v)[4]) {
  if (l * 8 < u.len) store8(p + u.off + l * 8, v);
}
template <typename T>
__device__ __forceinline__ void store_values(T* p, const Unit& u, int l, const float (&v)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (l + 32 * j < u.len) store1(p + u.off + l + 32 * j, v[j]);
}

// Codes and scale of one unit.
__device__ __forceinline__ void store_codes(const f32x2 (&v)[4], const Act8Scale& s, const Unit& u, int64_t idx, int l,
                                            int8_t* codes, float* scales) {
  if (l * 8 < u.len) *reinterpret_cast<uint2*>(codes + u.off + l * 8) = act8_codes8(v, s.inv);
  if (l == 0 && u.len > 0) scales[idx] = s.scale;
}
__device__ __forceinline__ void store_codes(const float (&v)[4], const Act8Scale& s, const Unit& u, int64_t idx, int l,
                                            int8_t* codes, float* scales) {
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (l + 32 * j < u.len) codes[u.off + l + 32 * j] = static_cast<int8_t>(act8_code(v[j], s.inv) & 0xFFu);
  if (l == 0 && u.len > 0) scales[idx] = s.scale;
}

// 1 / (1 + exp(-g)); for bf16 results by way of 2^24 times it (kSigmoidUnit puts
// the factor back: powers of two, so no bit of a normal value changes). For those
// the hardware's approximations (a few fp32 ulp) are far below the rounding to
// 8 bits, but its reciprocal flushes what is below 2^-126 to zero: from g =
// -87.4 to -88.7, where 1 + exp(-g) is still finite, a large `up` or dy makes
// that visible. fp32 results take expf and the rounded division.
constexpr float kSigmoidUnit = 1.0f / 16777216.0f;
__device__ __forceinline__ float ex2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_fast(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
template <typename T>
__device__ __forceinline__ float sigmoid(float g) {
  if constexpr (sizeof(T) == 2)
    return rcp_fast(fmaf(ex2_fast(g * -1.4426950408889634f), kSigmoidUnit, kSigmoidUnit)) * kSigmoidUnit;
  else
    return __fdiv_rn(1.0f, 1.0f + expf(-g));
}
template <typename T>
__device__ __forceinline__ f32x2 sigmoid(f32x2 g) {
  float a, b;
  if constexpr (sizeof(T) == 2) {
    const f32x2 unit = both2(kSigmoidUnit);
    split2(mul2(g, both2(-1.4426950408889634f)), a, b);
    split2(fma2(pair2(ex2_fast(a), ex2_fast(b)), unit, unit), a, b);
    return mul2(pair2(rcp_fast(a), rcp_fast(b)), unit);
  } else {
    split2(g, a, b);
    return pair2(sigmoid<T>(a), sigmoid<T>(b));
  }
}

// y = silu(g) u; and dg = d u s (1 + g (1 - s)), du = d g s.
template <typename T>
__device__ __forceinline__ void gate_forward(float g, float u, float& y) {
  y = g * sigmoid<T>(g) * u;
}
template <typename T>
__device__ __forceinline__ void gate_forward(f32x2 g, f32x2 u, f32x2& y) {
  y = mul2(mul2(g, sigmoid<T>(g)), u);
}
template <typename T>
__device__ __forceinline__ void gate_backward(float d, float g, float u, float& dg, float& du) {
  const float s = sigmoid<T>(g), ds = d * s;
  dg = ds * u * fmaf(g, 1.0f - s, 1.0f);
  du = ds * g;
}
template <typename T>
__device__ __forceinline__ void gate_backward(f32x2 d, f32x2 g, f32x2 u, f32x2& dg, f32x2& du) {
  const f32x2 one = both2(1.0f);
  const f32x2 s = sigmoid<T>(g), ds = mul2(d, s);
  dg = mul2(mul2(ds, u), fma2(g, fma2(s, both2(-1.0f), one), one));
  du = mul2(ds, g);
}

struct Act8Args {
  const void* a;     // x, gate, dy
  const void* b;     // up
  void* o0;          // decoded x, y, dgate
  void* o1;          // dup
  int8_t* c0;        // codes of x / gate
  float* s0;
  int8_t* c1;        // codes of up
  float* s1;
  int64_t units;     // M * G
  int groups, K;
};

enum class What { Encode, Decode, Fwd, FwdSave, Bwd };

template <What what, typename T, bool kVec, int kU>
__global__ void __launch_bounds__(kThreads) act8_kernel(const Act8Args p) {
  pdl_wait_primary();
  pdl_launch_dependents();
  constexpr int W = Act8Lane<kVec>::W, kRow = kThreads / W;  // units that the block takes at once
  constexpr int N = 4;  // pairs or single values per lane
  using Val = std::conditional_t<kVec, f32x2, float>;
  const int l = threadIdx.x % W, h = threadIdx.x / W;
  const T* a = static_cast<const T*>(p.a);
  const T* b = static_cast<const T*>(p.b);
  for (int64_t first = static_cast<int64_t>(blockIdx.x) * (kRow * kU); first < p.units;
       first += static_cast<int64_t>(gridDim.x) * (kRow * kU)) {
    const Units all(first, p.units, p.groups, p.K);
    const int64_t u0 = first + h;
    constexpr int T0 = kRow;
    Unit u[kU];
#pragma unroll
    for (int i = 0; i < kU; ++i) u[i] = all.at(h + i * kRow);
    if constexpr (what == What::Encode) {
      Loaded<T, kVec> x[kU];
#pragma unroll
      for (int i = 0; i < kU; ++i) x[i].load(a, u[i], l);
#pragma unroll
      for (int i = 0; i < kU; ++i) {
        Val v[N];
        x[i].get(v);
        store_codes(v, act8_scale(x[i].absmax()), u[i], u0 + i * T0, l, p.c0, p.s0);
      }
    } else if constexpr (what == What::Decode) {
      LoadedCodes<kVec> c[kU];
      float s[kU];
#pragma unroll
      for (int i = 0; i < kU; ++i) {
        c[i].load(p.c0, u[i], l);
        s[i] = u[i].len ? __ldg(p.s0 + u0 + i * T0) : 0.0f;
      }
#pragma unroll
      for (int i = 0; i < kU; ++i) {
        Val v[N];
        c[i].get(s[i], v);
        store_values(static_cast<T*>(p.o0), u[i], l, v);
      }
    } else if constexpr (what == What::Fwd || what == What::FwdSave) {
      Loaded<T, kVec> g[kU], q[kU];
#pragma unroll
      for (int i = 0; i < kU; ++i) {
        g[i].load(a, u[i], l);
        q[i].load(b, u[i], l);
      }
#pragma unroll
      for (int i = 0; i < kU; ++i) {
        Val gv[N], uv[N], y[N];
        g[i].get(gv);
        q[i].get(uv);
#pragma unroll
        for (int j = 0; j < N; ++j) gate_forward<T>(gv[j], uv[j], y[j]);
        store_values(static_cast<T*>(p.o0), u[i], l, y);
        if constexpr (what == What::FwdSave) {
          store_codes(gv, act8_scale(g[i].absmax()), u[i], u0 + i * T0, l, p.c0, p.s0);
          store_codes(uv, act8_scale(q[i].absmax()), u[i], u0 + i * T0, l, p.c1, p.s1);
        }
      }
    } else {
      Loaded<T, kVec> d[kU];
      LoadedCodes<kVec> cg[kU], cu[kU];
      float sg[kU], su[kU];
#pragma unroll
      for (int i = 0; i < kU; ++i) {
        d[i].load(a, u[i], l);
        cg[i].load(p.c0, u[i], l);
        cu[i].load(p.c1, u[i], l);
        sg[i] = u[i].len ? __ldg(p.s0 + u0 + i * T0) : 0.0f;
        su[i] = u[i].len ? __ldg(p.s1 + u0 + i * T0) : 0.0f;
      }
#pragma unroll
      for (int i = 0; i < kU; ++i) {
        Val dv[N], gv[N], uv[N], dg[N], du[N];
        d[i].get(dv);
        cg[i].get(sg[i], gv);
        cu[i].get(su[i], uv);
#pragma unroll
        for (int j = 0; j < N; ++j) gate_backward<T>(dv[j], gv[j], uv[j], dg[j], du[j]);
        store_values(static_cast<T*>(p.o0), u[i], l, dg);
        store_values(static_cast<T*>(p.o1), u[i], l, du);
      }
    }
  }
}

template <What what, typename T, bool kVec, int kU>
cudaError_t launch_one(const Act8Args& p, cudaStream_t s) {
  const int64_t per = static_cast<int64_t>(kThreads / Act8Lane<kVec>::W) * kU;
  const int64_t want = (p.units + per - 1) / per;
  // less than a block per SM: one unit per thread on more SMs (600 x 1000 bf16 in
  // 1.7 and 1.6 us for 2.4 and 1.9, A1 and A2 with 4; at 1200 x 1024 4 per thread
  // take 2.2 and 1.9)
  if constexpr (kU > 1) {
    if (want <= kPlanSms) return launch_one<what, T, kVec, 1>(p, s);
  }
  constexpr int64_t kMaxGrid = 1 << 20;
  return launch_pdl(act8_kernel<what, T, kVec, kU>, dim3(static_cast<unsigned>(want < kMaxGrid ? want : kMaxGrid)),
                    dim3(kThreads), 0, s, p);
}

template <What what, int kU>
cudaError_t launch_act8(Act8Args p, bool f32, int64_t M, int64_t K, cudaStream_t s) {
  p.K = static_cast<int>(K);
  p.groups = static_cast<int>((K + kAct8Group - 1) / kAct8Group);
  p.units = M * p.groups;
  const bool vec = K % 8 == 0;
  if (f32)
    return vec ? launch_one<what, float, true, kU>(p, s) : launch_one<what, float, false, kU>(p, s);
  return vec ? launch_one<what, __nv_bfloat16, true, kU>(p, s) : launch_one<what, __nv_bfloat16, false, kU>(p, s);
}

}  // namespace

cudaError_t launch_act8_encode(const void* x, int f32, int64_t M, int64_t K, int8_t* codes, float* scales,
                               cudaStream_t s) {
  Act8Args p{};
  p.a = x;
  p.c0 = codes;
  p.s0 = scales;
  return launch_act8<What::Encode, 4>(p, f32 != 0, M, K, s);
}

cudaError_t launch_act8_decode(const int8_t* codes, const float* scales, int64_t M, int64_t K, void* x, int f32,
                               cudaStream_t s) {
  Act8Args p{};
  p.c0 = const_cast<int8_t*>(codes);
  p.s0 = const_cast<float*>(scales);
  p.o0 = x;
  return launch_act8<What::Decode, 4>(p, f32 != 0, M, K, s);
}

cudaError_t launch_swiglu_forward(const void* gate, const void* up, int f32, int64_t M, int64_t K, void* y,
                                  int8_t* gate_codes, float* gate_scales, int8_t* up_codes, float* up_scales,
                                  cudaStream_t s) {
  Act8Args p{};
  p.a = gate;
  p.b = up;
  p.o0 = y;
  p.c0 = gate_codes;
  p.s0 = gate_scales;
  p.c1 = up_codes;
  p.s1 = up_scales;
  return gate_codes ? launch_act8<What::FwdSave, 2>(p, f32 != 0, M, K, s)
                    : launch_act8<What::Fwd, 2>(p, f32 != 0, M, K, s);
}

cudaError_t launch_swiglu_backward(const void* dy, const int8_t* gate_codes, const float* gate_scales,
                                   const int8_t* up_codes, const float* up_scales, int f32, int64_t M, int64_t K,
                                   void* dgate, void* dup, cudaStream_t s) {
  Act8Args p{};
  p.a = dy;
  p.o0 = dgate;
  p.o1 = dup;
  p.c0 = const_cast<int8_t*>(gate_codes);
  p.s0 = const_cast<float*>(gate_scales);
  p.c1 = const_cast<int8_t*>(up_codes);
  p.s1 = const_cast<float*>(up_scales);
  return launch_act8<What::Bwd, 2>(p, f32 != 0, M, K, s);
}

}  // namespace bl
