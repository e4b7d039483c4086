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
// bl_act8.cuh). Each thread takes kU units spaced one grid apart, so that
// every load of a warp is contiguous and all of a thread's loads are in
// flight before it computes.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "bl_act8.cuh"
#include "bl_device.cuh"
#include "bl_internal.h"

namespace bl {
namespace {

constexpr int kThreads = 256;

// One lane's share of a unit: `off` is the element offset of the lane's first
// value, n how many of its values exist (vector: 0 or 8; scalar: values l,
// l + 32, ... below the group's length).
struct Unit {
  int64_t off;
  int len;  // values of the group
};

__device__ __forceinline__ Unit unit_at(int64_t u, int groups, int K, bool narrow) {
  const int64_t row = narrow ? static_cast<int64_t>(static_cast<uint32_t>(u) / static_cast<uint32_t>(groups)) : u / groups;
  const int g = static_cast<int>(u - row * groups);
  const int left = K - g * kAct8Group;
  return {row * K + static_cast<int64_t>(g) * kAct8Group, left < kAct8Group ? left : kAct8Group};
}

// A lane's values of a unit, as loaded.
template <typename T, bool kVec>
struct Loaded;
template <typename T>
struct Loaded<T, true> {
  Raw8<T> r;
  __device__ __forceinline__ void load(const T* p, const Unit& u, int l) {
    if (l * 8 < u.len) r.load(p + u.off + l * 8);
    else r.clear();
  }
  __device__ __forceinline__ void get(float (&v)[8]) const { r.get(v); }
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
};

template <bool kVec>
struct LoadedCodes;
template <>
struct LoadedCodes<true> {
  uint2 c;
  __device__ __forceinline__ void load(const int8_t* p, const Unit& u, int l) {
    c = l * 8 < u.len ? *reinterpret_cast<const uint2*>(p + u.off + l * 8) : make_uint2(0u, 0u);
  }
  __device__ __forceinline__ void get(float scale, float (&v)[8]) const { act8_values8(c, scale, v); }
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
__device__ __forceinline__ void store_values(T* p, const Unit& u, int l, const float (&v)[8]) {
  if (l * 8 < u.len) store8(p + u.off + l * 8, v);
}
template <typename T>
__device__ __forceinline__ void store_values(T* p, const Unit& u, int l, const float (&v)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (l + 32 * j < u.len) store1(p + u.off + l + 32 * j, v[j]);
}

// Codes and scale of one unit (every lane of the warp takes part).
__device__ __forceinline__ void encode_unit(const float (&v)[8], bool live, const Unit& u, int64_t idx, int l,
                                            int8_t* codes, float* scales) {
  const Act8Scale s = act8_scale(act8_absmax_bits<true>(v));
  if (!live) return;
  if (l * 8 < u.len) *reinterpret_cast<uint2*>(codes + u.off + l * 8) = act8_codes8(v, s.inv);
  if (l == 0) scales[idx] = s.scale;
}
__device__ __forceinline__ void encode_unit(const float (&v)[4], bool live, const Unit& u, int64_t idx, int l,
                                            int8_t* codes, float* scales) {
  const Act8Scale s = act8_scale(act8_absmax_bits<false>(v));
  if (!live) return;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (l + 32 * j < u.len) codes[u.off + l + 32 * j] = static_cast<int8_t>(act8_code(v[j], s.inv) & 0xFFu);
  if (l == 0) scales[idx] = s.scale;
}

// 1 / (1 + exp(-g)). For bf16 results the hardware's approximations (a few
// fp32 ulp) are far below the rounding to 8 bits; fp32 results take expf and
// the rounded division.
template <typename T>
__device__ __forceinline__ float sigmoid(float g) {
  if constexpr (sizeof(T) == 2) return __fdividef(1.0f, 1.0f + __expf(-g));
  else return __fdiv_rn(1.0f, 1.0f + expf(-g));
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
  constexpr int W = Act8Lane<kVec>::W, N = Act8Lane<kVec>::N;
  const int l = threadIdx.x % W;
  const int64_t T0 = static_cast<int64_t>(gridDim.x) * (kThreads / W);
  const bool narrow = p.units <= 0xFFFFFFFFll;
  const T* a = static_cast<const T*>(p.a);
  const T* b = static_cast<const T*>(p.b);
  // the loop runs on the whole warp's first unit, so that every lane of the
  // warp takes part in its shuffles
  const int64_t first = static_cast<int64_t>(blockIdx.x) * (kThreads / W) + threadIdx.x / W;
  for (int64_t base = first - threadIdx.x % 32 / W; base < p.units; base += kU * T0) {
    const int64_t u0 = base + threadIdx.x % 32 / W;
    Unit u[kU];
    bool live[kU];
#pragma unroll
    for (int i = 0; i < kU; ++i) {
      const int64_t idx = u0 + i * T0;
      live[i] = idx < p.units;
      u[i] = live[i] ? unit_at(idx, p.groups, p.K, narrow) : Unit{0, 0};
    }
    if constexpr (what == What::Encode) {
      Loaded<T, kVec> x[kU];
#pragma unroll
      for (int i = 0; i < kU; ++i) x[i].load(a, u[i], l);
#pragma unroll
      for (int i = 0; i < kU; ++i) {
        float v[N];
        x[i].get(v);
        encode_unit(v, live[i], u[i], u0 + i * T0, l, p.c0, p.s0);
      }
    } else if constexpr (what == What::Decode) {
      LoadedCodes<kVec> c[kU];
      float s[kU];
#pragma unroll
      for (int i = 0; i < kU; ++i) {
        c[i].load(p.c0, u[i], l);
        s[i] = live[i] ? __ldg(p.s0 + u0 + i * T0) : 0.0f;
      }
#pragma unroll
      for (int i = 0; i < kU; ++i) {
        float v[N];
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
        float gv[N], uv[N], y[N];
        g[i].get(gv);
        q[i].get(uv);
#pragma unroll
        for (int j = 0; j < N; ++j) y[j] = gv[j] * sigmoid<T>(gv[j]) * uv[j];
        store_values(static_cast<T*>(p.o0), u[i], l, y);
        if constexpr (what == What::FwdSave) {
          encode_unit(gv, live[i], u[i], u0 + i * T0, l, p.c0, p.s0);
          encode_unit(uv, live[i], u[i], u0 + i * T0, l, p.c1, p.s1);
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
        sg[i] = live[i] ? __ldg(p.s0 + u0 + i * T0) : 0.0f;
        su[i] = live[i] ? __ldg(p.s1 + u0 + i * T0) : 0.0f;
      }
#pragma unroll
      for (int i = 0; i < kU; ++i) {
        float dv[N], gv[N], uv[N], dg[N], du[N];
        d[i].get(dv);
        cg[i].get(sg[i], gv);
        cu[i].get(su[i], uv);
#pragma unroll
        for (int j = 0; j < N; ++j) {
          const float s = sigmoid<T>(gv[j]);
          const float ds = dv[j] * s;
          dg[j] = ds * uv[j] * fmaf(gv[j], 1.0f - s, 1.0f);
          du[j] = ds * gv[j];
        }
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
