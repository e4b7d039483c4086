// Layer norm and RMS norm, forward and backward (N1, N2).
//
//   forward   mean, then sum (x - mean)^2 from the values in registers (two
//             reductions: no cancellation), y = (x - mean) rstd w + b, and the
//             8-bit form of x in the same pass
//   backward  g = dy w, xhat = (x - mean) rstd
//             dx = rstd (g - mean(g) - xhat mean(g xhat))
//             dweight = sum over rows of dy xhat, dbias = sum over rows of dy
//
// Both should be bound by HBM, but the work per value is near what an SM issues
// while its share of the bytes arrives, and a row's sums are a chain of shuffles
// and a barrier: no unit is saturated (ncu, 4096 x 2560 with the 8-bit x: SM 51
// and 36 %, L1 41 and 58 %). So a thread takes 16 or 32 columns of a row, that the
// row's sums, addresses and reciprocals cost little per value. A group of threads
// walks the rows of its own; each thread copies its columns of the next rows
// asynchronously into its own places of shared memory, which keeps the bytes
// in flight without registers and without barriers. Forward: several blocks
// per SM. Backward: one block per SM, whose threads keep their columns' sums
// of dweight and dbias in registers over all rows; the groups join them in
// shared memory and write one partial row per block to the workspace (148 x 2
// x K floats at most), which a second launch adds in a fixed order. Rows wider
// than 8192 columns take two passes in the backward: the row sums, then column
// strips.
//
// Measured on B200 (back to back in a graph, over inputs that rotate past L2), with
// the share of the copy rate: bf16 with the 8-bit x, 4096 x 2560: forward 13.2 us
// (0.62), backward 19.5 (0.42; of these 6 to 8 us are the start, the groups' joining
// and the second launch), 16384 x 2560: 41.2 (0.80) and 50.3 (0.65). 4096 x 2560 fp32:
// 16.1 (0.81) and 28.5 (0.68). Rows that fill every thread's places spare the column
// tests, a tenth of the time.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "bl_act8.cuh"
#include "bl_device.cuh"
#include "bl_internal.h"
#include "bl_rows.cuh"

namespace bl {
namespace {

struct NormArgs {
  const void* x;
  const void* weight;
  const void* bias;
  int p_f32;
  int64_t M;
  int K;
  int tpr;  // threads per row
  float eps;
  float k, inv_k;  // K and its reciprocal
  void* y;
  float* mean;
  float* rstd;
  int8_t* codes;
  float* scales;
};

// s / k, with inv = fp32(1 / k): the quotient's error is made good by one
// step with the exact remainder (a row of one value keeps its mean exactly).
// An infinite sum has no remainder: its mean is that infinity.
__device__ __forceinline__ float mean_of(float s, float k, float inv) {
  const float m = s * inv;
  return fabsf(m) < __uint_as_float(0x7F800000u) ? fmaf(fmaf(-m, k, s), inv, m) : m;
}

// group_sum of two values, whose buffer (a float2 per warp: 8-byte accesses) is
// given by its shared-memory address.
__device__ __forceinline__ void group_sum2(float (&v)[2], uint32_t buf, int t, int tpr, int barrier) {
  v[0] = warp_sum(v[0]);
  v[1] = warp_sum(v[1]);
  if (tpr == 32) return;
  if ((t & 31) == 0)
    asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(buf + (t >> 5) * 8), "f"(v[0]), "f"(v[1]) : "memory");
  group_barrier(barrier, tpr);
  f32x2 s = 0;
#pragma unroll 4
  for (int w = 0; w < (tpr >> 5); ++w) {
    f32x2 a;
    asm volatile("ld.shared.b64 %0, [%1];" : "=l"(a) : "r"(buf + w * 8) : "memory");
    s = add2(s, a);
  }
  split2(s, v[0], v[1]);
}

// ---------------------------------------------------------------- forward
constexpr int kFwdThreads = 256;  // most threads of a forward block
// Rows in flight per group: at most 96 and 128 KB per block (8 vectors).
template <typename T>
constexpr int kFwdDepth = sizeof(T) == 2 ? 3 : 2;

// Sum over the block's warps, at most 8: `buf` holds 8 floats, those of warps
// that the block does not have are 0. kWarp: the row is one warp's.
template <bool kWarp>
__device__ __forceinline__ float block_sum8(float v, float* buf, int t) {
  v = warp_sum(v);
  if constexpr (kWarp) return v;
  if ((t & 31) == 0) buf[t >> 5] = v;
  __syncthreads();
  const float4 a = reinterpret_cast<const float4*>(buf)[0], b = reinterpret_cast<const float4*>(buf)[1];
  return ((a.x + a.y) + (a.z + a.w)) + ((b.x + b.y) + (b.z + b.w));
}

// Vector rows: a block (kWarp: a warp) of tpr threads walks the rows first,
// first + step, ... with the next rows' loads in flight. kFull: the row fills
// every thread's vectors, so no column is tested (those tests cost a fifth of
// the instructions).
template <typename T, int kVecs, bool kRms, bool kSave, bool kFull, bool kWarp>
__global__ void __launch_bounds__(kFwdThreads, kVecs <= 2 ? 4 : kVecs == 4 ? 2 : 1)
    norm_forward_kernel(const NormArgs p) {
  pdl_wait_primary();
  pdl_launch_dependents();
  extern __shared__ uint4 ring[];
  __shared__ float4 sums[2][2];  // 8 floats each
  constexpr int kPieces = sizeof(T) / 2;  // 16-byte pieces per vector
  constexpr int kDepth = kFwdDepth<T>;
  const int K = p.K, tpr = kWarp ? 32 : blockDim.x;
  const int t = kWarp ? threadIdx.x & 31 : threadIdx.x;
  const uint32_t stride = blockDim.x * 16, row_stride = kVecs * kPieces * stride;
  const uint32_t mine = smem_u32(ring) + threadIdx.x * 16, end = mine + kDepth * row_stride;
  const int c0 = t * 8, cs = tpr * 8;  // the thread's vectors: columns c0 + j cs
  auto live = [&](int j) { return kFull || c0 + j * cs < K; };
  float* buf0 = reinterpret_cast<float*>(sums[0]);
  float* buf1 = reinterpret_cast<float*>(sums[1]);
  if constexpr (!kWarp) {
    if (threadIdx.x < 4) reinterpret_cast<float4*>(sums)[threadIdx.x] = make_float4(0.f, 0.f, 0.f, 0.f);
    __syncthreads();
  }
  const int64_t first = kWarp ? static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5) : blockIdx.x;
  const int64_t step = kWarp ? static_cast<int64_t>(gridDim.x) * (blockDim.x >> 5) : gridDim.x, step_k = step * K;
  int rows = first < p.M ? static_cast<int>((p.M - 1 - first) / step) + 1 : 0, left = rows;
  int64_t row = first, at = row * K + c0;            // the thread's place in this row
  const T* ahead = static_cast<const T*>(p.x) + at;  // and in the row to load next
  const int groups = (K + kAct8Group - 1) / kAct8Group;
  auto issue = [&](uint32_t slot) {
    if (left > 0) {
#pragma unroll
      for (int j = 0; j < kVecs; ++j)
        if (live(j)) issue8(slot + j * kPieces * stride, stride, ahead + j * cs);
      ahead += step_k;
      --left;
    }
    copy_async_commit();
  };
#pragma unroll
  for (int s = 0; s < kDepth; ++s) issue(mine + s * row_stride);
  f32x2 w[kVecs][4];
#pragma unroll
  for (int j = 0; j < kVecs; ++j) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[j][i] = both2(1.0f);
    if (p.weight && live(j)) load_params8(p.weight, p.p_f32, c0 + j * cs, w[j]);
  }
  for (uint32_t slot = mine; rows > 0; --rows, row += step, at += step_k) {
    copy_async_wait<kDepth - 1>();
    Raw8<T> raw[kVecs];
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      if (live(j)) read_raw(slot + j * kPieces * stride, stride, raw[j]);
      else raw[j].clear();
    }
    issue(slot);
    slot += row_stride;
    if (slot == end) slot = mine;
    float mean = 0.0f;
    if constexpr (!kRms) {
      f32x2 s2 = 0;
#pragma unroll
      for (int j = 0; j < kVecs; ++j) {
        f32x2 v[4];
        raw[j].get(v);
        s2 = add2(s2, add2(add2(v[0], v[1]), add2(v[2], v[3])));
      }
      mean = mean_of(block_sum8<kWarp>(sum2(s2), buf0, t), p.k, p.inv_k);
    }
    if constexpr (kSave) {
      // the 16 lanes of half a warp hold a group's 128 columns
#pragma unroll
      for (int j = 0; j < kVecs; ++j) {
        const Act8Scale a = act8_scale(act8_absmax<16>(raw[j].absmax()));
        if (live(j)) {
          f32x2 v[4];
          raw[j].get(v);
          *reinterpret_cast<uint2*>(p.codes + at + j * cs) = act8_codes8(v, a.inv);
          if ((t & 15) == 0) p.scales[row * groups + (c0 + j * cs) / kAct8Group] = a.scale;
        }
      }
    }
    const f32x2 nmean2 = both2(-mean);
    f32x2 q2 = 0;
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      if (live(j)) {
        f32x2 v[4];
        raw[j].get(v);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const f32x2 a = kRms ? v[i] : add2(v[i], nmean2);
          q2 = fma2(a, a, q2);
        }
      }
    }
    const float rstd = rsqrt_of(fmaf(block_sum8<kWarp>(sum2(q2), buf1, t), p.inv_k, p.eps));
    if (t == 0) {
      if constexpr (!kRms) p.mean[row] = mean;
      p.rstd[row] = rstd;
    }
    const f32x2 rstd2 = both2(rstd);
    T* y = static_cast<T*>(p.y) + at;
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      if (live(j)) {
        f32x2 o[4];
        raw[j].get(o);
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = mul2(mul2(kRms ? o[i] : add2(o[i], nmean2), rstd2), w[j][i]);
        if (p.bias) {
          f32x2 b[4];
          load_params8(p.bias, p.p_f32, c0 + j * cs, b);
#pragma unroll
          for (int i = 0; i < 4; ++i) o[i] = add2(o[i], b[i]);
        }
        store8(y + j * cs, o);
      }
    }
    // RMS norm has one sum per row: its buffer is free again only once every
    // warp has read it
    if constexpr (kRms && !kWarp) __syncthreads();
  }
}

// Scalar rows (K % 8 != 0: a row starts at any element): 8 columns per thread,
// one group per row.
template <typename T>
__global__ void __launch_bounds__(1024) norm_forward_scalar_kernel(const NormArgs p, int rms) {
  pdl_wait_primary();
  pdl_launch_dependents();
  __shared__ float sums[2][32];
  const int tpr = p.tpr, K = p.K;
  const int grp = threadIdx.x / tpr, t = threadIdx.x % tpr;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (blockDim.x / tpr) + grp;
  if (row >= p.M) return;  // whole groups leave
  const T* x = static_cast<const T*>(p.x) + row * K;
  const int warp0 = grp * (tpr >> 5);
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = t + i * tpr < K ? to_f32(x[t + i * tpr]) : 0.0f;
  float mean = 0.0f;
  if (!rms) {
    float s[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < 8; ++i) s[0] += v[i];
    group_sum(s, sums[0] + warp0, t, tpr, 1 + grp);
    mean = mean_of(s[0], p.k, p.inv_k);
  }
  float q[1] = {0.0f};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[i] -= mean;
    q[0] += t + i * tpr < K ? v[i] * v[i] : 0.0f;
  }
  group_sum(q, sums[1] + warp0, t, tpr, 1 + grp);
  const float rstd = rsqrt_of(fmaf(q[0], p.inv_k, p.eps));
  if (t == 0) {
    if (!rms) p.mean[row] = mean;
    p.rstd[row] = rstd;
  }
  T* y = static_cast<T*>(p.y) + row * K;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int c = t + i * tpr;
    if (c < K) {
      float o = v[i] * rstd;
      if (p.weight) o *= load_param(p.weight, p.p_f32, c);
      if (p.bias) o += load_param(p.bias, p.p_f32, c);
      store1(y + c, o);
    }
  }
}

// Rows that do not fit in a block's registers: one block per row, which is
// read three times (from L2 after the first).
template <typename T>
__global__ void __launch_bounds__(1024) norm_forward_wide_kernel(const NormArgs p, int rms) {
  pdl_wait_primary();
  pdl_launch_dependents();
  __shared__ float sums[2][32];
  const int t = threadIdx.x, K = p.K;
  for (int64_t row = blockIdx.x; row < p.M; row += gridDim.x) {
    const T* x = static_cast<const T*>(p.x) + row * K;
    float mean = 0.0f;
    if (!rms) {
      float s[1] = {0.0f};
      for (int c = t; c < K; c += 1024) s[0] += to_f32(x[c]);
      group_sum(s, sums[0], t, 1024, 1);
      mean = mean_of(s[0], p.k, p.inv_k);
    }
    float q[1] = {0.0f};
    for (int c = t; c < K; c += 1024) {
      const float d = to_f32(x[c]) - mean;
      q[0] += d * d;
    }
    group_sum(q, sums[1], t, 1024, 1);
    const float rstd = rsqrt_of(fmaf(q[0], p.inv_k, p.eps));
    if (t == 0) {
      if (!rms) p.mean[row] = mean;
      p.rstd[row] = rstd;
    }
    T* y = static_cast<T*>(p.y) + row * K;
    for (int c = t; c < K; c += 1024) {
      float o = (to_f32(x[c]) - mean) * rstd;
      if (p.weight) o *= load_param(p.weight, p.p_f32, c);
      if (p.bias) o += load_param(p.bias, p.p_f32, c);
      store1(y + c, o);
    }
    __syncthreads();  // the next row's sums reuse the buffers
  }
}

// ---------------------------------------------------------------- backward
struct NormBwdArgs {
  const void* dy;
  const void* x;  // or null: codes, scales
  const int8_t* codes;
  const float* scales;
  const void* weight;
  int p_f32;
  const float* mean;
  const float* rstd;
  int64_t M;
  int K;
  int tpr;
  float inv_k;
  int rms;
  void* dx;
  float* parts;      // [blocks][2][K], or null when neither sum is wanted
  float2* row_sums;  // wide rows: (c1, c2) per row
};

// A thread's 8 columns of a row of dy and x, as loaded.
template <typename T, bool kVec, bool kSaved>
struct RowIn;
template <typename T>
struct RowIn<T, true, false> {
  Raw8<T> d, x;
  __device__ __forceinline__ void load(const NormBwdArgs& p, int64_t row, int t, int tpr, int c0) {
    if (c0 < p.K) {
      d.load(static_cast<const T*>(p.dy) + row * p.K + c0);
      x.load(static_cast<const T*>(p.x) + row * p.K + c0);
    } else {
      d.clear();
      x.clear();
    }
  }
  __device__ __forceinline__ void get(f32x2 (&dv)[4], f32x2 (&xv)[4]) const {
    d.get(dv);
    x.get(xv);
  }
};
template <typename T>
struct RowIn<T, true, true> {
  Raw8<T> d;
  uint2 c;
  float s;
  __device__ __forceinline__ void load(const NormBwdArgs& p, int64_t row, int t, int tpr, int c0) {
    if (c0 < p.K) {
      d.load(static_cast<const T*>(p.dy) + row * p.K + c0);
      c = *reinterpret_cast<const uint2*>(p.codes + row * p.K + c0);
      s = __ldg(p.scales + row * ((p.K + kAct8Group - 1) / kAct8Group) + c0 / kAct8Group);
    } else {
      d.clear();
      c = make_uint2(0u, 0u);
      s = 0.0f;
    }
  }
  __device__ __forceinline__ void get(f32x2 (&dv)[4], f32x2 (&xv)[4]) const {
    d.get(dv);
    act8_values8(c, s, xv);
  }
};
template <typename T, bool kSaved>
struct RowIn<T, false, kSaved> {
  float d[8], x[8];
  __device__ __forceinline__ void load(const NormBwdArgs& p, int64_t row, int t, int tpr, int c0) {
    const int groups = (p.K + kAct8Group - 1) / kAct8Group;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = c0 + i * tpr;
      d[i] = x[i] = 0.0f;
      if (c < p.K) {
        d[i] = to_f32(static_cast<const T*>(p.dy)[row * p.K + c]);
        if constexpr (kSaved) x[i] = act8_value(p.codes[row * p.K + c], __ldg(p.scales + row * groups + c / kAct8Group));
        else x[i] = to_f32(static_cast<const T*>(p.x)[row * p.K + c]);
      }
    }
  }
  __device__ __forceinline__ void get(f32x2 (&dv)[4], f32x2 (&xv)[4]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) dv[i] = pair2(d[2 * i], d[2 * i + 1]), xv[i] = pair2(x[2 * i], x[2 * i + 1]);
  }
};

// Weights of the thread's 8 columns (zero outside the row).
template <bool kVec>
__device__ __forceinline__ void load_weights(const NormBwdArgs& p, int c0, int tpr, f32x2 (&w)[4]) {
  float f[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int c = kVec ? c0 + i : c0 + i * tpr;
    f[i] = c >= p.K ? 0.0f : p.weight ? load_param(p.weight, p.p_f32, c) : 1.0f;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = pair2(f[2 * i], f[2 * i + 1]);
}

template <typename T, bool kVec>
__device__ __forceinline__ void store_row(T* dx, int K, int c0, int tpr, const f32x2 (&o)[4]) {
  if constexpr (kVec) {
    if (c0 < K) store8(dx + c0, o);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float lo, hi;
      split2(o[i], lo, hi);
      if (c0 + 2 * i * tpr < K) store1(dx + c0 + 2 * i * tpr, lo);
      if (c0 + (2 * i + 1) * tpr < K) store1(dx + c0 + (2 * i + 1) * tpr, hi);
    }
  }
}

// Where a thread keeps rows in flight: 16-byte pieces of dy, then of x, or one
// piece with 8 codes and their scale.
template <typename T, bool kSaved>
struct RowRing {
  static constexpr int kVal = sizeof(T) / 2;
  static constexpr int kPieces = kVal + (kSaved ? 1 : kVal);
  // How far the places move from one row of the group to the next.
  struct Step {
    int64_t row, scale;
    __device__ __forceinline__ Step(int64_t step, int K, int groups) : row(step * K), scale(step * groups) {}
  };
  // The thread's places in the row to load next.
  struct From {
    const T* dy;
    const T* x;
    const int8_t* codes;
    const float* scale;
    int next_scale;  // from the first vector's scale to the second's
    __device__ __forceinline__ From(const NormBwdArgs& p, int64_t row, int c0, int cs, int groups) {
      const int64_t at = row * p.K + c0;
      dy = static_cast<const T*>(p.dy) + at;
      if constexpr (kSaved) {
        codes = p.codes + at;
        scale = p.scales + row * groups + c0 / kAct8Group;
        next_scale = (c0 + cs) / kAct8Group - c0 / kAct8Group;
      } else {
        x = static_cast<const T*>(p.x) + at;
      }
    }
    __device__ __forceinline__ void issue(int j, int cs, uint32_t at, uint32_t stride) const {
      issue8(at, stride, dy + j * cs);
      if constexpr (kSaved) {
        copy_async8(at + kVal * stride, codes + j * cs);
        copy_async4(at + kVal * stride + 8, scale + j * next_scale);
      } else {
        issue8(at + kVal * stride, stride, x + j * cs);
      }
    }
    __device__ __forceinline__ void advance(const Step& s) {
      dy += s.row;
      if constexpr (kSaved) codes += s.row, scale += s.scale;
      else x += s.row;
    }
  };
  __device__ static __forceinline__ void read(uint32_t at, uint32_t stride, f32x2 (&d)[4], f32x2 (&x)[4]) {
    Raw8<T> r;
    read_raw(at, stride, r);
    r.get(d);
    if constexpr (kSaved) {
      const uint4 c = lds16(at + kVal * stride);
      act8_values8(make_uint2(c.x, c.y), __uint_as_float(c.z), x);
    } else {
      read_raw(at + kVal * stride, stride, r);
      r.get(x);
    }
  }
};

// A row's part in the sums and in dx, for 8 columns of a thread (x becomes
// xhat; nmean = -mean).
__device__ __forceinline__ void row_sums(const f32x2 (&d)[4], f32x2 (&x)[4], const f32x2 (&w)[4], f32x2 nmean,
                                         f32x2 rstd, f32x2& s0, f32x2& s1, f32x2 (&dw)[4], f32x2 (&db)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[i] = mul2(add2(x[i], nmean), rstd);
    const f32x2 g = mul2(d[i], w[i]);
    s0 = add2(s0, g);
    s1 = fma2(g, x[i], s1);
    dw[i] = fma2(d[i], x[i], dw[i]);
    db[i] = add2(db[i], d[i]);
  }
}
// nc1, nc2: -c1 and -c2.
__device__ __forceinline__ void row_dx(const f32x2 (&d)[4], const f32x2 (&xhat)[4], const f32x2 (&w)[4], f32x2 rstd,
                                       f32x2 nc1, f32x2 nc2, f32x2 (&o)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = mul2(rstd, fma2(xhat[i], nc2, fma2(d[i], w[i], nc1)));
}

// The groups' sums of dweight and dbias, joined in order into the block's
// partial row. joint: [groups][2][width].
__device__ __forceinline__ void join_groups(const NormBwdArgs& p, const float* joint, int ngrp, int width) {
  __syncthreads();
  const int K = p.K;
  float* part = p.parts + static_cast<int64_t>(blockIdx.x) * 2 * K;
  for (int c = threadIdx.x; c < K; c += blockDim.x) {
    float a = 0.0f, b = 0.0f;
    for (int g = 0; g < ngrp; ++g) {
      a += joint[g * 2 * width + c];
      b += joint[g * 2 * width + width + c];
    }
    part[c] = a;
    part[K + c] = b;
  }
}

constexpr int kBwdThreads = 512;  // of a block of the vector kernel, one block per SM
constexpr int kBwdVecs = 2;       // vectors of 8 columns per thread
// Rows in flight: 512 threads x 2 vectors x depth x pieces x 16 bytes = 128,
// 128, 192 and 144 KB (bf16, bf16 from 8 bits, fp32, fp32 from 8 bits).
template <typename T>
constexpr int kBwdDepth = sizeof(T) == 2 ? 4 : 3;

// Vector rows. kFull: as in the forward.
template <typename T, bool kSaved, bool kFull>
__global__ void __launch_bounds__(kBwdThreads, 1) norm_backward_kernel(const NormBwdArgs p) {
  pdl_wait_primary();
  pdl_launch_dependents();
  extern __shared__ uint4 ring[];  // the rows in flight; afterwards the groups' sums
  __shared__ float2 sums[2][kBwdThreads / 32];
  using Ring = RowRing<T, kSaved>;
  constexpr int kDepth = kBwdDepth<T>;
  const int tpr = p.tpr, K = p.K;
  const int ngrp = blockDim.x / tpr;
  const int grp = threadIdx.x / tpr, t = threadIdx.x % tpr;
  const int c0 = t * 8, cs = tpr * 8;
  auto live = [&](int j) { return kFull || c0 + j * cs < K; };
  const uint32_t stride = blockDim.x * 16, row_stride = kBwdVecs * Ring::kPieces * stride;
  const uint32_t mine = smem_u32(ring) + threadIdx.x * 16, end = mine + kDepth * row_stride;
  uint32_t buf = smem_u32(sums[0] + grp * (tpr >> 5));
  const uint32_t bufs = buf ^ (buf + static_cast<uint32_t>(sizeof(sums[0])));
  const int64_t first = static_cast<int64_t>(blockIdx.x) * ngrp + grp;
  const int64_t step = static_cast<int64_t>(gridDim.x) * ngrp, step_k = step * K;
  int rows = first < p.M ? static_cast<int>((p.M - 1 - first) / step) + 1 : 0, left = rows;
  const int groups = (K + kAct8Group - 1) / kAct8Group;
  // the thread's places: in dx, and in what the row to load next reads
  T* dx = static_cast<T*>(p.dx) + (p.dx ? first * K + c0 : 0);
  typename Ring::From from(p, first, c0, cs, groups);
  const typename Ring::Step from_step(step, K, groups);
  auto issue = [&](uint32_t slot) {
    if (left > 0) {
#pragma unroll
      for (int j = 0; j < kBwdVecs; ++j)
        if (live(j)) from.issue(j, cs, slot + j * Ring::kPieces * stride, stride);
      from.advance(from_step);
      --left;
    }
    copy_async_commit();
  };
#pragma unroll
  for (int s = 0; s < kDepth; ++s) issue(mine + s * row_stride);
  const float* mean_at = p.rms ? p.rstd + first : p.mean + first;
  const float* rstd_at = p.rstd + first;
  float mean = 0.0f, rstd = 0.0f;
  if (rows > 0) {
    mean = __ldg(mean_at);
    rstd = __ldg(rstd_at);
  }
  f32x2 w[kBwdVecs][4], dw[kBwdVecs][4], db[kBwdVecs][4];
#pragma unroll
  for (int j = 0; j < kBwdVecs; ++j) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w[j][i] = both2(1.0f);
      dw[j][i] = db[j][i] = 0;
    }
    if (p.weight && live(j)) load_params8(p.weight, p.p_f32, c0 + j * cs, w[j]);
  }
  for (uint32_t slot = mine; rows > 0; --rows) {
    const f32x2 nmean2 = both2(p.rms ? 0.0f : -mean), rstd2 = both2(rstd);
    if (rows > 1) {
      mean = __ldg(mean_at += step);
      rstd = __ldg(rstd_at += step);
    }
    copy_async_wait<kDepth - 1>();
    f32x2 s0 = 0, s1 = 0, d[kBwdVecs][4], x[kBwdVecs][4];
#pragma unroll
    for (int j = 0; j < kBwdVecs; ++j) {
      if (live(j)) {
        Ring::read(slot + j * Ring::kPieces * stride, stride, d[j], x[j]);
        row_sums(d[j], x[j], w[j], nmean2, rstd2, s0, s1, dw[j], db[j]);
      }
    }
    issue(slot);
    slot += row_stride;
    if (slot == end) slot = mine;
    if (p.dx) {
      // two buffers in turn: one barrier per row
      float s[2] = {sum2(s0), sum2(s1)};
      group_sum2(s, buf, t, tpr, 1 + grp);
      buf ^= bufs;
      const f32x2 nc1 = both2(p.rms ? 0.0f : -s[0] * p.inv_k), nc2 = both2(-s[1] * p.inv_k);
#pragma unroll
      for (int j = 0; j < kBwdVecs; ++j) {
        if (live(j)) {
          f32x2 o[4];
          row_dx(d[j], x[j], w[j], rstd2, nc1, nc2, o);
          store8(dx + j * cs, o);
        }
      }
      dx += step_k;
    }
  }
  if (!p.parts) return;
  copy_async_wait<0>();
  __syncthreads();  // the ring becomes the joint sums
  float* joint = reinterpret_cast<float*>(ring);
  const int width = kBwdVecs * 8 * tpr;
#pragma unroll
  for (int j = 0; j < kBwdVecs; ++j) {
    float* at = joint + grp * 2 * width + c0 + j * cs;
    store8(at, dw[j]);
    store8(at + width, db[j]);
  }
  join_groups(p, joint, ngrp, width);
}

// Scalar rows.
template <typename T, bool kSaved>
__global__ void __launch_bounds__(1024, 1) norm_backward_scalar_kernel(const NormBwdArgs p) {
  pdl_wait_primary();
  pdl_launch_dependents();
  extern __shared__ uint4 ring[];  // the groups' sums
  __shared__ float2 sums[2][32];
  const int tpr = p.tpr, K = p.K;
  const int ngrp = blockDim.x / tpr;
  const int grp = threadIdx.x / tpr, t = threadIdx.x % tpr;
  const uint32_t sum0 = smem_u32(sums[0] + grp * (tpr >> 5));
  f32x2 w[4], dw[4] = {}, db[4] = {};
  load_weights<false>(p, t, tpr, w);
  int par = 0;
  const int64_t step = static_cast<int64_t>(gridDim.x) * ngrp;
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * ngrp + grp; row < p.M; row += step) {
    RowIn<T, false, kSaved> in;
    in.load(p, row, t, tpr, t);
    const f32x2 nmean2 = both2(p.rms ? 0.0f : -__ldg(p.mean + row)), rstd2 = both2(__ldg(p.rstd + row));
    f32x2 d[4], x[4], s0 = 0, s1 = 0;
    in.get(d, x);
    row_sums(d, x, w, nmean2, rstd2, s0, s1, dw, db);
    if (p.dx) {
      float s[2] = {sum2(s0), sum2(s1)};
      group_sum2(s, sum0 + par * static_cast<uint32_t>(sizeof(sums[0])), t, tpr, 1 + grp);
      par ^= 1;
      f32x2 o[4];
      row_dx(d, x, w, rstd2, both2(p.rms ? 0.0f : -s[0] * p.inv_k), both2(-s[1] * p.inv_k), o);
      store_row<T, false>(static_cast<T*>(p.dx) + row * K, K, t, tpr, o);
    }
  }
  if (!p.parts) return;
  float* joint = reinterpret_cast<float*>(ring) + grp * 16 * tpr + t;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    split2(dw[i], joint[2 * i * tpr], joint[(2 * i + 1) * tpr]);
    split2(db[i], joint[8 * tpr + 2 * i * tpr], joint[8 * tpr + (2 * i + 1) * tpr]);
  }
  join_groups(p, reinterpret_cast<float*>(ring), ngrp, 8 * tpr);
}

// Wide rows, first pass: the two sums of each row.
template <typename T, bool kSaved>
__global__ void __launch_bounds__(1024) norm_row_sums_kernel(const NormBwdArgs p) {
  pdl_wait_primary();
  pdl_launch_dependents();
  __shared__ float sums[32 * 2];
  const int t = threadIdx.x, K = p.K;
  for (int64_t row = blockIdx.x; row < p.M; row += gridDim.x) {
    const f32x2 nmean2 = both2(p.rms ? 0.0f : -__ldg(p.mean + row)), rstd2 = both2(__ldg(p.rstd + row));
    f32x2 s0 = 0, s1 = 0;
    for (int c0 = t; c0 < K; c0 += 8 * 1024) {
      RowIn<T, false, kSaved> in;
      in.load(p, row, t, 1024, c0);
      f32x2 w[4], d[4], x[4];
      load_weights<false>(p, c0, 1024, w);
      in.get(d, x);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const f32x2 g = mul2(d[i], w[i]);
        s0 = add2(s0, g);
        s1 = fma2(g, mul2(add2(x[i], nmean2), rstd2), s1);
      }
    }
    float s[2] = {sum2(s0), sum2(s1)};
    group_sum(s, sums, t, 1024, 1);
    if (t == 0) p.row_sums[row] = make_float2(p.rms ? 0.0f : s[0] * p.inv_k, s[1] * p.inv_k);
    __syncthreads();
  }
}

// Wide rows, second pass: block (strip, y) takes columns strip * 2048 .. of
// the rows y, y + gridDim.y, ...
template <typename T, bool kVec, bool kSaved>
__global__ void __launch_bounds__(256) norm_strip_kernel(const NormBwdArgs p) {
  pdl_wait_primary();
  pdl_launch_dependents();
  const int K = p.K, t = threadIdx.x;
  const int c0 = static_cast<int>(blockIdx.x) * 2048 + (kVec ? t * 8 : t);
  f32x2 w[4], dw[4] = {}, db[4] = {};
  load_weights<kVec>(p, c0, 256, w);
  for (int64_t row = blockIdx.y; row < p.M; row += gridDim.y) {
    RowIn<T, kVec, kSaved> in;
    in.load(p, row, t, 256, c0);
    const f32x2 nmean2 = both2(p.rms ? 0.0f : -__ldg(p.mean + row)), rstd2 = both2(__ldg(p.rstd + row));
    const float2 c = p.dx ? p.row_sums[row] : make_float2(0.0f, 0.0f);
    f32x2 d[4], x[4], s0 = 0, s1 = 0;
    in.get(d, x);
    row_sums(d, x, w, nmean2, rstd2, s0, s1, dw, db);
    if (p.dx) {
      f32x2 o[4];
      row_dx(d, x, w, rstd2, both2(-c.x), both2(-c.y), o);
      store_row<T, kVec>(static_cast<T*>(p.dx) + row * K, K, c0, 256, o);
    }
  }
  if (!p.parts) return;
  float* part = p.parts + static_cast<int64_t>(blockIdx.y) * 2 * K;
  float a[8], b[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    split2(dw[i], a[2 * i], a[2 * i + 1]);
    split2(db[i], b[2 * i], b[2 * i + 1]);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int c = kVec ? c0 + i : c0 + i * 256;
    if (c < K) {
      part[c] = a[i];
      part[K + c] = b[i];
    }
  }
}

// dweight, dbias from the blocks' partial rows: 32 columns per block, the
// partial rows (at most 148) spread over 32 threads of each column, whose
// loads are all in flight at once.
constexpr int kMaxParts = kPlanSms;

__global__ void __launch_bounds__(1024) norm_join_kernel(const float* __restrict__ parts, int nparts, int K,
                                                         void* dweight, void* dbias, int p_f32, int accumulate) {
  pdl_wait_primary();
  pdl_launch_dependents();
  __shared__ float sh[2][32][33];
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
  const int c = static_cast<int>(blockIdx.x) * 32 + x;
  constexpr int kU = (kMaxParts + 31) / 32;
  float a[kU], b[kU];
#pragma unroll
  for (int i = 0; i < kU; ++i) {
    const int r = y + 32 * i;
    a[i] = b[i] = 0.0f;
    if (c < K && r < nparts) {
      if (dweight) a[i] = parts[static_cast<int64_t>(r) * 2 * K + c];
      if (dbias) b[i] = parts[static_cast<int64_t>(r) * 2 * K + K + c];
    }
  }
#pragma unroll
  for (int i = 1; i < kU; ++i) a[0] += a[i], b[0] += b[i];
  sh[0][y][x] = a[0];
  sh[1][y][x] = b[0];
  __syncthreads();
  // warp y adds column y of either sum
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    void* out = which == 0 ? dweight : dbias;
    const int col = static_cast<int>(blockIdx.x) * 32 + y;
    if (!out || col >= K) continue;
    const float s = warp_sum(sh[which][x][y]);
    if (x != 0) continue;
    if (p_f32) {
      float* o = static_cast<float*>(out) + col;
      *o = accumulate ? s + *o : s;
    } else {
      __nv_bfloat16* o = static_cast<__nv_bfloat16*>(out) + col;
      *o = __float2bfloat16_rn(accumulate ? s + __bfloat162float(*o) : s);
    }
  }
}

// ---------------------------------------------------------------- host side
constexpr int kFwdMaxK = 16384;  // 256 threads x 8 vectors of 8
constexpr int kBwdMaxK = 8192;   // 512 threads x 16 columns (scalar: 1024 x 8)

template <typename T, int kVecs, bool kRms, bool kSave, bool kFull, bool kWarp>
cudaError_t forward_launch(const NormArgs& p, int tpr, cudaStream_t s) {
  const int block = kWarp ? kFwdThreads : tpr, per = kWarp ? kFwdThreads / 32 : 1;
  constexpr size_t kPerThread = static_cast<size_t>(kFwdDepth<T>) * kVecs * 8 * sizeof(T);
  auto kernel = norm_forward_kernel<T, kVecs, kRms, kSave, kFull, kWarp>;
  static bool done[64] = {};
  if (cudaError_t e = allow_smem(kernel, kPerThread * kFwdThreads, done); e != cudaSuccess) return e;
  // blocks resident on an SM: the launch bounds leave registers for 1024, 512
  // or 256 threads
  int blocks = (kVecs <= 2 ? 1024 : kVecs == 4 ? 512 : 256) / block;
  const int by_smem = static_cast<int>(size_t(227 * 1024) / (kPerThread * block + 1280));
  if (blocks > by_smem) blocks = by_smem;
  const int64_t want = (p.M + per - 1) / per, most = static_cast<int64_t>(blocks < 1 ? 1 : blocks) * device_sm_count();
  return launch_pdl(kernel, dim3(static_cast<unsigned>(want < most ? want : most)), dim3(block), kPerThread * block, s, p);
}

template <typename T, int kVecs, bool kRms, bool kSave>
cudaError_t forward_vec(const NormArgs& p, cudaStream_t s) {
  const int tpr = round32((p.K + 8 * kVecs - 1) / (8 * kVecs));
  const bool full = tpr * 8 * kVecs == p.K;
  if (tpr == 32) {
    if constexpr (kVecs <= 4)
      return full ? forward_launch<T, kVecs, kRms, kSave, true, true>(p, tpr, s)
                  : forward_launch<T, kVecs, kRms, kSave, false, true>(p, tpr, s);
  }
  return full ? forward_launch<T, kVecs, kRms, kSave, true, false>(p, tpr, s)
              : forward_launch<T, kVecs, kRms, kSave, false, false>(p, tpr, s);
}

template <typename T, bool kRms, bool kSave>
cudaError_t forward_rows(const NormArgs& p, cudaStream_t s) {
  // the most columns per thread (16, 32 or, for the widest rows, 64) that
  // leave at most a tenth of the group's places empty. Measured on B200 (bf16),
  // 32 against 16: 4096 x 4096 with codes 14.8 and 16.9 us, 4096 x 1024 4.3 and 4.7
  const int k2 = round32((p.K + 15) / 16) * 16, k4 = round32((p.K + 31) / 32) * 32;
  if (p.K > 8192) return forward_vec<T, 8, kRms, kSave>(p, s);
  if (p.K > 4096 || 10 * (k4 - p.K) <= k4 || k4 <= k2) return forward_vec<T, 4, kRms, kSave>(p, s);
  return forward_vec<T, 2, kRms, kSave>(p, s);
}

template <typename T>
cudaError_t forward(NormArgs p, int rms, cudaStream_t s) {
  const bool vec = p.K % 8 == 0 && p.K <= kFwdMaxK;
  cudaError_t e;
  if (vec) {
    if (p.codes) return rms ? forward_rows<T, true, true>(p, s) : forward_rows<T, false, true>(p, s);
    return rms ? forward_rows<T, true, false>(p, s) : forward_rows<T, false, false>(p, s);
  }
  if (p.K <= 8192) {
    p.tpr = round32((p.K + 7) / 8);
    const int groups = p.tpr >= 256 ? 1 : 256 / p.tpr;
    e = launch_pdl(norm_forward_scalar_kernel<T>, dim3(static_cast<unsigned>((p.M + groups - 1) / groups)),
                   dim3(groups * p.tpr), 0, s, p, rms);
  } else {
    const unsigned grid = static_cast<unsigned>(p.M < (1 << 20) ? p.M : (1 << 20));
    e = launch_pdl(norm_forward_wide_kernel<T>, dim3(grid), dim3(1024), 0, s, p, rms);
  }
  if (e != cudaSuccess || !p.codes) return e;
  return launch_act8_encode(p.x, sizeof(T) == 4, p.M, p.K, p.codes, p.scales, s);
}

template <typename T, bool kVec, bool kSaved>
cudaError_t backward(NormBwdArgs p, int* nparts, cudaStream_t s) {
  if (p.K > kBwdMaxK) {
    if (p.dx) {
      const unsigned grid = static_cast<unsigned>(p.M < (1 << 20) ? p.M : (1 << 20));
      if (cudaError_t e = launch_pdl(norm_row_sums_kernel<T, kSaved>, dim3(grid), dim3(1024), 0, s, p); e != cudaSuccess)
        return e;
    }
    const int rows = static_cast<int>(p.M < kMaxParts ? p.M : kMaxParts);
    *nparts = rows;
    return launch_pdl(norm_strip_kernel<T, kVec, kSaved>, dim3((p.K + 2047) / 2048, rows), dim3(256), 0, s, p);
  }
  // a thread's columns, the block's threads, and shared memory per thread: the
  // rows in flight, and afterwards the groups' sums (two floats per column)
  const int cols = kVec ? 8 * kBwdVecs : 8, threads = kVec ? kBwdThreads : 1024;
  const int tpr = round32((p.K + cols - 1) / cols);
  int groups = threads / tpr;
  if (tpr > 32 && groups > 15) groups = 15;  // named barriers 1..15 (a row of 32 threads needs none)
  // few rows: smaller blocks (128 threads at least) on more SMs, where that halves
  // them or more. Measured on B200: 333 x 1001 fp32 5.5 us for 7.2, 256 x 512 4.0
  // for 5.6; short of half of it the larger blocks win (2048 x 512: 6.8, 7.5 spread)
  const int64_t spread = (p.M + kMaxParts - 1) / kMaxParts, least = 128 / tpr > 1 ? 128 / tpr : 1;
  if (const int64_t few = spread > least ? spread : least; 2 * few <= groups) groups = static_cast<int>(few);
  const int block = groups * tpr;
  const int64_t want = (p.M + groups - 1) / groups;
  const int grid = static_cast<int>(want < kMaxParts ? want : kMaxParts);
  p.tpr = tpr;
  *nparts = grid;
  size_t per_thread = static_cast<size_t>(cols) * 8;
  if constexpr (kVec) {
    constexpr size_t kRing = 16 * RowRing<T, kSaved>::kPieces * kBwdVecs * kBwdDepth<T>;
    if (kRing > per_thread) per_thread = kRing;
  }
  auto go = [&](auto kernel, bool (&done)[64]) {
    if (cudaError_t e = allow_smem(kernel, threads * per_thread, done); e != cudaSuccess) return e;
    return launch_pdl(kernel, dim3(grid), dim3(block), block * per_thread, s, p);
  };
  static bool done[2][64] = {};
  if constexpr (kVec)
    return tpr * cols == p.K ? go(norm_backward_kernel<T, kSaved, true>, done[0])
                             : go(norm_backward_kernel<T, kSaved, false>, done[1]);
  else
    return go(norm_backward_scalar_kernel<T, kSaved>, done[0]);
}

}  // namespace

size_t norm_backward_workspace_bytes(int64_t M, int64_t K) {
  const size_t parts = static_cast<size_t>(kMaxParts) * 2 * static_cast<size_t>(K) * 4;
  return parts + (K > kBwdMaxK ? static_cast<size_t>(M) * 8 : 0);
}

cudaError_t launch_norm_forward(const void* x, int f32, const void* weight, const void* bias, int p_f32, int64_t M,
                                int64_t K, float eps, int rms, void* y, float* mean, float* rstd, int8_t* codes,
                                float* scales, cudaStream_t s) {
  NormArgs p{};
  p.x = x;
  p.weight = weight;
  p.bias = bias;
  p.p_f32 = p_f32;
  p.M = M;
  p.K = static_cast<int>(K);
  p.eps = eps;
  p.k = static_cast<float>(K);
  p.inv_k = 1.0f / p.k;
  p.y = y;
  p.mean = mean;
  p.rstd = rstd;
  p.codes = codes;
  p.scales = scales;
  return f32 ? forward<float>(p, rms, s) : forward<__nv_bfloat16>(p, rms, s);
}

cudaError_t launch_norm_backward(const void* dy, const void* x, const int8_t* codes, const float* scales, int f32,
                                 const void* weight, int p_f32, const float* mean, const float* rstd, int64_t M,
                                 int64_t K, int rms, void* dx, void* dweight, void* dbias, int accumulate,
                                 void* workspace, cudaStream_t s) {
  NormBwdArgs p{};
  p.dy = dy;
  p.x = x;
  p.codes = codes;
  p.scales = scales;
  p.weight = weight;
  p.p_f32 = p_f32;
  p.mean = mean;
  p.rstd = rstd;
  p.M = M;
  p.K = static_cast<int>(K);
  p.inv_k = 1.0f / static_cast<float>(K);
  p.rms = rms;
  p.dx = dx;
  const bool sums = dweight || dbias;
  if (M == 0 && accumulate) return cudaSuccess;
  p.parts = sums ? static_cast<float*>(workspace) : nullptr;
  p.row_sums = reinterpret_cast<float2*>(static_cast<float*>(workspace) + static_cast<size_t>(kMaxParts) * 2 * K);
  const bool vec = K % 8 == 0, saved = x == nullptr;
  int nparts = 0;
  cudaError_t e = cudaSuccess;
  if (M > 0) {
    auto go = [&](auto t) {
      using T = decltype(t);
      if (vec) return saved ? backward<T, true, true>(p, &nparts, s) : backward<T, true, false>(p, &nparts, s);
      return saved ? backward<T, false, true>(p, &nparts, s) : backward<T, false, false>(p, &nparts, s);
    };
    e = f32 ? go(float{}) : go(__nv_bfloat16{});
  }
  if (e != cudaSuccess || !sums) return e;
  return launch_pdl(norm_join_kernel, dim3(static_cast<unsigned>((K + 31) / 32)), dim3(1024), 0, s,
                    static_cast<const float*>(workspace), nparts, static_cast<int>(K), dweight, dbias, p_f32, accumulate);
}

}  // namespace bl
