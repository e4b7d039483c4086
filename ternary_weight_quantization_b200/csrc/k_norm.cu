// Layer norm and RMS norm, forward and backward (N1, N2).
//
//   forward   mean, then sum (x - mean)^2 from the values in registers (two
//             reductions: no cancellation), y = (x - mean) rstd w + b, and the
//             8-bit form of x in the same pass
//   backward  g = dy w, xhat = (x - mean) rstd
//             dx = rstd (g - mean(g) - xhat mean(g xhat))
//             dweight = sum over rows of dy xhat, dbias = sum over rows of dy
//
// Both are bound by HBM. Forward: a group of kTpr threads holds one row in
// registers. Backward: a group of threads covers one row with 8 columns per
// thread, so that each thread also keeps its columns' sums of dweight and
// dbias in registers over all rows of its group; one block per SM, whose
// groups join their sums in shared memory and write one partial row each to
// the workspace (148 x 2 x K floats at most), which a second launch adds in a
// fixed order. Rows wider than 8192 columns take two passes: the row sums,
// then column strips.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "bl_act8.cuh"
#include "bl_device.cuh"
#include "bl_internal.h"

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
  float k;  // K
  void* y;
  float* mean;
  float* rstd;
  int8_t* codes;
  float* scales;
};

// 8 consecutive parameters (vector) from column c, or the one at c.
__device__ __forceinline__ void load_params8(const void* p, int f32, int c, float (&v)[8]) {
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
  for (int w = 0; w < (tpr >> 5); ++w) {
#pragma unroll
    for (int i = 0; i < kN; ++i) v[i] += buf[w * kN + i];
  }
}

// ---------------------------------------------------------------- forward
// Column of value i (0..7) of the thread's vector v: vector layout, 8
// consecutive columns; scalar layout, one column every tpr.
template <bool kVec>
__device__ __forceinline__ int column(int v, int i, int t, int tpr) {
  return kVec ? (v * tpr + t) * 8 + i : t + (v * 8 + i) * tpr;
}

template <typename T, int kVecs, bool kVec, bool kRms, bool kSave>
__global__ void __launch_bounds__(1024) norm_forward_kernel(const NormArgs p) {
  pdl_wait_primary();
  pdl_launch_dependents();
  __shared__ float sums[2][32];
  const int tpr = p.tpr;
  const int grp = threadIdx.x / tpr, t = threadIdx.x % tpr;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (blockDim.x / tpr) + grp;
  if (row >= p.M) return;  // whole groups leave
  const int K = p.K;
  const T* x = static_cast<const T*>(p.x) + row * K;
  const int warp0 = grp * (tpr >> 5);
  float v[kVecs][8];
#pragma unroll
  for (int j = 0; j < kVecs; ++j) {
    if constexpr (kVec) {
      Raw8<T> r;
      const int c = column<true>(j, 0, t, tpr);
      if (c < K) r.load(x + c);
      else r.clear();
      r.get(v[j]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int c = column<false>(j, i, t, tpr);
        v[j][i] = c < K ? to_f32(x[c]) : 0.0f;
      }
    }
  }
  if constexpr (kSave) {
    // the 16 lanes of half a warp hold a group's 128 columns
    static_assert(kVec, "the 8-bit form is written from the vector layout");
    const int groups = (K + kAct8Group - 1) / kAct8Group;
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      const int c = column<true>(j, 0, t, tpr);
      const Act8Scale s = act8_scale(act8_absmax_bits<true>(v[j]));
      if (c < K) {
        *reinterpret_cast<uint2*>(p.codes + row * K + c) = act8_codes8(v[j], s.inv);
        if ((t & 15) == 0) p.scales[row * groups + c / kAct8Group] = s.scale;
      }
    }
  }
  float mean = 0.0f;
  if constexpr (!kRms) {
    float s[1] = {0.0f};
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
#pragma unroll
      for (int i = 0; i < 8; ++i) s[0] += v[j][i];
    }
    group_sum(s, sums[0] + warp0, t, tpr, 1 + grp);
    mean = __fdiv_rn(s[0], p.k);
  }
  float q[1] = {0.0f};
#pragma unroll
  for (int j = 0; j < kVecs; ++j) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[j][i] -= mean;
      q[0] += column<kVec>(j, i, t, tpr) < K ? v[j][i] * v[j][i] : 0.0f;
    }
  }
  group_sum(q, sums[1] + warp0, t, tpr, 1 + grp);
  const float rstd = __fdiv_rn(1.0f, __fsqrt_rn(__fdiv_rn(q[0], p.k) + p.eps));
  if (t == 0) {
    if constexpr (!kRms) p.mean[row] = mean;
    p.rstd[row] = rstd;
  }
  T* y = static_cast<T*>(p.y) + row * K;
#pragma unroll
  for (int j = 0; j < kVecs; ++j) {
    if constexpr (kVec) {
      const int c = column<true>(j, 0, t, tpr);
      if (c >= K) break;
      float w[8], o[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = v[j][i] * rstd;
      if (p.weight) {
        load_params8(p.weight, p.p_f32, c, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] *= w[i];
      }
      if (p.bias) {
        load_params8(p.bias, p.p_f32, c, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] += w[i];
      }
      store8(y + c, o);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int c = column<false>(j, i, t, tpr);
        if (c < K) {
          float o = v[j][i] * rstd;
          if (p.weight) o *= load_param(p.weight, p.p_f32, c);
          if (p.bias) o += load_param(p.bias, p.p_f32, c);
          store1(y + c, o);
        }
      }
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
      mean = __fdiv_rn(s[0], p.k);
    }
    float q[1] = {0.0f};
    for (int c = t; c < K; c += 1024) {
      const float d = to_f32(x[c]) - mean;
      q[0] += d * d;
    }
    group_sum(q, sums[1], t, 1024, 1);
    const float rstd = __fdiv_rn(1.0f, __fsqrt_rn(__fdiv_rn(q[0], p.k) + p.eps));
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
  __device__ __forceinline__ void get(float (&dv)[8], float (&xv)[8]) const {
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
  __device__ __forceinline__ void get(float (&dv)[8], float (&xv)[8]) const {
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
  __device__ __forceinline__ void get(float (&dv)[8], float (&xv)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) dv[i] = d[i], xv[i] = x[i];
  }
};

// Weights of the thread's 8 columns (zero outside the row).
template <bool kVec>
__device__ __forceinline__ void load_weights(const NormBwdArgs& p, int c0, int tpr, float (&w)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int c = kVec ? c0 + i : c0 + i * tpr;
    w[i] = c >= p.K ? 0.0f : p.weight ? load_param(p.weight, p.p_f32, c) : 1.0f;
  }
}

template <typename T, bool kVec>
__device__ __forceinline__ void store_row(T* dx, int K, int c0, int tpr, const float (&o)[8]) {
  if constexpr (kVec) {
    if (c0 < K) store8(dx + c0, o);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c0 + i * tpr < K) store1(dx + c0 + i * tpr, o[i]);
  }
}

// kRows rows of a group at a time.
template <typename T, bool kVec, bool kSaved, int kRows>
__global__ void __launch_bounds__(1024, 1) norm_backward_kernel(const NormBwdArgs p) {
  pdl_wait_primary();
  pdl_launch_dependents();
  extern __shared__ float joint[];  // [groups][2][8 tpr] after the rows
  __shared__ float sums[2][32 * 2 * kRows];
  const int tpr = p.tpr, K = p.K;
  const int ngrp = blockDim.x / tpr;
  const int grp = threadIdx.x / tpr, t = threadIdx.x % tpr;
  const int c0 = kVec ? t * 8 : t;
  float w[8], dw[8], db[8];
  load_weights<kVec>(p, c0, tpr, w);
#pragma unroll
  for (int i = 0; i < 8; ++i) dw[i] = db[i] = 0.0f;
  float* my_sums[2] = {sums[0] + grp * (tpr >> 5) * 2 * kRows, sums[1] + grp * (tpr >> 5) * 2 * kRows};
  int par = 0;
  const int64_t step = static_cast<int64_t>(gridDim.x) * ngrp * kRows;
  for (int64_t row = (static_cast<int64_t>(blockIdx.x) * ngrp + grp) * kRows; row < p.M; row += step) {
    RowIn<T, kVec, kSaved> in[kRows];
    float mean[kRows], rstd[kRows], s[2 * kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const int64_t m = row + r < p.M ? row + r : row;
      in[r].load(p, m, t, tpr, c0);
      mean[r] = p.rms ? 0.0f : __ldg(p.mean + m);
      rstd[r] = __ldg(p.rstd + m);
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      float d[8], x[8];
      in[r].get(d, x);
      const bool live = row + r < p.M;
      s[2 * r] = s[2 * r + 1] = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float xh = (x[i] - mean[r]) * rstd[r];
        const float g = d[i] * w[i];
        s[2 * r] += g;
        s[2 * r + 1] = fmaf(g, xh, s[2 * r + 1]);
        if (live) {
          dw[i] = fmaf(d[i], xh, dw[i]);
          db[i] += d[i];
        }
      }
    }
    if (p.dx) {
      group_sum(s, my_sums[par], t, tpr, 1 + grp);
      par ^= 1;
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        if (row + r >= p.M) break;
        const float c1 = p.rms ? 0.0f : s[2 * r] * p.inv_k, c2 = s[2 * r + 1] * p.inv_k;
        float d[8], x[8], o[8];
        in[r].get(d, x);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float xh = (x[i] - mean[r]) * rstd[r];
          o[i] = rstd[r] * (fmaf(d[i], w[i], -c1) - xh * c2);
        }
        store_row<T, kVec>(static_cast<T*>(p.dx) + (row + r) * K, K, c0, tpr, o);
      }
    }
  }
  if (!p.parts) return;
  // columns outside the row are never read back from the joint sums
  float* mine = joint + static_cast<int64_t>(grp) * 16 * tpr;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int c = kVec ? c0 + i : c0 + i * tpr;
    mine[c] = dw[i];
    mine[8 * tpr + c] = db[i];
  }
  __syncthreads();
  float* part = p.parts + static_cast<int64_t>(blockIdx.x) * 2 * K;
  for (int c = threadIdx.x; c < K; c += blockDim.x) {
    float a = 0.0f, b = 0.0f;
    for (int g = 0; g < ngrp; ++g) {
      a += joint[static_cast<int64_t>(g) * 16 * tpr + c];
      b += joint[static_cast<int64_t>(g) * 16 * tpr + 8 * tpr + c];
    }
    part[c] = a;
    part[K + c] = b;
  }
}

// Wide rows, first pass: the two sums of each row.
template <typename T, bool kSaved>
__global__ void __launch_bounds__(1024) norm_row_sums_kernel(const NormBwdArgs p) {
  pdl_wait_primary();
  pdl_launch_dependents();
  __shared__ float sums[32 * 2];
  const int t = threadIdx.x, K = p.K;
  for (int64_t row = blockIdx.x; row < p.M; row += gridDim.x) {
    const float mean = p.rms ? 0.0f : __ldg(p.mean + row), rstd = __ldg(p.rstd + row);
    float s[2] = {0.0f, 0.0f};
    for (int c0 = t; c0 < K; c0 += 8 * 1024) {
      RowIn<T, false, kSaved> in;
      in.load(p, row, t, 1024, c0);
      float w[8];
      load_weights<false>(p, c0, 1024, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float g = in.d[i] * w[i];
        s[0] += g;
        s[1] = fmaf(g, (in.x[i] - mean) * rstd, s[1]);
      }
    }
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
  float w[8], dw[8], db[8];
  load_weights<kVec>(p, c0, 256, w);
#pragma unroll
  for (int i = 0; i < 8; ++i) dw[i] = db[i] = 0.0f;
  for (int64_t row = blockIdx.y; row < p.M; row += gridDim.y) {
    RowIn<T, kVec, kSaved> in;
    in.load(p, row, t, 256, c0);
    const float mean = p.rms ? 0.0f : __ldg(p.mean + row), rstd = __ldg(p.rstd + row);
    const float2 c = p.dx ? p.row_sums[row] : make_float2(0.0f, 0.0f);
    float d[8], x[8], o[8];
    in.get(d, x);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float xh = (x[i] - mean) * rstd;
      o[i] = rstd * (fmaf(d[i], w[i], -c.x) - xh * c.y);
      dw[i] = fmaf(d[i], xh, dw[i]);
      db[i] += d[i];
    }
    if (p.dx) store_row<T, kVec>(static_cast<T*>(p.dx) + row * K, K, c0, 256, o);
  }
  if (!p.parts) return;
  float* part = p.parts + static_cast<int64_t>(blockIdx.y) * 2 * K;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int c = kVec ? c0 + i : c0 + i * 256;
    if (c < K) {
      part[c] = dw[i];
      part[K + c] = db[i];
    }
  }
}

// dweight, dbias from the blocks' partial rows: 32 columns per block, the
// partial rows spread over 16 threads of each column.
__global__ void __launch_bounds__(512) norm_join_kernel(const float* __restrict__ parts, int nparts, int K,
                                                        void* dweight, void* dbias, int p_f32, int accumulate) {
  pdl_wait_primary();
  pdl_launch_dependents();
  __shared__ float sh[2][16][33];
  const int x = threadIdx.x & 31, yy = threadIdx.x >> 5;
  const int c = static_cast<int>(blockIdx.x) * 32 + x;
  float a = 0.0f, b = 0.0f;
  if (c < K) {
#pragma unroll 4
    for (int r = yy; r < nparts; r += 16) {
      a += parts[static_cast<int64_t>(r) * 2 * K + c];
      b += parts[static_cast<int64_t>(r) * 2 * K + K + c];
    }
  }
  sh[0][yy][x] = a;
  sh[1][yy][x] = b;
  __syncthreads();
  if (yy < 2 && c < K) {
    void* out = yy == 0 ? dweight : dbias;
    if (!out) return;
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) s += sh[yy][i][x];
    if (p_f32) {
      float* o = static_cast<float*>(out) + c;
      *o = accumulate ? s + *o : s;
    } else {
      __nv_bfloat16* o = static_cast<__nv_bfloat16*>(out) + c;
      *o = __float2bfloat16_rn(accumulate ? s + __bfloat162float(*o) : s);
    }
  }
}

// ---------------------------------------------------------------- host side
constexpr int kFwdMaxK = 32768;  // 1024 threads x 4 vectors of 8
constexpr int kBwdMaxK = 8192;   // 1024 threads x 8 columns
constexpr int kMaxParts = 148;   // partial rows of dweight and dbias

template <typename T, bool kRms>
cudaError_t forward_rows(NormArgs p, bool vec, bool save, cudaStream_t s) {
  // threads per row: the fewest that hold the row with 4 vectors each (2 below
  // 512 columns)
  int tpr = 32;
  while (tpr * 32 < p.K) tpr *= 2;
  const int vecs = tpr * 16 >= p.K ? 2 : 4;
  p.tpr = tpr;
  const int block = tpr < 256 ? 256 : tpr;
  const int per = block / tpr;
  const dim3 grid(static_cast<unsigned>((p.M + per - 1) / per));
  auto go = [&](auto kernel) { return launch_pdl(kernel, grid, dim3(block), 0, s, p); };
  if (vec && save)
    return vecs == 2 ? go(norm_forward_kernel<T, 2, true, kRms, true>) : go(norm_forward_kernel<T, 4, true, kRms, true>);
  if (vec)
    return vecs == 2 ? go(norm_forward_kernel<T, 2, true, kRms, false>)
                     : go(norm_forward_kernel<T, 4, true, kRms, false>);
  return vecs == 2 ? go(norm_forward_kernel<T, 2, false, kRms, false>)
                   : go(norm_forward_kernel<T, 4, false, kRms, false>);
}

template <typename T>
cudaError_t forward(const NormArgs& p, int rms, cudaStream_t s) {
  const bool vec = p.K % 8 == 0, narrow = p.K <= kFwdMaxK;
  const bool fused = vec && narrow && p.codes;
  cudaError_t e;
  if (!narrow) {
    const unsigned grid = static_cast<unsigned>(p.M < (1 << 20) ? p.M : (1 << 20));
    e = launch_pdl(norm_forward_wide_kernel<T>, dim3(grid), dim3(1024), 0, s, p, rms);
  } else {
    e = rms ? forward_rows<T, true>(p, vec, fused, s) : forward_rows<T, false>(p, vec, fused, s);
  }
  if (e != cudaSuccess || !p.codes || fused) return e;
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
  constexpr int kRows = sizeof(T) == 2 ? 2 : 1;
  auto kernel = norm_backward_kernel<T, kVec, kSaved, kRows>;
  constexpr int kJoint = 1024 * 16 * 4;
  static int configured[64] = {};  // attribute set once per process per device
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !configured[dev]) {
    if (cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kJoint);
        e != cudaSuccess)
      return e;
    if (dev >= 0 && dev < 64) configured[dev] = 1;
  }
  const int tpr = ((p.K + 7) / 8 + 31) / 32 * 32;
  // named barriers 1..15 serve the groups (a row of 32 threads needs none)
  int groups = 1024 / tpr;
  if (tpr > 32 && groups > 15) groups = 15;
  const int64_t want = (p.M + static_cast<int64_t>(groups) * kRows - 1) / (static_cast<int64_t>(groups) * kRows);
  const int grid = static_cast<int>(want < kMaxParts ? want : kMaxParts);
  p.tpr = tpr;
  *nparts = grid;
  return launch_pdl(kernel, dim3(grid), dim3(groups * tpr), static_cast<size_t>(groups) * tpr * 16 * 4, s, p);
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
  return launch_pdl(norm_join_kernel, dim3(static_cast<unsigned>((K + 31) / 32)), dim3(512), 0, s,
                    static_cast<const float*>(workspace), nparts, static_cast<int>(K), dweight, dbias, p_f32, accumulate);
}

}  // namespace bl
