// RMS norm of a residual stream, with the projection's output added on the way
// in and the result left in INT8 with one scale per token (Q1), and its
// gradients (Q2).
//
//   forward   r = rn(x + residual)          kept in the stream's type
//             rstd = 1 / sqrt(mean(r^2) + eps)
//             t = r w, a = max(max |t| rstd, 1e-5)
//             xq = rint(t (127 / max |t|))    (t rstd 127 / 1e-5 where a is that)
//             sx = a / 127
//   backward  n = r rstd, g = dy w          (the quantiser's Jacobian is 1)
//             d = dsum + rstd (g - n mean(g n))
//             dresidual, dx = d, dweight = sum over rows of dy n
//
// Both sums of a row (of r^2, and the largest |t|) come from one pass: t is the
// normed value up to the factor rstd, which is not known yet, so its codes need
// no second pass and a row costs one barrier. y = r rstd w itself is never
// rounded to a type of its own.
//
// Bound by HBM (a row moves 2 to 4 times its own bytes), like the norms without
// the 8-bit result (k_norm.cu), whose way of walking rows this is: a group of
// threads takes rows in turn, each thread copies its own columns of the next
// rows asynchronously into its own places of shared memory (bytes in flight
// without registers or barriers). Forward: several blocks per SM, a block (or,
// for narrow rows, a warp) per row. Backward: one block per SM, columns' sums of
// dweight in registers over all of its rows, joined per block and then by a
// second launch in a fixed order.
//
// Measured on B200 (in a graph, inputs from HBM), with the share of the copy rate:
// bf16, 4096 x 2560: forward 13.8 us (0.81), backward 18.9 (0.68, of which some 6 are
// its start, the blocks' joins and the second launch); 16384 x 2560: 53.0 (0.85) and
// 53.3 (0.96). bf16 onto an fp32 stream, 4096 x 2560: 21.1 (0.83) and 31.3 (0.82). One
// token: 2.0 and 5.3 (launches). The forward issues 0.53 instructions a cycle and
// scheduler (ncu): next to HBM that is what it is short of.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "bl_act8.cuh"
#include "bl_device.cuh"
#include "bl_internal.h"
#include "bl_rows.cuh"

namespace bl {
namespace {

constexpr float kQuantFloor = 1e-5f;  // least absmax, as of S2

struct FwdArgs {
  const void* x;
  const void* residual;  // or null: x is the stream
  const void* weight;
  int p_f32;
  int64_t M;
  int K;
  float eps, inv_k;
  void* sum;
  float* rstd;
  int8_t* xq;
  float* sx;
};

// The larger of m and the absolute values of v; a NaN if there is one.
__device__ __forceinline__ float top_of(const f32x2 (&v)[4], float m) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float lo, hi;
    split2(v[i], lo, hi);
    asm("max.NaN.f32 %0, %0, %1, %2;" : "+f"(m) : "f"(fabsf(lo)), "f"(fabsf(hi)));
  }
  return m;
}

// The sum of 8 values of x and of the residual, rounded to the stream's type and
// stored. (Two bf16 numbers add exactly in fp32, or so far apart that the smaller
// one is lost in bf16 all the same: the packed bf16 addition, rounded once, gives
// what an fp32 addition and a rounding would.)
__device__ __forceinline__ uint32_t add_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ void add_keep(const Raw8<__nv_bfloat16>& x, const Raw8<__nv_bfloat16>& r, __nv_bfloat16* to,
                                         f32x2 (&v)[4]) {
  Raw8<__nv_bfloat16> o;
  o.a = make_uint4(add_bf16x2(x.a.x, r.a.x), add_bf16x2(x.a.y, r.a.y), add_bf16x2(x.a.z, r.a.z), add_bf16x2(x.a.w, r.a.w));
  *reinterpret_cast<uint4*>(to) = o.a;
  o.get(v);
}
template <typename TX>
__device__ __forceinline__ void add_keep(const Raw8<TX>& x, const Raw8<float>& r, float* to, f32x2 (&v)[4]) {
  f32x2 o[4];
  x.get(v);
  r.get(o);
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = add2(v[i], o[i]);
  store8(to, v);
}

constexpr int kFwdThreads = 512;  // most threads of a forward block
template <typename TX, typename TS>
constexpr int kFwdPieces = (sizeof(TX) + sizeof(TS)) / 2;  // 16-byte pieces of 8 columns
template <typename TX, typename TS>
constexpr int kFwdDepth = kFwdPieces<TX, TS> == 2 ? 3 : 2;  // rows in flight per group

// kFull: the row fills every thread's vectors. kWarp: a warp per row.
template <typename TX, typename TS, int kVecs, bool kFull, bool kWarp>
__global__ void __launch_bounds__(kFwdThreads, kVecs <= 2 ? 2 : 1) norm_quant_forward_kernel(const FwdArgs p) {
  pdl_wait_primary();
  pdl_launch_dependents();
  extern __shared__ uint4 ring[];
  __shared__ float4 sums[2][kFwdThreads / 64];  // (sum, maximum) of two warps each, two rows in turn
  constexpr int kPx = sizeof(TX) / 2, kPieces = kFwdPieces<TX, TS>, kDepth = kFwdDepth<TX, TS>;
  const int K = p.K, tpr = kWarp ? 32 : blockDim.x;
  const int t = kWarp ? threadIdx.x & 31 : threadIdx.x;
  const uint32_t stride = blockDim.x * 16, row_stride = kVecs * kPieces * stride;
  const uint32_t mine = smem_u32(ring) + threadIdx.x * 16, end = mine + kDepth * row_stride;
  const int c0 = t * 8, cs = tpr * 8;  // the thread's vectors: columns c0 + j cs
  auto live = [&](int j) { return kFull || c0 + j * cs < K; };
  if constexpr (!kWarp) {
    if (threadIdx.x < 2 * (kFwdThreads / 64)) sums[0][threadIdx.x] = make_float4(0.f, 0.f, 0.f, 0.f);
    __syncthreads();
  }
  const int64_t first = kWarp ? static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5) : blockIdx.x;
  const int64_t step = kWarp ? static_cast<int64_t>(gridDim.x) * (blockDim.x >> 5) : gridDim.x, step_k = step * K;
  int rows = first < p.M ? static_cast<int>((p.M - 1 - first) / step) + 1 : 0, left = rows;
  int64_t row = first, at = row * K + c0;  // the thread's place in this row
  const bool added = p.residual != nullptr;
  const TX* next_x = static_cast<const TX*>(p.x) + at;  // and in the row to load next
  const TS* next_r = static_cast<const TS*>(p.residual) + (added ? at : 0);
  auto issue = [&](uint32_t slot) {
    if (left > 0) {
#pragma unroll
      for (int j = 0; j < kVecs; ++j) {
        if (!live(j)) continue;
        const uint32_t to = slot + j * kPieces * stride;
        issue8(to, stride, next_x + j * cs);
        if (added) issue8(to + kPx * stride, stride, next_r + j * cs);
      }
      next_x += step_k;
      if (added) next_r += step_k;
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
  int par = 0;
  for (uint32_t slot = mine; rows > 0; --rows, row += step, at += step_k) {
    copy_async_wait<kDepth - 1>();
    f32x2 v[kVecs][4], q2 = 0;  // t, and the sum of r^2
    float most = 0.0f;
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      if (!live(j)) continue;
      const uint32_t from = slot + j * kPieces * stride;
      Raw8<TX> rx;
      read_raw(from, stride, rx);
      if (added) {
        Raw8<TS> rs;
        read_raw(from + kPx * stride, stride, rs);
        add_keep(rx, rs, static_cast<TS*>(p.sum) + at + j * cs, v[j]);
      } else {
        rx.get(v[j]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        q2 = fma2(v[j][i], v[j][i], q2);
        v[j][i] = mul2(v[j][i], w[j][i]);
      }
      most = top_of(v[j], most);
    }
    issue(slot);
    slot += row_stride;
    if (slot == end) slot = mine;
    float q = warp_sum(sum2(q2));
    // (as integers the bits of values from 0 on have the values' order, NaN last)
    uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(most));
    if constexpr (!kWarp) {
      // the buffers alternate, so one barrier per row is enough: a warp writes
      // one again only after a barrier that every reader of it has reached
      if ((t & 31) == 0) reinterpret_cast<float2*>(sums[par])[t >> 5] = make_float2(q, __uint_as_float(top));
      __syncthreads();
      q = 0.0f;
      const int n = (tpr + 63) >> 6;
#pragma unroll 4
      for (int i = 0; i < n; ++i) {
        const float4 two = sums[par][i];
        q += two.x + two.z;
        top = max(top, max(__float_as_uint(two.y), __float_as_uint(two.w)));
      }
      par ^= 1;
    }
    // a sum beyond fp32 (or a NaN) leaves NaN, not a row of zeros
    const float rstd = q < __uint_as_float(0x7F800000u) ? rsqrt_of(fmaf(q, p.inv_k, p.eps)) : __uint_as_float(0x7FC00000u);
    const float most_t = __uint_as_float(top), a = max_nan(__fmul_rn(most_t, rstd), kQuantFloor);
    // 127 / a of y is 127 / max |t| of t, but where a is the floor: the reciprocal's
    // approximation (an fp32 step off) and one product
    float f;
    asm("rcp.approx.f32 %0, %1;" : "=f"(f) : "f"(most_t));
    f = a > kQuantFloor ? f * 127.0f : rstd * (127.0f / kQuantFloor);
    if (t == 0) {
      p.rstd[row] = rstd;
      p.sx[row] = __fdiv_rn(a, 127.0f);
    }
    // f is a few fp32 steps from 127 / max |t| at most, so |t f| ends below 127.5
#pragma unroll
    for (int j = 0; j < kVecs; ++j)
      if (live(j)) *reinterpret_cast<uint2*>(p.xq + at + j * cs) = act8_codes8(v[j], f);
  }
}

// ---------------------------------------------------------------- backward
struct BwdArgs {
  const void* dy;
  const void* dsum;  // or null
  const void* sum;
  const void* weight;
  int p_f32;
  const float* rstd;
  int64_t M;
  int K;
  int tpr;
  float inv_k;
  void* dresidual;  // or null
  void* dx;         // or null
  float* parts;     // [blocks][K], or null
};

constexpr int kBwdThreads = 512;  // of a block, one block per SM
constexpr int kBwdVecs = 2;       // vectors of 8 columns per thread
template <typename TD, typename TS>
constexpr int kBwdPieces = (sizeof(TD) + 2 * sizeof(TS)) / 2;
// Rows in flight: 512 threads x 2 vectors x depth x pieces x 16 bytes = 192 KB
// at most.
template <typename TD, typename TS>
constexpr int kBwdDepth = kBwdPieces<TD, TS> <= 4 ? 12 / kBwdPieces<TD, TS> : 2;

template <typename TD, typename TS, typename TX, bool kFull>
__global__ void __launch_bounds__(kBwdThreads, 1) norm_quant_backward_kernel(const BwdArgs p) {
  pdl_wait_primary();
  pdl_launch_dependents();
  extern __shared__ uint4 ring[];  // the rows in flight; afterwards the groups' sums
  __shared__ float sums[2][kBwdThreads / 32];
  constexpr int kPd = sizeof(TD) / 2, kPs = sizeof(TS) / 2, kPieces = kBwdPieces<TD, TS>, kDepth = kBwdDepth<TD, TS>;
  const int tpr = p.tpr, K = p.K, ngrp = blockDim.x / tpr;
  const int grp = threadIdx.x / tpr, t = threadIdx.x % tpr;
  const int c0 = t * 8, cs = tpr * 8;
  auto live = [&](int j) { return kFull || c0 + j * cs < K; };
  const uint32_t stride = blockDim.x * 16, row_stride = kBwdVecs * kPieces * stride;
  const uint32_t mine = smem_u32(ring) + threadIdx.x * 16, end = mine + kDepth * row_stride;
  // neighbouring rows to neighbouring blocks, so that the blocks' rows differ by one
  const int64_t first = static_cast<int64_t>(grp) * gridDim.x + blockIdx.x;
  const int64_t step = static_cast<int64_t>(gridDim.x) * ngrp, step_k = step * K;
  int rows = first < p.M ? static_cast<int>((p.M - 1 - first) / step) + 1 : 0, left = rows;
  int64_t at = first * K + c0, next = at;  // the thread's place in this row, and in the row to load next
  auto issue = [&](uint32_t slot) {
    if (left > 0) {
#pragma unroll
      for (int j = 0; j < kBwdVecs; ++j) {
        if (!live(j)) continue;
        const uint32_t to = slot + j * kPieces * stride;
        issue8(to, stride, static_cast<const TD*>(p.dy) + next + j * cs);
        issue8(to + kPd * stride, stride, static_cast<const TS*>(p.sum) + next + j * cs);
        if (p.dsum) issue8(to + (kPd + kPs) * stride, stride, static_cast<const TS*>(p.dsum) + next + j * cs);
      }
      next += step_k;
      --left;
    }
    copy_async_commit();
  };
#pragma unroll
  for (int s = 0; s < kDepth; ++s) issue(mine + s * row_stride);
  const float* rstd_at = p.rstd + first;
  float rstd = rows > 0 ? __ldg(rstd_at) : 0.0f;
  f32x2 w[kBwdVecs][4], dw[kBwdVecs][4];
#pragma unroll
  for (int j = 0; j < kBwdVecs; ++j) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w[j][i] = both2(1.0f);
      dw[j][i] = 0;
    }
    if (p.weight && live(j)) load_params8(p.weight, p.p_f32, c0 + j * cs, w[j]);
  }
  const bool rows_out = p.dresidual || p.dx;
  int par = 0;
  for (uint32_t slot = mine; rows > 0; --rows, at += step_k) {
    const f32x2 rstd2 = both2(rstd);
    if (rows > 1) rstd = __ldg(rstd_at += step);
    copy_async_wait<kDepth - 1>();
    f32x2 g[kBwdVecs][4], n[kBwdVecs][4], s2 = 0;
    Raw8<TS> ds[kBwdVecs];
#pragma unroll
    for (int j = 0; j < kBwdVecs; ++j) {
      if (!live(j)) continue;
      const uint32_t from = slot + j * kPieces * stride;
      Raw8<TD> rd;
      Raw8<TS> rs;
      read_raw(from, stride, rd);
      read_raw(from + kPd * stride, stride, rs);
      ds[j].clear();
      if (p.dsum) read_raw(from + (kPd + kPs) * stride, stride, ds[j]);
      rd.get(g[j]);
      rs.get(n[j]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        n[j][i] = mul2(n[j][i], rstd2);
        dw[j][i] = fma2(g[j][i], n[j][i], dw[j][i]);
        g[j][i] = mul2(g[j][i], w[j][i]);
        s2 = fma2(g[j][i], n[j][i], s2);
      }
    }
    issue(slot);
    slot += row_stride;
    if (slot == end) slot = mine;
    if (rows_out) {
      float s[1] = {sum2(s2)};
      group_sum(s, sums[par] + grp * (tpr >> 5), t, tpr, 1 + grp);
      par ^= 1;
      const f32x2 nc = both2(-s[0] * p.inv_k);
#pragma unroll
      for (int j = 0; j < kBwdVecs; ++j) {
        if (!live(j)) continue;
        f32x2 o[4];
        ds[j].get(o);
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = fma2(rstd2, fma2(n[j][i], nc, g[j][i]), o[i]);
        if (p.dresidual) store8(static_cast<TS*>(p.dresidual) + at + j * cs, o);
        if (p.dx) store8(static_cast<TX*>(p.dx) + at + j * cs, o);
      }
    }
  }
  if (!p.parts) return;
  copy_async_wait<0>();
  __syncthreads();  // the ring becomes the groups' sums
  float* joint = reinterpret_cast<float*>(ring);
  const int width = kBwdVecs * 8 * tpr;
#pragma unroll
  for (int j = 0; j < kBwdVecs; ++j) store8(joint + grp * width + c0 + j * cs, dw[j]);
  __syncthreads();
  float* part = p.parts + static_cast<int64_t>(blockIdx.x) * K;
  for (int c = threadIdx.x; c < K; c += blockDim.x) {
    float a = 0.0f;
    for (int i = 0; i < ngrp; ++i) a += joint[i * width + c];
    part[c] = a;
  }
}

// dweight from the blocks' partial rows: 16 columns per block, the rows (at most
// kPlanSms) spread over 32 threads of each, whose loads are all in flight at once.
// (8 threads of each: 1.3 us more at 2560 columns.)
constexpr int kJoinCols = 16, kJoinSplit = 32;

__global__ void __launch_bounds__(kJoinCols* kJoinSplit)
    norm_quant_join_kernel(const float* __restrict__ parts, int nparts, int K, void* dweight, int p_f32, int accumulate) {
  __shared__ float sums[kJoinSplit][kJoinCols + 1];
  pdl_wait_primary();
  pdl_launch_dependents();
  const int x = threadIdx.x % kJoinCols, y = threadIdx.x / kJoinCols;
  const int c = static_cast<int>(blockIdx.x) * kJoinCols + x;
  constexpr int kMost = (kPlanSms + kJoinSplit - 1) / kJoinSplit;
  float a = 0.0f;
  if (c < K) {
    float v[kMost];
#pragma unroll
    for (int i = 0; i < kMost; ++i) {
      const int r = y + i * kJoinSplit;
      v[i] = r < nparts ? parts[static_cast<int64_t>(r) * K + c] : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < kMost; ++i) a += v[i];
  }
  sums[y][x] = a;
  __syncthreads();
  if (y != 0 || c >= K) return;
#pragma unroll
  for (int i = 1; i < kJoinSplit; ++i) a += sums[i][x];
  if (p_f32) {
    float* o = static_cast<float*>(dweight) + c;
    *o = accumulate ? a + *o : a;
  } else {
    __nv_bfloat16* o = static_cast<__nv_bfloat16*>(dweight) + c;
    *o = __float2bfloat16_rn(accumulate ? a + __bfloat162float(*o) : a);
  }
}

// ---------------------------------------------------------------- host side

template <typename TX, typename TS, int kVecs, bool kFull, bool kWarp>
cudaError_t forward_launch(const FwdArgs& p, int tpr, cudaStream_t s) {
  const int block = kWarp ? 256 : tpr, per = kWarp ? block / 32 : 1;
  constexpr size_t kPerThread = static_cast<size_t>(kFwdDepth<TX, TS>) * kVecs * kFwdPieces<TX, TS> * 16;
  auto kernel = norm_quant_forward_kernel<TX, TS, kVecs, kFull, kWarp>;
  static bool done[64] = {};
  constexpr size_t kMost = kPerThread * (kNormQuantMaxK / (8 * kVecs));  // of the widest rows' blocks (or a warp kernel's 256 threads)
  static_assert(kMost <= 227 * 1024 && kNormQuantMaxK / (8 * kVecs) <= kFwdThreads && kNormQuantMaxK / (8 * kVecs) >= 256, "blocks");
  if (cudaError_t e = allow_smem(kernel, kMost, done); e != cudaSuccess) return e;
  int blocks = (kVecs <= 2 ? 1024 : 512) / block;  // resident on an SM, by registers
  const int by_smem = static_cast<int>(size_t(227 * 1024) / (kPerThread * block + 1280));
  if (blocks > by_smem) blocks = by_smem;
  if (blocks < 1) blocks = 1;
  const int64_t want = (p.M + per - 1) / per, most = static_cast<int64_t>(blocks) * device_sm_count();
  return launch_pdl(kernel, dim3(static_cast<unsigned>(want < most ? want : most)), dim3(block), kPerThread * block, s, p);
}

template <typename TX, typename TS, int kVecs>
cudaError_t forward_vec(const FwdArgs& p, cudaStream_t s) {
  const int tpr = round32((p.K + 8 * kVecs - 1) / (8 * kVecs));
  const bool full = tpr * 8 * kVecs == p.K;
  if (tpr == 32)
    return full ? forward_launch<TX, TS, kVecs, true, true>(p, tpr, s)
                : forward_launch<TX, TS, kVecs, false, true>(p, tpr, s);
  return full ? forward_launch<TX, TS, kVecs, true, false>(p, tpr, s)
              : forward_launch<TX, TS, kVecs, false, false>(p, tpr, s);
}

template <typename TX, typename TS>
cudaError_t forward(const FwdArgs& p, cudaStream_t s) {
  // 32 columns per thread where that leaves at most a tenth of the group's
  // places empty, else 16
  const int k2 = round32((p.K + 15) / 16) * 16, k4 = round32((p.K + 31) / 32) * 32;
  if (10 * (k4 - p.K) <= k4 || k4 <= k2) return forward_vec<TX, TS, 4>(p, s);
  return forward_vec<TX, TS, 2>(p, s);
}

template <typename TD, typename TS, typename TX>
cudaError_t backward(BwdArgs p, int* nparts, cudaStream_t s) {
  constexpr int kCols = 8 * kBwdVecs;
  const int tpr = round32((p.K + kCols - 1) / kCols);
  int groups = kBwdThreads / tpr;
  if (tpr > 32 && groups > 15) groups = 15;  // named barriers 1..15 (a row of 32 threads needs none)
  // few rows: smaller blocks on more SMs (the rule of the norms without the
  // 8-bit result)
  const int64_t spread = (p.M + kPlanSms - 1) / kPlanSms, least = 128 / tpr > 1 ? 128 / tpr : 1;
  if (const int64_t few = spread > least ? spread : least; 2 * few <= groups) groups = static_cast<int>(few);
  const int block = groups * tpr;
  const int64_t want = (p.M + groups - 1) / groups;
  const int grid = static_cast<int>(want < kPlanSms ? want : kPlanSms);
  p.tpr = tpr;
  *nparts = grid;
  // per thread: the rows in flight, and afterwards one float per column
  constexpr size_t kRing = static_cast<size_t>(16) * kBwdPieces<TD, TS> * kBwdVecs * kBwdDepth<TD, TS>;
  static_assert(kRing >= kCols * 4 && kRing * kBwdThreads <= 196608, "shared memory");
  auto go = [&](auto kernel, bool (&done)[64]) {
    if (cudaError_t e = allow_smem(kernel, kBwdThreads * kRing, done); e != cudaSuccess) return e;
    return launch_pdl(kernel, dim3(grid), dim3(block), block * kRing, s, p);
  };
  static bool done[2][64] = {};
  return tpr * kCols == p.K ? go(norm_quant_backward_kernel<TD, TS, TX, true>, done[0])
                            : go(norm_quant_backward_kernel<TD, TS, TX, false>, done[1]);
}

}  // namespace

size_t norm_quant_backward_workspace_bytes(int64_t K) { return static_cast<size_t>(kPlanSms) * static_cast<size_t>(K) * 4; }

cudaError_t launch_norm_quant_forward(const void* x, int x_f32, const void* residual, int s_f32, const void* weight,
                                      int p_f32, int64_t M, int64_t K, float eps, void* sum, float* rstd, int8_t* xq,
                                      float* sx, cudaStream_t s) {
  FwdArgs p{};
  p.x = x;
  p.residual = residual;
  p.weight = weight;
  p.p_f32 = p_f32;
  p.M = M;
  p.K = static_cast<int>(K);
  p.eps = eps;
  p.inv_k = 1.0f / static_cast<float>(K);
  p.sum = sum;
  p.rstd = rstd;
  p.xq = xq;
  p.sx = sx;
  if (x_f32) return forward<float, float>(p, s);
  return s_f32 ? forward<__nv_bfloat16, float>(p, s) : forward<__nv_bfloat16, __nv_bfloat16>(p, s);
}

cudaError_t launch_norm_quant_backward(const void* dy, int dy_f32, const void* dsum, const void* sum, int s_f32,
                                       const void* weight, int p_f32, const float* rstd, int64_t M, int64_t K,
                                       void* dresidual, void* dx, int x_f32, void* dweight, int accumulate,
                                       void* workspace, cudaStream_t s) {
  BwdArgs p{};
  p.dy = dy;
  p.dsum = dsum;
  p.sum = sum;
  p.weight = weight;
  p.p_f32 = p_f32;
  p.rstd = rstd;
  p.M = M;
  p.K = static_cast<int>(K);
  p.inv_k = 1.0f / static_cast<float>(K);
  p.dresidual = dresidual;
  p.dx = dx;
  p.parts = dweight ? static_cast<float*>(workspace) : nullptr;
  int nparts = 0;
  if (M > 0) {
    using B = __nv_bfloat16;
    cudaError_t e;
    if (dy_f32)
      e = x_f32 ? backward<float, float, float>(p, &nparts, s)
                : s_f32 ? backward<float, float, B>(p, &nparts, s) : backward<float, B, B>(p, &nparts, s);
    else
      e = x_f32 ? backward<B, float, float>(p, &nparts, s)
                : s_f32 ? backward<B, float, B>(p, &nparts, s) : backward<B, B, B>(p, &nparts, s);
    if (e != cudaSuccess) return e;
  }
  if (!dweight) return cudaSuccess;
  return launch_pdl(norm_quant_join_kernel, dim3(static_cast<unsigned>((K + kJoinCols - 1) / kJoinCols)),
                    dim3(kJoinCols * kJoinSplit), 0, s, static_cast<const float*>(workspace), nparts, static_cast<int>(K),
                    dweight, p_f32, accumulate);
}

}  // namespace bl
