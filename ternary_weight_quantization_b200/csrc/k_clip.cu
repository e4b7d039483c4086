// The norm over all of a model's gradients, and the gradients scaled down to a
// largest norm (C1, C2).
//
//   norm = sqrt(sum over all tensors of g^2)
//   out  = rn(g * (most / norm)) where norm > most, else g
//
// Two launches over a list of tensors of any sizes and either type: one sums, the
// other adds the blocks' sums (every block for itself, in the same order), and
// scales. Bound by HBM: the first reads every gradient, the second reads it again
// and writes it; a user who only wants the norm pays for the first alone.
//
// The list travels in the launch's parameters (no table in memory, nothing to
// copy, and a captured graph keeps it); longer lists take several launches. The
// tensors are cut into segments of 4 KB, each warp takes an equal run of them (a
// run per block: a block whose run crosses small tensors waits for one after the
// other's loads, 8.7 us for 6.9 over 9 MB in 28 tensors), and the second launch
// walks its runs backwards, from what the first read last and L2 still holds.
//
// Measured on B200 (in a graph, gradients from HBM): 1279 MB of bf16 in 57 tensors:
// norm 215 us (0.91 of the copy rate), clipped copies 655 (0.9 of what the two
// launches move, 0.6 of reading once and writing once: a second reading is the price
// of a norm that has to be known first); 85 MB of fp32 in 39: 17.4 and 40.4; 9 MB in
// 30: 5.7 and 9.4 (two launches of 1.5 to 2 us, one HBM latency each).
//
// Sums: the squares of up to 32 values are added in fp32, such sums in fp64. A
// sum that leaves fp32's range (values around 1e19 and beyond, or so small that
// their squares vanish) is formed again in fp64, so the norm of any finite
// gradients is finite and right.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "bl_act8.cuh"
#include "bl_device.cuh"
#include "bl_internal.h"

namespace bl {
namespace {

constexpr int kThreads = 512;
constexpr int kSegment = 4096;  // bytes
constexpr int kBlocks = 2 * kPlanSms;  // resident at once
constexpr int kWarps = kThreads / 32;
constexpr int kU = 4;           // 16-byte vectors whose squares are added in fp32
constexpr int kGroups = 2;      // such groups in flight per thread where the squares are summed

struct Entry {
  const void* in;
  void* out;
  int64_t n2;  // 2 n + (fp32)
};

template <int kCap>
struct Table {
  Entry e[kCap];
  int first[kCap + 1];  // the tensor's first segment; at `count` the end
  int count;
  uint16_t from[kBlocks + 1];  // tensor that holds the first segment of a block's runs; at `blocks` the last tensor
};

// Elements [b, e) of a tensor that its segments [s, t) cover.
__device__ __forceinline__ void span(int64_t n, int esize, int s, int t, int64_t& b, int64_t& e) {
  const int64_t per = kSegment / esize;
  b = s * per;
  e = t * per < n ? t * per : n;
}

__device__ __forceinline__ double square(float x) { return static_cast<double>(x) * static_cast<double>(x); }

// Sum of squares of the 16-byte vectors v: as fp32, or again in fp64 where that
// left its range.
template <typename T>
__device__ __forceinline__ double squares(const uint4 (&v)[kU]) {
  f32x2 s = 0, s1 = 0;
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const f32x2 a = pair2(bf16_lo(w[i]), bf16_hi(w[i]));
        if (i & 1) s1 = fma2(a, a, s1);
        else s = fma2(a, a, s);
      }
    } else {
      const f32x2 a = pair2(__uint_as_float(w[0]), __uint_as_float(w[1]));
      const f32x2 b = pair2(__uint_as_float(w[2]), __uint_as_float(w[3]));
      s = fma2(a, a, s);
      s1 = fma2(b, b, s1);
    }
  }
  const float f = sum2(add2(s, s1));
  // 2^-80: 46 bits above the smallest normal square, so what vanished below is
  // less than 2^-40 of the sum
  if (f < __uint_as_float(0x7F800000u) && f >= 8.271806e-25f) return static_cast<double>(f);
  double d = 0.0;
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
    if ((w[0] | w[1] | w[2] | w[3]) == 0u) continue;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 2) d += square(bf16_lo(w[i])) + square(bf16_hi(w[i]));
      else d += square(__uint_as_float(w[i]));
    }
  }
  return d;
}

// Elements from `p` to the next 16-byte boundary, at most n.
template <typename T>
__device__ __forceinline__ int64_t to_boundary(const void* p, int64_t n) {
  const int64_t h = ((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / sizeof(T);
  return h < n ? h : n;
}

template <typename T>
__device__ __forceinline__ double sum_range(const T* p, int64_t n) {
  const int t = threadIdx.x & 31;
  const int64_t head = to_boundary<T>(p, n);
  double d = t < head ? square(to_f32(p[t])) : 0.0;
  p += head;
  n -= head;
  constexpr int kPer = 16 / sizeof(T);
  const int64_t vecs = n / kPer;
  const uint4* v = reinterpret_cast<const uint4*>(p);
  for (int64_t i = t; i < vecs; i += kGroups * kU * 32) {
    uint4 r[kGroups][kU];
#pragma unroll
    for (int u = 0; u < kGroups * kU; ++u)
      r[u / kU][u % kU] = i + u * 32 < vecs ? __ldg(v + i + u * 32) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int g = 0; g < kGroups; ++g) d += squares<T>(r[g]);
  }
  const int64_t tail = vecs * kPer + t;
  if (tail < n) d += square(to_f32(p[tail]));
  return d;
}

// Sum over the block, in a fixed order; every thread gets it.
__device__ __forceinline__ double block_sum(double d, double* buf) {
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) d += __shfl_xor_sync(0xffffffffu, d, s);
  if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = d;
  __syncthreads();
  d = buf[threadIdx.x % kWarps];
#pragma unroll
  for (int s = kWarps / 2; s > 0; s >>= 1) d += __shfl_xor_sync(0xffffffffu, d, s);
  return d;
}

// First segment of run i of n equal ones.
__host__ __device__ __forceinline__ int run_start(int segments, int i, int n) {
  return static_cast<int>(static_cast<int64_t>(segments) * i / n);
}

// The warp's run [s, end) of segments, and the tensor that its walk begins with
// (its first segment's, or with kBack its last one's). Read before the wait for
// the launches in front: the parameters' lines take their time to the SM.
struct Run {
  int s, end;
  int i, first, next;
  const void* in;
  void* out;
  int64_t n2;
  template <bool kBack, int kCap>
  __device__ __forceinline__ void begin(const Table<kCap>& t) {
    const int segments = t.first[t.count], n = gridDim.x * kWarps;
    const int w = blockIdx.x * kWarps + __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);  // (known to be the warp's)
    s = run_start(segments, w, n);
    end = run_start(segments, w + 1, n);
    const int at = kBack ? end - 1 : s;
    int lo = t.from[blockIdx.x], hi = t.from[blockIdx.x + 1];  // the last of them with first <= at
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (t.first[mid] <= at) lo = mid;
      else hi = mid - 1;
    }
    move(t, lo);
    asm volatile("" ::"r"(first), "r"(next), "l"(in), "l"(out), "l"(n2));
  }
  template <int kCap>
  __device__ __forceinline__ void move(const Table<kCap>& t, int to) {
    i = to, first = t.first[i], next = t.first[i + 1], in = t.e[i].in, out = t.e[i].out, n2 = t.e[i].n2;
  }
};

template <int kCap>
__global__ void __launch_bounds__(kThreads, 2) grad_sum_kernel(const __grid_constant__ Table<kCap> t, double* parts) {
  __shared__ double buf[kWarps];
  Run x{};
  x.begin<false>(t);
  pdl_wait_primary();
  pdl_launch_dependents();
  double d = 0.0;
  while (x.s < x.end) {
    const int last = x.next < x.end ? x.next : x.end;
    const bool f32 = x.n2 & 1;
    int64_t b, e;
    span(x.n2 >> 1, f32 ? 4 : 2, x.s - x.first, last - x.first, b, e);
    if (f32) d += sum_range(static_cast<const float*>(x.in) + b, e - b);
    else d += sum_range(static_cast<const __nv_bfloat16*>(x.in) + b, e - b);
    x.s = last;
    if (x.s < x.end) x.move(t, x.i + 1);
  }
  d = block_sum(d, buf);
  if (threadIdx.x == 0) parts[blockIdx.x] = d;
}

// The sum of all blocks' sums, in the same order in every block.
__device__ __forceinline__ double total_of(const double* parts, int nparts, double* buf) {
  double d = 0.0;
  for (int i = threadIdx.x; i < nparts; i += kThreads) d += parts[i];
  return block_sum(d, buf);
}

__global__ void __launch_bounds__(kThreads) grad_norm_kernel(const double* parts, int nparts, float* norm) {
  __shared__ double buf[kWarps];
  pdl_wait_primary();
  pdl_launch_dependents();
  const double d = total_of(parts, nparts, buf);
  if (threadIdx.x == 0) *norm = static_cast<float>(sqrt(d));
}

// A gradient's factor, as f * step: step is 1 but where the factor is too small
// for fp32 to hold well; there it is a power of two that f lacks.
struct Scale {
  float f, step;
  __device__ __forceinline__ float operator()(float g) const { return g * f * step; }
};

__device__ __forceinline__ uint4 scaled(const uint4& v, const Scale& k, __nv_bfloat16) {
  return make_uint4(pack_bf16x2(k(bf16_hi(v.x)), k(bf16_lo(v.x))), pack_bf16x2(k(bf16_hi(v.y)), k(bf16_lo(v.y))),
                    pack_bf16x2(k(bf16_hi(v.z)), k(bf16_lo(v.z))), pack_bf16x2(k(bf16_hi(v.w)), k(bf16_lo(v.w))));
}
__device__ __forceinline__ uint4 scaled(const uint4& v, const Scale& k, float) {
  return make_uint4(__float_as_uint(k(__uint_as_float(v.x))), __float_as_uint(k(__uint_as_float(v.y))),
                    __float_as_uint(k(__uint_as_float(v.z))), __float_as_uint(k(__uint_as_float(v.w))));
}

template <typename T>
__device__ __forceinline__ void scale_range(const T* in, T* out, int64_t n, const Scale& k, bool copy) {
  const int t = threadIdx.x & 31;
  auto one = [&](int64_t i) {
    if (copy) out[i] = in[i];
    else store1(out + i, k(to_f32(in[i])));
  };
  if (((reinterpret_cast<uintptr_t>(in) ^ reinterpret_cast<uintptr_t>(out)) & 15) != 0) {
    // the two start at different places of a 16-byte line
#pragma unroll 4
    for (int64_t i = t; i < n; i += 32) one(i);
    return;
  }
  const int64_t head = to_boundary<T>(in, n);
  if (t < head) one(t);
  in += head;
  out += head;
  n -= head;
  constexpr int kPer = 16 / sizeof(T);
  const int64_t vecs = n / kPer;
  const uint4* v = reinterpret_cast<const uint4*>(in);
  uint4* o = reinterpret_cast<uint4*>(out);
  for (int64_t i = t; i < vecs; i += kU * 32) {
    uint4 r[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u)
      if (i + u * 32 < vecs) r[u] = __ldcs(v + i + u * 32);
#pragma unroll
    for (int u = 0; u < kU; ++u)
      if (i + u * 32 < vecs) __stcs(o + i + u * 32, copy ? r[u] : scaled(r[u], k, T{}));
  }
  const int64_t tail = vecs * kPer + t;
  if (tail < n) one(tail);
}

template <int kCap>
__global__ void __launch_bounds__(kThreads, 2) grad_scale_kernel(const __grid_constant__ Table<kCap> t, const double* parts,
                                                                 int nparts, double most, int in_place, float* norm) {
  __shared__ double buf[kWarps];
  Run x{};
  x.begin<true>(t);
  pdl_wait_primary();
  pdl_launch_dependents();
  const double len = sqrt(total_of(parts, nparts, buf));
  if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = static_cast<float>(len);
  // an infinite or NaN norm scales nothing: the caller sees it in `norm`
  const bool clip = len > most && len < __longlong_as_double(0x7FF0000000000000ll);
  if (!clip && in_place) return;
  Scale k;
  const double factor = clip ? most / len : 1.0;
  const bool tiny = factor < 1e-30;
  k.f = static_cast<float>(tiny ? factor * 0x1p96 : factor);
  k.step = tiny ? 0x1p-96f : 1.0f;
  while (x.end > x.s) {
    const int from = x.end - 1;
    const bool f32 = x.n2 & 1;
    int64_t b, e;
    span(x.n2 >> 1, f32 ? 4 : 2, from - x.first, x.end - x.first, b, e);
    if (f32)
      scale_range(static_cast<const float*>(x.in) + b, static_cast<float*>(x.out) + b, e - b, k, !clip);
    else
      scale_range(static_cast<const __nv_bfloat16*>(x.in) + b, static_cast<__nv_bfloat16*>(x.out) + b, e - b, k, !clip);
    x.end = from;
    if (x.end > x.s && x.end == x.first) x.move(t, x.i - 1);
  }
}

// ---------------------------------------------------------------- host side
constexpr int kFew = 64, kMany = 1024;  // tensors per launch (parameters of 2 and 28 KB)

template <int kCap>
int grid_of(const Table<kCap>& t) {
  return t.first[t.count] < kBlocks ? t.first[t.count] : kBlocks;
}

// Fills `t` from the tensors [i, count) that hold something, up to its capacity;
// returns where to go on. (2^40 elements in all, the caller's limit, are 2^30
// segments and one more per tensor.)
template <int kCap>
int64_t fill(Table<kCap>& t, const ClipTensor* x, int64_t i, int64_t count) {
  t.count = 0;
  t.first[0] = 0;
  int64_t segments = 0;
  for (; i < count && t.count < kCap; ++i) {
    if (x[i].n == 0) continue;
    const int64_t per = kSegment / (x[i].f32 ? 4 : 2), more = (x[i].n + per - 1) / per;
    segments += more;
    t.e[t.count] = {x[i].in, x[i].out, 2 * x[i].n + (x[i].f32 ? 1 : 0)};
    t.first[++t.count] = static_cast<int>(segments);
  }
  if (t.count > 0) {
    const int blocks = grid_of(t);
    for (int b = 0, j = 0; b <= blocks; ++b) {
      const int at = run_start(t.first[t.count], b * kWarps, blocks * kWarps);
      while (j + 1 < t.count && t.first[j + 1] <= at) ++j;
      t.from[b] = static_cast<uint16_t>(j);
    }
  }
  return i;
}

template <int kCap>
cudaError_t launch_all(const ClipTensor* x, int64_t count, float* norm, double most, int clip, double* parts,
                       cudaStream_t s) {
  Table<kCap> t;
  int nparts = 0;
  for (int64_t i = 0; i < count;) {
    i = fill(t, x, i, count);
    if (t.count == 0) break;
    const int grid = grid_of(t);
    if (cudaError_t e = launch_pdl(grad_sum_kernel<kCap>, dim3(grid), dim3(kThreads), 0, s, t, parts + nparts); e != cudaSuccess)
      return e;
    nparts += grid;
  }
  if (!clip || nparts == 0)
    return launch_pdl(grad_norm_kernel, dim3(1), dim3(kThreads), 0, s, static_cast<const double*>(parts), nparts, norm);
  for (int64_t i = 0; i < count;) {
    const bool begin = i == 0;
    bool in_place = true;
    const int64_t next = fill(t, x, i, count);
    for (int j = 0; j < t.count; ++j) in_place = in_place && t.e[j].in == t.e[j].out;
    if (t.count == 0) break;
    const int grid = grid_of(t);
    if (cudaError_t e = launch_pdl(grad_scale_kernel<kCap>, dim3(grid), dim3(kThreads), 0, s, t,
                                   static_cast<const double*>(parts), nparts, most, in_place ? 1 : 0, begin ? norm : nullptr);
        e != cudaSuccess)
      return e;
    i = next;
  }
  return cudaSuccess;
}

}  // namespace

// One fp64 sum per block of the first launches.
size_t grad_norm_workspace_bytes(int64_t count) {
  const int64_t launches = (count + kMany - 1) / kMany;
  return static_cast<size_t>(launches) * kBlocks * sizeof(double);
}

cudaError_t launch_clip(const ClipTensor* tensors, int64_t count, float* norm, double most, int clip, void* workspace,
                        cudaStream_t s) {
  double* parts = static_cast<double*>(workspace);
  return count <= kFew ? launch_all<kFew>(tensors, count, norm, most, clip, parts, s)
                       : launch_all<kMany>(tensors, count, norm, most, clip, parts, s);
}

}  // namespace bl
