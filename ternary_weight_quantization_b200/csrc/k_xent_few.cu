// The head cross-entropy for a few tokens (X1, X2 with up to 16 tokens): a
// handful of tokens leaves the tensor-core tiles of 256 empty, and what counts
// is how fast W streams through. Here the rows of W are the 16-row operand of
// mma.sync and 8 or twice 8 tokens its columns; for the logits W goes from global
// memory to the operands' registers without shared memory in between.
//
//   logits    a warp takes 16 rows of W. The sum over K may take its terms in
//             any order, so a lane's 16 bytes of a row (8 consecutive values)
//             are the operands of two instructions, and the tokens' values are
//             read in the same order. Where there are few rows, the warps of a
//             block share a unit's K and join their sums in shared memory
//   forward   each lane keeps the running maximum and sum of its tokens; one
//             pair per token and block goes to the join
//   backward  one launch writes dz as two bf16 terms (hi + lo: 2^-17 relative),
//             32 bytes per row of W and 8 tokens. The second takes 64 columns
//             per warp and walks down the rows: dW = dz h in one instruction
//             per 16 x 8 tile (hi and lo are its 16 terms), dH += W^T dz in
//             registers, W's tiles transposed on their way out of shared memory.
//             The third joins dH over the row blocks, in a fixed order
//
// The join sums the target's logit once more in fp32 (the tensor cores' sums drop
// up to one step of fp32 per 16 terms).
//
// Bound by HBM where W is large, by the launches (two, three) where it is not.
// Measured on B200, forward / backward with a bf16 dW, next to the tiles' kernel:
// one token, 131072 x 4096: 172 / 575 us (206 / 650); the forward reads W at
// 6.2 TB/s. 4 tokens, 32000 x 2048: 24 / 70 (32 / 94). 8 tokens, 8192 x 512:
// 5.6 / 11.3 (8.2 / 19.3). 5 tokens, 68159 x 72: 7.4 / 16.5 (16.0 / 35.8).
// 16 tokens, 8192 x 512: 7.2 / 14.9 (8.1 / 19.2); 2000 x 1000: 6.1 / 12.3 (10.3 /
// 18.8); 32000 x 2560: 34.6 / 106 (35.5 / 105), with an fp32 dW 136 (134). With four
// groups 32 tokens, 8192 x 512 took 11.6 / 30.5 (8.4 / 19.6): the instructions grow
// with the tokens, and their sums leave registers for one block per SM. Above 16
// the tiles take over.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "bl_act8.cuh"
#include "bl_device.cuh"
#include "bl_internal.h"

namespace bl {
namespace {

constexpr int kWarps = 8;
constexpr float kLog2e = 1.4426950408889634f;

struct FewParams {
  const __nv_bfloat16* h;
  const __nv_bfloat16* W;
  const int64_t* targets;
  int M, V, K;
  int ksplit;      // logits: warps that share a unit's K (a power of two, <= kWarps)
  float2* part;    // forward: [block][M]
  float2* tlogit;  // forward: [M], the targets' logits (x)
  const float* lse;
  const float* dloss;
  uint32_t* dz;    // backward: [V][group of 8 tokens][4 words of hi, 4 of lo]
  float* dh_part;  // [row block][M][K], or null
  void* dW;        // or null
  int w_add;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Four 8 x 8 tiles of 16-bit values, lane l naming row l % 8 of tile l / 8: the
// lane gets elements 2 (l % 4) and the next of row l / 4 of each; kTrans: of
// column l / 4.
template <bool kTrans>
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t at) {
  if constexpr (kTrans)
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at)
                 : "memory");
  else
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at)
                 : "memory");
}

// 16 bytes to shared memory, zeros with in = false (src has to be readable).
__device__ __forceinline__ void copy16(uint32_t at, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(at), "l"(src), "r"(in ? 16 : 0) : "memory");
}

// W is read once (or once per launch): not kept in L1, where h stays.
__device__ __forceinline__ uint4 load_stream(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

__device__ __forceinline__ bool counts(const FewParams& p, int m) {
  if (m >= p.M) return false;
  const int64_t t = __ldg(p.targets + m);
  return t >= 0 && t < p.V;
}

// (maximum fl(z log2 e), sum of 2^(z log2 e - maximum)) joined with another pair,
// and with one logit. Where the maximum stays, the sum keeps its bits.
__device__ __forceinline__ void join(float& top, float& sum, float top2, float sum2) {
  const float n = fmaxf(top, top2), nl = n == __uint_as_float(0xFF800000u) ? 0.0f : n;
  sum = sum * ex2(top - nl) + sum2 * ex2(top2 - nl);
  top = n;
}
__device__ __forceinline__ void join(float& top, float& sum, float z) {
  const float n = fmaxf(top, z * kLog2e), nl = n == __uint_as_float(0xFF800000u) ? 0.0f : n;
  sum = fmaf(sum, ex2(top - nl), ex2(fmaf(z, kLog2e, -nl)));
  top = n;
}

// One step of 32 columns: two instructions per 8 tokens, two accumulators, so
// that instructions do not wait on each other and the sums' chains are short.
template <int NT>
__device__ __forceinline__ void logits_step(float (&acc)[2][NT][4], const uint4& w0, const uint4& w1,
                                            const uint4 (&x)[NT]) {
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    mma16816(acc[0][t], w0.x, w1.x, w0.y, w1.y, x[t].x, x[t].y);
    mma16816(acc[1][t], w0.z, w1.z, w0.w, w1.w, x[t].z, x[t].w);
  }
}

// The warp's share of the logits of 16 rows: c[t] holds (row lane / 4, tokens
// 8t + 2 (lane % 4) and the next), then the same 8 rows below.
template <int NT>
__device__ __forceinline__ void few_logits(const FewParams& p, int row0, int col0, int cols, const __nv_bfloat16* hp,
                                           const bool (&on)[NT], float (&c)[NT][4]) {
  const int lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  const int last = p.V - 1;
  const __nv_bfloat16* wa = p.W + static_cast<int64_t>(row0 + g < last ? row0 + g : last) * p.K;
  const __nv_bfloat16* wb = p.W + static_cast<int64_t>(row0 + g + 8 < last ? row0 + g + 8 : last) * p.K;
  const int64_t group = static_cast<int64_t>(8) * p.K;  // from a token to the one 8 below
  const uint4 zero = make_uint4(0, 0, 0, 0);
  float acc[2][NT][4] = {};
  constexpr int kAhead = NT == 1 ? 4 : 3;  // steps whose loads are in flight (128 registers)
  int k = col0;
#pragma unroll 1  // (unrolled, the registers run out: 178 us for 172)
  for (; k + 32 * kAhead <= cols; k += 32 * kAhead) {
    uint4 w0[kAhead], w1[kAhead], x[kAhead][NT];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      w0[i] = load_stream(wa + k + 32 * i + 8 * q);
      w1[i] = load_stream(wb + k + 32 * i + 8 * q);
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
#pragma unroll
      for (int t = 0; t < NT; ++t)
        x[i][t] = on[t] ? __ldg(reinterpret_cast<const uint4*>(hp + t * group + k + 32 * i + 8 * q)) : zero;
#pragma unroll
    for (int i = 0; i < kAhead; ++i) logits_step<NT>(acc, w0[i], w1[i], x[i]);
  }
  if (k < cols) {  // the last columns, all requested at once as well
    uint4 w0[kAhead], w1[kAhead], x[kAhead][NT];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int at = k + 32 * i + 8 * q;
      w0[i] = at < cols ? load_stream(wa + at) : zero;
      w1[i] = at < cols ? load_stream(wb + at) : zero;
#pragma unroll
      for (int t = 0; t < NT; ++t)
        x[i][t] = at < cols && on[t] ? __ldg(reinterpret_cast<const uint4*>(hp + t * group + at)) : zero;
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kAhead; ++i) logits_step<NT>(acc, w0[i], w1[i], x[i]);
  }
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i) c[t][i] = acc[0][t][i] + acc[1][t][i];
}

// dz as hi + lo, a pair of tokens.
__device__ __forceinline__ void split_pair(float a, float b, uint32_t& hi, uint32_t& lo) {
  hi = pack_bf16x2(b, a);
  lo = pack_bf16x2(b - bf16_hi(hi), a - bf16_lo(hi));
}

template <int NT, bool kGrad>
__global__ void __launch_bounds__(kWarps * 32, 2) few_logits_kernel(const FewParams p) {
  __shared__ float4 shares[2][kWarps][NT][32];
  __shared__ float2 pairs[kWarps][8 * NT];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  const int ks = p.ksplit, groups = kWarps / ks, grp = warp / ks, slice = warp % ks;
  const int steps = (p.K + 31) / 32, per = (steps + ks - 1) / ks;
  const int col0 = slice * per * 32, cols = col0 + per * 32 < p.K ? col0 + per * 32 : p.K;
  const float ninf = __uint_as_float(0xFF800000u);
  {
    const int row = (blockIdx.x * groups + grp) * 16 + (lane >> 1), c = col0 + (lane & 1) * 64;
    if (row < p.V && c < cols) prefetch_l2(p.W + static_cast<int64_t>(row) * p.K + c);
  }
  pdl_wait_primary();
  pdl_launch_dependents();

  const __nv_bfloat16* hp = p.h + static_cast<int64_t>(g) * p.K;
  bool on[NT];
  int tgt[NT][2];  // the lane's tokens, two of every 8: their targets, or -1
  float nlse[NT][2], gain[NT][2], top[NT][2], sum[NT][2];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    on[t] = kGrad ? counts(p, 8 * t + g) : 8 * t + g < p.M;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int m = 8 * t + 2 * q + e;
      const bool live = counts(p, m);
      tgt[t][e] = live ? static_cast<int>(__ldg(p.targets + m)) : -1;
      nlse[t][e] = kGrad && live ? -__ldg(p.lse + m) * kLog2e : 0.0f;
      gain[t][e] = kGrad && live ? __ldg(p.dloss + m) : 0.0f;
      top[t][e] = ninf;
      sum[t][e] = 0.0f;
    }
  }

  const int units = (p.V + 15) / 16, step = gridDim.x * groups;
  int buf = 0;
  for (int first = blockIdx.x * groups; first < units; first += step) {
    __syncwarp();
    const int row0 = (first + grp) * 16;
    float c[NT][4];
    if (row0 < p.V) few_logits<NT>(p, row0, col0, cols, hp, on, c);
    if (ks > 1) {
      if (row0 < p.V && slice != 0) {
#pragma unroll
        for (int t = 0; t < NT; ++t) shares[buf][warp][t][lane] = make_float4(c[t][0], c[t][1], c[t][2], c[t][3]);
      }
      __syncthreads();
      if (slice == 0 && row0 < p.V) {
        for (int s = 1; s < ks; ++s) {
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            const float4 o = shares[buf][warp + s][t][lane];
            c[t][0] += o.x, c[t][1] += o.y, c[t][2] += o.z, c[t][3] += o.w;
          }
        }
      }
      buf ^= 1;  // this one is free again after the next barrier
    }
    if (slice != 0 || row0 >= p.V) continue;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int row = row0 + g + 8 * half;
      if (row < p.V) {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          if constexpr (kGrad) {
            float d[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float x = ex2(fmaf(c[t][2 * half + e], kLog2e, nlse[t][e])) - (tgt[t][e] == row ? 1.0f : 0.0f);
              d[e] = tgt[t][e] >= 0 ? gain[t][e] * x : 0.0f;
            }
            uint32_t hi, lo;
            split_pair(d[0], d[1], hi, lo);
            uint32_t* at = p.dz + (static_cast<int64_t>(row) * NT + t) * 8 + q;
            at[0] = hi;
            at[4] = lo;
          } else {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float z = c[t][2 * half + e];
              join(top[t][e], sum[t][e], z);
              if (tgt[t][e] == row) p.tlogit[8 * t + 2 * q + e].x = z;
            }
          }
        }
      }
    }
  }
  if constexpr (!kGrad) {
    // 8 lanes hold rows of the same tokens; then the warps, in order
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int s = 4; s < 32; s *= 2) {
          const float t2 = __shfl_xor_sync(0xffffffffu, top[t][e], s), s2 = __shfl_xor_sync(0xffffffffu, sum[t][e], s);
          join(top[t][e], sum[t][e], t2, s2);
        }
        if (g == 0) pairs[warp][8 * t + 2 * q + e] = make_float2(top[t][e], sum[t][e]);
      }
    __syncthreads();
    if (threadIdx.x < p.M) {
      float2 a = make_float2(ninf, 0.0f);
      for (int w = 0; w < kWarps; w += ks) {
        const float2 b = pairs[w][threadIdx.x];
        join(a.x, a.y, b.x, b.y);
      }
      p.part[static_cast<int64_t>(blockIdx.x) * p.M + threadIdx.x] = a;
    }
  }
}

constexpr int kRing = 4;                     // units in flight per warp
template <int NT>
constexpr int kSlot = 16 * 128 + 16 * 32 * NT;  // a unit's 16 rows: 64 columns of W, dz
template <int NT>
constexpr int kProductsSmem = kWarps * kRing * kSlot<NT>;
static_assert(kProductsSmem<1> >= kWarps * 8 * 65 * 4, "the warps' sums take W's place");

template <int NT, bool kF32>
__global__ void __launch_bounds__(kWarps * 32, 2) few_products_kernel(const FewParams p) {
  extern __shared__ uint4 ring[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  const int c0 = blockIdx.x * 64;
  const bool want_dh = p.dh_part != nullptr;
  const int units = (p.V + 15) / 16, step = gridDim.y * kWarps;
  int u = blockIdx.y * kWarps + warp;
  const uint32_t mine = static_cast<uint32_t>(__cvta_generic_to_shared(ring)) + warp * kRing * kSlot<NT>;

  // W: 8 lanes copy a row's 128 bytes; chunk c of row r lies at place c ^ (r % 8)
  const int lr = lane >> 3, lc = c0 + 8 * (lane & 7);
  const bool want_w = want_dh && lc < p.K;
  const uint32_t w_to = mine + lr * 128;
  auto request_w = [&](int unit, int slot) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = lr + 4 * i, row = unit * 16 + r;
      const bool in = want_w && row < p.V;
      copy16(w_to + slot * kSlot<NT> + i * 512 + (((lane & 7) ^ (r & 7)) << 4),
             in ? p.W + static_cast<int64_t>(row) * p.K + lc : p.W, in);
    }
  };
  // dz: the unit's rows are one piece of memory; 16 bytes per lane and 8 tokens
  auto request_dz = [&](int unit, int slot) {
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int i = t * 32 + lane;
      const bool in = unit * 16 + i / (2 * NT) < p.V;
      copy16(mine + slot * kSlot<NT> + 2048 + i * 16, in ? p.dz + static_cast<int64_t>(unit) * 128 * NT + i * 4 : p.dz,
             in);
    }
  };
  // The launch before wrote dz alone, and began after all earlier ones had
  // ended: what this one reads besides dz needs no wait.
  if (want_dh) {
#pragma unroll
    for (int i = 0; i < kRing - 1; ++i)
      if (u + i * step < units) request_w(u + i * step, i);
  }
  // dW's operand: tokens 2q and 2q + 1 at the column that puts 16 consecutive
  // bytes of the result into one lane, 64 into four
  uint32_t hp[NT][8];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int m = 8 * t + 2 * q;
    const bool a = counts(p, m), b = counts(p, m + 1);
    const uint16_t* h0 = reinterpret_cast<const uint16_t*>(p.h) + static_cast<int64_t>(m) * p.K;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c = c0 + (kF32 ? 16 * (j >> 1) + 4 * (g >> 1) + 2 * (j & 1) : 32 * (j >> 2) + 8 * (g >> 1) + 2 * (j & 3)) + (g & 1);
      const uint32_t lo = a && c < p.K ? __ldg(h0 + c) : 0u, hi = b && c < p.K ? __ldg(h0 + p.K + c) : 0u;
      hp[t][j] = hi << 16 | lo;
    }
  }
  pdl_wait_primary();
  pdl_launch_dependents();
#pragma unroll
  for (int i = 0; i < kRing - 1; ++i) {
    if (u + i * step < units) request_dz(u + i * step, i);
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  // the rows that this lane names for the tiles: dz as [rows 0-7, 8-15] x [hi, lo];
  // W as [columns 16j + 0-7, 8-15] x [rows 0-7, 8-15]
  const int tr = lane & 7, tile = lane >> 3;
  const uint32_t dz_at = mine + 2048 + ((tile & 1) * 8 + tr) * (32 * NT) + (tile >> 1) * 16;
  const uint32_t w_at = mine + ((tile >> 1) * 8 + tr) * 128;
  float acc[NT][4][4] = {};
  for (int slot = 0; u < units; u += step, slot = slot + 1 < kRing ? slot + 1 : 0) {
    const int row0 = u * 16;
    asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 2) : "memory");
    __syncwarp();  // this unit is there for the whole warp, and the last one has been read
    if (const int ahead = u + (kRing - 1) * step; ahead < units) {
      const int to = slot ? slot - 1 : kRing - 1;
      if (want_dh) request_w(ahead, to);
      request_dz(ahead, to);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    if (want_dh) {
      uint32_t w[4][4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        ldmatrix4<true>(w[j], w_at + slot * kSlot<NT> + (((2 * j + (tile & 1)) ^ tr) << 4));
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        uint32_t d[4];  // hi of rows 0-7 and 8-15, then lo
        ldmatrix4<true>(d, dz_at + slot * kSlot<NT> + 32 * t);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          mma16816(acc[t][j], w[j][0], w[j][1], w[j][2], w[j][3], d[2], d[3]);
          mma16816(acc[t][j], w[j][0], w[j][1], w[j][2], w[j][3], d[0], d[1]);
        }
      }
    }
    if (p.dW) {
      uint32_t d[NT][4];
#pragma unroll
      for (int t = 0; t < NT; ++t) ldmatrix4<false>(d[t], dz_at + slot * kSlot<NT> + 32 * t);
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        __syncwarp();
        float o[4][4] = {};  // [pair of columns][row g: 2, row g + 8: 2]
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            mma16816(o[j], d[t][0], d[t][1], d[t][2], d[t][3], hp[t][4 * s + j], hp[t][4 * s + j]);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int row = row0 + g + 8 * half;
          if (row >= p.V) continue;
          if constexpr (kF32) {
#pragma unroll
            for (int b = 0; b < 2; ++b) {
              const int c = c0 + 32 * s + 16 * b + 4 * q;
              if (c >= p.K) continue;
              float4* out = reinterpret_cast<float4*>(static_cast<float*>(p.dW) + static_cast<int64_t>(row) * p.K + c);
              float4 v = make_float4(o[2 * b][2 * half], o[2 * b][2 * half + 1], o[2 * b + 1][2 * half],
                                     o[2 * b + 1][2 * half + 1]);
              if (p.w_add) {
                const float4 old = *out;
                v.x += old.x, v.y += old.y, v.z += old.z, v.w += old.w;
              }
              *out = v;
            }
          } else {
            const int c = c0 + 32 * s + 8 * q;
            if (c >= p.K) continue;
            __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.dW) + static_cast<int64_t>(row) * p.K + c;
            f32x2 v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = pair2(o[j][2 * half], o[j][2 * half + 1]);
            if (p.w_add) {
              f32x2 old[4];
              Raw8<__nv_bfloat16> r;
              r.load(out);
              r.get(old);
#pragma unroll
              for (int j = 0; j < 4; ++j) v[j] = add2(v[j], old[j]);
            }
            store8(out, v);
          }
        }
      }
    }
  }
  if (!want_dh) return;
  // the block's warps joined in order, where W was
  float(*joint)[8][65] = reinterpret_cast<float(*)[8][65]>(ring);
  asm volatile("cp.async.wait_group 0;" ::: "memory");
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) joint[warp][2 * q + (i & 1)][16 * j + g + 8 * (i >> 1)] = acc[t][j][i];
    __syncthreads();
    for (int i = threadIdx.x; i < 8 * 64; i += kWarps * 32) {
      const int m = 8 * t + (i >> 6), c = i & 63;
      float s = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) s += joint[w][i >> 6][c];
      if (m < p.M && c0 + c < p.K) p.dh_part[(static_cast<int64_t>(blockIdx.y) * p.M + m) * p.K + c0 + c] = s;
    }
  }
}

// dH from the row blocks' sums: 32 values per block, the row blocks spread over
// 16 threads of each.
__global__ void __launch_bounds__(512) few_dh_kernel(const float* __restrict__ parts, int nparts, int n,
                                                     __nv_bfloat16* __restrict__ dH) {
  pdl_wait_primary();
  pdl_launch_dependents();
  __shared__ float sh[16][33];
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
  const int i = blockIdx.x * 32 + x;
  float s = 0.0f;
  if (i < n) {
#pragma unroll 10
    for (int r = y; r < nparts; r += 16) s += parts[static_cast<int64_t>(r) * n + i];
  }
  sh[y][x] = s;
  __syncthreads();
  if (y == 0 && i < n) {
#pragma unroll
    for (int q = 1; q < 16; ++q) s += sh[q][x];
    dH[i] = __float2bfloat16_rn(s);
  }
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

constexpr int64_t kWave = 2 * kPlanSms;  // blocks at work at once, two per SM

// The logits' warps per unit of 16 rows: as many as it takes to give every SM
// 8 warps, as long as each has more than one round of loads (4 steps of 32).
// Measured on B200 (forward): 4000 x 4096 8.9 us with 8 warps, 27.9 with one;
// 8192 x 512 5.3 with 4, 6.9 with one; 32000 x 2048 25.2 with two, 23.7 with one.
int few_ksplit(int64_t V, int64_t K) {
  const int64_t units = ceil_div(V, 16), steps = ceil_div(K, 32);
  int ks = 1;
  while (ks < kWarps && units * ks < kPlanSms * 8 && steps > 4 * ks) ks *= 2;
  return ks;
}

int few_blocks(int64_t V, int64_t K) {
  const int64_t want = ceil_div(ceil_div(V, 16) * few_ksplit(V, K), kWarps);
  return static_cast<int>(want < kWave ? want : kWave);
}

// Row blocks of the products: one wave of two blocks per SM; two waves, which
// even out, where a warp still has 8 units in each. Measured on B200 (backward):
// 32000 x 2560 95.7 us in one wave, 87.9 in two; 8192 x 512 10.4 and 12.3.
int few_row_blocks(int64_t V, int64_t K) {
  const int64_t warps = ceil_div(ceil_div(V, 16), kWarps), tiles = ceil_div(K, 64);
  const int64_t one = kWave / tiles > 0 ? kWave / tiles : 1;
  const int64_t two = 2 * kWave / tiles > 0 ? 2 * kWave / tiles : 1;
  const int64_t most = warps >= 8 * two ? two : one;
  return static_cast<int>(warps < most ? warps : most);
}

int few_groups(int64_t M) { return M <= 8 ? 1 : 2; }  // of 8 tokens: the kernels' NT

size_t few_dz_bytes(int64_t M, int64_t V) { return static_cast<size_t>(V) * 32 * few_groups(M); }

FewParams few_params(const void* h, const void* W, const int64_t* targets, int64_t M, int64_t V, int64_t K) {
  FewParams p{};
  p.h = static_cast<const __nv_bfloat16*>(h);
  p.W = static_cast<const __nv_bfloat16*>(W);
  p.targets = targets;
  p.M = static_cast<int>(M);
  p.V = static_cast<int>(V);
  p.K = static_cast<int>(K);
  p.ksplit = few_ksplit(V, K);
  return p;
}

template <bool kGrad>
cudaError_t launch_logits(const FewParams& p, cudaStream_t s) {
  const dim3 grid(few_blocks(p.V, p.K)), block(kWarps * 32);
  return few_groups(p.M) == 1 ? launch_pdl(few_logits_kernel<1, kGrad>, grid, block, 0, s, p)
                              : launch_pdl(few_logits_kernel<2, kGrad>, grid, block, 0, s, p);
}

template <int NT, bool kF32>
cudaError_t launch_products(const FewParams& p, int row_blocks, cudaStream_t s) {
  static bool done[64] = {};  // per device: the kernel's shared memory is set
  int dev = 0;
  if (const cudaError_t e = cudaGetDevice(&dev); e != cudaSuccess) return e;
  if (dev >= 64 || !done[dev]) {
    const cudaError_t e = cudaFuncSetAttribute(few_products_kernel<NT, kF32>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, kProductsSmem<NT>);
    if (e != cudaSuccess) return e;
    if (dev < 64) done[dev] = true;
  }
  return launch_pdl(few_products_kernel<NT, kF32>, dim3(static_cast<unsigned>(ceil_div(p.K, 64)), row_blocks),
                    dim3(kWarps * 32), kProductsSmem<NT>, s, p);
}

template <bool kF32>
cudaError_t launch_products(const FewParams& p, int row_blocks, cudaStream_t s) {
  return few_groups(p.M) == 1 ? launch_products<1, kF32>(p, row_blocks, s) : launch_products<2, kF32>(p, row_blocks, s);
}

}  // namespace

int xent_few_parts(int64_t V, int64_t K) { return few_blocks(V, K); }

size_t xent_few_workspace_bytes(int64_t M, int64_t V, int64_t K) {
  return few_dz_bytes(M, V) + static_cast<size_t>(few_row_blocks(V, K)) * M * K * 4;
}

cudaError_t launch_xent_few_forward(const void* h, const void* W, const int64_t* targets, int64_t M, int64_t V,
                                    int64_t K, float2* part, float2* tlogit, cudaStream_t s) {
  FewParams p = few_params(h, W, targets, M, V, K);
  p.part = part;
  p.tlogit = tlogit;
  return launch_logits<false>(p, s);
}

cudaError_t launch_xent_few_backward(const void* h, const void* W, const int64_t* targets, const float* lse,
                                     const float* dloss, int64_t M, int64_t V, int64_t K, void* dH, void* dW,
                                     int dw_is_f32, int accumulate, void* workspace, cudaStream_t s) {
  FewParams p = few_params(h, W, targets, M, V, K);
  p.lse = lse;
  p.dloss = dloss;
  p.dz = static_cast<uint32_t*>(workspace);
  float* parts = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + few_dz_bytes(M, V));
  p.dh_part = dH ? parts : nullptr;
  p.dW = dW;
  p.w_add = accumulate;
  if (const cudaError_t e = launch_logits<true>(p, s); e != cudaSuccess) return e;
  const int row_blocks = few_row_blocks(V, K);
  const cudaError_t e =
      dw_is_f32 ? launch_products<true>(p, row_blocks, s) : launch_products<false>(p, row_blocks, s);
  if (e != cudaSuccess || !dH) return e;
  const int n = static_cast<int>(M * K);
  return launch_pdl(few_dh_kernel, dim3((n + 31) / 32), dim3(512), 0, s, static_cast<const float*>(parts), row_blocks,
                    n, static_cast<__nv_bfloat16*>(dH));
}

}  // namespace bl
