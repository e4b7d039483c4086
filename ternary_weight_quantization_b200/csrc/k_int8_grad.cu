// The straight-through gradients of the INT8 product (L2) for a few tokens, from the
// codes themselves: one reading of the weights gives both.
//
//   dX[m,k] = sum_n dY[m,n] w_hat[n,k]      w_hat = bf16(code * sw[n])
//   dW[n,k] = sum_m dY[m,n] x_hat[m,k]      x_hat = bf16(code * sx[m])
//
// A block has 32 kW columns of K and a slice of the channels; a warp takes 16 channels
// at a time. mma.sync.m16n8k16, fp32 sums:
//   dX   rows = tokens, columns = K, over the channels: a lane's codes of channels
//        2t, 2t + 1, 2t + 8, 2t + 9 (4 kW bytes of each, straight from global memory) are
//        its B operands of 4 kW instructions, whose columns are 4 kW apart
//   dW   rows = channels, columns = K, over the tokens: dY's operand transposed in
//        registers, x_hat from shared memory, laid out so that a lane's results are
//        8 consecutive columns
// dX's sums stay in registers over the warp's channels; the warps' are added in
// shared memory, the slices' by a second launch, both in order.
//
// The weights are read once and dW written once; at that it is short of instructions
// (ncu, 16 x 32000 x 2560: 430 of them for 2048 codes of dX, 0.5 issued a cycle and
// scheduler), and few tokens leave it a start, a wave and a join. Measured on B200 (in a
// graph, inputs from HBM; floor by bytes; before: by values written in bf16 and the
// products of k_xent.cu, which more tokens take):
//   tokens x channels x K   us      floor   before
//   1 x 6912 x 2560         16.3    8.1     31.5
//   16 x 6912 x 2560        18.1    8.2     29.9
//   32 x 6912 x 2560        23.8    8.2     30.0    (64: 45.8 for 31.1)
//   2 x 25128 x 208         13.0    2.4     19.2    (its 148 slices joined by one thread a place: 22.4)
//   64 x 512 x 512          6.0     0.2     9.7
//   5 x 11976 x 2704        26      14.9    54.1
//   16 x 32000 x 2560       102     62.7    134     (dW in fp32)
//   13 x 368 x 1984         6.5     0.4     8.6
// A ring of asynchronous copies for the codes measured 18.9 us at 1 x 6912 x 2560, and
// sums written to shared memory without `place` 20.4.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "bl_act8.cuh"
#include "bl_device.cuh"
#include "bl_internal.h"
#include "bl_rows.cuh"

namespace bl {
namespace {

constexpr int kGradWarps = 8, kGradThreads = 32 * kGradWarps;

struct FewGradParams {
  const __nv_bfloat16* dY;
  const int8_t* xq;
  const float* sx;
  const int8_t* wq;
  const float* sw;
  int M, N, K;
  int tiles_k, slices;
  __nv_bfloat16* dX;  // of a single slice
  float* sums;        // [slices][M][K], of more (or null: no dX)
  void* dW;           // or null
  int accumulate;
};

// kTok: 16 tokens each.
template <int kTok>
struct FewGrad {
  static constexpr int kW = 4 / kTok, kCols = 32 * kW, kTiles = kCols / 8;  // words of a channel per lane; tiles of 8 columns
  static constexpr int kXBytes = kTok * kTiles * 32 * 8;
  static constexpr int kSmemBytes = kXBytes + kGradWarps * 16 * kTok * kCols * 4;
};

__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

// Code j of two words (with their sign bits turned) times two scales, in bf16:
// 2^23 + 128 + code has the code in its low byte.
__device__ __forceinline__ uint32_t values2(uint32_t a, uint32_t b, int j, f32x2 scale) {
  const uint32_t lo = __byte_perm(a, 0x4B000000u, 0x7440u | j), hi = __byte_perm(b, 0x4B000000u, 0x7440u | j);
  return pack_bf16x2(mul2(add2(pair2(__uint_as_float(lo), __uint_as_float(hi)), both2(-8388736.0f)), scale));
}

__device__ __forceinline__ void load_words(const int8_t* p, uint32_t (&w)[4]) {
  const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
  w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
}
__device__ __forceinline__ void load_words(const int8_t* p, uint32_t (&w)[2]) {
  const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
  w[0] = v.x, w[1] = v.y;
}

__device__ __forceinline__ void load_words(const int8_t* p, uint32_t (&w)[1]) {
  w[0] = __ldg(reinterpret_cast<const uint32_t*>(p));
}

// Eight columns of a channel of dW.
__device__ __forceinline__ void write_dw(float* to, float (&v)[8], int add) {
  float4* q = reinterpret_cast<float4*>(to);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float4 r = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    if (add) {
      const float4 o = q[i];
      r.x += o.x, r.y += o.y, r.z += o.z, r.w += o.w;
    }
    q[i] = r;
  }
}
__device__ __forceinline__ void write_dw(__nv_bfloat16* to, float (&v)[8], int add) {
  uint4* q = reinterpret_cast<uint4*>(to);
  if (add) {
    const uint4 o = *q;
    const uint32_t w[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) v[2 * i] += bf16_lo(w[i]), v[2 * i + 1] += bf16_hi(w[i]);
  }
  *q = make_uint4(pack_bf16x2(v[1], v[0]), pack_bf16x2(v[3], v[2]), pack_bf16x2(v[5], v[4]), pack_bf16x2(v[7], v[6]));
}

// Place of 4 columns, the f-th, in a token's row of the sums: the lanes of a store (8
// apart in f or a row apart) fall on different banks.
__device__ __forceinline__ int place(int f, int token) { return f ^ ((f >> 3) << 1 | (token & 1)); }

template <int kTok, typename TW>
__global__ void __launch_bounds__(kGradThreads, 2) int8_few_grad_kernel(const FewGradParams p) {
  using G = FewGrad<kTok>;
  constexpr int kW = G::kW, kCols = G::kCols, kTiles = G::kTiles;
  extern __shared__ uint8_t smem[];
  uint2* xf = reinterpret_cast<uint2*>(smem);  // [kTok][kTiles][32]: x_hat as B operands
  float* red = reinterpret_cast<float*>(smem + G::kXBytes);  // [warps][tokens][columns]
  pdl_wait_primary();
  pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int kb = static_cast<int>(blockIdx.x) % p.tiles_k * kCols, slice = static_cast<int>(blockIdx.x) / p.tiles_k;
  const int chunks = (p.N + 15) >> 4;
  const int c0 = static_cast<int>(static_cast<int64_t>(chunks) * slice / p.slices),
            c1 = static_cast<int>(static_cast<int64_t>(chunks) * (slice + 1) / p.slices);
  const int kl = kb + g * 4 * kW;  // the lane's columns of the weights
  const bool dx = p.dX != nullptr || p.sums != nullptr, dw = p.dW != nullptr;

  // a chunk's codes, their scales, dY's operands
  uint32_t w[4][kW], a[kTok][4];
  float s[4];
  auto load = [&](int c) {
    const int n = c * 16 + 2 * t;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int nr = n + (r & 1) + (r >> 1) * 8;
      s[r] = 0.0f;
#pragma unroll
      for (int i = 0; i < kW; ++i) w[r][i] = 0u;
      if (dx && nr < p.N) {
        s[r] = __ldg(p.sw + nr);
        if (kl < p.K) load_words(p.wq + static_cast<int64_t>(nr) * p.K + kl, w[r]);
      }
    }
#pragma unroll
    for (int m = 0; m < kTok; ++m)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int token = 16 * m + g + (r & 1) * 8, nr = n + (r >> 1) * 8;
        a[m][r] = token < p.M && nr < p.N ? __ldg(reinterpret_cast<const uint32_t*>(p.dY + static_cast<int64_t>(token) * p.N + nr)) : 0u;
      }
  };
  int c = c0 + warp;
  if (c < c1) load(c);
  if (dw) {
    for (int i = threadIdx.x; i < kTok * kTiles * 32; i += kGradThreads) {
      const int l = i & 31, jj = i / 32 % kTiles, m = i / (32 * kTiles), lg = l >> 2, lt = l & 3;
      const int k = kb + 32 * (jj >> 2) + 8 * (lg >> 1) + 2 * (jj & 3) + (lg & 1);
      float v[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int token = 16 * m + 2 * lt + (r & 1) + (r >> 1) * 8;
        v[r] = token < p.M && k < p.K
                   ? __fmul_rn(static_cast<float>(__ldg(p.xq + static_cast<int64_t>(token) * p.K + k)), __ldg(p.sx + token))
                   : 0.0f;
      }
      xf[i] = make_uint2(pack_bf16x2(v[1], v[0]), pack_bf16x2(v[3], v[2]));
    }
    __syncthreads();
  }
  float acc[kTok][kTiles][4] = {};
  for (; c < c1; c += kGradWarps) {
    uint32_t tr[kTok][4];
#pragma unroll
    for (int m = 0; m < kTok; ++m) {
      // (of the four 8 x 8 parts the two off the diagonal change places)
      tr[m][0] = transpose8(a[m][0]), tr[m][1] = transpose8(a[m][2]);
      tr[m][2] = transpose8(a[m][1]), tr[m][3] = transpose8(a[m][3]);
    }
    if (dx) {
      const f32x2 lo = pair2(s[0], s[1]), hi = pair2(s[2], s[3]);
#pragma unroll
      for (int i = 0; i < kW; ++i) {
        uint32_t x[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) x[r] = w[r][i] ^ 0x80808080u;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t b0 = values2(x[0], x[1], j, lo), b1 = values2(x[2], x[3], j, hi);
#pragma unroll
          for (int m = 0; m < kTok; ++m) mma_bf16(acc[m][4 * i + j], a[m], b0, b1);
        }
      }
    }
    const int n0 = c * 16 + g;
    if (c + kGradWarps < c1) load(c + kGradWarps);
    if (dw) {
#pragma unroll
      for (int i = 0; i < kW; ++i) {
        float d[4][4] = {};
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int m = 0; m < kTok; ++m) {
            const uint2 b = xf[(m * kTiles + 4 * i + j) * 32 + lane];
            mma_bf16(d[j], tr[m], b.x, b.y);
          }
        const int k = kb + 32 * i + 8 * t;
        if (k < p.K) {
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            if (n0 + 8 * r < p.N) {
              float v[8];
#pragma unroll
              for (int j = 0; j < 4; ++j) v[2 * j] = d[j][2 * r], v[2 * j + 1] = d[j][2 * r + 1];
              write_dw(static_cast<TW*>(p.dW) + static_cast<int64_t>(n0 + 8 * r) * p.K + k, v, p.accumulate);
            }
          }
        }
      }
    }
  }
  if (!dx) return;
  // tile jj's column 2t + h is column (2t + h) 4 kW + jj of the block's
  float* own = red + warp * 16 * kTok * kCols;
#pragma unroll
  for (int m = 0; m < kTok; ++m)
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int i = 0; i < kW; ++i)
        *reinterpret_cast<float4*>(own + (16 * m + g + (r >> 1) * 8) * kCols + 4 * place((2 * t + (r & 1)) * kW + i, g)) =
            make_float4(acc[m][4 * i][r], acc[m][4 * i + 1][r], acc[m][4 * i + 2][r], acc[m][4 * i + 3][r]);
  __syncthreads();
  for (int i = threadIdx.x; i < 16 * kTok * kCols / 4; i += kGradThreads) {
    const int token = i / (kCols / 4), f = i % (kCols / 4), k = kb + 4 * f, at = i - f + place(f, token);
    if (token >= p.M || k >= p.K) continue;
    float4 v = reinterpret_cast<const float4*>(red)[at];
#pragma unroll
    for (int u = 1; u < kGradWarps; ++u) {
      const float4 o = reinterpret_cast<const float4*>(red + u * 16 * kTok * kCols)[at];
      v.x += o.x, v.y += o.y, v.z += o.z, v.w += o.w;
    }
    if (p.dX)
      *reinterpret_cast<uint2*>(p.dX + static_cast<int64_t>(token) * p.K + k) = make_uint2(pack_bf16x2(v.y, v.x), pack_bf16x2(v.w, v.z));
    else
      *reinterpret_cast<float4*>(p.sums + (static_cast<int64_t>(slice) * p.M + token) * p.K + k) = v;
  }
}

// dX from its slices. There may be few outputs of many slices, so 8 warps share 32
// places (of 4 columns): each adds every eighth slice, and the first one their sums.
__global__ void __launch_bounds__(256) int8_few_join_kernel(const float4* __restrict__ sums, int64_t vecs, int slices,
                                                            uint2* __restrict__ dX) {
  __shared__ float4 sh[8][32];
  pdl_wait_primary();
  pdl_launch_dependents();
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 32 + x;
  float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (i < vecs) {
    constexpr int kU = 4;
    for (int s = y; s < slices; s += 8 * kU) {
      float4 w[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u)
        w[u] = s + 8 * u < slices ? sums[(s + 8 * u) * vecs + i] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int u = 0; u < kU; ++u) v.x += w[u].x, v.y += w[u].y, v.z += w[u].z, v.w += w[u].w;
    }
  }
  sh[y][x] = v;
  __syncthreads();
  if (y > 0 || i >= vecs) return;
#pragma unroll
  for (int u = 1; u < 8; ++u) v.x += sh[u][x].x, v.y += sh[u][x].y, v.z += sh[u][x].z, v.w += sh[u][x].w;
  dX[i] = make_uint2(pack_bf16x2(v.y, v.x), pack_bf16x2(v.w, v.z));
}

template <int kTok, typename TW>
cudaError_t launch_few(FewGradParams p, cudaStream_t s) {
  using G = FewGrad<kTok>;
  auto kernel = int8_few_grad_kernel<kTok, TW>;
  static bool done[64] = {};
  if (cudaError_t e = allow_smem(kernel, G::kSmemBytes, done); e != cudaSuccess) return e;
  return launch_pdl(kernel, dim3(static_cast<unsigned>(p.tiles_k * p.slices)), dim3(kGradThreads), G::kSmemBytes, s, p);
}

}  // namespace

cudaError_t launch_int8_few_grads(const void* dY, const int8_t* xq, const float* sx, const int8_t* wq, const float* sw,
                                  int64_t M, int64_t N, int64_t K, void* dX, void* dW, int dw_is_f32, int accumulate,
                                  float* sums, cudaStream_t s) {
  FewGradParams p{};
  p.dY = static_cast<const __nv_bfloat16*>(dY);
  p.xq = xq;
  p.sx = sx;
  p.wq = wq;
  p.sw = sw;
  p.M = static_cast<int>(M);
  p.N = static_cast<int>(N);
  p.K = static_cast<int>(K);
  p.dW = dW;
  p.accumulate = accumulate;
  const int tok = M <= 16 ? 1 : M <= 32 ? 2 : 4, cols = 128 / tok;
  p.tiles_k = static_cast<int>((K + cols - 1) / cols);
  // slices of the channels: two blocks per SM, 16 channels per warp at least, and
  // no more than the sums have room for (2 bytes per weight)
  int64_t slices = 2 * device_sm_count() / p.tiles_k;
  const int64_t chunks = (N + 15) / 16, busy = (chunks + kGradWarps - 1) / kGradWarps, room = N / (2 * M);
  slices = slices < busy ? slices : busy;
  slices = slices < room ? slices : room;
  p.slices = slices < 1 ? 1 : static_cast<int>(slices);
  if (dX) {
    if (p.slices == 1) p.dX = static_cast<__nv_bfloat16*>(dX);
    else p.sums = sums;
  }
  cudaError_t e;
  if (tok == 1) e = dw_is_f32 ? launch_few<1, float>(p, s) : launch_few<1, __nv_bfloat16>(p, s);
  else if (tok == 2) e = dw_is_f32 ? launch_few<2, float>(p, s) : launch_few<2, __nv_bfloat16>(p, s);
  else e = dw_is_f32 ? launch_few<4, float>(p, s) : launch_few<4, __nv_bfloat16>(p, s);
  if (e != cudaSuccess || !p.sums) return e;
  const int64_t vecs = M * K / 4;
  return launch_pdl(int8_few_join_kernel, dim3(static_cast<unsigned>((vecs + 31) / 32)), dim3(256), 0, s,
                    reinterpret_cast<const float4*>(sums), vecs, p.slices, static_cast<uint2*>(dX));
}

}  // namespace bl
