// Product of two INT8 operands with a scale per token and per output channel
// (L1), and the operands' values for its straight-through gradients (L2).
//
//   acc[m,n] = sum_k xq[m,k] wq[n,k]              exact INT32
//   y[m,n]   = rn(fp32(acc) * fp32(sx[m] * sw[n]))
//
// Three kernels:
//   int8_tile_kernel  persistent CTA pairs, tcgen05.mma kind::i8 (cta_group::2),
//                     both operands by TMA, INT32 accumulators in TMEM
//   int8_few_kernel   a few tokens: the weights stream through mma.sync straight
//                     from global memory, in the order that makes a lane's
//                     16-byte loads the operands
//   int8_values_kernel  rn_bf16(code * scale) of both operands, for the gradients'
//                     products (k_xent.cu)
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <cstdint>

#include "bl_act8.cuh"
#include "bl_device.cuh"
#include "bl_internal.h"
#include "bl_rows.cuh"

namespace bl {
namespace {

// ---------------------------------------------------------------- tiles
// A pair tile is 256 tokens x BN channels; a stage is 128 of K: per CTA 128
// tokens' and BN / 2 channels' rows of 128 bytes, 128-byte swizzled. Everything
// outside the tensors loads as zeros (nothing in the sums) and is not stored.
//
// Roles (320 threads per CTA): warp 0 loads, warp 1 issues the MMAs (one lane of
// the leader CTA), warps 2..9 are the epilogue (two per TMEM lane quadrant, half
// the columns each; thread = token). Every wait is bounded: on expiry a CTA
// records a timeout in the device error word, tells its peer, drains what it has
// in flight, frees TMEM and exits.
constexpr int kRows = 256;             // tokens of a pair tile
constexpr int kBlockK = 128;           // K per stage
constexpr int kABytes = 128 * kBlockK; // one CTA's tokens of a stage
constexpr uint32_t kTmemCols = 512;    // two accumulators
constexpr int kEpiWarps = 8, kWarpEpi0 = 2, kTileThreads = 32 * (kWarpEpi0 + kEpiWarps);
constexpr int kEpiBox = 4096;          // output box: 32 rows x 128 bytes

template <int BN>
struct Geo {
  static constexpr int kBBytes = BN / 2 * kBlockK;
  static constexpr int kStageBytes = kABytes + kBBytes;
  static constexpr int kStages = BN == 256 ? 6 : 7;
  static constexpr int kSlots = BN == 256 ? 1 : 1;  // output boxes per epilogue warp
  static constexpr int kOffEpi = kStages * kStageBytes;
  static constexpr int kOffBar = kOffEpi + kEpiWarps * kSlots * kEpiBox;
  static constexpr int kNumBars = 2 * kStages + 5;  // full, empty, tmem_full[2], tmem_empty[2], done
  static constexpr int kOffMisc = kOffBar + kNumBars * 8;
  static constexpr int kSmemBytes = kOffMisc + 64 + 1024 /*base alignment*/;
  static_assert(kSmemBytes <= 232448, "shared memory budget");
};

struct TileParams {
  int M, N, K;
  int tiles_m, ntiles;
  const float* sx;
  const float* sw;
  void* y;
  int* err;
};

__device__ __forceinline__ void load_pair(const CUtensorMap* map, uint32_t bar_cluster, uint32_t dst, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], "
      "[%2];" ::"r"(dst),
      "l"(map), "r"(bar_cluster), "r"(x), "r"(y)
      : "memory");
}

__device__ __forceinline__ void st_shared_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// 16-byte chunk j of row `row` of a 32 x 128 byte box, 128-byte swizzled.
__device__ __forceinline__ uint32_t box_chunk(uint32_t box, int row, int j) {
  return box + static_cast<uint32_t>(row) * 128u + (static_cast<uint32_t>(j ^ (row & 7)) << 4);
}

// TY: type of y. kTma: y's rows start on 16-byte boundaries, so a box leaves by
// one TMA store; else the warp writes it row by row.
template <typename TY, int BN, bool kTma>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kTileThreads, 1)
    int8_tile_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w,
                     const __grid_constant__ CUtensorMap map_y, const __grid_constant__ TileParams p) {
  using G = Geo<BN>;
  constexpr int kStages = G::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + G::kOffBar);
  uint64_t* empty = full + kStages;
  uint64_t* tmem_full = full + 2 * kStages;
  uint64_t* tmem_empty = tmem_full + 2;
  uint64_t* done_bar = tmem_full + 4;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + G::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + G::kOffMisc + 4);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int pair = static_cast<int>(blockIdx.x >> 1), npairs = static_cast<int>(gridDim.x >> 1);

  if (threadIdx.x == 32 * kWarpEpi0) {
    prefetch_tensormap(&map_x);
    prefetch_tensormap(&map_w);
    if (kTma) prefetch_tensormap(&map_y);
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tmem_full[b], 1);
      mbar_init(&tmem_empty[b], 2 * kEpiWarps);
    }
    mbar_init(done_bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_holder, kTmemCols);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;
  pdl_wait_primary();
  pdl_launch_dependents();

  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    if (mbar_wait(bar, parity, abort_flag, p.err)) return true;
    st_cluster_u32(map_to_rank(smem_u32(const_cast<int*>(abort_flag)), rank ^ 1u), 1u);
    return false;
  };
  auto lead = [&](uint64_t* bar) -> uint32_t { return map_to_rank(smem_u32(bar), 0); };
  const int nkb = (p.K + kBlockK - 1) / kBlockK;
  // tokens fastest: the pairs at work share few tiles of the weights
  auto tile_row = [&](int u) { return u % p.tiles_m * kRows + static_cast<int>(rank) * 128; };
  auto tile_col = [&](int u) { return u / p.tiles_m * BN; };

  if (warp == 0) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0, issued = 0;  // stages requested so far
      const uint32_t bars = lead(full), smem0 = smem_u32(smem);
      bool ok = true;
      for (int u = pair; ok && u < p.ntiles; u += npairs) {
        const int a0 = tile_row(u), b0 = tile_col(u) + static_cast<int>(rank) * (BN / 2);
        for (int kb = 0; kb < nkb; ++kb) {
          if (!wait(&empty[stage], phase ^ 1)) {
            ok = false;
            break;
          }
          // both CTAs' boxes arrive on the leader's barrier
          if (leader) mbar_arrive_expect_tx(&full[stage], 2 * G::kStageBytes);
          const uint32_t at = smem0 + stage * G::kStageBytes, bar = bars + 8 * stage;
          load_pair(&map_x, bar, at, kb * kBlockK, a0);
          load_pair(&map_w, bar, at + kABytes, kb * kBlockK, b0);
          ++issued;
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
      if (leader && (!ok || *abort_flag)) {
        // let every copy already issued land before the pair exits
        const unsigned long long deadline = globaltimer_ns() + kWaitLimitNs;
        for (uint32_t s = 0; s < kStages && s < issued; ++s)
          mbar_drain_until(&full[s], (issued - s - 1) / kStages & 1, deadline);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (leader && lane == 0) {
      constexpr uint32_t kIdesc = make_idesc(2 /*s32*/, 1 /*s8*/, 0, 0, kRows, BN);
      const uint32_t s0 = smem_u32(smem);
      const uint64_t ad0 = smem_desc_sw128(s0, 16, 1024), bd0 = smem_desc_sw128(s0 + kABytes, 16, 1024);
      int stage = 0, buf = 0;
      uint32_t phase = 0, buf_phase = 0;
      bool ok = true;
      for (int u = pair; ok && u < p.ntiles; u += npairs) {
        if (!wait(&tmem_empty[buf], buf_phase ^ 1)) break;
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(buf * 256);
        for (int kb = 0; kb < nkb; ++kb) {
          if (!wait(&full[stage], phase)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t at = static_cast<uint64_t>(stage) * (G::kStageBytes >> 4);
#pragma unroll
          for (int kk = 0; kk < kBlockK / 32; ++kk)
            mma_i8_pair(d_tmem, ad0 + at + kk * 2, bd0 + at + kk * 2, kIdesc, (kb | kk) != 0);
          mma_commit_pair(&empty[stage], 0x3);
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1;
          }
        }
        if (ok) mma_commit_pair(&tmem_full[buf], 0x3);
        if (++buf == 2) {
          buf = 0;
          buf_phase ^= 1;
        }
      }
      mma_commit_pair(done_bar, 0x3);
    }
    if (lane == 0) mbar_drain(done_bar, 0);
    __syncwarp();
  } else {
    const int q = warp & 3, part = (warp - kWarpEpi0) >> 2, slot0 = warp - kWarpEpi0;
    constexpr int kChunks = BN / 64;  // 32-column chunks of a warp
    const uint32_t boxes = smem_u32(smem + G::kOffEpi + slot0 * G::kSlots * kEpiBox);
    uint32_t seq = 0, box = 0;
    int buf = 0;
    uint32_t buf_phase = 0;
    constexpr int kEsize = sizeof(TY), kPerBox = 128 / kEsize;  // columns of a box: 64 or 32
    for (int u = pair; u < p.ntiles; u += npairs) {
      const int row0 = tile_row(u) + q * 32, row = row0 + lane;
      const int col0 = tile_col(u) + part * (BN / 2);
      const float sx = row < p.M ? __ldg(p.sx + row) : 0.0f;
      const f32x2 sx2 = both2(sx);
      if (!wait(&tmem_full[buf], buf_phase)) break;
      tc_fence_after();
      const uint32_t tbase = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + buf * 256 + part * (BN / 2);
      auto chunk = [&](uint32_t (&r)[32], int c) {
        const int col = col0 + 32 * c;
        if (col >= p.N) return;
        f32x2 v[16];
        const float* sw = p.sw + col;
        if (col + 32 <= p.N) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float4 w = __ldg(reinterpret_cast<const float4*>(sw) + j);
            v[2 * j] = pair2(w.x, w.y);
            v[2 * j + 1] = pair2(w.z, w.w);
          }
        } else {
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const float a = col + 2 * j < p.N ? __ldg(sw + 2 * j) : 0.0f;
            const float b = col + 2 * j + 1 < p.N ? __ldg(sw + 2 * j + 1) : 0.0f;
            v[j] = pair2(a, b);
          }
        }
        // three roundings in fp32: of the sum, of the two scales' product, of y
#pragma unroll
        for (int j = 0; j < 16; ++j)
          v[j] = mul2(pair2(__int2float_rn(static_cast<int>(r[2 * j])), __int2float_rn(static_cast<int>(r[2 * j + 1]))),
                      mul2(v[j], sx2));
        const bool first = kEsize == 4 || (c & 1) == 0, last = kEsize == 4 || (c & 1) || col + 32 >= p.N;
        if (first) {
          if constexpr (kTma) {
            if (lane == 0) bulk_wait_group_read<G::kSlots - 1>();
          }
          __syncwarp();
          box = boxes + (seq++ % G::kSlots) * kEpiBox;
        }
        if constexpr (kEsize == 4) {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            asm volatile("st.shared.v2.b64 [%0], {%1, %2};" ::"r"(box_chunk(box, lane, j)), "l"(v[2 * j]), "l"(v[2 * j + 1])
                         : "memory");
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            st_shared_v4(box_chunk(box, lane, (c & 1) * 4 + j), pack_bf16x2(v[4 * j]), pack_bf16x2(v[4 * j + 1]),
                         pack_bf16x2(v[4 * j + 2]), pack_bf16x2(v[4 * j + 3]));
        }
        if (!last) return;
        const int bcol = col & ~(kPerBox - 1);  // (a warp's first column is a multiple of 64)
        if constexpr (kTma) {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_2d(&map_y, box, bcol, row0);
            bulk_commit_group();
          }
        } else {
          __syncwarp();
          const int rows = p.M - row0 < 32 ? p.M - row0 : 32;
          for (int i = 0; i < rows; ++i) {
#pragma unroll
            for (int h = 0; h < kPerBox; h += 32) {
              const int k = lane + h;
              if (bcol + k >= p.N) continue;
              const uint32_t from = box_chunk(box, i, k * kEsize / 16) + (k * kEsize & 15);
              TY* to = static_cast<TY*>(p.y) + static_cast<int64_t>(row0 + i) * p.N + bcol + k;
              if constexpr (kEsize == 4) {
                uint32_t w;
                asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w) : "r"(from) : "memory");
                *reinterpret_cast<uint32_t*>(to) = w;
              } else {
                uint16_t w;
                asm volatile("ld.shared.b16 %0, [%1];" : "=h"(w) : "r"(from) : "memory");
                *reinterpret_cast<uint16_t*>(to) = w;
              }
            }
          }
        }
      };
      auto release = [&] {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(lead(&tmem_empty[buf]));
      };
      if (row0 < p.M) {
        uint32_t ra[32], rb[32];
        tmem_ld_32x32b_x32(tbase, ra);
        tmem_ld_wait();
#pragma unroll 1
        for (int c = 0; c < kChunks; c += 2) {
          tmem_ld_32x32b_x32(tbase + 32 * (c + 1), rb);
          chunk(ra, c);
          tmem_ld_wait();
          if (c + 2 < kChunks) tmem_ld_32x32b_x32(tbase + 32 * (c + 2), ra);
          else release();  // every load of this buffer has landed
          chunk(rb, c + 1);
          tmem_ld_wait();
        }
      } else {
        release();
      }
      if (++buf == 2) {
        buf = 0;
        buf_phase ^= 1;
      }
    }
    if (kTma && lane == 0) bulk_wait_group_all();
    __syncwarp();
  }

  tc_fence_before();
  cluster_sync_all();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, kTmemCols);
  }
}

// ---------------------------------------------------------------- a few tokens
// A CTA takes 16 R channels, its warps consecutive shares of K in blocks of 64,
// whose INT32 sums they add in shared memory (exact in any order). Lane (g, t) =
// (lane / 4, lane % 4) loads bytes 16 t .. 16 t + 15 of the block of rows g and
// g + 8, and of token g of each group of 8: words 2 s and 2 s + 1 are its operands
// of step s of mma.sync.m16n8k32. The order of K within the block is another one
// than the instruction's, the same for both operands.
__device__ __forceinline__ void mma_s8(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

constexpr int kFewWarps = 8;   // most warps of a CTA
constexpr int64_t kFewMost = 32;  // most tokens

struct FewParams {
  const int8_t* xq;
  const float* sx;
  const int8_t* wq;
  const float* sw;
  int M, N, K;
  void* y;
};

// kTok: groups of 8 tokens; R: groups of 16 channels; kU: blocks of K in flight.
template <typename TY, int kTok, int R, int kU>
__global__ void __launch_bounds__(32 * kFewWarps) int8_few_kernel(const FewParams p) {
  extern __shared__ int sums[];  // [warps][8 kTok tokens][16 R channels]
  constexpr int kN = 16 * R, kM = 8 * kTok;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int warps = blockDim.x >> 5;
  const int n0 = static_cast<int>(blockIdx.x) * kN;
  const int nb = (p.K + 63) >> 6;
  const int b0 = nb * warp / warps, b1 = nb * (warp + 1) / warps;
  // rows outside read the last row, whose sums go nowhere
  const int8_t* w[2 * R];
#pragma unroll
  for (int i = 0; i < 2 * R; ++i) {
    const int n = n0 + g + 8 * i;
    w[i] = p.wq + static_cast<int64_t>(n < p.N ? n : p.N - 1) * p.K + 16 * t;
  }
  const int8_t* x[kTok];
#pragma unroll
  for (int i = 0; i < kTok; ++i) x[i] = p.xq + static_cast<int64_t>(g + 8 * i < p.M ? g + 8 * i : p.M - 1) * p.K + 16 * t;
  pdl_wait_primary();
  pdl_launch_dependents();
  int acc[R][kTok][4] = {};
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  for (int b = b0; b < b1; b += kU) {
    uint4 wv[kU][2 * R], xv[kU][kTok];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int k = (b + u) * 64;
      const bool in = b + u < b1 && k + 16 * t < p.K;  // K is a multiple of 16
#pragma unroll
      for (int i = 0; i < 2 * R; ++i) wv[u][i] = in ? __ldg(reinterpret_cast<const uint4*>(w[i] + k)) : zero;
#pragma unroll
      for (int i = 0; i < kTok; ++i) xv[u][i] = in ? __ldg(reinterpret_cast<const uint4*>(x[i] + k)) : zero;
    }
#pragma unroll
    for (int u = 0; u < kU; ++u)
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const uint4 a = wv[u][2 * r], c = wv[u][2 * r + 1];
#pragma unroll
        for (int i = 0; i < kTok; ++i) {
          mma_s8(acc[r][i], a.x, c.x, a.y, c.y, xv[u][i].x, xv[u][i].y);
          mma_s8(acc[r][i], a.z, c.z, a.w, c.w, xv[u][i].z, xv[u][i].w);
        }
      }
  }
  int* mine = sums + warp * kN * kM;
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int i = 0; i < kTok; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        // row g (+ 8), tokens 2 t and 2 t + 1
        const int n = 16 * r + g + (j >> 1) * 8, m = 8 * i + 2 * t + (j & 1);
        mine[m * kN + n] = acc[r][i][j];
      }
  __syncthreads();
  for (int i = threadIdx.x; i < kN * kM; i += blockDim.x) {
    const int n = n0 + i % kN, m = i / kN;
    if (m >= p.M || n >= p.N) continue;
    int s = 0;
    for (int v = 0; v < warps; ++v) s += sums[v * kN * kM + i];
    store1(static_cast<TY*>(p.y) + static_cast<int64_t>(m) * p.N + n,
           __int2float_rn(s) * __fmul_rn(__ldg(p.sx + m), __ldg(p.sw + n)));
  }
}

// ---------------------------------------------------------------- values for the gradients
struct ValuesParams {
  const uint2* q[2];      // codes of the two operands (null: not wanted)
  const float* scale[2];
  uint4* out[2];
  int64_t chunks[2];      // of 8 codes
  int per_row;
  float* one;
};

__global__ void __launch_bounds__(256) int8_values_kernel(const ValuesParams p) {
  pdl_wait_primary();
  pdl_launch_dependents();
  constexpr int kU = 4;
  const int64_t T = static_cast<int64_t>(gridDim.x) * 256, t = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (t == 0) *p.one = 1.0f;
#pragma unroll
  for (int o = 0; o < 2; ++o) {
    const int64_t n = p.chunks[o];
    const bool narrow = n <= 0xFFFFFFFFll;  // the row by a 32-bit division
    for (int64_t i0 = t; i0 < n; i0 += kU * T) {
      uint2 c[kU];
      float s[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int64_t i = i0 + u * T;
        if (i < n) {
          c[u] = __ldg(p.q[o] + i);
          s[u] = __ldg(p.scale[o] + (narrow ? static_cast<int64_t>(static_cast<uint32_t>(i) / static_cast<uint32_t>(p.per_row))
                                            : i / p.per_row));
        }
      }
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int64_t i = i0 + u * T;
        if (i < n) {
          f32x2 v[4];
          act8_values8(c[u], s[u], v);
          p.out[o][i] = make_uint4(pack_bf16x2(v[0]), pack_bf16x2(v[1]), pack_bf16x2(v[2]), pack_bf16x2(v[3]));
        }
      }
    }
  }
}

// ---------------------------------------------------------------- host side

bool make_map(CUtensorMap* m, const void* base, CUtensorMapDataType type, uint64_t inner, uint64_t outer,
              uint64_t row_bytes, uint32_t box_inner, uint32_t box_outer) {
  static const PFN_cuTensorMapEncodeTiled_v12000 encode = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  }();
  if (!encode) return false;
  const cuuint64_t dims[2] = {inner, outer}, strides[1] = {row_bytes};
  const cuuint32_t box[2] = {box_inner, box_outer}, steps[2] = {1, 1};
  return encode(m, type, 2, const_cast<void*>(base), dims, strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename TY, int BN, bool kTma>
cudaError_t launch_tiles(const CUtensorMap (&maps)[3], const TileParams& p, cudaStream_t s) {
  auto kernel = int8_tile_kernel<TY, BN, kTma>;
  constexpr int kSmem = Geo<BN>::kSmemBytes;
  static int pairs_of[64] = {};  // pairs resident at once, by device
  int dev = 0;
  cudaGetDevice(&dev);
  int pairs = dev >= 0 && dev < 64 ? pairs_of[dev] : 0;
  if (!pairs) {
    if (cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem); e != cudaSuccess)
      return e;
    pairs = device_sm_count() / 2;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(2 * pairs);
    cfg.blockDim = dim3(kTileThreads);
    cfg.dynamicSmemBytes = kSmem;
    int clusters = 0;
    if (cudaOccupancyMaxActiveClusters(&clusters, kernel, &cfg) == cudaSuccess && clusters > 0 && clusters < pairs)
      pairs = clusters;
    cudaGetLastError();
    if (dev >= 0 && dev < 64) pairs_of[dev] = pairs;
  }
  const int n = p.ntiles < pairs ? p.ntiles : pairs;
  return launch_pdl(kernel, dim3(2 * n), dim3(kTileThreads), kSmem, s, maps[0], maps[1], maps[2], p);
}

template <typename TY>
cudaError_t forward_tiles(const int8_t* xq, const int8_t* wq, TileParams p, cudaStream_t s) {
  p.tiles_m = (p.M + kRows - 1) / kRows;
  // narrow tiles where they still find a pair each: twice the SMs share the
  // weights' loads
  const int narrow = p.tiles_m * ((p.N + 127) / 128);
  const bool half = narrow <= device_sm_count() / 2;
  const int bn = half ? 128 : 256;
  p.ntiles = p.tiles_m * ((p.N + bn - 1) / bn);
  const bool tma = static_cast<int64_t>(p.N) * sizeof(TY) % 16 == 0;
  CUtensorMap maps[3] = {};
  if (!make_map(&maps[0], xq, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.K, p.M, p.K, kBlockK, 128) ||
      !make_map(&maps[1], wq, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.K, p.N, p.K, kBlockK, bn / 2) ||
      (tma && !make_map(&maps[2], p.y, sizeof(TY) == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                        p.N, p.M, static_cast<uint64_t>(p.N) * sizeof(TY), 128 / sizeof(TY), 32)))
    return cudaErrorInvalidValue;
  if (half) return tma ? launch_tiles<TY, 128, true>(maps, p, s) : launch_tiles<TY, 128, false>(maps, p, s);
  return tma ? launch_tiles<TY, 256, true>(maps, p, s) : launch_tiles<TY, 256, false>(maps, p, s);
}

template <typename TY, int kTok, int R, int kU>
cudaError_t launch_few(const FewParams& p, cudaStream_t s) {
  auto kernel = int8_few_kernel<TY, kTok, R, kU>;
  constexpr size_t kPerWarp = static_cast<size_t>(16 * R) * 8 * kTok * sizeof(int);
  static bool done[64] = {};
  if (cudaError_t e = allow_smem(kernel, kPerWarp * kFewWarps, done); e != cudaSuccess) return e;
  const int nb = (p.K + 63) / 64;
  int warps = kFewWarps;
  while (warps > 1 && 2 * warps > nb) warps /= 2;  // two blocks of K per warp at least
  return launch_pdl(kernel, dim3((p.N + 16 * R - 1) / (16 * R)), dim3(32 * warps), kPerWarp * warps, s, p);
}

template <typename TY>
cudaError_t forward_few(const FewParams& p, cudaStream_t s) {
  if (p.M <= 8) return launch_few<TY, 1, 1, 4>(p, s);
  if (p.M <= 16) return launch_few<TY, 2, 1, 4>(p, s);
  return launch_few<TY, 4, 1, 2>(p, s);
}

size_t align256(size_t n) { return (n + 255) & ~size_t(255); }

}  // namespace

cudaError_t launch_int8_forward(const int8_t* xq, const float* sx, const int8_t* wq, const float* sw, int64_t M,
                                int64_t N, int64_t K, void* y, int y_f32, int* err, cudaStream_t s) {
  if (M <= kFewMost) {
    FewParams p{xq, sx, wq, sw, static_cast<int>(M), static_cast<int>(N), static_cast<int>(K), y};
    return y_f32 ? forward_few<float>(p, s) : forward_few<__nv_bfloat16>(p, s);
  }
  TileParams p{};
  p.M = static_cast<int>(M);
  p.N = static_cast<int>(N);
  p.K = static_cast<int>(K);
  p.sx = sx;
  p.sw = sw;
  p.y = y;
  p.err = err;
  return y_f32 ? forward_tiles<float>(xq, wq, p, s) : forward_tiles<__nv_bfloat16>(xq, wq, p, s);
}

// The values of x and of w in bf16, the factor 1, dX's partial sums.
size_t int8_backward_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  return align256(static_cast<size_t>(M) * K * 2) + align256(static_cast<size_t>(N) * K * 2) + 256 +
         linear_grad_sum_bytes(M, N, K);
}

cudaError_t launch_int8_backward(const void* dY, const int8_t* xq, const float* sx, const int8_t* wq, const float* sw,
                                 int64_t M, int64_t N, int64_t K, void* dX, void* dW, int dw_is_f32, int accumulate,
                                 void* workspace, int* err, cudaStream_t s) {
  if (M == 0) {
    if (dW && !accumulate) return cudaMemsetAsync(dW, 0, static_cast<size_t>(N) * K * (dw_is_f32 ? 4 : 2), s);
    return cudaSuccess;
  }
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  uint8_t* x = ws;
  uint8_t* w = x + align256(static_cast<size_t>(M) * K * 2);
  float* one = reinterpret_cast<float*>(w + align256(static_cast<size_t>(N) * K * 2));
  ValuesParams v{};
  v.q[0] = reinterpret_cast<const uint2*>(xq);
  v.q[1] = reinterpret_cast<const uint2*>(wq);
  v.scale[0] = sx;
  v.scale[1] = sw;
  v.out[0] = reinterpret_cast<uint4*>(x);
  v.out[1] = reinterpret_cast<uint4*>(w);
  v.chunks[0] = dW ? M * K / 8 : 0;
  v.chunks[1] = dX ? N * K / 8 : 0;
  v.per_row = static_cast<int>(K / 8);
  v.one = one;
  const int64_t most = v.chunks[0] > v.chunks[1] ? v.chunks[0] : v.chunks[1];
  const int64_t want = (most + 1023) / 1024, cap = static_cast<int64_t>(8) * device_sm_count();
  if (cudaError_t e = launch_pdl(int8_values_kernel, dim3(static_cast<unsigned>(want < cap ? want : cap)), dim3(256), 0, s, v);
      e != cudaSuccess)
    return e;
  return launch_linear_grads(dY, x, w, M, N, K, dX, dW, dw_is_f32, accumulate, one,
                             reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(one) + 256), err, s);
}

}  // namespace bl
