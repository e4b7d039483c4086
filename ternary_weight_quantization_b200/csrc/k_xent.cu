// The LM head and its softmax cross-entropy over a large vocabulary, forward
// and backward, without the logits in memory (X1, X2).
//
//   z = h W^T           lse = log sum_v exp z       loss = lse - z[target]
//   dz = dloss (exp(z - lse) - [target])            dH = dz W      dW = dz^T h
//
// Three phases of one persistent CTA-pair GEMM template (bf16 operands, fp32
// accumulators in TMEM, tcgen05.mma cta_group::2):
//
//                D rows x columns   A            B            reduction  epilogue
//   Lse          tokens x vocab     h  K-major   W  K-major   K          max and sum of exp of the tile's columns, per token
//   Dz           tokens x vocab     h  K-major   W  K-major   K          dz of a vocabulary piece, bf16 (two terms for fp32 dW)
//   Grad: dH     tokens x K         dz K-major   W  MN-major  vocab      bf16, or fp32 partial sums over pieces and slices
//   Grad: dW     vocab x K          dz MN-major  h  MN-major  tokens     bf16 or fp32; of a linear with few tiles, fp32 sums over slices
//
// The backward walks the vocabulary in pieces: Dz forms the piece's logits
// again and leaves its dz in the workspace (128 MiB at most), Grad multiplies it
// into dH and dW. Nothing of size tokens x vocabulary is
// kept. That costs one product more than the three (z, dH, dW) the operator
// cannot do without; keeping lse from the forward saves the second one.
//
// A pair tile is 256 x 256; every operand tile is 128 rows x 64 of the
// reduction per CTA (two TMA boxes of 64 x 64, 128-byte swizzled: only the
// coordinates and the descriptors differ between K-major and MN-major). With
// 5 to 7 stages of 32 KB and two TMEM accumulators the tensor cores do not wait
// for an epilogue unless it takes longer than its tile's products: for Lse and Dz,
// with their exponentials, up to K of about 384 (forward of 2048 tokens, vocabulary
// 9472, four even waves: 17 to 18 us from K 192 to 384, 20.4 at 512, 31 at 1024).
// All bounds are handled by TMA: rows and columns outside a tensor load as zeros
// and are not stored.
//
// Roles (384 threads per CTA): warp 0 loads, warp 1 issues the MMAs (one lane
// of the leader CTA), warps 2 and 3 do side work on whole rows (the target's
// logit; h without the left-out rows), warps 4..11 are the epilogue (two per
// TMEM lane quadrant, half the columns each; thread = row of D, so a token's
// softmax statistics stay in one thread). Every wait is bounded: on expiry a
// CTA records a timeout in the device error word, tells its peer, drains what it
// has in flight, frees TMEM and exits.
//
// What bounds it (B200, 4096 tokens, K 2560, vocabulary 32000): a stage is 512
// cycles of MMA and 32 KB of loads per SM; loads alone take 573 cycles, MMAs
// alone 640, both together 690, so the two share the SM's memory path. Lse runs
// at 0.95 of the measured bf16 peak (ncu: 425 us), Dz at 0.97 and Grad at 0.9 of
// it (busiest pair 576 of 553 stages on average); back to back the step is held
// by the power cap at 0.90 of the sustained rate. Whole calls, forward + backward,
// back to back in a graph: 2048 tokens, K 512, vocabulary 8192 in 73 us (1.8 x the
// time of four products at the peak: 256 tiles on 74 pairs are four waves for 3.46
// waves of work, and each of five launches has its own start and end), 4096, 2560,
// 32000 in 2.05 to 2.11 ms; the forward alone at 2048, 2560, 131072 in 1.03 to 1.04
// ms (1320 to 1337 TFLOP/s).
// With few tiles the time is a tile's own: about 6 us of launch, fill and epilogue
// and 0.3 us per stage. Up to 16 tokens have kernels of their own
// (k_xent_few.cu).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <cstdint>
#include <type_traits>

#include "bl_act8.cuh"
#include "bl_device.cuh"
#include "bl_internal.h"
#include "bl_mma.cuh"

namespace bl {
namespace {

enum class Phase { Lse, Dz, Grad };

constexpr int kWarpLoad = 0, kWarpMma = 1, kWarpEpi0 = 4;
constexpr int kTile = 256;              // rows (and, where BN says nothing else, columns) of a pair tile
constexpr int kBlockR = 64;             // reduction per stage
constexpr int kBox = 8192;              // one 64 x 64 bf16 box
constexpr int kStageBytes = 4 * kBox;   // A and B: two boxes each
constexpr uint32_t kTmemCols = 512;     // two accumulators of 256 columns
constexpr int kEpiBox = 4096;           // output box: 32 rows x 128 bytes

// Stages, epilogue warps and output boxes per epilogue warp of each phase.
template <Phase P>
struct Geo {
  static constexpr int kStages = P == Phase::Lse ? 7 : P == Phase::Dz ? 5 : 6;
  static constexpr int kEpiWarps = 8;
  static constexpr int kSlots = P == Phase::Lse ? 0 : P == Phase::Dz ? 2 : 1;
  static constexpr int kParts = kEpiWarps / 4;        // warps that share a TMEM lane quadrant
  static constexpr int kThreads = 32 * (kWarpEpi0 + kEpiWarps);
  static constexpr int kOffEpi = kStages * kStageBytes;
  static constexpr int kOffBar = kOffEpi + kEpiWarps * kSlots * kEpiBox;
  static constexpr int kNumBars = 2 * kStages + 5;    // full, empty, tmem_full[2], tmem_empty[2], done
  static constexpr int kOffMisc = kOffBar + kNumBars * 8;
  // TMEM base, abort flag; epilogue maxima at 64
  static constexpr int kSmemBytes = kOffMisc + 128 + 1024 /*base alignment*/;
  static_assert(kSmemBytes <= 232448, "shared memory budget");
};

constexpr float kLog2e = 1.4426950408889634f;

struct XentParams {
  int M, V, K;
  int v0, vcount;        // this piece of the vocabulary
  const int64_t* targets;
  int* err;
  // The pairs' tiles: `ntiles_a` tiles taken round robin, then `ntiles_b`
  // cheaper ones, of which the pairs without a last tile of the first kind
  // (from `split_pair` on) take `more` each, before the others continue.
  int ntiles_a, ntiles_b, split_pair, more;
  int tiles_m, tiles_k;  // tiles over tokens and over K
  // Lse
  float2* part;          // [2 per vocab tile][M]: (maximum, sum) of half its columns, see LseState
  float2* tlogit;        // [M]: the target's logit, as the tile has it and as an fp32 dot product
  const uint4* W;        // rows of W
  // Dz
  const float* lse;
  const float* dloss;
  float* scale;          // max |dloss| of the tokens that count
  int find_scale;        // first piece: form it; later ones read it
  int split;             // dz also as its bf16 remainder
  const uint4* h;        // rows of h, copied to hm with left-out rows cleared
  uint4* hm;             // (first piece only, else null)
  // Grad
  int ntiles_h;          // tiles of dH (all slices); the rest are dW's
  int dw_first;          // dW's tiles are the costlier ones
  int cost_a, cost_b;    // k-blocks of a tile of either kind
  int slices;            // the reduction of dH is split over this many partial sums
  int rows_pad;          // rows between the slices' partial sums
  int h_f32;             // dH goes to the fp32 partial sums (else straight to bf16)
  int h_add;             // ... and is added to them (later pieces)
  int t0, tcount;        // tokens of this launch's share of dW
  int w_f32, w_add;      // dW is fp32; dW adds to its contents
  int w_slices, w_rows;  // the reduction of dW is split over this many fp32 partial sums (1: none), rows between them
  void* dW;              // for the bf16 sums that read dW back
};

struct Tile {
  int cls;         // Grad: 0 dH, 1 dW
  int a0, b0;      // first A row and B row of the pair tile
  int kb0, nkb;    // k-blocks
  int slice;
};

// The pair's i-th tile (false: none left).
__device__ __forceinline__ bool next_tile(const XentParams& p, int pair, int npairs, int i, int& u) {
  u = i * npairs + pair;
  if (u < p.ntiles_a) return true;
  const int own = pair < p.ntiles_a ? (p.ntiles_a - 1 - pair) / npairs + 1 : 0;
  const int j = i - own;  // its j-th tile of the second kind
  if (pair >= p.split_pair) {
    u = j * (npairs - p.split_pair) + pair - p.split_pair;
    if (j >= p.more) return false;
  } else {
    u = p.more * (npairs - p.split_pair) + j * p.split_pair + pair;
  }
  if (u >= p.ntiles_b) return false;
  u += p.ntiles_a;
  return true;
}

template <Phase P, int BN>
__device__ __forceinline__ Tile decode(const XentParams& p, int u) {
  Tile t{};
  if constexpr (P != Phase::Grad) {
    // tokens fastest: the pairs at work share few tiles of W, and h stays in L2
    t.a0 = (u % p.tiles_m) * kTile;
    t.b0 = (u / p.tiles_m) * BN;
    t.nkb = (p.K + kBlockR - 1) / kBlockR;
    return t;
  }
  // dH's tiles come first unless dW's are the costlier ones
  if (p.dw_first) u = u < p.ntiles_a ? u + p.ntiles_h : u - p.ntiles_a;
  if (u < p.ntiles_h) {
    const int per = p.tiles_m * p.tiles_k;
    t.slice = u / per;
    u -= t.slice * per;
    t.a0 = (u / p.tiles_k) * kTile;
    t.b0 = (u % p.tiles_k) * kTile;
    const int nkb = (p.vcount + kBlockR - 1) / kBlockR;
    t.kb0 = static_cast<int>(static_cast<int64_t>(nkb) * t.slice / p.slices);
    t.nkb = static_cast<int>(static_cast<int64_t>(nkb) * (t.slice + 1) / p.slices) - t.kb0;
  } else {
    u -= p.ntiles_h;
    t.cls = 1;
    t.nkb = (p.tcount + kBlockR - 1) / kBlockR;
    if (p.w_slices > 1) {
      const int per = (p.vcount + kTile - 1) / kTile * p.tiles_k, nkb = t.nkb;
      t.slice = u / per;
      u -= t.slice * per;
      t.kb0 = static_cast<int>(static_cast<int64_t>(nkb) * t.slice / p.w_slices);
      t.nkb = static_cast<int>(static_cast<int64_t>(nkb) * (t.slice + 1) / p.w_slices) - t.kb0;
    }
    t.a0 = (u / p.tiles_k) * kTile;
    t.b0 = (u % p.tiles_k) * kTile;
    if (p.split) t.nkb *= 2;  // the remainders first, while the sums are small
  }
  return t;
}

// Instruction descriptors and descriptor steps (16-byte units per 16 of the
// reduction): K-major 32 bytes along the row, MN-major 16 rows.
__host__ __device__ constexpr uint32_t idesc(int a_mn, int b_mn, int bn) {
  return make_idesc(1 /*f32*/, 1 /*bf16*/, a_mn, b_mn, kTile, bn);
}

__device__ __forceinline__ uint64_t operand_desc(uint32_t saddr, bool mn) {
  return smem_desc_sw128(saddr, mn ? kBox : 16, 1024);
}

template <bool kAMn, bool kBMn, int BN>
__device__ __forceinline__ void mma_stage(uint32_t d_tmem, uint64_t ad, uint64_t bd, int kb) {
  constexpr uint64_t as = kAMn ? 128 : 2, bs = kBMn ? 128 : 2;
#pragma unroll
  for (int kk = 0; kk < 4; ++kk)
    mma_f16_pair(d_tmem, ad + kk * as, bd + kk * bs, idesc(kAMn, kBMn, BN), (kb | kk) != 0);
}

// tma_load_2d_pair to a shared-memory address.
__device__ __forceinline__ void load_pair(const CUtensorMap* map, uint32_t bar_cluster, uint32_t dst, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], "
      "[%2];" ::"r"(dst),
      "l"(map), "r"(bar_cluster), "r"(x), "r"(y)
      : "memory");
}

// As tma_store_2d, adding the tile's fp32 values to what the tensor holds
// (each element one rounded fp32 addition at L2).
__device__ __forceinline__ void tma_add_2d(const CUtensorMap* map, uint32_t src_smem, int x, int y) {
  asm volatile("cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(map),
               "r"(src_smem), "r"(x), "r"(y)
               : "memory");
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void st_shared_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// 16-byte chunk j of row `lane` of a 32 x 128 byte box, 128-byte swizzled.
__device__ __forceinline__ uint32_t box_chunk(uint32_t box, int lane, int j) {
  return box + static_cast<uint32_t>(lane) * 128u + (static_cast<uint32_t>(j ^ (lane & 7)) << 4);
}

// An epilogue warp's output staging: kSlots boxes used in turn.
template <int kSlots>
struct Stager {
  uint32_t base;
  uint32_t seq;
  int lane;
  // A box whose last store has been read. kOpen: boxes taken before this one
  // whose stores are still to be issued.
  template <int kOpen = 0>
  __device__ __forceinline__ uint32_t next() {
    if (lane == 0) bulk_wait_group_read<kSlots - 1 - kOpen>();
    __syncwarp();
    return base + (seq++ % kSlots) * kEpiBox;
  }
  // (The box's first row lies inside the tensor: see `any`.)
  __device__ __forceinline__ void store(const CUtensorMap* map, uint32_t box, int x, int y, bool add) {
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      if (add) tma_add_2d(map, box, x, y);
      else tma_store_2d(map, box, x, y);
      bulk_commit_group();
    }
  }
};

// ---- Lse: running maximum and sum over the tile's columns of one token. The
// maximum is kept as m = fl(z log2 e) and the sum relative to 2^m, here and in
// the joins: rescaling takes ex2 of the difference of two such numbers, which is
// exactly 1 where the maximum stays. (With z kept instead, every join left the
// rounding of z log2 e in the sum, always to the same side.)
struct LseState {
  float m, s;
  __device__ __forceinline__ void chunk(uint32_t (&r)[32], int valid) {
    if (valid < 32) {
#pragma unroll
      for (int j = 0; j < 32; ++j) r[j] = j < valid ? r[j] : 0xFF800000u;  // -inf
    }
    float c = __uint_as_float(r[0]);
#pragma unroll
    for (int j = 1; j < 32; ++j) c = fmaxf(c, __uint_as_float(r[j]));
    const float n = fmaxf(m, c * kLog2e);
    // an empty maximum (all -inf) leaves exp(-inf - 0) = 0
    const float nl = n == __uint_as_float(0xFF800000u) ? 0.0f : n;
    float a0 = 0.0f, a1 = 0.0f;
#pragma unroll
    for (int j = 0; j < 32; j += 2) {
      a0 += ex2(fmaf(__uint_as_float(r[j]), kLog2e, -nl));
      a1 += ex2(fmaf(__uint_as_float(r[j + 1]), kLog2e, -nl));
    }
    s = fmaf(s, ex2(m - nl), a0 + a1);
    m = n;
  }
};

// Boxes of 64 rows, of the `most` that a CTA's share of an operand has, that
// hold rows below `limit`.
__device__ __forceinline__ int boxes(int limit, int row, int most) {
  const int n = (limit - row + 63) >> 6;
  return n < 0 ? 0 : n < most ? n : most;
}

// What CTA `rank` loads per stage in the logit phases: the boxes of A and of B
// that hold rows. The others are left out: rows of A and of B reach only their
// own rows and columns of D, which are not used there. (In Grad the tests cost
// more than they save: 4096 tokens, K 2560, vocabulary 32000: 2.34 ms with them,
// 2.26 without.) A CTA without any loads one all the same, of zeros or of rows
// that are not used: the leader's stages fill only with both CTAs' boxes, which is
// what keeps its loader from running rounds ahead of the peer's, whose waits tell
// one round from the next by a single bit.
template <int BN>
struct CtaBoxes {
  int a, b;
  __device__ __forceinline__ CtaBoxes(const XentParams& p, const Tile& t, int rank)
      : a(boxes(p.M, t.a0 + rank * 128, 2)), b(boxes(p.vcount, t.b0 + rank * (BN / 2), BN / 128)) {
    if (a + b == 0) b = 1;
  }
};

template <Phase P, int BN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(Geo<P>::kThreads, 1)
    xent_kernel(const __grid_constant__ CUtensorMap map_h, const __grid_constant__ CUtensorMap map_w,
                const __grid_constant__ CUtensorMap map_dz, const __grid_constant__ CUtensorMap map_dz_lo,
                const __grid_constant__ CUtensorMap out0, const __grid_constant__ CUtensorMap out1,
                const __grid_constant__ XentParams p) {
  using G = Geo<P>;
  static_assert(BN == 256 || (BN == 128 && P != Phase::Grad), "tile widths");
  constexpr int kChunks = BN / 32 / G::kParts;  // 32-column chunks of an epilogue warp
  constexpr int kStages = G::kStages, kEpiWarps = G::kEpiWarps;
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
    // the descriptors' fetch overlaps the set-up
    prefetch_tensormap(&map_h);
    prefetch_tensormap(&map_w);
    if constexpr (P == Phase::Grad) prefetch_tensormap(&map_dz);
    if (P == Phase::Grad && p.split) prefetch_tensormap(&map_dz_lo);
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
  if (warp == kWarpMma) {
    tmem_alloc_pair(tmem_holder, kTmemCols);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;
  pdl_wait_primary();
  pdl_launch_dependents();

  // a warp's; a failed wait also stops the peer CTA's
  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    if (mbar_wait_warp(bar, parity, abort_flag, p.err)) return true;
    st_cluster_u32(map_to_rank(smem_u32(const_cast<int*>(abort_flag)), rank ^ 1u), 1u);
    return false;
  };
  auto lead = [&](uint64_t* bar) -> uint32_t { return map_to_rank(smem_u32(bar), 0); };

  if (warp == kWarpLoad) {
    const bool one = elect_one();
    int stage = 0;
    uint32_t phase = 0, issued = 0;  // stages requested so far
    const uint32_t bars = lead(full), smem0 = smem_u32(smem);
    bool ok = true;
    int u;
    for (int i = 0; ok && next_tile(p, pair, npairs, i, u); ++i) {
      const Tile t = decode<P, BN>(p, u);
      const int a0 = t.a0 + static_cast<int>(rank) * 128, b0 = t.b0 + static_cast<int>(rank) * (BN / 2);
      // both CTAs' boxes arrive on the leader's barrier
      uint32_t bytes = 2 * kStageBytes;
      int na = 2, nb = 2;
      if constexpr (P != Phase::Grad) {
        const CtaBoxes<BN> first(p, t, 0), second(p, t, 1);
        na = leader ? first.a : second.a;
        nb = leader ? first.b : second.b;
        bytes = kBox * (first.a + first.b + second.a + second.b);
      }
      // one loop per kind of tile: a stage must be requested in the few hundred
      // cycles that the tensor cores take for one
      auto each = [&](int n, auto load) {
        for (int kb = 0; kb < n; ++kb) {
          if (!wait(&empty[stage], phase ^ 1)) {
            ok = false;
            return;
          }
          if (one) {
            if (leader) mbar_arrive_expect_tx(&full[stage], bytes);
            load(kb, bars + 8 * stage, smem0 + stage * kStageBytes);
          }
          __syncwarp();
          ++issued;
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1;
          }
        }
      };
      // K-major: (reduction, row); MN-major: (row, reduction)
      if constexpr (P != Phase::Grad) {
        const int w0 = p.v0 + b0;
        if (na == 2 && nb == BN / 128) {
          each(t.nkb, [&](int kb, uint32_t bar, uint32_t sa) {
            const int k0 = kb * kBlockR;
#pragma unroll
            for (int j = 0; j < 2; ++j) load_pair(&map_h, bar, sa + j * kBox, k0, a0 + 64 * j);
#pragma unroll
            for (int j = 0; j < BN / 128; ++j) load_pair(&map_w, bar, sa + (2 + j) * kBox, k0, w0 + 64 * j);
          });
        } else {
          each(t.nkb, [&](int kb, uint32_t bar, uint32_t sa) {
            const int k0 = kb * kBlockR;
#pragma unroll
            for (int j = 0; j < 2; ++j)
              if (j < na) load_pair(&map_h, bar, sa + j * kBox, k0, a0 + 64 * j);
#pragma unroll
            for (int j = 0; j < BN / 128; ++j)
              if (j < nb) load_pair(&map_w, bar, sa + (2 + j) * kBox, k0, w0 + 64 * j);
          });
        }
      } else if (t.cls == 0) {
        const int v0 = t.kb0 * kBlockR;
        each(t.nkb, [&](int kb, uint32_t bar, uint32_t sa) {
          const int v = v0 + kb * kBlockR;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            load_pair(&map_dz, bar, sa + j * kBox, v, a0 + 64 * j);
            load_pair(&map_w, bar, sa + (2 + j) * kBox, b0 + 64 * j, p.v0 + v);
          }
        });
      } else {
        auto of = [&](const CUtensorMap* dz) {
          return [&, dz](int kb, uint32_t bar, uint32_t sa) {
            const int m = p.t0 + (t.kb0 + kb) * kBlockR;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              load_pair(dz, bar, sa + j * kBox, a0 + 64 * j, m);
              load_pair(&map_h, bar, sa + (2 + j) * kBox, b0 + 64 * j, m);
            }
          };
        };
        if (p.split) {
          each(t.nkb >> 1, of(&map_dz_lo));
          if (ok) each(t.nkb >> 1, of(&map_dz));
        } else {
          each(t.nkb, of(&map_dz));
        }
      }
    }
    if (one && leader && (!ok || *abort_flag)) {
      // let every copy already issued land before the pair exits: the last
      // request of each stage that was requested at all
      const unsigned long long deadline = globaltimer_ns() + kWaitLimitNs;
      for (uint32_t s = 0; s < kStages && s < issued; ++s)
        mbar_drain_until(&full[s], (issued - s - 1) / kStages & 1, deadline);
    }
    __syncwarp();
  } else if (warp == kWarpMma) {
    if (leader) {
      const bool one = elect_one();
      const uint32_t s0 = smem_u32(smem);
      int stage = 0, buf = 0;
      uint32_t phase = 0, buf_phase = 0;
      bool ok = true;
      int u;
      for (int i = 0; ok && next_tile(p, pair, npairs, i, u); ++i) {
        const Tile t = decode<P, BN>(p, u);
        if (t.nkb == 0) continue;
        if (!wait(&tmem_empty[buf], buf_phase ^ 1)) break;
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(buf * kTile);
        auto each = [&](auto a_mn, auto b_mn) {
          constexpr bool kAMn = decltype(a_mn)::value, kBMn = decltype(b_mn)::value;
          const uint64_t ad0 = operand_desc(s0, kAMn), bd0 = operand_desc(s0 + 2 * kBox, kBMn);
          for (int kb = 0; kb < t.nkb; ++kb) {
            if (!wait(&full[stage], phase)) {
              ok = false;
              return;
            }
            tc_fence_after();
            const uint64_t at = static_cast<uint64_t>(stage) * (kStageBytes >> 4);
            if (one) {
              mma_stage<kAMn, kBMn, BN>(d_tmem, ad0 + at, bd0 + at, kb);
              mma_commit_pair(&empty[stage], 0x3);
            }
            __syncwarp();
            if (++stage == kStages) {
              stage = 0;
              phase ^= 1;
            }
          }
          if (one) mma_commit_pair(&tmem_full[buf], 0x3);
          __syncwarp();
        };
        using K = std::false_type;
        using MN = std::true_type;
        if constexpr (P != Phase::Grad) each(K{}, K{});
        else if (t.cls == 0) each(K{}, MN{});
        else each(MN{}, MN{});
        if (++buf == 2) {
          buf = 0;
          buf_phase ^= 1;
        }
      }
      if (one) mma_commit_pair(done_bar, 0x3);
      __syncwarp();
    }
    if (lane == 0) mbar_drain(done_bar, 0);
    __syncwarp();
  } else if (warp < kWarpEpi0) {
    // The loss is a difference with the target's logit, which the tensor
    // core's sum leaves up to K / 16 steps of fp32 low: these two warps form
    // it again as an fp32 dot product while the tiles run, and the join puts
    // it in the place of the tile's.
    if constexpr (P == Phase::Lse) {
      const int per_row = p.K / 8;
      for (int m = static_cast<int>(blockIdx.x) * 2 + warp - 2; m < p.M; m += 2 * static_cast<int>(gridDim.x)) {
        const int64_t t = __ldg(p.targets + m);
        if (t < 0 || t >= p.V) continue;
        const uint4* a = p.h + static_cast<int64_t>(m) * per_row;
        const uint4* b = p.W + t * per_row;
        float z0 = 0.0f, z1 = 0.0f;
#pragma unroll 4
        for (int i = lane; i < per_row; i += 32) {
          const uint4 x = __ldg(a + i), y = __ldg(b + i);
          const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            z0 = fmaf(bf16_lo(xs[j]), bf16_lo(ys[j]), z0);
            z1 = fmaf(bf16_hi(xs[j]), bf16_hi(ys[j]), z1);
          }
        }
        float z = z0 + z1;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
        if (lane == 0) p.tlogit[m].y = z;
      }
    }
    if constexpr (P == Phase::Dz) {
      if (p.hm) {
        // h with the left-out rows cleared, for dW (0 * NaN would be NaN)
        const int64_t n = static_cast<int64_t>(p.M) * (p.K / 8);
        const int64_t T = static_cast<int64_t>(gridDim.x) * 64;
        const uint32_t per_row = static_cast<uint32_t>(p.K / 8);
        const bool narrow = n <= 0xFFFFFFFFll;
        constexpr int kU = 8;
        for (int64_t i0 = static_cast<int64_t>(blockIdx.x) * 64 + (threadIdx.x - 64); i0 < n; i0 += kU * T) {
          uint4 v[kU];
          int64_t t[kU];
#pragma unroll
          for (int u = 0; u < kU; ++u) {
            const int64_t i = i0 + u * T;
            if (i < n) {
              v[u] = __ldg(p.h + i);
              t[u] = __ldg(p.targets + (narrow ? static_cast<int64_t>(static_cast<uint32_t>(i) / per_row) : i / per_row));
            }
          }
#pragma unroll
          for (int u = 0; u < kU; ++u) {
            const int64_t i = i0 + u * T;
            if (i < n) p.hm[i] = t[u] >= 0 && t[u] < p.V ? v[u] : make_uint4(0u, 0u, 0u, 0u);
          }
        }
      }
    }
  } else {
    const int q = warp & 3, part = (warp - kWarpEpi0) >> 2;
    float scale = 1.0f;
    if constexpr (P == Phase::Dz) {
      // dz is kept relative to the largest |dloss|: its target term -dloss
      // would otherwise round the same way for every token of a mean
      // (dloss = 1 / tokens), an error of up to 2^-8 of the whole gradient.
      // The products' epilogues put the factor back in fp32.
      if (p.find_scale) {
        const int e = threadIdx.x - kWarpEpi0 * 32;
        constexpr int kU = 8;  // tokens in flight per thread
        float top = 0.0f;
        for (int m0 = e; m0 < p.M; m0 += kU * kEpiWarps * 32) {
          int64_t t[kU];
          float a[kU];
#pragma unroll
          for (int i = 0; i < kU; ++i) {
            const int m = m0 + i * kEpiWarps * 32;
            t[i] = m < p.M ? __ldg(p.targets + m) : -1;
            a[i] = m < p.M ? fabsf(__ldg(p.dloss + m)) : 0.0f;
          }
#pragma unroll
          for (int i = 0; i < kU; ++i)
            if (t[i] >= 0 && t[i] < p.V && a[i] < __uint_as_float(0x7F800000u)) top = fmaxf(top, a[i]);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        float* tops = reinterpret_cast<float*>(smem + G::kOffMisc + 64);
        if (lane == 0) tops[warp - kWarpEpi0] = top;
        asm volatile("bar.sync 1, %0;" ::"n"(kEpiWarps * 32) : "memory");
#pragma unroll
        for (int w = 0; w < kEpiWarps; ++w) top = fmaxf(top, tops[w]);
        scale = top > 0.0f ? top : 1.0f;
        if (blockIdx.x == 0 && e == 0) *p.scale = scale;
      } else {
        scale = *p.scale;
      }
    }
    if constexpr (P == Phase::Grad) scale = __ldg(p.scale);
    Stager<G::kSlots> st{smem_u32(smem + G::kOffEpi + (warp - kWarpEpi0) * G::kSlots * kEpiBox), 0u, lane};
    int buf = 0;
    uint32_t buf_phase = 0;
    int u;
    for (int i = 0; next_tile(p, pair, npairs, i, u); ++i) {
      const Tile t = decode<P, BN>(p, u);
      if (t.nkb == 0) continue;
      const int row0 = t.a0 + static_cast<int>(rank) * 128 + q * 32;  // first D row of the warp
      const int row = row0 + lane;
      // the thread's token
      int tgt = -1;
      float nlse = 0.0f, g = 0.0f;
      uint32_t keep = 0u;
      LseState ls{__uint_as_float(0xFF800000u), 0.0f};
      if constexpr (P != Phase::Grad) {
        if (row < p.M) {
          const int64_t tt = __ldg(p.targets + row);
          if (tt >= 0 && tt < p.V) {
            tgt = static_cast<int>(tt) - (p.v0 + t.b0);
            keep = 0xFFFFFFFFu;
            if constexpr (P == Phase::Dz) {
              nlse = -__ldg(p.lse + row) * kLog2e;
              g = __fdiv_rn(__ldg(p.dloss + row), scale);
            }
          }
        }
      }
      if (!wait(&tmem_full[buf], buf_phase)) break;
      tc_fence_after();
      const uint32_t tbase = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + buf * kTile;
      const bool any = row0 < (P == Phase::Grad && t.cls == 1 ? p.vcount : p.M);  // rows of the warp that are used
      uint32_t box = 0, box_lo = 0;
      // one chunk of 32 columns in registers; the next one's TMEM load is
      // under way meanwhile
      auto chunk = [&](uint32_t (&r)[32], int c) {
        const int col = t.b0 + 32 * c;  // first column: of the piece (Lse, Dz) or of K (Grad)
        if constexpr (P == Phase::Lse) {
          if (static_cast<unsigned>(tgt - 32 * c) < 32u) {
            float z = 0.0f;
#pragma unroll
            for (int j = 0; j < 32; ++j) z = j == tgt - 32 * c ? __uint_as_float(r[j]) : z;
            p.tlogit[row].x = z;
          }
          if (p.v0 + col < p.V) ls.chunk(r, p.V - (p.v0 + col));
        } else if constexpr (P == Phase::Dz) {
          if (col >= p.vcount) return;
          const bool here = static_cast<unsigned>(tgt - 32 * c) < 32u;
          float d[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) d[j] = ex2(fmaf(__uint_as_float(r[j]), kLog2e, nlse));
          if (here) {
#pragma unroll
            for (int j = 0; j < 32; ++j) d[j] = j == tgt - 32 * c ? d[j] - 1.0f : d[j];
          }
          // dz to bf16: the type the products take (as the dY of the layer's
          // own backward); with `split` its remainder too, 16 bits in all
          uint32_t hi[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            d[2 * j] *= g;
            d[2 * j + 1] *= g;
            hi[j] = pack_bf16x2(d[2 * j + 1], d[2 * j]);
          }
          if ((c & 1) == 0) box = st.next();
#pragma unroll
          for (int j = 0; j < 4; ++j)
            st_shared_v4(box_chunk(box, lane, (c & 1) * 4 + j), hi[4 * j] & keep, hi[4 * j + 1] & keep,
                         hi[4 * j + 2] & keep, hi[4 * j + 3] & keep);
          const bool last = (c & 1) || col + 32 >= p.vcount;
          if (last) st.store(&out0, box, col & ~63, row0, false);
          if (p.split) {
            if ((c & 1) == 0) box_lo = st.template next<1>();
#pragma unroll
            for (int j = 0; j < 16; ++j)
              hi[j] = pack_bf16x2(d[2 * j + 1] - bf16_hi(hi[j]), d[2 * j] - bf16_lo(hi[j]));
#pragma unroll
            for (int j = 0; j < 4; ++j)
              st_shared_v4(box_chunk(box_lo, lane, (c & 1) * 4 + j), hi[4 * j] & keep, hi[4 * j + 1] & keep,
                           hi[4 * j + 2] & keep, hi[4 * j + 3] & keep);
            if (last) st.store(&out1, box_lo, col & ~63, row0, false);
          }
        } else {
          if (col >= p.K) return;
#pragma unroll
          for (int j = 0; j < 32; ++j) r[j] = __float_as_uint(__uint_as_float(r[j]) * scale);
          const bool f32 = t.cls == 0 ? p.h_f32 != 0 : p.w_f32 != 0 || p.w_slices > 1;
          if (f32) {
            box = st.next();
#pragma unroll
            for (int j = 0; j < 8; ++j) st_shared_v4(box_chunk(box, lane, j), r[4 * j], r[4 * j + 1], r[4 * j + 2], r[4 * j + 3]);
            if (t.cls == 0) st.store(&out0, box, col, t.slice * p.rows_pad + row0, p.h_add != 0);
            else st.store(&out1, box, col, p.v0 + t.slice * p.w_rows + row0, p.w_add != 0);
          } else {
            if (t.cls == 1 && p.w_add && row < p.vcount) {
              // one rounding: the bf16 contents are added to the fp32 sum
              const uint4* old = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.dW) +
                                                                static_cast<int64_t>(p.v0 + row) * p.K + col);
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                if (col + 8 * j < p.K) {
                  const uint4 o = old[j];
                  const uint32_t w[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
                  for (int i = 0; i < 4; ++i) {
                    r[8 * j + 2 * i] = __float_as_uint(__uint_as_float(r[8 * j + 2 * i]) + bf16_lo(w[i]));
                    r[8 * j + 2 * i + 1] = __float_as_uint(__uint_as_float(r[8 * j + 2 * i + 1]) + bf16_hi(w[i]));
                  }
                }
              }
            }
            if ((c & 1) == 0) box = st.next();
#pragma unroll
            for (int j = 0; j < 4; ++j)
              st_shared_v4(box_chunk(box, lane, (c & 1) * 4 + j),
                           pack_bf16x2(__uint_as_float(r[8 * j + 1]), __uint_as_float(r[8 * j])),
                           pack_bf16x2(__uint_as_float(r[8 * j + 3]), __uint_as_float(r[8 * j + 2])),
                           pack_bf16x2(__uint_as_float(r[8 * j + 5]), __uint_as_float(r[8 * j + 4])),
                           pack_bf16x2(__uint_as_float(r[8 * j + 7]), __uint_as_float(r[8 * j + 6])));
            if ((c & 1) || col + 32 >= p.K) {
              if (t.cls == 0) st.store(&out0, box, col & ~63, row0, false);
              else st.store(&out1, box, col & ~63, p.v0 + row0, false);
            }
          }
        }
      };
      constexpr int kLast = kChunks - 1;
      const int first = part * kChunks;
      auto release = [&] {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(lead(&tmem_empty[buf]));
      };
      if (any) {
        uint32_t ra[32], rb[32];
        tmem_ld_32x32b_x32(tbase + 32 * first, ra);
        tmem_ld_wait();
#pragma unroll 1
        for (int c = 0; c < kLast; c += 2) {
          tmem_ld_32x32b_x32(tbase + 32 * (first + c + 1), rb);
          chunk(ra, first + c);
          tmem_ld_wait();
          if (c + 1 < kLast) tmem_ld_32x32b_x32(tbase + 32 * (first + c + 2), ra);
          else release();  // every load of this buffer has landed
          chunk(rb, first + c + 1);
          tmem_ld_wait();
        }
      } else {
        release();
      }
      if constexpr (P == Phase::Lse) {
        if (row < p.M) p.part[static_cast<int64_t>(t.b0 / (BN / 2) + part) * p.M + row] = make_float2(ls.m, ls.s);
      }
      if (++buf == 2) {
        buf = 0;
        buf_phase ^= 1;
      }
    }
    if (lane == 0) bulk_wait_group_all();
    __syncwarp();
  }

  tc_fence_before();
  cluster_sync_all();
  if (warp == kWarpMma) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, kTmemCols);
  }
}

// lse and loss from the vocabulary tiles' (max, sum): kJoinTokens tokens per
// block, the tiles spread over kJoinSplit threads of each token, joined in a
// fixed order. (8 tokens, so that a few thousand tokens fill the SMs and a
// thread has few loads to wait for: at 2048 tokens and 1024 parts 10.8 us with
// 32 tokens and 32 threads each.) With h (the few tokens' forward), the warps
// that the last step leaves idle sum the targets' logits in fp32; they need
// nothing of the launch before, which began after all earlier ones had ended.
constexpr int kJoinTokens = 8, kJoinSplit = 64;

__device__ __forceinline__ float2 join_parts(float2 a, float2 b) {
  const float n = fmaxf(a.x, b.x);
  const float nl = n == __uint_as_float(0xFF800000u) ? 0.0f : n;
  return make_float2(n, a.y * ex2(a.x - nl) + b.y * ex2(b.x - nl));
}

__global__ void __launch_bounds__(kJoinTokens* kJoinSplit)
    xent_join_kernel(const float2* __restrict__ part, int tiles, int M, int V, const float2* __restrict__ tlogit,
                     const int64_t* __restrict__ targets, float* loss, float* lse, const __nv_bfloat16* h,
                     const __nv_bfloat16* W, int K) {
  __shared__ float2 sh[kJoinTokens][kJoinSplit + 1];
  __shared__ float target_logit[kJoinTokens];
  if (h && threadIdx.x >= 32 * kJoinTokens) {
    const int w = (threadIdx.x >> 5) - kJoinTokens, lane = threadIdx.x & 31;
    const int m = static_cast<int>(blockIdx.x) * kJoinTokens + w;
    const int64_t t = m < M ? targets[m] : -1;
    if (t >= 0 && t < V) {
      f32x2 a[2] = {};
#pragma unroll 2
      for (int k = lane * 8; k < K; k += 256) {
        Raw8<__nv_bfloat16> x, y;
        x.load(h + static_cast<int64_t>(m) * K + k);
        y.load(W + t * K + k);
        f32x2 xv[4], yv[4];
        x.get(xv);
        y.get(yv);
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i & 1] = fma2(xv[i], yv[i], a[i & 1]);
      }
      float z = sum2(add2(a[0], a[1]));
#pragma unroll
      for (int s = 16; s > 0; s >>= 1) z += __shfl_xor_sync(0xffffffffu, z, s);
      if (lane == 0) target_logit[w] = z;
    }
  }
  pdl_wait_primary();
  pdl_launch_dependents();
  const float2 none = make_float2(__uint_as_float(0xFF800000u), 0.0f);
  const int x = threadIdx.x % kJoinTokens, y = threadIdx.x / kJoinTokens;
  const int m = static_cast<int>(blockIdx.x) * kJoinTokens + x;
  // warp w joins token w's parts at the end; its target is read ahead
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int mm = static_cast<int>(blockIdx.x) * kJoinTokens + warp;
  int64_t t = -1;
  float2 tl = make_float2(0.0f, 0.0f);
  if (warp < kJoinTokens && mm < M && lane == 0) {
    t = targets[mm];
    tl = tlogit[mm];  // not written (and not used) for a left-out token
  }
  float2 a = none;
  if (m < M) {
    constexpr int kU = 4;
    for (int i = y; i < tiles; i += kU * kJoinSplit) {
      float2 v[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u)
        v[u] = i + u * kJoinSplit < tiles ? part[static_cast<int64_t>(i + u * kJoinSplit) * M + m] : none;
#pragma unroll
      for (int u = 0; u < kU; ++u) a = join_parts(a, v[u]);
    }
  }
  sh[x][y] = a;
  __syncthreads();
  if (warp >= kJoinTokens) return;
  a = sh[warp][lane];
#pragma unroll
  for (int i = 32; i < kJoinSplit; i += 32) a = join_parts(a, sh[warp][lane + i]);
#pragma unroll
  for (int s = 16; s > 0; s >>= 1)
    a = join_parts(a, make_float2(__shfl_xor_sync(0xffffffffu, a.x, s), __shfl_xor_sync(0xffffffffu, a.y, s)));
  if (lane == 0 && mm < M) {
    if (h) tl.y = target_logit[warp];
    float l = fmaf(a.x, 0.6931471805599453f, logf(a.y));
    float nll = 0.0f;
    if (t >= 0 && t < V) {
      // the fp32 target logit in the place of the tile's, in lse too: a token
      // whose target holds nearly all of the sum keeps a loss near 0
      const float d = __expf(tl.y - l) - __expf(tl.x - l);
      if (d > -0.5f) l += log1pf(d);
      nll = l - tl.y;
    }
    lse[mm] = l;
    loss[mm] = nll;
  }
}

// dH from the fp32 partial sums of its slices, added in order.
__global__ void __launch_bounds__(256) xent_dh_kernel(const float4* __restrict__ acc, int64_t slice_vecs, int slices,
                                                      int64_t nvecs, uint2* __restrict__ dH) {
  pdl_wait_primary();
  pdl_launch_dependents();
  const int64_t T = static_cast<int64_t>(gridDim.x) * 256;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < nvecs; i += T) {
    float4 v = acc[i];
    for (int s = 1; s < slices; ++s) {
      const float4 w = acc[s * slice_vecs + i];
      v.x += w.x, v.y += w.y, v.z += w.z, v.w += w.w;
    }
    dH[i] = make_uint2(pack_bf16x2(v.y, v.x), pack_bf16x2(v.w, v.z));
  }
}

// ---------------------------------------------------------------- host side

// Tensor map of a row-major 2D array of bf16 (f32: fp32) elements with 128-byte
// swizzled boxes; false when the driver rejects it.
bool make_map(CUtensorMap* m, const void* base, bool f32, uint64_t inner, uint64_t outer, uint64_t row_bytes,
              uint32_t box_inner, uint32_t box_outer) {
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
  return encode(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base),
                dims, strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Spreads the second kind of tiles so that the pairs end together: the least
// end time at which they all fit. With ntiles_a = qP + e, the first e pairs
// are busy with q + 1 of the first kind, the others with q.
void share_tiles(XentParams& p, int npairs) {
  p.split_pair = p.ntiles_a % npairs;
  p.more = 0;
  if (p.ntiles_b == 0) return;
  const int64_t ahead = p.cost_a / p.cost_b;  // tiles of the second kind in one of the first
  const int64_t e = p.split_pair, f = npairs - e;
  int64_t more = p.ntiles_b / npairs;
  while (f * more + (more > ahead ? e * (more - ahead) : 0) < p.ntiles_b) ++more;
  p.more = static_cast<int>(more);
}

template <Phase P, int BN>
cudaError_t launch_phase(const CUtensorMap (&maps)[6], XentParams& p, cudaStream_t s) {
  static int pairs_of[64] = {};  // pairs resident at once, by device
  int dev = 0;
  cudaGetDevice(&dev);
  int pairs = dev >= 0 && dev < 64 ? pairs_of[dev] : 0;
  if (!pairs) {
    if (cudaError_t e = cudaFuncSetAttribute(xent_kernel<P, BN>, cudaFuncAttributeMaxDynamicSharedMemorySize, Geo<P>::kSmemBytes);
        e != cudaSuccess)
      return e;
    pairs = device_sm_count() / 2;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(2 * pairs);
    cfg.blockDim = dim3(Geo<P>::kThreads);
    cfg.dynamicSmemBytes = Geo<P>::kSmemBytes;
    int clusters = 0;
    if (cudaOccupancyMaxActiveClusters(&clusters, xent_kernel<P, BN>, &cfg) == cudaSuccess && clusters > 0 && clusters < pairs)
      pairs = clusters;
    cudaGetLastError();
    if (dev >= 0 && dev < 64) pairs_of[dev] = pairs;
  }
  const int ntiles = p.ntiles_a + p.ntiles_b;
  if (ntiles == 0) return cudaSuccess;
  const int n = ntiles < pairs ? ntiles : pairs;
  share_tiles(p, n);
  return launch_pdl(xent_kernel<P, BN>, dim3(2 * n), dim3(Geo<P>::kThreads), Geo<P>::kSmemBytes, s, maps[0], maps[1],
                    maps[2], maps[3], maps[4], maps[5], p);
}

int tiles_of(int64_t n) { return static_cast<int>((n + kTile - 1) / kTile); }
size_t align256(size_t n) { return (n + 255) & ~size_t(255); }

// Where the backward's parts lie in the workspace, and how it cuts the work.
struct Plan {
  int64_t piece;   // vocabulary columns per piece (a multiple of 256)
  int pieces, slices;
  int64_t rows_pad;
  bool sums;       // dH goes through fp32 partial sums
  size_t off_lo, off_h, off_scale, off_sum, bytes;
};

// dz of a piece: larger pieces mean fewer launches and fewer additions to dH's
// partial sums, smaller ones a smaller workspace. Measured on B200 (backward, 4096
// tokens, K 2560, vocabulary 32000): 32 MiB 1.72 ms, 64 MiB 1.62, 128 MiB 1.57,
// 256 MiB (the whole vocabulary at once) 1.54.
constexpr int64_t kPieceBytes = int64_t(128) << 20;
constexpr int kPlanPairs = kPlanSms / 2;
constexpr int kF32Tokens = 1024;  // tokens per partial sum of an fp32 dW

// dH has few tiles, each with the whole piece to sum over, next to dW's many
// with the tokens (wkb k-blocks each): its reduction is cut into slices of at most two thirds of
// a pair's even share of all k-blocks (a tile's epilogue counted as 8), so
// that no pair is left alone with one. Measured on B200 (backward): 30 tokens,
// K 136, vocabulary 68684: 39 us, with at most 8 slices 63; 2048 tokens, K
// 512, vocabulary 8192: 59 us either way (4 slices).
int dh_slices(int64_t M, int64_t vcount, int64_t K, int64_t wkb) {
  const int64_t tiles = static_cast<int64_t>(tiles_of(M)) * tiles_of(K), nkb = (vcount + kBlockR - 1) / kBlockR;
  const int64_t share = (tiles * nkb + tiles_of(vcount) * tiles_of(K) * (wkb + 8)) / kPlanPairs + 8;
  int64_t slices = (3 * nkb + 2 * share - 1) / (2 * share);
  if (slices > 32) slices = 32;
  if (slices > nkb) slices = nkb;
  if (tiles >= kPlanPairs) slices = 1;
  return slices < 1 ? 1 : static_cast<int>(slices);
}

Plan make_plan(int64_t M, int64_t V, int64_t K, bool f32) {
  Plan q{};
  const int64_t per_col = M * (f32 ? 4 : 2);
  int64_t most = kPieceBytes / per_col / kTile * kTile;
  if (most < kTile) most = kTile;
  const int64_t all = (V + kTile - 1) / kTile * kTile;
  q.pieces = static_cast<int>((all + most - 1) / most);
  q.piece = ((V + q.pieces - 1) / q.pieces + kTile - 1) / kTile * kTile;
  q.pieces = static_cast<int>((V + q.piece - 1) / q.piece);
  q.rows_pad = (M + kTile - 1) / kTile * kTile;
  const int64_t vcount = V < q.piece ? V : q.piece;
  const int64_t tokens = M < kF32Tokens || !f32 ? M : kF32Tokens;
  q.slices = dh_slices(M, vcount, K, (tokens + kBlockR - 1) / kBlockR * (f32 ? 2 : 1));
  q.sums = q.pieces > 1 || q.slices > 1;
  size_t off = align256(static_cast<size_t>(M) * q.piece * 2);
  q.off_lo = off;
  if (f32) off += align256(static_cast<size_t>(M) * q.piece * 2);
  q.off_h = off;
  off += align256(static_cast<size_t>(M) * K * 2);
  q.off_scale = off;
  off += 256;
  q.off_sum = off;
  if (q.sums) off += static_cast<size_t>(q.slices) * q.rows_pad * K * 4;
  q.bytes = off;
  return q;
}

// Tiles of a Grad launch and their costs, from the vocabulary and the tokens set.
void grad_tiles(XentParams& p, bool dh, bool dw) {
  p.ntiles_h = dh ? p.slices * p.tiles_m * p.tiles_k : 0;
  const int ntiles_w = dw ? p.w_slices * tiles_of(p.vcount) * p.tiles_k : 0;
  const int cost_h = (p.vcount + kBlockR - 1) / kBlockR / p.slices;
  const int cost_w = (p.tcount + kBlockR - 1) / kBlockR * (p.split ? 2 : 1) / p.w_slices;
  p.dw_first = cost_w > cost_h || p.ntiles_h == 0;
  p.ntiles_a = p.dw_first ? ntiles_w : p.ntiles_h;
  p.ntiles_b = p.dw_first ? p.ntiles_h : ntiles_w;
  // a tile also costs its epilogue, about 4 k-blocks
  p.cost_a = (p.dw_first ? cost_w : cost_h) + 4;
  p.cost_b = (p.dw_first ? cost_h : cost_w) + 4;
}

// dH from its fp32 partial sums.
cudaError_t join_dh(const float* sum, int64_t rows_pad, int slices, int64_t M, int64_t K, void* dH, cudaStream_t s) {
  const int64_t nvecs = M * K / 4;
  const int64_t want = (nvecs + 255) / 256, cap = static_cast<int64_t>(8) * device_sm_count();
  return launch_pdl(xent_dh_kernel, dim3(static_cast<unsigned>(want < cap ? want : cap)), dim3(256), 0, s,
                    reinterpret_cast<const float4*>(sum), rows_pad * K / 4, slices, nvecs, static_cast<uint2*>(dH));
}

}  // namespace

// Columns of a tile of logits: 128 where such tiles still find a pair each, so
// that twice the SMs share the weights' loads and the epilogue (64 tokens, K
// 512, vocabulary 8192: forward 8.7 us, with 256 columns 9.8);
// else 256, which loads a third fewer bytes per product.
static int logit_columns(int64_t M, int64_t vocab) {
  return static_cast<int64_t>(tiles_of(M)) * ((vocab + 127) / 128) <= kPlanPairs ? 128 : 256;
}

// (maximum, sum) pairs per token: two per tile.
static int logit_parts(int64_t M, int64_t V) {
  const int bn = logit_columns(M, V);
  return 2 * static_cast<int>((V + bn - 1) / bn);
}

static size_t forward_bytes(int64_t M, int64_t parts) {
  return align256(static_cast<size_t>(parts) * M * 8) + align256(static_cast<size_t>(M) * 8);
}

// The workspaces never shrink as tokens are added, so that a loop's buffers
// serve its short last batch. The forward's bytes grow with the tokens except
// where the few tokens' kernels end and where the tiles turn from 128 to 256
// columns: the larger of the values just before those and of the call's own.
size_t xent_forward_workspace_bytes(int64_t M, int64_t V, int64_t K) {
  const int64_t few = M < kXentFew ? M : kXentFew;
  size_t most = forward_bytes(few, xent_few_parts(V, K));
  if (few == M) return most;
  const int64_t narrow = kPlanPairs / ((V + 127) / 128) * kTile;  // the most tokens with 128 columns
  for (const int64_t m : {M, narrow < M ? narrow : M}) {
    const size_t n = m > few ? forward_bytes(m, logit_parts(m, V)) : 0;
    if (n > most) most = n;
  }
  return most;
}

// A bound on the plan's bytes for up to M tokens, for either type of dW where
// that is fp32 (a call for dH alone plans as for bf16).
//   dz     a piece holds at most kPieceBytes, or 256 columns; at most the
//          whole vocabulary
//   sums   make_plan's slices are ceil(3 nkb / (2 share)) with share >=
//          tiles nkb / kPlanPairs, so at most ceil(1.5 kPlanPairs / tiles) (and
//          32, and nkb); a single slice takes sums only where the vocabulary is
//          in pieces, which more tokens (or bytes per entry) never undo
// Each part only grows with M and with the bytes per entry. At most 64 MiB of
// dz and about 30 MB of sums are more than the plan itself lays out (2048
// tokens, K 512, V 8192: 67 MB for 48; 4096, 2560, 32000: 197 for 195).
size_t xent_backward_workspace_bytes(int64_t M, int64_t V, int64_t K, int dw_is_f32) {
  if (xent_few(M)) return xent_few_workspace_bytes(M, V, K);
  const int64_t per = dw_is_f32 ? 4 : 2, all = (V + kTile - 1) / kTile * kTile;
  const int64_t piece = kPieceBytes > M * kTile * per ? kPieceBytes : M * kTile * per;
  const int64_t whole = M * all * per;
  const int64_t tm = tiles_of(M), tk = tiles_of(K), nkb = (V + kBlockR - 1) / kBlockR;
  const bool pieces = make_plan(M, V, K, dw_is_f32 != 0).pieces > 1;
  int64_t rows = pieces ? tm : 0;  // of dH's partial sums, in tiles
  for (int64_t m = 1; m <= tm && m * tk < kPlanPairs; ++m) {
    int64_t slices = (3 * kPlanPairs + 2 * m * tk - 1) / (2 * m * tk);
    slices = slices > 32 ? 32 : slices;
    slices = slices > nkb ? nkb : slices;
    if (slices > 1 && m * slices > rows) rows = m * slices;
  }
  const size_t bytes = align256(static_cast<size_t>(whole < piece ? whole : piece)) +
                       align256(static_cast<size_t>(M) * K * 2) + 256 + static_cast<size_t>(rows) * kTile * K * 4;
  const size_t few = xent_few_workspace_bytes(kXentFew, V, K);
  return bytes > few ? bytes : few;
}

cudaError_t launch_xent_forward(const void* h, const void* W, const int64_t* targets, int64_t M, int64_t V, int64_t K,
                                float* loss, float* lse, void* workspace, int* err, cudaStream_t s) {
  const bool few = xent_few(M);
  const int bn = logit_columns(M, V), parts = few ? xent_few_parts(V, K) : logit_parts(M, V);
  float2* part = static_cast<float2*>(workspace);
  float2* tlogit =
      reinterpret_cast<float2*>(static_cast<uint8_t*>(workspace) + align256(static_cast<size_t>(parts) * M * 8));
  cudaError_t e;
  if (few) {
    e = launch_xent_few_forward(h, W, targets, M, V, K, part, tlogit, s);
  } else {
    CUtensorMap maps[6] = {};
    if (!make_map(&maps[0], h, false, K, M, K * 2, 64, 64) || !make_map(&maps[1], W, false, K, V, K * 2, 64, 64))
      return cudaErrorInvalidValue;
    XentParams p{};
    p.M = static_cast<int>(M);
    p.V = static_cast<int>(V);
    p.K = static_cast<int>(K);
    p.vcount = p.V;
    p.targets = targets;
    p.err = err;
    p.tiles_m = tiles_of(M);
    p.tiles_k = tiles_of(K);
    p.ntiles_a = p.tiles_m * parts / 2;
    p.h = static_cast<const uint4*>(h);
    p.W = static_cast<const uint4*>(W);
    p.part = part;
    p.tlogit = tlogit;
    e = bn == 128 ? launch_phase<Phase::Lse, 128>(maps, p, s) : launch_phase<Phase::Lse, 256>(maps, p, s);
  }
  if (e != cudaSuccess) return e;
  return launch_pdl(xent_join_kernel, dim3(static_cast<unsigned>((M + kJoinTokens - 1) / kJoinTokens)),
                    dim3(kJoinTokens * kJoinSplit), 0, s, static_cast<const float2*>(part), parts, static_cast<int>(M),
                    static_cast<int>(V), static_cast<const float2*>(tlogit), targets, loss, lse,
                    few ? static_cast<const __nv_bfloat16*>(h) : nullptr, static_cast<const __nv_bfloat16*>(W),
                    static_cast<int>(K));
}

cudaError_t launch_xent_backward(const void* h, const void* W, const int64_t* targets, const float* lse,
                                 const float* dloss, int64_t M, int64_t V, int64_t K, void* dH, void* dW,
                                 int dw_is_f32, int accumulate, void* workspace, int* err, cudaStream_t s) {
  if (M == 0) {
    if (dW && !accumulate) return cudaMemsetAsync(dW, 0, static_cast<size_t>(V) * K * (dw_is_f32 ? 4 : 2), s);
    return cudaSuccess;
  }
  if (xent_few(M))
    return launch_xent_few_backward(h, W, targets, lse, dloss, M, V, K, dH, dW, dw_is_f32, accumulate, workspace, s);
  const bool f32 = dW && dw_is_f32;
  const Plan q = make_plan(M, V, K, dw_is_f32 != 0);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  void* dz = ws;
  void* lo = ws + q.off_lo;
  void* hm = ws + q.off_h;
  float* sum = reinterpret_cast<float*>(ws + q.off_sum);

  XentParams p{};
  p.M = static_cast<int>(M);
  p.V = static_cast<int>(V);
  p.K = static_cast<int>(K);
  p.targets = targets;
  p.err = err;
  p.tiles_m = tiles_of(M);
  p.tiles_k = tiles_of(K);
  p.lse = lse;
  p.dloss = dloss;
  p.split = f32;
  p.h = static_cast<const uint4*>(h);
  p.scale = reinterpret_cast<float*>(ws + q.off_scale);
  p.slices = q.slices;
  p.rows_pad = static_cast<int>(q.rows_pad);
  p.h_f32 = q.sums;
  p.w_f32 = f32;
  p.w_slices = 1;
  p.dW = dW;

  CUtensorMap zm[6] = {}, gm[6] = {};  // maps of Dz and of Grad
  if (!make_map(&zm[0], h, false, K, M, K * 2, 64, 64) ||
      !make_map(&zm[1], W, false, K, V, K * 2, 64, 64) ||
      !make_map(&gm[0], hm, false, K, M, K * 2, 64, 64))
    return cudaErrorInvalidValue;
  gm[1] = zm[1];
  if (dH && !(q.sums ? make_map(&gm[4], sum, true, K, static_cast<uint64_t>(q.slices) * q.rows_pad, K * 4, 32, 32)
                     : make_map(&gm[4], dH, false, K, M, K * 2, 64, 32)))
    return cudaErrorInvalidValue;
  if (dW && !make_map(&gm[5], dW, f32, K, V, K * (f32 ? 4 : 2), f32 ? 32 : 64, 32))
    return cudaErrorInvalidValue;

  for (int i = 0; i < q.pieces; ++i) {
    p.v0 = static_cast<int>(i * q.piece);
    p.vcount = static_cast<int>(V - p.v0 < q.piece ? V - p.v0 : q.piece);
    // dz of this piece: rows of `piece` elements, of which vcount are used
    // (the products read zeros beyond them)
    if (!make_map(&gm[2], dz, false, p.vcount, M, q.piece * 2, 64, 64) ||
        !make_map(&zm[4], dz, false, p.vcount, M, q.piece * 2, 64, 32))
      return cudaErrorInvalidValue;
    if (f32 && (!make_map(&gm[3], lo, false, p.vcount, M, q.piece * 2, 64, 64) ||
                !make_map(&zm[5], lo, false, p.vcount, M, q.piece * 2, 64, 32)))
      return cudaErrorInvalidValue;
    p.hm = i == 0 && dW ? static_cast<uint4*>(hm) : nullptr;
    p.find_scale = i == 0;
    const int bn = logit_columns(M, p.vcount);
    p.ntiles_a = p.tiles_m * ((p.vcount + bn - 1) / bn);
    p.ntiles_b = 0;
    const cudaError_t e = bn == 128 ? launch_phase<Phase::Dz, 128>(zm, p, s) : launch_phase<Phase::Dz, 256>(zm, p, s);
    if (e != cudaSuccess) return e;
    // an fp32 dW joins partial sums of 1024 tokens, one launch each (the
    // launches order the additions)
    const int step = f32 ? kF32Tokens : p.M;
    for (int t0 = 0; t0 < p.M; t0 += step) {
      p.t0 = t0;
      p.tcount = p.M - t0 < step ? p.M - t0 : step;
      p.h_add = i > 0;
      p.w_add = accumulate || t0 > 0;
      grad_tiles(p, dH && t0 == 0, dW != nullptr);
      if (cudaError_t e = launch_phase<Phase::Grad, 256>(gm, p, s); e != cudaSuccess) return e;
      if (!dW) break;
    }
  }
  if (!dH || !q.sums) return cudaSuccess;
  return join_dh(sum, q.rows_pad, q.slices, M, K, dH, s);
}

// ---- the gradients of y = x w^T from operands in bf16: Grad alone, with dY in
// the place of dz, x of h and w of the head
namespace {

// The fp32 partial sums of dX and of dW joined, each in order: to bf16 or fp32, and
// with `add` to what is there (one rounding to bf16). The first blocks take dX's.
struct JoinPart {
  const float4* sums;
  void* out;
  int64_t slice_vecs, vecs;  // from a slice to the next; outputs, in fours
  int slices, f32, add, blocks;
};

__device__ __forceinline__ void join_sums(const JoinPart& p, int block) {
  const int64_t T = static_cast<int64_t>(p.blocks) * 256;
  for (int64_t i = static_cast<int64_t>(block) * 256 + threadIdx.x; i < p.vecs; i += T) {
    float4 v = p.sums[i];
    for (int s = 1; s < p.slices; ++s) {
      const float4 w = p.sums[s * p.slice_vecs + i];
      v.x += w.x, v.y += w.y, v.z += w.z, v.w += w.w;
    }
    if (p.f32) {
      float4* to = static_cast<float4*>(p.out) + i;
      if (p.add) {
        const float4 o = *to;
        v.x += o.x, v.y += o.y, v.z += o.z, v.w += o.w;
      }
      *to = v;
    } else {
      uint2* to = static_cast<uint2*>(p.out) + i;
      if (p.add) {
        const uint2 o = *to;
        v.x += bf16_lo(o.x), v.y += bf16_hi(o.x), v.z += bf16_lo(o.y), v.w += bf16_hi(o.y);
      }
      *to = make_uint2(pack_bf16x2(v.y, v.x), pack_bf16x2(v.w, v.z));
    }
  }
}

__global__ void __launch_bounds__(256) linear_join_kernel(const __grid_constant__ JoinPart first, const __grid_constant__ JoinPart second) {
  pdl_wait_primary();
  pdl_launch_dependents();
  const int block = static_cast<int>(blockIdx.x);
  if (block < first.blocks) join_sums(first, block);
  else join_sums(second, block - first.blocks);
}

// Slices of dX's reduction: as of dH, and each at most 131072 columns (the
// tensor cores' sums lose up to a step of fp32 per 16 terms).
int linear_slices(int64_t M, int64_t N, int64_t K) {
  const int slices = dh_slices(M, N, K, (M + kBlockR - 1) / kBlockR), least = static_cast<int>((N + 131071) / 131072);
  return slices > least ? slices : least;
}
int64_t pad_rows(int64_t M) { return (M + kTile - 1) / kTile * kTile; }

// Slices of dW's reduction over the tokens, where its tiles are few: parts of at most
// two thirds of a pair's even share of all k-blocks, as of dH (4096 tokens, 512
// channels, K 2560: 20 tiles of 64 k-blocks next to dX's 160 of 8); an fp32 dW
// takes at most 1024 tokens in each, or, where those sums are too many, one launch
// for each 1024 tokens. 1: none. (As many without dX: dW is the same then.)
int linear_w_slices(int64_t M, int64_t N, int64_t K, bool f32) {
  const int64_t tiles = static_cast<int64_t>(tiles_of(N)) * tiles_of(K), nkb = (M + kBlockR - 1) / kBlockR;
  if (tiles >= kPlanPairs) return 1;
  const int64_t others = static_cast<int64_t>(tiles_of(M)) * tiles_of(K) * ((N + kBlockR - 1) / kBlockR + 8);
  const int64_t share = (tiles * nkb + others) / kPlanPairs + 8, most = (3 * kPlanPairs + 2 * tiles - 1) / (2 * tiles);
  int64_t slices = (3 * nkb + 2 * share - 1) / (2 * share);
  if (f32 && slices < (M + kF32Tokens - 1) / kF32Tokens) slices = (M + kF32Tokens - 1) / kF32Tokens;
  if (slices > 32 || slices > most || slices > nkb) {
    slices = most < nkb ? most : nkb;
    if (slices > 32) slices = 32;
    if (f32 && slices * kF32Tokens < M) return 1;
  }
  return slices < 1 ? 1 : static_cast<int>(slices);
}

}  // namespace

// Never shrinks as tokens are added, as the sizes of the head's backward: for
// every smaller number of token tiles a bound on its slices, those of
// make_plan's comment (up to kPlanPairs / tiles and a half, 32, and k-blocks).
// dW's slices are at most ceil(1.5 kPlanPairs / tiles), 32, and k-blocks.
static size_t linear_x_sum_bytes(int64_t M, int64_t N, int64_t K) {
  const int64_t tm = tiles_of(M), tk = tiles_of(K), nkb = (N + kBlockR - 1) / kBlockR, least = (N + 131071) / 131072;
  int64_t rows = least > 1 ? tm * least : 0;  // of the partial sums, in tiles
  for (int64_t m = 1; m <= tm && m * tk < kPlanPairs; ++m) {
    int64_t slices = (3 * kPlanPairs + 2 * m * tk - 1) / (2 * m * tk);
    slices = slices > 32 ? 32 : slices;
    slices = slices > nkb ? nkb : slices;
    if (slices > 1 && m * slices > rows) rows = m * slices;
  }
  return static_cast<size_t>(rows) * kTile * K * 4;
}

size_t linear_grad_sum_bytes(int64_t M, int64_t N, int64_t K) {
  const int64_t tiles = static_cast<int64_t>(tiles_of(N)) * tiles_of(K), nkb = (M + kBlockR - 1) / kBlockR;
  int64_t slices = tiles < kPlanPairs ? (3 * kPlanPairs + 2 * tiles - 1) / (2 * tiles) : 0;
  slices = slices > 32 ? 32 : slices;
  slices = slices > nkb ? nkb : slices;
  return linear_x_sum_bytes(M, N, K) + (slices > 1 ? static_cast<size_t>(slices * pad_rows(N)) * K * 4 : 0);
}

cudaError_t launch_linear_grads(const void* dY, const void* x, const void* w, int64_t M, int64_t N, int64_t K, void* dX,
                                void* dW, int dw_is_f32, int accumulate, float* one, float* sums, int* err,
                                cudaStream_t s) {
  const bool f32 = dW && dw_is_f32;
  XentParams p{};
  p.M = static_cast<int>(M);
  p.V = static_cast<int>(N);
  p.K = static_cast<int>(K);
  p.vcount = p.V;
  p.err = err;
  p.tiles_m = tiles_of(M);
  p.tiles_k = tiles_of(K);
  p.scale = one;
  p.slices = linear_slices(M, N, K);
  p.rows_pad = static_cast<int>(pad_rows(M));
  p.h_f32 = p.slices > 1;
  p.w_f32 = f32;
  p.dW = dW;
  p.w_slices = dW ? linear_w_slices(M, N, K, f32) : 1;
  p.w_rows = static_cast<int>(pad_rows(N));
  const bool split = p.w_slices > 1;
  float* w_sums = sums + linear_x_sum_bytes(M, N, K) / 4;
  CUtensorMap gm[6] = {};
  if (!make_map(&gm[2], dY, false, N, M, N * 2, 64, 64)) return cudaErrorInvalidValue;
  if (dW && (!make_map(&gm[0], x, false, K, M, K * 2, 64, 64) ||
             !(split ? make_map(&gm[5], w_sums, true, K, static_cast<uint64_t>(p.w_slices) * p.w_rows, K * 4, 32, 32)
                     : make_map(&gm[5], dW, f32, K, N, K * (f32 ? 4 : 2), f32 ? 32 : 64, 32))))
    return cudaErrorInvalidValue;
  if (dX && (!make_map(&gm[1], w, false, K, N, K * 2, 64, 64) ||
             !(p.h_f32 ? make_map(&gm[4], sums, true, K, static_cast<uint64_t>(p.slices) * p.rows_pad, K * 4, 32, 32)
                       : make_map(&gm[4], dX, false, K, M, K * 2, 64, 32))))
    return cudaErrorInvalidValue;
  // maps that no tile uses are prefetched all the same
  for (int i : {0, 1, 3, 4, 5})
    if ((i == 3) || (!dW && (i == 0 || i == 5)) || (!dX && (i == 1 || i == 4))) gm[i] = gm[2];
  const int step = f32 && !split ? kF32Tokens : p.M;
  for (int t0 = 0; t0 < p.M; t0 += step) {
    p.t0 = t0;
    p.tcount = p.M - t0 < step ? p.M - t0 : step;
    p.w_add = !split && (accumulate || t0 > 0);
    grad_tiles(p, dX && t0 == 0, dW != nullptr);
    if (cudaError_t e = launch_phase<Phase::Grad, 256>(gm, p, s); e != cudaSuccess) return e;
    if (!dW) break;
  }
  JoinPart parts[2] = {};
  if (dX && p.h_f32)
    parts[0] = {reinterpret_cast<const float4*>(sums), dX, static_cast<int64_t>(p.rows_pad) * K / 4, M * K / 4, p.slices, 0, 0, 0};
  if (split)
    parts[1] = {reinterpret_cast<const float4*>(w_sums), dW, static_cast<int64_t>(p.w_rows) * K / 4, N * K / 4, p.w_slices, f32, accumulate, 0};
  for (JoinPart& part : parts) {
    const int64_t want = (part.vecs + 255) / 256, cap = static_cast<int64_t>(8) * device_sm_count();
    part.blocks = static_cast<int>(want < cap ? want : cap);
  }
  const int blocks = parts[0].blocks + parts[1].blocks;
  if (blocks == 0) return cudaSuccess;
  return launch_pdl(linear_join_kernel, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, s, parts[0], parts[1]);
}

}  // namespace bl
