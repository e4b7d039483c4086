// Product of two INT8 operands with a scale per token and per output channel
// (L1), and the operands' values for its straight-through gradients (L2).
//
//   acc[m,n] = sum_k xq[m,k] wq[n,k]              exact INT32
//   y[m,n]   = rn(fp32(acc) * fp32(sx[m] * sw[n]))
//
// Four kernels:
//   int8_tile_kernel  persistent CTA pairs, tcgen05.mma kind::i8 (cta_group::2),
//                     both operands by TMA, INT32 accumulators in TMEM
//   int8_few_kernel   a few tokens: the weights stream through a deep TMA ring to
//                     mma.sync
//   int8_mid_kernel   tens of tokens: tiles of 128 channels by all tokens, whose K
//                     is split over a cluster
//   int8_values_kernel  rn_bf16(code * scale) of both operands, for the gradients'
//                     products (k_xent.cu)
//
// Measured on B200 (a call among others in a graph, inputs from HBM; the floor is
// the bytes at the copy rate or the operations at twice the bf16 rate):
//   tokens x channels x K    kernel   us      floor   bound by
//   1 x 6912 x 2560          few      6.0     2.7     the start (2.2) and one HBM latency
//   16 x 32000 x 2560, fp32  few      17.0    12.8    HBM (4.9 TB/s)
//   64 x 32000 x 2560        mid      17.4    13.2    HBM
//   64 x 6912 x 2560         mid      8.5     2.9     108 CTAs with 10 stages each (260 ns a stage: 4 in flight), their join
//   64 x 2560 x 6912         mid      8.5     2.8     120 CTAs (6 per tile), 9 stages each
//   333 x 5001 x 1040        tiles    8.1     1.4     one tile per pair: set-up, 9 stages, its end
//   768 x 768 x 16384        mid      21.2    5.9     144 CTAs reading 226 MB from L2
//   512 x 2560 x 6912        tiles    13.8    5.7     54 pairs with 54 stages each (165 ns a stage, of the loads)
//   2048 x 2560 x 6912       tiles    26.1    22.2    tensor cores (two rounds of tiles as 1.73)
//   2048 x 8192 x 512        tiles    12.2    5.9     the epilogue
//   4096 x 6912 x 2560       tiles    47.2    44.4    tensor cores (5.84 rounds as 6)
//   4096 x 32000 x 2560      tiles    208     205     tensor cores
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <atomic>
#include <cstdint>
#include <type_traits>

#include "bl_act8.cuh"
#include "bl_device.cuh"
#include "bl_internal.h"
#include "bl_mma.cuh"
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
constexpr int kBoxPitch = 176;
template <typename TY, int BN, bool kTma>
struct Geo {
  // an epilogue warp's output box, 32 rows of 32 columns; or of 128 bytes, where the
  // warp writes them itself, with 32 bytes in front and 16 behind that part the banks
  static constexpr int kBoxRow = kTma ? 32 * sizeof(TY) : kBoxPitch;
  static constexpr int kBox = 32 * kBoxRow;
  static constexpr int kBBytes = BN / 2 * kBlockK;
  static constexpr int kStageBytes = kABytes + kBBytes;
  static constexpr int kStages = (232448 - 1280 - kEpiWarps * (kBox + 128)) / kStageBytes;
  static constexpr int kOffEpi = kStages * kStageBytes;
  static constexpr int kOffScale = kOffEpi + kEpiWarps * kBox;  // a chunk's channel scales, per epilogue warp
  static constexpr int kOffBar = kOffScale + kEpiWarps * 128;
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

// 16-byte piece j of row `row` of an output box of 32 columns: rows of 128 bytes,
// 128-byte swizzled (fp32), or of 64 bytes, 64-byte swizzled (bf16).
template <int kEsize>
__device__ __forceinline__ uint32_t box_piece(uint32_t box, int row, int j) {
  const int turn = kEsize == 4 ? row & 7 : (row >> 1) & 3;
  return box + static_cast<uint32_t>(row) * (32 * kEsize) + (static_cast<uint32_t>(j ^ turn) << 4);
}

__device__ __forceinline__ void store_word_if(bool yes, char* to, uint32_t w) {
  asm volatile("{\n.reg .pred q;\nsetp.ne.b32 q, %2, 0;\n@q st.global.b32 [%0], %1;\n}" ::"l"(to), "r"(w), "r"(static_cast<int>(yes)) : "memory");
}

// A warp's 32 rows, of which 128 bytes from column col on stand in the box behind the
// 32 bytes in front of them, go to y in runs that start and end on its 32-byte sectors:
// of each row, from the last sector boundary up to col to the last one up to the end
// of the 128 bytes (kEnd: from there to col alone). A row whose columns do not start on
// a word's boundary stands a column further on in the box, so that its words are y's.
// Only words within columns lo .. hi - 1 and the first `rows` rows are written.
// (Runs that start where the 32 columns do: 139 us for 80 at 7788 x 10233 x 384
// fp32, for partly written sectors; the loop unrolled in full: 100, for instructions
// that no cache holds; branches around the stores: twice the time.)
template <typename TY, bool kEnd>
__device__ __forceinline__ void store_rows(uint32_t box, TY* y, int row0, int rows, int col, int lo, int hi, int N, int lane) {
  constexpr int kEsize = sizeof(TY), kPer = 4 / kEsize;        // elements of a word
  constexpr int kLanes = kEnd ? 8 : 32, kStep = 32 / kLanes;   // of a row; rows at once
  constexpr int kU = 8;                                        // words in flight
  const int r0 = lane / kLanes, l = lane % kLanes;
  const uintptr_t start = reinterpret_cast<uintptr_t>(y + static_cast<int64_t>(row0) * N + col);
  char* to = reinterpret_cast<char*>(start & ~uintptr_t(31)) + 4 * l;
  const uint32_t step = static_cast<uint32_t>(kStep * kEsize) * static_cast<uint32_t>(N);
  uint32_t rel = static_cast<uint32_t>(start & 31) + static_cast<uint32_t>(r0 * kEsize) * static_cast<uint32_t>(N);  // of the row
  uint32_t from = box + r0 * kBoxPitch + 32 + 4 * l;
#pragma unroll 1
  for (int r = r0; r < 32; r += kU * kStep) {
    uint32_t w[kU], at[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      at[u] = rel;
      asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[u]) : "r"(from + u * kStep * kBoxPitch - (rel & 28)));
      rel += step;
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int c = col + l * kPer - static_cast<int>((at[u] & 31) / kEsize);
      store_word_if(r + u * kStep < rows && c >= lo && c + kPer <= hi, to + (at[u] & ~31u), w[u]);
    }
    from += kU * kStep * kBoxPitch;
  }
}

// TY: type of y. kTma: y's rows start on 16-byte boundaries, so a box leaves by
// one TMA store; else the warp writes it row by row.
template <typename TY, int BN, bool kTma>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kTileThreads, 1)
    int8_tile_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w,
                     const __grid_constant__ CUtensorMap map_y, const __grid_constant__ TileParams p) {
  using G = Geo<TY, BN, kTma>;
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

  // a warp's; a failed wait also stops the peer CTA's
  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    if (mbar_wait_warp(bar, parity, abort_flag, p.err)) return true;
    st_cluster_u32(map_to_rank(smem_u32(const_cast<int*>(abort_flag)), rank ^ 1u), 1u);
    return false;
  };
  auto lead = [&](uint64_t* bar) -> uint32_t { return map_to_rank(smem_u32(bar), 0); };
  const int nkb = (p.K + kBlockK - 1) / kBlockK;
  // tokens fastest: the pairs at work share few tiles of the weights
  auto tile_row = [&](int u) { return u % p.tiles_m * kRows + static_cast<int>(rank) * 128; };
  auto tile_col = [&](int u) { return u / p.tiles_m * BN; };

  if (warp == 0) {
    const bool one = elect_one();
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
        if (one) {
          // both CTAs' boxes arrive on the leader's barrier
          if (leader) mbar_arrive_expect_tx(&full[stage], 2 * G::kStageBytes);
          const uint32_t at = smem0 + stage * G::kStageBytes, bar = bars + 8 * stage;
          load_pair(&map_x, bar, at, kb * kBlockK, a0);
          load_pair(&map_w, bar, at + kABytes, kb * kBlockK, b0);
        }
        __syncwarp();
        ++issued;
        if (++stage == kStages) {
          stage = 0;
          phase ^= 1;
        }
      }
    }
    if (one && leader && (!ok || *abort_flag)) {
      // let every copy already issued land before the pair exits
      const unsigned long long deadline = globaltimer_ns() + kWaitLimitNs;
      for (uint32_t s = 0; s < kStages && s < issued; ++s)
        mbar_drain_until(&full[s], (issued - s - 1) / kStages & 1, deadline);
    }
    __syncwarp();
  } else if (warp == 1) {
    if (leader) {
      const bool one = elect_one();
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
          if (one) {
#pragma unroll
            for (int kk = 0; kk < kBlockK / 32; ++kk)
              mma_i8_pair(d_tmem, ad0 + at + kk * 2, bd0 + at + kk * 2, kIdesc, (kb | kk) != 0);
            mma_commit_pair(&empty[stage], 0x3);
          }
          __syncwarp();
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1;
          }
        }
        if (ok && one) mma_commit_pair(&tmem_full[buf], 0x3);
        __syncwarp();
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
  } else {
    const int q = warp & 3, part = (warp - kWarpEpi0) >> 2, slot0 = warp - kWarpEpi0;
    // 32-column chunks of the warp: the first half of the tile's, or the second
    constexpr int kChunks = BN / 32, kFirst = (kChunks + 1) / 2;
    const int chunks = part == 0 ? kFirst : kChunks - kFirst;
    constexpr int kEsize = sizeof(TY);
    const uint32_t box = smem_u32(smem + G::kOffEpi + slot0 * G::kBox);
    const uint32_t table = smem_u32(smem + G::kOffScale + slot0 * 128);
    int buf = 0;
    uint32_t buf_phase = 0;
    // What the next tile needs, requested while this one is worked on: the token's
    // scale, and of each chunk's channels one scale per lane, which all lanes then
    // read from shared memory. (Every lane reading all 32 from global memory, a
    // chunk ahead: 50 us for 8192 x 8192 outputs of K 128.)
    float next_sx = 0.0f, next_sw[kFirst];
    auto prepare = [&](int u) {
      if (u >= p.ntiles) return;
      const int row = tile_row(u) + q * 32 + lane, col = tile_col(u) + part * kFirst * 32 + lane;
      if (row < p.M) asm volatile("ld.global.nc.f32 %0, [%1];" : "=f"(next_sx) : "l"(p.sx + row));
#pragma unroll
      for (int c = 0; c < kFirst; ++c)
        if (c < chunks && col + 32 * c < p.N)
          asm volatile("ld.global.nc.f32 %0, [%1];" : "=f"(next_sw[c]) : "l"(p.sw + col + 32 * c));
    };
#pragma unroll
    for (int c = 0; c < kFirst; ++c) next_sw[c] = 0.0f;
    prepare(pair);
    for (int u = pair; u < p.ntiles; u += npairs) {
      const int row0 = tile_row(u) + q * 32;
      const int col0 = tile_col(u) + part * kFirst * 32;
      const f32x2 sx2 = both2(next_sx);
      float sw[kFirst];
#pragma unroll
      for (int c = 0; c < kFirst; ++c) sw[c] = next_sw[c];
      prepare(u + npairs);
      // chunks that hold columns
      const int left = (p.N - col0 + 31) >> 5, live = row0 >= p.M || left < 0 ? 0 : left < chunks ? left : chunks;
      if (!wait(&tmem_full[buf], buf_phase)) break;
      tc_fence_after();
      const uint32_t tbase = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + buf * 256 + part * kFirst * 32;
      auto release = [&] {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(lead(&tmem_empty[buf]));
      };
      if (live == 0) release();
      uint32_t last[8], word = 0;  // of the chunk before: a row's last 32 bytes as the box had them; its last word
      uint32_t r[2][32];
      if (live > 0) {
        tmem_ld_32x32b_x32(tbase, r[0]);
        tmem_ld_wait();
      }
#pragma unroll
      for (int c = 0; c < kFirst; ++c) {
        if (c >= live) break;
        const int col = col0 + 32 * c;
        // (the buffer is released when every load of it has landed)
        if (c + 1 < live) tmem_ld_32x32b_x32(tbase + 32 * (c + 1), r[(c + 1) & 1]);
        else release();
        __syncwarp();
        asm volatile("st.shared.f32 [%0], %1;" ::"r"(table + lane * 4), "f"(sw[c]) : "memory");
        __syncwarp();
        // three roundings in fp32: of the sum, of the two scales' product, of y
        f32x2 v[16];
#pragma unroll
        for (int j = 0; j < 16; j += 2) {
          f32x2 w0, w1;
          asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(w0), "=l"(w1) : "r"(table + j * 8));
          const uint32_t* a = r[c & 1] + 2 * j;
          v[j] = mul2(pair2(__int2float_rn(static_cast<int>(a[0])), __int2float_rn(static_cast<int>(a[1]))), mul2(w0, sx2));
          v[j + 1] = mul2(pair2(__int2float_rn(static_cast<int>(a[2])), __int2float_rn(static_cast<int>(a[3]))), mul2(w1, sx2));
        }
        if (kTma && lane == 0) bulk_wait_group_read<0>();
        __syncwarp();
        uint32_t out[8 * kEsize];
        if constexpr (kEsize == 4) {
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            float lo, hi;
            split2(v[j], lo, hi);
            out[2 * j] = __float_as_uint(lo), out[2 * j + 1] = __float_as_uint(hi);
          }
        } else {
#pragma unroll
          for (int j = 0; j < 16; ++j) out[j] = pack_bf16x2(v[j]);
        }
        if constexpr (kTma) {
#pragma unroll
          for (int j = 0; j < 2 * kEsize; ++j)
            st_shared_v4(box_piece<kEsize>(box, lane, j), out[4 * j], out[4 * j + 1], out[4 * j + 2], out[4 * j + 3]);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_2d(&map_y, box, col, row0);
            bulk_commit_group();
          }
        } else {
          // 128 bytes of each row at a time (part h of them now)
          constexpr int kParts = 4 / kEsize;
          const int h = c % kParts, left = col - 32 * h, hi = col + 32 < p.N ? col + 32 : p.N;
          const bool end = c + 1 == live, whole = h == kParts - 1;
          const uint32_t to = box + lane * kBoxPitch;
          TY* y = static_cast<TY*>(p.y);
          const int rows = p.M - row0;
          auto front = [&] {
            st_shared_v4(to, last[0], last[1], last[2], last[3]);
            st_shared_v4(to + 16, last[4], last[5], last[6], last[7]);
          };
          if (h == 0 && c > 0) front();
          const uint32_t first = out[0], tail = out[8 * kEsize - 1];
          const bool odd = kEsize == 2 && (lane & p.N & 1);  // the row starts in the middle of a word
          if constexpr (kEsize == 2) {
            // (the word in front of the first one is written by nobody here)
            const uint32_t pick = odd ? 0x5432u : 0x7654u;
            uint32_t before = c > 0 ? word : 0u;
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const uint32_t w = out[j];
              out[j] = __byte_perm(before, w, pick);
              before = w;
            }
            word = tail;
          }
#pragma unroll
          for (int j = 0; j < 2 * kEsize; ++j)
            st_shared_v4(to + 32 + h * 64 + 16 * j, out[4 * j], out[4 * j + 1], out[4 * j + 2], out[4 * j + 3]);
#pragma unroll
          for (int j = 0; j < 8; ++j) last[j] = out[8 * kEsize - 8 + j];
          if constexpr (kEsize == 2) {
            // a row's first and last element, where they share their words with columns of others
            TY* line = y + static_cast<int64_t>(row0 + lane) * p.N;
            if (c == 0 && odd && lane < rows) *reinterpret_cast<uint16_t*>(line + col) = static_cast<uint16_t>(first);
            if (end && (odd != ((hi & 1) != 0)) && lane < rows) {
              uint16_t w = static_cast<uint16_t>(tail >> 16);
              if (hi < col + 32) asm volatile("ld.shared.b16 %0, [%1];" : "=h"(w) : "r"(to + 32 + 2 * (hi - 1 - left) + 2 * odd) : "memory");
              *reinterpret_cast<uint16_t*>(line + hi - 1) = w;
            }
          }
          if (whole || end) {
            __syncwarp();
            store_rows<TY, false>(box, y, row0, rows, left, col0, hi, p.N, lane);
            if (whole && end) {
              __syncwarp();
              front();
              __syncwarp();
              store_rows<TY, true>(box, y, row0, rows, col + 32, col0, hi, p.N, lane);
            }
          }
        }
        tmem_ld_wait();
      }
      if (++buf == 2) {
        buf = 0;
        buf_phase ^= 1;
      }
    }
    if (kTma && lane == 0) bulk_wait_group_read<0>();
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
// The weights are read once and hardly used: what counts is bytes in flight. A CTA
// (two fit on an SM, of this kernel or of the next one, whose first loads then
// overlap this one's end) takes tiles of 16 R channels in turn; up to four warps,
// each with every fourth stage, keep a ring of stages (256 of K: the channels' rows
// and the tokens', 128-byte swizzled boxes) filled by TMA, across the ends of
// tiles (one of them takes some 250 cycles for a stage's requests, which a CTA's
// share of HBM fills in fewer). R x S consumer warps: a
// warp takes one group of 16 channels and every S-th stage, mma.sync.m16n8k32 on
// operands that ldmatrix brings in the instruction's order; the S warps' INT32
// sums are added in shared memory (exact in any order).
constexpr int64_t kFewMost = 16;   // most tokens, with weights of any shape
constexpr int kFewSmem = 114688;   // of a CTA: half an SM's

struct FewParams {
  int M, N, K, ntiles;
  const float* sx;
  const float* sw;
  void* y;
  int* err;
};

template <int kTok, int R>
struct Few {
  static constexpr int S = kTok == 1 && R == 1 ? 8 : R == 1 || (R == 2 && kTok != 2) ? 4 : 2;
  static constexpr int kLoaders = S < 4 ? S : 4;
  static constexpr int kWarps = R * S, kThreads = 32 * (kLoaders + kWarps), kN = 16 * R, kM = 8 * kTok;
  static constexpr int kBoxW = kN * 128, kBoxX = kM * 128, kStageBytes = 2 * (kBoxW + kBoxX);
  static constexpr int kSums = S * kM * kN;  // ints
  static constexpr int kBufs = kTok == 4 ? 1 : 2;  // of them, in turn
  static constexpr int kFixed = kBufs * kSums * 4 + 512 /*barriers*/ + 1024 /*base alignment*/;
  // a multiple of S, so that a slot of the ring is always the same warps': they
  // have seen its last filling when they wait for the next
  static constexpr int kStages = (kFewSmem - kFixed) / kStageBytes / S * S;
  static constexpr int kOffSums = kStages * kStageBytes;
  static constexpr int kOffBar = kOffSums + kBufs * kSums * 4;  // full, empty, joined, read; the abort flag
  static constexpr int kSmemBytes = kOffBar + 512 + 1024;
  static_assert(kStages >= S && kSmemBytes <= kFewSmem && (2 * kStages + 2) * 8 + 8 <= 512, "shared memory");
};

__device__ __forceinline__ void mma_s8(int (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldmatrix4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix2(uint32_t addr, uint32_t& a, uint32_t& b) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x2.shared.b16 {%0, %1}, [%2];" : "=r"(a), "=r"(b) : "r"(addr) : "memory");
}
// 16-byte chunk c of row r of a box of 128-byte rows, 128-byte swizzled.
__device__ __forceinline__ uint32_t few_chunk(uint32_t box, int r, int c) {
  return box + static_cast<uint32_t>(r) * 128u + (static_cast<uint32_t>(c ^ (r & 7)) << 4);
}

template <typename TY, int kTok, int R>
__global__ void __launch_bounds__(Few<kTok, R>::kThreads, 2)
    int8_few_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w, const FewParams p) {
  using G = Few<kTok, R>;
  constexpr int kStages = G::kStages, S = G::S, kN = G::kN, kM = G::kM;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + G::kOffBar);
  uint64_t* empty = full + kStages;
  uint64_t* joined = empty + kStages;
  uint64_t* read = joined + 1;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(read + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int boxes = (p.K + 127) >> 7, nst = (boxes + 1) >> 1;  // boxes of 128 of K, stages of two
  if (threadIdx.x == 0) {
    prefetch_tensormap(&map_w);
    prefetch_tensormap(&map_x);
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], R);
    }
    mbar_init(joined, G::kWarps);
    mbar_init(read, G::kWarps);
    *abort_flag = 0;
    fence_mbar_init();
  }
  __syncthreads();
  pdl_wait_primary();
  pdl_launch_dependents();
  if (warp < G::kLoaders) {
    const bool one = elect_one();
    const int mine = ((p.ntiles - 1 - static_cast<int>(blockIdx.x)) / static_cast<int>(gridDim.x) + 1) * nst;  // the CTA's stages
    int it = warp, st = warp % nst, u = blockIdx.x + warp / nst * gridDim.x;
    bool ok = true;
    for (; it < mine; it += G::kLoaders) {
      const int stage = it % kStages;
      if (!mbar_wait_warp(&empty[stage], (it / kStages & 1) ^ 1, abort_flag, p.err)) {
        ok = false;
        break;
      }
      if (one) {
        const bool two = 2 * st + 1 < boxes;
        mbar_arrive_expect_tx(&full[stage], two ? G::kStageBytes : G::kStageBytes / 2);
        uint8_t* at = smem + stage * G::kStageBytes;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (h == 1 && !two) break;
          tma_load_2d(&map_w, &full[stage], at + h * G::kBoxW, (2 * st + h) * 128, u * kN);
          tma_load_2d(&map_x, &full[stage], at + 2 * G::kBoxW + h * G::kBoxX, (2 * st + h) * 128, 0);
        }
      }
      __syncwarp();
      for (st += G::kLoaders; st >= nst; st -= nst) u += gridDim.x;
    }
    // an early end: let this warp's copies land before the CTA exits
    if (one && (!ok || *abort_flag)) {
      const unsigned long long deadline = globaltimer_ns() + kWaitLimitNs;
      for (int i = it - G::kLoaders, n = 0; i >= 0 && n < kStages; i -= G::kLoaders, n += G::kLoaders)
        mbar_drain_until(&full[i % kStages], i / kStages & 1, deadline);
    }
    return;
  }
  const int cw = warp - G::kLoaders, group = cw % R, share = cw / R;
  const int steps = (p.K + 31) >> 5;  // of 32 of K
  // the lane's row and 16-byte half of a step, in the operands' four matrices
  const int wrow = group * 16 + (lane & 15), whalf = lane >> 4;
  const int xrow = kTok == 1 ? lane & 7 : (lane & 7) + (lane >> 4) * 8, xhalf = (lane >> 3) & 1;
  int tile = 0;
  uint32_t base = 0;  // stages of the tiles before
  for (int u = blockIdx.x; u < p.ntiles; u += gridDim.x, ++tile, base += nst) {
    int acc[kTok][4] = {};
    for (uint32_t st = (share - base) & (S - 1); st < static_cast<uint32_t>(nst); st += S) {
      const uint32_t stage = (base + st) % kStages;
      if (!mbar_wait_warp(&full[stage], (base + st) / kStages & 1, abort_flag, p.err)) return;
      const uint32_t at = smem_u32(smem) + stage * G::kStageBytes;
      const int left = steps - static_cast<int>(st) * 8;
#pragma unroll
      for (int step = 0; step < 8; ++step) {
        if (step >= left) break;
        const int box = step >> 2, c = (step & 3) * 2;
        uint32_t a[4];
        ldmatrix4(few_chunk(at + box * G::kBoxW, wrow, c + whalf), a);
        const uint32_t xbox = at + 2 * G::kBoxW + box * G::kBoxX;
        if constexpr (kTok == 1) {
          uint32_t b0, b1;
          ldmatrix2(few_chunk(xbox, xrow, c + xhalf), b0, b1);
          mma_s8(acc[0], a, b0, b1);
        } else {
#pragma unroll
          for (int i = 0; i < kTok; i += 2) {
            uint32_t b[4];
            ldmatrix4(few_chunk(xbox, xrow + 8 * i, c + xhalf), b);
            mma_s8(acc[i], a, b[0], b[1]);
            mma_s8(acc[i + 1], a, b[2], b[3]);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[stage]);
    }
    // two buffers in turn: a warp writes one again only after a join that every
    // reader of it has reached; a single one only when all have read it
    if (G::kBufs == 1 && tile > 0 && !mbar_wait_warp(read, (tile - 1) & 1, abort_flag, p.err)) return;
    int* sums = reinterpret_cast<int*>(smem + G::kOffSums) + tile % G::kBufs * G::kSums;
    int* own = sums + share * kN * kM + group * 16;
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int i = 0; i < kTok; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) own[(8 * i + 2 * t + (j & 1)) * kN + g + (j >> 1) * 8] = acc[i][j];
    __syncwarp();
    if (lane == 0) mbar_arrive(joined);
    if (!mbar_wait_warp(joined, tile & 1, abort_flag, p.err)) return;
    for (int i = threadIdx.x - 32 * G::kLoaders; i < kN * kM; i += 32 * G::kWarps) {
      const int n = u * kN + i % kN, m = i / kN;
      if (m >= p.M || n >= p.N) continue;
      int v = 0;
#pragma unroll
      for (int k = 0; k < S; ++k) v += sums[k * kN * kM + i];
      store1(static_cast<TY*>(p.y) + static_cast<int64_t>(m) * p.N + n,
             __int2float_rn(v) * __fmul_rn(__ldg(p.sx + m), __ldg(p.sw + n)));
    }
    if constexpr (G::kBufs == 1) {
      __syncwarp();
      if (lane == 0) mbar_arrive(read);
    }
  }
}

// ---------------------------------------------------------------- tens of tokens
// D = W x^T: 128 channels of one CTA by 32 or 64 tokens,
// tcgen05.mma kind::i8 (cta_group::1). There are few such tiles, so the CTAs of a
// cluster share one: each sums its part of K, leaves its INT32 sums in its shared
// memory, and turns its share of the tokens into y from all CTAs' sums. A warp reads
// 128 channels of a token at once from each CTA, 16 bytes a lane, and everything it
// needs before it adds (4 bytes a lane and one CTA after another: 1 us more over 2 or
// 4 CTAs, 2 over 8; 16 bytes a lane of one channel's tokens, so with the lanes apart:
// the same 1 to 2). A tile that is not shared goes from TMEM to y, a thread for each
// channel, so a warp writes 32 channels of a token at once, whatever N.
//
// Roles (192 threads): warp 0 loads, warp 1 issues the MMAs, warps 2..5 are the
// epilogue. Waits are bounded as in the tiles' kernel; every thread reaches the
// cluster's barriers whatever happened before.
constexpr int64_t kMidMost = 64;  // most tokens of a tile
constexpr int kMidThreads = 192;
constexpr int kMidShare = 8;  // most CTAs of a cluster

struct MidParams {
  int M, N, K;
  int tiles_n, share;  // tiles over the channels; CTAs per tile
  const float* sx;
  const float* sw;
  void* y;
  int* err;
};

template <int NT>
struct Mid {
  static constexpr int kW = 128 * kBlockK, kX = NT * kBlockK, kStageBytes = kW + kX;
  static constexpr int kStages = 110 * 1024 / kStageBytes;  // two CTAs to an SM
  static constexpr int kOffBar = kStages * kStageBytes;  // full, empty; done; TMEM base, abort flag
  static constexpr int kOffSx = (kOffBar + (2 * kStages + 1) * 8 + 8 + 15) / 16 * 16;  // the tokens' scales
  static constexpr int kSmemBytes = kOffSx + NT * 4 + 1024 /*base alignment*/;
  static_assert(kSmemBytes <= 232448 && NT * 512 <= kOffBar, "the sums fit in the ring");
};

__device__ __forceinline__ int4 ld_cluster_v4(uint32_t addr) {
  int4 v;
  asm volatile("ld.shared::cluster.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

__device__ __forceinline__ void store4(float* p, const float (&v)[4]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, const float (&v)[4]) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(pair2(v[0], v[1])), pack_bf16x2(pair2(v[2], v[3])));
}

// Channels n .. n + 3 (n a multiple of 4) of a token, those that there are.
template <typename TY>
__device__ __forceinline__ void store_channels(TY* to, const float (&v)[4], int n, int N) {
  if ((N & 3) == 0) {
    if (n < N) store4(to, v);
  } else {
#pragma unroll
    for (int h = 0; h < 4; ++h)
      if (n + h < N) store1(to + h, v[h]);
  }
}

template <typename TY, int NT>
__global__ void __launch_bounds__(kMidThreads)
    int8_mid_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w, const MidParams p) {
  using G = Mid<NT>;
  constexpr int kStages = G::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + G::kOffBar);
  uint64_t* empty = full + kStages;
  uint64_t* done = empty + kStages;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank()), share = p.share;
  const int tile = static_cast<int>(blockIdx.x) / share;
  const int n0 = tile % p.tiles_n * 128, t0 = tile / p.tiles_n * NT, M = p.M - t0 < NT ? p.M - t0 : NT;  // tokens t0 .. t0 + M - 1
  const int boxes = (p.K + kBlockK - 1) / kBlockK;
  const int kb0 = boxes * rank / share, nkb = boxes * (rank + 1) / share - kb0;
  if (threadIdx.x == 0) {
    prefetch_tensormap(&map_w);
    prefetch_tensormap(&map_x);
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(done, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc_one(tmem_holder, NT);
    tmem_relinquish_one();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  pdl_wait_primary();
  pdl_launch_dependents();  // (after the allocation: a dependent's must not come first)
  if (warp == 0) {
    const bool one = elect_one();
    int kb = 0;
    for (; kb < nkb; ++kb) {
      const int s = kb % kStages;
      if (!mbar_wait_warp(&empty[s], (kb / kStages & 1) ^ 1, abort_flag, p.err)) break;
      if (one) {
        mbar_arrive_expect_tx(&full[s], G::kStageBytes);
        uint8_t* at = smem + s * G::kStageBytes;
        tma_load_2d(&map_w, &full[s], at, (kb0 + kb) * kBlockK, n0);
        tma_load_2d(&map_x, &full[s], at + G::kW, (kb0 + kb) * kBlockK, t0);
      }
      __syncwarp();
    }
    if (one && (kb < nkb || *abort_flag)) {
      const unsigned long long deadline = globaltimer_ns() + kWaitLimitNs;
      for (int i = kb - 1; i >= 0 && i >= kb - kStages; --i)
        mbar_drain_until(&full[i % kStages], i / kStages & 1, deadline);
    }
  } else if (warp == 1) {
    const bool one = elect_one();
    constexpr uint32_t kIdesc = make_idesc(2 /*s32*/, 1 /*s8*/, 0, 0, 128, NT);
    const uint32_t s0 = smem_u32(smem);
    const uint64_t ad0 = smem_desc_sw128(s0, 16, 1024), bd0 = smem_desc_sw128(s0 + G::kW, 16, 1024);
    for (int kb = 0; kb < nkb; ++kb) {
      const int s = kb % kStages;
      if (!mbar_wait_warp(&full[s], kb / kStages & 1, abort_flag, p.err)) break;
      tc_fence_after();
      const uint64_t at = static_cast<uint64_t>(s) * (G::kStageBytes >> 4);
      if (one) {
#pragma unroll
        for (int kk = 0; kk < kBlockK / 32; ++kk) mma_i8_one(tmem, ad0 + at + kk * 2, bd0 + at + kk * 2, kIdesc, (kb | kk) != 0);
        mma_commit_one(&empty[s]);
      }
      __syncwarp();
    }
    if (one) mma_commit_one(done);
  }
  __syncwarp();
  const int q = warp & 3, row = q * 32 + lane, n = n0 + row;
  float* sx = reinterpret_cast<float*>(smem + G::kOffSx);
  if (warp >= 2) {
    if (row < NT) sx[row] = row < M ? __ldg(p.sx + t0 + row) : 0.0f;
    asm volatile("bar.sync 1, 128;" ::: "memory");
  }
  const float sw = warp >= 2 && n < p.N ? __ldg(p.sw + n) : 0.0f;
  bool ok = true;
  TY* y = static_cast<TY*>(p.y) + static_cast<int64_t>(t0) * p.N;
  if (warp >= 2) {
    ok = mbar_wait_warp(done, 0, abort_flag, p.err);
    tc_fence_after();
  } else if (lane == 0) {
    mbar_drain(done, 0);  // nothing reads the ring any more
  }
  __syncwarp();
  int* sums = reinterpret_cast<int*>(smem);  // [NT][128]
  if (warp >= 2 && ok) {
    const uint32_t base = tmem + (static_cast<uint32_t>(q * 32) << 16);
#pragma unroll 1
    for (int c = 0; c < M; c += 32) {
      uint32_t r[32];
      tmem_ld_32x32b_x32(base + c, r);
      tmem_ld_wait();
      if (share > 1) {
#pragma unroll
        for (int j = 0; j < 32; ++j)
          sums[(c + j) * 128 + row] = static_cast<int>(r[j]);
      } else if (n < p.N) {
#pragma unroll
        for (int j = 0; j < 32; j += 4) {
          const float4 s4 = *reinterpret_cast<const float4*>(sx + c + j);
          const float s[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (c + j + i < M)
              store1(y + static_cast<int64_t>(c + j + i) * p.N + n, __int2float_rn(static_cast<int>(r[j + i])) * __fmul_rn(s[i], sw));
        }
      }
    }
  }
  // freed in front of the cluster's barriers: a CTA that holds TMEM waits for no other
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_one(tmem, NT);
  }
  if (share > 1) {
    cluster_sync_all();
    if (warp >= 2 && ok) {
      // a warp takes every fourth token of the CTA's share, a lane 4 of the channels;
      // all CTAs' sums of them are requested at once
      const int m0 = M * rank / share + q, m1 = M * (rank + 1) / share, c0 = n0 + 4 * lane;
      const uint32_t at = smem_u32(sums + m0 * 128 + 4 * lane);
      float w[4];
#pragma unroll
      for (int h = 0; h < 4; ++h) w[h] = c0 + h < p.N ? __ldg(p.sw + c0 + h) : 0.0f;
      auto join = [&](auto ctas) {
        constexpr int kShare = decltype(ctas)::value, kU = (NT + 4 * kShare - 1) / (4 * kShare);
        int4 t[kU][kShare];
#pragma unroll
        for (int i = 0; i < kU; ++i) {
          if (m0 + 4 * i >= m1) break;
#pragma unroll
          for (int k = 0; k < kShare; ++k) t[i][k] = ld_cluster_v4(map_to_rank(at, k) + i * 2048);
        }
#pragma unroll
        for (int i = 0; i < kU; ++i) {
          const int m = m0 + 4 * i;
          if (m >= m1) break;
          int4 v = t[i][0];
#pragma unroll
          for (int k = 1; k < kShare; ++k) v.x += t[i][k].x, v.y += t[i][k].y, v.z += t[i][k].z, v.w += t[i][k].w;
          const float s = sx[m];
          const float o[4] = {__int2float_rn(v.x) * __fmul_rn(s, w[0]), __int2float_rn(v.y) * __fmul_rn(s, w[1]),
                              __int2float_rn(v.z) * __fmul_rn(s, w[2]), __int2float_rn(v.w) * __fmul_rn(s, w[3])};
          store_channels(y + static_cast<int64_t>(m) * p.N + c0, o, c0, p.N);
        }
      };
      switch (share) {
        case 2: join(std::integral_constant<int, 2>{}); break;
        case 4: join(std::integral_constant<int, 4>{}); break;
        case 6: join(std::integral_constant<int, 6>{}); break;
        default: join(std::integral_constant<int, 8>{});
      }
    }
    cluster_sync_all();  // a CTA's sums stay until all have read them
  }
}

// ---------------------------------------------------------------- values for the gradients
// The two operands' chunks of 8 codes are one range, cut evenly.
struct ValuesParams {
  const uint2* q[2];
  const float* scale[2];
  uint4* out[2];
  int64_t first, chunks;  // of the first operand, and of both (either may have none)
  int per_row;
  float* one;
};

constexpr int kValuesU = 4;  // chunks in flight per thread

__global__ void __launch_bounds__(256) int8_values_kernel(const ValuesParams p) {
  pdl_wait_primary();
  pdl_launch_dependents();
  const int64_t T = static_cast<int64_t>(gridDim.x) * 256, t = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (t == 0) *p.one = 1.0f;
  const bool narrow = p.chunks <= 0xFFFFFFFFll;  // the row by a 32-bit division
  for (int64_t i0 = t; i0 < p.chunks; i0 += kValuesU * T) {
    uint2 c[kValuesU];
    float s[kValuesU];
#pragma unroll
    for (int u = 0; u < kValuesU; ++u) {
      const int64_t at = i0 + u * T;
      if (at < p.chunks) {
        const bool second = at >= p.first;
        const int64_t i = second ? at - p.first : at;
        c[u] = __ldg((second ? p.q[1] : p.q[0]) + i);
        s[u] = __ldg((second ? p.scale[1] : p.scale[0]) +
                     (narrow ? static_cast<int64_t>(static_cast<uint32_t>(i) / static_cast<uint32_t>(p.per_row)) : i / p.per_row));
      }
    }
#pragma unroll
    for (int u = 0; u < kValuesU; ++u) {
      const int64_t at = i0 + u * T;
      if (at < p.chunks) {
        f32x2 v[4];
        act8_values8(c[u], s[u], v);
        const bool second = at >= p.first;
        (second ? p.out[1] : p.out[0])[second ? at - p.first : at] =
            make_uint4(pack_bf16x2(v[0]), pack_bf16x2(v[1]), pack_bf16x2(v[2]), pack_bf16x2(v[3]));
      }
    }
  }
}

// ---------------------------------------------------------------- host side

bool make_map(CUtensorMap* m, const void* base, CUtensorMapDataType type, uint64_t inner, uint64_t outer,
              uint64_t row_bytes, uint32_t box_inner, uint32_t box_outer,
              CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B) {
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
  // (Lines of 128 bytes, not pairs of them: where K is no multiple of 128 a box's rows lie
  // on two lines each, 12 x 3149 x 6672 11.3 us for 13.1; else the same.)
  return encode(m, type, 2, const_cast<void*>(base), dims, strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
                swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename TY, int BN, bool kTma>
cudaError_t launch_tiles(const CUtensorMap (&maps)[3], const TileParams& p, cudaStream_t s) {
  auto kernel = int8_tile_kernel<TY, BN, kTma>;
  constexpr int kSmem = Geo<TY, BN, kTma>::kSmemBytes;
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

template <typename TY, int BN>
cudaError_t forward_tiles(const int8_t* xq, const int8_t* wq, TileParams p, cudaStream_t s) {
  p.ntiles = p.tiles_m * ((p.N + BN - 1) / BN);
  // Boxes leave by TMA where rows start on 16 bytes, but not those of a y beyond some
  // half of L2 (fp32; bf16: all of it) whose rows do not start on 32 (7788 x 10236 x 384
  // fp32: 99.8 us by TMA, 77.7 in whole sectors; bf16, 10232: 63.4 and 56.9, and 16.6 and
  // 18.2 at 3809 x 4520 x 336).
  const int64_t row = static_cast<int64_t>(p.N) * sizeof(TY);
  const bool tma = row % 16 == 0 && (row % 32 == 0 || p.M * row < int64_t(1) << (sizeof(TY) == 4 ? 26 : 27));
  CUtensorMap maps[3] = {};
  if (!make_map(&maps[0], xq, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.K, p.M, p.K, kBlockK, 128) ||
      !make_map(&maps[1], wq, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.K, p.N, p.K, kBlockK, BN / 2) ||
      (tma && !make_map(&maps[2], p.y, sizeof(TY) == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                        p.N, p.M, static_cast<uint64_t>(p.N) * sizeof(TY), 32, 32,
                        sizeof(TY) == 4 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B)))
    return cudaErrorInvalidValue;
  return tma ? launch_tiles<TY, BN, true>(maps, p, s) : launch_tiles<TY, BN, false>(maps, p, s);
}

// The tiles' width: the least time of the busiest pair, its tiles times a stage's
// MMAs (measured with all SMs at work, in cycles of 1.9 GHz: 88 for 32 of K with 64
// columns, 109 with 128, 136 with 192, 183 with 256; so 45 + 0.5 a column) and 300 for
// each tile, and the end of one tile.
struct TilePlan {
  int columns;
  int64_t cycles;
};
TilePlan tile_plan(int64_t M, int64_t N, int64_t K) {
  const int64_t tiles_m = (M + kRows - 1) / kRows, pairs = device_sm_count() / 2, nkb = (K + kBlockK - 1) / kBlockK;
  TilePlan best{256, INT64_MAX};
  for (int bn = 256; bn >= 64; bn -= 32) {
    const int64_t rounds = (tiles_m * ((N + bn - 1) / bn) + pairs - 1) / pairs;
    const int64_t cycles = rounds * (nkb * (180 + 2 * bn) + 300) + 10 * bn;
    if (cycles < best.cycles) best = {bn, cycles};
  }
  return best;
}

template <typename TY>
cudaError_t forward_tiles(const int8_t* xq, const int8_t* wq, TileParams p, int columns, cudaStream_t s) {
  p.tiles_m = (p.M + kRows - 1) / kRows;
  switch (columns) {
    case 64: return forward_tiles<TY, 64>(xq, wq, p, s);
    case 96: return forward_tiles<TY, 96>(xq, wq, p, s);
    case 128: return forward_tiles<TY, 128>(xq, wq, p, s);
    case 160: return forward_tiles<TY, 160>(xq, wq, p, s);
    case 192: return forward_tiles<TY, 192>(xq, wq, p, s);
    case 224: return forward_tiles<TY, 224>(xq, wq, p, s);
    default: return forward_tiles<TY, 256>(xq, wq, p, s);
  }
}

template <typename TY, int kTok, int R>
cudaError_t launch_few(const int8_t* xq, const int8_t* wq, FewParams p, cudaStream_t s) {
  using G = Few<kTok, R>;
  auto kernel = int8_few_kernel<TY, kTok, R>;
  static bool done[64] = {};
  if (cudaError_t e = allow_smem(kernel, G::kSmemBytes, done); e != cudaSuccess) return e;
  CUtensorMap x, w;
  if (!make_map(&x, xq, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.K, p.M, p.K, 128, G::kM) ||
      !make_map(&w, wq, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.K, p.N, p.K, 128, G::kN))
    return cudaErrorInvalidValue;
  p.ntiles = (p.N + G::kN - 1) / G::kN;
  const int most = 2 * device_sm_count();
  return launch_pdl(kernel, dim3(p.ntiles < most ? p.ntiles : most), dim3(G::kThreads), G::kSmemBytes, s, x, w, p);
}

template <typename TY, int kTok>
cudaError_t forward_few(const int8_t* xq, const int8_t* wq, const FewParams& p, cudaStream_t s) {
  // the tiles' channels: those with the least to load (the channels' rows, and for
  // each tile the tokens', from L2, so half of them) for the busiest SM and for
  // the SMs at work on average
  constexpr int kWidest = kTok == 4 ? 3 : 4;
  const int sms = device_sm_count();
  int best = 1;
  int64_t least = INT64_MAX;
  for (int r = kWidest; r >= 1; --r) {
    const int64_t tiles = (p.N + 16 * r - 1) / (16 * r), rows = 16 * r + 4 * kTok;
    const int64_t cost = (tiles + sms - 1) / sms * rows * 16 + tiles * rows * 16 / (tiles < sms ? tiles : sms);
    if (cost < least) best = r, least = cost;
  }
  switch (best) {
    case 1: return launch_few<TY, kTok, 1>(xq, wq, p, s);
    case 2: return launch_few<TY, kTok, 2>(xq, wq, p, s);
    case 3: return launch_few<TY, kTok, 3>(xq, wq, p, s);
    default: return launch_few<TY, kTok, kWidest>(xq, wq, p, s);
  }
}

template <typename TY>
cudaError_t forward_few(const int8_t* xq, const int8_t* wq, const FewParams& p, cudaStream_t s) {
  if (p.M <= 8) return forward_few<TY, 1>(xq, wq, p, s);
  return p.M <= 16 ? forward_few<TY, 2>(xq, wq, p, s) : forward_few<TY, 4>(xq, wq, p, s);
}

// Shared memory of which an SM holds one CTA's: what the narrow tiles' kernels may ask
// for, as much as the question of how many clusters fit does. It is set here alone and
// always to this, so that no host thread takes from another what it is about to use.
constexpr int kMidLimit = 128 * 1024;

template <typename TY, int NT>
cudaError_t allow_mid() {
  static_assert(Mid<NT>::kSmemBytes <= kMidLimit, "shared memory");
  static bool done[64] = {};
  return allow_smem(int8_mid_kernel<TY, NT>, kMidLimit, done);
}

// Clusters of `share` CTAs that fit at once with an SM for each CTA (a cluster lies
// within one GPC: 15 of 8, 33 of 4). An answer is kept; where the question fails, what
// the SMs alone allow serves this call.
int clusters_at_once(int share) {
  static std::atomic<int> known[64][kMidShare + 1] = {};
  int dev = 0;
  cudaGetDevice(&dev);
  const bool keep = dev >= 0 && dev < 64;
  if (keep)
    if (const int n = known[dev][share].load(std::memory_order_relaxed)) return n;
  int clusters = 0;
  if (allow_mid<__nv_bfloat16, 64>() == cudaSuccess) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(share * device_sm_count()));
    cfg.blockDim = dim3(kMidThreads);
    cfg.dynamicSmemBytes = kMidLimit;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = share;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&clusters, int8_mid_kernel<__nv_bfloat16, 64>, &cfg) != cudaSuccess) clusters = 0;
  }
  cudaGetLastError();
  if (clusters <= 0) return device_sm_count() / share;
  if (keep) known[dev][share].store(clusters, std::memory_order_relaxed);
  return clusters;
}

// CTAs per tile (1 or even: 3, 5 and 7 measured 0.25 us more than their stages say), and
// the nanoseconds that follow from it: 260 per stage of a CTA, 550 + 75 per CTA for a
// join, 1300 where the clusters do not fit one CTA to an SM (64 tokens, 17 tiles, 32
// stages: 13.5 us alone, 9.8 over 2 CTAs, 7.9 over 4, 7.5 over 6, 8.5 over 8; 15 tiles:
// 7.3 over 8). There is no term for what many tiles read from L2: 768 x 768 x 16384 takes
// 21.2 us where this says 17.3 (in wide tiles 24.4, so the choice is right all the same).
struct MidPlan {
  int share;
  int64_t ns;
};
MidPlan mid_plan(int64_t tiles, int64_t K) {
  const int64_t boxes = (K + kBlockK - 1) / kBlockK, most = device_sm_count() * 5 / 4;
  MidPlan best{1, boxes * 260};
  for (int share = 2; share <= kMidShare && tiles * share <= most && share <= boxes; share += 2) {
    const int64_t ns = (boxes + share - 1) / share * 260 + 550 + 75 * share + (tiles > clusters_at_once(share) ? 1300 : 0);
    if (ns < best.ns) best = {share, ns};
  }
  return best;
}

// A programmatic dependent launch of clusters of `cluster` CTAs.
template <typename... Params, typename... Args>
cudaError_t launch_clusters(void (*kernel)(Params...), int grid, int cluster, int threads, int smem, cudaStream_t s, Args... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <typename TY, int NT>
cudaError_t launch_mid(const int8_t* xq, const int8_t* wq, MidParams p, cudaStream_t s) {
  using G = Mid<NT>;
  if (cudaError_t e = allow_mid<TY, NT>(); e != cudaSuccess) return e;
  CUtensorMap x, w;
  if (!make_map(&x, xq, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.K, p.M, p.K, kBlockK, NT) ||
      !make_map(&w, wq, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.K, p.N, p.K, kBlockK, 128))
    return cudaErrorInvalidValue;
  p.tiles_n = (p.N + 127) / 128;
  const int tiles = p.tiles_n * ((p.M + NT - 1) / NT);
  return launch_clusters(int8_mid_kernel<TY, NT>, tiles * p.share, p.share, kMidThreads, G::kSmemBytes, s, x, w, p);
}

template <typename TY>
cudaError_t forward_mid(const int8_t* xq, const int8_t* wq, const MidParams& p, cudaStream_t s) {
  return p.M <= 32 ? launch_mid<TY, 32>(xq, wq, p, s) : launch_mid<TY, 64>(xq, wq, p, s);
}

size_t align256(size_t n) { return (n + 255) & ~size_t(255); }

}  // namespace

cudaError_t launch_int8_forward(const int8_t* xq, const float* sx, const int8_t* wq, const float* sw, int64_t M,
                                int64_t N, int64_t K, void* y, int y_f32, int* err, cudaStream_t s) {
  // Up to 16 tokens stream the weights through mma.sync, up to 32 where K and the
  // weights are of middling size: its start is 0.5 us shorter, its stages are slower (17
  // to 32 tokens: 1000 x 768 3.1 us for 3.6, 2048 x 1024 3.3 for 3.7; 2560 x 2560 6.7
  // for 5.3, 8192 x 512 4.0 for 3.3).
  if (M <= kFewMost || (M <= 32 && K >= 512 && K <= 2048 && N <= 4096 && N * K <= int64_t(1) << 22)) {
    const FewParams p{static_cast<int>(M), static_cast<int>(N), static_cast<int>(K), 0, sx, sw, y, err};
    return y_f32 ? forward_few<float>(xq, wq, p, s) : forward_few<__nv_bfloat16>(xq, wq, p, s);
  }
  const TilePlan wide = tile_plan(M, N, K);
  // More tokens than one narrow tile has take the wide tiles, but where those are few
  // and K is long, so that splitting K over narrow ones is worth its join (at 1.9
  // cycles a nanosecond; 65 x 120 x 5824: 5.5 us for 10.3 in wide tiles, 412 x 332 x
  // 3200 5.6 for 7.6).
  const int64_t columns = M <= 32 ? 32 : kMidMost, tiles = (N + 127) / 128 * ((M + columns - 1) / columns);
  const MidPlan narrow = mid_plan(tiles, K);
  if (M <= kMidMost || (tiles * narrow.share <= device_sm_count() * 5 / 4 && narrow.ns + 400 < wide.cycles * 10 / 19)) {
    const MidParams p{static_cast<int>(M), static_cast<int>(N), static_cast<int>(K), 0, narrow.share, sx, sw, y, err};
    return y_f32 ? forward_mid<float>(xq, wq, p, s) : forward_mid<__nv_bfloat16>(xq, wq, p, s);
  }
  TileParams p{};
  p.M = static_cast<int>(M);
  p.N = static_cast<int>(N);
  p.K = static_cast<int>(K);
  p.sx = sx;
  p.sw = sw;
  p.y = y;
  p.err = err;
  return y_f32 ? forward_tiles<float>(xq, wq, p, wide.columns, s) : forward_tiles<__nv_bfloat16>(xq, wq, p, wide.columns, s);
}

// The values of x and of w in bf16, the factor 1, dX's and dW's partial sums.
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
  // Few tokens take the codes' own kernel: up to 32 in any case (32 x 6912 x 2560: 23.8 us
  // for 30.0 by values in bf16), up to 64 where it is the launches that count (64 tokens, 512
  // x 512: 6.0 for 9.7; 1000 x 2560: 12.2 for 13.2; 2560 x 2560: 21.5 for 17.9).
  if (M <= 32 || (M <= 64 && N * K <= int64_t(5) << 19))
    return launch_int8_few_grads(dY, xq, sx, wq, sw, M, N, K, dX, dW, dw_is_f32, accumulate, reinterpret_cast<float*>(w), s);
  float* one = reinterpret_cast<float*>(w + align256(static_cast<size_t>(N) * K * 2));
  ValuesParams v{};
  v.q[0] = reinterpret_cast<const uint2*>(xq);
  v.q[1] = reinterpret_cast<const uint2*>(wq);
  v.scale[0] = sx;
  v.scale[1] = sw;
  v.out[0] = reinterpret_cast<uint4*>(x);
  v.out[1] = reinterpret_cast<uint4*>(w);
  v.first = dW ? M * K / 8 : 0;
  v.chunks = v.first + (dX ? N * K / 8 : 0);
  v.per_row = static_cast<int>(K / 8);
  v.one = one;
  // as many rounds as fill the SMs, and a grid that fills the rounds
  const int64_t most = static_cast<int64_t>(8) * device_sm_count(), per = 256 * kValuesU;
  const int64_t rounds = (v.chunks + most * per - 1) / (most * per), grid = (v.chunks + rounds * per - 1) / (rounds * per);
  if (cudaError_t e = launch_pdl(int8_values_kernel, dim3(static_cast<unsigned>(grid)), dim3(256), 0, s, v);
      e != cudaSuccess)
    return e;
  return launch_linear_grads(dY, x, w, M, N, K, dX, dW, dw_is_f32, accumulate, one,
                             reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(one) + 256), err, s);
}

}  // namespace bl
