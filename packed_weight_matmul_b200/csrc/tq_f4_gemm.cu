// Product of two 4-bit matrices of one format (tq_linear_f4) on the
// block-scaled tensor cores of sm_100a:
//
//   y[b][n] = g_w g_x sum_k c_w[n][k] s_w[n][k/B] c_x[b][k] s_x[b][k/B]
//
// tcgen05.mma kind::mxf4 (MX4: E8M0 scale per 32) and kind::mxf4nvf4 (NV4:
// E4M3 scale per 16) multiply the packed codes as they lie in memory: codes
// go from global to shared memory by TMA and are never decoded. The block
// scales of both operands have to sit in tensor memory, row r of a 128-row
// operand at lane r % 32 (repeated in all four lane quarters) and column
// r / 32, one 32-bit column word per row holding the scales of 128 (MX4) or
// 64 (NV4) consecutive k.
//
// For more than 64 batch rows (fewer: tq_f4_decode.cu). A tile is CG * 128
// weight rows (M) times NT = 128 or 256 batch rows (N); CG = 2 pairs
// the CTAs of a cluster on one tile (each holds its 128 weight rows and half
// of the batch rows). Persistent, 16 (pair, NV4) or 18 warps per CTA:
//   warp 0       TMA producer: per stage of 256 k the 128-byte swizzled boxes
//                of the weight rows and of this CTA's batch rows; it also
//                allocates the tensor memory
//   warp 1       MMA issuer (first CTA of a pair): 4 MMAs of K = 64 per stage;
//                in the second CTA it passes "stage ready" on to the first
//   next         scales, see below
//   last 8       epilogue: tensor memory -> registers -> y
//
// Scales, stored: two groups of four warps take turns. A group reads the scales
// of every row for 4 stages (32 bytes of MX4, 64 of NV4) into registers one
// turn ahead, lays them down row by row in shared memory, and per stage every
// warp reads rows lane, lane + 32, ... and stores word w of row group i to
// column 4 w + i of its own lane quarter.
// Scales, copied (pairs with NV4): two groups of three warps take turns. Warp b
// has 128 rows (b = 0: of the weights); a lane reads 32 scale bytes (2 stages)
// of rows lane, lane + 32, + 64, + 96 into registers one turn ahead and per
// stage stores word w of its four rows as 16 bytes: the 512 bytes that one
// tcgen05.cp (32 lanes x 16 bytes, to all four lane quarters), issued before
// the stage's MMAs, takes to columns 4 w .. 4 w + 3.
// Storing reads every scale four times from shared memory, which the TMA and
// the MMAs need too; a copy takes the warp of the MMAs and the tensor core
// about 30 cycles. 21504 x 5376 x 2048 rows (256 x 256 tiles): NV4 142 us
// stored, 113 copied, MX4 99 either way, but one wave of such tiles, 18944 x
// 4096 x 256 rows, 16.3 and 17.3 us; 5376 x 8192 x 777 rows (128 x 128 tiles,
// half the MMA time per copy): NV4 24.0 and 26.3 us, MX4 21.4 and 23.1 us.
//
// A stage's barrier counts the scale warps of a group and the codes' bytes.
//
// Every wait is bounded; one that gives up leaves NaN in the outputs of the
// tiles that were not finished.
#include "tq_f4_digits.cuh"
#include "tq_f4_tc.cuh"

namespace tq {
using namespace f4;
namespace {

constexpr int kRowsM = 128;         // weight rows per CTA
constexpr uint32_t kStageRow = kF4StageRow;
constexpr uint32_t kTmemColumns = 512;
constexpr uint32_t kSmemLimit = 227u * 1024u;
constexpr uint32_t kReserve = 3u * 1024u;  // barriers, alignment, static
constexpr int kScaleGroups = 2, kDrainWarps = 8;
constexpr int kScaleWarps = 4;  // of a group, single CTA

template <int FMT, int NT, int CG>
struct Plan {
  static constexpr int kWords = FMT == TQ_FMT_MX4 ? 2 : 4;  // scale words/row
  static constexpr uint32_t kScaleRow = kWords * 4;  // scale bytes per stage
  static constexpr uint32_t kBCols = NT / 32 > 4 ? NT / 32 : 4;
  static constexpr uint32_t kScaleCols = kWords * (4 + kBCols);
  static constexpr uint32_t kA = kRowsM * kStageRow;
  static constexpr uint32_t kB = (NT / CG) * kStageRow;
  // scales by tcgen05.cp, see above
  static constexpr bool kCopied = CG == 2 && FMT == TQ_FMT_NV4;
  static constexpr int kScaleBlocks = 1 + (NT + 127) / 128;  // of 128 rows
  static constexpr int kArrivals = kCopied ? kScaleBlocks : kScaleWarps;
  static constexpr int kDrainWarp = 2 + kScaleGroups * kArrivals;
  static constexpr int kThreads = 32 * (kDrainWarp + kDrainWarps);
  // copied: 32 bytes of a row in turn, in the ring
  static constexpr uint32_t kS = kCopied ? kScaleBlocks * 128 * kScaleRow : 0;
  static constexpr uint32_t kStage = kA + kB + kS;
  // else scale bytes of a row that a group reads at once, four pieces of one
  // load each where the ring is long enough (see the assertion below), else
  // two
  static constexpr uint32_t kPiece = FMT == TQ_FMT_NV4 ? 16u : 8u;
  static constexpr uint32_t kUnit =
      kCopied ? 32u
              : kPiece * (5 * kStage + 2 * (kRowsM + NT) * 4 * kPiece + kReserve <=
                                  kSmemLimit
                              ? 4u
                              : 2u);
  static constexpr uint32_t kScales = kCopied ? 0 : (kRowsM + NT) * kUnit;
  static constexpr int kUnitStages = (int)(kUnit / kScaleRow);
  static constexpr int kFit =
      (int)((kSmemLimit - kReserve - kScaleGroups * kScales) / kStage);
  static constexpr int kFitT = (int)((kTmemColumns - NT) / kScaleCols);
  static constexpr int kStages0 = kFit < kFitT ? kFit : kFitT;
  static constexpr int kStages = kStages0 < 8 ? kStages0 : 8;
  // A wait by parity is right only one phase ahead. Between two units of a
  // group lie up to kUnitStages stages of the other one, so the MMAs of stage
  // it - 2 kStages are known to be done when a group waits for those of
  // it - kStages only with kStages > kUnitStages.
  static_assert(kStages > kUnitStages, "a group could run two phases ahead");
  // offsets from the 1024-byte aligned base
  static constexpr uint32_t kOffB = kStages * kA;
  static constexpr uint32_t kOffS = kOffB + kStages * kB;
  static constexpr uint32_t kOffBar = kOffS + kStages * kS +
                                      kScaleGroups * kScales;
  static constexpr uint32_t kSmem = kOffBar + 512 + 1024;
  static_assert(kSmem <= kSmemLimit, "shared memory");
};

struct Args {
  const uint8_t *wscales, *xscales;
  const float *wg, *xg;
  void *y;
  int64_t n, batch, ldy;
  int k, tiles_m, tiles_n, y_bf16;
  DigitArgs digits;
  const uint8_t *wcodes;
};

template <int CG>
__device__ __forceinline__ void alloc_columns(uint32_t dst, uint32_t cols) {
  if constexpr (CG == 1) {
    tmem_alloc(dst, cols);
  } else {
    asm volatile(
        "tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
            dst),
        "r"(cols)
        : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::
                     : "memory");
  }
}

template <int CG>
__device__ __forceinline__ void free_columns(uint32_t taddr, uint32_t cols) {
  if constexpr (CG == 1)
    tmem_dealloc(taddr, cols);
  else
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(
                     taddr),
                 "r"(cols)
                 : "memory");
}

// Two fp32 values as bf16, `lo` in the low half.
__device__ __forceinline__ uint32_t bf16_pair(uint32_t lo, uint32_t hi) {
  const __nv_bfloat162 p =
      __floats2bfloat162_rn(__uint_as_float(lo), __uint_as_float(hi));
  return *reinterpret_cast<const uint32_t *>(&p);
}

// Arrive on the barrier at this CTA's address `bar` in the pair's first CTA,
// when a warp has read its part of the accumulator. Relaxed: nothing was written
// that the other side reads. The loads from tensor memory are over
// (tcgen05.wait::ld) and the fence before the arrival keeps them before it; a
// release would wait for the stores of y too.
__device__ __forceinline__ void arrive_leader(uint32_t bar) {
  uint32_t remote;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(remote) : "r"(bar));
  asm volatile(
      "mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(
          remote)
      : "memory");
}

// The same with release: also what this thread knows to be written to shared
// memory.
__device__ __forceinline__ void announce_leader(uint32_t bar) {
  uint32_t remote;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(remote) : "r"(bar));
  asm volatile(
      "mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(remote)
      : "memory");
}

template <int FMT, int NT, int CG>
__global__ void __launch_bounds__(Plan<FMT, NT, CG>::kThreads, 1)
    product_f4_kernel(const __grid_constant__ CUtensorMap tmap_w,
                      const __grid_constant__ CUtensorMap tmap_x,
                      const Args args) {
  using P = Plan<FMT, NT, CG>;
  constexpr int S = P::kStages;
  extern __shared__ uint8_t smem_raw[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t bars = base + P::kOffBar;
  // ready: a stage's codes and scales are here (in the first CTA of a pair:
  // the second one's too); empty: its MMAs are done
  const uint32_t ready = bars, empty = bars + 8 * S;
  const uint32_t dfull = bars + 16 * S, dempty = dfull + 8;
  const uint32_t slot = dfull + 16, abort_addr = dfull + 20;
  const uint32_t rank = CG == 2 ? cluster_rank() : 0u;
  const int group = blockIdx.x / CG, groups = gridDim.x / CG;
  const int tiles = args.tiles_m * args.tiles_n;
  const int steps = (args.k + 255) / 256;

  pdl_launch_dependents();
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(ready + 8 * s,
                P::kArrivals + 1 + (CG == 2 && rank == 0));
      mbar_init(empty + 8 * s, 1);
    }
    mbar_init(dfull, 1);
    mbar_init(dempty, CG * kDrainWarps);
    st_volatile_s32(abort_addr, 0);
    mbar_init_fence();
  }
  if (warp == 0) alloc_columns<CG>(slot, kTmemColumns);
  tc_fence_before_sync();
  __syncthreads();
  if (CG == 2) {
    asm volatile("barrier.cluster.arrive.aligned;\n"
                 "barrier.cluster.wait.aligned;" ::: "memory");
  }
  tc_fence_after_sync();
  pdl_wait();  // user memory is read and written from here on
  // all columns are this CTA's, so they start at column 0
  constexpr uint32_t kTmem = 0;

  if (warp == 0) {
    if (lane == 0) {
      uint32_t it = 0;
      bool ok = true;
      for (int t = group; t < tiles && ok; t += groups) {
        const int m0 = (t / args.tiles_n) * (CG * kRowsM) + rank * kRowsM;
        const int b0 = (t % args.tiles_n) * NT + rank * (NT / CG);
        for (int i = 0; i < steps; ++i, ++it) {
          const uint32_t s = it % S, ph = (it / S) & 1u;
          ok = mbar_wait(empty + 8 * s, ph ^ 1u, abort_addr, kWaitLimitNs);
          if (!ok) break;
          mbar_arrive_expect_tx(ready + 8 * s, P::kA + P::kB);
          tma_load_2d(base + s * P::kA, &tmap_w, i * (int)kStageRow, m0,
                      ready + 8 * s);
          tma_load_2d(base + P::kOffB + s * P::kB, &tmap_x,
                      i * (int)kStageRow, b0, ready + 8 * s);
        }
      }
      // every copy issued has landed, and every MMA that read one is done
      for (uint32_t j = it > (uint32_t)S ? it - S : 0; j < it; ++j)
        mbar_wait(empty + 8 * (j % S), (j / S) & 1u);
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 1) {
      uint32_t it = 0;
      bool ok = true;
      for (int t = group; t < tiles && ok; t += groups) {
        for (int i = 0; i < steps && ok; ++i, ++it) {
          ok = mbar_wait(ready + 8 * (it % S), (it / S) & 1u, abort_addr,
                         kWaitLimitNs);
          if (ok) announce_leader(ready + 8 * (it % S));
        }
      }
    }
    if (rank == 0) {  // the whole warp, see mma_stage
      uint32_t it = 0, done = 0;
      bool ok = true, here = false;
      for (int t = group; t < tiles && ok; t += groups, ++done) {
        if (done > 0)
          ok = mbar_wait_cluster(dempty, (done - 1) & 1u, abort_addr,
                                 kWaitLimitNs);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) break;
        for (int i = 0; i < steps; ++i, ++it) {
          const uint32_t s = it % S, ph = (it / S) & 1u;
          if (!here) {
            ok = CG == 2 ? mbar_wait_cluster(ready + 8 * s, ph, abort_addr,
                                             kWaitLimitNs)
                         : mbar_wait(ready + 8 * s, ph, abort_addr,
                                     kWaitLimitNs);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok) break;
          }
          tc_fence_after_sync();
          // the next stage's barrier is asked before this one's MMAs go out (by
          // a test that never suspends the warp, as try_wait may)
          const uint32_t s1 = (it + 1) % S, ph1 = ((it + 1) / S) & 1u;
          const bool next = mbar_test<CG>(ready + 8 * s1, ph1);
          const uint32_t sa = kTmem + NT + s * P::kScaleCols;
          if constexpr (P::kCopied) {
            const uint64_t scales = smem_desc_rows16(base + P::kOffS + s * P::kS);
  #pragma unroll
            for (int b = 0; b < P::kScaleBlocks; ++b)
              copy_scales<CG, P::kWords>(
                  b == 0 ? sa : sa + P::kWords * 4 + 4 * (b - 1),
                  b == 0 ? 4 : P::kBCols, scales + b * P::kWords * 32);
          }
          mma_stage<FMT, CG>(
              kTmem, smem_desc_kmajor_sw128(base + s * P::kA),
              smem_desc_kmajor_sw128(base + P::kOffB + s * P::kB),
              idesc_f4<FMT>(CG * kRowsM, NT, 0u),
              idesc_f4<FMT>(CG * kRowsM, NT, FMT == TQ_FMT_MX4 ? 2u : 0u), sa,
              sa + P::kWords * 4, P::kBCols, i != 0 ? 1u : 0u, empty + 8 * s);
          here = __all_sync(0xFFFFFFFFu, next);
        }
        if (ok) commit<CG>(dfull);
      }
      // every MMA issued is done before the CTA goes on to free its memory
      for (uint32_t j = it > (uint32_t)S ? it - S : 0; j < it; ++j)
        mbar_wait(empty + 8 * (j % S), (j / S) & 1u);
    }
  } else if (warp < P::kDrainWarp) {
    if constexpr (P::kCopied) {
      const int turn = (warp - 2) / P::kScaleBlocks;  // this warp's group
      const int block = (warp - 2) % P::kScaleBlocks;
      const int64_t row_bytes = args.k / f4_block(FMT);
      const bool whole = args.k % 256 == 0;
      const int units = (steps + P::kUnitStages - 1) / P::kUnitStages;
      const uint8_t *const scales = block == 0 ? args.wscales : args.xscales;
      const int64_t last = (block == 0 ? args.n : args.batch) - 1;
      // unit `lu` of tile `lt`; rows past the matrix repeat the last one (their
      // outputs are not stored)
      auto load = [&](int lt, int lu, uint32_t (&v)[4][8]) {
        const int64_t row0 =
            block == 0 ? (int64_t)(lt / args.tiles_n) * (CG * kRowsM) +
                             rank * kRowsM
                       : (int64_t)(lt % args.tiles_n) * NT + 128 * (block - 1);
        const int off = 32 * lu, left = (int)row_bytes - off;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int64_t r = row0 + lane + 32 * i;
          const uint8_t *p = scales + (r < last ? r : last) * row_bytes + off;
          // rows whose length is a multiple of a stage's scale bytes (k a
          // multiple of 256) start on such a boundary
          if (whole)
            load_unit<P::kWords>(v[i], p, left);
          else
            load_unit<0>(v[i], p, left);
        }
      };
      // (tile, unit) of this group's next turn: every second unit in order
      int lt = group, lu = turn;
      auto settle = [&]() {
        while (lu >= units) {
          lu -= units;
          lt += groups;
        }
      };
      settle();
      uint32_t v[4][8], next[4][8] = {};
      if (lt < tiles) load(lt, lu, next);
      bool ok = true;
      while (lt < tiles && ok) {
        // stages before this unit
        const uint32_t first = (uint32_t)((lt - group) / groups) * steps +
                               lu * P::kUnitStages;
        const int count = steps - lu * P::kUnitStages;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int w = 0; w < 8; ++w)  // E4M3 scales are read without their sign
            v[i][w] = FMT == TQ_FMT_NV4 ? next[i][w] & 0x7F7F7F7Fu : next[i][w];
        lu += kScaleGroups;
        settle();
#pragma unroll
        for (int i = 0; i < P::kUnitStages; ++i) {
          if (i >= count || !ok) break;
          const uint32_t it = first + i, s = it % S, ph = (it / S) & 1u;
          // the MMAs that read this slot's scales before are done
          ok = mbar_wait(empty + 8 * s, ph ^ 1u, abort_addr, kWaitLimitNs);
          ok = __all_sync(0xFFFFFFFFu, ok);
          if (!ok) break;
          const uint32_t at = base + P::kOffS + s * P::kS +
                              block * 128 * P::kScaleRow + 16 * lane;
#pragma unroll
          for (int w = 0; w < P::kWords; ++w)
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                             at + 512 * w),
                         "r"(v[0][i * P::kWords + w]),
                         "r"(v[1][i * P::kWords + w]),
                         "r"(v[2][i * P::kWords + w]),
                         "r"(v[3][i * P::kWords + w])
                         : "memory");
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) mbar_arrive(ready + 8 * s);
          // not before the first stage's stores, which would queue up behind
          if (i == 0 && lt < tiles) load(lt, lu, next);
        }
      }
    } else {
      const int turn = (warp - 2) / kScaleWarps;  // this warp's group
      const int tid = (threadIdx.x - 64) & 127;
      constexpr uint32_t tmem_scales = kTmem + NT;
      const uint32_t quarter = (uint32_t)(warp & 3) << 21;  // lane 32 q, bits 16+
      const int row_bytes = args.k / (FMT == TQ_FMT_MX4 ? 32 : 16);
      const bool whole = args.k % 256 == 0;
      const uint32_t buf = base + P::kOffS + turn * P::kScales;
      const int units = (steps + P::kUnitStages - 1) / P::kUnitStages;
      // a row's unit is read by kPieces neighbouring threads
      constexpr int kPieces = (int)(P::kUnit / P::kPiece), kPass = 128 / kPieces;
      constexpr int kPieceWords = (int)P::kPiece / 4;
      constexpr int kRowsPer = (kRowsM + NT + kPass - 1) / kPass;
      const int my_row = tid / kPieces, my_piece = tid % kPieces;
      uint32_t v[kRowsPer][kPieceWords];
      // unit `lu` of tile `lt`, into registers; rows past the matrix repeat the
      // last one (their outputs are not stored)
      int at_tile = -1;
      const uint8_t *wrows = nullptr, *xrows = nullptr;
      int wlast = 0, xlast = 0;
      auto load = [&](int lt, int lu) {
        if (lt != at_tile) {
          at_tile = lt;
          const int64_t m0 =
              (int64_t)(lt / args.tiles_n) * (CG * kRowsM) + rank * kRowsM;
          const int64_t b0 = (int64_t)(lt % args.tiles_n) * NT;
          const int64_t m = m0 < args.n ? m0 : args.n - 1;
          wlast = (int)(args.n - 1 - m < kRowsM ? args.n - 1 - m : kRowsM);
          xlast = (int)(args.batch - 1 - b0 < NT ? args.batch - 1 - b0 : NT);
          wrows = args.wscales + m * row_bytes;
          xrows = args.xscales + b0 * row_bytes;
        }
        const int off = lu * (int)P::kUnit + (int)P::kPiece * my_piece;
        auto each = [&](auto read) {
#pragma unroll
          for (int j = 0; j < kRowsPer; ++j) {
            const bool of_w = kPass * (j + 1) <= kRowsM;
            int r = my_row + kPass * j - (of_w ? 0 : kRowsM);
            r = min(r, of_w ? wlast : xlast);
            read(v[j], (of_w ? wrows : xrows) + (int64_t)r * row_bytes + off);
          }
        };
        // rows whose length is a multiple of a piece (k a multiple of 256)
        // start on its boundary
        if (whole)
          each([&](uint32_t (&d)[kPieceWords], const uint8_t *p) {
            load_piece(d, p, row_bytes - off);
          });
        else
          each([&](uint32_t (&d)[kPieceWords], const uint8_t *p) {
            load_piece_shifted(d, p, row_bytes - off);
          });
      };
      // (tile, unit) of this group's next turn: every second unit in order
      int lt = group, lu = turn;
      auto settle = [&]() {
        while (lu >= units) {
          lu -= units;
          lt += groups;
        }
      };
      settle();
      if (lt < tiles) load(lt, lu);
      bool ok = true;
      while (lt < tiles) {
        const int u = lu;
        // stages before this unit
        const uint32_t first =
            (uint32_t)((lt - group) / groups) * steps + u * P::kUnitStages;
        const int count = steps - u * P::kUnitStages < P::kUnitStages
                              ? steps - u * P::kUnitStages
                              : P::kUnitStages;
        bar_sync(1 + turn, 128);  // the group has read its last unit
#pragma unroll
        for (int j = 0; j < kRowsPer; ++j) {
          if (FMT == TQ_FMT_NV4) {  // E4M3 scales are read without their sign
#pragma unroll
            for (int w = 0; w < kPieceWords; ++w) v[j][w] &= 0x7F7F7F7Fu;
          }
          if (my_row + kPass * j < kRowsM + NT)
            store_piece(buf + scale_at<kPieces, P::kPiece>(my_row + kPass * j,
                                                           my_piece),
                        v[j]);
        }
        bar_sync(1 + turn, 128);
        lu += kScaleGroups;
        settle();
        if (lt < tiles) load(lt, lu);
#pragma unroll 1
        for (int i = 0; i < count; ++i) {
          const uint32_t it = first + i, s = it % S, ph = (it / S) & 1u;
          // the MMAs that read this slot's scales before are done; after a wait
          // that gave up, the warps only keep meeting at the barriers above
          if (ok)
            ok = mbar_wait(empty + 8 * s, ph ^ 1u, abort_addr, kWaitLimitNs);
          ok = __all_sync(0xFFFFFFFFu, ok);
          if (!ok) continue;
          tc_fence_after_sync();
          const uint32_t cols = tmem_scales + s * P::kScaleCols + quarter;
#pragma unroll
          for (int r0 = 0; r0 < 4 + (int)P::kBCols; r0 += 4) {
            uint32_t a[4][4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              if (32 * (r0 + r) >= kRowsM + NT) {
                a[r][0] = a[r][1] = a[r][2] = a[r][3] = 0;
                continue;
              }
              const uint32_t at =
                  buf + scale_at<kPieces, P::kPiece>(32 * (r0 + r) + lane, i);
              if constexpr (P::kWords == 2)
                asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];"
                             : "=r"(a[r][0]), "=r"(a[r][1])
                             : "r"(at)
                             : "memory");
              else
                asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                             : "=r"(a[r][0]), "=r"(a[r][1]), "=r"(a[r][2]),
                               "=r"(a[r][3])
                             : "r"(at)
                             : "memory");
            }
#pragma unroll
            for (int w = 0; w < P::kWords; ++w)
              tmem_st4(r0 == 0 ? cols + 4 * w
                               : cols + P::kWords * 4 + P::kBCols * w + r0 - 4,
                       a[0][w], a[1][w], a[2][w], a[3][w]);
          }
          tmem_st_wait();
          tc_fence_before_sync();
          if (lane == 0) mbar_arrive(ready + 8 * s);
          __syncwarp();
        }
      }
    }
  } else {
    const int q = warp & 3, half = (warp - P::kDrainWarp) >> 2;  // lanes, columns
    constexpr int kCols = NT / 2;
    const float g = args.wg != nullptr ? *args.wg : 1.0f;
    const Factors both =
        FMT == TQ_FMT_NV4
            ? scale_factors(g, args.xg != nullptr ? *args.xg : 1.0f)
            : Factors{1.0f, 1.0f};
    // bf16 pairs need an even row pitch and a 4-byte aligned y
    const bool pairs = args.y_bf16 && args.ldy % 2 == 0 && args.n % 2 == 0 &&
                       (reinterpret_cast<uintptr_t>(args.y) & 3u) == 0;
    uint32_t done = 0;
    bool ok = true;
    for (int t = group; t < tiles; t += groups, ++done) {
      if (ok) ok = mbar_wait(dfull, done & 1u, abort_addr, kWaitLimitNs);
      ok = __all_sync(0xFFFFFFFFu, ok);
      tc_fence_after_sync();
      const int64_t row = (int64_t)(t / args.tiles_n) * (CG * kRowsM) +
                          rank * kRowsM + 32 * q + lane;
      const int64_t b0 = (int64_t)(t % args.tiles_n) * NT + half * kCols;
      const int cols = (int)(args.batch - b0 < kCols ? args.batch - b0 : kCols);
      const uint32_t src = kTmem + half * kCols + ((uint32_t)q << 21);
      const float gn = ok ? both.a : __int_as_float(0x7FC00000);
      // accumulators times the tensor scales, two at once
      auto scale = [&](uint32_t (&v)[16]) {
        const F2 a = pack2(gn, gn), b = pack2(both.b, both.b);
#pragma unroll
        for (int j = 0; j < 16; j += 2) {
          F2 p = pack2(__uint_as_float(v[j]), __uint_as_float(v[j + 1]));
          if (FMT == TQ_FMT_NV4) p = mul2(p, b);
          p = mul2(p, a);
          asm("mov.b64 {%0, %1}, %2;" : "=r"(v[j]), "=r"(v[j + 1]) : "l"(p.v));
        }
      };
      auto drained = [&]() {  // the accumulator may be written again
        tc_fence_before_sync();
        __syncwarp();
        if (!ok || lane != 0) return;
        if (CG == 2)
          arrive_leader(dempty);
        else
          mbar_arrive(dempty);
      };
      // Chunks past the batch are left out; the branch also keeps a chunk's
      // arithmetic behind its load (without it every column stayed in 32 bits
      // until the end and was spilled: 4900 cycles for the 128 columns of a
      // warp instead of 1150). As many columns as 64 registers hold are read
      // first, so that the next tile can start while they are stored: all of
      // them as bf16 pairs (two columns of this lane's row), 64 in fp32.
      uint32_t h[kCols / 2] = {};
      if (args.digits.exps != nullptr) {
        const DigitArgs &D = args.digits;
        const float one = ok ? g : __int_as_float(0x7FC00000);
        const TensorScale ts = FMT == TQ_FMT_NV4 ? tensor_scale(one)
                                                 : TensorScale{one, 0};
#pragma unroll
        for (int c = 0; c < kCols; c += 16) {
          if (c >= cols) break;
          uint32_t v[16];
          tmem_ld16(src + c, v);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int64_t b = (b0 + c) / 8 + j;
            const int e = c + 8 * j < cols ? __ldg(D.exps + b) : 0;
            h[c / 8 + j] =
                __float_as_uint(digit_sum<FMT>(&v[8 * j], e, ts));
          }
        }
        drained();
        float *p = static_cast<float *>(args.y) + b0 / 8 * args.ldy + row;
        if (row < args.n) {
#pragma unroll
          for (int j = 0; j < kCols / 8; ++j) {
            if (8 * j < cols) {
              float f = __uint_as_float(h[j]);
              const int64_t b = b0 / 8 + j;
              if (__ldg(D.odd + b))
                f += g * odd_products<FMT>(D.x + b * D.ldx, 0, args.k,
                                           args.wcodes, args.wscales, row,
                                           args.k);
              *p = f;
            }
            p += args.ldy;
          }
        }
        __syncwarp();
      } else if (args.y_bf16) {
#pragma unroll
        for (int c = 0; c < kCols; c += 16) {
          if (c >= cols) break;
          uint32_t v[16];
          tmem_ld16(src + c, v);
          tmem_ld_wait();
          scale(v);
#pragma unroll
          for (int j = 0; j < 8; ++j)
            h[c / 2 + j] = bf16_pair(v[2 * j], v[2 * j + 1]);
        }
        drained();
        __nv_bfloat16 *y = static_cast<__nv_bfloat16 *>(args.y);
        if (pairs) {
          // lanes 2i and 2i + 1 swap, so that each stores two neighbouring
          // rows of one column: the even lane column 2j, the odd lane 2j + 1
          const int odd = lane & 1;
          __nv_bfloat16 *p = y + (b0 + odd) * args.ldy + (row - odd);
#pragma unroll
          for (int j = 0; j < kCols / 2; ++j) {
            const uint32_t o = __shfl_xor_sync(0xFFFFFFFFu, h[j], 1);
            const uint32_t two =
                odd ? __byte_perm(o, h[j], 0x7632) : __byte_perm(h[j], o, 0x5410);
            if (row < args.n && 2 * j + odd < cols)
              *reinterpret_cast<uint32_t *>(p) = two;
            p += 2 * args.ldy;
          }
        } else if (row < args.n) {
          __nv_bfloat16 *p = y + b0 * args.ldy + row;
#pragma unroll
          for (int j = 0; j < kCols; ++j) {
            const uint32_t two = h[j / 2];
            if (j < cols)
              *p = __ushort_as_bfloat16(
                  (unsigned short)(j & 1 ? two >> 16 : two));
            p += args.ldy;
          }
        }
      } else {
        constexpr int kHeld = kCols / 2;
        float *p = static_cast<float *>(args.y) + b0 * args.ldy + row;
#pragma unroll 1
        for (int c = 0; c < kCols; c += kHeld) {
#pragma unroll
          for (int i = 0; i < kHeld; i += 16) {
            if (c + i >= cols) break;
            uint32_t v[16];
            tmem_ld16(src + c + i, v);
            tmem_ld_wait();
            scale(v);
#pragma unroll
            for (int j = 0; j < 16; ++j) h[i + j] = v[j];
          }
          if (c + kHeld >= kCols) drained();
          if (row < args.n) {
#pragma unroll
            for (int j = 0; j < kHeld; ++j) {
              if (c + j < cols) *p = __uint_as_float(h[j]);
              p += args.ldy;
            }
          }
          __syncwarp();
        }
      }
    }
  }

  __syncwarp();
  tc_fence_before_sync();
  __syncthreads();
  if (CG == 2) {
    asm volatile("barrier.cluster.arrive.aligned;\n"
                 "barrier.cluster.wait.aligned;" ::: "memory");
  }
  if (warp == 0) {
    tc_fence_after_sync();
    free_columns<CG>(kTmem, kTmemColumns);
  }
}

template <int FMT, int NT, int CG>
cudaError_t launch(const WeightsView &w, const WeightsView &x, Args a,
                   cudaStream_t stream) {
  using P = Plan<FMT, NT, CG>;
  int dev = 0, sms = 148;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  CUtensorMap mw, mx;
  if ((e = code_map(&mw, w, kRowsM)) != cudaSuccess) return e;
  if ((e = code_map(&mx, x, NT / CG)) != cudaSuccess) return e;
  a.tiles_m = (int)((w.n + CG * kRowsM - 1) / (CG * kRowsM));
  a.tiles_n = (int)((x.n + NT - 1) / NT);
  const int64_t tiles = (int64_t)a.tiles_m * a.tiles_n;
  const int groups = (int)(tiles < sms / CG ? tiles : sms / CG);
  auto kern = product_f4_kernel<FMT, NT, CG>;
  if ((e = ensure_smem_limit<product_f4_kernel<FMT, NT, CG>>(
           (int)P::kSmem)) != cudaSuccess)
    return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(groups * CG));
  cfg.blockDim = dim3(P::kThreads);
  cfg.dynamicSmemBytes = P::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = CG;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = CG == 1 ? 1 : 2;
  return cudaLaunchKernelEx(&cfg, kern, mw, mx, a);
}

template <int FMT>
cudaError_t dispatch(const WeightsView &w, const WeightsView &x, const Args &a,
                     cudaStream_t stream) {
  // A wave of 256 x 256 tiles takes about 7/5 of the time of a wave of 128 x
  // 128 tiles, two of which cover half of it, so the large tile wins where its
  // waves are full: MX4 (NV4) 101 (113) against 129 (150) us at 21504 x 5376 x
  // 2048 rows, but 30 (36) against 22 (25) us at 5376 x 8192 x 777 rows (84
  // tiles on 74 pairs) and 9.8 (9.2) against 5.8 (6.1) us at 1024 x 1024 x
  // 1024.
  int dev = 0, sms = 148;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  auto waves = [&](int64_t m, int64_t b, int64_t at_once) {
    const int64_t tiles = ((w.n + m - 1) / m) * ((x.n + b - 1) / b);
    return (tiles + at_once - 1) / at_once;
  };
  if (x.n > 128 && 7 * waves(256, 256, sms / 2) <= 5 * waves(128, 128, sms))
    return launch<FMT, 256, 2>(w, x, a, stream);
  return launch<FMT, 128, 1>(w, x, a, stream);
}

Args args_of(const WeightsView &w, const WeightsView &x, void *y, int64_t ldy) {
  Args a = {};
  a.wscales = reinterpret_cast<const uint8_t *>(w.scales);
  a.xscales = reinterpret_cast<const uint8_t *>(x.scales);
  a.wg = w.lut;
  a.xg = x.lut;
  a.y = y;
  a.n = w.n;
  a.batch = x.n;
  a.ldy = ldy;
  a.k = (int)w.k;
  a.wcodes = w.codes;
  return a;
}

}  // namespace

cudaError_t product_f4(const WeightsView &w, const WeightsView &x, void *y,
                       int64_t ldy, int y_type, const DigitArgs &digits,
                       cudaStream_t stream) {
  // up to 64 rows the kernel that splits K (8192 x 5376 x 16 rows: 8.6 against
  // 10.8 us); for 128 both take the same
  if (x.n <= 64)
    return decode_f4_packed(w, x, y, ldy, y_type, digits, stream);
  Args a = args_of(w, x, y, ldy);
  a.y_bf16 = y_type == TQ_Y_BF16;
  a.digits = digits;
  return w.format == TQ_FMT_MX4 ? dispatch<TQ_FMT_MX4>(w, x, a, stream)
                                : dispatch<TQ_FMT_NV4>(w, x, a, stream);
}

cudaError_t launch_linear_f4(const WeightsView &w, const WeightsView &x,
                             void *y, int64_t ldy, int y_type,
                             cudaStream_t stream) {
  return product_f4(w, x, y, ldy, y_type, DigitArgs{}, stream);
}

}  // namespace tq
