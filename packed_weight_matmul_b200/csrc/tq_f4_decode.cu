// Few rows of x times 4-bit weights on the block-scaled tensor cores, without
// decoding a weight:
//
//   y[b][n] = g sum_k c[n][k] s[n][k / B] x[b][k]
//
// The codes of 128 weight rows go from global to shared memory by TMA as they
// lie, their scales to tensor memory, and tcgen05.mma (kind mxf4 / mxf4nvf4)
// multiplies them by a 4-bit x. Packed x (tq_linear_f4) is such a matrix
// already. A bf16 x is written as a sum of 8 of them, exactly enough
// (tq_f4_digits.cuh: base-8 digits, row 8 b + i of the B operand holds digit i
// of row b of x).
//
// Bound by the codes' way from HBM: an MMA of 64 k takes 41 to 64 cycles for
// 8192 weights, 2 to 3 times the rate at which HBM delivers them. A digit
// costs 3 lane instructions per value of x and CTA, so a pass takes 4 bf16
// rows (packed ones: 32 or 64). MX4, 8192 x 5376: 1 row 10.0 us, 16 packed
// rows 8.7 us (HBM alone 3.6; 5 us are start-up and the sum over the cluster);
// 21504 x 5376, 1 row: 16.8 us, 3.7 TB/s; 64 rows over 128 experts of 768 x
// 2048: 18 us.
//
// One CTA per 128 weight rows and slice of K, two CTAs per SM (one starts up
// or ends while the other streams), the slices of a tile in a cluster that
// adds them in rank order through distributed shared memory. 14 warps:
//   warp 0       TMA producer (codes; packed x); tensor-memory allocation
//   warp 1       MMA issuer
//   warps 2-5    scales to tensor memory, as in tq_f4_gemm.cu (packed x: and
//                warps 6-9, in turn)
//   warps 6-13   bf16 x: exponents, digits into the swizzled B tiles; the first
//                four read the accumulator at the end
// Every wait is bounded; one that gives up leaves NaN in the CTA's outputs.
#include <cooperative_groups.h>

#include "tq_f4_digits.cuh"
#include "tq_f4_tc.cuh"

namespace tq {
using namespace f4;
namespace {

constexpr int kTile = 128;
constexpr int kThreads = 448, kXThreads = 256;
constexpr int kStageK = 256;
constexpr uint32_t kColumns = 256;            // tensor memory, half of an SM's
constexpr uint32_t kSmemLimit = 113u * 1024u;  // two CTAs per SM
constexpr int kSegment = 1024;                // ids looked through at once
constexpr int kMapExperts = 4096;

enum { kBf16 = 0, kPacked = 1 };

template <int FMT, int NT, int SRC>
struct DecodePlan {
  static constexpr int kTerms = SRC == kBf16 ? 8 : 1;
  static constexpr int kRows = NT / kTerms;  // rows of x per pass
  static constexpr int kWords = FMT == TQ_FMT_MX4 ? 2 : 4;  // scale words/row
  static constexpr uint32_t kBCols = NT / 32 > 4 ? NT / 32 : 4;
  static constexpr uint32_t kScaleCols = kWords * (4 + kBCols);
  static constexpr uint32_t kA = kTile * kF4StageRow;
  static constexpr uint32_t kB = NT * kF4StageRow;
  static constexpr uint32_t kPiece = kWords * 4;  // scale bytes of a stage
  // Packed x leaves warps free: a second group of four moves scales, and they
  // take turns by units of 2 stages. A wait by parity is right one phase
  // ahead, so the ring has to be longer than the other group's unit.
  static constexpr int kGroups = SRC == kPacked ? 2 : 1;
  static constexpr int kUnitStages = SRC == kPacked ? 2 : 4;
  static constexpr uint32_t kUnit = kUnitStages * kPiece;
  static constexpr int kScaleRows = kTile + (SRC == kPacked ? NT : 0);
  static constexpr uint32_t kScales = kScaleRows * kUnit;  // of one group
  static constexpr uint32_t kExp = SRC == kBf16 ? kRows * 16 : 0;
  static constexpr uint32_t kFixed = 2048 + kGroups * kScales +
                                     (SRC == kBf16 ? kSegment * 4 + 1024 : 0);
  static constexpr int kFit = (int)((kSmemLimit - kFixed) / (kA + kB + kExp));
  static constexpr int kFitT = (int)((kColumns - NT) / kScaleCols);
  static constexpr int kStages0 = kFit < kFitT ? kFit : kFitT;
  static constexpr int kStages = kStages0 < 8 ? kStages0 : 8;
  static_assert(kStages >= 3 && (kGroups == 1 || kStages > kUnitStages),
                "ring too short");
  static constexpr uint32_t kOffB = kStages * kA;
  static constexpr uint32_t kOffS = kOffB + kStages * kB;
  static constexpr uint32_t kOffE = kOffS + kGroups * kScales;
  static constexpr uint32_t kOffBar = kOffE + kStages * kExp;
  static constexpr uint32_t kSmem = kOffBar + 256 + 1024;
  static constexpr int kPitch = kTile + 4;  // of the partial tile
  static_assert(kRows * kPitch * 4 <= kOffS, "partial tile");
  static_assert(SRC == kPacked || kRows == 4, "rows that share a stage");
};

struct DecodeArgs {
  const uint8_t *codes, *wscales;  // of expert 0
  const float *wg;
  const __nv_bfloat16 *x;  // bf16
  int64_t ldx;
  const uint8_t *xscales;  // packed
  const float *xg;
  DigitArgs digits;  // packed
  void *y;
  int64_t n, batch, ldy;
  int k, y_bf16, ks;
  const int32_t *ids;  // null: one matrix, rows of x in order
  int n_experts, slots;
  int32_t *status;
};

__device__ __forceinline__ void mbar_arrive_n(uint32_t bar, uint32_t n) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(n)
               : "memory");
}

__device__ __forceinline__ void fence_async() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

template <int FMT, int NT, int SRC>
__global__ void __launch_bounds__(kThreads, 2)
    decode_f4_kernel(const __grid_constant__ CUtensorMap tmap_w,
                     const __grid_constant__ CUtensorMap tmap_x,
                     const DecodeArgs a) {
  using P = DecodePlan<FMT, NT, SRC>;
  constexpr int S = P::kStages;
  extern __shared__ uint8_t smem_raw[];
  __shared__ int s_rows[SRC == kBf16 ? kSegment : 1];
  __shared__ int s_count[kSegment / 32 + 2];
  __shared__ int s_exp[P::kRows], s_odd[P::kRows];
  __shared__ Factors s_both;  // packed x: both tensor scales
  __shared__ uint32_t s_map[SRC == kBf16 ? kMapExperts / 32 : 1];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t bars = base + P::kOffBar;
  const uint32_t ready = bars, empty = bars + 8 * S, xready = bars + 16 * S;
  const uint32_t dfull = bars + 24 * S, slot = dfull + 8;
  const uint32_t abort_addr = dfull + 12;
  const int ks = a.ks, rank = ks > 1 ? (int)cluster_rank() : 0;
  const int64_t row0 = (int64_t)(blockIdx.x / ks) * kTile;
  const int all = (a.k + kStageK - 1) / kStageK;
  const int st0 = (int)((int64_t)all * rank / ks);
  const int steps = (int)((int64_t)all * (rank + 1) / ks) - st0;

  pdl_launch_dependents();
  if (tid == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(ready + 8 * s, 4 + 1);
      mbar_init(empty + 8 * s, 1);
      mbar_init(xready + 8 * s, 8);
    }
    mbar_init(dfull, 1);
    st_volatile_s32(abort_addr, 0);
    mbar_init_fence();
    if (a.ids == nullptr)  // hint the L2 cache with the first codes
      for (int i = 0; i < 8 && i < steps; ++i)
        tma_prefetch_2d(&tmap_w, (st0 + i) * (int)kF4StageRow, (int)row0);
  }
  if (warp == 0) tmem_alloc(slot, kColumns);
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  // the same in every lane, which keeps it in a uniform register
  const uint32_t tmem =
      __reduce_max_sync(0xFFFFFFFFu, (uint32_t)ld_volatile_s32(slot));
  const uint32_t tmem_scales = tmem + NT;
  pdl_wait();

  int64_t expert = a.ids != nullptr ? blockIdx.y : 0;
  uint32_t done = 0;  // stages of the passes before

  // packed rows that make one row of y
  const int per = SRC == kPacked && a.digits.exps != nullptr ? 8 : 1;
  // `rows` rows of x (s_rows[first + i], or b0 + i): one pass over K
  auto pass = [&](int pass_no, int first, int64_t b0, int rows) {
    const int64_t wrow = expert * a.n + row0;  // first weight row
    // bf16 x: warps that share a stage's rows (their arrivals add up to 8),
    // one row each, and stages in work at once: a wait by parity is right one
    // phase ahead, so a warp skips S stages at most.
    const int per_stage = rows <= 1 ? 1 : rows <= 2 ? 2 : 4;
    const int at_once = 8 / per_stage < S ? 8 / per_stage : S;
    // Scales to tensor memory: group `turn` of four warps.
    auto move_scales = [&](int turn) {
      const int at = (tid - 64) & 127;
      const uint32_t quarter = (uint32_t)(warp & 3) << 21;
      const int row_bytes = a.k / f4_block(FMT);
      const bool whole = a.k % kStageK == 0;
      const uint32_t buf = base + P::kOffS + turn * P::kScales;
      constexpr int kPieces = P::kUnitStages, kPass = 128 / kPieces;
      constexpr int kPieceWords = (int)P::kPiece / 4;
      constexpr int kLoads = (P::kScaleRows + kPass - 1) / kPass;
      const int my_row = at / kPieces, my_piece = at % kPieces;
      const int64_t m = wrow < (expert + 1) * a.n ? wrow : (expert + 1) * a.n - 1;
      const int64_t wleft = (expert + 1) * a.n - 1 - m;
      const int wlast = (int)(wleft < kTile ? wleft : kTile);
      const int xlast = rows - 1;
      const uint8_t *wrows = a.wscales + m * row_bytes;
      const uint8_t *xrows =
          SRC == kPacked ? a.xscales + b0 * row_bytes : a.wscales;
      uint32_t v[kLoads][kPieceWords];
      auto load = [&](int u) {
        const int off =
            (st0 + u * P::kUnitStages + my_piece) * (int)P::kPiece;
        auto each = [&](auto read) {
#pragma unroll
          for (int j = 0; j < kLoads; ++j) {
            const bool of_w = kPass * (j + 1) <= kTile;
            int r = my_row + kPass * j - (of_w ? 0 : kTile);
            r = min(r, of_w ? wlast : xlast);
            read(v[j], (of_w ? wrows : xrows) + (int64_t)r * row_bytes + off);
          }
        };
        if (whole)
          each([&](uint32_t (&d)[kPieceWords], const uint8_t *p) {
            load_piece(d, p, row_bytes - off);
          });
        else
          each([&](uint32_t (&d)[kPieceWords], const uint8_t *p) {
            load_piece_shifted(d, p, row_bytes - off);
          });
      };
      const int units = (steps + P::kUnitStages - 1) / P::kUnitStages;
      if (turn < units) load(turn);
      bool ok = true;
#pragma unroll 1
      for (int u = turn; u < units; u += P::kGroups) {
        bar_sync(1 + 2 * turn, 128);  // the last unit has been read
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
          if (FMT == TQ_FMT_NV4) {  // E4M3 scales are read without their sign
#pragma unroll
            for (int w = 0; w < kPieceWords; ++w) v[j][w] &= 0x7F7F7F7Fu;
          }
          if (my_row + kPass * j < P::kScaleRows)
            store_piece(buf + scale_at<kPieces, P::kPiece>(my_row + kPass * j,
                                                           my_piece),
                        v[j]);
        }
        bar_sync(1 + 2 * turn, 128);
        if (u + P::kGroups < units) load(u + P::kGroups);
        const int left = steps - u * P::kUnitStages;
#pragma unroll 1
        for (int i = 0; i < left && i < P::kUnitStages; ++i) {
          const uint32_t it = done + u * P::kUnitStages + i;
          const uint32_t s = it % S, ph = (it / S) & 1u;
          // after a wait that gave up, the warps only keep meeting at the
          // barriers above
          if (ok)
            ok = mbar_wait(empty + 8 * s, ph ^ 1u, abort_addr, kWaitLimitNs);
          if (SRC == kBf16 && ok)
            ok = mbar_wait(xready + 8 * s, ph, abort_addr, kWaitLimitNs);
          ok = __all_sync(0xFFFFFFFFu, ok);
          if (!ok) continue;
          tc_fence_after_sync();
          const uint32_t cols = tmem_scales + s * P::kScaleCols + quarter;
#pragma unroll
          for (int r0 = 0; r0 < 4 + (int)P::kBCols; r0 += 4) {
            uint32_t w[4][4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const int row = 32 * (r0 + r);
              if (row >= kTile + NT) {
                w[r][0] = w[r][1] = w[r][2] = w[r][3] = 0;
                continue;
              }
              // x rows 8 b + i: the block scales of row b of x
              const int n_row = row - kTile + lane;
              const uint32_t from =
                  SRC == kPacked || r0 == 0
                      ? buf + scale_at<kPieces, P::kPiece>(row + lane, i)
                      : base + P::kOffE + s * P::kExp + (n_row >> 3) * 16;
              if constexpr (P::kWords == 2)
                asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];"
                             : "=r"(w[r][0]), "=r"(w[r][1])
                             : "r"(from)
                             : "memory");
              else
                asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                             : "=r"(w[r][0]), "=r"(w[r][1]), "=r"(w[r][2]),
                               "=r"(w[r][3])
                             : "r"(from)
                             : "memory");
              if (SRC == kBf16 && FMT == TQ_FMT_MX4 && r0 != 0) {
                const uint32_t lower = (uint32_t)(n_row & 7) * 0x03030303u;
                w[r][0] = __vsubus4(w[r][0], lower);
                w[r][1] = __vsubus4(w[r][1], lower);
              }
            }
#pragma unroll
            for (int j = 0; j < P::kWords; ++j)
              tmem_st4(r0 == 0 ? cols + 4 * j
                               : cols + P::kWords * 4 + P::kBCols * j + r0 - 4,
                       w[0][j], w[1][j], w[2][j], w[3][j]);
          }
          tmem_st_wait();
          tc_fence_before_sync();
          if (lane == 0) mbar_arrive(ready + 8 * s);
          __syncwarp();
        }
      }
    };

    if (FMT == TQ_FMT_NV4 && SRC == kPacked && tid == kThreads - 1)
      s_both = scale_factors(a.wg != nullptr ? *a.wg : 1.0f,
                             a.xg != nullptr ? *a.xg : 1.0f);
    if (warp == 0) {
      if (lane == 0) {
        bool ok = true;
        int i = 0;
        for (; i < steps; ++i) {
          const uint32_t it = done + i, s = it % S, ph = (it / S) & 1u;
          ok = mbar_wait(empty + 8 * s, ph ^ 1u, abort_addr, kWaitLimitNs);
          if (!ok) break;
          mbar_arrive_expect_tx(ready + 8 * s,
                                P::kA + (SRC == kPacked ? P::kB : 0u));
          tma_load_2d(base + s * P::kA, &tmap_w,
                      (st0 + i) * (int)kF4StageRow, (int)wrow, ready + 8 * s);
          if (SRC == kPacked)
            tma_load_2d(base + P::kOffB + s * P::kB, &tmap_x,
                        (st0 + i) * (int)kF4StageRow, (int)b0, ready + 8 * s);
        }
        // every copy issued has landed, and every MMA that read one is done
        for (int j = i > S ? i - S : 0; j < i; ++j)
          mbar_wait(empty + 8 * ((done + j) % S), ((done + j) / S) & 1u);
      }
    } else if (warp == 1) {
      bool ok = true, here = false;
      int i = 0;
      for (; i < steps; ++i) {  // the whole warp, see mma_stage
        const uint32_t it = done + i, s = it % S, ph = (it / S) & 1u;
        if (!here) {
          ok = mbar_wait(ready + 8 * s, ph, abort_addr, kWaitLimitNs);
          ok = __all_sync(0xFFFFFFFFu, ok);
          if (!ok) break;
        }
        tc_fence_after_sync();
        const bool next =
            mbar_test<1>(ready + 8 * ((it + 1) % S), ((it + 1) / S) & 1u);
        const uint32_t sa = tmem_scales + s * P::kScaleCols;
        mma_stage<FMT, 1>(
            tmem, smem_desc_kmajor_sw128(base + s * P::kA),
            smem_desc_kmajor_sw128(base + P::kOffB + s * P::kB),
            idesc_f4<FMT>(kTile, NT, 0u),
            idesc_f4<FMT>(kTile, NT, FMT == TQ_FMT_MX4 ? 2u : 0u), sa,
            sa + P::kWords * 4, P::kBCols, i != 0 ? 1u : 0u, empty + 8 * s);
        here = __all_sync(0xFFFFFFFFu, next);
      }
      if (ok) commit<1>(dfull);
      for (int j = i > S ? i - S : 0; j < i; ++j)
        mbar_wait(empty + 8 * ((done + j) % S), ((done + j) / S) & 1u);
    } else if (warp < 6) {
      move_scales(0);
    } else {
      if (P::kGroups == 2 && warp < 10) move_scales(1);
      const int xw = warp - 6, xt = tid - 192;
      const int64_t k0 = (int64_t)st0 * kStageK;
      const int64_t k1 = k0 + (int64_t)steps * kStageK < a.k
                             ? k0 + (int64_t)steps * kStageK
                             : a.k;
      auto x_row = [&](int r) {
        return a.x + (a.ids != nullptr ? s_rows[first + r] : b0 + r) * a.ldx;
      };
      if constexpr (SRC == kBf16) {
        // the first values to convert, on their way during what follows
        const int mine = xw % per_stage;  // this warp's row
        uint4 next;
        auto load = [&](int i) {
          const int64_t k = k0 + (int64_t)i * kStageK + 8 * lane;
          next = make_uint4(0, 0, 0, 0);
          if (mine < rows && i < steps && k < k1)
            next = __ldg(reinterpret_cast<const uint4 *>(x_row(mine) + k));
        };
        // warps past the last group of per_stage have no stages of their own
        const int start = xw / per_stage < at_once ? xw / per_stage : steps;
        load(start);
        // Exponent of each row's largest value in the slice; few rows are
        // shared by several warps.
        for (int r = xt; r < rows; r += kXThreads) {
          s_exp[r] = 1;
          s_odd[r] = 0;
        }
        bar_sync(2, kXThreads);
        const int parts = 8 / rows;
        for (int u = xw; u < rows * parts; u += 8) {
          const int r = u % rows, part = u / rows;
          const __nv_bfloat16 *p = x_row(r);
          uint32_t m = 0, odd = 0;
          for (int64_t k = k0 + 8 * lane + 1024 * part; k < k1;
               k += 1024 * parts) {
            uint4 v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              v[j] = make_uint4(0, 0, 0, 0);
              if (k + 256 * j < k1)
                v[j] = __ldg(reinterpret_cast<const uint4 *>(p + k + 256 * j));
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              uint32_t t = max_mag8(v[j]);
              if (t >= 0x7F80u) {
                odd = 1;
                t = max_mag8(only_finite8(v[j]));
              }
              m = max(m, t);
            }
          }
          m = __reduce_max_sync(0xFFFFFFFFu, m);
          odd = __reduce_max_sync(0xFFFFFFFFu, odd);
          if (lane == 0) {
            atomicMax(&s_exp[r], (int)(m >> 7));
            if (odd) s_odd[r] = 1;
          }
        }
        // B rows and exponents of rows of x that are not there
        for (int i = xt; i < S * (P::kRows - rows) * 64; i += kXThreads) {
          const int s = i / ((P::kRows - rows) * 64);
          const int j = i % ((P::kRows - rows) * 64);
          asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(
                           base + P::kOffB + s * P::kB + rows * 1024 + j * 16),
                       "r"(0)
                       : "memory");
          if (j < P::kRows - rows)
            asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(
                             base + P::kOffE + s * P::kExp + (rows + j) * 16),
                         "r"(0)
                         : "memory");
        }
        fence_async();
        bar_sync(2, kXThreads);
        int i = start;
#pragma unroll 1
        for (; i < steps; i += at_once) {
          const uint32_t it = done + i, s = it % S, ph = (it / S) & 1u;
          uint4 w = next;
          load(i + at_once);
          bool ok = mbar_wait(empty + 8 * s, ph ^ 1u, abort_addr, kWaitLimitNs);
          ok = __all_sync(0xFFFFFFFFu, ok);
          if (!ok) break;
          if (mine < rows) {
            if (s_odd[mine]) w = only_finite8(w);
            uint32_t m = max_mag8(w);
            m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
            if (FMT == TQ_FMT_MX4)
              m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
            uint32_t byte, field;
            digit_scale<FMT>(max((int)(m >> 7), 1), s_exp[mine], &byte,
                             &field);
            constexpr int kLanes = f4_block(FMT) / 8;
            if (lane % kLanes == 0)
              asm volatile("st.shared.u8 [%0], %1;" ::"r"(
                               base + P::kOffE + s * P::kExp + mine * 16 +
                               lane / kLanes),
                           "r"(byte)
                           : "memory");
            // row 8 mine + i: 16-byte chunk c (32 codes) lies at c ^ i
            const uint32_t at =
                base + P::kOffB + s * P::kB + mine * 1024 + (lane & 3) * 4;
            digits8(w, field, [&](int d, uint32_t codes) {
              asm volatile("st.shared.b32 [%0], %1;" ::"r"(
                               at + d * 128 + (((lane >> 2) ^ d) << 4)),
                           "r"(codes)
                           : "memory");
            });
          }
          fence_async();
          __syncwarp();
          if (lane == 0) mbar_arrive_n(xready + 8 * s, 8 / per_stage);
        }
      }
      if (warp < 10) {
        const float wg = a.wg != nullptr ? a.wg[expert] : 1.0f;
        const bool ok0 = mbar_wait(dfull, (uint32_t)pass_no & 1u, abort_addr,
                                   kWaitLimitNs);
        const bool ok = __all_sync(0xFFFFFFFFu, ok0);
        tc_fence_after_sync();
        const int q = warp & 3, r = 32 * q + lane;
        float *part = reinterpret_cast<float *>(smem_raw + (base - smem_u32(smem_raw)));
        const TensorScale ts = FMT == TQ_FMT_NV4 ? tensor_scale(wg)
                                                 : TensorScale{1.0f, 0};
#pragma unroll 1
        for (int c = 0; c < rows * P::kTerms; c += 16) {
          uint32_t v[16];
          tmem_ld16(tmem + c + ((uint32_t)q << 21), v);
          tmem_ld_wait();
          if (SRC == kPacked && per == 8) {
            const DigitArgs &D = a.digits;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int b = c / 8 + h;
              if (8 * b >= rows) break;
              const int64_t at = b0 / 8 + b;
              float t = digit_sum<FMT>(&v[8 * h], D.exps[at], ts);
              if (D.odd[at] && row0 + r < a.n)
                t += wg * odd_products<FMT>(D.x + at * D.ldx, (int)k0, (int)k1,
                                       a.codes, a.wscales, wrow + r, a.k);
              part[b * P::kPitch + r] = ok ? t : __int_as_float(0x7FC00000);
            }
          } else if constexpr (SRC == kPacked) {
#pragma unroll
            for (int j = 0; j < 16; ++j)
              if (c + j < rows)
                part[(c + j) * P::kPitch + r] =
                    ok ? __uint_as_float(v[j]) : __int_as_float(0x7FC00000);
          } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int b = c / 8 + h;
              if (b >= rows) break;
              float t = digit_sum<FMT>(&v[8 * h], s_exp[b], ts);
              if (s_odd[b] && row0 + r < a.n)
                t += wg * odd_products<FMT>(x_row(b), (int)k0, (int)k1, a.codes,
                                       a.wscales, wrow + r, a.k);
              part[b * P::kPitch + r] = ok ? t : __int_as_float(0x7FC00000);
            }
          }
        }
        tc_fence_before_sync();
      }
    }
    __syncwarp();
    if (ks > 1)
      cooperative_groups::this_cluster().sync();
    else
      __syncthreads();
    for (int i = tid + rank * kThreads; i < rows / per * kTile;
         i += ks * kThreads) {
      const int b = i / kTile, r = i % kTile;
      if (row0 + r >= a.n) continue;  // every read is stored, see below
      const uint32_t at = base + (uint32_t)(b * P::kPitch + r) * 4;
      float v = 0.0f;
      for (int c = 0; c < ks; ++c) {
        float u;
        if (ks == 1) {
          asm volatile("ld.shared.f32 %0, [%1];" : "=f"(u) : "r"(at) : "memory");
        } else {
          uint32_t remote;
          asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                       : "=r"(remote)
                       : "r"(at), "r"(c));
          asm volatile("ld.shared::cluster.f32 %0, [%1];"
                       : "=f"(u)
                       : "r"(remote)
                       : "memory");
        }
        v += u;
      }
      // (digit_sum has applied the tensor scale)
      if (FMT == TQ_FMT_NV4 && SRC == kPacked && per == 1)
        v = v * s_both.b * s_both.a;
      const int64_t row = a.ids != nullptr ? s_rows[first + b] : b0 / per + b;
      if (a.y_bf16)
        static_cast<__nv_bfloat16 *>(a.y)[row * a.ldy + row0 + r] =
            __float2bfloat16_rn(v);
      else
        static_cast<float *>(a.y)[row * a.ldy + row0 + r] = v;
    }
    // The partial tiles have been read (each value that was read has gone into
    // a store, which was issued before this barrier's arrival); what comes next
    // writes there by copies.
    fence_async();
    if (ks > 1)
      cluster_sync_relaxed();
    else
      __syncthreads();
    done += steps;
  };

  if (a.ids == nullptr) {
    const int64_t b0 = (int64_t)blockIdx.y * P::kRows;
    pass(0, 0, b0,
         (int)(a.batch - b0 < P::kRows ? a.batch - b0 : P::kRows));
  } else if constexpr (SRC == kBf16) {
    // The first slot looks for ids that name no expert: NaN in their rows.
    if (blockIdx.y == 0 && rank == 0) {
      for (int64_t i = tid; i < a.batch; i += kThreads) {
        const int32_t id = __ldg(a.ids + i);
        if (id >= 0 && id < a.n_experts) continue;
        const int64_t end = row0 + kTile < a.n ? row0 + kTile : a.n;
        for (int64_t r = row0; r < end; ++r)
          static_cast<float *>(a.y)[i * a.ldy + r] = __int_as_float(0x7FC00000);
        report(a.status, TQ_ERR_INVALID_ARG);
      }
    }
    bool mine = true;
    if (a.slots < a.n_experts) {
      // fewer rows than experts: slot j takes the j-th expert that has any
      for (int i = tid; i < kMapExperts / 32; i += kThreads) s_map[i] = 0;
      __syncthreads();
      for (int64_t i = tid; i < a.batch; i += kThreads) {
        const int32_t id = __ldg(a.ids + i);
        if (id >= 0 && id < a.n_experts)
          atomicOr(&s_map[id >> 5], 1u << (id & 31));
      }
      __syncthreads();
      if (warp == 0) {
        constexpr int kEach = kMapExperts / 32 / 32;
        int c = 0;
#pragma unroll
        for (int j = 0; j < kEach; ++j) c += __popc(s_map[lane * kEach + j]);
        int before = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int v = __shfl_up_sync(0xFFFFFFFFu, before, o);
          if (lane >= o) before += v;
        }
        if (lane == 31) s_count[kSegment / 32 + 1] = -1;
        __syncwarp();
        before -= c;
        int want = (int)blockIdx.y - before;
        if (want >= 0 && want < c) {
          for (int j = 0; j < kEach; ++j) {
            uint32_t w = s_map[lane * kEach + j];
            const int p = __popc(w);
            if (want >= p) {
              want -= p;
              continue;
            }
            for (; want > 0; --want) w &= w - 1;
            s_count[kSegment / 32 + 1] = (lane * kEach + j) * 32 + __ffs(w) - 1;
            break;
          }
        }
      }
      __syncthreads();
      mine = s_count[kSegment / 32 + 1] >= 0;
      expert = mine ? s_count[kSegment / 32 + 1] : 0;
      __syncthreads();
    }
    // Rows of x that picked this expert, in ascending order (every CTA of the
    // cluster finds the same list), a segment of the ids at a time.
    int passes = 0;
    for (int64_t seg = 0; mine && seg < a.batch; seg += kSegment) {
      constexpr int kPer = kSegment / 32 / 8;  // groups of 32 ids per warp
      uint32_t hit[kPer];
      if (warp < 8) {
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
          const int64_t i = seg + (j * 8 + warp) * 32 + lane;
          const bool is =
              i < a.batch && __ldg(a.ids + i) == (int32_t)expert;
          hit[j] = __ballot_sync(0xFFFFFFFFu, is);
          if (lane == 0) s_count[j * 8 + warp] = __popc(hit[j]);
        }
      }
      __syncthreads();
      if (warp == 0) {  // exclusive prefix sums, one count per lane
        static_assert(kSegment == 1024, "one count per lane");
        const int c = s_count[lane];
        int before = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int v = __shfl_up_sync(0xFFFFFFFFu, before, o);
          if (lane >= o) before += v;
        }
        if (lane == 31) s_count[32] = before;
        s_count[lane] = before - c;
      }
      __syncthreads();
      if (warp < 8) {
#pragma unroll
        for (int j = 0; j < kPer; ++j)
          if (hit[j] >> lane & 1u)
            s_rows[s_count[j * 8 + warp] +
                   __popc(hit[j] & ((1u << lane) - 1u))] =
                (int)(seg + (j * 8 + warp) * 32 + lane);
      }
      __syncthreads();
      const int total = s_count[32];
      for (int first = 0; first < total; first += P::kRows)
        pass(passes++, first, 0,
             total - first < P::kRows ? total - first : P::kRows);
      __syncthreads();  // the list has been read
    }
  }

  tc_fence_before_sync();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, kColumns);
  }
}

// Clusters of ks CTAs that are resident together, asked once per kernel, ks
// and device.
template <int FMT, int NT, int SRC>
int resident(int ks, int dev) {
  static std::atomic<int> known[16][9];  // 0: not asked yet
  using P = DecodePlan<FMT, NT, SRC>;
  if (dev < 16) {
    const int v = known[dev][ks].load(std::memory_order_relaxed);
    if (v != 0) return v;
  }
  const int n = max_clusters(reinterpret_cast<const void *>(decode_f4_kernel<FMT, NT, SRC>),
                             ks, kThreads, P::kSmem);
  if (dev < 16 && n > 0) known[dev][ks].store(n, std::memory_order_relaxed);
  return n;
}

// `copies`: how many products of n rows run at once (passes, experts).
template <int FMT, int NT, int SRC>
cudaError_t launch(const WeightsView &w, const WeightsView *x, DecodeArgs a,
                   int64_t copies, int64_t grid_y, cudaStream_t stream) {
  using P = DecodePlan<FMT, NT, SRC>;
  auto kern = decode_f4_kernel<FMT, NT, SRC>;
  cudaError_t e =
      ensure_smem_limit<decode_f4_kernel<FMT, NT, SRC>>((int)P::kSmem);
  if (e != cudaSuccess) return e;
  int dev = 0;
  if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
  CUtensorMap mw, mx;
  WeightsView every = w;
  every.n *= a.ids != nullptr ? a.n_experts : 1;
  if ((e = code_map(&mw, every, kTile)) != cudaSuccess) return e;
  if (SRC == kPacked) {
    if ((e = code_map(&mx, *x, NT)) != cudaSuccess) return e;
  } else {
    mx = mw;
  }
  // The widest split of K whose clusters are all resident at once, with two
  // stages at least per CTA: a second wave costs a whole start-up.
  const int64_t tiles = (a.n + kTile - 1) / kTile;
  const int stages = (a.k + kStageK - 1) / kStageK;
  a.ks = 1;
  for (int ks = 8; ks > 1; --ks)
    if (2 * ks <= stages &&
        tiles * copies <= resident<FMT, NT, SRC>(ks, dev)) {
      a.ks = ks;
      break;
    }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(tiles * a.ks), (unsigned)grid_y);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = P::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = a.ks;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = a.ks > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, mw, mx, a);
}

template <int NT, int SRC>
cudaError_t launch_format(const WeightsView &w, const WeightsView *x,
                          const DecodeArgs &a, int64_t copies, int64_t grid_y,
                          cudaStream_t stream) {
  return w.format == TQ_FMT_MX4
             ? launch<TQ_FMT_MX4, NT, SRC>(w, x, a, copies, grid_y, stream)
             : launch<TQ_FMT_NV4, NT, SRC>(w, x, a, copies, grid_y, stream);
}

DecodeArgs weight_args(const WeightsView &w) {
  DecodeArgs a = {};
  a.codes = w.codes;
  a.wscales = reinterpret_cast<const uint8_t *>(w.scales);
  a.wg = w.lut;
  a.n = w.n;
  a.k = (int)w.k;
  return a;
}

}  // namespace

bool decode_f4_supported(const WeightsView &w, int64_t copies) {
  return w.n * copies <= INT32_MAX / 2;  // rows of the tensor map
}

cudaError_t decode_f4_bf16(const WeightsView &w, const __nv_bfloat16 *x,
                           int64_t batch, int64_t ldx, float *y, int64_t ldy,
                           cudaStream_t stream) {
  DecodeArgs a = weight_args(w);
  a.x = x;
  a.ldx = ldx;
  a.y = y;
  a.ldy = ldy;
  a.batch = batch;
  const int64_t passes = (batch + 3) / 4;
  return launch_format<32, kBf16>(w, nullptr, a, passes, passes, stream);
}

cudaError_t decode_f4_experts(const WeightsView &w, int n_experts,
                              const int32_t *ids, int64_t tokens,
                              const __nv_bfloat16 *x, int64_t ldx, float *y,
                              int64_t ldy, int32_t *status,
                              cudaStream_t stream) {
  DecodeArgs a = weight_args(w);
  a.x = x;
  a.ldx = ldx;
  a.y = y;
  a.ldy = ldy;
  a.batch = tokens;
  a.ids = ids;
  a.n_experts = n_experts;
  a.status = status;
  const int64_t used = tokens < n_experts ? tokens : n_experts;
  a.slots = n_experts <= kMapExperts ? (int)used : n_experts;
  return launch_format<32, kBf16>(w, nullptr, a, used, a.slots, stream);
}

cudaError_t decode_f4_packed(const WeightsView &w, const WeightsView &x,
                             void *y, int64_t ldy, int y_type,
                             const DigitArgs &digits, cudaStream_t stream) {
  DecodeArgs a = weight_args(w);
  a.digits = digits;
  a.xscales = reinterpret_cast<const uint8_t *>(x.scales);
  a.xg = x.lut;
  a.y = y;
  a.ldy = ldy;
  a.y_bf16 = y_type == TQ_Y_BF16;
  a.batch = x.n;
  return x.n <= 32 ? launch_format<32, kPacked>(w, &x, a, 1, 1, stream)
                   : launch_format<64, kPacked>(w, &x, a, 1, 1, stream);
}

}  // namespace tq
