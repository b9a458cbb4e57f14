// Products of few rows of x with 4-bit weights:
//
//   y[b][n] = g sum_k c[n][k] s[n][k / B] x[b][k]
//
// for bf16 x (tq_linear) and for rows of x that pick their matrix
// (tq_linear_experts_f4).
// Meant to be bound by the codes' way from HBM (0.53 bytes per weight), which
// leaves about 3 lane instructions for a weight. The profiler counts 3.0 (NV4,
// 5376 x 21504, 4 rows) and 3.4 (128 experts of 768 x 2048, 500 rows), start
// and end among them, so issue slots and start-up bind first: 22.1 us, 2.9
// TB/s, and 45 us; 1003 x 4128, 13 rows: 8.0 us.
//
// Arithmetic. Codes become fp16 pairs by one conversion instruction each, are
// multiplied by their block's scale in fp16 (exact, see below) and go as the
// A operand into fp16 mma with fp32 sums; x is the B operand:
//   NV4  c s has at most 6 significant bits between 2^-10 and 2688: exact.
//   MX4  the scale is 2^(E - R + 5), exact for R - 19 <= E <= R + 8, with R an
//        exponent that this part of the row has met. A block above that moves
//        R to its own exponent, and the sums are scaled down; a stage with a
//        block below it multiplies its codes block by block, as they are, and
//        applies 2^(E - R + 5), at least 2^-126, to the fp32 sums. Blocks of
//        zero codes may carry any scale and do neither; R starts as a guess,
//        the largest scale of the first stage, and falls too while the sums
//        are 0.
//   x    bf16 has 8 significant bits, fp16 11 but a short range: x is held
//        as x 2^(14 - X) with X the exponent of the largest value of its row
//        so far, exact down to 2^(X - 31), off by at most 2^(X - 39) below.
//        When X rises the sums are scaled down.
// fp16 mma instead of bf16: the conversion instruction of sm_100a gives fp16;
// the way to bf16 pairs takes three more instructions per pair.
//
// Work. A CTA owns 128 weight rows, 16 per warp, and a slice of K; the CTAs of
// a cluster split K and add their partial tiles in rank order through
// distributed shared memory (deterministic). Every warp keeps its own ring of
// cp.async stages of 16 rows x 256 codes, so nothing but the rows of x is
// shared, and those are staged as fp16 by all warps, double-buffered, one
// block barrier per buffer.
//
// The k order inside an mma is free as long as A and B agree: lane (g, t)
// takes 16 consecutive bytes (32 codes) of rows g and g + 8, and its part of
// an x row is the same 32 k, 8 per 16-byte load.
#include <cooperative_groups.h>

#include "tq_f4_rows.cuh"

namespace tq {
namespace {

constexpr int kStageK = 256;    // codes of a row per stage
constexpr int kSegment = 1024;  // ids looked through at once
constexpr int kList = 2 * kSegment;  // rows of an expert gathered for its passes
constexpr int kPrefetch = 1024; // bytes of a row hinted to the L2 cache
// CTAs that run at once, two on each of a B200's SMs. A constant, since
// tq_linear_workspace, which follows the same rules, asks no GPU.
constexpr int kPlaces = 2 * 148;
constexpr int kTopR = 246;  // R at most: NaN (255) lies outside of its range

struct RowArgs {
  const uint8_t *codes, *scales;  // weights (of expert 0)
  const float *g;                 // tensor scale(s) or null
  int64_t n, k;
  const __nv_bfloat16 *x;
  int64_t ldx, batch;
  float *y;
  int64_t ldy;
  const int32_t *ids;  // null: one matrix, rows of x in order
  int n_experts;
  int32_t *status;
  int ks;  // CTAs of a cluster
};

template <int FMT, int NT>
struct RowPlan {
  static constexpr int kWarps = 8, kThreads = 32 * kWarps;
  static constexpr int kTile = 16 * kWarps;  // weight rows of a CTA
  static constexpr int kCtas = 2;  // per SM
  static constexpr int kRing = 3;  // stages of a warp's ring
  // buffers of x: with 64 rows there is room for one only
  static constexpr int kXBufs = NT == 64 ? 1 : 2;
  static constexpr int kScaleRow = FMT == TQ_FMT_MX4 ? 8 : 16;  // per stage
  static constexpr int kScalePitch = FMT == TQ_FMT_MX4 ? 16 : 32;
  static constexpr int kCodes = 16 * kStageK / 2;
  static constexpr int kStage = kCodes + 16 * kScalePitch;
  static constexpr int kXK = NT == 8 ? 512 : 256;
  static constexpr int kXStages = kXK / kStageK;
  static constexpr int kXPitch = kXK * 2 + 64;
  static constexpr int kXBuf = NT * kXPitch;
  static constexpr int kUnits = kXK / 8;  // 8-value units of a buffered x row
  static constexpr int kPer = NT * kUnits / kThreads;  // units per thread
  static_assert(kUnits % 32 == 0, "a warp's units share a row");
  static constexpr int kPartPitch = kTile + 4;
  static constexpr int kRingBytes = kWarps * kRing * kStage;
  static constexpr int kPart = NT * kPartPitch * 4;
  static constexpr int kBody = kRingBytes > kPart ? kRingBytes : kPart;
  static constexpr int kSmem = kBody + kXBufs * kXBuf;
};

__device__ __forceinline__ uint32_t scaled_h2(uint32_t w, float s) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;"
      : "=r"(r)
      : "f"(__uint_as_float(w & 0xFFFF0000u) * s),
        "f"(__uint_as_float(w << 16) * s));
  return r;
}

// WHOLE: k is a multiple of 256, so that every row's scale bytes start aligned
// and no stage is cut short.
template <int FMT, int NT, bool WHOLE>
__global__ void __launch_bounds__(RowPlan<FMT, NT>::kThreads,
                                  RowPlan<FMT, NT>::kCtas)
    rows_f4_kernel(const RowArgs a) {
  using P = RowPlan<FMT, NT>;
  constexpr int kWarps = P::kWarps, kThreads = P::kThreads, kTile = P::kTile;
  constexpr int kTiles = NT / 8;  // mma columns
  constexpr int kRing = P::kRing;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int s_rows[kList];
  __shared__ int s_count[kSegment / 32 + 1];
  __shared__ float s_fac[2][NT];
  __shared__ uint32_t s_max[2][NT * P::kUnits / 32];
  __shared__ int s_exp[NT];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  const int ks = a.ks, rank = ks > 1 ? (int)cluster_rank() : 0;
  const int64_t row0 = (int64_t)(blockIdx.x / ks) * kTile;
  const int64_t expert = a.ids != nullptr ? blockIdx.y : 0;
  const uint32_t ring = smem_u32(smem) + warp * kRing * P::kStage;
  const uint32_t xbuf = smem_u32(smem) + P::kBody;

  // slice of K, in stages
  const int stages = (int)((a.k + kStageK - 1) / kStageK);
  const int st0 = (int)((int64_t)stages * rank / ks);
  const int st1 = (int)((int64_t)stages * (rank + 1) / ks);
  const int count = st1 - st0;

  // this warp's 16 weight rows; rows past the matrix repeat the last one
  const int64_t code_pitch = a.k / 2;
  const int64_t blocks = a.k / f4_block(FMT);
  const int64_t first = row0 + 16 * warp < a.n ? row0 + 16 * warp : a.n - 1;
  const int last = (int)(a.n - 1 - first < 15 ? a.n - 1 - first : 15);
  const uint8_t *codes =
      a.codes + (expert * a.n + first) * code_pitch + (lane & 7) * 16;
  const uint8_t *scales = a.scales + (expert * a.n + first) * blocks;
  uint32_t off[4];  // of the four rows this lane copies (k < 2^27)
#pragma unroll
  for (int i = 0; i < 4; ++i)
    off[i] = (uint32_t)(min((lane >> 3) + 4 * i, last) * code_pitch);
  // chunks t and t + 4 of row g in a stage (the odd rows' halves are swapped)
  const uint32_t my_chunk =
      g * (kStageK / 2) + ((t ^ ((g & 1) << 2)) << 4);
  const uint32_t ring_at =
      ring + (lane >> 3) * (kStageK / 2) +
      (((lane & 7) ^ (((lane >> 3) & 1) << 2)) << 4);

  pdl_launch_dependents();
  // Hint the L2 cache with this warp's codes, so that they are on their way
  // while the kernel before finishes: lane r takes row r of the slice. Not for
  // experts, most of whose CTAs start long after that kernel's end: 500 rows
  // over 128 experts of 768 x 2048 (NV4) 50 us with it, 46 us without.
  if (a.ids == nullptr && lane <= last && count > 0) {
    const int64_t from = (int64_t)st0 * (kStageK / 2);
    const int64_t to = (int64_t)st1 * (kStageK / 2);
    const int64_t bytes = (to < code_pitch ? to : code_pitch) - from;
    prefetch_l2_bulk(a.codes + (expert * a.n + first + lane) * code_pitch + from,
                     (uint32_t)(bytes < kPrefetch ? bytes : kPrefetch));
  }
  pdl_wait();

  // WHOLE: lanes 0 .. 15 copy a row's scale bytes each
  const uint8_t *my_scales =
      scales + min(lane, last) * blocks + (int64_t)st0 * P::kScaleRow;
  codes += (int64_t)st0 * (kStageK / 2);
  auto issue = [&](int st, int slot) {  // stage st of the slice into the ring
    if (st < count) {
      const uint8_t *src = codes + st * (kStageK / 2);
      const uint32_t dst = ring_at + slot * P::kStage;
      const bool live =
          WHOLE || (int64_t)(st0 + st) * (kStageK / 2) + (lane & 7) * 16 <
                       code_pitch;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        cp_async<16>(dst + 4 * i * (kStageK / 2), live ? src + off[i] : a.codes,
                     live);
      const uint32_t sdst = ring + slot * P::kStage + P::kCodes;
      if constexpr (WHOLE) {
        if (lane < 16)
          cp_async<P::kScaleRow>(sdst + lane * P::kScalePitch,
                                 my_scales + st * P::kScaleRow, true);
      } else {
        // the aligned words around a row's bytes; a word that holds none of
        // them is not read
        const int64_t sat = (int64_t)(st0 + st) * P::kScaleRow;
        constexpr int kW = P::kScaleRow / 4 + 1;
#pragma unroll
        for (int j = 0; j < (16 * kW + 31) / 32; ++j) {
          const int e = lane + 32 * j, r = e / kW, w = e % kW;
          if (e < 16 * kW) {
            const uint8_t *p = scales + min(r, last) * blocks;
            const uint8_t *q = p + sat;
            q -= reinterpret_cast<uintptr_t>(q) & 3u;
            q += 4 * w;
            const bool in = q < p + blocks;
            cp_async<4>(sdst + r * P::kScalePitch + 4 * w, in ? q : a.scales,
                        in);
          }
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };

  auto start = [&] {
#pragma unroll 1
    for (int p = 0; p < kRing - 1; ++p) issue(p, p);
  };

  const float gw = a.g != nullptr ? a.g[expert] : 1.0f;
  // `rows` <= NT rows of x, s_rows[base + i] each (or b0 + i): one pass;
  // `started`: its first stages are on their way
  auto pass = [&](int base, int64_t b0, int rows, bool started) {
    float acc[kTiles][4];
#pragma unroll
    for (int i = 0; i < kTiles; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = 0.0f;
    uint32_t R = 0;  // MX4: R of row g in the low half, of row g + 8 above
    // X of the rows of this thread's units
    int ex[P::kPer];
#pragma unroll
    for (int j = 0; j < P::kPer; ++j) ex[j] = -112;

    if (!started) start();
    // Rows of x, kXK values of each per buffer. Thread tid holds units
    // tid + kThreads j, a warp's 32 units of one j lie in one row.
    const int64_t k_end =
        (int64_t)st1 * kStageK < a.k ? (int64_t)st1 * kStageK : a.k;
    const int buffers = (count + P::kXStages - 1) / P::kXStages;
    constexpr int kHeld = P::kPer < 4 ? P::kPer : 4;  // units in registers
    uint4 xr[kHeld];
    auto load_x = [&](int i, int j0, uint4 (&xr)[kHeld]) {
      if (i >= buffers) return;
      const int64_t k0 = (int64_t)st0 * kStageK + (int64_t)i * P::kXK;
#pragma unroll
      for (int j = 0; j < kHeld; ++j) {
        const int q = tid + kThreads * (j0 + j), r = q / P::kUnits;
        const int64_t k = k0 + 8 * (q % P::kUnits);
        const bool live = r < rows && k < k_end;
        const int64_t row =
            !live ? 0 : a.ids != nullptr ? s_rows[base + r] : b0 + r;
        xr[j] = make_uint4(0, 0, 0, 0);
        if (live)
          xr[j] = __ldg(reinterpret_cast<const uint4 *>(a.x + row * a.ldx + k));
      }
    };
    // The largest magnitude (bf16 bits) of a warp's units.
    constexpr bool kShared = P::kUnits > 32;  // a row's units lie in two warps
    auto warp_max = [&](int j) {
      uint32_t m = __reduce_max_sync(0xFFFFFFFFu, max_mag8(xr[j]));
      if (m >= 0x7F80u)  // NaN or Inf: take the largest finite value
        m = __reduce_max_sync(0xFFFFFFFFu, max_finite8(xr[j]));
      return m;
    };
    auto publish = [&](int i) {
      if constexpr (kShared) {
        if (i >= buffers) return;
#pragma unroll
        for (int j = 0; j < kHeld; ++j) {
          if ((warp * 32 + kThreads * j) / P::kUnits >= rows) break;
          const uint32_t m = warp_max(j);
          if (lane == 0) s_max[i & 1][warp + kWarps * j] = m;
        }
      }
    };
    // registers -> fp16 in buffer i; whether a row's exponent rose
    auto convert = [&](int i, int j0) {
      bool rose = false;
      if (i >= buffers) return rose;
#pragma unroll
      for (int j = 0; j < kHeld; ++j) {
        const int q = tid + kThreads * (j0 + j), r = q / P::kUnits;
        if ((warp * 32 + kThreads * (j0 + j)) / P::kUnits >= rows) break;
        const int unit = q % P::kUnits;
        int &x_exp = ex[j0 + j];
        uint32_t m = 0;
        if constexpr (kShared) {
#pragma unroll
          for (int u = 0; u < P::kUnits / 32; ++u)
            m = max(m, s_max[i & 1][r * (P::kUnits / 32) + u]);
        } else {
          m = warp_max(j);
        }
        const int now = max(x_exp, (int)(m >> 7) - 127);
        if (unit == 0) s_fac[i & 1][r] = pow2_down(x_exp - now);
        rose |= now != x_exp;
        x_exp = now;
        // 2^(14 - X), X >= -112
        const float f = __uint_as_float((uint32_t)(141 - x_exp) << 23);
        const uint4 h =
            make_uint4(scaled_h2(xr[j].x, f), scaled_h2(xr[j].y, f),
                       scaled_h2(xr[j].z, f), scaled_h2(xr[j].w, f));
        // unit 4 t + s of a group of 128 k lies at position 4 s + t, so that
        // the four lanes of a quad read 64 consecutive bytes
        const int pos = (unit & ~15) | ((unit & 3) << 2) | ((unit >> 2) & 3);
        sts128(xbuf + (P::kXBufs == 2 ? i & 1 : 0) * P::kXBuf +
                   r * P::kXPitch + pos * 16,
               h);
      }
      return rose;
    };

    uint4 then[kHeld];  // the second buffer's, on their way with the first's
    if (P::kXBufs == 2) {
      load_x(0, 0, xr);
      load_x(1, 0, then);
    }
    for (int i = tid; i < P::kXBufs * (NT - rows) * (P::kXPitch / 16);
         i += kThreads) {
      const int b = i / ((NT - rows) * (P::kXPitch / 16));
      sts128(xbuf + b * P::kXBuf + rows * P::kXPitch +
                 (i - b * (NT - rows) * (P::kXPitch / 16)) * 16,
             make_uint4(0, 0, 0, 0));  // rows that are not there
    }
    if (tid >= rows && tid < NT) s_fac[0][tid] = s_fac[1][tid] = 1.0f;
    int any = 0;
    if constexpr (P::kXBufs == 2) {
      publish(0);
      if (kShared) __syncthreads();
      any = convert(0, 0);
#pragma unroll
      for (int j = 0; j < kHeld; ++j) xr[j] = then[j];
      publish(1);
      any = __syncthreads_or(any);
    }
    int st = 0, slot = 0;
#pragma unroll 1
    for (int i = 0; i < buffers; ++i) {
      int rose = 0;
      if constexpr (P::kXBufs == 2) {
        rose = convert(i + 1, 0);
        load_x(i + 2, 0, xr);
      } else {
        // one buffer: filled between two barriers, while the other CTA of the
        // SM computes
        if (i > 0) __syncthreads();
#pragma unroll
        for (int j = 0; j < P::kPer; j += kHeld) {
          load_x(i, j, xr);
          rose |= convert(i, j);
        }
        any = __syncthreads_or(rose);
      }
      if (any) {
#pragma unroll
        for (int c = 0; c < kTiles; ++c) {
          const float f0 = s_fac[i & 1][8 * c + 2 * t];
          const float f1 = s_fac[i & 1][8 * c + 2 * t + 1];
          acc[c][0] *= f0;
          acc[c][1] *= f1;
          acc[c][2] *= f0;
          acc[c][3] *= f1;
        }
      }
      const int end = st + P::kXStages < count ? st + P::kXStages : count;
      uint32_t xat = xbuf + (P::kXBufs == 2 ? i & 1 : 0) * P::kXBuf +
                     g * P::kXPitch + t * 16;
#pragma unroll 1
      for (; st < end; ++st, xat += 2 * kStageK) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 2) : "memory");
        __syncwarp();
        issue(st + kRing - 1, slot == 0 ? kRing - 1 : slot - 1);
        const uint32_t src = ring + slot * P::kStage;
        slot = slot == kRing - 1 ? 0 : slot + 1;
        // fp16 factors of chunks t and t + 4 of rows g and g + 8
        uint32_t f[2][2][2];  // [half][row][block of the chunk]
        const uint32_t s0 = src + P::kCodes + g * P::kScalePitch;
        // rows that do not start on a word boundary lie shifted, and bytes
        // past the row's end belong to the next row
        auto odd_byte = [&](int r, int j) {
          const uint32_t shift =
              (uint32_t)(reinterpret_cast<uintptr_t>(
                             scales + min(g + 8 * r, last) * blocks) &
                         3u);
          const uint32_t b = lds_u8(s0 + 8 * r * P::kScalePitch + shift + j);
          return (int64_t)(st0 + st) * P::kScaleRow + j < blocks ? b : 0u;
        };
        if constexpr (FMT == TQ_FMT_MX4) {
          uint32_t e[2];  // [row]: chunk t in the low half, t + 4 above
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            if constexpr (WHOLE) {
              uint32_t lo, hi;
              asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];"
                           : "=r"(lo), "=r"(hi)
                           : "r"(s0 + 8 * r * P::kScalePitch)
                           : "memory");
              e[r] = __byte_perm(lo, hi, t | (t + 4) << 8) & 0x00FF00FFu;
            } else {
              e[r] = odd_byte(r, t) | odd_byte(r, t + 4) << 16;
            }
          }
          if (st == 0) {  // a guess: the largest exponent in the stage
            R = __vmaxu2(__byte_perm(e[0], e[1], 0x5410),
                         __byte_perm(e[0], e[1], 0x7632));
            R = __vmaxu2(R, __shfl_xor_sync(0xFFFFFFFFu, R, 1));
            R = __vmaxu2(R, __shfl_xor_sync(0xFFFFFFFFu, R, 2));
            R = __vminu2(R, kTopR * 0x00010001u);
          }
          // blocks outside of what fp16 holds beside R
          bool odd = false;
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const uint32_t top = __byte_perm(R, 0, r == 0 ? 0x1010 : 0x3232);
            odd |= __vmaxu2(e[r], top + 0x00080008u) != top + 0x00080008u ||
                   __vminu2(e[r] + 0x00130013u, top) != top;
          }
          if (__any_sync(0xFFFFFFFFu, odd)) {
            bool small = false;
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              // exponents of the blocks with any weight, else -1; NaN apart
              const int was = (int)(R >> (16 * r) & 0xFFFFu);
              int E[2], now = -1;
              bool nan = false;
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const uint4 c = lds128(src + 8 * r * (kStageK / 2) +
                                       (h == 0 ? my_chunk : my_chunk ^ 64u));
                const int b = (int)(e[r] >> (16 * h) & 0xFFu);
                nan |= b == 255;
                E[h] = b != 255 && ((c.x | c.y | c.z | c.w) & 0x77777777u) != 0
                           ? b
                           : -1;
                now = max(now, E[h]);
              }
              now = max(now, __shfl_xor_sync(0xFFFFFFFFu, now, 1));
              now = max(now, __shfl_xor_sync(0xFFFFFFFFu, now, 2));
              // with no sums yet (NaN and Inf have no scale) R may fall as well
              bool some = false;
#pragma unroll
              for (int c = 0; c < 2 * kTiles; ++c) {
                const uint32_t u =
                    __float_as_uint(acc[c / 2][2 * r + c % 2]) << 1;
                some |= u - 1u < 0xFEFFFFFFu;
              }
              const uint32_t sums = __ballot_sync(0xFFFFFFFFu, some);
              some = (sums >> (lane & 28) & 15u) != 0;
              now = now < 0 || (some && now <= was + 8) ? was : min(now, kTopR);
              const uint32_t nans = __ballot_sync(0xFFFFFFFFu, nan);
              // a NaN scale makes the row NaN, whatever the codes
              const bool gone = (nans >> (lane & 28) & 15u) != 0;
              const float f = pow2_down(min(was - now, 0));
#pragma unroll
              for (int c = 0; c < kTiles; ++c) {
                acc[c][2 * r] =
                    gone ? __int_as_float(0x7FC00000) : acc[c][2 * r] * f;
                acc[c][2 * r + 1] =
                    gone ? __int_as_float(0x7FC00000) : acc[c][2 * r + 1] * f;
              }
              R += (uint32_t)(now - was) << (16 * r);
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                if (E[h] < 0) E[h] = now;  // weighs nothing
                small |= E[h] + 19 < now;
              }
              e[r] = (uint32_t)E[0] | (uint32_t)E[1] << 16;
            }
            if (__any_sync(0xFFFFFFFFu, small)) {
              // Word i % 4 of block i / 4: the lanes that hold another block
              // feed zeros on both sides (0 times Inf would be NaN).
#pragma unroll 1
              for (int i = 0; i < 32; ++i) {
                const uint32_t here = t == (i >> 2 & 3) ? 0xFFFFFFFFu : 0u;
                const uint32_t at =
                    src + (my_chunk ^ (i >> 4 << 6)) + 4 * (i & 3);
                const uint32_t xs = xat + 256 * (i >> 4) + 64 * (i & 3);
                uint32_t p[4], q[4];
                f4x8_to_h2(lds32(at) & here, p);
                f4x8_to_h2(lds32(at + 8 * (kStageK / 2)) & here, q);
                float f[2];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                  const uint32_t both =
                      __shfl_sync(0xFFFFFFFFu, e[r], i >> 2 & 3, 4);
                  const int E = (int)(both >> (16 * (i >> 4)) & 0xFFu);
                  const int field = E - (int)(R >> (16 * r) & 0xFFFFu) + 132;
                  f[r] = __int_as_float(max(field, 1) << 23);
                }
#pragma unroll
                for (int c = 0; c < kTiles; ++c) {
                  const uint4 v = lds128(xs + 8 * c * P::kXPitch);
                  float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                  mma_f16(d, p[0], q[0], p[1], q[1], v.x & here, v.y & here);
                  mma_f16(d, p[2], q[2], p[3], q[3], v.z & here, v.w & here);
#pragma unroll
                  for (int k = 0; k < 4; ++k)
                    acc[c][k] = fmaf(d[k], f[k >> 1], acc[c][k]);
                }
              }
              continue;
            }
          }
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            // exponent fields E - R + 20 of both chunks, 1 to 28
            const uint32_t v = e[r] + 0x00140014u -
                               __byte_perm(R, 0, r == 0 ? 0x1010 : 0x3232);
            f[0][r][0] = f[0][r][1] = __byte_perm(v, 0, 0x1010) << 10;
            f[1][r][0] = f[1][r][1] = __byte_perm(v, 0, 0x3232) << 10;
          }
        } else {
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              uint32_t b, v;
              if constexpr (WHOLE)
                asm volatile("ld.shared.u16 %0, [%1];"
                             : "=r"(b)
                             : "r"(s0 + 8 * r * P::kScalePitch + 2 * t + 8 * h)
                             : "memory");
              else
                b = odd_byte(r, 2 * t + 8 * h) |
                    odd_byte(r, 2 * t + 8 * h + 1) << 8;
              asm("cvt.rn.f16x2.e4m3x2 %0, %1;"
                  : "=r"(v)
                  : "h"((uint16_t)(b & 0x7F7Fu)));
              f[h][r][0] = __byte_perm(v, 0, 0x1010);
              f[h][r][1] = __byte_perm(v, 0, 0x3232);
            }
        }
        // The tensor core cuts its sums instead of rounding them, so a stage
        // has sums of its own, which are added to the others with rounding.
        // NV4, 5376 x 21504: 1.2e-7 off instead of 1.2e-6, in the same time up
        // to 16 rows, in 44.6 instead of 43.3 us at 24. 64 rows have not the
        // registers: there the sums are those of half a stage and four column
        // tiles at a time, with the half's weights decoded before (83 instead
        // of 76 us; with a stage's sums of all tiles spilled 85, with one tile
        // at a time 82 and, 128 experts of 768 x 2048 at 4096 rows, 154 instead
        // of 147).
        constexpr bool kStageSums = NT <= 32;
        constexpr int kWords = kStageSums ? 1 : 4;  // decoded at once
        constexpr int kAtOnce = kStageSums ? kTiles : 4;  // column tiles
        float own[kAtOnce][4];
        if constexpr (kStageSums) {
#pragma unroll
          for (int c = 0; c < kAtOnce; ++c)
#pragma unroll
            for (int j = 0; j < 4; ++j) own[c][j] = 0.0f;
        }
        // not unrolled: the two halves together overran the instruction cache
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
          const uint32_t at = src + (h == 0 ? my_chunk : my_chunk ^ 64u);
          const uint4 c0 = lds128(at);
          const uint4 c1 = lds128(at + 8 * (kStageK / 2));
          const uint32_t w0[4] = {c0.x, c0.y, c0.z, c0.w};
          const uint32_t w1[4] = {c1.x, c1.y, c1.z, c1.w};
#pragma unroll
          for (int s0 = 0; s0 < 4; s0 += kWords) {
            uint32_t p[kWords][4], q[kWords][4];
#pragma unroll
            for (int s = 0; s < kWords; ++s) {
              f4x8_to_h2(w0[s0 + s], p[s]);
              f4x8_to_h2(w1[s0 + s], q[s]);
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                p[s][c] = hmul2(p[s][c], f[0][0][(s0 + s) >> 1]);
                q[s][c] = hmul2(q[s][c], f[0][1][(s0 + s) >> 1]);
              }
            }
#pragma unroll
            for (int tile = 0; tile < kTiles; tile += kAtOnce) {
              if constexpr (!kStageSums) {
#pragma unroll
                for (int c = 0; c < kAtOnce; ++c)
                  own[c][0] = own[c][1] = own[c][2] = own[c][3] = 0.0f;
              }
#pragma unroll
              for (int s = 0; s < kWords; ++s)
#pragma unroll
                for (int c = 0; c < kAtOnce; ++c) {
                  const uint4 v =
                      lds128(xat + 256 * h + 8 * (tile + c) * P::kXPitch +
                             64 * (s0 + s));
                  mma_f16(own[c], p[s][0], q[s][0], p[s][1], q[s][1], v.x, v.y);
                  mma_f16(own[c], p[s][2], q[s][2], p[s][3], q[s][3], v.z, v.w);
                }
              if constexpr (!kStageSums) {
#pragma unroll
                for (int c = 0; c < kAtOnce; ++c)
#pragma unroll
                  for (int j = 0; j < 4; ++j) acc[tile + c][j] += own[c][j];
              }
            }
          }
#pragma unroll
          for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int c = 0; c < 2; ++c) f[0][r][c] = f[1][r][c];
        }
        if constexpr (kStageSums) {
#pragma unroll
          for (int c = 0; c < kTiles; ++c)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[c][j] += own[c][j];
        }
      }
      if constexpr (P::kXBufs == 2) {
        publish(i + 2);
        any = __syncthreads_or(rose);
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
#pragma unroll
    for (int j = 0; j < P::kPer; ++j) {
      const int q = tid + kThreads * j;
      if (q % P::kUnits == 0) s_exp[q / P::kUnits] = ex[j];
    }
    __syncthreads();  // rings are free, exponents are there

    // partial sums in units of y, [row of x][weight row]
    float *part = reinterpret_cast<float *>(smem);
    const TensorScale ts = FMT == TQ_FMT_NV4 ? tensor_scale(gw)
                                             : TensorScale{1.0f, 0};
#pragma unroll
    for (int i = 0; i < kTiles; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int b = 8 * i + 2 * t + (j & 1);
        int e = s_exp[b] - 14 + ts.e;
        if (FMT == TQ_FMT_MX4) e += (int)(j < 2 ? R & 0xFFFFu : R >> 16) - 132;
        part[b * P::kPartPitch + 16 * warp + g + (j < 2 ? 0 : 8)] =
            times_pow2(acc[i][j] * ts.m, e);
      }
    if (ks > 1)
      cooperative_groups::this_cluster().sync();
    else
      __syncthreads();
    const uint32_t mine = smem_u32(part);
    for (int i = tid + rank * kThreads; i < rows * kTile; i += ks * kThreads) {
      const int b = i / kTile, r = i % kTile;
      if (row0 + r >= a.n) continue;  // every read is stored, see below
      const uint32_t at = mine + (b * P::kPartPitch + r) * 4;
      float v = 0.0f;
      if (ks == 1) {
        v = part[b * P::kPartPitch + r];
      } else {
        for (int c = 0; c < ks; ++c) {
          uint32_t remote;
          float u;
          asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                       : "=r"(remote)
                       : "r"(at), "r"(c));
          asm volatile("ld.shared::cluster.f32 %0, [%1];"
                       : "=f"(u)
                       : "r"(remote)
                       : "memory");
          v += u;
        }
      }
      const int64_t row = a.ids != nullptr ? s_rows[base + b] : b0 + b;
      a.y[row * a.ldy + row0 + r] = v;
    }
    // The partial tiles have been read (each value that was read has gone into
    // a store, which was issued before this barrier's arrival): shared memory
    // may change, or go.
    if (ks > 1)
      cluster_sync_relaxed();
    else
      __syncthreads();
  };

  if (a.ids == nullptr) {
    const int64_t b0 = (int64_t)blockIdx.y * NT;
    pass(0, b0, (int)(a.batch - b0 < NT ? a.batch - b0 : NT), false);
    return;
  }
  // Rows of x that picked this expert, in ascending order (every CTA of the
  // cluster finds the same list), a segment of the ids at a time; the passes
  // follow when the list is full or the ids are at their end. 128 experts of
  // 768 x 2048, 2048 and 4096 rows: 83 and 145 us, against 137 and 430 us
  // with passes after every segment.
  int held = 0;
  start();  // most experts have rows: the codes come while the ids are read
  bool started = true;
  for (int64_t seg = 0; seg < a.batch; seg += kSegment) {
    constexpr int kPer = kSegment / kThreads;
    uint32_t hit = 0;  // bit j: id j of this thread
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int64_t i = seg + (j * kWarps + warp) * 32 + lane;
      const int32_t id = i < a.batch ? __ldg(a.ids + i) : -2;
      const bool is = i < a.batch && id == (int32_t)expert;
      const uint32_t vote = __ballot_sync(0xFFFFFFFFu, is);
      if (lane == 0) s_count[j * kWarps + warp] = __popc(vote);
      if (is) hit |= 1u << j;
      if (expert == 0 && rank == 0 && blockIdx.z == 0 && i < a.batch &&
          (id < 0 || id >= a.n_experts)) {
        // nobody's row: NaN in this CTA's columns
        const int64_t end = row0 + kTile < a.n ? row0 + kTile : a.n;
        for (int64_t r = row0; r < end; ++r)
          a.y[i * a.ldy + r] = __int_as_float(0x7FC00000);
        report(a.status, TQ_ERR_INVALID_ARG);
      }
    }
    __syncthreads();
    if (warp == 0) {  // exclusive prefix sums, 4 counts per lane
      constexpr int kEach = kSegment / 32 / 32;
      static_assert(kEach * 32 * 32 == kSegment, "one count per 32 ids");
      int c[kEach], sum = 0;
#pragma unroll
      for (int j = 0; j < kEach; ++j) {
        c[j] = s_count[lane * kEach + j];
        sum += c[j];
      }
      int before = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xFFFFFFFFu, before, o);
        if (lane >= o) before += v;
      }
      if (lane == 31) s_count[kSegment / 32] = before;
      before -= sum;
#pragma unroll
      for (int j = 0; j < kEach; ++j) {
        s_count[lane * kEach + j] = before;
        before += c[j];
      }
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const bool is = hit >> j & 1u;
      const uint32_t vote = __ballot_sync(0xFFFFFFFFu, is);
      if (is)
        s_rows[held + s_count[j * kWarps + warp] +
               __popc(vote & ((1u << lane) - 1u))] =
            (int)(seg + (j * kWarps + warp) * 32 + lane);
    }
    __syncthreads();
    held += s_count[kSegment / 32];
    if (held > kList - kSegment || seg + kSegment >= a.batch) {
      // (the passes of an expert are shared by the CTAs along z)
      for (int base = NT * blockIdx.z; base < held; base += NT * gridDim.z) {
        pass(base, 0, held - base < NT ? held - base : NT, started);
        started = false;
      }
      held = 0;
    }
    __syncthreads();  // the list and the counts have been read
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// Clusters of ks CTAs that are resident together, asked once per kernel, ks
// and device.
template <int FMT, int NT, bool WHOLE>
int resident(int ks, int dev) {
  static std::atomic<int> known[16][9];  // 0: not asked yet
  using P = RowPlan<FMT, NT>;
  if (dev < 16) {
    const int v = known[dev][ks].load(std::memory_order_relaxed);
    if (v != 0) return v;
  }
  const int n = max_clusters(reinterpret_cast<const void *>(rows_f4_kernel<FMT, NT, WHOLE>),
                             ks, P::kThreads, P::kSmem);
  if (dev < 16 && n > 0) known[dev][ks].store(n, std::memory_order_relaxed);
  return n;
}

// `copies`: how many row products of n rows run at once (passes, experts).
template <int FMT, int NT, bool WHOLE>
cudaError_t launch_whole(RowArgs a, int64_t copies, dim3 grid,
                         cudaStream_t stream) {
  using P = RowPlan<FMT, NT>;
  auto kern = rows_f4_kernel<FMT, NT, WHOLE>;
  cudaError_t e =
      ensure_smem_limit<rows_f4_kernel<FMT, NT, WHOLE>>(P::kSmem);
  if (e != cudaSuccess) return e;
  int dev = 0;
  if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
  const int64_t tiles = (a.n + P::kTile - 1) / P::kTile;
  const int64_t stages = (a.k + kStageK - 1) / kStageK;
  // The widest split of K whose clusters are all resident at once, with two
  // stages at least per CTA: a second wave costs a whole pass of start-up and
  // reduction (8192 x 5376, batch 1: 17.5 us with 320 CTAs on 296 places).
  a.ks = 1;
  for (int ks = 8; ks > 1; --ks)
    if (2 * ks <= stages &&
        tiles * copies <= resident<FMT, NT, WHOLE>(ks, dev)) {
      a.ks = ks;
      break;
    }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(tiles * a.ks), grid.y, grid.z);
  cfg.blockDim = dim3(P::kThreads);
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
  return cudaLaunchKernelEx(&cfg, kern, a);
}

template <int FMT, int NT>
cudaError_t launch(const RowArgs &a, int64_t copies, dim3 grid,
                   cudaStream_t stream) {
  return a.k % kStageK == 0
             ? launch_whole<FMT, NT, true>(a, copies, grid, stream)
             : launch_whole<FMT, NT, false>(a, copies, grid, stream);
}

template <int NT>
cudaError_t launch_format(int format, const RowArgs &a, int64_t copies,
                          dim3 grid, cudaStream_t stream) {
  return format == TQ_FMT_MX4
             ? launch<TQ_FMT_MX4, NT>(a, copies, grid, stream)
             : launch<TQ_FMT_NV4, NT>(a, copies, grid, stream);
}

cudaError_t launch_nt(int format, int nt, const RowArgs &a, int64_t copies,
                      dim3 grid, cudaStream_t stream) {
  switch (nt) {
    case 8: return launch_format<8>(format, a, copies, grid, stream);
    case 16: return launch_format<16>(format, a, copies, grid, stream);
    case 32: return launch_format<32>(format, a, copies, grid, stream);
    default: return launch_format<64>(format, a, copies, grid, stream);
  }
}

RowArgs weight_args(const WeightsView &w) {
  RowArgs a = {};
  a.codes = w.codes;
  a.scales = reinterpret_cast<const uint8_t *>(w.scales);
  a.g = w.lut;
  a.n = w.n;
  a.k = w.k;
  return a;
}

}  // namespace

int rows_per_pass_f4(const WeightsView &w, int64_t copies, int64_t rows) {
  int nt = rows <= 8 ? 8 : rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
  const int64_t tiles = (w.n + 127) / 128;
  const int64_t split = (w.k + kStageK - 1) / kStageK / 2;  // of K, at most
  const int64_t each = tiles * copies * (split < 1 ? 1 : split < 8 ? split : 8);
  while (nt > 8 && each * ((rows + nt / 2 - 1) / (nt / 2)) <= kPlaces) nt /= 2;
  return nt;
}

cudaError_t linear_f4_bf16(const WeightsView &w, const __nv_bfloat16 *x,
                           int64_t batch, int64_t ldx, float *y, int64_t ldy,
                           cudaStream_t stream) {
  // Up to 3 (MX4: 4) rows the digits of x cost less than decoding the weights,
  // but for long rows of x: 21504 x 5376 (MX4) at 1, 2, 4, 8 rows 17.0, 18.8,
  // 23.7, 35.7 us there against 28.4, 28.7, 30.2, 32.3 us here; 5376 x 21504
  // (NV4) at 1, 2, 4 rows 21.4, 23.8, 28.8 against 21.9, 22.0, 23.3 us.
  if (batch <= (w.format == TQ_FMT_MX4 ? 4 : 3) && decode_f4_supported(w, 1))
    return decode_f4_bf16(w, x, batch, ldx, y, ldy, stream);
  RowArgs a = weight_args(w);
  a.x = x;
  a.ldx = ldx;
  a.batch = batch;
  a.y = y;
  a.ldy = ldy;
  const int nt = rows_per_pass_f4(w, 1, batch);
  const int64_t passes = (batch + nt - 1) / nt;
  cudaError_t e = cudaSuccess;
  // a grid's second dimension ends at 65535
  for (int64_t p = 0; p < passes && e == cudaSuccess; p += 65535) {
    const int64_t now = passes - p < 65535 ? passes - p : 65535;
    RowArgs b = a;
    b.x += p * nt * ldx;
    b.y = y + p * nt * ldy;
    b.batch -= p * nt;
    e = launch_nt(w.format, nt, b, now, dim3(1, (unsigned)now), stream);
  }
  return e;
}

cudaError_t launch_linear_experts_f4(const WeightsView &w, int n_experts,
                                     const int32_t *ids, int64_t tokens,
                                     const __nv_bfloat16 *x, int64_t ldx,
                                     float *y, int64_t ldy, int32_t *status,
                                     cudaStream_t stream) {
  // The same trade: 64 rows over 128 experts of 768 x 2048 (MX4) 18.5 us there
  // against 24.1 us here, 257 rows 37.8 against 35.8 us, 500 rows (NV4) 59
  // against 46 us.
  if (tokens <= n_experts && decode_f4_supported(w, n_experts))
    return decode_f4_experts(w, n_experts, ids, tokens, x, ldx, y, ldy, status,
                             stream);
  RowArgs a = weight_args(w);
  a.x = x;
  a.ldx = ldx;
  a.batch = tokens;
  a.y = y;
  a.ldy = ldy;
  a.ids = ids;
  a.n_experts = n_experts;
  a.status = status;
  // Experts that get rows at all, and the rows of one: room for twice the mean.
  // With room for four times the mean fewer experts need a second pass, but
  // every pass is wider: 128 experts of 768 x 2048 (MX4) at 257, 500, 1024
  // rows 43, 49.5, 74 us against 36, 46.5, 55 us, 32 experts of 1024 x 4096 at
  // 256 rows 47 against 34 us.
  const int64_t used = tokens < n_experts ? tokens : n_experts;
  const int64_t most = 2 * ((tokens + n_experts - 1) / n_experts);
  const int nt = rows_per_pass_f4(w, used, most);
  // CTAs that share an expert's passes: all of twice the mean where the passes
  // were cut for it, else what the mean needs (768 x 2048, 8 experts, 300 rows:
  // 18 us, with one for each pass of twice the mean 27 us).
  const int64_t room = kPlaces / (used * ((w.n + 127) / 128));
  int64_t z = nt < 64 && nt < most / 2 ? (most + nt - 1) / nt
                                       : (most / 2 + nt - 1) / nt;
  z = z < room ? z : room;
  z = z < 1 ? 1 : z;
  return launch_nt(w.format, nt, a, used * z,
                   dim3(1, (unsigned)n_experts, (unsigned)z), stream);
}

}  // namespace tq
