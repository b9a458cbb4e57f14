// Products of few rows of x with 4-bit weights:
//
//   y[b][n] = g sum_k c[n][k] s[n][k / B] x[b][k]
//
// for bf16 x (tq_linear), for rows of x that pick their matrix
// (tq_linear_experts_f4) and for up to 16 rows of 4-bit x (tq_linear_f4).
// Bound by the codes' way from HBM (0.53 bytes per weight), so a weight may
// cost about 3 lane instructions.
//
// Arithmetic. Codes become fp16 pairs by one conversion instruction each, are
// multiplied by their block's scale in fp16 (exact, see below) and go as the
// A operand into fp16 mma with fp32 sums; x is the B operand:
//   NV4  c s has at most 6 significant bits between 2^-10 and 2688: exact.
//   MX4  the scale is 2^(E - R + 13) with R the largest exponent that this
//        part of the row has met: c 2^(E - R + 13) is exact down to
//        2^(R - 27), smaller blocks (below 2^-27 of the row's largest) count
//        as 0. When R rises the sums are scaled down, exactly.
//   x    bf16 has 8 significant bits, fp16 11 but a short range: x is held
//        as x 2^(14 - X) with X the exponent of the largest value of its row
//        so far, exact down to 2^(X - 31), off by at most 2^(X - 39) below.
//        When X rises the sums are scaled down.
// fp16 mma instead of bf16: the conversion instruction of sm_100a gives fp16;
// the way to bf16 pairs takes three more instructions per pair.
//
// Work. A CTA owns 128 (256) weight rows, 16 per warp, and a slice of K; the CTAs
// of a cluster split K and add their partial tiles in rank order through
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
constexpr int kRing = 3;        // stages of a warp's ring
constexpr int kSegment = 2048;  // ids looked through at once

// Where the rows of x come from.
enum { kBf16 = 0, kPacked = 1 };

struct RowArgs {
  const uint8_t *codes, *scales;  // weights (of expert 0)
  const float *g;                 // tensor scale(s) or null
  int64_t n, k;
  const __nv_bfloat16 *x;  // kBf16
  int64_t ldx;
  const uint8_t *xcodes, *xscales;  // kPacked
  const float *xg;
  int64_t batch;
  void *y;
  int64_t ldy;
  int y_bf16;
  const int32_t *ids;  // null: one matrix, rows of x in order
  int n_experts;
  int32_t *status;
  int ks;  // CTAs of a cluster
};

template <int FMT, int NT>
struct RowPlan {
  // 8 warps, two CTAs per SM; 64 rows of x share one large CTA instead
  static constexpr int kWarps = NT == 64 ? 16 : 8;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kTile = 16 * kWarps;  // weight rows of a CTA
  static constexpr int kScaleRow = FMT == TQ_FMT_MX4 ? 8 : 16;  // per stage
  static constexpr int kScalePitch = FMT == TQ_FMT_MX4 ? 16 : 32;
  static constexpr int kCodes = 16 * kStageK / 2;
  static constexpr int kStage = kCodes + 16 * kScalePitch;
  static constexpr int kXK = NT == 8 ? 1024 : NT == 16 ? 512 : 256;
  static constexpr int kXStages = kXK / kStageK;
  static constexpr int kXPitch = kXK * 2 + 64;
  static constexpr int kXBuf = NT * kXPitch;
  static constexpr int kPerWarp = NT / kWarps;  // rows of x a warp stages
  static constexpr int kUnits = kXK / 256;      // 8-value units per lane
  static constexpr int kPartPitch = kTile + 4;
  static constexpr int kRingBytes = kWarps * kRing * kStage;
  static constexpr int kPart = NT * kPartPitch * 4;
  static constexpr int kBody = kRingBytes > kPart ? kRingBytes : kPart;
  static constexpr int kSmem = kBody + 2 * kXBuf;
};

// One lane's share of a buffer of x rows, in flight between global memory and
// the conversion.
template <int SRC, int COUNT>
struct XRegs;
template <int COUNT>
struct XRegs<kBf16, COUNT> {
  uint4 v[COUNT];
};
template <int COUNT>
struct XRegs<kPacked, COUNT> {
  uint32_t v[COUNT];  // 8 codes
  uint32_t s[COUNT];  // their scale byte
};

__device__ __forceinline__ uint32_t max_mag8(const uint4 &w) {
  const uint32_t m = __vmaxu2(__vmaxu2(w.x & 0x7FFF7FFFu, w.y & 0x7FFF7FFFu),
                              __vmaxu2(w.z & 0x7FFF7FFFu, w.w & 0x7FFF7FFFu));
  return max(m >> 16, m & 0xFFFFu);
}

// max_mag8 over the finite values.
__device__ __noinline__ uint32_t max_finite8(uint4 w) {
  const uint32_t v[4] = {w.x, w.y, w.z, w.w};
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t a = (v[i >> 1] >> (16 * (i & 1))) & 0x7FFFu;
    if (a < 0x7F80u) m = max(m, a);
  }
  return m;
}

__device__ __forceinline__ uint32_t scaled_h2(uint32_t w, float s) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;"
      : "=r"(r)
      : "f"(__uint_as_float(w & 0xFFFF0000u) * s),
        "f"(__uint_as_float(w << 16) * s));
  return r;
}

// fp16 pair of the MX4 factor 2^(E - R + 13): exponent field E - R + 28.
__device__ __forceinline__ uint32_t mx4_factor(int E, int R) {
  const int f = E - R + 28;
  const uint32_t h = f > 0 ? (uint32_t)f : 0u;
  return E == 255 ? 0x7E007E00u : h * 0x04000400u;
}

// fp16 pair of an E4M3 byte (its sign is not looked at).
__device__ __forceinline__ uint32_t nv4_factor(uint32_t b) {
  uint32_t h;
  b &= 0x7Fu;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)(b | b << 8)));
  return h;
}

template <int FMT, int NT, int SRC>
__global__ void __launch_bounds__(RowPlan<FMT, NT>::kThreads,
                                  NT == 64 ? 1 : 2)
    rows_f4_kernel(const RowArgs a) {
  using P = RowPlan<FMT, NT>;
  constexpr int kWarps = P::kWarps, kThreads = P::kThreads, kTile = P::kTile;
  constexpr int kTiles = NT / 8;  // mma columns
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int s_rows[kSegment];
  __shared__ int s_count[kSegment / 32 + 1];
  __shared__ float s_fac[2][NT];
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
  const bool whole = a.k % kStageK == 0;
  int64_t off[4];  // of the four rows this lane copies
#pragma unroll
  for (int i = 0; i < 4; ++i)
    off[i] = min((lane >> 3) + 4 * i, last) * code_pitch;

  pdl_launch_dependents();
  if ((lane & 7) == 0 && count > 0) {
#pragma unroll
    for (int p = 0; p < kRing - 1; ++p)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (p < count)
          asm volatile("prefetch.global.L2 [%0];" ::"l"(
              codes + off[i] + (int64_t)(st0 + p) * (kStageK / 2)));
  }
  pdl_wait();

  auto issue = [&](int st) {  // stage st of the slice into the ring
    if (st < count) {
      const uint32_t dst = ring + (st % kRing) * P::kStage;
      const int64_t at = (int64_t)(st0 + st) * (kStageK / 2);
      const bool live = at + (lane & 7) * 16 < code_pitch;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = (lane >> 3) + 4 * i;
        cp_async<16>(dst + r * (kStageK / 2) +
                         (((lane & 7) ^ ((r & 1) << 2)) << 4),
                     live ? codes + off[i] + at : codes, live);
      }
      const uint32_t sdst = dst + P::kCodes;
      const int64_t sat = (int64_t)(st0 + st) * P::kScaleRow;
      if (whole) {
        if (lane < 16)
          cp_async<P::kScaleRow>(sdst + lane * P::kScalePitch,
                                 scales + min(lane, last) * blocks + sat, true);
      } else {
        // the aligned words around a row's bytes; a word that holds none of
        // them is not read
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

  const float gw = a.g != nullptr ? a.g[expert] : 1.0f;
  // `rows` <= NT rows of x, s_rows[base + i] each (or b0 + i): one pass
  auto pass = [&](int base, int64_t b0, int rows) {
    float acc[kTiles][4];
#pragma unroll
    for (int i = 0; i < kTiles; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = 0.0f;
    int R0 = 0, R1 = 0;  // MX4: R of rows g and g + 8
    int ex[P::kPerWarp];  // X (bf16) or R (MX4 x) of the rows this warp stages
#pragma unroll
    for (int i = 0; i < P::kPerWarp; ++i) ex[i] = SRC == kBf16 ? -112 : 0;

#pragma unroll 1
    for (int p = 0; p < kRing - 1; ++p) issue(p);

    constexpr int kRegs = P::kPerWarp * P::kUnits;
    XRegs<SRC, kRegs> xr;
    auto load_x = [&](int st) {  // the buffer that starts with stage st
      const int64_t k0 = (int64_t)(st0 + st) * kStageK;
      const int64_t k_end =
          (int64_t)st1 * kStageK < a.k ? (int64_t)st1 * kStageK : a.k;
#pragma unroll
      for (int i = 0; i < P::kPerWarp; ++i) {
        const int r = warp * P::kPerWarp + i;
        const int64_t row =
            r < rows ? (a.ids != nullptr ? s_rows[base + r] : b0 + r) : 0;
#pragma unroll
        for (int u = 0; u < P::kUnits; ++u) {
          const int64_t k = k0 + 8 * (lane + 32 * u);
          const bool live = r < rows && k < k_end;
          const int j = i * P::kUnits + u;
          if constexpr (SRC == kBf16) {
            xr.v[j] = make_uint4(0, 0, 0, 0);
            if (live)
              xr.v[j] = __ldg(reinterpret_cast<const uint4 *>(a.x + row * a.ldx +
                                                              k));
          } else {
            xr.v[j] = 0;
            xr.s[j] = 0;
            if (live) {
              xr.v[j] = __ldg(reinterpret_cast<const uint32_t *>(
                  a.xcodes + row * code_pitch + k / 2));
              xr.s[j] = __ldg(a.xscales + row * blocks + k / f4_block(FMT));
            }
          }
        }
      }
    };
    // registers -> fp16 in buffer `buf`; whether a row's exponent rose
    auto stage_x = [&](int buf) {
      bool rose = false;
#pragma unroll
      for (int i = 0; i < P::kPerWarp; ++i) {
        const int r = warp * P::kPerWarp + i;
        float s = 0.0f;
        if constexpr (SRC == kBf16) {
          uint32_t m = 0;
#pragma unroll
          for (int u = 0; u < P::kUnits; ++u)
            m = max(m, max_mag8(xr.v[i * P::kUnits + u]));
          m = __reduce_max_sync(0xFFFFFFFFu, m);
          if (m >= 0x7F80u) {  // NaN or Inf: take the largest finite value
            m = 0;
#pragma unroll
            for (int u = 0; u < P::kUnits; ++u)
              m = max(m, max_finite8(xr.v[i * P::kUnits + u]));
            m = __reduce_max_sync(0xFFFFFFFFu, m);
          }
          const int e = (int)(m >> 7) - 127;
          const int now = max(ex[i], e);
          if (lane == 0) s_fac[buf][r] = pow2_down(ex[i] - now);
          rose |= now != ex[i];
          ex[i] = now;
          // 2^(14 - X), X >= -112
          s = __uint_as_float((uint32_t)(141 - now) << 23);
        } else if (FMT == TQ_FMT_MX4) {
          uint32_t m = 0;
#pragma unroll
          for (int u = 0; u < P::kUnits; ++u) {
            const uint32_t b = xr.s[i * P::kUnits + u];
            m = max(m, b == 255u ? 0u : b);
          }
          const int now =
              max(ex[i], (int)__reduce_max_sync(0xFFFFFFFFu, m));
          if (lane == 0) s_fac[buf][r] = pow2_down(ex[i] - now);
          rose |= now != ex[i];
          ex[i] = now;
        }
#pragma unroll
        for (int u = 0; u < P::kUnits; ++u) {
          const int j = i * P::kUnits + u;
          const int unit = lane + 32 * u;  // of 8 k
          uint4 h;
          if constexpr (SRC == kBf16) {
            h.x = scaled_h2(xr.v[j].x, s);
            h.y = scaled_h2(xr.v[j].y, s);
            h.z = scaled_h2(xr.v[j].z, s);
            h.w = scaled_h2(xr.v[j].w, s);
          } else {
            uint32_t q[4];
            f4x8_to_h2(xr.v[j], q);
            const uint32_t f = FMT == TQ_FMT_MX4
                                   ? mx4_factor((int)xr.s[j], ex[i])
                                   : nv4_factor(xr.s[j]);
            h = make_uint4(hmul2(q[0], f), hmul2(q[1], f), hmul2(q[2], f),
                           hmul2(q[3], f));
          }
          // unit 4 t + s of a group of 128 k lies at position 4 s + t, so
          // that the four lanes of a quad read 64 consecutive bytes
          const int pos = (unit & ~15) | ((unit & 3) << 2) | ((unit >> 2) & 3);
          sts128(xbuf + buf * P::kXBuf + r * P::kXPitch + pos * 16, h);
        }
      }
      return rose;
    };

    load_x(0);
    int buf = 0;
#pragma unroll 1
    for (int st = 0; st < count; buf ^= 1) {
      const bool rose = stage_x(buf);
      const int any = __syncthreads_or(rose);
      const int end = st + P::kXStages < count ? st + P::kXStages : count;
      if (end < count) load_x(end);
      if (any) {
#pragma unroll
        for (int i = 0; i < kTiles; ++i) {
          const float f0 = s_fac[buf][8 * i + 2 * t];
          const float f1 = s_fac[buf][8 * i + 2 * t + 1];
          acc[i][0] *= f0;
          acc[i][1] *= f1;
          acc[i][2] *= f0;
          acc[i][3] *= f1;
        }
      }
      uint32_t xat = xbuf + buf * P::kXBuf + g * P::kXPitch + t * 16;
#pragma unroll 1
      for (; st < end; ++st, xat += 2 * kStageK) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 2) : "memory");
        __syncwarp();
        issue(st + kRing - 1);
        const uint32_t src = ring + (st % kRing) * P::kStage;
        // scale bytes of chunks t and t + 4 of rows g and g + 8
        uint32_t f[2][2][2];  // [half][row][block of the chunk]
        {
          constexpr int kB = FMT == TQ_FMT_MX4 ? 1 : 2;
          uint32_t b[2][2][kB];
          const uint32_t s0 = src + P::kCodes;
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const int row = g + 8 * r;
            // rows that do not start on a word boundary lie shifted
            const uint32_t shift =
                whole ? 0u
                      : (uint32_t)(reinterpret_cast<uintptr_t>(
                                       scales + min(row, last) * blocks) &
                                   3u);
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int c = 0; c < kB; ++c) {
                const int j = (t + 4 * h) * kB + c;
                b[h][r][c] = lds_u8(s0 + row * P::kScalePitch + shift + j);
                if (!whole && (int64_t)(st0 + st) * P::kScaleRow + j >= blocks)
                  b[h][r][c] = 0;  // past the row's end
              }
          }
          if constexpr (FMT == TQ_FMT_MX4) {
            uint32_t m = 0;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t e0 = b[h][0][0] == 255u ? 0u : b[h][0][0];
              const uint32_t e1 = b[h][1][0] == 255u ? 0u : b[h][1][0];
              m = __vmaxu2(m, e0 | e1 << 16);
            }
            m = __vmaxu2(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
            m = __vmaxu2(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
            const int n0 = max(R0, (int)(m & 0xFFFFu));
            const int n1 = max(R1, (int)(m >> 16));
            if (__any_sync(0xFFFFFFFFu, n0 != R0 || n1 != R1)) {
              const float f0 = pow2_down(R0 - n0), f1 = pow2_down(R1 - n1);
#pragma unroll
              for (int i = 0; i < kTiles; ++i) {
                acc[i][0] *= f0;
                acc[i][1] *= f0;
                acc[i][2] *= f1;
                acc[i][3] *= f1;
              }
              R0 = n0;
              R1 = n1;
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              f[h][0][0] = f[h][0][1] = mx4_factor((int)b[h][0][0], R0);
              f[h][1][0] = f[h][1][1] = mx4_factor((int)b[h][1][0], R1);
            }
          } else {
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int r = 0; r < 2; ++r) {
                f[h][r][0] = nv4_factor(b[h][r][0]);
                f[h][r][1] = nv4_factor(b[h][r][kB - 1]);
              }
          }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t chunk = (uint32_t)(t + 4 * h) ^ ((g & 1) << 2);
          const uint4 c0 = lds128(src + g * (kStageK / 2) + chunk * 16);
          const uint4 c1 = lds128(src + (g + 8) * (kStageK / 2) + chunk * 16);
          const uint32_t w0[4] = {c0.x, c0.y, c0.z, c0.w};
          const uint32_t w1[4] = {c1.x, c1.y, c1.z, c1.w};
#pragma unroll
          for (int s = 0; s < 4; ++s) {
            uint32_t p[4], q[4];
            f4x8_to_h2(w0[s], p);
            f4x8_to_h2(w1[s], q);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              p[i] = hmul2(p[i], f[h][0][s >> 1]);
              q[i] = hmul2(q[i], f[h][1][s >> 1]);
            }
#pragma unroll
            for (int i = 0; i < kTiles; ++i) {
              const uint4 v =
                  lds128(xat + 256 * h + 8 * i * P::kXPitch + 64 * s);
              mma_f16(acc[i], p[0], q[0], p[1], q[1], v.x, v.y);
              mma_f16(acc[i], p[2], q[2], p[3], q[3], v.z, v.w);
            }
          }
        }
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (lane == 0) {
#pragma unroll
      for (int i = 0; i < P::kPerWarp; ++i)
        s_exp[warp * P::kPerWarp + i] = ex[i];
    }
    __syncthreads();  // rings are free, exponents are there

    // partial sums in units of y (without g), [row of x][weight row]
    float *part = reinterpret_cast<float *>(smem);
#pragma unroll
    for (int i = 0; i < kTiles; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int b = 8 * i + 2 * t + (j & 1);
        int e = 0;
        if (FMT == TQ_FMT_MX4) e += (j < 2 ? R0 : R1) - 140;
        if (SRC == kBf16)
          e += s_exp[b] - 14;
        else if (FMT == TQ_FMT_MX4)
          e += s_exp[b] - 140;
        part[b * P::kPartPitch + 16 * warp + g + (j < 2 ? 0 : 8)] =
            scalbnf(acc[i][j], e);
      }
    if (ks > 1)
      cooperative_groups::this_cluster().sync();
    else
      __syncthreads();
    float gs = gw;
    if (SRC == kPacked && a.xg != nullptr) gs *= *a.xg;
    const uint32_t mine = smem_u32(part);
    for (int i = tid + rank * kThreads; i < rows * kTile; i += ks * kThreads) {
      const int b = i / kTile, r = i % kTile;
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
      v *= gs;
      if (row0 + r < a.n) {
        const int64_t row = a.ids != nullptr ? s_rows[base + b] : b0 + b;
        if (a.y_bf16)
          static_cast<__nv_bfloat16 *>(a.y)[row * a.ldy + row0 + r] =
              __float2bfloat16_rn(v);
        else
          static_cast<float *>(a.y)[row * a.ldy + row0 + r] = v;
      }
    }
    // the partial tiles have been read: shared memory may change, or go
    if (ks > 1)
      cooperative_groups::this_cluster().sync();
    else
      __syncthreads();
  };

  if (a.ids == nullptr) {
    const int64_t b0 = (int64_t)blockIdx.y * NT;
    pass(0, b0, (int)(a.batch - b0 < NT ? a.batch - b0 : NT));
    return;
  }
  // Rows of x that picked this expert, in ascending order (every CTA of the
  // cluster finds the same list), a segment of the ids at a time.
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
      if (expert == 0 && rank == 0 && i < a.batch &&
          (id < 0 || id >= a.n_experts)) {
        // nobody's row: NaN in this CTA's columns
        const int64_t end = row0 + kTile < a.n ? row0 + kTile : a.n;
        for (int64_t r = row0; r < end; ++r)
          static_cast<float *>(a.y)[i * a.ldy + r] = __int_as_float(0x7FC00000);
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
        s_rows[s_count[j * kWarps + warp] +
               __popc(vote & ((1u << lane) - 1u))] =
            (int)(seg + (j * kWarps + warp) * 32 + lane);
    }
    __syncthreads();
    const int total = s_count[kSegment / 32];
    for (int base = 0; base < total; base += NT)
      pass(base, 0, total - base < NT ? total - base : NT);
    __syncthreads();  // the list has been read
  }
}

template <int FMT, int NT, int SRC>
cudaError_t launch(const RowArgs &a, int64_t grid_y, cudaStream_t stream) {
  using P = RowPlan<FMT, NT>;
  auto kern = rows_f4_kernel<FMT, NT, SRC>;
  cudaError_t e = ensure_smem_limit<rows_f4_kernel<FMT, NT, SRC>>(P::kSmem);
  if (e != cudaSuccess) return e;
  const int64_t tiles = (a.n + P::kTile - 1) / P::kTile;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(tiles * a.ks), (unsigned)grid_y);
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

template <int SRC>
cudaError_t launch_nt(int format, int nt, const RowArgs &a, int64_t grid_y,
                      cudaStream_t stream) {
  const bool mx = format == TQ_FMT_MX4;
  switch (nt) {
    case 8:
      return mx ? launch<TQ_FMT_MX4, 8, SRC>(a, grid_y, stream)
                : launch<TQ_FMT_NV4, 8, SRC>(a, grid_y, stream);
    case 16:
      return mx ? launch<TQ_FMT_MX4, 16, SRC>(a, grid_y, stream)
                : launch<TQ_FMT_NV4, 16, SRC>(a, grid_y, stream);
    default: break;
  }
  if constexpr (SRC == kBf16) {
    if (nt == 32)
      return mx ? launch<TQ_FMT_MX4, 32, SRC>(a, grid_y, stream)
                : launch<TQ_FMT_NV4, 32, SRC>(a, grid_y, stream);
    return mx ? launch<TQ_FMT_MX4, 64, SRC>(a, grid_y, stream)
              : launch<TQ_FMT_NV4, 64, SRC>(a, grid_y, stream);
  }
  return cudaErrorInvalidValue;
}

int rows_per_pass(int64_t rows) {
  return rows <= 8 ? 8 : rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
}

// CTAs of a cluster: enough for every place on the device, at least two
// stages of K each.
cudaError_t split(int64_t n, int64_t k, int nt, int64_t copies, int *ks) {
  int dev = 0, sms = 148;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  const int64_t stages = (k + kStageK - 1) / kStageK;
  const int64_t tile = nt == 64 ? 256 : 128, places = nt == 64 ? sms : 2 * sms;
  const int64_t tiles = (n + tile - 1) / tile * copies;
  int64_t c = (places + tiles - 1) / tiles;
  if (c > stages / 2) c = stages / 2;
  if (c > 8) c = 8;
  if (c < 1) c = 1;
  *ks = (int)c;
  return cudaSuccess;
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

cudaError_t linear_f4_bf16(const WeightsView &w, const __nv_bfloat16 *x,
                           int64_t batch, int64_t ldx, float *y, int64_t ldy,
                           cudaStream_t stream) {
  RowArgs a = weight_args(w);
  a.x = x;
  a.ldx = ldx;
  a.batch = batch;
  a.y = y;
  a.ldy = ldy;
  const int nt = rows_per_pass(batch);
  const int64_t passes = (batch + nt - 1) / nt;
  cudaError_t e = split(w.n, w.k, nt, passes, &a.ks);
  // a grid's second dimension ends at 65535
  for (int64_t p = 0; p < passes && e == cudaSuccess; p += 65535) {
    const int64_t now = passes - p < 65535 ? passes - p : 65535;
    RowArgs b = a;
    b.x += p * nt * ldx;
    b.y = y + p * nt * ldy;
    b.batch -= p * nt;
    e = launch_nt<kBf16>(w.format, nt, b, now, stream);
  }
  return e;
}

cudaError_t launch_linear_experts_f4(const WeightsView &w, int n_experts,
                                     const int32_t *ids, int64_t tokens,
                                     const __nv_bfloat16 *x, int64_t ldx,
                                     float *y, int64_t ldy, int32_t *status,
                                     cudaStream_t stream) {
  RowArgs a = weight_args(w);
  a.x = x;
  a.ldx = ldx;
  a.batch = tokens;
  a.y = y;
  a.ldy = ldy;
  a.ids = ids;
  a.n_experts = n_experts;
  a.status = status;
  // experts that get rows at all, and the rows of one
  const int64_t used = tokens < n_experts ? tokens : n_experts;
  const int nt = rows_per_pass(2 * ((tokens + n_experts - 1) / n_experts));
  const cudaError_t e = split(w.n, w.k, nt, used, &a.ks);
  if (e != cudaSuccess) return e;
  return launch_nt<kBf16>(w.format, nt, a, n_experts, stream);
}

bool rows_f4_packed_supported(const WeightsView &x) { return x.n <= 16; }

cudaError_t rows_f4_packed(const WeightsView &w, const WeightsView &x, void *y,
                           int64_t ldy, int y_type, cudaStream_t stream) {
  RowArgs a = weight_args(w);
  a.xcodes = x.codes;
  a.xscales = reinterpret_cast<const uint8_t *>(x.scales);
  a.xg = x.lut;
  a.batch = x.n;
  a.y = y;
  a.ldy = ldy;
  a.y_bf16 = y_type == TQ_Y_BF16;
  const int nt = rows_per_pass(x.n);
  const cudaError_t e = split(w.n, w.k, nt, 1, &a.ks);
  if (e != cudaSuccess) return e;
  return launch_nt<kPacked>(w.format, nt, a, 1, stream);
}

}  // namespace tq
