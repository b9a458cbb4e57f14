// 4-bit float quantizer and decoder (tq_quantize_f4; tq_unpack of
// TQ_FMT_MX4 / TQ_FMT_NV4).
//
// Quantize, per block of consecutive values v of a row ("OCP Microscaling
// Formats (MX) Specification" v1.0, section 6.3, for MX4):
//   MX4  scale 2^E, E = floor(log2 max|v|) - 2; code = E2M1_RNE(v 2^-E)
//   NV4  scale s g, s = E4M3_RNE(max|v| / (6 g)); code = E2M1_RNE(v / (s g))
// MX4: a lane holds 8 values (one 16-byte load), a block of 32 is 4 neighbouring
// lanes and its maximum two shuffles. NV4: a lane holds a whole block of 16 (two
// loads), since what a block costs (below) would be paid twice otherwise. Bound
// by HBM, 2 + 0.53 bytes per value, and nearly as much by arithmetic. With
// tq_unpack after it: MX4, 21504 x 5376: 105 us, 5.6 TB/s of 4.6 bytes per value
// both ways; NV4, 8192 x 5376 with a scale of its own: 66 us.
//
// Every decision equals exact arithmetic. MX4: v 2^-E is exact in fp32. NV4:
// quotients are taken as products with a reciprocal, relative error below
// 2^-21, so only those next to a border t between two codes need more. Such
// quotients are not rare: with g = max|W| / 2688 and values of 8 significant
// bits, many lie at a border but for the rounding of g. But at a border v is
// close to t d, d = s g, t one of 1, 3, 5, 7 (times a power of two) and v of 8
// bits, and two different v / t differ by 2^-13 or more: all the close ones of
// a block have one v / t, on one side of d. So a block asks once, per t,
// whether t d is close to an 8-bit number, takes the side from the sign of
// v - t d (exact in two fused multiply-adds, d held as an unrounded sum), and
// moves its reciprocal by 2^-19 to that side; on a tie it clears the last bits
// of the quotients instead. (8192 x 5376: 26 us; with each close
// quotient decided by itself 36 us, in fp64 133 us.) The block scale
// is settled in the same manner, quotient by quotient.
#include "tq_f4.cuh"

namespace tq {
namespace {

__device__ __forceinline__ float bf16_lo(uint32_t w) {
  return __uint_as_float(w << 16);
}
__device__ __forceinline__ float bf16_hi(uint32_t w) {
  return __uint_as_float(w & 0xFFFF0000u);
}

// The 8 E2M1 codes of q[0..7] (nearest even, at most 6), q[0] lowest.
__device__ __forceinline__ uint32_t e2m1x8(const float (&q)[8]) {
  uint32_t r;
  asm("{\n .reg .b8 t0, t1, t2, t3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 t0, %2, %1;\n"
      " cvt.rn.satfinite.e2m1x2.f32 t1, %4, %3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 t2, %6, %5;\n"
      " cvt.rn.satfinite.e2m1x2.f32 t3, %8, %7;\n"
      " mov.b32 %0, {t0, t1, t2, t3};\n}"
      : "=r"(r)
      : "f"(q[0]), "f"(q[1]), "f"(q[2]), "f"(q[3]), "f"(q[4]), "f"(q[5]),
        "f"(q[6]), "f"(q[7]));
  return r;
}

// E4M3 byte of a positive fp64 quotient, nearest even, at most 448. The
// quotient is scaled to units of its last place (2^-9 below 2^-6) and
// rounded to an integer there.
__device__ __noinline__ uint32_t e4m3_of_f64(double r) {
  if (r >= 448.0) return 0x7Eu;
  int e = (int)((__double_as_longlong(r) >> 52) & 0x7FF) - 1023;
  if (e < -6) e = -6;
  int m = __double2int_rn(scalbn(r, 3 - e));  // 8..16; below 8 subnormal
  if (m == 16) {
    m = 8;
    ++e;
  }
  return m >= 8 ? (uint32_t)((e + 7) * 8 + (m - 8)) : (uint32_t)m;
}

// E2M1 code of v / d decided in fp64 (d > 0).
__device__ __noinline__ uint32_t e2m1_of_f64(float v, double d) {
  const double q = fabs((double)v) / d;
  const uint32_t c = (uint32_t)(q > 0.25) + (q >= 0.75) + (q > 1.25) +
                     (q >= 1.75) + (q > 2.5) + (q >= 3.5) + (q > 5.0);
  return c | ((__float_as_uint(v) >> 28) & 8u);
}

// g of an NV4 matrix from max |W| (fp32 bits of a bf16 magnitude).
__device__ __forceinline__ float nv4_tensor_scale(float amax) {
  return amax == 0.0f ? 1.0f : (float)((double)amax / 2688.0);
}

// d = hi + lo exactly.
struct Two {
  float hi, lo;
};

__device__ __forceinline__ Two two_product(float a, float b) {
  Two d;
  d.hi = a * b;
  d.lo = fmaf(a, b, -d.hi);
  return d;
}

// A quotient q ~ v / d whose bits below the top BITS are within 16 of a
// border's (all zero): the border itself where v / d is exactly on it, else
// the number next to the border on the side of v / d.
template <uint32_t BITS>
__device__ __forceinline__ bool near_border(float q) {
  return ((__float_as_uint(q) + 16u) & ((1u << BITS) - 1u)) < 32u;
}

template <uint32_t BITS>
__device__ __forceinline__ float settle(float q, float v, const Two &d) {
  const uint32_t u =
      (__float_as_uint(q) + (1u << (BITS - 1))) & ~((1u << BITS) - 1u);
  const float t = __uint_as_float(u);
  if (t == 0.0f || fabsf(t) > 1e9f) return t;  // Inf among them: saturates
  const float r = fmaf(-t, d.lo, fmaf(-t, d.hi, v));
  if (r == 0.0f) return t;
  return __uint_as_float((r > 0.0f) == (t > 0.0f) ? u + 1u : u - 1u);
}

// What an NV4 call derives from g once per thread.
struct Nv4 {
  float g, inv_g, inv_6g;
  Two six_g;
  bool exact;  // g so large or small that the fp32 quotients may be off
};

__device__ __forceinline__ Nv4 nv4_make(float g) {
  Nv4 s;
  s.g = g;
  s.inv_g = 1.0f / g;
  s.inv_6g = s.inv_g * (1.0f / 6.0f);
  s.six_g = two_product(6.0f, g);
  s.exact = !(g > 1e-30f && g < 1e30f);
  return s;
}

// Block scale byte of an NV4 block with the largest magnitude `top`. Borders
// lie halfway between E4M3 values: at most 5 significant bits, and below 2^-6
// odd multiples of 2^-10, so their low 19 bits are clear.
__device__ __forceinline__ uint32_t nv4_scale(float top, const Nv4 &s) {
  if (s.exact) return e4m3_of_f64((double)top / (6.0 * (double)s.g));
  float r = top * s.inv_6g;
  if (near_border<19>(r)) r = settle<19>(r, top, s.six_g);
  uint16_t b;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
      : "=h"(b)
      : "f"(0.0f), "f"(r));
  return b;
}

// Words of 8 values that a lane takes at once.
template <int FMT>
constexpr int kWords = FMT == TQ_FMT_MX4 ? 1 : 2;

template <int FMT>
__device__ __forceinline__ void quantize_words(const uint4 (&w)[kWords<FMT>],
                                               const Nv4 &s,
                                               uint32_t (&codes)[kWords<FMT>],
                                               uint32_t *byte, bool *bad) {
  uint32_t m = max_mag8(w[0]);
  if constexpr (FMT == TQ_FMT_MX4) {
    m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
    m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
  } else {
    m = max(m, max_mag8(w[1]));
  }
  if (m >= 0x7F80u) {  // NaN or Inf in the block
    *bad = true;
#pragma unroll
    for (int h = 0; h < kWords<FMT>; ++h) codes[h] = 0;
    *byte = FMT == TQ_FMT_MX4 ? 0xFFu : 0x7Fu;
    return;
  }
  float inv;
  const float top = __uint_as_float(m << 16);
  float sf = 0.0f;
  bool tie = false;
  if (FMT == TQ_FMT_MX4) {
    // bf16 exponent field f: floor(log2 top) = f - 127, so the byte is
    // f - 2; subnormal maxima (f = 0) clamp to 0 as well
    const int f = (int)(m >> 7);
    *byte = (uint32_t)max(f - 2, 0);
    inv = __uint_as_float((254u - *byte) << 23);  // 2^(127 - byte)
  } else {
    *byte = nv4_scale(top, s);
    sf = e4m3_to_f32(*byte);
    inv = sf == 0.0f ? 0.0f : __fdividef(s.inv_g, sf);
    const Two d = two_product(sf, s.g);
#pragma unroll
    for (int t = 1; t < 8; t += 2) {
      const uint32_t u = __float_as_uint((float)t * d.hi) + 64u;
      if ((u & 0xFFFFu) < 128u) {  // within 64 units of an 8-bit number
        const float r = fmaf(-(float)t, d.lo,
                             fmaf(-(float)t, d.hi,
                                  __uint_as_float(u & 0xFFFF0000u)));
        if (r == 0.0f)
          tie = true;
        else
          inv = __uint_as_float(__float_as_uint(inv) + (r > 0.0f ? 16u : -16u));
        break;
      }
    }
  }
#pragma unroll
  for (int h = 0; h < kWords<FMT>; ++h) {
    const uint32_t v[4] = {w[h].x, w[h].y, w[h].z, w[h].w};
    float q[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      asm("{\n .reg .b64 a, b;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %4};\n"
          " mul.rn.f32x2 a, a, b;\n mov.b64 {%0, %1}, a;\n}"
          : "=f"(q[2 * i]), "=f"(q[2 * i + 1])
          : "f"(bf16_lo(v[i])), "f"(bf16_hi(v[i])), "f"(inv));
    }
    if (FMT == TQ_FMT_NV4 && tie) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        q[i] = __uint_as_float((__float_as_uint(q[i]) + 8u) & ~15u);
    }
    codes[h] = e2m1x8(q);
    if (FMT == TQ_FMT_NV4 && s.exact && sf != 0.0f) {
      const double d = (double)sf * (double)s.g;
      uint32_t c = 0;
#pragma unroll 1
      for (int i = 0; i < 8; ++i) {
        const uint32_t x = i < 2 ? v[0] : i < 4 ? v[1] : i < 6 ? v[2] : v[3];
        c |= e2m1_of_f64(i & 1 ? bf16_hi(x) : bf16_lo(x), d) << (4 * i);
      }
      codes[h] = c;
    }
  }
}

// `rows` rows of `units` 16-byte units (8 values), `pitch` units apart; a dense
// matrix comes as one row. A block takes kPer * 256 consecutive units of a
// row; a thread's kPer loads are in flight together.
constexpr int kPer = 4, kChunk = 256 * kPer;

template <int FMT>
__global__ void __launch_bounds__(256, 5)
    quantize_f4_kernel(const uint4 *__restrict__ W, int64_t rows,
                       int64_t units, int64_t pitch,
                       uint32_t *__restrict__ codes,
                       uint8_t *__restrict__ scales, const float *ts,
                       int32_t *status) {
  pdl_launch_dependents();
  pdl_wait();
  Nv4 s = {};
  bool bad = false, bad_g = false;
  if (FMT == TQ_FMT_NV4) {
    const float g = *ts;
    bad_g = !(g > 0.0f && g < __int_as_float(0x7F800000));
    s = nv4_make(bad_g ? 1.0f : g);
  }
  for (int64_t row = blockIdx.y; row < rows; row += gridDim.y) {
    const uint4 *src = W + row * pitch;
    // whole warps run the shuffles: the loop goes by the block's first unit
    for (int64_t first = (int64_t)blockIdx.x * kChunk; first < units;
         first += (int64_t)gridDim.x * kChunk) {
      const int64_t u0 = first + threadIdx.x * kWords<FMT>;
      constexpr int N = kWords<FMT>, kRounds = kPer / N;
      uint4 w[kRounds][N];
#pragma unroll
      for (int i = 0; i < kRounds; ++i) {
        const int64_t u = u0 + 256 * N * i;
#pragma unroll
        for (int h = 0; h < N; ++h) {
          w[i][h] = make_uint4(0, 0, 0, 0);
          if (u < units) w[i][h] = __ldg(src + u + h);  // units: a multiple of N
        }
      }
#pragma unroll
      for (int i = 0; i < kRounds; ++i) {
        const int64_t u = u0 + 256 * N * i;
        uint32_t c[N], b;
        quantize_words<FMT>(w[i], s, c, &b, &bad);
        if (u >= units) continue;
        const int64_t at = row * units + u;
        if constexpr (FMT == TQ_FMT_MX4) {
          codes[at] = c[0];
          if (threadIdx.x % 4 == 0) scales[at / 4] = (uint8_t)b;
        } else {
          if (bad_g) {
            c[0] = c[N - 1] = 0;
            b = 0x7Fu;
          }
          *reinterpret_cast<uint2 *>(codes + at) = make_uint2(c[0], c[N - 1]);
          scales[at / 2] = (uint8_t)b;
        }
      }
    }
  }
  if (bad) report(status, TQ_ERR_NONFINITE);
  if (bad_g && threadIdx.x == 0) report(status, TQ_ERR_INVALID_ARG);
}

// max |W| over the finite values, as bf16 bits (magnitudes order like them),
// in scratch[0]; the last block to arrive (scratch[1] counts them) turns it
// into g. Goes from the end of the matrix to its front.
__global__ void __launch_bounds__(256)
    amax_f4_kernel(const uint4 *__restrict__ W, int64_t rows, int64_t units,
                   int64_t pitch, uint32_t *scratch, float *ts) {
  pdl_launch_dependents();
  pdl_wait();
  uint32_t m = 0;
  const int64_t chunks = (units + kChunk - 1) / kChunk;
  for (int64_t r = blockIdx.y; r < rows; r += gridDim.y) {
    const uint4 *src = W + (rows - 1 - r) * pitch;
    for (int64_t c = blockIdx.x; c < chunks; c += gridDim.x) {
      const int64_t u0 = (chunks - 1 - c) * kChunk + threadIdx.x;
      uint4 w[kPer];
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        w[i] = make_uint4(0, 0, 0, 0);
        if (u0 + 256 * i < units) w[i] = __ldg(src + u0 + 256 * i);
      }
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        uint32_t t = max_mag8(w[i]);
        if (t >= 0x7F80u) t = max_finite8(w[i]);
        m = max(m, t);
      }
    }
  }
  m = __reduce_max_sync(0xFFFFFFFFu, m);
  __shared__ uint32_t s_m[8];
  if ((threadIdx.x & 31) == 0) s_m[threadIdx.x >> 5] = m;
  __syncthreads();
  if (threadIdx.x != 0) return;
#pragma unroll
  for (int i = 1; i < 8; ++i) m = max(m, s_m[i]);
  atomicMax(scratch, m);
  __threadfence();
  if (atomicAdd(scratch + 1, 1u) == gridDim.x * gridDim.y - 1) {
    __threadfence();
    const uint32_t all = atomicMax(scratch, 0u);
    *ts = nv4_tensor_scale(__uint_as_float(all << 16));
  }
}

// Decode: a thread turns kPer groups of 8 codes (4 bytes each) into bf16.
template <int FMT>
__global__ void __launch_bounds__(256)
    unpack_f4_kernel(const uint32_t *__restrict__ codes,
                     const uint8_t *__restrict__ scales,
                     const float *__restrict__ ts, int64_t units,
                     uint4 *__restrict__ out, int32_t *status) {
  pdl_launch_dependents();
  pdl_wait();
  const float g = FMT == TQ_FMT_NV4 && ts != nullptr ? *ts : 1.0f;
  bool bad = false;
  for (int64_t u0 = (int64_t)blockIdx.x * kChunk + threadIdx.x; u0 < units;
       u0 += (int64_t)gridDim.x * kChunk) {
    uint32_t w[kPer], b[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int64_t u = u0 + 256 * i;
      w[i] = b[i] = 0;
      if (u < units) {
        w[i] = __ldg(codes + u);
        b[i] = __ldg(scales + u / (f4_block(FMT) / 8));
      }
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int64_t u = u0 + 256 * i;
      if (FMT == TQ_FMT_NV4 && (b[i] & 0x80u)) bad = true;
      const float s = f4_scale<FMT>(b[i]);
      uint32_t h[4], o[4];
      f4x8_to_h2(w[i], h);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float2 f = __half22float2(*reinterpret_cast<__half2 *>(&h[j]));
        f.x *= s;  // exact: 2 significant bits times 1 or 4
        f.y *= s;
        if (FMT == TQ_FMT_NV4) {
          f.x *= g;
          f.y *= g;
        }
        const __nv_bfloat162 p = __floats2bfloat162_rn(f.x, f.y);
        o[j] = *reinterpret_cast<const uint32_t *>(&p);
      }
      if (u < units) __stcs(out + u, make_uint4(o[0], o[1], o[2], o[3]));
    }
  }
  if (bad) report(status, TQ_ERR_BAD_CODE);
}

// Blocks for `units` units of each of `rows` rows, 8 per SM at most.
cudaError_t grid_for(int64_t rows, int64_t units, dim3 *grid) {
  int dev = 0, sms = 148;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  const int64_t want = (units + kChunk - 1) / kChunk, most = (int64_t)sms * 8;
  const int64_t x = want < most ? want : most;
  const int64_t y = rows < most / x ? rows : most / x;
  *grid = dim3((unsigned)x, (unsigned)(y < 1 ? 1 : y));
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_quantize_f4(const uint16_t *W, int64_t n, int64_t k,
                               int64_t ldw, int format, uint8_t *codes,
                               uint8_t *scales, float *ts, bool given,
                               int32_t *status, cudaStream_t stream) {
  const bool own_scale = format == TQ_FMT_NV4 && !given;
  if (n == 0 || k == 0) {
    if (!own_scale) return cudaSuccess;
    static const float one = 1.0f;  // of an empty matrix
    return cudaMemcpyAsync(ts, &one, sizeof(one), cudaMemcpyHostToDevice,
                           stream);
  }
  const bool dense = ldw == k || n == 1;
  const int64_t rows = dense ? 1 : n, units = dense ? n * (k / 8) : k / 8;
  const uint4 *src = reinterpret_cast<const uint4 *>(W);
  uint32_t *c = reinterpret_cast<uint32_t *>(codes);
  dim3 grid;
  cudaError_t e = grid_for(rows, units, &grid);
  if (e != cudaSuccess) return e;
  if (own_scale) {
    // the front of the codes, not written yet, is the maximum's scratch
    if ((e = cudaMemsetAsync(codes, 0, 8, stream)) != cudaSuccess) return e;
    if ((e = launch_pdl(amax_f4_kernel, grid, dim3(256), 0, stream, src, rows,
                        units, ldw / 8, c, ts)) != cudaSuccess)
      return e;
    return launch_pdl(quantize_f4_kernel<TQ_FMT_NV4>, grid, dim3(256), 0,
                      stream, src, rows, units, ldw / 8, c, scales,
                      (const float *)ts, status);
  }
  if (format == TQ_FMT_NV4)
    return launch_pdl(quantize_f4_kernel<TQ_FMT_NV4>, grid, dim3(256), 0,
                      stream, src, rows, units, ldw / 8, c, scales,
                      (const float *)ts, status);
  return launch_pdl(quantize_f4_kernel<TQ_FMT_MX4>, grid, dim3(256), 0,
                    stream, src, rows, units, ldw / 8, c, scales,
                    (const float *)nullptr, status);
}

cudaError_t launch_unpack_f4(const WeightsView &w, uint16_t *out,
                             int32_t *status, cudaStream_t stream) {
  const int64_t units = w.n * (w.k / 8);
  dim3 grid;
  const cudaError_t e = grid_for(1, units, &grid);
  if (e != cudaSuccess) return e;
  const uint32_t *c = reinterpret_cast<const uint32_t *>(w.codes);
  const uint8_t *s = reinterpret_cast<const uint8_t *>(w.scales);
  uint4 *o = reinterpret_cast<uint4 *>(out);
  return w.format == TQ_FMT_MX4
             ? launch_pdl(unpack_f4_kernel<TQ_FMT_MX4>, grid, dim3(256), 0,
                          stream, c, s, (const float *)nullptr, units, o,
                          status)
             : launch_pdl(unpack_f4_kernel<TQ_FMT_NV4>, grid, dim3(256), 0,
                          stream, c, s, w.lut, units, o, status);
}

}  // namespace tq
