// 4-bit float quantizer and decoder (tq_quantize_f4; tq_unpack of
// TQ_FMT_MX4 / TQ_FMT_NV4).
//
// Quantize, per block of consecutive values v of a row ("OCP Microscaling
// Formats (MX) Specification" v1.0, section 6.3, for MX4):
//   MX4  scale 2^E, E = floor(log2 max|v|) - 2; code = E2M1_RNE(v 2^-E)
//   NV4  scale s g, s = E4M3_RNE(max|v| / (6 g)); code = E2M1_RNE(v / (s g))
// A lane holds 8 values (one 16-byte load), so a block of 32 (16) is 4 (2)
// neighbouring lanes and its maximum two (one) shuffles; codes leave as one
// 4-byte store per lane. Bound by HBM: 2 + 0.53 bytes per value.
//
// Every decision equals exact arithmetic. MX4: v 2^-E is exact in fp32. NV4:
// quotients are taken as products with a reciprocal (relative error below
// 2^-21), and where one lies within 2^-19 of a border between two results
// the block is decided again in fp64: s g has 28 significant bits and a
// border times it at most 31, v has 8, so v and a border that differ do so
// by more than 2^-40 relative, far above the 2^-53 of an fp64 quotient.
#include "tq_f4.cuh"

namespace tq {
namespace {

// Largest magnitude (bf16 bits) of the 8 values of a 16-byte word.
__device__ __forceinline__ uint32_t max_mag8(const uint4 &w) {
  const uint32_t m = __vmaxu2(__vmaxu2(w.x & 0x7FFF7FFFu, w.y & 0x7FFF7FFFu),
                              __vmaxu2(w.z & 0x7FFF7FFFu, w.w & 0x7FFF7FFFu));
  return max(m >> 16, m & 0xFFFFu);
}

__device__ __forceinline__ float bf16_lo(uint32_t w) {
  return __uint_as_float(w << 16);
}
__device__ __forceinline__ float bf16_hi(uint32_t w) {
  return __uint_as_float(w & 0xFFFF0000u);
}

// Two E2M1 codes (nearest even, at most 6): lo in bits 0-3, hi in bits 4-7.
__device__ __forceinline__ uint32_t e2m1x2(float lo, float hi) {
  uint32_t r;
  asm("{\n .reg .b8 t;\n cvt.rn.satfinite.e2m1x2.f32 t, %1, %2;\n"
      " mov.b32 %0, {t, 0, 0, 0};\n}"
      : "=r"(r)
      : "f"(hi), "f"(lo));
  return r;
}

// The 8 codes of q[0..7].
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

// What an NV4 call derives from g once per thread.
struct Nv4 {
  float g, inv_g, inv_6g;
  bool exact;  // g so large or small that the fp32 quotients may be off
};

__device__ __forceinline__ Nv4 nv4_make(float g) {
  Nv4 s;
  s.g = g;
  s.inv_g = 1.0f / g;
  s.inv_6g = s.inv_g * (1.0f / 6.0f);
  s.exact = !(g > 1e-30f && g < 1e30f);
  return s;
}

// Block scale byte of an NV4 block with the largest magnitude `top`.
__device__ __forceinline__ uint32_t nv4_scale(float top, const Nv4 &s) {
  const float r = top * s.inv_6g;
  // Borders lie halfway between E4M3 values: at most 5 significant bits, and
  // below 2^-6 odd multiples of 2^-10. Both have the low 19 bits clear.
  const bool near = ((__float_as_uint(r) + 16u) & 0x7FFFFu) < 32u;
  if ((near && r != 0.0f) || s.exact)
    return e4m3_of_f64((double)top / (6.0 * (double)s.g));
  uint16_t b;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
      : "=h"(b)
      : "f"(0.0f), "f"(r));
  return b;
}

template <int FMT>
__device__ __forceinline__ void quantize8(const uint4 &w, bool live,
                                          const Nv4 &s, uint32_t *codes,
                                          uint32_t *byte, bool *bad) {
  uint32_t m = live ? max_mag8(w) : 0u;
  m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
  if (FMT == TQ_FMT_MX4) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
  if (m >= 0x7F80u) {  // NaN or Inf in the block
    *bad = true;
    *codes = 0;
    *byte = FMT == TQ_FMT_MX4 ? 0xFFu : 0x7Fu;
    return;
  }
  float inv, q[8];
  const float top = __uint_as_float(m << 16);
  double d = 0.0;
  if (FMT == TQ_FMT_MX4) {
    // bf16 exponent field f: floor(log2 top) = f - 127, so the byte is
    // f - 2; subnormal maxima (f = 0) clamp to 0 as well
    const int f = (int)(m >> 7);
    *byte = (uint32_t)max(f - 2, 0);
    inv = __uint_as_float((254u - *byte) << 23);  // 2^(127 - byte)
  } else {
    *byte = nv4_scale(top, s);
    const float sf = e4m3_to_f32(*byte);
    inv = sf == 0.0f ? 0.0f : __fdividef(s.inv_g, sf);
    d = (double)sf * (double)s.g;
  }
  const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    q[2 * i] = bf16_lo(v[i]) * inv;
    q[2 * i + 1] = bf16_hi(v[i]) * inv;
  }
  *codes = e2m1x8(q);
  if (FMT == TQ_FMT_NV4) {
    // Borders are odd multiples of 1/4, 1/2, 1 with at most 3 significant
    // bits: the low 21 bits of q are clear there.
    uint32_t close = 0xFFFFFFFFu;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t u = max(__float_as_uint(q[i]) & 0x7FFFFFFFu, 0x3E010000u);
      close = min(close, (u + 16u) & 0x1FFFFFu);
    }
    if ((close < 32u || s.exact) && inv != 0.0f) {
      uint32_t c = 0;
#pragma unroll 1
      for (int i = 0; i < 8; ++i) {
        const uint32_t h = v[0] * (i < 2) + v[1] * (i >> 1 == 1) +
                           v[2] * (i >> 1 == 2) + v[3] * (i >> 1 == 3);
        c |= e2m1_of_f64(i & 1 ? bf16_hi(h) : bf16_lo(h), d) << (4 * i);
      }
      *codes = c;
    }
  }
}

// One lane per 8 values; `units` = n * k / 8. MODE 0: MX4; 1: NV4 with g in
// *ts; 2: NV4 with max |W| in *ts.
template <int FMT, bool AMAX>
__global__ void __launch_bounds__(256)
    quantize_f4_kernel(const uint16_t *__restrict__ W, int64_t units,
                       int64_t row_units, int64_t ldw,
                       uint32_t *__restrict__ codes,
                       uint8_t *__restrict__ scales, const float *ts,
                       int32_t *status) {
  Nv4 s = {};
  bool bad = false, bad_g = false;
  if (FMT == TQ_FMT_NV4) {
    const float g = AMAX ? nv4_tensor_scale(*ts) : *ts;
    bad_g = !(g > 0.0f && g < __int_as_float(0x7F800000));
    s = nv4_make(bad_g ? 1.0f : g);
  }
  const int64_t step = (int64_t)gridDim.x * blockDim.x;
  const int64_t first = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  // whole warps run the shuffles: the loop count is the block's
  const int64_t rounds =
      (units - (int64_t)blockIdx.x * blockDim.x + step - 1) / step;
  for (int64_t r = 0; r < rounds; ++r) {
    const int64_t u = first + r * step;
    const bool live = u < units;
    uint4 w = make_uint4(0, 0, 0, 0);
    if (live) {
      const int64_t row = u / row_units;
      w = __ldg(reinterpret_cast<const uint4 *>(W + row * ldw) +
                (u - row * row_units));
    }
    uint32_t c, b;
    quantize8<FMT>(w, live, s, &c, &b, &bad);
    if (!live) continue;
    if (bad_g) {
      c = 0;
      b = 0x7Fu;
    }
    codes[u] = c;
    constexpr int kLanes = FMT == TQ_FMT_MX4 ? 4 : 2;
    if (u % kLanes == 0) scales[u / kLanes] = (uint8_t)b;
  }
  if (bad) report(status, TQ_ERR_NONFINITE);
  if (bad_g && threadIdx.x == 0) report(status, TQ_ERR_INVALID_ARG);
}

// max |W| over the finite values, as fp32 bits (magnitudes order like them).
__global__ void __launch_bounds__(256)
    amax_f4_kernel(const uint16_t *__restrict__ W, int64_t units,
                   int64_t row_units, int64_t ldw, uint32_t *out) {
  uint32_t m = 0;
  for (int64_t u = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; u < units;
       u += (int64_t)gridDim.x * blockDim.x) {
    const int64_t row = u / row_units;
    const uint4 w = __ldg(reinterpret_cast<const uint4 *>(W + row * ldw) +
                          (u - row * row_units));
    const uint32_t t = max_mag8(w);
    if (t < 0x7F80u) {
      m = max(m, t);
    } else {  // some value is not finite: take the others one by one
      const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t a = (v[i >> 1] >> (16 * (i & 1))) & 0x7FFFu;
        if (a < 0x7F80u) m = max(m, a);
      }
    }
  }
  m = __reduce_max_sync(0xFFFFFFFFu, m);
  if ((threadIdx.x & 31) == 0 && m != 0) atomicMax(out, m << 16);
}

__global__ void tensor_scale_kernel(float *ts) { *ts = nv4_tensor_scale(*ts); }

// Decode: a thread turns 8 codes (one 4-byte load) into 8 bf16.
template <int FMT>
__global__ void __launch_bounds__(256)
    unpack_f4_kernel(const uint32_t *__restrict__ codes,
                     const uint8_t *__restrict__ scales,
                     const float *__restrict__ ts, int64_t units,
                     uint4 *__restrict__ out, int32_t *status) {
  const float g = FMT == TQ_FMT_NV4 && ts != nullptr ? *ts : 1.0f;
  bool bad = false;
  for (int64_t u = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; u < units;
       u += (int64_t)gridDim.x * blockDim.x) {
    const uint32_t w = __ldg(codes + u);
    const uint32_t b = __ldg(scales + u / (f4_block(FMT) / 8));
    if (FMT == TQ_FMT_NV4 && (b & 0x80u)) bad = true;
    const float s = f4_scale<FMT>(b);
    uint32_t h[4], o[4];
    f4x8_to_h2(w, h);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float2 f = __half22float2(*reinterpret_cast<__half2 *>(&h[i]));
      f.x *= s;  // exact: 2 significant bits times 1 or 4
      f.y *= s;
      if (FMT == TQ_FMT_NV4) {
        f.x *= g;
        f.y *= g;
      }
      const __nv_bfloat162 p = __floats2bfloat162_rn(f.x, f.y);
      o[i] = *reinterpret_cast<const uint32_t *>(&p);
    }
    __stcs(out + u, make_uint4(o[0], o[1], o[2], o[3]));
  }
  if (bad) report(status, TQ_ERR_BAD_CODE);
}

cudaError_t grid_for(int64_t units, int per_sm, int *grid) {
  int dev = 0, sms = 148;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  const int64_t want = (units + 255) / 256;
  *grid = (int)(want < (int64_t)sms * per_sm ? want : (int64_t)sms * per_sm);
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_quantize_f4(const uint16_t *W, int64_t n, int64_t k,
                               int64_t ldw, int format, uint8_t *codes,
                               uint8_t *scales, float *ts, bool given,
                               int32_t *status, cudaStream_t stream) {
  const int64_t units = n * (k / 8);
  const bool own_scale = format == TQ_FMT_NV4 && !given;
  if (units == 0 && !own_scale) return cudaSuccess;
  int grid = 1;
  cudaError_t e = grid_for(units, 16, &grid);
  if (e != cudaSuccess) return e;
  uint32_t *c = reinterpret_cast<uint32_t *>(codes);
  if (own_scale) {
    if ((e = cudaMemsetAsync(ts, 0, sizeof(float), stream)) != cudaSuccess)
      return e;
    if (units > 0) {
      amax_f4_kernel<<<grid, 256, 0, stream>>>(
          W, units, k / 8, ldw, reinterpret_cast<uint32_t *>(ts));
      if ((e = cudaGetLastError()) != cudaSuccess) return e;
      quantize_f4_kernel<TQ_FMT_NV4, true><<<grid, 256, 0, stream>>>(
          W, units, k / 8, ldw, c, scales, ts, status);
      if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    tensor_scale_kernel<<<1, 1, 0, stream>>>(ts);
    return cudaGetLastError();
  }
  if (format == TQ_FMT_NV4)
    quantize_f4_kernel<TQ_FMT_NV4, false><<<grid, 256, 0, stream>>>(
        W, units, k / 8, ldw, c, scales, ts, status);
  else
    quantize_f4_kernel<TQ_FMT_MX4, false><<<grid, 256, 0, stream>>>(
        W, units, k / 8, ldw, c, scales, ts, status);
  return cudaGetLastError();
}

cudaError_t launch_unpack_f4(const WeightsView &w, uint16_t *out,
                             int32_t *status, cudaStream_t stream) {
  const int64_t units = w.n * (w.k / 8);
  int grid = 1;
  const cudaError_t e = grid_for(units, 16, &grid);
  if (e != cudaSuccess) return e;
  const uint32_t *c = reinterpret_cast<const uint32_t *>(w.codes);
  const uint8_t *s = reinterpret_cast<const uint8_t *>(w.scales);
  uint4 *o = reinterpret_cast<uint4 *>(out);
  if (w.format == TQ_FMT_MX4)
    unpack_f4_kernel<TQ_FMT_MX4><<<grid, 256, 0, stream>>>(c, s, nullptr,
                                                           units, o, status);
  else
    unpack_f4_kernel<TQ_FMT_NV4><<<grid, 256, 0, stream>>>(c, s, w.lut, units,
                                                           o, status);
  return cudaGetLastError();
}

}  // namespace tq
