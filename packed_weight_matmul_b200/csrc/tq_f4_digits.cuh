// bf16 rows of x as sums of 4-bit ones, for the kernels that multiply on the
// block-scaled tensor cores (tq_f4_decode.cu, tq_f4_digits.cu, tq_f4_gemm.cu).
//
//   In a block of x let f be the exponent of its largest magnitude and
//   r = x 2^(1 - f) in (-4, 4). Digits in base 8: d_i = round(r_i) in
//   {-4 .. 4}, r_{i+1} = 8 (r_i - d_i), so x = 2^(f - 1) sum_i d_i 8^-i, and
//   after 8 digits the rest is at most 2^-23 of the block's largest value.
//   All of -4 .. 4 are E2M1 values. Row 8 b + i of the B operand holds d_i of
//   row b of x.
//   MX4: its block scale 2^(f - T - 1 - 3 i) is an E8M0 byte. T = 0, so that
//        the sums leave fp32's range only where y does, except for rows (slices
//        of K) whose largest value has an exponent X below -40: T = X + 40.
//        Digits whose scale falls below 2^-127 take that one: off by 2^-80 of
//        the row's largest at most.
//   NV4: an E4M3 byte reaches from 2^-9 to 2^8 only, so row i has a factor
//        2^(X - 9 - 3 i) of its own, applied to its sum, and the block scale
//        2^(f - X + 8); blocks below 2^-17 of the row's largest take the
//        smallest scale, which leaves them off by 2^-40 of it.
//   y = 2^T sum_i D_i (MX4) or 2^(X - 9) sum_i 8^-i D_i (NV4), D the fp32
//   accumulators. NaN and Inf count as 0 in the digits; their rows of x are
//   flagged and the products with them added to the sums afterwards.
#pragma once

#include "tq_f4.cuh"

namespace tq {
namespace f4 {

// NaN and Inf become 0.
__device__ __forceinline__ uint4 only_finite8(uint4 w) {
  uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if ((v[i] & 0x7F80u) == 0x7F80u) v[i] &= 0xFFFF0000u;
    if ((v[i] & 0x7F800000u) == 0x7F800000u) v[i] &= 0x0000FFFFu;
  }
  return make_uint4(v[0], v[1], v[2], v[3]);
}

struct F2 {
  uint64_t v;
};
__device__ __forceinline__ F2 pack2(float a, float b) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(r.v)
      : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
// E2M1 codes of 8 small integers, the first lowest.
__device__ __forceinline__ uint32_t codes8(const F2 (&q)[4]) {
  uint32_t r;
  asm("{\n .reg .b8 t0, t1, t2, t3;\n .reg .f32 a, b;\n"
      " mov.b64 {a, b}, %1;\n cvt.rn.satfinite.e2m1x2.f32 t0, b, a;\n"
      " mov.b64 {a, b}, %2;\n cvt.rn.satfinite.e2m1x2.f32 t1, b, a;\n"
      " mov.b64 {a, b}, %3;\n cvt.rn.satfinite.e2m1x2.f32 t2, b, a;\n"
      " mov.b64 {a, b}, %4;\n cvt.rn.satfinite.e2m1x2.f32 t3, b, a;\n"
      " mov.b32 %0, {t0, t1, t2, t3};\n}"
      : "=r"(r)
      : "l"(q[0].v), "l"(q[1].v), "l"(q[2].v), "l"(q[3].v));
  return r;
}

// 2^T of a row of exponent X (both biased).
__device__ __forceinline__ int mx4_reference(int X) { return min(X + 40, 127); }

// Block scale of exponent f (biased, at least 1) in a row of exponent X: the
// byte of digit 0 (the others of MX4 lie 3, 6, .. below, not under 0) and the
// exponent field of the factor that brings the block to (-4, 4).
template <int FMT>
__device__ __forceinline__ void digit_scale(int f, int X, uint32_t *byte,
                                            uint32_t *field) {
  if (FMT == TQ_FMT_MX4) {
    *byte = (uint32_t)(126 + f - mx4_reference(X));
    *field = (uint32_t)(255 - f);
  } else {
    const int e = max(f - X + 8, -9);
    *byte = e >= -6 ? (uint32_t)(e + 7) << 3 : 1u << (e + 9);
    *field = (uint32_t)(263 - X - e);
  }
}

// The 8 digits of 8 values, emit(i, codes of digit i) in order.
template <typename Emit>
__device__ __forceinline__ void digits8(const uint4 &w, uint32_t field,
                                        Emit emit) {
  const float f = __uint_as_float(field << 23);
  const F2 f2 = pack2(f, f);
  const F2 magic = pack2(12582912.0f, 12582912.0f);  // 1.5 2^23
  const F2 minus = pack2(-12582912.0f, -12582912.0f);
  const F2 neg = pack2(-1.0f, -1.0f), eight = pack2(8.0f, 8.0f);
  const uint32_t h[4] = {w.x, w.y, w.z, w.w};
  F2 q[4], v[4];
#pragma unroll
  for (int e = 0; e < 4; ++e)
    v[e] = mul2(pack2(__uint_as_float(h[e] << 16),
                      __uint_as_float(h[e] & 0xFFFF0000u)),
                f2);
#pragma unroll
  for (int d = 0; d < 8; ++d) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      q[e] = add2(add2(v[e], magic), minus);  // nearest integer
      v[e] = mul2(fma2(q[e], neg, v[e]), eight);
    }
    emit(d, codes8(q));
  }
}

// The sum behind a row's 8 accumulators (fp32 bits), times g; the smallest
// digits are added first.
template <int FMT>
__device__ __forceinline__ float digit_sum(const uint32_t *d, int X,
                                           const TensorScale &g) {
  float t = __uint_as_float(d[7]);
#pragma unroll
  for (int i = 6; i >= 0; --i)
    t = FMT == TQ_FMT_MX4 ? t + __uint_as_float(d[i])
                          : fmaf(t, 0.125f, __uint_as_float(d[i]));
  if (FMT == TQ_FMT_MX4)
    return t * g.m * __uint_as_float((uint32_t)mx4_reference(X) << 23);
  return times_pow2(t * g.m, X - 127 - 9 + g.e);
}

// One weight, for the rows of x that hold NaN or Inf.
template <int FMT>
__device__ float one_weight(const uint8_t *codes, const uint8_t *scales,
                            int64_t row, int64_t k_cols, int k) {
  const uint32_t b = codes[row * (k_cols / 2) + k / 2] >> (4 * (k & 1));
  const uint32_t m = b & 7u;
  const float mag =
      m < 2 ? 0.5f * m
            : __uint_as_float(((m >> 1) + 126u) << 23 | (m & 1u) << 22);
  const float s = f4_scale<FMT>(
      scales[row * (k_cols / f4_block(FMT)) + k / f4_block(FMT)]);
  return (b & 8u ? -mag : mag) * s;
}

// The products of a weight row with the NaN and Inf of a row of x between k0
// and k1.
template <int FMT>
__device__ __noinline__ float odd_products(const __nv_bfloat16 *x, int k0,
                                           int k1, const uint8_t *codes,
                                           const uint8_t *scales, int64_t row,
                                           int64_t k_cols) {
  float t = 0.0f;
  for (int k = k0; k < k1; ++k) {
    const float v = __bfloat162float(x[k]);
    if (!(fabsf(v) < __int_as_float(0x7F800000)))
      t += v * one_weight<FMT>(codes, scales, row, k_cols, k);
  }
  return t;
}

// Rows of a packed operand that are digits: every 8 of them belong to one row
// of x. exps null: they are not.
struct DigitArgs {
  const int *exps;  // exponent of each row of x
  const int *odd;   // whether it holds NaN or Inf
  const __nv_bfloat16 *x;
  int64_t ldx;
};

}  // namespace f4
}  // namespace tq
