// 4-bit floats with a scale per block (TQ_FMT_MX4, TQ_FMT_NV4): device
// helpers and launchers. E2M1 codes are decoded by the conversion
// instructions of sm_100a (two codes per byte -> two fp16, exact).
#pragma once

#include <cuda_fp16.h>

#include "tq_common.cuh"

namespace tq {

__host__ __device__ constexpr bool is_f4(int format) {
  return format == TQ_FMT_MX4 || format == TQ_FMT_NV4;
}
__host__ __device__ constexpr int f4_block(int format) {
  return format == TQ_FMT_MX4 ? 32 : 16;
}

// The 8 codes of a word as fp16 pairs: h[i] holds the codes of byte i, the
// low four bits in the low half.
__device__ __forceinline__ void f4x8_to_h2(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n .reg .b8 b0, b1, b2, b3;\n mov.b32 {b0, b1, b2, b3}, %4;\n"
      " cvt.rn.f16x2.e2m1x2 %0, b0;\n cvt.rn.f16x2.e2m1x2 %1, b1;\n"
      " cvt.rn.f16x2.e2m1x2 %2, b2;\n cvt.rn.f16x2.e2m1x2 %3, b3;\n}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

// E8M0 byte -> fp32: 2^(b - 127), 255 is NaN (b = 0 is the subnormal 2^-127).
__device__ __forceinline__ float e8m0_to_f32(uint32_t b) {
  return b == 255u ? __int_as_float(0x7FC00000)
                   : __uint_as_float(b == 0u ? 0x00400000u : b << 23);
}

// E4M3 byte without its sign bit -> fp32 (0x7F is NaN).
__device__ __forceinline__ float e4m3_to_f32(uint32_t b) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)(b & 0x7Fu)));
  return __half2float(__ushort_as_half((unsigned short)h));
}

template <int FMT>
__device__ __forceinline__ float f4_scale(uint32_t b) {
  return FMT == TQ_FMT_MX4 ? e8m0_to_f32(b) : e4m3_to_f32(b);
}

// Largest magnitude (bf16 bits) of the 8 values of a 16-byte word.
__device__ __forceinline__ uint32_t max_mag8(const uint4 &w) {
  const uint32_t m = __vmaxu2(__vmaxu2(w.x & 0x7FFF7FFFu, w.y & 0x7FFF7FFFu),
                              __vmaxu2(w.z & 0x7FFF7FFFu, w.w & 0x7FFF7FFFu));
  return max(m >> 16, m & 0xFFFFu);
}

// The same over the finite values, one by one.
static __device__ __noinline__ uint32_t max_finite8(uint4 w) {
  const uint32_t v[4] = {w.x, w.y, w.z, w.w};
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t a = (v[i >> 1] >> (16 * (i & 1))) & 0x7FFFu;
    if (a < 0x7F80u) m = max(m, a);
  }
  return m;
}

// A tensor scale g = m 2^e with |m| < 1 (0, NaN and Inf as they are): sums may
// lie outside of fp32's range where g brings them back, so m is applied first
// and e together with the other exponents.
struct TensorScale {
  float m;
  int e;
};

__device__ __forceinline__ TensorScale tensor_scale(float g) {
  TensorScale s = {g, 0};
  if (fabsf(g) < __int_as_float(0x7F800000)) s.m = frexpf(g, &s.e);
  return s;
}

// v 2^e in two steps, for |e| up to 284: below 2^-252 the power is that, which
// leaves 0 of a sum all the same.
__device__ __forceinline__ float times_pow2(float v, int e) {
  const int half = max(e >> 1, -126), rest = max(e - half, -126);
  return v * __int_as_float((half + 127) << 23) *
         __int_as_float((rest + 127) << 23);
}

// v g_w g_x = v b a. b is 1 unless g_w g_x lies outside of fp32's range; then
// each factor has half of its exponent (more than 2^127 changes no result).
struct Factors {
  float a, b;
};

__device__ __forceinline__ Factors scale_factors(float gw, float gx) {
  const TensorScale w = tensor_scale(gw), x = tensor_scale(gx);
  const int e = w.e + x.e;
  if (e >= -124 && e <= 128) return {scalbnf(w.m * x.m, e), 1.0f};
  return {scalbnf(w.m * x.m, e - e / 2), scalbnf(1.0f, min(e / 2, 127))};
}

// All threads of a cluster meet. Relaxed: it orders no memory (the ordinary
// barrier waits until this CTA's global stores are acknowledged, about 1 us),
// which is enough where CTAs only tell one another that they have finished
// reading, and every value read has gone into an instruction issued before.
__device__ __forceinline__ void cluster_sync_relaxed() {
  asm volatile("barrier.cluster.arrive.relaxed;\n"
               "barrier.cluster.wait;" ::: "memory");
}

cudaError_t launch_quantize_f4(const uint16_t *W, int64_t n, int64_t k,
                               int64_t ldw, int format, uint8_t *codes,
                               uint8_t *scales, float *tensor_scale,
                               bool given, int32_t *status,
                               cudaStream_t stream);
cudaError_t launch_unpack_f4(const WeightsView &w, uint16_t *out,
                             int32_t *status, cudaStream_t stream);
// y = x W^T, bf16 x (tq_linear with a 4-bit descriptor).
cudaError_t linear_f4_bf16(const WeightsView &w, const __nv_bfloat16 *x,
                           int64_t batch, int64_t ldx, float *y, int64_t ldy,
                           cudaStream_t stream);
cudaError_t launch_linear_experts_f4(const WeightsView &w, int n_experts,
                                     const int32_t *ids, int64_t tokens,
                                     const __nv_bfloat16 *x, int64_t ldx,
                                     float *y, int64_t ldy, int32_t *status,
                                     cudaStream_t stream);
// y = x W^T, both in 4 bits.
cudaError_t launch_linear_f4(const WeightsView &w, const WeightsView &x,
                             void *y, int64_t ldy, int y_type,
                             cudaStream_t stream);

// Few rows of x on the block-scaled tensor cores (tq_f4_decode.cu): bf16 rows,
// rows that pick an expert, packed rows. `copies` matrices of w.n rows lie
// behind one another.
bool decode_f4_supported(const WeightsView &w, int64_t copies);
cudaError_t decode_f4_bf16(const WeightsView &w, const __nv_bfloat16 *x,
                           int64_t batch, int64_t ldx, float *y, int64_t ldy,
                           cudaStream_t stream);
cudaError_t decode_f4_experts(const WeightsView &w, int n_experts,
                              const int32_t *ids, int64_t tokens,
                              const __nv_bfloat16 *x, int64_t ldx, float *y,
                              int64_t ldy, int32_t *status,
                              cudaStream_t stream);
namespace f4 {
struct DigitArgs;
}
cudaError_t decode_f4_packed(const WeightsView &w, const WeightsView &x,
                             void *y, int64_t ldy, int y_type,
                             const f4::DigitArgs &digits, cudaStream_t stream);

// tq_linear with a workspace (tq_f4_digits.cu): bytes (0: of no use), call.
int64_t digits_f4_workspace(const WeightsView &w, int64_t batch);
cudaError_t digits_f4(const WeightsView &w, const __nv_bfloat16 *x,
                      int64_t batch, int64_t ldx, float *y, int64_t ldy,
                      uint8_t *workspace, cudaStream_t stream);
// Rows of x per pass of the row kernel, for `copies` products with up to `rows`
// rows each: all of them, but fewer where the CTAs of the passes find room next
// to one another, K split as far as it goes. A pass of 8 rows takes about half
// the time of one of 32 and a quarter of one of 64. Without and with that (us):
// 1003 x 4128 at 32 rows 12.0 and 9.4; 2048 x 8192 at 32 rows 17.3 and 12.6;
// 2048 x 2048 at 32 rows 9.1 and 6.7; 198 rows over 4 experts of 111 x 576 22
// and 8. Fewer rows at the price of the split of K did not pay (4096 x 4096, 20
// rows: 11.9, with 16 instead of 32 rows per pass 16.0).
int rows_per_pass_f4(const WeightsView &w, int64_t copies, int64_t rows);

// Clusters of `ks` CTAs that are resident together; 0: not known.
inline int max_clusters(const void *kern, int ks, int threads, size_t smem) {
  // An error already pending belongs to the caller: leave it.
  if (cudaPeekAtLastError() != cudaSuccess) return 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ks);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)ks;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) {
    cudaGetLastError();  // the query's own error
    return 0;
  }
  return n;
}

// The product with packed rows of x, which may be digits (tq_f4_gemm.cu).
cudaError_t product_f4(const WeightsView &w, const WeightsView &x, void *y,
                       int64_t ldy, int y_type, const f4::DigitArgs &digits,
                       cudaStream_t stream);

}  // namespace tq
