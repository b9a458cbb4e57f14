// Products with 4-bit weights, simplest form: one warp per output row and
// group of 8 batch rows; codes decoded in registers, fp32 sums, a butterfly
// over the lanes at the end.
#include "tq_f4.cuh"

namespace tq {
namespace {

constexpr int kWarps = 8, kBatch = 8;

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// 8 decoded, block-scaled weights of row `row` at column 8 u.
template <int FMT>
__device__ __forceinline__ void weights8(const uint8_t *codes,
                                         const uint8_t *scales, int64_t k,
                                         int64_t row, int64_t u, float (&w)[8]) {
  const uint32_t c =
      __ldg(reinterpret_cast<const uint32_t *>(codes + row * (k / 2)) + u);
  const float s = f4_scale<FMT>(
      __ldg(scales + row * (k / f4_block(FMT)) + u / (f4_block(FMT) / 8)));
  uint32_t h[4];
  f4x8_to_h2(c, h);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<__half2 *>(&h[i]));
    w[2 * i] = f.x * s;
    w[2 * i + 1] = f.y * s;
  }
}

template <int FMT>
__global__ void __launch_bounds__(kWarps * 32)
    linear_kernel(const uint8_t *__restrict__ codes,
                  const uint8_t *__restrict__ scales, const float *ts,
                  int64_t n, int64_t k, const int32_t *__restrict__ ids,
                  int n_experts, const __nv_bfloat16 *__restrict__ x,
                  int64_t batch, int64_t ldx, float *__restrict__ y,
                  int64_t ldy, int32_t *status) {
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int64_t per = ids != nullptr ? 1 : kBatch;
  if (row >= n) return;
  for (int64_t b0 = blockIdx.y * per; b0 < batch; b0 += gridDim.y * per) {
    const int nb = (int)(batch - b0 < per ? batch - b0 : per);
    int64_t e = 0;
    if (ids != nullptr) {
      e = ids[b0];
      if (e < 0 || e >= n_experts) {
        if (lane == 0) {
          y[b0 * ldy + row] = __int_as_float(0x7FC00000);
          report(status, TQ_ERR_INVALID_ARG);
        }
        continue;
      }
    }
    float acc[kBatch] = {};
    for (int64_t u = lane; u < k / 8; u += 32) {
      float w[8];
      weights8<FMT>(codes, scales, k, e * n + row, u, w);
      for (int b = 0; b < nb; ++b) {
        const uint4 v =
            __ldg(reinterpret_cast<const uint4 *>(x + (b0 + b) * ldx) + u);
        const uint32_t q[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          acc[b] = fmaf(w[2 * i], __uint_as_float(q[i] << 16), acc[b]);
          acc[b] = fmaf(w[2 * i + 1], __uint_as_float(q[i] & 0xFFFF0000u),
                        acc[b]);
        }
      }
    }
    const float g = ts != nullptr ? ts[e] : 1.0f;
    for (int b = 0; b < nb; ++b) {
      const float v = warp_sum(acc[b]);
      if (lane == 0) y[(b0 + b) * ldy + row] = v * g;
    }
  }
}

dim3 grid_of(int64_t n, int64_t batch, int64_t per) {
  const int64_t gy = (batch + per - 1) / per;
  return dim3((unsigned)((n + kWarps - 1) / kWarps),
              (unsigned)(gy < 65535 ? gy : 65535));
}

}  // namespace

cudaError_t linear_f4_bf16(const WeightsView &w, const __nv_bfloat16 *x,
                           int64_t batch, int64_t ldx, float *y, int64_t ldy,
                           cudaStream_t stream) {
  auto kern = w.format == TQ_FMT_MX4 ? linear_kernel<TQ_FMT_MX4>
                                     : linear_kernel<TQ_FMT_NV4>;
  kern<<<grid_of(w.n, batch, kBatch), kWarps * 32, 0, stream>>>(
      w.codes, reinterpret_cast<const uint8_t *>(w.scales), w.lut, w.n, w.k,
      nullptr, 1, x, batch, ldx, y, ldy, nullptr);
  return cudaGetLastError();
}

cudaError_t launch_linear_experts_f4(const WeightsView &w, int n_experts,
                                     const int32_t *ids, int64_t tokens,
                                     const __nv_bfloat16 *x, int64_t ldx,
                                     float *y, int64_t ldy, int32_t *status,
                                     cudaStream_t stream) {
  auto kern = w.format == TQ_FMT_MX4 ? linear_kernel<TQ_FMT_MX4>
                                     : linear_kernel<TQ_FMT_NV4>;
  kern<<<grid_of(w.n, tokens, 1), kWarps * 32, 0, stream>>>(
      w.codes, reinterpret_cast<const uint8_t *>(w.scales), w.lut, w.n, w.k,
      ids, n_experts, x, tokens, ldx, y, ldy, status);
  return cudaGetLastError();
}

}  // namespace tq
