// bf16 rows of x written as 4-bit rows (tq_f4_digits.cuh) into a workspace, and
// the product of weights with them (tq_linear_ws): for batches where the digits
// are better made once than by every CTA that needs them.
//
// Workspace, for up to kDigitRows rows of x at a time: codes [8 rows][k/2],
// scales [8 rows][k/block], the rows' exponents and their flags for NaN / Inf.
// One block per row and 2048 columns; each finds the row's largest magnitude
// itself (the row is in the L2 cache) and turns 8 values per thread into 8
// words of codes. Bound by arithmetic, 59 lane instructions per value by the
// profiler: 64 x 5376 takes 6 us by itself, of the 40 us of a product with
// 21504 weight rows.
#include "tq_f4_digits.cuh"

namespace tq {
using namespace f4;
namespace {

constexpr int64_t kDigitRows = 512;

struct Layout {
  int64_t rows, codes, scales, exps, odd, total;  // offsets in bytes
};

Layout layout_of(int format, int64_t batch, int64_t k) {
  auto up = [](int64_t v) { return (v + 255) / 256 * 256; };
  Layout L;
  L.rows = batch < kDigitRows ? batch : kDigitRows;
  L.codes = 0;
  L.scales = up(8 * L.rows * (k / 2));
  L.exps = L.scales + up(8 * L.rows * (k / f4_block(format)));
  L.odd = L.exps + up(4 * L.rows);
  L.total = L.odd + up(4 * L.rows);
  return L;
}

template <int FMT>
__global__ void __launch_bounds__(256)
    digits_kernel(const __nv_bfloat16 *__restrict__ x, int64_t ldx, int k,
                  uint8_t *__restrict__ codes, uint8_t *__restrict__ scales,
                  int *__restrict__ exps, int *__restrict__ odds) {
  pdl_launch_dependents();
  pdl_wait();
  const int64_t row = blockIdx.y;
  const __nv_bfloat16 *p = x + row * ldx;
  uint32_t m = 0, odd = 0;
  // this block's values first, they are needed again
  const int at = blockIdx.x * 2048 + threadIdx.x * 8;
  uint4 w = make_uint4(0, 0, 0, 0);
  if (at < k) w = __ldg(reinterpret_cast<const uint4 *>(p + at));
  for (int i = threadIdx.x * 8; i < k; i += 4 * 2048) {
    uint4 v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[j] = make_uint4(0, 0, 0, 0);
      if (i + 2048 * j < k)
        v[j] = __ldg(reinterpret_cast<const uint4 *>(p + i + 2048 * j));
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
  __shared__ uint32_t s_m[8], s_odd[8];
  m = __reduce_max_sync(0xFFFFFFFFu, m);
  odd = __reduce_max_sync(0xFFFFFFFFu, odd);
  if ((threadIdx.x & 31) == 0) {
    s_m[threadIdx.x >> 5] = m;
    s_odd[threadIdx.x >> 5] = odd;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    m = max(m, s_m[i]);
    odd |= s_odd[i];
  }
  const int X = max((int)(m >> 7), 1);
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    exps[row] = X;
    odds[row] = (int)odd;
  }
  // k is a multiple of 32: the lanes of a block are in or out together
  if (odd) w = only_finite8(w);
  uint32_t b = max_mag8(w);
  b = max(b, __shfl_xor_sync(0xFFFFFFFFu, b, 1));
  if (FMT == TQ_FMT_MX4) b = max(b, __shfl_xor_sync(0xFFFFFFFFu, b, 2));
  if (at >= k) return;
  uint32_t byte, field;
  digit_scale<FMT>(max((int)(b >> 7), 1), X, &byte, &field);
  constexpr int kBlock = f4_block(FMT);
  if (at % kBlock == 0) {
    uint8_t *q = scales + 8 * row * (k / kBlock) + at / kBlock;
#pragma unroll
    for (int d = 0; d < 8; ++d)
      q[d * (int64_t)(k / kBlock)] =
          FMT == TQ_FMT_MX4 ? (uint8_t)max((int)byte - 3 * d, 0)
                            : (uint8_t)byte;
  }
  uint8_t *c = codes + 8 * row * (k / 2) + at / 2;
  digits8(w, field, [&](int d, uint32_t v) {
    *reinterpret_cast<uint32_t *>(c + d * (int64_t)(k / 2)) = v;
  });
}

}  // namespace

// 0 where the plain kernels do as well. Measured (us; plain, digits):
//   MX4  21504 x 5376 batch 4: 24, 18; 16: 43, 26; 64: 120, 40
//        5376 x 21504 batch 4: 28, 21.6; 16: 33, 33; 32: 48, 36
//        8192 x 5376 batch 4: 14.5, 12.2; 4096 x 4096 batch 8: 7.9, 9.7; 32:
//        12.6, 12.2; 48: 17.5, 12.6; 2048 x 8192 batch 16: 10.3, 16; 32: 12.6,
//        16
//   NV4  21504 x 5376 batch 4: 29, 21; 16: 42, 29; 64: 117, 42
//        8192 x 5376 batch 4: 12.7, 13.6; 16: 16.4, 16.1; 32: 24, 18
//        5376 x 21504 batch 4: 23, 25; 16: 32, 39; 24: 45, 39; 32: 48, 41
//        2048 x 21504 batch 16: 20, 37; 32: 25, 37
//        1000 x 4000 batch 64: 9.3, 15.5; 130: 18.2, 16.5
//        128 x 512 batch 64: 4.6, 7.3; 300: 4.8, 7.9
// The second launch costs 4 us, and long rows of x cost more digits for the
// same weights. The plain kernel slows down past 16 and again past 32 rows
// unless it has room for passes of 8 or 16 next to one another; the product
// of the digits, which does not split K, needs many weight rows to fill the
// GPU.
int64_t digits_f4_workspace(const WeightsView &w, int64_t batch) {
  const int64_t weights = w.n * w.k;
  const bool large = batch >= 3 && (w.format == TQ_FMT_MX4
                                        ? weights >= (1 << 25)
                                        : weights >= (1 << 26) && w.n >= w.k);
  const bool wide = batch > (w.n >= 4096 ? 16 : 32) &&
                    rows_per_pass_f4(w, 1, batch) > 16;
  if (!(large || wide) || !decode_f4_supported(w, 1)) return 0;
  return layout_of(w.format, batch, w.k).total;
}

cudaError_t digits_f4(const WeightsView &w, const __nv_bfloat16 *x,
                      int64_t batch, int64_t ldx, float *y, int64_t ldy,
                      uint8_t *workspace, cudaStream_t stream) {
  const Layout L = layout_of(w.format, batch, w.k);
  for (int64_t b = 0; b < batch; b += L.rows) {
    const int64_t rows = batch - b < L.rows ? batch - b : L.rows;
    // (the second dimension ends at 65535)
    const dim3 grid((unsigned)((w.k + 2047) / 2048), (unsigned)rows);
    int *exps = reinterpret_cast<int *>(workspace + L.exps);
    int *odd = reinterpret_cast<int *>(workspace + L.odd);
    auto kern = w.format == TQ_FMT_MX4 ? digits_kernel<TQ_FMT_MX4>
                                       : digits_kernel<TQ_FMT_NV4>;
    cudaError_t e = launch_pdl(kern, grid, dim3(256), 0, stream, x + b * ldx,
                               ldx, (int)w.k, workspace + L.codes,
                               workspace + L.scales, exps, odd);
    if (e != cudaSuccess) return e;
    WeightsView u = w;  // the digits, as a 4-bit matrix
    u.n = 8 * rows;
    u.codes = workspace + L.codes;
    u.scales = reinterpret_cast<const uint16_t *>(workspace + L.scales);
    u.lut = nullptr;
    DigitArgs digits = {exps, odd, x + b * ldx, ldx};
    if ((e = product_f4(w, u, y + b * ldy, ldy, TQ_Y_F32, digits, stream)) !=
        cudaSuccess)
      return e;
  }
  return cudaSuccess;
}

}  // namespace tq
