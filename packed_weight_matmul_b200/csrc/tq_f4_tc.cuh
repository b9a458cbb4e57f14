// Shared by the kernels that feed 4-bit codes to the block-scaled tensor cores
// (tq_f4_gemm.cu, tq_f4_decode.cu): MMA issue, tensor-memory stores, scale
// pieces, tensor maps of packed codes.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include <mutex>

#include "tq_f4.cuh"
#include "tq_sm100_async.cuh"
#include "tq_sm100_mma.cuh"

namespace tq {
namespace f4 {

// Code bytes of a row per stage (256 k).
constexpr uint32_t kF4StageRow = 128;

__device__ __forceinline__ void tmem_st4(uint32_t taddr, uint32_t a, uint32_t b,
                                         uint32_t c, uint32_t d) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};" ::
                   "r"(taddr),
               "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}

// Whether the phase of parity `parity` is over, without waiting; for a pair
// with acquire at cluster scope.
template <int CG>
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  if constexpr (CG == 1)
    asm volatile(
        "{\n .reg .pred p;\n"
        " mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
        " selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
  else
    asm volatile(
        "{\n .reg .pred p;\n"
        " mbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], "
        "%2;\n selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
  return ok != 0;
}

#define TQ_COMMIT_1                                                          \
  "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64"
#define TQ_COMMIT_2                                                          \
  "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster."       \
  "multicast::cluster.b64"

// Arrive on `bar` (of both CTAs of a pair) when all MMAs issued so far are
// complete. Whole warp; the elected lane is the one that issues the MMAs.
template <int CG>
__device__ __forceinline__ void commit(uint32_t bar) {
  if constexpr (CG == 1)
    asm volatile("{\n .reg .pred q;\n elect.sync _|q, 0xFFFFFFFF;\n"
                 " @q " TQ_COMMIT_1 " [%0];\n}" ::"r"(bar)
                 : "memory");
  else
    asm volatile("{\n .reg .pred q;\n elect.sync _|q, 0xFFFFFFFF;\n"
                 " @q " TQ_COMMIT_2 " [%0], %1;\n}" ::"r"(bar),
                 "h"((uint16_t)3)
                 : "memory");
}

// One stage: D (+)= (A * scale A)(B * scale B)^T over 4 x 64 k, then arrive
// on `bar` as commit does. id0 / id1 are the instruction descriptors of even
// and odd MMAs, whose scale words start at sa + 4 w and sb + bcols w, w = j
// (NV4) or j / 2 (MX4). The whole warp comes here together and one elected
// lane issues: that way the operands stay in uniform registers (issued from
// inside an `if (lane == 0)`, an MMA cost about 80 cycles of moving them
// there, more than the tensor core needed for it).
template <int FMT, int CG>
__device__ __forceinline__ void mma_stage(uint32_t d, uint64_t a, uint64_t b,
                                          uint32_t id0, uint32_t id1,
                                          uint32_t sa, uint32_t sb,
                                          uint32_t bcols, uint32_t accumulate,
                                          uint32_t bar) {
  constexpr uint32_t kW = FMT == TQ_FMT_NV4 ? 1u : 0u;
  const uint32_t sa1 = sa + 4 * kW, sb1 = sb + bcols * kW;
  const uint32_t sa2 = sa + 4 * (1 + kW), sb2 = sb + bcols * (1 + kW);
  const uint32_t sa3 = sa2 + 4 * kW, sb3 = sb2 + bcols * kW;
#define TQ_MMA(KIND, DA, DB, ID, SA, SB, P)                                   \
  " @q tcgen05.mma.cta_group::" KIND " [%0], " DA ", " DB ", " ID ", [" SA     \
  "], [" SB "], " P ";\n"
#define TQ_STAGE(KIND, COMMIT)                                                \
  asm volatile(                                                               \
      "{\n .reg .pred p, q, t;\n .reg .b64 a1, a2, a3, b1, b2, b3;\n"         \
      " elect.sync _|q, 0xFFFFFFFF;\n setp.ne.b32 p, %13, 0;\n"               \
      " setp.eq.b32 t, 0, 0;\n"                                               \
      " add.s64 a1, %1, 2;\n add.s64 a2, %1, 4;\n add.s64 a3, %1, 6;\n"       \
      " add.s64 b1, %2, 2;\n add.s64 b2, %2, 4;\n add.s64 b3, %2, 6;\n"       \
      TQ_MMA(KIND, "%1", "%2", "%3", "%5", "%9", "p")                         \
      TQ_MMA(KIND, "a1", "b1", "%4", "%6", "%10", "t")                        \
      TQ_MMA(KIND, "a2", "b2", "%3", "%7", "%11", "t")                        \
      TQ_MMA(KIND, "a3", "b3", "%4", "%8", "%12", "t")                        \
      " @q " COMMIT ";\n}" ::"r"(d),                                          \
      "l"(a), "l"(b), "r"(id0), "r"(id1), "r"(sa), "r"(sa1), "r"(sa2),        \
      "r"(sa3), "r"(sb), "r"(sb1), "r"(sb2), "r"(sb3), "r"(accumulate),       \
      "r"(bar), "h"((uint16_t)3)                                              \
      : "memory")
  if constexpr (FMT == TQ_FMT_MX4 && CG == 1)
    TQ_STAGE("1.kind::mxf4.block_scale.scale_vec::2X", TQ_COMMIT_1 " [%14]");
  else if constexpr (FMT == TQ_FMT_MX4)
    TQ_STAGE("2.kind::mxf4.block_scale.scale_vec::2X",
             TQ_COMMIT_2 " [%14], %15");
  else if constexpr (CG == 1)
    TQ_STAGE("1.kind::mxf4nvf4.block_scale.scale_vec::4X",
             TQ_COMMIT_1 " [%14]");
  else
    TQ_STAGE("2.kind::mxf4nvf4.block_scale.scale_vec::4X",
             TQ_COMMIT_2 " [%14], %15");
#undef TQ_STAGE
#undef TQ_MMA
}

// Descriptor of 32 rows x 16 bytes that lie one after another.
__device__ __forceinline__ uint64_t smem_desc_rows16(uint32_t addr) {
  return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)(128u >> 4) << 16) |
         ((uint64_t)(128u >> 4) << 32) | (1ull << 46);
}

// WORDS times 512 bytes of shared memory (of each CTA of a pair), described by
// `src` and following one another, to tensor-memory columns t, t + step, ...:
// 16 bytes of lane r to 4 columns of lanes r, r + 32, r + 64, r + 96. Ordered
// before the MMAs that the elected lane issues later. Whole warp.
template <int CG, int WORDS>
__device__ __forceinline__ void copy_scales(uint32_t t, uint32_t step,
                                            uint64_t src) {
#define TQ_CP(GROUP)                                                          \
  asm volatile(                                                               \
      "{\n .reg .pred q;\n .reg .b64 s1;\n elect.sync _|q, 0xFFFFFFFF;\n"     \
      " add.s64 s1, %2, 32;\n"                                                \
      " @q tcgen05.cp.cta_group::" GROUP ".32x128b.warpx4 [%0], %2;\n"        \
      " @q tcgen05.cp.cta_group::" GROUP ".32x128b.warpx4 [%1], s1;\n}" ::"r"(  \
          t + 2 * i * step),                                                  \
      "r"(t + (2 * i + 1) * step), "l"(src + 64 * i)                          \
      : "memory")
#pragma unroll
  for (uint32_t i = 0; i < WORDS / 2; ++i) {
    if constexpr (CG == 1)
      TQ_CP("1");
    else
      TQ_CP("2");
  }
#undef TQ_CP
}

// Instruction descriptor of the 4-bit kinds: scale byte of B at bits 4-5 and
// of A at 29-30 (first of the word's bytes that this MMA uses), E2M1 = 1 at
// 7-9 and 10-12, N >> 3 at 17-22, E8M0 scales at 23, M >> 4 at 24-28.
template <int FMT>
__host__ __device__ constexpr uint32_t idesc_f4(int M, int N, uint32_t byte) {
  return (byte << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) |
         ((FMT == TQ_FMT_MX4 ? 1u : 0u) << 23) | ((uint32_t)(M >> 4) << 24) |
         (byte << 29);
}

__device__ __forceinline__ void bar_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// One piece (8 or 16 scale bytes) of a row at `off`, `left` bytes before the
// row's end; bytes past it are 0 (their codes are zero too).
template <int WORDS>
__device__ __forceinline__ void load_piece(uint32_t (&v)[WORDS],
                                           const uint8_t *p, int left) {
#pragma unroll
  for (int w = 0; w < WORDS; ++w) v[w] = 0;
  if (left <= 0) return;
  if constexpr (WORDS == 2) {
    const uint2 u = __ldg(reinterpret_cast<const uint2 *>(p));
    v[0] = u.x;
    v[1] = u.y;
  } else {
    const uint4 u = __ldg(reinterpret_cast<const uint4 *>(p));
    v[0] = u.x;
    v[1] = u.y;
    v[2] = u.z;
    v[3] = u.w;
  }
}

// The same for any p, by the aligned words that hold the bytes; a word without
// any of them is not read.
template <int WORDS>
__device__ __forceinline__ void load_piece_shifted(uint32_t (&v)[WORDS],
                                                   const uint8_t *p, int left) {
  const int skip = (int)(reinterpret_cast<uintptr_t>(p) & 3u);
  const uint32_t *q = reinterpret_cast<const uint32_t *>(p - skip);
  uint32_t x[WORDS + 1];
#pragma unroll
  for (int w = 0; w <= WORDS; ++w) {
    x[w] = 0;
    if (4 * w < left + skip && (w < WORDS || skip != 0)) x[w] = __ldg(q + w);
  }
#pragma unroll
  for (int w = 0; w < WORDS; ++w) {
    const uint32_t u = __funnelshift_r(x[w], x[w + 1], 8 * skip);
    const int n = left - 4 * w;  // bytes of the row in this word
    v[w] = n >= 4 ? u : n <= 0 ? 0u : u & ((1u << (8 * n)) - 1u);
  }
}

// 32 scale bytes of a row: in pieces of WORDS words to whose size `p` is
// aligned, or of any alignment (WORDS = 0).
template <int WORDS>
__device__ __forceinline__ void load_unit(uint32_t (&v)[8], const uint8_t *p,
                                          int left) {
  if constexpr (WORDS == 0) {
    load_piece_shifted(v, p, left);
  } else {
#pragma unroll
    for (int c = 0; c < 8 / WORDS; ++c) {
      uint32_t d[WORDS];
      load_piece(d, p + 4 * WORDS * c, left - 4 * WORDS * c);
#pragma unroll
      for (int w = 0; w < WORDS; ++w) v[c * WORDS + w] = d[w];
    }
  }
}

template <int WORDS>
__device__ __forceinline__ void store_piece(uint32_t at,
                                            const uint32_t (&v)[WORDS]) {
  if constexpr (WORDS == 2)
    asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(at), "r"(v[0]),
                 "r"(v[1])
                 : "memory");
  else
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at),
                 "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3])
                 : "memory");
}

// Where piece c of row r's unit (PIECES of BYTES bytes) lies in a group's
// scale buffer: row after row, a row's pieces swapped so that the reads of
// one piece by consecutive rows hit different banks.
template <uint32_t PIECES, uint32_t BYTES>
__device__ __forceinline__ uint32_t scale_at(uint32_t r, uint32_t c) {
  constexpr uint32_t kRowsPer128 = 128u / (PIECES * BYTES);
  return (r * PIECES + (c ^ ((r / kRowsPer128) & (PIECES - 1)))) * BYTES;
}

// ---- host ------------------------------------------------------------------

inline PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault,
                                &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

// Packed codes [rows][k/2]; boxes of 128 bytes (256 k) x `box` rows, 128-byte
// swizzle. Rows and columns past the matrix read as zero codes.
inline cudaError_t code_map(CUtensorMap *map, const WeightsView &w, int box_rows) {
  auto encode = encode_fn();
  if (encode == nullptr) return cudaErrorNotSupported;
  const cuuint64_t dims[2] = {(cuuint64_t)(w.k / 2), (cuuint64_t)w.n};
  const cuuint64_t strides[1] = {(cuuint64_t)(w.k / 2)};
  const cuuint32_t box[2] = {kF4StageRow, (cuuint32_t)box_rows};
  const cuuint32_t estr[2] = {1u, 1u};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2,
                const_cast<uint8_t *>(w.codes), dims, strides, box, estr,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? cudaSuccess
             : cudaErrorInvalidValue;
}

}  // namespace f4
}  // namespace tq
