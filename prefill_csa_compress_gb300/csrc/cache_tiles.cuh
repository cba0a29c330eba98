// Pieces that the tcgen05 kernels of the latent cache and eviction calls share.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include <cstring>

#include "cache_common.cuh"
#include "paged_common.cuh"
#include "tc.cuh"

namespace csa {
namespace cache {

// Bounded wait that also gives up when another role of the CTA has.
__device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity, volatile int *abort,
                                     uint32_t *status) {
  if (tc::mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = tc::global_ns();
  for (uint32_t i = 1;; ++i) {
    if (tc::mbar_try_wait(bar, parity)) return true;
    if ((i & 255u) == 0) {
      if (*abort) return false;
      if (tc::global_ns() - t0 > 2000000000ull) {
        *abort = 1;
        flag(status, CSA_DEV_TIMEOUT);
        return false;
      }
    }
  }
}

// Four MMAs over 64 of K, the operands' descriptors AS and BS sixteen bytes further on
// each; acc = 0: the first overwrites.  One statement, for one elected lane: a loop of
// single ones takes 80 cycles each to issue, these the 32 or 48 that they run for.
#define CSA_MMA4(group)                                                                     \
  asm volatile(                                                                             \
      "{\n\t.reg .pred p, q;\n\t.reg .b64 x, y;\n\tsetp.ne.b32 p, %4, 0;\n\t"               \
      "setp.eq.b32 q, 0, 0;\n\t"                                                            \
      "tcgen05.mma.cta_group::" group ".kind::f16 [%0], %1, %2, %3, p;\n\t"                 \
      "add.u64 x, %1, %5;\n\tadd.u64 y, %2, %6;\n\t"                                        \
      "tcgen05.mma.cta_group::" group ".kind::f16 [%0], x, y, %3, q;\n\t"                   \
      "add.u64 x, %1, 2 * %5;\n\tadd.u64 y, %2, 2 * %6;\n\t"                                \
      "tcgen05.mma.cta_group::" group ".kind::f16 [%0], x, y, %3, q;\n\t"                   \
      "add.u64 x, %1, 3 * %5;\n\tadd.u64 y, %2, 3 * %6;\n\t"                                \
      "tcgen05.mma.cta_group::" group ".kind::f16 [%0], x, y, %3, q;\n\t}" ::"r"(d),        \
      "l"(a), "l"(b), "r"(idesc), "r"(acc), "n"(AS), "n"(BS)                                \
      : "memory")
template <int AS, int BS>
__device__ __forceinline__ void mma4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  CSA_MMA4("1");
}
// The same by a pair of CTAs, issued by its first.
template <int AS, int BS>
__device__ __forceinline__ void mma4_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                          uint32_t acc) {
  CSA_MMA4("2");
}
#undef CSA_MMA4

// Host: a BF16 tensor map of up to four dimensions, 128-byte swizzle; strides (bytes) of
// dimensions 1 ...
inline bool encode(CUtensorMap *map, const void *base, int rank, const cuuint64_t *dims,
                   const cuuint64_t *strides, const cuuint32_t *box, CUtensorMapL2promotion l2) {
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    cudaDriverEntryPointQueryResult q;
    void *f = nullptr;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                         &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  }();
  const cuuint32_t ones[4] = {1, 1, 1, 1};
  memset(map, 0, sizeof(*map));
  return fn && fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void *>(base), dims, strides,
                  box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, l2,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace cache
}  // namespace csa
