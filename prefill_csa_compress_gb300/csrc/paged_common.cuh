// Pieces shared by the kernels of csa_paged_attn.
#pragma once

#include <cuda.h>

#include "csa_internal.cuh"
#include "tc.cuh"

namespace csa {
namespace paged {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// Positions [lo, hi) that a row at position p sees in a cache of kv_len; neither is
// negative, so that a page's first position can be taken off both.
template <typename Args>  // (of the calls that read a paged cache)
__device__ __forceinline__ void visible_range(const Args &a, int kv_len, int p,
                                              int &lo, int &hi) {
  const int len = min(kv_len, a.max_blocks < 0x7FFFFFFF / kBlock ? a.max_blocks * kBlock : 0x7FFFFFFF);
  hi = max(a.causal && p < len ? p + 1 : len, 0);
  lo = a.window > 0 && p >= a.window ? p - a.window + 1 : 0;
}

// The parts of split rows, merged by paged_merge_kernel: part s of row t and
// head h holds o = sum_j 2^(x_j - m) v_j (FP32 [head_dim]), and m, l = sum_j
// 2^(x_j - m) in ml; m = -inf: nothing was seen there (o is not written).
struct Parts {
  float *o;
  float2 *ml;
  int n;  // parts per row
};

// The parts that the decode kernel's CTAs leave: CTA c's continuation of an
// item begun before it in slot 2 c, an item that it begins and does not end in
// slot 2 c + 1; a slot holds o and ml of the item's pairs.  item[row][sub]: the
// first and last CTA of the row's item and the item's first row; the first CTA
// is -1 where the row sees nothing.
constexpr int kDecodeRows = 512;  // rows of a call that the decode kernel takes, at most
struct DecodeParts {
  float *o;
  float2 *ml;
  int4 *item;
};

// Bit 15 or 31 of the result: that half of the BF16 pair is not finite.
__device__ __forceinline__ uint32_t not_finite2(uint32_t w) {
  return ((w & 0x7F807F80u) + 0x00800080u) & 0x80008000u;
}

__device__ __forceinline__ void tma_load_4d(void *dst, const void *tmap, int x, int y, int z, int w,
                                            uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(tc::smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(w),
      "r"(tc::smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ void prefetch_map(const void *tmap) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(tmap)) : "memory");
}

// Host: tensor maps of the pools [pages, 128, heads, head_dim], one page of one
// head and 64 channels a box, 128-byte swizzle; and of q, a group's heads of
// `rows` rows a box.
bool encode_pools(const csa_paged_attn_args &a, CUtensorMap *k, CUtensorMap *v);
bool encode_q(const csa_paged_attn_args &a, int rows, CUtensorMap *q);

// out and lse from m (log2 units) and l, with the sink in both.
struct Joined {
  float inv, lse;
};
__device__ __forceinline__ Joined finish(float m, float l, float sink) {
  // m = -inf: nothing was seen (l = 0; NaN if a logit was); sink = -inf: none
  if (m == -INFINITY) return {l, l == 0.f ? sink : l};
  const float s2 = sink * kLog2e, mm = fmaxf(m, s2);
  const float f = exp2f(m - mm), L = l * f + (s2 == mm ? 1.f : exp2f(s2 - mm));
  return {f / L, (mm + log2f(L)) * kLn2};
}

}  // namespace paged

// Attention of chunks: tcgen05 tiles of 128 (row, head) pairs (k_paged_chunk.cu).
int paged_chunk_parts(const csa_paged_attn_args &a, int sms);
cudaError_t launch_paged_chunk(const csa_paged_attn_args &a, const paged::Parts &parts, int sms,
                               cudaStream_t s);

// Few rows per request: a stream of pages (k_paged_decode.cu).
int paged_decode_items(const csa_paged_attn_args &a, int rows);  // per request and kv head
size_t paged_decode_workspace(const csa_paged_attn_args &a, int sms);
cudaError_t launch_paged_decode(const csa_paged_attn_args &a, int sms, cudaStream_t s);

}  // namespace csa
