// Pieces shared by the kernels of csa_paged_attn.
#pragma once

#include "csa_internal.cuh"

namespace csa {
namespace paged {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// Positions [lo, hi) of request b that a row at position p sees.
__device__ __forceinline__ void visible_range(const csa_paged_attn_args &a, int b, int p, int &lo,
                                              int &hi) {
  const long long cap = (long long)a.max_blocks * kBlock;
  const int len = (int)min((long long)a.kv_len[b], min(cap, 0x7FFFFFFFll));
  hi = a.causal && p < len ? p + 1 : len;
  const long long from = a.window > 0 ? (long long)p - a.window + 1 : 0;
  lo = (int)max(0ll, min(from, 0x7FFFFFFFll));
}

// The parts of split rows, merged by paged_merge_kernel: part s of row t and
// head h holds o = sum_j 2^(x_j - m) v_j (FP32 [head_dim]), and m, l = sum_j
// 2^(x_j - m) in ml; m = -inf: nothing was seen there (o is not written).
struct Parts {
  float *o;
  float2 *ml;
  int n;  // parts per row
};

// out and lse from m (log2 units) and l, with the sink in both.
struct Joined {
  float inv, lse;
};
__device__ __forceinline__ Joined finish(float m, float l, float s2) {
  // m = -inf: nothing was seen; s2: the sink in log2 units, -inf for none
  const float mm = fmaxf(m, s2);
  if (mm == -INFINITY) return {0.f, l == 0.f ? -INFINITY : l};  // l is NaN if a logit was
  const float f = m == -INFINITY ? (l == 0.f ? 0.f : l) : exp2f(m - mm);
  const float L = l * f + exp2f(s2 - mm);
  return {f / L, (mm + log2f(L)) * kLn2};
}

}  // namespace paged

// Attention of chunks: tcgen05 tiles of 128 (row, head) pairs (k_paged_chunk.cu).
int paged_chunk_parts(const csa_paged_attn_args &a, int sms);
cudaError_t launch_paged_chunk(const csa_paged_attn_args &a, const paged::Parts &parts, int sms,
                               cudaStream_t s);

}  // namespace csa
