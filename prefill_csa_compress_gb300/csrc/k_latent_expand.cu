// Keys and values of every head from a paged latent cache (csa_latent_expand).
#include "cache_common.cuh"

namespace csa {
namespace {

constexpr int LE_POS = 16;

// One CTA: 16 positions of one page, one head; a thread an output channel.
__global__ void __launch_bounds__(256) latent_expand_kernel(csa_latent_expand_args a) {
  __shared__ float c[LE_POS][kLatent];
  const int h = blockIdx.x, piece = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
  const int j0 = piece * LE_POS;
  const int lo = max(a.first ? a.first[b] : 0, j0);
  const int hi = (int)min((long long)min(a.kv_len[b], j0 + LE_POS), (long long)a.max_blocks * kBlock);
  if (lo >= hi) return;
  const long long src = page_row(a.block_table, a.max_blocks, a.n_blocks, b, j0, a.status_dev);
  const long long dst = page_row(a.out_table, a.out_max_blocks, a.n_out_blocks, b, j0, a.status_dev);
  if (src < 0 || dst < 0) return;
  const uint8_t *cp = static_cast<const uint8_t *>(a.c_pool) +
                      pool_offset(src, a.c_page_stride, a.c_token_stride);
  for (int i = tid; i < (hi - j0) * kLatent; i += 256)
    c[i / kLatent][i % kLatent] = __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(
        cp + (i / kLatent) * a.c_token_stride)[i % kLatent]);
  __syncthreads();
  const bool key = tid < kNope;
  const __nv_bfloat16 *w =
      reinterpret_cast<const __nv_bfloat16 *>(
          static_cast<const uint8_t *>(key ? a.w_uk : a.w_uv) +
          h * (key ? a.w_uk_head_stride : a.w_uv_head_stride)) +
      (tid & 127) * kLatent;
  float s[LE_POS] = {};
  for (int k = 0; k < kLatent; ++k) {
    const float x = __bfloat162float(w[k]);
#pragma unroll
    for (int i = 0; i < LE_POS; ++i) s[i] += x * c[i][k];
  }
  uint8_t *kp = static_cast<uint8_t *>(a.k_pool) + pool_offset(dst, a.k_page_stride, a.k_token_stride) +
                h * a.k_head_stride;
  uint8_t *vp = static_cast<uint8_t *>(a.v_pool) + pool_offset(dst, a.v_page_stride, a.v_token_stride) +
                h * a.v_head_stride;
  const uint8_t *rp = static_cast<const uint8_t *>(a.r_pool) +
                      pool_offset(src, a.r_page_stride, a.r_token_stride);
#pragma unroll
  for (int i = 0; i < LE_POS; ++i) {
    if (j0 + i < lo || j0 + i >= hi) continue;
    uint8_t *to = key ? kp + i * a.k_token_stride : vp + i * a.v_token_stride;
    reinterpret_cast<__nv_bfloat16 *>(to)[tid & 127] = __float2bfloat16_rn(s[i]);
    if (tid < kRopeDim)
      reinterpret_cast<__nv_bfloat16 *>(kp + i * a.k_token_stride)[kNope + tid] =
          reinterpret_cast<const __nv_bfloat16 *>(rp + i * a.r_token_stride)[tid];
  }
}

}  // namespace

cudaError_t launch_latent_expand(const csa_latent_expand_args &a, cudaStream_t s) {
  launch_begin(CSA_K_LATENT_EXPAND, s);
  latent_expand_kernel<<<dim3(a.n_heads, a.max_blocks * (kBlock / LE_POS), a.n_req), 256, 0, s>>>(a);
  launch_end(CSA_K_LATENT_EXPAND, s);
  return cudaGetLastError();
}

}  // namespace csa
