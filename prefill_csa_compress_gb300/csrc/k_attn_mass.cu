// The attention weight that every cached position received (csa_attn_mass).
#include "cache_common.cuh"
#include "paged_common.cuh"

namespace csa {
namespace {

// One CTA a page of a request, a thread a position.
template <int D>
__global__ void __launch_bounds__(128) attn_mass_kernel(csa_attn_mass_args a) {
  const int b = blockIdx.y, j = blockIdx.x * kBlock + threadIdx.x;
  if (blockIdx.x == 0 && b == 0)
    for (int t = threadIdx.x; t < a.n_rows; t += 128)
      if (a.row_req[t] >= a.n_req) flag(a.status_dev, CSA_DEV_BAD_POS);
  if (j >= a.kv_len[b]) return;
  const int page = a.block_table[(long long)b * a.max_blocks + blockIdx.x];
  const bool there = page >= 0 && page < a.n_blocks;
  bool read = false;
  float sum = 0.f;
  const float sl2 = a.softmax_scale * paged::kLog2e;
  const int g = a.n_heads / a.n_kv_heads;
  for (int kh = 0; kh < a.n_kv_heads; ++kh) {
    float k[D];
    if (there) {
      const __nv_bfloat16 *kp = reinterpret_cast<const __nv_bfloat16 *>(
          static_cast<const uint8_t *>(a.k_pool) + page * a.k_page_stride +
          threadIdx.x * a.k_token_stride + kh * a.k_head_stride);
#pragma unroll
      for (int i = 0; i < D; ++i) k[i] = __bfloat162float(kp[i]);
    }
    for (int t = 0; t < a.n_rows; ++t) {
      if (a.row_req[t] != b) continue;
      int lo, hi;
      paged::visible_range(a, a.kv_len[b], a.row_pos[t], lo, hi);
      if (j < lo || j >= hi) continue;
      read = true;
      if (!there) continue;
      for (int h = kh * g; h < kh * g + g; ++h) {
        const float lse = a.lse[(long long)t * a.n_heads + h];
        if (lse == -INFINITY) continue;
        const __nv_bfloat16 *q = reinterpret_cast<const __nv_bfloat16 *>(
                                     static_cast<const uint8_t *>(a.q) + t * a.q_row_stride) +
                                 h * D;
        float x = 0.f;
#pragma unroll
        for (int i = 0; i < D; ++i) x += k[i] * __bfloat162float(q[i]);
        sum += exp2f(x * sl2 - lse * paged::kLog2e);
      }
    }
  }
  if (read && !there) flag(a.status_dev, CSA_DEV_BAD_BLOCK);
  float *out = reinterpret_cast<float *>(reinterpret_cast<uint8_t *>(a.mass_out) +
                                         b * a.mass_out_row_stride) + j;
  if (a.decay != 0.f)
    sum += a.decay * reinterpret_cast<const float *>(reinterpret_cast<const uint8_t *>(a.mass) +
                                                     b * a.mass_row_stride)[j];
  *out = sum;
}

}  // namespace

size_t attn_mass_workspace(const csa_attn_mass_args &) { return 0; }

cudaError_t launch_attn_mass(const csa_attn_mass_args &a, cudaStream_t s) {
  launch_begin(CSA_K_ATTN_MASS, s);
  const dim3 grid(a.max_blocks, a.n_req);
  if (a.head_dim == 64)
    attn_mass_kernel<64><<<grid, 128, 0, s>>>(a);
  else
    attn_mass_kernel<128><<<grid, 128, 0, s>>>(a);
  launch_end(CSA_K_ATTN_MASS, s);
  return cudaGetLastError();
}

}  // namespace csa
