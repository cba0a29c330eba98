// Absorbed latent attention over a paged latent cache (csa_latent_attn).
#include "cache_common.cuh"
#include "paged_common.cuh"

namespace csa {
namespace {

// One CTA a (row, head): 256 positions at a time, a thread a logit, then two
// output channels a thread.
__global__ void __launch_bounds__(256) latent_attn_kernel(csa_latent_attn_args a) {
  __shared__ float q[kLatent + kRopeDim], p[256], red[8];
  __shared__ long long at[256];
  const int t = blockIdx.x / a.n_heads, h = blockIdx.x % a.n_heads, tid = threadIdx.x;
  const int b = a.row_req[t];
  if (b >= a.n_req && tid == 0) flag(a.status_dev, CSA_DEV_BAD_POS);
  if (b < 0 || b >= a.n_req) return;
  int lo, hi;
  paged::visible_range(a, a.kv_len[b], a.row_pos[t], lo, hi);
  const __nv_bfloat16 *qp = reinterpret_cast<const __nv_bfloat16 *>(
      static_cast<const uint8_t *>(a.q) + t * a.q_row_stride + h * a.q_head_stride);
  const __nv_bfloat16 *rp = reinterpret_cast<const __nv_bfloat16 *>(
      static_cast<const uint8_t *>(a.q_rope) + t * a.q_rope_row_stride + h * a.q_rope_head_stride);
  for (int i = tid; i < kLatent + kRopeDim; i += 256)
    q[i] = __bfloat162float(i < kLatent ? qp[i] : rp[i - kLatent]);
  __syncthreads();
  const float sl2 = a.softmax_scale * paged::kLog2e;
  float m = -INFINITY, l = 0.f, o[2] = {};
  for (int j0 = lo; j0 < hi; j0 += 256) {
    const int j = j0 + tid;
    const long long row =
        j < hi ? page_row(a.block_table, a.max_blocks, a.n_blocks, b, j, a.status_dev) : -1;
    float x = -INFINITY;
    if (row >= 0) {
      const __nv_bfloat16 *c = reinterpret_cast<const __nv_bfloat16 *>(
          static_cast<const uint8_t *>(a.c_pool) + pool_offset(row, a.c_page_stride, a.c_token_stride));
      const __nv_bfloat16 *r = reinterpret_cast<const __nv_bfloat16 *>(
          static_cast<const uint8_t *>(a.r_pool) + pool_offset(row, a.r_page_stride, a.r_token_stride));
      float s = 0.f;
      for (int i = 0; i < kLatent; ++i) s += q[i] * __bfloat162float(c[i]);
      for (int i = 0; i < kRopeDim; ++i) s += q[kLatent + i] * __bfloat162float(r[i]);
      x = s * sl2;
    }
    float mx = x;
    for (int k = 16; k; k >>= 1) mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, k));
    if ((tid & 31) == 0) red[tid >> 5] = mx;
    __syncthreads();
    mx = m;
    for (int k = 0; k < 8; ++k) mx = fmaxf(mx, red[k]);
    const float f = m == mx ? 1.f : exp2f(m - mx);
    m = mx;
    // (round the probabilities as the product with the latents takes them)
    p[tid] = row < 0 || x == -INFINITY ? 0.f : exp2f(x - (m == -INFINITY ? 0.f : m));
    at[tid] = row;
    __syncthreads();
    l *= f, o[0] *= f, o[1] *= f;
    for (int k = 0; k < 256 && j0 + k < hi; ++k) {
      if (at[k] < 0) continue;
      const __nv_bfloat162 c = reinterpret_cast<const __nv_bfloat162 *>(
          static_cast<const uint8_t *>(a.c_pool) +
          pool_offset(at[k], a.c_page_stride, a.c_token_stride))[tid];
      l += p[k];
      const float pr = round_bf16(p[k]);
      o[0] += pr * __low2float(c), o[1] += pr * __high2float(c);
    }
    __syncthreads();
  }
  const paged::Joined J = paged::finish(m, l, a.sink ? a.sink[h] : -INFINITY);
  const bool zero = m == -INFINITY && l == 0.f;
  reinterpret_cast<__nv_bfloat162 *>(a.out)[((long long)t * a.n_heads + h) * (kLatent / 2) + tid] =
      zero ? __floats2bfloat162_rn(0.f, 0.f) : __floats2bfloat162_rn(o[0] * J.inv, o[1] * J.inv);
  if (a.lse && tid == 0) a.lse[(long long)t * a.n_heads + h] = J.lse;
}

}  // namespace

size_t latent_attn_workspace(const csa_latent_attn_args &) { return 0; }

cudaError_t launch_latent_attn(const csa_latent_attn_args &a, cudaStream_t s) {
  launch_begin(CSA_K_LATENT_ATTN, s);
  latent_attn_kernel<<<a.n_rows * a.n_heads, 256, 0, s>>>(a);
  launch_end(CSA_K_LATENT_ATTN, s);
  return cudaGetLastError();
}

}  // namespace csa
