// Attention over a paged cache of separate keys and values (csa_paged_attn).
#include "csa_internal.cuh"
#include "tc.cuh"

namespace csa {
namespace {

constexpr int PA_THREADS = 256;

// One warp per (row, head): a running maximum m and sum l over the visible
// positions, out = sum_j 2^(x_j - m) v_j / l.
template <int D>
__global__ void __launch_bounds__(PA_THREADS) paged_attn_kernel(csa_paged_attn_args a) {
  tc::griddep_wait();
  tc::griddep_launch_dependents();
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const long long n = (long long)a.n_rows * a.n_heads;
  const float sl2 = a.softmax_scale * 1.4426950408889634f;
  for (long long i = (long long)blockIdx.x * (PA_THREADS / 32) + (threadIdx.x >> 5); i < n;
       i += (long long)gridDim.x * (PA_THREADS / 32)) {
    const int t = (int)(i / a.n_heads), h = (int)(i - (long long)t * a.n_heads);
    const int b = a.row_req[t], p = a.row_pos[t];
    if (b < 0) continue;
    if (b >= a.n_req) {
      if (lane == 0) flag(a.status_dev, CSA_DEV_BAD_POS);
      continue;
    }
    const int kvh = h / (a.n_heads / a.n_kv_heads);
    const long long len = min((long long)a.kv_len[b], (long long)a.max_blocks * kBlock);
    const int hi = (int)(a.causal ? min(len, (long long)p + 1) : len);
    const long long lo_w = a.window > 0 ? (long long)p - a.window + 1 : 0;
    const int lo = lo_w > 0 ? (int)min(lo_w, (long long)0x7FFFFFFF) : 0;
    const __nv_bfloat16 *q = reinterpret_cast<const __nv_bfloat16 *>(
        static_cast<const uint8_t *>(a.q) + t * a.q_row_stride) + h * D;
    float qv[E], acc[E];
    for (int e = 0; e < E; ++e) {
      qv[e] = __bfloat162float(q[lane * E + e]);
      acc[e] = 0.f;
    }
    float m = -INFINITY, l = 0.f;
    for (int j = lo; j < hi; ++j) {
      const long long row = page_row(a.block_table, a.max_blocks, a.n_blocks, b, j, a.status_dev);
      if (row < 0) continue;
      const __nv_bfloat16 *k = reinterpret_cast<const __nv_bfloat16 *>(
          static_cast<const uint8_t *>(a.k_pool) + (row >> 7) * a.k_page_stride +
          (row & 127) * a.k_token_stride + kvh * a.k_head_stride);
      const __nv_bfloat16 *v = reinterpret_cast<const __nv_bfloat16 *>(
          static_cast<const uint8_t *>(a.v_pool) + (row >> 7) * a.v_page_stride +
          (row & 127) * a.v_token_stride + kvh * a.v_head_stride);
      float x = 0.f;
      for (int e = 0; e < E; ++e) x = fmaf(qv[e], __bfloat162float(k[lane * E + e]), x);
      for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
      x *= sl2;
      const float mn = fmaxf(m, x);
      const float w = mn == -INFINITY ? 0.f : exp2f(x - mn), f = mn == -INFINITY ? 1.f : exp2f(m - mn);
      m = mn;
      l = l * f + w;
      for (int e = 0; e < E; ++e) acc[e] = acc[e] * f + w * __bfloat162float(v[lane * E + e]);
    }
    const float s2 = a.sink ? a.sink[h] * 1.4426950408889634f : -INFINITY;
    const float mm = fmaxf(m, s2);
    const float f = m == -INFINITY ? 0.f : exp2f(m - mm);
    const float L = l * f + (s2 == -INFINITY ? 0.f : exp2f(s2 - mm));
    __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(a.out) + ((long long)t * a.n_heads + h) * D;
    for (int e = 0; e < E; ++e)
      o[lane * E + e] = __float2bfloat16_rn(m == -INFINITY ? 0.f : acc[e] * f / L);
    if (a.lse && lane == 0)
      a.lse[(long long)t * a.n_heads + h] =
          mm == -INFINITY ? -INFINITY : (mm + log2f(L)) * 0.6931471805599453f;
  }
}

}  // namespace

size_t paged_attn_workspace(const csa_paged_attn_args &) { return 0; }

cudaError_t launch_paged_attn(const csa_paged_attn_args &a, cudaStream_t s) {
  const long long want = ((long long)a.n_rows * a.n_heads + 7) / 8;
  const dim3 grid((unsigned)(want < 152 * 64 ? want : 152 * 64));
  launch_begin(CSA_K_PAGED_ATTN, s);
  const cudaError_t e =
      a.head_dim == 64
          ? launch_kernel(paged_attn_kernel<64>, grid, dim3(PA_THREADS), 0, s, 0, false, a)
          : launch_kernel(paged_attn_kernel<128>, grid, dim3(PA_THREADS), 0, s, 0, false, a);
  launch_end(CSA_K_PAGED_ATTN, s);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace csa
