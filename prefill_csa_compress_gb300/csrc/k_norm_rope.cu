// csa_qk_norm_rope and csa_kv_append: every head of every row is normed over
// its channels and rotated at the row's position (headvec.cuh), then stored to
// its own tensor or into a paged cache.  Both only move memory: each element
// is read once and written once.
#include <type_traits>

#include "csa_internal.cuh"
#include "headvec.cuh"
#include "lowbit.cuh"
#include "tc.cuh"

namespace csa {
namespace {

using headvec::Rope;

constexpr int NR_THREADS = 256;

__device__ __forceinline__ const uint16_t *at(const void *base, long long bytes) {
  return reinterpret_cast<const uint16_t *>(static_cast<const uint8_t *>(base) + bytes);
}

template <int L, int C>
__global__ void __launch_bounds__(NR_THREADS) qk_norm_rope_kernel(csa_qk_norm_rope_args a) {
  tc::griddep_wait();
  tc::griddep_launch_dependents();
  constexpr int PER_BLOCK = NR_THREADS / L;
  const int H = a.n_q_heads + a.n_k_heads, n_chunks = a.head_dim / 8;
  const long long total = (long long)a.n_rows * H;
  const Rope R{a.rope_cos, a.rope_sin, a.rope_start, a.rope_dim, a.rope_cap,
               a.rope_layout == CSA_ROPE_HALF};
  for (long long i0 = (long long)blockIdx.x * PER_BLOCK; i0 < total;
       i0 += (long long)gridDim.x * PER_BLOCK) {
    const long long i = i0 + threadIdx.x / L;
    bool on = i < total;
    const int t = on ? (int)(i / H) : 0, h = on ? (int)(i - (long long)t * H) : 0;
    if (on && a.row_req && a.row_req[t] < 0) on = false;
    const bool is_q = h < a.n_q_heads;
    const int hh = is_q ? h : h - a.n_q_heads;
    const long long col = (long long)hh * a.head_dim * 2;
    const int trow = on ? headvec::table_row(R, a.row_pos[t], a.status_dev) : -1;
    float y[C][8];
    headvec::load<L, C>(is_q ? at(a.q, t * a.q_row_stride + col) : at(a.k, t * a.k_row_stride + col),
                        n_chunks, on, a.norm, a.norm, a.eps,
                        static_cast<const uint16_t *>(is_q ? a.q_gamma : a.k_gamma), R, trow, y);
    uint8_t *out = static_cast<uint8_t *>(is_q ? a.q_out : a.k_out) +
                   t * (is_q ? a.q_out_row_stride : a.k_out_row_stride) + col;
#pragma unroll
    for (int j = 0; j < C; ++j) {
      const int c = (threadIdx.x & (L - 1)) + L * j;
      if (on && c < n_chunks) reinterpret_cast<uint4 *>(out)[c] = headvec::pack8(y[j]);
    }
  }
}

template <int L, int C>
__global__ void __launch_bounds__(NR_THREADS) kv_append_kernel(csa_kv_append_args a) {
  tc::griddep_wait();
  tc::griddep_launch_dependents();
  constexpr int PER_BLOCK = NR_THREADS / L;
  const int HV = a.n_heads * (a.v ? 2 : 1), n_chunks = a.head_dim / 8;
  const long long total = (long long)a.n_rows * HV;
  const Rope R{a.rope_cos, a.rope_sin, a.rope_start, a.rope_dim, a.rope_cap,
               a.rope_layout == CSA_ROPE_HALF};
  for (long long i0 = (long long)blockIdx.x * PER_BLOCK; i0 < total;
       i0 += (long long)gridDim.x * PER_BLOCK) {
    const long long i = i0 + threadIdx.x / L;
    bool on = i < total;
    const int t = on ? (int)(i / HV) : 0, hv = on ? (int)(i - (long long)t * HV) : 0;
    const bool is_k = hv < a.n_heads;
    const int h = is_k ? hv : hv - a.n_heads;
    const int b = on ? a.row_req[t] : -1, p = on ? a.row_pos[t] : -1;
    if (b >= a.n_req) flag(a.status_dev, CSA_DEV_BAD_POS);
    on = on && b >= 0 && b < a.n_req && p >= 0;
    long long row = -1;
    if (on) row = page_row(a.block_table, a.max_blocks, a.n_blocks, b, p, a.status_dev);
    on = on && row >= 0;
    const int trow = on && is_k ? headvec::table_row(R, p, a.status_dev) : -1;
    const long long col = (long long)h * a.head_dim * 2;
    float y[C][8];
    headvec::load<L, C>(is_k ? at(a.k, t * a.k_row_stride + col) : at(a.v, t * a.v_row_stride + col),
                        n_chunks, on, a.norm, is_k && a.norm, a.eps,
                        static_cast<const uint16_t *>(a.k_gamma), R, trow, y);
    const long long page = row >> 7, in = row & 127;
    if (a.fmt == CSA_FMT_BF16) {
      uint8_t *out = is_k ? static_cast<uint8_t *>(a.k_pool) + page * a.k_page_stride +
                                in * a.k_token_stride + h * a.k_head_stride
                          : static_cast<uint8_t *>(a.v_pool) + page * a.v_page_stride +
                                in * a.v_token_stride + h * a.v_head_stride;
#pragma unroll
      for (int j = 0; j < C; ++j) {
        const int c = (threadIdx.x & (L - 1)) + L * j;
        if (on && c < n_chunks) reinterpret_cast<uint4 *>(out)[c] = headvec::pack8(y[j]);
      }
    } else if constexpr (L >= 4) {
      // groups of 32 channels: four neighbouring lanes share a scale
      uint8_t *codes = static_cast<uint8_t *>(is_k ? a.k_pool : a.v_pool);
      uint8_t *scales = is_k ? a.k_scale_pool : a.v_scale_pool;
      const long long vec = row * a.n_heads + h;
#pragma unroll
      for (int j = 0; j < C; ++j) {
        const int c = (threadIdx.x & (L - 1)) + L * j;
        float m = 0.f;
#pragma unroll
        for (int u = 0; u < 8; ++u) m = fmaxf(m, fabsf(y[j][u]));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
        const int e = m <= 3.4028235e38f ? lowbit::e8m0_exponent_448(m) : 127;
        // 2^-e as a factor: exact, in two steps where it leaves FP32's normal range
        const float s1 = lowbit::pow2f(-(e / 2)), s2 = lowbit::pow2f(-(e - e / 2));
        uint32_t w[2] = {0, 0};
#pragma unroll
        for (int u = 0; u < 8; ++u)
          w[u >> 2] |= (uint32_t)__nv_cvt_float_to_fp8(y[j][u] * s1 * s2, __NV_SATFINITE, __NV_E4M3)
                       << (8 * (u & 3));
        if (on && c < n_chunks) {
          reinterpret_cast<uint2 *>(codes + vec * a.head_dim)[c] = make_uint2(w[0], w[1]);
          if ((c & 3) == 0) scales[vec * (a.head_dim / 32) + (c >> 2)] = (uint8_t)(e + 127);
        }
      }
    }
  }
}

int grid_for(long long vectors, int per_block) {
  const long long want = (vectors + per_block - 1) / per_block;
  return (int)(want < 152 * 256 ? want : 152 * 256);
}

}  // namespace

cudaError_t launch_qk_norm_rope(const csa_qk_norm_rope_args &a, cudaStream_t s) {
  const long long n = (long long)a.n_rows * (a.n_q_heads + a.n_k_heads);
  launch_begin(CSA_K_NORM_ROPE, s);
  const cudaError_t e = headvec::dispatch(a.head_dim, [&](auto L, auto C) {
    return launch_kernel(qk_norm_rope_kernel<L(), C()>, dim3(grid_for(n, NR_THREADS / L())),
                         dim3(NR_THREADS), 0, s, 0, false, a);
  });
  launch_end(CSA_K_NORM_ROPE, s);
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_kv_append(const csa_kv_append_args &a, cudaStream_t s) {
  const long long n = (long long)a.n_rows * a.n_heads * (a.v ? 2 : 1);
  launch_begin(CSA_K_KV_APPEND, s);
  const cudaError_t e = headvec::dispatch(a.head_dim, [&](auto L, auto C) {
    return launch_kernel(kv_append_kernel<L(), C()>, dim3(grid_for(n, NR_THREADS / L())),
                         dim3(NR_THREADS), 0, s, 0, false, a);
  });
  launch_end(CSA_K_KV_APPEND, s);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace csa
