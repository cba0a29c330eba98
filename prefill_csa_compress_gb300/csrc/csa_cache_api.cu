// extern "C" entry points of the latent cache and eviction calls: host-side
// argument checks and kernel dispatch.  No entry point synchronises or allocates
// device memory.
#include <cmath>

#include "api_checks.cuh"
#include "cache_common.cuh"

namespace csa {
namespace {

constexpr int kMaxRows = 1 << 24, kMaxPages = 1 << 24;

// A row and a head stride in bytes, 0 meaning dense: any order, no overlap.
bool row_head_strides(int64_t *row, int64_t *head, int64_t n_rows, int64_t n_heads, int64_t bytes) {
  if (*head == 0) *head = bytes;
  if (*row == 0) *row = n_heads * bytes;
  if (*row % 16 != 0 || *head % 16 != 0 || *row < bytes || *head < bytes ||
      *row >= (int64_t(1) << 40) || *head >= (int64_t(1) << 40))
    return false;
  if (n_rows <= 1 || n_heads <= 1) return true;
  return *row >= *head ? *row >= *head * (n_heads - 1) + bytes : *head >= *row * (n_rows - 1) + bytes;
}

// A row stride in bytes of FP32 rows, 0 meaning dense.
bool float_row_stride(int64_t *s, int64_t n) {
  if (*s == 0) *s = n * 4;
  return *s % 4 == 0 && *s >= n * 4 && *s < (int64_t(1) << 40);
}

bool latent_pool_strides(int64_t *c_page, int64_t *c_token, int64_t *r_page, int64_t *r_token,
                         int64_t n_blocks) {
  int64_t c_head = 0, r_head = 0;
  return pool_strides(c_page, c_token, &c_head, n_blocks, 1, kLatent * 2) &&
         pool_strides(r_page, r_token, &r_head, n_blocks, 1, kRopeDim * 2);
}

bool scale_ok(float s) { return s > 0.f && std::isfinite(s); }

}  // namespace
}  // namespace csa

using namespace csa;

extern "C" {

CSA_API csa_status_t csa_latent_attn(csa_latent_attn_args *user, csa_stream_t stream) {
  if (!has_size(user, sizeof(csa_latent_attn_args))) return CSA_ERR_INVALID_ARG;
  csa_latent_attn_args a = *user;
  if (a.n_rows < 0 || a.n_heads < 1 || a.n_req <= 0 || a.max_blocks <= 0 || a.n_blocks <= 0)
    return CSA_ERR_INVALID_ARG;
  if (a.n_rows > kMaxRows || a.max_blocks > kMaxPages || a.n_heads > kMaxHeads)
    return CSA_ERR_UNSUPPORTED;
  if ((a.causal != 0 && a.causal != 1) || a.window < 0 || !scale_ok(a.softmax_scale))
    return CSA_ERR_INVALID_ARG;
  if (!row_head_strides(&a.q_row_stride, &a.q_head_stride, a.n_rows, a.n_heads, kLatent * 2) ||
      !row_head_strides(&a.q_rope_row_stride, &a.q_rope_head_stride, a.n_rows, a.n_heads,
                        kRopeDim * 2) ||
      !latent_pool_strides(&a.c_page_stride, &a.c_token_stride, &a.r_page_stride,
                           &a.r_token_stride, a.n_blocks))
    return CSA_ERR_INVALID_ARG;
  const size_t need = query_bytes(latent_attn_workspace(a));
  if (!a.workspace) {
    user->workspace_bytes = need;
    return CSA_OK;
  }
  if (a.workspace_bytes < need || !aligned(a.workspace, 256)) return CSA_ERR_INVALID_ARG;
  if (a.n_rows == 0) return CSA_OK;
  if (!a.q || !a.q_rope || !a.row_req || !a.row_pos || !a.kv_len || !a.block_table || !a.c_pool ||
      !a.r_pool || !a.out)
    return CSA_ERR_INVALID_ARG;
  if (!aligned(a.q, 16) || !aligned(a.q_rope, 16) || !aligned(a.c_pool, 16) ||
      !aligned(a.r_pool, 16) || !aligned(a.out, 16))
    return CSA_ERR_INVALID_ARG;
  return from_cuda(launch_latent_attn(a, static_cast<cudaStream_t>(stream)));
}

CSA_API csa_status_t csa_latent_expand(csa_latent_expand_args *user, csa_stream_t stream) {
  if (!has_size(user, sizeof(csa_latent_expand_args))) return CSA_ERR_INVALID_ARG;
  csa_latent_expand_args a = *user;
  if (a.n_heads < 1 || a.n_heads > 65536 || a.n_req < 0 || a.max_blocks <= 0 || a.n_blocks <= 0 ||
      a.out_max_blocks <= 0 || a.n_out_blocks <= 0)
    return CSA_ERR_INVALID_ARG;
  if (a.max_blocks >= kMaxPages) return CSA_ERR_UNSUPPORTED;
  const int64_t wb = (int64_t)kNope * kLatent * 2;
  if (!latent_pool_strides(&a.c_page_stride, &a.c_token_stride, &a.r_page_stride,
                           &a.r_token_stride, a.n_blocks) ||
      !row_stride(&a.w_uk_head_stride, wb) || !row_stride(&a.w_uv_head_stride, wb) ||
      !pool_strides(&a.k_page_stride, &a.k_token_stride, &a.k_head_stride, a.n_out_blocks,
                    a.n_heads, (kNope + kRopeDim) * 2) ||
      !pool_strides(&a.v_page_stride, &a.v_token_stride, &a.v_head_stride, a.n_out_blocks,
                    a.n_heads, kValue * 2))
    return CSA_ERR_INVALID_ARG;
  if (a.n_req == 0) return CSA_OK;
  if (!a.kv_len || !a.block_table || !a.out_table || !a.c_pool || !a.r_pool || !a.w_uk || !a.w_uv ||
      !a.k_pool || !a.v_pool)
    return CSA_ERR_INVALID_ARG;
  if (!aligned(a.c_pool, 16) || !aligned(a.r_pool, 16) || !aligned(a.w_uk, 16) ||
      !aligned(a.w_uv, 16) || !aligned(a.k_pool, 16) || !aligned(a.v_pool, 16))
    return CSA_ERR_INVALID_ARG;
  return from_cuda(launch_latent_expand(a, static_cast<cudaStream_t>(stream)));
}

CSA_API csa_status_t csa_attn_mass(csa_attn_mass_args *user, csa_stream_t stream) {
  if (!has_size(user, sizeof(csa_attn_mass_args))) return CSA_ERR_INVALID_ARG;
  csa_attn_mass_args a = *user;
  if (a.n_rows < 0 || a.n_req <= 0 || a.max_blocks <= 0 || a.n_blocks <= 0 || a.n_heads < 1 ||
      a.n_kv_heads < 1 || a.n_heads > 65536 || a.n_heads % a.n_kv_heads)
    return CSA_ERR_INVALID_ARG;
  if (a.n_rows > kMaxRows || a.max_blocks >= kMaxPages ||
      (a.head_dim != 64 && a.head_dim != 128) || a.n_heads / a.n_kv_heads > 128)
    return CSA_ERR_UNSUPPORTED;
  if ((a.causal != 0 && a.causal != 1) || a.window < 0 || !scale_ok(a.softmax_scale) ||
      !(a.decay >= 0.f) || !std::isfinite(a.decay))
    return CSA_ERR_INVALID_ARG;
  const int64_t bytes = (int64_t)a.head_dim * 2, cols = (int64_t)a.max_blocks * kBlock;
  if (!row_stride(&a.q_row_stride, a.n_heads * bytes) ||
      !pool_strides(&a.k_page_stride, &a.k_token_stride, &a.k_head_stride, a.n_blocks,
                    a.n_kv_heads, bytes) ||
      !float_row_stride(&a.mass_row_stride, cols) || !float_row_stride(&a.mass_out_row_stride, cols))
    return CSA_ERR_INVALID_ARG;
  const size_t need = query_bytes(attn_mass_workspace(a));
  if (!a.workspace) {
    user->workspace_bytes = need;
    return CSA_OK;
  }
  if (a.workspace_bytes < need || !aligned(a.workspace, 256)) return CSA_ERR_INVALID_ARG;
  if (!a.kv_len || !a.block_table || !a.k_pool || !a.mass_out || (a.decay != 0.f && !a.mass) ||
      (a.n_rows > 0 && (!a.q || !a.lse || !a.row_req || !a.row_pos)))
    return CSA_ERR_INVALID_ARG;
  if (!aligned(a.q, 16) || !aligned(a.k_pool, 16) || !aligned(a.mass, 4) || !aligned(a.mass_out, 4) ||
      !aligned(a.lse, 4))
    return CSA_ERR_INVALID_ARG;
  // (equal rows of equal stride are in place; anything else must not overlap)
  if (a.mass == a.mass_out && a.decay != 0.f && a.mass_row_stride != a.mass_out_row_stride)
    return CSA_ERR_INVALID_ARG;
  return from_cuda(launch_attn_mass(a, static_cast<cudaStream_t>(stream)));
}

CSA_API csa_status_t csa_kv_evict(csa_kv_evict_args *user, csa_stream_t stream) {
  if (!has_size(user, sizeof(csa_kv_evict_args))) return CSA_ERR_INVALID_ARG;
  csa_kv_evict_args a = *user;
  if (a.n_req < 0 || a.max_blocks <= 0 || a.n_blocks <= 0 || a.n_heads < 1 || a.n_heads > 65536 ||
      a.first < 0 || a.recent < 0)
    return CSA_ERR_INVALID_ARG;
  if (a.max_blocks >= kMaxPages / 2) return CSA_ERR_UNSUPPORTED;
  if (!a.v_pool) a.v_dim = 0, a.v_page_stride = a.v_token_stride = a.v_head_stride = 0;
  if (a.k_dim < 8 || a.k_dim > 512 || a.k_dim % 8 != 0 ||
      (a.v_pool && (a.v_dim < 8 || a.v_dim > 512 || a.v_dim % 8 != 0)))
    return CSA_ERR_UNSUPPORTED;
  const int64_t cols = (int64_t)a.max_blocks * kBlock;
  if (!pool_strides(&a.k_page_stride, &a.k_token_stride, &a.k_head_stride, a.n_blocks, a.n_heads,
                    (int64_t)a.k_dim * 2) ||
      (a.v_pool && !pool_strides(&a.v_page_stride, &a.v_token_stride, &a.v_head_stride, a.n_blocks,
                                 a.n_heads, (int64_t)a.v_dim * 2)) ||
      !float_row_stride(&a.mass_row_stride, cols) || !float_row_stride(&a.mass_out_row_stride, cols))
    return CSA_ERR_INVALID_ARG;
  const size_t need = query_bytes(kv_evict_workspace(a));
  if (!a.workspace) {
    user->workspace_bytes = need;
    return CSA_OK;
  }
  if (a.workspace_bytes < need || !aligned(a.workspace, 256)) return CSA_ERR_INVALID_ARG;
  if (a.n_req == 0) return CSA_OK;
  if (!a.mass || !a.kv_len || !a.budget || !a.block_table || !a.k_pool || !a.kv_len_out)
    return CSA_ERR_INVALID_ARG;
  if (!aligned(a.k_pool, 16) || !aligned(a.v_pool, 16) || !aligned(a.mass, 4) ||
      !aligned(a.mass_out, 4))
    return CSA_ERR_INVALID_ARG;
  if (a.mass_out == a.mass && a.mass_row_stride != a.mass_out_row_stride)
    return CSA_ERR_INVALID_ARG;
  return from_cuda(launch_kv_evict(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
