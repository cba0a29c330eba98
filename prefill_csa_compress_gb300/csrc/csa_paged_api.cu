// extern "C" entry points of the paged key/value cache operators: host-side
// argument checks and kernel dispatch.  No entry point synchronises or
// allocates device memory.
#include <cmath>
#include <cstring>

#include "api_checks.cuh"
#include "csa_internal.cuh"

namespace csa {
namespace {

// head_dim, rotation and norm arguments that csa_qk_norm_rope and
// csa_kv_append share.
template <typename A>
csa_status_t check_head(const A &a) {
  if (a.head_dim < 8 || a.head_dim > 512 || a.head_dim % 8 != 0) return CSA_ERR_UNSUPPORTED;
  if (a.norm != 0 && a.norm != 1) return CSA_ERR_INVALID_ARG;
  if (a.norm && !(a.eps >= 0.f && std::isfinite(a.eps))) return CSA_ERR_INVALID_ARG;
  if ((a.rope_cos == nullptr) != (a.rope_sin == nullptr)) return CSA_ERR_INVALID_ARG;
  if (a.rope_cos) {
    if (a.rope_layout != CSA_ROPE_ADJACENT && a.rope_layout != CSA_ROPE_HALF)
      return CSA_ERR_INVALID_ARG;
    if (a.rope_cap <= 0 || a.rope_dim <= 0 || a.rope_start < 0 || a.rope_dim > a.head_dim ||
        a.rope_start > a.head_dim - a.rope_dim)
      return CSA_ERR_INVALID_ARG;
    if (a.rope_start % 8 != 0 || a.rope_dim % (a.rope_layout == CSA_ROPE_HALF ? 16 : 8) != 0)
      return CSA_ERR_UNSUPPORTED;
    if (!aligned(a.rope_cos, 16) || !aligned(a.rope_sin, 16)) return CSA_ERR_INVALID_ARG;
  }
  return CSA_OK;
}

}  // namespace
}  // namespace csa

using namespace csa;

extern "C" {

CSA_API csa_status_t csa_rope_table(csa_rope_table_args *user, csa_stream_t stream) {
  if (!has_size(user, sizeof(csa_rope_table_args))) return CSA_ERR_INVALID_ARG;
  const csa_rope_table_args a = *user;
  if (a.n_pos < 0 || a.pos0 < 0 || (int64_t)a.pos0 + a.n_pos > (int64_t(1) << 31))
    return CSA_ERR_INVALID_ARG;
  if (a.rope_dim < 2 || a.rope_dim > 512 || a.rope_dim % 2 != 0) return CSA_ERR_UNSUPPORTED;
  if (!(a.theta > 1.0) || !std::isfinite(a.theta)) return CSA_ERR_INVALID_ARG;
  if (!(a.attn_factor > 0.0) || !std::isfinite(a.attn_factor)) return CSA_ERR_INVALID_ARG;
  switch (a.scaling) {
    case CSA_ROPE_NONE: break;
    case CSA_ROPE_NTK:
      if (a.rope_dim < 4) return CSA_ERR_UNSUPPORTED;
      [[fallthrough]];
    case CSA_ROPE_LINEAR:
    case CSA_ROPE_YARN:
      if (!(a.factor >= 1.0) || !std::isfinite(a.factor)) return CSA_ERR_INVALID_ARG;
      if (a.scaling == CSA_ROPE_YARN &&
          (a.orig_len <= 0 || !(a.beta_slow > 0.0) || !(a.beta_fast >= a.beta_slow) ||
           !std::isfinite(a.beta_fast)))
        return CSA_ERR_INVALID_ARG;
      break;
    default: return CSA_ERR_INVALID_ARG;
  }
  if (a.n_pos == 0) return CSA_OK;
  if (!a.cos || !a.sin || !aligned(a.cos, 4) || !aligned(a.sin, 4)) return CSA_ERR_INVALID_ARG;
  return from_cuda(launch_rope_table(a, static_cast<cudaStream_t>(stream)));
}

CSA_API csa_status_t csa_qk_norm_rope(csa_qk_norm_rope_args *user, csa_stream_t stream) {
  if (!has_size(user, sizeof(csa_qk_norm_rope_args))) return CSA_ERR_INVALID_ARG;
  csa_qk_norm_rope_args a = *user;
  if (a.n_rows < 0 || a.n_q_heads < 1 || a.n_k_heads < 0 || a.n_q_heads > 65536 ||
      a.n_k_heads > 65536)
    return CSA_ERR_INVALID_ARG;
  const csa_status_t st = check_head(a);
  if (st != CSA_OK) return st;
  const int64_t qb = (int64_t)a.n_q_heads * a.head_dim * 2, kb = (int64_t)a.n_k_heads * a.head_dim * 2;
  if (!row_stride(&a.q_row_stride, qb) || !row_stride(&a.q_out_row_stride, qb))
    return CSA_ERR_INVALID_ARG;
  if (kb && (!row_stride(&a.k_row_stride, kb) || !row_stride(&a.k_out_row_stride, kb)))
    return CSA_ERR_INVALID_ARG;
  if (a.n_rows == 0) return CSA_OK;
  if (!a.q || !a.q_out || !a.row_pos || (kb && (!a.k || !a.k_out))) return CSA_ERR_INVALID_ARG;
  if (!aligned(a.q, 16) || !aligned(a.q_out, 16) || !aligned(a.q_gamma, 16) ||
      !aligned(a.k_gamma, 16) || (kb && (!aligned(a.k, 16) || !aligned(a.k_out, 16))))
    return CSA_ERR_INVALID_ARG;
  return from_cuda(launch_qk_norm_rope(a, static_cast<cudaStream_t>(stream)));
}

CSA_API csa_status_t csa_kv_append(csa_kv_append_args *user, csa_stream_t stream) {
  if (!has_size(user, sizeof(csa_kv_append_args))) return CSA_ERR_INVALID_ARG;
  csa_kv_append_args a = *user;
  if (a.n_rows < 0 || a.n_heads < 1 || a.n_heads > 65536) return CSA_ERR_INVALID_ARG;
  const csa_status_t st = check_head(a);
  if (st != CSA_OK) return st;
  if (a.n_req <= 0 || a.max_blocks <= 0 || a.n_blocks <= 0) return CSA_ERR_INVALID_ARG;
  const int64_t bytes = (int64_t)a.head_dim * 2;
  if (!row_stride(&a.k_row_stride, a.n_heads * bytes) ||
      !row_stride(&a.v_row_stride, a.n_heads * bytes))
    return CSA_ERR_INVALID_ARG;
  if (a.fmt == CSA_FMT_BF16) {
    if (!pool_strides(&a.k_page_stride, &a.k_token_stride, &a.k_head_stride, a.n_blocks, a.n_heads,
                      bytes) ||
        !pool_strides(&a.v_page_stride, &a.v_token_stride, &a.v_head_stride, a.n_blocks, a.n_heads,
                      bytes))
      return CSA_ERR_INVALID_ARG;
  } else if (a.fmt == CSA_FMT_MXFP8) {
    if (a.head_dim % 32 != 0 || a.k_page_stride || a.k_token_stride || a.k_head_stride ||
        a.v_page_stride || a.v_token_stride || a.v_head_stride)
      return CSA_ERR_UNSUPPORTED;
  } else {
    return CSA_ERR_UNSUPPORTED;
  }
  if (a.n_rows == 0) return CSA_OK;
  if (!a.k || !a.row_req || !a.row_pos || !a.block_table || !a.k_pool || (a.v && !a.v_pool))
    return CSA_ERR_INVALID_ARG;
  if (a.fmt == CSA_FMT_MXFP8 && (!a.k_scale_pool || (a.v && !a.v_scale_pool)))
    return CSA_ERR_INVALID_ARG;
  if (!aligned(a.k, 16) || !aligned(a.v, 16) || !aligned(a.k_pool, 16) || !aligned(a.v_pool, 16) ||
      !aligned(a.k_gamma, 16))
    return CSA_ERR_INVALID_ARG;
  return from_cuda(launch_kv_append(a, static_cast<cudaStream_t>(stream)));
}

CSA_API csa_status_t csa_paged_attn(csa_paged_attn_args *user, csa_stream_t stream) {
  if (!has_size(user, offsetof(csa_paged_attn_args, v_dim))) return CSA_ERR_INVALID_ARG;
  csa_paged_attn_args a = {};
  memcpy(&a, user, user->struct_size < sizeof(a) ? user->struct_size : sizeof(a));
  if (user->struct_size < sizeof(a) || a.v_dim == 0) a.v_dim = a.head_dim;
  if (a.n_rows < 0 || a.n_req <= 0 || a.max_blocks <= 0 || a.n_blocks <= 0)
    return CSA_ERR_INVALID_ARG;
  if (a.n_rows > (1 << 24)) return CSA_ERR_UNSUPPORTED;
  if (a.max_blocks > (1 << 24) || a.n_heads < 1 || a.n_kv_heads < 1 || a.n_heads > 65536 ||
      a.n_heads % a.n_kv_heads)
    return CSA_ERR_INVALID_ARG;
  const bool same = (a.head_dim == 64 || a.head_dim == 128) && a.v_dim == a.head_dim;
  if (!(same || (a.head_dim == 192 && a.v_dim == 128)) || a.n_heads / a.n_kv_heads > 128)
    return CSA_ERR_UNSUPPORTED;
  if ((a.causal != 0 && a.causal != 1) || a.window < 0 || a.mode < CSA_MODE_AUTO ||
      a.mode > CSA_MODE_PREFILL)
    return CSA_ERR_INVALID_ARG;
  if (!(a.softmax_scale > 0.f) || !std::isfinite(a.softmax_scale)) return CSA_ERR_INVALID_ARG;
  const int64_t bytes = (int64_t)a.head_dim * 2;
  if (!row_stride(&a.q_row_stride, a.n_heads * bytes)) return CSA_ERR_INVALID_ARG;
  if (!pool_strides(&a.k_page_stride, &a.k_token_stride, &a.k_head_stride, a.n_blocks,
                    a.n_kv_heads, bytes) ||
      !pool_strides(&a.v_page_stride, &a.v_token_stride, &a.v_head_stride, a.n_blocks,
                    a.n_kv_heads, (int64_t)a.v_dim * 2))
    return CSA_ERR_INVALID_ARG;
  const size_t need = query_bytes(paged_attn_workspace(a));
  if (!a.workspace) {
    user->workspace_bytes = need;
    return CSA_OK;
  }
  if (a.workspace_bytes < need || !aligned(a.workspace, 256)) return CSA_ERR_INVALID_ARG;
  if (a.n_rows == 0) return CSA_OK;
  if (!a.q || !a.row_req || !a.row_pos || !a.kv_len || !a.block_table || !a.k_pool || !a.v_pool ||
      !a.out)
    return CSA_ERR_INVALID_ARG;
  if (!aligned(a.q, 16) || !aligned(a.k_pool, 16) || !aligned(a.v_pool, 16) || !aligned(a.out, 16))
    return CSA_ERR_INVALID_ARG;
  return from_cuda(launch_paged_attn(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
