// csa_paged_attn: which kernel, how many parts, and the join of the parts.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <cstring>

#include "csa_internal.cuh"
#include "paged_common.cuh"
#include "tc.cuh"

namespace csa {
namespace {

using paged::Parts;

constexpr int PM_THREADS = 256;

// W groups of D / 4 threads per (row, head), four channels a thread: out and lse
// from the row's parts.  Part weights 2^(m_s - m) with m the largest reference; sums
// in FP32, group w adding parts w, w + W, ... and the groups added in order.
// Latency bounds it: four parts of a group are in flight at a time, and where a row
// has many parts eight groups share them (63 parts of 8 rows of 16 heads: the whole
// call 30.1 -> 19.6 us).
template <int D, int W>
__global__ void __launch_bounds__(PM_THREADS)
    paged_merge_kernel(csa_paged_attn_args a, Parts parts) {
  tc::griddep_wait();
  tc::griddep_launch_dependents();
  constexpr int PER = D / 4, ROWS = PM_THREADS / (PER * W);
  __shared__ float sums[W > 1 ? W * ROWS : 1][PER][5];
  const long long rows = (long long)a.n_rows * a.n_heads;
  const int c = threadIdx.x % PER, w = threadIdx.x / PER % W, i = threadIdx.x / (PER * W);
  const long long r = (long long)blockIdx.x * ROWS + i;
  const int t = r < rows ? (int)(r / a.n_heads) : 0;
  const int h = (int)(r - (long long)t * a.n_heads);
  const int b = r < rows ? a.row_req[t] : -1;
  const bool on = b >= 0 && b < a.n_req;
  if (W == 1 && !on) return;
  float m = -INFINITY, acc[4] = {}, l = 0.f;
  if (on) {
#pragma unroll 8
    for (int s = 0; s < parts.n; ++s) m = fmaxf(m, parts.ml[s * rows + r].x);
#pragma unroll 4
    for (int s = w; s < parts.n; s += W) {
      const float2 ml = parts.ml[s * rows + r];
      const float4 o = reinterpret_cast<const float4 *>(parts.o + (s * rows + r) * D)[c];
      if (ml.x == -INFINITY && ml.y == 0.f) continue;  // nothing was seen there (o is not set)
      const float x = ml.x == -INFINITY ? ml.y : exp2f(ml.x - m);  // (l is NaN there)
      l += x * ml.y;
      acc[0] += x * o.x, acc[1] += x * o.y, acc[2] += x * o.z, acc[3] += x * o.w;
    }
  }
  if constexpr (W > 1) {
    float *mine = sums[w * ROWS + i][c];
#pragma unroll
    for (int e = 0; e < 4; ++e) mine[e] = acc[e];
    mine[4] = l;
    __syncthreads();
    if (w != 0 || !on) return;
    for (int k = 1; k < W; ++k) {
      const float *other = sums[k * ROWS + i][c];
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[e] += other[e];
      l += other[4];
    }
  }
  const paged::Joined J = paged::finish(m, l, a.sink ? a.sink[h] : -INFINITY);
  const bool zero = m == -INFINITY && l == 0.f;
  __nv_bfloat162 out[2];
#pragma unroll
  for (int e = 0; e < 2; ++e)
    out[e] = zero ? __floats2bfloat162_rn(0.f, 0.f)
                  : __floats2bfloat162_rn(acc[2 * e] * J.inv, acc[2 * e + 1] * J.inv);
  reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(a.out) + r * D)[c] =
      *reinterpret_cast<const uint2 *>(out);
  if (a.lse && c == 0) a.lse[r] = J.lse;
}

template <int D, int W>
cudaError_t launch_merge(const csa_paged_attn_args &a, const Parts &parts, cudaStream_t s) {
  constexpr int per_block = PM_THREADS / (D / 4 * W);
  const long long rows = (long long)a.n_rows * a.n_heads;
  const dim3 grid((unsigned)((rows + per_block - 1) / per_block));
  return launch_kernel(paged_merge_kernel<D, W>, grid, dim3(PM_THREADS), 0, s, 0, false, a, parts);
}

int sm_count() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms <= 0)
    sms = 152;
  return sms;
}

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static const PFN_cuTensorMapEncodeTiled_v12000 encode = [] {
    cudaDriverEntryPointQueryResult q;
    void *fn = nullptr;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault,
                                         &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      fn = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  }();
  return encode;
}

// BF16 tensor map of up to 4 dimensions, 128-byte swizzle; strides (bytes) of
// dimensions 1...  L2 fetches 256 bytes at a time, but 128 for heads of 64: with tokens
// first their rows lie beside other heads', which would come along (4 x 2 rows at
// 131,072 positions of 8 x 64: 255 -> 198 us; with heads first 168 either way).
bool encode(CUtensorMap *map, const void *base, int rank, const cuuint64_t *dims,
            const cuuint64_t *strides, const cuuint32_t *box) {
  const PFN_cuTensorMapEncodeTiled_v12000 fn = tensor_map_encoder();
  const cuuint32_t ones[4] = {1, 1, 1, 1};
  memset(map, 0, sizeof(*map));
  return fn && fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void *>(base), dims,
                  strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  dims[0] == 64 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B
                                : CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The decode kernel or the chunk kernel.  The decode kernel reads a request's
// pages once for every item of 16 (row, head) pairs of a key/value head (32 from 17
// heads on), the chunk kernel once for up to 256 pairs, but works through the
// requests of a CTA's rows one after the other.  With the average rows of a
// request: up to two items, decode (8 requests of 8 rows of 4 heads over 1000
// positions 20 us against 37, 64 requests of 1 row 52 against 165).  Several
// requests of more items too, while there are at most two an SM, a request's pages
// are not read too often, and a request does not fill a chunk CTA: 4 x 16 rows of 4
// heads over 600 positions 18 us against 26, 8 of them over 2000 43 against 44.  Else
// chunks: 24 of them over 600 (59 us against 37), 8 over 8000 (168 against 91), 12 x
// 8 rows of 32 heads over 400 (20 against 15).  The host does not know how the rows
// are spread.  With one chunk and single tokens for the rest, decode is the faster one
// wherever this takes it (64 requests, 512 rows of 32 heads over 600: 107 us against
// 453) and mostly where this takes chunks (of 64 heads: 162 against 407).  With all rows
// one request's it is the slower one from some 100,000 rows x positions on (16 rows over
// 8000: 24 us against 19, 512 over 600: 98 against 22).  Nor does the host know the
// caches' lengths: max_blocks stands for them.  Results do not depend on the choice but
// for rounding.
bool use_decode(const csa_paged_attn_args &a, int sms) {
  if (a.mode == CSA_MODE_PREFILL || a.n_rows > paged::kDecodeRows) return false;
  if (a.mode == CSA_MODE_DECODE) return true;
  const int per = (int)(((long long)a.n_rows + a.n_req - 1) / a.n_req);
  const long long items = paged_decode_items(a, per);
  return items <= 2 || (a.n_req > 1 && items * a.n_req * a.n_kv_heads <= 2 * sms &&
                        items * a.max_blocks <= 64 && per * (a.n_heads / a.n_kv_heads) < 256);
}

struct Layout {
  bool decode;
  int parts;
  size_t ml, total;  // parts' statistics after their outputs
};

Layout layout(const csa_paged_attn_args &a, int sms) {
  Layout L{use_decode(a, sms), 1, 0, 0};
  if (L.decode) {
    L.total = paged_decode_workspace(a, sms);
    return L;
  }
  L.parts = paged_chunk_parts(a, sms);
  if (L.parts > 1) {
    const size_t rows = (size_t)a.n_rows * a.n_heads * L.parts;
    L.ml = align_up(rows * a.head_dim * sizeof(float), 256);
    L.total = L.ml + align_up(rows * sizeof(float2), 256);
  }
  return L;
}

}  // namespace

namespace paged {

bool encode_pools(const csa_paged_attn_args &a, CUtensorMap *k, CUtensorMap *v) {
  const cuuint64_t dims[4] = {(cuuint64_t)a.head_dim, (cuuint64_t)a.n_kv_heads, (cuuint64_t)kBlock,
                              (cuuint64_t)a.n_blocks};
  const cuuint32_t box[4] = {64, 1, (cuuint32_t)kBlock, 1};
  const cuuint64_t ks[3] = {(cuuint64_t)a.k_head_stride, (cuuint64_t)a.k_token_stride,
                            (cuuint64_t)a.k_page_stride};
  const cuuint64_t vs[3] = {(cuuint64_t)a.v_head_stride, (cuuint64_t)a.v_token_stride,
                            (cuuint64_t)a.v_page_stride};
  return encode(k, a.k_pool, 4, dims, ks, box) && encode(v, a.v_pool, 4, dims, vs, box);
}

bool encode_q(const csa_paged_attn_args &a, int rows, CUtensorMap *q) {
  const cuuint64_t dims[3] = {(cuuint64_t)a.head_dim, (cuuint64_t)a.n_heads, (cuuint64_t)a.n_rows};
  const cuuint64_t st[2] = {(cuuint64_t)a.head_dim * 2, (cuuint64_t)a.q_row_stride};
  const cuuint32_t box[3] = {64, (cuuint32_t)(a.n_heads / a.n_kv_heads), (cuuint32_t)rows};
  return encode(q, a.q, 3, dims, st, box);
}

}  // namespace paged

size_t paged_attn_workspace(const csa_paged_attn_args &a) { return layout(a, sm_count()).total; }

cudaError_t launch_paged_attn(const csa_paged_attn_args &a, cudaStream_t s) {
  const int sms = sm_count();
  const Layout L = layout(a, sms);
  if (L.decode) {
    const cudaError_t e = launch_paged_decode(a, sms, s);
    return e != cudaSuccess ? e : cudaGetLastError();
  }
  uint8_t *ws = static_cast<uint8_t *>(a.workspace);
  const Parts parts{reinterpret_cast<float *>(ws), reinterpret_cast<float2 *>(ws + L.ml), L.parts};
  cudaError_t e = launch_paged_chunk(a, parts, sms, s);
  if (e != cudaSuccess || L.parts == 1) return e != cudaSuccess ? e : cudaGetLastError();
  launch_begin(CSA_K_PAGED_MERGE, s);
  const bool many = L.parts >= 8;
  if (a.head_dim == 64)
    e = many ? launch_merge<64, 8>(a, parts, s) : launch_merge<64, 1>(a, parts, s);
  else
    e = many ? launch_merge<128, 8>(a, parts, s) : launch_merge<128, 1>(a, parts, s);
  launch_end(CSA_K_PAGED_MERGE, s);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace csa
