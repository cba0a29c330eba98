// Cuts paged caches to their heaviest positions, in place (csa_kv_evict).
//
// The choice.  A mass maps to 32 bits in its order (NaN lowest, both zeros alike,
// protected positions as +inf); four passes over eight bits each find the key T of
// the n-th heaviest and how many positions equal to T are taken, lowest first.
// A position's rank among the kept ones is then the number of keys above T before
// it and of taken ties before it, so holes before n and kept positions behind it
// pair up by rank and no two moves touch the same slot: sources lie at n and
// behind, destinations before it.
#include "cache_common.cuh"

namespace csa {
namespace {

constexpr int EV_THREADS = 1024, EV_WARPS = EV_THREADS / 32;

// A request's moves in the workspace: (destination, source) pairs, and their number.
struct Moves {
  int2 *list;      // [n_req][cap]
  int *n;          // [n_req]
  long long cap;   // half of a request's slots: every move has a hole and a source
};

__device__ __forceinline__ int cache_len(const csa_kv_evict_args &a, int b) {
  return (int)max(min((long long)a.kv_len[b], (long long)a.max_blocks * kBlock), 0ll);
}

__device__ __forceinline__ const float *mass_row(const csa_kv_evict_args &a, int b) {
  return reinterpret_cast<const float *>(reinterpret_cast<const uint8_t *>(a.mass) +
                                         b * a.mass_row_stride);
}

__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return 0;
  const uint32_t u = __float_as_uint(x == 0.f ? 0.f : x);
  return u >> 31 ? ~u : u | 0x80000000u;
}

__global__ void __launch_bounds__(EV_THREADS) evict_plan_kernel(csa_kv_evict_args a, Moves mv) {
  __shared__ int hist[256], above[EV_WARPS], ties[EV_WARPS], above_n[EV_WARPS], ties_n[EV_WARPS];
  __shared__ uint32_t sh_prefix;
  __shared__ int sh_need;
  const int b = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int L = cache_len(a, b), n = min(L, max(a.budget[b], 0));
  const float *mass = mass_row(a, b);
  __syncthreads();  // (kv_len_out may be kv_len)
  if (tid == 0) a.kv_len_out[b] = n, mv.n[b] = 0;
  if (n == 0 || n == L) return;
  auto key_at = [&](int i) {
    return i < a.first || i >= L - a.recent ? 0xFF800000u : order_key(mass[i]);
  };
  uint32_t prefix = 0;
  int need = n;
  for (int shift = 24; shift >= 0; shift -= 8) {
    if (tid < 256) hist[tid] = 0;
    __syncthreads();
    for (int i = tid; i < L; i += EV_THREADS) {
      const uint32_t k = key_at(i);
      if (shift == 24 || (k >> (shift + 8)) == (prefix >> (shift + 8)))
        atomicAdd(&hist[k >> shift & 255], 1);
    }
    __syncthreads();
    if (tid == 0) {
      int d = 255;
      while (hist[d] < need) need -= hist[d--];
      sh_need = need;
      sh_prefix = prefix | (uint32_t)d << shift;
    }
    __syncthreads();
    prefix = sh_prefix, need = sh_need;
    __syncthreads();
  }
  // a warp's run of positions; keys above T and ties in it, in all and before n
  const int per = (L + EV_WARPS * 32 - 1) / (EV_WARPS * 32) * 32;
  const int i0 = warp * per, i1 = min(L, i0 + per);
  int c_a = 0, c_t = 0, n_a = 0, n_t = 0;
  for (int i = i0; i < i1; i += 32) {
    const uint32_t k = i + lane < i1 ? key_at(i + lane) : 0;
    const bool in = i + lane < i1;
    const uint32_t up = __ballot_sync(~0u, in && k > prefix), eq = __ballot_sync(~0u, in && k == prefix);
    const int before = n - i;
    const uint32_t m = before >= 32 ? ~0u : (before <= 0 ? 0u : (1u << before) - 1u);
    c_a += __popc(up), c_t += __popc(eq), n_a += __popc(up & m), n_t += __popc(eq & m);
  }
  if (lane == 0) above[warp] = c_a, ties[warp] = c_t, above_n[warp] = n_a, ties_n[warp] = n_t;
  __syncthreads();
  int a0 = 0, t0 = 0, k_a = 0, k_t = 0;
  for (int w = 0; w < EV_WARPS; ++w) {
    if (w < warp) a0 += above[w], t0 += ties[w];
    k_a += above_n[w], k_t += ties_n[w];
  }
  const int kept_n = k_a + min(k_t, need);  // kept positions that stay
  int2 *list = mv.list + b * mv.cap;
  for (int i = i0; i < i1; i += 32) {
    const bool in = i + lane < i1;
    const uint32_t k = in ? key_at(i + lane) : 0, under = (1u << lane) - 1u;
    const uint32_t up = __ballot_sync(~0u, in && k > prefix), eq = __ballot_sync(~0u, in && k == prefix);
    const int tie = t0 + __popc(eq & under);
    const bool kept = in && (k > prefix || (k == prefix && tie < need));
    const int rank = a0 + __popc(up & under) + min(tie, need);  // kept positions before
    const int j = i + lane;
    if (in && !kept && j < n) list[j - rank].x = j;
    if (kept && j >= n) list[rank - kept_n].y = j;
    a0 += __popc(up), t0 += __popc(eq);
  }
  if (tid == 0) mv.n[b] = n - kept_n;
}

// A warp a slot: what the slot holds now, and the row's move if there is one.
__global__ void __launch_bounds__(256) evict_move_kernel(csa_kv_evict_args a, Moves mv) {
  const int b = blockIdx.y, lane = threadIdx.x & 31;
  const int n = a.kv_len_out[b], H = mv.n[b];
  const float *mass = mass_row(a, b);
  float *mass_out = a.mass_out ? reinterpret_cast<float *>(reinterpret_cast<uint8_t *>(a.mass_out) +
                                                           b * a.mass_out_row_stride)
                               : nullptr;
  int *src_out = a.slot_src ? a.slot_src + (long long)b * a.max_blocks * kBlock : nullptr;
  const int2 *list = mv.list + b * mv.cap;
  for (int m = blockIdx.x * 8 + (threadIdx.x >> 5); m < H; m += gridDim.x * 8) {
    const int2 e = list[m];
    if (lane == 0) {
      if (mass_out) mass_out[e.x] = mass[e.y];
      if (src_out) src_out[e.x] = e.y;
    }
    const long long to = page_row(a.block_table, a.max_blocks, a.n_blocks, b, e.x, a.status_dev);
    const long long from = page_row(a.block_table, a.max_blocks, a.n_blocks, b, e.y, a.status_dev);
    if (to < 0 || from < 0) continue;
    for (int kv = 0; kv < 2; ++kv) {
      uint8_t *pool = static_cast<uint8_t *>(kv ? a.v_pool : a.k_pool);
      if (!pool) continue;
      const int vecs = (kv ? a.v_dim : a.k_dim) / 8;
      const long long ps = kv ? a.v_page_stride : a.k_page_stride,
                      ts = kv ? a.v_token_stride : a.k_token_stride,
                      hs = kv ? a.v_head_stride : a.k_head_stride;
      for (int v = lane; v < vecs * a.n_heads; v += 32) {
        const long long off = v / vecs * hs + v % vecs * 16;
        *reinterpret_cast<uint4 *>(pool + pool_offset(to, ps, ts) + off) =
            *reinterpret_cast<const uint4 *>(pool + pool_offset(from, ps, ts) + off);
      }
    }
  }
}

// Slots that keep what they hold.
__global__ void __launch_bounds__(256) evict_stay_kernel(csa_kv_evict_args a, Moves) {
  const int b = blockIdx.y, n = a.kv_len_out[b];
  const float *mass = mass_row(a, b);
  for (int j = blockIdx.x * 256 + threadIdx.x; j < n; j += gridDim.x * 256) {
    if (a.mass_out && a.mass_out != a.mass)
      reinterpret_cast<float *>(reinterpret_cast<uint8_t *>(a.mass_out) +
                                b * a.mass_out_row_stride)[j] = mass[j];
    if (a.slot_src) a.slot_src[(long long)b * a.max_blocks * kBlock + j] = j;
  }
}

}  // namespace

size_t kv_evict_workspace(const csa_kv_evict_args &a) {
  return align_up((size_t)a.n_req * a.max_blocks * (kBlock / 2) * sizeof(int2), 256) +
         align_up((size_t)a.n_req * sizeof(int), 256);
}

cudaError_t launch_kv_evict(const csa_kv_evict_args &a, cudaStream_t s) {
  Moves mv;
  mv.cap = (long long)a.max_blocks * (kBlock / 2);
  mv.list = static_cast<int2 *>(a.workspace);
  mv.n = reinterpret_cast<int *>(static_cast<uint8_t *>(a.workspace) +
                                 align_up((size_t)a.n_req * mv.cap * sizeof(int2), 256));
  launch_begin(CSA_K_EVICT_PLAN, s);
  evict_plan_kernel<<<a.n_req, EV_THREADS, 0, s>>>(a, mv);
  launch_end(CSA_K_EVICT_PLAN, s);
  launch_begin(CSA_K_EVICT_MOVE, s);
  evict_stay_kernel<<<dim3(32, a.n_req), 256, 0, s>>>(a, mv);
  evict_move_kernel<<<dim3(152, a.n_req), 256, 0, s>>>(a, mv);
  launch_end(CSA_K_EVICT_MOVE, s);
  return cudaGetLastError();
}

}  // namespace csa
