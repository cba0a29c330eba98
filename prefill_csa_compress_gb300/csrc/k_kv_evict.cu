// Cuts paged caches to their heaviest positions, in place (csa_kv_evict).
//
// The choice.  A mass maps to 32 bits in its order (NaN lowest, both zeros alike,
// protected positions as +inf); four passes over eight bits each find the key T of
// the n-th heaviest and how many positions equal to T are taken, lowest first.
// A position's rank among the kept ones is then the number of keys above T before
// it and of taken ties before it, so holes before n and kept positions behind it
// pair up by rank, and no two moves touch the same slot: sources lie at n and
// behind, destinations before it.
//
// A cluster of up to eight CTAs takes a request: each counts its stretch of positions
// (a warp a run of them, up to 16 keys a thread in registers, else read again for every
// pass), and all add up the cluster's counts from distributed shared memory, so that
// every CTA knows the same T.  What it takes is a dozen trips to memory and across the
// cluster.  The moves are a kernel of their own, bound by memory.  Eight caches of 32,768
// positions of 4 KB cut to half: 105 us, 17 of them the choice (2048 bins and three passes:
// 30, for the way of the bins across the cluster), 84 the moves (6.4 TB/s); three caches of
// 2049: 14 us.  Narrow rows keep less in flight, since a move is a warp's and values follow
// keys: moves of latent rows (1,152 bytes) 44 us, 3.4 TB/s, of 256 bytes 20, 1.7 TB/s.
#include <cooperative_groups.h>

#include "cache_common.cuh"
#include "tc.cuh"

namespace cg = cooperative_groups;

namespace csa {
namespace {

constexpr int EV_THREADS = 1024, EV_WARPS = EV_THREADS / 32;
constexpr int EV_KEYS = 16;      // of a thread, in registers
constexpr int EV_BINS = 256;
constexpr int EV_MOVE_WARPS = 8;

// A request's moves in the workspace: (destination, source) pairs, and their number.
struct Moves {
  int2 *list;      // [n_req][cap]
  int *n;          // [n_req]
  long long cap;   // half of a request's slots: every move has a hole and a source
};

__device__ __forceinline__ const float *mass_row(const csa_kv_evict_args &a, int b) {
  return reinterpret_cast<const float *>(reinterpret_cast<const uint8_t *>(a.mass) +
                                         b * a.mass_row_stride);
}
__device__ __forceinline__ float *mass_out_row(const csa_kv_evict_args &a, int b) {
  return reinterpret_cast<float *>(reinterpret_cast<uint8_t *>(a.mass_out) +
                                   b * a.mass_out_row_stride);
}

__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return 0;
  const uint32_t u = __float_as_uint(x == 0.f ? 0.f : x);
  return u >> 31 ? ~u : u | 0x80000000u;
}

// Keys above T and equal to it: in all, and before position n.
struct Count {
  int above, ties, above_n, ties_n;
};

// Cached: a thread's keys stay in registers (a CTA's stretch is at most EV_KEYS threads
// long).
template <bool Cached>
__global__ void __launch_bounds__(EV_THREADS) evict_plan_kernel(csa_kv_evict_args a, Moves mv) {
  __shared__ int hist[2][EV_BINS];  // (in turn: others still read the one before)
  __shared__ int warp_sum[EV_BINS / 32];
  __shared__ Count warp_n[EV_WARPS], cta_n;
  __shared__ int found[2];
  cg::cluster_group cluster = cg::this_cluster();
  tc::griddep_wait();
  tc::griddep_launch_dependents();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int C = cluster.num_blocks(), rank = cluster.block_rank();
  const int b = blockIdx.x / C;
  const int L = (int)max(min((long long)a.kv_len[b], (long long)a.max_blocks * kBlock), 0ll);
  const int n = min(L, max(a.budget[b], 0));
  const float *mass = mass_row(a, b);
  float *mass_out = a.mass_out && a.mass_out != a.mass ? mass_out_row(a, b) : nullptr;
  int *src_out = a.slot_src ? a.slot_src + (long long)b * a.max_blocks * kBlock : nullptr;
  // this warp's run of positions: per is a multiple of 32
  const long long all_warps = (long long)C * EV_WARPS;
  const int per = (int)((L + all_warps * 32 - 1) / (all_warps * 32)) * 32;
  const long long at = (long long)(rank * EV_WARPS + warp) * per;
  const int i0 = (int)min(at, (long long)L), i1 = (int)min(at + per, (long long)L);
  auto key_at = [&](int i) {
    return i < a.first || i >= L - a.recent ? 0xFF800000u : order_key(mass[i]);
  };
  const bool whole = n == 0 || n == L;  // (the same in the whole cluster)
  uint32_t prefix = 0;
  int need = n;
  uint32_t key[EV_KEYS];
  if (!whole) {
    if (Cached)
#pragma unroll
      for (int k = 0; k < EV_KEYS; ++k) key[k] = i0 + 32 * k + lane < i1 ? key_at(i0 + 32 * k + lane) : 0u;
    // every(f): f(position, key, inside) for this warp's run, 32 at a time
#define EV_EVERY(...)                                                        \
  if (Cached) {                                                              \
    _Pragma("unroll") for (int k = 0; k < EV_KEYS; ++k) {                    \
      if (i0 + 32 * k >= i1) break;                                          \
      const int i = i0 + 32 * k + lane;                                      \
      const bool in = i < i1;                                                \
      const uint32_t x = key[k];                                             \
      __VA_ARGS__                                                            \
    }                                                                        \
  } else {                                                                   \
    for (int i2 = i0; i2 < i1; i2 += 32) {                                   \
      const int i = i2 + lane;                                               \
      const bool in = i < i1;                                                \
      const uint32_t x = in ? key_at(i) : 0u;                                \
      __VA_ARGS__                                                            \
    }                                                                        \
  }
#pragma unroll 1
    for (int pass = 0; pass < 4; ++pass) {
      const int shift = 24 - 8 * pass;
      int *H = hist[pass & 1];
      if (tid < EV_BINS) H[tid] = 0;
      __syncthreads();
      EV_EVERY(if (in && (pass == 0 || x >> (shift + 8) == prefix >> (shift + 8)))
                   atomicAdd(&H[x >> shift & 255u], 1);)
      cluster.sync();
      // a bin a thread, the largest first, over the cluster; the bin where the count from
      // above reaches `need`
      int c = 0, x = 0;
      const int bin = EV_BINS - 1 - tid;
      if (tid < EV_BINS) {
        for (int r = 0; r < C; ++r) c += cluster.map_shared_rank(H, r)[bin];
        x = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, x, o);
          if (lane >= o) x += y;
        }
        if (lane == 31) warp_sum[warp] = x;
      }
      __syncthreads();
      if (tid < EV_BINS) {
        const int before =
            x - c + __reduce_add_sync(0xffffffffu, lane < warp ? warp_sum[lane] : 0);
        if (before < need && before + c >= need) found[0] = bin, found[1] = need - before;
      }
      __syncthreads();
      prefix |= (uint32_t)found[0] << shift;
      need = found[1];
    }
    // keys above T and ties, of the warp, the CTA, the CTAs before
    Count m = {0, 0, 0, 0};
    EV_EVERY(const uint32_t up = __ballot_sync(0xffffffffu, in && x > prefix);
             const uint32_t eq = __ballot_sync(0xffffffffu, in && x == prefix);
             const int room = n - (i - lane);
             const uint32_t early = room >= 32 ? ~0u : (room <= 0 ? 0u : (1u << room) - 1u);
             m.above += __popc(up); m.ties += __popc(eq); m.above_n += __popc(up & early);
             m.ties_n += __popc(eq & early);)
    if (lane == 0) warp_n[warp] = m;
    __syncthreads();
    if (warp == 0) {
      Count s = warp_n[lane];
      int v[4] = {s.above, s.ties, s.above_n, s.ties_n};
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = __reduce_add_sync(0xffffffffu, v[e]);
      if (lane == 0) cta_n = {v[0], v[1], v[2], v[3]};
    }
    cluster.sync();
    int a0 = 0, t0 = 0, k_a = 0, k_t = 0;
    for (int r = 0; r < C; ++r) {
      const Count s = *cluster.map_shared_rank(&cta_n, r);
      if (r < rank) a0 += s.above, t0 += s.ties;
      k_a += s.above_n, k_t += s.ties_n;
    }
    a0 += __reduce_add_sync(0xffffffffu, lane < warp ? warp_n[lane].above : 0);
    t0 += __reduce_add_sync(0xffffffffu, lane < warp ? warp_n[lane].ties : 0);
    const int kept_n = k_a + min(k_t, need);  // kept positions that stay
    int2 *list = mv.list + b * mv.cap;
    EV_EVERY(const uint32_t under = (1u << lane) - 1u;
             const uint32_t up = __ballot_sync(0xffffffffu, in && x > prefix);
             const uint32_t eq = __ballot_sync(0xffffffffu, in && x == prefix);
             const int tie = t0 + __popc(eq & under);
             const bool kept = in && (x > prefix || (x == prefix && tie < need));
             const int before = a0 + __popc(up & under) + min(tie, need);  // kept ones
             if (in && !kept && i < n) list[i - before].x = i;
             if (kept && i >= n) list[before - kept_n].y = i;
             if (kept && i < n) {
               if (src_out) src_out[i] = i;
               if (mass_out) mass_out[i] = mass[i];
             } a0 += __popc(up);
             t0 += __popc(eq);)
    if (rank == 0 && tid == 0) mv.n[b] = n - kept_n;
  } else {
    for (int i = i0 + lane; i < min(i1, n); i += 32) {
      if (src_out) src_out[i] = i;
      if (mass_out) mass_out[i] = mass[i];
    }
    if (rank == 0 && tid == 0) mv.n[b] = 0;
  }
#undef EV_EVERY
  cluster.sync();  // every CTA has read kv_len (kv_len_out may be it) and the others' counts
  if (rank == 0 && tid == 0) a.kv_len_out[b] = n;
}

// One row: `vecs` 16-byte pieces a head, all heads; four pieces of a lane in flight.
__device__ __forceinline__ void copy_row(uint8_t *to, const uint8_t *from, int vecs, int heads,
                                         long long head_stride, int lane) {
  const int total = vecs * heads;
  const bool dense = head_stride == vecs * 16;
  for (int v0 = lane; v0 < total; v0 += 128) {
    uint4 x[4];
    long long off[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int v = v0 + 32 * k;
      off[k] = dense ? v * 16ll : v / vecs * head_stride + v % vecs * 16;
      if (v < total) x[k] = *reinterpret_cast<const uint4 *>(from + off[k]);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (v0 + 32 * k < total) *reinterpret_cast<uint4 *>(to + off[k]) = x[k];
  }
}

// A warp a move: the row of every pool, its mass and its old position.
__global__ void __launch_bounds__(32 * EV_MOVE_WARPS)
    evict_move_kernel(csa_kv_evict_args a, Moves mv, int per_req) {
  tc::griddep_wait();
  tc::griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int b = blockIdx.x / per_req, part = blockIdx.x - b * per_req;
  const int H = mv.n[b];
  const float *mass = mass_row(a, b);
  float *mass_out = a.mass_out ? mass_out_row(a, b) : nullptr;
  int *src_out = a.slot_src ? a.slot_src + (long long)b * a.max_blocks * kBlock : nullptr;
  const int2 *list = mv.list + b * mv.cap;
  const int step = per_req * EV_MOVE_WARPS;
  int m = part * EV_MOVE_WARPS + (threadIdx.x >> 5);
  int2 e = m < H ? list[m] : make_int2(0, 0);
  for (; m < H; m += step) {
    const long long to = page_row(a.block_table, a.max_blocks, a.n_blocks, b, e.x, a.status_dev);
    const long long from = page_row(a.block_table, a.max_blocks, a.n_blocks, b, e.y, a.status_dev);
    const int2 next = m + step < H ? list[m + step] : make_int2(0, 0);
    if (lane == 0) {
      if (mass_out) mass_out[e.x] = mass[e.y];
      if (src_out) src_out[e.x] = e.y;
    }
    if (to >= 0 && from >= 0) {
      uint8_t *k = static_cast<uint8_t *>(a.k_pool), *v = static_cast<uint8_t *>(a.v_pool);
      copy_row(k + pool_offset(to, a.k_page_stride, a.k_token_stride),
               k + pool_offset(from, a.k_page_stride, a.k_token_stride), a.k_dim / 8, a.n_heads,
               a.k_head_stride, lane);
      if (v)
        copy_row(v + pool_offset(to, a.v_page_stride, a.v_token_stride),
                 v + pool_offset(from, a.v_page_stride, a.v_token_stride), a.v_dim / 8, a.n_heads,
                 a.v_head_stride, lane);
    }
    e = next;
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
  // a CTA for every 4096 slots, eight at most
  const long long cols = (long long)a.max_blocks * kBlock;
  int C = 1;
  while (C < 8 && (long long)C * 4096 < cols) C *= 2;
  if ((long long)a.n_req * C > 0x7FFFFFFF) return cudaErrorInvalidValue;
  const dim3 grid((unsigned)(a.n_req * C));
  launch_begin(CSA_K_EVICT_PLAN, s);
  cudaError_t e =
      cols <= (long long)C * EV_THREADS * EV_KEYS
          ? launch_kernel(evict_plan_kernel<true>, grid, dim3(EV_THREADS), 0, s, C, false, a, mv)
          : launch_kernel(evict_plan_kernel<false>, grid, dim3(EV_THREADS), 0, s, C, false, a, mv);
  launch_end(CSA_K_EVICT_PLAN, s);
  if (e != cudaSuccess) return e;
  // eight CTAs an SM over all requests, as far as a request has moves for them
  long long per = (8ll * sm_count() + a.n_req - 1) / a.n_req;
  const long long most = (mv.cap + EV_MOVE_WARPS - 1) / EV_MOVE_WARPS;
  per = per < most ? per : most;
  if (a.n_req * per > 0x7FFFFFFF) return cudaErrorInvalidValue;
  launch_begin(CSA_K_EVICT_MOVE, s);
  e = launch_kernel(evict_move_kernel, dim3((unsigned)(a.n_req * per)), dim3(32 * EV_MOVE_WARPS), 0, s,
                    0, false, a, mv, (int)per);
  launch_end(CSA_K_EVICT_MOVE, s);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace csa
