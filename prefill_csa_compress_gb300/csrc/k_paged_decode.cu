// Attention of few rows per request over a paged key/value cache
// (csa_paged_attn): a stream of pages at HBM speed.
//
// An item is the rows of one request that share a key/value head's pages: up to
// 16 MT (row, head) pairs.  A page of K and V costs 512 D bytes and 16 MT x 128
// x D x 4 operations, far below the tensor cores' share, so the pages bound the
// time and the products run as warp-level m16n8k16 (the 128-row tiles of
// tcgen05 would be seven eighths padding at 16 pairs):
//   S = Q K^T   warp w takes keys 16 w .. 16 w + 15 of the page
//   P = 2^(S scale log2(e) - ref), one reference per pair, shared by the CTA;
//               the item's first page sets it; it moves (and O is rescaled) only
//               when a logit exceeds it by more than 2^8, which a barrier votes on
//   O += P V    warp w takes D / 8 output channels, P through shared memory,
//               so no warp holds a partial O and an item ends without a merge.
// A ninth warp keeps a ring of pages in flight by TMA.
//
// All pages of all items are one list, cut into equal shares, one per CTA: ragged
// contexts and few rows load every SM alike.  A share that starts or ends inside an
// item leaves a part in the workspace, at most two per CTA, which
// paged_join_kernel puts together in page order.  One CTA per SM keeps 192 KB of
// pages in flight; for heads of 64, where a page is half as long and latency shows,
// two keep 96 KB each (64 requests over 1000 positions of 8 x 64 47 -> 38 us, 32
// to 16,384 of 4 x 64 104 -> 92; 4 x 2 rows at 131,072 194 -> 198).
// 32 requests of one row with contexts to 16,384 (64 heads on 8 of 128): 207 us, 6.6
// TB/s; 4 x 2 rows at 131,072 positions: 311 us, 6.9 TB/s, the rate of a plain copy;
// of 64 channels (rows of 128 bytes, 1 KB apart): 198 us, 5.4 TB/s.  A page takes a CTA
// 2,400 cycles, an item of one page 6,000 (its logits 900, the references 500, the
// product 1,100, the sums and the output 1,600).
#include <cuda.h>
#include <cudaTypedefs.h>

#include "attn_common.cuh"
#include "csa_internal.cuh"
#include "paged_common.cuh"
#include "tc.cuh"

namespace csa {
namespace {

using paged::DecodeParts;

constexpr int PD_WARPS = 8, PD_THREADS = 32 * (PD_WARPS + 1);
constexpr int PD_BAR = 1;
constexpr float kMove = 8.f;

template <int D, int MT, int ST>
struct Cfg {
  static constexpr int CHUNKS = D / 64;
  static constexpr int TILE = CHUNKS * 16384;  // bytes of a page of K (or V)
  static constexpr int STAGES = ST;
  static constexpr int CTAS = ST * 2 * TILE <= 98304 ? 2 : 1;  // an SM
  static constexpr int PAIRS = 16 * MT;
  static constexpr int Q_STRIDE = D + 8, P_STRIDE = kBlock + 8;  // elements, odd in 16 bytes
  static constexpr int OFF_Q = STAGES * 2 * TILE;
  static constexpr int OFF_P = OFF_Q + PAIRS * Q_STRIDE * 2;
  static constexpr int OFF_MISC = OFF_P + PAIRS * P_STRIDE * 2;
};

// The list of items, by row, behind everything else in shared memory.
struct Plan {
  long long *before;  // pages of all items of earlier rows; and of all rows
  int *req;           // -1: padding, or no such request
  int *pages;         // of an item that starts at this row, or 0
  int *first;         // its first page
  int *lo, *hi;       // positions that the row sees

  __device__ Plan(void *at, int n) {
    before = static_cast<long long *>(at);
    req = reinterpret_cast<int *>(before + n + 1);
    pages = req + n;
    first = pages + n;
    lo = first + n;
    hi = lo + n;
  }
  static constexpr int bytes(int n) { return 8 * (n + 1) + 5 * 4 * n; }
};

template <int PAIRS>
struct Misc {
  uint64_t full[6], empty[6];
  int phys[6];  // the page in the stage, -1: unmapped
  int abort;
  uint32_t bad[2][4];  // keys of the page whose values are not finite (pages in turn)
  int lo[2][PAIRS], hi[2][PAIRS];  // what a pair sees (items in turn)
  float top[PD_WARPS][PAIRS], sum[PD_WARPS][PAIRS];
};

// Shared memory of a CTA for a call of n rows.
template <int D, int MT, int ST>
constexpr int smem_bytes(int n) {
  return Cfg<D, MT, ST>::OFF_MISC + (int)sizeof(Misc<16 * MT>) + Plan::bytes(n);
}

__device__ __forceinline__ bool pd_wait(uint64_t *bar, uint32_t parity, volatile int *abort,
                                        uint32_t *status) {
  if (tc::mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = tc::global_ns();
  for (uint32_t i = 1;; ++i) {
    if (tc::mbar_try_wait(bar, parity)) return true;
    if ((i & 255u) == 0) {
      if (*abort) return false;
      if (tc::global_ns() - t0 > 2000000000ull) {
        *abort = 1;
        flag(status, CSA_DEV_TIMEOUT);
        return false;
      }
    }
  }
}

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// c += a b: a 16 x 16 (row major), b 16 x 8, BF16, FP32 sums
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int D, int MT, int ST>
__global__ void __launch_bounds__(PD_THREADS, (Cfg<D, MT, ST>::CTAS))
    paged_decode_kernel(csa_paged_attn_args a, DecodeParts parts,
                        const __grid_constant__ CUtensorMap kmap,
                        const __grid_constant__ CUtensorMap vmap) {
  using C = Cfg<D, MT, ST>;
  constexpr int PAIRS = C::PAIRS;
  // (a kernel without static shared memory gets it 1024-byte aligned; one that did
  // not would stop before touching it)
  extern __shared__ __align__(1024) uint8_t sm[];
  auto *M = reinterpret_cast<Misc<PAIRS> *>(sm + C::OFF_MISC);
  const Plan plan(M + 1, a.n_rows);
  tc::griddep_wait();
  tc::griddep_launch_dependents();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tc::smem_u32(sm) & 1023u) {
    if (tid == 0) flag(a.status_dev, CSA_DEV_TIMEOUT);
    return;
  }
  volatile int *abort = &M->abort;
  const int g = a.n_heads / a.n_kv_heads;
  const int gt = min(g, PAIRS), rows = PAIRS / gt;       // heads and rows of an item
  const int head_tiles = (g + gt - 1) / gt, subs = a.n_kv_heads * head_tiles;

  // ---- the list of items, the same in every CTA: what each row sees ...
  for (int t = tid; t < a.n_rows; t += PD_THREADS) {
    const int b = a.row_req[t], p = a.row_pos[t];
    int lo = 0, hi = 0;
    if (b >= a.n_req && blockIdx.x == 0) flag(a.status_dev, CSA_DEV_BAD_POS);
    if (b >= 0 && b < a.n_req) paged::visible_range(a, a.kv_len[b], p, lo, hi);
    plan.req[t] = b < a.n_req ? b : -1;
    plan.lo[t] = lo;
    plan.hi[t] = hi;
  }
  if (tid == 0) {
    for (int i = 0; i < C::STAGES; ++i) {
      tc::mbar_init(&M->full[i], 1);
      tc::mbar_init(&M->empty[i], PD_WARPS);
    }
    M->abort = 0;
    tc::mbar_fence_init();
  }
  if (tid < 8) M->bad[tid >> 2][tid & 3] = 0;
  __syncthreads();
  // ... and, for each row t that starts an item, the pages that it and the rows
  // after it see: up to the next multiple of `rows`, while they are the same request's
  for (int t = tid; t < a.n_rows; t += PD_THREADS) {
    const int b = plan.req[t];
    int n_pages = 0, first = 0;
    if (b >= 0 && (t % rows == 0 || plan.req[t - 1] != b)) {
      int lo = 0x7FFFFFFF, hi = 0, n = 0;
      for (; n == 0 || (t + n < a.n_rows && (t + n) % rows != 0 && plan.req[t + n] == b); ++n)
        if (plan.lo[t + n] < plan.hi[t + n]) {
          lo = min(lo, plan.lo[t + n]);
          hi = max(hi, plan.hi[t + n]);
        }
      if (lo < hi) {
        first = lo / kBlock;
        n_pages = (hi - 1) / kBlock - first + 1;
      } else if (blockIdx.x == t % gridDim.x) {  // nothing to see: the join writes the rows
        for (int i = 0; i < n * subs; ++i)
          parts.item[(long long)t * subs + i] = make_int4(-1, -1, t, 0);
      }
    }
    plan.pages[t] = n_pages;
    plan.first[t] = first;
  }
  __syncthreads();
  if (warp == 0) {
    long long sum = 0;
    for (int t0 = 0; t0 < a.n_rows; t0 += 32) {
      const int t = t0 + lane;
      const long long mine = t < a.n_rows ? (long long)plan.pages[t] * subs : 0;
      long long x = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (t < a.n_rows) plan.before[t] = sum + x - mine;
      sum += __shfl_sync(0xffffffffu, x, 31);
    }
    if (lane == 0) plan.before[a.n_rows] = sum;
  }
  __syncthreads();
  const long long W = plan.before[a.n_rows];
  const long long N = W < gridDim.x ? W : gridDim.x;
  if (blockIdx.x >= N) return;
  const long long w0 = blockIdx.x * W / N, w1 = (blockIdx.x + 1) * W / N;
  int row0;  // the row whose items hold page w0
  {
    int l = 0, h = a.n_rows;
    while (h - l > 1) {
      const int mid = (l + h) >> 1;
      if (plan.before[mid] <= w0)
        l = mid;
      else
        h = mid;
    }
    row0 = l;
  }
  const int sub0 = (int)((w0 - plan.before[row0]) / plan.pages[row0]);
  const int pa0 = (int)(w0 - plan.before[row0] - (long long)sub0 * plan.pages[row0]);
  // the item behind item sub of row t (the last row is followed by none)
  auto next_item = [&](int &t, int &sub) {
    if (++sub < subs) return;
    sub = 0;
    do
      ++t;
    while (t < a.n_rows && plan.pages[t] == 0);
  };

  if (warp == PD_WARPS) {
    // ================================================================ loads
    uint32_t it = 0;
    bool ok = true;
    int t = row0, sub = sub0, pa = pa0;
    for (long long w = w0; w < w1 && ok;) {
      const int P = plan.pages[t];
      const int pb = (int)min((long long)P, pa + (w1 - w));
      const int kvh = sub / head_tiles;
      const int32_t *table =
          a.block_table + (long long)plan.req[t] * a.max_blocks + plan.first[t];
      int entry = 0;
      for (int p = pa; p < pb && ok; ++p, ++it) {
        if (((p - pa) & 31) == 0) entry = p + lane < pb ? table[p + lane] : 0;
        const int phys = __shfl_sync(0xffffffffu, entry, (p - pa) & 31);
        const bool there = phys >= 0 && phys < a.n_blocks;
        const int st = it % C::STAGES;
        ok = __all_sync(0xffffffffu, pd_wait(&M->empty[st], ((it / C::STAGES) & 1) ^ 1, abort,
                                             a.status_dev));
        if (!ok) break;
        if (lane == 0) {
          M->phys[st] = there ? phys : -1;
          if (there) {
            uint8_t *dst = sm + st * 2 * C::TILE;
            tc::mbar_arrive_expect_tx(&M->full[st], 2 * C::TILE);
#pragma unroll
            for (int kv = 0; kv < 2; ++kv)
              for (int c = 0; c < C::CHUNKS; ++c)
                paged::tma_load_4d(dst + kv * C::TILE + c * 16384, kv ? &vmap : &kmap, c * 64, kvh,
                                   0, phys, &M->full[st]);
          } else {
            flag(a.status_dev, CSA_DEV_BAD_BLOCK);
            tc::mbar_arrive(&M->full[st]);
          }
        }
        __syncwarp();
      }
      w += pb - pa;
      pa = 0;
      next_item(t, sub);
    }
    if (*abort)  // whatever was asked for has landed before the CTA retires
      for (uint32_t k = it > C::STAGES ? it - C::STAGES : 0; k < it; ++k)
        tc::mbar_wait(&M->full[k % C::STAGES], (k / C::STAGES) & 1, 50000000ull);
    return;
  }

  // ================================================================ products and softmax
  const uint32_t kv_s = tc::smem_u32(sm), q_s = tc::smem_u32(sm + C::OFF_Q),
                 p_s = tc::smem_u32(sm + C::OFF_P);
  __nv_bfloat16 *Ps = reinterpret_cast<__nv_bfloat16 *>(sm + C::OFF_P);
  const float sl2 = a.softmax_scale * paged::kLog2e;
  const int mi = lane >> 3, ri = lane & 7;  // ldmatrix: matrix and row of this lane's address
  const int fr = lane >> 2, fc = (lane & 3) * 2;  // fragment row and column
  constexpr int NV = D / 64;  // 8-channel tiles of O per warp
  // Item sub of row t, from its page pa (page w of the list) on, and this thread's
  // 16-byte pieces of its q; rows and heads that it lacks are zero.
  struct Item {
    int t, sub, pa, pb, h0, n_rows, n_heads;
  };
  constexpr int QN = PAIRS * (D / 8) / (32 * PD_WARPS);  // pieces a thread
  auto item_at = [&](long long w, int t, int sub, int pa) {
    Item I;
    I.t = t;
    I.sub = sub;
    I.pa = pa;
    I.pb = (int)min((long long)plan.pages[t], pa + (w1 - w));
    const int kvh = head_tiles == 1 ? sub : sub / head_tiles;
    I.h0 = kvh * g + (sub - kvh * head_tiles) * gt;
    I.n_heads = min(gt, (kvh + 1) * g - I.h0);  // the last head tile may be short
    I.n_rows = 1;
    while (t + I.n_rows < a.n_rows && (t + I.n_rows) % rows != 0 &&
           plan.req[t + I.n_rows] == plan.req[t])
      ++I.n_rows;
    return I;
  };
  auto read_q = [&](const Item &I, uint4(&q)[QN > 0 ? QN : 1]) {
#pragma unroll
    for (int u = 0; u < (QN > 0 ? QN : 1); ++u) {
      const int i = u * 32 * PD_WARPS + tid, m = i / (D / 8), c = i % (D / 8);
      const int r = m / gt, h = m % gt;
      q[u] = make_uint4(0, 0, 0, 0);
      if (m < PAIRS && r < I.n_rows && h < I.n_heads)
        q[u] = *reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(a.q) +
                                                (I.t + r) * a.q_row_stride +
                                                (long long)(I.h0 + h) * D * 2 + c * 16);
    }
  };
  // q and what each pair (row i / gt, head i % gt) sees, for the item's first page
  auto set_item = [&](const Item &I, const uint4(&q)[QN > 0 ? QN : 1], int turn) {
#pragma unroll
    for (int u = 0; u < (QN > 0 ? QN : 1); ++u) {
      const int i = u * 32 * PD_WARPS + tid, m = i / (D / 8), c = i % (D / 8);
      if (m < PAIRS) *reinterpret_cast<uint4 *>(sm + C::OFF_Q + m * C::Q_STRIDE * 2 + c * 16) = q[u];
    }
    if (tid < PAIRS) {
      const int r = tid / gt, h = tid % gt;
      const bool on = r < I.n_rows && h < I.n_heads;
      M->lo[turn][tid] = on ? plan.lo[I.t + r] : 0;
      M->hi[turn][tid] = on ? plan.hi[I.t + r] : 0;
    }
  };
  uint32_t it = 0;
  bool ok = true;
  int turn = 0;
  Item I = item_at(w0, row0, sub0, pa0);
  uint4 q_next[QN > 0 ? QN : 1];
  read_q(I, q_next);
  set_item(I, q_next, turn);
  tc::bar_sync(PD_BAR, 32 * PD_WARPS);
  for (long long w = w0; w < w1 && ok; turn ^= 1) {
    const int t = I.t, sub = I.sub, pa = I.pa, pb = I.pb, h0 = I.h0, n_heads = I.n_heads;
    const int n_rows = I.n_rows, P = plan.pages[t], first = plan.first[t];
    const int kvh = head_tiles == 1 ? sub : sub / head_tiles;
    const bool more = w + (pb - pa) < w1;
    // positions that every pair of the item sees (padding pairs aside)
    int all_lo = 0, all_hi = 0x7FFFFFFF;
    for (int r = 0; r < n_rows; ++r) {
      all_lo = max(all_lo, plan.lo[t + r]);
      all_hi = min(all_hi, max(plan.lo[t + r], plan.hi[t + r]));
    }
    float sink[MT][2];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int h = (i * 16 + u * 8 + fr) % gt;
        sink[i][u] = a.sink && h < n_heads ? a.sink[h0 + h] : -INFINITY;
      }
    // the next item's q is on its way during this one
    if (more) {
      int t_next = t, sub_next = sub;
      next_item(t_next, sub_next);
      I = item_at(w + (pb - pa), t_next, sub_next, 0);
      read_q(I, q_next);
    }
    uint32_t qf[MT == 1 ? D / 16 : 1][4];
    if constexpr (MT == 1) {
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
        ldsm4(q_s + (((mi & 1) * 8 + ri) * C::Q_STRIDE + k * 16 + (mi >> 1) * 8) * 2, qf[k]);
    }
    float o[MT][NV][4] = {}, l[MT][2] = {}, refs[MT][2];
#pragma unroll
    for (int i = 0; i < MT; ++i) refs[i][0] = refs[i][1] = -INFINITY;

    for (int p = pa; p < pb; ++p, ++it) {
      const int st = it % C::STAGES;
      ok = pd_wait(&M->full[st], (it / C::STAGES) & 1, abort, a.status_dev) && ok;
      const uint32_t ks = kv_s + st * 2 * C::TILE, vs = ks + C::TILE;
      const int phys = M->phys[st], base = (first + p) * kBlock;
      const bool mixed = phys < 0 || base < all_lo || all_hi - base < kBlock;

      // ---- S = Q K^T over this warp's 16 keys
      float x[MT][2][4] = {};
      {
        const int key = warp * 16 + (mi >> 1) * 8 + ri;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const int c = 2 * k + (mi & 1);
          uint32_t kf[4];
          ldsm4(ks + (c >> 3) * 16384 + key * 128 + (((c & 7) ^ ri) << 4), kf);
#pragma unroll
          for (int i = 0; i < MT; ++i) {
            if constexpr (MT > 1) {
              uint32_t q1[4];
              ldsm4(q_s + ((i * 16 + (mi & 1) * 8 + ri) * C::Q_STRIDE + k * 16 + (mi >> 1) * 8) * 2,
                    q1);
              mma16816(x[i][0], q1, kf[0], kf[1]);
              mma16816(x[i][1], q1, kf[2], kf[3]);
            } else {
              mma16816(x[i][0], qf[k], kf[0], kf[1]);
              mma16816(x[i][1], qf[k], kf[2], kf[3]);
            }
          }
        }
      }
      // ---- logits in log2 units; what a pair does not see is -inf
      bool exceeds = false;
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int m = i * 16 + u * 8 + fr;
          const float ref = refs[i][u];
          int lo = 0, hi = kBlock;
          if (mixed) {
            lo = M->lo[turn][m] - base;
            hi = phys < 0 ? 0 : M->hi[turn][m] - base;
          }
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float &y = x[i][n][2 * u + e];
              const int c = warp * 16 + n * 8 + fc + e;
              y = mixed && (c < lo || c >= hi) ? -INFINITY : y * sl2;
              exceeds |= y > ref + kMove;  // with ref = -inf: any logit above -inf
            }
        }
      if (mixed) {
        // this warp's 16 rows of V: rows that nobody sees and values that are
        // not finite become zero, the latter are reported
        const int row = warp * 16 + (lane & 15), half = lane >> 4;
        uint4 *v = reinterpret_cast<uint4 *>(sm + st * 2 * C::TILE + C::TILE + row * 128);
        uint32_t bad = 0;
#pragma unroll
        for (int q = 0; q < C::CHUNKS * 4; ++q) {
          const uint4 y = v[(q >> 2) * 1024 + (((q & 3) + half * 4 + lane) & 7)];
          bad |= paged::not_finite2(y.x) | paged::not_finite2(y.y) | paged::not_finite2(y.z) |
                 paged::not_finite2(y.w);
        }
        // both halves of a row rotate through its eight pieces
        bad |= __shfl_xor_sync(0xffffffffu, bad, 16);
        if (bad) {
          for (int q = 0; q < C::CHUNKS * 4; ++q)
            v[(q >> 2) * 1024 + (q & 3) + half * 4] = make_uint4(0, 0, 0, 0);
          tc::fence_async_shared();
          if (half == 0 && phys >= 0) atomicOr(&M->bad[it & 1][row >> 5], 1u << (row & 31));
        }
      }
      // ---- references: set by the item's first page, and moved when a logit
      // exceeds one by too much, to the pairs' largest logits of the page
      const bool start = p == pa;
      if (start || tc::bar_or(PD_BAR, 32 * PD_WARPS, exceeds)) {
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            float top = fmaxf(fmaxf(x[i][0][2 * u], x[i][0][2 * u + 1]),
                              fmaxf(x[i][1][2 * u], x[i][1][2 * u + 1]));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            if ((lane & 3) == 0) M->top[warp][i * 16 + u * 8 + fr] = top;
          }
        tc::bar_sync(PD_BAR, 32 * PD_WARPS);
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int m = i * 16 + u * 8 + fr;
            float top = M->top[0][m];
#pragma unroll
            for (int q = 1; q < PD_WARPS; ++q) top = fmaxf(top, M->top[q][m]);
            const float ref = refs[i][u];
            if (top > ref + kMove) {
              const float f = ref > -INFINITY ? exp2f(ref - top) : 1.f;
              refs[i][u] = top;
              l[i][u] *= f;
#pragma unroll
              for (int n = 0; n < NV; ++n) {
                o[i][n][2 * u] *= f;
                o[i][n][2 * u + 1] *= f;
              }
            }
          }
      }
      if (tid < 4) M->bad[~it & 1][tid] = 0;  // for the next page
      // ---- P, rounded to BF16 for the product; the sums take it unrounded
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int m = i * 16 + u * 8 + fr;
          const float ref = refs[i][u], r0 = ref == -INFINITY ? 0.f : ref;
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            const float y0 = attn::exp2_sfu(x[i][n][2 * u] - r0);
            const float y1 = attn::exp2_sfu(x[i][n][2 * u + 1] - r0);
            l[i][u] += y0 + y1;
            *reinterpret_cast<uint32_t *>(Ps + m * C::P_STRIDE + warp * 16 + n * 8 + fc) =
                attn::pack2(y0, y1);
          }
        }
      // every wait of the page came through, or all stop
      if (tc::bar_or(PD_BAR, 32 * PD_WARPS, !ok)) {
        ok = false;
        break;
      }
      // ---- O += P V over this warp's channels
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        uint32_t vf[4];
        if constexpr (NV == 2) {
          const int key = k * 16 + (mi & 1) * 8 + ri, c = warp * 2 + (mi >> 1);
          ldsm4t(vs + (c >> 3) * 16384 + key * 128 + (((c & 7) ^ ri) << 4), vf);
        } else {
          const int key = (k & ~1) * 16 + mi * 8 + ri;  // two steps' keys at once
          ldsm4t(vs + key * 128 + ((warp ^ ri) << 4), vf);
        }
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          uint32_t pf[4];
          ldsm4(p_s + ((i * 16 + (mi & 1) * 8 + ri) * C::P_STRIDE + k * 16 + (mi >> 1) * 8) * 2, pf);
          if constexpr (NV == 2) {
            mma16816(o[i][0], pf, vf[0], vf[1]);
            mma16816(o[i][1], pf, vf[2], vf[3]);
          } else {
            mma16816(o[i][0], pf, vf[(k & 1) * 2], vf[(k & 1) * 2 + 1]);
          }
        }
      }
      if (mixed) {
        // values that are not finite go to the pairs that see them
#pragma unroll 1
        for (int w4 = 0; w4 < 4; ++w4)
#pragma unroll 1
          for (uint32_t bits = M->bad[it & 1][w4]; bits; bits &= bits - 1) {
            const int c = 32 * w4 + __ffs(bits) - 1;
            const __nv_bfloat16 *v = reinterpret_cast<const __nv_bfloat16 *>(
                static_cast<const uint8_t *>(a.v_pool) + phys * a.v_page_stride +
                c * a.v_token_stride + kvh * a.v_head_stride);
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
              for (int u = 0; u < 2; ++u) {
                const int m = i * 16 + u * 8 + fr;
                if (c + base < M->lo[turn][m] || c + base >= M->hi[turn][m]) continue;
                const float pr = __bfloat162float(Ps[m * C::P_STRIDE + c]);
#pragma unroll
                for (int n = 0; n < NV; ++n)
#pragma unroll
                  for (int e = 0; e < 2; ++e)
                    o[i][n][2 * u + e] +=
                        pr * __bfloat162float(v[warp * (D / 8) + n * 8 + fc + e]);
              }
          }
      }
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&M->empty[st]);
    }
    if (!ok) break;

    // ---- the sums of all warps' keys, then the result or a part of it; the next
    // item's q takes this one's place (all warps are past their last logits)
    if (more) set_item(I, q_next, turn ^ 1);
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        l[i][u] += __shfl_xor_sync(0xffffffffu, l[i][u], 1);
        l[i][u] += __shfl_xor_sync(0xffffffffu, l[i][u], 2);
        if ((lane & 3) == 0) M->sum[warp][i * 16 + u * 8 + fr] = l[i][u];
      }
    tc::bar_sync(PD_BAR, 32 * PD_WARPS);
    const bool whole = pa == 0 && pb == P;
    const long long slot = 2 * (long long)blockIdx.x + (pa == 0 ? 1 : 0);
    if (pa == 0 && tid < n_rows) {
      // which CTAs hold the item, for the join
      int last = blockIdx.x;
      if (pb < P)
        last = (int)(((plan.before[t] + (long long)(sub + 1) * P) * N - 1) / W);
      parts.item[(long long)(t + tid) * subs + sub] = make_int4((int)blockIdx.x, last, t, 0);
    }
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int m = i * 16 + u * 8 + fr, r = m / gt, h = m % gt;
        if (r >= n_rows || h >= n_heads) continue;
        float sum = M->sum[0][m];
#pragma unroll
        for (int q = 1; q < PD_WARPS; ++q) sum += M->sum[q][m];
        const float ref = refs[i][u];
        const bool zero = ref == -INFINITY && sum == 0.f;
        if (whole) {
          const long long row = (long long)(t + r) * a.n_heads + h0 + h;
          const paged::Joined J = paged::finish(ref, sum, sink[i][u]);
          uint32_t *out = reinterpret_cast<uint32_t *>(static_cast<__nv_bfloat16 *>(a.out) + row * D +
                                                       warp * (D / 8) + fc);
#pragma unroll
          for (int n = 0; n < NV; ++n)
            out[n * 4] = zero ? 0u : attn::pack2(o[i][n][2 * u] * J.inv, o[i][n][2 * u + 1] * J.inv);
          if (a.lse && warp == 0 && fc == 0) a.lse[row] = J.lse;
        } else {
          float *out = parts.o + (slot * PAIRS + m) * D + warp * (D / 8) + fc;
#pragma unroll
          for (int n = 0; n < NV; ++n)
            *reinterpret_cast<float2 *>(out + n * 8) =
                make_float2(o[i][n][2 * u], o[i][n][2 * u + 1]);
          if (warp == 0 && fc == 0) parts.ml[slot * PAIRS + m] = make_float2(ref, sum);
        }
      }
    w += pb - pa;
  }
}

// out and lse of the rows whose items were cut, and of those that see nothing.
// One CTA per (row, head): warp s takes every fourth part, lanes the channels.
template <int D>
__global__ void __launch_bounds__(128)
    paged_join_kernel(csa_paged_attn_args a, DecodeParts parts, int pairs, int n_ctas) {
  tc::griddep_wait();
  tc::griddep_launch_dependents();
  constexpr int E = D / 32, NW = 4;
  __shared__ float sh_o[NW][D], sh_l[NW];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long row = blockIdx.x;
  const int t = (int)(row / a.n_heads), h = (int)(row - (long long)t * a.n_heads);
  const int g = a.n_heads / a.n_kv_heads, gt = min(g, pairs), kvh = h / g;
  const int head_tiles = (g + gt - 1) / gt, sub = kvh * head_tiles + h % g / gt;
  // (three waits for memory in all: these, the references, the outputs)
  const int4 it = parts.item[(long long)t * (a.n_kv_heads * head_tiles) + sub];
  const int b = a.row_req[t];
  const float sink = a.sink ? a.sink[h] : -INFINITY;
  if (b < 0 || b >= a.n_req) return;      // (item is not set there)
  if (it.x == it.y && it.x >= 0) return;  // written whole
  // (an item that its CTA gave up before, after a wait that ran out, is not set)
  if (it.y >= n_ctas || it.z > t || it.z <= t - pairs / gt) return;
  const int m = (t - it.z) * gt + h % g % gt, n = it.x < 0 ? 0 : it.y - it.x + 1;
  auto slot = [&](int s) { return (2ll * (it.x + s) + (s == 0 ? 1 : 0)) * pairs + m; };
  // the part with the largest reference first, then the sums in part order
  float ref = -INFINITY;
  for (int s = lane; s < n; s += 32) ref = fmaxf(ref, parts.ml[slot(s)].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) ref = fmaxf(ref, __shfl_xor_sync(0xffffffffu, ref, o));
  float acc[E] = {}, l = 0.f;
#pragma unroll 4
  for (int s = warp; s < n; s += NW) {
    const float2 ml = parts.ml[slot(s)];
    float o[E];
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = parts.o[slot(s) * D + lane * E + e];
    if (ml.x == -INFINITY && ml.y == 0.f) continue;  // nothing was seen there
    const float w = ml.x == -INFINITY ? ml.y : exp2f(ml.x - ref);  // (l is NaN there)
    l += w * ml.y;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] += w * o[e];
  }
#pragma unroll
  for (int e = 0; e < E; ++e) sh_o[warp][lane * E + e] = acc[e];
  if (lane == 0) sh_l[warp] = l;
  __syncthreads();
  if (warp != 0) return;
  l = (sh_l[0] + sh_l[1]) + (sh_l[2] + sh_l[3]);
  const paged::Joined J = paged::finish(ref, l, sink);
  const bool zero = ref == -INFINITY && l == 0.f;
  __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(a.out) + row * D + lane * E;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int d = lane * E + e;
    const float v = (sh_o[0][d] + sh_o[1][d]) + (sh_o[2][d] + sh_o[3][d]);
    out[e] = __float2bfloat16_rn(zero ? 0.f : v * J.inv);
  }
  if (a.lse && lane == 0) a.lse[row] = J.lse;
}

template <int D, int MT, int ST>
cudaError_t launch(const csa_paged_attn_args &a, const DecodeParts &parts, int ctas,
                   cudaStream_t s) {
  using C = Cfg<D, MT, ST>;
  CUtensorMap kmap, vmap;
  if (!paged::encode_pools(a, &kmap, &vmap)) return cudaErrorInvalidValue;
  constexpr int most = smem_bytes<D, MT, ST>(paged::kDecodeRows);
  static_assert(most <= 227 * 1024, "shared memory");
  static_assert(sizeof(Misc<C::PAIRS>) % 8 == 0 && C::OFF_MISC % 8 == 0, "alignment");
  int dev = 0;
  cudaGetDevice(&dev);
  static bool attr[64] = {};
  if (dev < 0 || dev >= 64 || !attr[dev]) {
    const cudaError_t e = cudaFuncSetAttribute(
        paged_decode_kernel<D, MT, ST>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) attr[dev] = true;
  }
  launch_begin(CSA_K_PAGED_ATTN, s);
  cudaError_t e = launch_kernel(paged_decode_kernel<D, MT, ST>, dim3(ctas), dim3(PD_THREADS),
                                smem_bytes<D, MT, ST>(a.n_rows), s, 0, false, a, parts, kmap, vmap);
  launch_end(CSA_K_PAGED_ATTN, s);
  if (e != cudaSuccess) return e;
  launch_begin(CSA_K_PAGED_MERGE, s);
  e = launch_kernel(paged_join_kernel<D>, dim3((unsigned)(a.n_rows * a.n_heads)), dim3(128), 0, s, 0,
                    false, a, parts, C::PAIRS, ctas);
  launch_end(CSA_K_PAGED_MERGE, s);
  return e;
}

// 16-pair tiles of an item: one, or two where a row's heads or two rows fill them.
int pair_tiles(const csa_paged_attn_args &a) {
  return a.n_heads / a.n_kv_heads > 16 ? 2 : 1;
}

}  // namespace

int paged_decode_items(const csa_paged_attn_args &a, int rows) {
  const int pairs = 16 * pair_tiles(a), g = a.n_heads / a.n_kv_heads;
  return g < pairs ? (rows + pairs / g - 1) / (pairs / g) : rows * ((g + pairs - 1) / pairs);
}

namespace {

// Two CTAs an SM for heads of 64, where they fit: up to 330 rows in items of 16
// pairs, 48 in items of 32 (the figures are at the top).
bool two_ctas(const csa_paged_attn_args &a) {
  constexpr int half = 228 * 1024 / 2 - 1024;  // of an SM's shared memory
  return a.head_dim == 64 && (pair_tiles(a) == 1 ? smem_bytes<64, 1, 3>(a.n_rows)
                                                 : smem_bytes<64, 2, 3>(a.n_rows)) <= half;
}

}  // namespace

size_t paged_decode_workspace(const csa_paged_attn_args &a, int sms) {
  const int pairs = 16 * pair_tiles(a);
  const int g = a.n_heads / a.n_kv_heads, gt = g < pairs ? g : pairs;
  const size_t subs = (size_t)a.n_kv_heads * ((g + gt - 1) / gt);
  const size_t slots = 2 * (size_t)sms * (two_ctas(a) ? 2 : 1) * pairs;
  return align_up(slots * a.head_dim * sizeof(float), 256) + align_up(slots * sizeof(float2), 256) +
         align_up((size_t)a.n_rows * subs * sizeof(int4), 256);
}

cudaError_t launch_paged_decode(const csa_paged_attn_args &a, int sms, cudaStream_t s) {
  const int mt = pair_tiles(a), ctas = sms * (two_ctas(a) ? 2 : 1);
  const size_t slots = 2 * (size_t)ctas * 16 * mt;
  uint8_t *ws = static_cast<uint8_t *>(a.workspace);
  DecodeParts parts;
  parts.o = reinterpret_cast<float *>(ws);
  ws += align_up(slots * a.head_dim * sizeof(float), 256);
  parts.ml = reinterpret_cast<float2 *>(ws);
  parts.item = reinterpret_cast<int4 *>(ws + align_up(slots * sizeof(float2), 256));
  if (a.head_dim == 128)
    return mt == 1 ? launch<128, 1, 3>(a, parts, ctas, s) : launch<128, 2, 3>(a, parts, ctas, s);
  if (ctas > sms)
    return mt == 1 ? launch<64, 1, 3>(a, parts, ctas, s) : launch<64, 2, 3>(a, parts, ctas, s);
  return mt == 1 ? launch<64, 1, 6>(a, parts, ctas, s) : launch<64, 2, 6>(a, parts, ctas, s);
}

}  // namespace csa
