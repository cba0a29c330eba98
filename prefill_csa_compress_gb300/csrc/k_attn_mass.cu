// The attention weight that every cached position received (csa_attn_mass): tcgen05
// tiles of two pages of 128 positions against up to 128 (row, head) pairs.
//
//   S^T[j, n] = k_j . q_n          (2 x 128 x N x D, both operands K-major)
//   mass[j]  += sum_n 2^(S^T[j, n] scale log2(e) - lse_n log2(e))
// A lane of tensor memory is a position, so a thread adds up its position's weights
// over all columns, and no sum crosses threads but at the end (in an order that the
// arguments fix: no atomics).
//
// A CTA takes two pages of a request (up to eight such pairs, one after the other, in large
// calls), some of its key heads and a share of the rows that see them (heads and rows are
// split only as far as there are too few pages to fill the GPU; mass_join_kernel then adds
// the parts in order).  A step is one key head and one tile of consecutive rows with their
// heads stacked under them; its queries serve both pages, which halves what a prompt
// fetches from L2.  One CTA an SM.  Roles:
//   warps 0..15  the exponentials and the sums, eight warps a page, two of them 32
//                positions, 32 columns in turn; each page's logits have buffers and
//                barriers of their own, so that one page's warps wait for tensor memory
//                while the other's compute (with common ones a prompt 11 us more);
//   warp 16      loads (TMA): the pages' keys once a head, the queries of every step;
//   warp 17      issues the MMAs;
//   warp 18      walks the rows, leaves out tiles that do not see the pages and
//                describes each step to the rest: references and bounds a column.
//
// What bounds it.  Decode (32 rows over ragged contexts to 16,384, 64 heads on 8 of 128):
// 121 us, 5.7 TB/s, the pages' way through three stages of a CTA.  A prompt of 8192 rows of
// 32 heads on 8: 263 us, 1.05 PFLOP/s; a step takes a CTA some 1,900 cycles, of which the
// products fill 1,024 (they read shared memory at its full rate) and the exponentials 1,024
// of their unit; between them stand the issuing lane's waits and the sums' latency.  Set
// aside: one page a CTA and two CTAs an SM (prompt 303 us, decode 132); runtime divisions
// by the number of stages in the issuing lane (300); all of a warp's logits in registers
// before its exponentials, as two reads of 32 columns or one of 64, the buffer given back
// at once or at the end (2 to 20 % more); with one page, exponentials on the FMA pipe (a
// quarter of them: 347), 16 columns at a time with the next ones on their way (317), three
// or four groups of warps (312, 483 with spills).
#include <cstddef>

#include "attn_common.cuh"
#include "cache_tiles.cuh"

namespace csa {
namespace {

constexpr int AM_THREADS = 608;
constexpr int AM_LOAD = 16, AM_MMA = 17, AM_WALK = 18;  // warps; 0 .. 15 add up
constexpr int AM_PAIR = 2 * kBlock;  // positions of two pages
constexpr int AM_STEPS = 4;   // steps described ahead
constexpr int AM_RING = 4;    // stages of keys and of queries, at most

// (One read for what the issuing lane needs: it goes through every step by itself, and
// each access that it waits for is time without products.)
struct Step {
  int t0;        // its rows start here
  int kvh;       // key head, < 0: no products, the pages are done
  int flags;     // NEW_K, ...; from SEEN on bit p: page p is there and some column sees some
                 // of it, from MIXED on: some column does not see all of it
  int page;      // of the request the first
  int phys[2];   // in the pool, -1: it is not there
  int pad[2];
};
constexpr int NEW_K = 1, LAST_K = 2, NO_MORE = 4;  // the head's first step, its last; kvh < 0
constexpr int SEEN = 3, MIXED = 5;                 // shifts

struct Misc {
  uint64_t k_full[AM_RING], k_empty[AM_RING], q_full[AM_RING], q_empty[AM_RING];
  uint64_t s_full[2][2], s_empty[2][2], x_full[2][2], m_full[AM_STEPS], m_empty[AM_STEPS], drained;
  uint32_t tmem;
  int abort;
  int vmin, vmax;      // rows of the request that see some of the pages
  alignas(16) Step step[AM_STEPS];
  alignas(16) float lse[AM_STEPS][128];  // a column's -lse log2(e) (read four at a time)
  int2 see[AM_STEPS][128];  // a column's positions of the pages [x, y)
  float sum[2][2][128];     // (by the step's parity, and the page)
};

static_assert(offsetof(Misc, step) % 16 == 0 && sizeof(Step) % 16 == 0 &&
                  offsetof(Misc, lse) % 16 == 0 && offsetof(Misc, see) % 8 == 0,
              "vector reads");

// How the host splits a call, and its shared memory.
struct Split {
  int tr, n;          // rows of a step and its columns, rounded up to 32
  int pairs;          // of pages of a request that a CTA takes one after the other
  int kv, rows;       // parts by key heads (heads_per each) and by rows
  int heads_per;
  int k_stages, q_stages;
  int q_bytes;        // of a stage (a whole number of 1024)
};

// A box of a tensor map into L2.
__device__ __forceinline__ void prefetch_4d(const void *tmap, int x, int y, int z, int w) {
  asm volatile("cp.async.bulk.prefetch.tensor.4d.L2.global [%0, {%1, %2, %3, %4}];" ::"l"(
                   reinterpret_cast<uint64_t>(tmap)),
               "r"(x), "r"(y), "r"(z), "r"(w)
               : "memory");
}

// A position's mass, or its part.  (A function, since in the loop it costs registers: with
// one page a CTA 308 against 302 us for a prompt.)
__device__ __noinline__ void put_mass(const csa_attn_mass_args &a, float *parts, long long part, int b,
                                      int col, float sum) {
  if (parts) {
    parts[part * ((long long)a.max_blocks * kBlock) + col] = sum;
    return;
  }
  if (a.decay != 0.f)
    sum += a.decay * reinterpret_cast<const float *>(reinterpret_cast<const uint8_t *>(a.mass) +
                                                     b * a.mass_row_stride)[col];
  reinterpret_cast<float *>(reinterpret_cast<uint8_t *>(a.mass_out) + b * a.mass_out_row_stride)[col] = sum;
}

// A position's sum where it is NaN, once more by the columns' bounds.
__device__ __noinline__ float bounded_sum(uint32_t logits, const float *lse, const int2 *see, int c0,
                                          int n, int j, float sl2, float sum) {
  float again = 0.f;
#pragma unroll 1
  for (int c = c0; c < n; c += 64) {
    float x[32];
    tc::tmem_ld32(logits + c, x);
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (j >= see[c + i].x && j < see[c + i].y) again += attn::exp2_sfu(fmaf(x[i], sl2, lse[c + i]));
  }
  return sum == sum ? sum : again;
}

// Full: the rows of a step fill its columns.  Else some have no query and count on
// 2^(0 k - inf) = 0, which a key that is not finite makes NaN, so that sums that come out
// NaN are taken once more without them.  (In one kernel, asked for every step, a prompt
// whose columns are full takes 265 us for 262; with such columns' logits set to zero 269;
// by bounds from the first 256 -> 296 where 3 of 128 are empty.)  The last rows' tile,
// which may be short in either, goes by bounds.
template <int D, bool Full>
__global__ void __launch_bounds__(AM_THREADS, 1)
    attn_mass_kernel(const __grid_constant__ csa_attn_mass_args a, float *parts, Split G,
                     const __grid_constant__ CUtensorMap qmap,
                     const __grid_constant__ CUtensorMap kmap) {
  constexpr int BOXES = D / 64, K_TILE = BOXES * 16384;  // (of a page; a stage has two)
  extern __shared__ __align__(1024) uint8_t sm[];
  uint8_t *ks = sm, *qs = sm + G.k_stages * 2 * K_TILE;
  Misc *M = reinterpret_cast<Misc *>(qs + G.q_stages * G.q_bytes);
  tc::griddep_wait();
  tc::griddep_launch_dependents();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tc::smem_u32(sm) & 1023u) {
    if (tid == 0) flag(a.status_dev, CSA_DEV_TIMEOUT);
    return;
  }
  // key heads fastest, then rows, requests, pages: the first pages, which the most rows
  // see, first
  int u = blockIdx.x;
  const int kv_part = u % G.kv;
  u /= G.kv;
  const int row_part = u % G.rows;
  u /= G.rows;
  const int b = u % a.n_req, pair0 = u / a.n_req * G.pairs;
  const int len = min(a.kv_len[b], a.max_blocks * kBlock);
  if (b == 0 && pair0 == 0 && kv_part == 0 && row_part == 0)
    for (int t = tid; t < a.n_rows; t += AM_THREADS)
      if (a.row_req[t] >= a.n_req) flag(a.status_dev, CSA_DEV_BAD_POS);
  if ((long long)pair0 * AM_PAIR >= len) return;
  const int pair1 = min(pair0 + G.pairs, (len - 1) / AM_PAIR + 1);
  const int32_t *table = a.block_table + (long long)b * a.max_blocks;
  // a page's place in the pool; -1: it has no position, or none there
  auto place = [&](int page) {
    const int phys = (long long)page * kBlock < len ? table[page] : -1;
    return phys >= 0 && phys < a.n_blocks ? phys : -1;
  };
  // the first pages' keys are asked for while the rows are found (behind a window no row
  // may see them; later pages asked for ahead make it slower)
  if (warp < 2 && a.window == 0) {
    const int phys = place(2 * pair0 + warp);
    if (phys >= 0)
      for (int i = lane; i < BOXES * G.heads_per; i += 32) {
        const int h = kv_part * G.heads_per + i / BOXES;
        if (h < a.n_kv_heads) prefetch_4d(&kmap, i % BOXES * 64, h, 0, phys);
      }
  }
  if (tid == 0) {
    for (int i = 0; i < AM_RING; ++i) {
      tc::mbar_init(&M->k_full[i], 1);
      tc::mbar_init(&M->k_empty[i], 1);
      tc::mbar_init(&M->q_full[i], 1);
      tc::mbar_init(&M->q_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      for (int p = 0; p < 2; ++p) {
        tc::mbar_init(&M->s_full[i][p], 2);
        tc::mbar_init(&M->s_empty[i][p], 8);
        tc::mbar_init(&M->x_full[i][p], 4);
      }
    }
    for (int i = 0; i < AM_STEPS; ++i) {
      tc::mbar_init(&M->m_full[i], 1);
      tc::mbar_init(&M->m_empty[i], 18);  // loads, MMA, sixteen warps of sums
    }
    tc::mbar_init(&M->drained, 1);
    M->abort = 0;
    M->vmin = 0x7FFFFFFF, M->vmax = -1;
    tc::mbar_fence_init();
    paged::prefetch_map(&qmap);
    paged::prefetch_map(&kmap);
  }
  if (warp == AM_MMA) tc::tmem_alloc(&M->tmem, 512);
  const int g = a.n_heads / a.n_kv_heads;
  // columns that no query fills are zero, and their references +inf
  {
    const int tail = (G.n - G.tr * g) * 8, per = G.q_bytes / BOXES;
    for (int i = tid; i < tail * BOXES * G.q_stages; i += AM_THREADS)
      reinterpret_cast<uint4 *>(qs + i / tail * per + G.tr * g * 128)[i % tail] = make_uint4(0, 0, 0, 0);
    tc::fence_async_shared();
  }
  __syncthreads();
  // the rows that see some of the pages
  {
    int v0 = 0x7FFFFFFF, v1 = -1;
    const int from = pair0 * AM_PAIR, end = (long long)pair1 * AM_PAIR < len ? pair1 * AM_PAIR : len;
#pragma unroll 4
    for (int t = tid; t < a.n_rows; t += AM_THREADS) {
      const int req = a.row_req[t], pos = a.row_pos[t];
      int lo, hi;
      paged::visible_range(a, len, pos, lo, hi);
      if (req == b && max(lo, from) < min(hi, end)) v0 = min(v0, t), v1 = t;
    }
    v0 = __reduce_min_sync(0xffffffffu, v0);
    v1 = __reduce_max_sync(0xffffffffu, v1);
    if (lane == 0 && v1 >= 0) {
      atomicMin(&M->vmin, v0);
      atomicMax(&M->vmax, v1);
    }
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = __reduce_or_sync(0xffffffffu, M->tmem);
  volatile int *abort = &M->abort;
  const int kv0 = kv_part * G.heads_per, kv1 = min(a.n_kv_heads, kv0 + G.heads_per);
  // this part's tiles of rows
  const int vmin = M->vmin, n_all = M->vmax < 0 ? 0 : (M->vmax - vmin) / G.tr + 1;
  const int tile0 = (int)((long long)n_all * row_part / G.rows);
  const int tile1 = (int)((long long)n_all * (row_part + 1) / G.rows);

  if (warp == AM_WALK) {
    // ================================================================ the steps
    // four columns a lane: row and head within the tile
    int r[4], h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int n = 32 * i + lane;
      r[i] = n / g, h[i] = n % g;
      if (r[i] >= G.tr) r[i] = -1;
    }
    uint32_t it = 0;
    bool ok = true;
    int phys[2] = {place(2 * pair0), place(2 * pair0 + 1)};
    for (int pair = pair0; pair < pair1 && ok; ++pair) {
      const int base = pair * AM_PAIR;
      const int there = (phys[0] >= 0) + 2 * (phys[1] >= 0);
      for (int kvh = kv0; kvh < kv1 && ok; ++kvh) {
        // asked for a tile ahead
        int req[4], pos[4];
        float lse[4];
        auto ask = [&](int tile) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int t = vmin + tile * G.tr + r[i];
            const bool in = r[i] >= 0 && t < a.n_rows && tile < tile1;
            req[i] = in ? a.row_req[t] : -1;
            pos[i] = in ? a.row_pos[t] : 0;
            lse[i] = in ? a.lse[(long long)t * a.n_heads + kvh * g + h[i]] : INFINITY;
          }
        };
        // a step is published when the next one is known, or that there is none
        int pending = -1, first = 1;
        float p_lse[4];
        int2 p_see[4];
        int p_seen = 0, p_mixed = 0;
        auto publish = [&](bool last) {
          const int st = it % AM_STEPS;
          ok = __all_sync(0xffffffffu, cache::wait(&M->m_empty[st], ((it / AM_STEPS) & 1) ^ 1, abort,
                                               a.status_dev));
          if (!ok) return;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            M->lse[st][32 * i + lane] = p_lse[i];
            M->see[st][32 * i + lane] = p_see[i];
          }
          if (lane == 0) {
            Step &S = M->step[st];
            S.t0 = pending, S.kvh = kvh;
            S.flags = (first ? NEW_K : 0) | (last ? LAST_K : 0) | p_seen << SEEN | p_mixed << MIXED;
            S.page = 2 * pair, S.phys[0] = phys[0], S.phys[1] = phys[1];
          }
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&M->m_full[st]);
          ++it;
          first = 0;
        };
        ask(tile0);
        for (int tile = tile0; tile < tile1 && ok; ++tile) {
          bool any[2] = {false, false}, part[2] = {false, false};
          float x[4];
          int2 see[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            int lo, hi;
            paged::visible_range(a, len, pos[i], lo, hi);
            lo = max(lo - base, 0), hi = min(hi - base, AM_PAIR);
            if (req[i] != b || lo >= hi || lse[i] == -INFINITY) lo = hi = 0;
            const bool row = r[i] >= 0 && vmin + tile * G.tr + r[i] < a.n_rows;
#pragma unroll
            for (int p = 0; p < 2; ++p) {
              any[p] = any[p] || max(lo, p * kBlock) < min(hi, p * kBlock + kBlock);
              part[p] = part[p] || (row && (lo > p * kBlock || hi < p * kBlock + kBlock));
            }
            x[i] = -lse[i] * paged::kLog2e, see[i] = make_int2(lo, hi);
          }
          ask(tile + 1);
          const int seen = __any_sync(0xffffffffu, any[0]) + 2 * __any_sync(0xffffffffu, any[1]);
          const int mixed = vmin + (tile + 1) * G.tr > a.n_rows
                                ? 3
                                : __any_sync(0xffffffffu, part[0]) + 2 * __any_sync(0xffffffffu, part[1]);
          if ((seen & ~there) && lane == 0) flag(a.status_dev, CSA_DEV_BAD_BLOCK);
          if (!(seen & there)) continue;
          if (pending >= 0) publish(false);
          pending = vmin + tile * G.tr, p_seen = seen & there, p_mixed = mixed;
#pragma unroll
          for (int i = 0; i < 4; ++i) p_lse[i] = x[i], p_see[i] = see[i];
        }
        if (pending >= 0 && ok) publish(true);
      }
      if (pair + 1 < pair1) phys[0] = place(2 * pair + 2), phys[1] = place(2 * pair + 3);
      if (!ok) break;
      const int st = it % AM_STEPS;  // the pages are done
      ok = __all_sync(0xffffffffu, cache::wait(&M->m_empty[st], ((it / AM_STEPS) & 1) ^ 1, abort,
                                           a.status_dev));
      if (ok && lane == 0) {
        Step &S = M->step[st];
        S.kvh = -1, S.page = 2 * pair, S.flags = pair + 1 == pair1 ? NO_MORE : 0;
        tc::mbar_arrive(&M->m_full[st]);
      }
      ++it;
    }
    __syncwarp();
  } else if (warp == AM_LOAD) {
    // ================================================================ loads
    if (lane == 0) {
      uint32_t nk = 0, nq = 0;
      int sk = 0, sq = 0;               // stages
      uint32_t k_turn = 1, q_turn = 1;  // parities
      bool ok = true;
      for (uint32_t it = 0;; ++it) {
        const int st = it % AM_STEPS;
        ok = cache::wait(&M->m_full[st], (it / AM_STEPS) & 1, abort, a.status_dev);
        if (!ok) break;
        const Step S = M->step[st];
        tc::mbar_arrive(&M->m_empty[st]);
        if (S.kvh < 0) {
          if (S.flags & NO_MORE) break;
          continue;
        }
        if (S.flags & NEW_K) {
          ok = cache::wait(&M->k_empty[sk], k_turn, abort, a.status_dev);
          if (!ok) break;
          // (every page that is there: a later step of the head may see it)
          tc::mbar_arrive_expect_tx(&M->k_full[sk], K_TILE * ((S.phys[0] >= 0) + (S.phys[1] >= 0)));
          for (int p = 0; p < 2; ++p)
            if (S.phys[p] >= 0)
              for (int c = 0; c < BOXES; ++c)
                paged::tma_load_4d(ks + (2 * sk + p) * K_TILE + c * 16384, &kmap, c * 64, S.kvh, 0,
                                   S.phys[p], &M->k_full[sk]);
          ++nk;
          if (++sk == G.k_stages) sk = 0, k_turn ^= 1;
        }
        ok = cache::wait(&M->q_empty[sq], q_turn, abort, a.status_dev);
        if (!ok) break;
        tc::mbar_arrive_expect_tx(&M->q_full[sq], BOXES * 128 * g * G.tr);
        for (int c = 0; c < BOXES; ++c)
          tc::tma_load_3d(qs + sq * G.q_bytes + c * (G.q_bytes / BOXES), &qmap, c * 64, S.kvh * g,
                          S.t0, &M->q_full[sq]);
        ++nq;
        if (++sq == G.q_stages) sq = 0, q_turn ^= 1;
      }
      // whatever was asked for has landed before the CTA retires
      if (!ok) {
        for (uint32_t k = nk > (uint32_t)G.k_stages ? nk - G.k_stages : 0; k < nk; ++k)
          tc::mbar_wait(&M->k_full[k % G.k_stages], (k / G.k_stages) & 1, 50000000ull);
        for (uint32_t k = nq > (uint32_t)G.q_stages ? nq - G.q_stages : 0; k < nq; ++k)
          tc::mbar_wait(&M->q_full[k % G.q_stages], (k / G.q_stages) & 1, 50000000ull);
      }
    }
    __syncwarp();
  } else if (warp == AM_MMA) {
    // ================================================================ MMA
    if (tc::elect_one()) {
      const uint32_t idesc = tc::idesc_bf16_f32(128, G.n);
      const uint64_t dk = tc::desc_sw128(tc::smem_u32(ks)), dq = tc::desc_sw128(tc::smem_u32(qs));
      int sk = 0, sq = 0;               // stages
      uint32_t k_turn = 0, q_turn = 0;  // parities
      bool ok = true;
      for (uint32_t it = 0;; ++it) {
        const int st = it % AM_STEPS, buf = it & 1;
        ok = cache::wait(&M->m_full[st], (it / AM_STEPS) & 1, abort, a.status_dev);
        if (!ok) break;
        const int4 S = *reinterpret_cast<const int4 *>(&M->step[st]);  // t0, kvh, flags, page
        tc::mbar_arrive(&M->m_empty[st]);
        if (S.y >= 0)
          ok = (!(S.z & NEW_K) || cache::wait(&M->k_full[sk], k_turn, abort, a.status_dev)) &&
               cache::wait(&M->q_full[sq], q_turn, abort, a.status_dev);
        if (!ok) break;
        if (S.y >= 0) tc::tc_fence_after();
        const uint64_t k = dk + ((sk * 2 * K_TILE) >> 4), q = dq + ((sq * G.q_bytes) >> 4);
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          ok = ok && cache::wait(&M->s_empty[buf][p], ((it >> 1) & 1) ^ 1, abort, a.status_dev);
          if (!ok) break;
          tc::tc_fence_after();
          if (S.z >> (SEEN + p) & 1)
#pragma unroll
            for (int c = 0; c < BOXES; ++c)
              cache::mma4<2, 2>(tmem + buf * 256 + p * 128, k + ((p * K_TILE + c * 16384) >> 4),
                                q + ((c * (G.q_bytes / BOXES)) >> 4), idesc, c > 0);
          // (no logits: both arrivals are plain)
          if (S.y >= 0) tc::mma_commit(&M->s_full[buf][p]);
          else tc::mbar_arrive(&M->s_full[buf][p]);
          tc::mbar_arrive(&M->s_full[buf][p]);  // hands on the step's description
        }
        if (!ok) break;
        if (S.y < 0) {
          if (S.z & NO_MORE) break;
          continue;
        }
        tc::mma_commit(&M->q_empty[sq]);
        if (++sq == G.q_stages) sq = 0, q_turn ^= 1;
        if (S.z & LAST_K) {
          tc::mma_commit(&M->k_empty[sk]);
          if (++sk == G.k_stages) sk = 0, k_turn ^= 1;
        }
      }
      // every issued MMA has completed before tensor memory is released
      tc::mma_commit(&M->drained);
      tc::mbar_wait(&M->drained, 0, 100000000ull);
    }
    __syncwarp();
  } else {
    // ================================================================ exponentials and sums
    const int qd = warp & 3, grp = (warp >> 2) & 1, pg = warp >> 3;
    const int row = qd * 32 + lane, j = pg * kBlock + row;  // of the page, of both
    const uint32_t ts = tmem + ((uint32_t)(qd * 32) << 16) + pg * 128;
    const float sl2 = a.softmax_scale * paged::kLog2e;
    float total = 0.f;
    uint32_t outs0 = 0, outs1 = 0;  // pages done, by the step's parity
    bool ok = true;
    auto wait = [&](uint64_t *bar, uint32_t turn) {
      return (bool)__all_sync(0xffffffffu, cache::wait(bar, turn & 1, abort, a.status_dev));
    };
    for (uint32_t it = 0;; ++it) {
      const int st = it % AM_STEPS, buf = it & 1;
      ok = wait(&M->s_full[buf][pg], it >> 1);
      if (!ok) break;
      if (M->step[st].kvh < 0) {
        // the two halves of the columns, then the position's mass or its part
        const long long col = (long long)M->step[st].page * kBlock + j;
        const bool last = (M->step[st].flags & NO_MORE) != 0;
        if (grp == 1) {
          M->sum[buf][pg][row] = total;
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&M->x_full[buf][pg]);
        } else {
          ok = wait(&M->x_full[buf][pg], buf ? outs1++ : outs0++);
          if (!ok) break;
        }
        if (grp == 0 && col < len)
          put_mass(a, parts, (long long)(kv_part * G.rows + row_part) * a.n_req + b, b, (int)col,
                   total + M->sum[buf][pg][row]);
        total = 0.f;
        __syncwarp();
        if (lane == 0) {
          tc::mbar_arrive(&M->s_empty[buf][pg]);
          tc::mbar_arrive(&M->m_empty[st]);
        }
        if (last) break;
        continue;
      }
      const int flags = M->step[st].flags;
      const bool mixed = flags >> (MIXED + pg) & 1, seen = flags >> (SEEN + pg) & 1;
      tc::tc_fence_after();
      float2 sums[2] = {{0.f, 0.f}, {0.f, 0.f}};
#pragma unroll 1
      for (int c = 32 * grp; c < G.n && seen; c += 64) {
        float x[32];
        tc::tmem_ld32(ts + buf * 256 + c, x);
        const float4 *lse = reinterpret_cast<const float4 *>(M->lse[st] + c);
        if (!mixed) {
          const float2 one = make_float2(1.f, 1.f), scale = make_float2(sl2, sl2);
#pragma unroll
          for (int i = 0; i < 32; i += 4) {
            const float4 r = lse[i >> 2];
            float2 y = tc::ffma2(make_float2(x[i], x[i + 1]), scale, make_float2(r.x, r.y));
            float2 z = tc::ffma2(make_float2(x[i + 2], x[i + 3]), scale, make_float2(r.z, r.w));
            y.x = attn::exp2_sfu(y.x), y.y = attn::exp2_sfu(y.y);
            z.x = attn::exp2_sfu(z.x), z.y = attn::exp2_sfu(z.y);
            sums[0] = tc::ffma2(y, one, sums[0]);
            sums[1] = tc::ffma2(z, one, sums[1]);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const int2 see = M->see[st][c + i];
            const float y = attn::exp2_sfu(fmaf(x[i], sl2, M->lse[st][c + i]));
            if (j >= see.x && j < see.y) sums[i & 1].x += y;
          }
        }
      }
      float sum = (sums[0].x + sums[0].y) + (sums[1].x + sums[1].y);
      if (!Full && __any_sync(0xffffffffu, sum != sum))
        sum = bounded_sum(ts + buf * 256, M->lse[st], M->see[st], 32 * grp, seen ? G.n : 0, j, sl2, sum);
      total += sum;
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        tc::mbar_arrive(&M->s_empty[buf][pg]);
        tc::mbar_arrive(&M->m_empty[st]);
      }
    }
  }

  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  if (warp == AM_MMA) tc::tmem_dealloc(tmem, 512);
}

// mass_out from the parts, in order.
__global__ void __launch_bounds__(256)
    mass_join_kernel(csa_attn_mass_args a, const float *parts, int n_parts) {
  tc::griddep_wait();
  tc::griddep_launch_dependents();
  const long long cols = (long long)a.max_blocks * kBlock;
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  const int b = (int)(i / cols), j = (int)(i - b * cols);
  if (b >= a.n_req || j >= a.kv_len[b]) return;
  float sum = 0.f;
#pragma unroll 8
  for (int s = 0; s < n_parts; ++s) sum += parts[((long long)s * a.n_req + b) * cols + j];
  if (a.decay != 0.f)
    sum += a.decay * reinterpret_cast<const float *>(reinterpret_cast<const uint8_t *>(a.mass) +
                                                     b * a.mass_row_stride)[j];
  reinterpret_cast<float *>(reinterpret_cast<uint8_t *>(a.mass_out) + b * a.mass_out_row_stride)[j] = sum;
}

// Rows of a step: what a request has on average, as far as 128 columns go (the host
// does not know how rows are spread).  Parts, by key heads first (they share nothing), then
// by rows: a CTA for each SM at least, and up to two where each still has 32 steps (4096
// rows of 32 heads on 4 over 16,384: 505 us with one, 396 with two, 430 with four; 300 rows
// over 32,768 95, 101 and 106, since a CTA's start is paid for each).  With a handful of
// steps, as in decode, no second round for a few CTAs (one row over 32,768: 21 us with 256
// CTAs, 15 with 128; 3 x 500 rows over ragged 4000, which have more steps, 60 for 46).
// The host does not know the caches' lengths: the table's width stands for them, so that a
// table much wider than its caches leaves SMs idle (the prompt above with 4 times the
// columns it needs 743 us, with 16 times 1941).
Split split_of(const csa_attn_mass_args &a) {
  Split G;
  const int g = a.n_heads / a.n_kv_heads;
  const long long per = a.n_rows > 0 ? ((long long)a.n_rows + a.n_req - 1) / a.n_req : 1;
  const int most = 128 / g;
  G.tr = per < most ? (int)per : most;
  G.n = (G.tr * g + 31) / 32 * 32;
  const long long pairs = (long long)a.n_req * ((a.max_blocks + 1) / 2);
  const long long tiles = (per + G.tr - 1) / G.tr, steps = tiles * a.n_kv_heads, sms = sm_count();
  const long long hi = (2 * sms + pairs - 1) / pairs, fit = steps / 32;
  const long long lo = steps * pairs < 16 * sms ? (sms > pairs ? sms / pairs : 1)
                                                : (sms + pairs - 1) / pairs;
  const long long want = fit < lo ? lo : (fit < hi ? fit : hi);
  G.kv = (int)(want < a.n_kv_heads ? want : a.n_kv_heads);
  G.heads_per = (a.n_kv_heads + G.kv - 1) / G.kv;
  G.kv = (a.n_kv_heads + G.heads_per - 1) / G.heads_per;
  const long long left = (want + G.kv - 1) / G.kv;
  const long long row_parts = left < tiles / 8 ? left : tiles / 8;  // (at least eight tiles each)
  G.rows = (int)(row_parts < 1 ? 1 : (row_parts > 16 ? 16 : row_parts));
  // Several pairs of pages a CTA where that leaves four CTAs for each SM: a CTA's start
  // (the rows that see its pages, the first keys) is then paid once for them (the decode
  // above 129 us in a graph with six, 116 with four, 133, 123 and 153 with three, two and one).
  const long long run = pairs * G.kv * G.rows / (4 * sms);
  G.pairs = (int)(run < 1 ? 1 : (run > 8 ? 8 : run));
  // queries in two stages, keys in what is left (a prompt with four and one 1 % more
  // than with two and two)
  const int k_tile = 2 * a.head_dim * 256, boxes = a.head_dim / 64;
  G.q_bytes = boxes * (int)align_up((size_t)G.n * 128, 1024);
  const int room = 227 * 1024 - 1024 - (int)sizeof(Misc);
  G.q_stages = 2;
  G.k_stages = (room - G.q_stages * G.q_bytes) / k_tile;
  if (G.k_stages > AM_RING) G.k_stages = AM_RING;
  return G;
}

template <int D, bool Full>
cudaError_t launch(const csa_attn_mass_args &a, float *parts, const Split &G,
                   const CUtensorMap &qmap, const CUtensorMap &kmap, cudaStream_t s) {
  const size_t smem = G.k_stages * D * 512 + G.q_stages * G.q_bytes + sizeof(Misc);
  int dev = 0;
  cudaGetDevice(&dev);
  static bool attr[64] = {};
  if (dev < 0 || dev >= 64 || !attr[dev]) {
    const cudaError_t e = cudaFuncSetAttribute(
        attn_mass_kernel<D, Full>, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) attr[dev] = true;
  }
  const long long grid = (long long)a.n_req * (((a.max_blocks + 1) / 2 + G.pairs - 1) / G.pairs) * G.kv *
                         G.rows;
  if (grid > 0x7FFFFFFF) return cudaErrorInvalidValue;
  return launch_kernel(attn_mass_kernel<D, Full>, dim3((unsigned)grid), dim3(AM_THREADS), smem, s, 0,
                       false, a, parts, G, qmap, kmap);
}

}  // namespace

size_t attn_mass_workspace(const csa_attn_mass_args &a) {
  const Split G = split_of(a);
  const size_t n = (size_t)G.kv * G.rows;
  return n == 1 ? 0 : align_up(n * a.n_req * a.max_blocks * kBlock * sizeof(float), 256);
}

cudaError_t launch_attn_mass(const csa_attn_mass_args &a, cudaStream_t s) {
  const Split G = split_of(a);
  const int n_parts = G.kv * G.rows, g = a.n_heads / a.n_kv_heads;
  float *parts = n_parts > 1 ? static_cast<float *>(a.workspace) : nullptr;
  CUtensorMap qmap, kmap;
  const cuuint64_t rows = a.n_rows > 0 ? a.n_rows : 1;
  const cuuint64_t qd[3] = {(cuuint64_t)a.head_dim, (cuuint64_t)a.n_heads, rows};
  const cuuint64_t qs[2] = {(cuuint64_t)a.head_dim * 2, (cuuint64_t)a.q_row_stride};
  const cuuint32_t qb[3] = {64, (cuuint32_t)g, (cuuint32_t)G.tr};
  const cuuint64_t kd[4] = {(cuuint64_t)a.head_dim, (cuuint64_t)a.n_kv_heads, kBlock,
                            (cuuint64_t)a.n_blocks};
  const cuuint64_t kst[3] = {(cuuint64_t)a.k_head_stride, (cuuint64_t)a.k_token_stride,
                             (cuuint64_t)a.k_page_stride};
  const cuuint32_t kb[4] = {64, 1, kBlock, 1};
  // (without rows nothing is loaded: any address will do for the queries)
  // (heads of 64: the line beside theirs is another head's)
  const auto l2 = a.head_dim == 64 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B
                                   : CU_TENSOR_MAP_L2_PROMOTION_L2_256B;
  if (!cache::encode(&qmap, a.n_rows > 0 ? a.q : a.k_pool, 3, qd, qs, qb, l2) ||
      !cache::encode(&kmap, a.k_pool, 4, kd, kst, kb, l2))
    return cudaErrorInvalidValue;
  launch_begin(CSA_K_ATTN_MASS, s);
  const bool full = G.n == G.tr * g;
  cudaError_t e = a.head_dim == 64 ? full ? launch<64, true>(a, parts, G, qmap, kmap, s)
                                          : launch<64, false>(a, parts, G, qmap, kmap, s)
                  : full           ? launch<128, true>(a, parts, G, qmap, kmap, s)
                                   : launch<128, false>(a, parts, G, qmap, kmap, s);
  launch_end(CSA_K_ATTN_MASS, s);
  if (e != cudaSuccess || n_parts == 1) return e != cudaSuccess ? e : cudaGetLastError();
  launch_begin(CSA_K_MASS_JOIN, s);
  // (a call that is split has too few pages to come near a grid's limit)
  const long long all = (long long)a.n_req * a.max_blocks * kBlock;
  e = launch_kernel(mass_join_kernel, dim3((unsigned)((all + 255) / 256)), dim3(256), 0, s, 0, false,
                    a, (const float *)parts, n_parts);
  launch_end(CSA_K_MASS_JOIN, s);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace csa
