// Attention of a chunk of rows over a paged key/value cache (csa_paged_attn):
// tcgen05 tiles of 128 (row, head) pairs against one page of 128 keys.
//
// With the query heads of a group stacked under their row, a tile of R rows x G
// heads (R G <= 128) reads one key/value head:
//   S[m, c] = q_m . k_c      (128 x 128 x D, both operands K-major)
//   O[m, :] += P[m, c] v_c   (128 x D x 128, P from tensor memory, V MN-major)
// with P = 2^(S scale log2(e) - ref_m).  A page is exactly one key tile, so a
// page costs one block-table look-up and D / 64 TMA boxes for K and V each.
//
// A CTA owns two tiles of consecutive rows, so that one tile's products run
// while the other's softmax does, and both read each page once.  Roles:
//   warp 0      walks the requests of the CTA's rows and their pages, loads Q, K
//               and V by TMA (a ring of stages), and describes each page to the rest;
//   warp 1      issues the MMAs;
//   warp 3      looks through V on pages that some row does not see whole: rows
//               that no one sees are zeroed, values that are not finite are
//               zeroed and reported, since a zero probability times them is not zero;
//   warps 4..19 softmax, eight warps a tile, two threads a (row, head) pair with
//               64 logits each.  P is computed with the reference as it is; only
//               when some P of 32 pairs reaches 2 (the references are set so
//               that the largest is 2^-7) are the maxima taken, references moved
//               and O rescaled in tensor memory.  Bit 14 of a positive BF16 says
//               that it is 2 or more, so the test is an OR of the packed P, and
//               it rides on the barrier that both halves of S need before P
//               goes over them.
// Tensor memory: O (D columns a tile), and S (128 columns) with P in BF16 over it.
// D = 128 fills the 512 columns; with D = 64 there is room for a third S, and
// a tile's next logits then need not wait for its product (304 -> 298 us for a
// prompt of 8192, 142 -> 138 us for ragged chunks once only the pairs' two warps
// meet at a barrier and not the tile's eight).
// Rows of several requests in one CTA take turns: a page of another request is
// masked for the whole row.
//
// What bounds it is the chain of one tile.  D = 128: 2,900 cycles a page for both
// tiles, where their MMAs take 2,048 -- the softmax of a tile 1,500 (reading the
// logits 300, the probabilities 700, the barrier 250, storing them 200), its MMAs
// 1,024, the rest the way from role to role.  D = 64: 2,330 cycles, all of them the
// softmax's (the warps issue half of the time, the exponentials' unit is busy for
// 35 %).  A CTA's start and end take 14,000.  A prompt of 8192 (32 query heads on 8
// of 128) takes 381 us from L2 (1.44 PFLOP/s) and 398 from memory, of 64 channels 288
// us from L2 (0.95 PFLOP/s), 4096 rows of 64 heads of 128 over 65,536 positions 5.5 ms
// (1.54 PFLOP/s).
#include <cuda.h>

#include "attn_common.cuh"
#include "csa_internal.cuh"
#include "paged_common.cuh"
#include "tc.cuh"

namespace csa {
namespace {

using paged::Parts;

constexpr int PC_THREADS = 640;
constexpr int PC_LOAD = 0, PC_MMA = 1, PC_CLEAN = 3, PC_SOFT0 = 4;  // first warps
constexpr int PC_BAR_START = 9;  // named barriers: 1 .. 8 are the softmax warps'
constexpr int PC_META = 8;  // pages described ahead (the ring holds at most 4 of them)
constexpr float kLift = 7.f;  // log2 of the room below P = 2, where a reference moves

template <int D>
struct Cfg {
  static constexpr int CHUNKS = D / 64;                // 128-byte column groups of a row
  static constexpr int TILE = CHUNKS * 16384;          // bytes of a 128-row tile
  static constexpr int STAGES = D == 128 ? 5 : 8;      // K and V tiles in flight
  static constexpr int OFF_KV = 2 * TILE;
  static constexpr int OFF_MISC = OFF_KV + STAGES * TILE;
  // Tensor memory columns: buffers of 128 for S (with P over it), then O.  Two
  // buffers, one a tile, or with room for a third (ROTATE) three that the tiles
  // take in turn, so that a tile's next logits do not wait for its product.
  static constexpr bool ROTATE = D == 64;
  static constexpr int O_COL = ROTATE ? 384 : 256;
};

// One page as the consumers need it.
struct Page {
  int base;        // position of its first key
  int req;         // request it belongs to
  int r0, r1;      // the CTA's rows that read it (a request may have several runs)
  int mixed;       // some row of the CTA does not see all of it
  int lo, hi;      // columns [lo, hi) that at least one row sees
  uint32_t bad[4]; // columns whose values are not finite (mixed pages only)
};

struct Misc {
  // 32 barriers, initialised by a lane each
  uint64_t q_full, drained, kv_full[8], kv_empty[8], ready[4], pv_done[2], o_full[2];
  uint64_t s_full[3], p_full[3];  // a buffer each
  uint32_t tmem;
  int abort;
  int n_it;  // pages this CTA works through
  Page page[PC_META];
  float top[2][2][128];  // a pair's largest logit, or sum, of each half
};
// All of it but for a few hundred bytes, so nothing is set aside for aligning
// the start: a kernel without static shared memory gets it 1024-byte aligned,
// and one that did not would stop before touching it.
static_assert(Cfg<128>::OFF_MISC + sizeof(Misc) <= 227 * 1024, "shared memory");

// Bounded wait that also gives up when another role has.
__device__ __forceinline__ bool pc_wait(uint64_t *bar, uint32_t parity, volatile int *abort,
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
__device__ __forceinline__ bool pc_wait_warp(uint64_t *bar, uint32_t parity, volatile int *abort,
                                             uint32_t *status) {
  return __all_sync(0xffffffffu, pc_wait(bar, parity, abort, status));
}

// The CTA's rows in the load warp's registers: lane i holds rows 32 k + i.
// Read at once, so that the walk over them waits for memory twice, not once a row.
constexpr int PC_K = 8;
struct Rows {
  int req[PC_K], lo[PC_K], hi[PC_K];  // -2 past the last row; what a row sees
};

__device__ __forceinline__ void read_rows(const csa_paged_attn_args &a, int t0, int n, Rows &W) {
  const int lane = threadIdx.x & 31;
  int pos[PC_K], len[PC_K];
#pragma unroll
  for (int k = 0; k < PC_K; ++k) {
    const int r = 32 * k + lane;
    W.req[k] = r < n ? a.row_req[t0 + r] : -2;
    pos[k] = r < n ? a.row_pos[t0 + r] : 0;
  }
#pragma unroll
  for (int k = 0; k < PC_K; ++k)  // (one wait for all of them)
    len[k] = a.kv_len[W.req[k] >= 0 && W.req[k] < a.n_req ? W.req[k] : 0];
#pragma unroll
  for (int k = 0; k < PC_K; ++k) {
    paged::visible_range(a, len[k], pos[k], W.lo[k], W.hi[k]);
    if (W.req[k] < 0 || W.req[k] >= a.n_req) W.lo[k] = W.hi[k] = 0;
  }
}

// Consecutive rows of one request: what they see.
struct Run {
  int req, end;
  int lo, hi;          // positions [lo, hi) that at least one of them sees
  int all_lo, all_hi;  // positions that every one of them sees

  __device__ __forceinline__ void add(int l, int h) {
    if (l < h) {
      lo = min(lo, l);
      hi = max(hi, h);
      all_lo = max(all_lo, l);
      all_hi = min(all_hi, h);
    } else {
      all_lo = 0x7FFFFFFF;  // a row that sees nothing
    }
  }
  __device__ __forceinline__ void reduce() {
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    all_lo = __reduce_max_sync(0xffffffffu, all_lo);
    all_hi = __reduce_min_sync(0xffffffffu, all_hi);
  }
};

// All rows as one run, if they are one request's (the usual case, without the
// registers and the code of the walk: that code is fetched cold by every CTA).
// meanwhile() runs while the first rows are on their way.
template <typename F>
__device__ __forceinline__ bool one_run(const csa_paged_attn_args &a, int t0, int n, Run &R,
                                        F &&meanwhile) {
  const int lane = threadIdx.x & 31;
  R = {0, n, 0x7FFFFFFF, 0, 0, 0x7FFFFFFF};
  bool same = true;
#pragma unroll 1
  for (int r = lane; r - lane < n; r += 64) {
    int req[2], pos[2], len[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int t = t0 + min(r + 32 * k, n - 1);  // (past the last row: that row again)
      req[k] = a.row_req[t];
      pos[k] = a.row_pos[t];
    }
    if (r == lane) {
      meanwhile();
      R.req = __shfl_sync(0xffffffffu, req[0], 0);
    }
#pragma unroll
    for (int k = 0; k < 2; ++k)
      len[k] = a.kv_len[req[k] >= 0 && req[k] < a.n_req ? req[k] : 0];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      int lo, hi;
      paged::visible_range(a, len[k], pos[k], lo, hi);
      same = same && req[k] == R.req;
      R.add(lo, hi);
    }
  }
  R.reduce();
  return __all_sync(0xffffffffu, same);
}

// The run that starts at row r0 < n (whole warp; req < 0: padding).
__device__ __forceinline__ Run next_run(const Rows &W, int r0, int n) {
  const int lane = threadIdx.x & 31;
  int mine = 0;
#pragma unroll
  for (int k = 0; k < PC_K; ++k)
    if (r0 >> 5 == k) mine = W.req[k];
  Run R = {__shfl_sync(0xffffffffu, mine, r0 & 31), n, 0x7FFFFFFF, 0, 0, 0x7FFFFFFF};
#pragma unroll
  for (int k = 0; k < PC_K; ++k) {
    const int r = 32 * k + lane;
    const uint32_t other = __ballot_sync(0xffffffffu, r >= r0 && W.req[k] != R.req);
    if (other && R.end == n) R.end = min(n, 32 * k + __ffs(other) - 1);
    if (r >= r0 && r < R.end) R.add(W.lo[k], W.hi[k]);
  }
  R.reduce();
  return R;
}

__device__ __forceinline__ int run_pages(const Run &R) {
  return R.lo < R.hi ? (R.hi - 1) / kBlock - R.lo / kBlock + 1 : 0;
}

// The MMAs of one step and the commits behind them, for one elected lane.
#define PC_MMA_PTX "tcgen05.mma.cta_group::1.kind::f16 "
#define PC_COMMIT_PTX "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 "
#define PC_BEGIN_PTX \
  "{\n\t.reg .pred p, q;\n\t.reg .b32 a;\n\t.reg .b64 x, y;\n\t"
#define PC_COMMIT_IF_PTX(n) "setp.ne.u32 q, %" #n ", 0;\n\t@q " PC_COMMIT_PTX "[%" #n "];\n\t"
#define PC_PV_PTX(k) \
  "add.u32 a, %1, " #k " * 8;\n\tadd.u64 x, %2, " #k " * 128;\n\t" PC_MMA_PTX "[%0], [a], x, %3, p;\n\t"
#define PC_QK_PTX(c, k)                                                     \
  "add.u64 x, %1, " #c " * 1024 + " #k " * 2;\n\tadd.u64 y, %2, " #c " * 1024 + " #k " * 2;\n\t" \
  PC_MMA_PTX "[%0], x, y, %3, p;\n\tsetp.eq.b32 p, 0, 0;\n\t"

// O += P V over the page's 128 keys; the barriers `freed` and `done` (0: none)
// are arrived on when everything issued so far has completed.
__device__ __forceinline__ void issue_pv(uint32_t d, uint32_t p_tmem, uint64_t v, uint32_t idesc,
                                         uint32_t freed, uint32_t done) {
  asm volatile(PC_BEGIN_PTX "setp.eq.b32 p, 0, 0;\n\t" PC_PV_PTX(0) PC_PV_PTX(1) PC_PV_PTX(2)
                   PC_PV_PTX(3) PC_PV_PTX(4) PC_PV_PTX(5) PC_PV_PTX(6) PC_PV_PTX(7)
                       PC_COMMIT_IF_PTX(4) PC_COMMIT_IF_PTX(5) "}" ::"r"(d),
               "r"(p_tmem), "l"(v), "r"(idesc), "r"(freed), "r"(done)
               : "memory");
}
// S = Q K^T over D / 16 steps; `full` also gets a plain arrival, which hands on
// what this warp has seen (the page's description).
template <int D>
__device__ __forceinline__ void issue_qk(uint32_t d, uint64_t q, uint64_t k, uint32_t idesc,
                                         uint32_t full, uint32_t freed) {
#define PC_QK_END_PTX                                                                      \
  PC_COMMIT_PTX "[%4];\n\t{\n\t.reg .b64 st;\n\tmbarrier.arrive.shared::cta.b64 st, [%4];\n\t}\n\t" \
  PC_COMMIT_IF_PTX(5) "}"
  if constexpr (D == 64)
    asm volatile(PC_BEGIN_PTX "setp.ne.b32 p, 0, 0;\n\t" PC_QK_PTX(0, 0) PC_QK_PTX(0, 1)
                     PC_QK_PTX(0, 2) PC_QK_PTX(0, 3) PC_QK_END_PTX ::"r"(d),
                 "l"(q), "l"(k), "r"(idesc), "r"(full), "r"(freed)
                 : "memory");
  else
    asm volatile(PC_BEGIN_PTX "setp.ne.b32 p, 0, 0;\n\t" PC_QK_PTX(0, 0) PC_QK_PTX(0, 1)
                     PC_QK_PTX(0, 2) PC_QK_PTX(0, 3) PC_QK_PTX(1, 0) PC_QK_PTX(1, 1)
                         PC_QK_PTX(1, 2) PC_QK_PTX(1, 3) PC_QK_END_PTX ::"r"(d),
                 "l"(q), "l"(k), "r"(idesc), "r"(full), "r"(freed)
                 : "memory");
}

// Bits below n of a word (none for n <= 0, all for n >= 32).
__device__ __forceinline__ uint32_t below(int n) {
  return n <= 0 ? 0u : (n >= 32 ? ~0u : (1u << n) - 1u);
}

// 16 consecutive FP32 columns of this thread's lane, and back.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&v)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const float (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};\n\t"
      "tcgen05.wait::st.sync.aligned;" ::"r"(taddr),
      "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]),
      "f"(v[8]), "f"(v[9]), "f"(v[10]), "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15])
      : "memory");
}

struct ChunkGrid {
  int n_tiles;    // row tiles (of 2 R rows)
  int rows_tile;  // R
  int n_parts;    // parts of a tile's pages
};

template <int D>
__global__ void __launch_bounds__(PC_THREADS, 1)
    paged_chunk_kernel(csa_paged_attn_args a, Parts parts, ChunkGrid G,
                       const __grid_constant__ CUtensorMap qmap,
                       const __grid_constant__ CUtensorMap kmap,
                       const __grid_constant__ CUtensorMap vmap) {
  using C = Cfg<D>;
  extern __shared__ __align__(1024) uint8_t sm[];
  Misc *M = reinterpret_cast<Misc *>(sm + C::OFF_MISC);
  tc::griddep_wait();
  tc::griddep_launch_dependents();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tc::smem_u32(sm) & 1023u) {
    if (tid == 0) flag(a.status_dev, CSA_DEV_TIMEOUT);
    return;
  }
  volatile int *abort = &M->abort;

  // the CTA's item: key/value head fastest, parts next, the last rows (which
  // see the most) first
  const int kvh = blockIdx.x % a.n_kv_heads;
  const int part = blockIdx.x / a.n_kv_heads % G.n_parts;
  const int tile = G.n_tiles - 1 - blockIdx.x / a.n_kv_heads / G.n_parts;
  const int g = a.n_heads / a.n_kv_heads;
  const int t0 = tile * 2 * G.rows_tile;
  const int n_rows = min(2 * G.rows_tile, a.n_rows - t0);
  const int n_sub = n_rows > G.rows_tile ? 2 : 1;  // tiles with rows

  // The warp that loads sets up the barriers and finds the CTA's pages; its
  // loads of q and of the first page need no other warp, and it joins the others
  // once they are under way.
  if (warp == PC_LOAD) {
    // ================================================================ loads
    // Two walks over the runs of one request, the first to count the pages: this
    // part takes its share of them.
    Run R;
    Rows W;
    const bool single = one_run(a, t0, n_rows, R, [&] {
      // (q_full, ..., o_full: one arrival; s_full two; p_full a warp each)
      tc::mbar_init(&M->q_full + lane, lane < 26 ? 1 : (lane < 29 ? 2 : 8));
      if (lane == 0) M->abort = 0;
      tc::mbar_fence_init();
      __syncwarp();
      if (lane == 0) {
        const uint32_t box = (uint32_t)(G.rows_tile * g * 128);
        tc::mbar_arrive_expect_tx(&M->q_full, n_sub * C::CHUNKS * box);
        for (int s = 0; s < n_sub; ++s)
          for (int c = 0; c < C::CHUNKS; ++c)
            tc::tma_load_3d(sm + s * C::TILE + c * 16384, &qmap, c * 64, kvh * g,
                            t0 + s * G.rows_tile, &M->q_full);
      }
    });
    if (!single) read_rows(a, t0, n_rows, W);
    bool counting = true, many = false, ok = true;
    int total = 0, valid = 0, skip = 0, n_pages = 0, left = 0;
    uint32_t it = 0;  // tiles loaded
    for (int r = 0; ok;) {
      if (r >= n_rows || (!counting && left == 0)) {
        if (!counting) break;
        counting = false;
        skip = (int)((long long)total * part / G.n_parts);
        left = n_pages = (int)((long long)total * (part + 1) / G.n_parts) - skip;
        many = valid > 1;
        if (lane == 0) M->n_it = n_pages;
        r = 0;
        continue;
      }
      const int r0 = r;
      if (!single) R = next_run(W, r, n_rows);
      r = R.end;
      if (counting && R.req >= a.n_req && lane == 0) flag(a.status_dev, CSA_DEV_BAD_POS);
      if (R.req < 0 || R.req >= a.n_req) continue;
      const int np = run_pages(R);
      if (counting) {
        total += np;
        ++valid;
        continue;
      }
      if (skip >= np) {
        skip -= np;
        continue;
      }
      const int pg0 = R.lo / kBlock + skip, n = min(np - skip, left);
      skip = 0;
      left -= n;
      int entry = 0;
      for (int i = 0; i < n && ok; ++i) {
        if ((i & 31) == 0)
          entry = i + lane < n
                      ? a.block_table[(long long)R.req * a.max_blocks + pg0 + i + lane]
                      : 0;
        const int phys = __shfl_sync(0xffffffffu, entry, i & 31);
        const bool there = phys >= 0 && phys < a.n_blocks;
        const int base = (pg0 + i) * kBlock;
        // K, then V
#pragma unroll 1
        for (int kv = 0; kv < 2; ++kv, ++it) {
          const int st = it % C::STAGES;
          ok = pc_wait_warp(&M->kv_empty[st], ((it / C::STAGES) & 1) ^ 1, abort, a.status_dev);
          if (!ok) break;
          if (lane == 0) {
            if (kv == 0) {
              Page &P = M->page[(it >> 1) % PC_META];
              P.base = base;
              P.req = R.req;
              P.r0 = r0;
              P.r1 = there ? R.end : r0;  // an unmapped page is seen by no row
              P.mixed = many || !there || base < R.all_lo || R.all_hi - base < kBlock;
              P.lo = there ? max(R.lo - base, 0) : 0;
              P.hi = there ? min(R.hi - base, kBlock) : 0;
              if (!there) flag(a.status_dev, CSA_DEV_BAD_BLOCK);
            }
            uint8_t *dst = sm + C::OFF_KV + st * C::TILE;
            if (there) {
              tc::mbar_arrive_expect_tx(&M->kv_full[st], C::TILE);
              for (int c = 0; c < C::CHUNKS; ++c)
                paged::tma_load_4d(dst + c * 16384, kv ? &vmap : &kmap, c * 64, kvh, 0, phys,
                                   &M->kv_full[st]);
            } else {
              tc::mbar_arrive(&M->kv_full[st]);
            }
          }
          __syncwarp();
        }
        if (it == 2) tc::bar_sync(PC_BAR_START, PC_THREADS);  // n_it, barriers
      }
    }
    if (n_pages == 0) {
      // q has landed before the others put their zeros where it goes
      pc_wait_warp(&M->q_full, 0, abort, a.status_dev);
      tc::bar_sync(PC_BAR_START, PC_THREADS);
    }
    // whatever was asked for has landed before the CTA retires
    if (*abort) {
      tc::mbar_wait(&M->q_full, 0, 50000000ull);
      for (uint32_t k = it > C::STAGES ? it - C::STAGES : 0; k < it; ++k)
        tc::mbar_wait(&M->kv_full[k % C::STAGES], (k / C::STAGES) & 1, 50000000ull);
    }
  } else {
    if (warp == PC_MMA) tc::tmem_alloc(&M->tmem, 512);
    if (tid == PC_CLEAN * 32) {
      paged::prefetch_map(&qmap);
      paged::prefetch_map(&kmap);
      paged::prefetch_map(&vmap);
    }
    tc::tc_fence_before();
    tc::bar_sync(PC_BAR_START, PC_THREADS);
    tc::tc_fence_after();
  }
  const int n_it = M->n_it;
  const uint32_t tmem = __reduce_or_sync(0xffffffffu, M->tmem);  // (into a uniform register)
  if (warp == PC_MMA && n_it > 0) {
    // ================================================================ MMA
    // One lane does it all: a wait takes it 90 cycles where the whole warp, which has
    // to agree on each, takes 160 to 320 (prompt of 8192 with 64 channels a head: 341 ->
    // 302 us, with 128: 387 -> 381).
    if (tc::elect_one()) {
      constexpr uint32_t idesc_s = tc::idesc_bf16_f32(128, 128);
      constexpr uint32_t idesc_o = tc::idesc_bf16_f32(128, D) | (1u << 16);  // V is MN-major
      const uint32_t kvs = tc::smem_u32(sm) + C::OFF_KV;
      // descriptors of the first tiles; an address further on adds its sixteenths
      const uint64_t dq = tc::desc_sw128(tc::smem_u32(sm)), dk = tc::desc_sw128(kvs);
      const uint64_t dv = tc::desc_sw128_mn(kvs, 16384, 1024);
      const uint32_t bar_s = tc::smem_u32(M->s_full), bar_pv = tc::smem_u32(M->pv_done),
                     bar_kv = tc::smem_u32(M->kv_empty);
      int sk = 0, sv = 1;  // stages of the next K and V
      // The next logits, page qj of tile qs into buffer qb.
      int qj = 0, qs = 0, qb = 0;
      auto next_s = [&] {
        if (C::ROTATE && qs == 0 && !pc_wait(&M->kv_full[sk], (qj >> 2) & 1, abort, a.status_dev))
          return false;
        issue_qk<D>(tmem + qb * 128, dq + qs * (C::TILE >> 4), dk + sk * (C::TILE >> 4), idesc_s,
                    bar_s + 8 * qb, qs == n_sub - 1 ? bar_kv + 8 * sk : 0);
        if (++qs == n_sub) {
          qs = 0;
          ++qj;
          sk = sk + 2 >= C::STAGES ? sk + 2 - C::STAGES : sk + 2;
        }
        qb = C::ROTATE ? (qb == 2 ? 0 : qb + 1) : qs;
        return true;
      };
      bool ok = pc_wait(&M->q_full, 0, abort, a.status_dev) &&
                (C::ROTATE || pc_wait(&M->kv_full[0], 0, abort, a.status_dev));
      for (int n = 0; n < (C::ROTATE ? n_sub + 1 : n_sub) && qj < n_it && ok; ++n) ok = next_s();
      int pb = 0;  // buffer of the next P, and the parity of its turn
      uint32_t turn = 0;
      for (int j = 0; j < n_it && ok; ++j) {
        // the page's V and the next page's K
        ok = pc_wait(&M->ready[j & 3], (j >> 2) & 1, abort, a.status_dev);
        for (int s = 0; s < n_sub && ok; ++s) {
          ok = pc_wait(&M->p_full[pb], turn, abort, a.status_dev);
          if (!ok) break;
          tc::tc_fence_after();
          issue_pv(tmem + C::O_COL + s * D, tmem + pb * 128, dv + sv * (C::TILE >> 4), idesc_o,
                   s == n_sub - 1 ? bar_kv + 8 * sv : 0, C::ROTATE ? bar_pv + 8 * s : 0);
          if (++pb == (C::ROTATE ? 3 : n_sub)) {
            pb = 0;
            turn ^= 1;
          }
          if (qj < n_it) ok = next_s();  // over P, or over the P before it
        }
        sv = sv + 2 >= C::STAGES ? sv + 2 - C::STAGES : sv + 2;
      }
      for (int s = 0; s < n_sub && ok; ++s) tc::mma_commit(&M->o_full[s]);
      // every issued MMA has completed before tensor memory is released
      tc::mma_commit(&M->drained);
      tc::mbar_wait(&M->drained, 0, 100000000ull);
    }
    __syncwarp();
  } else if (warp == PC_CLEAN && n_it > 0) {
    // ================================================================ V on mixed pages
    bool ok = true;
    for (int j = 0; j < n_it && ok; ++j) {
      const uint32_t ik = 2 * j, iv = ik + 1;
      const int sv = iv % C::STAGES;
      // in the order of the loads: only then does a stage's parity tell this
      // load from the stage's one before
      if (j == 0) ok = pc_wait_warp(&M->kv_full[0], 0, abort, a.status_dev);
      ok = ok && pc_wait_warp(&M->kv_full[sv], (iv / C::STAGES) & 1, abort, a.status_dev);
      if (!ok) break;
      Page &P = M->page[j % PC_META];
      if (P.mixed) {
        uint8_t *v = sm + C::OFF_KV + sv * C::TILE;
        bool wrote = false;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int row = k * 32 + lane;
          uint4 *p = reinterpret_cast<uint4 *>(v + row * 128);
          uint32_t bad = 0;
#pragma unroll
          for (int c = 0; c < C::CHUNKS; ++c) {
            uint4 w[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) w[q] = p[c * 1024 + ((q + lane) & 7)];
#pragma unroll
            for (int q = 0; q < 8; ++q)
              bad |= paged::not_finite2(w[q].x) | paged::not_finite2(w[q].y) |
                     paged::not_finite2(w[q].z) | paged::not_finite2(w[q].w);
          }
          if (bad) {
            for (int c = 0; c < C::CHUNKS; ++c)
              for (int q = 0; q < 8; ++q) p[c * 1024 + q] = make_uint4(0, 0, 0, 0);
            wrote = true;
          }
          const uint32_t seen = __ballot_sync(0xffffffffu, bad != 0 && row >= P.lo && row < P.hi);
          if (lane == 0) P.bad[k] = seen;
        }
        if (wrote) tc::fence_async_shared();
      }
      if (j + 1 < n_it)  // the MMA warp waits once for both
        ok = pc_wait_warp(&M->kv_full[(ik + 2) % C::STAGES], ((ik + 2) / C::STAGES) & 1, abort,
                          a.status_dev);
      __syncwarp();
      if (lane == 0 && ok) tc::mbar_arrive(&M->ready[j & 3]);
    }
  } else if (warp >= PC_SOFT0) {
    // ================================================================ softmax
    const int s = (warp - PC_SOFT0) >> 3, half = ((warp - PC_SOFT0) >> 2) & 1;
    const int m = (warp & 3) * 32 + lane;
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    uint32_t ts = tmem + s * 128 + lane_off;
    const uint32_t to = tmem + C::O_COL + s * D + half * (D / 2) + lane_off;  // this half
    const int bar = 1 + s * 4 + (warp & 3);  // of the two warps that share 32 rows
    const float sl2 = a.softmax_scale * paged::kLog2e;
    const int rr = s * G.rows_tile + m / g, t = t0 + rr, h = kvh * g + m % g;
    int req = -1, lo = 0, hi = 0;
    if (m < G.rows_tile * g && rr < n_rows) {
      req = a.row_req[t];
      if (req >= a.n_req) req = -1;
      if (req >= 0) paged::visible_range(a, a.kv_len[req], a.row_pos[t], lo, hi);
    }
    const float sink = req >= 0 && a.sink ? a.sink[h] : -INFINITY;
    // P = 2^(x - ref): ref is kLift above the largest logit when it is set
    float ref = -INFINITY, l = 0.f;
    bool ok = true;
    int buf = s;  // of the logits, and the parity of its turn
    uint32_t turn = 0;
    if (s < n_sub && n_it > 0) {
      {
        uint32_t z[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) z[i] = 0;
        for (int c = 0; c < D / 2; c += 32) tc::tmem_st32u(to + c, z);
        tc::tmem_wait_st();
      }
      // the tile's product of the page before is complete
      auto o_settled = [&](int j) {
        if (C::ROTATE && j > 0) pc_wait_warp(&M->pv_done[s], (j - 1) & 1, abort, a.status_dev);
        tc::tc_fence_after();  // (else the logits were issued behind it)
      };
      for (int j = 0; j < n_it; ++j) {
        ok = pc_wait_warp(&M->s_full[buf], turn, abort, a.status_dev);
        Page &P = M->page[j % PC_META];
        const bool mixed = P.mixed != 0;
        // this half's columns that the row sees (all of them unless the page is mixed)
        uint32_t see[2] = {~0u, ~0u};
        if (mixed) {
          const int c_lo = max(lo - P.base, 0) - 64 * half;
          const int c_hi = (rr >= P.r0 && rr < P.r1 ? min(hi - P.base, kBlock) : 0) - 64 * half;
#pragma unroll
          for (int k = 0; k < 2; ++k)
            see[k] = below(c_hi - 32 * k) & ~below(c_lo - 32 * k);
        }
        // P and its sum, with the references as they are; where some P of the
        // tile comes out at 2 or more (bit 14 or 30), again with moved references.
        uint32_t w[32];
        float sum;
        for (bool move = j == 0;;) {
          float x[64];
          tc::tc_fence_after();
          tc::tmem_ld64(ts + 64 * half, x);
          if (mixed) {
#pragma unroll
            for (int i = 0; i < 64; ++i)
              if (!(see[i >> 5] >> (i & 31) & 1u)) x[i] = -INFINITY;
          }
          if (move) {
            float mx[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
            for (int i = 4; i < 64; ++i) mx[i & 3] = fmaxf(mx[i & 3], x[i]);
            float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sl2;
            M->top[s][half][m] = top;
            // (a wait that gave up is known to both warps here)
            if (tc::bar_or(bar, 64, !ok)) {
              ok = false;
              break;
            }
            top = fmaxf(top, M->top[s][half ^ 1][m]);
            float f = 1.f;
            if (req >= 0 && top > ref + 1.f) {
              f = ref == -INFINITY ? 1.f : exp2f(ref - (top + kLift));
              ref = top + kLift;
              l *= f;
            }
            if (__any_sync(0xffffffffu, f != 1.f)) {
              o_settled(j);
#pragma unroll 1
              for (int c = 0; c < D / 2; c += 16) {
                float o[16];
                tmem_ld16(to + c, o);
#pragma unroll
                for (int i = 0; i < 16; ++i) o[i] *= f;
                tmem_st16(to + c, o);
              }
            }
          }
          // with nothing seen yet, any logit makes an infinite P
          const float r0 = ref == -INFINITY ? 1e30f : -ref;
          float2 sums[2] = {{0.f, 0.f}, {0.f, 0.f}};
          uint32_t any = 0;
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            float2 y = tc::ffma2(make_float2(x[2 * i], x[2 * i + 1]), make_float2(sl2, sl2),
                                 make_float2(r0, r0));
            y.x = attn::exp2_sfu(y.x);
            y.y = attn::exp2_sfu(y.y);
            w[i] = attn::pack2(y.x, y.y);
            any |= w[i];
            sums[i & 1] = tc::ffma2(y, make_float2(1.f, 1.f), sums[i & 1]);
          }
          sum = (sums[0].x + sums[1].x) + (sums[0].y + sums[1].y);
          // Both halves have read S before P goes over it.  (A thread without a
          // row has whatever was in shared memory for q: it asks for nothing.)
          const bool again =
              tc::bar_or(bar, 64, !move && (((any & 0x40004000u) && req >= 0) || !ok));
          if (!again) break;
          move = true;
        }
        if (!ok) break;
        l += sum;
        if (mixed) {
          // values that are not finite are zero in the product; the rows that
          // see them add them here
          ok = pc_wait_warp(&M->ready[j & 3], (j >> 2) & 1, abort, a.status_dev);
          if (tc::bar_or(bar, 64, !ok)) {
            ok = false;
            break;
          }
          const uint32_t bad[4] = {P.bad[0], P.bad[1], P.bad[2], P.bad[3]};
          if (bad[0] | bad[1] | bad[2] | bad[3]) {
            o_settled(j);
            const int phys = a.block_table[(long long)P.req * a.max_blocks + P.base / kBlock];
            const float r0 = ref == -INFINITY ? 0.f : ref;
#pragma unroll 1
            for (int k = 0; k < 4; ++k)
#pragma unroll 1
              for (uint32_t b = bad[k]; b; b &= b - 1) {
                const int c = 32 * k + __ffs(b) - 1;
                const bool sees = c + P.base >= lo && c + P.base < hi && rr >= P.r0 && rr < P.r1;
                uint32_t raw;
                asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];"
                             : "=r"(raw)
                             : "r"(ts + c));
                asm volatile("tcgen05.wait::ld.sync.aligned;" : "+r"(raw)::"memory");
                const float p = exp2f(__uint_as_float(raw) * sl2 - r0);
                const __nv_bfloat16 *v = reinterpret_cast<const __nv_bfloat16 *>(
                                             static_cast<const uint8_t *>(a.v_pool) +
                                             phys * a.v_page_stride + c * a.v_token_stride +
                                             kvh * a.v_head_stride) +
                                         half * (D / 2);
#pragma unroll 1
                for (int d = 0; d < D / 2; d += 16) {
                  float o[16];
                  tmem_ld16(to + d, o);
#pragma unroll
                  for (int i = 0; i < 16; ++i)
                    if (sees) o[i] += p * __bfloat162float(v[d + i]);
                  tmem_st16(to + d, o);
                }
              }
            tc::bar_sync(bar, 64);  // both halves have read S before P goes over it
          }
        }
        tc::tmem_st32u(ts + 32 * half, w);
        tc::tmem_wait_st();
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&M->p_full[buf]);
        // the next page's buffer
        if (C::ROTATE) buf += n_sub;
        if (!C::ROTATE || buf >= 3) {
          if (C::ROTATE) buf -= 3;
          turn ^= 1;
        }
        if (C::ROTATE) ts = tmem + buf * 128 + lane_off;
      }
      // the row's sum over both halves
      M->top[s][half][m] = l;
      if (tc::bar_or(bar, 64, !ok)) ok = false;
      l = half ? M->top[s][0][m] + l : l + M->top[s][1][m];
    }
    // ---- the row's result, or its part
    const long long row = (long long)t * a.n_heads + h;
    const bool mine = req >= 0 && ok;
    float scale = 1.f;
    if (G.n_parts > 1) {
      if (mine && half == 0)
        parts.ml[(long long)part * a.n_rows * a.n_heads + row] = make_float2(ref, l);
    } else {
      const paged::Joined J = paged::finish(ref, l, sink);
      scale = J.inv;
      if (mine && half == 0 && a.lse) a.lse[row] = J.lse;
    }
    // (the last product has been under way all the while)
    if (s < n_sub && n_it > 0) {
      ok = ok && pc_wait_warp(&M->o_full[s], 0, abort, a.status_dev);
      tc::tc_fence_after();
    }
    const bool zero = ref == -INFINITY && l == 0.f;  // nothing seen: O may hold nothing
    if (s < n_sub && ok) {
      // Through shared memory (the tile's Q, which no MMA reads any more), 64
      // bytes of a row at a time: a thread holds a row, and four lanes store one
      // row's piece (every lane storing its own row took 3.7 us).
      const uint32_t rows_here = __ballot_sync(0xffffffffu, mine && !(G.n_parts > 1 && zero));
      uint4 *stage = reinterpret_cast<uint4 *>(sm + s * C::TILE +
                                               (half * 4 + (warp & 3)) * (C::TILE / 8));
#pragma unroll 1
      for (int c = 0; c < D / 2; c += 32) {
        float o[32];
        if (n_it > 0)
          tc::tmem_ld32(to + c, o);
        else
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = 0.f;
        const int d = half * (D / 2) + c;
        if (G.n_parts > 1) {
          // 32 rows of 64 bytes twice: D = 64 has 2 KB a warp
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 4; ++i)
              stage[lane * 4 + (i ^ ((lane >> 1) & 3))] = make_uint4(
                  __float_as_uint(o[16 * u + 4 * i]), __float_as_uint(o[16 * u + 4 * i + 1]),
                  __float_as_uint(o[16 * u + 4 * i + 2]), __float_as_uint(o[16 * u + 4 * i + 3]));
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int r = i * 8 + (lane >> 2), q = lane & 3;
              const uint4 v = stage[r * 4 + (q ^ ((r >> 1) & 3))];
              const long long to_row = __shfl_sync(0xffffffffu, row, r);
              if (rows_here >> r & 1)
                reinterpret_cast<uint4 *>(
                    parts.o + ((long long)part * a.n_rows * a.n_heads + to_row) * D + d + 16 * u)[q] = v;
            }
          }
        } else {
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t q[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              q[e] = zero ? 0u : attn::pack2(o[8 * i + 2 * e] * scale, o[8 * i + 2 * e + 1] * scale);
            stage[lane * 4 + (i ^ ((lane >> 1) & 3))] = make_uint4(q[0], q[1], q[2], q[3]);
          }
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int r = i * 8 + (lane >> 2), q = lane & 3;
            const uint4 v = stage[r * 4 + (q ^ ((r >> 1) & 3))];
            const long long to_row = __shfl_sync(0xffffffffu, row, r);
            if (rows_here >> r & 1)
              reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.out) + to_row * D + d)[q] = v;
          }
        }
      }
    }
  }

  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  if (warp == PC_MMA) tc::tmem_dealloc(tmem, 512);
}

template <int D>
cudaError_t launch(const csa_paged_attn_args &a, const Parts &parts, cudaStream_t s) {
  using C = Cfg<D>;
  const int g = a.n_heads / a.n_kv_heads;
  ChunkGrid G;
  G.rows_tile = 128 / g;
  G.n_tiles = (a.n_rows + 2 * G.rows_tile - 1) / (2 * G.rows_tile);
  G.n_parts = parts.n;
  CUtensorMap qmap, kmap, vmap;
  if (!paged::encode_q(a, G.rows_tile, &qmap) || !paged::encode_pools(a, &kmap, &vmap))
    return cudaErrorInvalidValue;
  const size_t smem = C::OFF_MISC + sizeof(Misc);
  int dev = 0;
  cudaGetDevice(&dev);
  static bool attr[64] = {};
  if (dev < 0 || dev >= 64 || !attr[dev]) {
    const cudaError_t e = cudaFuncSetAttribute(
        paged_chunk_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) attr[dev] = true;
  }
  const long long grid = (long long)G.n_tiles * a.n_kv_heads * G.n_parts;
  if (grid > 0x7FFFFFFF) return cudaErrorInvalidValue;
  launch_begin(CSA_K_PAGED_ATTN, s);
  const cudaError_t e = launch_kernel(paged_chunk_kernel<D>, dim3((unsigned)grid), dim3(PC_THREADS),
                                      smem, s, 0, false, a, parts, G, qmap, kmap, vmap);
  launch_end(CSA_K_PAGED_ATTN, s);
  return e;
}

}  // namespace

// Parts that a tile's pages are split into: as many as make waves x (pages of a
// part + 4) + 2 + p / 16 smallest, in units of a page: a CTA's fixed cost is about
// four pages, joining costs two and a sixteenth a part.  (2048 rows of 24 heads over
// 12345 positions: 1, 2, 3, 4, 8 parts 242, 210, 203, 231, 267 us; 16 rows of 64 heads
// over 32768: 8, 13, 19, 26 parts 58, 44, 44, 58 us; 8 rows of 16 over 8000: 8, 16, 32,
// 64 parts 22, 17, 16, 19 us.  The rule takes 3, 19 and 32.)
int paged_chunk_parts(const csa_paged_attn_args &a, int sms) {
  const int rows = 2 * (128 / (a.n_heads / a.n_kv_heads));
  const long long items = (long long)((a.n_rows + rows - 1) / rows) * a.n_kv_heads;
  long long pages = a.max_blocks;
  if (a.window > 0) {
    const long long seen = ((long long)a.window + rows + kBlock - 1) / kBlock + 1;
    pages = pages < seen ? pages : seen;
  }
  // the requests that a CTA's rows may belong to, each with pages of its own
  const long long per = ((long long)a.n_rows + a.n_req - 1) / a.n_req;
  const long long runs = per >= rows ? 1 : (rows + per - 1) / (per > 0 ? per : 1);
  pages *= runs < a.n_req ? runs : a.n_req;
  int best = 1;
  double cost = 1e30;
  for (int p = 1; p <= 64 && p <= pages; ++p) {
    const long long waves = (items * p + sms - 1) / sms;
    const double c = (double)waves * ((double)((pages + p - 1) / p) + 4.0) + (p > 1 ? 2.0 + p / 16.0 : 0.0);
    if (c < cost * 0.97) {
      cost = c;
      best = p;
    }
    if (waves > 8) break;
  }
  return best;
}

cudaError_t launch_paged_chunk(const csa_paged_attn_args &a, const Parts &parts, int /*sms*/,
                               cudaStream_t s) {
  return a.head_dim == 64 ? launch<64>(a, parts, s) : launch<128>(a, parts, s);
}

}  // namespace csa
