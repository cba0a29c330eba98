// Absorbed latent attention over a paged latent cache (csa_latent_attn): tcgen05
// tiles of up to 64 (row, head) pairs against 64 positions.
//
// A position is one row of 576 channels, key and value at once: the logits take all of
// it, the values are its first 512.  With the heads of a row stacked under it, an item of
// R rows x G heads (R G <= 64) of one request does
//   S[m, j]  = q_m . (c_j, r_j)      64 x 64 x 576, both operands K-major
//   O^T[:, m] += c^T P^T             512 x pairs x 64: the latents as they lie are the
//                                    M-major operand, P in shared memory
// so a tile is fetched once for both products, and O^T takes 4 x 64 columns of tensor
// memory beside two buffers of S.  P = 2^(S scale log2(e) - ref), one reference a pair,
// which moves (and O^T is rescaled) only when some P reaches 2; it is set so that the
// largest is 2^-7, so that is seldom.
//
// P goes over the tile's rotated keys, so that a tile's logits and its product are all
// that has to be complete before its shared memory is loaded again.
//
// Roles: warp 0 loads (TMA, nine boxes of 64 channels a tile, pairs with a barrier of their
// own, two tiles in flight; boxes are asked for again as soon as their last product is
// done); warp 1 issues the logits, warp 2 the products; warp 3 looks up what the rows of
// the next item see; warps 4 .. 11 do the softmax, two warps 16 pairs, and the outputs.
//
// Few items: all tiles of all items are one list, cut into equal shares, one per SM, so
// that ragged contexts load every SM alike; a cut item leaves parts that
// latent_join_kernel puts together in order.  Many: a CTA takes R rows whole.
//
// What bounds it: a tile takes 2,200 cycles, 1,920 of them the tensor cores' (36 products
// of 64 x 64 x 16 at 32 cycles, 16 of 128 x 64 x 16 at 48: an SM reads 128 bytes of shared
// memory a cycle, so that half of their rate is the most with 64 pairs; the O of 128 would
// fill the tensor memory of one CTA, not of two, but pairs of CTAs are not built).  4 x 2
// rows of 128 heads at 131,072 positions: 295 us, 0.99 PFLOP/s; 32 rows of 16 heads,
// contexts to 16,384: 81 us, 4.7 TB/s, 12 of them the start (the list, the first loads) and
// 8 the join; one row of 128 heads over 1001: 20 us.
#include "attn_common.cuh"
#include "cache_tiles.cuh"

namespace csa {
namespace {

constexpr int LA_THREADS = 384;
constexpr int LA_LOAD = 0, LA_MMA = 1, LA_SOFT0 = 4;  // first warps
constexpr int LA_PAIRS = 64, LA_KEYS = 64;
constexpr int LA_BOXES = 9;                   // of 64 channels; the last is the rotated key
constexpr int LA_BOX = LA_KEYS * 128;         // bytes (of 64 pairs or 64 positions)
constexpr int LA_TILE = LA_BOXES * LA_BOX;
constexpr int LA_ROWS = 4096;                 // of a call whose tiles are cut into shares
constexpr int OFF_KV = LA_TILE, OFF_MISC = OFF_KV + 2 * LA_TILE;
constexpr int BAR_SOFT = 1;                   // named barrier of the softmax warps
constexpr int O_COL = 0, S_COL = 256;         // tensor memory
constexpr float kLift = 7.f;                  // log2 of the room below P = 2

// A CTA's run of tiles of one item.
struct Seg {
  int t, nr;    // rows
  int req;      // of this request
  int sub;      // group of 64 heads
  int tile, n;  // first tile (of 64 positions) and how many
  int slot;     // where its part goes, -1: the item is whole
};
constexpr int LA_JOIN = 8;    // parts of a row that are asked for together
constexpr int LA_AHEAD = 3;  // tiles that L2 is asked for before they are loaded
constexpr int LA_NEAR = 64;  // segments kept in shared memory; the rest in the workspace
static_assert(LA_PAIRS <= LA_NEAR, "rows taken whole need no more");

struct Misc {
  uint64_t q_full, q_empty, o_free, drained[2], s_full[2], info[2], info_free[2];
  // Products that are complete, tiles in turn: whoever waits for one knows only that the
  // one two before is (its shared memory was loaded again), and a parity tells a phase from
  // no more than the one before it.
  uint64_t pv_done[2];
  // P of a tile, tiles in turn: the softmax may be done with the next tile before the
  // products' warp looks for this one (with one barrier it would have been overtaken by two
  // phases and never see its own), but not with the one after, which is loaded behind this
  // tile's product.
  uint64_t p_full[2];
  uint64_t full[2][4], empty[2][4];  // pairs of boxes of a tile; the rotated keys with the last
  uint32_t tmem;
  int abort;
  int n_seg;
  int there[2];                // the tile's page is in the pool
  uint32_t bad[2];             // positions of a tile with values that are not finite
  Seg near_[LA_NEAR];
  int2 see[2][LA_PAIRS];       // what a pair sees (segments in turn)
  int4 all[2];                 // positions that all rows see [x, y), that some do [z, w)
  float top[2][LA_PAIRS];
  alignas(8) float f[LA_PAIRS];  // (read two at a time)
  uint32_t row[2][LA_PAIRS];   // a pair's (row, head) in lse, kNone: it has none
};
constexpr uint32_t kNone = 0xFFFFFFFFu;
static_assert(OFF_MISC + sizeof(Misc) <= 227 * 1024, "shared memory");

struct Parts {
  float *o;      // [slots][64][512]
  float2 *ml;    // [slots][64]
  int4 *cut;     // [CTAs]: an item that the CTA begins and does not end: row, rows, sub, last CTA
  Seg *far_;     // [CTAs][n_far]: a CTA's segments behind those in shared memory
  int n_far;
};

struct Shape {
  int gt, R, subs;  // heads and rows of an item, head groups
  int n16;          // pairs, rounded up to 16
  int shares;       // 1: the list of tiles is cut into shares
};

// 32 columns of 16 lanes: thread i holds columns 2 (i % 4) + {0, 1} of every group of
// eight, of lane i / 4 (x[4 g], x[4 g + 1]) and of lane i / 4 + 8 (x[4 g + 2], ...).
__device__ __forceinline__ void tmem_ld_16x32(uint32_t taddr, float (&x)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])::"memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) x[i] = __uint_as_float(r[i]);
}

// A box of a tensor map into L2.
__device__ __forceinline__ void prefetch_3d(const void *tmap, int x, int y, int z) {
  asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global [%0, {%1, %2, %3}];" ::"l"(
                   reinterpret_cast<uint64_t>(tmap)),
               "r"(x), "r"(y), "r"(z)
               : "memory");
}

// 16 consecutive columns of this thread's lane.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&x)[16]) {
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
  for (int i = 0; i < 16; ++i) x[i] = __uint_as_float(r[i]);
}

// The CTA's rows while its segments are found, where the tiles land afterwards.
struct Plan {
  long long *before;  // tiles of all items of earlier rows
  int *req, *lo, *hi, *tiles, *first, *nr;
  uint32_t *starts;   // a bit a row that differs from the one before it in its request
  int *run;           // a word of these: the row that starts the run its first row is in
  __device__ Plan(uint8_t *at, int n) {
    before = reinterpret_cast<long long *>(at);
    req = reinterpret_cast<int *>(before + n + 1);
    lo = req + n, hi = lo + n, tiles = hi + n, first = tiles + n, nr = first + n;
    starts = reinterpret_cast<uint32_t *>(nr + n);
    run = reinterpret_cast<int *>(starts + (n + 31) / 32);
  }
  static constexpr int bytes(int n) { return 8 * (n + 1) + 24 * n + (n + 31) / 32 * 8; }
};

static_assert(Plan::bytes(LA_ROWS) <= 2 * LA_TILE, "the list of rows");

__global__ void __launch_bounds__(LA_THREADS, 1)
    latent_attn_kernel(csa_latent_attn_args a, Parts parts, Shape H,
                       const __grid_constant__ CUtensorMap qmap,
                       const __grid_constant__ CUtensorMap qrmap,
                       const __grid_constant__ CUtensorMap cmap,
                       const __grid_constant__ CUtensorMap rmap) {
  extern __shared__ __align__(1024) uint8_t sm[];
  Misc *M = reinterpret_cast<Misc *>(sm + OFF_MISC);
  tc::griddep_wait();
  tc::griddep_launch_dependents();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tc::smem_u32(sm) & 1023u) {
    if (tid == 0) flag(a.status_dev, CSA_DEV_TIMEOUT);
    return;
  }
  if (warp == LA_MMA) tc::tmem_alloc(&M->tmem, 512);
  if (warp == LA_SOFT0 && lane < 4)
    paged::prefetch_map(lane == 0 ? &qmap : (lane == 1 ? &qrmap : (lane == 2 ? &cmap : &rmap)));
  volatile int *abort = &M->abort;
  Seg *far_ = parts.far_ + (long long)blockIdx.x * parts.n_far;

  // ================================================================ the CTA's segments
  // rows [row0, row0 + n): all of the call, or this CTA's own
  const int own = H.shares ? 0 : (int)(gridDim.x - 1 - blockIdx.x);
  const int row0 = H.shares ? 0 : own / H.subs * H.R;
  const int n = H.shares ? a.n_rows : min(H.R, a.n_rows - row0);
  const int subs = H.shares ? H.subs : 1, sub0 = H.shares ? 0 : own % H.subs;
  {
    const Plan plan(sm + OFF_KV, n);
    for (int r = tid; r < ((n + 31) & ~31); r += LA_THREADS) {
      int b = -1, lo = 0, hi = 0;
      if (r < n) {
        b = a.row_req[row0 + r];
        if (b >= a.n_req) {
          if ((H.shares ? blockIdx.x : sub0) == 0) flag(a.status_dev, CSA_DEV_BAD_POS);
          b = -1;
        }
        if (b >= 0) paged::visible_range(a, a.kv_len[b], a.row_pos[row0 + r], lo, hi);
        plan.req[r] = b, plan.lo[r] = lo, plan.hi[r] = hi;
      }
      const bool start = r < n && (r == 0 || a.row_req[row0 + r - 1] != a.row_req[row0 + r]);
      const uint32_t bits = __ballot_sync(0xffffffffu, start);
      if (lane == 0) plan.starts[r >> 5] = bits;
    }
    if (tid == 0) {
      tc::mbar_init(&M->q_full, 1);
      tc::mbar_init(&M->q_empty, 1);
      tc::mbar_init(&M->o_free, 8);
      for (int i = 0; i < 2; ++i) {
        tc::mbar_init(&M->drained[i], 1);
        tc::mbar_init(&M->pv_done[i], 1);
        tc::mbar_init(&M->p_full[i], 8);
        tc::mbar_init(&M->info[i], 1);
        tc::mbar_init(&M->info_free[i], 8);
        tc::mbar_init(&M->s_full[i], 2);
        for (int c = 0; c < 4; ++c) tc::mbar_init(&M->full[i][c], 1);
        for (int c = 0; c < 4; ++c) tc::mbar_init(&M->empty[i][c], 1);
      }
      M->abort = 0;
      M->bad[0] = M->bad[1] = 0;
      tc::mbar_fence_init();
    }
    __syncthreads();
    if (n > 32) {
      if (warp == 0) {
        int last = 0;
        for (int w0 = 0; w0 * 32 < n; w0 += 32) {
          const int w = w0 + lane;
          const uint32_t bits = w * 32 < n ? plan.starts[w] : 0;
          int x = bits ? w * 32 + 31 - __clz(bits) : -1;  // the word's last start
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x = max(x, y);
          }
          const int before = __shfl_up_sync(0xffffffffu, x, 1);
          if (w * 32 < n) plan.run[w] = max(last, lane ? before : -1);
          last = max(last, __shfl_sync(0xffffffffu, x, 31));
        }
      }
      __syncthreads();
    }
    for (int r = tid; r < n; r += LA_THREADS) {
      const int b = plan.req[r];
      const uint32_t bits = plan.starts[r >> 5] & (0xffffffffu >> (31 - (r & 31)));
      const int run = bits ? (r & ~31) + 31 - __clz(bits) : plan.run[r >> 5];
      int tiles = 0, first = 0, k = 0;
      if (b >= 0 && (r - run) % H.R == 0) {
        int lo = 0x7FFFFFFF, hi = 0;
        for (; k < H.R && r + k < n && plan.req[r + k] == b; ++k)
          if (plan.lo[r + k] < plan.hi[r + k]) {
            lo = min(lo, plan.lo[r + k]);
            hi = max(hi, plan.hi[r + k]);
          }
        if (lo < hi) {
          first = lo / LA_KEYS;
          tiles = (hi - 1) / LA_KEYS - first + 1;
        }
      }
      plan.tiles[r] = tiles, plan.first[r] = first, plan.nr[r] = k;
    }
    __syncthreads();
    if (warp == 0) {
      long long sum = 0;
      int most = 0, items = 0;  // tiles of the longest item; items
      for (int r0 = 0; r0 < n; r0 += 32) {
        const int r = r0 + lane;
        const int tiles = r < n ? plan.tiles[r] : 0;
        const long long mine = (long long)tiles * subs;
        most = max(most, tiles);
        items += __popc(__ballot_sync(0xffffffffu, tiles > 0)) * subs;
        long long x = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const long long y = __shfl_up_sync(0xffffffffu, x, o);
          if (lane >= o) x += y;
        }
        if (r < n) plan.before[r] = sum + x - mine;
        sum += __shfl_sync(0xffffffffu, x, 31);
      }
      if (lane == 0) plan.before[n] = sum;
      most = __reduce_max_sync(0xffffffffu, most);
      __syncwarp();
      if (lane == 0) {
        const long long W = sum;
        long long N = H.shares ? (W < gridDim.x ? W : gridDim.x) : 1;
        // Items of one length: whole shares an item, so that the items of one cache (its
        // rows, its head groups) go over the same tiles at the same time and L2 serves
        // all but the first, where that leaves at most an eighth of the SMs out.
        if (items > 0 && W == (long long)items * most && N > items && N % items * 8 <= N) N -= N % items;
        const long long c = H.shares ? blockIdx.x : 0;
        int n_seg = 0;
        int4 cut = make_int4(-1, 0, 0, 0);
        if (W > 0 && c < N) {
          const long long w0 = c * W / N, w1 = (c + 1) * W / N;
          int l = 0, h = n;
          while (h - l > 1) {
            const int mid = (l + h) >> 1;
            if (plan.before[mid] <= w0)
              l = mid;
            else
              h = mid;
          }
          for (long long w = w0; w < w1;) {
            while (plan.tiles[l] == 0) ++l;
            const int P = plan.tiles[l], sub = (int)((w - plan.before[l]) / P);
            const int pa = (int)(w - plan.before[l] - (long long)sub * P);
            const int pb = (int)min((long long)P, pa + (w1 - w));
            Seg s;
            s.t = row0 + l, s.nr = plan.nr[l], s.req = plan.req[l], s.sub = sub0 + sub;
            s.tile = plan.first[l] + pa, s.n = pb - pa;
            s.slot = pa > 0 ? 2 * (int)c : (pb < P ? 2 * (int)c + 1 : -1);
            if (pa == 0 && pb < P)
              cut = make_int4(s.t, s.nr, s.sub, (int)(((w + P) * N - 1) / W));
            if (n_seg < LA_NEAR)
              M->near_[n_seg] = s;
            else
              far_[n_seg] = s;
            ++n_seg;
            w += pb - pa;
            if (pb == P && sub == subs - 1) ++l;
          }
        }
        M->n_seg = n_seg;
        if (H.shares) parts.cut[c] = cut;
      }
    }
    // rows of items that see nothing
    for (int r = H.shares ? (int)blockIdx.x : 0; r < n; r += H.shares ? (int)gridDim.x : 1) {
      if (plan.nr[r] == 0 || plan.tiles[r] != 0) continue;
      const int h0 = H.shares ? 0 : sub0 * H.gt, h1 = H.shares ? a.n_heads : min(a.n_heads, h0 + H.gt);
      for (int k = 0; k < plan.nr[r]; ++k) {
        const long long at = (long long)(row0 + r + k) * a.n_heads;
        for (int i = tid; i < (h1 - h0) * (kLatent / 8); i += LA_THREADS)
          reinterpret_cast<uint4 *>(a.out)[(at + h0) * (kLatent / 8) + i] = make_uint4(0, 0, 0, 0);
        if (a.lse)
          for (int h = h0 + tid; h < h1; h += LA_THREADS)
            a.lse[at + h] = a.sink ? a.sink[h] : -INFINITY;
      }
    }
    __syncthreads();
  }
  const int n_seg = M->n_seg;
  auto seg_at = [&](int i) { return i < LA_NEAR ? M->near_[i] : far_[i]; };
  tc::fence_async_shared();  // (the plan was where the tiles land)
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = __reduce_or_sync(0xffffffffu, M->tmem);

  if (warp == LA_LOAD) {
    // ================================================================ loads
    if (lane == 0) {
      bool ok = true;
      uint32_t it = 0, n_q = 0;
      for (int s = 0; s < n_seg && ok; ++s) {
        const Seg g = seg_at(s);
        const int32_t *table = a.block_table + (long long)g.req * a.max_blocks;
        const int end = g.tile + g.n;
        int asked = g.tile + 1, phys = table[g.tile >> 1];  // (prefetches keep to the segment)
        ok = cache::wait(&M->q_empty, (s & 1) ^ 1, abort, a.status_dev);
        if (!ok) break;
        ++n_q;
        tc::mbar_arrive_expect_tx(&M->q_full, LA_BOXES * 128 * H.gt * H.R);
        tc::tma_load_3d(sm + 8 * LA_BOX, &qrmap, 0, g.sub * H.gt, g.t, &M->q_full);
        for (int c = 0; c < 8; ++c)
          tc::tma_load_3d(sm + c * LA_BOX, &qmap, c * 64, g.sub * H.gt, g.t, &M->q_full);
        for (int i = 0; i < g.n && ok; ++i, ++it) {
          const int st = it & 1, tile = g.tile + i;
          const uint32_t par = ((it >> 1) & 1) ^ 1;
          const int next = i + 1 < g.n ? table[(tile + 1) >> 1] : 0;
          const bool there = phys >= 0 && phys < a.n_blocks;
          uint8_t *dst = sm + OFF_KV + st * LA_TILE;
          for (int c = 0; c < 4; ++c) {
            ok = cache::wait(&M->empty[st][c], par, abort, a.status_dev);
            if (!ok) break;
            if (c == 0) M->there[st] = there;
            if (there) {
              uint64_t *bar = &M->full[st][c];
              tc::mbar_arrive_expect_tx(bar, c == 3 ? 3 * LA_BOX : 2 * LA_BOX);
              for (int e = 2 * c; e < 2 * c + 2; ++e)
                tc::tma_load_3d(dst + e * LA_BOX, &cmap, e * 64, (tile & 1) * LA_KEYS, phys, bar);
              if (c == 3)
                tc::tma_load_3d(dst + 8 * LA_BOX, &rmap, 0, (tile & 1) * LA_KEYS, phys, bar);
            } else {
              tc::mbar_arrive(&M->full[st][c]);
            }
          }
          if (!there) flag(a.status_dev, CSA_DEV_BAD_BLOCK);
          for (; asked < min(tile + LA_AHEAD, end); ++asked) {
            const int pg = table[asked >> 1];
            if (asked < tile + 2 || pg < 0 || pg >= a.n_blocks) continue;
            for (int c = 0; c < 8; ++c)
              prefetch_3d(&cmap, c * 64, (asked & 1) * LA_KEYS, pg);
            prefetch_3d(&rmap, 0, (asked & 1) * LA_KEYS, pg);
          }
          phys = next;
        }
      }
      // whatever was asked for has landed before the CTA retires
      if (!ok || *abort) {
        if (n_q > 0) tc::mbar_wait(&M->q_full, (n_q - 1) & 1, 50000000ull);
        for (uint32_t k = it > 1 ? it - 2 : 0; k <= it; ++k)
          for (int c = 0; c < 4; ++c)
            tc::mbar_wait(&M->full[k & 1][c], (k >> 1) & 1, 5000000ull);
      }
    }
    __syncwarp();
  } else if (warp == LA_MMA) {
    // ================================================================ logits
    // (In order: a tile is loaded again only after its product, so its arrival also says
    // that the softmax has read the logits before in this buffer and that nothing reads
    // the P before.)
    if (tc::elect_one()) {
      constexpr uint32_t idesc = tc::idesc_bf16_f32(LA_PAIRS, LA_KEYS);
      const uint32_t base = tc::smem_u32(sm);
      const uint64_t dq = tc::desc_sw128(base), dk = tc::desc_sw128(base + OFF_KV);
      bool ok = true;
      int it = 0;
      for (int s = 0; s < n_seg && ok; ++s) {
        const int end = it + seg_at(s).n;
        ok = cache::wait(&M->q_full, s & 1, abort, a.status_dev);
        for (; it < end && ok; ++it) {
          const int st = it & 1;
          const uint32_t d = tmem + S_COL + st * 64;
          const uint64_t k = dk + ((st * LA_TILE) >> 4);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            ok = ok && cache::wait(&M->full[st][c], (it >> 1) & 1, abort, a.status_dev);
            if (!ok) break;
            tc::tc_fence_after();
#pragma unroll
            for (int e = 2 * c; e < (c == 3 ? 9 : 2 * c + 2); ++e)
              cache::mma4<2, 2>(d, dq + ((e * LA_BOX) >> 4), k + ((e * LA_BOX) >> 4), idesc, e > 0);
          }
          if (!ok) break;
          tc::mma_commit(&M->s_full[st]);
          tc::mbar_arrive(&M->s_full[st]);  // hands on what the loads were told
        }
        if (ok) tc::mma_commit(&M->q_empty);
      }
      // every issued MMA has completed before tensor memory is released
      tc::mma_commit(&M->drained[0]);
      tc::mbar_wait(&M->drained[0], 0, 100000000ull);
    }
    __syncwarp();
  } else if (warp == LA_MMA + 1) {
    // ================================================================ products
    // (A warp of their own: one that issues both has to ask which is ready, and each
    // question costs it a hundred cycles.)
    if (tc::elect_one()) {
      const uint32_t idesc = tc::idesc_bf16_f32(128, H.n16) | (1u << 15);  // c^T is M-major
      const uint32_t base = tc::smem_u32(sm);
      const uint64_t dv = tc::desc_sw128_mn(base + OFF_KV, LA_BOX, 1024);
      const uint64_t dp = tc::desc_sw128(base + OFF_KV + 8 * LA_BOX);
      bool ok = true;
      int it = 0;
      for (int s = 0; s < n_seg && ok; ++s) {
        const int n_it = seg_at(s).n;
        if (s > 0) ok = cache::wait(&M->o_free, (s - 1) & 1, abort, a.status_dev);
        for (int i = 0; i < n_it && ok; ++i, ++it) {
          ok = cache::wait(&M->p_full[it & 1], (it >> 1) & 1, abort, a.status_dev);
          if (!ok) break;
          tc::tc_fence_after();
          const uint64_t at = ((it & 1) * LA_TILE) >> 4;
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            cache::mma4<128, 2>(tmem + O_COL + b * 64, dv + at + ((2 * b * LA_BOX) >> 4), dp + at, idesc,
                         i > 0);
            tc::mma_commit(&M->empty[it & 1][b]);
          }
          tc::mma_commit(&M->pv_done[it & 1]);
        }
      }
      tc::mma_commit(&M->drained[1]);
      tc::mbar_wait(&M->drained[1], 0, 100000000ull);
    }
    __syncwarp();
  } else if (warp == LA_MMA + 2) {
    // ================================================================ what the rows see
    // (a segment ahead: the softmax would wait for memory twice at every item's start)
    for (int s = 0; s < n_seg; ++s) {
      const Seg g = seg_at(s);
      const int len = a.kv_len[g.req];
      int pos[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) pos[e] = 32 * e + lane < g.nr ? a.row_pos[g.t + 32 * e + lane] : 0;
      // (the tables of the segment before the last: its outputs are written)
      if (!__all_sync(0xffffffffu, cache::wait(&M->info_free[s & 1], ((s >> 1) & 1) ^ 1, abort,
                                           a.status_dev)))
        break;
      int all_lo = 0, all_hi = 0x7FFFFFFF, any_lo = 0x7FFFFFFF, any_hi = 0;
      int2 see[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        int lo, hi;
        paged::visible_range(a, len, pos[e], lo, hi);
        if (32 * e + lane < g.nr) {
          if (lo < hi) {
            all_lo = max(all_lo, lo), all_hi = min(all_hi, hi);
            any_lo = min(any_lo, lo), any_hi = max(any_hi, hi);
          } else {
            all_hi = 0;  // a row that sees nothing
          }
        }
        see[e] = make_int2(lo, hi);
      }
      all_lo = __reduce_max_sync(0xffffffffu, all_lo);
      all_hi = __reduce_min_sync(0xffffffffu, all_hi);
      any_lo = __reduce_min_sync(0xffffffffu, any_lo);
      any_hi = __reduce_max_sync(0xffffffffu, any_hi);
      if (lane == 0) M->all[s & 1] = make_int4(all_lo, all_hi, any_lo, any_hi);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        // pair m is row m / gt (a lane's register) and head m % gt
        const int m = 32 * e + lane, r = m / H.gt, h = g.sub * H.gt + m % H.gt;
        int2 x, y;
        x.x = __shfl_sync(0xffffffffu, see[0].x, r & 31), x.y = __shfl_sync(0xffffffffu, see[0].y, r & 31);
        y.x = __shfl_sync(0xffffffffu, see[1].x, r & 31), y.y = __shfl_sync(0xffffffffu, see[1].y, r & 31);
        const bool in = r < g.nr && h < a.n_heads;
        M->see[s & 1][m] = in ? (r < 32 ? x : y) : make_int2(0, 0);
        M->row[s & 1][m] = in ? (uint32_t)(g.t + r) * a.n_heads + h : kNone;
      }
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&M->info[s & 1]);
    }
  } else if (warp >= LA_SOFT0) {
    // ================================================================ softmax and outputs
    const int qd = warp & 3, half = (warp - LA_SOFT0) >> 2;
    const int ma = 16 * qd + (lane >> 2), fc = (lane & 3) * 2;  // pairs ma, ma + 8
    const uint32_t lane_off = (uint32_t)(qd * 32) << 16;
    const float sl2 = a.softmax_scale * paged::kLog2e;
    uint32_t it = 0;
    auto wait = [&](uint64_t *bar, uint32_t turn) {
      return (bool)__all_sync(0xffffffffu, cache::wait(bar, turn & 1, abort, a.status_dev));
    };
    // ok: no wait of this warp gave up; given_up: some warp's did
    bool ok = true, given_up = false;
    for (int s = 0; s < n_seg && !given_up; ++s) {
      const Seg g = seg_at(s);
      // what the item's rows see: all of them, some, and this thread's two
      ok = wait(&M->info[s & 1], s >> 1) && ok;
      const int4 all = M->all[s & 1];
      const int all_lo = all.x, all_hi = all.y, any_lo = all.z, any_hi = all.w;
      const int2 see[2] = {M->see[s & 1][ma], M->see[s & 1][ma + 8]};
      const int lo[2] = {see[0].x, see[1].x}, hi[2] = {see[0].y, see[1].y};
      float ref[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
      // bits of a P of 2 or more, of rows that see something
      const uint32_t big[2] = {hi[0] > lo[0] ? 0x40004000u : 0u, hi[1] > lo[1] ? 0x40004000u : 0u};
      const float2 one = make_float2(1.f, 1.f);
      for (int i = 0; i < g.n; ++i, ++it) {
        const int st = it & 1, base = (g.tile + i) * LA_KEYS;
        ok = wait(&M->s_full[st], it >> 1) && ok;
        const bool there = ok && M->there[st];
        const bool mixed = !there || base < all_lo || all_hi - base < LA_KEYS;
        tc::tc_fence_after();
        float x[16];
        tmem_ld_16x32(tmem + S_COL + st * 64 + 32 * half + lane_off, x);
        if (mixed) {
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const int e = (k >> 1) & 1, j = base + 32 * half + (k >> 2) * 8 + fc + (k & 1);
            if (!there || j < lo[e] || j >= hi[e]) x[k] = -INFINITY;
          }
        }
        float2 p[8];
        uint32_t w[8];
        for (bool move = i == 0;;) {
          if (move) {
            float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int k = 0; k < 16; ++k) top[(k >> 1) & 1] = fmaxf(top[(k >> 1) & 1], x[k]);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], 1));
              top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], 2));
              if ((lane & 3) == 0) M->top[half][ma + 8 * e] = top[e] * sl2;
            }
            tc::bar_sync(BAR_SOFT, 256);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float t = fmaxf(M->top[0][ma + 8 * e], M->top[1][ma + 8 * e]);
              float f = 1.f;
              if (t > ref[e] + 1.f && hi[e] > lo[e]) {
                f = ref[e] == -INFINITY ? 1.f : exp2f(ref[e] - (t + kLift));
                ref[e] = t + kLift;
                l[e] *= f;
              }
              if (half == 0 && (lane & 3) == 0) M->f[ma + 8 * e] = f;
            }
            if (i > 0) {
              // O^T of all pairs, once the product before is complete
              ok = wait(&M->pv_done[(it - 1) & 1], (it - 1) >> 1) && ok;
              tc::bar_sync(BAR_SOFT, 256);
              tc::tc_fence_after();
#pragma unroll 1
              for (int c = 0; c < 128; c += 32) {
                if ((c & 63) >= H.n16) continue;
                const uint32_t at = tmem + O_COL + half * 128 + c + lane_off;
                float o[32];
                tc::tmem_ld32(at, o);
#pragma unroll
                for (int k = 0; k < 32; ++k) o[k] *= M->f[(c & 63) + k];
                tc::tmem_st32(at, o);
              }
              tc::tmem_wait_st();
              tc::tc_fence_before();
            }
            // (the next reading of top and f is behind this barrier)
            tc::bar_sync(BAR_SOFT, 256);
          }
          uint32_t any = 0;
          const float r0[2] = {ref[0] == -INFINITY ? 1e30f : -ref[0],
                               ref[1] == -INFINITY ? 1e30f : -ref[1]};
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int e = k & 1;
            float2 y = tc::ffma2(make_float2(x[2 * k], x[2 * k + 1]), make_float2(sl2, sl2),
                                 make_float2(r0[e], r0[e]));
            y.x = attn::exp2_sfu(y.x), y.y = attn::exp2_sfu(y.y);
            p[k] = y;
            w[k] = attn::pack2(y.x, y.y);
            any |= w[k] & big[e];
          }
          // (a wait that gave up is known to all of them from here: every thread takes
          // the same way past the barriers)
          if (!tc::bar_or(BAR_SOFT, 256, !ok || (!move && any))) break;
          if (tc::bar_or(BAR_SOFT, 256, !ok)) {
            given_up = true;
            break;
          }
          if (move) break;
          move = true;
        }
        if (given_up) break;
        if (mixed) {
          // Positions that not every row sees: latents that are not finite become zero
          // (zero times them is not zero), and rows that see them NaN.
          // Four positions of a warp at a time, eight lanes a row of a box.
#pragma unroll 1
          for (int key4 = 4 * (warp - LA_SOFT0); key4 < LA_KEYS; key4 += 32) {
            const int key = key4 + (lane >> 3), j = base + key;
            const bool part = !there || j < all_lo || j >= all_hi;
            if (!__any_sync(0xffffffffu, part)) continue;
            bool zero = part && (!there || j < any_lo || j >= any_hi);
            const bool look = part && !zero;
            uint4 *row = reinterpret_cast<uint4 *>(sm + OFF_KV + st * LA_TILE + key * 128) + (lane & 7);
            if (__any_sync(0xffffffffu, look)) {
              uint32_t odd = 0;
#pragma unroll 4
              for (int u = 0; u < 8; ++u) {
                const uint4 v = row[u * (LA_BOX / 16)];
                odd |= paged::not_finite2(v.x) | paged::not_finite2(v.y) | paged::not_finite2(v.z) |
                       paged::not_finite2(v.w);
              }
#pragma unroll
              for (int o = 1; o < 8; o <<= 1) odd |= __shfl_xor_sync(0xffffffffu, odd, o);
              if (look && odd) {
                zero = true;
                if ((lane & 7) == 0) atomicOr(&M->bad[key >> 5], 1u << (key & 31));
              }
            }
            if (zero)
#pragma unroll 4
              for (int u = 0; u < 8; ++u) row[u * (LA_BOX / 16)] = make_uint4(0, 0, 0, 0);
          }
          tc::bar_sync(BAR_SOFT, 256);
          const uint32_t bad[2] = {M->bad[0], M->bad[1]};
          if (bad[0] | bad[1]) {
#pragma unroll 1
            for (int k = 0; k < LA_KEYS; ++k)
              if (bad[k >> 5] >> (k & 31) & 1u)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                  if (base + k >= lo[e] && base + k < hi[e]) l[e] = NAN;
            tc::bar_sync(BAR_SOFT, 256);
            if (tid == LA_SOFT0 * 32) M->bad[0] = M->bad[1] = 0;
          }
        }
        // P goes over the tile's rotated keys, which nothing reads any more
        uint8_t *P = sm + OFF_KV + st * LA_TILE + 8 * LA_BOX;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int m = ma + 8 * (k & 1), chunk = 4 * half + (k >> 1);
          *reinterpret_cast<uint32_t *>(P + m * 128 + ((chunk ^ (m & 7)) << 4) + fc * 2) = w[k];
        }
        tc::fence_async_shared();
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&M->p_full[st]);
        // (the sums while the product runs)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float2 y = tc::ffma2(tc::ffma2(p[e], one, p[2 + e]), one, tc::ffma2(p[4 + e], one, p[6 + e]));
          l[e] += y.x + y.y;
        }
      }
      // ---- the item's outputs, or its part
      if (given_up) break;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
        l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
        if ((lane & 3) == 0) M->top[half][ma + 8 * e] = l[e];
      }
      tc::bar_sync(BAR_SOFT, 256);
      if (half == 0 && (lane & 3) == 0)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int m = ma + 8 * e;
          const float sum = M->top[0][m] + M->top[1][m];
          float f = 0.f;
          const uint32_t row = M->row[s & 1][m];
          if (row != kNone) {
            const int h = g.sub * H.gt + m % H.gt;
            if (g.slot >= 0) {
              parts.ml[(long long)g.slot * LA_PAIRS + m] = make_float2(ref[e], sum);
            } else {
              const paged::Joined J = paged::finish(ref[e], sum, a.sink ? a.sink[h] : -INFINITY);
              f = ref[e] == -INFINITY && sum == 0.f ? 0.f : J.inv;
              if (a.lse) a.lse[row] = J.lse;
            }
          }
          M->f[m] = f;
        }
      ok = wait(&M->pv_done[(it - 1) & 1], (it - 1) >> 1) && ok;
      if (tc::bar_or(BAR_SOFT, 256, !ok)) break;
      tc::tc_fence_after();
#pragma unroll 1
      for (int blk = 2 * half; blk < 2 * half + 2; ++blk) {
        const int d = blk * 128 + 32 * qd + lane;
        // (16 pairs at a time: more take registers from the tiles' loop, 304 -> 317 us for
        // 4 x 2 rows of 128 heads at 131,072 positions)
#pragma unroll 1
        for (int c = 0; c < H.n16; c += 16) {
          float o[16];
          tmem_ld16(tmem + O_COL + blk * 64 + c + lane_off, o);
          if (g.slot >= 0) {
            float *to = parts.o + ((long long)g.slot * LA_PAIRS + c) * kLatent + d;
#pragma unroll
            for (int k = 0; k < 16; ++k)
              if (M->row[s & 1][c + k] != kNone) to[k * kLatent] = o[k];
          } else {
            // two pairs at a time: even lanes store two channels of the first, odd ones
            // of the second
            __nv_bfloat16 *to = static_cast<__nv_bfloat16 *>(a.out) + (d & ~1);
#pragma unroll
            for (int k = 0; k < 16; k += 2) {
              const float2 f = *reinterpret_cast<const float2 *>(M->f + c + k);  // (0: saw nothing)
              const uint32_t both = attn::pack2(f.x == 0.f ? 0.f : o[k] * f.x, f.y == 0.f ? 0.f : o[k + 1] * f.y);
              const uint32_t other = __shfl_xor_sync(0xffffffffu, both, 1);
              const uint32_t row = M->row[s & 1][c + k + (lane & 1)];
              if (row != kNone)
                *reinterpret_cast<uint32_t *>(to + (long long)row * kLatent) =
                    lane & 1 ? __byte_perm(other, both, 0x7632) : __byte_perm(both, other, 0x5410);
            }
          }
        }
      }
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        tc::mbar_arrive(&M->o_free);
        tc::mbar_arrive(&M->info_free[s & 1]);
      }
      tc::bar_sync(BAR_SOFT, 256);  // (before top and f are written again)
    }
  }

  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  if (warp == LA_MMA) tc::tmem_dealloc(tmem, 512);
}

// The pairs of items that were cut: CTA (m, c) joins pair m of the item that CTA c of
// the attention began and did not end, parts in order.
__global__ void __launch_bounds__(128)
    latent_join_kernel(csa_latent_attn_args a, Parts parts, Shape H, int n_ctas) {
  tc::griddep_wait();
  tc::griddep_launch_dependents();
  const int c = blockIdx.y, m = blockIdx.x, tid = threadIdx.x;
  const int4 it = parts.cut[c];
  if (it.x < 0 || it.w >= n_ctas) return;
  const int r = m / H.gt, h = it.z * H.gt + m % H.gt;
  if (r >= it.y || h >= a.n_heads) return;
  const int n = it.w - c + 1;
  auto slot = [&](int s) { return (2ll * (c + s) + (s == 0 ? 1 : 0)) * LA_PAIRS + m; };
  // LA_JOIN parts at a time, statistics and outputs asked for together: what this takes is
  // the way to memory.  The sums move to a larger reference as it comes.
  float ref = -INFINITY, acc[4] = {}, l = 0.f;
  for (int s0 = 0; s0 < n; s0 += LA_JOIN) {
    float2 ml[LA_JOIN];
    float4 o[LA_JOIN];
#pragma unroll
    for (int k = 0; k < LA_JOIN; ++k) {
      if (s0 + k >= n) break;
      ml[k] = parts.ml[slot(s0 + k)];
      o[k] = reinterpret_cast<const float4 *>(parts.o + slot(s0 + k) * kLatent)[tid];
    }
    float top = ref;
#pragma unroll
    for (int k = 0; k < LA_JOIN; ++k)
      if (s0 + k < n) top = fmaxf(top, ml[k].x);
    const float f = ref == -INFINITY ? 0.f : exp2f(ref - top);
    if (ref != -INFINITY) l *= f;  // (l is NaN where a logit was)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[e] *= f;
    ref = top;
#pragma unroll
    for (int k = 0; k < LA_JOIN; ++k) {
      if (s0 + k >= n || (ml[k].x == -INFINITY && ml[k].y == 0.f)) continue;  // nothing seen there
      const float w = ml[k].x == -INFINITY ? ml[k].y : exp2f(ml[k].x - ref);
      l += w * ml[k].y;
      acc[0] += w * o[k].x, acc[1] += w * o[k].y, acc[2] += w * o[k].z, acc[3] += w * o[k].w;
    }
  }
  const paged::Joined J = paged::finish(ref, l, a.sink ? a.sink[h] : -INFINITY);
  const bool zero = ref == -INFINITY && l == 0.f;
  const long long row = (long long)(it.x + r) * a.n_heads + h;
  __nv_bfloat162 out[2];
#pragma unroll
  for (int e = 0; e < 2; ++e)
    out[e] = zero ? __floats2bfloat162_rn(0.f, 0.f)
                  : __floats2bfloat162_rn(acc[2 * e] * J.inv, acc[2 * e + 1] * J.inv);
  reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(a.out) + row * kLatent)[tid] =
      *reinterpret_cast<const uint2 *>(out);
  if (a.lse && tid == 0) a.lse[row] = J.lse;
}

// CTAs of a call whose rows are taken whole.
long long blocks_of(const csa_latent_attn_args &a, const Shape &H) {
  return (long long)((a.n_rows + H.R - 1) / H.R) * H.subs;
}

Shape shape_of(const csa_latent_attn_args &a) {
  Shape H;
  H.gt = a.n_heads < LA_PAIRS ? a.n_heads : LA_PAIRS;
  H.R = LA_PAIRS / H.gt;
  H.subs = (a.n_heads + LA_PAIRS - 1) / LA_PAIRS;
  H.n16 = (H.gt * H.R + 15) / 16 * 16;
  // Whole rows where one request's items fill the SMs in their last round too (its rows
  // then go over the same tiles at the same time: 600 rows of 16 heads over 8000 positions
  // 147 us, in shares 175), and where there are many items of several (2000 rows of 32
  // heads, 4 requests over 2000: 160 against 185); else shares (1200 rows of 8 heads, 3
  // ragged requests to 4000: 80 us against 97).
  const long long items = blocks_of(a, H), sms = sm_count(), rounds = (items + sms - 1) / sms;
  const bool filled = a.n_req == 1 && items * 10 >= rounds * sms * 9;
  H.shares = !filled && (a.n_rows <= 512 || (a.n_rows <= LA_ROWS && items <= 2 * sms));
  return H;
}

struct Layout {
  size_t ml, cut, far_, total;
  int n_far;
};
Layout layout(const csa_latent_attn_args &a, int sms) {
  Layout L{0, 0, 0, 0, 0};
  const Shape H = shape_of(a);
  if (!H.shares) return L;  // (a CTA that takes its rows whole has no more segments than rows)
  const long long items = (long long)a.n_rows * H.subs;  // (of a CTA, at most)
  L.n_far = items > LA_NEAR ? (int)items : 0;
  const size_t slots = 2 * (size_t)sms * LA_PAIRS;
  L.ml = align_up(slots * kLatent * sizeof(float), 256);
  L.cut = L.ml + align_up(slots * sizeof(float2), 256);
  L.far_ = L.cut + align_up(sms * sizeof(int4), 256);
  L.total = L.far_ + align_up((size_t)sms * L.n_far * sizeof(Seg), 256);
  return L;
}

// [x, y, z] of the given strides (bytes).
bool encode(CUtensorMap *map, const void *base, const cuuint64_t (&dims)[3], int64_t s1, int64_t s2,
            const cuuint32_t (&box)[3]) {
  const cuuint64_t strides[2] = {(cuuint64_t)s1, (cuuint64_t)s2};
  return cache::encode(map, base, 3, dims, strides, box, CU_TENSOR_MAP_L2_PROMOTION_L2_128B);
}

}  // namespace

size_t latent_attn_workspace(const csa_latent_attn_args &a) { return layout(a, sm_count()).total; }

cudaError_t launch_latent_attn(const csa_latent_attn_args &a, cudaStream_t s) {
  const int sms = sm_count();
  const Shape H = shape_of(a);
  const Layout L = layout(a, sms);
  uint8_t *ws = static_cast<uint8_t *>(a.workspace);
  const Parts parts{reinterpret_cast<float *>(ws), reinterpret_cast<float2 *>(ws + L.ml),
                    reinterpret_cast<int4 *>(ws + L.cut), reinterpret_cast<Seg *>(ws + L.far_),
                    L.n_far};
  CUtensorMap qmap, qrmap, cmap, rmap;
  const cuuint64_t rows = a.n_rows, heads = a.n_heads, pages = a.n_blocks;
  const cuuint32_t qbox[3] = {64, (cuuint32_t)H.gt, (cuuint32_t)H.R}, kbox[3] = {64, LA_KEYS, 1};
  if (!encode(&qmap, a.q, {kLatent, heads, rows}, a.q_head_stride, a.q_row_stride, qbox) ||
      !encode(&qrmap, a.q_rope, {kRopeDim, heads, rows}, a.q_rope_head_stride, a.q_rope_row_stride,
              qbox) ||
      !encode(&cmap, a.c_pool, {kLatent, kBlock, pages}, a.c_token_stride, a.c_page_stride, kbox) ||
      !encode(&rmap, a.r_pool, {kRopeDim, kBlock, pages}, a.r_token_stride, a.r_page_stride, kbox))
    return cudaErrorInvalidValue;
  const size_t smem = OFF_MISC + sizeof(Misc);
  int dev = 0;
  cudaGetDevice(&dev);
  static bool attr[64] = {};
  if (dev < 0 || dev >= 64 || !attr[dev]) {
    const cudaError_t e = cudaFuncSetAttribute(
        latent_attn_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) attr[dev] = true;
  }
  const long long grid = H.shares ? sms : blocks_of(a, H);
  launch_begin(CSA_K_LATENT_ATTN, s);
  cudaError_t e = launch_kernel(latent_attn_kernel, dim3((unsigned)grid), dim3(LA_THREADS), smem, s,
                                0, false, a, parts, H, qmap, qrmap, cmap, rmap);
  launch_end(CSA_K_LATENT_ATTN, s);
  if (e != cudaSuccess || !H.shares) return e != cudaSuccess ? e : cudaGetLastError();
  launch_begin(CSA_K_LATENT_JOIN, s);
  e = launch_kernel(latent_join_kernel, dim3(H.gt * H.R, (unsigned)sms), dim3(128), 0, s, 0, false,
                    a, parts, H, sms);
  launch_end(CSA_K_LATENT_JOIN, s);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace csa
