// Keys and values of every head from a paged latent cache (csa_latent_expand): a
// tcgen05 product of two pages of latents with the heads' up-projections, by pairs of
// CTAs.
//
//   D[j, n] = c_j . w_n    (256 positions x 256 channels of a head x 512, K-major both)
// Each CTA of a pair (cta_group::2) keeps its page of latents (128 KB) in shared memory
// and the pair goes through some of the heads: of a head's 256 rows of 512 the first CTA
// loads the keys' half and the second the values', in eight pieces of 64 columns (16 KB),
// four in flight, and the tensor cores of both read both.  So every SM fetches 32 bytes
// a cycle, where a CTA by itself needs 64 for the same rate, more than it can keep in
// flight beside the latents (355 us for a prompt of 8192 and 128 heads).  A head's 256
// columns of sums take half of tensor memory: one head is written while the next one is
// computed.  Roles, in each CTA:
//   warp 0       loads (TMA): the page's latents, its half of the weights' pieces;
//   warp 1       of the first CTA: issues the MMAs of the pair (256 x 256 x 16);
//   warps 4..11  round the sums to BF16 and store them, two warps 32 positions: key
//                channels, or value channels.  The rotated key, which all heads share,
//                is loaded once and stored from shared memory for every head.
// A prompt of 8192 and 128 heads: 246 us (1.12 PFLOP/s), 159 without its stores; filling
// the 671 MB that it writes takes 168, so what is left is how far the two overlap.  2 x 1500
// positions, 32 heads: 29 us.
#include "attn_common.cuh"
#include "cache_tiles.cuh"

namespace csa {
namespace {

constexpr int LE_THREADS = 384;
constexpr int LE_LOAD = 0, LE_MMA = 1, LE_OUT0 = 4;  // first warps
constexpr int LE_BOX = 16384;                        // 64 columns of 128 rows
constexpr int LE_STAGES = 4;                         // pieces of the weights in flight
constexpr int LE_OUT = 2048;  // 32 channels of 32 positions, a warp's way to memory
constexpr int LE_OFF_W = 8 * LE_BOX, LE_OFF_R = LE_OFF_W + LE_STAGES * LE_BOX,
              LE_OFF_OUT = LE_OFF_R + LE_BOX, LE_OFF_MISC = LE_OFF_OUT + 8 * LE_OUT;

struct Misc {
  uint64_t r_full, c_full[8], w_full[LE_STAGES], w_empty[LE_STAGES], d_full[2], d_empty[2], drained;
  uint32_t tmem;
  int abort;
};
static_assert(LE_OFF_MISC + sizeof(Misc) <= 227 * 1024, "shared memory");

// ---- the pair: addresses of the first CTA's barriers, arrivals there, loads that
// complete there, commits that arrive at both

__device__ __forceinline__ uint32_t first_cta(const uint64_t *bar) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(tc::smem_u32(bar)));
  return r;
}
__device__ __forceinline__ void arrive_first(const uint64_t *bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(first_cta(bar))
               : "memory");
}
__device__ __forceinline__ void load_pair_3d(void *dst, const void *tmap, int x, int y, int z,
                                             const uint64_t *bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(tc::smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(first_cta(bar)), "l"(policy)
      : "memory");
}
__device__ __forceinline__ void commit_pair(uint64_t *bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
      "[%0], %1;" ::"r"(tc::smem_u32(bar)),
      "h"((uint16_t)3)
      : "memory");
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}

// A box of shared memory into a pool [channels, heads, 128, pages], as a bulk group; until
// the groups of this thread are complete.
__device__ __forceinline__ void store_4d(const void *tmap, int x, int y, int z, int w, const void *src) {
  asm volatile(
      "cp.async.bulk.tensor.4d.global.shared::cta.bulk_group [%0, {%1, %2, %3, %4}], [%5];\n\t"
      "cp.async.bulk.commit_group;" ::"l"(reinterpret_cast<uint64_t>(tmap)),
      "r"(x), "r"(y), "r"(z), "r"(w), "r"(tc::smem_u32(src))
      : "memory");
}
__device__ __forceinline__ void stores_done() {
  asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

__global__ void __launch_bounds__(LE_THREADS, 1)
    latent_expand_kernel(csa_latent_expand_args a, int heads_per,
                         const __grid_constant__ CUtensorMap cmap,
                         const __grid_constant__ CUtensorMap kmap,
                         const __grid_constant__ CUtensorMap vmap,
                         const __grid_constant__ CUtensorMap rmap,
                         const __grid_constant__ CUtensorMap kr_out) {
  extern __shared__ __align__(1024) uint8_t sm[];
  Misc *M = reinterpret_cast<Misc *>(sm + LE_OFF_MISC);
  tc::griddep_wait();
  tc::griddep_launch_dependents();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tc::smem_u32(sm) & 1023u) {
    if (tid == 0) flag(a.status_dev, CSA_DEV_TIMEOUT);
    return;
  }
  // pages fastest: CTAs that run together read the same weights
  const int rank = blockIdx.x & 1, pairs_req = (a.max_blocks + 1) / 2;
  const long long pairs = (long long)a.n_req * pairs_req;
  const int part = (int)((blockIdx.x >> 1) / pairs);
  const long long u = (blockIdx.x >> 1) - part * pairs;
  const int b = (int)(u / pairs_req), page0 = 2 * (int)(u - (long long)b * pairs_req);
  const int h0 = part * heads_per, h1 = min(a.n_heads, h0 + heads_per);
  // positions [lo, hi) of either page, and where they are and go; both CTAs know both
  int lo[2], hi[2], src[2], dst[2];
  bool on[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int page = page0 + e;
    lo[e] = hi[e] = src[e] = dst[e] = 0;
    on[e] = false;
    if (page >= a.max_blocks) continue;
    const int base = page * kBlock;
    lo[e] = max((a.first ? max(a.first[b], 0) : 0) - base, 0);
    hi[e] = min(max(a.kv_len[b], 0) - base, kBlock);
    if (lo[e] >= hi[e]) continue;
    src[e] = a.block_table[(long long)b * a.max_blocks + page];
    dst[e] = page < a.out_max_blocks ? a.out_table[(long long)b * a.out_max_blocks + page] : -1;
    on[e] = src[e] >= 0 && src[e] < a.n_blocks && dst[e] >= 0 && dst[e] < a.n_out_blocks;
    if (!on[e] && tid == 0) flag(a.status_dev, CSA_DEV_BAD_BLOCK);
  }
  if (!on[0] && !on[1]) return;
  const bool mine_on = on[rank];
  const int my_lo = lo[rank], my_hi = mine_on ? hi[rank] : my_lo, my_src = src[rank], my_dst = dst[rank];
  const bool full = mine_on && my_lo == 0 && my_hi == kBlock;
  if (tid == 0) {
    tc::mbar_init(&M->r_full, 1);
    for (int i = 0; i < 8; ++i) tc::mbar_init(&M->c_full[i], 1);
    for (int i = 0; i < LE_STAGES; ++i) {
      tc::mbar_init(&M->w_full[i], 1);
      tc::mbar_init(&M->w_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&M->d_full[i], 1);
      tc::mbar_init(&M->d_empty[i], 16);  // eight warps of either CTA
    }
    tc::mbar_init(&M->drained, 1);
    M->abort = 0;
    tc::mbar_fence_init();
  }
  __syncthreads();
  if (warp == LE_MMA) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     tc::smem_u32(&M->tmem)),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc::tc_fence_before();
  __syncthreads();
  cluster_sync();  // the other CTA's barriers are there
  tc::tc_fence_after();
  const uint32_t tmem = __reduce_or_sync(0xffffffffu, M->tmem);
  volatile int *abort = &M->abort;

  if (warp == LE_LOAD) {
    // ================================================================ loads
    if (lane == 0) {
      // (weights and latents are read again, what is written is not)
      const uint64_t keep = tc::l2_evict_last();
      uint32_t it = 0;
      bool ok = true;
      if (full) {
        tc::mbar_arrive_expect_tx(&M->r_full, LE_BOX);
        tc::tma_load_3d(sm + LE_OFF_R, &rmap, 0, 0, my_src, &M->r_full);
      }
      for (int h = h0; h < h1 && ok; ++h)
        for (int c = 0; c < 8; ++c, ++it) {
          const int st = it % LE_STAGES;
          ok = cache::wait(&M->w_empty[st], ((it / LE_STAGES) & 1) ^ 1, abort, a.status_dev);
          if (!ok) break;
          if (h == h0) {
            if (rank == 0) tc::mbar_arrive_expect_tx(&M->c_full[c], LE_BOX * (on[0] + on[1]));
            if (mine_on) load_pair_3d(sm + c * LE_BOX, &cmap, c * 64, 0, my_src, &M->c_full[c], keep);
          }
          if (rank == 0) tc::mbar_arrive_expect_tx(&M->w_full[st], 2 * LE_BOX);
          load_pair_3d(sm + LE_OFF_W + st * LE_BOX, rank ? &vmap : &kmap, c * 64, 0, h, &M->w_full[st],
                       keep);
        }
      // Whatever was asked for has landed before the CTA retires, and the last stages have
      // been handed back: the first CTA's commits arrive at the second's barriers too.
      if (full) tc::mbar_wait(&M->r_full, 0, 50000000ull);
      for (uint32_t k = it > LE_STAGES ? it - LE_STAGES : 0; k < it && ok; ++k)
        ok = cache::wait(&M->w_empty[k % LE_STAGES], (k / LE_STAGES) & 1, abort, a.status_dev);
    }
    __syncwarp();
  } else if (warp == LE_MMA) {
    // ================================================================ MMA
    if (rank == 0 && tc::elect_one()) {
      constexpr uint32_t idesc = tc::idesc_bf16_f32(256, 256);
      const uint64_t dc = tc::desc_sw128(tc::smem_u32(sm));
      const uint64_t dw = tc::desc_sw128(tc::smem_u32(sm) + LE_OFF_W);
      uint32_t it = 0;
      bool ok = true;
      for (int h = h0; h < h1 && ok; ++h) {
        const int n = h - h0, buf = n & 1;
        ok = cache::wait(&M->d_empty[buf], ((n >> 1) & 1) ^ 1, abort, a.status_dev);
        for (int c = 0; c < 8 && ok; ++c, ++it) {
          const int st = it % LE_STAGES;
          ok = (n > 0 || cache::wait(&M->c_full[c], 0, abort, a.status_dev)) &&
               cache::wait(&M->w_full[st], (it / LE_STAGES) & 1, abort, a.status_dev);
          if (!ok) break;
          tc::tc_fence_after();
          cache::mma4_pair<2, 2>(tmem + buf * 256, dc + ((c * LE_BOX) >> 4), dw + ((st * LE_BOX) >> 4), idesc, c > 0);
          commit_pair(&M->w_empty[st]);
        }
        if (ok) commit_pair(&M->d_full[buf]);
      }
      // What was asked for has landed, and every issued MMA has completed, before the
      // pair retires.  (Where a wait gave up, loads of the stages may be under way still.)
      if (!ok)
        for (int k = 0; k < 2 * LE_STAGES; ++k)
          tc::mbar_wait(&M->w_full[k % LE_STAGES], (it / LE_STAGES + k / LE_STAGES) & 1, 5000000ull);
      asm volatile(
          "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
              tc::smem_u32(&M->drained))
          : "memory");
      tc::mbar_wait(&M->drained, 0, 100000000ull);
    }
    __syncwarp();
  } else if (warp >= LE_OUT0) {
    // ================================================================ outputs
    // (a value's half: columns 128 and on of a head's sums)
    const int qd = warp & 3, value = (warp - LE_OUT0) >> 2, j = qd * 32 + lane;
    const bool mine = j >= my_lo && j < my_hi;
    const uint32_t from = tmem + ((uint32_t)(qd * 32) << 16) + value * 128;
    const long long ts = value ? a.v_token_stride : a.k_token_stride;
    uint8_t *to = value ? static_cast<uint8_t *>(a.v_pool) + my_dst * a.v_page_stride
                        : static_cast<uint8_t *>(a.k_pool) + my_dst * a.k_page_stride;
    const long long hs = value ? a.v_head_stride : a.k_head_stride;
    // 32 channels at a time a warp turns its 32 positions through shared memory (16-byte
    // chunk c of row j at c ^ (j / 2) % 4), so that four lanes store 64 bytes of a row
    // (by TMA instead, a store's buffer was free again after 1,500 cycles, behind the
    // loads: 7,000 a head).  The rotated key of a page that is written whole goes by TMA,
    // straight from where it was loaded, else from registers.
    uint4 *box = reinterpret_cast<uint4 *>(sm + LE_OFF_OUT + (warp - LE_OUT0) * LE_OUT);
    const bool rotated = full && warp == LE_OUT0;
    uint4 r[8];
    if (!full && !value && mine)
#pragma unroll
      for (int i = 0; i < 8; ++i)
        r[i] = reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(a.r_pool) +
                                               my_src * a.r_page_stride + j * a.r_token_stride)[i];
    bool ok = !rotated || __all_sync(0xffffffffu, cache::wait(&M->r_full, 0, abort, a.status_dev));
    for (int h = h0; h < h1 && ok; ++h) {
      const int n = h - h0, buf = n & 1;
      ok = __all_sync(0xffffffffu, cache::wait(&M->d_full[buf], (n >> 1) & 1, abort, a.status_dev));
      if (!ok) break;
      tc::tc_fence_after();
      uint8_t *out = to + h * hs;
      if (rotated && lane == 0) store_4d(&kr_out, kNope, h, 0, my_dst, sm + LE_OFF_R);
#pragma unroll 1
      for (int c = 0; c < 128; c += 32) {
        float x[32];
        tc::tmem_ld32(from + buf * 256 + c, x);
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i)
          box[lane * 4 + (i ^ ((lane >> 1) & 3))] =
              make_uint4(attn::pack2(x[8 * i], x[8 * i + 1]), attn::pack2(x[8 * i + 2], x[8 * i + 3]),
                         attn::pack2(x[8 * i + 4], x[8 * i + 5]),
                         attn::pack2(x[8 * i + 6], x[8 * i + 7]));
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int row = i * 8 + (lane >> 2), q = lane & 3, at = qd * 32 + row;
          const uint4 y = box[row * 4 + (q ^ ((row >> 1) & 3))];
          if (at >= my_lo && at < my_hi)
            reinterpret_cast<uint4 *>(out + at * ts)[c / 8 + q] = y;
        }
      }
      if (!full && !value && mine)
#pragma unroll
        for (int i = 0; i < 8; ++i) reinterpret_cast<uint4 *>(out + j * ts)[kNope / 8 + i] = r[i];
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_first(&M->d_empty[buf]);
    }
    if (rotated && lane == 0) stores_done();
  }

  tc::tc_fence_before();
  __syncthreads();
  cluster_sync();  // neither CTA goes while the other's products or arrivals need it
  tc::tc_fence_after();
  if (warp == LE_MMA)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512)
                 : "memory");
}

// [x, y, z], boxes of 64 x 128.
bool encode_in(CUtensorMap *map, const void *base, cuuint64_t x, cuuint64_t y, cuuint64_t z,
               int64_t s1, int64_t s2) {
  const cuuint64_t dims[3] = {x, y, z}, strides[2] = {(cuuint64_t)s1, (cuuint64_t)s2};
  const cuuint32_t box[3] = {64, 128, 1};
  return cache::encode(map, base, 3, dims, strides, box, CU_TENSOR_MAP_L2_PROMOTION_L2_128B);
}

}  // namespace

cudaError_t launch_latent_expand(const csa_latent_expand_args &a, cudaStream_t s) {
  CUtensorMap cmap, kmap, vmap, rmap, kr_out;
  const cuuint64_t pages = a.n_blocks, heads = a.n_heads;
  // the rotated keys' place in a page of one head of k_pool
  const cuuint64_t out_dims[4] = {kNope + kRopeDim, heads, kBlock, (cuuint64_t)a.n_out_blocks};
  const cuuint64_t out_strides[3] = {(cuuint64_t)a.k_head_stride, (cuuint64_t)a.k_token_stride,
                                     (cuuint64_t)a.k_page_stride};
  const cuuint32_t out_box[4] = {kRopeDim, 1, kBlock, 1};
  if (!encode_in(&cmap, a.c_pool, kLatent, kBlock, pages, a.c_token_stride, a.c_page_stride) ||
      !encode_in(&kmap, a.w_uk, kLatent, kNope, heads, kLatent * 2, a.w_uk_head_stride) ||
      !encode_in(&vmap, a.w_uv, kLatent, kValue, heads, kLatent * 2, a.w_uv_head_stride) ||
      !encode_in(&rmap, a.r_pool, kRopeDim, kBlock, pages, a.r_token_stride, a.r_page_stride) ||
      !cache::encode(&kr_out, a.k_pool, 4, out_dims, out_strides, out_box,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_128B))
    return cudaErrorInvalidValue;
  const size_t smem = LE_OFF_MISC + sizeof(Misc);
  int dev = 0;
  cudaGetDevice(&dev);
  static bool attr[64] = {};
  if (dev < 0 || dev >= 64 || !attr[dev]) {
    const cudaError_t e = cudaFuncSetAttribute(
        latent_expand_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) attr[dev] = true;
  }
  // Parts of the heads: as many as make waves x (heads of a part + 1) smallest, a CTA's
  // start and end being worth about one head.  (Every column of the tables counts as a page:
  // the host does not know the lengths.)
  const int places = sm_count() / 2;
  const long long n_pairs = (long long)a.n_req * ((a.max_blocks + 1) / 2);
  int per = a.n_heads, parts = 1;
  long long best = 0;
  for (int p = 1; p <= a.n_heads && p <= 128; ++p) {
    const long long k = (a.n_heads + p - 1) / p, n = (a.n_heads + k - 1) / k;
    const long long cost = (n_pairs * n + places - 1) / places * (k + 1);
    if (p == 1 || cost < best) best = cost, per = (int)k, parts = (int)n;
  }
  if (2 * n_pairs * parts > 0x7FFFFFFF) return cudaErrorInvalidValue;
  launch_begin(CSA_K_LATENT_EXPAND, s);
  const cudaError_t e =
      launch_kernel(latent_expand_kernel, dim3((unsigned)(2 * n_pairs * parts)), dim3(LE_THREADS), smem,
                    s, 2, false, a, per, cmap, kmap, vmap, rmap, kr_out);
  launch_end(CSA_K_LATENT_EXPAND, s);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace csa
