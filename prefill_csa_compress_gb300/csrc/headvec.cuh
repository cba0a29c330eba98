// Heads of one row: the RMS norm over each head's channels and the rotation of
// part of them, held in registers by groups of lanes.  A head of 8 n channels
// is n chunks of 16 bytes; lane l of its group of L lanes holds chunks l, l + L,
// ... (C of them).
//   y = x gamma / sqrt(mean(x^2) + eps), then pairs turned at the position.
// FP32 throughout; the caller rounds once.  A warp takes U heads of 32 / L groups
// of one row at a time: the row's rotation and gamma are loaded once for all of
// them, and all heads' loads are in flight together.
#pragma once

#include <type_traits>

#include "csa_internal.cuh"

namespace csa {
namespace headvec {

struct Rope {
  const float *cos, *sin;  // [cap, dim / 2], or null: no rotation
  int start, dim, cap;
};

__device__ __forceinline__ void unpack8(const uint4 &u, float (&x)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t *>(&v);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ uint4 ld16(const void *p) { return *static_cast<const uint4 *>(p); }

__device__ __forceinline__ void ld4f(const float *p, float *v) {
  const float4 f = *reinterpret_cast<const float4 *>(p);
  v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w;
}

__device__ __forceinline__ void times(uint4 &x, __nv_bfloat162 s) {
  uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 y = __hmul2(*reinterpret_cast<const __nv_bfloat162 *>(&w[i]), s);
    w[i] = *reinterpret_cast<const uint32_t *>(&y);
  }
  x = make_uint4(w[0], w[1], w[2], w[3]);
}

// The row's position as the tables take it: -1 for none (and the flag when it
// lies past the tables).
__device__ __forceinline__ int table_row(const Rope &R, int pos, uint32_t *status) {
  if (!R.cos || pos < 0) return -1;
  if (pos >= R.cap) {
    flag(status, CSA_DEV_POS_GE_CAP);
    return -1;
  }
  return pos;
}

// Heads first + u (32 / L) + lane / L, u < U, of a row of `n` heads of 8 n_chunks
// channels, one after the other.  Every lane of the warp takes part in both
// steps: load() asks for the row's channels, which needs no position, so that the
// position, its table row and its page are on their way at the same time; finish()
// norms and rotates head after head and hands each chunk to store(head, chunk,
// on, y).  Everything is read before store() runs, so that it may overwrite its
// own head.
template <int L, int C, int U, bool HALF>
struct Heads {
  static constexpr int PAIRS = HALF ? 8 : 4;  // angles of a chunk
  // A half-layout chunk's partner: with one chunk a lane, the partner's lane has
  // it; above 256 channels it comes along.
  static constexpr bool FETCH = HALF && C > 1;
  uint4 raw[U][C], mate[FETCH ? U : 1][C];
  uint4 g[C], gm[HALF ? C : 1];               // gamma of both
  int h0, n, n_chunks, c_lo, c_hi, hop;

  // Heads whose mean square leaves FP32, or whose smaller squares may have vanished in
  // it: their channels (and their partners') times a power of two, exactly but for
  // channels 2^115 times smaller than the head's largest, and the mean square and eps
  // in that measure.  The result does not see the factor.  Out of line, so that the
  // usual path is as short as without it (2 rows of 64 heads of 512: 3.36 us in line,
  // 3.20 like this, 3.17 without); the vote costs 16384 rows of 40 heads of 128 2 us of 66.
  struct Head {
    uint4 raw[C], mate[FETCH ? C : 1];
    float mean;
  };
  static constexpr float kSmall = 0x1p-80f, kLarge = 3.4028235e38f;
  static __device__ __noinline__ Head rescaled(Head H, float inv_n, float eps) {
    const float s = H.mean < kSmall ? 0x1p80f : (H.mean > kLarge ? 0x1p-70f : 1.f);
    const __nv_bfloat162 s2 = __float2bfloat162_rn(s);
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < C; ++j) {
      times(H.raw[j], s2);
      if constexpr (FETCH) times(H.mate[j], s2);
      float x[8];
      unpack8(H.raw[j], x);
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
    }
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    H.mean = fmaf(ss, inv_n, eps * s * s);
    return H;
  }
  __device__ __forceinline__ float rescale(int u, float mean, float inv_n, float eps) {
    Head H;
#pragma unroll
    for (int j = 0; j < C; ++j) {
      H.raw[j] = raw[u][j];
      if constexpr (FETCH) H.mate[j] = mate[u][j];
    }
    H.mean = mean;
    H = rescaled(H, inv_n, eps);
#pragma unroll
    for (int j = 0; j < C; ++j) {
      raw[u][j] = H.raw[j];
      if constexpr (FETCH) mate[u][j] = H.mate[j];
    }
    return H.mean;
  }

  __device__ __forceinline__ bool turned(int c) const { return c >= c_lo && c < c_hi; }
  __device__ __forceinline__ int partner(int c) const { return c - c_lo < hop ? c + hop : c - hop; }

  __device__ __forceinline__ void load(const uint16_t *src, int first, int n_heads, int chunks,
                                       const uint16_t *gamma, const Rope &R) {
    const int lane = threadIdx.x & 31, l = lane & (L - 1);
    h0 = first + lane / L;
    n = n_heads;
    n_chunks = chunks;
    c_lo = R.cos ? R.start >> 3 : 0;
    c_hi = R.cos ? (R.start + R.dim) >> 3 : 0;
    hop = R.dim >> 4;
    const uint4 ones = make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u);
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int j = 0; j < C; ++j) {
        const int c = l + L * j, h = h0 + u * (32 / L);
        const uint16_t *head = src + (long long)h * 8 * n_chunks;
        raw[u][j] = make_uint4(0, 0, 0, 0);
        if (h < n && c < n_chunks) raw[u][j] = ld16(head + 8 * c);
        if constexpr (FETCH) {
          mate[u][j] = make_uint4(0, 0, 0, 0);
          if (h < n && c < n_chunks && turned(c)) mate[u][j] = ld16(head + 8 * partner(c));
        }
      }
#pragma unroll
    for (int j = 0; j < C; ++j) {
      const int c = l + L * j;
      g[j] = gamma && c < n_chunks ? ld16(gamma + 8 * c) : ones;
      if constexpr (HALF)
        gm[j] = gamma && c < n_chunks && turned(c) ? ld16(gamma + 8 * partner(c)) : ones;
    }
  }

  // `trow` as table_row gives it; `norm` alike in all lanes.
  template <typename Store>
  __device__ __forceinline__ void finish(bool norm, float eps, const Rope &R, int trow,
                                         Store &&store) {
    const int l = threadIdx.x & (L - 1);
    float cs[C][PAIRS], sn[C][PAIRS], sign[C];
    bool rot[C];
#pragma unroll
    for (int j = 0; j < C; ++j) {
      const int c = l + L * j;
      rot[j] = trow >= 0 && c < n_chunks && turned(c);
      sign[j] = HALF && c - c_lo < hop ? -1.f : 1.f;
      if (rot[j]) {
        const long long t = (long long)trow * (R.dim >> 1) +
                            PAIRS * ((HALF ? min(c, partner(c)) : c) - c_lo);
#pragma unroll
        for (int i = 0; i < PAIRS; i += 4) {
          ld4f(R.cos + t + i, cs[j] + i);
          ld4f(R.sin + t + i, sn[j] + i);
        }
      }
    }
    __syncwarp();
    const float inv_n = 1.f / (float)(8 * n_chunks);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = h0 + u * (32 / L);
      float r = 1.f;
      if (norm) {
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < C; ++j) {
          float x[8];
          unpack8(raw[u][j], x);
#pragma unroll
          for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
        }
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        float mean = fmaf(ss, inv_n, eps);
        if (__builtin_expect(__any_sync(0xffffffffu, !(mean >= kSmall && mean <= kLarge)), 0))
          mean = rescale(u, mean, inv_n, eps);
        r = rsqrtf(mean);
      }
#pragma unroll
      for (int j = 0; j < C; ++j) {
        uint4 other = make_uint4(0, 0, 0, 0);
        if constexpr (HALF && !FETCH) {
          const int from = ((threadIdx.x & 31) & ~(L - 1)) + (turned(l) ? partner(l) : l);
          other.x = __shfl_sync(0xffffffffu, raw[u][j].x, from);
          other.y = __shfl_sync(0xffffffffu, raw[u][j].y, from);
          other.z = __shfl_sync(0xffffffffu, raw[u][j].z, from);
          other.w = __shfl_sync(0xffffffffu, raw[u][j].w, from);
        }
        float y[8], w[8];
        unpack8(raw[u][j], y);
        unpack8(g[j], w);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] *= r * w[i];
        if (rot[j]) {
          if constexpr (!HALF) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float a = y[2 * i], b = y[2 * i + 1];
              y[2 * i] = a * cs[j][i] - b * sn[j][i];
              y[2 * i + 1] = a * sn[j][i] + b * cs[j][i];
            }
          } else {
            float m[8];
            unpack8(FETCH ? mate[FETCH ? u : 0][j] : other, m);
            unpack8(gm[j], w);
#pragma unroll
            for (int i = 0; i < 8; ++i)
              y[i] = y[i] * cs[j][i] + sign[j] * (m[i] * (r * w[i])) * sn[j][i];
          }
        }
        // every lane calls it (it may exchange values with its neighbours)
        store(h, l + L * j, h < n && l + L * j < n_chunks, y);
      }
    }
  }
};

// Groups' lanes, chunks a lane and heads at once for n_heads heads of `dim`
// channels, and the layout: f(L, C, U, HALF) as constants.  Four heads at once
// where a row has them (two of the half layout above 256 channels, for the
// registers), else one.
template <int L, int C, typename F>
auto dispatch_heads(int n_heads, bool half, F &&f) {
  using std::integral_constant;
  constexpr integral_constant<int, L> l{};
  constexpr integral_constant<int, C> c{};
  constexpr integral_constant<int, 1> one{};
  if (half) {
    constexpr integral_constant<int, (C == 1 ? 4 : 2)> many{};
    return n_heads > 32 / L ? f(l, c, many, std::true_type()) : f(l, c, one, std::true_type());
  }
  constexpr integral_constant<int, 4> many{};
  return n_heads > 32 / L ? f(l, c, many, std::false_type()) : f(l, c, one, std::false_type());
}
template <typename F>
auto dispatch(int dim, int n_heads, bool half, F &&f) {
  const int n = dim / 8;
  if (n <= 1) return dispatch_heads<1, 1>(n_heads, half, f);
  if (n <= 2) return dispatch_heads<2, 1>(n_heads, half, f);
  if (n <= 4) return dispatch_heads<4, 1>(n_heads, half, f);
  if (n <= 8) return dispatch_heads<8, 1>(n_heads, half, f);
  if (n <= 16) return dispatch_heads<16, 1>(n_heads, half, f);
  if (n <= 32) return dispatch_heads<32, 1>(n_heads, half, f);
  return dispatch_heads<32, 2>(n_heads, half, f);
}

}  // namespace headvec
}  // namespace csa
