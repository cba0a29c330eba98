// One head's vector of a row: the RMS norm over its channels and the rotation
// of part of them, held in registers by a group of lanes.  A vector of
// head_dim = 8 n channels is n chunks of 16 bytes; lane l of its group of L
// lanes holds chunks l, l + L, ... (C of them).
//   y = x gamma / sqrt(mean(x^2) + eps), then pairs turned at the position.
// FP32 throughout; the caller rounds once.
#pragma once

#include <type_traits>

#include "csa_internal.cuh"

namespace csa {
namespace headvec {

struct Rope {
  const float *cos, *sin;  // [cap, dim / 2], or null: no rotation
  int start, dim, cap, half_layout;
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

// The normed, rotated vector at `src` (n_chunks chunks) into y.  Every lane of
// the warp calls it with the same `reduce`; `on` is false for lanes without a
// vector, and `norm` (which needs `reduce`) may differ between the warp's
// vectors.  `trow` as table_row gives it.  All loads of the vector happen before it returns and
// before any lane of the warp leaves it, so the caller may overwrite `src`.
template <int L, int C>
__device__ __forceinline__ void load(const uint16_t *src, int n_chunks, bool on, bool reduce,
                                     bool norm, float eps, const uint16_t *gamma, const Rope &R, int trow,
                                     float (&y)[C][8]) {
  const int l = threadIdx.x & (L - 1);
  const int c_lo = R.start >> 3, c_hi = (R.start + R.dim) >> 3, hop = R.dim >> 4;
  uint4 raw[C], mate[C];
#pragma unroll
  for (int j = 0; j < C; ++j) {
    const int c = l + L * j;
    raw[j] = mate[j] = make_uint4(0, 0, 0, 0);
    if (on && c < n_chunks) {
      raw[j] = ld16(src + 8 * c);
      if (R.half_layout && trow >= 0 && c >= c_lo && c < c_hi)
        mate[j] = ld16(src + 8 * (c - c_lo < hop ? c + hop : c - hop));
    }
  }
  float r = 1.f;
  if (reduce) {
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < C; ++j) {
      float x[8];
      unpack8(raw[j], x);
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
    }
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    r = rsqrtf(ss / (float)(8 * n_chunks) + eps);
  }
  __syncwarp();
#pragma unroll
  for (int j = 0; j < C; ++j) {
    const int c = l + L * j;
    unpack8(raw[j], y[j]);
    if (!on || c >= n_chunks) continue;
    if (norm) {
      float g[8];
      if (gamma) unpack8(ld16(gamma + 8 * c), g);
#pragma unroll
      for (int i = 0; i < 8; ++i) y[j][i] *= gamma ? r * g[i] : r;
    }
    if (trow < 0 || c < c_lo || c >= c_hi) continue;
    const long long t = (long long)trow * (R.dim >> 1);
    if (!R.half_layout) {
      float cs[4], sn[4];
      ld4f(R.cos + t + 4 * (c - c_lo), cs);
      ld4f(R.sin + t + 4 * (c - c_lo), sn);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float a = y[j][2 * i], b = y[j][2 * i + 1];
        y[j][2 * i] = a * cs[i] - b * sn[i];
        y[j][2 * i + 1] = a * sn[i] + b * cs[i];
      }
    } else {
      const bool first = c - c_lo < hop;
      const int i0 = 8 * (first ? c - c_lo : c - c_lo - hop);
      float cs[8], sn[8], m[8];
      ld4f(R.cos + t + i0, cs);
      ld4f(R.cos + t + i0 + 4, cs + 4);
      ld4f(R.sin + t + i0, sn);
      ld4f(R.sin + t + i0 + 4, sn + 4);
      unpack8(mate[j], m);
      if (norm) {
        float g[8];
        if (gamma) unpack8(ld16(gamma + 8 * (first ? c + hop : c - hop)), g);
#pragma unroll
        for (int i = 0; i < 8; ++i) m[i] *= gamma ? r * g[i] : r;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i)
        y[j][i] = first ? y[j][i] * cs[i] - m[i] * sn[i] : m[i] * sn[i] + y[j][i] * cs[i];
    }
  }
}

// Lanes and chunks of a head of `dim` channels: f(L, C) as constants.
template <typename F>
auto dispatch(int dim, F &&f) {
  using std::integral_constant;
  const int n = dim / 8;
  if (n <= 1) return f(integral_constant<int, 1>(), integral_constant<int, 1>());
  if (n <= 2) return f(integral_constant<int, 2>(), integral_constant<int, 1>());
  if (n <= 4) return f(integral_constant<int, 4>(), integral_constant<int, 1>());
  if (n <= 8) return f(integral_constant<int, 8>(), integral_constant<int, 1>());
  if (n <= 16) return f(integral_constant<int, 16>(), integral_constant<int, 1>());
  if (n <= 32) return f(integral_constant<int, 32>(), integral_constant<int, 1>());
  return f(integral_constant<int, 32>(), integral_constant<int, 2>());
}

}  // namespace headvec
}  // namespace csa
