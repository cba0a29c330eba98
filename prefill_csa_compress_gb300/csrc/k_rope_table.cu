// FP32 half-width RoPE tables (csa_rope_table).
//
// Entry (p, i) is cos and sin of p * f_i.  The host turns each f_i into turns
// per position as a 64-bit binary fraction F_i = f_i / (2 pi) * 2^64, rounded once;
// p * F_i modulo 2^64 is then the angle modulo one turn, in two integer
// multiplications.  At p = 2^31 the rounding of F_i moves it by 3.7e-10 radians (a
// quotient of 53 bits would by 2.4e-7); its top 32 bits are kept (1.5e-9 radians).
#include <math.h>

#include "csa_internal.cuh"
#include "tc.cuh"

namespace csa {
namespace {

constexpr int RT_THREADS = 256;
constexpr int RT_MAX_PAIRS = 256;

struct RopeTurns {
  uint64_t f[RT_MAX_PAIRS];  // turns per position, 64-bit fraction
};

// cos and sin of a signed angle in units of 2^-32 turns: the nearest quarter
// turn taken off leaves |r| <= pi/4, where
//   sin r = r + r z (s0 + s1 z + s2 z^2),  cos r = 1 - z/2 + z^2 (c0 + c1 z + c2 z^2)
// with z = r^2 and the polynomials that interpolate (sin(r)/r - 1)/z and (cos r -
// 1 + z/2)/z^2 at the three Chebyshev nodes of [0, pi^2/16].  In FP32 they are 0.95e-7
// and 1.22e-7 off at most, nearly all of it the arithmetic's rounding (a fourth
// coefficient leaves 0.88e-7 and 1.18e-7); scaled by an FP32 factor 1.82e-7 of it.
// The quarter turns swap and negate.
__device__ __forceinline__ float2 cos_sin(uint32_t phase) {
  const uint32_t quarter = (phase + 0x20000000u) >> 30;
  const float r = (float)(int32_t)(phase - (quarter << 30)) * 1.46291807927e-9f;  // 2 pi / 2^32
  const float z = r * r;
  const float s = fmaf(r * z, fmaf(fmaf(-1.958789e-4f, z, 8.332748e-3f), z, -1.6666664e-1f), r);
  const float c = fmaf(fmaf(fmaf(2.4547942e-5f, z, -1.3888302e-3f), z, 4.1666664e-2f) * z, z,
                       fmaf(-0.5f, z, 1.f));
  const float u = quarter & 1u ? s : c, v = quarter & 1u ? c : s;
  return make_float2(quarter + 1u & 2u ? -u : u, quarter & 2u ? -v : v);
}

// A thread keeps the rotations of V neighbouring pairs and walks down the rows.
// V = 4 stores 16 bytes at a time; V = 1 takes odd widths and any address.
// What bounds it is the writing: the million-position table of 64 channels is
// 268 MB, 39.5 us at the measured copy rate.
template <int V>
__global__ void __launch_bounds__(RT_THREADS)
    rope_table_kernel(const __grid_constant__ RopeTurns turns, int pairs, int n_pos, int pos0,
                      float amp, float *cos_out, float *sin_out) {
  tc::griddep_wait();
  tc::griddep_launch_dependents();
  const int per_row = pairs / V, rows = RT_THREADS / per_row;  // threads a row, rows a step
  const int r = threadIdx.x / per_row, i = (threadIdx.x - r * per_row) * V;
  if (r >= rows) return;
  uint64_t f[V];
#pragma unroll
  for (int v = 0; v < V; ++v) f[v] = turns.f[i + v];
  const long long step = (long long)gridDim.x * rows;
  for (long long j = (long long)blockIdx.x * rows + r; j < n_pos; j += step) {
    float c[V], s[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      // the top half of (pos * f) modulo 2^64
      const uint32_t pos = (uint32_t)(pos0 + j);
      const uint32_t phase = __umulhi(pos, (uint32_t)f[v]) + pos * (uint32_t)(f[v] >> 32);
      const float2 cs = cos_sin(phase);
      c[v] = cs.x * amp;
      s[v] = cs.y * amp;
    }
    const long long e = j * pairs + i;
    if constexpr (V == 4) {
      *reinterpret_cast<float4 *>(cos_out + e) = make_float4(c[0], c[1], c[2], c[3]);
      *reinterpret_cast<float4 *>(sin_out + e) = make_float4(s[0], s[1], s[2], s[3]);
    } else {
      cos_out[e] = c[0];
      sin_out[e] = s[0];
    }
  }
}

// Rotation per position of each pair (csa_rope_scaling_t in include/csa.h).
void frequencies(const csa_rope_table_args &a, double *f) {
  const double d = a.rope_dim, kPi = 3.14159265358979323846;
  double theta = a.theta;
  if (a.scaling == CSA_ROPE_NTK) theta *= pow(a.factor, d / (d - 2.0));
  double lo = 0.0, hi = 0.0;
  if (a.scaling == CSA_ROPE_YARN) {
    lo = floor(d * log(a.orig_len / (2.0 * kPi * a.beta_fast)) / (2.0 * log(theta)));
    hi = ceil(d * log(a.orig_len / (2.0 * kPi * a.beta_slow)) / (2.0 * log(theta)));
    lo = lo > 0.0 ? lo : 0.0;
    hi = hi < d - 1.0 ? hi : d - 1.0;
  }
  const double span = hi - lo > 0.001 ? hi - lo : 0.001;
  for (int i = 0; i < a.rope_dim / 2; ++i) {
    f[i] = pow(theta, -2.0 * i / d);
    if (a.scaling == CSA_ROPE_LINEAR) f[i] /= a.factor;
    if (a.scaling == CSA_ROPE_YARN) {
      double r = (i - lo) / span;
      r = r < 0.0 ? 0.0 : (r > 1.0 ? 1.0 : r);
      f[i] = f[i] * (1.0 - r) + f[i] / a.factor * r;
    }
  }
}

// Turns per position of a rotation of f <= 1 radians, as a 64-bit fraction (below
// 0.16 * 2^64): 1 / (2 pi) as the sum of two doubles, the product's own rounding taken
// along, and one rounding at the end.
uint64_t turn_fraction(double f) {
  constexpr double kInv = 0x1.45f306dc9c883p-3, kInvLow = -0x1.6b01ec5417056p-57;
  const double p = f * kInv, low = fma(f, kInvLow, fma(f, kInv, -p));
  const double s = ldexp(p, 64), whole = floor(s);
  return (uint64_t)whole + (uint64_t)llrint((s - whole) + ldexp(low, 64));
}

}  // namespace

cudaError_t launch_rope_table(const csa_rope_table_args &a, cudaStream_t s) {
  const int pairs = a.rope_dim / 2;
  double f[RT_MAX_PAIRS];
  frequencies(a, f);
  RopeTurns turns;
  for (int i = 0; i < RT_MAX_PAIRS; ++i) turns.f[i] = i < pairs ? turn_fraction(f[i]) : 0;
  const bool wide = pairs % 4 == 0 && ((reinterpret_cast<uintptr_t>(a.cos) |
                                        reinterpret_cast<uintptr_t>(a.sin)) & 15u) == 0;
  const int rows = RT_THREADS / (wide ? pairs / 4 : pairs);
  const long long want = ((long long)a.n_pos + rows - 1) / rows;
  const dim3 grid((unsigned)(want < 152 * 8 ? want : 152 * 8));  // eight blocks an SM
  launch_begin(CSA_K_ROPE_TABLE, s);
  const cudaError_t e = launch_kernel(wide ? rope_table_kernel<4> : rope_table_kernel<1>, grid,
                                      dim3(RT_THREADS), 0, s, 0, false, turns, pairs, a.n_pos,
                                      a.pos0, (float)a.attn_factor, a.cos, a.sin);
  launch_end(CSA_K_ROPE_TABLE, s);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace csa
