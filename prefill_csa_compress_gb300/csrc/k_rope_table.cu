// FP32 half-width RoPE tables (csa_rope_table).
//
// Entry (p, i) is cos and sin of p * f_i.  The host turns each f_i into turns
// per position as a 64-bit binary fraction F_i = f_i / (2 pi) * 2^64; p * F_i
// modulo 2^64 is then the angle modulo one turn, exactly, in one integer
// multiplication.  F_i is off by at most half a unit (2^-65 turns) and by the
// 53 bits of f_i, so the angle at p < 2^31 is off by less than 2^-22 * f_i
// turns of p's relative 2^-53, that is below 1e-6 of FP32's half step for p up
// to 2^20.
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

__global__ void __launch_bounds__(RT_THREADS)
    rope_table_kernel(const __grid_constant__ RopeTurns turns, int pairs, int n_pos, int pos0,
                      float amp, float *cos_out, float *sin_out) {
  tc::griddep_wait();
  tc::griddep_launch_dependents();
  const long long n = (long long)n_pos * pairs;
  for (long long e = (long long)blockIdx.x * RT_THREADS + threadIdx.x; e < n;
       e += (long long)gridDim.x * RT_THREADS) {
    const long long j = e / pairs;
    const int i = (int)(e - j * pairs);
    const uint64_t phase = (uint64_t)(pos0 + j) * turns.f[i];
    float s, c;
    sincospif((float)(int64_t)phase * 0x1p-63f, &s, &c);
    cos_out[e] = c * amp;
    sin_out[e] = s * amp;
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

}  // namespace

cudaError_t launch_rope_table(const csa_rope_table_args &a, cudaStream_t s) {
  const int pairs = a.rope_dim / 2;
  double f[RT_MAX_PAIRS];
  frequencies(a, f);
  RopeTurns turns;
  for (int i = 0; i < RT_MAX_PAIRS; ++i) {
    // f <= 1, so the fraction is below 0.16 * 2^64
    turns.f[i] = i < pairs ? (uint64_t)llrint(ldexp(f[i] / 6.283185307179586476925, 62)) << 2 : 0;
  }
  const long long n = (long long)a.n_pos * pairs;
  const long long want = (n + RT_THREADS - 1) / RT_THREADS;
  const int grid = (int)(want < 152 * 64 ? want : 152 * 64);
  launch_begin(CSA_K_ROPE_TABLE, s);
  const cudaError_t e = launch_kernel(rope_table_kernel, dim3(grid), dim3(RT_THREADS), 0, s, 0,
                                      false, turns, pairs, a.n_pos, a.pos0, (float)a.attn_factor,
                                      a.cos, a.sin);
  launch_end(CSA_K_ROPE_TABLE, s);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace csa
