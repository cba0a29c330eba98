// csa_qk_norm_rope and csa_kv_append: every head of every row is normed over
// its channels and rotated at the row's position (headvec.cuh), then stored to
// its own tensor or into a paged cache.  Both only move memory: each element
// is read once and written once (8192 rows of 64 heads of 512: 183 us, 6.0 TB/s).
#include <type_traits>

#include "csa_internal.cuh"
#include "headvec.cuh"
#include "lowbit.cuh"
#include "tc.cuh"

namespace csa {
namespace {

using headvec::Rope;

constexpr int NR_THREADS = 256;
// Blocks an SM, for the loads in flight within the registers that are left to a thread:
// above 256 channels three (85 registers; 8192 rows of 64 heads of 512: 183 us, 6.0
// TB/s; two blocks 223 us, and two heads at once instead of four with four blocks 196
// us), up to 256 five (48 registers; 16384 rows of 32 + 8 heads of 128, adjacent pairs:
// 66 us, 5.1 TB/s; three blocks 81, four 70, six 67), four for halves, whose partners'
// angles and gammas come along (85 us; three blocks 91, five 112).  Partners fetched
// beside their chunks (halves above 256 channels) need more registers.
template <int C, bool HALF>
constexpr int kBlocks = C == 1 ? (HALF ? 4 : 5) : (HALF ? 1 : 3);
// The publication kernel, its inputs from memory.  With one head a warp there are many
// short warps, and four blocks help (8192 rows of 512 to MXFP8, with the host's call:
// 10.0 -> 9.3 us; the kernel alone 8.4, to BF16 7.7).  With several heads a warp, of up
// to 256 channels: adjacent pairs four (8192 rows of 8 + 8 heads of 128 18.0 us; without
// the look at a head's scale 17.5, three blocks of that 19.0 and two 23.1), halves two
// (25.6; without 25.1, three 23.1 but 64 rows 3.5 for 2.9, one 42.7); above that two
// (8192 rows of 8 heads of 512, keys alone, 33.1 us; without 31.9, three 39.0, one 46.6).
// At these bounds some instances spill (at most 290 bytes a thread, the halves above
// 256 channels).
template <int C, int U, bool HALF>
constexpr int kAppendBlocks = U == 1 ? (C == 1 || !HALF ? 4 : 1) : (C == 1 && !HALF ? 4 : 2);

__device__ __forceinline__ const uint16_t *at(const void *base, long long bytes) {
  return reinterpret_cast<const uint16_t *>(static_cast<const uint8_t *>(base) + bytes);
}

__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }

// One warp a unit: a row's heads h .. h + PER - 1 of q, or of k.  What bounds
// it is the copying: each channel is read once and written once.
template <int L, int C, int U, bool HALF>
__global__ void __launch_bounds__(NR_THREADS, (kBlocks<C, HALF>)) qk_norm_rope_kernel(csa_qk_norm_rope_args a) {
  tc::griddep_wait();
  tc::griddep_launch_dependents();
  constexpr int PER = 32 / L * U;
  const unsigned uq = (a.n_q_heads + PER - 1) / PER, uk = (a.n_k_heads + PER - 1) / PER;
  const unsigned long long total = (unsigned long long)a.n_rows * (uq + uk);
  const Rope R{a.rope_cos, a.rope_sin, a.rope_start, a.rope_dim, a.rope_cap};
  for (unsigned long long i = (unsigned long long)blockIdx.x * (NR_THREADS / 32) + (threadIdx.x >> 5);
       i < total; i += (unsigned long long)gridDim.x * (NR_THREADS / 32)) {
    const long long t = total >> 32 ? (long long)(i / (uq + uk)) : (unsigned)i / (uq + uk);
    const unsigned unit = (unsigned)(i - t * (uq + uk));
    const bool is_q = unit < uq;
    headvec::Heads<L, C, U, HALF> V;
    V.load(is_q ? at(a.q, t * a.q_row_stride) : at(a.k, t * a.k_row_stride),
           (is_q ? unit : unit - uq) * PER, is_q ? a.n_q_heads : a.n_k_heads, a.head_dim / 8,
           static_cast<const uint16_t *>(!a.norm ? nullptr : (is_q ? a.q_gamma : a.k_gamma)), R);
    if (a.row_req && a.row_req[t] < 0) continue;
    const int trow = headvec::table_row(R, a.row_pos[t], a.status_dev);
    uint8_t *out = is_q ? static_cast<uint8_t *>(a.q_out) + t * a.q_out_row_stride
                        : static_cast<uint8_t *>(a.k_out) + t * a.k_out_row_stride;
    V.finish(a.norm, a.eps, R, trow, [&](int h, int c, bool on, const float(&y)[8]) {
      if (on) reinterpret_cast<uint4 *>(out + (long long)h * a.head_dim * 2)[c] = headvec::pack8(y);
    });
  }
}

// The same over k and v, to the row's slot.
template <int L, int C, int U, bool HALF>
__global__ void __launch_bounds__(NR_THREADS, (kAppendBlocks<C, U, HALF>)) kv_append_kernel(csa_kv_append_args a) {
  tc::griddep_wait();
  tc::griddep_launch_dependents();
  constexpr int PER = 32 / L * U;
  const unsigned uk = (a.n_heads + PER - 1) / PER, units = uk * (a.v ? 2 : 1);
  const unsigned long long total = (unsigned long long)a.n_rows * units;
  const Rope R{a.rope_cos, a.rope_sin, a.rope_start, a.rope_dim, a.rope_cap};
  for (unsigned long long i = (unsigned long long)blockIdx.x * (NR_THREADS / 32) + (threadIdx.x >> 5);
       i < total; i += (unsigned long long)gridDim.x * (NR_THREADS / 32)) {
    const long long t = total >> 32 ? (long long)(i / units) : (unsigned)i / units;
    const unsigned unit = (unsigned)(i - t * units);
    const bool is_k = unit < uk, norm = is_k && a.norm;
    headvec::Heads<L, C, U, HALF> V;
    V.load(is_k ? at(a.k, t * a.k_row_stride) : at(a.v, t * a.v_row_stride),
           (is_k ? unit : unit - uk) * PER, a.n_heads, a.head_dim / 8,
           norm ? static_cast<const uint16_t *>(a.k_gamma) : nullptr, R);
    const int b = a.row_req[t], p = a.row_pos[t];
    if (b >= a.n_req) flag(a.status_dev, CSA_DEV_BAD_POS);
    if (b < 0 || b >= a.n_req || p < 0) continue;
    const long long row = page_row(a.block_table, a.max_blocks, a.n_blocks, b, p, a.status_dev);
    const int trow = is_k ? headvec::table_row(R, p, a.status_dev) : -1;
    if (row < 0) continue;
    if (a.fmt == CSA_FMT_BF16) {
      uint8_t *out = is_k ? static_cast<uint8_t *>(a.k_pool) + (row >> 7) * a.k_page_stride +
                                (row & 127) * a.k_token_stride
                          : static_cast<uint8_t *>(a.v_pool) + (row >> 7) * a.v_page_stride +
                                (row & 127) * a.v_token_stride;
      const long long hs = is_k ? a.k_head_stride : a.v_head_stride;
      V.finish(norm, a.eps, R, trow, [&](int h, int c, bool on, const float(&y)[8]) {
        if (on) reinterpret_cast<uint4 *>(out + h * hs)[c] = headvec::pack8(y);
      });
    } else if constexpr (L >= 4) {
      // groups of 32 channels: four neighbouring lanes share a scale
      uint8_t *codes = static_cast<uint8_t *>(is_k ? a.k_pool : a.v_pool);
      uint8_t *scales = is_k ? a.k_scale_pool : a.v_scale_pool;
      V.finish(norm, a.eps, R, trow, [&](int h, int c, bool on, const float(&y)[8]) {
        float m = 0.f;
#pragma unroll
        for (int u = 0; u < 8; ++u) m = fmaxf(m, fabsf(y[u]));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
        const int e = m <= 3.4028235e38f ? lowbit::e8m0_exponent_448(m) : 127;
        // 2^-e as a factor: exact, in two steps where it leaves FP32's normal range
        const float s1 = pow2(-(e / 2)), s2 = pow2(-(e - e / 2));
        uint32_t w[2] = {0, 0};
#pragma unroll
        for (int u = 0; u < 8; u += 2) {
          const float2 x = make_float2(y[u] * s1 * s2, y[u + 1] * s1 * s2);
          w[u >> 2] |= (uint32_t)__nv_cvt_float2_to_fp8x2(x, __NV_SATFINITE, __NV_E4M3) << (8 * (u & 3));
        }
        if (!on) return;
        const long long vec = row * a.n_heads + h;
        reinterpret_cast<uint2 *>(codes + vec * a.head_dim)[c] = make_uint2(w[0], w[1]);
        if ((c & 3) == 0) scales[vec * (a.head_dim / 32) + (c >> 2)] = (uint8_t)(e + 127);
      });
    }
  }
}

// A warp a unit, and more than one only past 2^20 units.
int grid_for(unsigned long long units) {
  const unsigned long long want = (units + NR_THREADS / 32 - 1) / (NR_THREADS / 32);
  return (int)(want < (1u << 17) ? want : (1u << 17));
}

unsigned long long units_of(int heads, int per) { return (unsigned long long)((heads + per - 1) / per); }

}  // namespace

cudaError_t launch_qk_norm_rope(const csa_qk_norm_rope_args &a, cudaStream_t s) {
  const bool half = a.rope_cos && a.rope_layout == CSA_ROPE_HALF;
  launch_begin(CSA_K_NORM_ROPE, s);
  const cudaError_t e =
      headvec::dispatch(a.head_dim, a.n_q_heads, half, [&](auto L, auto C, auto U, auto HALF) {
        constexpr int per = 32 / L() * U();
        const auto n = a.n_rows * (units_of(a.n_q_heads, per) + units_of(a.n_k_heads, per));
        return launch_kernel(qk_norm_rope_kernel<L(), C(), U(), HALF()>, dim3(grid_for(n)),
                             dim3(NR_THREADS), 0, s, 0, false, a);
      });
  launch_end(CSA_K_NORM_ROPE, s);
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_kv_append(const csa_kv_append_args &a, cudaStream_t s) {
  const bool half = a.rope_cos && a.rope_layout == CSA_ROPE_HALF;
  launch_begin(CSA_K_KV_APPEND, s);
  const cudaError_t e =
      headvec::dispatch(a.head_dim, a.n_heads, half, [&](auto L, auto C, auto U, auto HALF) {
        constexpr int per = 32 / L() * U();
        const auto n = a.n_rows * units_of(a.n_heads, per) * (a.v ? 2 : 1);
        return launch_kernel(kv_append_kernel<L(), C(), U(), HALF()>, dim3(grid_for(n)),
                             dim3(NR_THREADS), 0, s, 0, false, a);
      });
  launch_end(CSA_K_KV_APPEND, s);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace csa
