// Launchers of the latent cache and eviction calls, for csa_cache_api.cu.
#pragma once

#include "csa_internal.cuh"

namespace csa {

constexpr int kLatent = CSA_LATENT_DIM;
constexpr int kNope = CSA_NOPE_DIM;
constexpr int kValue = CSA_VALUE_DIM;

// SMs of the current device.
inline int sm_count() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms <= 0)
    sms = 152;
  return sms;
}

// Absorbed latent attention (k_latent_attn.cu).
size_t latent_attn_workspace(const csa_latent_attn_args &a);
cudaError_t launch_latent_attn(const csa_latent_attn_args &a, cudaStream_t s);
// Keys and values from latents (k_latent_expand.cu).
cudaError_t launch_latent_expand(const csa_latent_expand_args &a, cudaStream_t s);
// Accumulated attention weights (k_attn_mass.cu).
size_t attn_mass_workspace(const csa_attn_mass_args &a);
cudaError_t launch_attn_mass(const csa_attn_mass_args &a, cudaStream_t s);
// Eviction (k_kv_evict.cu).
size_t kv_evict_workspace(const csa_kv_evict_args &a);
cudaError_t launch_kv_evict(const csa_kv_evict_args &a, cudaStream_t s);

}  // namespace csa
