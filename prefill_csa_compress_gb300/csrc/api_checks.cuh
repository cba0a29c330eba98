// Argument checks that the C entry points of the paged caches share.
#pragma once

#include <cstring>
#include <utility>

#include "csa_internal.cuh"

namespace csa {
namespace {

inline bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

inline csa_status_t from_cuda(cudaError_t e) { return e == cudaSuccess ? CSA_OK : CSA_ERR_CUDA; }

inline bool has_size(const void *args, size_t size) {
  uint32_t got = 0;
  if (args) memcpy(&got, args, sizeof(got));
  return args && got >= size;
}

// What a size query answers: never 0, since a call without a workspace is taken for a
// query, and a caller who allocates what it is told holds a pointer then.
inline size_t query_bytes(size_t need) { return need < 256 ? 256 : need; }

// A row stride in bytes, 0 meaning dense.
inline bool row_stride(int64_t *s, int64_t row_bytes) {
  if (*s == 0) *s = row_bytes;
  return *s % 16 == 0 && *s >= row_bytes && *s <= (int64_t(1) << 40);
}

// A pool's strides in bytes made explicit (0: dense); false unless they are
// multiples of 16 that keep every (page, token, head) slot apart: sorted, each
// spans at least what the smaller ones reach over.
inline bool pool_strides(int64_t *page, int64_t *token, int64_t *head, int64_t n_pages, int64_t n_heads,
                  int64_t bytes) {
  if (*head == 0) *head = bytes;
  if (*token == 0) *token = n_heads * bytes;
  if (*page == 0) *page = kBlock * *token;
  int64_t st[3] = {*page, *token, *head}, n[3] = {n_pages, kBlock, n_heads};
  for (int i = 0; i < 3; ++i)
    if (st[i] % 16 != 0 || st[i] < bytes || st[i] >= (int64_t(1) << 40)) return false;
  for (int i = 0; i < 3; ++i)
    for (int j = i + 1; j < 3; ++j)
      if (st[j] < st[i]) {
        std::swap(st[i], st[j]);
        std::swap(n[i], n[j]);
      }
  __int128 reach = bytes;  // (to 2^71: 2^31 pages, 2^40 bytes apart)
  for (int i = 0; i < 3; ++i) {
    if (n[i] == 1) continue;
    if (st[i] < reach) return false;
    reach += (__int128)st[i] * (n[i] - 1);
  }
  return true;
}

}  // namespace
}  // namespace csa
