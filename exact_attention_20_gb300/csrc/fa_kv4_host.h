// Host-side checks that the entry points of the paged 4-bit cache share.
#pragma once

#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "fa_gb300_serve.h"
#include "fa_internal.h"
#include "fa_kv4.cuh"

namespace fa_internal {

namespace kv = fa::kv4;

constexpr int kMaxDevices = 64;

inline bool overlaps(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
  return a0 < b0 + nb && b0 < a0 + na;
}

inline bool misaligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

// log2 of a page size the cache takes, or -1.
inline int page_shift(int page_size) {
  for (int s = 4; s <= 10; ++s)
    if (page_size == 1 << s) return s;
  return -1;
}

// A tensor's scale: a power of two from 2^-40 to 2^40.
inline bool power_of_two(float g) {
  int e = 0;
  return std::isfinite(g) && g > 0.f && std::frexp(g, &e) == 0.5f && e >= -39 && e <= 41;
}

// The cache's own sizes and the tables'; shared by every entry point.
inline int check_cache(const void* cache, const int* page_table, const int* seq_lens, int n_seqs, int max_pages,
                int num_pages, int page_size, int Hkv, int d, float k_scale, float v_scale, size_t* cache_bytes) {
  if (n_seqs < 0 || max_pages < 1 || num_pages < 1 || page_shift(page_size) < 0 || Hkv < 1 || Hkv > (1 << 16) ||
      (d != 64 && d != 128) || !power_of_two(k_scale) || !power_of_two(v_scale))
    return FA_ERR_INVALID_ARG;
  *cache_bytes = static_cast<size_t>(num_pages) * Hkv * page_size * kv::row_bytes(d);
  if (n_seqs == 0) return FA_OK;
  if (!cache || !page_table || !seq_lens) return FA_ERR_NULL;
  if (misaligned(cache, 16) || misaligned(page_table, 4) || misaligned(seq_lens, 4)) return FA_ERR_ALIGN;
  return FA_OK;
}

inline int current(int* dev, fa_internal::DeviceView* view) {
  if (cudaGetDevice(dev) != cudaSuccess || *dev < 0 || *dev >= kMaxDevices) return FA_ERR_LAUNCH;
  if (!fa_internal::current_device(view)) return FA_ERR_LAUNCH;
  return view->supported ? FA_OK : FA_ERR_DEVICE;
}

// Tokens of a CTA of the store and load kernels: enough CTAs for a few per
// SM while there are, so that a decoding step's few tokens are spread out.
inline int tokens_per_cta(int T, int num_sms) {
  int n = kv::kMaxTokensPerCta;
  while (n > 1 && T < 4ll * num_sms * n) n /= 2;
  return n;
}

}  // namespace fa_internal
