// C ABI of drafted tokens: verification, and keeping the accepted ones in the
// cache.  (Their attention is launched with the cache's other attention.)
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <mutex>

#include "fa_gb300_draft.h"
#include "fa_keep.cuh"
#include "fa_kv4_host.h"
#include "fa_verify.cuh"

namespace {

namespace vf = fa::verify;
using namespace fa_internal;

// What a device holds of verify_kernel.
struct Held {
  int cluster;  // the largest cluster; 0: not asked yet
  int wide;     // CTAs of such clusters that are on the card at once, of kThreads threads
};

std::mutex g_mu;
Held g_held[kMaxDevices];

Held held(int dev) {
  std::lock_guard<std::mutex> lock(g_mu);
  Held& h = g_held[dev];
  if (h.cluster == 0) {
    const auto a = vf::verify_kernel<true>;
    const auto b = vf::verify_kernel<false>;
    const bool large = cudaFuncSetAttribute(a, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
                       cudaFuncSetAttribute(b, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess;
    for (h.cluster = large ? vf::kMaxCluster : 8; h.cluster > 1; h.cluster /= 2) {
      cudaLaunchConfig_t cfg{};
      cfg.gridDim = dim3(h.cluster);
      cfg.blockDim = dim3(vf::kThreads);
      cudaLaunchAttribute attr{};
      attr.id = cudaLaunchAttributeClusterDimension;
      attr.val.clusterDim.x = h.cluster;
      attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
      cfg.attrs = &attr;
      cfg.numAttrs = 1;
      int n[2] = {0, 0};
      if (cudaOccupancyMaxActiveClusters(&n[0], a, &cfg) == cudaSuccess &&
          cudaOccupancyMaxActiveClusters(&n[1], b, &cfg) == cudaSuccess && std::min(n[0], n[1]) > 0) {
        h.wide = std::min(n[0], n[1]) * h.cluster;
        break;
      }
    }
    cudaGetLastError();  // what was refused there is no error of this call
  }
  return h;
}

// CTAs of a sequence's cluster, and their threads.  A walk's passes follow one another,
// so that a sequence wants as many warps as have a tile, but sequences that wait for
// others to end want fewer: 256 threads where all clusters are on the card at once, else
// 128 (fp32, 128000 tokens: 1, 16 and 48 sequences 30, 53 and 82 us with 256, 39, 66 and 75
// with 128).  Clusters of eight, not of 16, leave the card idle
// behind the sequences that are done (48 sequences, 164 us for 145 at the time).
void shape(const Held& h, int n_seqs, int V, int* cluster, int* threads) {
  const int tiles = (V + vf::kTile - 1) / vf::kTile;
  auto size = [&](int warps) {
    int c = h.cluster;
    while (c > 1 && tiles <= warps * (c - 1)) c /= 2;
    return c;
  };
  *cluster = size(vf::kWarps);
  *threads = vf::kThreads;
  if (static_cast<long long>(n_seqs) * *cluster > h.wide) *threads = vf::kThreads / 2, *cluster = size(vf::kWarps / 2);
}

}  // namespace

extern "C" {

int fa_verify_tree(const void* logits, int logits_fp32, const int* tokens, const int* parents, const float* uniforms,
                   const float* draft_probs, int* path, int* n_kept, int* next_token, int n_seqs, int n_nodes, int V,
                   long long logits_stride, long long draft_stride, float temperature, void* stream) {
  constexpr long long kMaxStride = 1ll << 32;
  const double c = 1.4426950408889634 / static_cast<double>(temperature);
  if ((logits_fp32 != 0 && logits_fp32 != 1) || n_seqs < 0 || n_seqs > (1 << 24) || n_nodes < 1 || n_nodes > vf::kMaxNodes ||
      V < 1 || V > vf::kMaxVocab || logits_stride < V || logits_stride > kMaxStride ||
      (draft_probs && (draft_stride < V || draft_stride > kMaxStride)) || !(temperature >= 0.f) || !std::isfinite(temperature) ||
      (temperature > 0.f && !(c < 1e30 && c > 1e-30)))
    return FA_ERR_INVALID_ARG;
  if (n_seqs == 0) return FA_OK;
  if (!logits || !tokens || !parents || !uniforms || !path || !n_kept || !next_token) return FA_ERR_NULL;
  if (misaligned(logits, logits_fp32 ? 4 : 2) || misaligned(tokens, 4) || misaligned(parents, 4) || misaligned(uniforms, 4) ||
      misaligned(draft_probs, 4) || misaligned(path, 4) || misaligned(n_kept, 4) || misaligned(next_token, 4))
    return FA_ERR_ALIGN;
  const size_t rows = static_cast<size_t>(n_seqs) * n_nodes, nb = rows * 4, sb = static_cast<size_t>(n_seqs) * 4;
  const void* in[5] = {logits, tokens, parents, uniforms, draft_probs};
  const size_t in_bytes[5] = {((rows - 1) * logits_stride + V) * (logits_fp32 ? 4 : 2), nb, nb, nb,
                              ((rows - 1) * draft_stride + V) * 4};
  const void* out[3] = {path, n_kept, next_token};
  const size_t out_bytes[3] = {nb, sb, sb};
  for (int i = 0; i < 3; ++i) {
    for (int j = 0; j < 5; ++j)
      if (in[j] && overlaps(out[i], out_bytes[i], in[j], in_bytes[j])) return FA_ERR_ALIAS;
    for (int j = i + 1; j < 3; ++j)
      if (overlaps(out[i], out_bytes[i], out[j], out_bytes[j])) return FA_ERR_ALIAS;
  }
  int dev = 0;
  DeviceView view;
  const int rc = current(&dev, &view);
  if (rc != FA_OK) return rc;
  vf::Params p{};
  p.logits = logits;
  p.tokens = tokens;
  p.parents = parents;
  p.uniforms = uniforms;
  p.draft = draft_probs;
  p.path = path;
  p.n_kept = n_kept;
  p.next_token = next_token;
  p.n_nodes = n_nodes;
  p.V = V;
  p.logits_stride = logits_stride;
  p.draft_stride = draft_stride;
  p.greedy = temperature == 0.f;
  if (!p.greedy) {
    p.c_hi = static_cast<float>(c);
    p.c_lo = static_cast<float>(c - static_cast<double>(p.c_hi));
    p.span = static_cast<float>(vf::kSpan / c);
  }
  int size = 0, threads = 0;
  shape(held(dev), n_seqs, V, &size, &threads);
  p.quick = vf::quick_bound(vf::lane_tiles(V, size, threads / 32));
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(n_seqs) * size);
  cfg.blockDim = dim3(threads);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = size;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  const cudaError_t err = logits_fp32 ? cudaLaunchKernelEx(&cfg, vf::verify_kernel<true>, p)
                                      : cudaLaunchKernelEx(&cfg, vf::verify_kernel<false>, p);
  return err == cudaSuccess ? FA_OK : FA_ERR_LAUNCH;
}

int fa_kv4_keep(void* cache, const int* page_table, const int* seq_lens, const int* path, const int* n_kept,
                int* new_lens, int n_seqs, int n_nodes, int max_pages, int num_pages, int page_size, int Hkv, int d,
                int* errors, void* stream) {
  size_t cb = 0;
  int rc = check_cache(cache, page_table, seq_lens, n_seqs, max_pages, num_pages, page_size, Hkv, d, 1.f, 1.f, &cb);
  if (rc != FA_OK) return rc;
  if (n_nodes < 1 || n_nodes > fa::kv4::kKeepNodes || static_cast<long long>(n_seqs) * Hkv > 0x7fffffffll) return FA_ERR_INVALID_ARG;
  if (n_seqs == 0) return FA_OK;
  if (!path || !n_kept || !new_lens) return FA_ERR_NULL;
  if (misaligned(path, 4) || misaligned(n_kept, 4) || misaligned(new_lens, 4) || misaligned(errors, 4)) return FA_ERR_ALIGN;
  const size_t sb = static_cast<size_t>(n_seqs) * 4;
  const void* out[3] = {cache, new_lens, errors};
  const size_t out_bytes[3] = {cb, sb, 4};
  const void* in[4] = {page_table, seq_lens, path, n_kept};
  const size_t in_bytes[4] = {sb * max_pages, sb, sb * n_nodes, sb};
  for (int i = 0; i < 3; ++i) {
    if (out[i] == nullptr) continue;
    for (int j = 0; j < 4; ++j)
      if (overlaps(out[i], out_bytes[i], in[j], in_bytes[j])) return FA_ERR_ALIAS;
    for (int j = i + 1; j < 3; ++j)
      if (out[j] && overlaps(out[i], out_bytes[i], out[j], out_bytes[j])) return FA_ERR_ALIAS;
  }
  int dev = 0;
  DeviceView view;
  rc = current(&dev, &view);
  if (rc != FA_OK) return rc;
  fa::kv4::KeepParams p{};
  p.cache = static_cast<uint8_t*>(cache);
  p.page_table = page_table;
  p.seq_lens = seq_lens;
  p.path = path;
  p.n_kept = n_kept;
  p.new_lens = new_lens;
  p.errors = errors;
  p.n_nodes = n_nodes;
  p.max_pages = max_pages;
  p.num_pages = num_pages;
  p.page_shift = page_shift(page_size);
  p.Hkv = Hkv;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const unsigned grid = static_cast<unsigned>(n_seqs) * Hkv;
  if (d == 128) fa::kv4::keep_kernel<128><<<grid, fa::kv4::kKeepThreads, 0, s>>>(p);
  else fa::kv4::keep_kernel<64><<<grid, fa::kv4::kKeepThreads, 0, s>>>(p);
  return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_LAUNCH;
}

}  // extern "C"
