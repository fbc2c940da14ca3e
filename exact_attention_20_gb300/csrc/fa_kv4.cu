// C ABI of the paged 4-bit cache: storing, loading, and the attention of the
// newest tokens over it.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <mutex>

#include "fa_gb300_serve.h"
#include "fa_internal.h"
#include "fa_kv4_decode.cuh"

namespace {

namespace kv = fa::kv4;

constexpr int kMaxDevices = 64;
std::mutex g_mu;
bool g_attr[kMaxDevices][2][3];  // shared-memory attribute set: [d == 128][row tiles of 8, 16, 32]

bool overlaps(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
  return a0 < b0 + nb && b0 < a0 + na;
}

bool misaligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

// log2 of a page size the cache takes, or -1.
int page_shift(int page_size) {
  for (int s = 4; s <= 10; ++s)
    if (page_size == 1 << s) return s;
  return -1;
}

// A tensor's scale: a power of two from 2^-40 to 2^40.
bool power_of_two(float g) {
  int e = 0;
  return std::isfinite(g) && g > 0.f && std::frexp(g, &e) == 0.5f && e >= -39 && e <= 41;
}

// The cache's own sizes and the tables'; shared by every entry point.
int check_cache(const void* cache, const int* page_table, const int* seq_lens, int n_seqs, int max_pages,
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

int current(int* dev, fa_internal::DeviceView* view) {
  if (cudaGetDevice(dev) != cudaSuccess || *dev < 0 || *dev >= kMaxDevices) return FA_ERR_LAUNCH;
  if (!fa_internal::current_device(view)) return FA_ERR_LAUNCH;
  return view->supported ? FA_OK : FA_ERR_DEVICE;
}

// Tokens of a CTA of the store and load kernels: enough CTAs for a few per
// SM while there are, so that a decoding step's few tokens are spread out.
int tokens_per_cta(int T, int num_sms) {
  int n = kv::kMaxTokensPerCta;
  while (n > 1 && T < 4ll * num_sms * n) n /= 2;
  return n;
}

int move(bool store, const void* k, const void* v, void* k_out, void* v_out, void* cache, const int* page_table,
         const int* seq_lens, const int* cu, int T, int n_seqs, int max_pages, int num_pages, int page_size, int Hkv,
         int d, long long k_stride, long long v_stride, float k_scale, float v_scale, int* errors, void* stream) {
  size_t cb = 0;
  int rc = check_cache(cache, page_table, seq_lens, n_seqs, max_pages, num_pages, page_size, Hkv, d, k_scale, v_scale,
                       &cb);
  if (rc != FA_OK) return rc;
  const long long row = static_cast<long long>(Hkv) * d;
  if (T < 0 || T > (1 << 30) || k_stride < row || v_stride < row || k_stride % 8 || v_stride % 8 ||
      k_stride > (1ll << 32) || v_stride > (1ll << 32))
    return FA_ERR_INVALID_ARG;
  if (T == 0 || n_seqs == 0) return FA_OK;
  const void* a = store ? k : k_out;
  const void* b = store ? v : v_out;
  if (!a || !b || !cu) return FA_ERR_NULL;
  if (misaligned(a, 16) || misaligned(b, 16) || misaligned(cu, 4) || misaligned(errors, 4)) return FA_ERR_ALIGN;
  const size_t ab = (static_cast<size_t>(T - 1) * k_stride + row) * 2, bb = (static_cast<size_t>(T - 1) * v_stride + row) * 2;
  const size_t pb = static_cast<size_t>(n_seqs) * max_pages * 4, lb = static_cast<size_t>(n_seqs) * 4;
  // what is written against everything else
  const void* out[2] = {store ? cache : a, store ? cache : b};
  const size_t out_bytes[2] = {store ? cb : ab, store ? cb : bb};
  const void* in[6] = {page_table, seq_lens, cu, store ? a : cache, store ? b : nullptr, errors};
  const size_t in_bytes[6] = {pb, lb, lb + 4, store ? ab : cb, bb, 4};
  for (int i = 0; i < 2; ++i)
    for (int j = 0; j < 6; ++j)
      if (in[j] && overlaps(out[i], out_bytes[i], in[j], in_bytes[j])) return FA_ERR_ALIAS;
  if (!store && overlaps(a, ab, b, bb)) return FA_ERR_ALIAS;
  for (int j = 0; j < 5; ++j)
    if (errors && in[j] && overlaps(errors, 4, in[j], in_bytes[j])) return FA_ERR_ALIAS;
  int dev = 0;
  fa_internal::DeviceView view;
  rc = current(&dev, &view);
  if (rc != FA_OK) return rc;
  kv::MoveParams p{};
  p.k = static_cast<const __nv_bfloat16*>(k);
  p.v = static_cast<const __nv_bfloat16*>(v);
  p.k_out = static_cast<__nv_bfloat16*>(k_out);
  p.v_out = static_cast<__nv_bfloat16*>(v_out);
  p.cache = static_cast<uint8_t*>(cache);
  p.page_table = page_table;
  p.seq_lens = seq_lens;
  p.cu = cu;
  p.errors = errors;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.T = T;
  p.n_seqs = n_seqs;
  p.max_pages = max_pages;
  p.num_pages = num_pages;
  p.page_shift = page_shift(page_size);
  p.Hkv = Hkv;
  p.k_scale = store ? 1.f / k_scale : k_scale;
  p.v_scale = store ? 1.f / v_scale : v_scale;
  p.tokens_per_cta = tokens_per_cta(T, view.num_sms);
  p.wide = !misaligned(a, 32) && !misaligned(b, 32) && k_stride % 16 == 0 && v_stride % 16 == 0;
  const int grid = (T + p.tokens_per_cta - 1) / p.tokens_per_cta;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (store) {
    if (d == 128) kv::store_kernel<128><<<grid, kv::kMoveThreads, 0, s>>>(p);
    else kv::store_kernel<64><<<grid, kv::kMoveThreads, 0, s>>>(p);
  } else {
    if (d == 128) kv::load_kernel<128><<<grid, kv::kMoveThreads, 0, s>>>(p);
    else kv::load_kernel<64><<<grid, kv::kMoveThreads, 0, s>>>(p);
  }
  return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_LAUNCH;
}

// How a call's query rows and its work are divided.
struct DecodePlan {
  int nt;         // row tiles of 8 nt rows
  int row_tiles;
  int split;      // ranges of equal tiles, merged afterwards; else one CTA per item
  long long grid;
  size_t bytes;   // workspace
};

DecodePlan decode_plan(int n_seqs, int Lq, int G, int Hkv, int d, int max_pages, int page_size, int num_sms) {
  DecodePlan pl{};
  const int rows = Lq * G;
  pl.nt = rows <= 8 ? 1 : rows <= 16 ? 2 : 4;
  pl.row_tiles = (rows + 8 * pl.nt - 1) / (8 * pl.nt);
  const long long items = static_cast<long long>(n_seqs) * Hkv * pl.row_tiles;
  const long long units = (static_cast<long long>(max_pages) * page_size + kv::kUnit - 1) / kv::kUnit;  // of an item, at most
  // Items that cannot be longer than a CTA's least share are taken whole.
  pl.split = units > kv::kMinUnits;
  if (!pl.split) {
    pl.grid = items;
    return pl;
  }
  pl.grid = std::min(static_cast<long long>(num_sms), (items * std::min(units, 1ll << 26) + kv::kMinUnits - 1) / kv::kMinUnits);
  // parts: two of a CTA and one of each warp (O), the CTAs' (m, l), and the cuts
  const size_t all_rows = static_cast<size_t>(pl.grid) * 8 * pl.nt;
  pl.bytes = all_rows * (2 + kv::kMaxWarps) * d * 4 + all_rows * 2 * 8 + static_cast<size_t>(pl.grid) * sizeof(kv::Cut);
  return pl;
}

template <int D, int NT>
int launch_decode(const kv::DecodeParams& p, const DecodePlan& pl, int dev, cudaStream_t stream) {
  auto kernel = kv::decode_kernel<D, NT>;
  constexpr int smem = kv::DecodeCfg<D, NT>::kSmemBytes;
  {
    std::lock_guard<std::mutex> lock(g_mu);
    bool& set = g_attr[dev][D == 128][NT / 2];
    if (!set) {
      if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
        return FA_ERR_LAUNCH;
      set = true;
    }
  }
  kernel<<<static_cast<int>(pl.grid), kv::DecodeCfg<D, NT>::kThreads, smem, stream>>>(p);
  if (cudaGetLastError() != cudaSuccess) return FA_ERR_LAUNCH;
  if (!pl.split) return FA_OK;
  // the merge may be set up while the first kernel runs; its CTAs wait for it
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(pl.grid), 8 * NT / kv::kMergeRows);
  cfg.blockDim = dim3(kv::kMergeThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kv::merge_kernel<D>, p, 8 * NT) != cudaSuccess)
    return FA_ERR_LAUNCH;
  return FA_OK;
}

int check_decode_sizes(int n_seqs, int Lq, int Hq, int Hkv, int d, int max_pages, int page_size) {
  if (n_seqs < 0 || Lq < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || Hkv > (1 << 16) || Hq / Hkv > 128 ||
      (d != 64 && d != 128) || max_pages < 1 || page_shift(page_size) < 0)
    return FA_ERR_INVALID_ARG;
  // rows of a KV head, items and output rows within 32 bits
  const long long rows = static_cast<long long>(Lq) * (Hq / Hkv);
  if (Lq > (1 << 16) || rows > (1 << 20) || static_cast<long long>(n_seqs) * Lq > (1 << 30)) return FA_ERR_INVALID_ARG;
  if (static_cast<long long>(n_seqs) * Hkv * ((rows + 7) / 8) > (1ll << 30)) return FA_ERR_INVALID_ARG;
  return FA_OK;
}

}  // namespace

extern "C" {

int fa_kv4_store(const void* k, const void* v, void* cache, const int* page_table, const int* seq_lens,
                 const int* cu_seqlens, int T, int n_seqs, int max_pages, int num_pages, int page_size, int Hkv, int d,
                 long long k_stride, long long v_stride, float k_scale, float v_scale, int* errors, void* stream) {
  return move(true, k, v, nullptr, nullptr, cache, page_table, seq_lens, cu_seqlens, T, n_seqs, max_pages, num_pages,
              page_size, Hkv, d, k_stride, v_stride, k_scale, v_scale, errors, stream);
}

int fa_kv4_load(const void* cache, const int* page_table, const int* seq_lens, const int* cu_seqlens, void* k, void* v,
                int T, int n_seqs, int max_pages, int num_pages, int page_size, int Hkv, int d, float k_scale,
                float v_scale, int* errors, void* stream) {
  const long long row = Hkv > 0 && Hkv <= (1 << 16) ? static_cast<long long>(Hkv) * d : 0;
  return move(false, nullptr, nullptr, k, v, const_cast<void*>(cache), page_table, seq_lens, cu_seqlens, T, n_seqs,
              max_pages, num_pages, page_size, Hkv, d, row, row, k_scale, v_scale, errors, stream);
}

int fa_kv4_attention_workspace(int n_seqs, int Lq, int Hq, int Hkv, int d, int max_pages, int page_size,
                               size_t* bytes) {
  if (bytes == nullptr) return FA_ERR_NULL;
  int rc = check_decode_sizes(n_seqs, Lq, Hq, Hkv, d, max_pages, page_size);
  if (rc != FA_OK) return rc;
  int dev = 0;
  fa_internal::DeviceView view;
  rc = current(&dev, &view);
  if (rc != FA_OK) return rc;
  *bytes = n_seqs == 0 ? 0 : decode_plan(n_seqs, Lq, Hq / Hkv, Hkv, d, max_pages, page_size, view.num_sms).bytes;
  return FA_OK;
}

int fa_kv4_attention(const void* q, const void* cache, const int* page_table, const int* seq_lens, void* o, float* lse,
                     int n_seqs, int Lq, int Hq, int Hkv, int d, int max_pages, int num_pages, int page_size,
                     long long q_stride, float scale, float k_scale, float v_scale, int* errors, void* workspace,
                     size_t workspace_bytes, void* stream) {
  int rc = check_decode_sizes(n_seqs, Lq, Hq, Hkv, d, max_pages, page_size);
  if (rc != FA_OK) return rc;
  size_t cb = 0;
  rc = check_cache(cache, page_table, seq_lens, n_seqs, max_pages, num_pages, page_size, Hkv, d, k_scale, v_scale, &cb);
  if (rc != FA_OK) return rc;
  const long long row = static_cast<long long>(Hq) * d;
  const float qk_scale = static_cast<float>(static_cast<double>(scale) * k_scale * 1.4426950408889634);
  if (!std::isfinite(scale) || !(scale > 0.f) || !std::isfinite(qk_scale) || !(qk_scale > 0.f) || q_stride < row ||
      q_stride % 8 || q_stride > (1ll << 32))
    return FA_ERR_INVALID_ARG;
  if (n_seqs == 0) return FA_OK;
  if (!q || !o || !lse) return FA_ERR_NULL;
  if (misaligned(q, 16) || misaligned(o, 16) || misaligned(lse, 4) || misaligned(errors, 4) ||
      misaligned(workspace, 256))
    return FA_ERR_ALIGN;
  const size_t T = static_cast<size_t>(n_seqs) * Lq;
  const void* in[5] = {q, cache, page_table, seq_lens, errors};
  const size_t in_bytes[5] = {((T - 1) * q_stride + row) * 2, cb, static_cast<size_t>(n_seqs) * max_pages * 4,
                              static_cast<size_t>(n_seqs) * 4, 4};
  const void* out[3] = {o, lse, workspace};
  const size_t out_bytes[3] = {T * row * 2, T * Hq * 4, workspace_bytes};
  for (int i = 0; i < 3; ++i) {
    if (out[i] == nullptr) continue;
    for (int j = 0; j < 5; ++j)
      if (in[j] && overlaps(out[i], out_bytes[i], in[j], in_bytes[j])) return FA_ERR_ALIAS;
    for (int j = i + 1; j < 3; ++j)
      if (out[j] && overlaps(out[i], out_bytes[i], out[j], out_bytes[j])) return FA_ERR_ALIAS;
  }
  for (int j = 0; j < 4; ++j)
    if (errors && overlaps(errors, 4, in[j], in_bytes[j])) return FA_ERR_ALIAS;
  int dev = 0;
  fa_internal::DeviceView view;
  rc = current(&dev, &view);
  if (rc != FA_OK) return rc;
  const DecodePlan pl = decode_plan(n_seqs, Lq, Hq / Hkv, Hkv, d, max_pages, page_size, view.num_sms);
  if (pl.bytes > 0 && (workspace == nullptr || workspace_bytes < pl.bytes)) return FA_ERR_SCRATCH;
  kv::DecodeParams p{};
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.cache = static_cast<const uint8_t*>(cache);
  p.page_table = page_table;
  p.seq_lens = seq_lens;
  p.o = static_cast<__nv_bfloat16*>(o);
  p.lse = lse;
  const long long rows = pl.grid * 8 * pl.nt;
  p.part_o = static_cast<float*>(workspace);
  p.first_o = p.part_o + 2 * rows * d;
  p.part_ml = reinterpret_cast<float2*>(p.first_o + kv::kMaxWarps * rows * d);
  p.cuts = reinterpret_cast<kv::Cut*>(p.part_ml + 2 * rows);
  p.errors = errors;
  p.status = view.status;
  p.q_stride = q_stride;
  p.wait_limit_ns = fa_internal::kWaitLimitNs;
  p.qk_scale = qk_scale;
  p.v_scale = v_scale;
  p.n_seqs = n_seqs;
  p.Lq = Lq;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.G = Hq / Hkv;
  p.row_tiles = pl.row_tiles;
  p.max_pages = max_pages;
  p.num_pages = num_pages;
  p.page_shift = page_shift(page_size);
  p.split = pl.split;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (d == 128)
    return pl.nt == 1 ? launch_decode<128, 1>(p, pl, dev, s)
         : pl.nt == 2 ? launch_decode<128, 2>(p, pl, dev, s) : launch_decode<128, 4>(p, pl, dev, s);
  return pl.nt == 1 ? launch_decode<64, 1>(p, pl, dev, s)
       : pl.nt == 2 ? launch_decode<64, 2>(p, pl, dev, s) : launch_decode<64, 4>(p, pl, dev, s);
}

}  // extern "C"
