// C ABI of the paged 4-bit cache: storing, loading, and the attention of the
// newest tokens over it.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <mutex>

#include "fa_gb300_draft.h"
#include "fa_internal.h"
#include "fa_kv4_decode.cuh"
#include "fa_kv4_host.h"
#include "fa_kv4_tree.cuh"

namespace {

namespace kv = fa::kv4;
using namespace fa_internal;

constexpr int kMaxNodes = kv::kMaxTreeNodes;
// Rows of a KV head above which a tree goes to the tensor core's 128-row tiles.
// 32 contexts of 250 to 12000 tokens, 8 KV heads, tiles against kv4::decode_kernel:
// 16 rows 65.2 and 47.8 us at d = 128, 55.1 and 29.5 at d = 64; 24 rows 66.9 and
// 78.5, 55.5 and 52.8; one context of 20000, d = 128: 16 rows 26.5 and 23.9, 24
// rows 26.3 and 28.8.
constexpr int kTreeRows = 16;
// Rows of a KV head above which it does so where that is little work: items taken
// whole, or key tiles for no more than a CTA each.  8 KV heads, tiles against
// kv4::decode_kernel: 12 rows over 600 tokens 13.2 and 18.2 us at d = 128, 11.7 and
// 13.8 at d = 64; over 2000 15.4 and 18.7, 14.0 and 14.0; two contexts of 2000 17.8 and
// 19.6, 15.5 and 14.6.  8 rows over 600 tokens 13.4 and 13.3, over 2000 15.3 and 13.6.
constexpr int kFewRows = 8;
// Key tiles up to which a tree's items are taken whole, one by each CTA, where
// all are on the card at once: 16 nodes, 8 KV heads, five tiles 13.2 us and 14.4
// in parts that are merged; six tiles 15.0 and 14.4.
// Both rules take an item to be as long as the page table is wide: the lengths are on
// the device.  Under a table of 2048 pages of 64 the same 16 nodes over 600 tokens
// take 14.7 us for 13.2 (d = 64: 13.1 for 11.9), 12 rows over them 16.8 for 13.4.
constexpr int kWholeTiles = 5;

std::mutex g_mu;
bool g_tree_attr[kMaxDevices][2];  // of tree_kernel: [d == 128]
bool g_attr[kMaxDevices][2][2][3];  // shared-memory attribute set: [tree][d == 128][row tiles of 8, 16, 32]

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

// The same for a tree's rows in tiles of 128, with keys in tiles of 128.
DecodePlan tree_plan(int n_seqs, int nodes, int G, int Hkv, int d, int max_pages, int page_size, int num_sms) {
  namespace tr = kv::tree;
  DecodePlan pl{};
  pl.row_tiles = (nodes * G + tr::kRows - 1) / tr::kRows;
  const long long items = static_cast<long long>(n_seqs) * Hkv * pl.row_tiles;
  const long long tiles = (static_cast<long long>(max_pages) * page_size + tr::kKeys - 1) / tr::kKeys;  // of an item, at most
  pl.split = items > num_sms || tiles > kWholeTiles;
  if (!pl.split) {
    pl.grid = items;
    return pl;
  }
  pl.grid = std::min(static_cast<long long>(num_sms),
                     (items * std::min(tiles + tr::kItemTiles, 1ll << 26) + tr::kMinTiles - 1) / tr::kMinTiles);
  const size_t rows = static_cast<size_t>(pl.grid) * 2 * tr::kRows;  // parts: two of a CTA, and their (m, l); then the cuts
  pl.bytes = rows * d * 4 + rows * 8 + static_cast<size_t>(pl.grid) * sizeof(kv::Cut);
  return pl;
}

// How a call is divided; *tiles: by the tensor core's 128-row tiles.
DecodePlan plan(bool tree, int n_seqs, int Lq, int G, int Hkv, int d, int max_pages, int page_size, int num_sms, bool* tiles) {
  *tiles = false;
  if (tree && Lq * G > kFewRows) {
    const DecodePlan pl = tree_plan(n_seqs, Lq, G, Hkv, d, max_pages, page_size, num_sms);
    const long long keys = static_cast<long long>(max_pages) * page_size;
    const long long work = static_cast<long long>(n_seqs) * Hkv * ((keys + kv::tree::kKeys - 1) / kv::tree::kKeys);
    *tiles = Lq * G > kTreeRows || !pl.split || work <= num_sms;
    if (*tiles) return pl;
  }
  return decode_plan(n_seqs, Lq, G, Hkv, d, max_pages, page_size, num_sms);
}

// ROWS: of a CTA.  Items of 128 rows are in few parts, so that a row's threads take
// them one after another: with two rows a CTA, as for small items, 32 contexts of
// 24 nodes took 8 us longer.
template <int D, int ROWS>
int launch_merge(const kv::DecodeParams& p, const DecodePlan& pl, int rows, cudaStream_t stream) {
  // the merge may be set up while the first kernel runs; its CTAs wait for it
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(pl.grid), rows / ROWS);
  cfg.blockDim = dim3(kv::kMergeThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv::merge_kernel<D, ROWS>, p, rows) == cudaSuccess ? FA_OK : FA_ERR_LAUNCH;
}

template <int D>
int launch_tree(const kv::DecodeParams& p, const DecodePlan& pl, int dev, cudaStream_t stream) {
  auto kernel = kv::tree::tree_kernel<D>;
  constexpr int smem = kv::tree::Cfg<D>::kSmemBytes;
  {
    std::lock_guard<std::mutex> lock(g_mu);
    bool& set = g_tree_attr[dev][D == 128];
    if (!set) {
      if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
        return FA_ERR_LAUNCH;
      set = true;
    }
  }
  kernel<<<static_cast<int>(pl.grid), kv::tree::kThreads, smem, stream>>>(p);
  if (cudaGetLastError() != cudaSuccess) return FA_ERR_LAUNCH;
  return pl.split ? launch_merge<D, 4 * kv::kMergeThreads / D>(p, pl, kv::tree::kRows, stream) : FA_OK;
}

template <int D, int NT, bool TREE>
int launch_decode(const kv::DecodeParams& p, const DecodePlan& pl, int dev, cudaStream_t stream) {
  auto kernel = kv::decode_kernel<D, NT, TREE>;
  constexpr int smem = kv::DecodeCfg<D, NT>::kSmemBytes;
  {
    std::lock_guard<std::mutex> lock(g_mu);
    bool& set = g_attr[dev][TREE][D == 128][NT / 2];
    if (!set) {
      if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
        return FA_ERR_LAUNCH;
      set = true;
    }
  }
  kernel<<<static_cast<int>(pl.grid), kv::DecodeCfg<D, NT>::kThreads, smem, stream>>>(p);
  if (cudaGetLastError() != cudaSuccess) return FA_ERR_LAUNCH;
  return pl.split ? launch_merge<D, 2>(p, pl, 8 * NT, stream) : FA_OK;
}

template <int D, bool TREE>
int launch_rows(const kv::DecodeParams& p, const DecodePlan& pl, int dev, cudaStream_t s) {
  if (pl.nt == 1) return launch_decode<D, 1, TREE>(p, pl, dev, s);
  if constexpr (!TREE) {  // (more rows of a tree go to its own kernel)
    if (pl.nt == 4) return launch_decode<D, 4, TREE>(p, pl, dev, s);
  }
  return launch_decode<D, 2, TREE>(p, pl, dev, s);
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

int attention_workspace(bool tree, int n_seqs, int Lq, int Hq, int Hkv, int d, int max_pages, int page_size, size_t* bytes) {
  if (bytes == nullptr) return FA_ERR_NULL;
  int rc = check_decode_sizes(n_seqs, Lq, Hq, Hkv, d, max_pages, page_size);
  if (rc != FA_OK) return rc;
  int dev = 0;
  fa_internal::DeviceView view;
  rc = current(&dev, &view);
  if (rc != FA_OK) return rc;
  bool tiles = false;
  *bytes = n_seqs == 0 ? 0 : plan(tree, n_seqs, Lq, Hq / Hkv, Hkv, d, max_pages, page_size, view.num_sms, &tiles).bytes;
  return FA_OK;
}

// The attention of the newest tokens, in order or as a tree's nodes.
int attention(bool tree, const void* q, const void* cache, const int* page_table, const int* seq_lens,
              const int* parents, void* o, float* lse, int n_seqs, int Lq, int Hq, int Hkv, int d, int max_pages,
              int num_pages, int page_size, long long q_stride, float scale, float k_scale, float v_scale, int* errors,
              void* workspace, size_t workspace_bytes, void* stream) {
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
  if (!q || !o || !lse || (tree && !parents)) return FA_ERR_NULL;
  if (misaligned(q, 16) || misaligned(o, 16) || misaligned(lse, 4) || misaligned(errors, 4) ||
      misaligned(parents, 4) || misaligned(workspace, 256))
    return FA_ERR_ALIGN;
  const size_t T = static_cast<size_t>(n_seqs) * Lq;
  const void* in[6] = {q, cache, page_table, seq_lens, parents, errors};
  const size_t in_bytes[6] = {((T - 1) * q_stride + row) * 2, cb, static_cast<size_t>(n_seqs) * max_pages * 4,
                              static_cast<size_t>(n_seqs) * 4, T * 4, 4};
  const void* out[3] = {o, lse, workspace};
  const size_t out_bytes[3] = {T * row * 2, T * Hq * 4, workspace_bytes};
  for (int i = 0; i < 3; ++i) {
    if (out[i] == nullptr) continue;
    for (int j = 0; j < 6; ++j)
      if (in[j] && overlaps(out[i], out_bytes[i], in[j], in_bytes[j])) return FA_ERR_ALIAS;
    for (int j = i + 1; j < 3; ++j)
      if (out[j] && overlaps(out[i], out_bytes[i], out[j], out_bytes[j])) return FA_ERR_ALIAS;
  }
  for (int j = 0; j < 5; ++j)
    if (errors && in[j] && overlaps(errors, 4, in[j], in_bytes[j])) return FA_ERR_ALIAS;
  int dev = 0;
  fa_internal::DeviceView view;
  rc = current(&dev, &view);
  if (rc != FA_OK) return rc;
  bool tiles = false;
  const DecodePlan pl = plan(tree, n_seqs, Lq, Hq / Hkv, Hkv, d, max_pages, page_size, view.num_sms, &tiles);
  if (pl.bytes > 0 && (workspace == nullptr || workspace_bytes < pl.bytes)) return FA_ERR_SCRATCH;
  kv::DecodeParams p{};
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.cache = static_cast<const uint8_t*>(cache);
  p.page_table = page_table;
  p.seq_lens = seq_lens;
  p.o = static_cast<__nv_bfloat16*>(o);
  p.lse = lse;
  const long long rows = pl.grid * (tiles ? kv::tree::kRows : 8 * pl.nt);
  p.part_o = static_cast<float*>(workspace);
  p.first_o = p.part_o + 2 * rows * d;
  p.part_ml = reinterpret_cast<float2*>(p.first_o + (tiles ? 0 : kv::kMaxWarps * rows * d));
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
  p.parents = parents;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (tiles) return d == 128 ? launch_tree<128>(p, pl, dev, s) : launch_tree<64>(p, pl, dev, s);
  if (tree) return d == 128 ? launch_rows<128, true>(p, pl, dev, s) : launch_rows<64, true>(p, pl, dev, s);
  return d == 128 ? launch_rows<128, false>(p, pl, dev, s) : launch_rows<64, false>(p, pl, dev, s);
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
  return attention_workspace(false, n_seqs, Lq, Hq, Hkv, d, max_pages, page_size, bytes);
}

int fa_kv4_attention(const void* q, const void* cache, const int* page_table, const int* seq_lens, void* o, float* lse,
                     int n_seqs, int Lq, int Hq, int Hkv, int d, int max_pages, int num_pages, int page_size,
                     long long q_stride, float scale, float k_scale, float v_scale, int* errors, void* workspace,
                     size_t workspace_bytes, void* stream) {
  return attention(false, q, cache, page_table, seq_lens, nullptr, o, lse, n_seqs, Lq, Hq, Hkv, d, max_pages, num_pages,
                   page_size, q_stride, scale, k_scale, v_scale, errors, workspace, workspace_bytes, stream);
}

int fa_kv4_tree_attention_workspace(int n_seqs, int n_nodes, int Hq, int Hkv, int d, int max_pages, int page_size,
                                    size_t* bytes) {
  if (n_nodes > kMaxNodes) return FA_ERR_INVALID_ARG;
  return attention_workspace(true, n_seqs, n_nodes, Hq, Hkv, d, max_pages, page_size, bytes);
}

int fa_kv4_tree_attention(const void* q, const void* cache, const int* page_table, const int* seq_lens,
                          const int* parents, void* o, float* lse, int n_seqs, int n_nodes, int Hq, int Hkv, int d,
                          int max_pages, int num_pages, int page_size, long long q_stride, float scale, float k_scale,
                          float v_scale, int* errors, void* workspace, size_t workspace_bytes, void* stream) {
  if (n_nodes > kMaxNodes) return FA_ERR_INVALID_ARG;
  return attention(true, q, cache, page_table, seq_lens, parents, o, lse, n_seqs, n_nodes, Hq, Hkv, d, max_pages,
                   num_pages, page_size, q_stride, scale, k_scale, v_scale, errors, workspace, workspace_bytes, stream);
}

}  // extern "C"
