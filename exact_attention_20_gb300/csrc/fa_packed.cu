// C ABI of the attention over packed prompts: argument checks, the work plan,
// TMA tensor maps and the launches (one per 1024 sequences).
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <mutex>

#include "fa_gb300_serve.h"
#include "fa_internal.h"
#include "fa_packed_plan.h"
#include "tma_host.h"

namespace {

namespace pk = fa::packed;

constexpr int kMaxDevices = 64;
std::mutex g_mu;
bool g_attr[kMaxDevices][2][2];  // shared-memory attribute set: [d == 128][causal]

bool overlaps(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
  return a0 < b0 + nb && b0 < a0 + na;
}

// Host checks of the sizes; *total = the sequences' tokens.
int check_sizes(const int* seq_lens, int n_seqs, int T, int Hq, int Hkv, int d, int causal, long long* total) {
  *total = 0;
  if (n_seqs < 0 || T < 0 || T > (1 << 30) || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || Hq / Hkv > fa::kBlockM)
    return FA_ERR_INVALID_ARG;
  if ((d != 64 && d != 128) || (causal != 0 && causal != 1)) return FA_ERR_INVALID_ARG;
  // heads x d: a token's row, whose byte size has to fit an int and TMA's limits
  if (Hq > (1 << 20)) return FA_ERR_INVALID_ARG;
  if (n_seqs > 0 && seq_lens == nullptr) return FA_ERR_NULL;
  for (int i = 0; i < n_seqs; ++i) {
    if (seq_lens[i] < 0) return FA_ERR_INVALID_ARG;
    *total += seq_lens[i];
    if (*total > T) return FA_ERR_INVALID_ARG;
  }
  return FA_OK;
}

int make_plan(const int* seq_lens, int n, int begin, int Hkv, int tpt, int causal, int num_ctas, pk::Params& p,
              int& n_slots, int& n_split) {
  p.cu[0] = begin;
  for (int i = 0; i < n; ++i) p.cu[i + 1] = p.cu[i] + seq_lens[i];
  return causal ? pk::make_plan<true>(n, Hkv, tpt, num_ctas, p, n_slots, n_split)
                : pk::make_plan<false>(n, Hkv, tpt, num_ctas, p, n_slots, n_split);
}

// Workspace: the parts' O, then their logsumexps, then the arrival counters.
size_t workspace_bytes(int n_slots, int n_split, int d) {
  return (static_cast<size_t>(n_slots) * fa::kItemRows * (d + 1) +
          static_cast<size_t>(n_split) * pk::kCountersPerItem) * 4;
}

template <int D, bool CAUSAL>
int launch(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const pk::Params& p, int grid, int dev,
           cudaStream_t stream) {
  auto kernel = pk::fa_packed_kernel<D, CAUSAL>;
  constexpr int smem = pk::PackedCfg<D>::kSmemBytes;
  {
    std::lock_guard<std::mutex> lock(g_mu);
    bool& set = g_attr[dev][D == 128][CAUSAL];
    if (!set) {
      if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
        return FA_ERR_LAUNCH;
      set = true;
    }
  }
  kernel<<<grid, fa::kNumThreads, smem, stream>>>(tq, tk, tv, p);
  return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_LAUNCH;
}

}  // namespace

extern "C" {

int fa_fwd_packed_workspace(const int* seq_lens, int n_seqs, int T, int Hq, int Hkv, int d, int causal,
                            size_t* bytes) {
  if (bytes == nullptr) return FA_ERR_NULL;
  long long total = 0;
  const int rc = check_sizes(seq_lens, n_seqs, T, Hq, Hkv, d, causal, &total);
  if (rc != FA_OK) return rc;
  fa_internal::DeviceView view;
  if (!fa_internal::current_device(&view)) return FA_ERR_LAUNCH;
  if (!view.supported) return FA_ERR_DEVICE;
  *bytes = 0;
  pk::Params p;
  int begin = 0;
  for (int i = 0; i < n_seqs; i += pk::kMaxSeqs) {
    const int n = std::min(pk::kMaxSeqs, n_seqs - i);
    int n_slots = 0, n_split = 0;
    make_plan(seq_lens + i, n, begin, Hkv, fa::kBlockM / (Hq / Hkv), causal, view.num_sms, p, n_slots, n_split);
    begin = p.cu[n];
    *bytes = std::max(*bytes, workspace_bytes(n_slots, n_split, d));
  }
  return FA_OK;
}

int fa_fwd_packed(const void* q, const void* k, const void* v, void* o, float* lse, const int* seq_lens, int n_seqs,
                  int T, int Hq, int Hkv, int d, long long q_stride, long long k_stride, long long v_stride,
                  int causal, float scale, void* workspace, size_t ws_bytes, void* stream) {
  long long total = 0;
  int rc = check_sizes(seq_lens, n_seqs, T, Hq, Hkv, d, causal, &total);
  if (rc != FA_OK) return rc;
  const float qk_scale = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
  if (!std::isfinite(qk_scale) || !(scale > 0.f)) return FA_ERR_INVALID_ARG;
  const long long q_row = static_cast<long long>(Hq) * d, kv_row = static_cast<long long>(Hkv) * d;
  constexpr long long kMaxStride = 1ll << 32;  // TMA takes byte strides below 2^40
  if (q_stride < q_row || k_stride < kv_row || v_stride < kv_row || q_stride % 8 || k_stride % 8 || v_stride % 8 ||
      q_stride > kMaxStride || k_stride > kMaxStride || v_stride > kMaxStride)
    return FA_ERR_INVALID_ARG;
  if (total == 0) return FA_OK;
  if (!q || !k || !v || !o || !lse) return FA_ERR_NULL;
  auto mis = [](const void* x, uintptr_t a) { return (reinterpret_cast<uintptr_t>(x) & (a - 1)) != 0; };
  if (mis(q, 16) || mis(k, 16) || mis(v, 16) || mis(o, 16) || mis(lse, 4) || mis(workspace, 256)) return FA_ERR_ALIGN;
  const size_t ob = static_cast<size_t>(T) * q_row * 2, lb = static_cast<size_t>(T) * Hq * 4;
  auto extent = [&](long long stride, long long row) { return (static_cast<size_t>(T - 1) * stride + row) * 2; };
  const void* ins[3] = {q, k, v};
  const size_t in_bytes[3] = {extent(q_stride, q_row), extent(k_stride, kv_row), extent(v_stride, kv_row)};
  for (int i = 0; i < 3; ++i) {
    if (overlaps(o, ob, ins[i], in_bytes[i]) || overlaps(lse, lb, ins[i], in_bytes[i])) return FA_ERR_ALIAS;
    if (workspace && overlaps(workspace, ws_bytes, ins[i], in_bytes[i])) return FA_ERR_ALIAS;
  }
  if (overlaps(o, ob, lse, lb)) return FA_ERR_ALIAS;
  if (workspace && (overlaps(workspace, ws_bytes, o, ob) || overlaps(workspace, ws_bytes, lse, lb))) return FA_ERR_ALIAS;

  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return FA_ERR_LAUNCH;
  fa_internal::DeviceView view;
  if (!fa_internal::current_device(&view)) return FA_ERR_LAUNCH;
  if (!view.supported) return FA_ERR_DEVICE;
  const int G = Hq / Hkv, tpt = fa::kBlockM / G;

  // the plans of all launches first, so that a workspace that is too small launches nothing
  pk::Params p;
  int begin = 0, grid = 0, n_slots = 0, n_split = 0;
  size_t need = 0;
  for (int i = 0; i < n_seqs; i += pk::kMaxSeqs) {
    const int n = std::min(pk::kMaxSeqs, n_seqs - i);
    grid = make_plan(seq_lens + i, n, begin, Hkv, tpt, causal, view.num_sms, p, n_slots, n_split);
    begin = p.cu[n];
    need = std::max(need, workspace_bytes(n_slots, n_split, d));
  }
  if (need > 0 && (workspace == nullptr || ws_bytes < need)) return FA_ERR_SCRATCH;

  CUtensorMap tq, tk, tv;
  if (!fa::encode_bf16_tokens(&tq, q, d, Hq, T, q_stride, 64, G, tpt) ||
      !fa::encode_bf16_tokens(&tk, k, d, Hkv, T, k_stride, 64, 1, fa::kBlockN) ||
      !fa::encode_bf16_tokens(&tv, v, d, Hkv, T, v_stride, 64, 1, fa::kBlockN))
    return FA_ERR_LAUNCH;
  p.o = static_cast<__nv_bfloat16*>(o);
  p.lse = lse;
  p.status = view.status;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k = static_cast<const __nv_bfloat16*>(k);
  p.v = static_cast<const __nv_bfloat16*>(v);
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.T = T;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.G = G;
  p.tpt = tpt;
  p.qk_scale = qk_scale;
  p.wait_limit_ns = fa_internal::kWaitLimitNs;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  begin = 0;
  for (int i = 0; i < n_seqs; i += pk::kMaxSeqs) {
    const int n = std::min(pk::kMaxSeqs, n_seqs - i);
    if (n_seqs > pk::kMaxSeqs)  // else p still holds the one launch's plan
      grid = make_plan(seq_lens + i, n, begin, Hkv, tpt, causal, view.num_sms, p, n_slots, n_split);
    begin = p.cu[n];
    if (grid == 0) continue;
    p.part_o = static_cast<float*>(workspace);
    p.part_lse = p.part_o + static_cast<size_t>(n_slots) * fa::kItemRows * d;
    p.counters = reinterpret_cast<int*>(p.part_lse + static_cast<size_t>(n_slots) * fa::kItemRows);
    if (n_split > 0 &&
        cudaMemsetAsync(p.counters, 0, static_cast<size_t>(n_split) * pk::kCountersPerItem * sizeof(int), s) != cudaSuccess)
      return FA_ERR_LAUNCH;
    rc = d == 128 ? (causal ? launch<128, true>(tq, tk, tv, p, grid, dev, s) : launch<128, false>(tq, tk, tv, p, grid, dev, s))
                  : (causal ? launch<64, true>(tq, tk, tv, p, grid, dev, s) : launch<64, false>(tq, tk, tv, p, grid, dev, s));
    if (rc != FA_OK) return rc;
  }
  return FA_OK;
}

}  // extern "C"
