// C ABI of rotary positions: rotating, and appending to the paged 4-bit cache.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "fa_gb300_rotary.h"
#include "fa_kv4_host.h"
#include "fa_rotary.cuh"

namespace {

namespace ro = fa::rotary;
using namespace fa_internal;

int check_turn(int d, int rot_dim, int interleaved, float magnitude) {
  if ((d != 64 && d != 128) || rot_dim < 16 || rot_dim > d || rot_dim % 16 || (interleaved != 0 && interleaved != 1) ||
      !std::isfinite(magnitude) || !(magnitude > 0.f))
    return FA_ERR_INVALID_ARG;
  return FA_OK;
}

// A tensor [B][N][H][d] with strides in elements.
struct Strided {
  const void* ptr;
  long long stride[3], count[3];  // batch, token, head
  int d;
  size_t bytes() const {
    long long e = d;
    for (int i = 0; i < 3; ++i) e += (count[i] - 1) * stride[i];
    return static_cast<size_t>(e) * 2;
  }
  bool same(const Strided& o) const {
    if (ptr != o.ptr) return false;
    for (int i = 0; i < 3; ++i)
      if (count[i] > 1 && stride[i] != o.stride[i]) return false;
    return true;
  }
  // Whether every element has a place of its own: from the smallest stride on, each passes what lies within.
  bool own_places() const {
    int order[3] = {0, 1, 2};
    std::sort(order, order + 3, [&](int a, int b) { return stride[a] < stride[b]; });
    long long within = d;
    for (int i : order) {
      if (count[i] < 2) continue;
      if (stride[i] < within) return false;
      within += (count[i] - 1) * stride[i];
    }
    return true;
  }
  // The elements that one run of them takes of every `every`, counted from ptr: dimensions whose stride is a
  // multiple of it fall on one another.
  long long run(long long every) const {
    long long e = d;
    for (int i = 0; i < 3; ++i)
      if (count[i] > 1 && stride[i] % every != 0) e += (count[i] - 1) * stride[i];
    return e;
  }
};

// Whether two tensors share an element (may say so where they interleave in ways that this does not see through).
bool share(const Strided& a, const Strided& b) {
  if (!overlaps(a.ptr, a.bytes(), b.ptr, b.bytes())) return false;
  const long long apart = static_cast<long long>(reinterpret_cast<uintptr_t>(b.ptr) - reinterpret_cast<uintptr_t>(a.ptr));
  // Apart in every period of some stride's length, as columns of the same rows are (q and k of one projection's output:
  // the token stride), or heads of the same batch entries (views of one [B, H, N, d]: the batch stride).
  for (const Strided* t : {&a, &b})
    for (int i = 0; i < 3; ++i) {
      if (t->count[i] < 2 || t->stride[i] == 0) continue;
      const long long s = t->stride[i] * 2, at = (apart % s + s) % s;  // bytes
      if (a.run(t->stride[i]) * 2 <= at && at + b.run(t->stride[i]) * 2 <= s) return false;
    }
  return true;
}

}  // namespace

extern "C" {

int fa_rotate(const void* q, const void* k, void* q_out, void* k_out, const int* positions, const long long* turns,
              int B, int N, int Hq, int Hk, int d, int rot_dim, int interleaved, float magnitude, int backward,
              const long long* strides, long long position_stride, void* stream) {
  int rc = check_turn(d, rot_dim, interleaved, magnitude);
  if (rc != FA_OK) return rc;
  if (B < 0 || B > 65535 || N < 0 || static_cast<long long>(B) * N > (1 << 30) || Hq < 1 || Hk < 0 || Hq > (1 << 16) ||
      Hk > (1 << 16) || (backward != 0 && backward != 1))
    return FA_ERR_INVALID_ARG;
  if (strides == nullptr) return FA_ERR_NULL;
  const int tensors = Hk > 0 ? 2 : 1;
  for (int i = 0; i < 12; ++i) {
    if (i / 3 % 2 >= tensors) continue;  // k's
    if (strides[i] < 0 || strides[i] % 8 || strides[i] > (1ll << 40)) return FA_ERR_INVALID_ARG;
  }
  if (position_stride < 0 || (positions && position_stride != 0 && position_stride < N) || position_stride > (1ll << 40))
    return FA_ERR_INVALID_ARG;
  if (B == 0 || N == 0) return FA_OK;
  if (!q || !q_out || !turns || (tensors == 2 && (!k || !k_out))) return FA_ERR_NULL;
  if (misaligned(q, 16) || misaligned(q_out, 16) || misaligned(turns, 8) || misaligned(positions, 4) ||
      (tensors == 2 && (misaligned(k, 16) || misaligned(k_out, 16))))
    return FA_ERR_ALIGN;
  Strided in[2], out[2];
  for (int i = 0; i < tensors; ++i) {
    const int heads = i ? Hk : Hq;
    in[i] = Strided{i ? k : q, {strides[3 * i], strides[3 * i + 1], strides[3 * i + 2]}, {B, N, heads}, d};
    out[i] = Strided{i ? k_out : q_out, {strides[6 + 3 * i], strides[7 + 3 * i], strides[8 + 3 * i]}, {B, N, heads}, d};
    if (!out[i].own_places()) return FA_ERR_INVALID_ARG;
  }
  const size_t pb = positions ? (static_cast<size_t>(B - 1) * position_stride + N) * 4 : 0, tb = static_cast<size_t>(rot_dim) * 4;
  bool in_place = true;
  for (int i = 0; i < tensors; ++i) {
    in_place = in_place && out[i].same(in[i]);
    for (int j = 0; j < tensors; ++j)
      if (!(i == j && out[i].same(in[i])) && share(out[i], in[j])) return FA_ERR_ALIAS;
    if ((positions && overlaps(out[i].ptr, out[i].bytes(), positions, pb)) || overlaps(out[i].ptr, out[i].bytes(), turns, tb))
      return FA_ERR_ALIAS;
  }
  if (tensors == 2 && share(out[0], out[1])) return FA_ERR_ALIAS;
  int dev = 0;
  DeviceView view;
  rc = current(&dev, &view);
  if (rc != FA_OK) return rc;
  ro::RotateParams p{};
  ro::View* views[2] = {&p.q, &p.k};
  for (int i = 0; i < tensors; ++i)
    *views[i] = ro::View{static_cast<const __nv_bfloat16*>(in[i].ptr), static_cast<__nv_bfloat16*>(const_cast<void*>(out[i].ptr)),
                         in[i].stride[0], in[i].stride[1], in[i].stride[2], out[i].stride[0], out[i].stride[1], out[i].stride[2]};
  p.positions = positions;
  p.turns = reinterpret_cast<const unsigned long long*>(turns);
  p.position_stride = position_stride;
  p.N = N;
  p.Hq = Hq;
  p.H = Hq + Hk;
  p.rot = rot_dim;
  p.interleaved = interleaved;
  p.copy_rest = !in_place;
  p.m = magnitude;
  p.sign = backward ? -1.f : 1.f;
  p.tokens_per_cta = std::min(ro::kMaxTokens, tokens_per_cta(static_cast<int>(static_cast<long long>(B) * N), view.num_sms));
  const dim3 grid((N + p.tokens_per_cta - 1) / p.tokens_per_cta, B);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (d == 128) ro::rotate_kernel<128><<<grid, ro::kThreads, 0, s>>>(p);
  else ro::rotate_kernel<64><<<grid, ro::kThreads, 0, s>>>(p);
  return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_LAUNCH;
}

int fa_kv4_append(const void* q, const void* k, const void* v, void* q_out, void* k_out, void* cache,
                  const int* page_table, const int* seq_lens, const int* cu_seqlens, const int* positions,
                  const long long* turns, int T, int n_seqs, int max_pages, int num_pages, int page_size, int Hq,
                  int Hkv, int d, int rot_dim, int interleaved, float magnitude, long long q_stride,
                  long long k_stride, long long v_stride, float k_scale, float v_scale, int* errors, void* stream) {
  size_t cb = 0;
  int rc = check_cache(cache, page_table, seq_lens, n_seqs, max_pages, num_pages, page_size, Hkv, d, k_scale, v_scale, &cb);
  if (rc != FA_OK) return rc;
  rc = check_turn(d, rot_dim, interleaved, magnitude);
  if (rc != FA_OK) return rc;
  const long long kv_row = static_cast<long long>(Hkv) * d, q_row = static_cast<long long>(Hq) * d;
  constexpr long long kMaxStride = 1ll << 32;
  if (T < 0 || T > (1 << 30) || Hq < 0 || Hq > (1 << 16) || k_stride < kv_row || v_stride < kv_row || k_stride % 8 ||
      v_stride % 8 || k_stride > kMaxStride || v_stride > kMaxStride ||
      (Hq > 0 && (q_stride < q_row || q_stride % 8 || q_stride > kMaxStride)))
    return FA_ERR_INVALID_ARG;
  if (T == 0 || n_seqs == 0) return FA_OK;
  if (!k || !v || !cu_seqlens || !turns || (Hq > 0 && (!q || !q_out))) return FA_ERR_NULL;
  if (Hq == 0) q = q_out = nullptr;
  if (misaligned(q, 16) || misaligned(k, 16) || misaligned(v, 16) || misaligned(q_out, 16) || misaligned(k_out, 16) ||
      misaligned(cu_seqlens, 4) || misaligned(positions, 4) || misaligned(turns, 8) || misaligned(errors, 4))
    return FA_ERR_ALIGN;
  auto extent = [&](long long stride, long long row) { return (static_cast<size_t>(T - 1) * stride + row) * 2; };
  const size_t pb = static_cast<size_t>(n_seqs) * max_pages * 4, lb = static_cast<size_t>(n_seqs) * 4;
  const void* out[4] = {cache, q_out, k_out, errors};
  const size_t out_bytes[4] = {cb, static_cast<size_t>(T) * q_row * 2, static_cast<size_t>(T) * kv_row * 2, 4};
  const void* in[8] = {q, k, v, page_table, seq_lens, cu_seqlens, positions, turns};
  const size_t in_bytes[8] = {Hq > 0 ? extent(q_stride, q_row) : 0, extent(k_stride, kv_row), extent(v_stride, kv_row), pb, lb,
                              lb + 4, static_cast<size_t>(T) * 4, static_cast<size_t>(rot_dim) * 4};
  for (int i = 0; i < 4; ++i) {
    if (out[i] == nullptr) continue;
    for (int j = 0; j < 8; ++j)
      if (in[j] && overlaps(out[i], out_bytes[i], in[j], in_bytes[j])) return FA_ERR_ALIAS;
    for (int j = i + 1; j < 4; ++j)
      if (out[j] && overlaps(out[i], out_bytes[i], out[j], out_bytes[j])) return FA_ERR_ALIAS;
  }
  int dev = 0;
  DeviceView view;
  rc = current(&dev, &view);
  if (rc != FA_OK) return rc;
  ro::AppendParams p{};
  p.m.k = static_cast<const __nv_bfloat16*>(k);
  p.m.v = static_cast<const __nv_bfloat16*>(v);
  p.m.cache = static_cast<uint8_t*>(cache);
  p.m.page_table = page_table;
  p.m.seq_lens = seq_lens;
  p.m.cu = cu_seqlens;
  p.m.errors = errors;
  p.m.k_stride = k_stride;
  p.m.v_stride = v_stride;
  p.m.T = T;
  p.m.n_seqs = n_seqs;
  p.m.max_pages = max_pages;
  p.m.num_pages = num_pages;
  p.m.page_shift = page_shift(page_size);
  p.m.Hkv = Hkv;
  p.m.k_scale = 1.f / k_scale;
  p.m.v_scale = 1.f / v_scale;
  p.m.tokens_per_cta = tokens_per_cta(T, view.num_sms);
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.q_out = static_cast<__nv_bfloat16*>(q_out);
  p.k_out = static_cast<__nv_bfloat16*>(k_out);
  p.positions = positions;
  p.turns = reinterpret_cast<const unsigned long long*>(turns);
  p.q_stride = q_stride;
  p.Hq = Hq;
  p.rot = rot_dim;
  p.interleaved = interleaved;
  p.scale = magnitude;
  const int grid = (T + p.m.tokens_per_cta - 1) / p.m.tokens_per_cta;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (d == 128) ro::append_kernel<128><<<grid, ro::kThreads, 0, s>>>(p);
  else ro::append_kernel<64><<<grid, ro::kThreads, 0, s>>>(p);
  return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_LAUNCH;
}

}  // extern "C"
