// Keeping the accepted nodes of a tree: their rows of the paged 4-bit cache move
// to the first places of the tree.
//
// A CTA takes one KV head of one sequence: all rows that move are read into
// shared memory, then written, so that a row may move onto one that moves too.
// A row of a head is 18 words of d / 16 bytes (8 of K codes, one of K scales,
// 8 of V codes, one of V scales), each contiguous, at offsets within its group
// that the format gives.  Bound by latency: lengths, the path, a page id and the
// rows are four loads one after another, 2.5 us for one sequence, 3.5 for 128
// paths of trees of 60.
#pragma once

#include "fa_kv4.cuh"

namespace fa {
namespace kv4 {

constexpr int kKeepThreads = 128;
constexpr int kKeepNodes = 64;
constexpr int kRowWords = 18;

struct KeepParams {
  uint8_t* cache;
  const int* page_table;
  const int* seq_lens;
  const int* path;      // [n_seqs][n_nodes]
  const int* n_kept;
  int* new_lens;
  int* errors;          // or null
  int n_nodes, max_pages, num_pages, page_shift, Hkv;
};

template <int D>
struct KeepWord;
template <>
struct KeepWord<64> { using Type = uint32_t; };
template <>
struct KeepWord<128> { using Type = uint2; };

// Byte offset of word w of a row within its group, the row's number aside.
template <int D>
__device__ __forceinline__ int word_at(int w, int row) {
  constexpr int kWord = D / 16;
  const int v = w >= kRowWords / 2, i = w - v * (kRowWords / 2);
  return i < 8 ? codes_at(D, v) + row * (D / 2) + i * kWord : scales_at(D, v) + row * kWord;
}

template <int D>
__global__ void __launch_bounds__(kKeepThreads) keep_kernel(const KeepParams p) {
  using Word = typename KeepWord<D>::Type;
  __shared__ Word s_rows[kKeepNodes * kRowWords];
  __shared__ long long s_from[kKeepNodes], s_to[kKeepNodes];  // offset of the group, plus the row; -1: does not move
  const int s = blockIdx.x / p.Hkv, h = blockIdx.x - s * p.Hkv;
  const long long first = static_cast<long long>(p.seq_lens[s]) - p.n_nodes;
  const int asked = p.n_kept[s], kept = min(max(asked, 0), p.n_nodes);
  const bool tells = h == 0 && p.errors != nullptr;
  if (h == 0 && threadIdx.x == 0) {
    p.new_lens[s] = static_cast<int>(max(0ll, first + kept));
    if (tells && asked != kept) atomicOr(p.errors, kErrPosition);
  }
  const long long head_bytes = static_cast<long long>(row_bytes(D)) << p.page_shift;
  auto place = [&](long long pos) -> long long {
    const long long page_at = pos >> p.page_shift;
    if (pos < 0 || page_at >= p.max_pages) {
      if (tells) atomicOr(p.errors, kErrPosition);
      return -1;
    }
    const int page = __ldg(p.page_table + static_cast<long long>(s) * p.max_pages + page_at);
    if (page < 0 || page >= p.num_pages) {
      if (tells) atomicOr(p.errors, kErrPage);
      return -1;
    }
    const int in_page = static_cast<int>(pos) & ((1 << p.page_shift) - 1);
    return (static_cast<long long>(page) * p.Hkv + h) * head_bytes + static_cast<long long>(in_page / kGroup) * group_bytes(D) +
           in_page % kGroup;
  };
  if (threadIdx.x < kept) {
    const int j = threadIdx.x, node = __ldg(p.path + static_cast<long long>(s) * p.n_nodes + j);
    long long from = -1, to = -1;
    if (node < 0 || node >= p.n_nodes) {
      if (tells) atomicOr(p.errors, kErrPosition);
    } else {
      from = place(first + node);
      to = place(first + j);
    }
    const bool moves = from >= 0 && to >= 0 && from != to;
    s_from[j] = moves ? from : -1;
    s_to[j] = to;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < kept * kRowWords; i += kKeepThreads) {
    const int j = i / kRowWords, w = i - j * kRowWords;
    const long long from = s_from[j];
    if (from < 0) continue;
    const int row = static_cast<int>(from & (kGroup - 1));
    s_rows[i] = *reinterpret_cast<const Word*>(p.cache + (from - row) + word_at<D>(w, row));
  }
  __syncthreads();
  for (int i = threadIdx.x; i < kept * kRowWords; i += kKeepThreads) {
    const int j = i / kRowWords, w = i - j * kRowWords;
    if (s_from[j] < 0) continue;
    const long long to = s_to[j];
    const int row = static_cast<int>(to & (kGroup - 1));
    *reinterpret_cast<Word*>(p.cache + (to - row) + word_at<D>(w, row)) = s_rows[i];
  }
}

}  // namespace kv4
}  // namespace fa
