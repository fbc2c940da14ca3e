// The paged 4-bit cache of keys and values: its format, and the kernels that
// store into it and load from it.
//
// Format.  BLOCK = 16 consecutive elements of one head of one token share an
// e4m3 scale s = e4m3(amax / (6 g)), 6 being e2m1's largest value and g the
// tensor's own power-of-two scale; an element's code is the e2m1 value nearest
// to x / (s g), ties to the even code, and stands for code * s * g.  A block
// with a NaN or an infinity in it gets the scale NaN (and reads back as NaN);
// where amax / (6 g) rounds to more than 448 the scale is 448 and large
// elements saturate; where it rounds to 0 the block reads back as zeros.
// Two significant bits times four fit bf16's eight and f16's eleven, so code
// * s is exact in either.
//
// A page holds page_size tokens (a power of two, 16 or more) of every KV head:
// cache[page][head][group of 16 tokens] of 18 d bytes each,
//     [K codes 16 x d/2][K scales 16 x d/16][V codes 16 x d/2][V scales 16 x d/16],
// the even element of a code byte in its low four bits.  A group is one
// contiguous piece, so that one bulk copy brings all a warp needs of it.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "sm103_ptx.cuh"

namespace fa {
namespace kv4 {

constexpr int kGroup = 16;  // tokens of a group
constexpr int kBlock = 16;  // elements that share a scale

__host__ __device__ constexpr int row_bytes(int d) { return d + d / 8; }  // one token of one head, K and V
__host__ __device__ constexpr int group_bytes(int d) { return kGroup * row_bytes(d); }
// offsets within a group
__host__ __device__ constexpr int codes_at(int d, int v) { return v * kGroup * row_bytes(d) / 2; }
__host__ __device__ constexpr int scales_at(int d, int v) { return codes_at(d, v) + kGroup * d / 2; }

// What a call's `errors` word may hold (bits).
constexpr int kErrPage = 1;      // a page id outside [0, num_pages)
constexpr int kErrPosition = 2;  // a token before position 0 or past the table's pages

// Two e4m3 values (low byte first) to f16, exact.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two) {
  uint32_t r;
  const uint16_t h = static_cast<uint16_t>(two);
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(h));
  return r;
}

// Four code bytes to eight f16 values, byte i's low code in the low half of r[i]: exact.
__device__ __forceinline__ void e2m1x8_to_f16x2(uint32_t w, uint32_t* r) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(w));
}

__device__ __forceinline__ uint32_t f16x2_mul(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Eight fp32 values to four code bytes (round to nearest even, saturating at
// 6), element 0 in the low four bits of byte 0.
__device__ __forceinline__ uint32_t pack_e2m1x8(const float* y) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]));
  return r;
}

// One block of 16 bf16 values (eight words) to eight code bytes and a scale
// byte.  inv_g = 1 / g, a power of two, so every product with it is exact.
//
// x / (s g) is taken as x * ((1 / s) / g), whose relative error is below
// 2^-22, then rounded to a multiple of 2^-13 by adding and subtracting 1.5 *
// 2^10: a quotient that is exactly halfway between two codes (all are
// multiples of 1/4) becomes exactly that again, so that ties go to the even
// code as with an exact division.  Any other quotient lies further from a
// halfway point t than that step: t s has at most seven significant bits and
// x eight, so they differ by at least 2^-8 of t, 2^-10 at the least.
__device__ __forceinline__ void quantise_block(const uint32_t* x, float inv_g, uint32_t* codes, uint32_t& scale) {
  // the largest magnitude, on bf16 pairs without their signs; an infinity or
  // NaN has the largest bit patterns, so integer maxima find it too
  uint32_t m2 = x[0] & 0x7fff7fffu;
#pragma unroll
  for (int i = 1; i < 8; ++i) m2 = __vmaxu2(m2, x[i] & 0x7fff7fffu);
  const uint32_t top = max(m2 & 0xffffu, m2 >> 16);
  if (top >= 0x7f80u) {
    scale = 0x7fu;  // NaN
    codes[0] = codes[1] = 0u;
    return;
  }
  const float amax = __uint_as_float(top << 16);
  uint16_t s2;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(s2) : "f"(0.f), "f"(__fdiv_rn(amax * inv_g, 6.f)));
  scale = s2 & 0xffu;
  const float s = __half2float(__ushort_as_half(static_cast<unsigned short>(e4m3x2_to_f16x2(scale) & 0xffffu)));
  const float r = s > 0.f ? __fdiv_rn(inv_g, s) : 0.f;
  constexpr float kMagic = 1536.f;  // 1.5 * 2^10: an fp32 sum near it is a multiple of 2^-13
  const uint64_t r2 = f2_pack(r, r), up = f2_pack(kMagic, kMagic), down = f2_pack(-kMagic, -kMagic);
  float y[16];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint64_t v = f2_pack(__uint_as_float(x[i] << 16), __uint_as_float(x[i] & 0xffff0000u));
    f2_unpack(f2_add(f2_add(f2_mul(v, r2), up), down), y[2 * i], y[2 * i + 1]);
  }
  codes[0] = pack_e2m1x8(y);
  codes[1] = pack_e2m1x8(y + 8);
}

// Eight words, read once; `ptr` 32-byte aligned.
__device__ __forceinline__ void ld_global_nc_v8(const void* ptr, uint32_t* r) {
  asm volatile("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "l"(ptr));
}

struct MoveParams {
  const __nv_bfloat16* k;  // store: [T][Hkv][D], token strides below
  const __nv_bfloat16* v;
  __nv_bfloat16* k_out;    // load: [T][Hkv][D], contiguous
  __nv_bfloat16* v_out;
  uint8_t* cache;
  const int* page_table;   // [n_seqs][max_pages]
  const int* seq_lens;     // [n_seqs]
  const int* cu;           // [n_seqs + 1]
  int* errors;             // or null
  long long k_stride, v_stride;
  int T, n_seqs, max_pages, num_pages, page_shift, Hkv;  // page_size = 1 << page_shift
  int tokens_per_cta;
  int wide;                // rows of k, v (store) or k_out, v_out (load) are 32-byte aligned
  float k_scale, v_scale;  // store: their inverses
};

constexpr int kMoveThreads = 256;
constexpr int kMaxTokensPerCta = 16;
constexpr int kCuCached = 2048;  // sequences whose cu entries a CTA keeps in shared memory

// Where token `tok` of a packed tensor lies in the cache: the byte offset of
// its group of head 0 plus its row in the low four bits, or -1 if it has no
// place (behind the last sequence, -2 where that is an error).
// cu_at(i) = cu[i].  The token's sequence is the last whose first token is
// not behind it, found by bisection.
template <class Cu>
__device__ __forceinline__ long long place_of(int tok, int D, const MoveParams& p, Cu cu_at) {
  const int n = p.n_seqs;
  if (n == 0 || tok < cu_at(0) || tok >= cu_at(n)) return -1;
  int lo = 0, hi = n;  // cu[lo] <= tok < cu[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (cu_at(mid) <= tok) lo = mid; else hi = mid;
  }
  // position: the sequence's last cu[lo+1] - cu[lo] positions
  const long long pos = static_cast<long long>(p.seq_lens[lo]) - cu_at(lo + 1) + tok;
  const long long page_at = pos >> p.page_shift;
  if (pos < 0 || page_at >= p.max_pages) {
    if (p.errors) atomicOr(p.errors, kErrPosition);
    return -2;
  }
  const int page = p.page_table[static_cast<long long>(lo) * p.max_pages + page_at];
  if (page < 0 || page >= p.num_pages) {
    if (p.errors) atomicOr(p.errors, kErrPage);
    return -2;
  }
  const int in_page = static_cast<int>(pos) & ((1 << p.page_shift) - 1);
  const long long page_bytes = (static_cast<long long>(p.Hkv) * row_bytes(D)) << p.page_shift;
  return page * page_bytes + static_cast<long long>(in_page / kGroup) * group_bytes(D) + in_page % kGroup;
}

// Places of the CTA's tokens, one thread each, the cu entries through shared memory.
__device__ __forceinline__ void find_places(int first, int count, int D, const MoveParams& p, int* s_cu,
                                            long long* s_place) {
  const bool cached = p.n_seqs < kCuCached;
  if (cached) {
    for (int i = threadIdx.x; i <= p.n_seqs; i += kMoveThreads) s_cu[i] = p.cu[i];
    __syncthreads();
  }
  if (threadIdx.x < count)
    s_place[threadIdx.x] = cached ? place_of(first + threadIdx.x, D, p, [&](int i) { return s_cu[i]; })
                                  : place_of(first + threadIdx.x, D, p, [&](int i) { return __ldg(p.cu + i); });
  __syncthreads();
}

// A thread stores one block: 32 bytes read, 8 code bytes and a scale byte
// written.  Consecutive threads take a token's blocks of one head, then the
// next token's, so that a warp writes whole runs of a group's rows.  Bound by
// the bytes: 107846 tokens of 8 heads, d = 128, 566 MB, 95 us, 6.0 TB/s (and
// loaded again 188 us in all; 203 with 16-byte accesses).
template <int D>
__global__ void __launch_bounds__(kMoveThreads) store_kernel(const MoveParams p) {
  constexpr int kBlocks = D / kBlock;
  __shared__ int s_cu[kCuCached];
  __shared__ long long s_place[kMaxTokensPerCta];
  const int first = blockIdx.x * p.tokens_per_cta;
  const int count = min(p.tokens_per_cta, p.T - first);
  find_places(first, count, D, p, s_cu, s_place);
  const int units = 2 * p.Hkv * count * kBlocks;  // [tensor][head][token][block]
  const int head_bytes = row_bytes(D) << p.page_shift;
  for (int u = threadIdx.x; u < units; u += kMoveThreads) {
    const int block = u % kBlocks;
    const int rest = u / kBlocks;
    const int i = rest % count;
    const int hv = rest / count;
    const int is_v = hv >= p.Hkv;
    const int h = is_v ? hv - p.Hkv : hv;
    const long long place = s_place[i];
    if (place < 0) continue;
    const int row = static_cast<int>(place & (kGroup - 1));
    const __nv_bfloat16* src = (is_v ? p.v + static_cast<long long>(first + i) * p.v_stride
                                     : p.k + static_cast<long long>(first + i) * p.k_stride) +
                               static_cast<long long>(h) * D + block * kBlock;
    uint32_t x[8];
    if (p.wide) {
      ld_global_nc_v8(src, x);
    } else {
      const uint4 a = __ldg(reinterpret_cast<const uint4*>(src)), b = __ldg(reinterpret_cast<const uint4*>(src) + 1);
      x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    }
    uint32_t codes[2], scale;
    quantise_block(x, is_v ? p.v_scale : p.k_scale, codes, scale);
    uint8_t* group = p.cache + (place - row) + static_cast<long long>(h) * head_bytes;
    *reinterpret_cast<uint2*>(group + codes_at(D, is_v) + row * (D / 2) + block * 8) = make_uint2(codes[0], codes[1]);
    group[scales_at(D, is_v) + row * kBlocks + block] = static_cast<uint8_t>(scale);
  }
}

// The other way: a thread reads a block's codes and scale and writes 16 bf16
// values; a token whose position or page is refused is written as zeros.
// 65536 tokens of 8 heads, d = 128, 344 MB, 59 us: 5.8 TB/s.  Several blocks
// in flight a thread, or 32 and 64 tokens a CTA, took 66 to 74 us.
template <int D>
__global__ void __launch_bounds__(kMoveThreads) load_kernel(const MoveParams p) {
  constexpr int kBlocks = D / kBlock;
  __shared__ int s_cu[kCuCached];
  __shared__ long long s_place[kMaxTokensPerCta];
  const int first = blockIdx.x * p.tokens_per_cta;
  const int count = min(p.tokens_per_cta, p.T - first);
  find_places(first, count, D, p, s_cu, s_place);
  const int units = 2 * p.Hkv * count * kBlocks;
  const int head_bytes = row_bytes(D) << p.page_shift;
  for (int u = threadIdx.x; u < units; u += kMoveThreads) {
    const int block = u % kBlocks;
    const int rest = u / kBlocks;
    const int i = rest % count;
    const int hv = rest / count;
    const int is_v = hv >= p.Hkv;
    const int h = is_v ? hv - p.Hkv : hv;
    const long long place = s_place[i];
    if (place == -1) continue;
    uint32_t out[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
    if (place >= 0) {
      const int row = static_cast<int>(place & (kGroup - 1));
      const uint8_t* group = p.cache + (place - row) + static_cast<long long>(h) * head_bytes;
      const uint2 c = *reinterpret_cast<const uint2*>(group + codes_at(D, is_v) + row * (D / 2) + block * 8);
      const uint32_t sb = group[scales_at(D, is_v) + row * kBlocks + block];
      const uint32_t s = e4m3x2_to_f16x2(sb | (sb << 8));
      uint32_t h2[8];
      e2m1x8_to_f16x2(c.x, h2);
      e2m1x8_to_f16x2(c.y, h2 + 4);
      const float g = is_v ? p.v_scale : p.k_scale;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t w = f16x2_mul(h2[e], s);
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
        out[e] = pack_bf16x2(f.x * g, f.y * g);
      }
    }
    __nv_bfloat16* dst = (is_v ? p.v_out : p.k_out) +
                         (static_cast<long long>(first + i) * p.Hkv + h) * D + block * kBlock;
    if (p.wide) {
      st_global_v8(dst, out);
    } else {
      reinterpret_cast<uint4*>(dst)[0] = make_uint4(out[0], out[1], out[2], out[3]);
      reinterpret_cast<uint4*>(dst)[1] = make_uint4(out[4], out[5], out[6], out[7]);
    }
  }
}

}  // namespace kv4
}  // namespace fa
