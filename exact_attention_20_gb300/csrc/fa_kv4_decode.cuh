// Attention of each sequence's newest tokens over the paged 4-bit cache.
//
// Query i of the Lq newest tokens of a sequence of len tokens stands at
// position len - Lq + i and sees the keys up to itself:
//
//     O = sum_j softmax_j(scale q . k_j) v_j,   L = ln sum_j exp(scale q . k_j),
//
// k_j and v_j being what the cache's codes and scales stand for.  The work is
// bound by reading 18 d bytes per 16 tokens and KV head once, so all query
// rows of a KV head (Lq tokens x G heads) are taken together, and the products
// run on the tensor core as mma.sync with keys (or d) as the 16-row dimension
// and the query rows as its 8 columns: a 128-row tcgen05 tile would be padding,
// and the operands would have to go through shared memory as 16-bit values.
// Here a lane's code bytes turn into its own operand registers:
//
// - S^T = K Q^T: A is K (16 keys x 16 of d).  Which d a k-index means is free
//   as long as K and Q agree, so lane t of a quad owns d = (D/4) t ... of its
//   two keys: whole 16-element blocks, one 16-byte load and one or two scales.
// - O^T += V^T P^T: A is V^T (16 of d x 16 keys).  Lane group g owns d =
//   (D/8) g ..., for four keys: 8 bytes and one scale each.  Codes of two keys
//   are interleaved nibble by nibble, so that one conversion gives a register
//   that pairs the keys.  P^T comes from S^T by an 8x8 transpose.
// - Codes times scales are exact in f16 (fa_kv4.cuh).  Q rows are brought to
//   [2^14, 2^15) by a power of two (exact, but for elements 2^-28 of the
//   row's largest), P = exp2(s - m) lies in [0, 2^15) with m set so that a
//   maximum gives 2^8: f16 then loses nothing above 2^-33 of the maximum.
//   P's rounding to f16 is 2^-11 relative; every sum is fp32.
//
// Work: the (sequence, KV head, row tile) items' 256-token tiles, concatenated,
// are cut into equal ranges, one per CTA, from the lengths on the device.
// Within a range each of the eight warps takes every eighth unit of 32 tokens
// through a ring of its own (bulk copies, one unit ahead of the arithmetic
// and across items), with its own online softmax; the warps' states are
// combined at the end of an item, and the parts of an item cut between CTAs
// by merge_kernel.
#pragma once

#include "fa_kv4.cuh"

namespace fa {
namespace kv4 {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kUnit = 2 * kGroup;       // tokens a warp takes at a time
constexpr int kTile = kWarps * kUnit;   // tokens of one step of a CTA
constexpr int kMinTiles = 2;            // tiles a CTA takes at least, where there are that many
constexpr float kLift = 8.f;            // log2 of P at a maximum
constexpr float kMove = 7.f;            // the reference moves on a jump above this many log2 units
constexpr float kNone = -3.0e38f;       // reference of a row without keys yet
constexpr int kSiteKv4 = 7;             // status code: a wait gave up

// An item cut by the start of a CTA's range, at its first cut: parts lie with
// CTAs c0 .. c1, the first in slot slot0, the others in slot 2 c.
struct Cut {
  int s, item, c0, c1, slot0;  // s < 0: none
};

struct DecodeParams {
  const __nv_bfloat16* q;  // [n_seqs * Lq][Hq][D], token stride q_stride
  const uint8_t* cache;
  const int* page_table;
  const int* seq_lens;
  __nv_bfloat16* o;        // [n_seqs * Lq][Hq][D]
  float* lse;              // [Hq][n_seqs * Lq]
  float* part_o;           // workspace: [2 grid][rows][D], parts' O, not normalised
  float2* part_ml;         // workspace: [2 grid][rows], (m, l) in log2 units
  Cut* cuts;               // workspace: [grid]
  int* errors;             // or null
  int* status;
  long long q_stride;
  unsigned long long wait_limit_ns;
  float qk_scale;          // scale * k_scale * log2(e)
  float v_scale;
  int n_seqs, Lq, Hq, Hkv, G;
  int row_tiles;           // row tiles of an item's Lq * G rows
  int max_pages, num_pages, page_shift;  // page_size = 1 << page_shift
  int split;               // ranges may cut items (the merge kernel follows)
};

template <int D, int NT>
struct DecodeCfg {
  static constexpr int kRows = 8 * NT;
  // O^T takes NT D / 4 registers of a lane.  Up to 64 of them, two CTAs (16
  // warps) fit an SM's registers, with Q in shared memory where it would take
  // 32 more; a CTA's ring then has two units a warp (147 KB in all, 74 KB at
  // the least in flight).
  static constexpr bool kWide = NT * D > 256;
  static constexpr int kCtasPerSm = kWide ? 1 : 2;
  static constexpr bool kSharedQ = NT * D >= 256;
  static constexpr int kStages = D == 128 && !kWide ? 2 : 4;
  static constexpr int kPad = 8;  // floats, so that rows of the combine buffer start in other banks
  static constexpr int kUnitBytes = 2 * group_bytes(D);
  static constexpr int kRingBytes = kWarps * kStages * kUnitBytes;
  static constexpr int kCombineAt = kRingBytes;                              // [warp][8 rows][D + pad] fp32
  static constexpr int kMlAt = kCombineAt + kWarps * 8 * (D + kPad) * 4;     // [warp][rows] (m, l)
  static constexpr int kQAt = kMlAt + kWarps * kRows * 8;                    // [NT][D / 16][lane] two words, then factors
  static constexpr int kBarAt = kQAt + (kSharedQ ? NT * (D / 16) * 32 * 8 + kRows * 4 : 0);
  static constexpr int kSmemBytes = kBarAt + kWarps * kStages * 8;
};

// The items' tiles: a sequence has ceil(len / 256), one at least (so that
// every output row has an item to write it).
__device__ __forceinline__ int tokens_of(int s, const DecodeParams& p) {
  const long long most = min(static_cast<long long>(p.max_pages) << p.page_shift, 0x7fffff00ll);
  return max(0, static_cast<int>(min(static_cast<long long>(p.seq_lens[s]), most)));
}
__device__ __forceinline__ int tiles_of(int len) { return max(1, (len + kTile - 1) / kTile); }

// Exclusive scan of one value per thread over the block, and the total.
__device__ __forceinline__ long long block_scan(long long v, long long* s_sums, long long& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long x = v;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, off);
    if (lane >= off) x += y;
  }
  if (lane == 31) s_sums[warp] = x;
  __syncthreads();
  long long before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += s_sums[w];
    total += s_sums[w];
  }
  return before + x - v;
}

// The sequences' tiles, counted for one item of each: this thread's sequences
// [lo, hi) with their sum, the sum before them, and the total.
struct Scan {
  long long mine, before, total;
  int lo, hi;
  __device__ __forceinline__ Scan(const DecodeParams& p, long long* s_sums) {
    const int per = (p.n_seqs + kThreads - 1) / kThreads;
    lo = min(static_cast<int>(threadIdx.x) * per, p.n_seqs);
    hi = min(lo + per, p.n_seqs);
    mine = 0;
    for (int s = lo; s < hi; ++s) mine += tiles_of(tokens_of(s, p));
    before = block_scan(mine, s_sums, total);
  }
};

// A CTA's place in the concatenated items: the segment (tiles of one item) it
// is at.  Only changed between segments.
struct Walk {
  int s, item;        // sequence, item within it (head * row_tiles + row tile)
  int len, tiles;     // the sequence's
  int t0, count;      // the segment's tiles: [t0, t0 + count)
  int left;           // tiles from t0 to the end of the CTA's range; 0: done
  __device__ __forceinline__ void set() { count = min(tiles - t0, left); }
  __device__ __forceinline__ void next(const DecodeParams& p) {
    left -= count;
    t0 = 0;
    if (left <= 0) return;
    if (++item == p.Hkv * p.row_tiles) {
      item = 0;
      ++s;
      len = tokens_of(s, p);
      tiles = tiles_of(len);
    }
    set();
  }
  // the segment's units of 32 tokens: [first, end)
  __device__ __forceinline__ int first_unit() const { return t0 * kWarps; }
  __device__ __forceinline__ int end_unit() const { return min((t0 + count) * kWarps, (len + kUnit - 1) / kUnit); }
};

__device__ __forceinline__ void mma_f16(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 8x8 transpose of 16-bit values across a warp.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Query rows to f16 fragments: lane (g, t) of row tile nt holds row 8 nt + g,
// d = (D/4) t ..., step i the elements 4i .. 4i+3 of those in two words; and
// each row's factor from a product of S^T to log2 units.
template <int D>
__device__ __forceinline__ void load_q_rows(int nt, int row_tile0, const Walk& w, const DecodeParams& p,
                                            uint32_t (*q)[2], float& factor) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int h = w.item / p.row_tiles;
  const int r = row_tile0 + nt * 8 + g;
  uint4 x[D / 32];
  const int i = r / p.G;
  const __nv_bfloat16* src = p.q + (static_cast<long long>(w.s) * p.Lq + i) * p.q_stride +
                             static_cast<long long>(h * p.G + r - i * p.G) * D + t * (D / 4);
#pragma unroll
  for (int n = 0; n < D / 32; ++n)
    x[n] = r < p.Lq * p.G ? __ldg(reinterpret_cast<const uint4*>(src) + n) : make_uint4(0, 0, 0, 0);
  uint32_t m2 = 0;
#pragma unroll
  for (int n = 0; n < D / 32; ++n) {
    m2 = __vmaxu2(m2, __vmaxu2(x[n].x & 0x7fff7fffu, x[n].y & 0x7fff7fffu));
    m2 = __vmaxu2(m2, __vmaxu2(x[n].z & 0x7fff7fffu, x[n].w & 0x7fff7fffu));
  }
  uint32_t top = max(m2 & 0xffffu, m2 >> 16);
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
  const int e = max(static_cast<int>(top >> 7) - 127, -100);  // floor(log2) of the row's largest element
  const float up = __uint_as_float(static_cast<uint32_t>(127 + 14 - e) << 23);
  factor = __uint_as_float(static_cast<uint32_t>(127 - 14 + e) << 23) * p.qk_scale;
#pragma unroll
  for (int n = 0; n < D / 32; ++n) {
    const uint32_t wds[4] = {x[n].x, x[n].y, x[n].z, x[n].w};
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int pair = n * 4 + c;  // d pair within the lane's D/4
      q[pair / 2][pair & 1] = pack_f16x2(__uint_as_float(wds[c] << 16) * up, __uint_as_float(wds[c] & 0xffff0000u) * up);
    }
  }
}

// One warp's state over the units it took of one item.
template <int D, int NT>
struct State {
  static constexpr bool kSharedQ = DecodeCfg<D, NT>::kSharedQ;
  float acc[NT][D / 16][4];  // O^T: d = (D/8) g + 2j (+1: elements 2, 3), rows 2t (+1: elements 1, 3)
  float m[NT][2], l[NT][2];  // rows 2t, 2t+1; l: this lane's keys only
  float f[NT][2];            // a product of S^T to log2 units, for rows 2t and 2t+1
  uint32_t q[kSharedQ ? 1 : NT][D / 16][2];
  const uint2* q_shared;     // this lane's words in shared memory, steps and row tiles 32 apart

  __device__ __forceinline__ void reset() {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int j = 0; j < D / 16; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[nt][j][e] = 0.f;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        m[nt][e] = kNone;
        l[nt][e] = 0.f;
      }
    }
  }

  // The item's query rows.  With Q in shared memory the whole CTA calls this
  // at the same point, after a barrier behind the last use of the item before.
  __device__ __forceinline__ void load_q(const Walk& w, const DecodeParams& p, uint8_t* smem) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, t = lane & 3;
    const int row0 = w.item % p.row_tiles * 8 * NT;
    if constexpr (kSharedQ) {
      uint2* words = reinterpret_cast<uint2*>(smem + DecodeCfg<D, NT>::kQAt);
      float* factors = reinterpret_cast<float*>(words + NT * (D / 16) * 32);
      if (warp < NT) {
        uint32_t x[D / 16][2];
        float factor;
        load_q_rows<D>(warp, row0, w, p, x, factor);
#pragma unroll
        for (int i = 0; i < D / 16; ++i) words[(warp * (D / 16) + i) * 32 + lane] = make_uint2(x[i][0], x[i][1]);
        if (t == 0) factors[warp * 8 + (lane >> 2)] = factor;
      }
      __syncthreads();
      q_shared = words + lane;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        f[nt][0] = factors[nt * 8 + 2 * t];
        f[nt][1] = factors[nt * 8 + 2 * t + 1];
      }
    } else {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float factor;
        load_q_rows<D>(nt, row0, w, p, q[nt], factor);
        f[nt][0] = __shfl_sync(0xffffffffu, factor, 8 * t);  // lanes 4 r hold row r's
        f[nt][1] = __shfl_sync(0xffffffffu, factor, 8 * t + 4);
      }
    }
  }

  // S^T of one group of 16 keys at `st`.  Row g of a product is key
  // (g >> 1) + 4 (g & 1), row g + 8 that plus 8: then a lane's four keys of the
  // second product are t, t + 4, t + 8, t + 12, and the four lanes of a quad
  // read four neighbouring rows.
  __device__ __forceinline__ void scores(const uint8_t* st, float (*c)[4]) const {
    constexpr int kHalf = D / 2, kBlocks = D / 16;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int key = (g >> 1) + 4 * (g & 1);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) c[nt][e] = 0.f;
    uint32_t wa[D / 32], wb[D / 32], sa, sb;
    const uint8_t* ka = st + codes_at(D, 0) + key * kHalf + t * (D / 8);
    const uint8_t* sc = st + scales_at(D, 0) + key * kBlocks + t * (kBlocks / 4);
    if constexpr (D == 128) {
      const uint4 a = *reinterpret_cast<const uint4*>(ka), b = *reinterpret_cast<const uint4*>(ka + 8 * kHalf);
      wa[0] = a.x, wa[1] = a.y, wa[2] = a.z, wa[3] = a.w;
      wb[0] = b.x, wb[1] = b.y, wb[2] = b.z, wb[3] = b.w;
      sa = *reinterpret_cast<const uint16_t*>(sc);
      sb = *reinterpret_cast<const uint16_t*>(sc + 8 * kBlocks);
    } else {
      const uint2 a = *reinterpret_cast<const uint2*>(ka), b = *reinterpret_cast<const uint2*>(ka + 8 * kHalf);
      wa[0] = a.x, wa[1] = a.y;
      wb[0] = b.x, wb[1] = b.y;
      sa = sc[0];
      sb = sc[8 * kBlocks];
    }
    const uint32_t ha = e4m3x2_to_f16x2(sa), hb = e4m3x2_to_f16x2(sb);
#pragma unroll
    for (int n = 0; n < D / 32; ++n) {  // a word: eight elements of d, two steps
      const uint32_t da = __byte_perm(ha, 0, n < 2 ? 0x1010 : 0x3232), db = __byte_perm(hb, 0, n < 2 ? 0x1010 : 0x3232);
      uint32_t xa[4], xb[4];
      e2m1x8_to_f16x2(wa[n], xa);
      e2m1x8_to_f16x2(wb[n], xb);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        xa[i] = f16x2_mul(xa[i], da);
        xb[i] = f16x2_mul(xb[i], db);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          uint32_t q0, q1;
          if constexpr (kSharedQ) {
            const uint2 x = q_shared[(nt * (D / 16) + 2 * n + i) * 32];
            q0 = x.x, q1 = x.y;
          } else {
            q0 = q[nt][2 * n + i][0], q1 = q[nt][2 * n + i][1];
          }
          mma_f16(c[nt], xa[2 * i], xb[2 * i], xa[2 * i + 1], xb[2 * i + 1], q0, q1);
        }
    }
  }

  // O^T += V^T P^T of one group.  tail: keys from `valid` on (counted within
  // the group) lie past the sequence's end, and what is there may be NaN,
  // which 0 * NaN would spread.
  __device__ __forceinline__ void values(const uint8_t* st, const uint32_t* b0, const uint32_t* b1, bool tail, int pos,
                                         const Walk& w, const DecodeParams& p) {
    constexpr int kHalf = D / 2, kBlocks = D / 16;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const uint8_t* va = st + codes_at(D, 1) + t * kHalf + g * (D / 16);
    const uint8_t* sc = st + scales_at(D, 1) + t * kBlocks + (D == 128 ? g : g >> 1);
    uint32_t s[4];
#pragma unroll
    for (int n = 0; n < 4; ++n) s[n] = sc[4 * n * kBlocks];
    if (tail) {
      uint32_t nan = 0;  // bit n: this lane's block of key t + 4n is NaN
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        if (pos + t + 4 * n >= w.len) s[n] = 0u;
        nan |= ((s[n] & 0x7fu) == 0x7fu ? 1u : 0u) << n;
      }
      if (__any_sync(0xffffffffu, nan != 0)) {
        // such a key must not reach the rows that do not see it: it is left
        // out of the product, and its block set to NaN in the others
        const int row0 = w.item % p.row_tiles * 8 * NT;
#pragma unroll 1
        for (int k = 0; k < kGroup; ++k) {
          if (!((__shfl_sync(0xffffffffu, nan, (lane & ~3) | (k & 3)) >> (k >> 2)) & 1u)) continue;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int r = min(row0 + nt * 8 + 2 * t + e, p.Lq * p.G - 1);
              if (pos + k > w.len - p.Lq + r / p.G) continue;
#pragma unroll
              for (int j = 0; j < D / 16; ++j) acc[nt][j][e] = acc[nt][j][2 + e] = __uint_as_float(0x7fffffffu);
            }
        }
#pragma unroll
        for (int n = 0; n < 4; ++n)
          if ((nan >> n) & 1u) s[n] = 0u;
      }
    }
    const uint32_t s01 = e4m3x2_to_f16x2(s[0] | (s[1] << 8)), s23 = e4m3x2_to_f16x2(s[2] | (s[3] << 8));
    constexpr int kWords = D / 64;  // words of codes of a lane and key
    uint32_t w4[4][kWords];
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      if constexpr (D == 128) {
        const uint2 x = *reinterpret_cast<const uint2*>(va + 4 * n * kHalf);
        w4[n][0] = x.x;
        w4[n][kWords - 1] = x.y;
      } else {
        w4[n][0] = *reinterpret_cast<const uint32_t*>(va + 4 * n * kHalf);
      }
    }
#pragma unroll
    for (int x = 0; x < kWords; ++x) {
      constexpr uint32_t kLow = 0x0f0f0f0fu;
      uint32_t lo01[4], hi01[4], lo23[4], hi23[4];
      e2m1x8_to_f16x2((w4[0][x] & kLow) | ((w4[1][x] << 4) & ~kLow), lo01);
      e2m1x8_to_f16x2(((w4[0][x] >> 4) & kLow) | (w4[1][x] & ~kLow), hi01);
      e2m1x8_to_f16x2((w4[2][x] & kLow) | ((w4[3][x] << 4) & ~kLow), lo23);
      e2m1x8_to_f16x2(((w4[2][x] >> 4) & kLow) | (w4[3][x] & ~kLow), hi23);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t a0 = f16x2_mul(lo01[i], s01), a1 = f16x2_mul(hi01[i], s01);
        const uint32_t a2 = f16x2_mul(lo23[i], s23), a3 = f16x2_mul(hi23[i], s23);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma_f16(acc[nt][4 * x + i], a0, a1, a2, a3, b0[nt], b1[nt]);
      }
    }
  }

  // A unit of 32 tokens, two groups at `st`: together, so that one's products
  // overlap the other's softmax, where the registers allow.
  __device__ __forceinline__ void unit(const uint8_t* st, int pos, bool tail, uint32_t skip, const Walk& w,
                                       const DecodeParams& p) {
    if constexpr (NT * D < 256) {
      groups<2>(st, pos, tail, skip, w, p);
    } else {
#pragma unroll 1
      for (int n = 0; n < 2; ++n) groups<1>(st + n * group_bytes(D), pos + n * kGroup, tail, skip >> n, w, p);
    }
  }

  // NG groups at `st`, the first token at position `pos`.  skip: bit n set
  // where group n is not to be looked at (its page was refused, or it lies
  // past the sequence).  tail: some keys may be past some row's own position.
  template <int NG>
  __device__ __forceinline__ void groups(const uint8_t* st, int pos, bool tail, uint32_t skip, const Walk& w,
                                         const DecodeParams& p) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int key = (g >> 1) + 4 * (g & 1);
    float c[NG][NT][4];
#pragma unroll
    for (int n = 0; n < NG; ++n) scores(st + n * group_bytes(D), c[n]);
    if (tail || skip != 0) {
      const int row0 = w.item % p.row_tiles * 8 * NT;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          // a row past the item's last is as its last
          const int r = min(row0 + nt * 8 + 2 * t + e, p.Lq * p.G - 1);
          const int last = w.len - p.Lq + r / p.G;  // the row's own position
#pragma unroll
          for (int n = 0; n < NG; ++n) {
            if (((skip >> n) & 1u) || pos + n * kGroup + key > last) c[n][nt][e] = -INFINITY;
            if (((skip >> n) & 1u) || pos + n * kGroup + key + 8 > last) c[n][nt][2 + e] = -INFINITY;
          }
        }
    }
    // log2 of P: the score in log2 units less the reference, which moves only
    // where one exceeds it by more than kMove + kLift
    bool move = false;
    float x[NG][NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int n = 0; n < NG; ++n) {
          x[n][nt][e] = fmaf(c[n][nt][e], f[nt][e], -m[nt][e]);
          x[n][nt][2 + e] = fmaf(c[n][nt][2 + e], f[nt][e], -m[nt][e]);
        }
        float top = fmaxf(x[0][nt][e], x[0][nt][2 + e]);
        if constexpr (NG == 2) top = fmax3(top, x[1][nt][e], x[1][nt][2 + e]);
        move |= top > kLift + kMove;
      }
    if (__any_sync(0xffffffffu, move)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float mx = fmaxf(c[0][nt][e], c[0][nt][2 + e]);
          if constexpr (NG == 2) mx = fmax3(mx, c[1][nt][e], c[1][nt][2 + e]);
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
          const float to = fmaxf(m[nt][e], mx * f[nt][e] - kLift);  // f > 0: the maximum commutes with it
          const float alpha = to == m[nt][e] ? 1.f : ex2_approx(m[nt][e] - to);  // 0 from kNone
          m[nt][e] = to;
          l[nt][e] *= alpha;
#pragma unroll
          for (int j = 0; j < D / 16; ++j) {
            acc[nt][j][e] *= alpha;
            acc[nt][j][2 + e] *= alpha;
          }
#pragma unroll
          for (int n = 0; n < NG; ++n) {
            x[n][nt][e] = fmaf(c[n][nt][e], f[nt][e], -to);
            x[n][nt][2 + e] = fmaf(c[n][nt][2 + e], f[nt][e], -to);
          }
        }
    }
#pragma unroll
    for (int n = 0; n < NG; ++n) {
      uint32_t b0[NT], b1[NT];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float p0 = ex2_approx(x[n][nt][0]), p1 = ex2_approx(x[n][nt][1]);
        const float p2 = ex2_approx(x[n][nt][2]), p3 = ex2_approx(x[n][nt][3]);
        l[nt][0] += p0 + p2;
        l[nt][1] += p1 + p3;
        b0[nt] = transpose8x8(pack_f16x2(p0, p1));
        b1[nt] = transpose8x8(pack_f16x2(p2, p3));
      }
      if ((skip >> n) & 1u) continue;  // a skipped group's bytes are not a group's
      values(st + n * group_bytes(D), b0, b1, tail, pos + n * kGroup, w, p);
    }
  }
};

// Row r (within the item's row tile) of item w: its place in O and LSE.
struct RowPlace {
  bool store;
  long long token;
  int head;
};
__device__ __forceinline__ RowPlace row_place(int s, int item, int r_in_tile, int rows, const DecodeParams& p) {
  const int h = item / p.row_tiles, rt = item - h * p.row_tiles;
  const int r = rt * rows + r_in_tile;
  const int i = r / p.G;
  return RowPlace{r < p.Lq * p.G, static_cast<long long>(s) * p.Lq + i, h * p.G + r - i * p.G};
}

// O = O_acc v_scale / l as bf16 and L = (m + log2 l) ln 2 of four elements of a row.
__device__ __forceinline__ void write_row(const RowPlace& rp, int D, int d4, float4 O, float M, float L,
                                          const DecodeParams& p) {
  const float inv = L == 0.f ? 0.f : p.v_scale / L;
  *reinterpret_cast<uint2*>(p.o + (rp.token * p.Hq + rp.head) * D + d4) =
      make_uint2(pack_bf16x2(O.x * inv, O.y * inv), pack_bf16x2(O.z * inv, O.w * inv));
  if (d4 == 0)
    p.lse[static_cast<long long>(rp.head) * p.n_seqs * p.Lq + rp.token] = (M + log2f(L)) * 0.69314718055994531f;
}

template <int D, int NT>
__global__ void __launch_bounds__(kThreads, DecodeCfg<D, NT>::kCtasPerSm) decode_kernel(const DecodeParams p) {
  using C = DecodeCfg<D, NT>;
  constexpr int kRows = C::kRows;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ long long s_sums[kWarps];
  __shared__ Walk s_walk;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint8_t* ring = smem + warp * C::kStages * C::kUnitBytes;
  const uint32_t ring_u32 = smem_u32(ring);
  const uint32_t bar0 = smem_u32(smem + C::kBarAt) + warp * C::kStages * 8;
  if (lane == 0) {
    for (int st = 0; st < C::kStages; ++st) mbar_init(bar0 + 8 * st, 1);
    fence_barrier_init();
  }

  // This CTA's range of the concatenated items' tiles.
  const int items = p.Hkv * p.row_tiles;  // of a sequence
  if (p.split) {
    const Scan sc(p, s_sums);
    const long long all = sc.total * items;
    const long long ctas = min(static_cast<long long>(gridDim.x), (all + kMinTiles - 1) / kMinTiles);
    const long long c = blockIdx.x;
    const long long begin = c < ctas ? all * c / ctas : all;
    const long long end = c < ctas ? all * (c + 1) / ctas : all;
    if (threadIdx.x == 0) {
      s_walk.left = 0;
      p.cuts[c].s = -1;
    }
    __syncthreads();
    // the thread whose sequences hold tile `begin`
    if (begin < end && begin >= sc.before * items && begin < (sc.before + sc.mine) * items) {
      long long at = sc.before * items;
      for (int s = sc.lo; s < sc.hi; ++s) {
        const int len = tokens_of(s, p), n = tiles_of(len);
        if (begin < at + static_cast<long long>(n) * items) {
          const int item = static_cast<int>((begin - at) / n);
          const long long a = at + static_cast<long long>(item) * n;  // the item's first tile
          Walk w{s, item, len, n, static_cast<int>(begin - a), 0, static_cast<int>(min(end - begin, 0x7fffffffll))};
          w.set();
          s_walk = w;
          const long long prev = all * (c - 1) / ctas;  // where the range before this one starts
          if (begin > a && prev <= a) {  // the item's first cut
            long long c1 = c;
            while (all * (c1 + 1) / ctas < a + n) ++c1;
            p.cuts[c] = Cut{s, item, static_cast<int>(c - 1), static_cast<int>(c1),
                            static_cast<int>(2 * (c - 1) + (prev == a ? 0 : 1))};
          }
          break;
        }
        at += static_cast<long long>(n) * items;
      }
    }
  } else if (threadIdx.x == 0) {
    // short items: CTA i takes item i whole
    const int s = blockIdx.x / items, len = tokens_of(s, p), n = tiles_of(len);
    s_walk = Walk{s, static_cast<int>(blockIdx.x) - s * items, len, n, 0, n, n};
  }
  __syncthreads();
  Walk w = s_walk;
  if (p.errors && blockIdx.x == 0) {
    for (int s = threadIdx.x; s < p.n_seqs; s += kThreads)
      if (p.seq_lens[s] != tokens_of(s, p)) atomicOr(p.errors, kErrPosition);
  }

  // The load cursor runs ahead of the arithmetic, through the same units; the
  // page ids of the unit it is at are already on their way.
  Walk lw = w;
  int lu = 0, l_end = 0;        // the next unit to load, the end of its segment
  const int* l_table = nullptr;
  long long l_head = 0;         // the item's KV head within a page, in bytes
  int page0 = -1, page1 = -1;   // its groups' pages
  const int group_shift = p.page_shift - 4;  // log2 of a page's groups
  const int group_mask = (1 << group_shift) - 1;
  const long long page_bytes = (static_cast<long long>(row_bytes(D)) << p.page_shift) * p.Hkv;
  auto enter = [&]() {  // to the first segment from lw on that has a unit for this warp
    while (lw.left > 0) {
      lu = lw.first_unit() + warp;
      l_end = lw.end_unit();
      if (lu < l_end) {
        l_table = p.page_table + static_cast<long long>(lw.s) * p.max_pages;
        l_head = (static_cast<long long>(row_bytes(D)) << p.page_shift) * (lw.item / p.row_tiles);
        return;
      }
      lw.next(p);
    }
  };
  auto look_up = [&]() {  // the unit's pages; its second group may lie past the sequence's last page
    if (lw.left <= 0) return;
    page0 = __ldg(l_table + (2 * lu >> group_shift));
    page1 = page0;
    if (group_shift == 0) page1 = (2 * lu + 1) * kGroup < lw.len ? __ldg(l_table + 2 * lu + 1) : -2;
  };
  enter();
  look_up();
  uint32_t loads = 0;  // units asked for
  uint32_t skips = 0;  // two bits per stage: groups that were not loaded
  auto issue = [&]() {
    if (lw.left <= 0) return;
    const uint32_t st = loads % C::kStages, dst = ring_u32 + st * C::kUnitBytes, bar = bar0 + 8 * st;
    const bool ok0 = static_cast<uint32_t>(page0) < static_cast<uint32_t>(p.num_pages);
    const bool ok1 = static_cast<uint32_t>(page1) < static_cast<uint32_t>(p.num_pages);
    skips = (skips & ~(3u << (2 * st))) | ((ok0 ? 0u : 1u) | (ok1 ? 0u : 2u)) << (2 * st);
    if (lane == 0) {
      const uint8_t* src = p.cache + page0 * page_bytes + l_head + (2 * lu & group_mask) * group_bytes(D);
      if (group_shift > 0) {  // both groups lie together
        if (ok0) {
          mbar_arrive_expect_tx(bar, C::kUnitBytes);
          bulk_load(dst, src, C::kUnitBytes, bar);
        } else {
          mbar_arrive(bar);
        }
      } else {
        mbar_arrive_expect_tx(bar, ((ok0 ? 1 : 0) + (ok1 ? 1 : 0)) * group_bytes(D));
        if (ok0) bulk_load(dst, src, group_bytes(D), bar);
        if (ok1) bulk_load(dst + group_bytes(D), p.cache + page1 * page_bytes + l_head, group_bytes(D), bar);
      }
      if (p.errors && (!ok0 || (!ok1 && page1 != -2))) atomicOr(p.errors, kErrPage);
    }
    ++loads;
    lu += kWarps;
    if (lu >= l_end) {
      lw.next(p);
      enter();
    }
    look_up();
  };
#pragma unroll 1
  for (int i = 0; i < C::kStages; ++i) issue();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  float* comb = reinterpret_cast<float*>(smem + C::kCombineAt);
  float2* s_ml = reinterpret_cast<float2*>(smem + C::kMlAt);
  uint32_t used = 0;  // units taken from the ring
  bool dead = false;  // a wait gave up
  int slot = 2 * blockIdx.x;
  State<D, NT> state;
  for (; w.left > 0; w.next(p), slot = 2 * blockIdx.x + 1) {
    state.reset();
    state.load_q(w, p, smem);
    const int end = w.end_unit();
    const int tail_from = w.len - p.Lq + 1;  // a unit that reaches past it is masked
    for (int u = w.first_unit() + warp; u < end && !dead; u += kWarps) {
      const uint32_t st = used % C::kStages;
      if (!__all_sync(0xffffffffu, mbar_wait_bounded(bar0 + 8 * st, (used / C::kStages) & 1, p.wait_limit_ns))) {
        dead = true;
        if (lane == 0) atomicCAS(p.status, 0, kSiteKv4);
        break;
      }
      state.unit(ring + st * C::kUnitBytes, u * kUnit, (u + 1) * kUnit > tail_from, (skips >> (2 * st)) & 3u, w, p);
      __syncwarp();  // every lane has read the stage
      ++used;
      issue();
    }
    // The warps' states: M = max m_w, O = sum O_w 2^(m_w - M), l likewise (a
    // warp without keys has m = kNone, l = 0 and O = 0).
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float l = state.l[nt][e];
        l += __shfl_xor_sync(0xffffffffu, l, 4);
        l += __shfl_xor_sync(0xffffffffu, l, 8);
        l += __shfl_xor_sync(0xffffffffu, l, 16);
        if (g == 0) s_ml[warp * kRows + nt * 8 + 2 * t + e] = make_float2(state.m[nt][e], l);
      }
    const bool whole = w.count == w.tiles;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int j = 0; j < D / 16; ++j) {
        float* dst = comb + (warp * 8 + 2 * t) * (D + C::kPad) + (D / 8) * g + 2 * j;
        *reinterpret_cast<float2*>(dst) = make_float2(state.acc[nt][j][0], state.acc[nt][j][2]);
        *reinterpret_cast<float2*>(dst + D + C::kPad) = make_float2(state.acc[nt][j][1], state.acc[nt][j][3]);
      }
      __syncthreads();
#pragma unroll 1
      for (int idx = threadIdx.x; idx < 8 * D / 4; idx += kThreads) {
        const int r = idx / (D / 4), d4 = idx % (D / 4) * 4;
        float M = kNone;
#pragma unroll
        for (int x = 0; x < kWarps; ++x) M = fmaxf(M, s_ml[x * kRows + nt * 8 + r].x);
        float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
        float L = 0.f;
#pragma unroll
        for (int x = 0; x < kWarps; ++x) {
          const float2 ml = s_ml[x * kRows + nt * 8 + r];
          const float f = exp2f(ml.x - M);
          const float4 a = *reinterpret_cast<const float4*>(comb + (x * 8 + r) * (D + C::kPad) + d4);
          L = fmaf(ml.y, f, L);
          O.x = fmaf(a.x, f, O.x);
          O.y = fmaf(a.y, f, O.y);
          O.z = fmaf(a.z, f, O.z);
          O.w = fmaf(a.w, f, O.w);
        }
        if (whole) {
          const RowPlace rp = row_place(w.s, w.item, nt * 8 + r, kRows, p);
          if (rp.store) write_row(rp, D, d4, O, M, L, p);
        } else {
          const long long row = static_cast<long long>(slot) * kRows + nt * 8 + r;
          *reinterpret_cast<float4*>(p.part_o + row * D + d4) = O;
          if (d4 == 0) p.part_ml[row] = make_float2(M, L);
        }
      }
      __syncthreads();
    }
  }
  // Copies still in flight land before the CTA exits (only after a wait gave up).
  for (; used < loads; ++used) mbar_wait_bounded(bar0 + 8 * (used % C::kStages), (used / C::kStages) & 1, p.wait_limit_ns);
}

constexpr int kMergeRows = 2;  // rows of a CTA of merge_kernel

// Block (c, y): rows 2y, 2y+1 of the item that the start of CTA c's range cuts
// first, if it does: its parts' states are merged as the warps' were.  D / 4
// threads take a row's part, several parts side by side.
template <int D>
__global__ void __launch_bounds__(kThreads) merge_kernel(const DecodeParams p, int rows) {
  constexpr int kLanes = D / 4;                               // threads of one row
  constexpr int kSide = kThreads / (kMergeRows * kLanes);     // parts side by side
  __shared__ float4 s_o[kSide][kMergeRows][kLanes];
  __shared__ float2 s_ml[kSide][kMergeRows];
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the kernel before has finished and its writes are here
  const Cut cut = p.cuts[blockIdx.x];
  if (cut.s < 0) return;
  const int lane = threadIdx.x % kLanes, rr = threadIdx.x / kLanes % kMergeRows, side = threadIdx.x / (kLanes * kMergeRows);
  const int r = blockIdx.y * kMergeRows + rr;
  auto row_of = [&](int c) { return static_cast<long long>(c == cut.c0 ? cut.slot0 : 2 * c) * rows + r; };
  float M = kNone, L = 0.f;
  float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
  constexpr int kAhead = 4;  // parts loaded together
  for (int c = cut.c0 + side; c <= cut.c1; c += kSide * kAhead) {
    float2 ml[kAhead];
    float4 o[kAhead];
#pragma unroll
    for (int n = 0; n < kAhead; ++n) {
      const int x = c + n * kSide;
      ml[n] = x <= cut.c1 ? p.part_ml[row_of(x)] : make_float2(kNone, 0.f);
      o[n] = x <= cut.c1 ? *reinterpret_cast<const float4*>(p.part_o + row_of(x) * D + lane * 4) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    float to = M;
#pragma unroll
    for (int n = 0; n < kAhead; ++n) to = fmaxf(to, ml[n].x);
    const float a = exp2f(M - to);
    M = to;
    L *= a;
    O = make_float4(O.x * a, O.y * a, O.z * a, O.w * a);
#pragma unroll
    for (int n = 0; n < kAhead; ++n) {
      const float f = exp2f(ml[n].x - M);
      L = fmaf(ml[n].y, f, L);
      O = make_float4(fmaf(o[n].x, f, O.x), fmaf(o[n].y, f, O.y), fmaf(o[n].z, f, O.z), fmaf(o[n].w, f, O.w));
    }
  }
  s_o[side][rr][lane] = O;
  if (lane == 0) s_ml[side][rr] = make_float2(M, L);
  __syncthreads();
  if (side > 0) return;
  float to = kNone;
#pragma unroll
  for (int n = 0; n < kSide; ++n) to = fmaxf(to, s_ml[n][rr].x);
  L = 0.f;
  O = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int n = 0; n < kSide; ++n) {
    const float f = exp2f(s_ml[n][rr].x - to);
    const float4 o = s_o[n][rr][lane];
    L = fmaf(s_ml[n][rr].y, f, L);
    O = make_float4(fmaf(o.x, f, O.x), fmaf(o.y, f, O.y), fmaf(o.z, f, O.z), fmaf(o.w, f, O.w));
  }
  const RowPlace rp = row_place(cut.s, cut.item, r, rows, p);
  if (rp.store) write_row(rp, D, lane * 4, O, to, L, p);
}

}  // namespace kv4
}  // namespace fa
