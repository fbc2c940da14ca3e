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
// Work: the (sequence, KV head, row tile) items' units of 32 tokens,
// concatenated, are cut into ranges of equal cost, one per CTA, and a CTA's
// range into one per warp, from the lengths on the device.  A warp goes through
// its range alone, with a ring of its own (bulk copies, two units ahead of the
// arithmetic and across items) and an online softmax per item: an item that
// lies within the range it writes itself.  Only the range's first and last
// items may be shared; their states are combined once, at the CTA's end, and
// what an item has in several CTAs by merge_kernel.
//
// Measured on a GB300 (8 KV heads of 4 query heads, d = 128): 96 contexts of
// 350 to 16000 tokens, 403 MB of cache, 79 us (59 at the copy rate); one of
// 131072, 151 MB, 39 us (22).  About 219 instructions a group of 16 tokens
// leave issue slots 60 % used; of a call's time 3 us go to finding the
// ranges, 4 to the first loads, 3 to the combination and 4 to the merge, and
// CTAs with equal ranges end up to a quarter of the loop apart.
#pragma once

#include "fa_kv4.cuh"

namespace fa {
namespace kv4 {

constexpr int kMaxWarps = 16;
constexpr int kUnit = 2 * kGroup;       // tokens a warp takes at a time
constexpr int kMinUnits = 16;           // units a CTA takes at least, where there are that many
// Ranges are equal in cost: an item costs its units and this many more (Q, the
// page ids, the state's start and end).  96 contexts of 350 to 16000 tokens
// took 82.8, 81.0, 79.6 and 80.0 us with 1, 2, 3 and 4.
constexpr int kItemUnits = 3;
constexpr float kLift = 8.f;            // log2 of P at a maximum
constexpr float kMove = 7.f;            // the reference moves on a jump above this many log2 units
constexpr float kNone = -3.0e38f;       // reference of a row without keys yet
constexpr int kSiteKv4 = 7;             // status code: a wait gave up

// An item cut by the start of a CTA's range, at its first cut: its parts lie
// with CTAs c0 .. c1.  A CTA's slot 2c holds its part of the item that began
// before its range, slot 2c + 1 that of the one that goes on behind it.
struct Cut {
  int s, item, c0, c1;  // s < 0: none
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
  float* first_o;          // workspace: [warps][rows][D], a warp's first item's O, not normalised
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
  // One CTA an SM (two of eight warps, whose ends an SM's preference for its
  // older warps draws 10 us apart, took 84 us where this takes 80).  O^T takes
  // NT D / 4 registers of a lane: with 128 of them a CTA has 8 warps, else 16,
  // whose 128 registers a lane hold everything at NT D / 4 = 16, 32 and, but
  // for spills (112 bytes stored at d = 128, 304 at d = 64), 64, with Q in
  // shared memory where it would take 32 more.  At d = 128 and 8 rows the ring
  // has three units a warp (216 KB, two thirds of it in flight).  The 96
  // contexts above, with 8 / 16 / 32 rows of a KV head: 80 / 122 / 191 us at d =
  // 128, 53 / 72 / 153 at d = 64; the cache alone would take 59 and 30.
  static constexpr bool kWide = NT * D > 256;
  static constexpr int kWarps = kWide ? 8 : kMaxWarps;
  static constexpr int kThreads = kWarps * 32;
  static constexpr bool kSharedQ = NT * D >= 256;
  static constexpr int kStages = D == 64 ? (kSharedQ ? 4 : 5) : kWide ? 4 : kSharedQ ? 2 : 3;
  static constexpr int kPad = 8;  // floats, so that rows of a state start in other banks
  static constexpr int kUnitBytes = 2 * group_bytes(D);
  static constexpr int kWarpRing = kStages * kUnitBytes;                  // at the end it holds the warp's last state:
  static_assert(kRows * (D + kPad) * 4 <= kWarpRing, "[rows][D + pad] fp32");
  static constexpr int kMlAt = kWarps * kWarpRing;                        // [warp][first, last][rows] (m, l)
  static constexpr int kQBytes = kSharedQ ? NT * (D / 16) * 32 * 8 : 0;   // a warp's Q: [NT][D / 16][lane] two words
  static constexpr int kQAt = kMlAt + kWarps * 2 * kRows * 8;
  static constexpr int kBarAt = kQAt + kWarps * kQBytes;
  static constexpr int kSmemBytes = kBarAt + kWarps * kStages * 8;
};

// The items' units: a sequence has ceil(len / 32), one at least (so that
// every output row has an item to write it).
__device__ __forceinline__ int tokens_of(int s, const DecodeParams& p) {
  const long long most = min(static_cast<long long>(p.max_pages) << p.page_shift, 0x7fffff00ll);
  return max(0, static_cast<int>(min(static_cast<long long>(p.seq_lens[s]), most)));
}
__device__ __forceinline__ int data_units(int len) { return (len + kUnit - 1) / kUnit; }
__device__ __forceinline__ int units_of(int len) { return max(1, data_units(len)); }
__device__ __forceinline__ int cost_of(int len) { return units_of(len) + kItemUnits; }

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
  for (int w = 0; w < kMaxWarps; ++w) {
    if (w * 32 >= static_cast<int>(blockDim.x)) break;
    if (w < warp) before += s_sums[w];
    total += s_sums[w];
  }
  return before + x - v;
}

// The sequences' costs, counted for one item of each: this thread's sequences
// [lo, hi) with their sum, the sum before them, and the total.
struct Scan {
  long long mine, before, total;
  int lo, hi;
  __device__ __forceinline__ Scan(const DecodeParams& p, long long* s_sums) {
    const int threads = static_cast<int>(blockDim.x), per = (p.n_seqs + threads - 1) / threads;
    lo = min(static_cast<int>(threadIdx.x) * per, p.n_seqs);
    hi = min(lo + per, p.n_seqs);
    mine = 0;
    for (int s = lo; s < hi; ++s) mine += cost_of(tokens_of(s, p));
    before = block_scan(mine, s_sums, total);
  }
};

// A warp's place in the concatenated items: the segment (units of one item) it
// is at.  Only changed between segments.
struct Walk {
  int s, item;     // sequence, item within it (head * row_tiles + row tile)
  int len, units;  // the sequence's
  int u0, count;   // the segment's units: [u0, u0 + count); none where the range ends within the item's own cost
  int take;        // the segment's cost
  int left;        // cost from here to the end of the warp's range; 0: done
  // from `at` of the item's cost on
  __device__ __forceinline__ void set(int at) {
    take = min(units + kItemUnits - at, left);
    u0 = max(0, at - kItemUnits);
    count = max(0, at + take - kItemUnits - u0);
  }
  __device__ __forceinline__ void next(const DecodeParams& p) {
    left -= take;
    if (left <= 0) return;
    if (++item == p.Hkv * p.row_tiles) {
      item = 0;
      ++s;
      len = tokens_of(s, p);
      units = units_of(len);
    }
    set(0);
  }
  __device__ __forceinline__ int end() const { return min(u0 + count, data_units(len)); }  // of the units that hold tokens
};

// Where a warp's loads are: a segment and its next unit.
struct LoadCursor {
  Walk w;
  int u;
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

  // The item's query rows (`words`: the warp's shared memory for them; every
  // lane reads its own words only).
  __device__ __forceinline__ void load_q(const Walk& w, const DecodeParams& p, uint2* words) {
    const int lane = threadIdx.x & 31, t = lane & 3;
    const int row0 = w.item % p.row_tiles * 8 * NT;
    q_shared = words + lane;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float factor;
      if constexpr (kSharedQ) {
        uint32_t x[D / 16][2];
        load_q_rows<D>(nt, row0, w, p, x, factor);
#pragma unroll
        for (int i = 0; i < D / 16; ++i) words[(nt * (D / 16) + i) * 32 + lane] = make_uint2(x[i][0], x[i][1]);
      } else {
        load_q_rows<D>(nt, row0, w, p, q[nt], factor);
      }
      factor = fmaxf(factor, 1.17549435e-38f);  // positive: a masked score is -inf times it
      f[nt][0] = __shfl_sync(0xffffffffu, factor, 8 * t);  // lanes 4 r hold row r's
      f[nt][1] = __shfl_sync(0xffffffffu, factor, 8 * t + 4);
    }
  }

  // l summed over the lanes that hold a row's keys.
  __device__ __forceinline__ void sum_l() {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], 4);
        l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], 8);
        l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], 16);
      }
  }

  // The state of a shared item, to [rows][stride] fp32 and [rows] (m, l).
  __device__ __forceinline__ void save(float* o, int stride, float2* ml) const {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = nt * 8 + 2 * t + e;
#pragma unroll
        for (int j = 0; j < D / 16; j += 2)
          *reinterpret_cast<float4*>(o + r * stride + (D / 8) * g + 2 * j) =
              make_float4(acc[nt][j][e], acc[nt][j][2 + e], acc[nt][j + 1][e], acc[nt][j + 1][2 + e]);
        if (g == 0) ml[r] = make_float2(m[nt][e], l[nt][e]);
      }
  }

  // The whole of an item: O = O_acc v_scale / l in bf16, L = (m + log2 l) ln 2.
  __device__ __forceinline__ void write(const Walk& w, const DecodeParams& p) const {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const RowPlace rp = row_place(w.s, w.item, nt * 8 + 2 * t + e, 8 * NT, p);
        if (!rp.store) continue;
        const float inv = l[nt][e] == 0.f ? 0.f : p.v_scale / l[nt][e];
        uint4* dst = reinterpret_cast<uint4*>(p.o + (rp.token * p.Hq + rp.head) * D + (D / 8) * g);
#pragma unroll
        for (int j = 0; j < D / 16; j += 4)
          dst[j / 4] = make_uint4(pack_bf16x2(acc[nt][j][e] * inv, acc[nt][j][2 + e] * inv),
                                  pack_bf16x2(acc[nt][j + 1][e] * inv, acc[nt][j + 1][2 + e] * inv),
                                  pack_bf16x2(acc[nt][j + 2][e] * inv, acc[nt][j + 2][2 + e] * inv),
                                  pack_bf16x2(acc[nt][j + 3][e] * inv, acc[nt][j + 3][2 + e] * inv));
        if (g == 0)
          p.lse[static_cast<long long>(rp.head) * p.n_seqs * p.Lq + rp.token] =
              (m[nt][e] + log2f(l[nt][e])) * 0.69314718055994531f;
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

  // O^T += V^T P^T of one group.  masked: keys may lie past the sequence's
  // end, or (skip) none of the group is to be looked at; the scales there may
  // be NaN, which 0 * NaN would spread (codes are always finite).
  __device__ __forceinline__ void values(const uint8_t* st, const uint32_t* b0, const uint32_t* b1, bool masked,
                                         uint32_t skip, int pos, const Walk& w, const DecodeParams& p) {
    constexpr int kHalf = D / 2, kBlocks = D / 16;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const uint8_t* va = st + codes_at(D, 1) + t * kHalf + g * (D / 16);
    const uint8_t* sc = st + scales_at(D, 1) + t * kBlocks + (D == 128 ? g : g >> 1);
    uint32_t s[4];
#pragma unroll
    for (int n = 0; n < 4; ++n) s[n] = sc[4 * n * kBlocks];
    if (masked) {
      uint32_t nan = 0;  // bit n: this lane's block of key t + 4n is NaN
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        if (skip != 0 || pos + t + 4 * n >= w.len) s[n] = 0u;
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
    const bool masked = tail || skip != 0;
    if (masked) {
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
      values(st + n * group_bytes(D), b0, b1, masked, (skip >> n) & 1u, pos + n * kGroup, w, p);
    }
  }
};

// O = O_acc v_scale / l as bf16 and L = (m + log2 l) ln 2 of four elements of a row.
__device__ __forceinline__ void write_row(const RowPlace& rp, int D, int d4, float4 O, float M, float L,
                                          const DecodeParams& p) {
  const float inv = L == 0.f ? 0.f : p.v_scale / L;
  *reinterpret_cast<uint2*>(p.o + (rp.token * p.Hq + rp.head) * D + d4) =
      make_uint2(pack_bf16x2(O.x * inv, O.y * inv), pack_bf16x2(O.z * inv, O.w * inv));
  if (d4 == 0)
    p.lse[static_cast<long long>(rp.head) * p.n_seqs * p.Lq + rp.token] = (M + log2f(L)) * 0.69314718055994531f;
}

// Where a CTA's range starts: a sequence, and the cost of its items before it.
struct From {
  int s;
  long long at;
};

// A warp's shared items: its range's first (where that is not its last too) and last.
struct Shared {
  int s, item, u0, count, units;  // the item's units [u0, u0 + count) of `units`; count = 0: none
};

// The combination of a CTA's shared items: M = max m_e, O = sum O_e 2^(m_e - M),
// l likewise (a state without keys has m = kNone, l = 0 and O = 0).  A warp
// takes 32 / (D / 4) rows of an item at a time, elements d4 .. d4+3 to a lane.
// Of an item's entries only the last may be a warp's first item, in the
// workspace; its load goes out a step ahead.  The loops are not unrolled: this
// runs once a launch, from a cold instruction cache.
template <int D, int NT>
__device__ __forceinline__ void combine(const int* entries, const int* starts, int groups, const uint8_t* smem,
                                        const Shared (*shared)[2], const DecodeParams& p) {
  using C = DecodeCfg<D, NT>;
  constexpr int kRows = C::kRows, kWarps = C::kWarps, kLanes = D / 4, kSide = 32 / kLanes, kSteps = kRows / kSide;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r0 = lane / kLanes, d4 = lane % kLanes * 4;
  const float2* s_ml = reinterpret_cast<const float2*>(smem + C::kMlAt);
  const float* first_o = p.first_o + static_cast<long long>(blockIdx.x) * kWarps * kRows * D + d4;
  auto fetch = [&](int idx) {  // the last entry's elements, where they are in the workspace
    if (idx >= groups * kSteps) return make_float4(0.f, 0.f, 0.f, 0.f);
    const int last = entries[starts[idx / kSteps + 1] - 1];
    if (last & 1) return make_float4(0.f, 0.f, 0.f, 0.f);
    return *reinterpret_cast<const float4*>(first_o + ((last >> 1) * kRows + idx % kSteps * kSide + r0) * D);
  };
  float4 ahead = fetch(warp);
#pragma unroll 1
  for (int idx = warp; idx < groups * kSteps; idx += kWarps) {
    const int group = idx / kSteps, r = idx % kSteps * kSide + r0;
    const int e0 = starts[group], e1 = starts[group + 1];
    const float4 stored = ahead;
    ahead = fetch(idx + kWarps);
    float M = kNone, L = 0.f;
    int count = 0;
#pragma unroll 4
    for (int x = e0; x < e1; ++x) {
      const int e = entries[x];
      count += shared[e >> 1][e & 1].count;
      M = fmaxf(M, s_ml[e * kRows + r].x);
    }
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int x = e0; x < e1; ++x) {
      const int e = entries[x];
      const float2 ml = s_ml[e * kRows + r];
      const float f = ex2_approx(ml.x - M);
      const float4 a = e & 1 ? *reinterpret_cast<const float4*>(smem + (e >> 1) * C::kWarpRing + (r * (D + C::kPad) + d4) * 4)
                             : stored;
      L = fmaf(ml.y, f, L);
      o = make_float4(fmaf(a.x, f, o.x), fmaf(a.y, f, o.y), fmaf(a.z, f, o.z), fmaf(a.w, f, o.w));
    }
    const Shared& x = shared[entries[e0] >> 1][entries[e0] & 1];
    if (count == x.units) {
      const RowPlace rp = row_place(x.s, x.item, r, kRows, p);
      if (rp.store) write_row(rp, D, d4, o, M, L, p);
    } else {
      const long long row = (2ll * blockIdx.x + (x.u0 > 0 ? 0 : 1)) * kRows + r;
      *reinterpret_cast<float4*>(p.part_o + row * D + d4) = o;
      if (d4 == 0) p.part_ml[row] = make_float2(M, L);
    }
  }
}

template <int D, int NT>
__global__ void __launch_bounds__(DecodeCfg<D, NT>::kThreads, 1) decode_kernel(const DecodeParams p) {
  using C = DecodeCfg<D, NT>;
  constexpr int kRows = C::kRows, kWarps = C::kWarps, kThreads = C::kThreads;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ long long s_sums[kMaxWarps];
  __shared__ From s_from;
  __shared__ LoadCursor s_load[kWarps];
  __shared__ Shared s_shared[kWarps][2];
  __shared__ int s_entry[2 * kWarps], s_group[2 * kWarps + 1], s_groups;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint8_t* ring = smem + warp * C::kWarpRing;
  const uint32_t ring_u32 = smem_u32(ring);
  const uint32_t bar0 = smem_u32(smem + C::kBarAt) + warp * C::kStages * 8;
  if (lane == 0) {
    for (int st = 0; st < C::kStages; ++st) mbar_init(bar0 + 8 * st, 1);
    fence_barrier_init();
    s_shared[warp][0].count = s_shared[warp][1].count = 0;
  }

  // This CTA's range of the concatenated items' cost, and from it this warp's.
  const int items = p.Hkv * p.row_tiles;  // of a sequence
  Walk w;
  w.left = 0;
  if (p.split) {
    if (threadIdx.x == 0) p.cuts[blockIdx.x].s = -1;
    const Scan sc(p, s_sums);  // a barrier, too
    const long long all = sc.total * items;
    const long long ctas = min(static_cast<long long>(gridDim.x), (all + kMinUnits - 1) / kMinUnits);
    const long long c = blockIdx.x;
    const long long begin = c < ctas ? all * c / ctas : all;
    const int n = c < ctas ? static_cast<int>(min(all * (c + 1) / ctas - begin, 0x7fffffffll)) : 0;
    const long long lo = sc.before * items, hi = (sc.before + sc.mine) * items;
    if (begin >= lo && begin < hi) {  // this thread's sequences hold the range's start
      long long at = lo;
      int s = sc.lo;
      for (;; ++s) {
        const long long after = at + static_cast<long long>(cost_of(tokens_of(s, p))) * items;
        if (begin < after) break;
        at = after;
      }
      s_from = From{s, begin - at};
    }
    __syncthreads();
    // this warp's share, from that sequence on
    const int from = static_cast<int>(static_cast<long long>(n) * warp / kWarps);
    w.left = static_cast<int>(static_cast<long long>(n) * (warp + 1) / kWarps) - from;
    if (w.left > 0) {
      w.s = s_from.s;
      long long at = s_from.at + from;  // counted from the sequence's start
      int cost;
      for (;; ++w.s) {
        w.len = tokens_of(w.s, p);
        w.units = units_of(w.len);
        cost = w.units + kItemUnits;
        if (at < static_cast<long long>(cost) * items) break;
        at -= static_cast<long long>(cost) * items;
      }
      w.item = at < 0x7fffffffll ? static_cast<int>(at) / cost : static_cast<int>(at / cost);
      const int in_item = static_cast<int>(at - static_cast<long long>(w.item) * cost);
      w.set(in_item);
      if (from == 0 && lane == 0 && w.u0 > 0) {
        // the CTA's range starts within an item: is this the item's first cut?
        const long long a = begin - in_item;  // its start
        if (all * (c - 1) / ctas <= a + kItemUnits)
          p.cuts[c] = Cut{w.s, w.item, static_cast<int>(c - 1), static_cast<int>(((a + cost) * ctas + all - 1) / all - 1)};
      }
    }
  } else {
    // short items: CTA i takes item i whole
    w.s = blockIdx.x / items;
    w.item = static_cast<int>(blockIdx.x) - w.s * items;
    w.len = tokens_of(w.s, p);
    w.units = units_of(w.len);
    const int from = w.units * warp / kWarps;
    w.left = w.units * (warp + 1) / kWarps - from;
    w.set(from + kItemUnits);
  }
  if (p.errors && blockIdx.x == 0) {
    for (int s = threadIdx.x; s < p.n_seqs; s += kThreads)
      if (p.seq_lens[s] != tokens_of(s, p)) atomicOr(p.errors, kErrPosition);
  }

  // The loads run ahead of the arithmetic, through the same units.  Up to 32
  // units of a segment are looked up together, one by each lane, which later
  // issues its unit's copies; the cursor is only touched then.
  if (lane == 0) s_load[warp] = LoadCursor{w, w.u0};
  __syncwarp();
  const int group_shift = p.page_shift - 4;  // log2 of a page's groups
  const long long page_bytes = (static_cast<long long>(row_bytes(D)) << p.page_shift) * p.Hkv;
  const uint8_t *src0 = nullptr, *src1 = nullptr;  // this lane's unit: its groups
  uint32_t bad0 = 0, bad1 = 0;                     // lanes whose first, second group is not loaded
  int batch = 0, next = 0;                         // units looked up, and issued of those
  auto look_up = [&]() {
    LoadCursor c = s_load[warp];
    batch = next = 0;
    while (c.w.left > 0 && c.u >= c.w.end()) {  // to the next segment that holds tokens
      c.w.next(p);
      c.u = c.w.u0;
    }
    if (c.w.left > 0) {
      batch = min(32, c.w.end() - c.u);
      const int group = 2 * (c.u + lane);
      int page0 = -1, page1 = -1;
      const bool second = (group + 1) * kGroup < c.w.len;  // else it may lie past the sequence's last page
      if (lane < batch) {
        const int* table = p.page_table + static_cast<long long>(c.w.s) * p.max_pages;
        page0 = __ldg(table + (group >> group_shift));
        page1 = group_shift > 0 ? page0 : second ? __ldg(table + group + 1) : -1;
      }
      const bool ok0 = static_cast<uint32_t>(page0) < static_cast<uint32_t>(p.num_pages);
      const bool ok1 = static_cast<uint32_t>(page1) < static_cast<uint32_t>(p.num_pages);
      const uint8_t* head = p.cache + (static_cast<long long>(row_bytes(D)) << p.page_shift) * (c.w.item / p.row_tiles);
      src0 = head + page0 * page_bytes + (group & ((1 << group_shift) - 1)) * group_bytes(D);
      src1 = group_shift > 0 ? src0 + group_bytes(D) : head + page1 * page_bytes;
      bad0 = __ballot_sync(0xffffffffu, lane < batch && !ok0);
      bad1 = __ballot_sync(0xffffffffu, lane < batch && !ok1);
      if (p.errors && lane < batch && (!ok0 || (!ok1 && second))) atomicOr(p.errors, kErrPage);
      c.u += batch;
    }
    __syncwarp();
    if (lane == 0) s_load[warp] = c;
    __syncwarp();
  };
  uint32_t loads = 0;     // units asked for
  uint32_t load_at = 0;   // the stage the next one goes to
  uint32_t skips = 0;     // two bits per stage: groups that were not loaded
  auto issue = [&]() {
    if (next == batch) {
      look_up();
      if (batch == 0) return;
    }
    const uint32_t st = load_at, dst = ring_u32 + st * C::kUnitBytes, bar = bar0 + 8 * st;
    if ((bad0 | bad1 | skips) == 0 && group_shift > 0) {  // the usual case: both groups lie together
      if (lane == next) {
        mbar_arrive_expect_tx(bar, C::kUnitBytes);
        bulk_load(dst, src0, C::kUnitBytes, bar);
      }
    } else {
      const uint32_t no0 = (bad0 >> next) & 1u, no1 = (bad1 >> next) & 1u;
      skips = (skips & ~(3u << (2 * st))) | (no0 | no1 << 1) << (2 * st);
      if (lane == next) {
        mbar_arrive_expect_tx(bar, (2 - no0 - no1) * group_bytes(D));
        if (no0 == 0) bulk_load(dst, src0, group_bytes(D), bar);
        if (no1 == 0) bulk_load(dst + group_bytes(D), src1, group_bytes(D), bar);
      }
    }
    load_at = st + 1 == C::kStages ? 0 : st + 1;
    ++next;
    ++loads;
  };
#pragma unroll 1
  for (int i = 0; i < C::kStages; ++i) issue();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  float2* s_ml = reinterpret_cast<float2*>(smem + C::kMlAt);
  float* first_o = p.first_o + (static_cast<long long>(blockIdx.x) * kWarps + warp) * kRows * D;
  uint32_t used = 0;            // units taken from the ring
  uint32_t at = 0, parity = 0;  // the stage of the next one, and its phase
  bool dead = false;            // a wait gave up
  State<D, NT> state;
#pragma unroll 1
  for (; w.left > 0; w.next(p)) {
    if (w.count == 0) continue;  // the range ends with an item's own cost
    state.reset();
    state.load_q(w, p, reinterpret_cast<uint2*>(smem + C::kQAt + warp * C::kQBytes));
    const int end = w.end();
    const int tail_from = w.len - p.Lq + 1;  // a unit that reaches past it is masked
#pragma unroll 1
    for (int u = w.u0; u < end && !dead; ++u) {
      if (!__all_sync(0xffffffffu, mbar_wait_bounded(bar0 + 8 * at, parity, p.wait_limit_ns))) {
        dead = true;
        if (lane == 0) atomicCAS(p.status, 0, kSiteKv4);
        break;
      }
      state.unit(ring + at * C::kUnitBytes, u * kUnit, (u + 1) * kUnit > tail_from, (skips >> (2 * at)) & 3u, w, p);
      __syncwarp();  // every lane has read the stage
      ++used;
      if (++at == C::kStages) at = 0, parity ^= 1u;
      issue();
    }
    state.sum_l();
    if (w.count == w.units) {
      state.write(w, p);
      continue;
    }
    // a shared item: the range's last goes where the ring was (nothing is on
    // its way there any more), its first to the workspace
    const int which = w.take == w.left ? 1 : 0;
    if (lane == 0) s_shared[warp][which] = Shared{w.s, w.item, w.u0, w.count, w.units};
    if (which == 1 && !dead)
      state.save(reinterpret_cast<float*>(ring), D + C::kPad, s_ml + (warp * 2 + 1) * kRows);
    else if (which == 0)
      state.save(first_o, D, s_ml + warp * 2 * kRows);
  }
  // Copies still in flight land before the CTA exits (only after a wait gave up).
  for (; used < loads; ++used) mbar_wait_bounded(bar0 + 8 * (used % C::kStages), (used / C::kStages) & 1, p.wait_limit_ns);
  __syncthreads();

  // The shared items: entries (warp, first / last) in order, an item's are
  // neighbours; the first warp lists them and where each item's start.
  if (warp == 0) {
    const Shared x = lane < 2 * kWarps ? s_shared[lane >> 1][lane & 1] : Shared{0, 0, 0, 0, 0};
    const uint32_t used_mask = __ballot_sync(0xffffffffu, x.count > 0);
    const uint32_t below = used_mask & ((1u << lane) - 1u);
    const int before = below ? 31 - __clz(below) : lane;  // the entry before this one
    const int s_before = __shfl_sync(0xffffffffu, x.s, before), item_before = __shfl_sync(0xffffffffu, x.item, before);
    const bool starts = x.count > 0 && (below == 0 || s_before != x.s || item_before != x.item);
    const uint32_t starts_mask = __ballot_sync(0xffffffffu, starts);
    if (x.count > 0) s_entry[__popc(below)] = lane;
    if (starts) s_group[__popc(starts_mask & ((1u << lane) - 1u))] = __popc(below);
    if (lane == 0) {
      s_groups = __popc(starts_mask);
      s_group[__popc(starts_mask)] = __popc(used_mask);
    }
  }
  __syncthreads();
  combine<D, NT>(s_entry, s_group, s_groups, smem, s_shared, p);
}

constexpr int kMergeRows = 2;  // rows of a CTA of merge_kernel
constexpr int kMergeThreads = 256;

// Block (c, y): rows 2y, 2y+1 of the item that the start of CTA c's range cuts
// first, if it does: its parts' states are merged as the warps' were.  D / 4
// threads take a row's part, several parts side by side.
template <int D>
__global__ void __launch_bounds__(kMergeThreads) merge_kernel(const DecodeParams p, int rows) {
  constexpr int kLanes = D / 4;                               // threads of one row
  constexpr int kSide = kMergeThreads / (kMergeRows * kLanes);     // parts side by side
  __shared__ float4 s_o[kSide][kMergeRows][kLanes];
  __shared__ float2 s_ml[kSide][kMergeRows];
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the kernel before has finished and its writes are here
  const Cut cut = p.cuts[blockIdx.x];
  if (cut.s < 0) return;
  const int lane = threadIdx.x % kLanes, rr = threadIdx.x / kLanes % kMergeRows, side = threadIdx.x / (kLanes * kMergeRows);
  const int r = blockIdx.y * kMergeRows + rr;
  auto row_of = [&](int c) { return (2ll * c + (c == cut.c0 ? 1 : 0)) * rows + r; };
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
