// Attention of a tree of drafted tokens over the paged 4-bit cache on the
// tensor core (tcgen05), for trees whose rows fill a good part of its 128.
//
// Row r of an item is node r / G of the tree and query head r % G of the item's
// KV head; it sees the context and the nodes on its line (tree_line):
//
//     O = sum_j softmax_j(scale q . k_j) v_j,   L = ln sum_j exp(scale q . k_j).
//
// fa_kv4_decode.cuh turns a lane's codes into its own operands of mma.sync, all
// over again for every 8 to 32 rows; here a tile of 128 keys is turned into f16
// once, in shared memory, for 128 rows:
//
// - Codes times scales are exact in f16 (fa_kv4.cuh).  Q rows are brought to
//   [2^14, 2^15) by a power of two, and P to a maximum of 2^8 when the reference is
//   set, which moves when P would leave f16's range: as in fa_kv4_decode.cuh, f16 then
//   loses nothing above 2^-33 of the maximum, P's rounding is 2^-11, every sum is fp32.
// - Two softmax warpgroups, one row a thread, take a CTA's tiles in turn, each
//   with its own S, P and O in tensor memory and its own running maximum and sum, so
//   that one's products overlap the other's exponentials and neither waits for the
//   other's maximum.  An item's two states meet at its end.
// - Eight warps turn codes into operands, K or V of 32 keys each, from a ring that
//   one warp fills (bulk copies some tiles ahead, across items).  A tile's K and V each
//   have two places in shared memory, one for each warpgroup.
//
// What a row does not see must not reach it: scores are replaced by -inf, bit by
// bit of the row's line; of V, keys past the sequence's end and blocks that are NaN
// at a tree's node are zeros in the product (0 * NaN is NaN), the latter being
// set to NaN at the end in the rows that see the node.
//
// Work: the (sequence, KV head, row tile) items' tiles, concatenated, are cut
// into ranges of equal cost, one per CTA, from the lengths on the device; an item
// cut between CTAs is merged by merge_kernel (fa_kv4_decode.cuh).
//
// Measured on a GB300 (8 KV heads of 4 query heads, d = 128): 60 nodes over 131000
// tokens 130 us, 990 TFLOP/s of visible products (58 us at cuBLAS' bf16 rate, 68
// with the rows that fill the second tile of 128; the cache read twice, 302 MB, 45
// us); 24 nodes over 32 contexts of 250 to 12000 tokens 67 us (17; 22 with the rows
// that fill a tile; 16 for the bytes).  A tile takes a CTA 1.07 us: the tensor core
// has work for 46 % of that, issue slots are 56 % used.  What bounds it is a
// warpgroup's own round, two tiles long: its products 0.6 us (the operands, the codes
// and their conversion move 196 KB through shared memory a tile, 0.75 us at the most),
// scores through tensor memory 0.2 us a half, exponentials 0.3 a half, four
// hand-overs of 0.1.  Without the softmax's arithmetic the long context takes 116 us,
// without the conversion of codes 120.  An item's start and end are 5 us, a launch's
// start 2.7.
// Items of 256 rows, each warpgroup with all key tiles for its own 128 (half the
// conversions and loads; K then has one place only): 137 us.
//
// Warps: 0-7 softmax; 8-15 codes to operands; 16 MMA issuer; 17 loads.
#pragma once

#include <type_traits>

#include "fa_kv4_decode.cuh"

namespace fa {
namespace kv4 {
namespace tree {

constexpr int kRows = 128;             // of an item
constexpr int kKeys = 128;             // of a tile
constexpr int kTurnWarps = 8;          // four for K, four for V; two groups of a tile each
constexpr int kThreads = 640;
// An item's own cost, in tiles.  The 32 contexts: 72, 68 and 72 us with 5, 8 and 11, the
// long one 133, 130 and 129.
constexpr int kItemTiles = 8;
// A CTA takes at least, where there are that many.  16 nodes over 2000 tokens: 15.6, 16.9
// and 20.5 us with 2, 4 and 8.
constexpr int kMinTiles = 2;
constexpr uint32_t kTmemCols = 512;
constexpr int kSiteTree = 8;           // status code: a wait gave up
// Registers: the launch gives every thread 96 (65536 / 640, rounded down to 8).
constexpr uint32_t kRegsSoftmax = 128, kRegsTurn = 80, kRegsIssue = 64;
static_assert(256 * kRegsSoftmax + 256 * kRegsTurn + 128 * kRegsIssue <= kThreads * 96, "register split exceeds the launch");

constexpr int kFixedBars = 18;         // beside the rings'

template <int D>
struct Cfg {
  static constexpr int kSlabs = D / 64;                 // 64 columns of d each
  static constexpr int kSlabBytes = 128 * 128;          // 128 rows of 128 bytes
  static constexpr int kTileBytes = kSlabs * kSlabBytes;
  static constexpr int kRing = D == 128 ? 3 : 6;        // tiles of codes and scales
  static constexpr int kQOff = 0;
  static constexpr int kKOff = kTileBytes;              // two places
  static constexpr int kVOff = kKOff + 2 * kTileBytes;  // two places
  static constexpr int kRawOff = kVOff + 2 * kTileBytes;
  static constexpr int kRawTile = kKeys / kGroup * group_bytes(D);
  static constexpr int kBarOff = kRawOff + kRing * kRawTile;
  static constexpr int kNumBars = kFixedBars + 2 * kRing;
  static constexpr int kMiscOff = kBarOff + (kNumBars * 8 + 15) / 16 * 16;
  static constexpr int kSmemBytes = kMiscOff + 16 + 1024;  // + alignment slack
  static_assert(kSmemBytes + 4096 <= 232448, "227 KB with the static part");
  // Tensor memory: S and O of each warpgroup; P over S, or at d = 64 beside O
  static constexpr int kTmemS = 0, kTmemO = 256, kTmemP = D == 64 ? kTmemO + 64 : kTmemS, kTmemGroup = 128;
};

// The barriers' shared addresses, all from one.
struct Bars {
  uint32_t at;
  volatile int* abort_flag;
  __device__ __forceinline__ uint32_t k_full(uint32_t g) const { return at + 8 * g; }
  __device__ __forceinline__ uint32_t k_empty(uint32_t g) const { return at + 16 + 8 * g; }
  __device__ __forceinline__ uint32_t v_full(uint32_t g) const { return at + 32 + 8 * g; }
  __device__ __forceinline__ uint32_t v_empty(uint32_t g) const { return at + 48 + 8 * g; }
  __device__ __forceinline__ uint32_t s_full(uint32_t g) const { return at + 64 + 8 * g; }
  __device__ __forceinline__ uint32_t p_ready(uint32_t g) const { return at + 80 + 8 * g; }
  __device__ __forceinline__ uint32_t o_done(uint32_t g) const { return at + 96 + 8 * g; }
  __device__ __forceinline__ uint32_t q_full() const { return at + 112; }
  __device__ __forceinline__ uint32_t states() const { return at + 120; }   // between the warpgroups: an item's states are there,
  __device__ __forceinline__ uint32_t written() const { return at + 128; }  // its O has been read
  __device__ __forceinline__ uint32_t drain() const { return at + 136; }
  __device__ __forceinline__ uint32_t raw(uint32_t st) const { return at + 144 + 16 * st; }  // a ring place is full, empty
  __device__ __forceinline__ uint32_t raw_empty(uint32_t st) const { return at + 152 + 16 * st; }
};
// kv4's costs and walk over the concatenated items, in tiles of 128 keys.
__device__ __forceinline__ int data_tiles(int len) { return (len + kKeys - 1) / kKeys; }
__device__ __forceinline__ int tiles_of(int len) { return max(1, data_tiles(len)); }
__device__ __forceinline__ int tile_cost(int len) { return tiles_of(len) + kItemTiles; }

// A CTA's place in the concatenated items: the segment (tiles of one item) it is at.
struct Segments {
  int s, item;     // sequence, item within it (head * row_tiles + row tile)
  int len, tiles;  // the sequence's
  int t0, count;   // the segment's tiles: [t0, t0 + count); none where the range ends within the item's own cost
  int take, left;  // the segment's cost; that from here to the end of the range (0: done)
  __device__ __forceinline__ void set(int at) {
    take = min(tiles + kItemTiles - at, left);
    t0 = max(0, at - kItemTiles);
    count = max(0, at + take - kItemTiles - t0);
  }
  __device__ __forceinline__ void next(const DecodeParams& p) {
    left -= take;
    if (left <= 0) return;
    if (++item == p.Hkv * p.row_tiles) {
      item = 0;
      ++s;
      len = tokens_of(s, p);
      tiles = tiles_of(len);
    }
    set(0);
  }
  // To the next segment with a share in its item, from the present one on.
  __device__ __forceinline__ void skip_empty(const DecodeParams& p) {
    while (left > 0 && count == 0) next(p);
  }
  __device__ __forceinline__ int data() const { return max(0, min(t0 + count, data_tiles(len)) - t0); }  // tiles with tokens
  __device__ __forceinline__ bool whole() const { return count == tiles; }
};

// Waits of a warp for a barrier's phase, for a limited time; false, in every lane,
// where one gave up.
__device__ __forceinline__ bool wait_on(uint32_t bar, uint32_t parity, const Bars b, int* status, unsigned long long limit_ns) {
  const uint64_t t0 = global_timer_ns();
  uint32_t polls = 0;
  while (true) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    if ((++polls & 31u) == 0u) {
      bool stop = *b.abort_flag != 0;
      if (!stop && global_timer_ns() - t0 > limit_ns) {
        stop = true;
        *b.abort_flag = 1;
        atomicCAS(status, 0, kSiteTree);
      }
      if (__any_sync(0xffffffffu, stop)) return false;
    }
  }
}
// The same of one thread.
__device__ __forceinline__ bool wait_alone(uint32_t bar, uint32_t parity, const Bars& b, const DecodeParams& p) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_timer_ns();
  uint32_t polls = 0;
  while (true) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((++polls & 31u) == 0u) {
      if (*b.abort_flag) return false;
      if (global_timer_ns() - t0 > p.wait_limit_ns) {
        *b.abort_flag = 1;
        atomicCAS(p.status, 0, kSiteTree);
        return false;
      }
    }
  }
}
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, const Bars& b, const DecodeParams& p) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  return wait_on(bar, parity, b, p.status, p.wait_limit_ns);
}

// What the warps pass each other beside the barriers.
struct Notes {
  uint32_t skip[4][2];                // a tile's groups whose page was refused (a byte each), by tile number mod 4
  uint32_t nan[4][kMaxTreeNodes];     // by item number mod 4: (item number << 8) | V blocks of a node that are NaN
  uint32_t any_nan[4];                // the item number + 1 where there is one
  float2 ml[2][kRows];                // the warpgroups' running maxima and sums
  float factor[kRows];                // of the item whose Q is in shared memory
  uint32_t raw[8];                    // by ring place: a bit for each group that was loaded, and from bit 8 for each refused
};

// ---------------------------------------------------------------------------
// Codes to operands (warps 0-3: K of a tile's keys 32 w ...; 4-7: V)
// ---------------------------------------------------------------------------
// K or V of two groups (32 keys x D) into rows key0 .. of a tile,
// blocks of 16 elements, eight or four a lane.  A row is 128 bytes of each
// 64-column slab, its 16-byte chunks permuted by the row's low bits as the 128-byte
// swizzle wants; the lanes' blocks are dealt so that eight lanes' chunks fall into
// all banks.  scale_of(key, block, byte) may change a block's scale.
template <int D, class Scale>
__device__ __forceinline__ void turn_keys(const uint8_t* raw, uint8_t* tile, int key0, Scale scale_of) {
  constexpr int kKeysAtOnce = 32 * 16 / D, kSteps = 32 / kKeysAtOnce;
  const int lane = threadIdx.x & 31;
  const int block = D == 128 ? (lane & 3) | (lane >> 1 & 4) : lane & 3;
  const int key_in = D == 128 ? (lane >> 2 & 1) | (lane >> 3 & 2) : lane >> 2;
  uint2 codes[kSteps];
  uint32_t scales[kSteps];
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int key = i * kKeysAtOnce + key_in;
    const uint8_t* half = raw + (i * kKeysAtOnce >= kGroup ? group_bytes(D) - kGroup * (D / 2) : 0);
    const uint8_t* half_s = raw + (i * kKeysAtOnce >= kGroup ? group_bytes(D) - kGroup * (D / 16) : 0);
    codes[i] = *reinterpret_cast<const uint2*>(half + key * (D / 2) + block * 8);
    scales[i] = half_s[kGroup * D / 2 + key * (D / 16) + block];
  }
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int key = i * kKeysAtOnce + key_in, row = key0 + key;
    const uint32_t sb = scale_of(key, block, scales[i]);
    const uint32_t s = e4m3x2_to_f16x2(sb | (sb << 8));
    uint32_t x[8];
    e2m1x8_to_f16x2(codes[i].x, x);
    e2m1x8_to_f16x2(codes[i].y, x + 4);
#pragma unroll
    for (int n = 0; n < 8; ++n) x[n] = f16x2_mul(x[n], s);
    uint8_t* at = tile + (block >> 2) * Cfg<D>::kSlabBytes + row * 128;
    const int chunk = (block & 3) * 2;
    *reinterpret_cast<uint4*>(at + ((chunk ^ (row & 7)) << 4)) = make_uint4(x[0], x[1], x[2], x[3]);
    *reinterpret_cast<uint4*>(at + (((chunk + 1) ^ (row & 7)) << 4)) = make_uint4(x[4], x[5], x[6], x[7]);
  }
}

// The same where not all keys are context: keys that are not in `on` (bit per
// group: behind the sequence or refused) or not below `live` are zeros; a V block
// that is NaN at a node (the first key's is node0) is zeros, too, and noted.  A
// call, so that the plain conversion's loop stays short.
template <int D>
__device__ __noinline__ void turn_tail(const uint8_t* raw, uint8_t* tile, int key0, uint32_t on, int v, int live, int node0,
                                       uint32_t number, Notes& notes, int nodes) {
  const int lane = threadIdx.x & 31;
  uint32_t* noted = notes.nan[number & 3u];
  if (v && node0 + lane >= 0 && node0 + lane < nodes) noted[node0 + lane] = number << 8;
  __syncwarp();
  turn_keys<D>(raw, tile, key0, [&](int key, int block, uint32_t s) {
    if (key >= live || !(on >> (key >> 4) & 1u)) return 0u;
    if (v && (s & 0x7fu) == 0x7fu && node0 + key >= 0) {
      atomicOr(noted + node0 + key, 1u << block);
      notes.any_nan[number & 3u] = number + 1;
      return 0u;
    }
    return s;
  });
}

template <int D>
__device__ __forceinline__ void run_turn(int w, uint8_t* smem, Segments seg, const Bars& b, Notes& notes, const DecodeParams& p) {
  using C = Cfg<D>;
  const int lane = threadIdx.x & 31, v = w >> 2, pair = w & 3;
  uint32_t c = 0;             // tiles taken
  uint32_t st = 0, phase = 0; // the ring place of the next one, and its barrier's phase
  uint32_t number = 0;        // items with tiles
  bool ok = true;
  const int key0 = pair * 2 * kGroup;
  const uint8_t* raw = smem + C::kRawOff + pair * 2 * group_bytes(D) + codes_at(D, v);
  const uint32_t full = v ? b.v_full(0) : b.k_full(0), empty = v ? b.v_empty(0) : b.k_empty(0);
  uint8_t* tiles = smem + (v ? C::kVOff : C::kKOff);
#pragma unroll 1
  for (; seg.left > 0 && ok; seg.next(p)) {
    const int n = seg.data();
    if (n == 0) continue;
    const int prefix = seg.len - p.Lq;
#pragma unroll 1
    for (int t = seg.t0; t < seg.t0 + n; ++t, ++c) {
      const uint32_t place = c & 1u;
      const int pos = t * kKeys + key0;
      ok = wait(b.raw(st), phase, b, p) && wait(empty + 8 * place, (c >> 1 & 1u) ^ 1u, b, p);
      if (!ok) break;
      const uint32_t has = notes.raw[st] >> (2 * pair);
      if (v == 0 && lane < 2) reinterpret_cast<uint8_t*>(notes.skip[c & 3u])[2 * pair + lane] = has >> (8 + lane) & 1u ? 0xffu : 0u;
      const uint8_t* keys = raw + st * C::kRawTile;
      uint8_t* tile = tiles + place * C::kTileBytes;
      if ((has & 3u) == 3u && pos + 2 * kGroup <= prefix) turn_keys<D>(keys, tile, key0, [](int, int, uint32_t s) { return s; });
      else turn_tail<D>(keys, tile, key0, has & 3u, v, seg.len - pos, pos - prefix, number, notes, p.Lq);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(full + 8 * place);
        mbar_arrive(b.raw_empty(st));
      }
      if (++st == C::kRing) st = 0, phase ^= 1u;
    }
    ++number;
  }
}

// ---------------------------------------------------------------------------
// Loads (one warp): tiles of codes and scales, a copy for each group
// ---------------------------------------------------------------------------
template <int D>
__device__ __forceinline__ void run_load(uint32_t sbase, Segments seg, const Bars& b, Notes& notes, const DecodeParams& p) {
  using C = Cfg<D>;
  constexpr int kGroups = kKeys / kGroup, kAtOnce = 32 / kGroups;  // tiles looked up together
  const int lane = threadIdx.x & 31, group_in = lane % kGroups, tile_in = lane / kGroups;
  const int group_shift = p.page_shift - 4;
  const long long head_bytes = static_cast<long long>(row_bytes(D)) << p.page_shift, page_bytes = head_bytes * p.Hkv;
  // a batch: up to kAtOnce tiles of one segment, and what this lane has to copy of them
  struct Batch {
    const uint8_t* head;  // the KV head's part of page 0
    int count, group, page;
    bool exists;
  };
  int at = 0;  // tiles of the segment that were looked up
  auto look_up = [&]() {
    Batch x{nullptr, 0, 0, -1, false};
    while (seg.left > 0 && at >= seg.data()) {
      seg.next(p);
      at = 0;
    }
    if (seg.left <= 0) return x;
    x.count = min(kAtOnce, seg.data() - at);
    x.group = (seg.t0 + at + tile_in) * kGroups + group_in;
    x.exists = tile_in < x.count && x.group * kGroup < seg.len;
    if (x.exists) x.page = __ldg(p.page_table + static_cast<long long>(seg.s) * p.max_pages + (x.group >> group_shift));
    x.head = p.cache + head_bytes * (seg.item / p.row_tiles);
    at += x.count;
    return x;
  };
  uint32_t st = 0, phase = 0, issued = 0;
  bool ok = true;
  Batch now = look_up();
#pragma unroll 1
  while (now.count > 0 && ok) {
    const Batch next = look_up();  // on its way while this one is issued
    const bool on = static_cast<uint32_t>(now.page) < static_cast<uint32_t>(p.num_pages);
    const uint32_t loaded = __ballot_sync(0xffffffffu, on), refused = __ballot_sync(0xffffffffu, now.exists && !on);
    if (p.errors && now.exists && !on) atomicOr(p.errors, kErrPage);
    const uint8_t* src = now.head + now.page * page_bytes + static_cast<long long>(now.group & ((1 << group_shift) - 1)) * group_bytes(D);
#pragma unroll 1
    for (int i = 0; i < now.count; ++i, ++issued) {
      ok = wait(b.raw_empty(st), phase ^ 1u, b, p);
      if (!ok) break;
      const uint32_t has = loaded >> (i * kGroups) & 0xffu;
      if (lane == 0) {
        notes.raw[st] = has | (refused >> (i * kGroups) & 0xffu) << 8;
        mbar_arrive_expect_tx(b.raw(st), __popc(has) * group_bytes(D));
      }
      __syncwarp();
      if (tile_in == i && on) bulk_load(sbase + C::kRawOff + st * C::kRawTile + group_in * group_bytes(D), src, group_bytes(D), b.raw(st));
      if (++st == C::kRing) st = 0, phase ^= 1u;
    }
    now = next;
  }
  // Every copy that was started lands before the CTA exits, also after a wait gave up.
  const uint32_t first = issued > static_cast<uint32_t>(C::kRing) ? issued - C::kRing : 0;
  for (uint32_t i = first; i < issued; ++i) mbar_wait_bounded(b.raw(i % C::kRing), i / C::kRing & 1u, p.wait_limit_ns);
}

// ---------------------------------------------------------------------------
// MMA issuer
// ---------------------------------------------------------------------------
// Instruction descriptor for kind::f16 with f16 A and B and an fp32 accumulator.
__host__ __device__ constexpr uint32_t idesc_f16_f32(uint32_t M, uint32_t N, bool b_mn_major) {
  return (1u << 4) | ((b_mn_major ? 1u : 0u) << 16) | ((N >> 3) << 17) | ((M >> 4) << 24);
}

// The products with descriptors put together from words: the upper one is a
// constant of the operand's layout, the lower one the address (>> 4) and the
// leading offset.  Held as 64-bit values, 24 of them would fill the warp's registers.
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t hi, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
      "mov.b64 a, {%1, %3};\n\t"
      "mov.b64 b, {%2, %3};\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n\t}\n" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t hi, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\t"
      "mov.b64 b, {%2, %3};\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}\n" ::"r"(d),
      "r"(a), "r"(b_lo), "r"(hi), "r"(idesc), "r"(accumulate)
      : "memory");
}

// One thread for both warpgroups, tile after tile: O += P V of the tile before the
// last (the same warpgroup's) and S = Q K^T of this one go to the tensor core in
// one piece, so that one warpgroup has its softmax while the other has the tensor
// core.  (Two issuers, each for one of them, drifted into step: both softmaxes at
// the same time, with the tensor core idle.)
template <int D>
__device__ __forceinline__ void run_issue(uint32_t sbase, uint32_t tmem, Segments seg, const Bars& b, const DecodeParams& p) {
  using C = Cfg<D>;
  const uint32_t hi = static_cast<uint32_t>(sdesc_sw128(0, 0, 1024) >> 32);
  const uint32_t q_lo = static_cast<uint32_t>(sdesc_sw128(sbase + C::kQOff, 16, 1024));
  const uint32_t k_lo0 = static_cast<uint32_t>(sdesc_sw128(sbase + C::kKOff, 16, 1024));
  const uint32_t v_lo0 = static_cast<uint32_t>(sdesc_sw128(sbase + C::kVOff, C::kSlabBytes, 1024));
  bool ok = true;
  uint32_t c = 0, items = 0;  // tiles; items with tiles
#pragma unroll 1
  for (; seg.left > 0 && ok; seg.next(p)) {
    const int n = seg.data();
    if (n == 0) continue;
    ok = wait_alone(b.q_full(), items & 1u, b, p);
    ++items;
    // step i: P V of tile i - 2 and Q K^T of tile i, where there are such
#pragma unroll 1
    for (int i = 0; i < n + 2 && ok; ++i, ++c) {
      const bool pv = i >= 2, qk = i < n;
      if (i == 1 && n == 1) continue;  // nothing of the other warpgroup
      const uint32_t g = c & 1u;  // of tile i, and of tile i - 2
      if (qk) ok = wait_alone(b.k_full(g), c >> 1 & 1u, b, p);
      if (pv) ok = ok && wait_alone(b.v_full(g), (c - 2) >> 1 & 1u, b, p) && wait_alone(b.p_ready(g), (c - 2) >> 1 & 1u, b, p);
      if (!ok) break;
      tc_fence_after_sync();
      const uint32_t tm = tmem + g * C::kTmemGroup, place = g * (C::kTileBytes >> 4);
      if (pv) {
#pragma unroll
        for (int kk = 0; kk < kKeys / 16; ++kk)
          mma_ts(tm + C::kTmemO, tm + C::kTmemP + kk * 8, v_lo0 + place + kk * 128, hi, idesc_f16_f32(kRows, D, true),
                 i > 3 || kk > 0 ? 1u : 0u);
        umma_commit(b.v_empty(g));
      }
      if (qk) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (kk / 4) * C::kSlabBytes + (kk % 4) * 32;
          mma_ss(tm + C::kTmemS, q_lo + (off >> 4), k_lo0 + place + (off >> 4), hi, idesc_f16_f32(kRows, kKeys, false), kk > 0 ? 1u : 0u);
        }
        umma_commit(b.s_full(g));
        umma_commit(b.k_empty(g));
      } else {
        umma_commit(b.o_done(g));
      }
    }
    c -= 2;
  }
  // Every MMA this thread issued must finish before tensor memory is released.
  umma_commit(b.drain());
  mbar_wait_bounded(b.drain(), 0, p.wait_limit_ns);
}

// ---------------------------------------------------------------------------
// Softmax and output (warpgroup g: one row a thread)
// ---------------------------------------------------------------------------
// Q rows of an item to shared memory as f16 (K-major slabs, 128-byte swizzle),
// and each row's factor from its scores to log2 units: warp w of eight takes rows
// 16 w ..., D / 8 lanes a row, all loads in flight at once.
template <int D>
__device__ __forceinline__ void load_q(int w, uint8_t* smem, const Segments& seg, Notes& notes, const DecodeParams& p) {
  constexpr int kLanes = D / 8, kAtOnce = 32 / kLanes, kSteps = 16 / kAtOnce;
  const int lane = threadIdx.x & 31, chunk = lane % kLanes;
  const int h = seg.item / p.row_tiles, r0 = (seg.item - h * p.row_tiles) * kRows;
  const __nv_bfloat16* q = p.q + static_cast<long long>(seg.s) * p.Lq * p.q_stride + static_cast<long long>(h) * p.G * D + chunk * 8;
  uint4 x[kSteps];
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int r = r0 + w * 16 + i * kAtOnce + lane / kLanes, node = r / p.G;
    x[i] = make_uint4(0, 0, 0, 0);
    if (node < p.Lq) x[i] = __ldg(reinterpret_cast<const uint4*>(q + node * p.q_stride + (r - node * p.G) * D));
  }
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int row = w * 16 + i * kAtOnce + lane / kLanes;
    const uint32_t wds[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
    uint32_t m2 = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) m2 = __vmaxu2(m2, wds[k] & 0x7fff7fffu);
    uint32_t top = max(m2 & 0xffffu, m2 >> 16);
#pragma unroll
    for (int off = 1; off < kLanes; off <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, off));
    const int e = max(static_cast<int>(top >> 7) - 127, -100);  // floor(log2) of the row's largest element
    const float up = __uint_as_float(static_cast<uint32_t>(127 + 14 - e) << 23);
    uint32_t y[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) y[k] = pack_f16x2(__uint_as_float(wds[k] << 16) * up, __uint_as_float(wds[k] & 0xffff0000u) * up);
    *reinterpret_cast<uint4*>(smem + Cfg<D>::kQOff + (chunk >> 3) * Cfg<D>::kSlabBytes + row * 128 +
                              (((chunk & 7) ^ (row & 7)) << 4)) = make_uint4(y[0], y[1], y[2], y[3]);
    if (chunk == 0)  // positive: a masked score is -inf times it
      notes.factor[row] = fmaxf(__uint_as_float(static_cast<uint32_t>(127 - 14 + e) << 23) * p.qk_scale, 1.17549435e-38f);
  }
}

// tree_line of each lane's node (-1: no such row), the tree's parents two to a lane.
__device__ __forceinline__ unsigned long long tree_line_warp(const int* parents, int nodes, int node, int first_position) {
  const int lane = threadIdx.x & 31;
  const int lo = lane < nodes ? __ldg(parents + lane) : -2, hi = lane + 32 < nodes ? __ldg(parents + lane + 32) : -2;
  unsigned long long line = 0;
  bool going = node >= 0;
  while (__any_sync(0xffffffffu, going)) {
    const int a = __shfl_sync(0xffffffffu, lo, node & 31), b = __shfl_sync(0xffffffffu, hi, node & 31);
    if (!going) continue;
    const int parent = node < 32 ? a : b;
    line |= 1ull << node;
    const bool absent = first_position + node < 0 || parent < -1 || parent >= node;
    if (absent) line = 0;
    going = !absent && parent >= 0;
    node = parent;
  }
  return line;
}

// 4 x 4 transpose of 16-byte pieces over four neighbouring lanes: v[k] becomes
// piece (lane & 3) of the k-th of them.
__device__ __forceinline__ void transpose_quad(uint4* v) {
  const bool odd = threadIdx.x & 1, upper = threadIdx.x & 2;
  auto swap = [](uint4& a, uint4& b, bool low, int off) {  // the one that this lane does not keep
    uint4 x = low ? a : b;
    x.x = __shfl_xor_sync(0xffffffffu, x.x, off);
    x.y = __shfl_xor_sync(0xffffffffu, x.y, off);
    x.z = __shfl_xor_sync(0xffffffffu, x.z, off);
    x.w = __shfl_xor_sync(0xffffffffu, x.w, off);
    if (low) a = x;
    else b = x;
  };
  swap(v[0], v[1], odd, 1);
  swap(v[2], v[3], odd, 1);
  swap(v[0], v[2], upper, 2);
  swap(v[1], v[3], upper, 2);
}

template <int D>
__device__ __forceinline__ void run_softmax(int g, uint8_t* smem, uint32_t tmem, Segments seg, const Bars& b, Notes& notes,
                                            const DecodeParams& p) {
  using C = Cfg<D>;
  const int lane = threadIdx.x & 31, quad = (threadIdx.x >> 5) & 3, row = quad * 32 + lane;
  const uint32_t lane_off = static_cast<uint32_t>(quad * 32) << 16;
  const uint32_t tS = tmem + lane_off + C::kTmemS + g * C::kTmemGroup, tP = tmem + lane_off + C::kTmemP + g * C::kTmemGroup;
  const uint32_t tO = tmem + lane_off + C::kTmemO;  // warpgroup 0's; 1's kTmemGroup further on
  bool ok = true;
  uint32_t c = 0, uses = 0, items = 0, done[2] = {0, 0}, number = 0;
  auto wait_voted = [&](uint32_t bar, uint32_t parity) { ok = ok && wait(bar, parity, b, p); };
  auto arrive = [&](uint32_t bar) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
  };
  seg.skip_empty(p);
  auto load = [&](const Segments& at) {
    load_q<D>(g * 4 + quad, smem, at, notes, p);
    fence_proxy_async_smem();
    arrive(b.q_full());
  };
  if (seg.left > 0 && seg.data() > 0) load(seg);
#pragma unroll 1
  while (seg.left > 0 && ok) {
    const int n = seg.data();
    const int h = seg.item / p.row_tiles, r0 = (seg.item - h * p.row_tiles) * kRows;
    const bool live = r0 + quad * 32 < p.Lq * p.G;  // the warp has rows
    float m = kNone, l = 0.f, factor = 1.f;
    unsigned long long line = 0;
    if (live) {
      const int node = (r0 + row) / p.G;
      line = tree_line_warp(p.parents + static_cast<long long>(seg.s) * p.Lq, p.Lq, node < p.Lq ? node : -1, seg.len - p.Lq);
    }
    if (n > 0) {
      wait_voted(b.q_full(), number & 1u);
      if (!ok) break;
      factor = notes.factor[row];
    }
    int mine[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) mine[i] = (n + (static_cast<int>(c & 1u) == i ? 1 : 0)) / 2;
    const int first = seg.t0 + (static_cast<int>(c & 1u) == g ? 0 : 1);  // this warpgroup's tiles: every other one
    const int prefix = seg.len - p.Lq;
    const uint64_t f2 = f2_pack(factor, factor);
#pragma unroll 1
    for (int i = 0; i < (g ? mine[1] : mine[0]) && ok; ++i) {
      const int t = first + 2 * i;
      wait_voted(b.s_full(g), uses & 1u);
      if (!ok) break;
      ++uses;
      if (live) {
        tc_fence_after_sync();
        const volatile uint32_t* refusals = notes.skip[(c + static_cast<uint32_t>(t - seg.t0)) & 3u];
        const uint32_t skip_lo = refusals[0], skip_hi = refusals[1];
        const bool masked = (t + 1) * kKeys > prefix || (skip_lo | skip_hi) != 0;
        // Half of the tile at a time, in a loop: code that the instruction cache
        // holds beside the other warps'.  (Where P lies over S, its columns go over
        // some read before.)
        float sum = 0.f;
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          // Against the present reference first: a sum within f16's range holds no P
          // above it.  Else the half's maximum is found, the reference moved, and P
          // taken again (an item's first tile, and later hardly ever).
          uint32_t pk[32];
          uint64_t sum2;
          bool again = false;
#pragma unroll 1
          for (;;) {
            uint32_t x[64];
            tmem_ld64_wait(tS + half * 64, x);
            if (masked) {
              // bit e: the row sees key 64 half + e
              const int node0 = t * kKeys + half * 64 - prefix;
              unsigned long long v = node0 >= 64 ? 0ull : node0 >= 0 ? line >> node0
                                     : node0 <= -64 ? ~0ull : (line << -node0) | ((1ull << -node0) - 1ull);
              const uint32_t refused = half ? skip_hi : skip_lo;
#pragma unroll
              for (int q = 0; q < 4; ++q)
                if (refused >> (8 * q) & 1u) v &= ~(0xffffull << (16 * q));
              const uint32_t lo = static_cast<uint32_t>(v), hi = static_cast<uint32_t>(v >> 32);
#pragma unroll
              for (int e = 0; e < 32; ++e) {
                if (!(lo >> e & 1u)) x[e] = __float_as_uint(-INFINITY);
                if (!(hi >> e & 1u)) x[32 + e] = __float_as_uint(-INFINITY);
              }
            }
            if (again) {
              float top[4];
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                top[q] = fmaxf(__uint_as_float(x[16 * q]), __uint_as_float(x[16 * q + 1]));
#pragma unroll
                for (int e = 2; e < 16; e += 2) top[q] = fmax3(top[q], __uint_as_float(x[16 * q + e]), __uint_as_float(x[16 * q + e + 1]));
              }
              const float most = fmaxf(fmax3(top[0], top[1], top[2]), top[3]) * factor;  // factor > 0: the maximum commutes with it
              const float to = fmaxf(m, most - kLift);
              const float alpha = to == m ? 1.f : ex2_approx(m - to);  // 0 from kNone
              m = to;
              l *= alpha;
              sum *= alpha;
              // what was summed with the old reference is brought to the new:
              if (i > 0) {  // O, whose last product was done before S was,
                const uint32_t own = tO + g * C::kTmemGroup;
#pragma unroll 1
                for (int e = 0; e < D / 16; ++e) {
                  uint32_t o[16];
                  tmem_ld16_wait(own + e * 16, o);
#pragma unroll
                  for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
                  tmem_st16(own + e * 16, o);
                }
              }
              if (half > 0) {  // and P of the first half
                tmem_st_wait();
#pragma unroll 1
                for (int e = 0; e < 2; ++e) {
                  uint32_t o[16];
                  tmem_ld16_wait(tP + e * 16, o);
#pragma unroll
                  for (int k = 0; k < 16; ++k) {
                    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&o[k]));
                    o[k] = pack_f16x2(f.x * alpha, f.y * alpha);
                  }
                  tmem_st16(tP + e * 16, o);
                }
              }
            }
            const uint64_t neg_m2 = f2_pack(-m, -m);
            sum2 = f2_pack(0.f, 0.f);
#pragma unroll
            for (int k = 0; k < 32; ++k) {
              float a, d;
              f2_unpack(f2_fma(f2_pack(__uint_as_float(x[2 * k]), __uint_as_float(x[2 * k + 1])), f2, neg_m2), a, d);
              a = ex2_approx(a);
              d = ex2_approx(d);
              sum2 = f2_add(sum2, f2_pack(a, d));
              pk[k] = pack_f16x2(a, d);
            }
            if (again) break;
            float sa, sb;
            f2_unpack(sum2, sa, sb);
            again = __any_sync(0xffffffffu, sa + sb > 65504.f);
            if (!again) break;
          }
          tmem_st32(tP + half * 32, pk);
          float sa, sb;
          f2_unpack(sum2, sa, sb);
          sum += sa + sb;
        }
        l += sum;
        tmem_st_wait();
        tc_fence_before_sync();
      }
      arrive(b.p_ready(g));
    }
    if (!ok) break;
    c += n;
    // both warpgroups' scores of this item are done with: Q may change
    notes.ml[g][row] = make_float2(m, l);
    arrive(b.states());
    wait_voted(b.states(), items & 1u);
    if (!ok) break;
    const float2 other = notes.ml[g ^ 1][row];
    const Segments was = seg;
    seg.next(p);
    seg.skip_empty(p);
    if (seg.left > 0 && seg.data() > 0) load(seg);

    // The item's output: this warpgroup writes half of the columns.
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (mine[i] > 0) {
        wait_voted(b.o_done(i), done[i] & 1u);
        ++done[i];
      }
    if (!ok) break;
    if (live) {
      tc_fence_after_sync();
      const bool whole = was.whole(), none = n == 0 || line == 0;
      const float M = none ? kNone : fmaxf(m, other.x);
      const float f_own = ex2_approx(m - M), f_other = ex2_approx(other.x - M);
      const float L = none ? 0.f : fmaf(l, f_own, other.y * f_other);
      const float inv = !whole ? 1.f : L == 0.f ? 0.f : p.v_scale / L;
      float f[2];
      f[0] = none ? 0.f : (g ? f_other : f_own) * inv, f[1] = none ? 0.f : (g ? f_own : f_other) * inv;
      const RowPlace rp = row_place(was.s, was.item, row, kRows, p);
      const uint32_t slot = number & 3u;
      const bool any_nan = n > 0 && *reinterpret_cast<volatile uint32_t*>(&notes.any_nan[slot]) == number + 1;
      uint32_t bad = 0;  // blocks that are NaN at a node that this row sees
      if (any_nan) {
        for (int j = 0; j < p.Lq; ++j) {
          const uint32_t note = notes.nan[slot][j];
          if ((line >> j & 1ull) && note >> 8 == (number & 0xffffffu)) bad |= note & 0xffu;
        }
      }
      const long long part_row = (2ll * blockIdx.x + (was.t0 > 0 ? 0 : 1)) * kRows + row;
      // where this row's piece of 16 bytes goes, and, from the lanes that hold them, the quad's four rows'
      constexpr int kHalf = D / 2;
      uint8_t* mine_at = whole ? reinterpret_cast<uint8_t*>(p.o + (rp.token * p.Hq + rp.head) * D + g * kHalf)
                               : reinterpret_cast<uint8_t*>(p.part_o + part_row * D + g * kHalf);
      if (!rp.store) mine_at = nullptr;
      uint8_t* at[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        at[k] = reinterpret_cast<uint8_t*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(mine_at), (lane & ~3) | k));
      const int piece = (lane & 3) * 16;
      auto columns = [&](int col, float* o) {  // 16 of them, from column `col` of the half on
        uint32_t x[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) o[k] = 0.f;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (mine[i] == 0) continue;  // the same for the warp
          tmem_ld16_wait(tO + i * C::kTmemGroup + g * kHalf + col, x);
          if (f[i] != 0.f) {
#pragma unroll
            for (int k = 0; k < 16; ++k) o[k] = fmaf(__uint_as_float(x[k]), f[i], o[k]);
          }
        }
        if (bad >> ((g * kHalf + col) / 16) & 1u) {
#pragma unroll
          for (int k = 0; k < 16; ++k) o[k] = __uint_as_float(0x7fffffffu);
        }
      };
      // 64 bytes of a row at a time, transposed within the quad so that four lanes store them together
#pragma unroll 1
      for (int e = 0; e < (whole ? kHalf / 32 : kHalf / 16); ++e) {
        uint4 v[4];
        if (whole) {
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            float o[16];
            columns(e * 32 + half * 16, o);
            v[2 * half] = make_uint4(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]), pack_bf16x2(o[4], o[5]), pack_bf16x2(o[6], o[7]));
            v[2 * half + 1] = make_uint4(pack_bf16x2(o[8], o[9]), pack_bf16x2(o[10], o[11]), pack_bf16x2(o[12], o[13]),
                                         pack_bf16x2(o[14], o[15]));
          }
        } else {
          float o[16];
          columns(e * 16, o);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            v[k] = make_uint4(__float_as_uint(o[4 * k]), __float_as_uint(o[4 * k + 1]), __float_as_uint(o[4 * k + 2]),
                              __float_as_uint(o[4 * k + 3]));
        }
        transpose_quad(v);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (at[k] != nullptr) *reinterpret_cast<uint4*>(at[k] + e * 64 + piece) = v[k];
      }
      if (g == 0 && rp.store) {
        if (whole) p.lse[static_cast<long long>(rp.head) * p.n_seqs * p.Lq + rp.token] = (M + log2f(L)) * 0.69314718055994531f;
        else p.part_ml[part_row] = make_float2(M, L);
      }
    }
    if (n > 0) ++number;
    ++items;
    // the other warpgroup has read this one's O and state, too
    tc_fence_before_sync();
    arrive(b.written());
    wait_voted(b.written(), (items - 1) & 1u);
  }
}

// ---------------------------------------------------------------------------
// Kernel
// ---------------------------------------------------------------------------
template <int D>
__global__ void __launch_bounds__(kThreads, 1) tree_kernel(const DecodeParams p) {
  using C = Cfg<D>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Notes notes;
  __shared__ long long s_sums[kThreads / 32];
  __shared__ Segments s_seg;
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sbase = smem_u32(smem);
  const int warp = threadIdx.x >> 5;

  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kMiscOff);
  const Bars b{sbase + C::kBarOff, reinterpret_cast<volatile int*>(smem + C::kMiscOff + 4)};
  if (threadIdx.x == 0) s_seg.left = 0;
  if (threadIdx.x == 18 * 32) {
    for (int i = 0; i < C::kRing; ++i) {
      mbar_init(b.raw(i), 1);
      mbar_init(b.raw_empty(i), kTurnWarps);
    }
    for (int g = 0; g < 2; ++g) {
      mbar_init(b.k_full(g), kTurnWarps / 2);
      mbar_init(b.v_full(g), kTurnWarps / 2);
      mbar_init(b.k_empty(g), 1);
      mbar_init(b.v_empty(g), 1);
      mbar_init(b.s_full(g), 1);
      mbar_init(b.p_ready(g), 4);
      mbar_init(b.o_done(g), 1);
    }
    mbar_init(b.q_full(), 8);
    mbar_init(b.states(), 8);
    mbar_init(b.written(), 8);
    mbar_init(b.drain(), 1);
    *b.abort_flag = 0;
    for (int i = 0; i < 4; ++i) notes.any_nan[i] = 0;
    fence_barrier_init();
  }
  if (threadIdx.x >= 256 && threadIdx.x < 256 + 4 * kMaxTreeNodes) notes.nan[(threadIdx.x - 256) / kMaxTreeNodes][threadIdx.x % kMaxTreeNodes] = 0xffffffffu;
  if (warp == 16) {
    tmem_alloc(smem_u32(tmem_slot), kTmemCols);
    tmem_relinquish_alloc_permit();
  }

  // This CTA's range of the concatenated items' cost.
  const int items = p.Hkv * p.row_tiles;  // of a sequence
  if (p.split) {
    if (threadIdx.x == 0) p.cuts[blockIdx.x].s = -1;
    const int per = (p.n_seqs + kThreads - 1) / kThreads;
    const int lo = min(static_cast<int>(threadIdx.x) * per, p.n_seqs), hi = min(lo + per, p.n_seqs);
    long long mine = 0, total;
    for (int s = lo; s < hi; ++s) mine += tile_cost(tokens_of(s, p));
    const long long before = block_scan<kThreads / 32>(mine, s_sums, total);
    const long long all = total * items;
    const long long ctas = min(static_cast<long long>(gridDim.x), (all + kMinTiles - 1) / kMinTiles);
    const long long c = blockIdx.x;
    auto share = [&](long long i) {  // all * i / ctas; a 64-bit division takes a few hundred cycles
      const long long x = all * i;
      return x <= 0xffffffffll ? static_cast<long long>(static_cast<uint32_t>(x) / static_cast<uint32_t>(ctas)) : x / ctas;
    };
    const long long begin = c < ctas ? share(c) : all;
    const int n = c < ctas ? static_cast<int>(min(share(c + 1) - begin, 0x7fffffffll)) : 0;
    if (n > 0 && begin >= before * items && begin < (before + mine) * items) {  // this thread's sequences hold the range's start
      long long at = begin - before * items;
      Segments w;
      w.s = lo;
      int cost;
      for (;; ++w.s) {
        w.len = tokens_of(w.s, p);
        cost = tile_cost(w.len);
        if (at < static_cast<long long>(cost) * items) break;
        at -= static_cast<long long>(cost) * items;
      }
      w.tiles = tiles_of(w.len);
      w.left = n;
      w.item = at <= 0x7fffffffll ? static_cast<int>(at) / cost : static_cast<int>(at / cost);
      const int in_item = static_cast<int>(at - static_cast<long long>(w.item) * cost);
      w.set(in_item);
      s_seg = w;
      if (w.t0 > 0) {
        // the range starts within an item: is this the item's first cut?
        const long long a = begin - in_item;  // its start
        if (share(c - 1) <= a + kItemTiles)
          p.cuts[c] = Cut{w.s, w.item, static_cast<int>(c - 1), static_cast<int>(((a + cost) * ctas + all - 1) / all - 1)};
      }
    }
  } else if (threadIdx.x == 0) {
    // short items: CTA i takes item i whole
    Segments w;
    w.s = blockIdx.x / items;
    w.item = static_cast<int>(blockIdx.x) - w.s * items;
    w.len = tokens_of(w.s, p);
    w.tiles = tiles_of(w.len);
    w.left = w.tiles + kItemTiles;
    w.set(0);
    s_seg = w;
  }
  if (p.errors && blockIdx.x == 0) {
    for (int s = threadIdx.x; s < p.n_seqs; s += kThreads)
      if (p.seq_lens[s] != tokens_of(s, p)) atomicOr(p.errors, kErrPosition);
    for (int i = threadIdx.x; i < p.n_seqs * p.Lq; i += kThreads)
      if (p.parents[i] >= i % p.Lq) atomicOr(p.errors, kErrTree);
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const uint32_t tmem = *tmem_slot;

  if (warp < 8) {
    setmaxnreg_inc<kRegsSoftmax>();
    run_softmax<D>(warp >> 2, smem, tmem, s_seg, b, notes, p);
  } else if (warp < 16) {
    setmaxnreg_dec<kRegsTurn>();
    run_turn<D>(warp - 8, smem, s_seg, b, notes, p);
  } else {
    setmaxnreg_dec<kRegsIssue>();
    if (warp == 16 && (threadIdx.x & 31) == 0) run_issue<D>(sbase, tmem, s_seg, b, p);
    else if (warp == 17) run_load<D>(sbase, s_seg, b, notes, p);
  }
  __syncwarp();
  tc_fence_before_sync();
  __syncthreads();
  if (warp == 16) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, kTmemCols);
  }
}

}  // namespace tree
}  // namespace kv4
}  // namespace fa
