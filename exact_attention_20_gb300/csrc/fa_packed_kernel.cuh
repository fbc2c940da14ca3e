// Attention over packed prompts for sm_103a: sequences of different lengths
// one after another in [T][heads][d] tensors, with grouped heads.
//
// For token t of a sequence of L tokens and query head h (KV head h / G)
//
//     O[t,h] = sum_j softmax_j(scale q[t,h] . k[j,h/G]) v[j,h/G],
//
// j over the sequence's tokens, up to t under the causal mask; L[h,t] is the
// logsumexp.  The tile pipeline is the one of fa_fwd_kernel.cuh (two 128-row
// query tiles per CTA, S and O in tensor memory, one softmax warpgroup per
// tile, two MMA issuers taking turns); what differs is what a tile is and how
// work is divided:
//
// - A query tile holds all G query heads of one KV head for floor(128 / G)
//   tokens, token after token (row = token * G + head).  The heads of a group
//   share every K/V tile, so a K/V tile read once serves 256 rows whatever G
//   is, and a short prompt fills G times as many rows as it has tokens.  G
//   need not divide 128: the tile's last rows then stay unused.
// - A work item is two such tiles, 2 floor(128 / G) tokens of one (sequence,
//   KV head).  Where there are more items than CTAs and none is long, the host
//   sorts them by length and deals them out; else it cuts the concatenated
//   items into ranges of equal cost, one per CTA, as for the dense forward,
//   and an item cut between CTAs is computed in parts that meet in a workspace.
// - K/V tiles start at their sequence's first token, wherever that lies in
//   the packed tensors (the token is an outer TMA coordinate, so any start is
//   fine).  The last tile runs past the item's visible keys, into later
//   tokens, the next sequence or rows behind the last one.  Their scores are
//   replaced by -inf; P is 0 there, but 0 * NaN is NaN: the V rows past the
//   item's last visible key are zeroed in shared memory, and a row that comes
//   out NaN under the mask is looked at again (mend_rows).  That is slow: where
//   the last of 131072 tokens alone has a NaN, the 127 rows before it take 0.55
//   s, with finite values the whole prompt of one head 3 ms.
//
// Warps: 0-7 softmax, one row a thread; 8 TMA; 9 and 10 MMA; 11 dispatcher.
// Measured on a GB300: 16384 tokens, 2 KV heads of 8 query heads, d = 128,
// causal, 735 us: 1495 TFLOP/s of visible products, 78 % of cuBLAS' bf16
// rate; 24 prompts of 40 to 1901 tokens, 32 / 8 heads, 118 us (55 at that
// rate; two products of 256 rows and the softmax between them are 1.6 us a
// step, an item's start and end 3.5 us).  What bounds long prompts is the
// turn from S to P and back in a tile's softmax warps: the tensor pipe is
// active 62 % of the time, issue slots are 47 % used.  Without a mask at d =
// 64, 8 x 1024 tokens of 16 heads take 60 us: 134 M exponentials, 27 us of
// the MUFU's rate, in 3.4 rounds of items that cost four.
#pragma once

#include <type_traits>

#include "fa_fwd_kernel.cuh"

namespace fa {
namespace packed {

constexpr int kMaxCtas = 160;         // one CTA per SM
constexpr int kMaxSeqs = 1024;        // sequences of one launch
constexpr int kMaxPairs = 2048;       // (sequence, block) pairs of a dealt launch
constexpr int kMaxParts = 8;          // parts of one split item
constexpr int kCountersPerItem = 8;   // per query tile and warp quadrant
constexpr int kItemsAhead = 4;        // items that the dispatcher has written and not all warps read
constexpr int kSitePacked = 6;        // status code: a wait gave up

// Shared memory: Q tiles, the K/V ring, and (d = 128) 4 KB a softmax warp to
// bring output rows into whole 128-byte lines.  At d = 128 that takes the place of
// the dense forward's fifth ring stage, which costs prompts of any length
// less than 1 %, while lane-by-lane rows (32 lines touched by each store) held
// an item up by 1.0 us of its 1.9 us per step plus 3 us.
template <int D>
struct PackedCfg {
  static constexpr int kSlabs = Cfg<D>::kSlabs, kTileBytes = Cfg<D>::kTileBytes;
  static constexpr int kQkInstr = Cfg<D>::kQkInstr, kPvInstr = Cfg<D>::kPvInstr;
  static constexpr int kStages = D == 128 ? 4 : 9;
  // P in two halves: the product with V's first 64 keys starts while the other
  // half's exponentials are taken.  8 x 1024 tokens of 16 heads at d = 64 without
  // a mask: 59 us, 62 in one piece (both with P over S, below; with P beside it
  // 60).  At d = 128, where the tensor core has twice
  // the work, an issuer that holds its turn between the halves is in the other's
  // way: 16384 tokens 823 us, 744 in one piece.
  static constexpr bool kHalves = D == 64;
  // Tensor memory columns of query tile 0, tile 1's 128 further on.  At d = 64
  // P has the columns that O leaves free: no product writes where another, not
  // known to be done, still reads.  At d = 128 there are none, and P lies over
  // S, as in the dense forward: the next S is issued behind the P V that reads
  // P by the same thread, and of the same shape, which keeps their order.
  static constexpr int kTmemS = 0, kTmemO = 256, kTmemP = D == 64 ? kTmemO + D : kTmemS;
  static constexpr int kTmemTile = 128;
  static_assert(kTmemP == kTmemS || (kTmemO + D <= kTmemP && kTmemP + kBlockN / 2 <= kTmemO + kTmemTile), "P's columns");
  static constexpr int kQOff = 0;
  static constexpr int kKVOff = kQTiles * kTileBytes;
  static constexpr int kOutOff = kKVOff + kStages * kTileBytes;
  static constexpr int kWarpOut = 32 * 128;
  static constexpr int kBarOff = kOutOff + (D == 128 ? 8 * kWarpOut : 0);
  static constexpr int kNumBars = 2 * 2 + 2 * kStages + 2 * 5 + 1 + 2 + 2 * kItemsAhead;
  static constexpr int kMiscOff = kBarOff + (kNumBars * 8 + 15) / 16 * 16;
  static constexpr int kItemsOff = kMiscOff + 16;
  static constexpr int kSmemBytes = kItemsOff + kItemsAhead * 64 + 1024;  // + alignment slack
  static_assert(kSmemBytes <= 232448, "227 KB");
};

// The kernel's shared memory, from the first 1024-byte boundary on.
__device__ __forceinline__ uint8_t* shared_base() {
  extern __shared__ uint8_t smem_raw[];
  return smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
}

// One part of a split item: its workspace slot, the item's first slot and
// number of parts (consecutive slots), and the item's counters.  slot < 0:
// the chunk is the whole item.
struct Part {
  int slot, slot0, count, k;
};

// A CTA's share: n_items consecutive items from (s, h, b), the first from
// step_begin, the last up to step_end (a step is one 128-key tile).
struct Range {
  int s, h, b;
  int n_items, step_begin, step_end;
  Part first, last;
};

// A dealt launch's item, for every KV head.
struct Pair {
  uint16_t s, b;
};

struct Params {
  __nv_bfloat16* o;   // [T][Hq][D]
  float* lse;         // [Hq][T]
  int* status;        // device status word (0 = ok)
  float* part_o;      // workspace: [slot][256 rows] of D fp32, a part's O normalised within it
  float* part_lse;    // workspace: [slot][256], the part's natural-log logsumexp
  int* counters;      // workspace: part arrivals, zero when the launch starts
  const __nv_bfloat16 *q, *k, *v;  // for mend_rows alone; token strides below
  long long q_stride, k_stride, v_stride;
  int T, Hq, Hkv, G;
  int tpt;            // tokens of a query tile: floor(128 / G)
  float qk_scale;     // scale * log2(e)
  unsigned long long wait_limit_ns;
  int cu[kMaxSeqs + 1];  // first token of each sequence, and the end of the last
  int dealt;          // items of a dealt launch, whose pairs are by length, longest first; 0: ranges
  union {
    Range range[kMaxCtas];
    Pair pair[kMaxPairs];
  };
};

// Key tiles that query tile t of block b visits (0 past the sequence's end).
template <bool CAUSAL>
__host__ __device__ __forceinline__ int tiles_for(int b, int t, int len, int tpt) {
  const int t0 = (2 * b + t) * tpt;
  if (t0 >= len) return 0;
  const int last = CAUSAL ? (t0 + tpt < len ? t0 + tpt : len) - 1 : len - 1;
  return last / kBlockN + 1;
}

// Steps of an item: the key tiles its longer query tile visits (under the
// mask the later one, where it has tokens).
template <bool CAUSAL>
__host__ __device__ __forceinline__ int item_steps(int b, int len, int tpt) {
  const int a = tiles_for<CAUSAL>(b, 0, len, tpt), c = tiles_for<CAUSAL>(b, 1, len, tpt);
  return a > c ? a : c;
}

// A CTA's i-th item among those dealt: one of each row of gridDim.x items, in
// the rows' order back and forth, so that who got a row's longest item gets
// the next row's shortest.  The pair's KV heads follow one another.
__device__ __forceinline__ int dealt_at(int i) {
  return i * gridDim.x + (i & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
}

__device__ __forceinline__ bool has_item(int i, const Params& p) {
  return p.dealt > 0 ? dealt_at(i) < p.dealt : i < p.range[blockIdx.x].n_items;
}

// The items of a CTA in turn.
struct Cursor {
  int s, h, b;
  int begin, len;  // the sequence's first token and length
  __device__ __forceinline__ void at(const Params& p) {
    begin = p.cu[s];
    len = p.cu[s + 1] - begin;
  }
  __device__ __forceinline__ explicit Cursor(const Params& p) {
    if (p.dealt > 0) {
      deal(0, p);
    } else {
      const Range& r = p.range[blockIdx.x];
      s = r.s, h = r.h, b = r.b;
      at(p);
    }
  }
  __device__ __forceinline__ void deal(int i, const Params& p) {
    const int item = dealt_at(i), n = item / p.Hkv;
    s = p.pair[n].s, h = item - n * p.Hkv, b = p.pair[n].b;
    at(p);
  }
  __device__ __forceinline__ void next(int i, const Params& p) {  // to item i, from the one before
    if (p.dealt > 0) return deal(i, p);
    if (++b * 2 * p.tpt < len) return;
    b = 0;
    if (++h < p.Hkv) return;
    h = 0;
    do {  // sequences without tokens have no items
      ++s;
      at(p);
    } while (len == 0);
  }
};

// What the warps read of an item, or of the part of it that is this CTA's.
struct alignas(16) Item {
  int begin, len, h, b;  // the sequence's first token and length, the KV head, the block
  int kb, ke, steps;     // key tiles [kb, ke) of `steps`
  int more;              // whether another item follows
  int ne[2];             // the key tiles that query tile t visits here: [kb, ne)
  int plain[2];          // those before this one need no mask
  int seen[2];           // keys that some row of query tile t sees
  int visible;           // keys of the item's last tile that some row sees
  int i;                 // the CTA's items before this one
  __device__ __forceinline__ bool whole() const { return kb == 0 && ke == steps; }
};
static_assert(sizeof(Item) == 64, "kItemsOff");

struct PackedSync : Sync {
  uint32_t p_half[2];  // kHalves: as p_ready, for P's first 64 keys
  uint32_t item_full0, item_empty0;
  const Item* items;
};

// When a warp was last seen in mend_rows; beside the abort flag.
__device__ __forceinline__ volatile unsigned long long* alive_word(volatile int* abort_flag) {
  return reinterpret_cast<volatile unsigned long long*>(abort_flag + 1);
}

// Bounded wait, as the dense forward's.  A warp in mend_rows, which only the
// mask needs, holds the others up for as long as its keys take: its last sign
// of life counts.  (Without a mask that check alone, never reached, cost 8192
// tokens 4 %.)
template <bool CAUSAL>
__device__ __forceinline__ bool wait_phase(uint32_t bar, uint32_t parity, const PackedSync& sy, const Params& p,
                                           unsigned long long more_ns = 0) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_timer_ns();
  uint32_t polls = 0;
  while (true) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((++polls & 31u) == 0u) {
      if (*sy.abort_flag) return false;
      uint64_t since = t0;
      if constexpr (CAUSAL) {
        const uint64_t alive = *alive_word(sy.abort_flag);  // read before the clock
        if (alive > since) since = alive;
      }
      if (global_timer_ns() - since > p.wait_limit_ns + more_ns) {
        *sy.abort_flag = 1;
        atomicCAS(p.status, 0, kSitePacked);
        return false;
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Dispatcher (one thread)
// ---------------------------------------------------------------------------
// Writes the CTA's items into a ring that all other warps read.  With each
// warp finding its own way (registers that the issuers and the softmax lack,
// and waits for parameters between items) a prompt of 16384 tokens took 753 us
// instead of 745, 24 ragged prompts 125 instead of 121.
template <bool CAUSAL>
__device__ __forceinline__ void run_dispatcher(Item* items, const PackedSync& sy, const Params& p) {
  Cursor c(p);
  const Range& r = p.range[blockIdx.x];  // read where the launch is not dealt
  unsigned long long steps = 0;          // of all items so far
  for (int i = 0;; ++i) {
    if (i > 0) c.next(i, p);
    Item it;
    it.begin = c.begin, it.len = c.len, it.h = c.h, it.b = c.b;
    it.steps = item_steps<CAUSAL>(c.b, c.len, p.tpt);
    it.more = has_item(i + 1, p);
    it.kb = p.dealt == 0 && i == 0 ? r.step_begin : 0;
    it.ke = p.dealt == 0 && !it.more ? r.step_end : it.steps;
    it.i = i;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      it.ne[t] = min(it.ke, tiles_for<CAUSAL>(c.b, t, c.len, p.tpt));
      it.seen[t] = CAUSAL ? min((2 * c.b + t + 1) * p.tpt, c.len) : c.len;
      // the first tile with a key that some row does not see
      const int masked = (CAUSAL ? min((2 * c.b + t) * p.tpt + 1, c.len) : c.len) / kBlockN;
      it.plain[t] = min(it.ne[t], masked);
    }
    it.visible = it.seen[1] - (it.steps - 1) * kBlockN;
    // free once the item kItemsAhead before is done; a step takes far less than 16 us
    const uint32_t n = i % kItemsAhead;
    if (!wait_phase<CAUSAL>(sy.item_empty0 + 8 * n, ((i / kItemsAhead) & 1u) ^ 1u, sy, p, steps << 14)) return;
    items[n] = it;
    mbar_arrive(sy.item_full0 + 8 * n);
    if (!it.more) return;
    steps += it.steps;
  }
}

// ---------------------------------------------------------------------------
// TMA producer (one thread)
// ---------------------------------------------------------------------------
template <int D, bool CAUSAL>
__device__ __forceinline__ void run_producer(const CUtensorMap* tmQ, const CUtensorMap* tmK, const CUtensorMap* tmV,
                                             uint32_t sbase, const PackedSync& sy, const Params& p) {
  using C = PackedCfg<D>;
  uint32_t q_loads[2] = {0, 0};
  uint32_t kv_count = 0;
  const uint64_t pol_q = l2_policy_evict_first();
  const uint64_t pol_kv = l2_policy_evict_last();
  const uint32_t q_bytes = static_cast<uint32_t>(p.G * p.tpt) * D * 2;
  bool ok = true;
  bool more = true;
  for (uint32_t i = 0; more && ok; ++i) {
    const uint32_t n = i % kItemsAhead;
    ok = wait_phase<CAUSAL>(sy.item_full0 + 8 * n, (i / kItemsAhead) & 1u, sy, p);
    if (!ok) break;
    const Item it = sy.items[n];
    mbar_arrive(sy.item_empty0 + 8 * n);
    more = it.more;
    for (int t = 0; t < kQTiles; ++t) {
      if (it.ne[t] <= it.kb) continue;  // no key tile of its own here
      ok = wait_phase<CAUSAL>(sy.q_empty[t], (q_loads[t] & 1u) ^ 1u, sy, p);
      if (!ok) break;
      ++q_loads[t];
      mbar_arrive_expect_tx(sy.q_full[t], q_bytes);
      const uint32_t dst = sbase + C::kQOff + t * C::kTileBytes;
      const int token = it.begin + (2 * it.b + t) * p.tpt;
#pragma unroll
      for (int s = 0; s < C::kSlabs; ++s)
        tma_load_3d_hint(dst + s * kSlabBytes, tmQ, sy.q_full[t], s * 64, it.h * p.G, token, pol_q);
    }
    for (int j = it.kb; j < it.ke && ok; ++j) {
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        if (!ok) break;
        const uint32_t slot = kv_count % C::kStages;
        ok = wait_phase<CAUSAL>(sy.kv_empty0 + 8 * slot, ((kv_count / C::kStages) & 1u) ^ 1u, sy, p);
        if (!ok) break;
        const uint32_t full = sy.kv_full0 + 8 * slot;
        mbar_arrive_expect_tx(full, C::kTileBytes);
        const uint32_t dst = sbase + C::kKVOff + slot * C::kTileBytes;
#pragma unroll
        for (int s = 0; s < C::kSlabs; ++s)
          tma_load_3d_hint(dst + s * kSlabBytes, n == 0 ? tmK : tmV, full, s * 64, it.h, it.begin + j * kBlockN, pol_kv);
        ++kv_count;
      }
    }
  }
  // Every copy this thread started lands before the CTA exits, also after an abort.
  const uint32_t first = kv_count > (uint32_t)C::kStages ? kv_count - C::kStages : 0;
  for (uint32_t n = first; n < kv_count; ++n)
    mbar_wait_bounded(sy.kv_full0 + 8 * (n % C::kStages), (n / C::kStages) & 1u, p.wait_limit_ns);
  for (int t = 0; t < kQTiles; ++t)
    if (q_loads[t] > 0) mbar_wait_bounded(sy.q_full[t], (q_loads[t] - 1) & 1u, p.wait_limit_ns);
}

// ---------------------------------------------------------------------------
// MMA issuers (one warp per query tile, strict turns, as in the dense forward)
// ---------------------------------------------------------------------------
template <int D, bool CAUSAL>
__device__ __forceinline__ void run_mma(int t, uint8_t* smem, uint32_t sbase, uint32_t tmem, const PackedSync& sy,
                                        const Params& p) {
  using C = PackedCfg<D>;
  const uint32_t bar_q_full = t ? sy.q_full[1] : sy.q_full[0];
  const uint32_t bar_q_empty = t ? sy.q_empty[1] : sy.q_empty[0];
  const uint32_t bar_s_full = t ? sy.s_full[1] : sy.s_full[0];
  const uint32_t bar_p_ready = t ? sy.p_ready[1] : sy.p_ready[0];
  const uint32_t bar_p_half = t ? sy.p_half[1] : sy.p_half[0];
  const uint32_t bar_o_done = t ? sy.o_done[1] : sy.o_done[0];
  const uint32_t bar_o_free = t ? sy.o_free[1] : sy.o_free[0];
  const uint32_t my_turn = t ? sy.turn[1] : sy.turn[0];
  const uint32_t next_turn = t ? sy.turn[0] : sy.turn[1];
  const uint64_t q_desc = sdesc_advance(sdesc_sw128(sbase + C::kQOff, 16, 1024), t * C::kTileBytes);
  const uint64_t k_desc0 = sdesc_sw128(sbase + C::kKVOff, 16, 1024);
  const uint64_t v_desc0 = sdesc_sw128(sbase + C::kKVOff, kSlabBytes, 1024);
  const uint32_t tm_s = tmem + C::kTmemS + t * C::kTmemTile;
  const uint32_t tm_p = tmem + C::kTmemP + t * C::kTmemTile;
  const uint32_t tm_o = tmem + C::kTmemO + t * C::kTmemTile;
  constexpr uint32_t idesc_qk = idesc_bf16_f32(kBlockM, kBlockN, /*b_mn_major=*/false);
  uint32_t q_uses = 0, kv_count = 0, pr_par = 0, of_par = 1, turn_par = 0;
  bool ok = true;
  auto full = [&](uint32_t c) { return sy.kv_full0 + 8 * (c % C::kStages); };
  auto empty = [&](uint32_t c) { return sy.kv_empty0 + 8 * (c % C::kStages); };
  const int lane = threadIdx.x & 31;
  const bool leader = lane == 0;
  auto wait_voted = [&](uint32_t bar, uint32_t par) {
    ok = __all_sync(0xffffffffu, ok && wait_phase<CAUSAL>(bar, par, sy, p));
  };
  // Both issuers wait for every position of the ring, in order: a full
  // barrier's wait is by parity and tells a fill only from the one before.
  auto wait_full = [&](uint32_t c) { wait_voted(full(c), (c / C::kStages) & 1u); };
  auto release_unused = [&](uint32_t c) {  // a K/V tile this query tile skips
    wait_full(c);
    if (ok && leader) mbar_arrive(empty(c));
  };
  if (t == 1 && leader) mbar_arrive(sy.turn[0]);  // tile 0 takes the first turn

  bool more = true;
  for (uint32_t i = 0; more && ok; ++i) {
    const uint32_t slot = i % kItemsAhead;
    wait_voted(sy.item_full0 + 8 * slot, (i / kItemsAhead) & 1u);
    if (!ok) break;
    const Item& it = sy.items[slot];
    // the same in every lane, and said to be: computed with once for the warp (740 us; else 744)
    auto uniform = [&](int x) { return __reduce_max_sync(0xffffffffu, x); };
    more = uniform(it.more);
    const int kb = uniform(it.kb), ke = uniform(it.ke);
    const int ne = uniform(t ? it.ne[1] : it.ne[0]);  // this tile's key tiles: [kb, ne)
    // The item's last V tile, where it is in this chunk: its rows from
    // `visible` on belong to no visible key.  The first issuer that uses the
    // tile zeroes those that the products, 16 keys at a time, still reach (the
    // other is ordered behind it by the turn).
    const int visible = uniform(it.visible);
    const int zero_rows = min(kBlockN, (visible + 15) & ~15) - visible;
    const int zero_at = uniform(ke == it.steps && zero_rows > 0 && (t == 0 || it.ne[0] < ke) ? ke - 1 : -1);
    // keys that some row of this query tile sees: its last tile's products stop there
    const int seen = uniform(t ? it.seen[1] : it.seen[0]);
    __syncwarp();
    if (leader) mbar_arrive(sy.item_empty0 + 8 * slot);
    if (ne > kb) {
      wait_voted(bar_q_full, q_uses & 1u);
      ++q_uses;
    }
    // step s issues O_t += P_t(s-1) V_{s-1} (if kb <= s-1 < ne) and S_t(s) (if s < ne)
    for (int s = kb; s <= ke && ok; ++s) {
      const bool do_pv = s - 1 >= kb && s - 1 < ne;
      const bool do_s = s < ne;
      const uint32_t cv = kv_count + 2 * (s - 1 - kb) + 1;  // V_{s-1}
      const uint32_t ck = kv_count + 2 * (s - kb);          // K_s
      if (do_pv) {
        wait_full(cv);
        if (s - 1 == zero_at && ok) {
          uint8_t* tile = smem + C::kKVOff + (cv % C::kStages) * C::kTileBytes;
#pragma unroll
          for (int slab = 0; slab < C::kSlabs; ++slab)  // whole 128-byte rows, so the swizzle is no matter
            for (int n = lane; n < zero_rows * 8; n += 32)
              *reinterpret_cast<uint4*>(tile + slab * kSlabBytes + visible * 128 + n * 16) = make_uint4(0, 0, 0, 0);
          fence_proxy_async_smem();
          __syncwarp();
        }
      }
      if (do_s) wait_full(ck);
      uint64_t dv[C::kPvInstr], dq[C::kQkInstr], dk[C::kQkInstr];
      {
        const uint64_t v0 = sdesc_advance(v_desc0, (cv % C::kStages) * C::kTileBytes);
        const uint64_t k0 = sdesc_advance(k_desc0, (ck % C::kStages) * C::kTileBytes);
#pragma unroll
        for (int kk = 0; kk < C::kPvInstr; ++kk) dv[kk] = sdesc_advance(v0, kk * 2048);
#pragma unroll
        for (int kk = 0; kk < C::kQkInstr; ++kk) {
          const uint32_t off = (kk / 4) * kSlabBytes + (kk % 4) * 32;
          dq[kk] = sdesc_advance(q_desc, off);
          dk[kk] = sdesc_advance(k0, off);
        }
      }
      const uint32_t acc0 = s > kb + 1 ? 1u : 0u;
      // Groups of 16 keys that P V takes.  (Q K^T always takes all 128: with fewer
      // columns it measured slower, and at d = 128 S and P V have to be of one shape.)
      int groups_pv = min(kBlockN, seen - (s - 1) * kBlockN + 15) / 16;
      // All of it in registers before the turn, which is what the other issuer
      // waits for (16384 tokens: 740 us; computed where it is used: 752).
#pragma unroll
      for (int kk = 0; kk < C::kPvInstr; ++kk) asm volatile("" : "+l"(dv[kk]));
#pragma unroll
      for (int kk = 0; kk < C::kQkInstr; ++kk) asm volatile("" : "+l"(dq[kk]), "+l"(dk[kk]));
      asm volatile("" : "+r"(groups_pv));
      // Which wait is last decides how the two tiles fall into step.  Without a
      // mask at d = 128 the turn is taken before P is waited for: 4 heads of 4,
      // 8192 tokens, 386 us and 397 the other way round; under the mask 16384
      // tokens take 771 us so and 740 the other way round.
      constexpr bool kTurnFirst = !CAUSAL && !C::kHalves;
      if (do_pv && s == kb + 1) {
        wait_voted(bar_o_free, of_par);
        of_par ^= 1u;
      }
      if constexpr (kTurnFirst) wait_voted(my_turn, turn_par);
      if (do_pv) {
        wait_voted(C::kHalves ? bar_p_half : bar_p_ready, pr_par);
        if constexpr (!C::kHalves) pr_par ^= 1u;
      }
      if constexpr (!kTurnFirst) wait_voted(my_turn, turn_par);
      turn_par ^= 1u;
      if (!ok) break;
      tc_fence_after_sync();
      // P V's instructions [FROM, TO), as far as some row sees
      auto issue_pv = [&](auto from, auto to) {
        constexpr int kFrom = decltype(from)::value, kTo = decltype(to)::value;
        constexpr uint32_t idesc_pv = idesc_bf16_f32(kBlockM, D, /*b_mn_major=*/true);
        if (groups_pv >= kTo) {
#pragma unroll
          for (int kk = kFrom; kk < kTo; ++kk) umma_ts(tm_o, tm_p + kk * 8, dv[kk], idesc_pv, kk > 0 ? 1u : acc0);
        } else {
#pragma unroll
          for (int kk = kFrom; kk < kTo - 1; ++kk)
            if (kk < groups_pv) umma_ts(tm_o, tm_p + kk * 8, dv[kk], idesc_pv, kk > 0 ? 1u : acc0);
        }
      };
      using Begin = std::integral_constant<int, 0>;
      using Half = std::integral_constant<int, C::kHalves ? C::kPvInstr / 2 : 0>;
      using End = std::integral_constant<int, C::kPvInstr>;
      if constexpr (C::kHalves) {
        if (do_pv) {
          if (leader) issue_pv(Begin{}, Half{});
          __syncwarp();
          wait_voted(bar_p_ready, pr_par);
          pr_par ^= 1u;
          if (!ok) break;
          tc_fence_after_sync();
        }
      }
      if (leader) {
        if (do_pv) issue_pv(Half{}, End{});
        if (do_s) {
#pragma unroll
          for (int kk = 0; kk < C::kQkInstr; ++kk) umma_ss(tm_s, dq[kk], dk[kk], idesc_qk, kk > 0 ? 1u : 0u);
        }
        mbar_arrive(next_turn);
        if (do_s) umma_commit(bar_s_full);
        if (do_pv && !do_s) umma_commit(bar_o_done);
        if (do_s && s == ne - 1) umma_commit(bar_q_empty);
        if (do_pv) umma_commit(empty(cv));
        if (do_s) umma_commit(empty(ck));
      }
      __syncwarp();
      if (!do_pv && s - 1 >= kb) release_unused(cv);
      if (!do_s && s < ke) release_unused(ck);
    }
    kv_count += 2 * (ke - kb);
  }
  // Every MMA this thread issued must finish before tensor memory is released.
  if (leader) umma_commit(sy.drain);
  __syncwarp();
  mbar_wait_bounded(sy.drain, 0, p.wait_limit_ns);
}

// ---------------------------------------------------------------------------
// Parts of split items
// ---------------------------------------------------------------------------
// A slot holds one part of an item, 256 rows of D fp32 values in groups of
// eight columns, each group with its 256 rows one after the other, so that a
// warp's 32-byte accesses to one group cover 1 KB.
template <int D>
__device__ __forceinline__ size_t part_index(int slot, int row, int group) {
  return static_cast<size_t>(slot) * kItemRows * D + (static_cast<size_t>(group) * kItemRows + row) * 8;
}

// The larger of two values (fp32 bits, or two bf16), NaN where either is.
__device__ __forceinline__ uint32_t max_nan(uint32_t a, uint32_t b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(__uint_as_float(a)), "f"(__uint_as_float(b)));
  return __float_as_uint(r);
}
__device__ __forceinline__ uint32_t max_nan_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ bool is_nan(uint32_t x) { return (x & 0x7fffffffu) > 0x7f800000u; }

// What this warp has of a split item: its state as the end of a chunk left it.
constexpr int kStored = 0;  // in the workspace, like the others
constexpr int kInTmem = 1;  // in tensor memory
constexpr int kEmpty = 2;   // no key tile: nothing anywhere
struct Own {
  int where;    // the same in every lane
  float lse;    // natural-log logsumexp of the part, -inf without keys
  float inv_l;  // the accumulator's factor
  uint32_t tO;  // the accumulator
};

// Merges one warp's 32 rows of a split item through the parts' logsumexps:
// L = ln sum_r exp(L_r), O = sum_r exp(L_r - L) O_r, the largest L_r
// subtracted first; a part without keys for a row has L_r = -inf and weighs 0.
// Every other part's rows are in the workspace.  Parts are added in key
// order, so the result does not depend on who merges.  Returns NaN (fp32 bits)
// where an element of the own part in tensor memory is.
template <int D>
__device__ __forceinline__ uint32_t merge_rows(const Part part, const Own own, int r, bool store, __nv_bfloat16* orow,
                                        float* lse_dst, const float* part_o, const float* part_lse) {
  constexpr float kLog2e = 1.4426950408889634f;
  const int mine = own.where == kStored ? -1 : part.slot - part.slot0;
  const float* lse_in = part_lse + static_cast<size_t>(part.slot0) * kItemRows + r;
  auto lse_of = [&](int i) { return i == mine ? own.lse : __ldcg(lse_in + i * kItemRows); };
  // -inf: no key (m may be -inf too); a row whose scores are NaN stays NaN
  auto weight = [&](float l, float m) { return l == -INFINITY ? 0.f : exp2f((l - m) * kLog2e); };
  float m = -INFINITY;
#pragma unroll 1
  for (int i = 0; i < part.count; ++i) m = fmaxf(m, lse_of(i));
  float sum = 0.f;
#pragma unroll 1
  for (int i = 0; i < part.count; ++i) sum += weight(lse_of(i), m);
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  uint32_t top = 0;
#pragma unroll 1
  for (int c = 0; c < D / 32; ++c) {
    float acc[32];
#pragma unroll
    for (int e = 0; e < 32; ++e) acc[e] = 0.f;
#pragma unroll 1
    for (int i = 0; i < part.count; ++i) {
      if (i == mine && own.where == kEmpty) continue;
      const float w = weight(lse_of(i), m) * inv;
      float x[32];
      if (i == mine) {
        uint32_t o[32];
        tmem_ld32_wait(own.tO + c * 32, o);
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          top = max_nan(top, o[e]);
          x[e] = __uint_as_float(o[e]) * own.inv_l;
        }
      } else {
#pragma unroll
        for (int n = 0; n < 4; ++n) ld_global_cg_v8(part_o + part_index<D>(part.slot0 + i, r, 4 * c + n), x + 8 * n);
      }
      if (w != 0.f) {  // an empty part's rows were never written
#pragma unroll
        for (int e = 0; e < 32; ++e) acc[e] = fmaf(w, x[e], acc[e]);
      }
    }
    if (store) {
      uint4* dst = reinterpret_cast<uint4*>(orow + c * 32);
#pragma unroll
      for (int n = 0; n < 4; ++n)
        dst[n] = make_uint4(pack_bf16x2(acc[8 * n], acc[8 * n + 1]), pack_bf16x2(acc[8 * n + 2], acc[8 * n + 3]),
                            pack_bf16x2(acc[8 * n + 4], acc[8 * n + 5]), pack_bf16x2(acc[8 * n + 6], acc[8 * n + 7]));
    }
  }
  if (store) *lse_dst = m + logf(sum);
  return top;
}

// The warp's arrival for a part whose rows are in the workspace: true for the
// warp that completes the item, which then merges it.
__device__ __forceinline__ bool part_arrive(int* ctr, int count, int lane) {
  __threadfence();
  __syncwarp();
  int old = 0;
  if (lane == 0) old = atomicAdd(ctr, 1);
  if (__shfl_sync(0xffffffffu, old, 0) != count - 1) return false;
  (void)ld_acquire_gpu(ctr);  // every lane: the other parts' rows were fenced before their arrivals
  return true;
}

// A row's place in O and LSE; rows without a query (past the sequence's end,
// or past the G * tpt rows of a tile) are not stored.
struct Row {
  bool store;
  __nv_bfloat16* o;
  float* lse;
  __device__ __forceinline__ Row(int begin, int len, int h, int t0, int row_in_tile, int D, const Params& p) {
    const int in_tile = row_in_tile / p.G, token = t0 + in_tile, head = h * p.G + row_in_tile - in_tile * p.G;
    store = in_tile < p.tpt && token < len;
    o = store ? p.o + (static_cast<size_t>(begin + token) * p.Hq + head) * D : p.o;
    lse = store ? p.lse + static_cast<size_t>(head) * p.T + begin + token : p.lse;
  }
};

// Where a chunk's rows are stored: bf16 rows of O, or fp32 rows of a part.
struct Mend {
  __nv_bfloat16* o;  // the row in O, or null
  float* part;       // the row's first group in the workspace, groups kItemRows * 8 apart
  float m_ref, inv_l;  // inv_l = 0: no visible score above -inf
};

// Rows with NaN among their columns, stored by their warp.  A row without
// weight is 0 whatever V holds: zeros in O; of a part nothing, since the merge
// leaves a part of weight 0 out.  In the others a NaN that comes from keys
// that the row does not see (0 * NaN or 0 * infinity in the product with P) is
// replaced by what the visible keys give.  A column needs that
// where V is not finite at a key behind the row's token within the chunk's
// tiles; its sum over the chunk's visible keys is then taken anew, key by key,
// the warp together on one row.  Only values that are not finite lead here, so
// it is a call: inlined it cost 24 ragged prompts 3 us of 150.
template <int D>
__device__ __noinline__ void mend_rows(uint32_t rows, int lane, int quad, int t0, const Item& c, const Mend mine,
                                       const Params& p) {
  constexpr int kPer = D / 32;  // columns of a lane
  constexpr int kRound = 128;   // keys between signs of life, about 20 us
  const int behind = min(min(2 * (c.b + 1) * p.tpt, c.len), c.ke * kBlockN);  // V rows from here on were zeroed or not read
  volatile unsigned long long* alive = alive_word(reinterpret_cast<volatile int*>(shared_base() + PackedCfg<D>::kMiscOff + 4));
  auto load = [&](const __nv_bfloat16* row, float* x) {
#pragma unroll
    for (int e = 0; e < kPer; ++e) x[e] = __bfloat162float(row[lane * kPer + e]);
  };
  __syncwarp();
  while (rows != 0) {
    const int src = __ffs(rows) - 1;
    rows &= rows - 1;
    const int in_tile = (quad * 32 + src) / p.G, token = t0 + in_tile;
    const int head = c.h * p.G + quad * 32 + src - in_tile * p.G;
    const float m_ref = __shfl_sync(0xffffffffu, mine.m_ref, src), inv_l = __shfl_sync(0xffffffffu, mine.inv_l, src);
    const unsigned long long o = __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(mine.o), src);
    const unsigned long long part = __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(mine.part), src);
    if (inv_l == 0.f) {
#pragma unroll
      for (int e = 0; e < kPer; ++e)
        if (o != 0) reinterpret_cast<__nv_bfloat16*>(o)[lane * kPer + e] = __float2bfloat16_rn(0.f);
      continue;
    }
    const __nv_bfloat16* v = p.v + static_cast<long long>(c.begin) * p.v_stride + c.h * D;
    bool need[kPer] = {};
    for (int key = max(token + 1, c.kb * kBlockN); key < behind; ++key) {
      float x[kPer];
      load(v + key * p.v_stride, x);
#pragma unroll
      for (int e = 0; e < kPer; ++e) need[e] |= !(fabsf(x[e]) < INFINITY);
    }
    bool any = false;
#pragma unroll
    for (int e = 0; e < kPer; ++e) any |= need[e];
    if (!__any_sync(0xffffffffu, any)) continue;
    float q[kPer], acc[kPer];
    load(p.q + (c.begin + token) * p.q_stride + static_cast<long long>(head) * D, q);
#pragma unroll
    for (int e = 0; e < kPer; ++e) acc[e] = 0.f;
    const __nv_bfloat16* k = p.k + static_cast<long long>(c.begin) * p.k_stride + c.h * D;
    const int to = min(token + 1, c.ke * kBlockN);
    // 32 rows over a million keys take a warp seconds: the others wait while it
    // shows that it goes on.  Columns that are NaN from visible keys stay so.
    bool open = true;
    for (int key = c.kb * kBlockN; key < to && __any_sync(0xffffffffu, open);) {
      if (lane == 0) *alive = global_timer_ns();
      const int stop = min(key + kRound, to);
#pragma unroll 4
      for (; key < stop; ++key) {
        float x[kPer], y[kPer], dot = 0.f;
        load(k + key * p.k_stride, x);
        load(v + key * p.v_stride, y);
#pragma unroll
        for (int e = 0; e < kPer; ++e) dot = fmaf(q[e], x[e], dot);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, off);
        const float w = exp2f(fmaf(dot, p.qk_scale, -m_ref));
#pragma unroll
        for (int e = 0; e < kPer; ++e) acc[e] = fmaf(w, y[e], acc[e]);
      }
      open = false;
#pragma unroll
      for (int e = 0; e < kPer; ++e) open |= need[e] && !isnan(acc[e]);
    }
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      const int col = lane * kPer + e;
      if (!need[e]) continue;
      if (o != 0) reinterpret_cast<__nv_bfloat16*>(o)[col] = __float2bfloat16_rn(acc[e] * inv_l);
      else reinterpret_cast<float*>(part)[col / 8 * kItemRows * 8 + col % 8] = acc[e] * inv_l;
    }
  }
  __syncwarp();
}

// ---------------------------------------------------------------------------
// Softmax / correction / epilogue warpgroup (128 threads, one row each)
// ---------------------------------------------------------------------------
template <int D, bool CAUSAL>
__device__ __forceinline__ void run_softmax(int t, uint32_t tmem, const PackedSync& sy, const Params& p) {
  using C = PackedCfg<D>;
  const int lane = threadIdx.x & 31;
  const int quad = (threadIdx.x >> 5) & 3;  // TMEM lanes 32*quad .. 32*quad+31
  const int row_in_tile = quad * 32 + lane;
  const uint32_t lane_off = static_cast<uint32_t>(quad * 32) << 16;
  const uint32_t tS = tmem + lane_off + C::kTmemS + t * C::kTmemTile;
  const uint32_t tP = tmem + lane_off + C::kTmemP + t * C::kTmemTile;
  const uint32_t tO = tmem + lane_off + C::kTmemO + t * C::kTmemTile;
  const float qk = p.qk_scale;
  const uint32_t bar_s_full = t ? sy.s_full[1] : sy.s_full[0];
  const uint32_t bar_p_ready = t ? sy.p_ready[1] : sy.p_ready[0];
  const uint32_t bar_p_half = t ? sy.p_half[1] : sy.p_half[0];
  const uint32_t bar_o_done = t ? sy.o_done[1] : sy.o_done[0];
  const uint32_t bar_o_free = t ? sy.o_free[1] : sy.o_free[0];
  uint32_t s_par = 0, od_par = 0;
  bool ok = true;
  uint32_t items = 0;
  for (bool more = true; more && ok; ++items) {
    // read from shared memory where it is needed: 128 scores of a row and what the
    // loop over key tiles needs beside them fill the registers
    const uint32_t n = items % kItemsAhead;
    ok = wait_phase<CAUSAL>(sy.item_full0 + 8 * n, (items / kItemsAhead) & 1u, sy, p);
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) break;
    const Item& it = sy.items[n];
    const int kb = it.kb;
    if (it.i == 1 && p.dealt == 0 && p.range[blockIdx.x].first.slot >= 0) {
      // The range's first chunk was a part and has stored its rows; its arrival
      // is made here, while this chunk's first scores are on their way.
      const Range& r = p.range[blockIdx.x];
      if (part_arrive(p.counters + r.first.k * kCountersPerItem + t * 4 + quad, r.first.count, lane)) {
        const Row row(p.cu[r.s], p.cu[r.s + 1] - p.cu[r.s], r.h, (2 * r.b + t) * p.tpt, row_in_tile, D, p);
        merge_rows<D>(r.first, Own{kStored, 0.f, 0.f, 0u}, t * kBlockM + row_in_tile, row.store, row.o, row.lse,
                      p.part_o, p.part_lse);
      }
    }
    float m_ref = -INFINITY;  // reference maximum, in log2 units; moves on a jump above kRescaleThreshold
    float l = 0.f;            // running sum of exp2(s*qk - m_ref), for the logsumexp
    float lq = 0.f;           // the same terms rounded to bf16 (what P.V multiplies), for O

    // One key tile; the masked ones, at the end, have a loop and registers of their own.
    auto step = [&](auto masked_tile, int j) {
      ok = wait_phase<CAUSAL>(bar_s_full, s_par, sy, p);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) return;
      s_par ^= 1u;
      tc_fence_after_sync();

      constexpr bool kMasked = decltype(masked_tile)::value;
      const uint64_t qk2 = f2_pack(qk, qk);
      float alpha = 1.f;
      float sa, sb, lq_tile;
      // O_t holds the sum up to tile j-1: brought to the new reference, 32
      // columns at a time where the tile's scores are still in registers
      auto rescale = [&]() {
        if (j == kb || !__any_sync(0xffffffffu, alpha != 1.f)) return;
        const uint64_t a2 = f2_pack(alpha, alpha);
        constexpr int kCols = C::kHalves ? 32 : 64, kUnroll = C::kHalves ? 1 : 2;
#pragma unroll kUnroll
        for (int e = 0; e < D / kCols; ++e) {
          uint32_t o[kCols];
          if constexpr (kCols == 64) tmem_ld64_wait(tO + e * 64, o);
          else tmem_ld32_wait(tO + e * 32, o);
#pragma unroll
          for (int n = 0; n < kCols / 2; ++n) {
            float lo, hi;
            f2_unpack(f2_mul(f2_pack(__uint_as_float(o[2 * n]), __uint_as_float(o[2 * n + 1])), a2), lo, hi);
            o[2 * n] = __float_as_uint(lo);
            o[2 * n + 1] = __float_as_uint(hi);
          }
#pragma unroll
          for (int n = 0; n < kCols; n += 32) tmem_st32(tO + e * kCols + n, o + n);
        }
      };
      auto hand_over = [&](uint32_t bar) {
        tmem_st_wait();
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar);  // one arrival per warp
      };
      if constexpr (kMasked) {
        // A masked tile: 32 columns at a time, up to the last that some row of
        // the tile sees; the maximum first, then the exponentials from S read
        // again (where P lies over S, its 16 columns over some read before).
        const int len = it.len, t0 = (2 * it.b + t) * p.tpt;  // the tile's first token
        const int lim = (CAUSAL ? min(t0 + row_in_tile / p.G, len - 1) : len - 1) - j * kBlockN;  // the row's last visible key
        const int cols = (CAUSAL ? min(t0 + p.tpt, len) : len) - j * kBlockN;
        const int all = CAUSAL ? __reduce_min_sync(0xffffffffu, lim) : lim;  // what every row of the warp sees
        // Only columns that some row of the warp does not see are compared (24
        // ragged prompts 118 us, with all compared 121).
        auto load = [&](int c4, uint32_t* x) {
          tmem_ld32_wait(tS + c4 * 32, x);
          if (c4 * 32 + 31 > all) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (c4 * 32 + e > lim) x[e] = __float_as_uint(-INFINITY);
          }
        };
        float m_tile = -INFINITY;
#pragma unroll 1
        for (int c4 = 0; c4 < 4 && c4 * 32 < cols; ++c4) {
          uint32_t x[32];
          load(c4, x);
          float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
          for (int e = 0; e < 32; e += 2) mx[e >> 1 & 1] = fmax3(mx[e >> 1 & 1], __uint_as_float(x[e]), __uint_as_float(x[e + 1]));
          m_tile = fmax3(m_tile, mx[0], mx[1]);
        }
        m_tile *= qk;  // qk > 0: max commutes with the scale
        if (m_tile > m_ref + kRescaleThreshold<2>) {
          alpha = ex2_approx(m_ref - m_tile);  // 0 when m_ref = -inf
          m_ref = m_tile;
        }
        const float m_use = m_ref == -INFINITY ? 0.f : m_ref;  // 0: no key of this part visible yet, P = 0
        const uint64_t negm2 = f2_pack(-m_use, -m_use);
        uint64_t sum2 = f2_pack(0.f, 0.f);
        float lqs[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
        for (int c4 = 0; c4 < 4 && c4 * 32 < cols; ++c4) {
          uint32_t x[32], pk[16];
          load(c4, x);
#pragma unroll
          for (int n = 0; n < 16; ++n) {
            float xa, xb;
            f2_unpack(f2_fma(f2_pack(__uint_as_float(x[2 * n]), __uint_as_float(x[2 * n + 1])), qk2, negm2), xa, xb);
            const float a = ex2_approx(xa), b = ex2_approx(xb);
            pk[n] = pack_bf16x2(a, b);
            sum2 = f2_add(sum2, f2_pack(a, b));
            add_bf16x2_halves(lqs[(n & 1) * 2], lqs[(n & 1) * 2 + 1], pk[n]);
          }
          tmem_st16(tP + c4 * 16, pk);
        }
        f2_unpack(sum2, sa, sb);
        lq_tile = (lqs[0] + lqs[1]) + (lqs[2] + lqs[3]);
      } else {
        uint32_t s[128];
        tmem_ld128_wait(tS, s);
        // One pass over the tile: exponentials against m_use, P stored to
        // tensor memory, the fp32 and bf16 row sums, and (if asked) the
        // tile's row maximum from the same values.
        auto exp_pass = [&](float m_use, bool with_max) -> float {
          const uint64_t negm2 = f2_pack(-m_use, -m_use);
          uint64_t sum2 = f2_pack(0.f, 0.f);
          float lqs[4] = {0.f, 0.f, 0.f, 0.f};
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int c4 = 0; c4 < 4; ++c4) {
            uint32_t pk[16];
#pragma unroll
            for (int n = 0; n < 16; ++n) {
              const int e = c4 * 32 + 2 * n;
              const uint64_t x = f2_fma(f2_pack(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), qk2, negm2);
              float xa, xb;
              f2_unpack(x, xa, xb);
              const float a = ex2_approx(xa);
              const float b = ex2_approx(xb);
              pk[n] = pack_bf16x2(a, b);
              sum2 = f2_add(sum2, f2_pack(a, b));
              add_bf16x2_halves(lqs[(n & 1) * 2], lqs[(n & 1) * 2 + 1], pk[n]);
              if (with_max) mx[c4] = fmax3(mx[c4], __uint_as_float(s[e]), __uint_as_float(s[e + 1]));
            }
            tmem_st16(tP + c4 * 16, pk);
            if (C::kHalves && c4 == 1) hand_over(bar_p_half);
          }
          f2_unpack(sum2, sa, sb);
          lq_tile = (lqs[0] + lqs[1]) + (lqs[2] + lqs[3]);
          return fmaxf(fmax3(mx[0], mx[1], mx[2]), mx[3]) * qk;  // qk > 0: max commutes with the scale
        };
        auto row_max = [&]() -> float {
          float mx[4];
#pragma unroll
          for (int q4 = 0; q4 < 4; ++q4)
            mx[q4] = fmax3(__uint_as_float(s[32 * q4]), __uint_as_float(s[32 * q4 + 1]), __uint_as_float(s[32 * q4 + 2]));
#pragma unroll
          for (int e = 3; e < 31; e += 2) {
#pragma unroll
            for (int q4 = 0; q4 < 4; ++q4)
              mx[q4] = fmax3(mx[q4], __uint_as_float(s[32 * q4 + e]), __uint_as_float(s[32 * q4 + e + 1]));
          }
#pragma unroll
          for (int q4 = 0; q4 < 4; ++q4) mx[q4] = fmaxf(mx[q4], __uint_as_float(s[32 * q4 + 31]));
          return fmaxf(fmax3(mx[0], mx[1], mx[2]), mx[3]) * qk;
        };
        if constexpr (CAUSAL || C::kHalves) {
          // the maximum first, then one pass (faster under the mask, with its many first tiles;
          // and where the first half of P goes to its product before the second is known)
          const float m_tile = row_max();
          if (m_tile > m_ref + kRescaleThreshold<2>) {
            alpha = ex2_approx(m_ref - m_tile);  // 0 when m_ref = -inf
            m_ref = m_tile;
          }
          if (C::kHalves) rescale();
          exp_pass(m_ref == -INFINITY ? 0.f : m_ref, false);  // 0: no key of this part visible yet, P = 0
        } else {
          // the exponentials against the current reference while the tile's
          // maximum is found in the same pass; taken again where a row moved
          if (m_ref == -INFINITY) {
            m_ref = row_max();
            alpha = 0.f;
          }
#pragma unroll 1
          for (int pass = 0; pass < 2; ++pass) {
            const float m_tile = exp_pass(m_ref == -INFINITY ? 0.f : m_ref, true);
            const bool move = m_tile > m_ref + kRescaleThreshold<2>;
            if (!__any_sync(0xffffffffu, move)) break;
            if (move) {
              alpha = ex2_approx(m_ref - m_tile);
              m_ref = m_tile;
            }
            tmem_st_wait();  // the repeated pass stores P over this one's
          }
        }
      }
      l = l * alpha + (sa + sb);
      lq = lq * alpha + lq_tile;

      if (!C::kHalves || kMasked) rescale();
      if (C::kHalves && kMasked) hand_over(bar_p_half);
      hand_over(bar_p_ready);
    };
    int j = kb;
    for (const int plain = it.plain[t]; j < plain && ok; ++j) step(std::false_type{}, j);
    const int ne = it.ne[t];
    for (; j < ne && ok; ++j) step(std::true_type{}, j);
    if (!ok) break;

    // a part may have no key tile of this query tile; it still reports its rows, as an empty part
    const bool empty = ne <= kb;
    Own own{kEmpty, -INFINITY, 0.f, tO};
    if (!empty) {
      ok = wait_phase<CAUSAL>(bar_o_done, od_par, sy, p);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      od_par ^= 1u;
      tc_fence_after_sync();
      // a part may hold no visible key of a row (l = 0): its O is 0 and its logsumexp -inf
      own = Own{kInTmem, (m_ref + log2f(l)) * 0.69314718055994531f, l == 0.f ? 0.f : 1.f / lq, tO};
    }
    const bool whole = it.whole();
    const Row row(it.begin, it.len, it.h, (2 * it.b + t) * p.tpt, row_in_tile, D, p);
    // whether the chunk's last V tiles held keys that some of the item's rows do not see
    const bool masked = CAUSAL && !empty && it.ke > 2 * it.b * p.tpt / kBlockN;
    if (!whole) {
      const Range& r = p.range[blockIdx.x];
      const Part part = it.i == 0 ? r.first : r.last;
      const int r_item = t * kBlockM + row_in_tile;  // row within the item, and its slot
      // The end of a chunk that is a part: where every other part is in already
      // (as a rule for the range's last chunk, whose item's other parts were
      // other CTAs' first work), the warp merges from where its rows are;
      // else it stores them and arrives.
      int* ctr = p.counters + part.k * kCountersPerItem + t * 4 + quad;
      bool merge = (it.i > 0 || !it.more) && __all_sync(0xffffffffu, ld_acquire_gpu(ctr) == part.count - 1);
      bool store = !merge;
#pragma unroll 1
      for (;;) {
        if (store) {
          if (own.where == kInTmem) {
            uint32_t top = 0;  // NaN where an element of the row is
#pragma unroll
            for (int e = 0; e < D / 32; ++e) {
              uint32_t o[32];
              tmem_ld32_wait(tO + e * 32, o);
#pragma unroll
              for (int n = 0; n < 32; ++n) {
                top = max_nan(top, o[n]);
                o[n] = __float_as_uint(__uint_as_float(o[n]) * own.inv_l);
              }
#pragma unroll
              for (int n = 0; n < 4; ++n) st_global_v8(p.part_o + part_index<D>(part.slot, r_item, e * 4 + n), o + n * 8);
            }
            const uint32_t rows = __ballot_sync(0xffffffffu, row.store && is_nan(top));
            if (masked && rows != 0)
              mend_rows<D>(rows, lane, quad, (2 * it.b + t) * p.tpt, it,
                           Mend{nullptr, p.part_o + part_index<D>(part.slot, r_item, 0), m_ref, own.inv_l}, p);
          }
          p.part_lse[static_cast<size_t>(part.slot) * kItemRows + r_item] = own.lse;
          own.where = kStored;
          // merged already, but for NaN rows; or arrive (in the range's first chunk: with the next one)
          if (!merge && (it.i > 0 || !it.more)) merge = part_arrive(ctr, part.count, lane);
        }
        if (!merge) break;
        __syncwarp();
        const uint32_t top = merge_rows<D>(part, own, r_item, row.store, row.o, row.lse, p.part_o, p.part_lse);
        // a NaN row is mended in the workspace, and merged again
        store = masked && own.where == kInTmem && __any_sync(0xffffffffu, row.store && is_nan(top));
        if (!store) break;
      }
    } else if (!empty) {
      uint32_t top = 0;  // NaN where an element of the row is
      const uint64_t il2 = f2_pack(own.inv_l, own.inv_l);
      auto to_bf16 = [&](const uint32_t* o) {  // two elements of the row
        float lo, hi;
        f2_unpack(f2_mul(f2_pack(__uint_as_float(o[0]), __uint_as_float(o[1])), il2), lo, hi);
        return pack_bf16x2(lo, hi);
      };
      if constexpr (D == 128) {
        // The warp's 32 rows, 64 columns at a time: each lane writes its row's
        // 128 bytes to shared memory (16-byte pieces swizzled by row), then
        // eight lanes store a row's line, four rows an instruction.
        uint8_t* out = shared_base() + C::kOutOff + (threadIdx.x >> 5) * C::kWarpOut;
        const uint32_t stores = __ballot_sync(0xffffffffu, row.store);
#pragma unroll
        for (int e = 0; e < D / 64; ++e) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t o[32];
            tmem_ld32_wait(tO + e * 64 + h * 32, o);
#pragma unroll
            for (int n = 0; n < 4; ++n) {
              const uint4 w = make_uint4(to_bf16(o + 8 * n), to_bf16(o + 8 * n + 2), to_bf16(o + 8 * n + 4),
                                         to_bf16(o + 8 * n + 6));
              if (CAUSAL) top = max_nan_bf16x2(top, max_nan_bf16x2(max_nan_bf16x2(w.x, w.y), max_nan_bf16x2(w.z, w.w)));
              *reinterpret_cast<uint4*>(out + lane * 128 + (((h * 4 + n) ^ (lane & 7)) * 16)) = w;
            }
          }
          __syncwarp();
#pragma unroll
          for (int x = 0; x < 8; ++x) {
            const int from = (lane >> 3) + 4 * x, piece = lane & 7;
            const uint4 v = *reinterpret_cast<const uint4*>(out + from * 128 + ((piece ^ (from & 7)) * 16));
            const unsigned long long dst = __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(row.o), from);
            if ((stores >> from) & 1u) *reinterpret_cast<uint4*>(dst + (e * 64 + piece * 8) * 2) = v;
          }
          __syncwarp();
        }
      } else {
        // 128-byte rows: each lane its own, which measured faster here
        const bool wide = (reinterpret_cast<uintptr_t>(p.o) & 31u) == 0;  // the API promises 16
#pragma unroll
        for (int e = 0; e < D / 32; ++e) {
          uint32_t o[32], w[16];
          tmem_ld32_wait(tO + e * 32, o);
#pragma unroll
          for (int n = 0; n < 16; ++n) w[n] = to_bf16(o + 2 * n);
          if constexpr (CAUSAL) {
#pragma unroll
            for (int n = 0; n < 16; n += 4)
              top = max_nan_bf16x2(top, max_nan_bf16x2(max_nan_bf16x2(w[n], w[n + 1]), max_nan_bf16x2(w[n + 2], w[n + 3])));
          }
          if (row.store && wide) {
            st_global_v8(row.o + e * 32, w);
            st_global_v8(row.o + e * 32 + 16, w + 8);
          } else if (row.store) {
            uint4* dst = reinterpret_cast<uint4*>(row.o + e * 32);
#pragma unroll
            for (int n = 0; n < 4; ++n) dst[n] = make_uint4(w[4 * n], w[4 * n + 1], w[4 * n + 2], w[4 * n + 3]);
          }
        }
      }
      if (row.store) *row.lse = own.lse;
      if constexpr (CAUSAL) {
        const uint32_t rows = __ballot_sync(0xffffffffu, row.store && ((top & 0x7fffu) > 0x7f80u || (top & 0x7fff0000u) > 0x7f800000u));
        if (rows != 0)
          mend_rows<D>(rows, lane, quad, (2 * it.b + t) * p.tpt, it, Mend{row.o, nullptr, m_ref, own.inv_l}, p);
      } else if (__any_sync(0xffffffffu, own.inv_l == 0.f)) {
        // a row without weight is 0 whatever V holds; NaN is right in any other, since it sees all of V
        if (row.store && own.inv_l == 0.f) {
#pragma unroll 1
          for (int n = 0; n < D / 8; ++n) reinterpret_cast<uint4*>(row.o)[n] = make_uint4(0, 0, 0, 0);
        }
      }
    }
    more = it.more;
    tc_fence_before_sync();
    __syncwarp();
    if (lane == 0) {  // one arrival per warp
      if (!empty) mbar_arrive(bar_o_free);
      mbar_arrive(sy.item_empty0 + 8 * n);
    }
  }
}

// ---------------------------------------------------------------------------
// Kernel
// ---------------------------------------------------------------------------
template <int D, bool CAUSAL>
__global__ void __launch_bounds__(kNumThreads, 1)
fa_packed_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                 const __grid_constant__ CUtensorMap tmV, const __grid_constant__ Params p) {
  using C = PackedCfg<D>;
  uint8_t* smem = shared_base();
  const uint32_t sbase = smem_u32(smem);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  PackedSync sy;
  {
    uint32_t b = sbase + C::kBarOff;
    auto take = [&](int n) {
      const uint32_t at = b;
      b += 8 * n;
      return at;
    };
    for (int t = 0; t < 2; ++t) sy.q_full[t] = take(1);
    for (int t = 0; t < 2; ++t) sy.q_empty[t] = take(1);
    sy.kv_full0 = take(C::kStages);
    sy.kv_empty0 = take(C::kStages);
    for (int t = 0; t < 2; ++t) sy.s_full[t] = take(1);
    for (int t = 0; t < 2; ++t) sy.p_ready[t] = take(1);
    for (int t = 0; t < 2; ++t) sy.o_done[t] = take(1);
    for (int t = 0; t < 2; ++t) sy.o_free[t] = take(1);
    sy.drain = take(1);
    for (int t = 0; t < 2; ++t) sy.turn[t] = take(1);
    for (int t = 0; t < 2; ++t) sy.p_half[t] = take(1);
    sy.item_full0 = take(kItemsAhead);
    sy.item_empty0 = take(kItemsAhead);
  }
  Item* items = reinterpret_cast<Item*>(smem + C::kItemsOff);
  sy.items = items;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kMiscOff);
  sy.abort_flag = reinterpret_cast<volatile int*>(smem + C::kMiscOff + 4);

  if (threadIdx.x == 0) {
    for (int t = 0; t < 2; ++t) {
      mbar_init(sy.q_full[t], 1);
      mbar_init(sy.q_empty[t], 1);
      mbar_init(sy.s_full[t], 1);
      mbar_init(sy.p_ready[t], kBlockM / 32);
      mbar_init(sy.p_half[t], kBlockM / 32);
      mbar_init(sy.o_done[t], 1);
      mbar_init(sy.o_free[t], kBlockM / 32);
      mbar_init(sy.turn[t], 1);
    }
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(sy.kv_full0 + 8 * s, 1);
      mbar_init(sy.kv_empty0 + 8 * s, 2);  // released by both MMA issuers
    }
    mbar_init(sy.drain, 2);
    for (int n = 0; n < kItemsAhead; ++n) {
      mbar_init(sy.item_full0 + 8 * n, 1);
      mbar_init(sy.item_empty0 + 8 * n, 1 + 2 + 8);  // the producer, the issuers, the softmax warps
    }
    *sy.abort_flag = 0;
    *alive_word(sy.abort_flag) = 0;
    fence_barrier_init();
  }
  if (warp == kLoadWarp && lane == 0) {
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(tmem_slot), kTmemCols);
    tmem_relinquish_alloc_permit();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;

  if (warp >= 8) {
    setmaxnreg_dec<kRegsAux>();
    if (warp == kLoadWarp) {
      if (lane == 0) run_producer<D, CAUSAL>(&tmQ, &tmK, &tmV, sbase, sy, p);
      __syncwarp();
    } else if (warp == kMmaWarp || warp == kMmaWarp + 1) {
      run_mma<D, CAUSAL>(warp - kMmaWarp, smem, sbase, tmem, sy, p);
      __syncwarp();
    } else {
      if (lane == 0) run_dispatcher<CAUSAL>(items, sy, p);
      __syncwarp();
    }
  } else {
    setmaxnreg_inc<kRegsSoftmax>();
    run_softmax<D, CAUSAL>(warp >> 2, tmem, sy, p);
  }

  tc_fence_before_sync();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, kTmemCols);
  }
}

}  // namespace packed
}  // namespace fa
