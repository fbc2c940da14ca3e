// Work division of the packed forward, on the host: the items of one launch
// dealt out by length, or their concatenation cut into contiguous ranges of
// about equal cost, one per CTA.
#pragma once

#include "fa_packed_kernel.cuh"

namespace fa {
namespace packed {

// What an item costs beyond its steps, in steps: loading Q, the pipeline's
// start, writing O.
constexpr int kItemCost = 2;
// An item is cut only where both sides keep this many steps: a part costs a
// write and a read of 256 rows in fp32 besides.
constexpr int kMinPartSteps = 8;
// With no more items than CTAs, items are cut only while every CTA keeps this
// many steps.
constexpr int kMinStepsPerCta = 16;
// Long items are dealt where the CTA with the most work has at most so many
// steps more than its equal share; cutting them leaves an overhead like that.
// A prompt of 4096 tokens at 8 KV heads, 4 query heads each: 109 us dealt, 127
// cut; 8192 tokens at 2 heads, where the excess is 8 steps: 120 and 121.
constexpr int kDealtSlack = 8;

// item_steps in one step, for the loops over all blocks: the last query tile
// that has tokens visits the most key tiles.
template <bool CAUSAL>
inline int plan_steps(int b, int len, int tpt) {
  const int end = (2 * b + 2) * tpt;
  return ((CAUSAL && end < len ? end : len) - 1) / kBlockN + 1;
}

// Fills p.pair with the pairs of all sequences, those with the most steps first.
template <bool CAUSAL>
inline void deal(int n, int tpt, int longest, Params& p) {
  // Pairs of each number of steps, then where the next one goes.  A block has
  // 2 tpt <= 256 tokens, a step 128: kMaxPairs blocks make at most so many.
  int at[2 * kMaxPairs + 1];
  for (int steps = 0; steps <= longest; ++steps) at[steps] = 0;
  auto each = [&](auto&& f) {
    for (int s = 0; s < n; ++s) {
      const int len = p.cu[s + 1] - p.cu[s];
      for (int b = 0; b * 2ll * tpt < len; ++b) f(s, b, plan_steps<CAUSAL>(b, len, tpt));
    }
  };
  each([&](int, int, int steps) { ++at[steps]; });
  for (int steps = longest, next = 0; steps >= 0; --steps) {
    const int k = at[steps];
    at[steps] = next;
    next += k;
  }
  each([&](int s, int b, int steps) { p.pair[at[steps]++] = Pair{static_cast<uint16_t>(s), static_cast<uint16_t>(b)}; });
}

// The most work that a CTA of a dealt launch gets.
template <bool CAUSAL>
inline long long most_dealt(int items, int Hkv, int tpt, int grid, const Params& p) {
  long long load[kMaxCtas] = {}, top = 0;
  int cta = 0, by = 1, pair = 0, left = 0, w = 0;
  for (int i = 0; i < items; ++i, --left) {
    if (left == 0) {
      const Pair x = p.pair[pair++];
      w = plan_steps<CAUSAL>(x.b, p.cu[x.s + 1] - p.cu[x.s], tpt) + kItemCost;
      left = Hkv;
    }
    load[cta] += w;
    cta += by;
    if (cta < 0 || cta == grid) {  // the next row goes back
      cta -= by;
      by = -by;
    }
  }
  for (int c = 0; c < grid; ++c) top = load[c] > top ? load[c] : top;
  return top;
}

// Sequences cu[0..n] (n <= kMaxSeqs): fills p.pair or p.range and returns the
// grid; the number of workspace slots and of split items go to n_slots and
// n_split.
template <bool CAUSAL>
inline int make_plan(int n, int Hkv, int tpt, int num_ctas, Params& p, int& n_slots, int& n_split) {
  n_slots = n_split = p.dealt = 0;
  const int most = num_ctas < kMaxCtas ? num_ctas : kMaxCtas;
  long long weight = 0, pairs = 0;
  int longest = 0, shortest = 1 << 30;
  for (int s = 0; s < n; ++s) {
    const int len = p.cu[s + 1] - p.cu[s];
    long long w = 0, k = 0;
    for (int b = 0; b * 2ll * tpt < len; ++b, ++k) {
      const int steps = plan_steps<CAUSAL>(b, len, tpt);
      longest = steps > longest ? steps : longest;
      shortest = steps < shortest ? steps : shortest;
      w += steps + kItemCost;
    }
    weight += w * Hkv;
    pairs += k;
  }
  const long long items = pairs * Hkv;
  if (items == 0) return 0;
  // Items too short to be cut are dealt where they differ (24 ragged prompts,
  // up to 15 steps: 121 us, 147 in contiguous ranges; items of one length are
  // as even in ranges), long ones where the CTA with the most work has little
  // more than its share.
  if (items > most && shortest < longest && pairs <= kMaxPairs && items < (1 << 30)) {
    const bool short_items = longest < 2 * kMinPartSteps;
    if (short_items || (longest + kItemCost) * static_cast<long long>(most) <= weight) {
      deal<CAUSAL>(n, tpt, longest, p);
      if (short_items || most_dealt<CAUSAL>(static_cast<int>(items), Hkv, tpt, most, p) <= weight / most + kDealtSlack) {
        p.dealt = static_cast<int>(items);
        return most;
      }
    }
  }
  long long ctas = items;
  if (ctas < most) {
    const long long by_work = weight / kMinStepsPerCta;
    ctas = by_work > ctas ? by_work : ctas;
    // an item meets at most kMaxParts ranges
    const long long by_parts = weight * (kMaxParts - 2) / (longest + kItemCost);
    if (ctas > items && ctas > by_parts) ctas = by_parts > items ? by_parts : items;
  }
  if (ctas > most) ctas = most;

  int grid = 0;             // ranges closed so far
  bool open = false;        // p.range[grid] has a first chunk
  long long cut = 1, at = 0;
  long long next = weight / ctas;  // where cut lies
  for (int s = 0; s < n; ++s) {
    const int len = p.cu[s + 1] - p.cu[s];
    for (int h = 0; h < Hkv; ++h) {
      for (int b = 0; b * 2ll * tpt < len; ++b) {
        const int steps = plan_steps<CAUSAL>(b, len, tpt);
        const long long w = steps + kItemCost;
        if (next >= at + w || cut >= ctas) {  // the usual case: no cut in it
          Range& r = p.range[grid];
          if (!open) {
            r = Range{s, h, b, 0, 0, 0, Part{-1, 0, 0, 0}, Part{-1, 0, 0, 0}};
            open = true;
          }
          ++r.n_items;
          r.step_end = steps;
          at += w;
          continue;
        }
        // this item's parts: their ranges, patched when their number is known
        int part_range[kMaxParts];
        bool part_first[kMaxParts];
        int parts = 0, done = 0;  // steps of the item already given to a range
        auto begin = [&](int step) {
          Range& r = p.range[grid];
          if (!open) {
            r = Range{s, h, b, 0, step, 0, Part{-1, 0, 0, 0}, Part{-1, 0, 0, 0}};
            open = true;
          }
          ++r.n_items;
        };
        auto take = [&](int to) {  // the open range gets steps [done, to) of this item
          begin(done);
          p.range[grid].step_end = to;
          if (done > 0 || to < steps) {
            part_range[parts] = grid;
            part_first[parts] = p.range[grid].n_items == 1;
            ++parts;
          }
          done = to;
        };
        for (; cut < ctas && next < at + w; next = weight * ++cut / ctas) {
          const int off = static_cast<int>(next - at) - kItemCost / 2;
          int step = off < 0 ? 0 : off > steps ? steps : off;
          // a cut in an item too short for it goes to the nearer end, with
          // fewer than kMinPartSteps steps (below) always in front
          if (steps < 2 * kMinPartSteps) step = 2 * step < steps ? 0 : steps;
          if (step - done < kMinPartSteps) step = done;
          if (steps - step < kMinPartSteps && step > done) step = steps;
          if (parts >= kMaxParts - 1 && step > done && step < steps) step = done;
          if (step > done) take(step);
          if (open && (step > 0 || done == 0)) {  // close the range here
            ++grid;
            open = false;
          }
        }
        if (done < steps) take(steps);
        at += w;
        if (parts > 0) {
          for (int i = 0; i < parts; ++i) {
            Range& r = p.range[part_range[i]];
            (part_first[i] ? r.first : r.last) = Part{n_slots + i, n_slots, parts, n_split};
          }
          n_slots += parts;
          ++n_split;
        }
      }
    }
  }
  return grid + (open ? 1 : 0);
}

}  // namespace packed
}  // namespace fa
