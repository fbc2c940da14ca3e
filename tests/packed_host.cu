// The packed forward's host plan and layout constants for the CPU tests (tests/packed_host.py builds this file).
#include "fa_packed_plan.h"

namespace pk = fa::packed;

extern "C" {

// S's, P's or O's first tensor memory column in query tile t (which = 0, 1, 2).
int packed_tmem(int d, int which, int t) {
  using A = pk::PackedCfg<64>;
  using B = pk::PackedCfg<128>;
  const int at[2][3] = {{A::kTmemS, A::kTmemP, A::kTmemO}, {B::kTmemS, B::kTmemP, B::kTmemO}};
  return at[d == 128][which] + t * (d == 128 ? B::kTmemTile : A::kTmemTile);
}

// The plan of n sequences: info = {grid, dealt, slots, split items}; ranges [grid][14] as in pk::Range, or pairs
// [dealt / Hkv][2].
void packed_plan(const int* lens, int n, int Hkv, int tpt, int causal, int num_ctas, int* info, int* ranges, int* pairs) {
  static pk::Params p;
  p.cu[0] = 0;
  for (int i = 0; i < n; ++i) p.cu[i + 1] = p.cu[i] + lens[i];
  info[0] = causal ? pk::make_plan<true>(n, Hkv, tpt, num_ctas, p, info[2], info[3])
                   : pk::make_plan<false>(n, Hkv, tpt, num_ctas, p, info[2], info[3]);
  info[1] = p.dealt;
  if (p.dealt > 0) {
    for (int i = 0; i < p.dealt / Hkv; ++i) pairs[2 * i] = p.pair[i].s, pairs[2 * i + 1] = p.pair[i].b;
    return;
  }
  for (int c = 0; c < info[0]; ++c) {
    const pk::Range& r = p.range[c];
    const int x[14] = {r.s, r.h, r.b, r.n_items, r.step_begin, r.step_end,
                       r.first.slot, r.first.slot0, r.first.count, r.first.k,
                       r.last.slot, r.last.slot0, r.last.count, r.last.k};
    for (int i = 0; i < 14; ++i) ranges[14 * c + i] = x[i];
  }
}

int packed_halves(int d) { return d == 128 ? pk::PackedCfg<128>::kHalves : pk::PackedCfg<64>::kHalves; }
}
