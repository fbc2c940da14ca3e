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

int packed_halves(int d) { return d == 128 ? pk::PackedCfg<128>::kHalves : pk::PackedCfg<64>::kHalves; }
}
