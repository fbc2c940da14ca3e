// Constants of the verification for the CPU tests (tests/test_verify_bound_cpu.py builds this file; host code alone runs).
#include "fa_verify.cuh"

namespace vf = fa::verify;

extern "C" {

float verify_quick_bound(int tiles) { return vf::quick_bound(tiles); }

int verify_lane_tiles(int V, int ctas, int warps) { return vf::lane_tiles(V, ctas, warps); }

}  // extern "C"
