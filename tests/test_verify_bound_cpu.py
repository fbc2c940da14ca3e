"""The bound on the quick pass's sum covers what its roundings may add up to, for clusters of any size.

The pass is run in 64 bits with every rounding at its largest and of one sign: a power of two is off by 2^-22 (the
documented error of ex2.approx), a product and an addition by 2^-24, a power's argument, of up to 17, by 2^-22.4 of it.
"""
import ctypes
import os
import subprocess

import pytest

from exact_attention_20_gb300 import build as fa_build

EX2, ROUND, ARGUMENT = 2.0 ** -22, 2.0 ** -24, 2.0 ** -22.4


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("verify") / "verify_host.so")
    src = os.path.join(os.path.dirname(os.path.abspath(__file__)), "verify_host.cu")
    subprocess.run([fa_build.nvcc(), *fa_build.COMPILE_FLAGS, "-shared", "-cudart", "static", "-I",
                    os.path.join(fa_build.ROOT, "include"), "-I", os.path.join(fa_build.PKG, "csrc"), "-o", out, src], check=True)
    lib = ctypes.CDLL(out)
    lib.verify_quick_bound.restype = ctypes.c_float
    return lib


def quick_error(tiles, rises):
    """The relative error of a lane's and the reductions' sum: the maximum rises by `rises` binary orders in all."""
    weight = 1 + EX2                        # of a token, when it is taken
    got = want = 0.0
    step = 2.0 ** (-rises / tiles)
    for _ in range(tiles):
        got *= step * (1 + EX2) * (1 + ROUND)
        want *= step
        got = (got + 8 * weight * (1 + ROUND) ** 4) * (1 + ROUND)
        want += 8
    for _ in range(3):                      # the warp's, the CTA's and the cluster's
        got *= (1 + EX2) * (1 + ROUND) * (1 + ROUND) ** 5
    return got * (1 + 17 * 0.6931471805599453 * ARGUMENT) / want - 1


def test_bound_covers_the_roundings(host):
    for tiles in range(1, 300):
        bound = host.verify_quick_bound(tiles)
        for rises in (0.0, 1e-3, 1.0, 17.0):
            assert quick_error(tiles, rises) <= 0.75 * bound, (tiles, rises)
        assert bound < 2.0 ** -11  # small enough that hardly any child is in doubt


def test_tiles_of_a_lane(host):
    # a row starts up to seven tokens into a tile; CTAs take equal parts of its tiles, warps every so many of those
    for V in (1, 2, 249, 250, 256, 257, 32000, 128000, 1 << 18):
        for ctas in (1, 2, 4, 8, 16):
            for warps in (4, 8):
                most = 0
                for shift in range(8):
                    tiles = -(-(V + shift) // 256)
                    per = -(-tiles // ctas)
                    most = max(most, len(range(0, min(per, tiles), warps)))
                assert host.verify_lane_tiles(V, ctas, warps) == most


def test_clusters_of_sixteen_keep_two_to_the_minus_fifteen(host):
    for warps in (4, 8):
        most = host.verify_lane_tiles(1 << 18, 16, warps)
        assert most <= 17 and host.verify_quick_bound(most) == 2.0 ** -15
    alone = host.verify_lane_tiles(1 << 18, 1, 4)
    assert alone == 257 and 2.0 ** -13 < host.verify_quick_bound(alone) < 2.0 ** -12
    # a bound that did not follow the tiles would not cover it
    assert quick_error(alone, 0.0) > 2.0 ** -15
