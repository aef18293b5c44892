"""The choice of kernel, tile and split of the 8-bit products (gbm_get_plan), without a GPU."""
import ctypes

import pytest

import tiled_dense_gemm_bias_amd as gba
from tests import moe_cases as cases
from tiled_dense_gemm_bias_amd import moe

OK, NULL, SHAPE, ALIGN = 0, 1, 2, 5


def raw(T=64, E=4, N=64, K=64, ws=0, cus=256, out=True):
    p = moe._Plan()
    return moe.moe_lib().gbm_get_plan(T, E, N, K, ws, cus, ctypes.byref(p) if out else None)


def test_refusals():
    assert raw() == OK and raw(out=False) == NULL
    for bad in (dict(T=0), dict(E=0), dict(N=0), dict(K=0), dict(T=-1), dict(E=4097), dict(T=(1 << 29) + 1), dict(N=(1 << 23) + 8),
                dict(K=(1 << 22) + 16), dict(cus=0), dict(cus=-5)):
        assert raw(**bad) == SHAPE, bad
    assert raw(N=60) == ALIGN and raw(K=24) == ALIGN
    assert raw(T=1 << 29, E=4096, N=1 << 23, K=1 << 22, ws=(1 << 64) - 1, cus=(1 << 31) - 1) == OK
    with pytest.raises(gba.GbaError):
        moe.plan(64, 0, 64, 64)


def test_plans_are_ones_that_can_run():
    """Over sizes of every order: a tile that is built, splits that fit the workspace and the depth, two slices at least
    for the persistent kernel, and few rows for the streaming one; every kernel is taken by some sizes."""
    tiles = {(16, 64), (32, 64), (64, 64), (64, 128), (128, 64), (128, 128)}
    seen = set()
    for T in (1, 5, 33, 260, 1000, 2000, 17000, 1 << 29):
        for E in (1, 3, 8, 40, 65, 4096):
            for N in (8, 72, 520, 1000, 14336, 1 << 21):
                for K in (16, 96, 1024, 4096, 8208, 16400, 1 << 22):
                    for ws in (0, 4096, 8 << 20, 1 << 40):
                        p = moe.plan(T, E, N, K, ws)
                        tile, slices = (p["tile_m"], p["tile_n"]), -(-K // 128)
                        seen.add((p["kind"],) + tile + (p["splits"] > 1,))
                        if p["kind"] == "ring":
                            assert tile in tiles and (p["splits"] == 1 or 2 * p["splits"] <= slices)
                            assert p["splits"] == 1 or 4 * T * N * p["splits"] <= ws
                        else:
                            assert p["splits"] == 1
                            assert tile == ((256, 256) if p["kind"] == "persistent" else (16, 16))
                            assert slices >= 2 if p["kind"] == "persistent" else T <= 8 * min(E, T)
    want = {("ring",) + t + (s,) for t in tiles for s in (False, True)} | {("persistent", 256, 256, False), ("stream", 16, 16, False)}
    assert seen == want


@pytest.mark.parametrize("case", cases.PRODUCTS, ids=lambda c: "%s-%d" % ("-".join(map(str, c[0])), sum(c[1])))
def test_cases_take_the_kernels_that_they_are_for(case):
    want, sizes, lead, tail, N, K, mib = case
    p = moe.plan(lead + sum(sizes) + tail, len(sizes), N, K, mib * cases.MIB)
    assert (p["kind"], p["tile_m"], p["tile_n"], p["splits"] > 1) == want
    assert min(sizes) >= 0


def test_every_kernel_has_a_case():
    assert len({c[0] for c in cases.PRODUCTS}) == 14
