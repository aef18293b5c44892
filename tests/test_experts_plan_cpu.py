"""The choice of kernel, tile and split of the grouped and 4-bit products (gbx_get_plan), without a GPU."""
import ctypes

import pytest

import tiled_dense_gemm_bias_amd as gba

experts = gba.experts
plan = experts.plan
OK, NULL, SHAPE, ALIGN = 0, 1, 2, 5
OPS = ("forward", "act_grad", "wgrad", "wgrad_bias", "mx4")
MIB = 1 << 20


def raw(op=0, T=64, E=4, N=64, K=64, ws=0, cus=256, out=True):
    p = experts._Plan()
    return experts.experts_lib().gbx_get_plan(op, T, E, N, K, ws, cus, ctypes.byref(p) if out else None)


def test_refusals():
    for op in range(5):
        assert raw(op) == OK
        assert raw(op, out=False) == NULL
        for bad in (dict(T=0), dict(E=0), dict(N=0), dict(K=0), dict(T=-1), dict(E=4097), dict(T=(1 << 29) + 1),
                    dict(N=1 << 24), dict(K=1 << 24), dict(cus=0)):
            assert raw(op, **bad) == SHAPE, (op, bad)
        assert raw(op, N=60) == ALIGN
        assert raw(op, K=36) == ALIGN
    assert raw(-1) == SHAPE and raw(5) == SHAPE
    assert raw(0, K=(1 << 21) + 8) == SHAPE and raw(1, K=(1 << 21) + 8) == OK      # the depth: K
    assert raw(1, N=(1 << 21) + 8) == SHAPE and raw(0, N=(1 << 21) + 8) == OK      # the depth: N
    assert raw(4, K=1 << 23) == OK and raw(4, K=(1 << 23) + 32) == SHAPE
    with pytest.raises(gba.GbaError):
        plan("forward", 64, 0, 64, 64)


@pytest.mark.parametrize("op", OPS)
def test_plans_are_ones_that_can_run(op):
    """Over sizes of every order: a tile that is built, splits that fit the workspace and the depth, two
    slices at least for the persistent kernel of a row product."""
    grad = op.startswith("wgrad")
    tiles = {(64, 64), (128, 128)} if grad else {(16, 64), (32, 64), (64, 64), (64, 128), (128, 64), (128, 128)}
    seen = set()
    for T in (1, 5, 33, 260, 2000, 17000, 1 << 29):
        for E in (1, 3, 64, 65, 4096):
            for N in (8, 72, 1000, 14336, 1 << 21):
                for K in (32, 96, 1024, 8224, 1 << 21):
                    for ws in (0, 4096, 8 * MIB, 1 << 40):
                        p = plan(op, T, E, N, K, ws)
                        words, cols = {"act_grad": (N, K), "mx4": (K // 4, N)}.get(op, (K, N))
                        slices = -(-words // 64)
                        tile = (p["tile_m"], p["tile_n"])
                        seen.add((tile, p["splits"] > 1))
                        if p["persistent"]:
                            assert tile == (256, 256) and p["splits"] == 1 and (grad or slices >= 2)
                        else:
                            assert tile in tiles
                        values = E * N * K if grad else T * cols
                        assert p["splits"] == 1 or 4 * values * p["splits"] <= ws
                        if not grad:
                            assert p["splits"] == 1 or p["splits"] * 2 <= slices
                        assert not (p["non_temporal"] and (grad or p["persistent"] or tile[0] > 64))
    assert len(seen) >= (4 if grad else 8), seen


def test_workspaces_and_devices():
    """No workspace, no split; with fewer compute units there is less to fill."""
    assert plan("forward", 3, 1, 72, 4096)["splits"] == 1
    assert plan("forward", 3, 1, 72, 4096, 8 * MIB)["splits"] == 16
    assert plan("forward", 3, 1, 72, 4096, 8 * MIB, cus=1)["splits"] == 1


def test_only_what_one_call_reads_counts_as_streamed():
    """One token reads one expert: 4 MiB of 64 experts of 1024 x 2048. Twelve of 32 experts of 2816 x 2048
    do not fit the cache, and neither does one expert of 14336 x 8192."""
    assert not plan("forward", 1, 64, 1024, 2048)["non_temporal"]
    assert not plan("forward", 8, 128, 1024, 2560)["non_temporal"]
    assert plan("forward", 16, 32, 2816, 2048)["non_temporal"]
    assert plan("forward", 1, 8, 14336, 8192)["non_temporal"]


def test_streamed_weights_are_split_where_that_pays():
    """Measured, whole against split in four, microseconds: 8 rows on 8 of 15 experts of
    4096 x 2560: 27.7 and 30.4; 240 rows on 12 of 27 experts of 2816 x 2048: 40.9 and 43.8; 16 rows on 12 of 32 of
    2816 x 2048: 34.3 and 28.1; of 2816 x 4096: 60.3 and 47.0."""
    streamed = dict(workspace=64 * MIB)
    assert plan("forward", 8, 15, 4096, 2560, **streamed) == dict(
        tile_m=16, tile_n=64, persistent=0, splits=1, non_temporal=1)
    assert plan("forward", 240, 27, 2816, 2048, **streamed)["splits"] == 1
    for K in (2048, 4096):
        p = plan("forward", 16, 32, 2816, K, **streamed)
        assert p["splits"] == 4 and p["non_temporal"]
    # not at one depth only: rows of 4 KiB a little longer or shorter, and long rows of any pitch
    assert plan("forward", 16, 32, 2816, 2040, **streamed)["splits"] == 1
    assert plan("forward", 16, 32, 2816, 4480, **streamed)["splits"] == 4
