"""The sizes of tests/experts_cases.py reach the kernels they stand for, all of them, without a GPU."""
import pytest

import tiled_dense_gemm_bias_amd as gba
from tests import experts_cases as cases

TILES = {(16, 64), (32, 64), (64, 64), (64, 128), (128, 64), (128, 128)}


def reached(op, groups, cols, depth, mib):
    sizes, lead, tail = groups
    N, K = (depth, cols) if op == "act_grad" else (cols, depth)
    p = gba.experts.plan(op, lead + sum(sizes) + tail, len(sizes), N, K, mib * cases.MIB)
    return p["tile_m"], p["tile_n"], p["persistent"], int(p["splits"] > 1), p["non_temporal"]


@pytest.mark.parametrize("op,table", [("forward", cases.ROWS), ("act_grad", cases.ROWS), ("mx4", cases.MX4),
                                      ("wgrad", cases.GRADS)])
def test_each_case_reaches_its_kernel(op, table):
    for want, groups, cols, depth, mib in table:
        assert reached(op, groups, cols, depth, mib) == want, (op, groups[0][:6], cols, depth)


@pytest.mark.parametrize("op,table", [("forward", cases.ROWS), ("mx4", cases.MX4), ("wgrad", cases.GRADS)])
def test_every_kernel_is_reached(op, table):
    """With the smallest tile whole, which the small shapes of the other tests reach."""
    have = {c[0] for c in table} | {(16, 64, 0, 0, 0), (64, 64, 0, 0, 0)}
    if op == "wgrad":
        assert {(t, u, 0, s, 0) for t, u in ((64, 64), (128, 128)) for s in (0, 1)} | {(256, 256, 1, 0, 0)} <= have
        return
    assert {(t, u, 0, 0, 0) for t, u in TILES} | {(256, 256, 1, 0, 0)} <= have
    splits = {(t, u) for t, u, _, s, _ in have if s}
    assert splits == TILES - ({(128, 64)} if op == "mx4" else set())     # its operands there are gigabytes
    streamed = {(t, u) for t, u, _, s, nt in have if nt}
    assert {(32, 64), (64, 128)} <= streamed
    assert {(t, u) for t, u, _, s, nt in have if nt and s} >= ({(16, 64)} if op == "mx4" else {(16, 64), (32, 64)})


def test_depths_and_searches_of_the_persistent_kernel():
    """Two slices with and without a partial one, six or more (the loads that warm the L2), and
    more experts than a wave has lanes."""
    for table, per in ((cases.ROWS, 1), (cases.MX4, 4)):
        big = [(len(g[0]), d // per) for (_, _, p, _, _), g, _, d, _ in table if p]
        assert {-(-d // 64) for e, d in big if e <= 64} >= {2, 6} or {-(-d // 64) for e, d in big if e <= 64} >= {2, 9}
        assert any(d % 64 for e, d in big if -(-d // 64) == 2) and any(d == 128 for e, d in big)
        assert any(e > 64 for e, d in big) and any(1 < e <= 64 and d > 320 for e, d in big)
