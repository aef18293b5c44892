"""The sizes of the persistent 8-bit kernel's tests are ones that it takes, and reach what they are for, without a GPU."""
import pytest

from tests import moe_large_cases as cases
from tests import test_gpu_fp8_block_large as large
from tiled_dense_gemm_bias_amd import moe


@pytest.mark.parametrize("case", cases.LARGE, ids=lambda c: "%d-%d-%d-%d" % (sum(c[1]), len(c[1]), c[4], c[5]))
def test_cases_take_the_persistent_kernel(case):
    want, sizes, lead, tail, N, K, mib = case
    p = moe.plan(lead + sum(sizes) + tail, len(sizes), N, K, mib)
    assert (p["kind"], p["tile_m"], p["tile_n"], p["splits"] > 1) == want and min(sizes) >= 0


def test_what_they_reach():
    some = [(len(c[1]), c[4], -(-c[5] // 128), c[5] % 128 != 0, sum(-(-n // 256) for n in c[1]) * -(-c[4] // 256)) for c in cases.LARGE]
    for slices, cut in ((2, True), (2, False), (3, True), (3, False), (4, True)):
        assert any(s[2:4] == (slices, cut) for s in some), (slices, cut)
    for experts in (False, True):                                      # up to 64 experts and more: lines whole, several tiles a CU
        assert any((s[0] > 64) == experts and s[1] % 64 == 0 and s[4] > 512 for s in some)
    assert any(s[1] % 64 for s in some) and any(s[1] % 256 and s[1] % 64 == 0 for s in some)
    assert sum(n % 256 != 0 for c in cases.LARGE for n in c[1]) > 100 and any(n == 0 for c in cases.LARGE for n in c[1])


def test_the_other_sizes():
    for T, E, N, K in large.OFFSETS + large.NAN:
        assert moe.plan(T, E, N, K)["kind"] == "persistent", (T, E, N, K)
    assert {E > 64 for T, E, N, K in large.OFFSETS} == {E > 64 for T, E, N, K in large.NAN} == {False, True}
