"""Products whose scales are far from 1: the two scales meet in one 32-bit product, which is exact here, so that whole numbers
come out bit for bit in every kernel, and what the product's range cannot hold is an infinity, in its own places."""
import math

import pytest

import tiled_dense_gemm_bias_amd as gba
from tests import moe_oracle as orc
from tests.gpu_util import say
from tests.test_gpu_experts import guarded as guarded16
from tests.test_gpu_experts import make_offsets
from tests.test_gpu_fp8_block import F8

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

# rows by expert, columns, depth, the kernel
SIZES = [([5, 0, 3], 264, 528, "stream"), ([40, 70, 3], 264, 272, "ring"), ([3500, 10], 4160, 272, "persistent")]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def product(sizes, N, K, kind, sa, sw):
    """(c, the exact sums in 64 bits) of whole numbers up to 8 with scales of 2^sa and 2^sw, or twice that."""
    g = torch.Generator(device="cuda").manual_seed(N + K)
    T, E = sum(sizes), len(sizes)
    assert gba.moe.plan(T, E, N, K, 0, torch.cuda.get_device_properties(0).multi_processor_count)["kind"] == kind
    whole = lambda *s: (torch.randint(-8, 9, s, generator=g, device="cuda") / 1.0).to(F8)
    two = lambda p, s: torch.exp2(torch.randint(0, 2, s, generator=g, device="cuda").double() + p).float()
    ac, asc, wc, wsc = whole(T, K), two(sa, gba.fp8_scales_shape(T, K)), whole(E, N, K), two(sw, gba.fp8_weight_scales_shape(E, N, K))
    a64 = orc.values(ac.view(torch.uint8), asc.T.contiguous())
    w64 = torch.stack([orc.values(wc[e].view(torch.uint8), wsc[e], 128) for e in range(E)])
    off = make_offsets(sizes)
    want, _, owned = orc.product(a64, off.tolist(), w64, None)
    assert owned.all()
    c, intact = guarded16((T, N), torch.bfloat16)
    gba.grouped_gemm_bias_act_fp8_block(ac, asc, off, wc, wsc, None, c, "none")
    torch.cuda.synchronize()
    intact()
    return c, want


@pytest.mark.parametrize("sa,sw", [(-60, -60), (100, -100), (-120, 118), (54, 54), (-70, -70), (-126, 60), (118, -126)])
@pytest.mark.parametrize("sizes,N,K,kind", SIZES)
def test_whole_numbers(sizes, N, K, kind, sa, sw):
    """Sums are multiples of 2^(sa + sw), from 2^-140 on exact in 32 bits (subnormal products of scales among them); compared
    where the result is a normal number of 16 bits."""
    say("scales", sizes, N, K, kind, sa, sw)
    c, want = product(sizes, N, K, kind, sa, sw)
    normal = (want.abs() >= 2.0 ** -125) | (want == 0)
    assert normal.any() and torch.equal(c[normal], want.float().bfloat16()[normal])
    assert (c[~normal].double().abs() <= 2.0 ** -125).all()


@pytest.mark.parametrize("sizes,N,K,kind", SIZES)
def test_scales_whose_product_is_infinite(sizes, N, K, kind):
    say("infinite", sizes, N, K, kind)
    c, want = product(sizes, N, K, kind, 70, 70)
    assert (want.abs().max() > 2.0 ** 145) and not torch.isfinite(c).any()
