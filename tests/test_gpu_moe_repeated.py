"""Gradients of routing where a caller's own indices name an expert several times in a row: the terms add up in the order of the
slots, bit for bit."""
import pytest

import tiled_dense_gemm_bias_amd as gba
from tests import experts_oracle as eo
from tests import moe_oracle as orc
from tests.gpu_util import say
from tests.test_gpu_moe_route import guarded, logits

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def grad(x, idx, dw, **kw):
    dx, intact = guarded(x.shape, torch.float32, 5)
    gba.moe_route_grad(x, idx, dw, dx, **kw)
    torch.cuda.synchronize()
    intact()
    return dx


@pytest.mark.parametrize("T,E,k", [(5, 6, 5), (33, 20, 16), (9, 20, 17), (70, 40, 32), (17, 200, 32), (6, 300, 32), (7, 1000, 32)])
def test_in_the_order_of_the_slots(T, E, k):
    """Sigmoid scores without renormalisation: a slot's term depends on its expert and weight alone, and is what a call with the
    other slots taken away leaves."""
    say("repeated", T, E, k)
    x, g = logits(T + E, T, E, "f32")
    # few different experts, some rows with all alike, some with none twice
    idx = torch.randint(-1, 3, (T, k), generator=g, device="cuda", dtype=torch.int32)
    idx[0] = E - 1
    idx[1] = -1
    idx[2, :min(k, E)] = torch.randperm(E, generator=g, device="cuda")[:min(k, E)].to(torch.int32)
    idx[3, ::2] = 4
    dw = torch.randn(T, k, generator=g, device="cuda") * torch.exp2(torch.randint(-12, 12, (T, k), generator=g, device="cuda").float())
    kw = dict(score="sigmoid", renormalize=False)
    want = torch.zeros(T, E, device="cuda")
    for j in range(k):
        one = torch.full_like(idx, -1)
        one[:, j] = idx[:, j]
        want = want + grad(x, one, dw, **kw)
    dx = grad(x, idx, dw, **kw)
    assert torch.equal(dx, want)
    assert all(torch.equal(grad(x, idx, dw, **kw), dx) for _ in range(3))


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k", [(33, 20, 17), (9, 300, 8)])
def test_against_the_formulas(T, E, k, score, renorm):
    say("repeated", T, E, k, score, renorm)
    x, g = logits(T + E, T, E, "f32")
    idx = torch.randint(0, 4, (T, k), generator=g, device="cuda", dtype=torch.int32)
    dw = torch.randn(T, k, generator=g, device="cuda")
    dx = grad(x, idx, dw, score=score, renormalize=renorm)
    want, size, depth = orc.route_grad(x, idx, dw, score, renorm)
    # k additions beside the roundings of a term
    eo.check("dx", dx, want, eo.with_rounding(want, (2 * depth[:, None] + 60 + k) * 2.0 ** -24 * size + 2.0 ** -120, torch.float32))
