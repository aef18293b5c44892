"""combine with its sums in 32 bits, and its gradient from 32 bits: against plain 64-bit forms, and as the example's layer
uses them, whose loss no 16-bit sums may stand behind."""
import pytest

import tiled_dense_gemm_bias_amd as gba
from tests import experts_oracle as eo
from tests.gpu_util import say
from tests.test_gpu_moe_move import DT, SIZES, case, gathered, valid
from tests.test_gpu_moe_route import guarded
from tests.test_gpu_moe_use import example

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("T,k,H,R", SIZES)
def test_sums(T, k, H, R, dtype, weighted):
    """k products and additions, one rounding each (2^-24 of the magnitudes), and no other."""
    say("combine f32", T, k, H, R, dtype, weighted)
    rows, _, y, w = case(T, k, H, R, dtype)
    out, intact = guarded((T, H), torch.float32, float("nan"))
    assert gba.moe_combine(y, rows, w if weighted else None, out) is out
    torch.cuda.synchronize()
    intact()
    v = gathered(y, rows)
    if weighted:
        v = v * w.double()[:, :, None]
    eo.check("out", out, v.sum(1), k * 2.0 ** -24 * v.abs().sum(1) + 2.0 ** -149)
    short = torch.empty(T, H, dtype=DT[dtype], device="cuda")
    assert torch.equal(gba.moe_combine(y, rows, w if weighted else None, short), out.to(DT[dtype]))


@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("T,k,H,R", SIZES)
def test_gradients(T, k, H, R, dtype, weighted):
    say("combine grad f32", T, k, H, R, dtype, weighted)
    rows, _, y, w = case(T, k, H, R, dtype)
    w = w if weighted else None
    dout = torch.randn(T, H, generator=torch.Generator(device="cuda").manual_seed(T + H), device="cuda")
    dy, i1 = guarded((R, H), DT[dtype], 5)
    dw, i2 = guarded((T, k), torch.float32, float("nan"))
    gba.moe_combine_grad(dout, y, rows, w, dy, dw)
    torch.cuda.synchronize()
    i1(), i2()
    ok = valid(rows, R)
    v = dout.double()[:, None] * (1.0 if w is None else w.double()[:, :, None])
    want = torch.full((R, H), 5.0, dtype=torch.float64, device="cuda")
    want[rows[ok].long()] = v.expand(T, k, H)[ok]
    eo.check("dy", dy, want, eo.with_rounding(want, 2.0 ** -24 * want.abs(), DT[dtype]))
    terms = gathered(y, rows) * dout.double()[:, None]
    eo.check("dw", dw, terms.sum(2), (H / 256 + 20) * 2.0 ** -24 * terms.abs().sum(2) + 2.0 ** -120)
    one = torch.full((R, H), 5, dtype=DT[dtype], device="cuda")
    gba.moe_combine_grad(dout, y, rows, w, one, None)
    other = torch.empty_like(dw)
    gba.moe_combine_grad(dout, y, rows, w, None, other)
    assert torch.equal(one, dy) and torch.equal(other, dw)


def test_a_captured_pass():
    say("graph f32")
    T, k, H, R = 40, 3, 520, 100
    rows, x, y, w = case(T, k, H, R, "bf16")
    out, dy, dw = torch.empty(T, H, device="cuda"), torch.zeros_like(y), torch.empty_like(w)

    def step():
        gba.moe_combine(y, rows, w, out)
        gba.moe_combine_grad(out, y, rows, w, dy, dw)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for r in range(3):
        y.copy_(torch.randn(y.shape, device="cuda"))
        step()
        want = [t.clone() for t in (out, dy, dw)]
        out.fill_(7), dw.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((out, dy, dw), want)), r


def test_the_examples_loss_and_first_gradient_are_of_unrounded_sums():
    """From the experts' outputs as the layer leaves them: the sums of k products (k 2^-24 of the magnitudes), a difference
    (2^-24) and its square; the gradient of the experts' rows, of the same difference (times 2 / tokens, itself rounded, and the weight: three roundings), is rounded to 16 bits once."""
    say("example f32")
    ex = example()
    tokens, experts, top, width, hidden = 257, 6, 2, 128, 192
    g = torch.Generator(device="cuda").manual_seed(6)
    layer = ex.ExpertLayer(experts, width, hidden, seed=9)
    router = torch.randn(experts, width, generator=g, device="cuda")
    x = torch.randn(tokens, width, generator=g, device="cuda").to(layer.dtype)
    to = ex.Routing(x.float() @ router.T, top)
    y, _ = layer.forward(to.dispatch(x), to.offsets)
    goal = to.combine(y).to(layer.dtype) * 1.01     # near the sums: what their rounding would lose is most of the loss
    loss, _ = ex.gradients(layer, router, x, goal, top)
    v = gathered(y, to.rows) * to.weights.double()[:, :, None]
    off, err = v.sum(1) - goal.double(), (top + 2) * 2.0 ** -24 * (v.abs().sum(1) + goal.double().abs())
    want = off.square().sum(1).mean()
    tol = (2 * off.abs() * err + err.square()).sum(1).mean() + want * (eo.sum_rel(width) + eo.sum_rel(tokens)) * 2
    assert abs(loss.item() - want.item()) <= tol.item()
    scale = 2.0 / tokens
    dy, _ = to.backward((to.combine(y) - goal) * scale, y)
    ok = to.rows >= 0
    at = to.rows[ok].long()
    d = (off[:, None] * scale * to.weights.double()[:, :, None])[ok]
    e = ((err + 4 * 2.0 ** -24 * off.abs())[:, None] * scale * to.weights.double()[:, :, None])[ok]
    eo.check("dy", dy[at], d, eo.with_rounding(d, e, layer.dtype))
