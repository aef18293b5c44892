"""Dispatch, combine and its gradients against plain 64-bit forms: odd widths, slots without a row, rows of no slot, row numbers
out of range, every k."""
import pytest

import tiled_dense_gemm_bias_amd as gba
from tests import experts_oracle as eo
from tests.gpu_util import say
from tests.test_gpu_moe_route import guarded

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

DT = {"bf16": torch.bfloat16, "f16": torch.float16}
SIZES = [(1, 1, 8, 1), (3, 2, 72, 10), (8, 2, 2048, 16), (5, 8, 4104, 40), (17, 9, 1000, 200), (2, 32, 264, 64), (33, 3, 8192, 99), (4, 2, 8200, 9),
         (2, 1, 20000, 2), (40000, 1, 16, 40000), (2050, 3, 2312, 5000), (2048, 9, 520, 15000), (3001, 2, 4088, 5000)]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def case(T, k, H, R, dtype, seed=1):
    """Distinct rows for most slots, some without a row, some out of range; rows that no slot names."""
    g = torch.Generator(device="cuda").manual_seed(seed + T + H)
    rows = torch.full((T * k,), -1, dtype=torch.int32, device="cuda")
    n = min(R, T * k)
    slots = torch.randperm(T * k, generator=g, device="cuda")[:n]
    rows[slots] = torch.randperm(R, generator=g, device="cuda")[:n].to(torch.int32)
    if T * k > 4:
        rows[0], rows[1], rows[2], rows[3] = R, -1, 2 ** 31 - 1, -2 ** 31
    draw = lambda *s: torch.randn(s, generator=g, device="cuda").to(DT[dtype])
    return rows.view(T, k), draw(T, H), draw(R, H), torch.randn(T, k, generator=g, device="cuda")


def valid(rows, R):
    return (rows >= 0) & (rows < R)


def gathered(y, rows):
    ok = valid(rows, y.shape[0])
    return torch.where(ok[:, :, None], y[torch.where(ok, rows, 0).long()].double(), 0.0)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("T,k,H,R", SIZES)
def test_dispatch(T, k, H, R, dtype):
    say("dispatch", T, k, H, R, dtype)
    rows, x, _, _ = case(T, k, H, R, dtype)
    out, intact = guarded((R, H), DT[dtype], 5)
    assert gba.moe_dispatch(x, rows, out) is out
    torch.cuda.synchronize()
    intact()
    want = torch.full((R, H), 5, dtype=DT[dtype], device="cuda")
    ok = valid(rows, R)
    t = torch.arange(T, device="cuda")[:, None].expand(T, k)
    want[rows[ok].long()] = x[t[ok]]
    assert torch.equal(out, want)


@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("T,k,H,R", SIZES)
def test_combine(T, k, H, R, dtype, weighted):
    say("combine", T, k, H, R, dtype, weighted)
    rows, _, y, w = case(T, k, H, R, dtype)
    out, intact = guarded((T, H), DT[dtype], float("nan"))
    assert gba.moe_combine(y, rows, w if weighted else None, out) is out
    torch.cuda.synchronize()
    intact()
    v = gathered(y, rows)
    if weighted:
        v = v * w.double()[:, :, None]
    want = v.sum(1)
    eo.check("out", out, want, eo.with_rounding(want, k * 2.0 ** -24 * v.abs().sum(1), DT[dtype]))


@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("T,k,H,R", SIZES)
def test_combine_grad(T, k, H, R, dtype, weighted):
    say("combine grad", T, k, H, R, dtype, weighted)
    rows, dout, y, w = case(T, k, H, R, dtype)
    w = w if weighted else None
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
    # either alone
    one = torch.full((R, H), 5, dtype=DT[dtype], device="cuda")
    gba.moe_combine_grad(dout, y, rows, w, one, None)
    assert torch.equal(one, dy)
    other = torch.empty_like(dw)
    gba.moe_combine_grad(dout, y, rows, w, None, other)
    assert torch.equal(other, dw)


def test_a_weight_of_nan_shows_without_a_row():
    say("nan weight")
    rows, _, y, w = case(6, 2, 64, 12, "bf16")
    rows[2] = -1
    w[2, 1] = float("nan")
    out = torch.empty(6, 64, dtype=torch.bfloat16, device="cuda")
    gba.moe_combine(y, rows, w, out)
    assert torch.isnan(out[2]).all() and not torch.isnan(out[[0, 1, 3, 4, 5]]).any()


def test_nothing_to_do():
    say("nothing")
    e = lambda *s, dt=torch.bfloat16: torch.full(s, 3, dtype=dt, device="cuda")
    i = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")
    out = e(4, 16)
    gba.moe_dispatch(e(0, 16), i(0, 2), out)
    assert (out == 3).all()
    gba.moe_dispatch(e(2, 16), i(2, 2), e(0, 16))
    none = e(2, 16)
    gba.moe_combine(e(0, 16), i(2, 2), None, none)
    assert (none == 0).all()
    dw = torch.ones(2, 2, device="cuda")
    gba.moe_combine_grad(e(2, 16), e(0, 16), i(2, 2), None, e(0, 16), dw)
    assert (dw == 0).all()
    dw = torch.ones(2, 2, device="cuda")
    gba.moe_combine_grad(e(2, 0), e(3, 0), i(2, 2), None, e(3, 0), dw)
    assert (dw == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_the_moves_are_each_others_gradients(dtype):
    """<dispatch(x), y> = <x, combine(y)> and combine's gradients, against torch's of the plain form in 64 bits."""
    say("adjoint", dtype)
    T, k, H, R = 9, 3, 40, 30
    rows, x, y, w = case(T, k, H, R, dtype)
    x64, y64, w64 = (t.double().requires_grad_() for t in (x, y, w))
    ok = valid(rows, R)
    v = torch.where(ok[:, :, None], y64[torch.where(ok, rows, 0).long()], 0.0)
    (v * w64[:, :, None] * x64[:, None].detach()).sum().backward()
    dy, dw = torch.zeros_like(y), torch.empty_like(w)
    gba.moe_combine_grad(x, y, rows, w, dy, dw)
    eo.check("dy", dy, y64.grad, eo.with_rounding(y64.grad, 2.0 ** -24 * y64.grad.abs(), DT[dtype]))
    eo.check("dw", dw, w64.grad, 21 * 2.0 ** -24 * (v.detach() * x.double()[:, None]).abs().sum(2) + 2.0 ** -120)
    out, back = torch.zeros_like(y), torch.empty_like(x)
    gba.moe_dispatch(x, rows, out)
    gba.moe_combine(y, rows, None, back)
    a, b = (out.double() * y.double()).sum().item(), (x.double() * v.detach().sum(1)).sum().item()
    assert abs(a - b) <= 1e-12 * (out.double() * y.double()).abs().sum().item()
