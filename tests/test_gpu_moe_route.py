"""Routing, its gradient and the sorting of slots against plain 64-bit forms: experts around the lanes'
edges, ties, masks that leave nothing, groups, NaN and infinities, every type and score."""
import math

import pytest

import tiled_dense_gemm_bias_amd as gba
from tests import experts_oracle as eo
from tests import moe_oracle as orc
from tests.gpu_util import say

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def guarded(shape, dtype, fill):
    n = math.prod(shape)
    whole = torch.full((n + 2048,), fill, dtype=dtype, device="cuda")
    whole[:1024] = 77
    whole[1024 + n:] = 77

    def intact():
        assert (whole[:1024] == 77).all() and (whole[1024 + n:] == 77).all(), "written outside the output"
    return whole[1024:1024 + n].view(shape), intact


def logits(seed, T, E, dtype, std=1.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(T, E, generator=g, device="cuda") * std).to(DT[dtype]), g


def run(x, k, bias=None, sort=True, **kw):
    T, E = x.shape
    idx, i1 = guarded((T, k), torch.int32, 12345)
    w, i2 = guarded((T, k), torch.float32, float("nan"))
    if not sort:
        gba.moe_route(x, idx, w, bias, **kw)
        torch.cuda.synchronize()
        i1(), i2()
        return idx, w
    off, i3 = guarded((E + 1,), torch.int32, 12345)
    rows, i4 = guarded((T, k), torch.int32, 12345)
    slots, i5 = guarded((T * k,), torch.int32, 12345)
    need = gba.moe_sort_workspace(T, E, k)
    ws, i6 = guarded((max(need, 4),), torch.uint8, 255)
    gba.moe_route(x, idx, w, bias, off, rows, slots, workspace=ws if need else None, **kw)
    torch.cuda.synchronize()
    for i in (i1, i2, i3, i4, i5, i6):
        i()
    return idx, w, off, rows, slots


def check_sorted(idx, off, rows, slots, E):
    o, r, s = orc.sort(idx.cpu(), E)
    assert off.tolist() == o
    assert rows.reshape(-1).tolist() == r
    assert slots is None or slots.tolist() == s


def check(x, k, bias=None, **kw):
    okw = {("renorm" if n == "renormalize" else n): v for n, v in kw.items()}
    want_idx, want_w, depth = orc.route(x, bias, k, **okw)
    idx, w, off, rows, slots = run(x, k, bias, **kw)
    same = idx.long() == want_idx
    assert same.all(), "first other choice at %s" % torch.nonzero(~same)[0].tolist()
    nan = torch.isnan(want_w)
    assert torch.equal(torch.isnan(w), nan)
    zero = torch.zeros_like(want_w)
    eo.check("weights", torch.where(nan, zero, w.double()), torch.where(nan, zero, want_w), orc.route_tol(torch.where(nan, zero, want_w), depth))
    check_sorted(idx, off, rows, slots, x.shape[1])
    i2, w2 = run(x, k, bias, sort=False, **kw)
    assert torch.equal(i2, idx) and torch.equal(w2.nan_to_num(7), w.nan_to_num(7))
    return idx, w


SIZES = [(1, 1, 1), (1, 8, 2), (3, 16, 16), (5, 17, 3), (33, 32, 32), (7, 33, 8), (64, 64, 6), (65, 65, 8), (31, 128, 17), (129, 129, 10),
         (300, 256, 8), (9, 257, 8), (40, 512, 10), (11, 513, 32), (17, 1000, 4), (5, 1024, 32), (1, 60, 4), (1000, 160, 6), (4099, 24, 3)]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k", SIZES)
def test_route(T, E, k, score, dtype):
    say("route", T, E, k, score, dtype)
    x, g = logits(T * 7 + E, T, E, dtype)
    check(x, k, score=score, renormalize=bool((T + E) % 2), scale=1.0 if k % 2 else 2.5)
    bias = torch.randn(E, generator=g, device="cuda") * 0.2
    check(x, k, bias, score=score, renormalize=bool((T + E + 1) % 2))


GROUPED = [(5, 8, 2, 2, 1), (33, 256, 8, 8, 4), (129, 160, 6, 8, 3), (17, 60, 4, 4, 2), (3, 512, 8, 8, 4), (9, 1024, 16, 16, 5), (65, 32, 3, 16, 2),
           (40, 24, 3, 8, 1), (7, 300, 10, 5, 2), (2, 1000, 5, 2, 1), (31, 16, 1, 16, 1), (8, 64, 8, 1, 1), (8, 64, 8, 4, 4)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k,groups,top", GROUPED)
def test_groups(T, E, k, groups, top, score, dtype):
    say("groups", T, E, k, groups, top, score, dtype)
    x, g = logits(T + E + k, T, E, dtype)
    x[0, : E // groups] = -math.inf                       # a group without experts
    if T > 2:
        x[1, 1:] = -math.inf                              # one expert left
        x[2] = -math.inf                                  # none
    bias = torch.randn(E, generator=g, device="cuda") * 0.2
    for best in (1, 2):
        for b in (None, bias):
            check(x, k, b, score=score, groups=groups, top_groups=top, group_best=best, renormalize=best == 1)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_ties_go_to_the_lowest_expert(dtype):
    say("ties", dtype)
    for E in (8, 40, 256, 1024):
        x = torch.zeros(4, E, dtype=DT[dtype], device="cuda")
        x[1] = -0.0
        x[1, ::2] = 0.0
        x[2] = -3.0
        x[3] = torch.arange(E, device="cuda") % 3
        bias = torch.zeros(E, device="cuda")
        for b in (None, bias):
            for score in ("softmax", "sigmoid"):
                idx, _ = check(x, min(E, 7), b, score=score)
                assert idx[0].tolist() == idx[1].tolist() == idx[2].tolist() == list(range(min(E, 7)))
        check(x, 4, bias, groups=4, top_groups=2, group_best=2)


def test_near_ties_are_settled_in_64_bits():
    """Values that 32-bit scores do not tell apart: pairs of logits a few steps apart under biases that
    almost cancel the difference."""
    say("near ties")
    g = torch.Generator(device="cuda").manual_seed(5)
    T, E = 2000, 64
    base = torch.randn(T, E // 2, generator=g, device="cuda")
    x = torch.stack([base, torch.nextafter(base, torch.full_like(base, 9.0))], 2).reshape(T, E)
    flip = torch.rand(T, E // 2, 1, generator=g, device="cuda") < 0.5
    x = torch.where(flip, x.view(T, -1, 2).flip(2), x.view(T, -1, 2)).reshape(T, E).contiguous()
    for score in ("sigmoid", "softmax"):
        check(x, 8, torch.zeros(E, device="cuda"), score=score)
        check(x, 8, torch.full((E,), -0.5, device="cuda"), score=score, groups=8, top_groups=3, group_best=2)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("E", [8, 100, 256, 700])
def test_masks_infinities_and_nan(E, dtype):
    say("masks", E, dtype)
    x, _ = logits(E, 12, E, dtype)
    low = torch.finfo(DT[dtype]).min
    x[0] = -math.inf
    x[1, 3:] = -math.inf
    x[2] = low
    x[3, 1:] = low
    x[4, 5] = math.nan
    x[5, 0] = math.inf
    x[6] = -200.0 if dtype != "f16" else -20.0
    x[7, :] = -math.inf
    x[7, E - 1] = low
    x[8] = 50.0
    k = 6
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            idx, w = check(x, k, score=score, renormalize=renorm)
            assert idx[0].tolist() == [-1] * k and w[0].tolist() == [0.0] * k
            assert idx[1].tolist()[3:] == [-1] * (k - 3)
            assert idx[4].tolist() == [-1] * k and torch.isnan(w[4]).all()
            if renorm and score == "sigmoid":
                assert abs(w[6].sum().item() - 1) < 1e-5          # scores that underflow keep their ratios
    bias = torch.zeros(E, device="cuda")
    bias[2], bias[3] = -math.inf, math.inf
    idx, _ = check(x, k, bias, score="sigmoid")
    assert not (idx == 2).any() and (idx[8, 0] == 3)
    bias[4] = math.nan
    idx, w = check(x, k, bias, score="softmax")
    assert (idx == -1).all() and torch.isnan(w).all()


@pytest.mark.parametrize("T,E,k", [(1, 4, 1), (100, 8, 8), (64, 300, 32), (65, 300, 32), (2049, 16, 1), (5000, 1024, 3), (16384, 2, 2), (20000, 7, 5),
                                   (300, 1000, 8), (40000, 64, 4)])
def test_sort(T, E, k):
    say("sort", T, E, k)
    g = torch.Generator(device="cuda").manual_seed(T + E)
    idx = torch.randint(-1, E, (T, k), generator=g, device="cuda", dtype=torch.int32)
    idx[T // 2:, 0] = E - 1
    if T > 10:
        idx[3:9] = torch.tensor([E, -5, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32, device="cuda")[:k].repeat(1, -(-k // 4))[:, :k]
    off, i1 = guarded((E + 1,), torch.int32, 5)
    rows, i2 = guarded((T, k), torch.int32, 5)
    slots, i3 = guarded((T * k,), torch.int32, 5)
    need = gba.moe_sort_workspace(T, E, k)
    ws, i4 = guarded((need + 8,), torch.uint8, 3)
    gba.moe_sort(idx, off, rows, slots, workspace=ws[:need] if need else None)
    torch.cuda.synchronize()
    for i in (i1, i2, i3, i4):
        i()
    check_sorted(idx, off, rows, slots, E)
    off2, rows2 = torch.empty_like(off), torch.empty_like(rows)
    gba.moe_sort(idx, off2, rows2, workspace=ws[:need] if need else None)
    assert torch.equal(off, off2) and torch.equal(rows, rows2)


def test_no_tokens():
    say("no tokens")
    e = lambda *s, dt=torch.int32: torch.full(s, 9, dtype=dt, device="cuda")
    off = e(6)
    gba.moe_route(e(0, 5, dt=torch.float32), e(0, 2), e(0, 2, dt=torch.float32), offsets=off, rows=e(0, 2))
    assert off.tolist() == [0] * 6
    off = e(6)
    gba.moe_sort(e(0, 2), off, e(0, 2), e(0))
    assert off.tolist() == [0] * 6
    gba.moe_route(e(0, 5, dt=torch.float32), e(0, 2), e(0, 2, dt=torch.float32))
    gba.moe_route_grad(e(0, 5, dt=torch.float32), e(0, 2), e(0, 2, dt=torch.float32), e(0, 5, dt=torch.float32))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (3, 8, 2), (33, 17, 5), (65, 64, 8), (129, 160, 17), (70, 256, 8), (9, 300, 32), (5, 1024, 10)])
def test_route_grad(T, E, k, renorm, score, dtype):
    say("route grad", T, E, k, renorm, score, dtype)
    x, g = logits(T + 3 * E, T, E, dtype)
    if T > 4:
        x[1, 1:] = -math.inf
        x[2] = -math.inf
        x[3] *= 20
    idx, _ = run(x, k, sort=False, score=score)
    dw = torch.randn(T, k, generator=g, device="cuda")
    dx, intact = guarded((T, E), DT[dtype], 5)
    assert gba.moe_route_grad(x, idx, dw, dx, score=score, renormalize=renorm, scale=1.5) is dx
    torch.cuda.synchronize()
    intact()
    want, size, depth = orc.route_grad(x, idx, dw, score, renorm, 1.5)
    err = (2 * depth[:, None] + 60) * 2.0 ** -24 * size + 2.0 ** -120
    eo.check("dx", dx, want, eo.with_rounding(want, err, DT[dtype]))
    if T > 4:
        assert (dx[2] == 0).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_grad_against_differences(score, renorm):
    """Central differences of the weights (in 64 bits, by the formulas of the forward pass): the step's square, 1e-8,
    and the differences' rounding, 2^-53 / 1e-4, are far below the 32-bit kernel's error."""
    say("differences", score, renorm)
    T, E, k, h = 6, 12, 3, 1e-4
    x, g = logits(11, T, E, "f32", std=1.0)
    idx, _ = run(x, k, sort=False, score=score)
    dw = torch.randn(T, k, generator=g, device="cuda")
    dx = torch.empty_like(x)
    gba.moe_route_grad(x, idx, dw, dx, score=score, renormalize=renorm)

    def loss(x64):
        s = torch.softmax(x64, 1) if score == "softmax" else torch.sigmoid(x64)
        w = s.gather(1, idx.long())
        if renorm:
            w = w / w.sum(1, keepdim=True)
        return (w * dw.double()).sum()
    for t in range(T):
        for e in range(E):
            d = torch.zeros(T, E, dtype=torch.float64, device="cuda")
            d[t, e] = h
            diff = ((loss(x.double() + d) - loss(x.double() - d)) / (2 * h)).item()
            assert abs(diff - dx[t, e].item()) < 1e-6 * (1 + dw.abs().max().item())


def test_a_repeated_expert_and_numbers_out_of_range():
    say("repeated")
    x, g = logits(3, 4, 20, "f32")
    idx = torch.tensor([[1, 1, 5], [20, -7, 3], [-1, -1, -1], [0, 19, 0]], dtype=torch.int32, device="cuda")
    dw = torch.randn(4, 3, generator=g, device="cuda")
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            dx = torch.empty_like(x)
            gba.moe_route_grad(x, idx, dw, dx, score=score, renormalize=renorm)
            legal = torch.where((idx >= 0) & (idx < 20), idx, -1)
            want, size, depth = orc.route_grad(x, legal, dw, score, renorm)
            eo.check("dx", dx, want, eo.with_rounding(want, (2 * depth[:, None] + 60) * 2.0 ** -24 * size + 2.0 ** -120, torch.float32))


# Around the sizes where the launches change: one workgroup for routing and sorting, tokens a workgroup, lanes a row.
BORDERS = [(32, 256, 8, 8, 4), (33, 256, 8, 8, 4), (32, 200, 6, 1, 1), (33, 200, 6, 1, 1), (64, 32, 4, 4, 2), (65, 32, 4, 4, 2), (63, 31, 3, 1, 1),
           (5, 288, 8, 8, 3), (64, 288, 32, 4, 2), (100, 512, 9, 16, 5), (70, 513, 9, 3, 2), (12300, 72, 3, 8, 3), (13001, 264, 4, 8, 2),
           (4097, 1024, 2, 16, 4), (20001, 96, 2, 12, 3)]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k,groups,top", BORDERS)
def test_borders(T, E, k, groups, top, score):
    say("borders", T, E, k, groups, top, score)
    x, g = logits(T + 5 * E, T, E, "f32")
    bias = torch.randn(E, generator=g, device="cuda") * 0.1
    x[T // 2, E // 3:] = -math.inf
    x[T - 1] = -math.inf
    check(x, k, bias, score=score, groups=groups, top_groups=top, group_best=2 if groups > 1 else 1, scale=2.5)
    check(x.bfloat16(), k, None, score=score, groups=groups, top_groups=top, renormalize=False)
