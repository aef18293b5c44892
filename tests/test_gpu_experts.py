"""Grouped products against plain 64-bit forms: group sizes around the tiles'
edges, empty experts, rows of no expert, odd depths and widths, both weight
layouts, both types, all activations, guards around every output."""
import pytest

import tiled_dense_gemm_bias_amd as gba
from tests import experts_oracle as orc
from tests.gpu_util import say

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

DT = {"f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def draw(g, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def guarded(shape, dtype, fill=float("nan")):
    """A tensor filled with `fill` inside a larger one, and a check that nothing around it was written."""
    n = 1
    for d in shape:
        n *= d
    whole = torch.full((n + 4096,), fill, dtype=dtype, device="cuda")
    whole[:2048] = 7.0
    whole[2048 + n:] = 7.0

    def intact():
        assert (whole[:2048] == 7).all() and (whole[2048 + n:] == 7).all(), "written outside the output"
    return whole[2048:2048 + n].view(shape), intact


def workspace(size=8 << 20):
    """A workspace of NaN, and a check that nothing past it was written."""
    whole = torch.full((size // 4 + 1024,), float("nan"), device="cuda")
    whole[size // 4:] = 7.0

    def intact():
        assert (whole[size // 4:] == 7).all(), "written outside the workspace"
    return whole[:size // 4], intact


def make_offsets(sizes, lead=0):
    o = [lead]
    for n in sizes:
        o.append(o[-1] + n)
    return torch.tensor(o, dtype=torch.int32, device="cuda")


# (rows by expert, rows before the first, rows after the last, N, K)
SHAPES = [
    ([1], 0, 0, 8, 8),
    ([1], 0, 0, 1000, 520),
    ([0, 3, 0], 0, 0, 72, 64),
    ([5, 0, 16, 17, 1], 0, 0, 136, 72),
    ([15, 1, 0, 2], 2, 3, 264, 200),
    ([63, 65, 64], 0, 0, 200, 136),
    ([0, 0, 300, 0], 1, 5, 64, 1000),
    ([127, 129, 128, 1], 0, 0, 264, 328),
    ([257, 0, 255, 511], 3, 0, 520, 264),
    ([1] * 70 + [0] * 30 + [2] * 30, 0, 1, 40, 128),
    ([400, 37], 0, 0, 1032, 64),
    ([0, 0], 0, 4, 16, 16),
]


# Sizes that the 256 x 256 persistent kernels take (many row tiles, wide outputs),
# with row, column and depth edges, empty experts, more experts than lanes, one tile more than a round.
BIG = [
    ([257, 0, 511, 300, 1000], 0, 0, 8200, 72),
    ([513, 255], 3, 7, 12296, 200),
    ([1, 700, 0, 0, 900], 0, 0, 8192, 128),
    ([200] * 70, 0, 0, 1032, 136),
    ([4096], 1, 0, 3080, 264),
    ([300, 2000, 1, 0, 1000, 640], 0, 2, 4104, 1000),
]
# Few output tiles and a long sum: split over K where a workspace is given.
DEEP = [
    ([3, 0, 20], 1, 2, 264, 4096),
    ([100], 0, 0, 256, 4104),
    ([1], 0, 0, 72, 3080),
    ([0, 70, 0, 1], 0, 3, 520, 2056),
]
DEEP_GRAD = [
    ([5000], 0, 0, 136, 200),
    ([1500, 0, 3], 1, 1, 72, 264),
    ([3000, 700], 0, 2, 512, 320),
]
BIG_GRAD = [
    ([257, 0, 511, 1, 64], 0, 0, 2056, 1544),
    ([65, 1000, 63, 300], 2, 5, 1800, 2048),
    ([2000], 0, 0, 4104, 3080),
]


def build(seed, sizes, lead, tail, dtype):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return g, make_offsets(sizes, lead), lead + sum(sizes) + tail, len(sizes)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("tb", [True, False])
@pytest.mark.parametrize("i", range(len(SHAPES + BIG + DEEP)))
def test_forward(i, tb, dtype):
    sizes, lead, tail, N, K = (SHAPES + BIG + DEEP)[i]
    dt, act = DT[dtype], orc.ACTS[(i + tb) % 6]
    say("forward", i, sizes[:8], N, K, tb, dtype, act)
    g, off, T, E = build(100 + i, sizes, lead, tail, dt)
    a = draw(g, (T, K), dt)
    w = draw(g, (E, N, K) if tb else (E, K, N), dt, K ** -0.5)
    bias = draw(g, (E, N), dt) if i % 3 else None
    z, z_intact = guarded((T, N), dt)
    c, c_intact = guarded((T, N), dt)
    want_z, err, owned = orc.product(a, off.tolist(), w, bias, tb)
    # What belongs to no expert, or to an empty one, may hold anything.
    a[~owned] = float("nan")
    for e, n in enumerate(sizes):
        if n == 0:
            w[e] = float("inf")
    assert gba.grouped_gemm_bias_act(a, off, w, bias, c, act, transpose_b=tb, preact=z) is c
    torch.cuda.synchronize()
    z_intact(), c_intact()
    orc.check("preact", z, want_z, orc.with_rounding(want_z, err, dt), owned)
    want = orc.act(act, want_z)
    orc.check("c", c, want, orc.with_rounding(want, orc.LIPSCHITZ[act] * err + orc.ACT_TOL, dt), owned)
    c2, _ = guarded((T, N), dt)
    gba.grouped_gemm_bias_act(a, off, w, bias, c2, act, transpose_b=tb)
    assert torch.equal(c2[owned], c[owned])
    c3, intact = guarded((T, N), dt)
    z3, z3_intact = guarded((T, N), dt)
    ws, ws_intact = workspace()
    gba.grouped_gemm_bias_act(a, off, w, bias, c3, act, transpose_b=tb, preact=z3, workspace=ws)
    torch.cuda.synchronize()
    intact(), z3_intact(), ws_intact()
    orc.check("preact, workspace", z3, want_z, orc.with_rounding(want_z, err, dt), owned)
    orc.check("c, workspace", c3, want, orc.with_rounding(want, orc.LIPSCHITZ[act] * err + orc.ACT_TOL, dt), owned)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("tb", [True, False])
@pytest.mark.parametrize("i", range(len(SHAPES + BIG + DEEP)))
def test_act_grad(i, tb, dtype):
    sizes, lead, tail, K, N = (SHAPES + BIG + DEEP)[i]
    dt, act = DT[dtype], orc.ACTS[(i + 2 * tb) % 6]
    say("act_grad", i, sizes[:8], N, K, tb, dtype, act)
    g, off, T, E = build(200 + i, sizes, lead, tail, dt)
    dc = draw(g, (T, N), dt)
    w = draw(g, (E, N, K) if tb else (E, K, N), dt, N ** -0.5)
    z = draw(g, (T, K), dt, 1.5) if act != "none" else None
    d, err, owned = orc.product(dc, off.tolist(), w, None, not tb)
    dc[~owned] = float("nan")
    da, intact = guarded((T, K), dt)
    assert gba.grouped_gemm_act_grad(dc, off, w, z, da, act, transpose_b=tb) is da
    torch.cuda.synchronize()
    intact()
    s = orc.slope(act, z.double()) if z is not None else torch.ones_like(d)
    tol = 0.0 if z is None else orc.SLOPE_TOL
    bound = orc.with_rounding(d * s, s.abs() * err + tol * (d.abs() + err), dt)
    orc.check("da", da, d * s, bound, owned)
    da2, intact = guarded((T, K), dt)
    ws, ws_intact = workspace()
    gba.grouped_gemm_act_grad(dc, off, w, z, da2, act, transpose_b=tb, workspace=ws)
    torch.cuda.synchronize()
    intact(), ws_intact()
    orc.check("da, workspace", da2, d * s, bound, owned)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("tb", [True, False])
@pytest.mark.parametrize("out", ["own", "f32", "add"])
@pytest.mark.parametrize("i", range(len(SHAPES + BIG_GRAD + DEEP_GRAD)))
def test_wgrad(i, out, tb, dtype):
    sizes, lead, tail, N, K = (SHAPES + BIG_GRAD + DEEP_GRAD)[i]
    dt = DT[dtype]
    say("wgrad", i, sizes[:8], N, K, out, tb, dtype)
    g, off, T, E = build(300 + i, sizes, lead, tail, dt)
    a, dc = draw(g, (T, K), dt), draw(g, (T, N), dt)
    odt = dt if out == "own" else torch.float32
    fill = 0.5 if out == "add" else float("nan")
    dw, w_intact = guarded((E, N, K) if tb else (E, K, N), odt, fill)
    db, b_intact = guarded((E, N), odt, fill)
    start = 0.5 if out == "add" else 0.0
    want, bound = torch.empty(E, N, K, dtype=torch.float64, device="cuda"), torch.empty(E, N, K, dtype=torch.float64, device="cuda")
    want_b, bound_b = torch.empty(E, N, dtype=torch.float64, device="cuda"), torch.empty(E, N, dtype=torch.float64, device="cuda")
    owned = torch.zeros(T, dtype=torch.bool, device="cuda")
    for e, b, n in orc.groups(off.tolist(), T):
        x, d = a[b:b + n].double(), dc[b:b + n].double()
        want[e], want_b[e] = d.T.contiguous() @ x + start, d.sum(0) + start
        size = d.T.abs().contiguous() @ x.abs() + start
        bound[e] = orc.with_rounding(want[e], size * orc.sum_rel(n), odt)
        bound_b[e] = orc.with_rounding(want_b[e], (d.abs().sum(0) + start) * orc.sum_rel(n), odt)
        owned[b:b + n] = True
    a[~owned], dc[~owned] = float("nan"), float("inf")
    assert gba.grouped_gemm_wgrad(a, dc, off, dw, db, accumulate=out == "add", transpose_b=tb) is dw
    torch.cuda.synchronize()
    w_intact(), b_intact()
    orc.check("dw", dw if tb else dw.transpose(1, 2), want, bound)
    orc.check("dbias", db, want_b, bound_b)
    dw2, intact = guarded(dw.shape, odt, fill)
    ws, ws_intact = workspace()
    gba.grouped_gemm_wgrad(a, dc, off, dw2, None, accumulate=out == "add", transpose_b=tb, workspace=ws)
    torch.cuda.synchronize()
    intact(), ws_intact()
    orc.check("dw, workspace", dw2 if tb else dw2.transpose(1, 2), want, bound)
    again = torch.full_like(dw, fill)
    gba.grouped_gemm_wgrad(a, dc, off, again, None, accumulate=out == "add", transpose_b=tb)
    assert torch.equal(again, dw)


@pytest.mark.parametrize("act", orc.ACTS)
def test_slopes_over_all_values(act):
    """act' of every finite bf16 value and of the infinities: dc . 1 . act'(z)."""
    say("slopes", act)
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).cuda()
    z = bits[:65536].reshape(-1, 8).contiguous()
    T = z.shape[0]
    dc = torch.zeros(T, 8, dtype=torch.bfloat16, device="cuda")
    dc[:, 0] = 1
    w = torch.zeros(1, 8, 8, dtype=torch.bfloat16, device="cuda")
    w[0, 0] = 1
    da = torch.empty_like(z)
    gba.grouped_gemm_act_grad(dc, make_offsets([T]), w, z, da, act, transpose_b=True)
    zf = z.double()
    want = orc.slope(act, zf.clamp(-1e4, 1e4))
    nan = torch.isnan(zf)
    if act != "none":
        assert torch.isnan(da[nan]).all()
    ok = ~nan
    orc.check(act, da[ok], want[ok], orc.with_rounding(want[ok], torch.full_like(want[ok], orc.SLOPE_TOL), torch.bfloat16))


def test_offsets_outside_the_rows_are_clamped():
    T, E, N, K = 40, 4, 64, 64
    g = torch.Generator(device="cuda").manual_seed(5)
    a, w = draw(g, (T, K), torch.float16), draw(g, (E, N, K), torch.float16, K ** -0.5)
    for o in ([-7, 10, 10, 30, 4000], [0, 0, 0, 0, 2 ** 31 - 1], [2 ** 31 - 1] * 5, [-2 ** 31] * 5):
        say("clamp", o)
        off = torch.tensor(o, dtype=torch.int32, device="cuda")
        want, err, owned = orc.product(a, o, w, None, True)
        c, intact = guarded((T, N), torch.float16)
        gba.grouped_gemm_bias_act(a, off, w, None, c, "none", transpose_b=True)
        torch.cuda.synchronize()
        intact()
        orc.check("c", c, want, orc.with_rounding(want, err, torch.float16), owned)


def test_depth_zero_and_no_rows():
    off = make_offsets([3, 2])
    bias = torch.randn(2, 16, device="cuda").half()
    c, z = (torch.empty(5, 16, dtype=torch.float16, device="cuda") for _ in range(2))
    gba.grouped_gemm_bias_act(torch.empty(5, 0, dtype=torch.float16, device="cuda"), off,
                              torch.empty(2, 16, 0, dtype=torch.float16, device="cuda"), bias, c, "relu", transpose_b=True, preact=z)
    want = bias.repeat_interleave(torch.tensor([3, 2], device="cuda"), 0)
    assert torch.equal(z, want) and torch.equal(c, want.clamp(min=0))
    none = torch.empty(0, 16, dtype=torch.float16, device="cuda")
    dw, db = (torch.full(s, 9.0, dtype=torch.float16, device="cuda") for s in ((2, 16, 16), (2, 16)))
    gba.grouped_gemm_wgrad(none, none, make_offsets([0, 0]), dw, db)
    assert (dw == 0).all() and (db == 0).all()
    gba.grouped_gemm_bias_act(none, make_offsets([0, 0]), dw, db, none.clone(), "gelu")


def test_non_finite_values_stay_in_their_rows():
    T, E, N, K = 70, 2, 136, 264
    g = torch.Generator(device="cuda").manual_seed(6)
    a, w = draw(g, (T, K), torch.bfloat16), draw(g, (E, N, K), torch.bfloat16, K ** -0.5)
    off = make_offsets([33, 37])
    clean = torch.empty(T, N, dtype=torch.bfloat16, device="cuda")
    gba.grouped_gemm_bias_act(a, off, w, None, clean, "none", transpose_b=True)
    a[32, 5], a[40, 7], w[1, 9, 3] = float("inf"), float("nan"), float("nan")
    c = torch.empty_like(clean)
    gba.grouped_gemm_bias_act(a, off, w, None, c, "none", transpose_b=True)
    assert torch.isnan(c[40]).all() and torch.isnan(c[33:, 9]).all() and not torch.isfinite(c[32]).any()
    rows = [r for r in range(T) if r not in (32, 40)]
    cols = [n for n in range(N) if n != 9]
    assert torch.equal(c[rows][:, cols], clean[rows][:, cols]) and torch.equal(c[:32, 9], clean[:32, 9])


def test_gradients_match_differences():
    """The three calls together are the gradient of sum(g . gelu(a w1 + b1) w2): against central
    differences of the 64-bit function, with the kernels' 16-bit roundings allowed for."""
    sizes, D, F = [9, 0, 30], 64, 96
    g = torch.Generator(device="cuda").manual_seed(11)
    off, T, E = make_offsets(sizes), sum(sizes), len(sizes)
    dt = torch.float16
    a, w1, b1, w2 = (draw(g, s, dt, f) for s, f in (((T, D), 1), ((E, F, D), D ** -0.5), ((E, F), 0.3), ((E, D, F), F ** -0.5)))
    dy = draw(g, (T, D), dt)
    z, h = torch.empty(T, F, dtype=dt, device="cuda"), torch.empty(T, F, dtype=dt, device="cuda")
    gba.grouped_gemm_bias_act(a, off, w1, b1, h, "gelu", transpose_b=True, preact=z)
    dz, da = torch.empty_like(z), torch.empty_like(a)
    gba.grouped_gemm_act_grad(dy, off, w2, z, dz, "gelu", transpose_b=True)
    gba.grouped_gemm_act_grad(dz, off, w1, None, da, "none", transpose_b=True)
    dw1, db1 = torch.empty(E, F, D, dtype=torch.float32, device="cuda"), torch.empty(E, F, dtype=torch.float32, device="cuda")
    gba.grouped_gemm_wgrad(a, dz, off, dw1, db1, transpose_b=True)

    def loss(a, w1, b1):
        total = 0.0
        for e, b, n in orc.groups(off.tolist(), T):
            hh = orc.act("gelu", a[b:b + n] @ w1[e].T + b1[e])
            total = total + (dy[b:b + n].double() * (hh @ w2[e].double().T)).sum()
        return total
    args = [t.double() for t in (a, w1, b1)]
    for k, grad in enumerate((da, dw1, db1)):
        way = torch.randn(args[k].shape, generator=g, device="cuda", dtype=torch.float64)
        h_ = 1e-5
        plus, minus = list(args), list(args)
        plus[k], minus[k] = args[k] + h_ * way, args[k] - h_ * way
        diff = (loss(*plus) - loss(*minus)) / (2 * h_)
        got = (grad.double() * way).sum()
        # Each of the products' inputs was rounded to 2^-11 of itself: a random
        # sum of that size, four of them, against the norm of what is summed.
        assert abs(got - diff) <= 8 * 2.0 ** -11 * (grad.double() * way).norm(), (k, got.item(), diff.item())


def test_another_stream_and_the_same_bits_again():
    T, E, N, K = 300, 5, 264, 520
    g = torch.Generator(device="cuda").manual_seed(7)
    a, w = draw(g, (T, K), torch.bfloat16), draw(g, (E, N, K), torch.bfloat16, K ** -0.5)
    off = make_offsets([10, 0, 200, 89, 1])
    first = torch.empty(T, N, dtype=torch.bfloat16, device="cuda")
    gba.grouped_gemm_bias_act(a, off, w, None, first, "gelu", transpose_b=True)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(3):
        c = torch.empty_like(first)
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            gba.grouped_gemm_bias_act(a, off, w, None, c, "gelu", transpose_b=True)
        s.synchronize()
        assert torch.equal(c, first)
