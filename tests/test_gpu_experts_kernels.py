"""Every kernel of the grouped and 4-bit products against the plain 64-bit forms, at sizes that reach it
(tests/experts_cases.py): both weight layouts, both types, all activations, with bias and
pre-activations, NaN in the rows of no expert and infinities in the weights of empty experts."""
import pytest

import tiled_dense_gemm_bias_amd as gba
from tests import experts_cases as cases
from tests import experts_oracle as orc
from tests.gpu_util import say
from tests.test_gpu_experts import DT, draw, guarded, make_offsets, workspace

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.empty_cache()


def here(op, want, T, E, N, K, mib):
    """On this device too the call takes the kernel that the case is for."""
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    p = gba.experts.plan(op, T, E, N, K, mib * cases.MIB, cus)
    assert (p["tile_m"], p["tile_n"], p["persistent"], int(p["splits"] > 1), p["non_temporal"]) == want


def setup(what, i, case, seed):
    want, (sizes, lead, tail), cols, depth, mib = case
    say(what, i, want, sizes[:6], len(sizes), cols, depth)
    g = torch.Generator(device="cuda").manual_seed(seed + i)
    ws, intact = workspace(mib * cases.MIB) if mib else (None, lambda: None)
    return g, want, sizes, make_offsets(sizes, lead), lead + sum(sizes) + tail, len(sizes), cols, depth, mib, ws, intact


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("tb", [True, False])
@pytest.mark.parametrize("i", range(len(cases.ROWS)))
def test_forward(i, tb, dtype):
    g, plan, sizes, off, T, E, N, K, mib, ws, ws_intact = setup("kernel forward", i, cases.ROWS[i], 1000)
    here("forward", plan, T, E, N, K, mib)
    dt, act = DT[dtype], orc.ACTS[(i + 3 * tb) % 6]
    a, w = draw(g, (T, K), dt), draw(g, (E, N, K) if tb else (E, K, N), dt, K ** -0.5)
    bias = draw(g, (E, N), dt) if i % 4 != 3 else None
    want_z, err, owned = orc.product(a, off.tolist(), w, bias, tb)
    a[~owned] = float("nan")
    for e, n in enumerate(sizes):
        if n == 0:
            w[e] = float("inf")
    (c, c_intact), (z, z_intact) = guarded((T, N), dt), guarded((T, N), dt)
    gba.grouped_gemm_bias_act(a, off, w, bias, c, act, transpose_b=tb, preact=z, workspace=ws)
    torch.cuda.synchronize()
    c_intact(), z_intact(), ws_intact()
    orc.check("preact", z, want_z, orc.with_rounding(want_z, err, dt), owned)
    want = orc.act(act, want_z)
    orc.check("c", c, want, orc.with_rounding(want, orc.LIPSCHITZ[act] * err + orc.ACT_TOL, dt), owned)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("tb", [True, False])
@pytest.mark.parametrize("i", range(len(cases.ROWS)))
def test_act_grad(i, tb, dtype):
    g, plan, sizes, off, T, E, K, N, mib, ws, ws_intact = setup("kernel act_grad", i, cases.ROWS[i], 2000)
    here("act_grad", plan, T, E, N, K, mib)
    dt, act = DT[dtype], orc.ACTS[(i + 2 * tb + 1) % 6]
    dc, w = draw(g, (T, N), dt), draw(g, (E, N, K) if tb else (E, K, N), dt, N ** -0.5)
    z = draw(g, (T, K), dt, 1.5) if act != "none" else None
    d, err, owned = orc.product(dc, off.tolist(), w, None, not tb)
    s = orc.slope(act, z.double()) if z is not None else torch.ones_like(d)
    tol = 0.0 if z is None else orc.SLOPE_TOL
    dc[~owned] = float("nan")
    if z is not None:
        z[~owned] = float("nan")
    da, intact = guarded((T, K), dt)
    gba.grouped_gemm_act_grad(dc, off, w, z, da, act, transpose_b=tb, workspace=ws)
    torch.cuda.synchronize()
    intact(), ws_intact()
    orc.check("da", da, d * s, orc.with_rounding(d * s, s.abs() * err + tol * (d.abs() + err), dt), owned)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("i", range(len(cases.MX4)))
def test_mx4(i, dtype):
    g, plan, sizes, off, T, E, N, K, mib, ws, ws_intact = setup("kernel mx4", i, cases.MX4[i], 3000)
    here("mx4", plan, T, E, N, K, mib)
    dt, act = DT[dtype], orc.ACTS[(i + 4) % 6]
    x, w = draw(g, (T, K), dt), draw(g, (E * N, K), dt, K ** -0.5)
    bias = draw(g, (E, N), dt)

    def quantised(v):
        codes = torch.empty(v.shape[0], K // 2, dtype=torch.uint8, device="cuda")
        scales = torch.empty(gba.mx4_scales_shape(v.shape[0], K), dtype=torch.uint8, device="cuda")
        return gba.mx4_quantize(v, codes, scales)

    def values(v):
        return torch.cat([orc.mx4_values(*orc.mx4_quantize(p)) for p in v.split(max(1, (1 << 24) // K))])
    (ac, asc), (wc, wsc) = quantised(x), quantised(w)
    lead = off[0].item()
    owned = torch.zeros(T, dtype=torch.bool, device="cuda")
    owned[lead:lead + sum(sizes)] = True
    asc[:, ~owned] = 255                                   # rows of no expert: NaN
    (c, intact), dense = guarded((T, N), dt), E == 1
    if dense:
        gba.gemm_bias_act_mx4(ac, asc, wc, wsc, bias[0], c, act, workspace=ws)
    else:
        gba.grouped_gemm_bias_act_mx4(ac, asc, off, wc.view(E, N, K // 2), wsc, bias, c, act, workspace=ws)
    torch.cuda.synchronize()
    intact(), ws_intact()
    begin = lead
    for e, n in enumerate(sizes):                          # by expert: the 64-bit weights of all are gigabytes
        if n:
            z, err, _ = orc.product(values(x[begin:begin + n]), [0, n], values(w[e * N:(e + 1) * N])[None], bias[e:e + 1],
                                    True, mx4=True)
            want = orc.act(act, z)
            orc.check("c of expert %d" % e, c[begin:begin + n], want,
                      orc.with_rounding(want, orc.LIPSCHITZ[act] * err + orc.ACT_TOL, dt))
        begin += n
    assert torch.isnan(c[~owned]).all(), "rows of no expert were written"


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("tb", [True, False])
@pytest.mark.parametrize("out", ["own", "f32", "add"])
@pytest.mark.parametrize("i", range(len(cases.GRADS)))
def test_wgrad(i, out, tb, dtype):
    g, plan, sizes, off, T, E, N, K, mib, ws, ws_intact = setup("kernel wgrad", i, cases.GRADS[i], 4000)
    here("wgrad", plan, T, E, N, K, mib)
    dt = DT[dtype]
    a, dc = draw(g, (T, K), dt), draw(g, (T, N), dt)
    odt, start = dt if out == "own" else torch.float32, 0.5 if out == "add" else 0.0
    fill = 0.5 if out == "add" else float("nan")
    lead = off[0].item()
    owned = torch.zeros(T, dtype=torch.bool, device="cuda")
    owned[lead:lead + sum(sizes)] = True
    a64, dc64 = a.double(), dc.double()
    a[~owned], dc[~owned] = float("nan"), float("inf")
    results = []
    for with_bias in (False, True):
        dw, w_intact = guarded((E, N, K) if tb else (E, K, N), odt, fill)
        db, b_intact = guarded((E, N), odt, fill) if with_bias else (None, lambda: None)
        gba.grouped_gemm_wgrad(a, dc, off, dw, db, accumulate=out == "add", transpose_b=tb, workspace=ws)
        torch.cuda.synchronize()
        w_intact(), b_intact(), ws_intact()
        results.append((dw, db))
    for e, b, n in orc.groups(off.tolist(), T):
        x, d = a64[b:b + n], dc64[b:b + n]
        want, size = d.T.contiguous() @ x + start, d.T.abs().contiguous() @ x.abs() + start
        for dw, db in results:
            orc.check("dw of expert %d" % e, dw[e] if tb else dw[e].T, want,
                      orc.with_rounding(want, size * orc.sum_rel(n), odt))
        want = d.sum(0) + start
        orc.check("dbias of expert %d" % e, db[e], want, orc.with_rounding(want, (d.abs().sum(0) + start) * orc.sum_rel(n), odt))
