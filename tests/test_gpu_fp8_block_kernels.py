"""Every kernel of the 8-bit products against the 64-bit definition, at sizes that reach it (tests/moe_cases.py), forward
and as a gradient: both types, all activations, NaN in the rows of no expert and in the scales of empty experts."""
import pytest

import tiled_dense_gemm_bias_amd as gba
from tests import experts_oracle as eo
from tests import moe_cases as cases
from tests import moe_oracle as orc
from tests.gpu_util import say
from tests.test_gpu_experts import draw, make_offsets, workspace
from tests.test_gpu_experts import guarded as guarded16
from tests.test_gpu_fp8_block import DT, F8, quantised, spread
from tiled_dense_gemm_bias_amd import moe

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.empty_cache()


def setup(what, case, dtype, seed):
    want, sizes, lead, tail, N, K, mib = case
    say(what, want, sizes[:8], len(sizes), N, K, dtype)
    T, E, dt = lead + sum(sizes) + tail, len(sizes), DT[dtype]
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    p = moe.plan(T, E, N, K, mib * cases.MIB, cus)
    assert (p["kind"], p["tile_m"], p["tile_n"], p["splits"] > 1) == want
    g = torch.Generator(device="cuda").manual_seed(seed + T + N + K)
    x, w = spread(g, (T, K), dt), draw(g, (E, N, K), dt, K ** -0.5)
    ac, asc = quantised(x)
    wc, wsc = torch.empty(E, N, K, dtype=F8, device="cuda"), torch.empty(gba.fp8_weight_scales_shape(E, N, K), device="cuda")
    gba.fp8_quantize_weights(w, wc, wsc)
    a64 = orc.values(ac.view(torch.uint8), asc.T.contiguous())
    w64 = torch.stack([orc.values(wc[e].view(torch.uint8), wsc[e], 128) for e in range(E)])
    off = make_offsets(sizes, lead)
    sums, err, owned = orc.product(a64, off.tolist(), w64, None)
    asc[:, ~owned] = float("nan")
    for e, n in enumerate(sizes):
        if n == 0:
            wsc[e] = float("nan")
    ws, intact = workspace(mib * cases.MIB) if mib else (None, lambda: None)
    return g, T, E, N, (ac, asc, off, wc, wsc), sums, err, owned, ws, intact


def check_forward(s, dt, act, preact):
    g, T, E, N, args, sums, err, owned, ws, ws_intact = s
    bias = draw(g, (E, N), dt)
    owner = torch.zeros(T, dtype=torch.long, device="cuda")
    off = args[2].tolist()
    for e in range(E):
        owner[off[e]:off[e + 1]] = e
    want_z = sums + bias.double()[owner]
    zerr = err + 2.0 ** -23 * (sums.abs() + bias.double()[owner].abs())    # the bias' sum, rounded to 32 bits
    (c, c_intact), (z, z_intact) = guarded16((T, N), dt), guarded16((T, N), dt)
    gba.grouped_gemm_bias_act_fp8_block(*args, bias, c, act, preact=z if preact else None, workspace=ws)
    torch.cuda.synchronize()
    c_intact(), z_intact(), ws_intact()
    want = eo.act(act, want_z)
    eo.check("c", c, want, eo.with_rounding(want, eo.LIPSCHITZ[act] * zerr + eo.ACT_TOL, dt), owned)
    if preact:
        eo.check("z", z, want_z, eo.with_rounding(want_z, zerr, dt), owned)
    assert torch.isnan(c[~owned]).all()


def check_grad(s, dt, act):
    g, T, E, N, args, sums, err, owned, ws, ws_intact = s
    z = draw(g, (T, N), dt, 1.5) if act != "none" else None
    slope = eo.slope(act, z.double()) if z is not None else torch.ones_like(sums)
    if z is not None:
        z[~owned] = float("nan")
    da, intact = guarded16((T, N), dt)
    gba.grouped_gemm_act_grad_fp8_block(*args, z, da, act, workspace=ws)
    torch.cuda.synchronize()
    intact(), ws_intact()
    want = sums * slope
    eo.check("da", da, want, eo.with_rounding(want, err * slope.abs() + eo.SLOPE_TOL * (sums.abs() + err), dt), owned)
    assert torch.isnan(da[~owned]).all()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("i", range(len(cases.PRODUCTS)))
def test_each_kernel(i, dtype):
    s = setup("kernel", cases.PRODUCTS[i], dtype, 100)
    check_forward(s, DT[dtype], eo.ACTS[i % 6], i % 2 == 0)
    check_grad(s, DT[dtype], eo.ACTS[(i + 2) % 6])


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("kind", ["persistent", "stream", "ring"])
def test_each_activation(kind, dtype):
    s = setup("activations", next(c for c in reversed(cases.PRODUCTS) if c[0][0] == kind and not c[0][3]), dtype, 200)
    for act in eo.ACTS:
        for preact in (False, True):
            check_forward(s, DT[dtype], act, preact)
        check_grad(s, DT[dtype], act)
