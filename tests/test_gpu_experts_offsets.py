"""Offsets in order that reach outside the rows, for every product: the rows are those of the clamped
offsets, and nothing else is written. (Offsets that decrease are the business of tests/test_experts_groups_cpu.py:
their rows are not defined, only that they lie in the arrays.)"""
import pytest

import tiled_dense_gemm_bias_amd as gba
from tests import experts_oracle as orc
from tests.gpu_util import say
from tests.test_gpu_experts import DT, draw, guarded, workspace

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

LOW, HIGH, MIB = -2 ** 31, 2 ** 31 - 1, 1 << 20


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.empty_cache()


def lists(T, E):
    """E + 1 entries each, in order."""
    inner = [T * i // E for i in range(1, E)]
    yield [-7] + inner + [T + 4000]
    yield [LOW] + inner[:-1] + [HIGH, HIGH] if E > 1 else [LOW, HIGH]
    yield [T // 2] * E + [HIGH]
    yield [LOW] * E + [T // 3]
    yield [HIGH] * (E + 1)
    yield [LOW] * (E + 1)


# rows, experts, columns, depth of 16-bit operands, workspace MiB, persistent, splits
SIZES = [(40, 4, 72, 4104, 8, 0, 1), (2600, 4, 3080, 416, 0, 1, 0), (2600, 6, 3080, 416, 8, 1, 0), (500, 70, 136, 264, 0, 0, 0)]


def setup(what, op, size, dtype, scale=1):
    T, E, cols, depth, mib, big, split = size
    depth *= scale
    N, K = (depth, cols) if op == "act_grad" else (cols, depth)
    p = gba.experts.plan(op, T, E, N, K, mib * MIB, torch.cuda.get_device_properties(0).multi_processor_count)
    assert p["persistent"] == big and (p["splits"] > 1) == bool(split)
    return T, E, N, K, DT[dtype], workspace(mib * MIB) if mib else (None, lambda: None), torch.Generator(device="cuda").manual_seed(T + E)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("size", SIZES)
def test_forward_and_input_gradient(size, dtype):
    for op in ("forward", "act_grad"):
        T, E, N, K, dt, (ws, ws_intact), g = setup(op, op, size, dtype)
        x = draw(g, (T, K if op == "forward" else N), dt)
        w = draw(g, (E, N, K), dt, x.shape[1] ** -0.5)
        z = draw(g, (T, K), dt)
        for o in lists(T, E):
            say("offsets", op, size, dtype, o[:8])
            off = torch.tensor(o, dtype=torch.int32, device="cuda")
            out, intact = guarded((T, N if op == "forward" else K), dt)
            if op == "forward":
                want, err, owned = orc.product(x, o, w, None, True)
                gba.grouped_gemm_bias_act(x, off, w, None, out, "none", transpose_b=True, workspace=ws)
            else:
                d, err, owned = orc.product(x, o, w, None, False)
                s = orc.slope("sigmoid", z.double())
                want, err = d * s, s * err + orc.SLOPE_TOL * (d.abs() + err)
                gba.grouped_gemm_act_grad(x, off, w, z, out, "sigmoid", transpose_b=True, workspace=ws)
            torch.cuda.synchronize()
            intact(), ws_intact()
            orc.check(op, out, want, orc.with_rounding(want, err, dt), owned)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("size", [(8000, 4, 72, 136, 8, 0, 1), (2600, 4, 3080, 416, 0, 1, 0), (500, 70, 72, 104, 0, 0, 0)])
def test_weight_and_bias_gradients(size, dtype):
    T, E, N, K, dt, (ws, ws_intact), g = setup("wgrad", "wgrad_bias", size, dtype)
    a, dc = draw(g, (T, K), dt), draw(g, (T, N), dt)
    for o in lists(T, E):
        say("offsets", "wgrad", size, dtype, o[:8])
        (dw, w_intact), (db, b_intact) = guarded((E, N, K), torch.float32), guarded((E, N), torch.float32)
        gba.grouped_gemm_wgrad(a, dc, torch.tensor(o, dtype=torch.int32, device="cuda"), dw, db, transpose_b=True, workspace=ws)
        torch.cuda.synchronize()
        w_intact(), b_intact(), ws_intact()
        for e, b, n in orc.groups(o, T):
            x, d = a[b:b + n].double(), dc[b:b + n].double()
            want, size64 = d.T.contiguous() @ x, d.T.abs().contiguous() @ x.abs()
            orc.check("dw", dw[e], want, orc.with_rounding(want, size64 * orc.sum_rel(n), torch.float32))
            orc.check("db", db[e], d.sum(0), orc.with_rounding(d.sum(0), d.abs().sum(0) * orc.sum_rel(n), torch.float32))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("size", SIZES)
def test_product_in_4_bits(size, dtype):
    T, E, N, K, dt, (ws, ws_intact), g = setup("mx4", "mx4", size, dtype, 4)
    x, w = draw(g, (T, K), dt), draw(g, (E * N, K), dt, K ** -0.5)
    (ac, asc), (wc, wsc) = (gba.mx4_quantize(v, torch.empty(v.shape[0], K // 2, dtype=torch.uint8, device="cuda"),
                                             torch.empty(gba.mx4_scales_shape(v.shape[0], K), dtype=torch.uint8, device="cuda"))
                            for v in (x, w))
    a64, w64 = (torch.cat([orc.mx4_values(*orc.mx4_quantize(p)) for p in v.split(max(1, (1 << 24) // K))]) for v in (x, w))
    for o in lists(T, E):
        say("offsets", "mx4", size, dtype, o[:8])
        want, err, owned = orc.product(a64, o, w64.view(E, N, K), None, True, mx4=True)
        c, intact = guarded((T, N), dt)
        gba.grouped_gemm_bias_act_mx4(ac, asc, torch.tensor(o, dtype=torch.int32, device="cuda"), wc.view(E, N, K // 2), wsc,
                                      None, c, "none", workspace=ws)
        torch.cuda.synchronize()
        intact(), ws_intact()
        orc.check("c", c, want, orc.with_rounding(want, err, dt), owned)
