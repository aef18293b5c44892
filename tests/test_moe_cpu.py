"""Refusals of libgba_moe and of its binding, without a GPU: every argument error is reported
before a device is touched. Also the plain forms themselves, against values worked out by hand."""
import ctypes
import math
import re

import pytest

import tiled_dense_gemm_bias_amd as gba
from tests.test_abi_cpu import _gpu_present

moe = gba.moe
torch = pytest.importorskip("torch")

OK, NULL, SHAPE, DTYPE, ACT, ALIGN, ALIAS, DEVICE = range(8)
SCRATCH = 12
BIG = 1 << 40


def at(i):
    """16-byte aligned fake addresses, far apart, never followed."""
    return 0x10000 + i * BIG


@pytest.fixture(scope="module")
def lib():
    return moe.moe_lib()


def route(lib, x=at(1), bias=at(2), idx=at(3), w=at(4), off=at(5), rows=at(6), slots=at(7), T=64, E=16, k=2, groups=1, top=1, best=1,
          score=0, scale=1.0, dt=2, flags=1, ws=None, nb=0):
    return lib.moe_route(x, bias, idx, w, off, rows, slots, T, E, k, groups, top, best, score, scale, dt, flags, ws, nb)


def grad(lib, x=at(1), idx=at(2), dw=at(3), dx=at(4), T=64, E=16, k=2, score=0, scale=1.0, dt=2, flags=1):
    return lib.moe_route_grad(x, idx, dw, dx, T, E, k, score, scale, dt, flags)


def sort(lib, idx=at(1), off=at(2), rows=at(3), slots=at(4), T=64, E=16, k=2, ws=None, nb=0):
    return lib.moe_sort(idx, off, rows, slots, T, E, k, ws, nb)


def dispatch(lib, x=at(1), rows=at(2), out=at(3), T=8, k=2, H=64, R=16, dt=0):
    return lib.moe_dispatch(x, rows, out, T, k, H, R, dt)


def combine(lib, y=at(1), rows=at(2), w=at(4), out=at(3), T=8, k=2, H=64, R=16, dt=0):
    return lib.moe_combine(y, rows, w, out, T, k, H, R, dt)


def cgrad(lib, x=at(1), y=at(5), rows=at(2), w=at(4), out=at(3), dw=at(6), T=8, k=2, H=64, R=16, dt=0):
    return lib.moe_combine_grad(x, y, rows, w, out, dw, T, k, H, R, dt)


def quant(lib, x=at(1), rows=at(2), out=at(3), s=at(4), T=8, k=2, H=64, R=16, dt=0, flags=0):
    return lib.fp8_quantize(x, rows, out, s, T, k, H, R, dt, flags)


def weights(lib, w=at(1), c=at(2), s=at(3), ct=at(4), st=at(5), E=2, N=64, K=64, dt=0, flags=0):
    return lib.fp8_quantize_weights(w, c, s, ct, st, E, N, K, dt, flags)


def fwd(lib, a=at(1), asc=at(2), off=at(3), w=at(4), wsc=at(5), bias=at(6), C=at(7), z=at(8), T=64, E=4, N=64, K=64, act=3, dt=0, ws=None, nb=0):
    return lib.grouped_gemm_bias_act_fp8_block(a, asc, off, w, wsc, bias, C, z, T, E, N, K, act, dt, ws, nb)


def dense(lib, a=at(1), asc=at(2), w=at(4), wsc=at(5), bias=at(6), C=at(7), z=at(8), T=64, N=64, K=64, act=3, dt=0, ws=None, nb=0):
    return lib.gemm_bias_act_fp8_block(a, asc, w, wsc, bias, C, z, T, N, K, act, dt, ws, nb)


def dgrad(lib, a=at(1), asc=at(2), off=at(3), w=at(4), wsc=at(5), z=at(6), C=at(7), T=64, E=4, N=64, K=64, act=3, dt=0, ws=None, nb=0):
    return lib.grouped_gemm_act_grad_fp8_block(a, asc, off, w, wsc, z, C, T, E, N, K, act, dt, ws, nb)


def dense_dgrad(lib, a=at(1), asc=at(2), w=at(4), wsc=at(5), z=at(6), C=at(7), T=64, N=64, K=64, act=3, dt=0, ws=None, nb=0):
    return lib.gemm_act_grad_fp8_block(a, asc, w, wsc, z, C, T, N, K, act, dt, ws, nb)


PRODUCTS = [fwd, dense, dgrad, dense_dgrad]


def test_exports_and_version(lib):
    src = re.sub(r"/\*.*?\*/", "", open(moe.MOE_HEADER).read(), flags=re.S)
    names = re.findall(r"^\s*(?:const\s+)?\w+\s*\*?\s*(\w+)\s*\(", src, flags=re.M)
    assert len(names) == 19 and "moe_sort_workspace" in names
    cdll = ctypes.CDLL(moe.MOE_LIB_PATH)
    assert not [n for n in names if not hasattr(cdll, n)]
    assert moe.moe_version().count(".") == 2


def test_route_refusals(lib):
    assert route(lib, dt=3) == DTYPE and route(lib, dt=-1) == DTYPE
    assert route(lib, score=2) == ACT
    assert route(lib, flags=2) == SHAPE
    for bad in (dict(T=-1), dict(T=(1 << 28) + 1), dict(E=0), dict(E=1025), dict(k=0), dict(k=17), dict(E=64, k=33), dict(scale=math.inf),
                dict(scale=math.nan), dict(groups=0), dict(groups=3), dict(E=64, groups=32), dict(groups=4, top=0), dict(groups=4, top=5),
                dict(groups=4, top=2, k=9), dict(best=0), dict(best=3)):
        assert route(lib, **bad) == SHAPE, bad
    for null in ("x", "idx", "w", "off", "rows"):
        assert route(lib, **{null: None}) == NULL, null
    assert route(lib, off=None, rows=None) == NULL          # slots alone
    assert route(lib, x=at(1) + 2) == ALIGN and route(lib, x=at(1) + 2, dt=0, idx=at(3) + 2) == ALIGN
    assert route(lib, idx=at(4)) == ALIAS and route(lib, w=at(1)) == ALIAS and route(lib, rows=at(2)) == ALIAS
    assert route(lib, slots=at(6) + 4) == ALIAS
    need = lib.moe_sort_workspace(10000, 16, 2)
    assert need > 0
    assert route(lib, T=10000, ws=at(9), nb=need - 1) == SCRATCH
    assert route(lib, T=10000, ws=None, nb=need) == NULL
    assert route(lib, T=10000, ws=at(9) + 2, nb=need) == ALIGN
    assert route(lib, T=10000, ws=at(1), nb=need) == ALIAS
    assert route(lib, T=0, off=None, rows=None, slots=None, x=None, idx=None, w=None) == OK


def test_route_grad_refusals(lib):
    assert grad(lib, dt=3) == DTYPE and grad(lib, score=-1) == ACT and grad(lib, flags=4) == SHAPE
    for bad in (dict(T=-1), dict(E=0), dict(E=1025), dict(k=0), dict(k=17), dict(scale=math.inf)):
        assert grad(lib, **bad) == SHAPE, bad
    for null in ("x", "idx", "dw", "dx"):
        assert grad(lib, **{null: None}) == NULL
    assert grad(lib, dx=at(1)) == ALIAS and grad(lib, dx=at(3) + 4) == ALIAS and grad(lib, dw=at(3) + 1) == ALIGN
    assert grad(lib, T=0, x=None, idx=None, dw=None, dx=None) == OK


def test_sort_refusals(lib):
    for bad in (dict(T=-1), dict(T=1 << 29), dict(E=0), dict(E=1025), dict(k=0), dict(k=33)):
        assert sort(lib, **bad) == SHAPE, bad
    for null in ("idx", "off", "rows"):
        assert sort(lib, **{null: None}) == NULL
    assert sort(lib, rows=at(1)) == ALIAS and sort(lib, slots=at(2)) == ALIAS and sort(lib, off=at(2) + 1) == ALIGN
    assert sort(lib, T=1 << 20, ws=at(8), nb=4) == SCRATCH


def test_sort_workspace(lib):
    size = lib.moe_sort_workspace
    assert size(0, 16, 2) == 0 and size(8, 32, 2) == 0 and size(1024, 1024, 2) == 0
    assert size(16384, 256, 8) == 256 * 256 * 4
    assert size(1 << 24, 1024, 32) == 256 * 1024 * 4
    assert size(-1, 16, 2) == size(8, 0, 2) == size(8, 16, 40) == 0
    assert gba.moe_sort_workspace(16384, 256, 8) == size(16384, 256, 8)


@pytest.mark.parametrize("call", [dispatch, combine, cgrad, quant])
def test_move_refusals(lib, call):
    assert call(lib, dt=2) == DTYPE
    for bad in (dict(T=-1), dict(k=0), dict(k=33), dict(H=-16), dict(H=(1 << 23) + 16), dict(R=-1), dict(R=(1 << 29) + 1), dict(T=(1 << 28) + 1)):
        assert call(lib, **bad) == SHAPE, bad
    assert call(lib, H=60) == ALIGN
    assert call(lib, out=at(3) + 8) == ALIGN
    assert call(lib, out=at(2)) == ALIAS
    if call is not quant:
        assert call(lib, rows=None) == NULL
    if call is not cgrad:
        assert call(lib, out=None) == NULL
        assert call(lib, out=at(1)) == ALIAS
        assert call(lib, H=0, **({"y": None} if call is combine else {"x": None})) == OK
    assert call(lib, rows=at(2) + 2) == ALIGN
    assert call(lib, T=0, R=0) == OK


def test_more_move_refusals(lib):
    assert cgrad(lib, out=at(5)) == ALIAS and cgrad(lib, dw=at(4)) == ALIAS and cgrad(lib, out=at(6)) == ALIAS
    assert cgrad(lib, out=None, dw=None) == OK
    assert quant(lib, flags=2) == SHAPE
    assert quant(lib, rows=None) == SHAPE and quant(lib, rows=None, k=1) == SHAPE          # R is not T
    assert quant(lib, s=None) == NULL and quant(lib, s=at(3)) == ALIAS
    assert quant(lib, H=72) == ALIGN                                                       # whole 16 codes
    deq = lambda c=at(1), s=at(2), x=at(3), R=4, K=64, dt=0: lib.fp8_dequantize(c, s, x, R, K, dt)  # noqa: E731
    assert deq(dt=2) == DTYPE and deq(R=-1) == SHAPE and deq(K=24) == ALIGN and deq(c=None) == NULL and deq(x=at(2)) == ALIAS
    assert deq(R=0, c=None, s=None, x=None) == OK


def test_weights_refusals(lib):
    assert weights(lib, dt=2) == DTYPE and weights(lib, flags=4) == SHAPE
    for bad in (dict(E=-1), dict(E=4097), dict(N=-8), dict(N=(1 << 23) + 16), dict(K=(1 << 23) + 16), dict(E=4096, N=1 << 20, K=1 << 20)):
        assert weights(lib, **bad) == SHAPE, bad
    assert weights(lib, K=24) == ALIGN and weights(lib, N=24) == ALIGN
    for one in ("c", "s", "ct", "st"):
        assert weights(lib, **{one: None}) == NULL
    assert weights(lib, c=None, s=None, ct=None, st=None) == NULL
    assert weights(lib, ct=at(2)) == ALIAS and weights(lib, s=at(5)) == ALIAS and weights(lib, c=at(1)) == ALIAS
    assert weights(lib, E=0, w=None) == OK
    deq = lambda c=at(1), s=at(2), x=at(3), E=2, N=64, K=64, dt=0: lib.fp8_dequantize_weights(c, s, x, E, N, K, dt)  # noqa: E731
    assert deq(dt=2) == DTYPE and deq(E=-1) == SHAPE and deq(K=24) == ALIGN and deq(s=None) == NULL and deq(x=at(1)) == ALIAS


@pytest.mark.parametrize("call", PRODUCTS)
def test_product_refusals(lib, call):
    assert call(lib, dt=2) == DTYPE and call(lib, dt=-1) == DTYPE
    assert call(lib, act=6) == ACT and call(lib, act=-1) == ACT
    for bad in (dict(T=-1), dict(T=(1 << 29) + 1), dict(N=-8), dict(K=-16), dict(K=(1 << 22) + 16), dict(N=(1 << 23) + 8)):
        assert call(lib, **bad) == SHAPE, bad
    assert call(lib, N=60) == ALIGN and call(lib, K=40) == ALIGN
    for null in ("a", "asc", "w", "wsc", "C"):
        assert call(lib, **{null: None}) == NULL, null
    assert call(lib, a=at(1) + 8) == ALIGN and call(lib, asc=at(2) + 2) == ALIGN and call(lib, wsc=at(5) + 1) == ALIGN
    for other in (1, 2, 4, 5, 6):
        assert call(lib, C=at(other)) == ALIAS
    assert call(lib, ws=at(9) + 8, nb=1 << 20) == ALIGN and call(lib, ws=at(1), nb=1 << 20) == ALIAS
    assert call(lib, T=0) == OK and call(lib, N=0, w=None, wsc=None, C=None) == OK
    if call in (fwd, dgrad):
        assert call(lib, E=0) == SHAPE and call(lib, E=4097) == SHAPE
        assert call(lib, off=None) == NULL and call(lib, off=at(3) + 2) == ALIGN
    if call in (fwd, dense):
        assert call(lib, z=at(7)) == ALIAS and call(lib, bias=at(6) + 2) == ALIGN
    else:
        assert call(lib, z=None) == NULL


def test_no_device_gives_device_error(lib):
    if _gpu_present():
        pytest.skip("a GPU is present; this checks the GPU-less path")
    for call in [route, grad, sort, dispatch, combine, cgrad, quant, weights] + PRODUCTS:
        assert call(lib) == DEVICE
    assert lib.fp8_dequantize(at(1), at(2), at(3), 4, 64, 0) == DEVICE
    assert lib.fp8_dequantize_weights(at(1), at(2), at(3), 1, 4, 64, 0) == DEVICE


def test_binding_refusals():
    f, h, i = torch.float32, torch.bfloat16, torch.int32
    z = lambda *s, dt=f: torch.zeros(s, dtype=dt)  # noqa: E731
    with pytest.raises(ValueError, match="device"):
        gba.moe_route(z(4, 8), z(4, 2, dt=i), z(4, 2))
    with pytest.raises(ValueError, match="device"):
        gba.moe_dispatch(z(4, 8, dt=h), z(4, 2, dt=i), z(8, 8, dt=h))
    with pytest.raises(ValueError, match="score"):
        moe._score("tanh")
    with pytest.raises(TypeError, match="logits"):
        moe._logits(z(2, 2, dt=torch.float64))
    with pytest.raises(TypeError, match="indices"):
        moe._typed("indices", z(2, dt=torch.int64), i)
    with pytest.raises(TypeError, match="float8"):
        moe._f8("a", z(2, 16, dt=torch.uint8), z(1, 2))
    f8 = torch.float8_e4m3fn
    with pytest.raises(ValueError, match="scales"):
        moe._f8_rows("a", z(2, 160, dt=f8), z(1, 2), (2, 160))
    with pytest.raises(ValueError, match="scales"):
        moe._f8_weights("w", z(3, 200, 160, dt=f8), z(3, 2, 1), (3, 200, 160))
    with pytest.raises(ValueError, match="rows"):
        moe._sorted(z(9, dt=i), z(4, 3, dt=i), None, 4, 8, 2)
    assert gba.fp8_scales_shape(5, 160) == (2, 5) and gba.fp8_weight_scales_shape(3, 129, 16) == (3, 2, 1)


# ------------------------------------------------------- the plain forms ----

def test_plain_route():
    from tests import moe_oracle as orc
    x = torch.tensor([[0.0, math.log(3), -math.inf, math.log(2)], [1.0, 1.0, 1.0, 1.0], [-math.inf] * 4])
    idx, w, _ = orc.route(x, None, 2, renorm=False)
    assert idx.tolist() == [[1, 3], [0, 1], [-1, -1]]
    assert torch.allclose(w, torch.tensor([[0.5, 1 / 3], [0.25, 0.25], [0, 0]], dtype=torch.float64), rtol=1e-6)
    idx, w, _ = orc.route(x, torch.tensor([2.0, 0, 9, 0]), 2, scale=2.0)
    assert idx.tolist() == [[0, 1], [2, 0], [-1, -1]]
    assert torch.allclose(w[0], torch.tensor([0.5, 1.5], dtype=torch.float64), rtol=1e-6)
    y = torch.tensor([[5.0, -9, 4, 4.5, 3, 3, 0, 0]])
    assert orc.route(y, None, 2, score="sigmoid", groups=4, top_groups=1, group_best=1)[0].tolist() == [[0, 1]]
    assert orc.route(y, None, 2, score="sigmoid", groups=4, top_groups=1, group_best=2)[0].tolist() == [[3, 2]]
    assert orc.sort(torch.tensor([[1, 0], [-1, 1], [0, 7]]), 3) == ([0, 2, 4, 4], [2, 0, -1, 3, 1, -1], [1, 4, 0, 3, -1, -1])


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_plain_route_grad_is_the_derivative(score, renorm):
    from tests import moe_oracle as orc
    g = torch.Generator().manual_seed(4)
    x = torch.randn(5, 9, generator=g, dtype=torch.float64)
    x[1, 4:] = -math.inf
    idx, _, _ = orc.route(x, None, 3, score)
    dw = torch.randn(5, 3, generator=g)
    leaf = x.clone().requires_grad_()
    s = torch.softmax(leaf, 1) if score == "softmax" else torch.sigmoid(leaf)
    w = s.gather(1, idx)
    if renorm:
        w = w / w.sum(1, keepdim=True)
    (w * dw.double() * 1.5).sum().backward()
    dx, size, _ = orc.route_grad(x, idx, dw, score, renorm, 1.5)
    assert torch.allclose(dx, leaf.grad, rtol=1e-9, atol=1e-12)
    assert (dx.abs() <= size * (1 + 1e-9)).all()


def test_plain_8_bits():
    from tests import moe_oracle as orc
    table = orc.e4m3_values()
    codes = torch.arange(127, dtype=torch.uint8)
    assert torch.equal(table.float(), codes.view(torch.float8_e4m3fn).float())
    near = torch.cat([table, (table[1:] + table[:-1]) / 2])   # every value and every border
    assert torch.equal(orc.to_codes(near).view(torch.float8_e4m3fn).float(), near.float().to(torch.float8_e4m3fn).float())
    for q, c in ((0.0, 0), (448.0, 126), (336.0, 0x7a), (-2.0 ** -10, 128), (3 * 2.0 ** -10, 2), (17.0, 0x58), (19.0, 0x5a)):
        assert orc.to_codes(torch.tensor([q], dtype=torch.float64)).item() == c, q
    x = torch.zeros(2, 160, dtype=torch.bfloat16)
    x[0, 0], x[0, 1], x[0, 130], x[1, 3] = 1.0, 0.75, -7.0, float("nan")
    c, s = orc.quantize(x)
    assert s.shape == (2, 2) and s[0, 0] == torch.tensor(1 / 448) and s[0, 1] == 7 / 448 and s[1, 1] == 2.0 ** -126 and s[1, 0].isnan()
    assert c[0, 0] == 126 and c[0, 1] == 0x7a and c[0, 130] == 254 and (c[1] == 0).all()
    assert orc.quantize(x, 1, True)[1][0].tolist() == [2.0 ** -8, 2.0 ** -6]
    assert orc.quantize(x, 128)[1].isnan()[0].tolist() == [True, False]
    assert torch.equal(orc.values(c, s)[0, :2].float(), torch.tensor([1.0, 320 / 448]))
