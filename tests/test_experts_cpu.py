"""Refusals of libgba_experts and of its binding, without a GPU: every argument
error is reported before a device is touched."""
import ctypes
import re

import pytest

import tiled_dense_gemm_bias_amd as gba
from tests.test_abi_cpu import _gpu_present

experts = gba.experts
torch = pytest.importorskip("torch")

OK, NULL, SHAPE, DTYPE, ACT, ALIGN, ALIAS, DEVICE = range(8)
P = 0x10000                    # 16-byte aligned fake addresses, far apart, never followed
BIG = 1 << 40


def at(i):
    return P + i * BIG


@pytest.fixture(scope="module")
def lib():
    return gba.experts.experts_lib()


def fwd(lib, A=at(1), off=at(2), W=at(3), bias=at(4), C=at(5), z=at(6), T=64, E=4, N=64, K=64, act=0, dt=0,
        flags=1, ws=None, nb=0):
    return lib.grouped_gemm_bias_act(A, off, W, bias, C, z, T, E, N, K, act, dt, flags, ws, nb)


def grad(lib, dC=at(1), off=at(2), W=at(3), z=at(4), dA=at(5), T=64, E=4, N=64, K=64, act=3, dt=0, flags=1,
         ws=None, nb=0):
    return lib.grouped_gemm_act_grad(dC, off, W, z, dA, T, E, N, K, act, dt, flags, ws, nb)


def wgrad(lib, A=at(1), dC=at(2), off=at(3), dW=at(4), db=at(5), T=64, E=4, N=64, K=64, dt=0, flags=1, ws=None,
          nb=0):
    return lib.grouped_gemm_wgrad(A, dC, off, dW, db, T, E, N, K, dt, flags, ws, nb)


def mx4(lib, ac=at(1), asc=at(2), off=at(3), wc=at(4), wsc=at(5), bias=at(6), C=at(7), T=64, E=4, N=64, K=64,
        act=0, dt=0, ws=None, nb=0):
    return lib.grouped_gemm_bias_act_mx4(ac, asc, off, wc, wsc, bias, C, T, E, N, K, act, dt, ws, nb)


def dense4(lib, ac=at(1), asc=at(2), wc=at(4), wsc=at(5), bias=at(6), C=at(7), M=64, N=64, K=64, act=0, dt=0,
           ws=None, nb=0):
    return lib.gemm_bias_act_mx4(ac, asc, wc, wsc, bias, C, M, N, K, act, dt, ws, nb)


def test_exports_and_version(lib):
    src = re.sub(r"/\*.*?\*/", "", open(experts.EXPERTS_HEADER).read(), flags=re.S)
    names = re.findall(r"^\s*(?:const\s+)?\w+\s*\*?\s*(\w+)\s*\(", src, flags=re.M)
    assert len(names) >= 10
    cdll = ctypes.CDLL(experts.EXPERTS_LIB_PATH)
    assert not [n for n in names if not hasattr(cdll, n)]
    assert gba.experts.experts_version().count(".") == 2


@pytest.mark.parametrize("call", [fwd, grad, wgrad, mx4, dense4])
def test_common_refusals(lib, call):
    rows = "M" if call is dense4 else "T"
    assert call(lib, dt=2) == DTYPE
    assert call(lib, dt=-1) == DTYPE
    if call is not wgrad:
        assert call(lib, act=6) == ACT
        assert call(lib, act=-1) == ACT
    assert call(lib, **{rows: -1}) == SHAPE
    assert call(lib, **{rows: 1 << 31}) == SHAPE
    assert call(lib, N=-8) == SHAPE
    assert call(lib, K=-32) == SHAPE
    assert call(lib, K=(1 << 24)) == SHAPE
    assert call(lib, N=(1 << 24)) == SHAPE
    assert call(lib, N=60) == ALIGN
    assert call(lib, K=36) == ALIGN
    if call is not dense4:
        assert call(lib, E=0) == SHAPE
        assert call(lib, E=4097) == SHAPE
        assert call(lib, off=None) == NULL
        assert call(lib, off=at(8) + 2) == ALIGN
    assert call(lib, ws=at(9) + 8, nb=1 << 20) == ALIGN
    assert call(lib, ws=at(1), nb=1 << 20) == ALIAS


def test_forward_refusals(lib):
    assert fwd(lib, A=None) == NULL
    assert fwd(lib, W=None) == NULL
    assert fwd(lib, C=None) == NULL
    assert fwd(lib, A=at(1) + 8) == ALIGN
    assert fwd(lib, bias=at(4) + 4) == ALIGN
    assert fwd(lib, z=at(6) + 2) == ALIGN
    assert fwd(lib, C=at(1) + 64) == ALIAS
    assert fwd(lib, z=at(5) + 64) == ALIAS
    assert fwd(lib, C=at(4)) == ALIAS
    assert fwd(lib, C=at(2)) == ALIAS            # the offsets
    assert fwd(lib, flags=2) == SHAPE
    assert fwd(lib, T=0) == OK
    assert fwd(lib, N=0, W=None, C=None) == OK
    assert fwd(lib, T=0, A=None, C=None, z=None, off=None) == OK


def test_gradient_refusals(lib):
    assert grad(lib, z=None) == NULL
    assert grad(lib, dA=None) == NULL
    assert grad(lib, dC=None) == NULL
    assert grad(lib, W=None) == NULL
    assert grad(lib, z=at(4) + 8) == ALIGN
    assert grad(lib, dA=at(4)) == ALIAS          # over z
    assert grad(lib, flags=16) == SHAPE
    assert grad(lib, N=(1 << 21) + 8) == SHAPE   # the depth of this product
    assert grad(lib, T=0) == OK
    assert grad(lib, K=0, W=None, dA=None) == OK
    assert wgrad(lib, A=None) == NULL
    assert wgrad(lib, dC=None) == NULL
    assert wgrad(lib, dW=None) == NULL
    assert wgrad(lib, dW=at(1) + 16) == ALIAS
    assert wgrad(lib, db=at(4) + 16) == ALIAS
    assert wgrad(lib, db=at(5) + 2) == ALIGN
    assert wgrad(lib, flags=64) == SHAPE
    assert wgrad(lib, flags=32) == DTYPE         # accumulate without fp32
    assert wgrad(lib, N=0, dC=None, dW=None, db=None) == OK


def test_mx4_refusals(lib):
    for call in (mx4, dense4):
        assert call(lib, ac=None) == NULL
        assert call(lib, asc=None) == NULL
        assert call(lib, wc=None) == NULL
        assert call(lib, wsc=None) == NULL
        assert call(lib, C=None) == NULL
        assert call(lib, asc=at(2) + 4) == ALIGN
        assert call(lib, C=at(5)) == ALIAS
        assert call(lib, C=at(6)) == ALIAS
        assert call(lib, K=(1 << 23) + 32) == SHAPE
        assert call(lib, N=0, wc=None, wsc=None, C=None) == OK
    q = lambda X=at(1), c=at(2), s=at(3), M=4, K=64, dt=0: lib.mx4_quantize(X, c, s, M, K, dt)  # noqa: E731
    d = lambda X=at(1), c=at(2), s=at(3), M=4, K=64, dt=0: lib.mx4_dequantize(c, s, X, M, K, dt)  # noqa: E731
    for f in (q, d):
        assert f(dt=3) == DTYPE
        assert f(M=-1) == SHAPE
        assert f(M=1 << 31) == SHAPE
        assert f(K=(1 << 23) + 32) == SHAPE
        assert f(K=48) == ALIGN
        assert f(X=None) == NULL
        assert f(c=None) == NULL
        assert f(s=None) == NULL
        assert f(X=at(1) + 8) == ALIGN
        assert f(M=0) == OK
        assert f(K=0, X=None, c=None, s=None) == OK
    assert q(c=at(1)) == ALIAS
    assert q(s=at(2)) == ALIAS
    assert d(X=at(3)) == ALIAS


@pytest.mark.parametrize("call", [fwd, grad, wgrad, mx4, dense4])
def test_most_rows(lib, call):
    """2^29 rows pass the size check (the next one, an output over an input, answers); one more does not."""
    rows, out = ("M", "C") if call is dense4 else ("T", {fwd: "C", grad: "dA", wgrad: "dW", mx4: "C"}[call])
    assert call(lib, **{rows: 1 << 29, out: at(1)}) == ALIAS
    assert call(lib, **{rows: (1 << 29) + 1, out: at(1)}) == SHAPE


def test_no_device_gives_device_error(lib):
    if _gpu_present():
        pytest.skip("a GPU is present; this checks the GPU-less path")
    for call in (fwd, grad, wgrad, mx4, dense4):
        assert call(lib) == DEVICE
    assert lib.mx4_quantize(at(1), at(2), at(3), 4, 64, 0) == DEVICE


def test_binding_refusals():
    h = torch.float16
    a, off, w = torch.zeros(4, 8, dtype=h), torch.zeros(3, dtype=torch.int32), torch.zeros(2, 16, 8, dtype=h)
    c = torch.zeros(4, 16, dtype=h)
    with pytest.raises(ValueError, match="device"):
        gba.grouped_gemm_bias_act(a, off, w, None, c, transpose_b=True)
    with pytest.raises(ValueError, match="device"):
        gba.mx4_quantize(torch.zeros(2, 32, dtype=h), torch.zeros(2, 16, dtype=torch.uint8),
                         torch.zeros(1, 2, 4, dtype=torch.uint8))
    with pytest.raises(TypeError, match="int32"):
        experts._offsets(torch.zeros(3, dtype=torch.int64), 2)
    with pytest.raises(ValueError, match="entries"):
        experts._offsets(off, 3)
    with pytest.raises(TypeError, match="dtype"):
        experts._same_dtype(a, c.bfloat16())
    with pytest.raises(ValueError, match="c is"):
        experts._expect("c", c, (4, 8))
    with pytest.raises(ValueError, match="multiple of 32"):
        experts._mx4("a", torch.zeros(2, 8, dtype=torch.uint8), torch.zeros(1, 2, 4, dtype=torch.uint8), 2, 16)
    with pytest.raises(ValueError, match="bytes"):
        experts._mx4("a", torch.zeros(2, 8, dtype=torch.uint8), torch.zeros(1, 2, 4, dtype=torch.uint8), 2, 32)
    with pytest.raises(ValueError, match="scales"):
        experts._mx4("a", torch.zeros(2, 16, dtype=torch.uint8), torch.zeros(2, 1, 4, dtype=torch.uint8), 2, 32)
    with pytest.raises(TypeError, match="uint8"):
        experts._mx4("a", torch.zeros(2, 16, dtype=torch.int8), torch.zeros(1, 2, 4, dtype=torch.uint8), 2, 32)


def test_scale_planes_of_rows():
    assert gba.mx4_scales_shape(5, 160) == (2, 5, 4)
    rows = torch.arange(5 * 5, dtype=torch.uint8).view(5, 5)
    planes = gba.mx4_pack_scales(rows)
    assert tuple(planes.shape) == (2, 5, 4)
    assert planes[1, 3, 0] == rows[3, 4] and planes[0, 2, 3] == rows[2, 3] and (planes[1, :, 1:] == 0).all()
    assert torch.equal(gba.mx4_unpack_scales(planes, 160), rows)
