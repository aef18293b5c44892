"""combine with tokens in 32 bits (GBM_F32_TOKENS): what is accepted and refused, without a GPU."""
import pytest

import tiled_dense_gemm_bias_amd as gba
from tests.test_abi_cpu import _gpu_present
from tests.test_moe_cpu import ALIAS, ALIGN, DEVICE, DTYPE, OK, at, cgrad, combine, dispatch, quant

torch = pytest.importorskip("torch")
F32 = gba.moe.F32_TOKENS


@pytest.fixture(scope="module")
def lib():
    return gba.moe.moe_lib()


def test_which_calls_take_it(lib):
    for call in (combine, cgrad):
        for dt in (0, 1):
            assert call(lib, dt=dt | F32, T=0, R=0) == OK
            assert call(lib, dt=dt | F32, out=at(3) + 8) == ALIGN
            if not _gpu_present():
                assert call(lib, dt=dt | F32) == DEVICE
        for dt in (2, 3, 512, 1 | 512, -1):
            assert call(lib, dt=dt | F32) == DTYPE
    assert dispatch(lib, dt=F32) == DTYPE and quant(lib, dt=1 | F32) == DTYPE


def test_the_tokens_take_twice_the_bytes(lib):
    """8 tokens of 64: 1024 bytes in 16 bits, 2048 in 32."""
    for call in (combine, cgrad):
        y = "y"
        where = "out" if call is combine else "x"
        if call is cgrad:   # dout is an input: an output of dy behind it
            assert call(lib, x=at(1), out=at(1) + 1024, dt=F32) == ALIAS
            assert call(lib, x=at(1), out=at(1) + 2048, dt=F32 | 1, T=0, R=0) == OK
            if not _gpu_present():
                assert call(lib, x=at(1), out=at(1) + 1024) == call(lib, x=at(1), out=at(1) + 2048, dt=F32) == DEVICE
        else:
            assert call(lib, **{where: at(1) - 1024, y: at(1)}, dt=F32) == ALIAS
            if not _gpu_present():
                assert call(lib, **{where: at(1) - 1024, y: at(1)}) == call(lib, **{where: at(1) - 2048, y: at(1)}, dt=F32) == DEVICE


def test_the_bindings_types():
    h, b, f = (torch.zeros(2, 8, dtype=t) for t in (torch.float16, torch.bfloat16, torch.float32))
    code = gba.moe._tokens_dtype
    assert (code(h, h), code(b, b, None), code(h, f), code(b, f, b)) == (0, 1, F32, 1 | F32)
    for bad in ((h, b), (h, f, b), (f, f), (h, h.double())):
        with pytest.raises(TypeError):
            code(*bad)
