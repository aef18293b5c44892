"""Rows that two slots name: every place holds a value of either slot (which one is not promised, and may differ from run to
run), rows of one slot hold theirs, and nothing else is written."""
import pytest

import tiled_dense_gemm_bias_amd as gba
from tests import moe_oracle as orc
from tests.gpu_util import say
from tests.test_gpu_moe_route import guarded

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def rows_and_values(T, H):
    """Tokens 2 i and 2 i + 1 share row i in slot 0; slot 1 of token t is row T + t. Distinct values a token."""
    g = torch.Generator(device="cuda").manual_seed(T + H)
    t = torch.arange(T, device="cuda", dtype=torch.int32)
    rows = torch.stack([t // 2, T + t], 1).contiguous()
    return rows, (torch.randn(T, H, generator=g, device="cuda") + 3 * (t % 7)[:, None]).bfloat16()


def check(out, rows, of_token, T):
    assert torch.equal(out[T:2 * T], of_token)
    a, b = of_token[0::2], of_token[1::2]
    assert ((out[:T // 2] == a) | (out[:T // 2] == b)).all()
    assert (out[T // 2:T] == 5).all()


@pytest.mark.parametrize("T,H", [(2, 16), (64, 2064), (512, 4112), (2048, 1040)])
def test_each_place_is_one_of_the_two(T, H):
    say("twice", T, H)
    rows, x = rows_and_values(T, H)
    out, i1 = guarded((2 * T, H), torch.bfloat16, 5)
    gba.moe_dispatch(x, rows, out)
    dy, i2 = guarded((2 * T, H), torch.bfloat16, 5)
    gba.moe_combine_grad(x, out, rows, None, dy, None)
    torch.cuda.synchronize()
    i1(), i2()
    check(out, rows, x, T)
    check(dy, rows, x, T)


@pytest.mark.parametrize("T,H", [(2, 16), (64, 2064), (512, 4112)])
def test_quantised(T, H):
    say("quantised twice", T, H)
    rows, x = rows_and_values(T, H)
    raw, i1 = guarded((2 * T, H), torch.uint8, 5)
    scales, i2 = guarded(gba.fp8_scales_shape(2 * T, H), torch.float32, 5)
    gba.fp8_quantize(x, raw.view(torch.float8_e4m3fn), scales, rows=rows)
    torch.cuda.synchronize()
    i1(), i2()
    codes, s = orc.quantize(x)
    check(raw, rows, codes, T)
    check(scales.T, rows, s, T)
