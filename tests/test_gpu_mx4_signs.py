"""Signs of the 4-bit format's values, zeros among them: every code under every scale, and every 16-bit
pattern there and back, compared bit for bit wherever the value is a number."""
import pytest

import tiled_dense_gemm_bias_amd as gba
from tests import experts_oracle as orc
from tests.gpu_util import say
from tests.test_gpu_experts import DT, guarded

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def same(got, values):
    """got has the bits of the 64-bit values rounded to its type (they are exact in 32 bits but for overflow), and
    NaN where they are NaN."""
    want = values.float().to(got.dtype)
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got), nan)
    assert torch.equal(got.view(torch.int16)[~nan], want.view(torch.int16)[~nan])
    return nan


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_every_code_under_every_scale(dtype):
    say("signs, codes", dtype)
    codes = torch.arange(16, device="cuda").repeat(256, 2)                  # [256, 32]
    s = torch.arange(256, device="cuda").view(256, 1)
    packed, planes = orc.mx4_pack(codes, s)
    x, intact = guarded((256, 32), DT[dtype])
    gba.mx4_dequantize(packed, planes, x)
    torch.cuda.synchronize()
    intact()
    nan = same(x, orc.mx4_values(codes, s))
    assert nan.sum() == 32
    assert torch.equal(torch.signbit(x[:255]), (codes[:255] >= 8))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_every_pattern_there_and_back(dtype):
    """With infinities and NaN in their blocks and without, so that every finite value is in a block of finite ones too."""
    say("signs, patterns", dtype)
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16).cuda().view(-1, 32)
    x = bits.view(DT[dtype])
    x = torch.cat([x, torch.where(torch.isfinite(x), x, torch.zeros_like(x))]).contiguous()
    codes = torch.empty(x.shape[0], 16, dtype=torch.uint8, device="cuda")
    scales = torch.empty(gba.mx4_scales_shape(*x.shape), dtype=torch.uint8, device="cuda")
    gba.mx4_quantize(x, codes, scales)
    c, s = orc.mx4_quantize(x)
    want_codes, want_scales = orc.mx4_pack(c, s)
    assert torch.equal(codes, want_codes) and torch.equal(scales, want_scales)
    y = torch.empty_like(x)
    gba.mx4_dequantize(codes, scales, y)
    nan = same(y, orc.mx4_values(c, s))
    finite = torch.isfinite(x).view(-1, 32).all(1)
    assert not nan[finite].any() and nan[~finite].all()
    assert torch.equal(torch.signbit(y[finite]), torch.signbit(x[finite]))
