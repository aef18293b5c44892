"""The derivatives that grouped_gemm_act_grad multiplies by, as fractions of themselves: every finite
16-bit pre-activation, outputs scaled up so that small derivatives keep their digits.

Bounds: the argument of the exponential, A in nats (z^2/2, |z|, or 2 y of the tanh form), is off by two
fp32 roundings, A 2^-23 of the result; the other steps are eight of 2^-23 at most. Where a derivative
passes through zero or 1 the terms it is the difference of are below 1.2 each: 4e-7, three steps. Below
2^-126 the hardware's exponential and reciprocal give 0, and the tanh form is held at its
value at z = -10, below 1e-30. Then one rounding of the output."""
import math

import pytest

import tiled_dense_gemm_bias_amd as gba
from tests import experts_oracle as orc
from tests.gpu_util import say
from tests.test_gpu_experts import DT, make_offsets

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def exact(act, z):
    """orc.slope without its cancellations in 64 bits."""
    if act != "gelu":
        return orc.slope(act, z)
    x = z.abs()
    phi = torch.exp(-x * x / 2) / math.sqrt(2 * math.pi)
    low = phi * (math.sqrt(math.pi / 2) * torch.special.erfcx(x / math.sqrt(2)) - x)
    return torch.where(z < 0, low, orc.slope(act, z))


def bound(act, z, want):
    x = z.abs()
    if act == "relu":
        return torch.zeros_like(want)
    if act in ("sigmoid", "softplus"):
        return ((x + 8) * 2.0 ** -23) * want.abs() + 2.0 ** -126
    if act == "gelu":
        nats, tiny = x * x / 2, 2.0 ** -126
    else:
        nats, tiny = 2 * math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3), 1e-30
    return torch.where(z > -1.5, torch.full_like(want, 4e-7), ((nats + 8) * 2.0 ** -23) * want.abs() + tiny)


@pytest.mark.parametrize("rows,width,depth", [(8192, 8, 8), (8192, 4096, 72)])
@pytest.mark.parametrize("dtype,scale", [("f16", 1.0), ("f16", 16384.0), ("bf16", 1.0)])
@pytest.mark.parametrize("act", ["relu", "sigmoid", "gelu", "softplus", "gelu_tanh"])
def test_derivatives_keep_their_digits(act, dtype, scale, rows, width, depth):
    say("derivatives", act, dtype, scale, rows, width)
    dt = DT[dtype]
    z = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(dt).cuda()
    z = torch.where(torch.isfinite(z), z, torch.zeros_like(z)).repeat(rows * width // 65536).view(rows, width).contiguous()
    dc = torch.zeros(rows, depth, dtype=dt, device="cuda")
    dc[:, 3] = scale
    w = torch.zeros(1, depth, width, dtype=dt, device="cuda")
    w[0, 3] = 1
    da = torch.empty_like(z)
    gba.grouped_gemm_act_grad(dc, make_offsets([rows]), w, z, da, act, transpose_b=True)
    # Every value once, then the same bits wherever else it stands.
    one, got = z.view(-1)[:65536].double(), da.view(-1, 65536)
    want = exact(act, one)
    orc.check(act, got[0], scale * want, orc.with_rounding(scale * want, scale * bound(act, one, want), dt))
    assert torch.equal(got, got[:1].expand_as(got))
