"""The gradient of routing for rows without any slot: zeros for padding, NaN where the forward pass had NaN weights, in every type
and score, at every number of lanes a row; rows beside them as ever."""
import math

import pytest

import tiled_dense_gemm_bias_amd as gba
from tests import experts_oracle as eo
from tests import moe_oracle as orc
from tests.gpu_util import say
from tests.test_gpu_moe_route import DT, guarded, logits, run

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,E,k", [(9, 1, 1), (9, 8, 2), (13, 40, 20), (70, 100, 8), (33, 256, 8), (11, 300, 17), (9, 1000, 4)])
def test_nan_rows(T, E, k, dtype, score, renorm):
    say("nan gradient", T, E, k, dtype, score, renorm)
    x, g = logits(T + E, T, E, dtype)
    x[1] = -math.inf                     # padding
    x[2, E - 1] = math.nan
    x[3, 0] = math.inf                   # a score of 1 by sigmoid, NaN by softmax
    x[5] = math.nan
    x[6, E // 2] = math.nan
    x[6, :E // 2] = -math.inf
    idx, w = run(x, k, sort=False, score=score, renormalize=renorm, scale=1.5)
    bad = torch.isnan(w).all(1)
    want_bad = [2, 5, 6] + ([3] if score == "softmax" else [])
    assert sorted(torch.nonzero(bad)[:, 0].tolist()) == sorted(want_bad)
    dw = torch.randn(T, k, generator=g, device="cuda")
    dx, intact = guarded((T, E), DT[dtype], 5)
    gba.moe_route_grad(x, idx, dw, dx, score=score, renormalize=renorm, scale=1.5)
    torch.cuda.synchronize()
    intact()
    assert torch.isnan(dx[bad]).all() and (dx[1] == 0).all()
    fine = ~bad
    fine[3] = False                      # (the plain form's softmax of an infinity)
    want, size, depth = orc.route_grad(x[fine], idx[fine], dw[fine], score, renorm, 1.5)
    eo.check("dx", dx[fine], want, eo.with_rounding(want, (2 * depth[:, None] + 60) * 2.0 ** -24 * size + 2.0 ** -120, DT[dtype]))
    if score == "sigmoid":
        assert torch.isfinite(dx[3]).all()


def test_no_slot_and_finite_logits():
    """Indices that a caller took away: zeros, as before."""
    say("no slots")
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            x, g = logits(1, 6, 70, "f32")
            idx = torch.full((6, 3), -1, dtype=torch.int32, device="cuda")
            dx = torch.full_like(x, 9)
            gba.moe_route_grad(x, idx, torch.full((6, 3), math.nan, device="cuda"), dx, score=score, renormalize=renorm)
            assert (dx == 0).all()
