"""Routing and combine's gradients on both sides of the sizes where one launch becomes two, and where a token's waves change."""
import math

import pytest

from tests.gpu_util import say
from tests.test_gpu_moe_f32 import test_gradients as combine_grad_f32
from tests.test_gpu_moe_move import test_combine_grad as combine_grad
from tests.test_gpu_moe_route import check, logits

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


ROUTED = [(16, 129, 6, 1, 1), (17, 129, 6, 1, 1), (16, 256, 8, 8, 4), (17, 256, 8, 8, 4), (31, 256, 3, 1, 1), (32, 128, 16, 8, 4), (33, 128, 16, 8, 4),
          (32, 33, 5, 1, 1), (33, 33, 5, 1, 1), (64, 32, 32, 4, 4), (65, 32, 31, 4, 4), (64, 16, 2, 1, 1), (65, 16, 2, 1, 1)]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k,groups,top", ROUTED)
def test_routed(T, E, k, groups, top, score):
    say("routed", T, E, k, groups, top, score)
    x, g = logits(T + 3 * E, T, E, "f32")
    x[T // 2, E // 3:] = -math.inf
    x[T - 1] = -math.inf
    bias = torch.randn(E, generator=g, device="cuda") * 0.1
    check(x, k, bias, score=score, groups=groups, top_groups=top, group_best=2 if groups > 1 else 1)
    check(x.bfloat16(), k, None, score=score, groups=groups, top_groups=top, renormalize=False)


# Tokens, slots, columns, rows: around the sizes where a token gets four waves, or one.
GRADIENTS = [(512, 3, 1024, 1700), (513, 3, 1024, 1700), (1024, 2, 2048, 2100), (1025, 2, 2048, 2100), (513, 9, 1032, 4000), (2304, 1, 2056, 2600),
             (2305, 1, 2056, 2600), (2049, 1, 3584, 2049), (3001, 1, 4096, 3001)]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("T,k,H,R", GRADIENTS)
def test_combine_gradients(T, k, H, R, dtype):
    for weighted in (True, False):
        combine_grad(T, k, H, R, dtype, weighted)
        combine_grad_f32(T, k, H, R, dtype, weighted)
