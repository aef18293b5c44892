"""Sorting of more slots a token than experts, as on a device that holds some of a token's experts; dispatch and combine on it."""
import pytest

import tiled_dense_gemm_bias_amd as gba
from tests import experts_oracle as eo
from tests.gpu_util import say
from tests.test_gpu_moe_route import check_sorted, guarded

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("T,experts,k,E", [(1, 8, 8, 1), (5, 16, 8, 2), (300, 256, 8, 4), (64, 64, 32, 3), (65, 64, 32, 3), (5000, 256, 8, 1), (9000, 256, 24, 5)])
def test_a_devices_share(T, experts, k, E):
    """Experts 1 .. E of a token's k different ones of `experts`; the others' slots are -1."""
    say("share", T, experts, k, E)
    g = torch.Generator(device="cuda").manual_seed(T + k)
    idx = torch.rand(T, experts, generator=g, device="cuda").topk(k, 1).indices.to(torch.int32) - 1
    idx[idx >= E] = -1
    off, i1 = guarded((E + 1,), torch.int32, 5)
    rows, i2 = guarded((T, k), torch.int32, 5)
    slots, i3 = guarded((T * k,), torch.int32, 5)
    need = gba.moe_sort_workspace(T, E, k)
    ws, i4 = guarded((need + 8,), torch.uint8, 3)
    gba.moe_sort(idx, off, rows, slots, workspace=ws[:need] if need else None)
    torch.cuda.synchronize()
    for i in (i1, i2, i3, i4):
        i()
    check_sorted(idx, off, rows, slots, E)
    x = torch.randn(T, 64, generator=g, device="cuda").bfloat16()
    n = int(off[-1])
    xs = gba.moe_dispatch(x, rows, torch.full((T * k, 64), 5, dtype=x.dtype, device="cuda"))
    assert torch.equal(xs[:n], x[slots[:n].long() // k]) and (xs[n:] == 5).all()
    out = gba.moe_combine(xs, rows, None, torch.empty(T, 64, device="cuda"))
    want = x.double() * (idx >= 0).sum(1, keepdim=True)
    eo.check("out", out, want, k * 2.0 ** -24 * want.abs() + 2.0 ** -149)


def test_an_expert_in_every_slot():
    """All slots of a token on one expert: rows in the order of the slots."""
    say("every slot")
    T, k = 700, 16
    idx = torch.zeros(T, k, dtype=torch.int32, device="cuda")
    off, rows = torch.empty(2, dtype=torch.int32, device="cuda"), torch.empty_like(idx)
    gba.moe_sort(idx, off, rows, workspace=torch.empty(gba.moe_sort_workspace(T, 1, k), dtype=torch.uint8, device="cuda"))
    assert off.tolist() == [0, T * k] and torch.equal(rows.view(-1).long(), torch.arange(T * k, device="cuda"))
