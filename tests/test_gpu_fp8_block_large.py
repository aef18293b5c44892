"""The persistent kernel of the 8-bit products at the sizes of moe_large_cases.LARGE, each of which is asserted to be taken by it:
against the 64-bit definition, bit for bit on whole numbers, with NaN scales and with offsets that reach outside the rows."""
import math

import pytest

import tiled_dense_gemm_bias_amd as gba
from tests import experts_oracle as eo
from tests import moe_cases
from tests import moe_large_cases as cases
from tests import moe_oracle as orc
from tests.gpu_util import say
from tests.test_gpu_experts import draw, make_offsets
from tests.test_gpu_experts import guarded as guarded16
from tests.test_gpu_experts_offsets import lists
from tests.test_gpu_fp8_block import DT, F8, quantised
from tests.test_gpu_fp8_block_kernels import check_forward, check_grad, setup
from tiled_dense_gemm_bias_amd import moe

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

# rows, experts, columns, depth
OFFSETS = [(3500, 2, 4160, 272), (12000, 66, 4096, 272)]
NAN = [(3500, 2, 4160, 272), (3000, 8, 4096, 384), (12000, 66, 4096, 272)]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.empty_cache()


def persistent(T, E, N, K):
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    return moe.plan(T, E, N, K, 0, cus)["kind"] == "persistent"


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("i", range(len(cases.LARGE)))
def test_each_size(i, dtype):
    s = setup("large", cases.LARGE[i], dtype, 300)
    check_forward(s, DT[dtype], eo.ACTS[i % 6], i % 2 == 1)
    check_forward(s, DT[dtype], eo.ACTS[(i + 3) % 6], i % 2 == 0)
    check_grad(s, DT[dtype], eo.ACTS[(i + 2) % 6])


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("i", [2, 8])
def test_each_activation(i, dtype):
    """Whole lines, ragged groups: every epilogue, with and without stored pre-activations."""
    s = setup("large activations", cases.LARGE[i], dtype, 400)
    for act in eo.ACTS:
        for preact in (False, True):
            check_forward(s, DT[dtype], act, preact)
        check_grad(s, DT[dtype], act)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("i", range(len(cases.LARGE)))
def test_whole_numbers_bit_for_bit(i, dtype):
    """Codes of whole numbers up to 8 and scales of 1 and 2 (every sum is a whole number below 2^18, exact in 32 bits):
    the exact sum plus the bias (a whole number too), rounded once; pre-activations, and the gradient of ReLU."""
    _, sizes, lead, tail, N, K, _ = cases.LARGE[i]
    dt = DT[dtype]
    say("large exact", i, len(sizes), N, K, dtype)
    g = torch.Generator(device="cuda").manual_seed(900 + i)
    T, E = lead + sum(sizes) + tail, len(sizes)
    assert persistent(T, E, N, K)
    whole = lambda *s: (torch.randint(-8, 9, s, generator=g, device="cuda") / 1.0).to(F8)
    two = lambda *s: torch.exp2(torch.randint(0, 2, s, generator=g, device="cuda").float())
    ac, asc, wc, wsc = whole(T, K), two(*gba.fp8_scales_shape(T, K)), whole(E, N, K), two(*gba.fp8_weight_scales_shape(E, N, K))
    bias = torch.randint(-100, 101, (E, N), generator=g, device="cuda").to(dt)
    a64 = orc.values(ac.view(torch.uint8), asc.T.contiguous())
    w64 = torch.stack([orc.values(wc[e].view(torch.uint8), wsc[e], 128) for e in range(E)])
    off = make_offsets(sizes, lead)
    for b in (None, bias):
        want, _, owned = orc.product(a64, off.tolist(), w64, b)
        (c, c_intact), (z, z_intact) = guarded16((T, N), dt), guarded16((T, N), dt)
        gba.grouped_gemm_bias_act_fp8_block(ac, asc, off, wc, wsc, b, c, "relu", preact=z)
        torch.cuda.synchronize()
        c_intact(), z_intact()
        assert torch.equal(z[owned], want.to(dt)[owned]) and torch.equal(c[owned], want.clamp(min=0).to(dt)[owned])
        assert torch.isnan(c[~owned]).all() and torch.isnan(z[~owned]).all()
    want, _, owned = orc.product(a64, off.tolist(), w64, None)
    z = torch.randn(T, N, generator=g, device="cuda").to(dt)
    da, intact = guarded16((T, N), dt)
    gba.grouped_gemm_act_grad_fp8_block(ac, asc, off, wc, wsc, z, da, "relu")
    torch.cuda.synchronize()
    intact()
    assert torch.equal(da[owned], torch.where(z > 0, want, torch.zeros_like(want)).to(dt)[owned]) and torch.isnan(da[~owned]).all()
    if E == 1 and off.tolist() == [0, T]:
        c, intact = guarded16((T, N), dt)
        gba.gemm_bias_act_fp8_block(ac, asc, wc[0], wsc[0], bias[0], c, "none")
        torch.cuda.synchronize()
        intact()
        assert torch.equal(c, (want + bias[0].double()).to(dt))
        gba.gemm_act_grad_fp8_block(ac, asc, wc[0], wsc[0], z, c, "relu")
        torch.cuda.synchronize()
        intact()
        assert torch.equal(c, torch.where(z > 0, want, torch.zeros_like(want)).to(dt))


@pytest.mark.parametrize("T,E,N,K", NAN)
def test_a_scale_of_nan_stays_in_its_rows_and_columns(T, E, N, K):
    say("large nan", T, E, N, K)
    assert persistent(T, E, N, K)
    g = torch.Generator(device="cuda").manual_seed(8)
    sizes = moe_cases.shares(T, E, T + N)
    first = next(e for e in range(E) if sizes[e])
    x, w = draw(g, (T, K), torch.bfloat16), draw(g, (E, N, K), torch.bfloat16, K ** -0.5)
    x[1, K - 3] = x[T - 1, 0] = math.nan
    w[first, N - 1, 130] = math.inf
    ac, asc = quantised(x)
    wc, wsc = torch.empty(E, N, K, dtype=F8, device="cuda"), torch.empty(gba.fp8_weight_scales_shape(E, N, K), device="cuda")
    gba.fp8_quantize_weights(w, wc, wsc)
    want = torch.zeros(T, N, dtype=torch.bool, device="cuda")
    want[1] = want[T - 1] = True
    want[:sizes[first], (N - 1) // 128 * 128:] = True
    c = torch.zeros(T, N, dtype=torch.bfloat16, device="cuda")
    gba.grouped_gemm_bias_act_fp8_block(ac, asc, make_offsets(sizes), wc, wsc, None, c, "none")
    assert torch.equal(torch.isnan(c), want)
    da = torch.zeros_like(c)
    gba.grouped_gemm_act_grad_fp8_block(ac, asc, make_offsets(sizes), wc, wsc, None, da, "none")
    assert torch.equal(torch.isnan(da), want)


@pytest.mark.parametrize("T,E,N,K", OFFSETS)
def test_offsets_that_reach_outside_the_rows(T, E, N, K):
    """Offsets in order: the rows are those of the clamped offsets, and nothing else is written."""
    assert persistent(T, E, N, K)
    g = torch.Generator(device="cuda").manual_seed(T + E)
    dt = torch.bfloat16
    a = quantised(draw(g, (T, K), dt))
    w = draw(g, (E, N, K), dt, K ** -0.5)
    wc, wsc = torch.empty(E, N, K, dtype=F8, device="cuda"), torch.empty(gba.fp8_weight_scales_shape(E, N, K), device="cuda")
    gba.fp8_quantize_weights(w, wc, wsc)
    z = draw(g, (T, N), dt)
    a64 = orc.values(a[0].view(torch.uint8), a[1].T.contiguous())
    w64 = torch.stack([orc.values(wc[e].view(torch.uint8), wsc[e], 128) for e in range(E)])
    for o in lists(T, E):
        say("large offsets", T, E, N, K, o[:8])
        off = torch.tensor(o, dtype=torch.int32, device="cuda")
        (c, c_intact), (da, da_intact) = guarded16((T, N), dt), guarded16((T, N), dt)
        gba.grouped_gemm_bias_act_fp8_block(*a, off, wc, wsc, None, c, "none")
        gba.grouped_gemm_act_grad_fp8_block(*a, off, wc, wsc, z, da, "relu")
        torch.cuda.synchronize()
        c_intact(), da_intact()
        want, err, owned = orc.product(a64, [min(max(v, 0), T) for v in o], w64, None)
        eo.check("c", c, want, eo.with_rounding(want, err, dt), owned)
        s = (z > 0).double()
        eo.check("da", da, want * s, eo.with_rounding(want * s, err, dt), owned)
        assert torch.isnan(c[~owned]).all() and torch.isnan(da[~owned]).all()
