"""Microscaled 4-bit quantisation (bit for bit) and product against the 64-bit definition."""
import pytest

import tiled_dense_gemm_bias_amd as gba
from tests import experts_oracle as orc
from tests.gpu_util import say
from tests.test_gpu_experts import DT, draw, guarded, make_offsets, workspace

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def bytes_guarded(shape):
    n = 1
    for d in shape:
        n *= d
    whole = torch.full((n + 4096,), 0xA5, dtype=torch.uint8, device="cuda")

    def intact():
        assert (whole[:2048] == 0xA5).all() and (whole[2048 + n:] == 0xA5).all(), "written outside the output"
    return whole[2048:2048 + n].view(shape), intact


def quantised(x):
    M, K = x.shape
    codes, i1 = bytes_guarded((M, K // 2))
    scales, i2 = bytes_guarded(gba.mx4_scales_shape(M, K))
    gba.mx4_quantize(x, codes, scales)
    torch.cuda.synchronize()
    i1(), i2()
    return codes, scales


def check_quantise(x):
    codes, scales = quantised(x)
    c, s = orc.mx4_quantize(x)
    want_codes, want_scales = orc.mx4_pack(c, s)
    assert torch.equal(scales, want_scales)
    assert torch.equal(codes, want_codes)
    assert torch.equal(gba.mx4_unpack_scales(scales, x.shape[1]), s.to(torch.uint8))
    assert torch.equal(gba.mx4_pack_scales(s.to(torch.uint8)), scales)
    for dt in (torch.bfloat16, torch.float16):
        y, intact = guarded(x.shape, dt)
        assert gba.mx4_dequantize(codes, scales, y) is y
        torch.cuda.synchronize()
        intact()
        want = orc.mx4_values(c, s).to(torch.float32).to(dt)   # exact in fp32 but for overflow
        assert torch.equal(torch.nan_to_num(y, nan=77.0), torch.nan_to_num(want, nan=77.0))
        assert torch.equal(torch.signbit(y), torch.signbit(want)) or torch.isnan(want).any()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("M,K", [(1, 32), (1, 4096), (3, 64), (7, 160), (16, 128), (17, 96), (33, 1056), (200, 544)])
def test_quantise(M, K, dtype):
    say("quantise", M, K, dtype)
    g = torch.Generator(device="cuda").manual_seed(M * 1000 + K)
    x = draw(g, (M, K), DT[dtype]) * torch.exp2(torch.randint(-12, 8, (M, 1), generator=g, device="cuda")).to(DT[dtype])
    x[0, :32] = 0
    x[0, 5] = -0.0
    check_quantise(x)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_quantise_every_value(dtype):
    """Every 16-bit pattern, in blocks led by every exponent: ties, saturation, subnormals, infinities, NaN."""
    say("every value", dtype)
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16).cuda()
    step = 128 if dtype == "bf16" else 1024
    exponents = 65536 // 2 // step                     # of the positive half
    rows = []
    for e in range(0, exponents, 7 if dtype == "bf16" else 3):
        lead = torch.full((65536 // 16, 2), e * step, dtype=torch.int16, device="cuda")
        other = bits.view(-1, 16)
        # values below the leader's next exponent, so that the leader sets the scale in many blocks
        rows.append(torch.cat([lead, other, other[:, :14]], 1))
    x = torch.cat(rows).view(DT[dtype]).reshape(-1, 32 * 32).contiguous()
    check_quantise(x)
    near = torch.cat([((bits & 0x7fff) % ((e + 1) * step) | (bits & -0x8000)).to(torch.int16) for e in range(1, exponents, 5)])
    check_quantise(near.view(DT[dtype]).reshape(-1, 32 * 64).contiguous())


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("M,N,K", [(1, 8, 32), (1, 1000, 4096), (5, 264, 96), (16, 64, 256), (17, 72, 288), (63, 136, 544),
                                   (65, 200, 1024), (129, 264, 160), (300, 520, 2080), (513, 1032, 128),
                                   (1025, 10248, 288), (3000, 5128, 544), (4096, 4096, 512), (8200, 2056, 1312),
                                   (3, 264, 8192), (40, 136, 4128), (150, 72, 10240)])
def test_product(M, N, K, dtype):
    dt, act = DT[dtype], orc.ACTS[(M + N) % 6]
    say("mx4 product", M, N, K, dtype, act)
    g = torch.Generator(device="cuda").manual_seed(M + N + K)
    x, w = draw(g, (M, K), dt), draw(g, (N, K), dt, K ** -0.5)
    bias = draw(g, (N,), dt) if M % 2 else None
    ac, asc = quantised(x)
    wc, wsc = quantised(w)
    a64, w64 = orc.mx4_values(*orc.mx4_quantize(x)), orc.mx4_values(*orc.mx4_quantize(w))
    want_z, err, _ = orc.product(a64, [0, M], w64[None], None if bias is None else bias[None], True, mx4=True)
    c, intact = guarded((M, N), dt)
    assert gba.gemm_bias_act_mx4(ac, asc, wc, wsc, bias, c, act) is c
    torch.cuda.synchronize()
    intact()
    want = orc.act(act, want_z)
    orc.check("c", c, want, orc.with_rounding(want, orc.LIPSCHITZ[act] * err + orc.ACT_TOL, dt))
    c2, intact = guarded((M, N), dt)
    ws, ws_intact = workspace()
    gba.gemm_bias_act_mx4(ac, asc, wc, wsc, bias, c2, act, workspace=ws)
    torch.cuda.synchronize()
    intact(), ws_intact()
    orc.check("c, workspace", c2, want, orc.with_rounding(want, orc.LIPSCHITZ[act] * err + orc.ACT_TOL, dt))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("sizes,lead,tail,N,K", [
    ([1], 0, 0, 8, 32), ([0, 3, 0, 1], 1, 0, 72, 160), ([5, 0, 16, 17], 0, 3, 136, 96), ([63, 0, 65, 2], 2, 1, 200, 544),
    ([129, 255, 0, 130], 0, 5, 264, 288), ([1] * 70 + [0] * 20 + [3] * 20, 0, 0, 40, 128),
    ([257, 0, 511, 300, 1000], 0, 0, 8200, 288), ([200] * 70, 0, 3, 1032, 544), ([300, 2000, 1, 0, 1000, 640], 5, 0, 4104, 1056),
    ([3, 0, 20], 1, 2, 264, 8224)])
def test_grouped_product(sizes, lead, tail, N, K, dtype):
    dt, act = DT[dtype], orc.ACTS[len(sizes) % 6]
    say("mx4 grouped", sizes[:8], lead, tail, N, K, dtype, act)
    g = torch.Generator(device="cuda").manual_seed(N + K)
    E, T = len(sizes), lead + sum(sizes) + tail
    off = make_offsets(sizes, lead)
    x, w = draw(g, (T, K), dt), draw(g, (E * N, K), dt, K ** -0.5)
    bias = draw(g, (E, N), dt)
    ac, asc = quantised(x)
    wc, wsc = quantised(w)
    a64 = orc.mx4_values(*orc.mx4_quantize(x))
    w64 = orc.mx4_values(*orc.mx4_quantize(w)).view(E, N, K)
    want_z, err, owned = orc.product(a64, off.tolist(), w64, bias, True, mx4=True)
    asc[:, ~owned] = 255                                   # rows of no expert: NaN
    c, intact = guarded((T, N), dt)
    assert gba.grouped_gemm_bias_act_mx4(ac, asc, off, wc.view(E, N, K // 2), wsc, bias, c, act) is c
    torch.cuda.synchronize()
    intact()
    want = orc.act(act, want_z)
    orc.check("c", c, want, orc.with_rounding(want, orc.LIPSCHITZ[act] * err + orc.ACT_TOL, dt), owned)
    c2, intact = guarded((T, N), dt)
    ws, ws_intact = workspace()
    gba.grouped_gemm_bias_act_mx4(ac, asc, off, wc.view(E, N, K // 2), wsc, bias, c2, act, workspace=ws)
    torch.cuda.synchronize()
    intact(), ws_intact()
    orc.check("c, workspace", c2, want, orc.with_rounding(want, orc.LIPSCHITZ[act] * err + orc.ACT_TOL, dt), owned)


def test_product_of_scales_over_the_whole_range():
    """Blocks of very different scales, a zero block, and a NaN block that reaches its own row only."""
    M, N, K = 20, 24, 256
    g = torch.Generator(device="cuda").manual_seed(3)
    x = draw(g, (M, K), torch.bfloat16) * torch.exp2(torch.randint(-30, 30, (M, 1), generator=g, device="cuda")).to(torch.bfloat16)
    x[3, 64:96] = 0
    x[4, 40] = float("nan")
    x[5, 200] = float("-inf")
    w = draw(g, (N, K), torch.bfloat16)
    ac, asc = quantised(x)
    wc, wsc = quantised(w)
    c = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    gba.gemm_bias_act_mx4(ac, asc, wc, wsc, None, c, "none")
    assert torch.isnan(c[4]).all() and torch.isnan(c[5]).all()
    keep = [r for r in range(M) if r not in (4, 5)]
    a64 = orc.mx4_values(*orc.mx4_quantize(x))[keep]
    want, err, _ = orc.product(a64, [0, len(keep)], orc.mx4_values(*orc.mx4_quantize(w))[None], None, True, mx4=True)
    orc.check("c", c[keep], want, orc.with_rounding(want, err, torch.bfloat16))
