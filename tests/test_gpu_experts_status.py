"""An error that an earlier HIP call of the thread left behind is not this library's: calls after it run, whole, and
report their own status."""
import ctypes

import pytest

import tiled_dense_gemm_bias_amd as gba
from tests.gpu_util import say
from tests.test_gpu_experts import make_offsets, workspace

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture
def hip():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    lib = ctypes.CDLL("libamdhip64.so")
    yield lib
    lib.hipGetLastError()


def test_calls_after_another_calls_error(hip):
    say("stale error")
    g = torch.Generator(device="cuda").manual_seed(1)
    dt = torch.bfloat16
    new = lambda *s, dt=dt: torch.empty(s, dtype=dt, device="cuda")  # noqa: E731
    T, E, N, K = 24, 3, 72, 4096
    off, ws = make_offsets([4, 0, 20]), workspace(4 << 20)[0]
    x = torch.randn(T, K, generator=g, device="cuda").to(dt)
    w = torch.randn(E, N, K, generator=g, device="cuda").to(dt)
    wide = torch.randn(1, 4096, 72, generator=g, device="cuda").to(dt)
    many = torch.randn(8192, 72, generator=g, device="cuda").to(dt)
    out = dict(c=new(T, N), da=new(T, K), dw=new(E, N, K, dt=torch.float32), db=new(E, N, dt=torch.float32),
               codes=new(T, K // 2, dt=torch.uint8), scales=new(*gba.mx4_scales_shape(T, K), dt=torch.uint8), back=new(T, K),
               c4=new(T, N), g4=new(T, N), big=new(8192, 4096))
    wq, wsc = new(E * N, K // 2, dt=torch.uint8), new(*gba.mx4_scales_shape(E * N, K), dt=torch.uint8)
    one, onesc = new(N, K // 2, dt=torch.uint8), new(*gba.mx4_scales_shape(N, K), dt=torch.uint8)
    gba.mx4_quantize(w.view(E * N, K), wq, wsc)
    gba.mx4_quantize(w[0], one, onesc)
    whole = make_offsets([8192])
    assert gba.experts.plan("forward", T, E, N, K, ws.nbytes)["splits"] > 1          # two launches
    assert gba.experts.plan("forward", 8192, 1, 4096, 72)["persistent"]
    calls = [lambda: gba.grouped_gemm_bias_act(x, off, w, None, out["c"], "gelu", transpose_b=True, workspace=ws),
             lambda: gba.grouped_gemm_act_grad(out["c"], off, w, x, out["da"], "relu", transpose_b=True),
             lambda: gba.grouped_gemm_wgrad(x, out["c"], off, out["dw"], out["db"], transpose_b=True),
             lambda: gba.mx4_quantize(x, out["codes"], out["scales"]),
             lambda: gba.mx4_dequantize(out["codes"], out["scales"], out["back"]),
             lambda: gba.gemm_bias_act_mx4(out["codes"], out["scales"], one, onesc, None, out["c4"], "none"),
             lambda: gba.grouped_gemm_bias_act_mx4(out["codes"], out["scales"], off, wq.view(E, N, K // 2), wsc, None, out["g4"], "none"),
             lambda: gba.grouped_gemm_bias_act(many, whole, wide, None, out["big"], "none", transpose_b=True)]
    for t in out.values():
        t.fill_(3)
    for call in calls:
        call()
    torch.cuda.synchronize()
    want = [t.clone() for t in out.values()]
    for t in out.values():
        t.fill_(3)
    torch.cuda.synchronize()
    for call in calls:
        assert hip.hipSetDevice(1000) != 0 and hip.hipPeekAtLastError() != 0
        call()
    assert hip.hipPeekAtLastError() != 0          # still the caller's to read
    hip.hipGetLastError()
    torch.cuda.synchronize()
    for t, ref in zip(out.values(), want):
        assert torch.equal(t.view(torch.uint8), ref.view(torch.uint8))
