"""Grouped and 4-bit products as a program uses them: captured into a graph whose
inputs and offsets change between replays, called by several threads on streams of
their own, with the most experts a call takes, and with arrays of more than 2^31
values."""
import threading

import pytest

import tiled_dense_gemm_bias_amd as gba
from tests import experts_oracle as orc
from tests.gpu_util import say
from tests.test_gpu_experts import DT, draw, make_offsets, workspace

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.empty_cache()


class Layer:
    """One layer's tensors: every entry point once, forward, backward and in 4 bits."""

    def __init__(self, E, T, D, F, dtype, with_workspace):
        self.ws = workspace(16 << 20)[0] if with_workspace else None
        e = lambda *s, dt=dtype: torch.empty(s, dtype=dt, device="cuda")
        self.w1, self.b1, self.w2 = e(E, F, D), e(E, F), e(E, F, D)
        self.h, self.z, self.y = e(T, F), e(T, F), e(T, D)
        self.dh, self.dx = e(T, F), e(T, D)
        self.dw, self.db = e(E, F, D, dt=torch.float32), e(E, F, dt=torch.float32)
        u = lambda *s: e(*s, dt=torch.uint8)
        self.xq, self.xs = u(T, D // 2), u(*gba.mx4_scales_shape(T, D))
        self.wq, self.wsc = u(E * F, D // 2), u(*gba.mx4_scales_shape(E * F, D))
        self.h4, self.d4, self.back = e(T, F), e(T, F), e(T, D)
        self.E, self.F, self.D = E, F, D

    def fill(self, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        for t in (self.w1, self.b1, self.w2):
            t.copy_(torch.randn(t.shape, generator=g, device="cuda") * self.D ** -0.5)

    def run(self, x, dy, off):
        k = dict(workspace=self.ws)
        gba.grouped_gemm_bias_act(x, off, self.w1, self.b1, self.h, "gelu", transpose_b=True, preact=self.z, **k)
        gba.grouped_gemm_bias_act(self.h, off, self.w2, None, self.y, "none", **k)
        gba.grouped_gemm_act_grad(dy, off, self.w2, self.z, self.dh, "gelu", **k)
        gba.grouped_gemm_act_grad(self.dh, off, self.w1, None, self.dx, "none", transpose_b=True, **k)
        gba.grouped_gemm_wgrad(x, self.dh, off, self.dw, self.db, transpose_b=True, **k)
        gba.mx4_quantize(x, self.xq, self.xs)
        gba.mx4_quantize(self.w1.view(-1, self.D), self.wq, self.wsc)
        gba.mx4_dequantize(self.xq, self.xs, self.back)
        gba.grouped_gemm_bias_act_mx4(self.xq, self.xs, off, self.wq.view(self.E, self.F, -1), self.wsc, self.b1, self.h4, "gelu", **k)
        gba.gemm_bias_act_mx4(self.xq, self.xs, self.wq[:self.F], self.first_scales(), self.b1[0], self.d4, "relu", **k)

    def first_scales(self):
        return self.one

    def set_dense(self):
        """Expert 0 alone, for the dense product."""
        self.one = self.wsc[:, :self.F].contiguous()

    def outputs(self):
        return [self.h, self.z, self.y, self.dh, self.dx, self.dw, self.db, self.xq, self.xs, self.back, self.h4, self.d4]


CASES = [
    ("f16", 3, 60, 64, 136, False, ([20, 0, 40], [0, 1, 59])),
    ("bf16", 4, 40, 2048, 264, True, ([10, 10, 20, 0], [0, 0, 0, 40])),
    ("bf16", 5, 3000, 288, 4104, False, ([1000, 0, 700, 300, 1000], [1, 2999, 0, 0, 0])),
]


@pytest.mark.parametrize("i", range(len(CASES)))
def test_graphs_replay_like_eager(i):
    dtype, E, T, D, F, with_ws, sizes = CASES[i]
    dt = DT[dtype]
    say("graph", CASES[i])
    g = torch.Generator(device="cuda").manual_seed(40 + i)
    layer = Layer(E, T, D, F, dt, with_ws)
    layer.fill(50 + i)
    gba.mx4_quantize(layer.w1.view(-1, D), layer.wq, layer.wsc)
    layer.set_dense()
    inputs = [(draw(g, (T, D), dt), draw(g, (T, D), dt), make_offsets(s)) for s in sizes]
    want = []
    for args in inputs:
        layer.run(*args)
        want.append([t.clone() for t in layer.outputs()])
    torch.cuda.synchronize()
    static = [t.clone() for t in inputs[0]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.run(*static)
    torch.cuda.synchronize()
    for r in range(4):
        for s, t in zip(static, inputs[r % 2]):
            s.copy_(t)
        for t in layer.outputs():
            t.fill_(3)
        if layer.ws is not None:
            layer.ws.fill_(float("nan"))
        say("replay", r)
        graph.replay()
        torch.cuda.synchronize()
        for k, (got, ref) in enumerate(zip(layer.outputs(), want[r % 2])):
            assert torch.equal(got.view(torch.uint8), ref.view(torch.uint8)), (r, k)


def test_threads_on_their_own_streams():
    """Four threads, a layer and a stream each: every call's bits are those of the same call alone."""
    say("threads")
    jobs = []
    for i in range(4):
        dtype, E, T, D, F, with_ws, sizes = CASES[i % len(CASES)]
        g = torch.Generator(device="cuda").manual_seed(70 + i)
        layer = Layer(E, T, D, F, DT[dtype], with_ws)
        layer.fill(80 + i)
        gba.mx4_quantize(layer.w1.view(-1, D), layer.wq, layer.wsc)
        layer.set_dense()
        args = (draw(g, (T, D), DT[dtype]), draw(g, (T, D), DT[dtype]), make_offsets(sizes[0]))
        layer.run(*args)
        jobs.append((layer, args, [t.clone() for t in layer.outputs()], torch.cuda.Stream()))
    torch.cuda.synchronize()
    wrong = []

    def work(n):
        layer, args, want, stream = jobs[n]
        try:
            with torch.cuda.stream(stream):
                for r in range(6):
                    for t in layer.outputs():
                        t.fill_(5)
                    layer.run(*args)
                    stream.synchronize()
                    wrong.extend((n, r, k) for k, (a, b) in enumerate(zip(layer.outputs(), want))
                                 if not torch.equal(a.view(torch.uint8), b.view(torch.uint8)))
        except Exception as e:   # shown by the test's thread
            wrong.append((n, repr(e)))
    threads = [threading.Thread(target=work, args=(n,)) for n in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not wrong


def test_the_most_experts():
    E, N, K, dt = 4096, 72, 136, torch.bfloat16
    say("4096 experts")
    g = torch.Generator(device="cuda").manual_seed(9)
    sizes = torch.randint(0, 3, (E,), generator=g, device="cuda").tolist()
    sizes[4000] = 300
    off, T = make_offsets(sizes), sum(sizes)
    a, w = draw(g, (T, K), dt), draw(g, (E, N, K), dt, K ** -0.5)
    c = torch.empty(T, N, dtype=dt, device="cuda")
    gba.grouped_gemm_bias_act(a, off, w, None, c, "none", transpose_b=True)
    owner = torch.repeat_interleave(torch.arange(E, device="cuda"), torch.tensor(sizes, device="cuda"))
    picked = w[owner]
    prods = picked.double() * a.double()[:, None, :]
    want = prods.sum(-1)
    size = prods.abs().sum(-1)
    orc.check("c", c, want, orc.with_rounding(want, size * orc.sum_rel(K), dt))
    dw = torch.empty(E, N, K, dtype=torch.float32, device="cuda")
    db = torch.empty(E, N, dtype=torch.float32, device="cuda")
    gba.grouped_gemm_wgrad(a, c, off, dw, db, transpose_b=True)
    outer = c.double()[:, :, None] * a.double()[:, None, :]
    want = torch.zeros(E, N, K, dtype=torch.float64, device="cuda").index_add_(0, owner, outer)
    size = torch.zeros(E, N, K, dtype=torch.float64, device="cuda").index_add_(0, owner, outer.abs())
    orc.check("dw", dw, want, orc.with_rounding(want, size * orc.sum_rel(300), torch.float32))
    want = torch.zeros(E, N, dtype=torch.float64, device="cuda").index_add_(0, owner, c.double())
    size = torch.zeros(E, N, dtype=torch.float64, device="cuda").index_add_(0, owner, c.double().abs())
    orc.check("db", db, want, orc.with_rounding(want, size * orc.sum_rel(300), torch.float32))
    with pytest.raises(gba.GbaError):
        gba.grouped_gemm_bias_act(a, make_offsets([0] * 4097), torch.empty(4097, 8, K, dtype=dt, device="cuda"), None,
                                  torch.empty(T, 8, dtype=dt, device="cuda"), "none", transpose_b=True)


# ------------------------------------------------- arrays of more than 2^31 values --

@pytest.mark.parametrize("F", [64, 520])
def test_many_rows(F):
    """270000 rows of 8200 values: inputs, outputs and pre-activations past 2^31 values and 2^32 bytes."""
    T, D, dt = 270000, 8200, torch.bfloat16
    sizes, tail = [100000, 162200, 7800], 300
    say("many rows", F)
    g = torch.Generator(device="cuda").manual_seed(21)
    off, E = make_offsets(sizes), len(sizes)
    x = torch.randn(T, D, generator=g, device="cuda", dtype=dt)
    w = draw(g, (E, F, D), dt, D ** -0.5)
    c = torch.empty(T, F, dtype=dt, device="cuda")
    gba.grouped_gemm_bias_act(x, off, w, None, c, "none", transpose_b=True)
    want, err, _ = orc.product(x[-tail:], [0, tail], w[-1:], None, True)
    orc.check("c", c[-tail:], want, orc.with_rounding(want, err, dt))
    # x as pre-activations; the gradient has its size
    dx = torch.empty(T, D, dtype=dt, device="cuda")
    gba.grouped_gemm_act_grad(c, off, w, x, dx, "sigmoid", transpose_b=True)
    d, err, _ = orc.product(c[-tail:], [0, tail], w[-1:], None, False)
    s = orc.slope("sigmoid", x[-tail:].double())
    orc.check("dx", dx[-tail:], d * s, orc.with_rounding(d * s, s * err + orc.SLOPE_TOL * (d.abs() + err), dt))
    dw, db = torch.empty(E, F, D, dtype=dt, device="cuda"), torch.empty(E, D, dtype=dt, device="cuda")
    gba.grouped_gemm_wgrad(x, c, off, dw, None, transpose_b=True)
    n = sizes[-1]
    cd, xd = c[-n:].double().T.contiguous(), x[-n:].double()
    want = cd @ xd
    orc.check("dw", dw[-1], want, orc.with_rounding(want, (cd.abs() @ xd.abs()) * orc.sum_rel(n), dt))
    dw2 = torch.empty(E, F, D, dtype=dt, device="cuda")
    gba.grouped_gemm_wgrad(c, x, off, dw2, db)      # x as the output's gradient: its column sums
    orc.check("dw2", dw2[-1], want, orc.with_rounding(want, (cd.abs() @ xd.abs()) * orc.sum_rel(n), dt))
    want = xd.sum(0)
    orc.check("db", db[-1], want, orc.with_rounding(want, xd.abs().sum(0) * orc.sum_rel(n), dt))


@pytest.mark.parametrize("tb", [True, False])
def test_many_weights(tb):
    """80 experts of 4096 x 8200: weights and their gradients past 2^31 values."""
    E, N, K, dt = 80, 4096, 8200, torch.bfloat16
    sizes = [30] + [0] * (E - 2) + [170]
    say("many weights", tb)
    g = torch.Generator(device="cuda").manual_seed(22)
    off, T = make_offsets(sizes), sum(sizes)
    w = torch.randn(E, N, K, generator=g, device="cuda", dtype=dt) if tb else torch.randn(E, K, N, generator=g, device="cuda", dtype=dt)
    x = draw(g, (T, K), dt, K ** -0.5)
    c = torch.empty(T, N, dtype=dt, device="cuda")
    want, err, _ = orc.product(x, off.tolist(), w, None, tb)
    for ws in (None, workspace(32 << 20)[0]):
        c.fill_(9)
        gba.grouped_gemm_bias_act(x, off, w, None, c, "none", transpose_b=tb, workspace=ws)
        orc.check("c", c, want, orc.with_rounding(want, err, dt))
    dx = torch.empty(T, K, dtype=dt, device="cuda")
    gba.grouped_gemm_act_grad(c, off, w, None, dx, "none", transpose_b=tb)
    want, err, _ = orc.product(c, off.tolist(), w, None, not tb)
    orc.check("dx", dx, want, orc.with_rounding(want, err, dt))
    dw = w.fill_(7)
    gba.grouped_gemm_wgrad(x, c, off, dw, None, transpose_b=tb)
    p, q = (c[30:].double(), x[30:].double()) if tb else (x[30:].double(), c[30:].double())
    p = p.T.contiguous()
    want = p @ q
    orc.check("dw", dw[-1], want, orc.with_rounding(want, (p.abs() @ q.abs()) * orc.sum_rel(170), dt))
    assert (dw[40] == 0).all() and (dw[-2] == 0).all()


def test_many_rows_in_4_bits():
    M, K, tail, dt = 600000, 8192, 200, torch.bfloat16
    say("many rows in 4 bits")
    g = torch.Generator(device="cuda").manual_seed(23)
    x = torch.randn(M, K, generator=g, device="cuda", dtype=dt)
    codes, scales = torch.empty(M, K // 2, dtype=torch.uint8, device="cuda"), torch.empty(gba.mx4_scales_shape(M, K), dtype=torch.uint8, device="cuda")
    gba.mx4_quantize(x, codes, scales)
    want_codes, want_scales = orc.mx4_pack(*orc.mx4_quantize(x[-tail:]))
    assert torch.equal(codes[-tail:], want_codes) and torch.equal(scales[:, -tail:], want_scales)
    a64 = orc.mx4_values(*orc.mx4_quantize(x[-tail:]))
    gba.mx4_dequantize(codes, scales, x)
    assert torch.equal(x[-tail:].double(), a64)
    for N in (64, 520):
        w = draw(g, (N, K), dt, K ** -0.5)
        wq, ws = torch.empty(N, K // 2, dtype=torch.uint8, device="cuda"), torch.empty(gba.mx4_scales_shape(N, K), dtype=torch.uint8, device="cuda")
        gba.mx4_quantize(w, wq, ws)
        c = torch.empty(M, N, dtype=dt, device="cuda")
        gba.gemm_bias_act_mx4(codes, scales, wq, ws, None, c, "none")
        want, err, _ = orc.product(a64, [0, tail], orc.mx4_values(*orc.mx4_quantize(w))[None], None, True, mx4=True)
        orc.check("c", c[-tail:], want, orc.with_rounding(want, err, dt))


def test_many_short_rows_in_4_bits():
    """More 16-row groups than one grid dimension is given."""
    M, K = (1 << 24) + (1 << 22) + 5, 32
    say("many short rows in 4 bits")
    g = torch.Generator(device="cuda").manual_seed(24)
    x = torch.randn(M, K, generator=g, device="cuda", dtype=torch.float16)
    codes, scales = torch.full((M, K // 2), 0xA5, dtype=torch.uint8, device="cuda"), torch.full(gba.mx4_scales_shape(M, K), 0xA5, dtype=torch.uint8, device="cuda")
    gba.mx4_quantize(x, codes, scales)
    y = torch.empty_like(x)
    gba.mx4_dequantize(codes, scales, y)
    for lo in (0, M // 2, (1 << 24) - 50, M - 100):
        c, s = orc.mx4_quantize(x[lo:lo + 100])
        want_codes, want_scales = orc.mx4_pack(c, s)
        assert torch.equal(codes[lo:lo + 100], want_codes) and torch.equal(scales[:, lo:lo + 100], want_scales)
        assert torch.equal(y[lo:lo + 100].double(), orc.mx4_values(c, s))


def test_the_example_learns_and_serves():
    """The layer of examples/expert_layer.py: its loss falls, its outputs in 4 bits stay near the 16-bit ones."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "expert_layer.py")
    spec = importlib.util.spec_from_file_location("expert_layer", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    say("example")
    losses, error = ex.run(tokens=1000, experts=6, top=2, width=256, hidden=320, steps=12)
    assert losses[-1] < 0.9 * losses[0], losses
    # A code is off by up to a quarter of its value (5 of 4 .. 6), its root mean square about a
    # tenth; four roundings (inputs, weights, twice) add up to some 0.2.
    assert 0 < error < 0.4, error


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_large_products_of_more_experts_than_lanes(dtype):
    """70 experts, empty ones among them, at sizes that the persistent kernels take: all three products."""
    E, N, K, dt = 70, 2056, 1032, DT[dtype]
    sizes = [(37 * e * e + 300) % 700 if e % 9 else 0 for e in range(E)]
    say("70 experts", dtype, sum(sizes))
    g = torch.Generator(device="cuda").manual_seed(31)
    off, T = make_offsets(sizes, 3), sum(sizes) + 8
    a, dc = draw(g, (T, K), dt), draw(g, (T, N), dt)
    w, bias = draw(g, (E, N, K), dt, K ** -0.5), draw(g, (E, N), dt)
    c, da = torch.full((T, N), float("nan"), dtype=dt, device="cuda"), torch.full((T, K), float("nan"), dtype=dt, device="cuda")
    gba.grouped_gemm_bias_act(a, off, w, bias, c, "sigmoid", transpose_b=True)
    z, err, owned = orc.product(a, off.tolist(), w, bias, True)
    want = orc.act("sigmoid", z)
    orc.check("c", c, want, orc.with_rounding(want, 0.25 * err + orc.ACT_TOL, dt), owned)
    gba.grouped_gemm_act_grad(dc, off, w, a, da, "softplus", transpose_b=True)
    d, err, _ = orc.product(dc, off.tolist(), w, None, False)
    s = orc.slope("softplus", a.double())
    orc.check("da", da, d * s, orc.with_rounding(d * s, s * err + orc.SLOPE_TOL * (d.abs() + err), dt), owned)
    for tb in (True, False):
        dw = torch.empty((E, N, K) if tb else (E, K, N), dtype=dt, device="cuda")
        db = torch.empty(E, N, dtype=dt, device="cuda")
        gba.grouped_gemm_wgrad(a, dc, off, dw, db, transpose_b=tb)
        for e, b, n in orc.groups(off.tolist(), T):
            x, y = a[b:b + n].double(), dc[b:b + n].double()
            p = y.T.contiguous()
            want, size = p @ x, p.abs() @ x.abs()
            orc.check("dw", dw[e] if tb else dw[e].T, want, orc.with_rounding(want, size * orc.sum_rel(n), dt))
            orc.check("db", db[e], y.sum(0), orc.with_rounding(y.sum(0), y.abs().sum(0) * orc.sum_rel(n), dt))
