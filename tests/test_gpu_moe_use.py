"""Routing, movement and 8-bit products as a program uses them: a whole expert layer forward and backward, each stage
against its definition on what the stage before left; captured into graphs whose inputs change between
replays; by several threads on streams of their own; with the most experts, offsets that reach outside the rows and arrays of
more than 2^31 values; and the example's layer."""
import importlib.util
import os
import threading

import pytest

import tiled_dense_gemm_bias_amd as gba
from tests import experts_oracle as eo
from tests import moe_oracle as orc
from tests.gpu_util import say
from tests.test_gpu_experts import DT, draw, make_offsets
from tests.test_gpu_experts_offsets import lists

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.empty_cache()


class Layer:
    """An expert layer in 8 bits and all that a step of it needs: y = combine(gelu(x W1^T + b1) W2^T), forward and backward,
    weight gradients in 16 bits."""

    def __init__(self, T, E, k, H, F, dtype, groups=1, score="softmax", logits=torch.float32):
        R = T * k
        e = lambda *s, dt=dtype: torch.empty(s, dtype=dt, device="cuda")
        f = lambda *s: e(*s, dt=torch.float32)
        self.T, self.E, self.k, self.H, self.F, self.R, self.dtype = T, E, k, H, F, R, dtype
        self.route = dict(score=score, scale=1.5, groups=groups, top_groups=max(1, groups // 2), group_best=2 if groups > 1 else 1)
        self.x, self.logits, self.bias, self.dout = e(T, H), e(T, E, dt=logits), f(E), e(T, H)
        self.w1, self.b1, self.w2 = e(E, F, H), e(E, F), e(E, H, F)
        self.idx, self.rows, self.off = e(T, k, dt=torch.int32), e(T, k, dt=torch.int32), e(E + 1, dt=torch.int32)
        self.slots, self.weights = e(R, dt=torch.int32), f(T, k)
        self.sort_ws = e(gba.moe_sort_workspace(T, E, k), dt=torch.uint8)
        self.ws = e(8 << 20, dt=torch.uint8)

        def coded(M, K):
            return e(M, K, dt=F8), f(*gba.fp8_scales_shape(M, K))

        def weights(N, K):
            return e(E, N, K, dt=F8), f(*gba.fp8_weight_scales_shape(E, N, K))
        self.c1, self.c1t, self.c2, self.c2t = weights(F, H), weights(H, F), weights(H, F), weights(F, H)
        self.xq, self.hq, self.dyq, self.dzq = coded(R, H), coded(R, F), coded(R, H), coded(R, F)
        self.h, self.z, self.y, self.out = e(R, F), e(R, F), e(R, H), e(T, H)
        self.dy, self.dz, self.dxs, self.dx = e(R, H), e(R, F), e(R, H), e(T, H)
        self.xs, self.dweights, self.dlogits = e(R, H), f(T, k), e(T, E, dt=logits)
        self.dw1, self.db1, self.dw2 = f(E, F, H), f(E, F), f(E, H, F)

    def inputs(self):
        return [self.x, self.logits, self.bias, self.dout, self.w1, self.b1, self.w2]

    def outputs(self):
        return [self.idx, self.weights, self.off, self.rows, self.slots, self.h, self.z, self.y, self.out, self.dy, self.dweights,
                self.dlogits, self.dz, self.dxs, self.dx, self.xs, self.dw1, self.db1, self.dw2, *self.xq, *self.hq, *self.dyq, *self.dzq,
                *self.c1, *self.c1t, *self.c2, *self.c2t]

    def fill(self, seed, padding=0):
        """Inputs of a seed; the last `padding` tokens go to no expert."""
        g = torch.Generator(device="cuda").manual_seed(seed)
        for t, std in zip(self.inputs(), (1.0, 1.5, 0.1, 1.0, self.H ** -0.5, 0.3, self.F ** -0.5)):
            t.copy_(torch.randn(t.shape, generator=g, device="cuda") * std)
        if padding:
            self.logits[-padding:] = float("-inf")

    def dirty(self):
        for t in self.outputs() + [self.ws, self.sort_ws]:
            t.view(torch.uint8).fill_(0xff)    # NaN in every type

    def run(self):
        gba.moe_route(self.logits, self.idx, self.weights, self.bias, self.off, self.rows, self.slots, workspace=self.sort_ws, **self.route)
        gba.fp8_quantize_weights(self.w1, *self.c1, *self.c1t)
        gba.fp8_quantize_weights(self.w2, *self.c2, *self.c2t)
        gba.fp8_quantize(self.x, *self.xq, rows=self.rows)
        k = dict(workspace=self.ws)
        gba.grouped_gemm_bias_act_fp8_block(*self.xq, self.off, *self.c1, self.b1, self.h, "gelu", preact=self.z, **k)
        gba.fp8_quantize(self.h, *self.hq)
        gba.grouped_gemm_bias_act_fp8_block(*self.hq, self.off, *self.c2, None, self.y, "none", **k)
        gba.moe_combine(self.y, self.rows, self.weights, self.out)

        gba.moe_combine_grad(self.dout, self.y, self.rows, self.weights, self.dy, self.dweights)
        r = self.route
        gba.moe_route_grad(self.logits, self.idx, self.dweights, self.dlogits, score=r["score"], scale=r["scale"])
        gba.fp8_quantize(self.dy, *self.dyq, pow2=True)
        gba.grouped_gemm_act_grad_fp8_block(*self.dyq, self.off, *self.c2t, self.z, self.dz, "gelu", **k)
        gba.fp8_quantize(self.dz, *self.dzq)
        gba.grouped_gemm_act_grad_fp8_block(*self.dzq, self.off, *self.c1t, None, self.dxs, "none", **k)
        gba.moe_combine(self.dxs, self.rows, None, self.dx)
        gba.moe_dispatch(self.x, self.rows, self.xs)
        gba.grouped_gemm_wgrad(self.xs, self.dz, self.off, self.dw1, self.db1, transpose_b=True, **k)
        gba.grouped_gemm_wgrad(self.h, self.dy, self.off, self.dw2, None, transpose_b=True, **k)


def check_product(what, codes, scales, off, wc, wsc, bias, act, out, preact=None, z=None):
    E, dt = wc.shape[0], out.dtype
    a64 = orc.values(codes.view(torch.uint8), scales.T.contiguous())
    n = int(off[-1])
    a64[n:] = 0
    w64 = torch.stack([orc.values(wc[e].view(torch.uint8), wsc[e], 128) for e in range(E)])
    sums, err, owned = orc.product(a64, off.tolist(), w64, bias)
    assert torch.equal(owned, torch.arange(len(owned), device="cuda") < n)
    if z is not None or act == "none" and preact is None:
        s = eo.slope(act, z.double()) if z is not None else torch.ones_like(sums)
        want, tol = sums * s, err * s.abs() + (eo.SLOPE_TOL * (sums.abs() + err) if z is not None else 0)
    else:
        want, tol = eo.act(act, sums), eo.LIPSCHITZ[act] * err + eo.ACT_TOL
        eo.check(what + " preact", preact, sums, eo.with_rounding(sums, err, dt), owned)
    eo.check(what, out, want, eo.with_rounding(want, tol, dt), owned)
    assert torch.isnan(out[n:]).all()


def check_rows_codes(x, codes, scales, pow2=False):
    want, s = orc.quantize(x, 1, pow2)
    assert torch.equal(codes.view(torch.uint8), want) and torch.equal(scales, s.T.contiguous())


# tokens, experts, top, width, hidden, padding tokens, groups, score, type, logits' type
LAYERS = [(1, 4, 2, 64, 144, 0, 1, "softmax", "bf16", torch.float32), (77, 8, 2, 272, 400, 5, 1, "softmax", "f16", torch.float32),
          (300, 40, 6, 528, 1040, 17, 8, "sigmoid", "bf16", torch.bfloat16), (1100, 300, 8, 64, 80, 1, 4, "sigmoid", "bf16", torch.float32),
          (2100, 6, 3, 1056, 2064, 0, 1, "softmax", "f16", torch.float16), (9, 16, 4, 144, 64, 9, 1, "softmax", "bf16", torch.float32)]


@pytest.mark.parametrize("i", range(len(LAYERS)))
def test_a_layer_stage_by_stage(i):
    T, E, k, H, F, padding, groups, score, dtype, logits = LAYERS[i]
    say("layer", LAYERS[i])
    m = Layer(T, E, k, H, F, DT[dtype], groups, score, logits)
    m.fill(10 + i, padding)
    m.dirty()
    m.run()
    torch.cuda.synchronize()
    dt = DT[dtype]
    # routing
    idx, w, depth = orc.route(m.logits, m.bias, k, **m.route)
    assert torch.equal(m.idx.long(), idx)
    eo.check("weights", m.weights, w, orc.route_tol(w, depth))
    o, rows, slots = orc.sort(m.idx.cpu(), E)
    assert m.off.tolist() == o and m.rows.reshape(-1).tolist() == rows and m.slots.tolist() == slots
    n = (T - padding) * k
    assert o[-1] == n
    # forward
    there = m.slots[:n].long()
    token = there // k
    assert torch.equal(m.xs[:n], m.x[token]) and torch.isnan(m.xs[n:]).all()
    check_rows_codes(m.x[token], m.xq[0][:n], m.xq[1][:, :n])
    assert (m.xq[0].view(torch.uint8)[n:] == 0xff).all() and torch.isnan(m.xq[1][:, n:]).all()
    check_product("h", *m.xq, m.off, *m.c1, m.b1, "gelu", m.h, m.z)
    check_rows_codes(m.h[:n], m.hq[0][:n], m.hq[1][:, :n])
    check_product("y", *m.hq, m.off, *m.c2, None, "none", m.y)

    def combined(v, weights):
        """Sums over a token's rows, and their errors: k products and additions in 32 bits."""
        want, size = (torch.zeros(T, H, dtype=torch.float64, device="cuda") for _ in range(2))
        p = v[:n].double() * weights.reshape(-1)[there, None]
        want.index_add_(0, token, p)
        size.index_add_(0, token, p.abs())
        return want, eo.with_rounding(want, size * (k + 1) * 2.0 ** -24, dt)
    eo.check("out", m.out, *combined(m.y, m.weights.double()))
    # backward
    d = m.dout.double()
    want = d[token] * m.weights.reshape(-1)[there, None].double()
    eo.check("dy", m.dy[:n], want, eo.with_rounding(want, want.abs() * 2.0 ** -24, dt))
    assert torch.isnan(m.dy[n:]).all()
    dots, size = (torch.zeros(T * k, dtype=torch.float64, device="cuda") for _ in range(2))
    p = d[token] * m.y[:n].double()
    dots[there], size[there] = p.sum(1), p.abs().sum(1)
    eo.check("dweights", m.dweights.reshape(-1), dots, size * eo.sum_rel(H) + 1e-30)
    want, size, depth = orc.route_grad(m.logits, m.idx, m.dweights, score, True, 1.5)
    eo.check("dlogits", m.dlogits, want, eo.with_rounding(want, (2 * depth[:, None] + 60) * 2.0 ** -24 * size + 2.0 ** -120, logits))
    check_rows_codes(m.dy[:n], m.dyq[0][:n], m.dyq[1][:, :n], True)
    check_product("dz", *m.dyq, m.off, *m.c2t, None, "gelu", m.dz, z=m.z)
    check_rows_codes(m.dz[:n], m.dzq[0][:n], m.dzq[1][:, :n])
    check_product("dxs", *m.dzq, m.off, *m.c1t, None, "none", m.dxs)
    eo.check("dx", m.dx, *combined(m.dxs, torch.ones(T * k, dtype=torch.float64, device="cuda")))
    # weights and their gradients
    for wt, (c, s), (ct, st) in ((m.w1, m.c1, m.c1t), (m.w2, m.c2, m.c2t)):
        for e in range(0, E, 7):
            want, s64 = orc.quantize(wt[e], 128)
            assert torch.equal(c[e].view(torch.uint8), want) and torch.equal(s[e], s64)
            assert torch.equal(ct[e].view(torch.uint8), want.T) and torch.equal(st[e], s64.T)
    for e in range(0, E, 5):
        lo, hi = o[e], o[e + 1]
        for dw, a, b in ((m.dw1, m.dz, m.xs), (m.dw2, m.dy, m.h)):
            p, q = a[lo:hi].double().T.contiguous(), b[lo:hi].double()
            eo.check("dw", dw[e], p @ q, (p.abs() @ q.abs()) * eo.sum_rel(hi - lo) + 1e-30)


# ------------------------------------------------------------ graphs, threads --

def same(got, want):
    return [i for i, (a, b) in enumerate(zip(got, want)) if not torch.equal(a.view(torch.uint8), b.view(torch.uint8))]


@pytest.mark.parametrize("i", range(len(LAYERS)))
def test_two_graphs_replay_like_eager(i):
    """Two layers' steps, each captured with workspaces of its own and replayed in turn with inputs that change."""
    T, E, k, H, F, padding, groups, score, dtype, logits = LAYERS[i]
    say("graphs", LAYERS[i])
    both = []
    for n in range(2):
        m = Layer(T, E, k, H, F, DT[dtype], groups, score, logits)
        want = []
        for seed in (20 + n, 30 + n):
            m.fill(seed, padding)
            m.dirty()
            m.run()
            want.append([t.clone() for t in m.outputs()])
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            m.run()
        torch.cuda.synchronize()
        both.append((m, graph, want))
    for r in range(4):
        for n, (m, graph, want) in enumerate(both):
            m.fill((20, 30)[r % 2] + n, padding)
            m.dirty()
        torch.cuda.synchronize()
        say("replay", r)
        for m, graph, want in both:
            graph.replay()
        torch.cuda.synchronize()
        for m, graph, want in both:
            assert not same(m.outputs(), want[r % 2])


def test_threads_on_their_own_streams():
    """Four threads, a layer and a stream each: every call's bits are those of the same call alone."""
    say("threads")
    jobs = []
    for i in range(4):
        T, E, k, H, F, padding, groups, score, dtype, logits = LAYERS[i + 1]
        m = Layer(T, E, k, H, F, DT[dtype], groups, score, logits)
        m.fill(60 + i, padding)
        m.dirty()
        m.run()
        jobs.append((m, [t.clone() for t in m.outputs()], torch.cuda.Stream()))
    torch.cuda.synchronize()
    wrong = []

    def work(n):
        m, want, stream = jobs[n]
        try:
            with torch.cuda.stream(stream):
                for r in range(5):
                    m.dirty()
                    m.run()
                    stream.synchronize()
                    wrong.extend((n, r, j) for j in same(m.outputs(), want))
        except Exception as e:   # shown by the test's thread
            wrong.append((n, repr(e)))
    threads = [threading.Thread(target=work, args=(n,)) for n in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not wrong


# ------------------------------------------------------------------- extremes --

def weights8(w):
    c, s = torch.empty(w.shape, dtype=F8, device="cuda"), torch.empty(gba.fp8_weight_scales_shape(*w.shape), device="cuda")
    return gba.fp8_quantize_weights(w, c, s)


def rows8(x):
    c, s = torch.empty(x.shape, dtype=F8, device="cuda"), torch.empty(gba.fp8_scales_shape(*x.shape), device="cuda")
    return gba.fp8_quantize(x, c, s)


@pytest.mark.parametrize("rows", [3, 40])
def test_the_most_experts(rows):
    """4096 experts of up to `rows` rows: the streaming kernel, and the staged ones."""
    E, N, K, dt = 4096, 72, 144, torch.bfloat16
    say("4096 experts", rows)
    g = torch.Generator(device="cuda").manual_seed(9)
    sizes = torch.randint(0, rows, (E,), generator=g, device="cuda").tolist()
    sizes[4000] = 300
    off, T = make_offsets(sizes, 2), sum(sizes) + 2
    a, w, bias = rows8(draw(g, (T, K), dt)), weights8(draw(g, (E, N, K), dt, K ** -0.5)), draw(g, (E, N), dt)
    c = torch.full((T, N), float("nan"), dtype=dt, device="cuda")
    gba.grouped_gemm_bias_act_fp8_block(*a, off, *w, bias, c, "none")
    a64 = orc.values(a[0].view(torch.uint8), a[1].T.contiguous())
    w64 = orc.values(w[0].view(torch.uint8).view(E * N, K), torch.repeat_interleave(w[1].view(E, -1), N, 0), 1).view(E, N, K)
    want, err, owned = orc.product(a64, off.tolist(), w64, bias)
    eo.check("c", c, want, eo.with_rounding(want, err, dt), owned)
    assert torch.isnan(c[:2]).all()
    with pytest.raises(gba.GbaError):
        gba.grouped_gemm_bias_act_fp8_block(*a, make_offsets([0] * 4097), torch.empty(4097, 8, K, dtype=F8, device="cuda"),
                                            torch.empty(4097, 1, 2, device="cuda"), None, torch.empty(T, 8, dtype=dt, device="cuda"), "none")


# rows, experts, columns, depth, the kernel
OFFSETS = [(40, 4, 72, 4112, "ring"), (30, 8, 264, 528, "stream"), (2600, 4, 4104, 528, "persistent"), (500, 70, 136, 272, "stream"), (9000, 70, 136, 272, "ring"),
           (9000, 66, 4104, 272, None)]


@pytest.mark.parametrize("T,E,N,K,kind", OFFSETS)
def test_offsets_that_reach_outside_the_rows(T, E, N, K, kind):
    """Offsets in order: the rows are those of the clamped offsets, and nothing else is written."""
    p = gba.moe.plan(T, E, N, K, 0, torch.cuda.get_device_properties(0).multi_processor_count)
    assert kind in (None, p["kind"])
    g = torch.Generator(device="cuda").manual_seed(T + E)
    dt = torch.bfloat16
    a, w = rows8(draw(g, (T, K), dt)), weights8(draw(g, (E, N, K), dt, K ** -0.5))
    z = draw(g, (T, N), dt)
    a64 = orc.values(a[0].view(torch.uint8), a[1].T.contiguous())
    w64 = torch.stack([orc.values(w[0][e].view(torch.uint8), w[1][e], 128) for e in range(E)])
    for o in lists(T, E):
        say("offsets", T, E, N, K, o[:8])
        off = torch.tensor(o, dtype=torch.int32, device="cuda")
        c, da = (torch.full((T, N), float("nan"), dtype=dt, device="cuda") for _ in range(2))
        gba.grouped_gemm_bias_act_fp8_block(*a, off, *w, None, c, "none")
        gba.grouped_gemm_act_grad_fp8_block(*a, off, *w, z, da, "relu")
        want, err, owned = orc.product(a64, [min(max(v, 0), T) for v in o], w64, None)
        eo.check("c", c, want, eo.with_rounding(want, err, dt), owned)
        s = (z > 0).double()
        eo.check("da", da, want * s, eo.with_rounding(want * s, err, dt), owned)
        assert torch.isnan(c[~owned]).all() and torch.isnan(da[~owned]).all()


@pytest.mark.parametrize("N,kind", [(72, "ring"), (520, "persistent")])
def test_many_rows(N, kind):
    """270000 rows of 16400 values: 8-bit and 16-bit arrays past 2^32 bytes, in every movement and product."""
    T, K, tail, dt = 270000, 16400, 200, torch.bfloat16
    depth = 64 if kind == "ring" else 512
    say("many rows", N)
    assert gba.moe.plan(T, 3, N, K)["kind"] == gba.moe.plan(T, 3, K, depth)["kind"] == kind
    g = torch.Generator(device="cuda").manual_seed(21)
    x = torch.empty(T, K, dtype=dt, device="cuda").normal_(generator=g)
    codes, scales = torch.empty(T, K, dtype=F8, device="cuda"), torch.empty(gba.fp8_scales_shape(T, K), device="cuda")
    gba.fp8_quantize(x, codes, scales)
    check_rows_codes(x[-tail:], codes[-tail:], scales[:, -tail:])
    sizes = [100000, 162200, 7800]
    off, w = make_offsets(sizes), weights8(draw(g, (3, N, K), dt, K ** -0.5))
    c = torch.empty(T, N, dtype=dt, device="cuda")
    gba.grouped_gemm_bias_act_fp8_block(codes, scales, off, *w, None, c, "none")
    a64 = orc.values(codes[-tail:].view(torch.uint8), scales[:, -tail:].T.contiguous())
    want, err, _ = orc.product(a64, [0, tail], orc.values(w[0][2].view(torch.uint8), w[1][2], 128)[None], None)
    eo.check("c", c[-tail:], want, eo.with_rounding(want, err, dt))
    # as a gradient: outputs and pre-activations of 16400 columns
    dc, wt = rows8(c[:, :depth].contiguous()), weights8(draw(g, (3, K, depth), dt, depth ** -0.5))
    da = torch.empty(T, K, dtype=dt, device="cuda")
    gba.grouped_gemm_act_grad_fp8_block(*dc, off, *wt, x, da, "relu")
    a64 = orc.values(dc[0][-tail:].view(torch.uint8), dc[1][:, -tail:].T.contiguous())
    want, err, _ = orc.product(a64, [0, tail], orc.values(wt[0][2].view(torch.uint8), wt[1][2], 128)[None], None)
    s = (x[-tail:] > 0).double()
    eo.check("da", da[-tail:], want * s, eo.with_rounding(want * s, err, dt))
    # movement: a row of the last tokens comes from, and goes to, the end
    rows = torch.randperm(T, generator=g, device="cuda").to(torch.int32).view(-1, 2)
    half = T // 2
    y = da
    gba.moe_dispatch(x[:half], rows, y)
    assert all(torch.equal(y[rows[-tail:, j].long()], x[half - tail:half]) for j in range(2))
    gba.fp8_quantize(x[:half], codes, scales, rows=rows)
    last = rows[-tail:, 1].long()
    check_rows_codes(x[half - tail:half], codes.view(torch.uint8)[last], scales[:, last])
    weights = torch.rand(half, 2, generator=g, device="cuda")
    out = torch.empty(half, K, dtype=dt, device="cuda")
    gba.moe_combine(y, rows, weights, out)
    exact = x[half - tail:half].double() * weights[-tail:].double().sum(1)[:, None]
    eo.check("out", out[-tail:], exact, eo.with_rounding(exact, exact.abs() * 3 * 2.0 ** -24, dt))
    dweights = torch.empty_like(weights)
    gba.moe_combine_grad(x[half:], y, rows, weights, None, dweights)
    p = x[T - tail:].double() * x[half - tail:half].double()
    eo.check("dweights", dweights[-tail:], p.sum(1)[:, None].expand(-1, 2), (p.abs().sum(1) * eo.sum_rel(K))[:, None].expand(-1, 2))
    gba.fp8_dequantize(codes, scales, y)
    v = (codes[-tail:].float() * scales[:, -tail:].T.repeat_interleave(128, 1)[:, :K]).to(dt)
    assert torch.equal(y[-tail:], v)


def test_many_weights():
    """80 experts of 4096 x 16400: 8-bit weights past 2^32 bytes."""
    E, N, K, dt = 80, 4096, 16400, torch.bfloat16
    say("many weights")
    g = torch.Generator(device="cuda").manual_seed(22)
    w = torch.empty(E, N, K, dtype=dt, device="cuda").normal_(generator=g)
    c, s = weights8(w)
    ct, st = torch.empty(E, K, N, dtype=F8, device="cuda"), torch.empty(gba.fp8_weight_scales_shape(E, K, N), device="cuda")
    gba.fp8_quantize_weights(w, None, None, ct, st)
    want, s64 = orc.quantize(w[-1], 128)
    assert torch.equal(c[-1].view(torch.uint8), want) and torch.equal(s[-1], s64)
    assert torch.equal(ct[-1].view(torch.uint8), want.T) and torch.equal(st[-1], s64.T)
    w64 = orc.values(want, s64, 128)[None]
    gba.fp8_dequantize_weights(c, s, w)
    assert torch.equal(w[-1], w64[0].to(dt))
    for n, kind in ((1, "stream"), (40, "ring"), (3800, "persistent")):
        assert gba.moe.plan(2 * n, E, N, K)["kind"] == kind
        sizes = [n] + [0] * (E - 2) + [n]
        off = make_offsets(sizes)
        a = rows8(draw(g, (2 * n, K), dt))
        a64 = orc.values(a[0].view(torch.uint8), a[1].T.contiguous())[n:]
        out = torch.empty(2 * n, N, dtype=dt, device="cuda")
        gba.grouped_gemm_bias_act_fp8_block(*a, off, c, s, None, out, "none")
        want, err, _ = orc.product(a64, [0, n], w64, None)
        eo.check("c", out[n:], want, eo.with_rounding(want, err, dt))
        back = torch.empty(2 * n, K, dtype=dt, device="cuda")
        d = rows8(out)
        gba.grouped_gemm_act_grad_fp8_block(*d, off, ct, st, None, back, "none")
        want, err, _ = orc.product(orc.values(d[0].view(torch.uint8), d[1].T.contiguous())[n:], [0, n], w64.transpose(1, 2).contiguous(), None)
        eo.check("da", back[n:], want, eo.with_rounding(want, err, dt))


# -------------------------------------------------------------------- example --

def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "expert_layer.py")
    spec = importlib.util.spec_from_file_location("expert_layer", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    return ex


def test_the_example_runs():
    say("example")
    ex = example()
    losses, layer, router, x = ex.train(tokens=300, experts=6, top=2, width=128, hidden=192, steps=2, seed=3)
    assert len(losses) == 2 and all(torch.isfinite(v) for v in losses)
    four, eight = ex.served_errors(layer, router, x, 2)
    # A code of 8 bits is off by up to 2^-4 of its value, its root mean square about half; four roundings
    # (inputs, weights, twice) add up to some 2^-4.
    assert 0 < eight < 0.125 and eight < four < 0.4


@pytest.mark.parametrize("tokens,experts,top,width,hidden", [(40, 4, 2, 64, 72), (257, 6, 3, 128, 96)])
def test_the_examples_gradients(tokens, experts, top, width, hidden):
    """Against the formulas in 64 bits. With every value goes the bound on its error, formed from those of its factors
    (|a b - a' b'| <= |a| eb + |b| ea + ea eb), the sums' and one rounding wherever the layer stores."""
    say("example's gradients", tokens, experts)
    ex = example()
    g = torch.Generator(device="cuda").manual_seed(5)
    layer = ex.ExpertLayer(experts, width, hidden, seed=8)
    router = torch.randn(experts, width, generator=g, device="cuda")
    x = torch.randn(tokens, width, generator=g, device="cuda").to(layer.dtype)
    goal = torch.randn(tokens, width, generator=g, device="cuda").to(layer.dtype)
    loss, drouter = ex.gradients(layer, router, x, goal, top)
    half = torch.finfo(layer.dtype).eps / 2

    def stored(v, e):
        return v, e + half * (v.abs() + e)

    def mul(a, b):
        return a[0] * b[0], a[0].abs() * b[1] + b[0].abs() * a[1] + a[1] * b[1]

    def mm(a, b, n):
        """Product of matrices and its error, n terms summed in 32 bits."""
        size = (a[0].abs() + a[1]) @ (b[0].abs() + b[1])
        return a[0] @ b[0], a[0].abs() @ b[1] + a[1] @ b[0].abs() + a[1] @ b[1] + size * (eo.sum_rel(n) + 2.0 ** -23)
    exact = lambda v: (v.double(), torch.zeros_like(v, dtype=torch.float64))
    T = lambda p: (p[0].T.contiguous(), p[1].T.contiguous())
    logits = mm(exact(x), T(exact(router)), width)
    idx = logits[0].topk(top, 1).indices
    chosen = logits[0].gather(1, idx)
    w = chosen.softmax(1)
    # softmax: d w_i <= w_i (1 - w_i) (e_i + e_j), twice that for the second order; and the weights' own tolerance
    el = logits[1].gather(1, idx).amax(1, keepdim=True)
    w = (w, w * (4 * el) + 2.0 ** -20 * w + 2.0 ** -60)
    y = torch.zeros(tokens, top, width, dtype=torch.float64, device="cuda"), torch.zeros(tokens, top, width, dtype=torch.float64, device="cuda")
    h, z = ((torch.zeros(tokens, top, hidden, dtype=torch.float64, device="cuda"), torch.zeros(tokens, top, hidden, dtype=torch.float64, device="cuda"))
            for _ in range(2))
    masks = [idx == e for e in range(experts)]
    for e, at in enumerate(masks):
        xe = x[at.nonzero()[:, 0]]
        ze = mm(exact(xe), T(exact(layer.w1[e])), width + 1)
        b = layer.b1[e].double()
        ze = ze[0] + b, ze[1] + 2.0 ** -22 * b.abs()
        he = stored(eo.act("gelu", ze[0]), eo.LIPSCHITZ["gelu"] * ze[1] + eo.ACT_TOL)
        ye = stored(*mm(he, T(exact(layer.w2[e])), hidden))
        for dst, src in ((z, stored(*ze)), (h, he), (y, ye)):
            dst[0][at], dst[1][at] = src
    wy = mul((w[0][..., None], w[1][..., None]), y)
    out = stored(wy[0].sum(1), wy[1].sum(1) + (wy[0].abs() + wy[1]).sum(1) * (top + 1) * 2.0 ** -23)
    off = out[0] - goal.double(), out[1] + 2.0 ** -23 * (out[0].abs() + goal.double().abs() + out[1])
    want = off[0].square().sum(1).mean()
    tol = (2 * off[0].abs() * off[1] + off[1] ** 2).sum(1).mean() + want * (eo.sum_rel(width) + eo.sum_rel(tokens)) * 2
    assert abs(loss.item() - want.item()) <= tol.item()
    dout = stored(off[0] * 2 / tokens, off[1] * 2 / tokens + off[0].abs() * 2.0 ** -22 / tokens)
    # the router
    p = mul((dout[0][:, None], dout[1][:, None]), y)
    dw = p[0].sum(2), p[1].sum(2) + (p[0].abs() + p[1]).sum(2) * (eo.sum_rel(width) + 2.0 ** -23)
    wdw = mul(w, dw)
    mean = wdw[0].sum(1, keepdim=True), wdw[1].sum(1, keepdim=True) + wdw[0].abs().sum(1, keepdim=True) * 2.0 ** -20
    centred = dw[0] - mean[0], dw[1] + mean[1] + 2.0 ** -20 * (dw[0].abs() + mean[0].abs())
    dl = mul(w, centred)
    dlogits = [torch.zeros(tokens, experts, dtype=torch.float64, device="cuda").scatter(1, idx, v) for v in (dl[0], dl[1] + 2.0 ** -20 * dl[0].abs())]
    want, tol = mm(T(dlogits), exact(x), tokens)
    eo.check("drouter", drouter, want, tol)
    # the experts. d gelu' / dz is at most 1.2: (2 - z^2) phi(z), 0.8 at 0, below that in size elsewhere
    dy = stored(*mul((w[0][..., None], w[1][..., None]), (dout[0][:, None].expand(-1, top, -1), dout[1][:, None].expand(-1, top, -1))))
    slope = eo.slope("gelu", z[0]), 1.2 * z[1] + eo.SLOPE_TOL
    for e, at in enumerate(masks):
        pick = lambda v: (v[0][at], v[1][at])
        xe, n = exact(x[at.nonzero()[:, 0]]), max(int(at.sum()), 1)
        want, tol = mm(T(pick(dy)), pick(h), n)
        eo.check("dw2", layer.grads[2][e], want, tol + 1e-30)
        d = mm(pick(dy), exact(layer.w2[e]), width)
        dz = stored(*mul(d, pick(slope)))
        want, tol = mm(T(dz), xe, n)
        eo.check("dw1", layer.grads[0][e], want, tol + 1e-30)
        eo.check("db1", layer.grads[1][e], dz[0].sum(0), dz[1].sum(0) + (dz[0].abs() + dz[1]).sum(0) * (eo.sum_rel(n) + 2.0 ** -23) + 1e-30)
