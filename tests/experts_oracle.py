"""Plain 64-bit forms of the grouped products and of the microscaled 4-bit format,
and the tolerances their kernels are held to.

Tolerances, derived from the number of roundings:
  * one rounding of the output: half a step, eps/2 of the value (bf16 2^-8, fp16
    2^-11, fp32 2^-24 of it) and half the smallest subnormal;
  * the fp32 sum of K products of 16-bit values: 2 sqrt(K + 1) 2^-24 of the sum of
    magnitudes S (statistical; the products are exact in fp32);
  * 4-bit products: 128 exact products an instruction, each addition off by at
    most one step (2^-23 of S), then one addition an instruction;
  * activations: slope bound L times the sum's error, and 2^-19 for the
    polynomial of GELU (8e-6 of |z| Phi(-|z|) <= 0.17) and the exp2 and reciprocal
    of the others; derivatives: 5e-6 (8e-6 of Phi(-|z|) <= 1/2, and a few fp32
    roundings of values below 1.13).
"""
import math

import torch

ACTS = ("none", "relu", "sigmoid", "gelu", "softplus", "gelu_tanh")
LIPSCHITZ = {"none": 1.0, "relu": 1.0, "sigmoid": 0.25, "gelu": 1.13, "softplus": 1.0, "gelu_tanh": 1.13}
ACT_TOL = 2.0 ** -19
SLOPE_TOL = 5e-6
CODE_VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def act(name, z):
    if name == "none":
        return z
    if name == "relu":
        return torch.where(z > 0, z, torch.where(torch.isnan(z), z, torch.zeros_like(z)))
    if name == "sigmoid":
        return torch.special.expit(z)
    if name == "gelu":
        return 0.5 * z * torch.special.erfc(-z / math.sqrt(2))
    if name == "softplus":
        return torch.clamp(z, min=0) + torch.log1p(torch.exp(-z.abs()))
    return z * torch.special.expit(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))


def slope(name, z):
    if name == "none":
        return torch.ones_like(z)
    if name == "relu":
        return (z > 0).double()
    if name == "sigmoid":
        return torch.special.expit(z) * torch.special.expit(-z)
    if name == "gelu":
        return 0.5 * torch.special.erfc(-z / math.sqrt(2)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if name == "softplus":
        return torch.special.expit(z)
    c = math.sqrt(2 / math.pi)
    u = 2 * c * (z + 0.044715 * z ** 3)
    return torch.special.expit(u) + z * torch.special.expit(u) * torch.special.expit(-u) * 2 * c * (1 + 3 * 0.044715 * z * z)


def groups(offsets, T):
    """(expert, first row, rows) with the offsets clamped as the library clamps them."""
    o = [min(max(int(v), 0), T) for v in offsets]
    return [(e, o[e], max(o[e + 1] - o[e], 0)) for e in range(len(o) - 1)]


def _nk(w, transpose_b):
    """w as [K, N] in 64 bits."""
    return w.double().T if transpose_b else w.double()


def sum_rel(K, mx4=False):
    if mx4:
        return (127 + -(-max(K, 1) // 128) + 1) * 2.0 ** -23
    return 2 * math.sqrt(K + 1) * 2.0 ** -24


def rounding(r, dtype):
    """Half a step of `dtype` at r."""
    tiny = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134, torch.float32: 2.0 ** -150}[dtype]
    return torch.finfo(dtype).eps / 2 * r.abs() + tiny


def with_rounding(r, err, dtype):
    """Bound on |rounded(v) - r| for |v - r| <= err."""
    return err + rounding(r.abs() + err, dtype)


def product(a, offsets, w, bias, transpose_b, mx4=False):
    """(sums [T,N], error bounds of the fp32 sums, rows that some expert owns)."""
    T, K = a.shape
    N = w.shape[1] if transpose_b else w.shape[2]
    r = torch.zeros(T, N, dtype=torch.float64, device=a.device)
    err = torch.zeros_like(r)
    owned = torch.zeros(T, dtype=torch.bool, device=a.device)
    for e, b, n in groups(offsets, T):
        if n:
            x, m = a[b:b + n].double(), _nk(w[e], transpose_b)
            r[b:b + n] = x @ m.contiguous()
            size = x.abs() @ m.abs().contiguous()
            if bias is not None:
                r[b:b + n] += bias[e].double()
                size += bias[e].double().abs()
            err[b:b + n] = size * sum_rel(K, mx4)
            owned[b:b + n] = True
    return r, err, owned


def check(what, got, want, bound, owned=None, sentinel=None):
    """Every owned row of got within bound of want; the others still `sentinel`."""
    g = got.double()
    if owned is not None:
        rest = got[~owned]
        assert torch.isnan(rest).all() if sentinel is None else (rest == sentinel).all(), "%s: rows of no expert were written" % what
        g, want, bound = g[owned], want[owned], bound[owned]
    off = (g - want).abs()
    bad = ~(off <= bound)
    if bad.any():
        at = torch.nonzero(bad)[0].tolist()
        raise AssertionError("%s: %d of %d values out of bounds, first at %s: got %r, want %r, bound %.3g" % (
            what, int(bad.sum()), bad.numel(), at, g[tuple(at)].item(), want[tuple(at)].item(), bound[tuple(at)].item()))


# ------------------------------------------------------------------ 4 bits ----

def mx4_quantize(x):
    """(codes [M,K] of 0..15, scale bytes [M,K/32]) of 16-bit values, by the definition."""
    M, K = x.shape
    b = x.double().reshape(M, K // 32, 32)
    top = b.abs().amax(-1)
    finite = torch.isfinite(b).all(-1)
    t = torch.where(finite & (top > 0), top, torch.ones_like(top))
    s = torch.frexp(t).exponent.long() - 1 - 2 + 127          # floor(log2) = exponent - 1
    s = torch.where(top > 0, s.clamp(min=0), torch.zeros_like(s))
    s = torch.where(finite, s, torch.full_like(s, 255))
    unit = ((s - 127 + 1023) << 52).view(torch.float64)
    y = torch.where(finite[..., None], b / unit[..., None], torch.zeros_like(b))
    table = torch.tensor(CODE_VALUES, dtype=torch.float64, device=x.device)
    d = (y.abs()[..., None] - table).abs()
    code = d.argmin(-1)                                        # the lower of two equally near
    near = d.gather(-1, code[..., None])[..., 0]
    up = (code + 1).clamp(max=7)
    tie = (d.gather(-1, up[..., None])[..., 0] == near) & (up != code) & (up % 2 == 0)
    code = torch.where(tie, up, code)
    code = code + 8 * torch.signbit(y).long()
    return code.reshape(M, K), s


def mx4_values(codes, s):
    """64-bit values of codes [M,K] and scale bytes [M,K/32]."""
    table = torch.tensor(CODE_VALUES + tuple(-v for v in CODE_VALUES), dtype=torch.float64, device=codes.device)
    unit = ((s.long() - 127 + 1023) << 52).view(torch.float64)
    unit = torch.where(s == 255, torch.full_like(unit, float("nan")), unit)
    return table[codes.long()] * unit.repeat_interleave(32, 1)


def mx4_pack(codes, s):
    """The stored form: packed codes and scale planes."""
    M, K = codes.shape
    c = codes.to(torch.uint8)
    planes = -(-K // 128)
    p = torch.zeros(planes, M, 4, dtype=torch.uint8, device=codes.device)
    for b in range(K // 32):
        p[b // 4, :, b % 4] = s[:, b].to(torch.uint8)
    return c[:, 0::2] | (c[:, 1::2] << 4), p
