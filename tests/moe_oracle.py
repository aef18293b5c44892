"""Plain 64-bit forms of routing, of the movement of rows and of the 8-bit format by blocks,
and the tolerances their kernels are held to.

Tolerances, derived from the number of roundings:
  * 32-bit scores and weights: the argument of an exponential is rounded (2^-24 of it, which is as much
    of the result), expf is off by 2^-22 at most, a sum over 1024 experts is 16 additions in a lane and 6
    across lanes, then a reciprocal or division and a product or two: (2 D + 40) 2^-24 of the value, D the
    largest argument, for a quotient of two such;
  * gradients: a weight and the difference of two terms, (2 D + 60) 2^-24 of the sum of magnitudes;
  * sums over k slots: one rounding a term, k 2^-24 of the sum of magnitudes;
  * dot products over H: at most H / 256 + 8 terms a lane, 6 additions across lanes, 4 across waves: (H / 256 +
    20) 2^-24 of the sum of magnitudes;
  * 8-bit products: the matrix instruction takes each eight consecutive products together and cuts them towards
    zero to multiples of 2^(e - 13), 2^e at most the largest of their magnitudes (test_the_matrix_instructions_rule
    measures this): at most seven of them lose less than 2^-13 of the largest each. The largest is at most the
    product of the eight places' largest values of either side. Then 16 sums an instruction and one for
    each block, each off by at most one step (2^-23 of the magnitudes), and the rounding of the scales' product and of
    the product by it.
"""
import math

import torch

from tests import experts_oracle as eo


def route(x, bias, k, score="softmax", renorm=True, scale=1.0, groups=1, top_groups=1, group_best=1):
    """(indices [T,k] int64, weights [T,k] in 64 bits, D: the largest argument of an exponential a row)."""
    x64 = x.double()
    T, E = x64.shape
    bad = torch.isnan(x64).any(1)
    if score == "softmax":
        bad |= (x64 == math.inf).any(1)
    if bias is not None:
        bad |= torch.isnan(bias).any()
    x64 = torch.where(bad[:, None], torch.zeros_like(x64), x64)
    if score == "softmax":
        m = x64.amax(1, keepdim=True)
        m = torch.where(m == -math.inf, torch.zeros_like(m), m)
        e = torch.exp(x64 - m)
        s = e / e.sum(1, keepdim=True).clamp(min=1e-300)
        depth = torch.where(x64 == -math.inf, m, x64).sub(m).abs().amax(1)
    else:
        s = 1 / (1 + torch.exp(-x64))
        depth = torch.where(torch.isinf(x64), torch.zeros_like(x64), x64).abs().amax(1)
    left = x64 != -math.inf
    if bias is not None:
        left &= (bias != -math.inf)[None]
    plain = bias is None and (groups == top_groups or group_best == 1)
    value = x64 if plain else s + (0 if bias is None else bias.double())
    value = torch.where(left, value.clamp(-1e300, 1e300), torch.full_like(value, -math.inf))
    if groups > top_groups:
        by = value.view(T, groups, -1)
        best = by.sort(dim=2, descending=True).values[:, :, :group_best]
        total = torch.where(best == -math.inf, torch.zeros_like(best), best).sum(2)
        total = torch.where(best[:, :, 0] == -math.inf, torch.full_like(total, -math.inf), total)
        kept = torch.zeros_like(total, dtype=torch.bool).scatter(1, total.sort(dim=1, descending=True, stable=True).indices[:, :top_groups], True)
        value = torch.where(kept[:, :, None], by, torch.full_like(by, -math.inf)).view(T, E)
    v, idx = value.sort(dim=1, descending=True, stable=True)
    v, idx = v[:, :k], idx[:, :k]
    none = (v == -math.inf) | bad[:, None]
    log_s = torch.log_softmax(x64, 1) if score == "softmax" else -torch.logaddexp(torch.zeros_like(x64), -x64)
    ls = log_s.gather(1, idx).masked_fill(none, -math.inf)
    if renorm:
        top = ls.amax(1, keepdim=True)
        ls = ls - torch.where(top == -math.inf, torch.zeros_like(top), torch.logsumexp(ls, 1, keepdim=True))
    w = torch.where(none, torch.zeros_like(ls), torch.exp(ls) * scale)
    w = torch.where(bad[:, None], torch.full_like(w, math.nan), w)
    return torch.where(none, torch.full_like(idx, -1), idx), w, depth


def route_tol(w, depth):
    return (2 * depth[:, None] + 40) * 2.0 ** -24 * w.abs() + 2.0 ** -120


def route_grad(x, idx, dw, score="softmax", renorm=True, scale=1.0):
    """(dx in 64 bits by the formulas, sums of magnitudes, D)."""
    x64 = x.double()
    T, E = x64.shape
    ok = idx >= 0
    at = idx.clamp(min=0).long()
    g = torch.where(ok, dw.double() * scale, torch.zeros(()).double().to(dw.device))
    if score == "softmax":
        m = x64.amax(1, keepdim=True).clamp(min=-1e300)
        p = torch.exp(x64 - m)
        p = p / p.sum(1, keepdim=True).clamp(min=1e-300)
        depth = torch.where(x64 == -math.inf, m, x64).sub(m).abs().amax(1)
    else:
        p = torch.special.expit(x64)
        depth = torch.where(torch.isinf(x64), torch.zeros_like(x64), x64).abs().amax(1)
    s = torch.where(ok, p.gather(1, at), torch.zeros_like(g))
    z = torch.zeros_like(x64)
    if renorm:
        if score == "softmax":
            ls = torch.where(ok, x64.gather(1, at), torch.full_like(g, -math.inf))
        else:
            ls = torch.where(ok, -torch.logaddexp(torch.zeros_like(g), -x64.gather(1, at)), torch.full_like(g, -math.inf))
        q = torch.exp(ls - ls.amax(1, keepdim=True).clamp(min=-1e300))
        q = q / q.sum(1, keepdim=True).clamp(min=1e-300)
        slope = torch.special.expit(-x64.gather(1, at)) if score == "sigmoid" else torch.ones_like(q)
        mean, size = (q * g).sum(1, keepdim=True), (q * g.abs()).sum(1, keepdim=True)
        d, a = q * slope * (g - mean), q * slope * (g.abs() + size)
    elif score == "softmax":
        mean, size = (s * g).sum(1, keepdim=True), (s * g.abs()).sum(1, keepdim=True)
        some = ok.any(1, keepdim=True)
        full = torch.zeros_like(z).scatter_add(1, at, torch.where(ok, g, torch.zeros_like(g)))
        dx = torch.where(some, p * (full - mean), z)
        return dx, torch.where(some, p * (full.abs() + size), z), depth
    else:
        d = g * s * torch.special.expit(-x64.gather(1, at))
        a = d.abs()
    zero = torch.zeros_like(d)
    return z.scatter_add(1, at, torch.where(ok, d, zero)), z.scatter_add(1, at, torch.where(ok, a, zero)), depth


def sort(idx, E):
    """(offsets, rows, slots) as lists, by a loop over the slots."""
    flat = idx.reshape(-1).tolist()
    by = [[] for _ in range(E)]
    for i, e in enumerate(flat):
        if 0 <= e < E:
            by[e].append(i)
    offsets, rows, slots = [0], [-1] * len(flat), []
    for e in range(E):
        for i in by[e]:
            rows[i] = len(slots)
            slots.append(i)
        offsets.append(len(slots))
    return offsets, rows, slots + [-1] * (len(flat) - len(slots))


# -------------------------------------------------------------- 8 bits ----

def e4m3_values():
    """The 127 magnitudes of codes 0 .. 126 in order, in 64 bits."""
    out = []
    for c in range(127):
        e, m = c >> 3, c & 7
        out.append(m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))
    return torch.tensor(out, dtype=torch.float64)


def to_codes(q):
    """Codes (uint8) of 64-bit values, nearest, ties to the even code, by a search in the table."""
    table = e4m3_values().to(q.device)
    m = q.abs().clamp(max=448.0)
    hi = torch.searchsorted(table, m.contiguous()).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    down, up = m - table[lo], table[hi] - m
    code = torch.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi)
    return (code + 128 * torch.signbit(q).long()).to(torch.uint8)


def _block_scale(top, pow2):
    """(fp32 scale, what a value is multiplied by, as numerator and denominator) of 64-bit maxima."""
    finite = torch.isfinite(top)
    t = torch.where(finite, top, torch.ones_like(top))
    tiny = t < 448 * 2.0 ** -126
    if pow2:
        s = torch.exp2(torch.ceil(torch.log2(torch.where(tiny, torch.ones_like(t), t) / 448)))
        s = torch.where(s * 448 < t, s * 2, s)                      # the logarithm's rounding
        s = torch.where(s * 224 >= torch.where(tiny, torch.full_like(t, 1e30), t), s / 2, s)
        num, den = torch.ones_like(t), s
    else:
        s = t / 448
        num, den = torch.full_like(t, 448.0), torch.where(tiny, torch.ones_like(t), t)
    num = torch.where(tiny, torch.full_like(t, 2.0 ** 126), num)
    den = torch.where(tiny, torch.ones_like(t), den)
    s = torch.where(tiny, torch.full_like(t, 2.0 ** -126), s)
    return torch.where(finite, s, torch.full_like(s, math.nan)).float(), num, den, finite


def quantize(x, rows_a_block=1, pow2=False):
    """(codes [R,K] uint8, scales [row blocks, K blocks] fp32) of 16-bit values by blocks of rows_a_block x 128."""
    R, K = x.shape
    up, wide = -(-R // rows_a_block) * rows_a_block, -(-K // 128) * 128
    full = torch.zeros(up, wide, dtype=torch.float64, device=x.device)
    full[:R, :K] = x.double()
    b = full.view(up // rows_a_block, rows_a_block, wide // 128, 128)
    top = torch.nan_to_num(b.abs(), nan=math.inf, posinf=math.inf).amax((1, 3), keepdim=True)
    s, num, den, finite = _block_scale(top, pow2)
    q = torch.where(finite, b, torch.zeros_like(b)) * num / den
    codes = torch.where(finite, to_codes(q.reshape(-1)).view(b.shape), torch.zeros((), dtype=torch.uint8, device=x.device))
    return codes.reshape(up, wide)[:R, :K].contiguous(), s[:, 0, :, 0].contiguous()


def values(codes, scales, rows_a_block=1):
    """64-bit values of codes [R,K] and scales [row blocks, K blocks]."""
    R, K = codes.shape
    table = e4m3_values().to(codes.device)
    c = codes.long()
    v = torch.where(c >= 128, -1.0, 1.0).double() * table[(c & 127).clamp(max=126)]
    return v * scales.double().repeat_interleave(rows_a_block, 0)[:R].repeat_interleave(128, 1)[:, :K]


def eights(v):
    """The largest magnitude of each eight consecutive values: [R,K] to [R,ceil(K/8)] (K a multiple of 8)."""
    return v.abs().unflatten(1, (-1, 8)).amax(2) if v.shape[1] else v


def product(a, offsets, w, bias, T=None):
    """(sums [T,N], error bounds, rows that some expert owns) of 64-bit values a [T,K], w [E,N,K]."""
    T, K = a.shape
    N = w.shape[1]
    r = torch.zeros(T, N, dtype=torch.float64, device=a.device)
    err, owned = torch.zeros_like(r), torch.zeros(T, dtype=torch.bool, device=a.device)
    for e, b, n in eo.groups(offsets, T):
        if n:
            m, x = w[e].T.contiguous(), a[b:b + n]
            r[b:b + n] = x @ m
            size = x.abs() @ m.abs()
            if bias is not None:
                r[b:b + n] += bias[e].double()
                size += bias[e].double().abs()
            cut = eights(x) @ eights(w[e]).T.contiguous()
            err[b:b + n] = size * (16 + -(-max(K, 1) // 128) + 4) * 2.0 ** -23 + 7 * 2.0 ** -13 * cut
            owned[b:b + n] = True
    return r, err, owned
