"""Cases of a mixture of experts' routing, of the movement of its rows, and of the 8-bit
products scaled by blocks of 128.

Four kinds of case, all on the GPU:

  route    a router's logits [T, E] to each token's k experts and their weights, and the
           sorting of the T k (token, expert) pairs by expert: group offsets, and each
           pair's row; where the case trains, the logits' gradient too;
  move     tokens copied to their rows (dispatch), rows summed back by weight (combine);
           where the case trains, the gradients of both;
  quant    16-bit values to 8-bit floats (E4M3) with one fp32 scale a block of 128, and
           back: activations in blocks along a row, moved to their experts' rows on the
           way where the case says so, or weights in blocks of 128 x 128, and transposed;
  product  c = act(a . w^T + bias) with both operands in that format, dense or by expert,
           or (act' in place of act) the gradient of a product's input; where the case
           says so the 16-bit activations are quantised first.

A token's slot (t, j) goes to expert indices[t, j], -1 where none is left (a padded row of a
batch has logits of -inf). Rows are sorted by expert, a row's place within its expert by (t, j).
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
F8 = torch.float8_e4m3fn


# ---------------------------------------------------------------- cases ----

def listed():
    return [
        # One decoding step of 8 sequences: latency.
        {"name": "route decode", "kind": "route", "dtype": "bf16", "T": 8, "E": 32, "k": 2, "score": "softmax", "renorm": True,
         "scale": 1.0, "bias": False, "groups": 1, "top_groups": 1, "group_best": 1, "masked": 0, "padded": 0, "train": False},
        # A prompt's odd number of tokens through a router with a bias for balance, limited to 4 of 8 groups
        # of experts; the batch is padded and some experts are switched off.
        {"name": "route prompt", "kind": "route", "dtype": "fp32", "T": 999, "E": 256, "k": 8, "score": "sigmoid", "renorm": True,
         "scale": 2.5, "bias": True, "groups": 8, "top_groups": 4, "group_best": 2, "masked": 3, "padded": 37, "train": False},
        # A training step: forward, sorting, and the gradient.
        {"name": "route train", "kind": "route", "dtype": "fp32", "T": 16384, "E": 256, "k": 8, "score": "softmax", "renorm": False,
         "scale": 1.0, "bias": True, "groups": 1, "top_groups": 1, "group_best": 1, "masked": 0, "padded": 0, "train": True},
        # 8 tokens' rows to two experts each, and back: latency.
        {"name": "move decode", "kind": "move", "dtype": "bf16", "T": 8, "E": 32, "k": 2, "H": 2048, "missing": 0, "train": False},
        # A training step's tokens, forward and backward: bandwidth.
        {"name": "move train", "kind": "move", "dtype": "bf16", "T": 8192, "E": 64, "k": 4, "H": 4096, "missing": 100, "train": True},
        # Activations of 7 tokens, to two experts each.
        {"name": "quant tokens", "kind": "quant", "dtype": "fp16", "T": 7, "E": 16, "k": 2, "H": 2048, "missing": 0},
        # The activations of a long batch, dispatched in 8 bits.
        {"name": "quant batch", "kind": "quant", "dtype": "bf16", "T": 8192, "E": 32, "k": 4, "H": 4096, "missing": 0},
        # The weights of 8 experts, for the product and (transposed) for the gradient of its input.
        {"name": "quant weights", "kind": "quant", "dtype": "bf16", "E": 8, "N": 8192, "K": 4096, "weights": True},
        # One decoding step of 8 tokens with two experts each: 12 of 32 experts have one or two rows.
        {"name": "fp8 decode", "kind": "product", "dtype": "bf16", "T": 16, "E": 32, "active": 12, "N": 2816, "K": 2048, "act": "gelu",
         "grad": False, "preact": False, "from16": True},
        # A prompt's rows through a dense 4096 -> 14336 projection.
        {"name": "fp8 prompt", "kind": "product", "dtype": "bf16", "T": 8192, "E": 0, "active": 0, "N": 14336, "K": 4096, "act": "gelu",
         "grad": False, "preact": False, "from16": False},
        # A training step's up projection with the pre-activations kept: about 2048 rows for each of 8 experts.
        {"name": "fp8 train", "kind": "product", "dtype": "bf16", "T": 16384, "E": 8, "active": 8, "N": 8192, "K": 4096, "act": "gelu",
         "grad": False, "preact": True, "from16": False},
        # Fine-tuning on a short batch: the input's gradient through tanh-GELU, ragged, one expert empty.
        {"name": "fp8 dgrad", "kind": "product", "dtype": "fp16", "T": 2001, "E": 16, "active": 15, "N": 2048, "K": 1408,
         "act": "gelu_tanh", "grad": True, "preact": False, "from16": True},
    ]


def _spread(rng, low, high, step=1):
    """A multiple of step, evenly over the logarithm of [low, high]."""
    v = math.exp(rng.uniform(math.log(low), math.log(high)))
    return max(low, int(v) // step * step)


def draw(rng):
    kind = rng.choice(["route", "route", "move", "quant", "product", "product", "product"])
    if kind == "route":
        E = rng.choice([8, 16, 24, 32, 60, 64, 128, 160, 256, 384, 512])
        groups = rng.choice([1, 1, 2, 4, 8])
        if E % groups or E // groups < 2:
            groups = 1
        top = rng.randint(1, groups)
        room = E // groups * top
        T = _spread(rng, 1, 16384 if E <= 256 else 8192)
        return {"kind": kind, "dtype": rng.choice(["fp32", "fp32", "bf16", "fp16"]), "T": T, "E": E, "k": rng.randint(1, min(10, room)),
                "score": rng.choice(["softmax", "sigmoid"]), "renorm": rng.random() < 0.5, "scale": rng.choice([1.0, 2.5]),
                "bias": rng.random() < 0.5, "groups": groups, "top_groups": top, "group_best": rng.choice([1, 2]),
                "masked": rng.choice([0, 0, E // 5]), "padded": rng.choice([0, T // 9]), "train": rng.random() < 0.5}
    dtype = rng.choice(["bf16", "fp16"])
    if kind == "quant" and rng.random() < 0.4:
        N, K = _spread(rng, 64, 8192, 16), _spread(rng, 64, 8192, 16)
        return {"kind": kind, "dtype": dtype, "E": rng.randint(1, max(1, min(16, 268_000_000 // (N * K)))), "N": N, "K": K, "weights": True}
    if kind in ("move", "quant"):
        E, k = rng.choice([8, 16, 32, 64, 128]), rng.randint(1, 8)
        H = _spread(rng, 128, 8192, 16 if kind == "quant" else 8)
        T = _spread(rng, 1, max(1, min(16384, 134_000_000 // (H * k))))
        c = {"kind": kind, "dtype": dtype, "T": T, "E": E, "k": k, "H": H, "missing": rng.choice([0, T // 7])}
        if kind == "move":
            c["train"] = rng.random() < 0.5
        return c
    T, E = _spread(rng, 1, 16384), rng.choice([0, 0, 1, 5, 8, 16, 32, 64])
    K = _spread(rng, 256, 4096, 16)
    N = _spread(rng, 256, min(8192, 268_000_000 // (K * max(E, 1))), 8)
    grad = rng.random() < 0.35
    return {"kind": kind, "dtype": dtype, "T": T, "E": E, "active": min(T, rng.randint(max(1, E // 2), E)) if E else 0, "N": N, "K": K,
            "act": rng.choice(["none", "relu", "sigmoid", "gelu", "softplus", "gelu_tanh"]), "grad": grad,
            "preact": not grad and rng.random() < 0.5, "from16": rng.random() < 0.5}


def work(case):
    c = case
    if c["kind"] == "route":
        T, E, k = c["T"], c["E"], c["k"]
        size = 4 if c["dtype"] == "fp32" else 2
        n = size * T * E + 12 * T * k + 4 * E
        if c["train"]:   # the logits are in hand; the gradient of the weights in, that of the logits out
            n += size * T * E + 4 * T * k
        return {"bytes": n, "flops": (8 if c["train"] else 4) * T * E}
    if c["kind"] == "move":
        T, H, R = c["T"], c["H"], (c["T"] - c["missing"]) * c["k"]
        forward = 2 * H * (2 * T + 2 * R) + 4 * c["T"] * c["k"] * 3
        if not c["train"]:
            return {"bytes": forward, "flops": 2 * R * H}
        # dispatch and its gradient, combine, and its two gradients
        return {"bytes": 2 * H * (4 * T + 5 * R) + 4 * c["T"] * c["k"] * 6, "flops": 6 * R * H}
    if c["kind"] == "quant":
        if c.get("weights"):
            n = c["E"] * c["N"] * c["K"]
            return {"bytes": 2 * n + 2 * n + 4 * n, "flops": 6 * n}   # both orders, and both back
        T, H, R = c["T"], c["H"], (c["T"] - c["missing"]) * c["k"]
        return {"bytes": 2 * T * H + (R * H + R * H // 32) + 2 * R * H, "flops": 4 * T * H + R * H}
    T, N, K = c["T"], c["N"], c["K"]
    groups = c["active"] if c["E"] else 1
    a = 2 * T * K if c["from16"] else T * K * 33 // 32
    outs = 2 if c["preact"] or (c["grad"] and c["act"] != "none") else 1
    bias = 0 if c["grad"] else 2 * N
    return {"bytes": a + groups * (N * K + bias) + 2 * T * N * outs, "flops": 2 * T * N * K}


# --------------------------------------------------------------- inputs ----

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, shape, dtype, std=1.0):
    """Normal values, drawn in pieces so that no 32-bit copy of a large tensor is held."""
    out = torch.empty(shape, dtype=dtype, device="cuda")
    for piece in out.view(-1).split(1 << 26):
        piece.copy_(torch.randn(piece.shape, generator=g, device="cuda").mul_(std))
    return out


def _sizes(seed, rows, experts, active):
    """Rows of each expert: `active` of them have some, in uneven shares, the others none."""
    g = torch.Generator().manual_seed(seed)
    share = torch.rand(active, generator=g) + 0.25
    extra = torch.multinomial(share, rows - active, replacement=True, generator=g) if rows > active else torch.empty(0, dtype=torch.int64)
    sizes = torch.zeros(experts, dtype=torch.int64)
    sizes[torch.randperm(experts, generator=g)[:active]] = torch.bincount(extra, minlength=active) + 1
    return sizes


def _sorted_rows(indices, E):
    """(offsets [E + 1], rows [T, k]) of the slots' experts: a stable sort."""
    flat = indices.reshape(-1).long()
    key = torch.where(flat < 0, E, flat)
    order = torch.sort(key, stable=True).indices
    rows = torch.empty_like(flat)
    rows[order] = torch.arange(flat.numel(), device=flat.device)
    offsets = torch.zeros(E + 1, dtype=torch.int64, device=flat.device)
    offsets[1:] = (key[:, None] == torch.arange(E, device=flat.device)).sum(0).cumsum(0)
    rows = torch.where(flat < 0, -1, rows)
    return offsets.to(torch.int32), rows.view(indices.shape).to(torch.int32)


def _pieces(n, row_values):
    """Ranges of rows of about 2^25 values."""
    step = max(1, (1 << 25) // max(1, row_values))
    return [(i, min(n, i + step)) for i in range(0, n, step)]


def _row_blocks(x):
    """x [R, K] as [R, blocks, 128], the last block filled up with zeros."""
    R, K = x.shape
    return torch.nn.functional.pad(x, (0, -K % 128)).unflatten(1, (-1, 128))


def _tile_blocks(w):
    """w [N, K] as [N blocks, 128, K blocks, 128], filled up with zeros."""
    N, K = w.shape
    return torch.nn.functional.pad(w, (0, -K % 128, 0, -N % 128)).unflatten(0, (-1, 128)).unflatten(2, (-1, 128))


def _scaled(blocks, dims):
    """(8-bit values, fp32 scales) of blocks whose maximum is taken over dims: the scale is max / 448, and the
    value nearest to 448 x / max (in 64 bits, as many x lie on a border)."""
    big = blocks.abs().amax(dims, keepdim=True).double()
    tiny = 448 * 2.0 ** -126
    q = torch.where(big < tiny, blocks.double() * 2.0 ** 126, blocks.double() * 448 / big.clamp(min=tiny))
    return q.float().to(F8), (big / 448).clamp(min=2.0 ** -126).float()


def _quantised_rows(x):
    """Codes [R, K] and scale planes [K blocks, R]."""
    R, K = x.shape
    codes = torch.empty(R, K, dtype=F8, device=x.device)
    scales = torch.empty(-(-K // 128), R, dtype=torch.float32, device=x.device)
    for i, j in _pieces(R, K):
        q, s = _scaled(_row_blocks(x[i:j]), 2)
        codes[i:j] = q.flatten(1)[:, :K]
        scales[:, i:j] = s[:, :, 0].T
    return codes, scales


def _quantised_weights(w):
    """Codes [E, N, K] and scales [E, N blocks, K blocks]."""
    E, N, K = w.shape
    codes, scales = [], []
    for e in range(E):
        q, s = _scaled(_tile_blocks(w[e]), (1, 3))
        codes.append(q.flatten(2).flatten(0, 1)[:N, :K])
        scales.append(s[:, 0, :, 0])
    return torch.stack(codes), torch.stack(scales)


def prepare(case, seed):
    c = case
    g, s = _generator(seed), {"case": c}
    dt = DTYPES[c["dtype"]]
    if c["kind"] == "route":
        T, E, k = c["T"], c["E"], c["k"]
        x = _normal(g, (T, E), torch.float32, 1.5)
        if c["masked"]:
            x[:, torch.randperm(E, generator=g, device="cuda")[:c["masked"]]] = -math.inf
        if c["padded"]:
            x[T - c["padded"]:] = -math.inf
        s["logits"] = x.to(dt)
        s["bias"] = _normal(g, (E,), torch.float32, 0.1) if c["bias"] else None
        s["indices"] = torch.empty(T, k, dtype=torch.int32, device="cuda")
        s["weights"] = torch.empty(T, k, device="cuda")
        s["offsets"] = torch.empty(E + 1, dtype=torch.int32, device="cuda")
        s["rows"] = torch.empty(T, k, dtype=torch.int32, device="cuda")
        s["workspace"] = torch.empty(4 << 20, dtype=torch.uint8, device="cuda")
        if c["train"]:
            s["dweights"] = _normal(g, (T, k), torch.float32)
            s["dlogits"] = torch.empty(T, E, dtype=dt, device="cuda")
        return s
    if c["kind"] == "move" or (c["kind"] == "quant" and not c.get("weights")):
        T, E, k, H = c["T"], c["E"], c["k"], c["H"]
        indices = torch.rand(T, E, generator=g, device="cuda").topk(k, 1).indices.to(torch.int32)
        if c["missing"]:
            indices[torch.randperm(T, generator=g, device="cuda")[:c["missing"]]] = -1
        s["offsets"], s["rows"] = _sorted_rows(indices, E)
        s["x"] = _normal(g, (T, H), dt)
        if c["kind"] == "quant":
            s["x"] *= torch.exp2(torch.randint(-6, 4, (T, 1), generator=g, device="cuda")).to(dt)
            s["codes"] = torch.zeros(T * k, H, dtype=torch.uint8, device="cuda").view(F8)
            s["scales"] = torch.zeros(-(-H // 128), T * k, device="cuda")
            s["y"] = torch.empty(T * k, H, dtype=dt, device="cuda")
            return s
        s["y"] = _normal(g, (T * k, H), dt)
        s["weights"] = torch.rand(T, k, generator=g, device="cuda") + 0.1
        s["xs"] = torch.zeros(T * k, H, dtype=dt, device="cuda")
        s["out"] = torch.empty(T, H, dtype=dt, device="cuda")
        if c["train"]:
            s["dout"] = _normal(g, (T, H), dt)
            s["dxs"] = _normal(g, (T * k, H), dt)
            s["dy"] = torch.zeros(T * k, H, dtype=dt, device="cuda")
            s["dweights"] = torch.empty(T, k, device="cuda")
            s["dx"] = torch.empty(T, H, dtype=dt, device="cuda")
        return s
    if c["kind"] == "quant":
        E, N, K = c["E"], c["N"], c["K"]
        s["w"] = _normal(g, (E, N, K), dt, K ** -0.5)
        for name, a, b in (("", N, K), ("_t", K, N)):
            s["codes" + name] = torch.empty(E, a, b, dtype=F8, device="cuda")
            s["scales" + name] = torch.empty(E, -(-a // 128), -(-b // 128), device="cuda")
            s["y" + name] = torch.empty(E, a, b, dtype=dt, device="cuda")
        return s
    T, N, K, E = c["T"], c["N"], c["K"], c["E"]
    # One workspace for all of a program's products, for splitting a long sum.
    s["workspace"] = torch.empty(32 << 20, dtype=torch.uint8, device="cuda")
    s["a"] = _normal(g, (T, K), dt)
    w = _normal(g, (max(E, 1), N, K), dt, K ** -0.5)
    s["w_codes"], s["w_scales"] = _quantised_weights(w)
    if not E:
        s["w_codes"], s["w_scales"] = s["w_codes"][0], s["w_scales"][0]
    if c["from16"]:
        s["codes"] = torch.empty(T, K, dtype=F8, device="cuda")
        s["scales"] = torch.empty(-(-K // 128), T, device="cuda")
    else:
        s["codes"], s["scales"] = _quantised_rows(s["a"])
    if E:
        s["sizes"] = _sizes(seed, T, E, c["active"]).tolist()
        s["offsets"] = torch.tensor([0] + s["sizes"], device="cuda").cumsum(0).to(torch.int32)
    s["bias"] = None if c["grad"] else _normal(g, (E, N) if E else (N,), dt, 0.14)
    s["z"] = None
    if c["preact"]:
        s["z"] = torch.empty(T, N, dtype=dt, device="cuda")
    elif c["grad"] and c["act"] != "none":
        s["z"] = _normal(g, (T, N), dt)
    s["c"] = torch.empty(T, N, dtype=dt, device="cuda")
    return s


# ----------------------------------------------------------- plain forms ----

def _route(c, x, bias):
    """(indices, weights fp32): the choice in 64 bits, as values lie next to a border."""
    T, E = x.shape
    x = x.double()
    masked = x == -math.inf
    if c["score"] == "softmax":
        m = x.amax(1, keepdim=True).clamp(min=-1e300)
        p = torch.exp(x - m)
        score = p / p.sum(1, keepdim=True).clamp(min=1.0)     # the largest is e^0 = 1
    else:
        score = 1 / (1 + torch.exp(-x))
    value = score if bias is None else score + bias.double()
    value = torch.where(masked, -math.inf, value)
    G, best = c["groups"], c["group_best"]
    if G > 1:
        top = value.view(T, G, E // G).sort(dim=2, descending=True).values[:, :, :best]
        total = torch.where(top[:, :, :1] == -math.inf, -math.inf, torch.where(top == -math.inf, 0.0, top).sum(2, keepdim=True))[:, :, 0]
        order = total.sort(dim=1, descending=True, stable=True).indices
        keep = torch.zeros(T, G, dtype=torch.bool, device=x.device).scatter_(1, order[:, :c["top_groups"]], True)
        value = torch.where(keep.repeat_interleave(E // G, 1), value, -math.inf)
    v, indices = value.sort(dim=1, descending=True, stable=True)
    v, indices = v[:, :c["k"]], indices[:, :c["k"]]
    w = torch.where(v == -math.inf, 0.0, score.gather(1, indices))
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
    return torch.where(v == -math.inf, -1, indices).to(torch.int32), (w * c["scale"]).float()


def _route_grad(c, x, indices, dweights):
    """The logits' gradient from the weights' (the choice has none)."""
    x = x.float()
    valid = indices >= 0
    at = indices.clamp(min=0).long()
    g = torch.where(valid, dweights, 0.0) * c["scale"]
    if c["score"] == "softmax":
        m = x.amax(1, keepdim=True).clamp(min=-3e38)
        p = torch.exp(x - m)
        p = p / p.sum(1, keepdim=True).clamp(min=1.0)
    else:
        p = 1 / (1 + torch.exp(-x))
    s = torch.where(valid, p.gather(1, at), 0.0)
    if c["renorm"]:
        total = s.sum(1, keepdim=True).clamp(min=1e-30)
        q = s / total
        ds = (g - (q * g).sum(1, keepdim=True)) / total
    else:
        ds = g
    dp = torch.zeros_like(x).scatter_add_(1, at, torch.where(valid, ds, 0.0))
    if c["score"] == "softmax":
        dx = p * (dp - (dp * p).sum(1, keepdim=True))
    else:
        dx = dp * p * (1 - p)
    return dx


def _act(name, z):
    if name == "relu":
        return z.clamp(min=0)
    if name == "sigmoid":
        return 1 / (1 + torch.exp(-z))
    if name == "gelu":
        return z * (0.5 * torch.special.erfc(z * -math.sqrt(0.5)))
    if name == "softplus":
        return z.clamp(min=0) + torch.log1p(torch.exp(-z.abs()))
    if name == "gelu_tanh":
        return z / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _act_slope(name, z):
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "sigmoid":
        s = 1 / (1 + torch.exp(-z))
        return s * (1 - s)
    if name == "gelu":
        return 0.5 * torch.special.erfc(z * -math.sqrt(0.5)) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if name == "softplus":
        return 1 / (1 + torch.exp(-z))
    r = math.sqrt(2 / math.pi)
    s = 1 / (1 + torch.exp(-2 * r * (z + 0.044715 * z * z * z)))
    return s + z * s * (1 - s) * 2 * r * (1 + 3 * 0.044715 * z * z)


def _row_values(codes, scales):
    """32-bit values of codes [R, K] and scale planes [K blocks, R]."""
    return codes.float() * scales.T.repeat_interleave(128, 1)[:, :codes.shape[1]]


def _weight_values(codes, scales):
    """32-bit values of codes [N, K] and scales [N blocks, K blocks]."""
    N, K = codes.shape
    return codes.float() * scales.repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]


def _gathered(src, rows, weights=None):
    """sum over j of weights[t, j] src[rows[t, j]] in 32 bits, rows of -1 left out."""
    out = torch.empty(rows.shape[0], src.shape[1], device=src.device)
    for i, j in _pieces(rows.shape[0], rows.shape[1] * src.shape[1]):
        r = rows[i:j]
        v = src[r.clamp(min=0).long()].float()
        if weights is not None:
            v = v * weights[i:j, :, None]
        out[i:j] = torch.where(r[:, :, None] >= 0, v, 0.0).sum(1)
    return out


def _moved(src, rows, out, weights=None):
    """out[rows[t, j]] = (weights[t, j]) src[t]; other rows of out stay."""
    slots = torch.nonzero(rows.reshape(-1) >= 0)[:, 0]
    to, k = rows.reshape(-1)[slots].long(), rows.shape[1]
    for i, j in _pieces(slots.numel(), src.shape[1]):
        v = src[slots[i:j] // k].float()
        if weights is not None:
            v = v * weights.reshape(-1)[slots[i:j], None]
        out[to[i:j]] = v.to(out.dtype)
    return out


def _plain(s):
    c = s["case"]
    dt = DTYPES[c["dtype"]]
    if c["kind"] == "route":
        indices, weights = _route(c, s["logits"], s["bias"])
        offsets, rows = _sorted_rows(indices, c["E"])
        if not c["train"]:
            return indices, weights, offsets, rows
        return indices, weights, offsets, rows, _route_grad(c, s["logits"], indices, s["dweights"]).to(dt)
    if c["kind"] == "move":
        xs = _moved(s["x"], s["rows"], s["xs"])
        out = _gathered(s["y"], s["rows"], s["weights"]).to(dt)
        if not c["train"]:
            return xs, out
        dy = _moved(s["dout"], s["rows"], s["dy"], s["weights"])
        dw = torch.empty_like(s["weights"])
        for i, j in _pieces(c["T"], c["k"] * c["H"]):
            r = s["rows"][i:j]
            d = (s["y"][r.clamp(min=0).long()].float() * s["dout"][i:j, None].float()).sum(2)
            dw[i:j] = torch.where(r >= 0, d, 0.0)
        return xs, out, dy, dw, _gathered(s["dxs"], s["rows"]).to(dt)
    if c["kind"] == "quant" and c.get("weights"):
        codes, scales = _quantised_weights(s["w"])
        for e in range(c["E"]):
            v = _weight_values(codes[e], scales[e]).to(dt)
            s["y"][e], s["y_t"][e] = v, v.T
        return s["y"], s["y_t"]
    if c["kind"] == "quant":
        codes, scales = _quantised_rows(s["x"])
        values = torch.cat([_row_values(codes[i:j], scales[:, i:j]).to(dt) for i, j in _pieces(c["T"], c["H"])])
        s["y"].zero_()
        return _moved(values, s["rows"], s["y"])
    codes, scales = _quantised_rows(s["a"]) if c["from16"] else (s["codes"], s["scales"])
    a = _row_values(codes, scales)
    if not c["E"]:
        z = a @ _weight_values(s["w_codes"], s["w_scales"]).T
        if s["bias"] is not None:
            z = z + s["bias"].float()
    else:
        parts = []
        for e, p in enumerate(a.split(s["sizes"])):
            if len(p):
                z = p @ _weight_values(s["w_codes"][e], s["w_scales"][e]).T
                parts.append(z if s["bias"] is None else z + s["bias"][e].float())
        z = torch.cat(parts)
    if c["grad"]:
        return (z if s["z"] is None else z * _act_slope(c["act"], s["z"].float())).to(dt)
    return (_act(c["act"], z).to(dt), z.to(dt)) if c["preact"] else _act(c["act"], z).to(dt)


# ------------------------------------------------------------------ run ----

def run(state):
    s = state
    if not own:
        return _plain(s)
    import tiled_dense_gemm_bias_amd as gba
    c = s["case"]
    if c["kind"] == "route":
        gba.moe_route(s["logits"], s["indices"], s["weights"], s["bias"], offsets=s["offsets"], rows=s["rows"],
                      workspace=s["workspace"], score=c["score"], renormalize=c["renorm"], scale=c["scale"], groups=c["groups"],
                      top_groups=c["top_groups"], group_best=c["group_best"])
        if not c["train"]:
            return s["indices"], s["weights"], s["offsets"], s["rows"]
        gba.moe_route_grad(s["logits"], s["indices"], s["dweights"], s["dlogits"], score=c["score"], renormalize=c["renorm"],
                           scale=c["scale"])
        return s["indices"], s["weights"], s["offsets"], s["rows"], s["dlogits"]
    if c["kind"] == "move":
        gba.moe_dispatch(s["x"], s["rows"], s["xs"])
        gba.moe_combine(s["y"], s["rows"], s["weights"], s["out"])
        if not c["train"]:
            return s["xs"], s["out"]
        gba.moe_combine_grad(s["dout"], s["y"], s["rows"], s["weights"], s["dy"], s["dweights"])
        gba.moe_combine(s["dxs"], s["rows"], None, s["dx"])
        return s["xs"], s["out"], s["dy"], s["dweights"], s["dx"]
    if c["kind"] == "quant" and c.get("weights"):
        gba.fp8_quantize_weights(s["w"], s["codes"], s["scales"], s["codes_t"], s["scales_t"])
        gba.fp8_dequantize_weights(s["codes"], s["scales"], s["y"])
        gba.fp8_dequantize_weights(s["codes_t"], s["scales_t"], s["y_t"])
        return s["y"], s["y_t"]
    if c["kind"] == "quant":
        gba.fp8_quantize(s["x"], s["codes"], s["scales"], rows=s["rows"])
        return gba.fp8_dequantize(s["codes"], s["scales"], s["y"])
    if c["from16"]:
        gba.fp8_quantize(s["a"], s["codes"], s["scales"])
    if c["grad"] and c["E"]:
        return gba.grouped_gemm_act_grad_fp8_block(s["codes"], s["scales"], s["offsets"], s["w_codes"], s["w_scales"], s["z"], s["c"],
                                                   c["act"], workspace=s["workspace"])
    if c["grad"]:
        return gba.gemm_act_grad_fp8_block(s["codes"], s["scales"], s["w_codes"], s["w_scales"], s["z"], s["c"], c["act"],
                                           workspace=s["workspace"])
    if c["E"]:
        gba.grouped_gemm_bias_act_fp8_block(s["codes"], s["scales"], s["offsets"], s["w_codes"], s["w_scales"], s["bias"], s["c"],
                                            c["act"], preact=s["z"], workspace=s["workspace"])
    else:
        gba.gemm_bias_act_fp8_block(s["codes"], s["scales"], s["w_codes"], s["w_scales"], s["bias"], s["c"], c["act"], preact=s["z"],
                                    workspace=s["workspace"])
    return (s["c"], s["z"]) if c["preact"] else s["c"]


# ---------------------------------------------------------------- exact ----

def _exact_act(name, z):
    return {"none": lambda: z, "relu": lambda: torch.maximum(z, torch.zeros_like(z)), "sigmoid": lambda: torch.special.expit(z),
            "gelu": lambda: z * torch.special.ndtr(z), "softplus": lambda: torch.logaddexp(z, torch.zeros_like(z)),
            "gelu_tanh": lambda: 0.5 * z * (1 + torch.tanh((2 / math.pi) ** 0.5 * (z + 0.044715 * z ** 3)))}[name]()


def _exact_slope(name, z):
    """By differentiating the definition."""
    z = z.clone().requires_grad_(True)
    with torch.enable_grad():
        (slope,) = torch.autograd.grad(_exact_act(name, z).sum(), z)
    return slope


def _exact_e4m3(q):
    """The nearest multiple of the format's step at q (2^-9 below 2^-6), ties to the even one, at most 448."""
    exponent = torch.frexp(q)[1].long() - 1
    step = ((exponent.clamp(min=-6) - 3 + 1023) << 52).view(torch.float64)
    return (torch.round(q / step) * step).clamp(-448, 448)


def _exact_blocks(x, rows_a_block):
    """The values that x [R, K] has in 8 bits, by blocks of rows_a_block x 128."""
    R, K = x.shape
    up, wide = -(-R // rows_a_block) * rows_a_block, -(-K // 128) * 128
    full = torch.zeros(up, wide, dtype=torch.float64, device=x.device)
    full[:R, :K] = x.double()
    b = full.view(up // rows_a_block, rows_a_block, wide // 128, 128)
    top = b.abs().amax((1, 3), keepdim=True)
    unit = torch.maximum(top / 448, torch.full_like(top, 2.0 ** -126))
    q = torch.where(top / 448 < 2.0 ** -126, b * 2.0 ** 126, 448 * b / torch.where(top > 0, top, torch.ones_like(top)))
    return (_exact_e4m3(q) * unit.float().double()).reshape(up, wide)[:R, :K]


def _exact_route(c, s):
    x = s["logits"].double()
    T, E = x.shape
    k, G = c["k"], c["groups"]
    log_score = torch.log_softmax(x, 1) if c["score"] == "softmax" else -torch.logaddexp(torch.zeros_like(x), -x)
    log_score = torch.where(torch.isnan(log_score), -math.inf, log_score)
    if s["bias"] is None and (G == 1 or c["group_best"] == 1):
        value = x                                                # the scores' order
    else:
        value = torch.exp(log_score) + (0 if s["bias"] is None else s["bias"].double())
        value = value.masked_fill(x == -math.inf, -math.inf)
    if G > 1:
        by_group = value.reshape(T, G, -1)
        first = by_group.amax(2)
        total = first
        if c["group_best"] == 2:
            at = by_group.argmax(2, keepdim=True)
            second = by_group.scatter(2, at, -math.inf).amax(2)
            total = first + second.masked_fill(second == -math.inf, 0.0)
        # a group's place: how many are better, or as good and earlier
        earlier = torch.ones(G, G, dtype=torch.bool, device=x.device).tril(-1)
        better = (total[:, None, :] > total[:, :, None]) | ((total[:, None, :] == total[:, :, None]) & earlier)
        keep = better.sum(2) < c["top_groups"]
        value = value.reshape(T, G, -1).masked_fill(~keep[:, :, None], -math.inf).reshape(T, E)
    indices = torch.empty(T, k, dtype=torch.int64, device=x.device)
    number = torch.arange(E, device=x.device)
    for j in range(k):
        top = value.amax(1, keepdim=True)
        at = torch.where(value == top, number, E).amin(1, keepdim=True)
        indices[:, j:j + 1] = torch.where(top == -math.inf, -1, at)
        value = value.scatter(1, at, -math.inf)
    ls = log_score.gather(1, indices.clamp(min=0)).masked_fill(indices < 0, -math.inf)
    if c["renorm"]:
        ls = ls - torch.logsumexp(ls, 1, keepdim=True)
    weights = torch.where(indices < 0, 0.0, torch.exp(ls)) * c["scale"]
    flat = indices.reshape(-1)
    counts = torch.bincount(flat + 1, minlength=E + 1)[1:]
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    rows = torch.full_like(flat, -1)
    place = torch.argsort(flat, stable=True)[(flat < 0).sum():]
    rows[place] = torch.arange(place.numel(), device=x.device)
    out = [indices.to(torch.int32), weights, offsets.to(torch.int32), rows.view(T, k).to(torch.int32)]
    if c["train"]:
        leaf = s["logits"].double().requires_grad_(True)
        valid = indices >= 0
        with torch.enable_grad():
            used = valid.any(1)
            ls = torch.log_softmax(leaf[used], 1) if c["score"] == "softmax" else torch.nn.functional.logsigmoid(leaf[used])
            ls = ls.gather(1, indices[used].clamp(min=0)).masked_fill(~valid[used], -math.inf)
            if c["renorm"]:
                ls = torch.log_softmax(ls, 1)
            total = (torch.exp(ls) * s["dweights"][used].double() * c["scale"]).masked_fill(~valid[used], 0.0).sum()
            (grad,) = torch.autograd.grad(total, leaf)
        out.append(torch.nan_to_num(grad))
    return tuple(out)


def exact(case, seed):
    s, c = prepare(case, seed), case
    if c["kind"] == "route":
        return _exact_route(c, s)
    if c["kind"] == "quant" and c.get("weights"):
        w = torch.stack([_exact_blocks(m, 128) for m in s["w"]])
        return w, w.transpose(1, 2).contiguous()
    if c["kind"] in ("move", "quant"):
        T, k, H, rows = c["T"], c["k"], c["H"], s["rows"].long()

        def placed(of_token):
            """[T k, H] with of_token(j) in the rows of the slots (., j)."""
            out = torch.zeros(T * k, H, dtype=torch.float64, device="cuda")
            for j in range(k):
                there = rows[:, j] >= 0
                out[rows[there, j]] = of_token(j)[there]
            return out

        def taken(src, j):
            return torch.where(rows[:, j, None] >= 0, src[rows[:, j].clamp(min=0)].double(), 0.0)
        if c["kind"] == "quant":
            values = _exact_blocks(s["x"], 1)
            return placed(lambda j: values)
        x, w = s["x"].double(), s["weights"].double()
        xs = placed(lambda j: x)
        out = sum(taken(s["y"], j) * w[:, j, None] for j in range(k))
        if not c["train"]:
            return xs, out
        d = s["dout"].double()
        return (xs, out, placed(lambda j: d * w[:, j, None]), torch.stack([(taken(s["y"], j) * d).sum(1) for j in range(k)], 1),
                sum(taken(s["dxs"], j) for j in range(k)))
    E, N, K = c["E"], c["N"], c["K"]
    if c["from16"]:
        a = _exact_blocks(s["a"], 1)
    else:
        a = s["codes"].double() * s["scales"].T.double()[:, torch.arange(K, device="cuda") // 128]
    at_n, at_k = torch.arange(N, device="cuda") // 128, torch.arange(K, device="cuda") // 128
    begin, parts = 0, []
    for e, n in enumerate(s["sizes"] if E else [c["T"]]):
        if n:
            codes, scales, bias = (s["w_codes"], s["w_scales"], s["bias"])
            if E:
                codes, scales, bias = codes[e], scales[e], None if bias is None else bias[e]
            w = codes.double() * scales.double()[at_n][:, at_k]
            z = a[begin:begin + n] @ w.T.contiguous()
            parts.append(z if bias is None else z + bias.double())
        begin += n
    z = torch.cat(parts)
    if c["grad"]:
        return z if s["z"] is None else z * _exact_slope(c["act"], s["z"].double())
    return (_exact_act(c["act"], z), z) if c["preact"] else _exact_act(c["act"], z)
