"""Cases of the expert-grouped products and the microscaled 4-bit operators.

Five kinds of case, all on the GPU:

  fwd    c = act(a_e . w_e^T + bias_e) for the rows of each expert e, with the
         pre-activation beside it where the case trains;
  dgrad  da = (dc_e . w_e) * act'(z): the gradient of a product's input, through
         the activation that made that input;
  wgrad  dw_e = dc_e^T . a_e and db_e = the column sums of dc_e;
  quant  16-bit values to microscaled 4-bit floats (blocks of 32 along a row, one
         power-of-two scale each) and back;
  mx4    c = act(x . w^T + bias) with both operands in that format, dense or by
         expert; where the case says so the 16-bit activations are quantised first.

Rows are sorted by expert: those of expert e are offsets[e] .. offsets[e+1] - 1.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
CODE_VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


# ---------------------------------------------------------------- cases ----

def listed():
    return [
        # One decoding step of 8 tokens with two experts each: 12 of 32 experts have
        # one or two rows, and the pass is the reading of their weights.
        {"name": "fwd decode", "kind": "fwd", "dtype": "bf16", "T": 16, "E": 32, "active": 12, "N": 2816, "K": 2048,
         "act": "gelu", "preact": False},
        # A short prompt over 16 experts, ragged: some tens of rows each, one expert empty.
        {"name": "fwd prompt", "kind": "fwd", "dtype": "fp16", "T": 999, "E": 16, "active": 15, "N": 1408, "K": 2048,
         "act": "gelu_tanh", "preact": False},
        # A training step's up projection: about 2048 rows for each of 8 experts; the
        # pre-activation is kept for the backward pass.
        {"name": "fwd train", "kind": "fwd", "dtype": "bf16", "T": 16384, "E": 8, "active": 8, "N": 8192, "K": 4096,
         "act": "gelu", "preact": True},
        # Fine-tuning on a short batch: the input's gradient through tanh-GELU.
        {"name": "dgrad small", "kind": "dgrad", "dtype": "fp16", "T": 515, "E": 16, "active": 13, "N": 2048, "K": 1408,
         "act": "gelu_tanh"},
        # The same training step backwards: the down projection's input gradient.
        {"name": "dgrad train", "kind": "dgrad", "dtype": "bf16", "T": 16384, "E": 8, "active": 8, "N": 4096, "K": 8192,
         "act": "gelu"},
        # Weight gradients of the short batch: few rows, the writing of all weights' gradients.
        {"name": "wgrad small", "kind": "wgrad", "dtype": "fp16", "T": 515, "E": 16, "active": 13, "N": 1408, "K": 2048},
        # Weight gradients of the training step.
        {"name": "wgrad train", "kind": "wgrad", "dtype": "bf16", "T": 16384, "E": 8, "active": 8, "N": 8192, "K": 4096},
        # Activations of 7 tokens: latency.
        {"name": "quant tokens", "kind": "quant", "dtype": "fp16", "M": 7, "K": 2048},
        # A weight matrix or the activations of a long batch: bandwidth.
        {"name": "quant matrix", "kind": "quant", "dtype": "bf16", "M": 16384, "K": 8192},
        # A decoding step of 5 sequences through a 4096 -> 14336 projection in 4 bits.
        {"name": "mx4 decode", "kind": "mx4", "dtype": "bf16", "M": 5, "E": 0, "active": 0, "N": 14336, "K": 4096,
         "act": "gelu", "from16": True},
        # A prompt's rows through the same projection, already in 4 bits.
        {"name": "mx4 prompt", "kind": "mx4", "dtype": "bf16", "M": 8192, "E": 0, "active": 0, "N": 14336, "K": 4096,
         "act": "gelu", "from16": False},
        # 4-bit experts serving a batch of prompts: 16 experts, ragged, two empty.
        {"name": "mx4 experts", "kind": "mx4", "dtype": "fp16", "M": 2001, "E": 16, "active": 14, "N": 4096, "K": 2048,
         "act": "relu", "from16": True},
    ]


def _spread(rng, low, high, step):
    """A multiple of step, evenly over the logarithm of [low, high]."""
    v = math.exp(rng.uniform(math.log(low), math.log(high)))
    return max(low, int(v) // step * step)


def draw(rng):
    kind = rng.choice(["fwd", "fwd", "dgrad", "wgrad", "quant", "mx4", "mx4"])
    dtype = rng.choice(sorted(DTYPES))
    act = rng.choice(["none", "relu", "sigmoid", "gelu", "softplus", "gelu_tanh"])
    if kind == "quant":
        return {"kind": kind, "dtype": dtype, "M": _spread(rng, 1, 16384, 1), "K": _spread(rng, 256, 8192, 32)}
    if kind == "mx4":
        M, K = _spread(rng, 1, 8192, 1), _spread(rng, 256, 8192, 32)
        E = rng.choice([0, 0, 1, 4, 7, 16, 32])
        N = _spread(rng, 256, min(14336, 234_000_000 // (K * max(E, 1))), 8)
        return {"kind": kind, "dtype": dtype, "M": M, "E": E, "active": min(M, rng.randint(max(1, E // 2), E)) if E else 0,
                "N": N, "K": K, "act": act, "from16": rng.random() < 0.5}
    T, E = _spread(rng, 1, 16384, 1), rng.choice([1, 2, 5, 8, 16, 32, 64])
    K = _spread(rng, 256, 4096, 8)
    N = _spread(rng, 256, min(8192, 268_000_000 // (K * E)), 8)
    c = {"kind": kind, "dtype": dtype, "T": T, "E": E, "active": min(T, rng.randint(max(1, E // 2), E)), "N": N, "K": K}
    if kind == "dgrad":
        c["N"], c["K"] = K, N
    if kind != "wgrad":
        c["act"] = act
    if kind == "fwd":
        c["preact"] = rng.random() < 0.5
    return c


def work(case):
    c = case
    if c["kind"] == "quant":
        n = c["M"] * c["K"]
        return {"bytes": 4 * n, "flops": 4 * n}
    if c["kind"] == "mx4":
        M, N, K = c["M"], c["N"], c["K"]
        groups = c["active"] if c["E"] else 1
        x = 2 * M * K if c["from16"] else M * K * 17 // 32
        return {"bytes": x + groups * (N * K * 17 // 32 + 2 * N) + 2 * M * N, "flops": 2 * M * N * K}
    T, N, K = c["T"], c["N"], c["K"]
    flops = 2 * T * N * K
    if c["kind"] == "fwd":
        return {"bytes": 2 * (T * K + c["active"] * N * (K + 1) + T * N * (2 if c["preact"] else 1)), "flops": flops}
    if c["kind"] == "dgrad":
        return {"bytes": 2 * (T * N + c["active"] * N * K + T * K * (1 if c["act"] == "none" else 2)), "flops": flops}
    return {"bytes": 2 * (T * (N + K) + c["E"] * N * (K + 1)), "flops": flops}


# --------------------------------------------------------------- inputs ----

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, shape, dtype, std=1.0):
    """Normal values in a 16-bit type, drawn in pieces so that no 32-bit copy of a large tensor is held."""
    out = torch.empty(shape, dtype=dtype, device="cuda")
    for piece in out.view(-1).split(1 << 26):
        piece.copy_(torch.randn(piece.shape, generator=g, device="cuda").mul_(std))
    return out


def _sizes(seed, rows, experts, active):
    """Rows of each expert: `active` of them have some, in uneven shares, the others none."""
    g = torch.Generator().manual_seed(seed)
    share = torch.rand(active, generator=g) + 0.25
    extra = torch.multinomial(share, rows - active, replacement=True, generator=g) if rows > active else torch.empty(0, dtype=torch.int64)
    counts = torch.bincount(extra, minlength=active) + 1
    sizes = torch.zeros(experts, dtype=torch.int64)
    sizes[torch.randperm(experts, generator=g)[:active]] = counts
    return sizes


def _offsets(sizes):
    return torch.cat([torch.zeros(1, dtype=torch.int64), sizes.cumsum(0)]).to(torch.int32).cuda()


def _block_scales(x):
    """The power of two of each block of 32 values, as its exponent: that of the block's
    largest magnitude less 2 (the largest 4-bit value is 1.5 * 2^2)."""
    big = x.abs().amax(-1, keepdim=True)
    exponent = torch.frexp(big).exponent - 3          # frexp's mantissa lies in [0.5, 1)
    return torch.where(big > 0, exponent, -127).clamp(-127, 127)


def _to_codes(x):
    """Codes [rows, K] (one 4-bit code a byte) and exponents [rows, K / 32] of 16-bit values
    [rows, K]: nearest code, ties to the even one, magnitudes over 6 to 6."""
    blocks = x.float().unflatten(-1, (-1, 32))
    e = _block_scales(blocks)
    y = blocks * _power_of_two(-e)
    m = y.abs()
    code = ((m > 0.25).int() + (m >= 0.75).int() + (m > 1.25).int() + (m >= 1.75).int() + (m > 2.5).int() + (m >= 3.5).int() + (m > 5.0).int())
    code += 8 * (torch.signbit(y)).int()
    return code.flatten(-2).to(torch.uint8), e.squeeze(-1)


def _power_of_two(e):
    """2^e in 32 bits for -128 < e < 128, from its bits."""
    e = e.to(torch.int32)
    normal = (e + 127).clamp(min=1) << 23
    return torch.where(e < -126, 1 << 22, normal).to(torch.int32).view(torch.float32)


def _packed(codes, exponents):
    """The stored form: two codes a byte, the even one low; scale bytes (exponent + 127) in
    planes of 4 blocks, [ceil(K / 128), rows, 4], blocks past K zero."""
    rows, blocks = exponents.shape
    planes = -(-blocks // 4)
    s = torch.zeros(rows, planes * 4, dtype=torch.uint8, device=codes.device)
    s[:, :blocks] = (exponents + 127).to(torch.uint8)
    return codes[:, 0::2] | (codes[:, 1::2] << 4), s.view(rows, planes, 4).transpose(0, 1).contiguous()


def _quantised(x):
    """_packed(_to_codes(x)) in pieces of rows."""
    pieces = [_packed(*_to_codes(p)) for p in x.split(max(1, (1 << 25) // x.shape[1]))]
    return torch.cat([p[0] for p in pieces]), torch.cat([p[1] for p in pieces], 1)


def prepare(case, seed):
    c = case
    g, dt = _generator(seed), DTYPES[c["dtype"]]
    s = {"case": c}
    if c["kind"] != "quant":
        # One workspace for all of a program's products, for splitting a long sum.
        s["workspace"] = torch.empty(32 << 20, dtype=torch.uint8, device="cuda")
    if c["kind"] == "quant":
        M, K = c["M"], c["K"]
        # Rows of different magnitude, as activations have.
        s["x"] = _normal(g, (M, K), dt) * torch.exp2(torch.randint(-6, 4, (M, 1), generator=g, device="cuda")).to(dt)
        s["codes"] = torch.empty(M, K // 2, dtype=torch.uint8, device="cuda")
        s["scales"] = torch.empty(-(-K // 128), M, 4, dtype=torch.uint8, device="cuda")
        s["y"] = torch.empty(M, K, dtype=dt, device="cuda")
        return s
    if c["kind"] == "mx4":
        M, N, K, E = c["M"], c["N"], c["K"], c["E"]
        s["x"] = _normal(g, (M, K), dt)
        w = _normal(g, (max(E, 1) * N, K), dt, K ** -0.5)
        s["w_codes"], s["w_scales"] = _quantised(w)
        s["bias"] = _normal(g, (E, N) if E else (N,), dt, 0.14)
        if c["from16"]:
            s["codes"] = torch.empty(M, K // 2, dtype=torch.uint8, device="cuda")
            s["scales"] = torch.empty(-(-K // 128), M, 4, dtype=torch.uint8, device="cuda")
        else:
            s["codes"], s["scales"] = _quantised(s["x"])
        if E:
            sizes = _sizes(seed, M, E, c["active"])
            s["sizes"], s["offsets"] = sizes.tolist(), _offsets(sizes)
            s["w_codes"] = s["w_codes"].view(E, N, K // 2)
        s["c"] = torch.empty(M, N, dtype=dt, device="cuda")
        return s
    T, N, K, E = c["T"], c["N"], c["K"], c["E"]
    sizes = _sizes(seed, T, E, c["active"])
    s["sizes"], s["offsets"] = sizes.tolist(), _offsets(sizes)
    if c["kind"] == "fwd":
        s["a"] = _normal(g, (T, K), dt)
        s["w"] = _normal(g, (E, N, K), dt, K ** -0.5)
        s["bias"] = _normal(g, (E, N), dt, 0.14)
        s["c"] = torch.empty(T, N, dtype=dt, device="cuda")
        s["z"] = torch.empty(T, N, dtype=dt, device="cuda") if c["preact"] else None
    elif c["kind"] == "dgrad":
        s["dc"] = _normal(g, (T, N), dt)
        s["w"] = _normal(g, (E, N, K), dt, N ** -0.5)
        s["z"] = _normal(g, (T, K), dt) if c["act"] != "none" else None
        s["da"] = torch.empty(T, K, dtype=dt, device="cuda")
    else:
        s["a"] = _normal(g, (T, K), dt)
        s["dc"] = _normal(g, (T, N), dt, T ** -0.5)
        s["dw"] = torch.empty(E, N, K, dtype=dt, device="cuda")
        s["db"] = torch.empty(E, N, dtype=dt, device="cuda")
    return s


# ----------------------------------------------------------- plain forms ----

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


def _by_expert(state, rows, product):
    """product(rows of e, e) for each expert that has rows, joined again."""
    parts = rows.split(state["sizes"])
    return torch.cat([product(p, e) for e, p in enumerate(parts) if len(p)])


def _values(codes, scales):
    """32-bit values [rows, K] of stored codes and scale planes."""
    table = torch.tensor(CODE_VALUES, device=codes.device)
    v = table[torch.stack([codes & 15, codes >> 4], -1).int()].flatten(-2).unflatten(-1, (-1, 32))
    e = scales.transpose(0, 1).flatten(1)[:, : v.shape[1]].int() - 127
    return (v * _power_of_two(e).unsqueeze(-1)).flatten(-2)


def _plain(s):
    c = s["case"]
    dt = DTYPES[c["dtype"]]
    if c["kind"] == "quant":
        codes, e = _to_codes(s["x"])
        table = torch.tensor(CODE_VALUES, device=codes.device)
        return (table[codes.int()].unflatten(-1, (-1, 32)) * _power_of_two(e).unsqueeze(-1)).flatten(-2).to(dt)
    if c["kind"] == "mx4":
        x = _values(*_packed(*_to_codes(s["x"]))) if c["from16"] else _values(s["codes"], s["scales"])
        if not c["E"]:
            w = _values(s["w_codes"], s["w_scales"])
            return _act(c["act"], x @ w.T + s["bias"].float()).to(dt)
        w = _values(s["w_codes"].flatten(0, 1), s["w_scales"]).view(c["E"], c["N"], c["K"])
        return _by_expert(s, x, lambda p, e: _act(c["act"], p @ w[e].T + s["bias"][e].float()).to(dt))
    if c["kind"] == "fwd":
        z = _by_expert(s, s["a"], lambda p, e: p.float() @ s["w"][e].float().T + s["bias"][e].float())
        return (_act(c["act"], z).to(dt), z.to(dt)) if c["preact"] else _act(c["act"], z).to(dt)
    if c["kind"] == "dgrad":
        d = _by_expert(s, s["dc"], lambda p, e: p.float() @ s["w"][e].float())
        return (d if s["z"] is None else d * _act_slope(c["act"], s["z"].float())).to(dt)
    pairs = list(zip(s["dc"].split(s["sizes"]), s["a"].split(s["sizes"])))
    return (torch.stack([(d.float().T @ a.float()).to(dt) for d, a in pairs]),
            torch.stack([d.float().sum(0).to(dt) for d, a in pairs]))


# ------------------------------------------------------------------ run ----

def run(state):
    s = state
    if not own:
        return _plain(s)
    import tiled_dense_gemm_bias_amd as gba
    c = s["case"]
    if c["kind"] == "quant":
        gba.mx4_quantize(s["x"], s["codes"], s["scales"])
        return gba.mx4_dequantize(s["codes"], s["scales"], s["y"])
    if c["kind"] == "mx4":
        if c["from16"]:
            gba.mx4_quantize(s["x"], s["codes"], s["scales"])
        if not c["E"]:
            return gba.gemm_bias_act_mx4(s["codes"], s["scales"], s["w_codes"], s["w_scales"], s["bias"], s["c"], c["act"],
                                         workspace=s["workspace"])
        return gba.grouped_gemm_bias_act_mx4(s["codes"], s["scales"], s["offsets"], s["w_codes"], s["w_scales"], s["bias"],
                                             s["c"], c["act"], workspace=s["workspace"])
    if c["kind"] == "fwd":
        gba.grouped_gemm_bias_act(s["a"], s["offsets"], s["w"], s["bias"], s["c"], c["act"], transpose_b=True, preact=s["z"],
                                  workspace=s["workspace"])
        return (s["c"], s["z"]) if c["preact"] else s["c"]
    if c["kind"] == "dgrad":
        return gba.grouped_gemm_act_grad(s["dc"], s["offsets"], s["w"], s["z"], s["da"], c["act"], transpose_b=True,
                                         workspace=s["workspace"])
    gba.grouped_gemm_wgrad(s["a"], s["dc"], s["offsets"], s["dw"], s["db"], transpose_b=True, workspace=s["workspace"])
    return s["dw"], s["db"]


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


def _exact_power(e):
    """2^e in 64 bits for -1023 < e < 1024, from its bits (a power function may round)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_mx4(x):
    """The format's definition on 64-bit values: of each block, scale 2^(floor(log2(max)) - 2), then the nearest value of
    the table, ties to the even code."""
    x = x.double()
    b = x.reshape(x.shape[0], -1, 32)
    top = b.abs().max(-1, keepdim=True).values
    scale = torch.where(top > 0, _exact_power(torch.frexp(top)[1].clamp(min=-124) - 3), torch.zeros_like(top))
    y = torch.where(scale > 0, b / torch.where(scale > 0, scale, torch.ones_like(scale)), torch.zeros_like(b))
    # The spacing of the values is 0.5 below 2, 1 from 2 to 4 and 2 above; round() takes ties to even multiples of it.
    step = torch.where(y.abs() < 2, 0.5, torch.where(y.abs() < 4, 1.0, 2.0))
    return ((torch.round(y / step) * step).clamp(-6, 6) * scale).reshape(x.shape)


def _exact_stored(codes, scales, K):
    nibble = torch.empty(codes.shape[0], K, dtype=torch.int64, device=codes.device)
    nibble[:, 0::2], nibble[:, 1::2] = (codes % 16).long(), (codes // 16).long()
    sign, power, half = 1 - 2 * (nibble // 8), nibble // 2 % 4, nibble % 2
    size = torch.where(power == 0, 0.5 * half.double(), (1 + 0.5 * half.double()) * _exact_power(power - 1))
    at = torch.arange(K, device=codes.device) // 32
    return sign * size * _exact_power(scales[at // 4, :, at % 4].T.long() - 127)


def exact(case, seed):
    s, c = prepare(case, seed), case
    if c["kind"] == "quant":
        return torch.cat([_exact_mx4(p) for p in s["x"].split(2048)])
    begin, parts = 0, []
    if c["kind"] == "mx4":
        x = _exact_mx4(s["x"]) if c["from16"] else _exact_stored(s["codes"], s["scales"], c["K"])
        if not c["E"]:
            w = _exact_stored(s["w_codes"], s["w_scales"], c["K"])
            return _exact_act(c["act"], torch.addmm(s["bias"].double(), x, w.T.contiguous()))
        for e, n in enumerate(s["sizes"]):
            if n:
                w = _exact_stored(s["w_codes"][e], s["w_scales"][:, e * c["N"]:(e + 1) * c["N"]], c["K"])
                parts.append(_exact_act(c["act"], torch.addmm(s["bias"][e].double(), x[begin:begin + n], w.T.contiguous())))
            begin += n
        return torch.cat(parts)
    if c["kind"] == "wgrad":
        dw, db = torch.zeros(c["E"], c["N"], c["K"], dtype=torch.float64, device="cuda"), torch.zeros(c["E"], c["N"], dtype=torch.float64, device="cuda")
        for e, n in enumerate(s["sizes"]):
            d = s["dc"][begin:begin + n].double()
            torch.mm(d.T.contiguous(), s["a"][begin:begin + n].double(), out=dw[e])
            db[e] = d.sum(0)
            begin += n
        return dw, db
    for e, n in enumerate(s["sizes"]):
        if n:
            w = s["w"][e].double()
            if c["kind"] == "fwd":
                parts.append(s["a"][begin:begin + n].double() @ w.T.contiguous() + s["bias"][e].double())
            else:
                parts.append(s["dc"][begin:begin + n].double() @ w)
        begin += n
    r = torch.cat(parts)
    if c["kind"] == "dgrad":
        return r if s["z"] is None else r * _exact_slope(c["act"], s["z"].double())
    return (_exact_act(c["act"], r), r) if c["preact"] else _exact_act(c["act"], r)
