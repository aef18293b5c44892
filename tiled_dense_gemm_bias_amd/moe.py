"""Python binding of libgba_moe: routing of tokens to experts, movement of their rows, and
products in 8-bit floating point with a scale for each block of 128 (see include/gba_moe.h
for the C ABI). The names here are also names of the package.

    gba.moe_route(logits, indices, weights, bias, offsets=offsets, rows=rows)
    gba.fp8_quantize(x, xs_codes, xs_scales, rows=rows)
    gba.grouped_gemm_bias_act_fp8_block(xs_codes, xs_scales, offsets, w_codes, w_scales, b, h, "gelu")
    gba.moe_combine(y, rows, weights, out)

Slot (t, j) is token t's j-th expert; rows are sorted by expert, and rows[t, j] is the row of
slot (t, j), or -1. A row belongs to one slot at most: one that a caller's own rows name twice is
written as a mixture of both. As in the rest of the package the caller owns every tensor, work runs
on the current stream, and tensors used on another stream than the one they were made on are the
caller's to keep alive (torch's record_stream).
"""
from __future__ import annotations

import ctypes
import os

import torch

from . import GbaError, _act
from .experts import _addr, _device, _expect, _offsets, _same_dtype, _workspace

_HERE = os.path.dirname(os.path.abspath(__file__))
MOE_LIB_PATH = os.path.join(_HERE, "libgba_moe.so")
MOE_HEADER = os.path.join(os.path.dirname(_HERE), "include", "gba_moe.h")

SCORES = {"softmax": 0, "sigmoid": 1}
RENORMALIZE = 1
POW2_SCALES = 1
F32_TOKENS = 256

_LIB = None


class _Plan(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("kind", "tile_m", "tile_n", "splits")]


def _lib():
    global _LIB
    if _LIB is None:
        if not os.path.exists(MOE_LIB_PATH):
            raise ImportError("libgba_moe.so is not built; run: python -m tiled_dense_gemm_bias_amd.build")
        lib = ctypes.CDLL(MOE_LIB_PATH)
        p, i64, ci, sz, cf = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t, ctypes.c_float
        sig = {
            "moe_route": [p] * 7 + [i64] * 5 + [ci, ci, cf, ci, ci, p, sz],
            "moe_route_grad": [p] * 4 + [i64] * 3 + [ci, cf, ci, ci],
            "moe_sort": [p] * 4 + [i64] * 3 + [p, sz],
            "moe_sort_workspace": [i64] * 3,
            "moe_dispatch": [p] * 3 + [i64] * 4 + [ci],
            "moe_combine": [p] * 4 + [i64] * 4 + [ci],
            "moe_combine_grad": [p] * 6 + [i64] * 4 + [ci],
            "fp8_quantize": [p] * 4 + [i64] * 4 + [ci, ci],
            "fp8_dequantize": [p] * 3 + [i64] * 2 + [ci],
            "fp8_quantize_weights": [p] * 5 + [i64] * 3 + [ci, ci],
            "fp8_dequantize_weights": [p] * 3 + [i64] * 3 + [ci],
            "gemm_bias_act_fp8_block": [p] * 7 + [i64] * 3 + [ci, ci, p, sz],
            "grouped_gemm_bias_act_fp8_block": [p] * 8 + [i64] * 4 + [ci, ci, p, sz],
            "gemm_act_grad_fp8_block": [p] * 6 + [i64] * 3 + [ci, ci, p, sz],
            "grouped_gemm_act_grad_fp8_block": [p] * 7 + [i64] * 4 + [ci, ci, p, sz],
            "gbm_set_stream": [p],
            "gbm_get_plan": [i64] * 4 + [sz, ci, ctypes.POINTER(_Plan)],
            "gbm_last_hip_error": [],
            "gbm_version": [],
        }
        for name, args in sig.items():
            fn = getattr(lib, name)
            fn.argtypes = args
            fn.restype = ci
        lib.gbm_version.restype = ctypes.c_char_p
        lib.moe_sort_workspace.restype = sz
        _LIB = lib
    return _LIB


def moe_lib():
    """The raw ctypes handle of libgba_moe.so (C ABI of include/gba_moe.h)."""
    return _lib()


def moe_version() -> str:
    return _lib().gbm_version().decode()


def _call(fn_name, d, *args):
    """Run entry point fn_name on device d's current stream (see the package's _call)."""
    lib = _LIB or _lib()
    C = torch._C
    if d == C._cuda_getDevice():
        lib.gbm_set_stream(C._cuda_getCurrentRawStream(d))
        st = getattr(lib, fn_name)(*args)
    else:
        with torch.cuda.device(d):
            lib.gbm_set_stream(C._cuda_getCurrentRawStream(d))
            st = getattr(lib, fn_name)(*args)
    if st != 0:
        raise GbaError(st, fn_name)


def _typed(what, t, dtype):
    if t is not None and t.dtype is not dtype:
        raise TypeError("%s has dtype %s, expected %s" % (what, t.dtype, dtype))


# ------------------------------------------------------------------ routing ----

_LOGITS = {torch.float16: 0, torch.bfloat16: 1, torch.float32: 2}


def _score(score):
    if score not in SCORES:
        raise ValueError("unknown score %r; one of %s" % (score, sorted(SCORES)))
    return SCORES[score]


def _logits(logits):
    if logits.dtype not in _LOGITS:
        raise TypeError("logits are float16, bfloat16 or float32, got %s" % logits.dtype)
    return _LOGITS[logits.dtype]


def moe_sort_workspace(T: int, E: int, k: int) -> int:
    """Bytes of workspace that sorting T k slots of E experts needs (0 for few slots)."""
    return _lib().moe_sort_workspace(T, E, k)


def moe_route(logits, indices, weights, bias=None, offsets=None, rows=None, slots=None, score="softmax",
              renormalize=True, scale=1.0, groups=1, top_groups=1, group_best=1, workspace=None):
    """Each token's k experts and their weights. Returns (indices, weights).

    logits [T,E] float16, bfloat16 or float32; indices int32 and weights float32 [T,k]. Scores are
    softmax(logits) or the logits' sigmoid; the choice is by score + bias (float32 [E] or None), ties to the lower
    number; weights are scale * score, divided by the chosen scores' sum where renormalize. groups > 1: only the experts
    of the top_groups best groups are left, a group's value being the sum of its group_best (1 or 2) best.
    Experts with a logit or bias of -inf are never chosen; slots left over have index -1 and weight 0.

    offsets (int32 [E+1]) and rows (int32 [T,k]), with slots (int32 [T k]) or without: the slots are
    sorted too, as by moe_sort, with moe_sort_workspace(T, E, k) bytes of workspace."""
    d = _device(logits, indices, weights, bias, offsets, rows, slots)
    T, E = logits.shape
    k = indices.shape[-1]
    _typed("indices", indices, torch.int32)
    _typed("weights", weights, torch.float32)
    _typed("bias", bias, torch.float32)
    _expect("indices", indices, (T, k))
    _expect("weights", weights, (T, k))
    _expect("bias", bias, (E,))
    if offsets is not None or rows is not None or slots is not None:
        if offsets is None or rows is None:
            raise ValueError("offsets and rows come together")
        _sorted(offsets, rows, slots, T, E, k)
    ws, nb = _workspace(workspace, d)
    _call("moe_route", d, logits.data_ptr(), _addr(bias), indices.data_ptr(), weights.data_ptr(), _addr(offsets), _addr(rows),
          _addr(slots), T, E, k, groups, top_groups, group_best, _score(score), scale, _logits(logits),
          RENORMALIZE if renormalize else 0, ws, nb)
    return indices, weights


def moe_route_grad(logits, indices, dweights, dlogits, score="softmax", renormalize=True, scale=1.0):
    """dlogits [T,E] (the logits' dtype) from dweights (float32 [T,k]): the gradient of moe_route's
    weights, for the experts that it chose. A token without any slot gets zeros, or NaN where moe_route's weights are NaN for
    its logits. Returns dlogits."""
    d = _device(logits, indices, dweights, dlogits)
    T, E = logits.shape
    k = indices.shape[-1]
    _typed("indices", indices, torch.int32)
    _typed("dweights", dweights, torch.float32)
    _typed("dlogits", dlogits, logits.dtype)
    _expect("indices", indices, (T, k))
    _expect("dweights", dweights, (T, k))
    _expect("dlogits", dlogits, (T, E))
    _call("moe_route_grad", d, logits.data_ptr(), indices.data_ptr(), dweights.data_ptr(), dlogits.data_ptr(), T, E, k,
          _score(score), scale, _logits(logits), RENORMALIZE if renormalize else 0)
    return dlogits


def _sorted(offsets, rows, slots, T, E, k):
    _offsets(offsets, E)
    _typed("rows", rows, torch.int32)
    _typed("slots", slots, torch.int32)
    _expect("rows", rows, (T, k))
    _expect("slots", slots, (T * k,))


def moe_sort(indices, offsets, rows, slots=None, workspace=None):
    """Sorts the slots of indices (int32 [T,k], -1: none) by expert, stably. Returns (offsets, rows).

    offsets int32 [E+1]: expert e owns rows offsets[e] .. offsets[e+1] - 1; rows int32 [T,k]: each slot's row, or -1;
    slots int32 [T k] or None: each row's slot t k + j, -1 past the last. workspace: moe_sort_workspace(T, E, k) bytes."""
    d = _device(indices, offsets, rows, slots)
    T, k = indices.shape
    E = offsets.shape[0] - 1
    _typed("indices", indices, torch.int32)
    _sorted(offsets, rows, slots, T, E, k)
    ws, nb = _workspace(workspace, d)
    _call("moe_sort", d, indices.data_ptr(), offsets.data_ptr(), rows.data_ptr(), _addr(slots), T, E, k, ws, nb)
    return offsets, rows


# --------------------------------------------------------- movement of rows ----

def _tokens_dtype(y, tokens, *rest):
    """The code of y's dtype, which rest share; tokens (combine's sums, or their gradient) may be float32 beside it."""
    if tokens.dtype is torch.float32:
        return _same_dtype(y, *rest) | F32_TOKENS
    return _same_dtype(y, tokens, *rest)


def moe_dispatch(x, rows, out):
    """out[rows[t, j]] = x[t]; other rows of out stay. x [T,H], rows int32 [T,k], out [R,H]. Returns out."""
    d = _device(x, rows, out)
    dt = _same_dtype(x, out)
    (T, H), k, R = x.shape, rows.shape[-1], out.shape[0]
    _typed("rows", rows, torch.int32)
    _expect("rows", rows, (T, k))
    _expect("out", out, (R, H))
    _call("moe_dispatch", d, x.data_ptr(), rows.data_ptr(), out.data_ptr(), T, k, H, R, dt)
    return out


def moe_combine(y, rows, weights, out):
    """out[t] = sum over j of weights[t, j] * y[rows[t, j]]; weights float32 [T,k], or None for ones (the gradient of
    moe_dispatch). A slot of -1 adds its weight times 0, so that weight has to be finite: moe_route leaves 0 there, and NaN in
    rows whose logits hold a NaN, which then shows in out. y [R,H], out [T,H], of y's dtype or float32. Returns out."""
    d = _device(y, rows, weights, out)
    dt = _tokens_dtype(y, out)
    (R, H), (T, k) = y.shape, rows.shape
    _typed("rows", rows, torch.int32)
    _typed("weights", weights, torch.float32)
    _expect("weights", weights, (T, k))
    _expect("out", out, (T, H))
    _call("moe_combine", d, y.data_ptr(), rows.data_ptr(), _addr(weights), out.data_ptr(), T, k, H, R, dt)
    return out


def moe_combine_grad(dout, y, rows, weights, dy, dweights):
    """moe_combine's gradients: dy[rows[t, j]] = weights[t, j] * dout[t] (other rows stay) and dweights[t, j] =
    <dout[t], y[rows[t, j]]>. dout [T,H] of y's dtype or float32; either of dy [R,H] and dweights (float32 [T,k]) may be
    None. Returns (dy, dweights)."""
    d = _device(dout, y, rows, weights, dy, dweights)
    dt = _tokens_dtype(y, dout, dy)
    (R, H), (T, k) = y.shape, rows.shape
    _typed("rows", rows, torch.int32)
    _typed("weights", weights, torch.float32)
    _typed("dweights", dweights, torch.float32)
    _expect("dout", dout, (T, H))
    _expect("weights", weights, (T, k))
    _expect("dy", dy, (R, H))
    _expect("dweights", dweights, (T, k))
    _call("moe_combine_grad", d, dout.data_ptr(), y.data_ptr(), rows.data_ptr(), _addr(weights), _addr(dy), _addr(dweights),
          T, k, H, R, dt)
    return dy, dweights


# ------------------------------------------------- 8-bit floats by blocks ----

def _blocks(n):
    return (n + 127) // 128


def fp8_scales_shape(R: int, K: int) -> tuple:
    """Shape of the scales of an [R,K] matrix by rows: [ceil(K/128), R]."""
    return (_blocks(K), R)


def fp8_weight_scales_shape(E: int, N: int, K: int) -> tuple:
    """Shape of the scales of E weights [N,K]: [E, ceil(N/128), ceil(K/128)]."""
    return (E, _blocks(N), _blocks(K))


def _f8(what, codes, scales):
    if codes.dtype is not torch.float8_e4m3fn:
        raise TypeError("%s: codes are float8_e4m3fn, got %s" % (what, codes.dtype))
    _typed(what + " scales", scales, torch.float32)


def _f8_rows(what, codes, scales, shape):
    _f8(what, codes, scales)
    _expect(what + " codes", codes, shape)
    _expect(what + " scales", scales, ((shape[1] + 127) // 128, shape[0]))


def _f8_weights(what, codes, scales, shape):
    _f8(what, codes, scales)
    _expect(what + " codes", codes, shape)
    _expect(what + " scales", scales, shape[:-2] + ((shape[-2] + 127) // 128, (shape[-1] + 127) // 128))


def fp8_quantize(x, codes, scales, rows=None, pow2=False):
    """x [T,K] (float16 or bfloat16, K a multiple of 16) to 8-bit floats with a scale for each 128 values of a row:
    codes float8_e4m3fn [R,K], scales float32 [ceil(K/128),R]. rows: None (R = T), or int32 [T,k], and x[t] goes to every
    row rows[t, j] (moe_dispatch in 8 bits; other rows stay). pow2: scales are powers of two. Returns (codes, scales)."""
    d = _device(x, codes, scales, rows)
    (T, K), R = x.shape, codes.shape[0]
    _f8_rows("x", codes, scales, (R, K))
    k = 1
    if rows is not None:
        _typed("rows", rows, torch.int32)
        k = rows.shape[-1]
        _expect("rows", rows, (T, k))
    elif R != T:
        raise ValueError("shape mismatch: x has %d rows, codes %d" % (T, R))
    _call("fp8_quantize", d, x.data_ptr(), _addr(rows), codes.data_ptr(), scales.data_ptr(), T, k, K, R, _same_dtype(x),
          POW2_SCALES if pow2 else 0)
    return codes, scales


def fp8_dequantize(codes, scales, x):
    """x [R,K] (float16 or bfloat16) = the values of codes and scales. Returns x."""
    d = _device(codes, scales, x)
    R, K = x.shape
    _f8_rows("x", codes, scales, (R, K))
    _call("fp8_dequantize", d, codes.data_ptr(), scales.data_ptr(), x.data_ptr(), R, K, _same_dtype(x))
    return x


def fp8_quantize_weights(w, codes, scales, codes_t=None, scales_t=None, pow2=False):
    """w [E,N,K] or [N,K] to 8-bit floats with a scale for each 128 x 128 block: codes like w, scales
    [E,ceil(N/128),ceil(K/128)] (w's leading dimensions); codes_t, scales_t: the same of w's last two dimensions
    transposed, for the gradient of a product's input. Either pair may be None. Returns (codes, scales)."""
    d = _device(w, codes, scales, codes_t, scales_t)
    N, K = w.shape[-2:]
    lead = w.shape[:-2]
    if len(lead) > 1:
        raise ValueError("w is [E,N,K] or [N,K], got %s" % (tuple(w.shape),))
    if (codes is None) != (scales is None) or (codes_t is None) != (scales_t is None) or (codes is None and codes_t is None):
        raise ValueError("codes and scales come in pairs, one at least")
    if codes is not None:
        _f8_weights("w", codes, scales, lead + (N, K))
    if codes_t is not None:
        _f8_weights("transposed w", codes_t, scales_t, lead + (K, N))
    _call("fp8_quantize_weights", d, w.data_ptr(), _addr(codes), _addr(scales), _addr(codes_t), _addr(scales_t),
          lead[0] if lead else 1, N, K, _same_dtype(w), POW2_SCALES if pow2 else 0)
    return codes, scales


def fp8_dequantize_weights(codes, scales, w):
    """w [E,N,K] or [N,K] (float16 or bfloat16) = the values of codes and scales. Returns w."""
    d = _device(codes, scales, w)
    if w.dim() not in (2, 3):
        raise ValueError("w is [E,N,K] or [N,K], got %s" % (tuple(w.shape),))
    _f8_weights("w", codes, scales, tuple(w.shape))
    N, K = w.shape[-2:]
    _call("fp8_dequantize_weights", d, codes.data_ptr(), scales.data_ptr(), w.data_ptr(), w.shape[0] if w.dim() == 3 else 1, N, K,
          _same_dtype(w))
    return w


# ---------------------------------------------------------- products in 8 bits ----

def gemm_bias_act_fp8_block(a_codes, a_scales, w_codes, w_scales, bias, c, act="gelu", preact=None, workspace=None):
    """c[M,N] = act(a @ w.T + bias), a [M,K] as fp8_quantize and w [N,K] as fp8_quantize_weights leave them; bias [N] or
    None, c and preact ([M,N] or None, receives a @ w.T + bias rounded) float16 or bfloat16. workspace: optional device
    tensor (a few MiB) that lets calls with few output tiles split K. Returns c."""
    d = _device(a_codes, a_scales, w_codes, w_scales, bias, c, preact)
    dt = _same_dtype(c, bias, preact)
    (M, K), N = a_codes.shape, c.shape[-1]
    _f8_rows("a", a_codes, a_scales, (M, K))
    _f8_weights("w", w_codes, w_scales, (N, K))
    _expect("c", c, (M, N))
    _expect("bias", bias, (N,))
    _expect("preact", preact, (M, N))
    ws, nb = _workspace(workspace, d)
    _call("gemm_bias_act_fp8_block", d, a_codes.data_ptr(), a_scales.data_ptr(), w_codes.data_ptr(), w_scales.data_ptr(), _addr(bias),
          c.data_ptr(), _addr(preact), M, N, K, _act(act), dt, ws, nb)
    return c


def grouped_gemm_bias_act_fp8_block(a_codes, a_scales, offsets, w_codes, w_scales, bias, c, act="gelu", preact=None, workspace=None):
    """gemm_bias_act_fp8_block by expert: a [T,K] sorted by expert, w [E,N,K], bias [E,N] or None, offsets int32 [E+1].
    Rows of no expert are not written. Returns c."""
    d = _device(a_codes, a_scales, offsets, w_codes, w_scales, bias, c, preact)
    dt = _same_dtype(c, bias, preact)
    (T, K), (E, N, _) = a_codes.shape, w_codes.shape
    _f8_rows("a", a_codes, a_scales, (T, K))
    _f8_weights("w", w_codes, w_scales, (E, N, K))
    _expect("c", c, (T, N))
    _expect("bias", bias, (E, N))
    _expect("preact", preact, (T, N))
    _offsets(offsets, E)
    ws, nb = _workspace(workspace, d)
    _call("grouped_gemm_bias_act_fp8_block", d, a_codes.data_ptr(), a_scales.data_ptr(), offsets.data_ptr(), w_codes.data_ptr(),
          w_scales.data_ptr(), _addr(bias), c.data_ptr(), _addr(preact), T, E, N, K, _act(act), dt, ws, nb)
    return c


def gemm_act_grad_fp8_block(dc_codes, dc_scales, w_codes, w_scales, z, da, act="gelu", workspace=None):
    """da[M,N] = (dc @ w.T) * act'(z): the gradient of a product's input, through the activation that made it. dc [M,K] as
    fp8_quantize leaves it; w [N,K]: the product's weights transposed (codes_t, scales_t of fp8_quantize_weights). act
    "none": z may be None. Returns da."""
    d = _device(dc_codes, dc_scales, w_codes, w_scales, z, da)
    dt = _same_dtype(da, z)
    (M, K), N = dc_codes.shape, da.shape[-1]
    _f8_rows("dc", dc_codes, dc_scales, (M, K))
    _f8_weights("w", w_codes, w_scales, (N, K))
    _expect("da", da, (M, N))
    _expect("z", z, (M, N))
    ws, nb = _workspace(workspace, d)
    _call("gemm_act_grad_fp8_block", d, dc_codes.data_ptr(), dc_scales.data_ptr(), w_codes.data_ptr(), w_scales.data_ptr(), _addr(z),
          da.data_ptr(), M, N, K, _act(act), dt, ws, nb)
    return da


def grouped_gemm_act_grad_fp8_block(dc_codes, dc_scales, offsets, w_codes, w_scales, z, da, act="gelu", workspace=None):
    """gemm_act_grad_fp8_block by expert: dc [T,K] sorted by expert, w [E,N,K], offsets int32 [E+1]. Returns da."""
    d = _device(dc_codes, dc_scales, offsets, w_codes, w_scales, z, da)
    dt = _same_dtype(da, z)
    (T, K), (E, N, _) = dc_codes.shape, w_codes.shape
    _f8_rows("dc", dc_codes, dc_scales, (T, K))
    _f8_weights("w", w_codes, w_scales, (E, N, K))
    _expect("da", da, (T, N))
    _expect("z", z, (T, N))
    _offsets(offsets, E)
    ws, nb = _workspace(workspace, d)
    _call("grouped_gemm_act_grad_fp8_block", d, dc_codes.data_ptr(), dc_scales.data_ptr(), offsets.data_ptr(), w_codes.data_ptr(),
          w_scales.data_ptr(), _addr(z), da.data_ptr(), T, E, N, K, _act(act), dt, ws, nb)
    return da


_KINDS = ("ring", "persistent", "stream")


def plan(T: int, E: int, N: int, K: int, workspace: int = 0, cus: int = 256) -> dict:
    """Kernel ("ring", "persistent" or "stream"), tile and splits of a product in 8 bits of T rows, E experts of [N,K],
    with `workspace` bytes on a device of `cus` compute units."""
    p = _Plan()
    st = _lib().gbm_get_plan(T, E, N, K, workspace, cus, ctypes.byref(p))
    if st != 0:
        raise GbaError(st, "gbm_get_plan")
    return {"kind": _KINDS[p.kind], "tile_m": p.tile_m, "tile_n": p.tile_n, "splits": p.splits}
