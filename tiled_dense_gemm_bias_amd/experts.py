"""Python binding of libgba_experts: products grouped by expert, forward and
backward, and microscaled 4-bit floating point (see include/gba_experts.h for the
C ABI). The names here are also names of the package.

Rows are sorted by expert: rows offsets[e] .. offsets[e+1] - 1 belong to expert
e, with offsets an int32 device tensor of E + 1 entries that the host never reads.

    gba.grouped_gemm_bias_act(a, offsets, w, bias, h, "gelu", transpose_b=True, preact=z)
    gba.grouped_gemm_act_grad(dy, offsets, w2, z, dz, "gelu", transpose_b=True)
    gba.grouped_gemm_wgrad(a, dz, offsets, dw, db, transpose_b=True)

As in the rest of the package the caller owns every tensor, work runs on the
current stream, and tensors used on another stream than the one they were made
on are the caller's to keep alive (torch's record_stream).
"""
from __future__ import annotations

import ctypes
import os

import torch

from . import GbaError, TRANSPOSE_B, _act, _check_dev, _dtype_code

_HERE = os.path.dirname(os.path.abspath(__file__))
EXPERTS_LIB_PATH = os.path.join(_HERE, "libgba_experts.so")
EXPERTS_HEADER = os.path.join(os.path.dirname(_HERE), "include", "gba_experts.h")

OUT_F32 = 16
ACCUMULATE = 32

_LIB = None


class _Plan(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("tile_m", "tile_n", "persistent", "splits", "non_temporal")]


def _lib():
    global _LIB
    if _LIB is None:
        if not os.path.exists(EXPERTS_LIB_PATH):
            raise ImportError("libgba_experts.so is not built; run: python -m tiled_dense_gemm_bias_amd.build")
        lib = ctypes.CDLL(EXPERTS_LIB_PATH)
        p, i64, ci, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
        sig = {
            "grouped_gemm_bias_act": [p] * 6 + [i64] * 4 + [ci, ci, ci, p, sz],
            "grouped_gemm_act_grad": [p] * 5 + [i64] * 4 + [ci, ci, ci, p, sz],
            "grouped_gemm_wgrad": [p] * 5 + [i64] * 4 + [ci, ci, p, sz],
            "mx4_quantize": [p, p, p, i64, i64, ci],
            "mx4_dequantize": [p, p, p, i64, i64, ci],
            "gemm_bias_act_mx4": [p] * 6 + [i64] * 3 + [ci, ci, p, sz],
            "grouped_gemm_bias_act_mx4": [p] * 7 + [i64] * 4 + [ci, ci, p, sz],
            "gbx_get_plan": [ci] + [i64] * 4 + [sz, ci, ctypes.POINTER(_Plan)],
            "gbx_set_stream": [p],
            "gbx_last_hip_error": [],
            "gbx_version": [],
        }
        for name, args in sig.items():
            fn = getattr(lib, name)
            fn.argtypes = args
            fn.restype = ci
        lib.gbx_version.restype = ctypes.c_char_p
        _LIB = lib
    return _LIB


def experts_lib():
    """The raw ctypes handle of libgba_experts.so (C ABI of include/gba_experts.h)."""
    return _lib()


def experts_version() -> str:
    return _lib().gbx_version().decode()


_OPS = {"forward": 0, "act_grad": 1, "wgrad": 2, "wgrad_bias": 3, "mx4": 4}


def plan(op, T, E, N, K, workspace=0, cus=256) -> dict:
    """What a call of these sizes runs on a device of `cus` compute units, given a workspace of
    that many bytes: tile_m, tile_n, persistent, splits, non_temporal. op: "forward", "act_grad", "wgrad",
    "wgrad_bias" (with dbias) or "mx4" (dense: E = 1). Needs no device."""
    p = _Plan()
    st = _lib().gbx_get_plan(_OPS[op], T, E, N, K, workspace, cus, ctypes.byref(p))
    if st != 0:
        raise GbaError(st, "gbx_get_plan")
    return {n: getattr(p, n) for n, _ in _Plan._fields_}


# The calls below run in a few microseconds of host time, as long as the smallest
# kernels: the checks are written for that (attributes once, torch.Size compared as
# the tuple it is, no copies of shapes).

def _device(*ts):
    """The index of the tensors' one device; _check_dev's refusals otherwise."""
    d = ts[0].get_device()
    if d >= 0:
        for t in ts:
            if t is not None and (t.get_device() != d or not t.is_contiguous()):
                break
        else:
            return d
    _check_dev(*ts)
    raise ValueError("gba works on device tensors")


def _call(fn_name, d, *args):
    """Run entry point fn_name on device d's current stream (see the package's _call)."""
    lib = _LIB or _lib()
    C = torch._C
    if d == C._cuda_getDevice():
        lib.gbx_set_stream(C._cuda_getCurrentRawStream(d))
        st = getattr(lib, fn_name)(*args)
    else:
        with torch.cuda.device(d):
            lib.gbx_set_stream(C._cuda_getCurrentRawStream(d))
            st = getattr(lib, fn_name)(*args)
    if st != 0:
        raise GbaError(st, fn_name)


def _addr(t):
    return None if t is None else t.data_ptr()


def _workspace(workspace, d):
    if workspace is None:
        return None, 0
    if workspace.get_device() != d or not workspace.is_contiguous():
        raise ValueError("the workspace is a contiguous tensor on the operands' device")
    return workspace.data_ptr(), workspace.nbytes


def _offsets(offsets, E):
    if offsets.dtype is not torch.int32:
        raise TypeError("offsets are int32, got %s" % offsets.dtype)
    if offsets.shape != (E + 1,):
        raise ValueError("offsets has E + 1 = %d entries, got shape %s" % (E + 1, tuple(offsets.shape)))


_CODES = {torch.float16: 0, torch.bfloat16: 1}


def _same_dtype(first, *rest):
    dtype = first.dtype
    for t in rest:
        if t is not None and t.dtype is not dtype:
            raise TypeError("all operands must share one dtype")
    dt = _CODES.get(dtype)
    return _dtype_code(first) if dt is None else dt


def _expect(what, t, shape):
    if t is not None and t.shape != shape:
        raise ValueError("shape mismatch: %s is %s, expected %s" % (what, tuple(t.shape), shape))


def grouped_gemm_bias_act(a, offsets, w, bias, c, act="gelu", transpose_b=False, preact=None,
                          workspace=None):
    """c[r] = act(a[r] @ w[e] + bias[e]) for the rows r of each expert e. Returns c.

    a [T,K]; offsets int32 [E+1]; w [E,K,N], or [E,N,K] with transpose_b; bias
    [E,N] or None; c [T,N]. preact: [T,N] or None, receives a[r] @ w[e] + bias[e]
    rounded (grouped_gemm_act_grad's z). Rows of no expert are not written.
    workspace: optional device tensor (a few MiB) that lets calls with few output
    tiles split K."""
    d = _device(a, offsets, w, bias, c, preact)
    dt = _same_dtype(a, w, bias, c, preact)
    T, K = a.shape
    if transpose_b:
        E, N, k = w.shape
    else:
        E, k, N = w.shape
    if k != K:
        raise ValueError("shape mismatch: a is %s, w %s" % (tuple(a.shape), tuple(w.shape)))
    _expect("c", c, (T, N))
    _expect("bias", bias, (E, N))
    _expect("preact", preact, (T, N))
    _offsets(offsets, E)
    ws, nb = _workspace(workspace, d)
    _call("grouped_gemm_bias_act", d, a.data_ptr(), offsets.data_ptr(), w.data_ptr(), _addr(bias),
          c.data_ptr(), _addr(preact), T, E, N, K, _act(act), dt, TRANSPOSE_B if transpose_b else 0, ws, nb)
    return c


def grouped_gemm_act_grad(dc, offsets, w, z, da, act="gelu", transpose_b=False, workspace=None):
    """da[r] = (dc[r] @ w[e].T) * act'(z[r]): the input gradient of
    grouped_gemm_bias_act, carried through the activation that made its input
    (a = act(z)). Returns da.

    w and transpose_b as in the forward call; dc [T,N]; z, da [T,K]. act "none":
    da = dc @ w[e].T, and z may be None."""
    d = _device(dc, offsets, w, z, da)
    dt = _same_dtype(dc, w, z, da)
    T, N = dc.shape
    if transpose_b:
        E, n, K = w.shape
    else:
        E, K, n = w.shape
    if n != N:
        raise ValueError("shape mismatch: dc is %s, w %s" % (tuple(dc.shape), tuple(w.shape)))
    _expect("da", da, (T, K))
    _expect("z", z, (T, K))
    _offsets(offsets, E)
    ws, nb = _workspace(workspace, d)
    _call("grouped_gemm_act_grad", d, dc.data_ptr(), offsets.data_ptr(), w.data_ptr(), _addr(z),
          da.data_ptr(), T, E, N, K, _act(act), dt, TRANSPOSE_B if transpose_b else 0, ws, nb)
    return da


def grouped_gemm_wgrad(a, dc, offsets, dw, dbias=None, accumulate=False, transpose_b=False,
                       workspace=None):
    """dw[e] = a_e.T @ dc_e ([E,K,N]), or dc_e.T @ a_e ([E,N,K]) with transpose_b:
    the layout w has in the forward call; dbias[e] = dc_e.sum(0). Returns dw.

    a [T,K], dc [T,N], of one 16-bit dtype; dw and dbias of that dtype or both
    float32. accumulate (float32 only): added to what they hold. An empty expert's
    gradients are zero."""
    d = _device(a, dc, offsets, dw, dbias)
    dt = _same_dtype(a, dc)
    T, K = a.shape
    N, E = dc.shape[1], dw.shape[0]
    _expect("dc", dc, (T, N))
    _expect("dw", dw, (E, N, K) if transpose_b else (E, K, N))
    _expect("dbias", dbias, (E, N))
    _offsets(offsets, E)
    flags = TRANSPOSE_B if transpose_b else 0
    if dw.dtype is torch.float32:
        flags |= OUT_F32
    elif dw.dtype is not a.dtype:
        raise TypeError("dw has the operands' dtype or float32")
    if dbias is not None and dbias.dtype is not dw.dtype:
        raise TypeError("dbias has dw's dtype")
    if accumulate:
        if dw.dtype is not torch.float32:
            raise TypeError("accumulate needs float32 gradients")
        flags |= ACCUMULATE
    ws, nb = _workspace(workspace, d)
    _call("grouped_gemm_wgrad", d, a.data_ptr(), dc.data_ptr(), offsets.data_ptr(), dw.data_ptr(),
          _addr(dbias), T, E, N, K, dt, flags, ws, nb)
    return dw


def mx4_scales_shape(M: int, K: int) -> tuple:
    """Shape of the scale planes of an [M,K] matrix: [ceil(K/128), M, 4]."""
    return (-(-K // 128), M, 4)


def mx4_pack_scales(rows):
    """Scale planes of scale bytes given by rows ([M, K/32] uint8, the layout of the
    OCP MX specification's blocks in row order)."""
    M, blocks = rows.shape
    planes = -(-blocks // 4)
    full = torch.zeros(M, planes * 4, dtype=torch.uint8, device=rows.device)
    full[:, :blocks] = rows
    return full.view(M, planes, 4).transpose(0, 1).contiguous()


def mx4_unpack_scales(scales, K: int):
    """Scale bytes by rows ([M, K/32]) of scale planes."""
    return scales.transpose(0, 1).reshape(scales.shape[1], -1)[:, :K // 32].contiguous()


def _mx4(what, codes, scales, M, K):
    if codes.dtype is not torch.uint8 or scales.dtype is not torch.uint8:
        raise TypeError("4-bit codes and scales are uint8 tensors")
    if K % 32:
        raise ValueError("%s: K must be a multiple of 32, got %d" % (what, K))
    if codes.numel() != M * K // 2:
        raise ValueError("%s: %d rows of %d codes are %d bytes, got shape %s" % (what, M, K, M * K // 2,
                                                                                 tuple(codes.shape)))
    if scales.shape != (-(-K // 128), M, 4):
        raise ValueError("shape mismatch: %s scales are %s, expected %s" % (what, tuple(scales.shape),
                                                                          mx4_scales_shape(M, K)))


def mx4_quantize(x, codes, scales):
    """Quantise x [M,K] (float16 or bfloat16, K a multiple of 32) to microscaled 4-bit
    floats: codes uint8 [M,K/2], scales uint8 [ceil(K/128),M,4]. Returns (codes, scales)."""
    d = _device(x, codes, scales)
    M, K = x.shape
    _mx4("codes", codes, scales, M, K)
    _call("mx4_quantize", d, x.data_ptr(), codes.data_ptr(), scales.data_ptr(), M, K, _same_dtype(x))
    return codes, scales


def mx4_dequantize(codes, scales, x):
    """x [M,K] (float16 or bfloat16) = the values of codes and scales. Returns x."""
    d = _device(codes, scales, x)
    M, K = x.shape
    _mx4("codes", codes, scales, M, K)
    _call("mx4_dequantize", d, codes.data_ptr(), scales.data_ptr(), x.data_ptr(), M, K, _same_dtype(x))
    return x


def gemm_bias_act_mx4(a_codes, a_scales, w_codes, w_scales, bias, c, act="gelu", workspace=None):
    """c[M,N] = act(a @ w.T + bias) with a [M,K] and w [N,K] as mx4_quantize leaves
    them; bias [N] or None and c float16 or bfloat16. Returns c."""
    d = _device(a_codes, a_scales, w_codes, w_scales, bias, c)
    dt = _same_dtype(c, bias)
    (M, half), N = a_codes.shape, c.shape[1]
    K = 2 * half
    _expect("c", c, (M, N))
    _expect("w_codes", w_codes, (N, half))
    _expect("bias", bias, (N,))
    _mx4("a", a_codes, a_scales, M, K)
    _mx4("w", w_codes, w_scales, N, K)
    ws, nb = _workspace(workspace, d)
    _call("gemm_bias_act_mx4", d, a_codes.data_ptr(), a_scales.data_ptr(), w_codes.data_ptr(),
          w_scales.data_ptr(), _addr(bias), c.data_ptr(), M, N, K, _act(act), dt, ws, nb)
    return c


def grouped_gemm_bias_act_mx4(a_codes, a_scales, offsets, w_codes, w_scales, bias, c, act="gelu",
                              workspace=None):
    """gemm_bias_act_mx4 by expert: a [T,K] sorted by expert, w_codes [E,N,K/2] with the
    scale planes of the [E*N,K] matrix, bias [E,N] or None. Returns c."""
    d = _device(a_codes, a_scales, offsets, w_codes, w_scales, bias, c)
    dt = _same_dtype(c, bias)
    (T, half), (E, N, wide) = a_codes.shape, w_codes.shape
    if wide != half:
        raise ValueError("shape mismatch: a is %s, w %s" % (tuple(a_codes.shape), tuple(w_codes.shape)))
    K = 2 * half
    _expect("c", c, (T, N))
    _expect("bias", bias, (E, N))
    _mx4("a", a_codes, a_scales, T, K)
    _mx4("w", w_codes, w_scales, E * N, K)
    _offsets(offsets, E)
    ws, nb = _workspace(workspace, d)
    _call("grouped_gemm_bias_act_mx4", d, a_codes.data_ptr(), a_scales.data_ptr(), offsets.data_ptr(),
          w_codes.data_ptr(), w_scales.data_ptr(), _addr(bias), c.data_ptr(), T, E, N, K, _act(act), dt, ws, nb)
    return c
