"""Operators of a feed-forward block (``include/pipelined_ffn.h``).

    h, gate, up = pg.gated_projection(x, Wg, Wu, save=True)           # act(x Wg) * (x Wu)
    dx, dWg, dWu = pg.gated_projection_backward(dh, x, Wg, Wu, gate, up)

    hq, hs = pg.quantize_fp8(h)                                       # a scale for every 128 of a row
    Wq, Ws = pg.quantize_fp8(Wd, "block")                             # ... for every 128 x 128
    y = pg.gemm_fp8(hq, Wq, hs, Ws, dtype=torch.bfloat16)             # the product in 8 bits

Argument checks and marshalling only; the kernels are in the CUDA library.
CUDA tensors in, CUDA tensors out, enqueued on `stream` (default: torch's
current stream) without synchronising.  Ordinary calls (operands on the
current device, results allocated, no stream given) go through the native
binding, csrc/feedforward_binding.cpp, which returns None for any other; those,
and what is to be refused, are dealt with here.  Where there is no binding a warning
says so, and all calls are.
"""
from __future__ import annotations

import ctypes
import functools
import importlib.machinery
import importlib.util
import os
import types
import warnings

from . import training as _t

__all__ = ["gated_projection", "gated_projection_backward", "quantize_fp8", "gemm_fp8"]

ACTIVATION = {"silu": 0, "gelu": 1, "gelu_tanh": 2}  # enum gemm_activation
GROUP = {"row": 0, "column": 1, "block": 2}  # enum gemm_fp8_group
BLOCK = 128
SIDE_MAX = 1 << 30


def bind(l):
    I, L, P, S = ctypes.c_int, ctypes.c_longlong, ctypes.c_void_p, ctypes.c_size_t
    l.gated_projection.argtypes = [I, I, I] + [P, L] * 6 + [I, P]
    l.gated_projection.restype = I
    l.gated_projection_backward_workspace.argtypes = [I, I, I, ctypes.POINTER(S)]
    l.gated_projection_backward_workspace.restype = I
    l.gated_projection_backward.argtypes = [I, I, I] + [P, L] * 9 + [I, P, S, P]
    l.gated_projection_backward.restype = I
    l.quantize_fp8.argtypes = [I, I, P, L, I, I, I, P, L, P, L, P]
    l.quantize_fp8.restype = I
    l.gemm_fp8.argtypes = [I, I, I] + [P, L, I, I, P, L, L, I] * 2 + [P, L, I, P]
    l.gemm_fp8.restype = I
    return l


_FORMATS, _RESULTS = {}, {}
_torch = _bf16 = _f32 = _native = None
_NATIVE_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_build", "_feedforward.so")


def _load_native():
    """The native binding, given the library's functions."""
    if not os.path.exists(_NATIVE_PATH):
        raise RuntimeError(f"native binding not built ({_NATIVE_PATH} missing): run "
                           "`python -m async_copy_pipelined_gb300.buildlib` or __graft_entry__.build()")
    loader = importlib.machinery.ExtensionFileLoader("_feedforward", _NATIVE_PATH)
    module = importlib.util.module_from_spec(importlib.util.spec_from_loader("_feedforward", loader))
    loader.exec_module(module)
    if module.torch_build != str(_t._load().__version__):
        raise RuntimeError(f"native binding was built for torch {module.torch_build}: build it again with "
                           "`python -m async_copy_pipelined_gb300.buildlib --force`")
    l = _t._lib()
    module.entries(*(ctypes.cast(f, ctypes.c_void_p).value for f in (
        l.gated_projection, l.gated_projection_backward, l.gated_projection_backward_workspace, l.quantize_fp8,
        l.gemm_fp8)))
    return module


def _no_native():
    """In the native binding's place: leaves every call to Python."""
    def leave(*args):
        return None
    return types.SimpleNamespace(gated_projection=leave, gated_projection_backward=leave, quantize_fp8=leave,
                                 gemm_fp8=leave)


def _load():
    """torch and the native binding, on the first call."""
    global _torch, _bf16, _f32, _native
    if _torch is None:
        torch = _t._load()
        _t._lib()  # without the library there is no call at all
        try:
            _native = _load_native()
        except (RuntimeError, ImportError) as e:
            warnings.warn(f"{e}.  Calls of the feed-forward operators take the host 10 to 25 us longer without it",
                          RuntimeWarning, stacklevel=3)
            _native = _no_native()
        _FORMATS[torch.float8_e4m3fn] = 0  # enum gemm_fp8_format
        _FORMATS[torch.float8_e5m2] = 1
        _bf16, _f32 = torch.bfloat16, torch.float32
        _RESULTS[_f32], _RESULTS[_bf16] = _t.F32, _t.BF16
        _torch = torch
    return _torch


def _activation(name):
    code = ACTIVATION.get(name)
    if code is None:
        raise ValueError(f"activation must be one of {sorted(ACTIVATION)}")
    return code


def _format(dtype, name):
    code = _FORMATS.get(dtype)
    if code is None:
        raise TypeError(f"{name} must be float8_e4m3fn or float8_e5m2, not {dtype}")
    return code


def _sides(what, *sizes):
    """Sizes that the library takes (ctypes would silently cut larger ones)."""
    for n in sizes:
        if n > SIDE_MAX:
            raise ValueError(f"{what} has a size of {n}: at most 2^30")


def _at(t, device, name):
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}: all operands must be on one device")


def _tokens(t, name, last):
    """(rows, pitch) of a bfloat16 tensor seen as rows of its last dimension;
    last: what that dimension must be (None: anything)."""
    if t.dtype is not _bf16:
        raise TypeError(f"{name} must be bfloat16, not {t.dtype}")
    shape = t.shape
    if len(shape) == 0 or (last is not None and shape[-1] != last):
        raise ValueError(f"{name} must have a last dimension of {'its own' if last is None else last}")
    cols = shape[-1]
    if len(shape) == 2 and cols > 0:  # a matrix, most often
        rows, pitch = shape[0], t.stride(0)
        if rows <= SIDE_MAX and cols <= SIDE_MAX and (cols == 1 or t.stride(1) == 1):
            if rows <= 1:
                return rows, cols
            if pitch >= cols:
                return rows, pitch
    if t.numel() == 0:
        rows = 1
        for n in shape[:-1]:
            rows *= n
        _sides(name, rows)
        return rows, max(cols, 1)
    rows, cols, pitch = _t._rows(t, name)
    _sides(name, rows, cols)
    return rows, pitch


def _weight(t, name, device, rows, cols):
    """Pitch of a width x hidden bfloat16 weight."""
    if t.device != device:
        _at(t, device, name)
    if t.dtype is not _bf16:
        raise TypeError(f"{name} must be bfloat16, not {t.dtype}")
    shape = t.shape
    if len(shape) != 2 or shape[0] != rows or shape[1] != cols:
        raise ValueError(f"{name} must be a {rows} x {cols} matrix")
    return _matrix(t, name)


def _matrix(t, name):
    """Row pitch of a matrix whose rows are contiguous."""
    rows, cols = t.shape
    if rows > SIDE_MAX or cols > SIDE_MAX:
        _sides(name, rows, cols)
    sr, sc = t.stride()
    if rows == 0 or cols == 0:
        return max(cols, 1)
    if cols > 1 and sc != 1:
        raise ValueError(f"{name} must have unit column stride (row-major rows)")
    if rows == 1:
        return cols
    if sr < cols:
        raise ValueError(f"the rows of {name} overlap in memory")
    return sr


def _up_to(n, step):
    return -(-n // step) * step


def _pitch(cols, step):
    """Pitch of new rows of `cols` elements, for `step` elements in 16 bytes:
    the rows' own length where that aligns the next row, so that the result is
    contiguous, else up to 32 bytes, which are written at once (6606 x 143 x 897
    to float32 in 8 bits: 19.1 us at a pitch of 900, 12.2 at 904).  Rows of an odd
    number of 16 bytes do without that: 897's neighbour 900 takes 18.7 us at its
    own length, where 12.2 could be had at 904 by giving the call such a C."""
    return cols if cols % step == 0 else -(-cols // (2 * step)) * 2 * step


def _new_rows(torch, shape, dtype, device, step):
    """A tensor whose rows start at multiples of `step` elements, so that a
    product can read it: contiguous where the last dimension is one."""
    pitch = _pitch(shape[-1], step)
    if pitch == shape[-1]:
        return torch.empty(shape, dtype=dtype, device=device)
    if len(shape) == 2:
        return torch.empty_strided(shape, (pitch, 1), dtype=dtype, device=device)
    return torch.empty((*shape[:-1], pitch), dtype=dtype, device=device)[..., :shape[-1]]


def _refuse_shared(out, name, *inputs):
    """The output is written while inputs are still read: it may share no byte
    with one.  Each: (tensor, name)."""
    if out.numel() == 0:
        return
    for t, other in inputs:
        if t is None or t.numel() == 0:
            continue
        if _t._share_bytes(_extent(out), _extent(t)):
            raise ValueError(f"{name} overlaps {other} in memory")


def _extent(t):
    """A tensor as training._share_bytes takes it: a matrix of rows at one
    distance, or all from its first to its last byte where it is none."""
    if t.dim() == 2 and t.stride(0) == 1 and t.shape[1] > 1:
        t = t.t()
    size, dims = t.element_size(), [(n, d) for n, d in zip(t.shape, t.stride()) if n > 1]
    cols = dims.pop()[0] if dims and dims[-1][1] == 1 else 1
    rows, pitch = 1, cols
    for n, d in reversed(dims):
        if rows == 1:
            pitch = d
        elif d != pitch * rows:
            pitch = 0
            break
        rows *= n
    if pitch < cols:
        span = 1 + sum((n - 1) * d for n, d in zip(t.shape, t.stride()))
        return t.data_ptr(), 1, 1, span, span, 0, size
    return t.data_ptr(), 1, rows, cols, pitch, 0, size


def gated_projection(x, w_gate, w_up, out=None, *, activation="silu", save=False, stream=None):
    """h = act(x w_gate) * (x w_up) in one kernel, bfloat16.

    x: (..., width), its rows at any common distance; w_gate and w_up: width x
    hidden, row-major (as gemm_bf16 takes B).  Their bases and row pitches must
    be multiples of 16 bytes.  Both projections are float32 sums; the
    activation and the product take the unrounded sums and round once.

    activation: "silu", "gelu" (by the normal distribution's function) or
    "gelu_tanh".  out: where h goes; allocated if None, with rows at multiples
    of 16 bytes, so that the next product can read them.

    save: return (h, gate, up) with the two projections rounded to bfloat16,
    which gated_projection_backward takes; otherwise h alone."""
    torch = _torch or _load()
    act = _activation(activation)
    if out is None and stream is None:
        done = _native.gated_projection(x, w_gate, w_up, act, save)
        if done is not None:
            return done
    device, shape = x.device, x.shape
    handle, other = _t._enter(device, stream)
    rows, ldx = _tokens(x, "x", None)
    width = shape[-1]
    if len(w_gate.shape) != 2 or w_gate.shape[0] != width:
        raise ValueError(f"w_gate must be a matrix of {width} rows, as x's last dimension")
    hidden = w_gate.shape[1]
    ldwg = _weight(w_gate, "w_gate", device, width, hidden)
    ldwu = _weight(w_up, "w_up", device, width, hidden)
    shape = (*shape[:-1], hidden)
    pitch = _pitch(hidden, 8)
    if out is None:
        out = _new_rows(torch, shape, _bf16, device, 8)
        ldh = pitch
    else:
        _at(out, device, "out")
        if tuple(out.shape) != shape:
            raise ValueError(f"out must have the shape {shape}")
        _, ldh = _tokens(out, "out", hidden)
        _refuse_shared(out, "out", (x, "x"), (w_gate, "w_gate"), (w_up, "w_up"))
    gate = up = p_gate = p_up = None
    if save:
        gate = _new_rows(torch, shape, _bf16, device, 8)
        up = _new_rows(torch, shape, _bf16, device, 8)
        p_gate, p_up = gate.data_ptr(), up.data_ptr()
    _t._call(device, "gated_projection", _t._lib().gated_projection, rows, width, hidden, x.data_ptr(), ldx,
             w_gate.data_ptr(), ldwg, w_up.data_ptr(), ldwu, out.data_ptr(), ldh, p_gate, pitch, p_up, pitch, act,
             handle)
    if other is not None:
        _t._record(other, x, w_gate, w_up, out, gate, up)
    return (out, gate, up) if save else out


@functools.lru_cache(maxsize=256)
def _gated_bytes(device, rows, width, hidden):
    need = ctypes.c_size_t()
    _t._call(device, "gated_projection_backward_workspace", _t._lib().gated_projection_backward_workspace, rows, width,
             hidden, ctypes.byref(need))
    return need.value


def gated_projection_backward(dh, x, w_gate, w_up, gate, up, *, activation="silu", input_grad=True, weight_grad=True,
                              stream=None):
    """(dx, dw_gate, dw_up) of gated_projection from dh, its operands and the
    gate and up it kept (all bfloat16).

    The gradients of the two projections, dh * up * act'(gate) and dh *
    act(gate), are computed in float32 and rounded to bfloat16 as operands of
    the three products, which sum in float32 and round once.

    input_grad, weight_grad: False where dx, or dw_gate and dw_up, are not
    wanted (None is returned for them, and nothing is computed)."""
    torch = _torch or _load()
    act = _activation(activation)
    if stream is None:
        done = _native.gated_projection_backward(dh, x, w_gate, w_up, gate, up, act, input_grad, weight_grad)
        if done is not None:
            return done
    device, shape = x.device, x.shape
    handle, other = _t._enter(device, stream)
    rows, ldx = _tokens(x, "x", None)
    width = shape[-1]
    if len(w_gate.shape) != 2 or w_gate.shape[0] != width:
        raise ValueError(f"w_gate must be a matrix of {width} rows, as x's last dimension")
    hidden = w_gate.shape[1]
    ldwg = _weight(w_gate, "w_gate", device, width, hidden)
    ldwu = _weight(w_up, "w_up", device, width, hidden)
    pitches = []
    for name, t in (("dh", dh), ("gate", gate), ("up", up)):
        if t.device != device:
            _at(t, device, name)
        if t.shape[-1:] != (hidden,) or t.shape[:-1] != shape[:-1]:
            raise ValueError(f"{name} must have x's shape with a last dimension of {hidden}")
        pitches.append(_tokens(t, name, hidden)[1])
    dx = dw_gate = dw_up = px = pwg = pwu = None
    if input_grad:
        dx = _new_rows(torch, shape, _bf16, device, 8)
        px = dx.data_ptr()
    if weight_grad:
        dw_gate = _new_rows(torch, w_gate.shape, _bf16, device, 8)
        dw_up = _new_rows(torch, w_gate.shape, _bf16, device, 8)
        pwg, pwu = dw_gate.data_ptr(), dw_up.data_ptr()
    ws = _t._workspace(device, _gated_bytes(device, rows, width, hidden), other)
    _t._call(device, "gated_projection_backward", _t._lib().gated_projection_backward, rows, width, hidden,
             dh.data_ptr(), pitches[0], x.data_ptr(), ldx, w_gate.data_ptr(), ldwg, w_up.data_ptr(), ldwu,
             gate.data_ptr(), pitches[1], up.data_ptr(), pitches[2], px, _pitch(width, 8), pwg, _pitch(hidden, 8), pwu,
             _pitch(hidden, 8), act, ws.data_ptr(), ws.numel(), handle)
    if other is not None:
        _t._record(other, dh, x, w_gate, w_up, gate, up, dx, dw_gate, dw_up)
    return dx, dw_gate, dw_up


def quantize_fp8(x, group="row", *, dtype=None, stream=None):
    """(q, scale): the matrix x (float32 or bfloat16) as 8-bit floating point
    numbers and float32 scales, q * scale being close to x.

    group: what shares a scale: "row" (128 consecutive elements of a row, scale
    rows x ceil(cols / 128)), "column" (128 of a column, ceil(rows / 128) x
    cols) or "block" (128 x 128, ceil(rows / 128) x ceil(cols / 128)).  dtype:
    torch.float8_e4m3fn (default) or torch.float8_e5m2.

    scale = max(largest |x| / the type's largest value, 2^-126) in float32, and
    q the value nearest to the exact x / scale, ties to even.  q's rows start
    at multiples of 16 bytes, so that gemm_fp8 can read them, as q or as q.t().
    A group with a NaN or an infinity gets a scale that is not finite."""
    torch = _torch or _load()
    code = GROUP.get(group)
    if code is None:
        raise ValueError(f"group must be one of {sorted(GROUP)}")
    fmt = 0
    if dtype is None:
        dtype = torch.float8_e4m3fn
    else:
        fmt = _format(dtype, "dtype")
    if stream is None:
        done = _native.quantize_fp8(x, code, fmt)
        if done is not None:
            return done
    dt = _t._dtype(x, "x")
    if len(x.shape) != 2:
        raise ValueError("x must be a matrix")
    device = x.device
    handle, other = _t._enter(device, stream)
    rows, cols = x.shape
    ldx = _matrix(x, "x")
    q = _new_rows(torch, (rows, cols), dtype, device, 16)
    lds = cols if code == 1 else -(-cols // BLOCK)
    scale = torch.empty((rows if code == 0 else -(-rows // BLOCK), lds), dtype=_f32, device=device)
    _t._call(device, "quantize_fp8", _t._lib().quantize_fp8, rows, cols, x.data_ptr(), ldx, dt, code, fmt,
             q.data_ptr(), _pitch(cols, 16), scale.data_ptr(), lds, handle)
    if other is not None:
        _t._record(other, x, q, scale)
    return q, scale


def _operand(t, name):
    """(pitch, transposed) of a matrix whose rows or columns are contiguous."""
    if len(t.shape) != 2:
        raise ValueError(f"{name} must be a matrix")
    rows, cols = t.shape
    if rows > SIDE_MAX or cols > SIDE_MAX:
        _sides(name, rows, cols)
    if rows == 0 or cols == 0:
        return max(cols, 1), 0
    sr, sc = t.stride()
    if cols == 1 and rows > 1 and sr == 1:
        return _up_to(rows, 16), 1  # one row's transpose
    if (cols == 1 or sc == 1) and (rows == 1 or sr >= cols):
        return (sr if rows > 1 else _up_to(cols, 16)), 0
    if (rows == 1 or sr == 1) and (cols == 1 or sc >= rows):
        return (sc if cols > 1 else _up_to(rows, 16)), 1
    raise ValueError(f"{name} must be row-major or the transpose of a row-major matrix")


def _scales(s, name, device, sides, blocks, along):
    """(elements that share one, stride along the sides, along the blocks) of an
    operand's scales; along: which dimension is the sides'."""
    if s.device != device:
        _at(s, device, name)
    if s.dtype is not _f32:
        raise TypeError(f"{name} must be float32, not {s.dtype}")
    shape = s.shape
    if len(shape) == 2 and shape[1 - along] == blocks:
        stride = s.stride()
        if shape[along] == sides:
            return 1, stride[along], stride[1 - along]
        if shape[along] == -(-sides // BLOCK):
            return BLOCK, stride[along], stride[1 - along]
    want = [(n, blocks) if along == 0 else (blocks, n) for n in (sides, -(-sides // BLOCK))]
    raise ValueError(f"{name} must be {want[0][0]} x {want[0][1]} or {want[1][0]} x {want[1][1]}, not {tuple(shape)}")


def gemm_fp8(A, B, a_scale, b_scale, C=None, *, dtype=None, stream=None):
    """C = A @ B for 8-bit floating point A (M x K) and B (K x N) with a scale
    for every 128 elements along K:

        C_mn = sum over blocks b of 128 of
               a_scale(m, b) * b_scale(b, n) * (A's row m . B's column n in block b)

    A and B: float8_e4m3fn or float8_e5m2, each row-major or the transpose
    (`.t()`) of a row-major matrix, rows in memory at multiples of 16 bytes (as
    quantize_fp8 leaves them).

    a_scale: float32, M x ceil(K / 128), or ceil(M / 128) x ceil(K / 128) where
    128 rows share one.  b_scale: ceil(K / 128) x N, or ceil(K / 128) x
    ceil(N / 128).  Any strides, so the scales of q.t() are scale.t().

    Products within a block are exact and summed in float32, blocks are scaled
    and summed in float32, and C is rounded once.  C: M x N, float32 or
    bfloat16; allocated if None, of `dtype` (default float32), with rows at
    multiples of 16 bytes, so that the next product can read them.  Scales
    whose products with each other or a block's sum leave float32's range give
    infinities or zeros."""
    torch = _torch or _load()
    if C is None and stream is None:
        done = _native.gemm_fp8(A, B, a_scale, b_scale, 0 if dtype is None else _RESULTS.get(dtype, -1))
        if done is not None:
            return done
    device = A.device
    handle, other = _t._enter(device, stream)
    if B.device != device:
        _at(B, device, "B")
    fa, fb = _format(A.dtype, "A"), _format(B.dtype, "B")
    lda, ta = _operand(A, "A")
    ldb, tb = _operand(B, "B")
    M, K = A.shape
    N = B.shape[1]
    if B.shape[0] != K:
        raise ValueError(f"inner dimensions differ: A is {M}x{K}, B is {B.shape[0]}x{N}")
    blocks = -(-K // BLOCK)
    ga, sam, sak = _scales(a_scale, "a_scale", device, M, blocks, 0)
    gb, sbn, sbk = _scales(b_scale, "b_scale", device, N, blocks, 1)
    if C is None:
        dtype = _f32 if dtype is None else dtype
        if dtype is not _f32 and dtype is not _bf16:
            raise TypeError(f"dtype must be float32 or bfloat16, not {dtype}")
        step = 4 if dtype is _f32 else 8
        C = _new_rows(torch, (M, N), dtype, device, step)
        ldc = _pitch(N, step)
    else:
        _at(C, device, "C")
        if tuple(C.shape) != (M, N) or (dtype is not None and C.dtype != dtype):
            raise ValueError(f"C must be a {M} x {N} tensor of the type asked for")
        ldc = _matrix(C, "C")
        _refuse_shared(C, "C", (A, "A"), (B, "B"), (a_scale, "a_scale"), (b_scale, "b_scale"))
    odt = _t._dtype(C, "C")
    _t._call(device, "gemm_fp8", _t._lib().gemm_fp8, M, N, K, A.data_ptr(), lda, fa, ta, a_scale.data_ptr(), sam,
             sak, ga, B.data_ptr(), ldb, fb, tb, b_scale.data_ptr(), sbk, sbn, gb, C.data_ptr(), ldc, odt,
             handle)
    if other is not None:
        _t._record(other, A, B, a_scale, b_scale, C)
    return C
