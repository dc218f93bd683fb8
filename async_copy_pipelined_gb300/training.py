"""Operators around a projection that is being trained (``include/pipelined_train.h``).

    y, mean, rstd = pg.layer_norm(x, weight, bias, stats=True)
    C = pg.gemm_bf16(y, W)                                       # the projection itself
    dx, dweight, dbias = pg.layer_norm_backward(dy, x, mean, rstd, weight)
    update = pg.orthogonalize(momentum, dtype=torch.bfloat16)    # the orthogonalised step for W

Argument checks and marshalling only; the kernels are in the CUDA library.
CUDA tensors in, CUDA tensors out, enqueued on `stream` (default: torch's
current stream) without synchronising.
"""
from __future__ import annotations

import ctypes
import functools

import async_copy_pipelined_gb300 as _pg

__all__ = ["layer_norm", "layer_norm_backward", "orthogonalize"]

F32, BF16 = 0, 1  # enum gemm_dtype
INT_MAX = 0x7FFFFFFF

def bind(l):
    I, L, P, F, S = ctypes.c_int, ctypes.c_longlong, ctypes.c_void_p, ctypes.c_float, ctypes.c_size_t
    l.layer_norm.argtypes = [I, I, P, L, I, P, P, I, P, L, P, P, F, P]
    l.layer_norm.restype = I
    l.layer_norm_backward_workspace.argtypes = [I, I, ctypes.POINTER(S)]
    l.layer_norm_backward_workspace.restype = I
    l.layer_norm_backward.argtypes = [I, I, P, L, P, L, I, P, P, P, I, P, L, P, P, P, S, P]
    l.layer_norm_backward.restype = I
    l.orthogonalize_workspace.argtypes = [I, I, I, I, ctypes.POINTER(S)]
    l.orthogonalize_workspace.restype = I
    l.orthogonalize.argtypes = [I, I, I, P, L, L, I, P, L, L, I, I, ctypes.POINTER(F), F, P, S, P]
    l.orthogonalize.restype = I
    return l


_torch = _short = None
_CODES = {}


def _load():
    """torch, on the first call: importing this package does not import it."""
    global _torch, _short
    if _torch is None:
        import torch
        _short = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        _CODES[torch.float32] = F32
        _CODES[torch.bfloat16] = BF16
        _torch = torch
    return _torch


def _raw_stream(index):
    """The current stream's handle (torch's own short cut to it where it has
    one: building a Stream object takes longer than the launch)."""
    return _short(index) if _short is not None else _torch.cuda.current_stream(index).cuda_stream


def _dtype(t, name):
    code = _CODES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be float32 or bfloat16, not {t.dtype}")
    return code


def _lib():
    """The loaded library (without the lock once it is there)."""
    return _pg._lib or _pg.lib()


def _counts(name, *sizes):
    """Sizes that the library takes as C ints, of which ctypes would silently
    keep the lower 32 bits."""
    for n in sizes:
        if n > INT_MAX:
            raise ValueError(f"{name} has a size of {n}: at most 2^31 - 1")


def _rows(t, name):
    """(rows, cols, pitch) of a tensor seen as rows of its last dimension:
    the rows' elements contiguous, the rows at one common distance."""
    shape = t.shape
    if len(shape) == 0:
        raise ValueError(f"{name} needs at least one dimension")
    cols = shape[-1]
    if cols < 1:
        raise ValueError(f"{name} has empty rows")
    count = t.numel() // cols
    if count > INT_MAX or cols > INT_MAX:
        _counts(name, count, cols)
    if t.is_contiguous():
        return count, cols, cols
    stride = t.stride()
    if cols > 1 and stride[-1] != 1:
        raise ValueError(f"{name} must have unit column stride (row-major rows)")
    rows, pitch, step = 1, cols, None  # step: the distance the next dimension out must have
    for n, d in zip(reversed(shape[:-1]), reversed(stride[:-1])):
        if n == 1:
            continue
        if step is None:
            pitch = d
        elif d != step:
            raise ValueError(f"the rows of {name} must lie at one common distance")
        rows *= n
        step = d * n
    if rows > 1 and pitch < cols:
        raise ValueError(f"the rows of {name} overlap in memory")
    return rows, cols, pitch


def _vector(t, name, n, device):
    """Pointer and type of an n-element parameter vector (None: absent)."""
    if t is None:
        return None
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, x on {device}: all operands must be on one device")
    if t.shape != (n,) or not t.is_contiguous():
        raise ValueError(f"{name} must be {n} contiguous elements")
    return t.data_ptr()


def _share_bytes(a, b):
    """Whether two stacks of matrices may share a byte.  Each: address, then
    matrices, rows, columns, row pitch, matrix pitch and element size.  Views
    of one buffer at the same pitches are told apart by their place within a
    pitch; what this does not show to be apart counts as shared."""
    (pa, na, ma, ca, la, ba, ea), (pb, nb, mb, cb, lb, bb, eb) = a, b
    wide_a, wide_b = ca * ea, cb * eb  # bytes of a row, of a matrix, of all
    tall_a, tall_b = ((ma - 1) * la) * ea + wide_a, ((mb - 1) * lb) * eb + wide_b
    if pa + (na - 1) * ba * ea + tall_a <= pb or pb + (nb - 1) * bb * eb + tall_b <= pa:
        return False

    def apart(pitch, size_a, size_b):
        at = (pb - pa) % pitch
        return at >= size_a and at + size_b <= pitch

    # A single row or matrix fits any pitch.
    if ma == 1 or mb == 1 or la * ea == lb * eb:
        pitch = la * ea if ma > 1 else lb * eb
        whole = all(n == 1 or (d * e) % pitch == 0 for n, d, e in ((na, ba, ea), (nb, bb, eb)))
        if pitch > 0 and whole and apart(pitch, wide_a, wide_b):
            return False
    if na == 1 or nb == 1 or ba * ea == bb * eb:
        pitch = ba * ea if na > 1 else bb * eb
        if (na > 1 or nb > 1) and pitch > 0 and apart(pitch, tall_a, tall_b):
            return False
    return True


def _refuse_overlap(out, out_rows, t, t_rows, name, what):
    """An output may be an input itself, row on row, but not overlap it otherwise."""
    if out_rows[0] == 0:
        return
    if out.data_ptr() == t.data_ptr() and out_rows == t_rows and out.dtype == t.dtype:
        return
    if _share_bytes(*((x.data_ptr(), 1, *rows, 0, x.element_size()) for x, rows in ((out, out_rows), (t, t_rows)))):
        raise ValueError(f"{what} overlaps {name} in memory; it may only be {name} itself")


def _enter(device, stream):
    """The launch stream's handle, and the stream itself where it is another
    than the device's current one (whose allocator order has to be kept)."""
    torch = _torch
    if device.type != "cuda":
        raise ValueError("operands must be CUDA tensors")
    if stream is None:
        return _raw_stream(device.index), None
    cur = torch.cuda.current_stream(device)
    if getattr(stream, "device", device) != device:
        raise ValueError(f"stream belongs to {stream.device}, operands to {device}")
    handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    if handle == cur.cuda_stream:
        return handle, None
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(handle, device=device)
    # What this call allocates may reuse memory that work on the current
    # stream still touches.
    stream.wait_stream(cur)
    return handle, stream


def _record(other, *tensors):
    """Memory used on a stream that is not the current one is not handed out
    again before that stream has passed this point."""
    if other is not None:
        for t in tensors:
            if t is not None:
                t.record_stream(other)


def _call(device, what, fn, *args):
    """A library call with `device` current, and its status checked."""
    if _torch.cuda.current_device() == device.index:
        st = fn(*args)
    else:
        with _torch.cuda.device(device):
            st = fn(*args)
    if st != _pg.GEMM_OK:
        raise _pg.GemmError(st, what)


def _workspace(device, nbytes, other):
    """This call's own buffer, from the launch stream's memory (other None:
    the current stream's).  A call makes several launches, between which
    another thread's may come on the same stream: calls share no buffer.
    Released on return, the memory goes only to work ordered behind them."""
    if other is None:
        return _torch.empty(nbytes, dtype=_torch.uint8, device=device)
    with _torch.cuda.stream(other):
        return _torch.empty(nbytes, dtype=_torch.uint8, device=device)


@functools.lru_cache(maxsize=256)
def _norm_bytes(device, rows, cols):
    """Workspace of layer_norm_backward for these sizes (a pure function of
    them and the device)."""
    need = ctypes.c_size_t()
    _call(device, "layer_norm_backward_workspace", _lib().layer_norm_backward_workspace, rows, cols,
          ctypes.byref(need))
    return need.value


@functools.lru_cache(maxsize=256)
def _orthogonalize_bytes(device, batch, m, n, dtype):
    need = ctypes.c_size_t()
    _call(device, "orthogonalize_workspace", _lib().orthogonalize_workspace, batch, m, n, dtype, ctypes.byref(need))
    return need.value


@functools.lru_cache(maxsize=64)
def _triples(coefficients, steps):
    """coefficients as the library takes them: 3 * steps floats."""
    per_step = coefficients if hasattr(coefficients[0], "__len__") else (coefficients,) * steps
    flat = [float(v) for c in per_step for v in c]
    if len(flat) != 3 * steps or steps < 1:
        raise ValueError("coefficients must be one (a, b, c), or one for each of one or more steps")
    return (ctypes.c_float * len(flat))(*flat)


def layer_norm(x, weight=None, bias=None, out=None, *, eps=1e-5, stats=False, stream=None):
    """Layer norm over the last dimension of x (float32 or bfloat16).

    y = (x - mean) * rstd * weight + bias in float32, rounded once to x's
    type; rstd = 1 / sqrt(var + eps) with the biased variance.  weight and
    bias (each optional) are float32 or bfloat16 vectors, both of one type.
    Rows may lie at any common distance (a column slice of a wider buffer).
    out: where y goes (x itself for an in-place call); allocated if None.

    stats: return (y, mean, rstd) with the rows' float32 statistics, which
    layer_norm_backward takes; otherwise y alone."""
    torch = _load()
    dt = _dtype(x, "x")
    rows, cols, ldx = _rows(x, "x")
    device = x.device
    handle, other = _enter(device, stream)
    pw, pb = _vector(weight, "weight", cols, device), _vector(bias, "bias", cols, device)
    wdt = F32
    if weight is not None:
        wdt = _dtype(weight, "weight")
        if bias is not None and bias.dtype != weight.dtype:
            raise TypeError("weight and bias must have one type")
    elif bias is not None:
        wdt = _dtype(bias, "bias")
    if out is None:
        out = torch.empty_like(x, memory_format=torch.contiguous_format)
        ldy = cols
    else:
        if out.device != device:
            raise ValueError(f"out is on {out.device}, x on {device}: all operands must be on one device")
        if out.shape != x.shape or out.dtype != x.dtype:
            raise ValueError("out must have x's shape and type")
        out_rows = _rows(out, "out")
        _refuse_overlap(out, out_rows, x, (rows, cols, ldx), "x", "out")
        ldy = out_rows[2]
    mean = rstd = pm = pr = None
    if stats:
        shape = x.shape[:-1]
        mean = torch.empty(shape, dtype=torch.float32, device=device)
        rstd = torch.empty(shape, dtype=torch.float32, device=device)
        pm, pr = mean.data_ptr(), rstd.data_ptr()
    _call(device, "layer_norm", _lib().layer_norm, rows, cols, x.data_ptr(), ldx, dt, pw, pb, wdt, out.data_ptr(), ldy,
          pm, pr, eps, handle)
    if other is not None:
        _record(other, x, weight, bias, out, mean, rstd)
    return (out, mean, rstd) if stats else out


def layer_norm_backward(dy, x, mean, rstd, weight=None, out=None, *, bias=None, stream=None):
    """(dx, dweight, dbias) of layer_norm from dy, its input x, the mean and
    rstd it returned, and its weight.

    dx has x's type; dweight and dbias have weight's.  Without a weight
    dweight is None, and dbias too unless bias, the one layer_norm was given,
    says that there is one (its values are not read).  All sums are float32 in an order fixed by the sizes: the
    same inputs give the same bits.  out: where dx goes (dy or x itself for an
    in-place call); allocated if None."""
    torch = _load()
    dt = _dtype(x, "x")
    rows = _rows(x, "x")
    device = x.device
    handle, other = _enter(device, stream)
    if dy.device != device:
        raise ValueError(f"dy is on {dy.device}, x on {device}: all operands must be on one device")
    if dy.shape != x.shape or dy.dtype != x.dtype:
        raise ValueError("dy must have x's shape and type")
    dy_rows = _rows(dy, "dy")
    for name, t in (("mean", mean), ("rstd", rstd)):
        if t.device != device:
            raise ValueError(f"{name} is on {t.device}, x on {device}: all operands must be on one device")
        if t.dtype != torch.float32 or t.numel() != rows[0] or not t.is_contiguous():
            raise ValueError(f"{name} must be {rows[0]} contiguous float32 values")
    pw = _vector(weight, "weight", rows[1], device)
    if out is None:
        out = torch.empty_like(x, memory_format=torch.contiguous_format)
        lddx = rows[1]
    else:
        if out.device != device:
            raise ValueError(f"out is on {out.device}, x on {device}: all operands must be on one device")
        if out.shape != x.shape or out.dtype != x.dtype:
            raise ValueError("out must have x's shape and type")
        out_rows = _rows(out, "out")
        _refuse_overlap(out, out_rows, x, rows, "x", "out")
        _refuse_overlap(out, out_rows, dy, dy_rows, "dy", "out")
        lddx = out_rows[2]
    l = _lib()
    wdt, ws_bytes = F32, 0
    dweight = dbias = ws = pdw = pdb = pws = None
    parameter = weight if weight is not None else bias
    if bias is not None:
        _vector(bias, "bias", rows[1], device)
        if bias.dtype != parameter.dtype:
            raise TypeError("weight and bias must have one type")
    if parameter is not None:
        wdt = _dtype(parameter, "weight" if weight is not None else "bias")
        if weight is not None:
            dweight = torch.empty_like(weight)
            pdw = dweight.data_ptr()
        dbias = torch.empty_like(parameter)
        ws = _workspace(device, _norm_bytes(device, rows[0], rows[1]), other)
        ws_bytes = ws.numel()
        pdb, pws = dbias.data_ptr(), ws.data_ptr()
    _call(device, "layer_norm_backward", l.layer_norm_backward, rows[0], rows[1], dy.data_ptr(), dy_rows[2],
          x.data_ptr(), rows[2], dt, mean.data_ptr(), rstd.data_ptr(), pw, wdt, out.data_ptr(), lddx, pdw, pdb, pws,
          ws_bytes, handle)
    if other is not None:
        _record(other, dy, x, mean, rstd, weight, out, dweight, dbias)
    return out, dweight, dbias


# Singular values from (0, 1] to around 1 in five steps: the quintic of the
# widest use, steep at zero (a = 3.44) at the price of ending within 0.68 .. 1.2.
COEFFICIENTS = (3.4445, -4.7750, 2.0315)


def _matrices(t, name):
    """(batch, m, n, row pitch, matrix pitch) of one matrix or a stack."""
    if t.dim() not in (2, 3):
        raise ValueError(f"{name} must be a matrix or a stack of matrices")
    m, n = t.shape[-2:]
    batch = t.shape[0] if t.dim() == 3 else 1
    _counts(name, batch, m, n)
    if t.numel() == 0:
        return batch, m, n, max(n, 1), max(m * n, 1)
    if n > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name} must have unit column stride (row-major rows)")
    pitch = t.stride(-2) if m > 1 else n
    if pitch < n:
        raise ValueError(f"the rows of {name} overlap in memory")
    return batch, m, n, pitch, t.stride(0) if batch > 1 else pitch * (m - 1) + n


def orthogonalize(G, out=None, *, steps=5, coefficients=COEFFICIENTS, eps=1e-7, dtype=None, workspace="auto",
                  stream=None):
    """The orthogonalised form of a weight's update G, by Newton-Schulz products.

    X <- G / (|G|_F + eps), then `steps` times X <- a X + (b A + c A A) X with
    A = X X^T (on the shorter side of G).  G: one matrix or a stack of them,
    float32 or bfloat16, rows at any pitch.  The result has G's shape and
    `dtype` (default: G's), which also sets the precision of the products: a
    bfloat16 result is within a small part of bfloat16's rounding of the
    exact one, a float32 result what float32 arithmetic gives, at about four
    times the cost.

    coefficients: one (a, b, c) for every step, or `steps` of them.  out:
    where the result goes (G itself for an in-place call).  workspace: "auto"
    allocates one for the call; or a uint8 CUDA tensor of at least
    orthogonalize_workspace() bytes (the C header), which serves one call at
    a time."""
    torch = _load()
    dt = _dtype(G, "G")
    batch, m, n, ldg, g_batch = _matrices(G, "G")
    device = G.device
    handle, other = _enter(device, stream)
    if out is None:
        dtype = G.dtype if dtype is None else dtype
        if dtype not in (torch.float32, torch.bfloat16):
            raise TypeError(f"dtype must be float32 or bfloat16, not {dtype}")
        out = torch.empty(G.shape, dtype=dtype, device=device)
    elif out.device != device:
        raise ValueError(f"out is on {out.device}, G on {device}: all operands must be on one device")
    elif out.shape != G.shape or (dtype is not None and out.dtype != dtype):
        raise ValueError("out must have G's shape and the type asked for")
    odt = _dtype(out, "out")
    _, _, _, ldo, o_batch = _matrices(out, "out")
    if out.numel() and not (out.data_ptr() == G.data_ptr() and odt == dt and (ldo, o_batch) == (ldg, g_batch)):
        if _share_bytes((out.data_ptr(), batch, m, n, ldo, o_batch, out.element_size()),
                        (G.data_ptr(), batch, m, n, ldg, g_batch, G.element_size())):
            raise ValueError("out overlaps G in memory; it may only be G itself")
    if batch > 1 and out.numel() and o_batch < ldo * (m - 1) + n and (o_batch < n or ldo < o_batch * (batch - 1) + n):
        raise ValueError("the matrices of out overlap in memory")
    triples = _triples(tuple(tuple(c) if hasattr(c, "__len__") else c for c in coefficients), steps)
    l = _lib()
    need = _orthogonalize_bytes(device, batch, m, n, odt)
    if isinstance(workspace, str):
        if workspace != "auto":
            raise ValueError('workspace must be "auto" or a uint8 CUDA tensor')
        ws = _workspace(device, need, other)
    else:
        ws = workspace
        if ws.device != device:
            raise ValueError(f"workspace is on {ws.device}, G on {device}")
        if not ws.is_contiguous():
            raise ValueError("workspace must be contiguous")
    _call(device, "orthogonalize", l.orthogonalize, batch, m, n, G.data_ptr(), ldg, g_batch, dt, out.data_ptr(), ldo,
          o_batch, odt, steps, triples, eps, ws.data_ptr(),
          ws.numel() * ws.element_size(), handle)
    if other is not None:
        _record(other, G, out, ws)
    return out
