"""Layer norm and its gradient against float64 on the host, at the sizes,
pitches and values where they can go wrong.

Tolerances.  u = 2^-24.  A float32 sum of n terms whose longest chain of
additions is d has an error of at most d u times the sum of the terms'
magnitudes (first order); the kernels' chains over a row are no longer than
n/32 + 16 (a row is shared by at least a warp), over the rows no longer than
rows + 16.  The rest are the roundings of the few operations per element,
counted generously, and the one rounding to the output's type."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
EPS = 1e-5


def _rounding(dtype):
    """Largest relative error of one rounding to nearest: 24 and 8 significant bits."""
    return U if dtype == "f32" else 2.0 ** -8


def _torch_dtype(dtype):
    import torch
    return {"f32": torch.float32, "bf16": torch.bfloat16}[dtype]


def _make(rows, cols, dtype, pad, seed, offset=0, scale=1.0, shift=0.0):
    """rows x cols on the GPU inside a buffer with `pad` more columns and
    `offset` leading elements, and the same values in float64."""
    import torch
    rng = np.random.default_rng(seed)
    pitch = cols + pad
    buf = torch.full((offset + rows * pitch,), float("nan"), dtype=_torch_dtype(dtype))
    view = buf[offset:].view(rows, pitch)[:, :cols]
    view.copy_(torch.from_numpy(rng.standard_normal((rows, cols)) * scale + shift))
    dev = buf.cuda()
    view = dev[offset:].view(rows, pitch)[:, :cols]
    return view, view.double().cpu().numpy(), dev


def _vec(cols, dtype, seed, base):
    import torch
    rng = np.random.default_rng(seed)
    v = torch.from_numpy(base + 0.3 * rng.standard_normal(cols)).to(_torch_dtype(dtype)).cuda()
    return v, v.double().cpu().numpy()


def _forward64(x, w, b, eps=EPS):
    n = x.shape[1]
    mean = x.sum(1) / n
    d = x - mean[:, None]
    rstd = 1.0 / np.sqrt((d * d).sum(1) / n + eps)
    return d * rstd[:, None] * w + b, mean, rstd


def _forward_bounds(x, w, b, dtype, eps=EPS):
    n = x.shape[1]
    d = n / 32 + 16
    y, mean, rstd = _forward64(x, w, b, eps)
    e_mean = d * U * np.abs(x).sum(1) / n
    # var is a sum of squares of differences that carry e_mean and a rounding;
    # e_mean enters var squared, the roundings as relative errors.
    e_diff = e_mean[:, None] + U * np.abs(x - mean[:, None])
    e_var = 2 * np.abs(x - mean[:, None]) * U * np.abs(x - mean[:, None])
    e_var = e_var.sum(1) / n + e_mean ** 2 + (d + 4) * U * (1 / rstd ** 2)
    rel_rstd = 0.5 * e_var * rstd ** 2 + 4 * U
    xhat = (x - mean[:, None]) * rstd[:, None]
    e_y = np.abs(w) * (e_diff * rstd[:, None] + np.abs(xhat) * (rel_rstd[:, None] + 2 * U)) + 2 * U * (
        np.abs(xhat * w) + np.abs(b))
    return y, mean, rstd, e_y * 1.01 + (_rounding(dtype) * 1.01) * np.abs(y) + 1e-38, e_mean * 1.01 + U * np.abs(
        mean) + 1e-38, rel_rstd * 1.01 * rstd


def _close(got, want, bound, what):
    err = np.abs(got - want)
    bad = ~(err <= bound)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst ratio {np.nanmax(err / bound):.3g}"


FORWARD = [
    # rows, cols, dtype, weight dtype, pad, offset
    (1, 1, "f32", "f32", 0, 0), (3, 1, "bf16", "bf16", 0, 0), (1, 2, "bf16", "f32", 0, 0),
    (5, 7, "f32", "f32", 0, 0), (5, 8, "bf16", "bf16", 0, 0), (2, 31, "bf16", "f32", 1, 0),
    (9, 33, "f32", "f32", 3, 1), (4, 64, "bf16", "bf16", 8, 0), (70, 128, "f32", "f32", 0, 0),
    (33, 255, "bf16", "bf16", 0, 1), (17, 256, "bf16", "f32", 0, 0), (300, 264, "bf16", "bf16", 8, 8),
    (64, 512, "f32", "f32", 4, 0), (63, 513, "f32", "f32", 0, 0), (40, 768, "bf16", "bf16", 0, 0),
    (300, 1000, "f32", "f32", 3, 0), (77, 1000, "bf16", "f32", 0, 0), (50, 1023, "bf16", "bf16", 0, 0),
    (50, 1024, "bf16", "bf16", 0, 0), (7, 1025, "bf16", "bf16", 7, 0), (1, 4096, "bf16", "bf16", 0, 0),
    (321, 2048, "f32", "f32", 0, 0), (19, 4104, "bf16", "f32", 0, 0), (610, 4096, "bf16", "bf16", 0, 0),
    (11, 5000, "f32", "f32", 0, 0), (5, 8191, "bf16", "bf16", 0, 0), (160, 8192, "bf16", "f32", 0, 0),
    (3, 16384, "bf16", "bf16", 0, 0), (3, 16384, "f32", "f32", 0, 0), (2, 16385, "f32", "f32", 0, 0),
    (2, 16392, "bf16", "bf16", 0, 0), (2, 50001, "bf16", "f32", 0, 0), (1, 70000, "f32", "f32", 0, 0),
    (3000, 40, "bf16", "f32", 0, 0), (70000, 8, "f32", "f32", 0, 0),
]


@pytest.mark.parametrize("rows,cols,dtype,wdtype,pad,offset", FORWARD)
def test_forward(rows, cols, dtype, wdtype, pad, offset):
    import torch
    import async_copy_pipelined_gb300 as pg
    x, x64, buf = _make(rows, cols, dtype, pad, seed=rows * 131 + cols, offset=offset, scale=1.5, shift=0.7)
    w, w64 = _vec(cols, wdtype, 5, 1.0)
    b, b64 = _vec(cols, wdtype, 6, 0.0)
    before = buf.clone()
    y, mean, rstd = pg.layer_norm(x, w, b, eps=EPS, stats=True)
    assert torch.equal(buf.nan_to_num(9.0), before.nan_to_num(9.0)), "an input was written"
    want, m64, r64, e_y, e_m, e_r = _forward_bounds(x64, w64, b64, dtype)
    assert y.shape == x.shape and y.dtype == x.dtype and mean.shape == (rows,)
    _close(y.double().cpu().numpy(), want, e_y, "y")
    _close(mean.double().cpu().numpy(), m64, e_m, "mean")
    _close(rstd.double().cpu().numpy(), r64, e_r, "rstd")
    # without statistics, without parameters, and in place: the same bits where the same is computed
    assert torch.equal(pg.layer_norm(x, w, b, eps=EPS), y)
    plain = pg.layer_norm(x, eps=EPS)
    want, _, _, e_y, _, _ = _forward_bounds(x64, np.ones(cols), np.zeros(cols), dtype)
    _close(plain.double().cpu().numpy(), want, e_y, "y without parameters")
    inplace = pg.layer_norm(x, w, b, x, eps=EPS)
    assert inplace.data_ptr() == x.data_ptr() and torch.equal(inplace, y)
    tail = buf.clone()
    buf[offset:].view(rows, cols + pad)[:, :cols] = 0
    tail[offset:].view(rows, cols + pad)[:, :cols] = 0
    assert tail[:offset].isnan().all() and tail[offset:].view(rows, cols + pad)[:, cols:].isnan().all()


@pytest.mark.parametrize("only", ["weight", "bias"])
def test_one_parameter_alone(only):
    import async_copy_pipelined_gb300 as pg
    x, x64, _ = _make(9, 300, "f32", 0, seed=3)
    v, v64 = _vec(300, "bf16", 4, 1.0)
    y = pg.layer_norm(x, **{only: v}, eps=EPS)
    w64, b64 = (v64, np.zeros(300)) if only == "weight" else (np.ones(300), v64)
    want, _, _, e_y, _, _ = _forward_bounds(x64, w64, b64, "f32")
    _close(y.double().cpu().numpy(), want, e_y, only)


@pytest.mark.parametrize("cols", [33, 1000, 4096, 20000])
def test_large_mean_small_spread(cols):
    """A mean two thousand times the spread: the variance must not come from
    a difference of two large sums."""
    import async_copy_pipelined_gb300 as pg
    x, x64, _ = _make(6, cols, "f32", 0, seed=cols, scale=0.5, shift=1000.0)
    y = pg.layer_norm(x, eps=EPS)
    want, _, _, e_y, _, _ = _forward_bounds(x64, np.ones(cols), np.zeros(cols), "f32")
    _close(y.double().cpu().numpy(), want, e_y, "y")
    assert e_y.max() < 0.2  # the bound itself still tells a wrong variance


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cols", [8, 1000, 4096, 20000])
def test_constant_rows_and_non_finite_rows(dtype, cols):
    import torch
    import async_copy_pipelined_gb300 as pg
    x = torch.randn((6, cols), device="cuda").to(_torch_dtype(dtype))
    clean = pg.layer_norm(x, eps=EPS)
    x[1] = 3.0  # no spread at all: xhat is zero, rstd 1/sqrt(eps)
    x[2, cols // 2] = float("inf")
    x[3, 0] = float("nan")
    x[4, -1] = float("-inf")
    w, b = torch.full((cols,), 2.0, device="cuda"), torch.full((cols,), 0.5, device="cuda")
    y, mean, rstd = pg.layer_norm(x, w, b, eps=EPS, stats=True)
    assert torch.equal(y[1], torch.full_like(y[1], 0.5))
    assert mean[1] == 3.0 and abs(rstd[1].item() * EPS ** 0.5 - 1) < 1e-6
    for r in (2, 3, 4):
        assert y[r].isnan().all()
    got = pg.layer_norm(x, eps=EPS)
    for r in (0, 5):  # the rows between are not touched by their neighbours
        assert torch.equal(got[r], clean[r])


def _backward64(dy, x, mean, rstd, w):
    n = x.shape[1]
    xhat = (x - mean[:, None]) * rstd[:, None]
    t = dy * w
    c1, c2 = t.sum(1) / n, (t * xhat).sum(1) / n
    dx = rstd[:, None] * (t - c1[:, None] - xhat * c2[:, None])
    return dx, (dy * xhat).sum(0), dy.sum(0)


def _backward_bounds(dy, x, mean, rstd, w, dtype, wdtype):
    rows, n = x.shape
    d = n / 32 + 16
    xhat = (x - mean[:, None]) * rstd[:, None]
    e_xhat = 3 * U * np.abs(xhat)  # difference, product; the difference of two float32 values is rounded once
    t = dy * w
    c1, c2 = t.sum(1) / n, (t * xhat).sum(1) / n
    e_c1 = (d + 3) * U * np.abs(t).sum(1) / n
    e_c2 = ((d + 4) * U * np.abs(t * xhat) + np.abs(t) * e_xhat).sum(1) / n
    dx, dw, db = _backward64(dy, x, mean, rstd, w)
    e_dx = rstd[:, None] * (e_c1[:, None] + np.abs(xhat) * e_c2[:, None] + np.abs(c2)[:, None] * e_xhat +
                            5 * U * (np.abs(t) + np.abs(c1)[:, None] + np.abs(xhat * c2[:, None])))
    e_dx = 1.01 * e_dx + 1.01 * _rounding(dtype) * np.abs(dx) + 1e-38
    e_dw = 1.01 * ((rows + 16) * U * np.abs(dy * xhat).sum(0) + (np.abs(dy) * e_xhat).sum(0))
    e_db = 1.01 * (rows + 16) * U * np.abs(dy).sum(0)
    r = 1.01 * _rounding(wdtype)
    return (dx, dw, db), (e_dx, e_dw + r * np.abs(dw) + 1e-38, e_db + r * np.abs(db) + 1e-38)


BACKWARD = [
    (1, 1, "f32", "f32", 0, 0), (2, 3, "bf16", "bf16", 0, 0), (1, 8, "bf16", "f32", 0, 0),
    (5, 31, "f32", "f32", 2, 1), (40, 64, "bf16", "bf16", 0, 0), (3000, 40, "f32", "f32", 0, 0),
    (33, 255, "bf16", "bf16", 0, 0), (32, 256, "bf16", "f32", 8, 8), (200, 512, "f32", "f32", 0, 0),
    (155, 1000, "f32", "f32", 3, 0), (310, 1000, "bf16", "f32", 0, 0), (32, 1024, "bf16", "bf16", 0, 0),
    (47, 1025, "bf16", "bf16", 0, 0), (700, 2048, "bf16", "f32", 0, 0), (21, 4096, "f32", "f32", 0, 0),
    (330, 4096, "bf16", "bf16", 0, 0), (1, 4096, "bf16", "bf16", 0, 0), (40, 5000, "f32", "f32", 0, 0),
    (9, 8191, "bf16", "f32", 0, 0), (25, 8192, "bf16", "bf16", 0, 0), (7, 16384, "bf16", "f32", 0, 0),
    (5, 16384, "f32", "f32", 0, 0), (3, 16385, "bf16", "bf16", 0, 0), (2, 40000, "f32", "f32", 0, 0),
]


@pytest.mark.parametrize("rows,cols,dtype,wdtype,pad,offset", BACKWARD)
def test_backward(rows, cols, dtype, wdtype, pad, offset):
    import torch
    import async_copy_pipelined_gb300 as pg
    x, x64, _ = _make(rows, cols, dtype, pad, seed=rows + cols, offset=offset, scale=1.3, shift=0.4)
    dy, dy64, _ = _make(rows, cols, dtype, 0, seed=rows + cols + 1, scale=0.01)
    w, w64 = _vec(cols, wdtype, 7, 1.0)
    _, mean, rstd = pg.layer_norm(x, w, None, eps=EPS, stats=True)
    m64, r64 = mean.double().cpu().numpy(), rstd.double().cpu().numpy()
    dx, dw, db = pg.layer_norm_backward(dy, x, mean, rstd, w)
    assert dx.shape == x.shape and dx.dtype == x.dtype and dw.dtype == w.dtype == db.dtype and dw.shape == (cols,)
    want, bound = _backward_bounds(dy64, x64, m64, r64, w64, dtype, wdtype)
    for got, ref, e, what in zip((dx, dw, db), want, bound, ("dx", "dweight", "dbias")):
        _close(got.double().cpu().numpy(), ref, e, what)
    # The same inputs give the same bits; no weight; gradients in place.
    again = pg.layer_norm_backward(dy, x, mean, rstd, w)
    assert all(torch.equal(a, b) for a, b in zip((dx, dw, db), again))
    bare, none_w, none_b = pg.layer_norm_backward(dy, x, mean, rstd)
    assert none_w is None and none_b is None
    want, bound = _backward_bounds(dy64, x64, m64, r64, np.ones(cols), dtype, wdtype)
    _close(bare.double().cpu().numpy(), want[0], bound[0], "dx without weight")
    into_dy = dy.clone()
    r = pg.layer_norm_backward(into_dy, x, mean, rstd, w, into_dy)
    assert r[0].data_ptr() == into_dy.data_ptr()
    assert all(torch.equal(a, b) for a, b in zip((dx, dw, db), r))
    r = pg.layer_norm_backward(dy, x, mean, rstd, w, x)
    assert r[0].data_ptr() == x.data_ptr()
    assert all(torch.equal(a, b) for a, b in zip((dx, dw, db), r))


@pytest.mark.parametrize("rows,cols", [(3, 16), (4, 130), (2, 1000)])
def test_gradient_against_differences(rows, cols):
    """<dx, v>, <dw, v> and <db, v> against central differences of the float64
    layer norm along v.  The differences' own error is what halving the step
    changes, three times over for a second-order formula."""
    import async_copy_pipelined_gb300 as pg
    x, x64, _ = _make(rows, cols, "f32", 0, seed=cols)
    dy, dy64, _ = _make(rows, cols, "f32", 0, seed=cols + 1)
    w, w64 = _vec(cols, "f32", 8, 1.0)
    _, mean, rstd = pg.layer_norm(x, w, None, eps=EPS, stats=True)
    got = [g.double().cpu().numpy() for g in pg.layer_norm_backward(dy, x, mean, rstd, w)]
    _, bound = _backward_bounds(dy64, x64, mean.double().cpu().numpy(), rstd.double().cpu().numpy(), w64, "f32",
                                "f32")
    rng = np.random.default_rng(1)

    def loss(x_, w_, b_):
        return (_forward64(x_, w_, b_)[0] * dy64).sum()

    b0 = np.zeros(cols)
    for k, base in enumerate((x64, w64, b0)):
        v = rng.standard_normal(base.shape)

        def slope(h):
            a = [x64, w64, b0]
            hi, lo = list(a), list(a)
            hi[k], lo[k] = base + h * v, base - h * v
            return (loss(*hi) - loss(*lo)) / (2 * h)

        d1, d2 = slope(2e-4), slope(1e-4)
        # mean and rstd reach the kernel rounded to float32: u of each, through x's gradient
        stats = 4 * U * np.abs(got[0] * v).sum() + 40 * U * np.abs(dy64).sum() if k < 2 else 0.0
        tol = (bound[k] * np.abs(v)).sum() + 3 * abs(d1 - d2) + 1e-9 * (1 + abs(d2)) + stats
        assert abs((got[k] * v).sum() - d2) <= tol, (k, (got[k] * v).sum(), d2, tol)


def test_empty_and_many_dimensions():
    import torch
    import async_copy_pipelined_gb300 as pg
    w = torch.ones(64, device="cuda")
    y, mean, rstd = pg.layer_norm(torch.empty((0, 64), device="cuda"), w, w, stats=True)
    assert y.shape == (0, 64) and mean.shape == (0,)
    dx, dw, db = pg.layer_norm_backward(torch.empty((0, 64), device="cuda"), torch.empty((0, 64), device="cuda"), mean,
                                        rstd, w)
    assert dx.shape == (0, 64) and torch.equal(dw, torch.zeros_like(w)) and torch.equal(db, torch.zeros_like(w))
    x = torch.randn((3, 5, 2, 64), device="cuda")
    y, mean, rstd = pg.layer_norm(x, w, stats=True)
    assert y.shape == x.shape and mean.shape == (3, 5, 2)
    flat = pg.layer_norm(x.view(30, 64), w)
    assert torch.equal(y.view(30, 64), flat)
    dx, _, _ = pg.layer_norm_backward(x, x, mean, rstd, w)
    assert dx.shape == x.shape
    one = pg.layer_norm(x[0, 0, 0], w)
    assert one.shape == (64,) and torch.equal(one, flat[0])
    sliced = x[:, :1, 1]  # 3 x 1 x 64 with one common distance between its rows
    assert torch.equal(pg.layer_norm(sliced, w), y[:, :1, 1])


def test_another_stream_and_a_captured_graph():
    import torch
    import async_copy_pipelined_gb300 as pg
    x = torch.randn((500, 4096), device="cuda")
    dy = torch.randn((500, 4096), device="cuda")
    w = torch.randn(4096, device="cuda")
    want, mean, rstd = pg.layer_norm(x, w, stats=True)
    want_b = pg.layer_norm_backward(dy, x, mean, rstd, w)
    s = torch.cuda.Stream()
    y = pg.layer_norm(x, w, stream=s)
    got_b = pg.layer_norm_backward(dy, x, mean, rstd, w, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(y, want) and all(torch.equal(a, b) for a, b in zip(want_b, got_b))
    g = torch.cuda.CUDAGraph()
    x2, dy2 = x.clone(), dy.clone()
    with torch.cuda.graph(g):
        y2, m2, r2 = pg.layer_norm(x2, w, stats=True)
        b2 = pg.layer_norm_backward(dy2, x2, m2, r2, w)
    for _ in range(2):
        x2.copy_(x.flip(0))
        dy2.copy_(dy.flip(0))
        g.replay()
        assert torch.equal(y2, want.flip(0)) and torch.equal(b2[0], want_b[0].flip(0))
        x2.copy_(x)
        dy2.copy_(dy)
        g.replay()
        assert torch.equal(y2, want) and all(torch.equal(a, b) for a, b in zip(want_b, b2))


def test_refusals_on_device():
    import torch
    import async_copy_pipelined_gb300 as pg
    x = torch.randn((8, 64), device="cuda")
    w = torch.ones(64, device="cuda")
    _, mean, rstd = pg.layer_norm(x, w, stats=True)
    with pytest.raises(TypeError):
        pg.layer_norm(x.half(), w)
    with pytest.raises(TypeError):
        pg.layer_norm(x, w, w.bfloat16())
    with pytest.raises(ValueError, match="64 contiguous"):
        pg.layer_norm(x, torch.ones(63, device="cuda"))
    with pytest.raises(ValueError, match="one device"):
        pg.layer_norm(x, w.cpu())
    with pytest.raises(ValueError, match="unit column stride"):
        pg.layer_norm(x.t())
    with pytest.raises(ValueError, match="overlap"):
        pg.layer_norm(x[:1].expand(8, 64))
    buf = torch.zeros(9 * 64, device="cuda")
    with pytest.raises(ValueError, match="overlaps x"):
        pg.layer_norm(buf[:512].view(8, 64), w, None, buf[64:].view(8, 64))
    with pytest.raises(ValueError, match="shape and type"):
        pg.layer_norm(x, w, None, x.bfloat16())
    with pytest.raises(pg.GemmError) as e:
        pg.layer_norm(x, w, eps=-1.0)
    assert e.value.status == 1
    with pytest.raises(ValueError, match="dy must"):
        pg.layer_norm_backward(x[:7], x, mean, rstd, w)
    with pytest.raises(ValueError, match="mean must"):
        pg.layer_norm_backward(x, x, mean[:7], rstd, w)
    with pytest.raises(ValueError, match="overlaps dy"):
        pg.layer_norm_backward(buf[:512].view(8, 64), x, mean, rstd, w, buf[64:].view(8, 64))
    with pytest.raises(ValueError, match="empty rows"):
        pg.layer_norm(torch.empty((3, 0), device="cuda"))
    torch.cuda.synchronize()
    assert pg.device_status() == (0, 0)


# Enough rows that every CTA's groups take several in turn: the rows come
# through shared memory, as whole vectors, as rows without a rest, or shifted
# where pitch or base is not 16-byte aligned.
MANY = [
    # rows, cols, dtype, weight dtype, pad, offset
    (5200, 512, "bf16", "bf16", 0, 0), (9000, 264, "f32", "f32", 0, 0), (4000, 1024, "bf16", "f32", 0, 0),
    (8000, 1000, "bf16", "bf16", 0, 0), (5000, 1001, "bf16", "f32", 0, 0), (5000, 999, "f32", "bf16", 0, 1),
    (2600, 1024, "bf16", "bf16", 1, 3), (1300, 4096, "bf16", "f32", 0, 0), (1300, 4096, "f32", "f32", 8, 4),
    (1300, 4100, "f32", "f32", 0, 0), (1500, 4097, "bf16", "bf16", 0, 0), (700, 8192, "bf16", "bf16", 0, 0),
    (650, 8200, "bf16", "f32", 0, 0), (620, 8192, "f32", "f32", 0, 0), (640, 5003, "f32", "f32", 2, 1),
    (320, 16384, "bf16", "bf16", 0, 0), (320, 12000, "bf16", "f32", 0, 0), (320, 12000, "f32", "f32", 0, 0),
    (40000, 7, "bf16", "bf16", 0, 1), (20000, 33, "f32", "f32", 0, 0),
]


@pytest.mark.parametrize("rows,cols,dtype,wdtype,pad,offset", MANY)
def test_many_rows_forward(rows, cols, dtype, wdtype, pad, offset):
    test_forward(rows, cols, dtype, wdtype, pad, offset)


@pytest.mark.parametrize("rows,cols,dtype,wdtype,pad,offset", MANY)
def test_many_rows_backward(rows, cols, dtype, wdtype, pad, offset):
    test_backward(rows, cols, dtype, wdtype, pad, offset)


def test_neighbouring_rows_of_an_unaligned_matrix_stay_apart():
    """Only whole 16-byte granules inside a row are copied ahead: what lies
    between the rows, and before and behind them, is never part of one."""
    import torch
    import async_copy_pipelined_gb300 as pg
    rows, cols, pad = 4000, 1001, 3
    x, x64, buf = _make(rows, cols, "bf16", pad, seed=1, offset=5)  # NaN in the gaps
    y, mean, rstd = pg.layer_norm(x, eps=EPS, stats=True)
    assert y.isfinite().all() and mean.isfinite().all()
    dx, dw, db = pg.layer_norm_backward(x, x, mean, rstd, torch.ones(cols, device="cuda"))
    assert dx.isfinite().all() and dw.isfinite().all() and db.isfinite().all()


def test_a_wait_that_runs_out_is_reported():
    """A row the ring never fills: the kernels give up on it, say so, and the
    next call is right."""
    import torch
    import async_copy_pipelined_gb300 as pg
    x = torch.randn((16000, 1024), device="cuda")
    w = torch.ones(1024, device="cuda")
    want, mean, rstd = pg.layer_norm(x, w, stats=True)
    want_b = pg.layer_norm_backward(x, x, mean, rstd, w)
    assert pg.device_status() == (0, 0)
    for call in (lambda: pg.layer_norm(x, w), lambda: pg.layer_norm_backward(x, x, mean, rstd, w)):
        try:
            pg.testing_set_hooks(20_000_000, 3)  # 20 ms
            call()
        finally:
            pg.testing_set_hooks()
        status, detail = pg.device_status()
        assert status == 6 and detail & 0xFF == 8
    assert torch.equal(pg.layer_norm(x, w), want)
    assert all(torch.equal(a, b) for a, b in zip(pg.layer_norm_backward(x, x, mean, rstd, w), want_b))
    assert pg.device_status() == (0, 0)


# Enough rows for the ring, at pitches that bring every alignment of a row's
# start, and rows that end inside a vector: 1 to 8 groups of threads a CTA.
UNALIGNED = [
    # rows, cols, dtype, weight dtype, pad of x, offset of x, pad and offset of the output
    (9000, 1, "bf16", "f32", 0, 1, 0, 0), (9000, 2, "f32", "f32", 1, 0, 2, 3), (9000, 7, "bf16", "bf16", 2, 3, 0, 0),
    (9000, 8, "bf16", "f32", 1, 0, 0, 0), (9000, 9, "bf16", "f32", 0, 0, 4, 5), (9000, 15, "f32", "f32", 0, 1, 1, 2),
    (9000, 250, "bf16", "bf16", 3, 0, 0, 1), (9000, 257, "bf16", "f32", 0, 0, 0, 0),
    (5200, 513, "bf16", "bf16", 0, 7, 3, 0), (5200, 520, "f32", "f32", 3, 0, 0, 0),
    (5200, 1000, "bf16", "f32", 3, 0, 0, 0), (5200, 1000, "f32", "bf16", 1, 2, 5, 1),
    (1700, 2500, "bf16", "f32", 0, 0, 0, 0), (1700, 2498, "f32", "f32", 0, 0, 1, 0),
    (1300, 4095, "bf16", "bf16", 2, 0, 0, 0), (1300, 4099, "f32", "f32", 2, 0, 0, 0),
    (700, 8191, "bf16", "f32", 1, 0, 0, 3), (700, 8192, "bf16", "f32", 3, 0, 0, 0),
    (700, 8190, "f32", "f32", 0, 1, 1, 0), (400, 12289, "bf16", "f32", 0, 0, 2, 0),
    (400, 9001, "f32", "f32", 0, 0, 0, 0), (400, 16383, "bf16", "bf16", 0, 5, 0, 0),
]


def _guarded(rows, cols, dtype, pad, offset):
    """An output amid guards: the view, and a check that nothing around it was written."""
    import torch
    buf = torch.full((offset + rows * (cols + pad) + 16,), 7.0, dtype=_torch_dtype(dtype), device="cuda")
    view = buf[offset:offset + rows * (cols + pad)].view(rows, cols + pad)

    def check():
        assert (buf[:offset] == 7.0).all() and (view[:, cols:] == 7.0).all() and (buf[-16:] == 7.0).all()

    return view[:, :cols], check


@pytest.mark.parametrize("rows,cols,dtype,wdtype,pad,offset,out_pad,out_offset", UNALIGNED)
def test_unaligned_rows(rows, cols, dtype, wdtype, pad, offset, out_pad, out_offset):
    import torch
    import async_copy_pipelined_gb300 as pg
    x, x64, _ = _make(rows, cols, dtype, pad, seed=rows + 3 * cols, offset=offset, scale=1.2, shift=0.6)
    w, w64 = _vec(cols, wdtype, 5, 1.0)
    b, b64 = _vec(cols, wdtype, 6, 0.0)
    out, check = _guarded(rows, cols, dtype, out_pad, out_offset)
    y, mean, rstd = pg.layer_norm(x, w, b, out, eps=EPS, stats=True)
    check()
    want, m64, r64, e_y, e_m, e_r = _forward_bounds(x64, w64, b64, dtype)
    _close(y.double().cpu().numpy(), want, e_y, "y")
    _close(mean.double().cpu().numpy(), m64, e_m, "mean")
    _close(rstd.double().cpu().numpy(), r64, e_r, "rstd")
    dy, dy64, _ = _make(rows, cols, dtype, 5 - pad, seed=cols, offset=2, scale=0.01)
    m64, r64 = mean.double().cpu().numpy(), rstd.double().cpu().numpy()
    want, bound = _backward_bounds(dy64, x64, m64, r64, w64, dtype, wdtype)
    out, check = _guarded(rows, cols, dtype, out_pad, out_offset)
    got = pg.layer_norm_backward(dy, x, mean, rstd, w, out)
    check()
    for g, ref, e, what in zip(got, want, bound, ("dx", "dweight", "dbias")):
        _close(g.double().cpu().numpy(), ref, e, what)
    # In place, on top of rows whose neighbours share granules: the same bits.
    gx = x.clone(memory_format=torch.preserve_format) if x.is_contiguous() else x
    assert torch.equal(pg.layer_norm_backward(dy, gx, mean, rstd, w, dy)[0], got[0])
    assert torch.equal(pg.layer_norm(x, w, b, x, eps=EPS), y)
    assert pg.device_status() == (0, 0)


def test_a_captured_call_on_a_side_stream_keeps_its_workspace():
    """The launch stream is a branch of the capture: what the capturing stream
    allocates and writes beside it must not be the memory the branch works in."""
    import torch
    import async_copy_pipelined_gb300 as pg
    x = torch.randn((3000, 1000), device="cuda")
    w = torch.ones(1000, device="cuda")
    _, mean, rstd = pg.layer_norm(x, w, stats=True)
    want = pg.layer_norm_backward(x, x, mean, rstd, w)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = pg.layer_norm_backward(x, x, mean, rstd, w, stream=side)
        others = [torch.full((k << 17,), 7, dtype=torch.uint8, device="cuda") for k in range(1, 33)]
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(5):
        graph.replay()
        torch.cuda.synchronize()
        assert all((o == 7).all() for o in others)
        assert all(torch.equal(a, b) for a, b in zip(captured, want))
    assert pg.device_status() == (0, 0)


def test_as_many_rows_as_an_int_counts():
    """2^31 - 1 rows of one element, each its own mean: y is the bias."""
    import torch
    import async_copy_pipelined_gb300 as pg
    rows = 2 ** 31 - 1
    x = torch.full((rows, 1), 5.0, dtype=torch.bfloat16, device="cuda")
    x[-1] = -2.0
    y = pg.layer_norm(x, torch.ones(1, device="cuda"), torch.full((1,), 3.0, device="cuda"), x)
    assert all((part == 3.0).all() for part in y.split(1 << 28))
    assert pg.device_status() == (0, 0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols,gap", [(4, 64, 0), (40, 100, 0), (40, 101, 3), (5000, 512, 0), (5000, 333, 1)])
def test_a_slice_of_the_same_buffer_may_be_the_output(rows, cols, gap, dtype):
    """Column slices side by side share no byte: x, dy and the output in one
    buffer, whose other columns stay as they are."""
    import torch
    import async_copy_pipelined_gb300 as pg
    wide = 3 * (cols + gap)
    buf = torch.full((rows, wide), 9.0, device="cuda").to(_torch_dtype(dtype))
    x, out, dy = (buf[:, k * (cols + gap):k * (cols + gap) + cols] for k in range(3))
    x.copy_(torch.randn((rows, cols), device="cuda"))
    dy.copy_(torch.randn((rows, cols), device="cuda"))
    w = torch.randn(cols, device="cuda")
    want, mean, rstd = pg.layer_norm(x.clone(), w, stats=True)
    want_b = pg.layer_norm_backward(dy.clone(), x.clone(), mean, rstd, w)
    before = buf.clone()
    assert pg.layer_norm(x, w, None, out) is out and torch.equal(out, want)
    got = pg.layer_norm_backward(dy, x, mean, rstd, w, out)
    assert all(torch.equal(a, b) for a, b in zip(got, want_b))
    out.copy_(before[:, cols + gap:2 * cols + gap])
    assert torch.equal(buf, before)
    with pytest.raises(ValueError, match="overlaps x"):
        pg.layer_norm(x, w, None, buf[:, 1:cols + 1])
    assert pg.device_status() == (0, 0)


@pytest.mark.parametrize("rows,cols", [(0, 8), (1, 300), (30, 1000), (400, 1000), (9000, 264), (700, 8200), (3, 20000)])
@pytest.mark.parametrize("dtype,bdtype", [("f32", "f32"), ("bf16", "f32"), ("f32", "bf16")])
def test_the_gradient_of_a_bias_alone(rows, cols, dtype, bdtype):
    """layer_norm takes a bias without a weight, and so does its gradient."""
    import torch
    import async_copy_pipelined_gb300 as pg
    x, x64, _ = _make(rows, cols, dtype, 0, seed=rows + cols)
    dy, dy64, _ = _make(rows, cols, dtype, 0, seed=rows + cols + 1)
    b, _ = _vec(cols, bdtype, 8, 0.0)
    _, mean, rstd = pg.layer_norm(x, None, b, eps=EPS, stats=True)
    dx, dw, db = pg.layer_norm_backward(dy, x, mean, rstd, bias=b)
    assert dw is None and db.dtype == b.dtype and db.shape == b.shape
    m64, r64 = mean.double().cpu().numpy(), rstd.double().cpu().numpy()
    want, bound = _backward_bounds(dy64, x64, m64, r64, np.ones(cols), dtype, bdtype)
    _close(dx.double().cpu().numpy(), want[0], bound[0], "dx")
    _close(db.double().cpu().numpy(), want[2], bound[2], "dbias")
    assert torch.equal(dx, pg.layer_norm_backward(dy, x, mean, rstd)[0])
    w, _ = _vec(cols, bdtype, 9, 1.0)
    both = pg.layer_norm_backward(dy, x, mean, rstd, w, bias=b)
    assert all(torch.equal(p, q) for p, q in zip(both, pg.layer_norm_backward(dy, x, mean, rstd, w)))
    with pytest.raises(TypeError):
        pg.layer_norm_backward(dy, x, mean, rstd, w, bias=b.half())
    with pytest.raises(ValueError, match="bias must be"):
        pg.layer_norm_backward(dy, x, mean, rstd, bias=torch.ones(cols + 1, device="cuda"))
    assert pg.device_status() == (0, 0)


# Rows on both sides of where a gradient leaves its one CTA.
FEW = [(r * g, c) for c, g in ((1, 16), (64, 16), (500, 16), (513, 8), (1024, 8), (1025, 5), (2048, 4), (5000, 1),
                               (8192, 1), (8193, 1), (16384, 1)) for r in (1, 2, 3, 4, 5)]


@pytest.mark.parametrize("rows,cols", FEW)
@pytest.mark.parametrize("dtype,pad", [("f32", 0), ("bf16", 0), ("bf16", 3)])
def test_few_rows_backward(rows, cols, dtype, pad):
    test_backward(rows, cols, dtype, "f32", pad, 0)
