"""Newton-Schulz orthogonalisation against float64.

Tolerances, as |got - exact|_F / |exact|_F.  The exact iteration in float64
multiplies a perturbation of the iterate by at most the polynomial's slope in
each direction, so the floor of any arithmetic with unit roundoff u is a small
multiple of u and depends on the spectrum; what the planes keep is u = 2^-11
(one float16 plane) beyond which X's extra plane and the diagonal's carry
eleven bits more.

  bfloat16 result: rounding the exact result alone errs by at most 2^-8 per
  element, in the mean by 2^-8 / sqrt(12) * 1.44 = 0.0017 (uniform mantissas).
  The result must be within 1.3 times that: 0.0022; of fewer than 1024
  elements, whose mean says little, 1.3 times 2^-8.
  float32 result: 2^-22 per product (two planes hold 22 bits), five steps of
  three products and a gain of up to 3.4445 a step on what is lost early: at
  most 5 * 3 * 2^-22 * 3.4445^2 = 4.2e-5 where small singular values are
  present, and 2e-5 for the well-conditioned matrices below."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

TRIPLE = (3.4445, -4.7750, 2.0315)


def _tol(out, x):
    return 4.2e-5 if out == "f32" else 0.0022 if x.numel() >= 1024 else 1.3 * 2.0 ** -8


def _torch_dtype(dtype):
    import torch
    return {"f32": torch.float32, "bf16": torch.bfloat16}[dtype]


def _exact(g, steps=5, coefficients=TRIPLE, eps=1e-7):
    """float64, on the device for speed: g (m x n) as given."""
    x = g.double()
    tall = x.shape[0] > x.shape[1]
    x = x.T if tall else x
    x = x / (x.square().sum().sqrt() + eps)
    for k in range(steps):
        a, b, c = coefficients if not hasattr(coefficients[0], "__len__") else coefficients[k]
        s = x @ x.T
        x = a * x + (b * s + c * (s @ s)) @ x
    return x.T if tall else x


def _rel(got, want):
    d = got.double() - want
    return (d.square().sum().sqrt() / want.square().sum().sqrt()).item()


def _gradient(m, n, kind, seed, scale=1e-3):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((m, n), generator=g, device="cuda")
    if kind == "decay":  # strong directions over a weak floor
        k = max(1, min(m, n) // 8)
        left = torch.randn((m, k), generator=g, device="cuda") * torch.arange(1, k + 1, device="cuda") ** -1.0
        x = 0.05 * x + left @ torch.randn((k, n), generator=g, device="cuda")
    return x * scale


def _check_status():
    import async_copy_pipelined_gb300 as pg
    assert pg.device_status() == (0, 0)


SHAPES = [(1, 1), (1, 7), (9, 1), (2, 3), (8, 8), (17, 33), (64, 64), (65, 63), (128, 128), (129, 127), (100, 300),
          (300, 100), (256, 256), (255, 257), (257, 513), (640, 384), (1000, 1000), (1024, 768), (333, 2100),
          (2100, 333), (1536, 1536), (2056, 3080)]


@pytest.mark.parametrize("m,n", SHAPES)
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16"), ("bf16", "f32")])
def test_against_float64(m, n, dtype, out):
    import async_copy_pipelined_gb300 as pg
    for kind in ("flat", "decay"):
        g = _gradient(m, n, kind, m * 7 + n).to(_torch_dtype(dtype))
        before = g.clone()
        o = pg.orthogonalize(g, dtype=_torch_dtype(out))
        assert o.shape == g.shape and o.dtype == _torch_dtype(out)
        assert (g == before).all()
        assert _rel(o, _exact(g)) <= _tol(out, g), kind
        again = pg.orthogonalize(g, dtype=_torch_dtype(out))
        assert (again == o).all()
    _check_status()


@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_is_orthogonal(out):
    """Singular values of the result lie in 0.68 .. 1.2 and its singular
    vectors are G's: O G^T is symmetric positive."""
    import torch
    import async_copy_pipelined_gb300 as pg
    g = _gradient(200, 500, "flat", 3)
    o = pg.orthogonalize(g, dtype=_torch_dtype(out)).double()
    s = torch.linalg.svdvals(o)
    assert 0.66 < s.min() and s.max() < 1.22
    p = o @ g.double().T
    assert (p - p.T).norm() < 0.01 * p.norm() and torch.linalg.eigvalsh((p + p.T) / 2).min() > 0


@pytest.mark.parametrize("batch,m,n", [(1, 40, 60), (3, 100, 260), (5, 260, 100), (12, 128, 128), (2, 700, 700),
                                       (40, 33, 65)])
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("f32", "f32")])
def test_batch_equals_single_matrices(batch, m, n, dtype, out):
    import torch
    import async_copy_pipelined_gb300 as pg
    g = torch.stack([_gradient(m, n, "decay", 50 + b, scale=10.0 ** (b - 2)) for b in range(batch)])
    g = g.to(_torch_dtype(dtype))
    o = pg.orthogonalize(g, dtype=_torch_dtype(out))
    for b in range(batch):
        assert _rel(o[b], _exact(g[b])) <= _tol(out, g[b])
    _check_status()


@pytest.mark.parametrize("m,n", [(100, 300), (300, 100), (130, 130)])
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("pad,offset", [(0, 1), (3, 0), (8, 8), (5, 3)])
def test_pitches_alignment_and_bounds(m, n, dtype, out, pad, offset):
    """Column slices at any offset, for G and for out; nothing outside out's
    elements is written."""
    import torch
    import async_copy_pipelined_gb300 as pg
    batch = 2

    def slices(values, dt):
        buf = torch.full((offset + batch * m * (n + pad),), 77.0, dtype=dt, device="cuda")
        view = buf[offset:].view(batch, m, n + pad)[:, :, :n]
        if values is not None:
            view.copy_(values)
        return buf, view

    plain = torch.stack([_gradient(m, n, "decay", b) for b in range(batch)]).to(_torch_dtype(dtype))
    want = pg.orthogonalize(plain, dtype=_torch_dtype(out))
    _, g = slices(plain, plain.dtype)
    buf, o = slices(None, _torch_dtype(out))
    assert pg.orthogonalize(g, o) is o
    assert torch.equal(o, want)
    o.fill_(77.0)
    assert (buf == 77.0).all()
    if dtype == out:
        pg.orthogonalize(g, g)  # in place
        assert torch.equal(g, want)
    _check_status()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [1e-30, 1e-12, 1.0, 1e15, 1e25, 1e37])
def test_scale_of_G(dtype, scale):
    """From gradients whose squares vanish in float32 to ones whose squares
    overflow it (eps 0 so that the smallest still count)."""
    import async_copy_pipelined_gb300 as pg
    g = _gradient(96, 160, "flat", 11, scale=1.0).clamp(-3, 3)
    g = (g * scale).to(_torch_dtype(dtype))
    if scale == 1e-30:
        eps = 1e-28  # squares are zero in float32: the norm reads 0, X = G / eps
        want = _exact(g * 0 + g, eps=1e-28)
        got = pg.orthogonalize(g, eps=eps)
        assert got.isfinite().all() and want.isfinite().all()
        return
    got = pg.orthogonalize(g, eps=0.0)
    assert _rel(got, _exact(g, eps=0.0)) <= _tol(dtype, g)


def test_zero_and_non_finite_matrices():
    import torch
    import async_copy_pipelined_gb300 as pg
    g = torch.stack([_gradient(130, 200, "flat", b) for b in range(5)])
    clean = pg.orthogonalize(g)
    g[1] = 0.0
    g[2, 129, 199] = float("nan")
    g[3, 0, 0] = float("inf")
    o = pg.orthogonalize(g)
    assert (o[1] == 0).all() and o[2].isnan().all() and o[3].isnan().all()
    assert torch.equal(o[0], clean[0]) and torch.equal(o[4], clean[4])
    b = pg.orthogonalize(g.bfloat16())
    assert (b[1] == 0).all() and b[2].isnan().all() and b[3].isnan().all() and b[0].isfinite().all()
    zeroed = _gradient(130, 200, "flat", 9)
    zeroed[10:20] = 0.0
    zeroed[:, 50] = 0.0
    z = pg.orthogonalize(zeroed)
    assert (z[10:20] == 0).all() and (z[:, 50] == 0).all() and _rel(z, _exact(zeroed)) <= _tol("f32", zeroed)
    _check_status()


def test_small_singular_values():
    """16 directions at 1 over a floor at 1e-3: what one rounding to eleven
    bits loses would come out hundreds of times larger."""
    import torch
    import async_copy_pipelined_gb300 as pg
    g = torch.Generator(device="cuda").manual_seed(2)
    u = torch.linalg.qr(torch.randn((384, 384), generator=g, device="cuda").double())[0]
    v = torch.linalg.qr(torch.randn((640, 384), generator=g, device="cuda").double())[0]
    s = torch.full((384,), 1e-3, device="cuda", dtype=torch.float64)
    s[:16] = 1.0
    x = ((u * s) @ v.T).float()
    for dt, out in (("bf16", "bf16"), ("f32", "bf16"), ("f32", "f32")):
        gx = x.to(_torch_dtype(dt))
        assert _rel(pg.orthogonalize(gx, dtype=_torch_dtype(out)), _exact(gx)) <= _tol(out, gx), (dt, out)


@pytest.mark.parametrize("steps,coefficients", [
    (1, TRIPLE), (2, TRIPLE), (3, TRIPLE), (9, (1.5, -0.5, 0.0)), (6, (1.875, -1.25, 0.375)), (1, (1.5, -0.5, 0.0)),
    (3, [(3.4445, -4.7750, 2.0315), (1.5, -0.5, 0.0), (1.875, -1.25, 0.375)]), (2, (1.0, 0.0, 0.0)),
])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_steps_and_coefficients(steps, coefficients, out):
    import async_copy_pipelined_gb300 as pg
    for m, n in ((150, 270), (270, 150)):
        g = _gradient(m, n, "decay", steps).to(_torch_dtype(out))
        o = pg.orthogonalize(g, steps=steps, coefficients=coefficients)
        assert _rel(o, _exact(g, steps, coefficients)) <= _tol(out, g)


def test_streams_graphs_and_workspace():
    import torch
    import async_copy_pipelined_gb300 as pg
    g = _gradient(300, 500, "decay", 1).bfloat16()
    want = pg.orthogonalize(g)
    s = torch.cuda.Stream()
    o = pg.orthogonalize(g, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(o, want)
    ws = torch.full((64 << 20,), 255, dtype=torch.uint8, device="cuda")  # float16 NaN everywhere
    assert torch.equal(pg.orthogonalize(g, workspace=ws), want)
    graph = torch.cuda.CUDAGraph()
    static = g.clone()
    with torch.cuda.graph(graph):
        captured = pg.orthogonalize(static, workspace=ws)
    for k in range(3):
        static.copy_(g if k != 1 else g.flip(0))
        graph.replay()
        assert torch.equal(captured, want if k != 1 else pg.orthogonalize(g.flip(0)))
    _check_status()


def test_refusals_on_device():
    import torch
    import async_copy_pipelined_gb300 as pg
    g = _gradient(64, 96, "flat", 1)
    with pytest.raises(TypeError):
        pg.orthogonalize(g.half())
    with pytest.raises(TypeError):
        pg.orthogonalize(g, dtype=torch.float16)
    with pytest.raises(ValueError, match="stack of matrices"):
        pg.orthogonalize(g[0])
    with pytest.raises(ValueError, match="unit column stride"):
        pg.orthogonalize(g.t())
    with pytest.raises(ValueError, match="shape"):
        pg.orthogonalize(g, g[:32])
    with pytest.raises(ValueError, match="one device"):
        pg.orthogonalize(g, torch.empty((64, 96)))
    with pytest.raises(ValueError, match="coefficients"):
        pg.orthogonalize(g, coefficients=[TRIPLE] * 4)
    with pytest.raises(ValueError, match="overlap"):
        pg.orthogonalize(torch.stack([g, g]), torch.empty_like(g).expand(2, 64, 96))
    for kw, status in ((dict(steps=40), 1), (dict(eps=-1.0), 1), (dict(coefficients=(9.0, -8.0, 2.0)), 3),
                       (dict(coefficients=(2.0, -1.0, 0.01)), 3), (dict(coefficients=(float("nan"), 0.0, 0.0)), 1),
                       (dict(workspace=torch.empty(1024, dtype=torch.uint8, device="cuda")), 1)):
        with pytest.raises(pg.GemmError) as e:
            pg.orthogonalize(g, **kw)
        assert e.value.status == status, kw
    empty = pg.orthogonalize(torch.empty((0, 5), device="cuda"))
    assert empty.shape == (0, 5)
    assert pg.orthogonalize(torch.empty((0, 5, 6), device="cuda")).shape == (0, 5, 6)
    torch.cuda.synchronize()
    _check_status()


def test_a_wait_that_runs_out_is_reported():
    """A ring position nothing fills: the kernels give up, say so, and the
    next call is right."""
    import async_copy_pipelined_gb300 as pg
    g = _gradient(200, 300, "flat", 1)
    want = pg.orthogonalize(g)
    _check_status()
    try:
        pg.testing_set_hooks(20_000_000, 1)  # 20 ms
        pg.orthogonalize(g)
    finally:
        pg.testing_set_hooks()
    status, detail = pg.device_status()
    assert status == 6 and detail & 0xFF == 7
    assert (pg.orthogonalize(g) == want).all()
    _check_status()


@pytest.mark.parametrize("m,n", [(128, 128), (128, 256), (127, 257), (100, 511), (512, 90), (65, 700), (64, 1024),
                                 (1025, 64), (120, 1500), (128, 2048), (2048, 128), (128, 2049), (3, 2000), (1, 64),
                                 (1500, 2), (40, 1)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_short_side(m, n, dtype):
    """A side of at most 128: one CTA or a cluster holds the matrix."""
    import torch
    import async_copy_pipelined_gb300 as pg
    for kind in ("flat", "decay"):
        g = torch.stack([_gradient(m, n, kind, m + n + b, scale=10.0 ** (2 * b)) for b in range(3)])
        g = g.to(_torch_dtype(dtype))
        o = pg.orthogonalize(g, dtype=torch.bfloat16)
        for b in range(3):
            assert _rel(o[b], _exact(g[b])) <= _tol("bf16", g[b]), (kind, b)
        assert torch.equal(o, pg.orthogonalize(g, dtype=torch.bfloat16))
    _check_status()


@pytest.mark.parametrize("m,n", [(60, 90), (90, 700), (700, 90)])
def test_a_short_side_in_place_strided_and_not_finite(m, n):
    import torch
    import async_copy_pipelined_gb300 as pg
    g = torch.stack([_gradient(m, n, "flat", b) for b in range(6)]).bfloat16()
    want = pg.orthogonalize(g)
    for pad, offset in ((0, 1), (8, 8), (3, 0)):
        buf = torch.full((offset + 6 * m * (n + pad),), 77.0, dtype=torch.bfloat16, device="cuda")
        view = buf[offset:].view(6, m, n + pad)[:, :, :n]
        view.copy_(g)
        assert torch.equal(pg.orthogonalize(view), want)
        pg.orthogonalize(view, view)
        assert torch.equal(view, want)
        view.fill_(77.0)
        assert (buf == 77.0).all()
    g[1] = 0.0
    g[2, m - 1, n - 1] = float("nan")
    g[4, 0, 0] = float("inf")
    o = pg.orthogonalize(g)
    assert (o[1] == 0).all() and o[2].isnan().all() and o[4].isnan().all()
    assert all(torch.equal(o[k], want[k]) for k in (0, 3, 5))
    _check_status()


@pytest.mark.parametrize("m,n", [(100, 200), (100, 900)])
def test_a_short_side_reports_a_wait_that_runs_out(m, n):
    import torch
    import async_copy_pipelined_gb300 as pg
    g = _gradient(m, n, "flat", 1).bfloat16()
    want = pg.orthogonalize(g)
    try:
        pg.testing_set_hooks(20_000_000, 4)
        pg.orthogonalize(g)
    finally:
        pg.testing_set_hooks()
    status, detail = pg.device_status()
    assert status == 6 and detail & 0xFF == 7
    assert torch.equal(pg.orthogonalize(g), want)
    _check_status()


def test_out_may_be_G_but_not_overlap_it():
    import torch
    import async_copy_pipelined_gb300 as pg
    buf = _gradient(65, 96, "flat", 1).bfloat16()
    with pytest.raises(ValueError, match="overlaps G"):
        pg.orthogonalize(buf[:64], buf[1:])
    want = pg.orthogonalize(buf[:64])
    assert torch.equal(pg.orthogonalize(buf[:64], buf[:64]), want)


def test_a_captured_call_keeps_its_workspace():
    """What a graph works in is the graph's: not the stream's buffer, which a
    larger call replaces and whose memory then goes to other tensors."""
    import torch
    import async_copy_pipelined_gb300 as pg
    g = _gradient(300, 500, "decay", 1).bfloat16()
    x = torch.randn((3000, 1000), device="cuda")
    w = torch.ones(1000, device="cuda")
    _, mean, rstd = pg.layer_norm(x, w, stats=True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        want = pg.orthogonalize(g)
        want_b = pg.layer_norm_backward(x, x, mean, rstd, w)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            captured = pg.orthogonalize(g)
            captured_b = pg.layer_norm_backward(x, x, mean, rstd, w)
        pg.orthogonalize(_gradient(700, 1900, "decay", 1).bfloat16())
        y = torch.randn((3000, 9000), device="cuda")
        _, m2, r2 = pg.layer_norm(y, stats=True)
        pg.layer_norm_backward(y, y, m2, r2, torch.ones(9000, device="cuda"))
        torch.cuda.synchronize()
        others = [torch.full((k << 18,), 7, dtype=torch.uint8, device="cuda") for k in range(1, 40)]
        graph.replay()
        torch.cuda.synchronize()
        assert all((o == 7).all() for o in others)
        assert torch.equal(captured, want)
        assert all(torch.equal(a, b) for a, b in zip(captured_b, want_b))
    _check_status()


def test_two_threads_on_one_stream():
    """Launches of two threads' calls mix on the stream they share; neither
    may work in the other's memory."""
    import threading

    import torch
    import async_copy_pipelined_gb300 as pg
    stream = torch.cuda.Stream()
    work = []
    for seed, (m, n) in ((1, (300, 500)), (2, (300, 500))):
        g = _gradient(m, n, "decay", seed).bfloat16()
        x = torch.randn((3000, 1000), device="cuda")
        w = torch.randn(1000, device="cuda")
        _, mean, rstd = pg.layer_norm(x, w, stats=True)
        work.append((g, x, mean, rstd, w, pg.orthogonalize(g), pg.layer_norm_backward(x, x, mean, rstd, w)))
    torch.cuda.synchronize()
    start, wrong = threading.Barrier(2), []

    def run(g, x, mean, rstd, w, want, want_b):
        with torch.cuda.stream(stream):
            start.wait()
            for _ in range(100):
                got = pg.orthogonalize(g)
                got_b = pg.layer_norm_backward(x, x, mean, rstd, w)
                if not (torch.equal(got, want) and all(torch.equal(a, b) for a, b in zip(got_b, want_b))):
                    wrong.append(threading.get_ident())

    threads = [threading.Thread(target=run, args=a) for a in work]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
    _check_status()


def test_workspaces_are_given_back():
    """What a call works in, 40 MB here, is free for other tensors afterwards;
    the allocator's block for the result may be up to 1 MiB larger than it."""
    import torch
    import async_copy_pipelined_gb300 as pg
    g = _gradient(1000, 2048, "flat", 1)
    with torch.cuda.stream(torch.cuda.Stream()):
        before = torch.cuda.memory_allocated()
        o = pg.orthogonalize(g)
        assert torch.cuda.memory_allocated() - before <= o.numel() * o.element_size() + (1 << 20)
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("m,n", [(96, 160), (130, 500), (300, 140)])
@pytest.mark.parametrize("scale,eps", [(1e-38, 0.0), (1e-36, 1e-37), (1e-30, 1e-28), (1e-30, 0.0), (1e-23, 1e-24),
                                       (1e-20, 0.0), (1e-12, 1e-12), (1e-10, 1e-10)])
def test_a_small_norm(dtype, m, n, scale, eps):
    """Squares that vanish in float32, in part or all of them, still make the
    norm, down to elements that are float32's last denormals."""
    import async_copy_pipelined_gb300 as pg
    g = (_gradient(m, n, "flat", 11, scale=1.0) * scale).to(_torch_dtype(dtype))
    assert _rel(pg.orthogonalize(g, eps=eps), _exact(g, eps=np.float32(eps).item())) <= _tol(dtype, g)
    assert (pg.orthogonalize(g * 0, eps=max(eps, 1e-40)) == 0).all()
    _check_status()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("m,n", [(96, 160), (120, 900), (130, 500), (300, 140), (1000, 700)])
@pytest.mark.parametrize("scale", [1e-9, 3e-11, 1e-12, 1e-15, 1e-20, 1e-28])
@pytest.mark.parametrize("steps,coefficients", [(5, TRIPLE), (1, TRIPLE), (9, (1.5, -0.5, 0.0)),
                                                (12, (1.875, -1.25, 0.375))])
def test_eps_beyond_the_norm(dtype, m, n, scale, steps, coefficients):
    """|G|_F far below eps: X starts at |G|_F / eps, and what the result keeps
    of it is relative to its own size."""
    import async_copy_pipelined_gb300 as pg
    g = (_gradient(m, n, "flat", 12, scale=1.0) * scale).to(_torch_dtype(dtype))
    want = _exact(g, steps, coefficients, eps=np.float32(1e-7).item())
    assert _rel(pg.orthogonalize(g, steps=steps, coefficients=coefficients), want) <= _tol(dtype, g)
    _check_status()


def test_eps_beyond_the_norm_of_some_matrices():
    import torch
    import async_copy_pipelined_gb300 as pg
    for m, n in ((100, 400), (200, 300)):
        g = torch.stack([_gradient(m, n, "decay", b, scale=10.0 ** -(4 * b)) for b in range(5)])
        o = pg.orthogonalize(g)
        for b in range(5):
            assert _rel(o[b], _exact(g[b], eps=np.float32(1e-7).item())) <= _tol("f32", g[b])
            assert torch.equal(o[b], pg.orthogonalize(g[b])) or m > 128  # larger ones may be cut otherwise


@pytest.mark.parametrize("m,n", [(60, 96), (200, 136), (130, 131)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_slice_of_the_same_buffer_may_be_the_output(m, n, dtype):
    """G and out side by side in one buffer: as columns, and as matrices."""
    import torch
    import async_copy_pipelined_gb300 as pg
    g = torch.stack([_gradient(m, n, "flat", b) for b in range(3)]).to(_torch_dtype(dtype))
    want = pg.orthogonalize(g)
    for buf in (torch.full((3, m, 2 * n), 7.0, dtype=g.dtype, device="cuda"),
                torch.full((3, 2 * m, n), 7.0, dtype=g.dtype, device="cuda")):
        columns = buf.shape[2] > n
        G, out = (buf[:, :, :n], buf[:, :, n:]) if columns else (buf[:, :m], buf[:, m:])
        G.copy_(g)
        assert pg.orthogonalize(G, out) is out
        assert torch.equal(out, want) and torch.equal(G, g)
        with pytest.raises(ValueError, match="overlaps G"):
            pg.orthogonalize(G, buf[:, :, 1:n + 1] if columns else buf[:, 1:m + 1])
    _check_status()


@pytest.mark.parametrize("batch,m,n", [(3, 60, 96), (2, 200, 136), (4, 1, 40), (5, 33, 700), (3, 300, 131)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_matrices_row_by_row_in_turn(batch, m, n, dtype):
    """A (m, batch, n) buffer seen as a stack: for G, for out, and in place."""
    import torch
    import async_copy_pipelined_gb300 as pg
    g = torch.stack([_gradient(m, n, "flat", b) for b in range(batch)]).to(_torch_dtype(dtype))
    want = pg.orthogonalize(g)
    buf = torch.full((m, batch, n + 8), 7.0, dtype=g.dtype, device="cuda")
    view = buf[:, :, :n].transpose(0, 1)
    assert torch.equal(pg.orthogonalize(g, view), want)
    assert torch.equal(view, want)
    view.copy_(g)
    assert torch.equal(pg.orthogonalize(view), want)
    pg.orthogonalize(view, view)
    assert torch.equal(view, want)
    view.fill_(7.0)
    assert (buf == 7.0).all()
    _check_status()


def test_a_workspace_with_gaps_or_repeats_is_refused():
    """numel() of a view that is not contiguous says nothing of the memory
    behind its address."""
    import torch
    import async_copy_pipelined_gb300 as pg
    g = _gradient(200, 300, "flat", 1)
    one = torch.empty(256, dtype=torch.uint8, device="cuda")
    for ws in (one.expand(1 << 16, 256), torch.empty((1 << 20, 32), dtype=torch.uint8, device="cuda")[:, :16]):
        with pytest.raises(ValueError, match="contiguous"):
            pg.orthogonalize(g, workspace=ws)
    assert _rel(pg.orthogonalize(g, workspace=torch.empty((1 << 16, 256), dtype=torch.uint8, device="cuda")),
                _exact(g)) <= _tol("f32", g)
    _check_status()


STEEP = [(8.28721201814563, -23.595886519098837, 17.300387312530933),
         (4.107059111542203, -2.9478499167379106, 0.5448431082926601),
         (3.9486908534822946, -2.908902115962949, 0.5518191394370137),
         (3.3184196573706015, -2.488488024314874, 0.51004894012372),
         (2.300652019954817, -1.6689039845747493, 0.4188073119525673)]


@pytest.mark.parametrize("m,n", [(100, 180), (200, 330), (700, 300)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("coefficients", [STEEP, [(2.7, 0.0, 0.0), (1.0, -0.24, 0.03)]])
def test_steps_that_pass_two(m, n, dtype, coefficients):
    """Singular values near 2 and up to 2.7 on the way: a matrix of one strong
    direction, whose value starts at 1, over weak ones."""
    import torch
    import async_copy_pipelined_gb300 as pg
    coefficients = [tuple(float(np.float32(v)) for v in c) for c in coefficients]
    g = _gradient(m, n, "flat", 5, scale=0.02)
    torch.manual_seed(m)
    u, v = (torch.nn.functional.normalize(torch.randn(k, device="cuda"), dim=0) for k in (m, n))
    g = (g + 40.0 * u[:, None] * v).to(_torch_dtype(dtype))
    o = pg.orthogonalize(g, steps=len(coefficients), coefficients=coefficients)
    assert o.isfinite().all()
    assert _rel(o, _exact(g, len(coefficients), coefficients)) <= _tol(dtype, g)
    _check_status()


@pytest.mark.parametrize("m,n", [(1, 50), (20, 30), (64, 64), (100, 300), (128, 1000), (129, 127), (300, 200),
                                 (700, 300), (500, 1500), (1000, 3000), (2100, 900)])
@pytest.mark.parametrize("kind", ["flat", "decay", "spaced"])
def test_float32_results_err_like_float32_arithmetic(m, n, kind):
    """Not only within the bound above, which accumulators added by truncation
    meet too: at most one and a half times as far from float64 as the formula
    in float32 arithmetic, plus 2^-21 for the 22 bits of two planes."""
    import torch
    import async_copy_pipelined_gb300 as pg
    assert torch.get_float32_matmul_precision() == "highest" and not torch.backends.cuda.matmul.allow_tf32
    if kind == "spaced":  # singular values from 1 to 1e-3
        torch.manual_seed(m + n)
        r = min(m, n)
        u, v = (torch.linalg.qr(torch.randn((k, r), device="cuda").double())[0] for k in (m, n))
        g = ((u * torch.logspace(0, -3, r, device="cuda").double()) @ v.T).float()
    else:
        g = _gradient(m, n, kind, m + n)
    want = _exact(g)
    x = g.T if m > n else g
    x = x / (x.square().sum().sqrt() + 1e-7)
    for _ in range(5):
        a, b, c = TRIPLE
        s = x @ x.T
        x = a * x + (b * s + c * (s @ s)) @ x
    plain = _rel(x.T if m > n else x, want)
    assert _rel(pg.orthogonalize(g), want) <= 1.5 * plain + 2.0 ** -21
    _check_status()
