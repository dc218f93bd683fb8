"""The training operators' checks that need no GPU: the C ABI's argument
validation (made before any device is asked) and the binding's refusals."""
import ctypes

import pytest

import async_copy_pipelined_gb300 as pg

INVALID, MISALIGNED = 1, 2


@pytest.fixture(scope="module")
def lib():
    pg.build()
    return pg.lib()


def _forward(lib, rows=4, cols=8, x=256, ldx=8, dtype=0, w=256, b=256, wdtype=0, y=512, ldy=8, mean=1024, rstd=2048,
             eps=1e-5):
    return lib.layer_norm(rows, cols, x, ldx, dtype, w, b, wdtype, y, ldy, mean, rstd, eps, None)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), INVALID), (dict(cols=0), INVALID), (dict(dtype=2), INVALID), (dict(wdtype=-1), INVALID),
    (dict(ldx=7), INVALID), (dict(ldy=7), INVALID), (dict(x=None), INVALID), (dict(y=None), INVALID),
    (dict(mean=None), INVALID), (dict(eps=-1e-5), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(eps=float("inf")), INVALID), (dict(x=258), MISALIGNED), (dict(w=257, wdtype=1), MISALIGNED),
    (dict(y=513, dtype=1), MISALIGNED), (dict(mean=1026), MISALIGNED),
    (dict(cols=(1 << 28) + 1, ldx=1 << 29, ldy=1 << 29), 3),
])
def test_layer_norm_validation(lib, kw, status):
    assert _forward(lib, **kw) == status


def _backward(lib, rows=4, cols=8, dy=256, lddy=8, x=256, ldx=8, dtype=0, mean=1024, rstd=2048, w=256, wdtype=0, dx=512,
              lddx=8, dw=4096, db=8192, ws=16384, ws_bytes=1 << 20):
    return lib.layer_norm_backward(rows, cols, dy, lddy, x, ldx, dtype, mean, rstd, w, wdtype, dx, lddx, dw, db, ws,
                                   ws_bytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), INVALID), (dict(cols=0), INVALID), (dict(dtype=3), INVALID), (dict(lddy=7), INVALID),
    (dict(lddx=7), INVALID), (dict(mean=None), INVALID), (dict(dx=None), INVALID), (dict(ws=None), INVALID),
    (dict(ws_bytes=255), INVALID), (dict(ws=16392), MISALIGNED), (dict(dx=514), MISALIGNED),
    (dict(dw=4097, wdtype=1), MISALIGNED),
])
def test_layer_norm_backward_validation(lib, kw, status):
    assert _backward(lib, **kw) == status


def test_layer_norm_backward_workspace(lib):
    n = ctypes.c_size_t()
    assert lib.layer_norm_backward_workspace(4, 8, ctypes.byref(n)) == 0
    assert n.value >= 4 * 2 * 8 * 4
    assert lib.layer_norm_backward_workspace(-1, 8, ctypes.byref(n)) == INVALID
    assert lib.layer_norm_backward_workspace(4, 0, ctypes.byref(n)) == INVALID
    assert lib.layer_norm_backward_workspace(4, 8, None) == INVALID


def test_host_tensors_are_refused(lib):
    import torch
    x = torch.ones((4, 8))
    with pytest.raises(ValueError, match="CUDA tensors"):
        pg.layer_norm(x)
    with pytest.raises(ValueError, match="CUDA tensors"):
        pg.layer_norm_backward(x, x, torch.ones(4), torch.ones(4))
    with pytest.raises(TypeError):
        pg.layer_norm(x.double())


def _orthogonalize(lib, batch=2, m=8, n=16, G=256, ldg=16, gb=128, dtype=0, out=512, ldo=16, ob=128, odt=0, steps=1,
                   co=(1.5, -0.5, 0.0), eps=1e-7, ws=1024, ws_bytes=1 << 30):
    arr = None if co is None else (ctypes.c_float * len(co))(*co)
    return lib.orthogonalize(batch, m, n, G, ldg, gb, dtype, out, ldo, ob, odt, steps, arr, eps, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(batch=-1), INVALID), (dict(m=-1), INVALID), (dict(n=-5), INVALID), (dict(ldg=15), INVALID),
    (dict(ldo=15), INVALID), (dict(ob=127), INVALID), (dict(gb=-1), INVALID), (dict(G=None), INVALID),
    (dict(out=None), INVALID), (dict(dtype=2), INVALID), (dict(odt=-1), INVALID), (dict(steps=0), INVALID),
    (dict(steps=33), INVALID), (dict(co=None), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(co=(float("inf"), 0.0, 0.0)), INVALID), (dict(co=(3.0, 0.0, 0.0)), 3), (dict(co=(2.0, -1.0, 0.1)), 3),
    (dict(G=257), MISALIGNED), (dict(out=513, odt=1), MISALIGNED), (dict(ws=1040), MISALIGNED),
    (dict(m=1 << 21, n=1), 3), (dict(m=1 << 16, n=1 << 16), 3),
])
def test_orthogonalize_validation(lib, kw, status):
    assert _orthogonalize(lib, **kw) == status


def test_orthogonalize_workspace(lib):
    n = ctypes.c_size_t()
    sizes = []
    for dt in (1, 0):
        assert lib.orthogonalize_workspace(1, 1000, 3000, dt, ctypes.byref(n)) == 0
        sizes.append(n.value)
    # two iterates of two planes, A and Q of one; three and two for float32
    assert sizes[0] > 2 * 2 * 1000 * 3000 * 2 + 2 * 1000 * 1000 * 2
    assert sizes[1] > 2 * 3 * 1000 * 3000 * 2 + 2 * 2 * 1000 * 1000 * 2
    assert lib.orthogonalize_workspace(1, 3000, 1000, 0, ctypes.byref(n)) == 0 and n.value == sizes[1]
    assert lib.orthogonalize_workspace(3, 0, 10, 0, ctypes.byref(n)) == 0 and n.value == 0
    assert lib.orthogonalize_workspace(1, -1, 10, 0, ctypes.byref(n)) == INVALID
    assert lib.orthogonalize_workspace(1, 10, 10, 5, ctypes.byref(n)) == INVALID
    assert lib.orthogonalize_workspace(1, 10, 10, 0, None) == INVALID


def test_orthogonalize_refuses_host_tensors(lib):
    import torch
    with pytest.raises(ValueError, match="CUDA tensors"):
        pg.orthogonalize(torch.ones((4, 8)))


@pytest.mark.parametrize("shape", [(2 ** 32 + 5, 8), (2 ** 31, 1), (3, 2 ** 32 + 8), (2 ** 16, 2 ** 16, 4)])
def test_counts_beyond_a_c_int_are_refused(lib, shape):
    """What ctypes would cut to its lower 32 bits: 2^32 + 5 rows to 5."""
    import torch
    x = torch.empty(shape, dtype=torch.bfloat16, device="meta")
    with pytest.raises(ValueError, match="2\\^31 - 1"):
        pg.layer_norm(x)
    with pytest.raises(ValueError, match="2\\^31 - 1"):
        pg.layer_norm_backward(x, x, x, x)


@pytest.mark.parametrize("shape", [(2 ** 32 + 5, 8), (8, 2 ** 32 + 5), (2 ** 32 + 1, 2, 3)])
def test_sides_beyond_a_c_int_are_refused(lib, shape):
    import torch
    with pytest.raises(ValueError, match="2\\^31 - 1"):
        pg.orthogonalize(torch.empty(shape, device="meta"))


def _bytes_of(view):
    address, batch, m, n, ld, pitch, size = view
    return {address + (b * pitch + i * ld + j) * size + k
            for b in range(batch) for i in range(m) for j in range(n) for k in range(size)}


def test_shared_bytes():
    """Against the sets of bytes: never missed, and siblings told apart."""
    import random

    from async_copy_pipelined_gb300 import training
    rng = random.Random(1)
    found = {True: 0, False: 0}
    for _ in range(4000):
        views = []
        for k in range(2):
            batch, m, n = rng.choice((1, 1, 2, 3)), rng.choice((1, 2, 3, 4)), rng.randint(1, 5)
            ld = n + rng.choice((0, 0, 1, 5, n))
            pitch = rng.choice((ld * m, ld * m + 3, 2 * ld * m, n, 0)) if batch > 1 else ld * (m - 1) + n
            views.append((rng.randint(0, 60) * 2, batch, m, n, ld if m > 1 else n, pitch, rng.choice((2, 4))))
            if k == 1 and rng.random() < 0.6:  # a sibling: the same pitches and type
                views[1] = (views[1][0], *views[0][1:3], min(views[1][3], views[0][4]), *views[0][4:])
        shared = bool(_bytes_of(views[0]) & _bytes_of(views[1]))
        said = training._share_bytes(*views)
        assert said or not shared, views
        found[said] += 1
    assert min(found.values()) > 500
    for other, shared in (((8, 3, 4, 8, 16, 64, 1), False), ((4, 3, 4, 8, 16, 64, 1), True),
                          ((64 * 3, 3, 4, 8, 16, 64, 1), False), ((8, 1, 1, 8, 8, 8, 1), False)):
        assert training._share_bytes((0, 3, 4, 8, 16, 64, 1), other) == shared
    # neighbours in a buffer of matrices side by side, and one after the other
    assert not training._share_bytes((0, 3, 4, 8, 8, 64, 2), (64, 3, 4, 8, 8, 64, 2))
    assert training._share_bytes((0, 3, 4, 8, 8, 64, 2), (62, 3, 4, 8, 8, 64, 2))


@pytest.mark.parametrize("kw,status", [
    (dict(ldo=32, ob=16, eps=-1.0), INVALID), (dict(ldo=32, ob=16, out=514), MISALIGNED),
    (dict(ldo=31, ob=16, out=514), INVALID), (dict(ldo=32, ob=15, out=514), INVALID),
    (dict(batch=3, ldo=47, ob=16, out=514), INVALID), (dict(batch=3, ldo=48, ob=16, out=514), MISALIGNED),
])
def test_orthogonalize_rows_in_turn(lib, kw, status):
    """out's matrices row by row in turn: its pitches are right (the next
    check speaks) unless rows overlap."""
    assert _orthogonalize(lib, **kw) == status


# A schedule of five steps whose first peaks at 1.9917 (Polar Express).
STEEP = (8.28721201814563, -23.595886519098837, 17.300387312530933, 4.107059111542203, -2.9478499167379106,
         0.5448431082926601, 3.9486908534822946, -2.908902115962949, 0.5518191394370137, 3.3184196573706015,
         -2.488488024314874, 0.51004894012372, 2.300652019954817, -1.6689039845747493, 0.4188073119525673)


@pytest.mark.parametrize("steps,co,status", [
    (1, STEEP[:3], MISALIGNED), (5, STEEP, MISALIGNED), (1, (2.79, 0.0, 0.0), MISALIGNED), (1, (2.81, 0.0, 0.0), 3),
    (1, (5.3, -8.0, 4.0), MISALIGNED), (2, (2.7, 0.0, 0.0, 0.3, 0.08, 0.01), 3),
    (2, (2.7, 0.0, 0.0, 0.9, -0.08, 0.01), MISALIGNED),  # x x + b / 2c ends at 11.3 and at 3.3
    (1, (15.6, -42.0, 28.0), 3), (1, (0.0, 0.0, 0.0), MISALIGNED),
])
def test_orthogonalize_coefficients(lib, steps, co, status):
    """Accepted ones come to the next check, of an address."""
    assert _orthogonalize(lib, steps=steps, co=co, out=514) == status
