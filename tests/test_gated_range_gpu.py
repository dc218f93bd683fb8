"""The gated projection's gradient at gates of any size that bfloat16 holds.

Tolerances: v = 2^-8 for one rounding to bfloat16.  act(gate) and act'(gate) are
off by at most 2^-16 relative in float32 (an exponential's argument of up to 100,
off by half a unit of 100, and some units of the values), and where an activation
has vanished, by at most 1e-12, as 1 + tanh in 64 bits cancels there."""
import pytest

pytestmark = pytest.mark.gpu

V = 2.0 ** -8
ACTS = ("silu", "gelu", "gelu_tanh")


def _act64(g, act):
    """act(g) and act'(g) in 64 bits."""
    import torch
    if act == "silu":
        s = torch.sigmoid(g)
        return g * s, s * (1 + g * (1 - s))
    if act == "gelu":
        c = 0.5 * torch.special.erfc(-g * 0.5 ** 0.5)
        return g * c, c + g * torch.exp(-0.5 * g * g) / (2 * torch.pi) ** 0.5
    k = (2 / torch.pi) ** 0.5
    t = torch.tanh(k * (g + 0.044715 * g ** 3))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * k * (1 + 3 * 0.044715 * g * g)


def _gates():
    """Zero, every power of two from 2^-126 to 2^127 and 1.75 times it, and the
    largest number, of both signs."""
    import torch
    e = torch.arange(-126, 128, dtype=torch.float64)
    g = torch.cat([torch.zeros(1, dtype=torch.float64), 2.0 ** e, 1.75 * 2.0 ** e,
                   torch.tensor([torch.finfo(torch.bfloat16).max], dtype=torch.float64)])
    return torch.cat([g, -g]).to("cuda", torch.bfloat16)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("rows", [1, 3, 200])
def test_gradient_at_gates_of_any_size(act, rows):
    """One row meets the gates; the others' gate is 1.  dh is 2^-10, so that no
    product leaves float32's range."""
    import torch
    import async_copy_pipelined_gb300 as pg
    at, one = rows // 2, torch.ones((), dtype=torch.bfloat16, device="cuda")
    gates = _gates()
    n = gates.numel()
    gate = one.expand(rows, n).clone()
    gate[at] = gates
    up = one.expand(rows, n).clone()
    dh = torch.full_like(up, 2.0 ** -10)
    x = torch.zeros((rows, 16), dtype=torch.bfloat16, device="cuda")
    x[at, 0], x[:, 1] = 1.0, 1.0
    pitch = n + -n % 8
    w_gate, w_up = (torch.zeros((16, pitch), dtype=torch.bfloat16, device="cuda")[:, :n] for _ in range(2))
    w_gate[2] = 2.0 ** -12
    dx, dw_gate, dw_up = pg.gated_projection_backward(dh, x, w_gate, w_up, gate, up, activation=act)
    value, slope = _act64(gate.double(), act)
    dg, du = slope * 2.0 ** -10, value * 2.0 ** -10
    # Row 0 of the weights' gradients is the one row's, once rounded to an operand
    # and once to the result; column 2 of dx sums a row's.
    for got, want, floor in ((dw_gate, dg[at], 1e-6 * 2.0 ** -10), (dw_up, du[at], 1e-12 * 2.0 ** -10)):
        assert got.isfinite().all()
        assert ((got[0].double() - want).abs() <= 1.01 * (2 * V + 2.0 ** -16) * want.abs() + floor).all()
        assert not got[2:].any()
    # Sums over the rows: terms rounded to operands, sums in float32, one rounding more.
    for got, terms in ((dw_gate, dg), (dw_up, du)):
        most, want = terms.abs().sum(0), terms.sum(0)
        bound = V * want.abs() + (V + 2.0 ** -16 + 4 * rows * 2.0 ** -24) * most
        assert ((got[1].double() - want).abs() <= 1.01 * bound + 1e-6 * 2.0 ** -10 * rows).all()
    want, most = dg.sum(1) * 2.0 ** -12, dg.abs().sum(1) * 2.0 ** -12
    bound = V * want.abs() + (V + 2.0 ** -16 + 4 * n * 2.0 ** -24) * most
    assert ((dx[:, 2].double() - want).abs() <= 1.01 * bound + 1e-6 * 2.0 ** -22 * n).all()
    assert not dx[:, 3:].any()
    assert pg.device_status()[0] == 0
