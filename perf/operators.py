"""What the training operators beside the GEMM are measured on.

Three operators around a projection C = A·B that is being trained:

  layer_norm            y = (x - mean) * rstd * weight + bias, row by row: what
                        feeds the projection, for a whole batch of tokens or
                        for a single one.
  layer_norm_backward   dx, dweight and dbias from dy: what the projection's
                        input gradient goes through.
  orthogonalize         the Newton-Schulz iteration X <- a X + (b A + c A A) X
                        with A = X X^T, started from G / (|G|_F + eps): the
                        orthogonalised update of the projection's weight.

`own` False: the plain form, elementary torch operations in 32 bits, rounded
once at the end.  `own` True: the calls a user makes of the library.  Both
take what prepare() returns.  exact() gives the same outputs from the
definition in 64 bits.
"""
import math

import torch

own = False

LN_EPS = 1e-5
NS_EPS = 1e-7
NS_STEPS = 5
NS_COEFFICIENTS = (3.4445, -4.7750, 2.0315)

_DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def _norm(name, op, rows, cols, dtype, weight_dtype, pad=0, stats=True):
    """pad: elements between the end of a row of x and the start of the next
    (a column slice of a wider buffer)."""
    return {"name": name, "op": op, "rows": rows, "cols": cols, "dtype": dtype, "weight_dtype": weight_dtype,
            "pad": pad, "stats": stats}


def _orth(name, batch, m, n, dtype, out_dtype):
    return {"name": name, "op": "orthogonalize", "batch": batch, "m": m, "n": n, "dtype": dtype,
            "out_dtype": out_dtype}


def listed():
    return [
        # One token of a model being sampled: pure latency, no statistics kept.
        _norm("norm token", "layer_norm", 1, 4096, "bf16", "bf16", stats=False),
        # A small float32 batch of ragged rows cut out of a wider buffer.
        _norm("norm ragged f32", "layer_norm", 300, 1000, "f32", "f32", pad=3),
        # A long batch of wide tokens, float32 master weights.
        _norm("norm batch", "layer_norm", 8192, 8192, "bf16", "f32"),
        # A few rows: the gradient of a short sequence.
        _norm("norm backward small", "layer_norm_backward", 32, 1024, "bf16", "bf16"),
        # Ragged float32 rows, not a power of two in either direction.
        _norm("norm backward ragged f32", "layer_norm_backward", 3000, 5000, "f32", "f32"),
        # A training batch: 16384 tokens.
        _norm("norm backward batch", "layer_norm_backward", 16384, 4096, "bf16", "f32"),
        # The weight of one small layer.
        _orth("orthogonalize 256", 1, 256, 256, "bf16", "bf16"),
        # The equal weights of twelve layers, updated together.
        _orth("orthogonalize 12 x 1024", 12, 1024, 1024, "bf16", "bf16"),
        # float32 in and out, ragged and wide.
        _orth("orthogonalize 1000x3000 f32", 1, 1000, 3000, "f32", "f32"),
        # A tall weight whose momentum is kept in float32.
        _orth("orthogonalize 5000x1000", 1, 5000, 1000, "f32", "bf16"),
        # An ordinary square projection.
        _orth("orthogonalize 4096", 1, 4096, 4096, "bf16", "bf16"),
        # The largest projection of the benchmark's sizes.
        _orth("orthogonalize 8192", 1, 8192, 8192, "bf16", "bf16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("layer_norm", "layer_norm_backward", "orthogonalize", "orthogonalize"))
    if op == "orthogonalize":
        dtype, out = rng.choice((("bf16", "bf16"), ("bf16", "bf16"), ("f32", "bf16"), ("f32", "f32")))
        m, n = _log_int(rng, 32, 8192), _log_int(rng, 32, 8192)
        if rng.random() < 0.5:  # whole multiples of 64 are as common as odd sizes
            m, n = -(-m // 64) * 64, -(-n // 64) * 64
        case = _orth("", 1, m, n, dtype, out)
        most = int(work(_orth("", 1, 4096, 4096, "bf16", "bf16"))["flops"] / work(case)["flops"])
        case["batch"] = _log_int(rng, 1, max(1, min(16, most)))
    else:
        dtype = rng.choice(("bf16", "f32"))
        cols = _log_int(rng, 64, 16384)
        if rng.random() < 0.6:
            cols = -(-cols // 64) * 64
        rows = _log_int(rng, 1, max(1, min(16384, (1 << 26) // cols)))
        case = _norm("", op, rows, cols, dtype, rng.choice(("f32", dtype)), pad=rng.choice((0, 0, 0, 8, 3)),
                     stats=op == "layer_norm_backward" or rng.random() < 0.7)
    del case["name"]
    return case


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _rows(g, rows, cols, pad, dtype):
    """Activations: rows of different means and spreads, in a buffer with
    `pad` more columns."""
    buf = torch.randn((rows, cols + pad), generator=g, device="cuda")
    buf *= torch.exp(0.5 * torch.randn((rows, 1), generator=g, device="cuda"))
    buf += 0.5 * torch.randn((rows, 1), generator=g, device="cuda")
    return buf.to(_DTYPES[dtype])[:, :cols]


def prepare(case, seed):
    g = _generator(seed)
    if case["op"] == "orthogonalize":
        # A gradient: a few strong directions over a floor of weak ones.
        b, m, n = case["batch"], case["m"], case["n"]
        k = max(1, min(m, n) // 16)
        left = torch.randn((b, m, k), generator=g, device="cuda")
        left *= torch.arange(1, k + 1, device="cuda").float() ** -0.5
        grad = torch.bmm(left, torch.randn((b, k, n), generator=g, device="cuda"))
        grad += 0.1 * torch.randn((b, m, n), generator=g, device="cuda")
        grad *= 1e-3
        grad = grad.to(_DTYPES[case["dtype"]])
        return {"case": case, "G": grad[0] if b == 1 else grad}
    rows, cols, pad, dtype = case["rows"], case["cols"], case["pad"], case["dtype"]
    wdt = _DTYPES[case["weight_dtype"]]
    state = {"case": case, "x": _rows(g, rows, cols, pad, dtype)}
    state["weight"] = (1.0 + 0.1 * torch.randn(cols, generator=g, device="cuda")).to(wdt)
    state["bias"] = (0.1 * torch.randn(cols, generator=g, device="cuda")).to(wdt)
    if case["op"] == "layer_norm_backward":
        # What the forward pass has left: the rows' statistics, in 32 bits.
        xf = state["x"].double()
        mean = xf.mean(1)
        var = (xf - mean[:, None]).square().mean(1)
        state["mean"], state["rstd"] = mean.float(), (var + LN_EPS).rsqrt().float()
        state["dy"] = (1e-2 * torch.randn((rows, cols + pad), generator=g, device="cuda")).to(_DTYPES[dtype])[:, :cols]
    return state


def run(state):
    case = state["case"]
    if own:
        import async_copy_pipelined_gb300 as pg
        if case["op"] == "orthogonalize":
            return pg.orthogonalize(state["G"], steps=NS_STEPS, coefficients=NS_COEFFICIENTS, eps=NS_EPS,
                                    dtype=_DTYPES[case["out_dtype"]])
        if case["op"] == "layer_norm":
            return pg.layer_norm(state["x"], state["weight"], state["bias"], eps=LN_EPS, stats=case["stats"])
        return pg.layer_norm_backward(state["dy"], state["x"], state["mean"], state["rstd"], state["weight"])
    if case["op"] == "orthogonalize":
        return _plain_orthogonalize(state["G"], _DTYPES[case["out_dtype"]])
    if case["op"] == "layer_norm":
        y, mean, rstd = _plain_norm(state["x"], state["weight"], state["bias"])
        return (y, mean, rstd) if case["stats"] else y
    return _plain_norm_backward(state["dy"], state["x"], state["mean"], state["rstd"], state["weight"])


def _plain_norm(x, weight, bias):
    xf = x.float()
    mean = xf.mean(1)
    d = xf - mean[:, None]
    rstd = torch.rsqrt((d * d).mean(1) + LN_EPS)
    y = d * rstd[:, None] * weight.float() + bias.float()
    return y.to(x.dtype), mean, rstd


def _plain_norm_backward(dy, x, mean, rstd, weight):
    g = dy.float()
    xhat = (x.float() - mean[:, None]) * rstd[:, None]
    gw = g * weight.float()
    dx = (gw - gw.mean(1, keepdim=True) - xhat * (gw * xhat).mean(1, keepdim=True)) * rstd[:, None]
    return dx.to(x.dtype), (g * xhat).sum(0).to(weight.dtype), g.sum(0).to(weight.dtype)


def _plain_orthogonalize(grad, out_dtype):
    a, b, c = NS_COEFFICIENTS
    x = grad.float()
    x = x / ((x * x).sum((-2, -1), keepdim=True).sqrt() + NS_EPS)
    tall = x.shape[-2] > x.shape[-1]
    if tall:
        x = x.mT
    for _ in range(NS_STEPS):
        s = x @ x.mT
        x = a * x + (b * s + c * (s @ s)) @ x
    return (x.mT if tall else x).to(out_dtype).contiguous()


def exact(case, seed):
    if case["op"] == "orthogonalize":
        if work(case)["flops"] > 4e12:
            return None  # 64-bit products of this size take too long
        g = prepare(case, seed)["G"].to(torch.float64)
        g = g.reshape(-1, g.shape[-2], g.shape[-1])
        outs = []
        for one in g:
            # p(S) = a I + b S + c S S applied to the shorter side.
            wide = one if one.shape[0] <= one.shape[1] else one.t()
            wide = wide / (torch.linalg.vector_norm(wide) + NS_EPS)
            eye = torch.eye(wide.shape[0], dtype=torch.float64, device=wide.device)
            for _ in range(NS_STEPS):
                gram = torch.mm(wide, wide.t())
                poly = torch.addmm(NS_COEFFICIENTS[1] * gram, gram, gram, alpha=NS_COEFFICIENTS[2])
                wide = torch.mm(poly + NS_COEFFICIENTS[0] * eye, wide)
            outs.append(wide if one.shape[0] <= one.shape[1] else wide.t())
        return outs[0].contiguous() if case["batch"] == 1 else torch.stack(outs)
    s = prepare(case, seed)
    x, w = s["x"].to(torch.float64), s["weight"].to(torch.float64)
    n = case["cols"]
    if case["op"] == "layer_norm":
        mean = torch.sum(x, 1) / n
        rstd = 1.0 / torch.sqrt(torch.sum((x - mean.unsqueeze(1)) ** 2, 1) / n + LN_EPS)
        y = (x - mean.unsqueeze(1)) * rstd.unsqueeze(1) * w.unsqueeze(0) + s["bias"].to(torch.float64).unsqueeze(0)
        return (y, mean, rstd) if case["stats"] else y
    # The gradient takes the saved statistics as given.
    xhat = (x - s["mean"].to(torch.float64).unsqueeze(1)) * s["rstd"].to(torch.float64).unsqueeze(1)
    dy = s["dy"].to(torch.float64)
    t = dy * w.unsqueeze(0)
    c1, c2 = torch.sum(t, 1) / n, torch.sum(t * xhat, 1) / n
    dx = s["rstd"].to(torch.float64).unsqueeze(1) * (t - c1.unsqueeze(1) - xhat * c2.unsqueeze(1))
    return dx, torch.sum(dy * xhat, 0), torch.sum(dy, 0)


def work(case):
    size = {"f32": 4, "bf16": 2}
    if case["op"] == "orthogonalize":
        r, c = sorted((case["m"], case["n"]))
        # Per step X X^T and A A (symmetric: half of each) and one full product.
        flops = NS_STEPS * (r * (r + 1) * c + r * (r + 1) * r + 2 * r * r * c)
        return {"bytes": case["batch"] * r * c * (size[case["dtype"]] + size[case["out_dtype"]]),
                "flops": case["batch"] * flops}
    rows, cols, e, w = case["rows"], case["cols"], size[case["dtype"]], size[case["weight_dtype"]]
    if case["op"] == "layer_norm":
        return {"bytes": rows * cols * 2 * e + cols * 2 * w + (rows * 8 if case["stats"] else 0),
                "flops": rows * cols * 8}
    return {"bytes": rows * cols * 3 * e + cols * 3 * w + rows * 8, "flops": rows * cols * 14}
