"""Train one normed projection on synthetic data with the library's operators.

    python examples/train_projection.py [--steps 60] [--width 1024] [--dtype bf16]

The layer is y = layer_norm(x) W.  Each step runs what training it takes:

    xn, mean, rstd = layer_norm(x, gain, shift)     rows normalised
    y              = gemm(xn, W)                    the projection
    dW             = gemm(xn^T, dy)                 its gradients
    dxn            = gemm(dy, W^T)
    dx, dg, ds     = layer_norm_backward(dxn, x, mean, rstd, gain)
    W             -= lr * orthogonalize(momentum)   the weight's update

against a fixed random target layer, and prints the loss.  gain and shift
follow their plain gradients; dx is what a layer below would get.  width and
batch: multiples of 8, as the GEMM's TMA fill asks of a bfloat16 pitch.
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))


def train(steps=60, width=1024, batch=2048, dtype="bf16", lr=0.02, momentum=0.9, seed=0, report=None):
    """Losses of each step, the last one evaluated after the last update."""
    import torch
    import async_copy_pipelined_gb300 as pg

    dt = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
    gemm = {"bf16": pg.gemm_bf16, "f32": pg.gemm_f32}[dtype]
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    target = torch.linalg.qr(randn(width, width))[0].to(dt).contiguous()
    weight = randn(width, width) * width ** -0.5  # float32 master weight
    gain, shift = torch.ones(width, device="cuda"), torch.zeros(width, device="cuda")
    speed = torch.zeros_like(weight)
    losses = []
    for step in range(steps + 1):
        x = (randn(batch, width) * torch.exp(0.5 * randn(batch, 1)) + randn(batch, 1)).to(dt)
        xn, mean, rstd = pg.layer_norm(x, gain, shift, stats=True)
        w = weight.to(dt)
        want = gemm(pg.layer_norm(x), target)
        diff = gemm(xn, w) - want
        losses.append(diff.square().mean())
        if report:
            report(step, losses[-1])
        if step == steps:
            break
        dy = (diff * (2.0 / batch)).to(dt)
        dw = gemm(xn.t().contiguous(), dy)
        dxn = gemm(dy, w.t().contiguous()).to(dt)
        _, dgain, dshift = pg.layer_norm_backward(dxn, x, mean, rstd, gain)
        speed.mul_(momentum).add_(dw)
        weight.add_(pg.orthogonalize(speed, dtype=torch.bfloat16), alpha=-lr * (1 - step / steps))
        gain.add_(dgain, alpha=-lr / width)
        shift.add_(dshift, alpha=-lr / width)
    torch.cuda.synchronize()
    status, detail = pg.device_status()
    if status != 0:
        raise RuntimeError(f"device status {status} ({detail:#x})")
    return [float(v) for v in losses]


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--width", type=int, default=1024)
    ap.add_argument("--batch", type=int, default=2048)
    ap.add_argument("--dtype", choices=("bf16", "f32"), default="bf16")
    args = ap.parse_args(argv)
    train(args.steps, args.width, args.batch, args.dtype,
          report=lambda step, loss: print(f"step {step:4d}  loss {loss.item():.5f}") if step % 10 == 0 else None)


if __name__ == "__main__":
    main()
