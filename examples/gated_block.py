"""A pre-norm gated feed-forward block with dropout in the residual stream,
    h = r + dropout1(x),  u = silu(G) U with [G | U] = W1 layernorm(h) + b1,
    y = h + dropout2(W2 u + b2),
on the layer norm, the gated linear layer, the linear layer and dropout: a training step (forward
and every gradient) and 8-bit serving. The masks are drawn from a seed and an offset, and drawn
again in the backward pass.

    python examples/gated_block.py [tokens] [width] [hidden]

prints how far both are from the same block in 64 bits and what a pass takes.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import tile_primitive_tensor_gb300 as tp  # noqa: E402


def make_params(width, hidden, dtype=torch.bfloat16, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)
    return {"gamma": 1 + normal(width, std=0.1), "beta": normal(width, std=0.1),
            "W1": normal(2 * hidden, width, std=width ** -0.5), "b1": normal(2 * hidden, std=0.1),
            "W2": normal(width, hidden, std=hidden ** -0.5), "b2": normal(width, std=0.1)}


def forward(p, x, r, drops):
    """The block's output and what its backward pass needs."""
    n = tp.layernorm(x, p["gamma"], p["beta"], r, dropout=drops[0], need_stats=True)
    pre = torch.empty(x.shape[0], p["W1"].shape[0], dtype=x.dtype, device=x.device)
    u = tp.gated_linear(n.y, p["W1"], p["b1"], pre=pre)
    y = tp.dropout(tp.linear(u, p["W2"], p["b2"]), drops[1], n.h)
    return y, (n, pre, u)


def backward(p, saved, dy, drops):
    """Gradients of x, of r and of every parameter."""
    n, pre, u = saved
    du, dW2, db2 = tp.linear_backward(tp.dropout_backward(dy, drops[1]), u, p["W2"])
    dn, dW1, db1 = tp.gated_linear_backward(du, n.y, p["W1"], pre)
    g = tp.layernorm_backward(dn, n.h, n.mean, n.rstd, p["gamma"], dy, dropout=drops[0])
    return {"x": g.dx, "r": g.dresidual, "gamma": g.dweight, "beta": g.dbias, "W1": dW1, "b1": db1,
            "W2": dW2, "b2": db2}


def quantise_rows(W):
    """e4m3 codes of W's rows and their float32 scales: laid out once, for serving."""
    scale = W.float().abs().amax(1).clamp_min(2.0 ** -126) / 448
    return (W.float() / scale[:, None]).to(torch.float8_e4m3fn), scale


def serve(p, q, x, r):
    """The block without dropout, W1 and the normalised rows in 8 bits; q = quantise_rows(W1)."""
    n = tp.layernorm(x, p["gamma"], p["beta"], r, quant="row")
    u = tp.gated_linear(n.y, q[0], p["b1"], scale_a=n.scale, scale_w=q[1], out_dtype=x.dtype)
    return tp.linear(u, p["W2"], p["b2"], residual=n.h)


def masks(drop, rows, cols):
    """What a dropout multiplies each element by, in 64 bits."""
    return tp.dropout(torch.ones(rows, cols, device="cuda"), drop).double().bool() / (1 - drop.p)


def reference(p, x, r, dy, keep, eps=1e-5):
    """Output and gradients in 64 bits, by torch's own differentiation; keep: the factors of the
    two dropouts."""
    t = {k: v.double().requires_grad_() for k, v in p.items()}
    x64, r64 = x.double().requires_grad_(), r.double().requires_grad_()
    h = r64 + x64 * keep[0]
    d = h - h.mean(1, keepdim=True)
    n = d * torch.rsqrt(d.square().mean(1, keepdim=True) + eps) * t["gamma"] + t["beta"]
    g, u = (n @ t["W1"].T + t["b1"]).chunk(2, 1)
    y = h + (torch.nn.functional.silu(g) * u @ t["W2"].T + t["b2"]) * keep[1]
    y.backward(dy.double())
    return y.detach(), {"x": x64.grad, "r": r64.grad, **{k: v.grad for k, v in t.items()}}


def distance(a, b):
    return float((a.double() - b).norm() / b.norm())


def errors(tokens, width, hidden, seed=0, p_drop=0.1):
    """Relative distances from the 64-bit block: the output, each gradient, and the 8-bit output."""
    p = make_params(width, hidden, seed=seed)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    x, r, dy = [torch.randn(tokens, width, generator=g, device="cuda").bfloat16() for _ in range(3)]
    drops = [tp.Dropout(p_drop, seed, 1), tp.Dropout(p_drop, seed, 2)]
    y, saved = forward(p, x, r, drops)
    grads = backward(p, saved, dy, drops)
    ref, ref_grads = reference(p, x, r, dy, [masks(d, tokens, width) for d in drops])
    plain, _ = reference(p, x, r, dy, [1.0, 1.0])
    e = {"out": distance(y, ref), "served": distance(serve(p, quantise_rows(p["W1"]), x, r), plain)}
    e.update({"d" + k: distance(v, ref_grads[k]) for k, v in grads.items()})
    return e


def main(tokens=1024, width=1024, hidden=4096):
    for name, e in errors(tokens, width, hidden).items():
        print(f"{name:8s} {e:.2e} from 64 bits")
    p = make_params(width, hidden)
    q = quantise_rows(p["W1"])
    x, r = [torch.randn(tokens, width, device="cuda").bfloat16() for _ in range(2)]
    step = torch.zeros(1, dtype=torch.int64, device="cuda")  # moved on from step to step, graphs too
    drops = [tp.Dropout(0.1, 1, step), tp.Dropout(0.1, 2, step)]

    def train():
        y, saved = forward(p, x, r, drops)
        grads = backward(p, saved, y, drops)
        step.add_(1)
        return grads
    for name, run in (("training step", train), ("serving pass", lambda: serve(p, q, x, r))):
        for _ in range(3):
            run()
        begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        torch.cuda.synchronize()
        begin.record()
        for _ in range(20):
            run()
        end.record()
        torch.cuda.synchronize()
        print(f"{name} of {tokens} tokens: {begin.elapsed_time(end) / 20 * 1e3:.1f} us")
    tp.check(tp.tpgemm_last_device_error())


if __name__ == "__main__":
    main(*map(int, sys.argv[1:]))
