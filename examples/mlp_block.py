"""A pre-norm feed-forward block, h = x + r, out = h + W2 gelu(W1 norm(h) + b1) + b2, on the norm and
the linear layer: a training step (forward and every gradient) and 8-bit serving.

    python examples/mlp_block.py [tokens] [width] [hidden]

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
    return {"gamma": 1 + normal(width, std=0.1), "W1": normal(hidden, width, std=width ** -0.5),
            "b1": normal(hidden, std=0.1), "W2": normal(width, hidden, std=hidden ** -0.5),
            "b2": normal(width, std=0.1)}


def forward(p, x, r):
    """The block's output and what its backward pass needs."""
    n = tp.rmsnorm(x, p["gamma"], r, need_rstd=True)
    pre = torch.empty(x.shape[0], p["W1"].shape[0], dtype=x.dtype, device=x.device)
    u = tp.linear(n.y, p["W1"], p["b1"], act="gelu", pre=pre)
    out = tp.linear(u, p["W2"], p["b2"], residual=n.h)
    return out, (n, pre, u)


def backward(p, saved, dout):
    """Gradients of x (and r) and of every parameter."""
    n, pre, u = saved
    du, dW2, db2 = tp.linear_backward(dout, u, p["W2"])
    dy, dW1, db1 = tp.linear_backward(du, n.y, p["W1"], pre, act="gelu")
    dx, dgamma = tp.rmsnorm_backward(dy, n.h, n.rstd, p["gamma"], dout)
    return {"x": dx, "gamma": dgamma, "W1": dW1, "b1": db1, "W2": dW2, "b2": db2}


def quantise_rows(W):
    """e4m3 codes of W's rows and their float32 scales: laid out once, for serving."""
    scale = W.float().abs().amax(1).clamp_min(2.0 ** -126) / 448
    return (W.float() / scale[:, None]).to(torch.float8_e4m3fn), scale


def serve(p, q, x, r):
    """The block with W1 and the normalised rows in 8 bits; q = quantise_rows(W1)."""
    n = tp.rmsnorm(x, p["gamma"], r, quant="row")
    u = tp.linear(n.y, q[0], p["b1"], act="gelu", scale_a=n.scale, scale_w=q[1], out_dtype=x.dtype)
    return tp.linear(u, p["W2"], p["b2"], residual=n.h)


def reference(p, x, r, dout, eps=1e-6):
    """Output and gradients in 64 bits, by torch's own differentiation."""
    t = {k: v.double().requires_grad_() for k, v in p.items()}
    x64 = x.double().requires_grad_()
    h = x64 + r.double()
    y = h * torch.rsqrt(h.square().mean(1, keepdim=True) + eps) * t["gamma"]
    u = torch.nn.functional.gelu(y @ t["W1"].T + t["b1"])
    out = h + u @ t["W2"].T + t["b2"]
    out.backward(dout.double())
    return out.detach(), {"x": x64.grad, **{k: v.grad for k, v in t.items()}}


def distance(a, b):
    return float((a.double() - b).norm() / b.norm())


def errors(tokens, width, hidden, seed=0):
    """Relative distances from the 64-bit block: the output, each gradient, and the 8-bit output."""
    p = make_params(width, hidden, seed=seed)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    x, r, dout = [torch.randn(tokens, width, generator=g, device="cuda").bfloat16() for _ in range(3)]
    out, saved = forward(p, x, r)
    grads = backward(p, saved, dout)
    ref, ref_grads = reference(p, x, r, dout)
    e = {"out": distance(out, ref), "served": distance(serve(p, quantise_rows(p["W1"]), x, r), ref)}
    e.update({"d" + k: distance(v, ref_grads[k]) for k, v in grads.items()})
    return e


def main(tokens=1024, width=1024, hidden=4096):
    for name, e in errors(tokens, width, hidden).items():
        print(f"{name:8s} {e:.2e} from 64 bits")
    p = make_params(width, hidden)
    q = quantise_rows(p["W1"])
    x, r = [torch.randn(tokens, width, device="cuda").bfloat16() for _ in range(2)]

    def train():
        out, saved = forward(p, x, r)
        return backward(p, saved, out)
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
