"""64-bit statements of the operators around the multiply, and the error bounds that the tests
of their kernels use. Written from the formulas; nothing here comes from the library.

Unit roundoffs: f16 2^-11, bf16 2^-8, f32 2^-24, e4m3 2^-4, e5m2 2^-3. A 32-bit accumulation of K
products, however ordered, in steps of at least 8 products that may truncate, is off by at most
(K / 8 + 64) 2^-23 of the sum of |products|. The hardware exponential is good to 2^-20 relative
over the arguments that matter here, and each activation and its derivative moves by at most 1.2
(second derivative 0.8) per unit of its argument."""
import math

import torch

U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134, torch.float32: 2.0 ** -150}
ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]
FP8 = {torch.float8_e4m3fn: (448.0, 8, -6, 3), torch.float8_e5m2: (57344.0, 15, -14, 2)}


def act(z, name):
    if name == "relu":
        return z.clamp_min(0)
    if name == "silu":
        return z / (1 + torch.exp(-z))
    if name == "gelu":
        return z * 0.5 * torch.erfc(-z / math.sqrt(2))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    return z


def act_grad(z, name):
    if name == "none":
        return torch.ones_like(z)
    if name == "relu":
        return (z > 0).double()
    z = z.detach().clone().requires_grad_(True)
    act(z, name).sum().backward()
    return z.grad


def acc(K):
    return (K / 8 + 64) * 2.0 ** -23


def linear(A, W, bias, residual, name, scale_a, scale_w, out):
    """(y, z, bound of y, bound of z)."""
    a, w = A.double(), W.double()
    if scale_a is not None:
        a = a * scale_a.double()[:, None]
    if scale_w is not None:
        w = w * scale_w.double()[:, None]
    z = a @ w.t()
    s = a.abs() @ w.abs().t()
    if bias is not None:
        z = z + bias.double()
        s = s + bias.double().abs()
    y = act(z, name)
    err = acc(A.shape[1]) * s
    bound_z = err + U[out] * z.abs() + TINY[out]
    r = torch.zeros_like(y) if residual is None else residual.double()
    y = y + r
    bound_y = 1.2 * err + 2.0 ** -19 * (z.abs() + r.abs()) + U[out] * y.abs() + TINY[out]
    return y, z, bound_y, bound_z


def linear_backward(dY, A, W, pre, name, grad):
    """((dA, dW, dbias), their bounds). dA is of A's type, the others of `grad`."""
    dt = A.dtype
    g = act_grad(pre.double(), name) if name != "none" else 1.0
    dz = dY.double() * g
    # act' is evaluated in 32 bits (its terms may cancel, so the error is absolute), and the
    # products read dz rounded to the operands' type.
    err = 2.0 ** -18 * dY.double().abs() * (name not in ("none", "relu"))
    rounded = err + (0 if name == "none" else U[dt]) * dz.abs() + (name != "none") * TINY[dt]
    a, w = A.double(), W.double()
    dA, dW, db = dz @ w, dz.t() @ a, dz.sum(0)
    bA = rounded @ w.abs() + acc(W.shape[0]) * (dz.abs() @ w.abs()) + U[dt] * dA.abs() + TINY[dt]
    bW = (rounded.t() @ a.abs() + acc(A.shape[0]) * (dz.abs().t() @ a.abs()) + U[grad] * dW.abs()
          + TINY[grad])
    bb = err.sum(0) + acc(8 * A.shape[0]) * dz.abs().sum(0) + U[grad] * db.abs() + TINY[grad]
    return (dA, dW, db), (bA, bW, bb)


def rmsnorm(x, weight, residual, eps):
    """(y, h, rstd)."""
    h = x.double() if residual is None else x.double() + residual.double()
    rstd = 1 / torch.sqrt(h.square().mean(1) + eps)
    return h * rstd[:, None] * weight.double(), h, rstd


def rmsnorm_backward(dy, h, rstd, weight, dh):
    """((dx, dweight), their bounds before the outputs' rounding)."""
    dy, h, r, g = dy.double(), h.double(), rstd.double()[:, None], weight.double()
    n, w = h * r, dy * g
    cols = h.shape[1]
    dot = (w * n).sum(1, keepdim=True) / cols
    mag = (w * n).abs().sum(1, keepdim=True) / cols
    dx = r * (w - n * dot)
    # a few roundings per term, and the sum's (any order, in 32 bits)
    bx = 2.0 ** -21 * r * (w.abs() + n.abs() * mag) + acc(8 * cols) * r * n.abs() * mag
    if dh is not None:
        dx = dx + dh.double()
        bx = bx + 2.0 ** -23 * dh.double().abs()
    dg = (dy * n).sum(0)
    bg = acc(8 * h.shape[0]) * (dy * n).abs().sum(0)
    return (dx, dg), (bx, bg)


def decode_mx(codes, scale):
    """Values of 8-bit codes [rows, cols] with E8M0 scales [rows, ceil(cols / 32)]."""
    s = torch.exp2(scale.double() - 127)
    s[scale == 255] = float("nan")
    return codes.double() * s.repeat_interleave(32, 1)[:, : codes.shape[1]]


def quantum(v, kind):
    """Spacing of an 8-bit type's values around v."""
    _, _, emin, bits = FP8[kind]
    e = torch.frexp(v.abs().double())[1].double() - 1
    return torch.exp2(e.clamp_min(emin) - bits)


def within(got, ref, bound):
    """Whether got is within bound of ref everywhere, NaN and infinities in the same places."""
    got = got.double()
    odd = ~torch.isfinite(ref)
    same = torch.where(torch.isnan(ref), torch.isnan(got), got == ref)
    bad = torch.where(odd, ~same, ~((got - ref).abs() <= bound))
    if bad.any():
        i = tuple(int(v) for v in bad.nonzero()[0])
        return False, f"{int(bad.sum())} of {bad.numel()} off, first at {i}: {got[i]} for {ref[i]}"
    return True, ""
