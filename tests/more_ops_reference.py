"""64-bit statements of the layer norm, dropout and the gated linear layer, and the error bounds that
the tests of their kernels use. Written from the formulas; nothing here comes from the library.

Dropout's words are those of Philox4x32-10 (Salmon et al., 2011), in Python's whole numbers on
numpy; its known answers are checked on the CPU."""
import numpy as np
import torch

import ops_reference as ref

E32 = 2.0 ** -24  # half a step of a 32-bit value, relative


def philox(c0, c1, c2, c3, k0, k1):
    """The four words of counters given as uint64 arrays of 32-bit values."""
    low = np.uint64(0xFFFFFFFF)
    c = [np.asarray(v, dtype=np.uint64) for v in (c0, c1, c2, c3)]
    for i in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        k = [np.uint64((k0 + i * 0x9E3779B9) & 0xFFFFFFFF), np.uint64((k1 + i * 0xBB67AE85) & 0xFFFFFFFF)]
        c = [(b >> np.uint64(32)) ^ c[1] ^ k[0], b & low, (a >> np.uint64(32)) ^ c[3] ^ k[1], a & low]
    return c


def kept(rows, cols, p, seed, offset):
    """The mask [rows, cols] of kept elements, on the CPU."""
    n = -(-cols // 4)
    b, r = np.meshgrid(np.arange(n, dtype=np.uint64), np.arange(rows, dtype=np.uint64))
    o = [np.full_like(b, offset & 0xFFFFFFFF), np.full_like(b, offset >> 32)]
    w = np.stack(philox(b, r, *o, seed & 0xFFFFFFFF, seed >> 32), -1).reshape(rows, 4 * n)[:, :cols]
    return torch.from_numpy(w >= np.uint64(round(p * 2 ** 32)))


def drop(x, numbers):
    """x in 64 bits after dropout, and what the 32-bit result is off by at most: the factor's
    rounding and the product's."""
    if numbers is None or numbers[0] == 0:
        return x.double(), 0 * x.double()
    p, seed, offset = numbers
    keep = kept(x.shape[0], x.shape[1], p, seed, int(offset)).to(x.device)
    y = torch.where(keep, x.double() / (1 - p), torch.zeros((), dtype=torch.float64, device=x.device))
    return y, 2 * E32 * y.abs()


def steps(n):
    """Roundings that one term of a row's 32-bit sum goes through: a thread adds at most 16 terms,
    or n / 1024 of a row that a block of 1024 shares, and a tree joins the threads."""
    return n / 1024 + 32


def layernorm(x, weight, bias, residual, eps, numbers=None):
    """(y, h, mean, rstd) and the bounds of all four before their own roundings."""
    h, eh = drop(x, numbers)
    if residual is not None:
        h = h + residual.double()
        eh = eh + E32 * h.abs()
    n = h.shape[1]
    mean = h.mean(1, keepdim=True)
    d = h - mean
    var = d.square().mean(1, keepdim=True)
    rstd = 1 / torch.sqrt(var + eps)
    y = d * rstd * weight.double() + (0 if bias is None else bias.double())
    a = steps(n) * E32
    # The first mean's error comes back as the mean of h - mean; what stays is the sum's own, of terms
    # as large as d (and that first error, second order), and the mean's last rounding.
    first = a * h.abs().mean(1, keepdim=True)
    emean = eh.mean(1, keepdim=True) + a * (d.abs().mean(1, keepdim=True) + first) + 2 * E32 * mean.abs()
    evar = 2 * (a + 2 * E32) * (var + first.square()) + 2 * (var.sqrt() * eh.square().mean(1, keepdim=True).sqrt())
    rel = 0.5 * evar / (var + eps) + 4 * E32
    w = weight.double().abs()
    # (h - mean, which the second value of the mean corrects: two roundings of d.)
    ey = rstd * w * (eh + emean + 2 * E32 * (d.abs() + first)) + d.abs() * rstd * w * (rel + 3 * E32) + 2 * E32 * y.abs()
    return (y, h, mean[:, 0], rstd[:, 0]), (ey, eh, emean[:, 0], (rel * rstd)[:, 0])


def layernorm_backward(dy, h, mean, rstd, weight, dh, numbers=None):
    """(dx, dresidual, dweight, dbias) and their bounds before the outputs' roundings."""
    dy, h, r = dy.double(), h.double(), rstd.double()[:, None]
    n = (h - mean.double()[:, None]) * r
    w = dy * weight.double()
    cols = h.shape[1]
    m1, m2 = w.mean(1, keepdim=True), (w * n).mean(1, keepdim=True)
    a1, a2 = w.abs().mean(1, keepdim=True), (w * n).abs().mean(1, keepdim=True)
    dt = r * (w - m1 - n * m2)
    a = steps(cols) * E32
    e = r * (8 * E32 * (w.abs() + a1 + n.abs() * a2) + a * (a1 + n.abs() * a2))
    if dh is not None:
        dt = dt + dh.double()
        e = e + 2 * E32 * dh.double().abs()
    e = e + 2 * E32 * dt.abs()
    dx, ex = drop(dt, numbers)
    if numbers is not None and numbers[0] > 0:
        ex = torch.where(dx == 0, 0 * ex, ex + e / (1 - numbers[0]))
    else:
        ex = e
    rows = ref.acc(8 * h.shape[0])
    return ((dx, dt, (dy * n).sum(0), dy.sum(0)),
            (ex, e, (rows + 4 * E32) * (dy * n).abs().sum(0), rows * dy.abs().sum(0)))


def rounded(bound, value, dtype):
    """A bound with the output's own rounding."""
    return bound * (1 + 2.0 ** -7) + ref.U[dtype] * value.abs() + ref.TINY[dtype]


def gated(A, W, bias, name, scale_a, scale_w, out):
    """(y, z, bound of y, bound of z) of Y = act(Z[:, :N]) Z[:, N:]."""
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
    err = ref.acc(A.shape[1]) * s
    g, u = z.chunk(2, 1)
    eg, eu = err.chunk(2, 1)
    f = ref.act(g, name)
    # the activation moves by at most 1.2 of its argument and is good to 2^-19 of it
    ef = 1.2 * eg + 2.0 ** -19 * g.abs()
    y = f * u
    bound = ef * (u.abs() + eu) + f.abs() * eu + 2 * E32 * y.abs()
    return y, z, rounded(bound, y, out), err + ref.U[out] * z.abs() + ref.TINY[out]


def gated_backward(dY, A, W, pre, name, grad):
    """((dA, dW, dbias), their bounds). dA is of A's type, the others of `grad`."""
    dt = A.dtype
    g, u = pre.double().chunk(2, 1)
    dy = dY.double()
    f, df = ref.act(g, name), ref.act_grad(g, name)
    dz = torch.cat([dy * u * df, dy * f], 1)
    # act and act' are evaluated in 32 bits (act' with an absolute error), and the products read dz
    # rounded to the operands' type.
    exact = name in ("none", "relu")
    err = torch.cat([dy.abs() * u.abs() * (0 if exact else 2.0 ** -18),
                     dy.abs() * (0 if exact else 2.0 ** -19) * g.abs()], 1) + 4 * E32 * dz.abs()
    cast = err + ref.U[dt] * dz.abs() + ref.TINY[dt]
    a, w = A.double(), W.double()
    dA, dW, db = dz @ w, dz.t() @ a, dz.sum(0)
    bA = cast @ w.abs() + ref.acc(W.shape[0]) * (dz.abs() @ w.abs())
    bW = cast.t() @ a.abs() + ref.acc(A.shape[0]) * (dz.abs().t() @ a.abs())
    bb = err.sum(0) + ref.acc(8 * A.shape[0]) * dz.abs().sum(0)
    return (dA, dW, db), (rounded(bA, dA, dt), rounded(bW, dW, grad), rounded(bb, db, grad))
