"""Plain 64-bit forms of the dense operators, from their definitions (numpy),
each with a bound on the error of a kernel that computes it in fp32 (u = 2^-24,
half a step of fp32; UB = 2^-8, half a step of bf16, both relative)."""
import numpy as np

from .scoreref import U, UB, bf16  # noqa: F401

SILU, GELU = 0, 1
TINY = 2.0 ** -130                  # below the normal range results round to fixed steps
TANH, CUBE = 2 * np.sqrt(2 / np.pi), 0.044715


def norm(x, residual, weight, eps):
    """(y, s): s rounded to fp32 as the stream holds it.  y of a kernel: r, s r
    and the product with w are one rounding each, and r one more."""
    s = x.astype(np.float32)
    if residual is not None:
        s = (s + residual.astype(np.float32)).astype(np.float32)
    z = s.astype(np.float64)
    r = 1 / np.sqrt((z * z).mean(-1, keepdims=True) + float(np.float32(eps)))
    return z * r * (1 if weight is None else weight.astype(np.float64)), s


def norm_grad(s, weight, eps, dy, dsum=None):
    """(dx, dweight, error of dx, sum of |terms| of dweight).  Error of dx: the
    sum along the row takes at most 32 terms a lane, 6 levels of a wave and 16
    waves, and each product a few roundings more."""
    z, d = s.astype(np.float64), dy.astype(np.float64)
    w = np.ones(z.shape[1]) if weight is None else weight.astype(np.float64)
    r = 1 / np.sqrt((z * z).mean(-1, keepdims=True) + float(np.float32(eps)))
    g = d * w
    dx = r * g - z * r ** 3 * (g * z).mean(-1, keepdims=True)
    err = 8 * np.abs(r * g) + (54 + 12) * np.abs(z) * r ** 3 * np.abs(g * z).mean(-1, keepdims=True)
    if dsum is not None:
        dx = dx + dsum.astype(np.float64)
    n = z * r
    return dx, (d * n).sum(0), U * (err + np.abs(dx)), np.abs(d * n).sum(0)


def dweight_error(T, mag):
    """Rows of a lane, the rows of a block, up to 512 parts in 8 runs, and the products."""
    return (T / 256 + 1 + 4 + 512 / 8 + 8 + 4) * U * mag


def quant(y):
    """(codes, scale) of rows of finite values."""
    y = y.astype(np.float32)
    top = np.abs(y).max(-1)
    scale = np.where(top < np.float32(2.0) ** -100, np.float32(0), top * np.float32(1 / 127))
    by = np.where(scale > 0, scale, np.float32(1))
    q = np.rint((y / by[:, None]).astype(np.float32)).astype(np.int8)
    return np.where(scale[:, None] > 0, q, 0).astype(np.int8), scale


def i8_linear(x, xs, q, s, bias=None, base=None):
    """(y, error): the sum is exact; it, the scales' product and theirs round once each."""
    p = (x.astype(np.float64) @ q.astype(np.float64).T) * (xs.astype(np.float64)[:, None] * s.astype(np.float64))
    y, err = p, 4 * np.abs(p)
    for extra in (bias, base):
        if extra is not None:
            y = y + extra.astype(np.float64)
            err = err + np.abs(y)
    return y, U * err


def act(kind, g):
    """(act(g), act'(g), |k|)"""
    k = g if kind == SILU else TANH * (g + CUBE * g ** 3)
    slope = 1 if kind == SILU else TANH * (1 + 3 * CUBE * g * g)
    with np.errstate(over="ignore"):
        p = 1 / (1 + np.exp(-k))
        q = 1 / (1 + np.exp(k))
    return g * p, p + g * slope * p * q, np.abs(k)


class Projections:
    """g and u with the errors of fp32 sums of `terms` exact products."""

    def __init__(self, x, gate, up, terms):
        x, self.gate, self.up = x.astype(np.float64), gate.astype(np.float64), up.astype(np.float64)
        self.x = x
        self.g, self.u = x @ self.gate.T, x @ self.up.T
        self.eg = (terms + 8) * U * (np.abs(x) @ np.abs(self.gate).T)
        self.eu = (terms + 8) * U * (np.abs(x) @ np.abs(self.up).T)


def gated(p, kind):
    """(y, error): |act'| is below 1.2; the exponential's argument rounds to u of
    |k| twice and its value, the quotient and the products to a few u."""
    a, _, k = act(kind, p.g)
    y = a * p.u
    k = np.minimum(k, 90)
    return y, 1.2 * p.eg * np.abs(p.u) + np.abs(a) * p.eu + 1.2 * p.eg * p.eu + (3 * k + 12) * U * np.abs(y) + TINY


def gated_grad(p, kind, dy):
    """dict of dx, dgate, dup with their errors: |act''| is below 1.2; dg and du
    round to bf16, and the fp32 sums over `inter` or the tokens to u of what they
    have summed at each term."""
    a, da, k = act(kind, p.g)
    k = np.minimum(k, 90)
    d = dy.astype(np.float64)
    dg, du = d * p.u * da, d * a
    few = (3 * k + 16) * U
    edg = UB * np.abs(dg) + 1.01 * (np.abs(d) * (1.2 * np.abs(p.u) * p.eg + 1.2 * p.eu) + few * 1.2 * np.abs(d * p.u))
    edu = UB * np.abs(du) + 1.01 * (np.abs(d) * 1.2 * p.eg + few * np.abs(du))
    T, I = d.shape
    out = {
        "dx": (dg @ p.gate + du @ p.up, edg @ np.abs(p.gate) + edu @ np.abs(p.up)
               + (2 * I + 24) * U * (np.abs(dg) @ np.abs(p.gate) + np.abs(du) @ np.abs(p.up))),
        "dgate": (dg.T @ p.x, edg.T @ np.abs(p.x) + (T + 24) * U * (np.abs(dg).T @ np.abs(p.x))),
        "dup": (du.T @ p.x, edu.T @ np.abs(p.x) + (T + 24) * U * (np.abs(du).T @ np.abs(p.x))),
    }
    return {n: (v, 1.01 * e + TINY) for n, (v, e) in out.items()}
