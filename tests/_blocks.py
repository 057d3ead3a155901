"""Plain 64-bit forms of the operators between blocks and of attention to shared
keys (numpy), and the error bounds their kernels are held to.

Bounds, with u = 2^-24 (half a step of fp32) and r the half step of a result's
type (bf16: 2^-8, fp32: u):
* block norm: a mean of K values in a tree below chains of at most 64 is off by at
  most (64 + 16) u of the mean magnitude, and so is a mean square; the
  reciprocal root halves that relatively.  Products, the gated sum and the
  modulation bring 8 u of the magnitudes that enter, and where a mean is taken off,
  what remains carries the error of both.  100 u of the magnitudes of h, of the
  norm's terms |h| + |mean| over the root, and of the modulation bound each
  stage; errors of h reach z through the norm multiplied by 2 / root (its own
  value, and the mean and the root it shares).
* attention: a score is a sum of D products, off by at most (D + 8) u of the sum
  of its terms' magnitudes (any order; + 8 for scale, code scale and the
  exponent's argument).  A weight is off by twice the largest such error
  relatively; sums of n weights or products in any order by n u, exponentials and
  the division by 64 u more.  bf16 results: every weight is rounded to bf16
  first, r of its own size.
"""
import numpy as np

from tests._attention import U, bf16   # noqa: F401


def half_step(dtype):
    return 2.0 ** -8 if dtype == "bf16" else U


def norm_rows(x, kind, weight, bias, eps, dx):
    """(norm of rows, bound of its error when x is off by dx)."""
    if kind is None:
        return x, dx
    mag = np.abs(x)
    mean = x.mean(-1, keepdims=True) if kind == "layer" else 0.0
    c = x - mean
    dc = dx + (dx.mean(-1, keepdims=True) + 100 * U * mag.mean(-1, keepdims=True) if kind == "layer" else 0.0)
    root = np.sqrt((c * c).mean(-1, keepdims=True) + eps)
    y = c / root
    # d root <= rms(dc) + 50 u root
    dy = dc / root + np.abs(y) * (np.sqrt((dc * dc).mean(-1, keepdims=True)) / root + 100 * U)
    if weight is not None:
        y, dy = y * weight, dy * np.abs(weight)
    if bias is not None:
        y = y + bias
    return y, dy + 4 * U * (np.abs(y) + (0.0 if bias is None else np.abs(bias)))


def block_norm(x, y, post, pre, gate, shift, scale, alpha, beta):
    """post, pre: None or (kind, weight, bias, eps); gate, shift, scale: None or
    the rows of every token.  Returns h, z and the bounds before rounding."""
    x = x.astype(np.float64)
    h, dh = alpha * x, 2 * U * np.abs(alpha * x)
    if y is not None:
        y = y.astype(np.float64)
        b, db = norm_rows(y, *(post or (None,) * 4), np.zeros_like(y))
        g = beta if gate is None else beta * gate
        h = h + g * b
        dh = dh + np.abs(g) * db + 8 * U * np.abs(g * b) + 2 * U * np.abs(h)
    z, dz = norm_rows(h, *(pre or (None,) * 4), dh)
    if scale is not None:
        z, dz = z * (1 + scale), dz * np.abs(1 + scale) + 4 * U * np.abs(z * (1 + scale))
    if shift is not None:
        z = z + shift
        dz = dz + 4 * U * (np.abs(z) + np.abs(shift))
    return h, z, dh, dz + 4 * U * np.abs(z)


def attention(q, k, v, scale, dtype):
    """q [rows][D], k, v [n][D] fp64 (the keys that count): out, lse and their
    bounds, rounding of the results included."""
    R, D = q.shape
    n = k.shape[0]
    if n == 0:
        return np.zeros((R, D)), np.full(R, -np.inf), np.zeros((R, D)), np.zeros(R)
    s = scale * (q @ k.T)
    m = s.max(-1, keepdims=True)
    e = np.exp(s - m)
    total = e.sum(-1, keepdims=True)
    lse = (m + np.log(total))[:, 0]
    p = e / total
    out, mag = p @ v, p @ np.abs(v)
    ds = (D + 8) * U * abs(scale) * (np.abs(q) @ np.abs(k).T).max(-1)
    rel = 2 * ds + (n + 64) * U
    r = half_step(dtype)
    d_out = mag * (rel[:, None] + (r if dtype == "bf16" else 0.0)) * (1 + r) + r * np.abs(out)
    return out, lse, d_out, ds + (n + 64) * U + 4 * U * np.abs(lse)
