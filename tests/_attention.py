"""Plain 64-bit forms of the attention operators (numpy, loops over rows) and
the error bounds their kernels are held to.

Bounds, with u = 2^-24 (fp32 arithmetic) and r = 2^-8 for a bf16 result (its
half-ulp rounding is 2^-9; one ulp is allowed where fp32 noise moves a value
over a rounding boundary) or 2u for an fp32 one:
* head norm: the mean square of D <= 256 values, summed in any tree of depth
  <= 12 above chains of <= 8, is off by at most 20 u relatively, its square
  root by 10 u; reciprocal, root, two products and the rotation's multiply and
  add bring 8 u more: under 40 u of the magnitudes that enter.
* attention: a score is a sum of D products, off by at most (D + 8) u of the
  sum of its terms' magnitudes (any order; + 8 for scale, code scale and the
  exponent's argument).  A weight is off by twice the largest such error
  relatively, plus 64 u for exponentials, their sum and the division.
"""
import numpy as np

U = 2.0 ** -24


def bf16(x):
    """Round fp32 values to bf16 (nearest even), as fp32."""
    b = np.ascontiguousarray(x, np.float32).view(np.uint32)
    return ((b + 0x7FFF + ((b >> 16) & 1)) & 0xFFFF0000).astype(np.uint32).view(np.float32)


def unit(dtype):
    return 2.0 ** -8 if dtype == "bf16" else 2 * U


def norm_rope(x, w, eps, cos, sin, positions, interleaved):
    """x [T][heads][D] -> (y fp64, magnitudes that enter each y)."""
    x = x.astype(np.float64)
    T, H, D = x.shape
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    if w is not None:
        y = y * w.astype(np.float64)
    if cos is None:
        return y, np.abs(y)
    half = cos.shape[1]
    i = np.arange(half)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    z, mag = y.copy(), np.abs(y)
    for t in range(T):
        p = positions[t]
        if not 0 <= p < cos.shape[0]:
            z[t][:, a] = z[t][:, b] = np.nan
            continue
        c, s = cos[p].astype(np.float64), sin[p].astype(np.float64)
        z[t][:, a] = y[t][:, a] * c - y[t][:, b] * s
        z[t][:, b] = y[t][:, b] * c + y[t][:, a] * s
        mag[t][:, a] = mag[t][:, b] = np.abs(y[t][:, a]) + np.abs(y[t][:, b])
    return z, mag


def int8_rule(x):
    """The symmetric 8-bit rule on fp32 rows, in fp32 arithmetic: codes, scales."""
    x = np.ascontiguousarray(x, np.float32)
    amax = np.abs(x).max(-1)
    with np.errstate(divide="ignore"):
        inv = np.where(amax > 0, np.float32(127) / amax, np.float32(0)).astype(np.float32)
    codes = np.clip(np.rint(x * inv[..., None]), -127, 127).astype(np.int8)
    return codes, (amax / np.float32(127)).astype(np.float32)


def attention(q, k, v, keep, scale):
    """One (sequence, kv head): q [G][D], k, v [n][D] fp64, keep [n] bool.
    Returns out, lse, weights [G][n] and the bounds (score error, out scale)."""
    G, D = q.shape
    n = k.shape[0]
    out, lse, w = np.zeros((G, D)), np.full(G, -np.inf), np.zeros((G, n))
    ds, mag = np.zeros(G), np.zeros((G, D))
    at = np.nonzero(keep)[0]
    if at.size:
        kk, vv = k[at], v[at]
        s = scale * (q @ kk.T)
        m = s.max(-1, keepdims=True)
        e = np.exp(s - m)
        lse = (m + np.log(e.sum(-1, keepdims=True)))[:, 0]
        p = e / e.sum(-1, keepdims=True)
        w[:, at] = p
        out = p @ vv
        mag = p @ np.abs(vv)
        ds = (D + 8) * U * abs(scale) * (np.abs(q) @ np.abs(kk).T).max(-1)
    return out, lse, w, ds, mag


def evict_row(weight, pos, n, keep, recent, sink):
    """(moves as (to, from) pairs, slot that ends in each place below keep) of one row."""
    if n <= keep:
        return [], list(range(n))
    newest = max(int(p) for p in pos[:n])

    def order(j):
        held = pos[j] < sink or pos[j] > newest - recent
        w = float(weight[j])
        return (0, 0.0, j) if held else (2, 0.0, j) if np.isnan(w) else (1, -w, j)

    kept = set(sorted(range(n), key=order)[:keep])
    free = [j for j in range(keep) if j not in kept]
    up = [j for j in range(keep, n) if j in kept]
    assert len(free) == len(up)
    come = list(range(keep))
    for to, at in zip(free, up):
        come[to] = at
    return list(zip(free, up)), come
