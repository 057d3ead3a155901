"""Which kernels attention to shared keys takes for a case: the rules of choice
written out again for 256 CUs, so that the tests can tell that their cases reach
every kernel that a call can; and the bounds its results are held to.

A weight enters its product as two bf16 parts for bf16 results: the second is
exact in fp32 before it is rounded, r of at most r of the weight (r = 2^-8, half a
step of bf16), so 2^-16 of each weight is lost; three parts lose less than fp32's
own rounding.  int8 caches multiply the weight by the value's scale first, one
rounding of u = 2^-24 more.  The rest is tests/_blocks.py's."""
import numpy as np

from tests import _blocks as A

CUS = 256


def attention(q, k, v, scale, dtype):
    """tests/_blocks.py's attention() with the weights' parts in the bound of out."""
    out, lse, d, dl = A.attention(q, k, v, scale, "f32")
    if dtype == "bf16" and k.shape[0]:
        s = scale * (q @ k.T)
        p = np.exp(s - lse[:, None])
        r = A.half_step("bf16")
        d = (d + (r * r + A.U) * (p @ np.abs(v))) * (1 + r) + r * np.abs(out)
    return out, lse, d, dl


def padded(D):
    return next(n for n in (64, 96, 128, 256) if D <= n)


def kind(DP, R, problems, keys):
    """Waves along the tokens (2 or 4), or 0: along the rows."""
    if R > 32:
        return 0
    return 4 if DP == 64 or (DP <= 128 and problems * -(-keys // 128) <= CUS) else 2


def parts(jobs, keys, step, least, twice):
    steps, enough = -(-keys // step), (2 if twice else 1) * CUS
    if jobs >= enough or jobs < 1:
        return 1
    return max(1, min(steps // least, 2 * enough // jobs, 64))


def step(k):
    return k * 32 if k else 64


def join(n, rows):
    return "few" if n <= 8 else "rows 64" if rows >= 8 * CUS else "rows 256"


def cross(B, Tq, S, hq, hkv, D, dtype, lens=None):
    """(kernels and orders, bytes of workspace)"""
    G = hq // hkv
    R, DP = Tq * G, padded(D)
    k = kind(DP, R, hkv * B, S)
    tiles = -(-R // (32 if k else 128))
    jobs = tiles * hkv * B
    n = parts(jobs, S, step(k), 4, dtype == "f32" and DP == 64)
    rows = R * hkv * B
    names = {("cross", DP, dtype, k)}
    each = tiles * hkv * n
    if lens and 1 < B <= 16 and each % 8 == 0:
        names |= {("longest first", "rows" if not k else "tokens", "several tiles" if tiles > 1 else "one", "parts" if n > 1 else "whole")}
        if each > 8:
            names |= {("longest first", "several jobs")}
    if n > 1:
        names |= {("join", "cross", join(n, rows), dtype), ("parts", "cross", k)}
    return names, round16(n * rows * D * 4) + round16(n * rows * 8) if n > 1 else 0


def prefix(B, P, L, hq, hkv, D, dtype, cache):
    G = hq // hkv
    R, DP = B * G, padded(D)
    k = kind(DP, R, hkv, P)
    tiles = -(-R // (32 if k else 128))
    n = parts(tiles * hkv, P, step(k), 1, dtype == "f32" and DP == 64) if P else 0
    own_tiles = -(-G // 32)
    own = kind(DP, 1, own_tiles * hkv * B, L)
    m = parts(own_tiles * hkv * B, L, step(own), 4, False)
    rows = R * hkv
    names = {("own", DP, dtype, cache, own)}
    if P:
        names |= {("prefix", DP, dtype, cache, k)}
    if m > 1:
        names |= {("join", "prefix", join(n + m, rows), dtype), ("own parts", dtype, cache)}
    every = n + (m if m > 1 else 0)
    return names, round16(every * rows * D * 4) + round16(every * rows * 8)


def round16(n):
    return -(-n // 16) * 16


def every():
    """What a call can reach."""
    names = set()
    for dtype in ("bf16", "f32"):
        for DP in (64, 96, 128, 256):
            narrow = {64: (4,), 256: (2,)}.get(DP, (4, 2))
            names |= {("cross", DP, dtype, k) for k in (0, *narrow)}
            for cache in ("bf16", "int8"):
                names |= {("prefix", DP, dtype, cache, k) for k in (0, *narrow)}
                names |= {("own", DP, dtype, cache, k) for k in narrow}
        names |= {("join", op, form, dtype) for op in ("cross", "prefix") for form in ("few", "rows 64", "rows 256")}
        names |= {("own parts", dtype, cache) for cache in ("bf16", "int8")}
    names |= {("parts", "cross", k) for k in (0, 2, 4)}
    names |= {("longest first", "several jobs")}
    names |= {("longest first", along, tiles, whole) for along in ("rows", "tokens") for whole in ("parts", "whole")
              for tiles in (("several tiles", "one") if along == "rows" else ("one",))}
    return names
