"""The operators between blocks and attention to shared keys on the GPU, against
plain 64-bit forms, at the sizes, types, strides, masks and lengths where they can
go wrong.  The bounds are derived in tests/_blocks.py."""
import numpy as np
import pytest

from rotated_w4a4_quantized_amd import rq
from tests import _blocks as A

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
MARK = 77.0    # what rows that must not be written hold


def rand(rng, shape, dtype, scale=1.0):
    """(device tensor of dtype, its exact values as fp32 numpy)."""
    x = (rng.standard_normal(shape) * scale).astype(np.float32)
    if dtype == "bf16":
        x = A.bf16(x)
    return torch.from_numpy(x).cuda().to(TYPES[dtype]), x


def num(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def same_bits(a, b):
    view = {4: torch.int32, 2: torch.int16, 1: torch.int8}[a.element_size()]
    return torch.equal(a.contiguous().view(view), b.contiguous().view(view))


def within(got, want, bound, name):
    with np.errstate(invalid="ignore"):
        off = np.where(got == want, 0.0, np.abs(got - want))
    bad = ~(off <= bound) & ~(np.isnan(got) & np.isnan(want))
    assert not bad.any(), (f"{name}: {bad.sum()} of {bad.size} outside, worst {np.nanmax(off / np.maximum(bound, 1e-300))} "
                           f"times the bound at {np.argwhere(bad)[0]}")


# ------------------------------------------------------------------ block_norm

NORM = [
    # T, K, post, pre, gate, shift, scale, groups, residual type, type, weights, biases
    (1, 8, None, "rms", False, False, False, 1, "bf16", "bf16", True, False),
    (1, 4096, "rms", "rms", False, False, False, 1, "bf16", "bf16", True, False),
    (3, 24, "layer", "layer", True, True, True, 2, "f32", "f32", True, True),
    (2, 504, None, "layer", True, True, True, 1, "bf16", "bf16", False, False),
    (5, 512, "rms", None, True, False, False, 5, "f32", "bf16", True, False),
    (7, 520, None, "rms", False, True, False, 3, "bf16", "f32", True, True),
    (65, 1024, "layer", "rms", True, False, True, 4, "f32", "f32", False, True),
    (130, 1152, None, "layer", True, True, True, 2, "bf16", "bf16", False, False),
    (33, 1536, None, "layer", True, True, True, 33, "f32", "bf16", False, False),
    (9, 2048, "rms", "rms", True, True, True, 2, "bf16", "bf16", True, True),
    (4, 2056, "layer", "layer", False, True, True, 2, "f32", "f32", True, True),
    (6, 4096, None, "layer", True, True, True, 3, "bf16", "f32", False, False),
    (5, 5000, "rms", "rms", True, False, False, 1, "f32", "bf16", True, False),
    (3, 8192, "rms", "layer", True, True, True, 1, "bf16", "bf16", True, True),
    (4, 8960, "rms", "rms", True, True, True, 2, "f32", "f32", True, False),
    (2, 12288, None, "rms", False, False, True, 1, "bf16", "bf16", True, False),
    (3, 16384, "layer", "layer", True, True, True, 3, "f32", "f32", True, True),
    (2, 16376, "rms", "rms", True, False, False, 1, "bf16", "bf16", True, False),
    (4099, 64, None, "layer", True, True, True, 7, "bf16", "bf16", False, False),
    (9001, 256, "rms", "rms", True, True, True, 3, "f32", "bf16", True, False),
]


def norm_case(rng, T, K, post, pre, gate, shift, scale, groups, res, io, weights, biases, index=False):
    x, xn = rand(rng, (T, K), res, 2.0)
    xn = xn + 1.0        # a mean worth taking off
    if res == "bf16":
        xn = A.bf16(xn)
    x = torch.from_numpy(xn).cuda().to(TYPES[res])
    y, yn = rand(rng, (T, K), io)
    norms, plain = {}, {}
    for name, kind, eps in (("post", post, 1e-5), ("pre", pre, 1e-6)):
        if kind is None:
            norms[name], plain[name] = None, None
            continue
        w, wn = rand(rng, K, "f32") if weights else (None, None)
        b, bn = rand(rng, K, "f32") if biases else (None, None)
        norms[name] = rq.Norm(K, kind, weight=w, bias=b, eps=eps)
        plain[name] = (kind, wn, bn, float(np.float32(eps)))
    table, tn = rand(rng, (groups, 3, K), "f32", 0.5)
    per = -(-T // groups)
    row = rng.integers(0, groups, T) if index else np.arange(T) // per
    use = (gate, shift, scale)
    mod = None
    if any(use):
        parts = [table[:, i] if u else None for i, u in enumerate(use)]
        mod = rq.Modulation(*parts, per=None if index else per,
                            index=torch.from_numpy(row.astype(np.int32)).cuda() if index else None)
    rows = [tn[row, i].astype(np.float64) if u else None for i, u in enumerate(use)]
    return x, xn, y, yn, norms, plain, mod, rows


@pytest.mark.parametrize("case", NORM, ids=str)
def test_block_norm(case):
    T, K = case[:2]
    res, io = case[8:10]
    rng = np.random.default_rng(T * 31 + K)
    for index in (False, True):
        x, xn, y, yn, norms, plain, mod, rows = norm_case(rng, *case, index=index)
        alpha, beta = (1.0, 1.0) if not index else (0.75, -1.5)
        h, z = torch.empty_like(x), torch.empty_like(y)
        rq.block_norm(x, z, norms["pre"], y=y, post=norms["post"], h=h, mod=mod, alpha=alpha, beta=beta)
        hn, zn, dh, dz = A.block_norm(xn, yn, plain["post"], plain["pre"], *rows, alpha, beta)
        within(num(h), hn, dh * 1.01 + A.half_step(res) * np.abs(hn), "h")
        within(num(z), zn, dz * 1.01 + A.half_step(io) * np.abs(zn), "z")


@pytest.mark.parametrize("res,io", [("bf16", "bf16"), ("f32", "bf16"), ("f32", "f32")])
def test_block_norm_parts_strides_and_in_place(res, io):
    rng = np.random.default_rng(5)
    T, K = 37, 1160
    x, xn, y, yn, norms, plain, mod, rows = norm_case(rng, T, K, "rms", "layer", True, True, True, 4, res, io, True, True)
    h0, z0 = torch.empty_like(x), torch.empty_like(y)
    rq.block_norm(x, z0, norms["pre"], y=y, post=norms["post"], h=h0, mod=mod)
    # only one of the results
    h, z = torch.empty_like(x), torch.empty_like(y)
    rq.block_norm(x, y=y, post=norms["post"], h=h, mod=mod)
    assert same_bits(h, h0)
    rq.block_norm(x, z, norms["pre"], y=y, post=norms["post"], mod=mod)
    assert same_bits(z, z0)
    # nothing added: the first norm of a network
    rq.block_norm(x, z, norms["pre"], mod=mod)
    hn, zn, dh, dz = A.block_norm(xn, None, None, plain["pre"], *rows, 1.0, 1.0)
    within(num(z), zn, dz * 1.01 + A.half_step(io) * np.abs(zn), "z alone")
    # rows inside wider ones, what lies between them left alone
    wide = {n: torch.full((T, K + 24), MARK, device="cuda", dtype=t.dtype) for n, t in (("x", x), ("y", y), ("h", x), ("z", y))}
    wide["x"][:, 8:8 + K], wide["y"][:, 16:16 + K] = x, y
    rq.block_norm(wide["x"][:, 8:8 + K], wide["z"][:, 8:8 + K], norms["pre"], y=wide["y"][:, 16:16 + K], post=norms["post"],
                  h=wide["h"][:, 16:16 + K], mod=mod)
    assert same_bits(wide["z"][:, 8:8 + K], z0) and same_bits(wide["h"][:, 16:16 + K], h0)
    for n, a in (("h", 16), ("z", 8)):
        assert (wide[n][:, :a] == MARK).all() and (wide[n][:, a + K:] == MARK).all()
    # in place
    xi, yi = x.clone(), y.clone()
    rq.block_norm(xi, yi, norms["pre"], y=yi, post=norms["post"], h=xi, mod=mod)
    assert same_bits(xi, h0) and same_bits(yi, z0)


def test_block_norm_rows_of_modulations_and_what_is_not_finite():
    rng = np.random.default_rng(6)
    T, K = 12, 128
    x, xn, y, yn, norms, plain, _, _ = norm_case(rng, T, K, None, "rms", False, False, False, 1, "f32", "f32", False, False)
    table, tn = rand(rng, (3, K), "f32")
    index = torch.tensor([0, 1, 2, 3, -1, 0, 2, 2, 1 << 30, 1, 0, -(1 << 31)], dtype=torch.int32, device="cuda")
    out = (index < 0) | (index >= 3)
    h, z = torch.empty_like(x), torch.empty_like(y)
    rq.block_norm(x, z, norms["pre"], y=y, h=h, mod=rq.Modulation(shift=table, index=index))
    assert torch.isnan(z[out]).all() and torch.isfinite(z[~out]).all() and torch.isfinite(h).all()
    rq.block_norm(x, z, norms["pre"], y=y, h=h, mod=rq.Modulation(gate=table, index=index))
    assert torch.isnan(h[out]).all() and torch.isnan(z[out]).all() and torch.isfinite(z[~out]).all()
    # a NaN or an infinity stays in its token; rows of zeros with eps 0 are 0 / 0
    x2 = x.clone()
    x2[3, 5], x2[7, 100] = float("nan"), float("inf")
    rq.block_norm(x2, z, norms["pre"], y=y, h=h)
    hn, zn, dh, dz = A.block_norm(xn, yn, None, plain["pre"], None, None, None, 1.0, 1.0)
    fine = [t for t in range(T) if t not in (3, 7)]
    within(num(z)[fine], zn[fine], dz[fine] * 1.01 + A.U * np.abs(zn[fine]), "z")
    assert torch.isnan(z[3]).all() and torch.isnan(z[7, 100])
    zero = torch.zeros_like(x)
    rq.block_norm(zero, z, rq.Norm(K, "rms", eps=0.0))
    assert torch.isnan(z).all()
    rq.block_norm(zero, z, rq.Norm(K, "layer", eps=1e-6))
    assert (z == 0).all()
    # no tokens
    rq.block_norm(x[:0], z[:0], norms["pre"], y=y[:0], h=h[:0])


def test_block_norm_means_far_from_zero():
    # the mean is taken off before squares are summed: 2^12 + small numbers keep them
    rng = np.random.default_rng(7)
    for K in (256, 4096, 16384):
        small = rng.integers(-8, 9, (5, K)).astype(np.float32) / 16
        x = torch.from_numpy(small + 4096).cuda()
        z = torch.empty_like(x)
        rq.block_norm(x, z, rq.Norm(K, "layer", eps=1e-6))
        xn = (small + 4096).astype(np.float64)
        _, zn, _, dz = A.block_norm(xn, None, None, ("layer", None, None, float(np.float32(1e-6))), None, None, None, 1.0, 1.0)
        within(num(z), zn, dz * 1.01 + A.U * np.abs(zn), "z")


# ------------------------------------------------------------------ cross_attention

CROSS = [
    # B, Tq, S, hq, hkv, D, type, lens, mask, q_lens, scale
    (1, 1, 1, 1, 1, 16, "bf16", None, False, False, None),
    (1, 1, 1, 1, 1, 64, "f32", None, False, False, None),
    (2, 1, 31, 4, 1, 64, "bf16", "some", False, False, None),
    (3, 1, 300, 16, 4, 64, "bf16", "some", True, False, None),
    (3, 1, 129, 8, 8, 128, "f32", "some", True, False, None),
    (1, 1, 5000, 32, 8, 128, "bf16", None, False, False, None),
    (2, 1, 700, 32, 1, 128, "bf16", "some", False, False, None),
    (2, 1, 500, 64, 1, 96, "bf16", None, True, False, None),
    (5, 1, 33, 4, 2, 256, "bf16", "some", True, False, None),
    (2, 1, 257, 4, 2, 256, "f32", "some", False, False, None),
    (2, 2, 65, 3, 3, 24, "bf16", None, False, False, None),
    (2, 5, 127, 6, 2, 40, "f32", "some", False, True, None),
    (1, 31, 128, 2, 2, 72, "bf16", None, True, False, None),
    (4, 33, 120, 2, 1, 72, "bf16", "some", True, True, None),
    (2, 100, 64, 5, 1, 80, "bf16", None, False, False, None),
    (2, 129, 63, 2, 2, 96, "f32", "some", False, True, None),
    (1, 257, 65, 3, 3, 104, "bf16", None, False, False, -0.2),
    (3, 257, 300, 4, 2, 128, "bf16", "some", True, True, None),
    (1, 130, 1000, 2, 2, 128, "bf16", None, False, False, None),
    (1, 300, 191, 2, 1, 128, "f32", None, True, False, 0.0),
    (2, 140, 70, 1, 1, 136, "bf16", "some", False, False, None),
    (1, 33, 2100, 1, 1, 200, "bf16", None, False, False, None),
    (2, 129, 129, 2, 1, 256, "bf16", "some", True, False, 0.3),
    (1, 150, 200, 2, 2, 256, "f32", None, False, False, -0.1),
    (1, 513, 513, 2, 2, 64, "bf16", None, False, False, None),
    (2, 40, 0, 2, 2, 64, "bf16", None, False, False, None),
    (1, 64, 9000, 1, 1, 64, "f32", None, True, False, None),
]


def cross_inputs(rng, B, Tq, S, hq, hkv, D, dtype, lens, mask, q_lens, scale):
    q, qn = rand(rng, (B, Tq, hq, D), dtype, 1.5)
    kv, kvn = rand(rng, (B, S, 2, hkv, D), "bf16")
    ln = np.full(B, S)
    lt = None
    if lens:
        raw = rng.integers(0, S + 1, B)
        raw[0] = S + 5 if B > 1 else S           # past the bound: cut
        if B > 2:
            raw[1], raw[2] = 0, -3               # nothing
        ln = np.clip(raw, 0, S)
        lt = torch.from_numpy(raw.astype(np.int32)).cuda()
    mt, mn = None, np.ones((B, S), bool)
    if mask:
        mn = rng.random((B, S)) < 0.7
        mn[B - 1, :S // 2] = False               # whole steps that do not count
        if B > 3:
            mn[3] = False
        mt = torch.from_numpy(mn).cuda()
    qt, qln = None, np.full(B, Tq)
    if q_lens:
        raw = rng.integers(0, Tq + 1, B)
        raw[0] = Tq + 7
        if B > 1:
            raw[1] = 0
        qln = np.clip(raw, 0, Tq)
        qt = torch.from_numpy(raw.astype(np.int32)).cuda()
    keep = mn & (np.arange(S)[None] < ln[:, None])
    # what does not count holds anything
    junk = torch.from_numpy(~keep).cuda()
    kv[junk] = torch.tensor([float("nan"), float("inf"), -float("inf")], device="cuda").to(torch.bfloat16)[
        torch.randint(0, 3, (int(junk.sum()), 2, hkv, D), device="cuda")]
    return q, qn, kv, kvn, lt, mt, qt, qln, keep


def check_cross(out, lse, qn, kvn, keep, qln, hq, hkv, scale, dtype):
    B, Tq, _, D = qn.shape
    scale = D ** -0.5 if scale is None else scale
    G = hq // hkv
    got, gl = num(out), None if lse is None else num(lse)
    for b in range(B):
        n = int(qln[b])
        assert (got[b, n:] == MARK).all(), "rows behind the last query were written"
        if gl is not None:
            assert (gl[b, n:] == MARK).all()
        at = np.nonzero(keep[b])[0]
        for h in range(hkv):
            k, v = (kvn[b, at, i, h].astype(np.float64) for i in (0, 1))
            q = qn[b, :n, h * G:(h + 1) * G].astype(np.float64).reshape(-1, D)
            o, l, do, dl = A.attention(q, k, v, scale, dtype)
            within(got[b, :n, h * G:(h + 1) * G].reshape(-1, D), o, do, f"out of sequence {b}, head {h}")
            if gl is not None:
                within(gl[b, :n, h * G:(h + 1) * G].reshape(-1), l, dl, f"lse of sequence {b}, head {h}")


def run_cross(q, k, v, lt, mt, qt, scale, lse=True, out=None, stream=None):
    B, Tq, hq, D = q.shape
    st = rq.States(k, v, lens=lt, mask=mt)
    out = torch.full_like(q, MARK) if out is None else out
    lse = torch.full((B, Tq, hq), MARK, device="cuda") if lse else None
    n = rq.cross_attention_workspace_bytes(st, Tq, hq, q.dtype)
    ws = torch.full((max(n, 16),), 255, dtype=torch.uint8, device="cuda")   # (as NaN: what is not written must not be read)
    rq.cross_attention(q, st, out, scale=scale, q_lens=qt, lse=lse, workspace=ws, stream=stream)
    return out, lse


@pytest.mark.parametrize("case", CROSS, ids=str)
def test_cross_attention(case):
    B, Tq, S, hq, hkv, D, dtype, _, _, _, scale = case
    rng = np.random.default_rng(sum(case[:6]) * 7)
    q, qn, kv, kvn, lt, mt, qt, qln, keep = cross_inputs(rng, *case)
    out, lse = run_cross(q, kv[:, :, 0], kv[:, :, 1], lt, mt, qt, scale)
    check_cross(out, lse, qn, kvn, keep, qln, hq, hkv, scale, dtype)
    again, lse2 = run_cross(q, kv[:, :, 0], kv[:, :, 1], lt, mt, qt, scale)
    assert same_bits(out, again) and same_bits(lse, lse2)


@pytest.mark.parametrize("Tq,S", [(1, 400), (40, 70), (300, 130)])
def test_cross_attention_strides(Tq, S):
    rng = np.random.default_rng(11)
    B, hq, hkv, D = 3, 4, 2, 64
    qkv, qn = rand(rng, (Tq, B, hq + 3, D), "bf16")       # token-major, other heads beside
    q = qkv[:, :, 1:1 + hq].transpose(0, 1)
    one, on = rand(rng, (1, S, hkv, 2 * D), "bf16")       # one sequence of states for all
    k, v = one[..., :D], one[..., D:]
    k, v = (t.contiguous().expand(B, S, hkv, D) for t in (k, v))
    mask = torch.zeros(1, S, dtype=torch.uint8, device="cuda")
    mask[0, ::2] = 1
    buf = torch.full((Tq, B, hq + 1, D), MARK, device="cuda", dtype=torch.bfloat16)
    out, lse = run_cross(q, k, v, None, mask.expand(B, S), None, None, out=buf[:, :, :hq].transpose(0, 1))
    keep = np.tile(np.arange(S) % 2 == 0, (B, 1))
    kvn = np.stack([on[..., :D], on[..., D:]], 2)
    check_cross(out, lse, qn[:, :, 1:1 + hq].transpose(1, 0, 2, 3), np.tile(kvn, (B, 1, 1, 1, 1)), keep, np.full(B, Tq), hq, hkv, None, "bf16")
    assert (buf[:, :, hq:] == MARK).all()


@pytest.mark.parametrize("Tq,S", [(1, 300), (3, 2000), (200, 300)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_cross_attention_scores_far_apart_and_not_finite(Tq, S, dtype):
    rng = np.random.default_rng(12)
    hq, hkv, D = 2, 1, 64
    # rising scores move the running maximum in every step
    q, qn = rand(rng, (1, Tq, hq, D), dtype, 0.1)
    kv, kvn = rand(rng, (1, S, 2, hkv, D), "bf16")
    qn[..., 0] = 16.0
    ramp = A.bf16(np.linspace(-40, 60, S).astype(np.float32))
    kvn[0, :, 0, 0, 0] = ramp
    q, kv = torch.from_numpy(qn).cuda().to(TYPES[dtype]), torch.from_numpy(kvn).cuda().bfloat16()
    keep = np.ones((1, S), bool)
    out, lse = run_cross(q, kv[:, :, 0], kv[:, :, 1], None, None, None, None)
    check_cross(out, lse, qn, kvn, keep, [Tq], hq, hkv, None, dtype)
    # and falling ones never do
    kvn = kvn[:, ::-1].copy()
    kv = torch.from_numpy(kvn).cuda().bfloat16()
    out, lse = run_cross(q, kv[:, :, 0], kv[:, :, 1], None, None, None, None)
    check_cross(out, lse, qn, kvn, keep, [Tq], hq, hkv, None, dtype)
    # a NaN query is NaN in its own row only; a NaN key in all
    q2 = q.clone()
    q2[0, Tq - 1, 1, 3] = float("nan")
    o2, l2 = run_cross(q2, kv[:, :, 0], kv[:, :, 1], None, None, None, None)
    assert torch.isnan(o2[0, Tq - 1, 1]).all() and torch.isnan(l2[0, Tq - 1, 1])
    keep_rows = torch.ones(Tq, hq, dtype=torch.bool)
    keep_rows[Tq - 1, 1] = False
    assert torch.equal(o2[0].cpu()[keep_rows], out[0].cpu()[keep_rows]) and torch.equal(l2[0].cpu()[keep_rows], lse[0].cpu()[keep_rows])
    for j in (0, S // 2, S - 1):
        kv2 = kv.clone()
        kv2[0, j, 0, 0, 5] = float("nan")
        o3, l3 = run_cross(q, kv2[:, :, 0], kv2[:, :, 1], None, None, None, None)
        assert torch.isnan(o3).all() and torch.isnan(l3).all()


def test_cross_attention_to_one_token():
    # A single key: the output is its value.  Its weight p is the exponential of what
    # rounding the maximum left over, within |s| u of 1: it rounds to 1 in bf16.  fp32:
    # p's three bf16 parts hold its 24 bits, so sum and division by l = p leave the
    # value up to their own rounding, u for each of the three products' sums and the
    # division's reciprocal and product: 4 u.
    rng = np.random.default_rng(13)
    for Tq in (1, 200):
        for dtype in ("bf16", "f32"):
            q, _ = rand(rng, (2, Tq, 2, 128), dtype, 3.0)
            kv, kvn = rand(rng, (2, 1, 2, 2, 128), "bf16")
            out, _ = run_cross(q, kv[:, :, 0], kv[:, :, 1], None, None, None, None)
            want = np.broadcast_to(kvn[:, :, 1].astype(np.float64), (2, Tq, 2, 128))
            within(num(out), want, 0.0 if dtype == "bf16" else 4 * A.U * np.abs(want), "out")


# ------------------------------------------------------------------ prefix_attention

PREFIX = [
    # B, prefix, own, hq, hkv, D, type, cache, page, mask
    (1, 1, 1, 1, 1, 16, "bf16", "bf16", 16, False),
    (1, 0, 40, 4, 2, 64, "bf16", "bf16", 16, False),
    (3, 33, 0, 4, 2, 64, "f32", "bf16", 16, False),
    (4, 64, 20, 8, 2, 64, "bf16", "bf16", 64, True),
    (5, 100, 37, 8, 8, 128, "bf16", "int8", 16, False),
    (6, 1000, 130, 32, 8, 128, "bf16", "bf16", 64, False),
    (7, 999, 130, 32, 8, 128, "f32", "int8", 32, True),
    (33, 257, 65, 4, 4, 72, "bf16", "bf16", 16, True),
    (40, 300, 20, 16, 2, 80, "bf16", "int8", 128, False),
    (70, 2000, 150, 8, 2, 128, "bf16", "bf16", 16, False),
    (130, 129, 33, 4, 1, 96, "f32", "bf16", 16, False),
    (9, 500, 300, 4, 1, 256, "bf16", "bf16", 32, True),
    (40, 500, 70, 4, 1, 256, "f32", "int8", 32, False),
    (66, 200, 70, 2, 1, 200, "bf16", "int8", 16, True),
    (3, 90, 70, 40, 1, 64, "bf16", "bf16", 16, False),
    (2, 3, 5000, 8, 2, 64, "bf16", "bf16", 16, False),
    (300, 130, 9, 1, 1, 64, "bf16", "bf16", 16, False),
]


def prefix_inputs(rng, B, P, L, hq, hkv, D, dtype, kind, page, mask):
    front, per = -(-P // page), max(1, -(-(P + L) // page))
    pages = front + B * (per - P // page) + 3
    order = rng.permutation(pages).astype(np.int32)
    own = order[front:front + B * (per - P // page)].reshape(B, -1)
    table = np.concatenate([np.full((B, P // page), -7, np.int32), own], 1)   # (below the prefix: not read)
    shape = (pages, hkv, page, D)
    t = {}
    if kind == "int8":
        codes = {n: rng.integers(-127, 128, shape).astype(np.int8) for n in "kv"}
        scale = {n: ((rng.random(shape[:3]) + 0.5) / 73).astype(np.float32) for n in "kv"}
        val = {n: codes[n].astype(np.float64) * scale[n][..., None] for n in "kv"}
        t = {n: torch.from_numpy(codes[n]).cuda() for n in "kv"}
        t.update({n + "_scale": torch.from_numpy(scale[n]).cuda() for n in "kv"})
    else:
        val = {}
        for n in "kv":
            t[n], x = rand(rng, shape, "bf16")
            val[n] = x.astype(np.float64)
    lens = P + rng.integers(0, L + 1, B)
    lens[0] = P + L
    if B > 2:
        lens[1], lens[2] = 0, P                  # not in the batch; nothing of its own
    if B > 4 and P > 1:
        lens[3], lens[4] = P - 1, P + L + 9      # shorter than the prefix: not in the batch; past the bound: cut
    q, qn = rand(rng, (B, hq * D), dtype, 1.5)
    m = rng.random((B, P + L)) < 0.7 if mask else None
    return table, order, t, val, lens, q, qn, m


def prefix_plain(b, table, order, val, n, P, page, pages, m, h):
    """Keys and values of sequence b that count, head h."""
    j = np.arange(n)
    pg = np.where(j < P, order[np.minimum(j // page, max(0, -(-P // page) - 1))], table[b][np.minimum(j // page, table.shape[1] - 1)])
    keep = (pg >= 0) & (pg < pages)
    if m is not None:
        keep &= (j < P) | m[b, :n]
    return (val[x][pg[keep], h, j[keep] % page] for x in "kv")


def run_prefix(q, cache, order, P, lens, max_len, hq, mask=None, scale=None, lse=True, stream=None, ws=None):
    B = q.shape[0]
    out = torch.full_like(q, MARK)
    lse = torch.full((B, hq), MARK, device="cuda") if lse else None
    if ws is None:
        n = rq.prefix_attention_workspace_bytes(cache, hq, P, max_len, q.dtype)
        ws = torch.full((max(n, 16),), 255, dtype=torch.uint8, device="cuda")
    rq.prefix_attention(q, cache, order, P, lens, out, scale=scale, max_len=max_len, mask=mask, lse=lse, workspace=ws, stream=stream)
    return out, lse


def check_prefix(out, lse, qn, table, order, val, lens, P, L, page, pages, hq, hkv, D, m, dtype, scale=None):
    G, B = hq // hkv, qn.shape[0]
    got, gl = num(out).reshape(B, hq, D), num(lse)
    for b in range(B):
        n = min(int(lens[b]), P + L)
        for h in range(hkv):
            if n < P or n < 1:
                assert (got[b] == 0).all() and (gl[b] == -np.inf).all()
                continue
            k, v = prefix_plain(b, table, order, val, n, P, page, pages, m, h)
            q = qn[b].reshape(hq, D)[h * G:(h + 1) * G].astype(np.float64)
            o, l, do, dl = A.attention(q, k, v, D ** -0.5 if scale is None else scale, dtype)
            within(got[b, h * G:(h + 1) * G], o, do, f"out of sequence {b}, head {h}")
            within(gl[b, h * G:(h + 1) * G], l, dl, f"lse of sequence {b}, head {h}")


@pytest.mark.parametrize("case", PREFIX, ids=str)
def test_prefix_attention(case):
    B, P, L, hq, hkv, D, dtype, kind, page, mask = case
    rng = np.random.default_rng(sum(case[:6]) * 3)
    table, order, t, val, lens, q, qn, m = prefix_inputs(rng, *case)
    pages = t["k"].shape[0]
    cache = rq.KVCache(t["k"], t["v"], torch.from_numpy(table).cuda(), k_scale=t.get("k_scale"), v_scale=t.get("v_scale"))
    front = torch.from_numpy(order[:max(1, -(-P // page))].copy()).cuda()
    lt = torch.from_numpy(lens.astype(np.int32)).cuda()
    mt = None if m is None else torch.from_numpy(m).cuda()
    out, lse = run_prefix(q, cache, front, P, lt, P + L, hq, mask=mt)
    check_prefix(out, lse, qn, table, order, val, lens, P, L, page, pages, hq, hkv, D, m, dtype)
    again, lse2 = run_prefix(q, cache, front, P, lt, P + L, hq, mask=mt)
    assert same_bits(out, again) and same_bits(lse, lse2)


@pytest.mark.parametrize("B,kind", [(3, "bf16"), (3, "int8"), (50, "bf16"), (50, "int8")])
def test_prefix_attention_missing_pages_and_junk(B, kind):
    # pages that are not there are passed over, and so is what lies behind lengths and
    # in front of a sequence's own slots, whatever it holds
    rng = np.random.default_rng(21)
    P, L, hq, hkv, D, page = 90, 60, 8, 2, 64, 16
    table, order, t, val, lens, q, qn, _ = prefix_inputs(rng, B, P, L, hq, hkv, D, "bf16", kind, page, False)
    pages = t["k"].shape[0]
    order = order.copy()
    order[2], order[4] = -1, pages
    table[B - 1, P // page + 1] = 1 << 30
    lens[B - 1] = P + L
    used = np.zeros((pages, page), bool)
    for j in range(P):
        if 0 <= order[j // page] < pages:
            used[order[j // page], j % page] = True
    for b in range(B):
        for j in range(P, min(int(lens[b]), P + L)):
            if 0 <= table[b, j // page] < pages:
                used[table[b, j // page], j % page] = True
    un = torch.from_numpy(~used).cuda()
    if kind == "int8":
        for n in "kv":
            t[n + "_scale"].transpose(1, 2)[un] = float("nan")
    else:
        for n in "kv":
            t[n].transpose(1, 2)[un] = float("nan")
    cache = rq.KVCache(t["k"], t["v"], torch.from_numpy(table).cuda(), k_scale=t.get("k_scale"), v_scale=t.get("v_scale"))
    front = torch.from_numpy(order[:-(-P // page)].copy()).cuda()
    out, lse = run_prefix(q, cache, front, P, torch.from_numpy(lens.astype(np.int32)).cuda(), P + L, hq)
    check_prefix(out, lse, qn, table, order, val, lens, P, L, page, pages, hq, hkv, D, None, "bf16")
    # no page at all: nothing to look at
    none = torch.full_like(front, -1)
    cache2 = rq.KVCache(t["k"], t["v"], torch.full_like(cache.table, -1), k_scale=t.get("k_scale"), v_scale=t.get("v_scale"))
    out, lse = run_prefix(q, cache2, none, P, torch.from_numpy(lens.astype(np.int32)).cuda(), P + L, hq)
    assert (out == 0).all() and (lse == -float("inf")).all()


@pytest.mark.parametrize("Tq, S", [(3, 150), (70, 150), (3, 4100)])
def test_cross_attention_queries_that_are_not_finite(Tq, S):
    """With no token left such a row is 0, too; else it is NaN, and its alone."""
    hq, hkv, D = 4, 2, 72
    for dtype in (torch.bfloat16, torch.float32):
        rng = np.random.default_rng(Tq + S)
        mask = np.ones((2, S), bool)
        mask[1] = False
        q = torch.from_numpy(rng.standard_normal((2, Tq, hq, D)).astype(np.float32)).cuda().to(dtype)
        kv = torch.from_numpy(rng.standard_normal((2, S, 2, hkv, D)).astype(np.float32)).cuda().to(torch.bfloat16)
        want, wl = run_cross(q, kv[:, :, 0], kv[:, :, 1], None, torch.from_numpy(mask).cuda(), None, None)
        odd = q.clone()
        odd[:, 1, 2, 5] = float("nan")
        odd[:, 2, 1, 70] = float("inf")
        got, gl = run_cross(odd, kv[:, :, 0], kv[:, :, 1], None, torch.from_numpy(mask).cuda(), None, None)
        assert (got[1] == 0).all() and (gl[1] == -float("inf")).all()
        for t, h in ((1, 2), (2, 1)):
            assert got[0, t, h].isnan().all() and gl[0, t, h].isnan()
            got[0, t, h], gl[0, t, h] = want[0, t, h], wl[0, t, h]
        assert torch.equal(got, want) and torch.equal(gl, wl)


def test_prefix_attention_equals_paged_attention_on_shared_pages():
    rng = np.random.default_rng(22)
    B, P, L, hq, hkv, D, page = 20, 192, 100, 8, 2, 128, 32
    table, order, t, val, lens, q, qn, _ = prefix_inputs(rng, B, P, L, hq, hkv, D, "f32", "bf16", page, False)
    lens[:] = P + rng.integers(0, L + 1, B)
    lens[1] = 0
    lt = torch.from_numpy(lens.astype(np.int32)).cuda()
    front = torch.from_numpy(order[:P // page].copy()).cuda()
    cache = rq.KVCache(t["k"], t["v"], torch.from_numpy(table).cuda())
    out, lse = run_prefix(q, cache, front, P, lt, P + L, hq)
    table[:, :P // page] = order[:P // page]
    whole = rq.KVCache(t["k"], t["v"], torch.from_numpy(table).cuda())
    o2, l2 = torch.empty_like(q), torch.empty_like(lse)
    ws = torch.empty(max(16, rq.paged_attention_workspace_bytes(whole, hq, P + L)), dtype=torch.uint8, device="cuda")
    rq.paged_attention(q, whole, lt, o2, max_len=P + L, lse=l2, workspace=ws)
    G = hq // hkv
    for b in range(B):
        n = int(lens[b])
        for h in range(hkv):
            if n == 0:
                continue
            k, v = prefix_plain(b, table, order, val, n, P, page, t["k"].shape[0], None, h)
            _, _, do, dl = A.attention(qn[b].reshape(hq, D)[h * G:(h + 1) * G].astype(np.float64), k, v, D ** -0.5, "f32")
            s = slice(h * G, (h + 1) * G)
            within(num(out)[b].reshape(hq, D)[s], num(o2)[b].reshape(hq, D)[s], 2 * do, "out")
            within(num(lse)[b, s], num(l2)[b, s], 2 * dl, "lse")
