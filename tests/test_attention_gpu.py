"""Attention operators on the GPU against plain 64-bit forms, at the sizes,
types, strides, masks and lengths where they can go wrong.  The bounds are
derived in tests/_attention.py."""
import numpy as np
import pytest

from rotated_w4a4_quantized_amd import rq
from tests import _attention as A

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
U = A.U


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


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


# ------------------------------------------------------------------ qk_norm_rope

NORM = [
    # T, hq, hkv, D, rot, interleaved, type, cache, page
    (1, 1, 1, 16, 16, False, "bf16", None, 16),
    (1, 32, 8, 128, 128, False, "bf16", "bf16", 64),
    (1, 32, 8, 128, 128, True, "f32", "int8", 16),
    (3, 5, 0, 24, 8, True, "f32", None, 16),
    (7, 12, 12, 128, 128, True, "bf16", None, 16),
    (13, 4, 2, 72, 72, False, "bf16", "bf16", 16),
    (13, 4, 2, 72, 72, True, "bf16", "int8", 16),
    (33, 3, 1, 80, 40, False, "f32", "bf16", 32),
    (33, 3, 1, 80, 40, False, "bf16", "int8", 32),
    (65, 16, 2, 64, 32, False, "f32", "int8", 128),
    (65, 16, 2, 64, 64, True, "bf16", "bf16", 16),
    (130, 7, 7, 96, 48, True, "f32", "bf16", 16),
    (257, 2, 1, 256, 256, False, "bf16", "bf16", 16),
    (257, 2, 1, 256, 128, True, "f32", "int8", 256),
    (1031, 12, 4, 128, 128, False, "bf16", "bf16", 16),
    (2500, 24, 24, 128, 128, True, "bf16", None, 16),
    (2500, 20, 4, 64, 0, False, "f32", "bf16", 64),
    (4099, 1, 1, 40, 16, False, "bf16", "int8", 16),
    (20001, 2, 1, 64, 64, True, "bf16", "bf16", 64),      # more tokens than waves: each walks over several
]


def check_heads(got, want, mag, dtype, what):
    got = num(got)
    bound = A.unit(dtype) * np.abs(want) + 40 * U * mag + 1e-37
    bad = ~(np.abs(got - want) <= bound) & ~(np.isnan(want) & np.isnan(got))
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {np.nanmax(np.abs(got - want) / bound):.3g} of the bound"


@pytest.mark.parametrize("T,hq,hkv,D,rot,inter,dtype,kind,page", NORM)
@pytest.mark.parametrize("weights", [True, False])
def test_qk_norm_rope(T, hq, hkv, D, rot, inter, dtype, kind, page, weights):
    rng = np.random.default_rng(T * 131 + D)
    row = (hq + 2 * hkv) * D
    ld = row + 24                                   # rows further apart than their width
    full, x = rand(rng, (T, ld), dtype, 2.0)
    x[T // 2, :D] = 0                               # a head of zeros
    full[T // 2, :D] = 0
    qkv = full[:, :row]
    rows = 300
    cos = sin = None
    if rot:
        ang = rng.uniform(-4, 4, (rows, rot // 2))
        cos, sin = np.cos(ang).astype(np.float32), np.sin(ang).astype(np.float32)
    qw, kw = (rng.standard_normal((2, D)) + 1).astype(np.float32) if weights else (None, None)
    dev = lambda a: None if a is None else torch.from_numpy(a).cuda()  # noqa: E731
    nrm = rq.QKNorm(hq, hkv, D, dev(qw), dev(kw), dev(cos), dev(sin), eps=1e-5, interleaved=inter)
    positions = rng.integers(0, rows, T).astype(np.int32)
    if T > 5 and rot:
        positions[3], positions[4] = -1, rows       # outside the table
    q_out = torch.full((T, hq * D + 8), 7.0, dtype=TYPES[dtype], device="cuda")
    k_out = torch.full((T, hkv * D), 7.0, dtype=TYPES[dtype], device="cuda") if hkv else None
    cache = seq = place = None
    if kind:
        # sequences of uneven share of the tokens, with gaps and tokens that go nowhere
        B = 3
        seq = rng.integers(0, B, T).astype(np.int32)
        need = T + 5
        per = -(-need // page)
        place = rng.permutation(need)[:T].astype(np.int32)
        if T > 10:
            place[7], place[8], seq[9] = -1, per * page, B
        table = rng.permutation(B * per + 3)[:B * per].reshape(B, per).astype(np.int32)
        table[B - 1, -1] = -1
        table[0, -1] = B * per + 3
        shape = (B * per + 3, hkv, page, D)
        i8 = kind == "int8"
        new = lambda: torch.full(shape, 5, dtype=torch.int8 if i8 else torch.bfloat16, device="cuda")  # noqa: E731
        sc = lambda: torch.full(shape[:3], 5.0, device="cuda") if i8 else None  # noqa: E731
        meta = (B, hkv, per * page)
        cache = rq.KVCache(new(), new(), dev(table), sc(), sc(), torch.full(meta, 5.0, device="cuda"),
                           torch.full(meta, 5, dtype=torch.int32, device="cuda"))
    rq.qk_norm_rope(nrm, qkv, q_out[:, :hq * D], k_out=k_out, positions=dev(positions), cache=cache, seq=dev(seq), place=dev(place))
    xh = x[:, :row].reshape(T, hq + 2 * hkv, D)
    wq, mq = A.norm_rope(xh[:, :hq], qw, 1e-5, cos, sin, positions, inter)
    wk, mk = A.norm_rope(xh[:, hq:hq + hkv], kw, 1e-5, cos, sin, positions, inter)
    check_heads(q_out[:, :hq * D].reshape(T, hq, D), wq, mq, dtype, "q")
    assert (q_out[:, hq * D:] == 7).all(), "wrote past a row of q_out"
    if hkv:
        check_heads(k_out.reshape(T, hkv, D), wk, mk, dtype, "k")
    assert same_bits(full[:, row:], torch.from_numpy(x).cuda().to(TYPES[dtype])[:, row:])
    if not kind:
        return
    at = {}
    for t in range(T):
        if 0 <= seq[t] < B and 0 <= place[t] < per * page and 0 <= table[seq[t], place[t] // page] < shape[0]:
            at[t] = (int(table[seq[t], place[t] // page]), int(place[t] % page), int(seq[t]), int(place[t]))
    ts = np.array(sorted(at))
    pg, off = np.array([at[t][0] for t in ts], dtype=int), np.array([at[t][1] for t in ts], dtype=int)
    v = xh[:, hq + hkv:].astype(np.float64)
    seen = np.zeros(shape[:3], bool)
    if len(ts):
        seen[pg, :, off] = True
    for name, y, mag in (("k", wk, mk), ("v", v, np.abs(v))):
        store = getattr(cache, name).cpu()
        assert (store.float().numpy()[~seen] == 5).all(), f"{name}: wrote a slot that is no token's"
        if not len(ts):
            continue
        got = store.float().numpy().astype(np.float64)[pg, :, off]
        if not i8:
            check_heads(torch.from_numpy(got), y[ts], mag[ts], "bf16", "cache " + name)
            continue
        s = getattr(cache, name + "_scale").cpu().numpy()[pg, :, off].astype(np.float64)
        if name == "v":     # the input's own values: the rule bit for bit
            codes, scales = A.int8_rule(x[:, :row].reshape(T, -1, D)[ts][:, hq + hkv:])
            assert np.array_equal(got.astype(np.int8), codes) and np.array_equal(s.astype(np.float32), scales)
            continue
        ok = np.isfinite(y[ts]).all(-1)     # (a token outside the table stores NaN's codes)
        amax = np.abs(y[ts]).max(-1)
        # the scale follows the fp32 values' largest, within their own bound
        assert (np.abs(s - amax / 127) <= (40 * U * mag[ts].max(-1) + 4 * U * amax) / 127 + 1e-37)[ok].all()
        assert (np.abs(got * s[..., None] - y[ts]) <= s[..., None] * 0.5001 + 80 * U * mag[ts])[ok].all()
    w, p = cache.weight.cpu().numpy(), cache.pos.cpu().numpy()
    want_w, want_p = np.full(meta, 5.0, np.float32), np.full(meta, 5, np.int32)
    for t in ts:
        want_w[at[t][2], :, at[t][3]], want_p[at[t][2], :, at[t][3]] = 0, positions[t]
    assert np.array_equal(w, want_w) and np.array_equal(p, want_p)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_qk_norm_rope_in_place_and_default_positions(dtype):
    rng = np.random.default_rng(5)
    T, hq, hkv, D = 70, 6, 2, 64
    qkv, x = rand(rng, (T, (hq + 2 * hkv) * D), dtype)
    ang = rng.uniform(-4, 4, (T, D // 2))
    cos, sin = (torch.from_numpy(f(ang).astype(np.float32)).cuda() for f in (np.cos, np.sin))
    nrm = rq.QKNorm(hq, hkv, D, cos=cos, sin=sin, interleaved=True)
    q, k = torch.empty(T, hq, D, dtype=TYPES[dtype], device="cuda"), torch.empty(T, hkv * D, dtype=TYPES[dtype], device="cuda")
    rq.qk_norm_rope(nrm, qkv, q, k_out=k)
    before = qkv.clone()
    rq.qk_norm_rope(nrm, qkv, qkv[:, :hq * D], k_out=qkv[:, hq * D:(hq + hkv) * D])
    assert same_bits(qkv[:, :hq * D].reshape(T, hq, D), q) and same_bits(qkv[:, hq * D:(hq + hkv) * D], k)
    assert same_bits(qkv[:, (hq + hkv) * D:], before[:, (hq + hkv) * D:])


def test_qk_norm_rope_no_tokens():
    nrm = rq.QKNorm(4, 2, 64)
    x = torch.zeros(0, 512, dtype=torch.bfloat16, device="cuda")
    rq.qk_norm_rope(nrm, x, torch.zeros(0, 256, dtype=torch.bfloat16, device="cuda"),
                    k_out=torch.zeros(0, 128, dtype=torch.bfloat16, device="cuda"))


# ------------------------------------------------------------------ paged_attention

def build(rng, B, hkv, D, page, lens, kind, track, spare=2, junk=True):
    """A cache with random pages; slots past the lengths hold NaN (junk)."""
    per = max(1, -(-max(max(lens), 1) // page)) + 1
    table = rng.permutation(B * per + spare)[:B * per].reshape(B, per).astype(np.int32)
    n = B * per + spare
    k, v = (rng.standard_normal((n, hkv, page, D)).astype(np.float32) for _ in range(2))
    used = np.zeros((n, page), bool)
    for b in range(B):
        for j in range(max(0, min(lens[b], per * page))):
            used[table[b, j // page], j % page] = True
    t = lambda a, dt: torch.from_numpy(np.ascontiguousarray(a)).cuda().to(dt)  # noqa: E731
    if kind == "int8":
        codes = [np.clip(np.rint(a * 40), -127, 127) for a in (k, v)]
        scale = [(rng.uniform(0.5, 2, a.shape[:3]) / 40).astype(np.float32) for a in (k, v)]
        k, v = (c * s[..., None].astype(np.float64) for c, s in zip(codes, scale))
        if junk:
            for s in scale:
                s[np.broadcast_to(~used[:, None], s.shape)] = np.nan
        c = dict(k=t(codes[0], torch.int8), v=t(codes[1], torch.int8), k_scale=t(scale[0], torch.float32),
                 v_scale=t(scale[1], torch.float32))
    else:
        k, v = A.bf16(k), A.bf16(v)
        dirty = [a.copy() for a in (k, v)]
        if junk:
            for a in dirty:
                a[np.broadcast_to(~used[:, None], a.shape[:3])] = np.nan
        c = dict(k=t(dirty[0], torch.bfloat16), v=t(dirty[1], torch.bfloat16))
    meta = (B, hkv, per * page)
    weight = rng.uniform(0, 3, meta).astype(np.float32)
    cache = rq.KVCache(c["k"], c["v"], t(table, torch.int32), c.get("k_scale"), c.get("v_scale"),
                       t(weight, torch.float32) if track else None)
    return cache, k.astype(np.float64), v.astype(np.float64), table, weight


def run_attend(cache, q, lens, max_len, mask=None, track=False, scale=None, stream=None, weight_out=None):
    hq = q.shape[1] // cache.head_dim
    out, lse = torch.full_like(q, 7.0), torch.full((cache.batch, hq), 7.0, device="cuda")
    ws = torch.full((max(16, rq.paged_attention_workspace_bytes(cache, hq, max_len, track)),), 255, dtype=torch.uint8, device="cuda")
    rq.paged_attention(q, cache, lens, out, lse=lse, max_len=max_len, mask=mask, track=track, scale=scale, workspace=ws,
                       weight_out=weight_out, stream=stream)
    return out, lse


def check_attend(cache, k, v, table, weight, q, qx, lens, max_len, mask, scale, out, lse, dtype, weight_out=None, limit=None, check_lse=True):
    B, D, hkv, page = cache.batch, cache.head_dim, cache.heads, cache.page
    hq = qx.shape[1] // D
    G = hq // hkv
    out, lse = num(out), num(lse)
    wo = None if weight_out is None else num(weight_out)
    pairs = [(b, h) for b in range(B) for h in range(hkv)]
    for b, h in pairs[:limit]:
        n = max(0, min(int(lens[b]), max_len))
        j = np.arange(n)
        pg = table[b, j // page]
        keep = (pg >= 0) & (pg < k.shape[0])
        if mask is not None:
            keep &= mask[b, :n] != 0
        pg = np.clip(pg, 0, k.shape[0] - 1)
        qq = qx.reshape(B, hkv, G, D)[b, h].astype(np.float64)
        o, ls, w, ds, mag = A.attention(qq, k[pg, h, j % page], v[pg, h, j % page], keep, scale)
        got = out.reshape(B, hkv, G, D)[b, h]
        rel = 2 * ds[:, None] + 64 * U
        bound = A.unit(dtype) * np.abs(o) + rel * mag + 1e-37
        if dtype == "bf16":     # weights are carried in two bf16 parts: 2^-16 of each
            bound = bound + 2.0 ** -16 * mag
        bad = ~(np.abs(got - o) <= bound)
        assert not bad.any(), f"b {b} h {h} n {n}: {bad.sum()} outputs off, worst {np.nanmax(np.abs(got - o) / bound):.3g}, nan {np.isnan(got).sum()}"
        gl = lse.reshape(B, hkv, G)[b, h]
        if not check_lse:
            continue
        if not keep.any():
            assert (gl == -np.inf).all() and (got == 0).all()
        else:
            assert (np.abs(gl - ls) <= ds + 16 * U * (np.abs(ls) + 1)).all(), (b, h, gl - ls)
        if wo is not None:
            want = weight[b, h].astype(np.float64).copy()
            want[:n] += w.sum(0)
            lim = np.full(want.shape, 0.0)
            lim[:n] = (w * rel).sum(0) + 4 * U * np.abs(want[:n])
            assert (np.abs(wo[b, h] - want) <= lim).all(), f"b {b} h {h}: weights off"


ATT = [
    # B, hq, hkv, D, page, lengths, type, cache
    (1, 1, 1, 16, 16, [1], "bf16", "bf16"),
    (1, 1, 1, 128, 16, [1], "f32", "int8"),
    (1, 12, 12, 128, 16, [333], "bf16", "bf16"),
    (1, 32, 8, 128, 64, [5000], "bf16", "bf16"),
    (1, 32, 8, 128, 64, [5000], "f32", "int8"),
    (4, 8, 2, 64, 16, [0, 17, 31, 300], "bf16", "bf16"),
    (4, 8, 2, 64, 16, [0, 16, 32, 299], "f32", "bf16"),
    (4, 8, 2, 64, 32, [0, 33, 63, 300], "bf16", "int8"),
    (3, 28, 4, 128, 16, [129, 2, 640], "bf16", "bf16"),
    (3, 20, 4, 80, 16, [129, 15, 77], "f32", "bf16"),
    (3, 20, 4, 72, 16, [129, 15, 77], "bf16", "int8"),
    (2, 5, 5, 96, 128, [250, 511], "bf16", "bf16"),
    (2, 6, 1, 256, 16, [250, 1025], "bf16", "bf16"),
    (2, 6, 1, 256, 64, [250, 1025], "f32", "int8"),
    (2, 6, 3, 200, 32, [250, 100], "bf16", "bf16"),
    (2, 32, 1, 128, 32, [700, 64], "bf16", "bf16"),
    (2, 40, 2, 64, 32, [700, 64], "f32", "int8"),
    (33, 4, 4, 32, 16, list(range(33)), "bf16", "bf16"),
    (70, 16, 4, 64, 16, [(37 * i) % 400 for i in range(70)], "f32", "bf16"),
]


@pytest.mark.parametrize("B,hq,hkv,D,page,lens,dtype,kind", ATT)
@pytest.mark.parametrize("mode", ["plain", "mask", "track"])
def test_paged_attention(B, hq, hkv, D, page, lens, dtype, kind, mode):
    rng = np.random.default_rng(B * 1000 + D + hq)
    cache, k, v, table, weight = build(rng, B, hkv, D, page, lens, kind, mode == "track")
    q, qx = rand(rng, (B, hq * D), dtype, 2.0)
    max_len = max(1, max(lens))
    mask = tm = None
    if mode == "mask":
        mask = (rng.random((B, max_len + 3)) < 0.6).astype(np.uint8) * 3
        mask[B - 1] = 0                                  # nothing is left of the last sequence
        tm = torch.from_numpy(mask).cuda()
    tl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out, lse = run_attend(cache, q, tl, max_len, tm, mode == "track")
    check_attend(cache, k, v, table, weight, q, qx, lens, max_len, mask, D ** -0.5, out, lse, dtype,
                 cache.weight if mode == "track" else None)


@pytest.mark.parametrize("B,hkv,top,track,dtype,kind", [
    (130, 2, 1500, False, "bf16", "bf16"),     # shares that span rows and end inside them
    (130, 2, 1500, True, "f32", "bf16"),
    (300, 4, 700, True, "bf16", "int8"),       # several rows, and empty sequences, in a share
    (300, 4, 700, False, "bf16", "bf16"),      # many rows: one workgroup each
    (70, 4, 1100, False, "f32", "int8"),
])
def test_paged_attention_many_uneven_rows(B, hkv, top, track, dtype, kind):
    rng = np.random.default_rng(B + top)
    D, page = 64, 16
    lens = (rng.integers(1, top + 1, B) * (rng.random(B) < 0.7)).tolist()
    lens[0], lens[1], lens[-1] = 0, top, 0
    cache, k, v, table, weight = build(rng, B, hkv, D, page, lens, kind, track)
    q, qx = rand(rng, (B, 2 * hkv * D), dtype, 2.0)
    out, lse = run_attend(cache, q, torch.tensor(lens, dtype=torch.int32, device="cuda"), top, None, track)
    check_attend(cache, k, v, table, weight, q, qx, lens, top, None, D ** -0.5, out, lse, dtype, cache.weight if track else None)


def test_paged_attention_without_tokens():
    """No sequence has a token, by length or by max_len 0."""
    rng = np.random.default_rng(17)
    for track in (False, True):
        for max_len, lens in ((0, [5, 9]), (600, [0, 0]), (100, [0, -3])):
            cache, *_ = build(rng, 2, 2, 64, 16, [600, 600], "bf16", track)
            before = None if cache.weight is None else cache.weight.clone()
            q, _ = rand(rng, (2, 4 * 64), "bf16")
            out, lse = run_attend(cache, q, torch.tensor(lens, dtype=torch.int32, device="cuda"), max_len, None, track)
            assert (out == 0).all() and (lse == -float("inf")).all()
            assert before is None or same_bits(before, cache.weight)


@pytest.mark.parametrize("kind", ["bf16", "int8"])
def test_paged_attention_values_in_masked_places(kind):
    """NaN and infinities where the mask leaves out, in keys and in values."""
    rng = np.random.default_rng(8)
    B, hq, hkv, D, page, lens = 2, 8, 2, 64, 16, [200, 77]
    cache, k, v, table, weight = build(rng, B, hkv, D, page, lens, kind, True)
    mask = (rng.random((B, 200)) < 0.5).astype(np.uint8)
    for b in range(B):
        for j in range(lens[b]):
            if not mask[b, j]:
                bad = float([np.nan, np.inf, -np.inf][j % 3])
                for t in (cache.k, cache.v) if kind == "bf16" else (cache.k_scale, cache.v_scale):
                    t[int(table[b, j // page]), :, j % page] = bad
    q, qx = rand(rng, (B, hq * D), "bf16")
    out, lse = run_attend(cache, q, torch.tensor(lens, dtype=torch.int32, device="cuda"), 200, torch.from_numpy(mask).cuda() != 0, True)
    check_attend(cache, k, v, table, weight, q, qx, lens, 200, mask, D ** -0.5, out, lse, "bf16", cache.weight)


def test_paged_attention_lengths_beyond_their_bounds_and_missing_pages():
    rng = np.random.default_rng(9)
    B, hq, hkv, D, page = 4, 4, 2, 64, 16
    lens = [-5, 100, 64, 90]
    cache, k, v, table, weight = build(rng, B, hkv, D, page, [0, 100, 64, 90], "bf16", True)
    table = table.copy()
    table[2, 1], table[2, 2] = -1, 10 ** 9              # pages that are not there
    table[3, :] = -7                                     # nothing is there
    cache.table.copy_(torch.from_numpy(table))
    q, qx = rand(rng, (B, hq * D), "bf16")
    out, lse = run_attend(cache, q, torch.tensor(lens, dtype=torch.int32, device="cuda"), 80, None, True)
    check_attend(cache, k, v, table, weight, q, qx, lens, 80, None, D ** -0.5, out, lse, "bf16", cache.weight)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_paged_attention_rows_apart_and_scales(dtype):
    rng = np.random.default_rng(10)
    B, hq, hkv, D, page, lens = 3, 6, 2, 64, 32, [50, 1, 130]
    cache, k, v, table, weight = build(rng, B, hkv, D, page, lens, "bf16", False)
    wide, wx = rand(rng, (B, hq * D + 128), dtype)
    q, qx = wide[:, 64:64 + hq * D], np.ascontiguousarray(wx[:, 64:64 + hq * D])
    o = torch.full((B, hq * D + 64), 7.0, dtype=TYPES[dtype], device="cuda")
    lse = torch.empty(B, hq, device="cuda")
    tl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    ws = torch.empty(max(16, rq.paged_attention_workspace_bytes(cache, hq, 130)), dtype=torch.uint8, device="cuda")
    for scale in (0.0, -0.3, 0.9):
        rq.paged_attention(q, cache, tl, o[:, :hq * D], scale=scale, max_len=130, lse=lse, workspace=ws)
        check_attend(cache, k, v, table, weight, q, qx, lens, 130, None, scale, o[:, :hq * D].contiguous(), lse, dtype)
        assert (o[:, hq * D:] == 7).all()


def test_paged_attention_sharp_softmax_and_large_scores():
    """Scores of some hundreds: one token takes all, wherever it lies."""
    rng = np.random.default_rng(11)
    B, hq, hkv, D, page, n = 1, 4, 1, 128, 16, 3000
    cache, k, v, table, weight = build(rng, B, hkv, D, page, [n], "bf16", True)
    q, qx = rand(rng, (B, hq * D), "bf16", 60.0)
    out, lse = run_attend(cache, q, torch.tensor([n], dtype=torch.int32, device="cuda"), n, None, True)
    check_attend(cache, k, v, table, weight, q, qx, [n], n, None, D ** -0.5, out, lse, "bf16", cache.weight)


def test_paged_attention_long_cache_past_32_bits():
    """Rows of k and v that start past 2^32 bytes and 2^31 elements."""
    rng = np.random.default_rng(12)
    hq, hkv, D, page, n = 8, 2, 128, 64, 1000
    pages = (1 << 31) // (hkv * page * D) + 64
    small, k, v, table, weight = build(rng, 1, hkv, D, page, [n], "bf16", False)
    big_k = torch.empty(pages, hkv, page, D, dtype=torch.bfloat16, device="cuda")
    big_v = torch.empty_like(big_k)
    count = small.k.shape[0]
    big_k[-count:], big_v[-count:] = small.k, small.v
    cache = rq.KVCache(big_k, big_v, small.table + (pages - count))
    q, qx = rand(rng, (1, hq * D), "bf16", 2.0)
    out, lse = run_attend(cache, q, torch.tensor([n], dtype=torch.int32, device="cuda"), n)
    check_attend(small, k, v, table, weight, q, qx, [n], n, None, D ** -0.5, out, lse, "bf16")
    # a store at the far end of the same cache
    nrm = rq.QKNorm(hq, hkv, D)
    row, x = rand(rng, (1, (hq + 2 * hkv) * D), "bf16")
    place = torch.tensor([5], dtype=torch.int32, device="cuda")
    rq.qk_norm_rope(nrm, row, torch.empty(1, hq * D, dtype=torch.bfloat16, device="cuda"), cache=cache, place=place)
    pg = int(cache.table[0, 0])
    assert np.array_equal(num(big_v[pg, :, 5]).ravel(), x[0, (hq + hkv) * D:].astype(np.float64))


def test_paged_attention_long_sequence():
    rng = np.random.default_rng(13)
    hq, hkv, D, page, n = 8, 2, 64, 16, 70001
    cache, k, v, table, weight = build(rng, 1, hkv, D, page, [n], "bf16", True)
    q, qx = rand(rng, (1, hq * D), "bf16", 2.0)
    out, lse = run_attend(cache, q, torch.tensor([n], dtype=torch.int32, device="cuda"), n, None, True)
    check_attend(cache, k, v, table, weight, q, qx, [n], n, None, D ** -0.5, out, lse, "bf16", cache.weight)


def test_paged_attention_shared_pages_same_bits_and_streams():
    """Sequences that share pages; the same bits again, on another stream, and
    for a sequence whatever else is in the batch's other rows' contents."""
    rng = np.random.default_rng(14)
    hq, hkv, D, page, lens = 8, 2, 128, 16, [900, 900, 333]
    cache, k, v, table, weight = build(rng, 3, hkv, D, page, lens, "bf16", True)
    table = table.copy()
    table[1] = table[0]
    cache.table.copy_(torch.from_numpy(table))
    q, qx = rand(rng, (3, hq * D), "bf16")
    tl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    w1, w2 = torch.zeros_like(cache.weight), torch.zeros_like(cache.weight)
    a = run_attend(cache, q, tl, 900, None, True, weight_out=w1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b = run_attend(cache, q, tl, 900, None, True, weight_out=w2, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    assert same_bits(a[0], b[0]) and same_bits(a[1], b[1]) and same_bits(w1, w2)
    check_attend(cache, k, v, table, weight, q, qx, lens, 900, None, D ** -0.5, a[0], a[1], "bf16")


def test_paged_attention_refuses_small_workspace():
    rng = np.random.default_rng(15)
    cache, *_ = build(rng, 1, 1, 64, 16, [4000], "bf16", True)
    q = torch.zeros(1, 64, dtype=torch.bfloat16, device="cuda")
    tl = torch.tensor([4000], dtype=torch.int32, device="cuda")
    need = rq.paged_attention_workspace_bytes(cache, 1, 4000, True)
    assert need > 0
    for ws in (None, torch.empty(need - 1, dtype=torch.uint8, device="cuda")):
        with pytest.raises(rq.RQError) as e:
            rq.paged_attention(q, cache, tl, torch.empty_like(q), max_len=4000, track=True, workspace=ws)
        assert e.value.status == -2


# ------------------------------------------------------------------ cache_evict

EVICT = [
    # B, hkv, D, page, lengths, keep, recent, sink, cache, what the weights are
    (1, 1, 16, 16, [2], 1, 0, 0, "bf16", "random"),
    (1, 8, 128, 16, [300], 256, 32, 4, "bf16", "random"),
    (1, 8, 128, 16, [300], 256, 256, 0, "int8", "random"),
    (3, 2, 64, 32, [0, 100, 40], 64, 8, 4, "bf16", "random"),
    (3, 2, 64, 32, [500, 65, 64], 64, 0, 0, "int8", "random"),
    (2, 3, 72, 16, [333, 200], 100, 10, 3, "int8", "ties"),
    (2, 3, 72, 16, [333, 200], 100, 10, 3, "bf16", "ties"),
    (2, 2, 80, 64, [700, 701], 350, 0, 0, "bf16", "zeros"),
    (2, 2, 64, 16, [129, 1000], 128, 1000, 0, "bf16", "random"),     # everything is protected
    (2, 2, 64, 16, [129, 1000], 1, 0, 0, "bf16", "odd"),
    (1, 2, 64, 16, [5000], 1500, 100, 4, "bf16", "odd"),
    (2, 4, 32, 128, [20000, 9000], 4096, 512, 4, "bf16", "random"),
    (1, 1, 16, 1024, [70000], 40000, 100, 0, "int8", "ties"),
    (40, 2, 32, 16, [17 * i % 160 for i in range(40)], 50, 5, 1, "bf16", "random"),
]


@pytest.mark.parametrize("B,hkv,D,page,lens,keep,recent,sink,kind,what", EVICT)
@pytest.mark.parametrize("in_place", [True, False])
def test_cache_evict(B, hkv, D, page, lens, keep, recent, sink, kind, what, in_place):
    rng = np.random.default_rng(B * 100 + D + keep)
    base, _, _, table, _ = build(rng, B, hkv, D, page, lens, kind, False, junk=False)
    meta = (B, hkv, table.shape[1] * page)
    weight = {"random": lambda: np.exp(2 * rng.standard_normal(meta)), "ties": lambda: rng.integers(0, 4, meta) / 2.0,
              "zeros": lambda: np.zeros(meta),
              "odd": lambda: rng.choice([np.nan, np.inf, -np.inf, -1.0, -0.0, 0.0, 1e-42, 3.0], meta)}[what]().astype(np.float32)
    pos = np.stack([rng.permutation(meta[2]) for _ in range(B * hkv)]).reshape(meta).astype(np.int32)
    dev = lambda a: torch.from_numpy(a.copy()).cuda()  # noqa: E731
    cache = rq.KVCache(base.k, base.v, base.table, base.k_scale, base.v_scale, dev(weight), dev(pos))
    before = {n: getattr(cache, n).clone() for n in ("k", "v", "k_scale", "v_scale") if getattr(cache, n) is not None}
    tl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    max_len = max(lens)
    ws = torch.full((max(16, rq.cache_evict_workspace_bytes(cache, keep, max_len)),), 255, dtype=torch.uint8, device="cuda")
    outs = {}
    if not in_place:
        outs = dict(lens_out=torch.full_like(tl, 9), weight_out=torch.full_like(cache.weight, 9.0), pos_out=torch.full_like(cache.pos, 9))
    rq.cache_evict(cache, tl, keep, recent=recent, sink=sink, max_len=max_len, workspace=ws, **outs)
    got_l = (tl if in_place else outs["lens_out"]).cpu().tolist()
    got_w = (cache.weight if in_place else outs["weight_out"]).cpu().numpy()
    got_p = (cache.pos if in_place else outs["pos_out"]).cpu().numpy()
    assert got_l == [min(n, keep) for n in lens]
    want_w = weight.copy() if in_place else np.full(meta, 9.0, np.float32)
    want_p = pos.copy() if in_place else np.full(meta, 9, np.int32)
    want = {n: t.cpu().clone() for n, t in before.items()}
    for b in range(B):
        for h in range(hkv):
            moves, come = A.evict_row(weight[b, h], pos[b, h], lens[b], keep, recent, sink)
            n = len(come)
            want_w[b, h, :n], want_p[b, h, :n] = weight[b, h, come], pos[b, h, come]
            if moves:
                to, at = np.array(moves).T
                for name, t in before.items():
                    src = t.cpu()[table[b, at // page], h, at % page]
                    want[name][table[b, to // page], h, to % page] = src
    assert np.array_equal(got_p, want_p), "positions"
    assert np.array_equal(got_w.view(np.int32), want_w.view(np.int32)), "weights"
    for name, t in want.items():
        assert same_bits(getattr(cache, name).cpu(), t), name
    if not in_place:
        assert np.array_equal(cache.weight.cpu().numpy().view(np.int32), weight.view(np.int32))
        assert np.array_equal(cache.pos.cpu().numpy(), pos) and tl.cpu().tolist() == lens


@pytest.mark.parametrize("n", [3000, 40000])
@pytest.mark.parametrize("apart", ["weight", "pos", "lens"])
def test_cache_evict_some_outputs_in_place(n, apart):
    rng = np.random.default_rng(n)
    hkv, D, page, keep, recent = 2, 16, 64, n // 3, 50
    base, _, _, table, _ = build(rng, 1, hkv, D, page, [n], "bf16", False, junk=False)
    meta = (1, hkv, base.slots)
    weight, pos = rng.uniform(0, 1, meta).astype(np.float32), np.stack([rng.permutation(base.slots) for _ in range(hkv)])[None].astype(np.int32)
    cache = rq.KVCache(base.k, base.v, base.table, weight=torch.from_numpy(weight.copy()).cuda(), pos=torch.from_numpy(pos.copy()).cuda())
    tl = torch.tensor([n], dtype=torch.int32, device="cuda")
    outs = {"weight": dict(weight_out=torch.zeros_like(cache.weight)), "pos": dict(pos_out=torch.zeros_like(cache.pos)),
            "lens": dict(lens_out=torch.zeros_like(tl))}[apart]
    rq.cache_evict(cache, tl, keep, recent=recent, max_len=n, workspace=torch.empty(rq.cache_evict_workspace_bytes(cache, keep, n), dtype=torch.uint8, device="cuda"), **outs)
    got_w, got_p = outs.get("weight_out", cache.weight).cpu().numpy(), outs.get("pos_out", cache.pos).cpu().numpy()
    assert outs.get("lens_out", tl).item() == keep
    for h in range(hkv):
        _, come = A.evict_row(weight[0, h], pos[0, h], n, keep, recent, 0)
        assert np.array_equal(got_w[0, h, :keep], weight[0, h, come]) and np.array_equal(got_p[0, h, :keep], pos[0, h, come])


def test_cache_evict_keeps_attention_of_survivors():
    """A cache whose lighter half has weight zero for this query attends the
    same after eviction, whatever the order of its slots."""
    rng = np.random.default_rng(21)
    B, hq, hkv, D, page, n, keep = 2, 8, 2, 64, 16, 400, 250
    cache, k, v, table, _ = build(rng, B, hkv, D, page, [n, n], "bf16", True)
    cache = rq.KVCache(cache.k, cache.v, cache.table, weight=torch.zeros_like(cache.weight),
                       pos=torch.arange(cache.slots, dtype=torch.int32, device="cuda").expand(B, hkv, -1).contiguous())
    q, qx = rand(rng, (B, hq * D), "f32", 6.0)
    tl = torch.full((B,), n, dtype=torch.int32, device="cuda")
    full, _ = run_attend(cache, q, tl, n, None, True)
    w = cache.weight[:, :, :n].cpu().numpy().astype(np.float64)
    lost = np.sort(w, -1)[..., :n - keep].sum(-1)               # at most this share of any head's weight is evicted
    rq.cache_evict(cache, tl, keep, max_len=n, workspace=torch.empty(rq.cache_evict_workspace_bytes(cache, keep, n), dtype=torch.uint8, device="cuda"))
    assert tl.tolist() == [keep, keep]
    left, _ = run_attend(cache, q, tl, keep)
    vmax = np.abs(v).max()
    d = np.abs(num(full) - num(left)).reshape(B, hkv, -1).max(-1)
    assert (d <= 2 * lost * vmax + 1e-4).all()
    assert lost.max() < 0.1


# ------------------------------------------------------------------ together, under a graph

def test_step_in_a_graph_replays_like_eager():
    """store + attend (tracked) + evict captured once and replayed with eager
    work between: every replay gives the eager result."""
    rng = np.random.default_rng(31)
    B, hq, hkv, D, page, n, keep = 3, 8, 2, 64, 16, 150, 120
    cache, *_ = build(rng, B, hkv, D, page, [n] * B, "bf16", True, junk=False)
    pos = torch.arange(cache.slots, dtype=torch.int32, device="cuda").expand(B, hkv, -1).contiguous()
    cache = rq.KVCache(cache.k, cache.v, cache.table, weight=cache.weight, pos=pos)
    ang = torch.from_numpy(rng.uniform(-3, 3, (400, D // 2)).astype(np.float32)).cuda()
    nrm = rq.QKNorm(hq, hkv, D, cos=ang.cos(), sin=ang.sin())
    qkv = rand(rng, (B, (hq + 2 * hkv) * D), "bf16")[0]
    place = torch.full((B,), n - 1, dtype=torch.int32, device="cuda")
    position = place.clone()
    lens, lens_out = torch.full((B,), n, dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
    q, out = (torch.empty(B, hq * D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    lse = torch.empty(B, hq, device="cuda")
    ws1 = torch.empty(max(16, rq.paged_attention_workspace_bytes(cache, hq, n, True)), dtype=torch.uint8, device="cuda")
    ws2 = torch.empty(max(16, rq.cache_evict_workspace_bytes(cache, keep, n)), dtype=torch.uint8, device="cuda")
    state = [cache.k, cache.v, cache.weight, cache.pos, lens_out, q, out, lse]

    def step():
        rq.qk_norm_rope(nrm, qkv, q, positions=position, cache=cache, place=place)
        rq.paged_attention(q, cache, lens, out, lse=lse, max_len=n, track=True, workspace=ws1)
        rq.cache_evict(cache, lens, keep, recent=16, max_len=n, lens_out=lens_out, workspace=ws2)

    start = [t.clone() for t in state]
    step()
    eager = [t.clone() for t in state]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        step()
        with torch.cuda.graph(g, stream=s):
            step()
    torch.cuda.current_stream().wait_stream(s)
    for _ in range(4):
        for t, x in zip(state, start):
            t.copy_(x)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for i, (t, x) in enumerate(zip(state, eager)):
            assert same_bits(t, x), i


# ------------------------------------------------------------------ the decode block

@pytest.mark.parametrize("int8", [False, True])
def test_decode_block_attends_to_what_it_stored(int8):
    """Steps of the decode block: every step's attention equals the formula's
    over the cache's own contents, before and after evictions, and without
    evictions over the tokens of its own projections."""
    from rotated_w4a4_quantized_amd.attention import DecodeAttention
    rng = np.random.default_rng(40)
    hidden, hq, hkv, D, B, steps = 256, 8, 2, 64, 3, 70
    Ws = [(rng.standard_normal(s) * 0.05).astype(np.float32) for s in (((hq + 2 * hkv) * D, hidden), (hidden, hq * D))]
    for budget in (None, 24):
        blk = DecodeAttention(*Ws, hq, hkv, D, B, max_len=steps, budget=budget, slack=8, recent=4, sink=2, page=16, int8=int8)
        c = blk.cache
        seen = []                                       # (position, value) of every token, fp64
        for t in range(steps):
            x, _ = rand(rng, (B, hidden), "bf16")
            before = blk.length
            y = blk.step(x)
            n = before + 1
            seen.append(num(blk.qkv)[:, (hq + hkv) * D:].reshape(B, hkv, D))
            assert torch.isfinite(y.float()).all()
            evicted = blk.length != n
            assert blk.length <= (steps if budget is None else budget + 8)
            assert blk.lens.tolist() == [blk.length] * B and blk.place.tolist() == [blk.length] * B
            if c.pos is not None:
                pos = c.pos.cpu().numpy()[:, :, :blk.length]
                assert (np.sort(pos, -1)[..., -min(4, blk.length):] == np.arange(t - min(4, blk.length) + 1, t + 1)).all(), "the newest stay"
                assert all((np.isin([0, 1][:t + 1], pos[b, h])).all() for b in range(B) for h in range(hkv)), "the first stay"
                assert all(len(set(pos[b, h])) == blk.length for b in range(B) for h in range(hkv))
                # what lies in a slot is the value of the token that pos names
                at = np.arange(blk.length)
                for b in range(B):
                    pg = c.table[b].cpu().numpy()[at // 16]
                    for h in range(hkv):
                        v = c.v.float().cpu().numpy()[pg, h, at % 16].astype(np.float64)
                        want = np.stack([seen[p][b, h] for p in pos[b, h]])
                        if int8:
                            s = c.v_scale.cpu().numpy()[pg, h, at % 16].astype(np.float64)
                            assert (np.abs(v * s[:, None] - want) <= 0.5001 * s[:, None]).all()
                        else:
                            assert np.array_equal(v, want)
            if evicted:
                continue
            full = {}
            for name in ("k", "v"):
                full[name] = num(getattr(c, name))
                if int8:
                    full[name] *= num(getattr(c, name + "_scale"))[..., None]
            check_attend(c, full["k"], full["v"], c.table.cpu().numpy(), None, blk.q, num(blk.q).astype(np.float32), [n] * B, n, None,
                         D ** -0.5, blk.attn, torch.full((B, hq), -1.0), "bf16", check_lse=False)
        assert blk.length == (steps if budget is None else 24 + (steps - 32) % 8)


def test_decode_command_runs(capsys):
    from rotated_w4a4_quantized_amd import attention
    attention.main(["--steps", "40", "--batch", "2", "--budget", "16"])
    assert "40 steps of 2 sequences" in capsys.readouterr().out


def test_decode_block_steps_on_another_stream():
    """Steps on a side stream give the bits of steps on the default one,
    through evictions, while the default stream is kept busy."""
    from rotated_w4a4_quantized_amd.attention import DecodeAttention
    rng = np.random.default_rng(41)
    hidden, hq, hkv, D, B, steps = 256, 8, 2, 64, 3, 60
    Ws = [(rng.standard_normal(s) * 0.05).astype(np.float32) for s in (((hq + 2 * hkv) * D, hidden), (hidden, hq * D))]
    x, _ = rand(rng, (steps, B, hidden), "bf16")
    got = {}
    for how in ("default", "stream", "address"):
        blk = DecodeAttention(*Ws, hq, hkv, D, B, max_len=steps, budget=24, slack=8, recent=4, sink=2, page=16)
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        busy = torch.ones(2048, 2048, device="cuda")
        ys = []
        for t in range(steps):
            if how == "default":
                ys.append(blk.step(x[t]).clone())
                continue
            busy @ busy                                   # (work that a stray operation would queue behind)
            y = blk.step(x[t], stream=s if how == "stream" else s.cuda_stream)
            with torch.cuda.stream(s):
                ys.append(y.clone())
        torch.cuda.synchronize()
        got[how] = ys + [blk.cache.k, blk.cache.v, blk.cache.weight, blk.cache.pos, blk.lens, blk.place, blk.position]
    for how in ("stream", "address"):
        for i, (a, b) in enumerate(zip(got["default"], got[how])):
            assert same_bits(a, b), (how, i)


def test_decode_block_with_a_budget_below_its_protected_tokens():
    """Defaults that protect more than the budget: the first and the newest
    tokens stay, the one just added among them."""
    from rotated_w4a4_quantized_amd.attention import DecodeAttention
    rng = np.random.default_rng(42)
    hidden, hq, hkv, D, B, steps = 128, 4, 2, 32, 2, 100
    Ws = [(rng.standard_normal(s) * 0.05).astype(np.float32) for s in (((hq + 2 * hkv) * D, hidden), (hidden, hq * D))]
    blk = DecodeAttention(*Ws, hq, hkv, D, B, max_len=steps, budget=16, slack=20, page=16)   # recent 32, sink 4
    evictions = 0
    for t in range(steps):
        n = blk.length + 1
        blk.step(rand(rng, (B, hidden), "bf16")[0])
        if blk.length == n:
            continue
        evictions += 1
        pos = np.sort(blk.cache.pos.cpu().numpy()[:, :, :16], -1)
        assert (pos == np.concatenate([np.arange(4), np.arange(t - 11, t + 1)])).all()
    assert evictions == 1 + (steps - 36) // 20


def test_decode_command_evicts(capsys):
    from rotated_w4a4_quantized_amd import attention
    attention.main(["--steps", "100", "--batch", "2", "--budget", "16"])
    assert "100 steps of 2 sequences" in (text := capsys.readouterr().out) and "36 tokens of 100 kept" in text


@pytest.mark.parametrize("host", ["tables", "weights"])
def test_qk_norm_rope_refuses_tables_in_host_memory(host):
    tables = dict(cos=torch.zeros(8, 32), sin=torch.zeros(8, 32)) if host == "tables" else dict(q_weight=torch.ones(64), k_weight=torch.ones(64))
    x = torch.zeros(2, 512, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        rq.qk_norm_rope(rq.QKNorm(4, 2, 64, **tables), x, torch.zeros_like(x[:, :256]), k_out=torch.zeros_like(x[:, :128]))


def test_workspaces_that_repeat_or_skip_memory_are_refused():
    rng = np.random.default_rng(43)
    cache, *_ = build(rng, 1, 1, 64, 16, [4000], "bf16", True)
    cache = rq.KVCache(cache.k, cache.v, cache.table, weight=cache.weight, pos=torch.zeros_like(cache.weight, dtype=torch.int32))
    q = torch.zeros(1, 64, dtype=torch.bfloat16, device="cuda")
    tl = torch.tensor([4000], dtype=torch.int32, device="cuda")
    n = max(rq.paged_attention_workspace_bytes(cache, 1, 4000, True), rq.cache_evict_workspace_bytes(cache, 100, 4000))
    one = torch.zeros(16, dtype=torch.uint8, device="cuda")
    for ws in (one[:1].expand(n), torch.zeros(2 * n, dtype=torch.uint8, device="cuda")[::2]):
        with pytest.raises(ValueError):
            rq.paged_attention(q, cache, tl, torch.empty_like(q), max_len=4000, track=True, workspace=ws)
        with pytest.raises(ValueError):
            rq.cache_evict(cache, tl, 100, max_len=4000, workspace=ws)


@pytest.mark.parametrize("D,rot,inter", [(64, 64, False), (128, 128, True), (80, 40, False)])
def test_int8_cache_keeps_what_is_not_finite(D, rot, inter):
    """Heads with NaN or infinities read back as NaN from an int8 cache, others
    as without them, and attention over such a sequence is NaN, not a number."""
    rng = np.random.default_rng(D)
    T, hq, hkv, page, rows = 12, 4, 2, 16, 50
    x = (rng.standard_normal((T, hq + 2 * hkv, D)) * 2).astype(np.float32)
    clean = x.copy()
    v = x[:, hq + hkv:]
    x[1, hq, 3] = np.nan
    x[2, hq + 1, D - 1] = np.inf
    v[3, 0, 0], v[4, 1, 5], v[5, 0, 7] = np.nan, np.inf, -np.inf
    v[6, 0, :], v[6, 0, 4] = 0, 1e-38                    # 127 / amax overflows: zeros stay zeros
    positions = rng.integers(0, rows, T).astype(np.int32)
    outside = positions.copy()
    outside[7], outside[8] = -1, rows
    ang = rng.uniform(-4, 4, (rows, rot // 2))
    dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    nrm = rq.QKNorm(hq, hkv, D, cos=dev(np.cos(ang).astype(np.float32)), sin=dev(np.sin(ang).astype(np.float32)), interleaved=inter)
    place = torch.zeros(T, dtype=torch.int32, device="cuda")
    got = []
    for data, pos in ((clean, positions), (x, outside)):
        c = rq.KVCache.alloc(T, hkv, D, page, page=page, int8=True)
        q = torch.empty(T, hq * D, device="cuda")
        rq.qk_norm_rope(nrm, dev(data).reshape(T, -1), q, positions=dev(pos), cache=c, place=place)
        got.append((c, q))
    bad = {"k": [(1, 0), (2, 1), (7, 0), (7, 1), (8, 0), (8, 1)], "v": [(3, 0), (4, 1), (5, 0)]}
    (c0, q0), (c1, q1) = got
    for n in "kv":
        codes, scale = getattr(c1, n)[:, :, 0].cpu().numpy(), getattr(c1, n + "_scale")[:, :, 0].cpu().numpy()
        with np.errstate(invalid="ignore"):
            back = codes * scale[..., None]
        for t in range(T):
            for h in range(hkv):
                if (t, h) in bad[n]:
                    assert np.isnan(back[t, h]).all() and (codes[t, h] == 0).all(), (n, t, h)
                elif (n, t, h) != ("v", 6, 0):
                    assert np.array_equal(codes[t, h], getattr(c0, n)[t, h, 0].cpu().numpy()), (n, t, h)
                    assert scale[t, h] == getattr(c0, n + "_scale")[t, h, 0].item()
    assert c1.v[6, 0, 0].tolist() == [127 if d == 4 else 0 for d in range(D)]
    out, lse = run_attend(c1, q0, torch.ones(T, dtype=torch.int32, device="cuda"), 1)
    nan = torch.isnan(out.reshape(T, hkv, hq // hkv, D)).all(-1).all(-1).cpu().numpy()
    finite = torch.isfinite(out.reshape(T, hkv, hq // hkv, D)).all(-1).all(-1).cpu().numpy()
    for t in range(T):
        for h in range(hkv):
            assert (nan if (t, h) in bad["k"] + bad["v"] else finite)[t, h], (t, h)


NANS = [
    # B, hq, hkv, D, page, lengths, type, cache: one workgroup a row, then shares, then many shares a row
    (3, 8, 2, 64, 16, [300, 17, 211], "bf16", "bf16"),
    (3, 8, 2, 128, 32, [300, 64, 500], "f32", "int8"),
    (3, 6, 1, 256, 16, [300, 65, 40], "bf16", "bf16"),
    (2, 8, 2, 64, 16, [3000, 900], "f32", "bf16"),
    (2, 4, 2, 128, 64, [9000, 4000], "bf16", "int8"),
    (2, 48, 2, 64, 16, [700, 2100], "bf16", "bf16"),
    (130, 4, 2, 64, 16, [1500 if i == 1 else 200 + 7 * i for i in range(130)], "bf16", "bf16"),
]


@pytest.mark.parametrize("B,hq,hkv,D,page,lens,dtype,kind", NANS)
@pytest.mark.parametrize("track", [False, True])
def test_paged_attention_nan_scores_show_everywhere(B, hq, hkv, D, page, lens, dtype, kind, track):
    """A NaN query, or a NaN key that is not masked: out, lse and weights of its
    heads are NaN, however tokens are dealt out to waves and workgroups; masked
    slots receive nothing and other rows are as ever."""
    rng = np.random.default_rng(B + D + hq)
    cache, k, v, table, weight = build(rng, B, hkv, D, page, lens, kind, track)
    q, qx = rand(rng, (B, hq * D), dtype, 2.0)
    n = max(lens)
    G = hq // hkv
    mask = (rng.random((B, n)) < 0.7).astype(np.uint8)
    mask[0, 5], mask[:, 0] = 1, 1
    h1 = hkv - 1
    q[1, h1 * G * D + 3] = np.nan                       # the first query head of the last key-value head
    at = int(table[0, 5 // page]), 0, 5 % page          # token 5 of key-value head 0 of sequence 0
    if kind == "int8":
        cache.k_scale[at] = np.nan
    else:
        cache.k[at][D // 2] = np.nan
    out, lse = run_attend(cache, q, torch.tensor(lens, dtype=torch.int32, device="cuda"), n, torch.from_numpy(mask).cuda(), track)
    o, ls = num(out).reshape(B, hkv, G, D), num(lse).reshape(B, hkv, G)
    bad = np.zeros((B, hkv, G), bool)
    bad[0, 0, :], bad[1, h1, 0] = True, True
    assert np.isnan(o[bad]).all() and np.isnan(ls[bad]).all()
    assert np.isfinite(o[~bad]).all() and np.isfinite(ls[~bad]).all()
    wo = num(cache.weight) if track else None
    for b, h in [(0, 0), (0, h1), (1, 0), (1, h1), (B - 1, h1)]:
        j = np.arange(lens[b])
        keep = mask[b, :lens[b]] != 0
        pg = table[b, j // page]
        want, wl, w, ds, mag = A.attention(qx.reshape(B, hkv, G, D)[b, h].astype(np.float64), k[pg, h, j % page], v[pg, h, j % page], keep, D ** -0.5)
        rel = 2 * ds[:, None] + 64 * U
        bound = A.unit(dtype) * np.abs(want) + rel * mag + 1e-37 + (2.0 ** -16 * mag if dtype == "bf16" else 0)
        ok = ~bad[b, h]
        assert (np.abs(o[b, h] - want) <= bound)[ok].all()
        assert (np.abs(ls[b, h] - wl) <= ds + 16 * U * (np.abs(wl) + 1))[ok].all()
        if not track:
            continue
        left_out = np.ones(wo.shape[2], bool)
        left_out[j[keep]] = False
        assert np.array_equal(wo[b, h][left_out], weight[b, h][left_out].astype(np.float64)), "slots left out receive nothing"
        if bad[b, h].any():
            assert np.isnan(wo[b, h][~left_out]).all()
        else:
            sums = weight[b, h, j] + w.sum(0)
            assert (np.abs(wo[b, h, j] - sums) <= (w * rel).sum(0) + 4 * U * np.abs(sums))[keep].all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_qk_norm_rope_of_tiny_heads(dtype):
    """Mean squares below 2^-126 (eps 0, or as small) give heads of mean square
    1 like any others.  Bound: each square and each sum of the mean is off by half
    the least fp32 step, 2^-150, in sum over D values and the division by D by less
    than 2^-148 absolutely, so a root by half of 2^-148 / mean relatively."""
    rng = np.random.default_rng(44)
    D, scales = 64, [1e-17, 3e-19, 1e-19, 5e-20, 2e-20, 1e-20]
    q, x = rand(rng, (len(scales), D), "f32")
    x = (x * np.array(scales, np.float32)[:, None]).astype(np.float32)
    if dtype == "bf16":
        x = A.bf16(x)
    q = torch.from_numpy(x).cuda().to(TYPES[dtype])
    for eps in (0.0, 1e-40):
        out = torch.empty_like(q)
        rq.qk_norm_rope(rq.QKNorm(1, 0, D, eps=eps), q, out)
        ms = (x.astype(np.float64) ** 2).mean(-1, keepdims=True) + float(np.float32(eps))
        want = x / np.sqrt(ms)
        rel = A.unit(dtype) + 40 * U + 2.0 ** -148 / ms
        assert (np.abs(num(out) - want) <= rel * np.abs(want)).all(), np.abs(num(out) / want - 1).max(-1)


def test_one_row_with_an_odd_number_of_elements_behind_it():
    rng = np.random.default_rng(45)
    hq, hkv, D = 4, 2, 64
    n = (hq + 2 * hkv) * D
    wide, x = rand(rng, (1, n + 3), "bf16")
    ref, got = torch.empty(1, hq * D, dtype=torch.bfloat16, device="cuda"), torch.zeros(1, hq * D + 5, dtype=torch.bfloat16, device="cuda")
    cache, *_ = build(rng, 1, hkv, D, 16, [40], "bf16", False)
    place = torch.tensor([39], dtype=torch.int32, device="cuda")
    rq.qk_norm_rope(rq.QKNorm(hq, hkv, D), wide[:, :n].clone(), ref, cache=cache, place=place)
    k = cache.k.clone()
    rq.qk_norm_rope(rq.QKNorm(hq, hkv, D), wide, got, cache=cache, place=place)
    assert same_bits(got[:, :hq * D], ref) and (got[:, hq * D:] == 0).all() and same_bits(cache.k, k)
