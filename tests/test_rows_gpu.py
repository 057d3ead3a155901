"""Attention to shared keys on the GPU: every kernel that a call can reach, against
plain 64-bit forms.  The bounds are derived in tests/_rows.py and tests/_blocks.py."""
import numpy as np
import pytest

from rotated_w4a4_quantized_amd import rq
from tests import _blocks as A
from tests import _rows as R
from tests.test_blocks_gpu import MARK, cross_inputs, num, prefix_inputs, prefix_plain, rand, run_cross, run_prefix, same_bits, within

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


TYPES, CACHES = ("bf16", "f32"), ("bf16", "int8")

CROSS = [
    # B, Tq, S, hq, hkv, D, type, lens, mask, q_lens, scale
    # waves along the tokens: two a workgroup where there is much work, four with parts
    *[(40, 1, 500, 4, 2, D, t, "some", m, False, None) for t in TYPES for D, m in ((96, True), (120, False))],
    *[(2, 2, 2000, 16, 8, 64, t, "some", False, True, None) for t in TYPES],
    (2, 3, 200, 2, 2, 80, "f32", None, True, False, None),
    (1, 2, 2000, 4, 2, 256, "f32", None, False, False, None),
    # few and many parts, few and many rows of them
    *[(1, 300, 600, 1, 1, D, t, None, True, False, None) for t in TYPES for D in (128, 200)],
    *[(1, 600, 3000, 4, 1, 16, t, "some", False, False, None) for t in TYPES],
    # sequences of uneven lengths, the longest first
    *[(3, 100, 90, 8, 8, 64, t, "some", False, True, None) for t in TYPES],
    (2, 100, 600, 8, 8, 64, "bf16", "some", True, False, 0.3),
    (3, 520, 200, 8, 8, 64, "bf16", "some", True, True, None),
    (5, 140, 190, 4, 4, 72, "bf16", "some", False, False, None),
    (3, 520, 1000, 4, 2, 72, "f32", "some", False, True, None),
    # as many sequences as are ranked, and more
    (16, 40, 100, 8, 8, 64, "bf16", "some", False, False, None),
    (17, 40, 100, 8, 8, 64, "bf16", "some", True, False, None),
    (70, 5, 150, 4, 2, 128, "bf16", "some", False, True, -0.1),
]

PREFIX = [
    # B, prefix, own, hq, hkv, D, type, cache, page, mask
    *[(B, P, L, hq, hkv, D, t, c, page, m) for t in TYPES for c in CACHES for D in (64, 72, 128, 256)
      for B, P, L, hq, hkv, page, m in ((3, 150, 30, 4, 2, 16, True), (2, 2100, 20, 16, 16, 64, False), (130, 140, 20, 2, 2, 32, False))],
    # own slots in several parts: behind a few and many of the prefix's, few and many rows
    *[(3, 60, 1200, 4, 2, D, t, c, 16, D == 64) for t in TYPES for c in CACHES for D in (64, 128)],
    *[(3, 1500, 1200, 8, 2, 40, t, c, 64, False) for t in TYPES for c in CACHES],
    *[(32, 2000, 1200, 64, 4, 16, t, c, 128, False) for t in TYPES for c in CACHES],
    (40, 300, 1100, 4, 2, 256, "bf16", "bf16", 64, True),
]


@pytest.mark.parametrize("case", CROSS, ids=str)
def test_cross_attention(case):
    B, Tq, S, hq, hkv, D, dtype, _, _, _, scale = case
    rng = np.random.default_rng(sum(case[:6]) * 5)
    q, qn, kv, kvn, lt, mt, qt, qln, keep = cross_inputs(rng, *case)
    out, lse = run_cross(q, kv[:, :, 0], kv[:, :, 1], lt, mt, qt, scale)
    got, gl, G = num(out), num(lse), hq // hkv
    for b in range(B):
        n = int(qln[b])
        assert (got[b, n:] == MARK).all() and (gl[b, n:] == MARK).all(), "rows behind the last query were written"
        at = np.nonzero(keep[b])[0]
        for h in range(hkv):
            k, v = (kvn[b, at, i, h].astype(np.float64) for i in (0, 1))
            s = slice(h * G, (h + 1) * G)
            o, l, do, dl = R.attention(qn[b, :n, s].astype(np.float64).reshape(-1, D), k, v, D ** -0.5 if scale is None else scale, dtype)
            within(got[b, :n, s].reshape(-1, D), o, do, f"out of sequence {b}, head {h}")
            within(gl[b, :n, s].reshape(-1), l, dl, f"lse of sequence {b}, head {h}")
    again, lse2 = run_cross(q, kv[:, :, 0], kv[:, :, 1], lt, mt, qt, scale)
    assert same_bits(out, again) and same_bits(lse, lse2)


def check_prefix(out, lse, qn, table, order, val, lens, P, L, page, pages, hq, hkv, D, m, dtype, scale=None, skip=()):
    """skip: (sequence, head) pairs that are not compared."""
    G, B = hq // hkv, qn.shape[0]
    got, gl = num(out).reshape(B, hq, D), num(lse)
    for b in range(B):
        n = min(int(lens[b]), P + L)
        if n < P or n < 1:
            assert (got[b] == 0).all() and (gl[b] == -np.inf).all()
            continue
        for h in range(hkv):
            k, v = prefix_plain(b, table, order, val, n, P, page, pages, m, h)
            heads = [i for i in range(h * G, (h + 1) * G) if (b, i) not in skip]
            q = qn[b].reshape(hq, D)[heads].astype(np.float64)
            o, l, do, dl = R.attention(q, k, v, D ** -0.5 if scale is None else scale, dtype)
            within(got[b, heads], o, do, f"out of sequence {b}, head {h}")
            within(gl[b, heads], l, dl, f"lse of sequence {b}, head {h}")


def prefix_case(rng, case):
    """Inputs on the device and what check_prefix() takes of them."""
    B, P, L, hq, hkv, D, dtype, kind, page, mask = case
    table, order, t, val, lens, q, qn, m = prefix_inputs(rng, *case)
    cache = rq.KVCache(t["k"], t["v"], torch.from_numpy(table).cuda(), k_scale=t.get("k_scale"), v_scale=t.get("v_scale"))
    front = torch.from_numpy(order[:max(1, -(-P // page))].copy()).cuda()
    lt = torch.from_numpy(lens.astype(np.int32)).cuda()
    mt = None if m is None else torch.from_numpy(m).cuda()
    return q, cache, front, lt, mt, (qn, table, order, val, lens, P, L, page, t["k"].shape[0], hq, hkv, D, m, dtype)


@pytest.mark.parametrize("case", PREFIX, ids=str)
def test_prefix_attention(case):
    B, P, L, hq = case[:4]
    q, cache, front, lt, mt, plain = prefix_case(np.random.default_rng(sum(case[:6]) * 3), case)
    out, lse = run_prefix(q, cache, front, P, lt, P + L, hq, mask=mt)
    check_prefix(out, lse, *plain)
    again, lse2 = run_prefix(q, cache, front, P, lt, P + L, hq, mask=mt)
    assert same_bits(out, again) and same_bits(lse, lse2)


@pytest.mark.parametrize("kind", CACHES)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("B,L", [(5, 70), (50, 70), (5, 1200)])
def test_prefix_attention_scales_strides_and_queries_that_are_not_finite(B, L, dtype, kind):
    P, hq, hkv, D = 100, 8, 2, 72
    case = (B, P, L, hq, hkv, D, dtype, kind, 16, True)
    q, cache, front, lt, mt, plain = prefix_case(np.random.default_rng(B + L), case)
    for scale in (-0.2, 0.0, 0.4):
        out, lse = run_prefix(q, cache, front, P, lt, P + L, hq, mask=mt, scale=scale)
        check_prefix(out, lse, *plain, scale=scale)
    # rows inside wider ones
    out, lse = run_prefix(q, cache, front, P, lt, P + L, hq, mask=mt)
    wide = torch.full((B, hq * D + 40), MARK, device="cuda", dtype=q.dtype)
    wide[:, 8:8 + hq * D] = q
    into = torch.full((B, hq * D + 16), MARK, device="cuda", dtype=q.dtype)
    ws = torch.empty(max(16, rq.prefix_attention_workspace_bytes(cache, hq, P, P + L, q.dtype)), dtype=torch.uint8, device="cuda")
    rq.prefix_attention(wide[:, 8:8 + hq * D], cache, front, P, lt, into[:, 16:], max_len=P + L, mask=mt, workspace=ws)
    assert same_bits(into[:, 16:], out) and (into[:, :16] == MARK).all()
    # a NaN or an infinity among a head's queries stays in its row, and where nothing is left the row is 0
    odd = q.view(B, hq, D).clone()
    odd[0, 3, 70], odd[4, 1, 0] = float("nan"), -float("inf")
    odd[1] = float("nan")                        # (the sequence of length 0)
    out, lse = run_prefix(odd.view(B, -1), cache, front, P, lt, P + L, hq, mask=mt)
    for b, i in ((0, 3), (4, 1)):
        assert out.view(B, hq, D)[b, i].isnan().all() and lse[b, i].isnan()
    check_prefix(out, lse, *plain, skip={(0, 3), (4, 1)})


@pytest.mark.parametrize("kind", CACHES)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("B,L", [(6, 40), (40, 40)])
def test_prefix_attention_is_as_exact_as_paged_attention(B, L, dtype, kind):
    """Both lie within the same bounds of the 64-bit result."""
    P, hq, hkv, D, page = 64, 8, 2, 128, 32
    case = (B, P, L, hq, hkv, D, dtype, kind, page, False)
    q, cache, front, lt, _, plain = prefix_case(np.random.default_rng(B), case)
    out, lse = run_prefix(q, cache, front, P, lt, P + L, hq)
    check_prefix(out, lse, *plain)
    table = cache.table.clone()
    table[:, :P // page] = front
    whole = rq.KVCache(cache.k, cache.v, table, k_scale=cache.k_scale, v_scale=cache.v_scale)
    short = torch.where(lt < P, torch.zeros_like(lt), lt)     # (not in the batch)
    o2, l2 = torch.empty_like(q), torch.empty_like(lse)
    ws = torch.empty(max(16, rq.paged_attention_workspace_bytes(whole, hq, P + L)), dtype=torch.uint8, device="cuda")
    rq.paged_attention(q, whole, short, o2, max_len=P + L, lse=l2, workspace=ws)
    check_prefix(o2, l2, *plain)


def test_more_workgroups_than_a_launch_holds_along_one_axis():
    # 2^24 and more (one each for a sequence and head): the same bits as a part of the sequences at a time
    B, H, D, page, each = 65535, 300, 16, 16, 16000
    g = torch.Generator(device="cuda").manual_seed(3)
    q = torch.randn(B, 1, H, D, generator=g, device="cuda", dtype=torch.bfloat16)
    kv = torch.randn(2, page, H, D, generator=g, device="cuda", dtype=torch.bfloat16)
    lens = torch.randint(0, page + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    k, v = (kv[i, None].expand(B, page, H, D) for i in (0, 1))
    out, lse = run_cross(q, k, v, lens, None, None, None)
    pages = kv.transpose(1, 2)[:, None].contiguous()
    table = torch.zeros(B, 1, dtype=torch.int32, device="cuda")
    o2, l2 = run_prefix(q.view(B, -1), rq.KVCache(pages[0], pages[1], table), None, 0, lens, page, H)
    for b in range(0, B, each):
        s = slice(b, min(b + each, B))
        part, part_lse = run_cross(q[s], k[s], v[s], lens[s].contiguous(), None, None, None)
        assert same_bits(part, out[s]) and same_bits(part_lse, lse[s])
        part, part_lse = run_prefix(q[s].view(-1, H * D), rq.KVCache(pages[0], pages[1], table[s]), None, 0, lens[s].contiguous(), page, H)
        assert same_bits(part, o2[s]) and same_bits(part_lse, l2[s])
    kn, vn = (num(t) for t in kv)
    for b in (0, 1, each - 1, 40000, B - 1):
        n = int(lens[b])
        for h in (0, 7, H - 1):
            o, l, do, dl = R.attention(num(q[b, :, h]), kn[:n, h], vn[:n, h], D ** -0.5, "bf16")
            for got, gl in ((out[b, :, h], lse[b, :, h]), (o2[b].view(H, D)[h:h + 1], l2[b, h:h + 1])):
                within(num(got), o, do, "out")
                within(num(gl), l, dl, "lse")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("Tq,S", [(2, 150), (60, 150), (2, 2000)])
def test_cross_attention_to_infinities(Tq, S, dtype):
    """What a score of +-infinity and an infinite value lead to."""
    rng = np.random.default_rng(S)
    H, D = 2, 64
    q, qn = rand(rng, (1, Tq, H, D), dtype)
    kv, kvn = rand(rng, (1, S, 2, H, D), "bf16")
    j = S // 3
    # a key of infinity in one coordinate: +-infinity times the query's, of either sign
    q[..., 3], qn[..., 3] = 1.5, 1.5
    q[0, 1, :, 3], qn[0, 1, :, 3] = -1.5, -1.5
    inf = kv.clone()
    inf[0, j, 0, :, 3] = float("inf")
    out, lse = run_cross(q, inf[:, :, 0], inf[:, :, 1], None, None, None, None)
    assert out[0, 0].isnan().all() and lse[0, 0].isnan().all()              # a score of +infinity
    if dtype == "bf16":                                                     # a score of -infinity: the token does not count
        at = np.delete(np.arange(S), j)
        for h in range(H):
            o, l, do, dl = R.attention(qn[0, 1:2, h].astype(np.float64), kvn[0, at, 0, h].astype(np.float64),
                                       kvn[0, at, 1, h].astype(np.float64), D ** -0.5, dtype)
            within(num(out[0, 1:2, h]), o, do, "out")
            within(num(lse[0, 1:2, h]), l, dl, "lse")
    # an infinite value: its column alone
    inf = kv.clone()
    inf[0, j, 1, 0, 5] = float("inf")
    want, wl = run_cross(q, kv[:, :, 0], kv[:, :, 1], None, None, None, None)
    out, lse = run_cross(q, inf[:, :, 0], inf[:, :, 1], None, None, None, None)
    assert not out[0, :, 0, 5].isfinite().any()
    out[0, :, 0, 5] = want[0, :, 0, 5]
    assert same_bits(out, want) and same_bits(lse, wl)
