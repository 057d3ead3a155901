"""The operators between blocks and attention to shared keys without a GPU:
refusals of the C ABI (every check runs before any HIP call), workspace sizes,
struct layouts and the binding's own checks; and the plain 64-bit forms against
independent values."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

from rotated_w4a4_quantized_amd import rq
from tests import _blocks as A

torch = pytest.importorskip("torch")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PTR = 1 << 20   # never dereferenced: every call here is rejected or has no work
NULL, SHAPE, DTYPE, ALIGN = -1, -2, -3, -4
BF16, F32 = rq.RQ_BF16, rq.RQ_F32


def ref(s):
    return None if s is None else ctypes.byref(s)


def fill(cls, base, kw):
    d = dict(base, **kw)
    return cls(*[d[f] for f, _ in cls._fields_])


def norm(**kw):
    return fill(rq.c_norm, dict(kind=0, eps=1e-6, weight=PTR, bias=None), kw)


def modulation(**kw):
    return fill(rq.c_modulation, dict(rows=4, reserved=0, ld=256, per=1, index=None, gate=PTR, shift=PTR, scale=PTR), kw)


def states(**kw):
    return fill(rq.c_states, dict(heads=4, head_dim=64, batch=2, reserved=0, keys=100, k_ld=512, v_ld=512, k_stride=51200,
                                  v_stride=51200, mask_ld=100, k=PTR, v=PTR, lens=None, mask=None), kw)


def cache(**kw):
    return fill(rq.c_kv_cache, dict(dtype=BF16, heads=4, head_dim=64, page=16, batch=2, table_ld=8, pages=32, k=PTR, v=PTR,
                                    k_scale=None, v_scale=None, table=PTR, weight=None, pos=None), kw)


def call_norm(post=None, pre=None, mod=None, width=256, x=PTR, x_dtype=BF16, x_ld=256, y=PTR, dtype=BF16, y_ld=256, T=4,
              alpha=1.0, beta=1.0, h=PTR, h_ld=256, z=PTR, z_ld=256):
    return rq.load().rq_block_norm(ref(post), ref(pre), ref(mod), width, x, x_dtype, x_ld, y, dtype, y_ld, T, alpha, beta, h,
                                   h_ld, z, z_ld, None)


def call_cross(s=None, q=PTR, dtype=BF16, q_ld=512, q_stride=25600, queries=50, heads=8, scale=0.125, q_lens=None, out=PTR,
               out_ld=512, out_stride=25600, lse=None, ws=PTR, wsb=1 << 40):
    s = states() if s is None else s
    return rq.load().rq_cross_attention(ref(s), q, dtype, q_ld, q_stride, queries, heads, scale, q_lens, out, out_ld,
                                        out_stride, lse, ws, wsb, None)


def call_prefix(c=None, table=PTR, prefix=40, q=PTR, dtype=BF16, q_ld=512, heads=8, scale=0.125, lens=PTR, max_len=100,
                mask=None, mask_ld=0, out=PTR, out_ld=512, lse=None, ws=PTR, wsb=1 << 40):
    c = cache() if c is None else c
    return rq.load().rq_prefix_attention(ref(c), table, prefix, q, dtype, q_ld, heads, scale, lens, max_len, mask, mask_ld,
                                         out, out_ld, lse, ws, wsb, None)


def test_struct_layouts(tmp_path):
    structs = {"rq_norm": rq.c_norm, "rq_modulation": rq.c_modulation, "rq_states": rq.c_states}
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "rq.h"', 'int main(void) {']
    for cname, ct in structs.items():
        lines.append(f'printf("{cname} %zu\\n", sizeof({cname}));')
        lines += [f'printf("{cname}.{f} %zu\\n", offsetof({cname}, {f}));' for f, _ in ct._fields_]
    src, exe = tmp_path / "probe.c", tmp_path / "probe"
    src.write_text("\n".join(lines + ["return 0;", "}"]))
    subprocess.check_call(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)])
    got = dict(l.split() for l in subprocess.check_output([str(exe)]).decode().splitlines())
    for cname, ct in structs.items():
        assert int(got[cname]) == ctypes.sizeof(ct)
        for f, _ in ct._fields_:
            assert int(got[f"{cname}.{f}"]) == getattr(ct, f).offset, (cname, f)


# ------------------------------------------------------------------ refusals

@pytest.mark.parametrize("kw,status", [
    (dict(width=0), SHAPE), (dict(width=4), SHAPE), (dict(width=252), SHAPE), (dict(width=16392), SHAPE),
    (dict(x_dtype=rq.RQ_I8), DTYPE), (dict(dtype=rq.RQ_I32), DTYPE), (dict(T=-1), SHAPE), (dict(T=1 << 31), SHAPE),
    (dict(alpha=float("nan")), SHAPE), (dict(beta=float("inf")), SHAPE), (dict(x_ld=248), SHAPE), (dict(y_ld=255), SHAPE),
    (dict(h_ld=0), SHAPE), (dict(z_ld=-256), SHAPE), (dict(x_ld=(1 << 31) + 8), SHAPE), (dict(x=None), NULL),
    (dict(h=None, z=None), NULL), (dict(x=PTR + 8), ALIGN), (dict(y=PTR + 8), ALIGN), (dict(h=PTR + 2), ALIGN),
    (dict(z=PTR + 4), ALIGN), (dict(x_ld=260), ALIGN), (dict(y_ld=260), ALIGN), (dict(h_ld=260), ALIGN), (dict(z_ld=257), ALIGN),
    (dict(x_dtype=F32, x_ld=258, h_ld=256), ALIGN),
])
def test_block_norm_refusals(kw, status):
    assert call_norm(**kw) == status
    assert rq.load().rq_last_error()


def test_block_norm_refuses_descriptors():
    for bad, status in ((dict(kind=2), SHAPE), (dict(kind=-1), SHAPE), (dict(eps=-1.0), SHAPE), (dict(eps=float("nan")), SHAPE),
                        (dict(eps=float("inf")), SHAPE), (dict(weight=PTR + 4), ALIGN), (dict(bias=PTR + 8), ALIGN)):
        assert call_norm(pre=norm(**bad)) == status
        assert call_norm(post=norm(**bad)) == status
    assert call_norm(post=norm(), y=None) == NULL
    assert call_norm(pre=norm(), z=None) == NULL
    for bad, status in ((dict(rows=0), SHAPE), (dict(rows=-3), SHAPE), (dict(ld=248), SHAPE), (dict(per=0), SHAPE),
                        (dict(rows=3), SHAPE), (dict(rows=1, per=3), SHAPE), (dict(ld=258), ALIGN), (dict(gate=PTR + 4), ALIGN),
                        (dict(shift=PTR + 8), ALIGN), (dict(scale=PTR + 12), ALIGN)):
        assert call_norm(mod=modulation(**bad)) == status, bad
    assert call_norm(T=0, x=None) == 0
    assert call_norm(T=0, mod=modulation(rows=1), post=norm(), pre=norm()) == 0


STATES = [
    (dict(heads=0), SHAPE), (dict(heads=1025), SHAPE), (dict(head_dim=8), SHAPE), (dict(head_dim=68), SHAPE),
    (dict(head_dim=264), SHAPE), (dict(batch=-1), SHAPE), (dict(batch=65536), SHAPE), (dict(keys=-1), SHAPE),
    (dict(keys=(1 << 24) + 1), SHAPE), (dict(heads=3), SHAPE),
]


@pytest.mark.parametrize("kw,status", STATES + [
    (dict(k_ld=255), SHAPE), (dict(v_ld=255), SHAPE), (dict(k_stride=-8), SHAPE), (dict(v_stride=-8), SHAPE),
    (dict(k=None), NULL), (dict(v=None), NULL), (dict(mask=PTR, mask_ld=99), SHAPE), (dict(k=PTR + 8), ALIGN),
    (dict(v=PTR + 2), ALIGN), (dict(k_ld=516), ALIGN), (dict(v_ld=516), ALIGN), (dict(k_stride=51204), ALIGN),
    (dict(v_stride=51201), ALIGN),
])
def test_states_refusals(kw, status):
    assert call_cross(states(**kw)) == status
    assert rq.load().rq_last_error()


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=rq.RQ_I8), DTYPE), (dict(heads=0), SHAPE), (dict(heads=6), SHAPE), (dict(heads=1028), SHAPE),
    (dict(queries=-1), SHAPE), (dict(queries=(1 << 24) + 1), SHAPE), (dict(queries=(1 << 25) // 16), SHAPE),
    (dict(scale=float("nan")), SHAPE), (dict(scale=float("-inf")), SHAPE), (dict(q_ld=511), SHAPE), (dict(out_ld=511), SHAPE),
    (dict(q_stride=-8), SHAPE), (dict(out_stride=-8), SHAPE), (dict(out_stride=512), SHAPE), (dict(out_stride=0), SHAPE),
    (dict(q=None), NULL), (dict(out=None), NULL), (dict(q=PTR + 8), ALIGN), (dict(out=PTR + 8), ALIGN), (dict(q_ld=516), ALIGN),
    (dict(out_ld=516, out_stride=25800), ALIGN), (dict(q_stride=25604), ALIGN), (dict(out_stride=25604), ALIGN),
])
def test_cross_attention_refusals(kw, status):
    assert call_cross(**kw) == status
    assert rq.load().rq_last_error()


def test_cross_attention_without_work_and_workspace():
    assert rq.load().rq_cross_attention(None, PTR, BF16, 512, 0, 1, 8, 1.0, None, PTR, 512, 0, None, None, 0, None) == NULL
    assert call_cross(states(batch=0), q=None, out=None, ws=None) == 0
    assert call_cross(queries=0, q=None, out=None, ws=None) == 0
    n = ctypes.c_size_t(0)
    size = rq.load().rq_cross_attention_workspace_bytes
    for kw, status in STATES:
        assert size(ref(states(**kw)), 50, 8, BF16, ctypes.byref(n)) == status
    assert size(ref(states()), 50, 8, BF16, None) == NULL
    assert size(None, 50, 8, BF16, ctypes.byref(n)) == NULL
    assert size(ref(states()), 50, 8, rq.RQ_I8, ctypes.byref(n)) == DTYPE
    # a long call of few rows takes a workspace, and is refused without
    long = states(keys=5000, k=PTR, batch=1)
    assert size(ref(long), 1, 8, BF16, ctypes.byref(n)) == 0 and n.value > 0
    assert call_cross(long, queries=1, ws=None, wsb=0) == SHAPE
    assert call_cross(long, queries=1, wsb=n.value - 1) == SHAPE
    assert call_cross(long, queries=1, ws=PTR + 8) == ALIGN
    # sequences of out one after another or token by token, but not into each other
    assert call_cross(out_ld=1024, out_stride=256) == SHAPE


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=F32), DTYPE), (dict(heads=0), SHAPE), (dict(head_dim=68), SHAPE), (dict(page=24), SHAPE), (dict(batch=65536), SHAPE),
    (dict(table_ld=0), SHAPE), (dict(pages=0), SHAPE), (dict(k=None), NULL), (dict(table=None), NULL), (dict(dtype=rq.RQ_I8), NULL),
    (dict(v=PTR + 4), ALIGN), (dict(table=PTR + 4), ALIGN),
])
def test_prefix_attention_refuses_caches(kw, status):
    assert call_prefix(cache(**kw)) == status


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=rq.RQ_I8), DTYPE), (dict(heads=0), SHAPE), (dict(heads=6), SHAPE), (dict(heads=1028), SHAPE), (dict(prefix=-1), SHAPE),
    (dict(prefix=101), SHAPE), (dict(max_len=129), SHAPE), (dict(max_len=-1), SHAPE), (dict(q_ld=511), SHAPE),
    (dict(out_ld=511), SHAPE), (dict(scale=float("nan")), SHAPE), (dict(mask=PTR, mask_ld=99), SHAPE), (dict(q=None), NULL),
    (dict(lens=None), NULL), (dict(out=None), NULL), (dict(table=None), NULL), (dict(q=PTR + 8), ALIGN), (dict(out=PTR + 8), ALIGN),
    (dict(q_ld=516), ALIGN), (dict(out_ld=516), ALIGN), (dict(table=PTR + 4), ALIGN), (dict(ws=None, wsb=0), SHAPE),
    (dict(ws=PTR + 8), ALIGN),
])
def test_prefix_attention_refusals(kw, status):
    assert call_prefix(**kw) == status
    assert rq.load().rq_last_error()


def test_prefix_attention_without_work_and_workspace():
    assert call_prefix(cache(batch=0), q=None, lens=None, out=None, ws=None) == 0
    assert rq.load().rq_prefix_attention(None, PTR, 1, PTR, BF16, 512, 8, 1.0, PTR, 9, None, 0, PTR, 512, None, PTR, 9, None) == NULL
    n = ctypes.c_size_t(0)
    size = rq.load().rq_prefix_attention_workspace_bytes
    assert size(ref(cache()), 8, BF16, 40, 100, ctypes.byref(n)) == 0
    assert call_prefix(wsb=n.value - 1) == SHAPE
    assert size(ref(cache()), 8, BF16, 101, 100, ctypes.byref(n)) == SHAPE
    assert size(ref(cache()), 8, BF16, 40, 100, None) == NULL
    assert size(None, 8, BF16, 40, 100, ctypes.byref(n)) == NULL


def test_workspaces_grow_with_the_keys():
    """A workspace for the longest call holds every shorter one."""
    n = ctypes.c_size_t(0)
    lengths = [*range(0, 700, 13), 1000, 1023, 1024, 1025, 2000, 5000, 20000, 100000]
    for D in (64, 72, 128, 256):
        for dtype in (BF16, F32):
            for batch, heads, queries in ((1, 1, 1), (3, 4, 1), (40, 8, 1), (1, 12, 77), (2, 4, 300)):
                last = 0
                for keys in lengths:
                    assert rq.load().rq_cross_attention_workspace_bytes(ref(states(head_dim=D, heads=heads, batch=batch, keys=keys)), queries,
                                                                        heads * 2, dtype, ctypes.byref(n)) == 0
                    assert n.value >= last
                    last = n.value
            for batch, heads in ((1, 1), (5, 8), (64, 8)):
                for prefix in (0, 40, 999):
                    last = 0
                    for more in lengths:
                        c = cache(head_dim=D, heads=heads, batch=batch, table_ld=1 << 14)
                        assert rq.load().rq_prefix_attention_workspace_bytes(ref(c), heads * 2, dtype, prefix, prefix + more, ctypes.byref(n)) == 0
                        assert n.value >= last
                        last = n.value


# ------------------------------------------------------------------ the binding

def test_binding_norm_and_modulation():
    f = torch.zeros
    with pytest.raises(ValueError):
        rq.Norm(64, "batch")
    with pytest.raises(ValueError):
        rq.Norm(64, weight=f(63))
    with pytest.raises(ValueError):
        rq.Norm(64, bias=f(64, dtype=torch.float64))
    with pytest.raises(ValueError):
        rq.Modulation()
    with pytest.raises(ValueError):
        rq.Modulation(gate=f(2, 64), shift=f(2, 32))
    with pytest.raises(ValueError):
        rq.Modulation(gate=f(2, 64), shift=f(3, 64))
    with pytest.raises(ValueError):
        rq.Modulation(gate=f(64, 2).t())
    with pytest.raises(ValueError):
        rq.Modulation(gate=f(2, 64).bfloat16())
    with pytest.raises(ValueError):
        rq.Modulation(gate=f(2, 64), shift=f(2, 128)[:, :64])       # two strides
    with pytest.raises(ValueError):
        rq.Modulation(gate=f(2, 64), index=f(4, dtype=torch.int64))
    m = rq.Modulation(*f(3, 6, 64).unbind(1)[:3], per=5)
    assert (m.c.rows, m.c.ld, m.c.per) == (3, 384, 5)
    x, n = f(4, 64), rq.Norm(64)
    for bad in (lambda: rq.block_norm(x, x, rq.Norm(32)), lambda: rq.block_norm(x, x, n, mod=rq.Modulation(gate=f(1, 32))),
                lambda: rq.block_norm(x, x, n, mod=rq.Modulation(gate=f(1, 64), index=f(3, dtype=torch.int32))),
                lambda: rq.block_norm(x[None], x[None], n), lambda: rq.block_norm(x, x, n)):   # (the last: host memory)
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        rq.block_norm(x, x, n, h=x.bfloat16())
    with pytest.raises(TypeError):
        rq.block_norm(x, x, n, y=x.bfloat16())


def test_binding_states():
    kv = torch.zeros(2, 10, 2, 4, 64, dtype=torch.bfloat16)
    s = rq.States(kv[:, :, 0], kv[:, :, 1])
    assert (s.c.k_ld, s.c.k_stride, s.c.heads, s.c.keys, s.c.batch) == (512, 5120, 4, 10, 2)
    assert s.c.v == s.c.k + 512
    one = kv[:1, :, 0].expand(3, 10, 4, 64)
    assert rq.States(one, one).c.k_stride == 0
    for bad in (dict(k=kv[:, :, 0], v=kv[:, :5, 1]), dict(k=kv[0], v=kv[0, :, :1]),
                dict(k=kv[:, :, 0].transpose(1, 2), v=kv[:, :, 0].transpose(1, 2)),
                dict(k=kv[:, :, 0], v=kv[:, :, 1], lens=torch.zeros(3, dtype=torch.int32)),
                dict(k=kv[:, :, 0], v=kv[:, :, 1], lens=torch.zeros(2, dtype=torch.int64)),
                dict(k=kv[:, :, 0], v=kv[:, :, 1], mask=torch.zeros(2, 9, dtype=torch.uint8)),
                dict(k=kv[:, :, 0], v=kv[:, :, 1], mask=torch.zeros(10, 2, dtype=torch.uint8).t())):
        with pytest.raises(ValueError):
            rq.States(**bad)
    with pytest.raises(TypeError):
        rq.States(kv[:, :, 0].float(), kv[:, :, 1].float())
    with pytest.raises(TypeError):
        rq.States(kv[:, :, 0], kv[:, :, 1], mask=torch.zeros(2, 10))
    q = torch.zeros(2, 3, 8, 64)
    for bad in (dict(q=q, out=q[:, :2]), dict(q=q[0], out=q[0]), dict(q=q[:1], out=q[:1]), dict(q=q[..., :32], out=q[..., :32]),
                dict(q=q, out=q.clone())):      # (the last: host memory)
        with pytest.raises(ValueError):
            rq.cross_attention(states=s, **bad)
    with pytest.raises(TypeError):
        rq.cross_attention(q, s, q.bfloat16())
    with pytest.raises(TypeError):
        rq.cross_attention_workspace_bytes(s, 3, 8, torch.float16)
    assert rq.cross_attention_workspace_bytes(s, 3, 8, torch.bfloat16) >= 0
    with pytest.raises(rq.RQError):
        rq.cross_attention_workspace_bytes(s, 3, 9, torch.bfloat16)


# ------------------------------------------------------------------ the plain forms

def test_plain_norm_against_torch():
    rng = np.random.default_rng(0)
    x, y = rng.standard_normal((2, 6, 40))
    w, b = rng.standard_normal((2, 40))
    g, s, c = rng.standard_normal((3, 6, 40))
    h, z, dh, dz = A.block_norm(x, y, ("layer", w, b, 1e-5), ("rms", w, None, 1e-3), g, s, c, 0.5, 2.0)
    t = torch.from_numpy
    branch = torch.nn.functional.layer_norm(t(y), (40,), t(w), t(b), 1e-5) * t(g) * 2
    th = t(x) * 0.5 + branch
    tz = th * torch.rsqrt((th ** 2).mean(-1, keepdim=True) + 1e-3) * t(w) * (1 + t(c)) + t(s)
    np.testing.assert_allclose(h, th.numpy(), rtol=1e-12, atol=1e-12)
    np.testing.assert_allclose(z, tz.numpy(), rtol=1e-12, atol=1e-12)
    assert (dh > 0).all() and (dh < 1e-3).all() and (dz > 0).all() and (dz < 5e-3).all()


def test_plain_attention_against_torch():
    rng = np.random.default_rng(1)
    q, k, v = rng.standard_normal((5, 16)), rng.standard_normal((9, 16)), rng.standard_normal((9, 16))
    out, lse, d, dl = A.attention(q, k, v, -0.3, "f32")
    s = torch.from_numpy(-0.3 * q @ k.T)
    np.testing.assert_allclose(out, (torch.softmax(s, -1) @ torch.from_numpy(v)).numpy(), rtol=1e-12)
    np.testing.assert_allclose(lse, torch.logsumexp(s, -1).numpy(), rtol=1e-12)
    assert (d > 0).all() and (d < 1e-4).all() and (dl < 1e-4).all()
    out, lse, d, dl = A.attention(q, k[:0], v[:0], 1.0, "f32")
    assert (out == 0).all() and np.isneginf(lse).all()


# ------------------------------------------------------------------ the blocks' own bookkeeping

def _weights(*shapes):
    rng = np.random.default_rng(0)
    return [rng.standard_normal(s).astype(np.float32) for s in shapes]


def test_decode_block_behind_a_prefix(monkeypatch):
    from rotated_w4a4_quantized_amd import attention
    calls = []
    hidden, hq, hkv, D, B, page = 128, 4, 2, 32, 3, 16
    Ws = _weights(((hq + 2 * hkv) * D, hidden), (hidden, hq * D))
    blk = attention.DecodeAttention(*Ws, hq, hkv, D, B, max_len=50, page=page, device="cpu", prefix=40)
    for name in ("rotate_quant", "w4a4_linear", "paged_attention", "cache_evict"):
        monkeypatch.setattr(rq, name, lambda *a, _n=name, **k: calls.append((_n, a, k)))
    monkeypatch.setattr(rq, "qk_norm_rope", lambda *a, **k: calls.append(("store", k["cache"], {n: k[n].tolist() for n in ("positions", "place")},
                                                                          k["seq"].tolist() if k.get("seq") is not None else None)))
    monkeypatch.setattr(rq, "prefix_attention", lambda *a, **k: calls.append(("prefix", a[3], k["max_len"], a[4].tolist())))
    x = torch.zeros(B, hidden, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        blk.step(x)                                    # no prefix yet
    for bad in (torch.zeros(39, hidden, dtype=torch.bfloat16), torch.zeros(41, hidden, dtype=torch.bfloat16)):
        with pytest.raises(ValueError):
            blk.set_prefix(bad)
    assert not calls
    for _ in range(2):                                 # anew
        calls.clear()
        blk.set_prefix(torch.zeros(40, hidden, dtype=torch.bfloat16))
        stored = [c for c in calls if c[0] == "store"]
        assert sum((c[2]["place"] for c in stored), []) == list(range(40)) and all(c[1] is blk.prefix_cache for c in stored)
        assert all(c[2]["place"] == c[2]["positions"] and set(c[3]) == {0} for c in stored)
        calls.clear()
        for t in range(10):
            blk.step(x)
        stored = [c for c in calls if c[0] == "store"]
        assert [c[2]["place"] for c in stored] == [[40 + t] * B for t in range(10)] and all(c[1] is blk.cache for c in stored)
        assert [c for c in calls if c[0] == "prefix"] == [("prefix", 40, 41 + t, [41 + t] * B) for t in range(10)]
        assert not [c for c in calls if c[0] in ("paged_attention", "cache_evict")]
        with pytest.raises(ValueError):
            blk.step(x)                                # past max_len
    # two full pages are shared; the third, which the prefix ends in, has copies, and no page is in two tables' own parts
    t = blk.cache.table
    assert (t[:, :2] == blk.prefix_table[:2]).all() and blk.prefix_table.tolist() == [0, 1, 2]
    own = t[:, 2:].flatten().tolist()
    assert len(set(own)) == len(own) and not set(own) & {0, 1, 2} and max(own) < blk.cache.k.shape[0]
    plain = attention.DecodeAttention(*Ws, hq, hkv, D, B, max_len=50, page=page, device="cpu")
    with pytest.raises(ValueError):
        plain.set_prefix(x)
    for kw in (dict(prefix=50), dict(prefix=-1), dict(prefix=8, budget=20)):
        with pytest.raises(ValueError):
            attention.DecodeAttention(*Ws, hq, hkv, D, B, max_len=50, page=page, device="cpu", **kw)


def test_diffusion_block_refusals(monkeypatch):
    from rotated_w4a4_quantized_amd import attention
    hidden, heads, D, batch, tokens, states, caption = 128, 2, 64, 2, 5, 7, 64
    inner = heads * D
    Ws = _weights((3 * inner, hidden), (hidden, inner), (inner, hidden), (2 * inner, caption), (hidden, inner))
    calls = []
    for name in ("rotate_quant", "w4a4_linear", "qk_norm_rope", "block_norm", "cross_attention"):
        monkeypatch.setattr(rq, name, lambda *a, _n=name, **k: calls.append((_n, a, k)))
    blk = attention.DiffusionAttention(*Ws, heads, D, batch, tokens, states, device="cpu")
    bf16 = torch.bfloat16
    x, mod = torch.zeros(batch * tokens, hidden, dtype=bf16), torch.zeros(batch, 5, hidden)
    with pytest.raises(ValueError):
        blk.step(x, mod)                               # no captions yet
    for bad in (torch.zeros(batch, 8, caption), torch.zeros(1, 3, caption), torch.zeros(batch, 0, caption), torch.zeros(batch, caption),
                torch.zeros(batch, caption, 3).transpose(1, 2)):
        with pytest.raises(ValueError):
            blk.set_caption(bad.to(bf16))
    assert not calls
    blk.set_caption(torch.zeros(batch, 3, caption, dtype=bf16), lens=torch.ones(batch, dtype=torch.int32))
    assert blk.states.keys == 3 and blk.states.c.k_stride == 3 * 2 * inner
    calls.clear()
    for bad in ((x[:-1], mod), (x, mod[:1]), (x, mod[:, :4]), (x, mod[..., :64])):
        with pytest.raises(ValueError):
            blk.step(*bad)
    assert not calls
    s = object()
    blk.step(x, mod, stream=s)
    assert [c[0] for c in calls if c[0] != "rotate_quant"] == [
        "block_norm", "w4a4_linear", "qk_norm_rope", "cross_attention", "w4a4_linear", "block_norm", "w4a4_linear",
        "cross_attention", "w4a4_linear", "block_norm"]
    assert all(c[2]["stream"] is s for c in calls)
    for i in range(5):
        with pytest.raises(ValueError):
            attention.DiffusionAttention(*[np.zeros((w.shape[0] + 8, w.shape[1]), np.float32) if j == i else w for j, w in enumerate(Ws)],
                                         heads, D, batch, tokens, states, device="cpu")
