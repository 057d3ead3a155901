"""Attention entry points without a GPU: refusals of the C ABI (every check
runs before any HIP call), workspace sizes, struct layouts and the binding's
own checks; and the plain 64-bit forms against independent values."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

from rotated_w4a4_quantized_amd import rq
from tests import _attention as A

torch = pytest.importorskip("torch")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PTR = 1 << 20   # never dereferenced: every call here is rejected or has no work


def cache(**kw):
    d = dict(dtype=rq.RQ_BF16, heads=4, head_dim=64, page=16, batch=2, table_ld=8, pages=32, k=PTR, v=PTR,
             k_scale=None, v_scale=None, table=PTR, weight=PTR, pos=PTR)
    d.update(kw)
    return rq.c_kv_cache(*[d[f] for f, _ in rq.c_kv_cache._fields_])


def norm(**kw):
    d = dict(q_heads=8, kv_heads=4, head_dim=64, rot_dim=64, interleaved=0, table_rows=100, eps=1e-6, reserved=0,
             q_weight=PTR, k_weight=PTR, cos=PTR, sin=PTR)
    d.update(kw)
    return rq.c_qk_norm(*[d[f] for f, _ in rq.c_qk_norm._fields_])


def call_norm(d=None, c=None, qkv=PTR, dtype=rq.RQ_BF16, ld=1024, T=4, positions=None, q=PTR, q_ld=512, k=PTR, k_ld=256,
              seq=None, place=PTR):
    d = norm() if d is None else d
    return rq.load().rq_qk_norm_rope(ctypes.byref(d), qkv, dtype, ld, T, positions, q, q_ld, k, k_ld,
                                     None if c is None else ctypes.byref(c), seq, place, None)


def call_attend(c=None, q=PTR, dtype=rq.RQ_BF16, q_ld=512, heads=8, scale=0.125, lens=PTR, max_len=100, mask=None, mask_ld=0,
                out=PTR, out_ld=512, lse=None, track=0, weight_out=None, ws=PTR, wsb=1 << 40):
    c = cache() if c is None else c
    return rq.load().rq_paged_attention(ctypes.byref(c), q, dtype, q_ld, heads, scale, lens, max_len, mask, mask_ld, out,
                                        out_ld, lse, track, weight_out, ws, wsb, None)


def call_evict(c=None, lens=PTR, max_len=100, keep=10, recent=2, sink=1, lens_out=PTR, weight_out=PTR, pos_out=PTR,
               ws=PTR, wsb=1 << 40):
    c = cache() if c is None else c
    return rq.load().rq_cache_evict(ctypes.byref(c), lens, max_len, keep, recent, sink, lens_out, weight_out, pos_out, ws,
                                    wsb, None)


NULL, SHAPE, DTYPE, ALIGN = -1, -2, -3, -4


def test_struct_layouts(tmp_path):
    structs = {"rq_kv_cache": rq.c_kv_cache, "rq_qk_norm": rq.c_qk_norm}
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


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=rq.RQ_F32), DTYPE), (dict(dtype=rq.RQ_I32), DTYPE), (dict(heads=0), SHAPE), (dict(heads=1025), SHAPE),
    (dict(head_dim=8), SHAPE), (dict(head_dim=68), SHAPE), (dict(head_dim=264), SHAPE), (dict(page=8), SHAPE),
    (dict(page=24), SHAPE), (dict(page=2048), SHAPE), (dict(batch=-1), SHAPE), (dict(batch=65536), SHAPE),
    (dict(table_ld=0), SHAPE), (dict(table_ld=(1 << 24) // 16 + 1), SHAPE), (dict(pages=0), SHAPE),
    (dict(pages=1 << 31), SHAPE), (dict(k=None), NULL), (dict(v=None), NULL), (dict(table=None), NULL),
    (dict(dtype=rq.RQ_I8), NULL), (dict(dtype=rq.RQ_I8, k_scale=PTR), NULL), (dict(k=PTR + 8), ALIGN),
    (dict(v=PTR + 4), ALIGN), (dict(weight=PTR + 4), ALIGN), (dict(pos=PTR + 4), ALIGN), (dict(table=PTR + 4), ALIGN),
])
def test_cache_refusals(kw, status):
    assert call_attend(cache(**kw)) == status
    assert call_evict(cache(**kw)) == status
    if "heads" not in kw and "head_dim" not in kw:
        assert call_norm(c=cache(**kw)) == status
    assert rq.load().rq_last_error()


@pytest.mark.parametrize("d,kw,status", [
    (dict(q_heads=0), {}, SHAPE), (dict(kv_heads=-1), {}, SHAPE), (dict(head_dim=60), {}, SHAPE), (dict(rot_dim=12), {}, SHAPE),
    (dict(rot_dim=72), {}, SHAPE), (dict(rot_dim=-8), {}, SHAPE), (dict(interleaved=2), {}, SHAPE),
    (dict(table_rows=0), {}, SHAPE), (dict(eps=-1.0), {}, SHAPE), (dict(eps=float("nan")), {}, SHAPE),
    (dict(eps=float("inf")), {}, SHAPE), ({}, dict(dtype=rq.RQ_I8), DTYPE), ({}, dict(dtype=rq.RQ_I32), DTYPE),
    ({}, dict(T=-1), SHAPE), ({}, dict(T=1 << 31), SHAPE), ({}, dict(ld=767), SHAPE), ({}, dict(q_ld=511), SHAPE),
    ({}, dict(k_ld=255), SHAPE), ({}, dict(qkv=None), NULL), ({}, dict(q=None), NULL), ({}, dict(k=None), NULL),
    (dict(cos=None), {}, NULL), (dict(sin=None), {}, NULL), ({}, dict(qkv=PTR + 2), ALIGN), ({}, dict(q=PTR + 8), ALIGN),
    ({}, dict(k=PTR + 8), ALIGN), ({}, dict(ld=1028), ALIGN), ({}, dict(q_ld=516), ALIGN), (dict(cos=PTR + 4), {}, ALIGN),
])
def test_qk_norm_rope_refusals(d, kw, status):
    assert call_norm(norm(**d), **kw) == status


def test_qk_norm_rope_cache_refusals():
    assert call_norm(c=cache(heads=2)) == SHAPE
    assert call_norm(c=cache(head_dim=128)) == SHAPE
    assert call_norm(c=cache(), ld=1023) == SHAPE   # the values belong to the row
    assert call_norm(c=cache(), place=None) == NULL
    assert rq.load().rq_qk_norm_rope(None, PTR, 1, 1024, 4, None, PTR, 512, PTR, 256, None, None, None, None) == NULL


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=rq.RQ_I8), DTYPE), (dict(heads=0), SHAPE), (dict(heads=6), SHAPE), (dict(heads=1028), SHAPE),
    (dict(q_ld=511), SHAPE), (dict(out_ld=511), SHAPE), (dict(max_len=-1), SHAPE), (dict(max_len=129), SHAPE),
    (dict(scale=float("nan")), SHAPE), (dict(scale=float("inf")), SHAPE), (dict(mask=PTR, mask_ld=99), SHAPE),
    (dict(track=2), SHAPE), (dict(track=1), NULL), (dict(q=None), NULL), (dict(lens=None), NULL), (dict(out=None), NULL),
    (dict(q=PTR + 8), ALIGN), (dict(out=PTR + 8), ALIGN), (dict(q_ld=516), ALIGN), (dict(out_ld=516), ALIGN),
    (dict(track=1, weight_out=PTR + 4), ALIGN),
])
def test_paged_attention_refusals(kw, status):
    assert call_attend(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(max_len=-1), SHAPE), (dict(max_len=129), SHAPE), (dict(keep=0), SHAPE), (dict(recent=-1), SHAPE),
    (dict(sink=-1), SHAPE), (dict(lens=None), NULL), (dict(lens_out=None), NULL), (dict(weight_out=None), NULL),
    (dict(pos_out=None), NULL), (dict(weight_out=PTR + 4), ALIGN), (dict(pos_out=PTR + 4), ALIGN),
    (dict(ws=None), SHAPE), (dict(wsb=4), SHAPE), (dict(ws=PTR + 4), ALIGN),
])
def test_cache_evict_refusals(kw, status):
    assert call_evict(**kw) == status


def test_evict_needs_weight_and_pos():
    assert call_evict(cache(weight=None)) == NULL
    assert call_evict(cache(pos=None)) == NULL


def test_no_work_is_ok():
    assert call_norm(T=0, qkv=None, q=None, k=None) == 0
    assert call_attend(cache(batch=0, k=None, v=None, table=None), q=None, out=None, lens=None) == 0
    assert call_evict(cache(batch=0, k=None, v=None, table=None), lens=None) == 0


def test_workspace_sizes():
    L = rq.load()
    n = ctypes.c_size_t(123)
    c = cache()
    assert L.rq_paged_attention_workspace_bytes(ctypes.byref(c), 8, 129, 0, ctypes.byref(n)) == SHAPE
    assert L.rq_paged_attention_workspace_bytes(ctypes.byref(c), 7, 100, 0, ctypes.byref(n)) == SHAPE
    assert L.rq_paged_attention_workspace_bytes(ctypes.byref(c), 8, 100, 0, None) == NULL
    assert L.rq_paged_attention_workspace_bytes(None, 8, 100, 0, ctypes.byref(n)) == NULL
    assert L.rq_cache_evict_workspace_bytes(ctypes.byref(c), 0, 100, ctypes.byref(n)) == SHAPE
    assert L.rq_cache_evict_workspace_bytes(ctypes.byref(c), 10, 100, None) == NULL
    assert L.rq_cache_evict_workspace_bytes(ctypes.byref(c), 10, 100, ctypes.byref(n)) == 0 and n.value > 0


@pytest.mark.parametrize("batch,heads,q_heads", [(1, 1, 1), (1, 8, 32), (40, 8, 8), (600, 4, 32), (3, 2, 80)])
@pytest.mark.parametrize("track", [0, 1])
def test_workspace_does_not_shrink_with_max_len(batch, heads, q_heads, track):
    """A caller that sizes its workspace for the longest call may make shorter ones."""
    L = rq.load()
    c = cache(batch=batch, heads=heads, table_ld=4096, page=16)
    last = last_evict = 0
    for max_len in [0, 1, 15, 64, 65, 128, 500, 512, 513, 1000, 2399, 2400, 2401, 5000, 9600, 20000, 65536]:
        n = ctypes.c_size_t(0)
        assert L.rq_paged_attention_workspace_bytes(ctypes.byref(c), q_heads, max_len, track, ctypes.byref(n)) == 0
        assert n.value >= last, max_len
        last = n.value
        assert L.rq_cache_evict_workspace_bytes(ctypes.byref(c), 1000, max_len, ctypes.byref(n)) == 0
        assert n.value >= last_evict
        last_evict = n.value


def test_binding_refusals():
    k = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    table = torch.zeros(1, 4, dtype=torch.int32)
    with pytest.raises(TypeError):
        rq.KVCache(k.float(), k.float(), table)
    with pytest.raises(ValueError):
        rq.KVCache(k, k[:2], table)
    with pytest.raises(ValueError):
        rq.KVCache(k, k, table.long())
    with pytest.raises(ValueError):
        rq.KVCache(k.transpose(1, 2), k.transpose(1, 2), table)
    with pytest.raises(ValueError):
        rq.KVCache(k.to(torch.int8), k.to(torch.int8), table)          # no scales
    with pytest.raises(ValueError):
        rq.KVCache(k, k, table, k_scale=torch.zeros(4, 2, 16))
    with pytest.raises(ValueError):
        rq.KVCache(k, k, table, weight=torch.zeros(1, 2, 63))
    with pytest.raises(ValueError):
        rq.QKNorm(4, 2, 64, cos=torch.zeros(8, 32))
    with pytest.raises(ValueError):
        rq.QKNorm(4, 2, 64, q_weight=torch.ones(32))
    c = rq.KVCache(k, k, table)
    q = torch.zeros(1, 256, dtype=torch.bfloat16)
    lens = torch.ones(1, dtype=torch.int32)
    with pytest.raises(ValueError):                                     # not on a GPU
        rq.paged_attention(q, c, lens, torch.zeros_like(q))
    with pytest.raises(TypeError):
        rq.paged_attention(q.half(), c, lens, q.half())
    with pytest.raises(TypeError):
        rq.paged_attention(q, c, lens, q.float())
    with pytest.raises(ValueError):
        rq.cache_evict(c, lens, 4)                                      # no weight, no pos


# ---- the plain forms themselves

def test_plain_rotation_keeps_norms_and_angles():
    """A rotation keeps the head's norm, and the product of a query and a key
    depends on the difference of their positions only."""
    rng = np.random.default_rng(0)
    D, half = 32, 16
    ang = np.arange(64)[:, None] * (100.0 ** (-np.arange(half) / half))
    cos, sin = np.cos(ang), np.sin(ang)
    x, y = rng.standard_normal((2, 1, 1, D))
    for inter in (False, True):
        f = lambda z, p: A.norm_rope(z, None, 0.0, cos, sin, [p], inter)[0][0, 0]  # noqa: E731
        assert abs(np.linalg.norm(f(x, 17)) - np.sqrt(D)) < 1e-12
        assert abs(f(x, 20) @ f(y, 13) - f(x, 40) @ f(y, 33)) < 1e-9
        assert abs(f(x, 20) @ f(y, 13) - f(x, 20) @ f(y, 14)) > 1e-6


def test_plain_attention_against_products_in_exact_cases():
    v = np.arange(12.0).reshape(4, 3)
    k = np.zeros((4, 3))
    q = np.ones((2, 3))
    out, lse, w, _, _ = A.attention(q, k, v, np.array([1, 0, 1, 0], bool), 1.0)
    assert np.allclose(out, v[[0, 2]].mean(0)) and np.allclose(lse, np.log(2)) and np.allclose(w[:, [1, 3]], 0)
    out, lse, w, _, _ = A.attention(q, k, v, np.zeros(4, bool), 1.0)
    assert not out.any() and np.all(lse == -np.inf) and not w.any()


def test_plain_eviction_by_hand():
    w = np.array([5, 1, 4, 0, 9, 2, 2, 7], np.float32)
    pos = np.arange(8)
    # budget 4, the newest one protected: 4 (9), 7 (protected), 0 (5), 2 (4)
    assert A.evict_row(w, pos, 8, 4, 1, 0) == ([(1, 4), (3, 7)], [0, 4, 2, 7])
    # order 4, 0, 2, then the two weights of 2: the lower slot
    assert A.evict_row(w, pos, 7, 4, 0, 0) == ([(1, 4), (3, 5)], [0, 4, 2, 5])
    assert A.evict_row(w, pos, 3, 4, 1, 0) == ([], [0, 1, 2])


def test_int8_rule_by_hand():
    codes, s = A.int8_rule(np.array([[0, 0, 0], [-2, 1.25, 0.005], [127, 1, -0.5]], np.float32))
    assert codes.tolist() == [[0, 0, 0], [-127, 79, 0], [127, 1, 0]]
    assert s[0] == 0 and s[2] == 1


@pytest.mark.parametrize("apart", ["cos", "sin", "q_weight", "k_weight"])
def test_head_norm_of_tables_on_several_devices_is_refused(apart):
    """The kernel takes addresses; one of host memory among the GPU's would be read there."""
    parts = dict(cos=torch.zeros(8, 32), sin=torch.zeros(8, 32), q_weight=torch.ones(64), k_weight=torch.ones(64))
    rq.QKNorm(4, 2, 64, **parts)
    parts[apart] = parts[apart].to("meta")
    with pytest.raises(ValueError):
        rq.QKNorm(4, 2, 64, **parts)


def test_workspace_of_the_binding():
    """A repeated element claims bytes that are not there."""
    ws = torch.zeros(64, dtype=torch.uint8)
    assert rq._workspace(None) == (None, 0) and rq._workspace(ws) == (ws.data_ptr(), 64)
    for bad in (ws[:1].expand(1 << 20), ws[::2], ws.reshape(8, 8).t()):
        with pytest.raises(ValueError):
            rq._workspace(bad)


@pytest.mark.parametrize("batch,heads,q_heads,max_len,track,status", [
    (65535, 1024, 1024, 64, 0, 0), (65535, 16, 16, 2048, 0, 0), (4096, 64, 64, 65536, 0, 0),
    (65535, 1024, 1024, 1024, 1, SHAPE), (4096, 64, 64, 65536, 1, 0),   # (one workgroup a row: nothing to join)
    (8192, 32, 1024, 65536, 1, SHAPE), (16384, 1024, 1024, 513, 1, SHAPE),
    (16384, 512, 512, 513, 1, 0)])
def test_attention_grids_that_no_launch_holds(batch, heads, q_heads, max_len, track, status):
    """Refused by their sizes, also when the workspace is asked for, before anything is launched."""
    n = ctypes.c_size_t(0)
    c = cache(batch=batch, heads=heads, table_ld=4096)
    assert rq.load().rq_paged_attention_workspace_bytes(ctypes.byref(c), q_heads, max_len, track, ctypes.byref(n)) == status
    if status:
        row = q_heads * 64
        assert call_attend(c, heads=q_heads, max_len=max_len, track=track, weight_out=PTR, q_ld=row, out_ld=row, wsb=1 << 62) == status
        assert b"launch" in rq.load().rq_last_error()


@pytest.mark.parametrize("batch,heads,keep,max_len,status", [
    (4096, 1023, 1, 2, 0), (4096, 1024, 1, 2, SHAPE), (65535, 1024, 100, 100, SHAPE), (65535, 64, 256, 1000, SHAPE),
    (65535, 32, 448, 1000, 0), (65535, 32, 512, 1000, SHAPE), (16384, 1, 65536, 65536, 0), (1024, 64, 30000, 65536, SHAPE)])
def test_eviction_grids_that_no_launch_holds(batch, heads, keep, max_len, status):
    n = ctypes.c_size_t(0)
    c = cache(batch=batch, heads=heads, table_ld=4096)
    assert rq.load().rq_cache_evict_workspace_bytes(ctypes.byref(c), keep, max_len, ctypes.byref(n)) == status
    if status:
        assert call_evict(c, keep=keep, max_len=max_len, wsb=1 << 62) == status
        assert b"launch" in rq.load().rq_last_error()


def test_a_single_row_may_be_followed_by_any_number_of_elements():
    """The row stride of one row is never used, so its multiple does not matter."""
    row = torch.zeros(1, 67)
    assert rq._rows(row, 1, 64, "q") == (row.data_ptr(), 64)
    two = torch.zeros(2, 67)
    assert rq._rows(two, 2, 64, "q") == (two.data_ptr(), 67)
    assert rq._rows(two[:0], 0, 64, "q")[1] == 64
    with pytest.raises(ValueError):
        rq._rows(torch.zeros(1, 63), 1, 64, "q")
