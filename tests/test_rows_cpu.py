"""Attention to shared keys, and the diffusion block on it, without a GPU: that the GPU tests' cases reach every
kernel that a call can (by the rules of choice written out in tests/_rows.py, which
the library's workspace sizes confirm)."""
import ctypes

import pytest

from rotated_w4a4_quantized_amd import rq
from tests import _rows as R
from tests import test_blocks_gpu, test_rows_gpu
from tests.test_blocks_cpu import BF16, F32, SHAPE, _weights, cache, call_cross, call_prefix, ref, states

torch = pytest.importorskip("torch")


def test_the_cases_reach_every_kernel():
    names = set()
    for c in test_blocks_gpu.CROSS + test_rows_gpu.CROSS:
        names |= R.cross(*c[:7], lens=c[7])[0]
    for c in test_blocks_gpu.PREFIX + test_rows_gpu.PREFIX:
        names |= R.prefix(*c[:8])[0]
    assert names == R.every()


@pytest.mark.skipif(torch.cuda.is_available(), reason="the rules are written out for 256 CUs, which the library assumes without a GPU")
def test_the_rules_are_the_library_s():
    n = ctypes.c_size_t(0)
    for c in test_blocks_gpu.CROSS + test_rows_gpu.CROSS:
        B, Tq, S, hq, hkv, D, dtype = c[:7]
        st = states(batch=B, keys=S, heads=hkv, head_dim=D)
        assert rq.load().rq_cross_attention_workspace_bytes(ref(st), Tq, hq, BF16 if dtype == "bf16" else F32, ctypes.byref(n)) == 0
        assert n.value == R.cross(*c[:7], lens=c[7])[1], c
    for c in test_blocks_gpu.PREFIX + test_rows_gpu.PREFIX:
        B, P, L, hq, hkv, D, dtype, kind, page = c[:9]
        ch = cache(batch=B, heads=hkv, head_dim=D, page=page, table_ld=-(-(P + L) // page), dtype=BF16 if kind == "bf16" else rq.RQ_I8,
                   k_scale=1 << 20, v_scale=1 << 20)
        assert rq.load().rq_prefix_attention_workspace_bytes(ref(ch), hq, BF16 if dtype == "bf16" else F32, P, P + L, ctypes.byref(n)) == 0
        assert n.value == R.prefix(*c[:8])[1], c


@pytest.mark.parametrize("heads,G,fits", [(256, 1, True), (300, 1, True), (512, 1, True), (513, 1, False), (256, 2, True), (171, 3, False)])
def test_the_limit_of_rows_is_the_stated_one(heads, G, fits):
    """batch * queries * q_heads < 2^25, however many workgroups that takes."""
    n = ctypes.c_size_t(0)
    assert (65535 * heads * G < 1 << 25) == fits
    want = 0 if fits else SHAPE
    st = states(batch=65535, heads=heads, head_dim=16, keys=3)
    assert rq.load().rq_cross_attention_workspace_bytes(ref(st), 1, heads * G, BF16, ctypes.byref(n)) == want
    for prefix, max_len in ((0, 16), (3, 16)):
        c = cache(batch=65535, heads=heads, head_dim=16, table_ld=1, pages=1)
        assert rq.load().rq_prefix_attention_workspace_bytes(ref(c), heads * G, BF16, prefix, max_len, ctypes.byref(n)) == want
    if not fits:
        assert b"2^25" in rq.load().rq_last_error()


@pytest.mark.parametrize("scale", [3e38, -2.0 ** 127 * 1.001, float("inf"), float("nan")])
def test_scales_that_overflow_are_refused(scale):
    """scale log2(e) has to be finite, too, or a score of 0 would be 0 times infinity."""
    assert call_cross(scale=scale) == SHAPE
    assert call_prefix(scale=scale) == SHAPE
    assert call_cross(states(batch=0), scale=2.0 ** 127) == 0 and call_prefix(cache(batch=0), scale=-2.0 ** 127) == 0


def test_diffusion_block_refuses_a_stream_of_another_type(monkeypatch):
    """Before anything runs."""
    from rotated_w4a4_quantized_amd import attention
    hidden, heads, D, batch, tokens, caption = 128, 2, 64, 2, 5, 64
    inner, calls = heads * D, []
    for name in ("rotate_quant", "w4a4_linear", "qk_norm_rope", "block_norm", "cross_attention"):
        monkeypatch.setattr(rq, name, lambda *a, _n=name, **k: calls.append(_n))
    blk = attention.DiffusionAttention(*_weights((3 * inner, hidden), (hidden, inner), (inner, hidden), (2 * inner, caption), (hidden, inner)),
                                       heads, D, batch, tokens, 7, device="cpu")
    blk.set_caption(torch.zeros(batch, 3, caption, dtype=torch.bfloat16))
    calls.clear()
    for dtype in (torch.float32, torch.float16):
        with pytest.raises(TypeError):
            blk.step(torch.zeros(batch * tokens, hidden, dtype=dtype), torch.zeros(batch, 5, hidden))
    assert not calls
