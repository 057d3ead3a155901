"""The operators between blocks and attention to shared keys as they are used: in
runs with the linears, on other streams, captured into graphs and replayed, and at
offsets past 32 bits.  The bounds are derived in tests/_blocks.py."""
import numpy as np
import pytest

from rotated_w4a4_quantized_amd import attention, rq
from tests import _blocks as A
from tests.test_blocks_gpu import check_prefix, num, prefix_plain, rand, run_cross, run_prefix, same_bits, within

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def weights(rng, *shapes):
    return [(rng.standard_normal(s) * 0.05).astype(np.float32) for s in shapes]


# ------------------------------------------------------------------ runs

@pytest.mark.parametrize("batch,tokens,states", [(1, 40, 9), (3, 130, 33)])
def test_diffusion_block_is_its_stages(batch, tokens, states, monkeypatch):
    """Every operator of a step gets the bits that the one before it left, and
    gives the formula's values for them."""
    rng = np.random.default_rng(batch)
    hidden, heads, D, caption = 256, 4, 72, 128
    inner, T = heads * D, batch * tokens
    blk = attention.DiffusionAttention(*weights(rng, (3 * inner, hidden), (hidden, inner), (inner, hidden), (2 * inner, caption),
                                                (hidden, inner)), heads, D, batch, tokens, states)
    text = rand(rng, (batch, states, caption), "bf16")[0]
    lens = rng.integers(1, states + 1, batch)
    lens[-1] = states
    blk.set_caption(text, lens=torch.from_numpy(lens.astype(np.int32)).cuda())
    x, xn = rand(rng, (T, hidden), "bf16", 2.0)
    mod, modn = rand(rng, (batch, 5, hidden), "f32", 0.3)
    seen = []

    def spy(name, outs):
        real = getattr(rq, name)

        def f(*a, **k):
            real(*a, **k)
            seen.append((name, a, dict(k), [o.clone() for o in outs(a, k)]))
        monkeypatch.setattr(rq, name, f)

    spy("block_norm", lambda a, k: [t for t in (k.get("h"), a[1]) if t is not None])
    spy("qk_norm_rope", lambda a, k: [a[2], k["k_out"], a[1]])
    spy("cross_attention", lambda a, k: [a[2], a[0]])
    spy("w4a4_linear", lambda a, k: [a[3]])
    h, z = blk.step(x, mod)
    assert [s[0] for s in seen] == ["block_norm", "w4a4_linear", "qk_norm_rope", "cross_attention", "w4a4_linear", "block_norm",
                                    "w4a4_linear", "cross_attention", "w4a4_linear", "block_norm"]
    out = [s[3] for s in seen]
    row = np.arange(T) // tokens
    shift, scale, gate, mlp_shift, mlp_scale = (modn[row, i].astype(np.float64) for i in range(5))
    ln = ("layer", None, None, float(np.float32(1e-6)))

    def norms(got_h, got_z, xv, yv, gate, shift, scale):
        hn, zn, dh, dz = A.block_norm(xv, yv, None, ln, gate, shift, scale, 1.0, 1.0)
        if got_h is not None:
            within(num(got_h), hn, dh * 1.01 + A.half_step("bf16") * np.abs(hn), "h")
        within(num(got_z), zn, dz * 1.01 + A.half_step("bf16") * np.abs(zn), "z")

    norms(None, out[0][0], xn, None, None, shift, scale)
    # the projections, recomputed from what came before, give the same bits
    def linear(layer, X, N):
        Y = torch.empty((T, N), dtype=torch.bfloat16, device="cuda")
        layer(X.contiguous(), Y)
        return Y
    real_seen = len(seen)
    assert same_bits(linear(blk.qkv_proj, out[0][0], 3 * inner), out[1][0])
    q, k_rot, qkv = out[2]
    v = qkv[:, 2 * inner:]
    assert same_bits(v, out[1][0][:, 2 * inner:]), "values pass the head norm"

    def attend(got, q, k, v, lens):
        g, qn, kn, vn = (num(t).reshape(batch, -1, heads, D) for t in (got, q, k, v))
        for b in range(batch):
            for i in range(heads):
                n = int(lens[b])
                o, _, d, _ = A.attention(qn[b, :, i], kn[b, :n, i], vn[b, :n, i], D ** -0.5, "bf16")
                within(g[b, :, i], o, d, f"attention of sample {b}, head {i}")

    attend(out[3][0], q, k_rot, v, [tokens] * batch)
    assert same_bits(linear(blk.out_proj, out[3][0].view(T, inner), hidden), out[4][0])
    norms(out[5][0], out[5][1], xn, num(out[4][0]), gate, None, None)
    assert same_bits(linear(blk.q_proj, out[5][1], inner), out[6][0])
    kv = blk.kv.view(batch, states, 2, inner)
    attend(out[7][0], out[6][0], kv[:, :, 0], kv[:, :, 1], lens)
    assert same_bits(linear(blk.caption_out, out[7][0].view(T, inner), hidden), out[8][0])
    norms(out[9][0], out[9][1], num(out[5][0]), num(out[8][0]), None, mlp_shift, mlp_scale)
    assert same_bits(h, out[9][0]) and same_bits(z, out[9][1]) and real_seen == 10
    # the stream that a step returned may go into the next, and another stream gives the same bits
    twice = blk.step(h, mod)[0].clone()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    blk.step(x, mod, stream=s)
    blk.step(blk.h, mod, stream=s.cuda_stream)
    s.synchronize()
    assert same_bits(blk.h, twice)


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("B,prefix", [(3, 33), (40, 64)])
def test_decode_block_with_a_shared_prefix(B, prefix, int8):
    """Steps behind a shared prefix: keys and values are those of a block that
    stores the prefix for every sequence, and attention is the formula's."""
    rng = np.random.default_rng(50)
    hidden, hq, hkv, D, steps, page = 128, 8, 2, 64, 20, 16
    Ws = weights(rng, ((hq + 2 * hkv) * D, hidden), (hidden, hq * D))
    blk = attention.DecodeAttention(*Ws, hq, hkv, D, B, max_len=prefix + steps, page=page, int8=int8, prefix=prefix)
    each = attention.DecodeAttention(*Ws, hq, hkv, D, B, max_len=prefix + steps, page=page, int8=int8)
    front, _ = rand(rng, (prefix, hidden), "bf16")
    for again in range(2):
        blk.set_prefix(front)
        if not again:
            for t in range(prefix):
                each.step(front[t].expand(B, hidden).contiguous())
        for t in range(steps if again else 3):
            x, _ = rand(rng, (B, hidden), "bf16")
            y = blk.step(x)
            assert torch.isfinite(y.float()).all() and blk.lens.tolist() == [prefix + t + 1] * B
            c, n = blk.cache, prefix + t + 1
            val = {"k": num(c.k), "v": num(c.v)}
            if int8:
                val = {m: val[m] * num(getattr(c, m + "_scale"))[..., None] for m in "kv"}
            lse = torch.full((B, hq), 0.0, device="cuda")
            got, lse = run_prefix(blk.q, c, blk.prefix_table, prefix, blk.lens, n, hq)
            assert same_bits(got, blk.attn)
            check_prefix(blk.attn, lse, num(blk.q).astype(np.float32), c.table.cpu().numpy(), blk.prefix_table.cpu().numpy(), val,
                         [n] * B, prefix, n - prefix, page, c.k.shape[0], hq, hkv, D, None, "bf16")
    # the prefix's keys and values are those of the tokens stored one by one
    for h in range(hkv):
        k, v = prefix_plain(1, blk.cache.table.cpu().numpy(), blk.prefix_table.cpu().numpy(), val, prefix, prefix, page, blk.cache.k.shape[0], None, h)
        e = each.cache
        at = torch.arange(prefix, device="cuda")
        pg = e.table[1].long()[at // page]
        for got, name in ((k, "k"), (v, "v")):
            w = num(getattr(e, name)[pg, h, at % page])
            if int8:
                w = w * num(getattr(e, name + "_scale")[pg, h, at % page])[:, None]
            assert np.array_equal(got, w)


def test_commands_run(capsys):
    attention.main(["--steps", "6", "--batch", "2", "--prefix", "100"])
    assert "6 steps of 2 sequences" in capsys.readouterr().out
    attention.main(["--steps", "3", "--batch", "2", "--diffusion"])
    assert "3 steps of 2 samples" in capsys.readouterr().out


# ------------------------------------------------------------------ graphs and streams

def _program(rng):
    """Inputs, results and a function that runs every operator on them."""
    T, K, B, hq, hkv, D = 50, 256, 2, 4, 2, 64
    x, y = rand(rng, (T, K), "f32")[0], rand(rng, (T, K), "bf16")[0]
    mod = rq.Modulation(*rand(rng, (2, 3, K), "f32")[0].unbind(1), per=25)
    pre = rq.Norm(K, "layer")
    q = rand(rng, (B, 300, hq, D), "bf16")[0]
    few = rand(rng, (B, 3, hq, D), "f32")[0]
    kv = rand(rng, (B, 1500, 2, hkv, D), "bf16")[0]
    lens = torch.tensor([1500, 700], dtype=torch.int32, device="cuda")
    st = rq.States(kv[:, :, 0], kv[:, :, 1], lens=lens)
    pool = rand(rng, (60, hkv, 16, D), "bf16")[0]
    cache = rq.KVCache(pool, pool.clone(), torch.arange(48, dtype=torch.int32, device="cuda").reshape(4, 12))
    front = torch.arange(50, 58, dtype=torch.int32, device="cuda")
    q1 = rand(rng, (4, hq * D), "bf16")[0]
    lens1 = torch.tensor([190, 128, 0, 150], dtype=torch.int32, device="cuda")
    bf16, f32 = torch.bfloat16, torch.float32
    n = max(rq.cross_attention_workspace_bytes(st, 300, hq, bf16), rq.cross_attention_workspace_bytes(st, 3, hq, f32),
            rq.prefix_attention_workspace_bytes(cache, hq, 128, 192, bf16))
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    outs = [torch.zeros_like(t) for t in (x, y, q, few, q1)]

    def run():
        rq.block_norm(x, outs[1], pre, y=y, h=outs[0], mod=mod)
        rq.cross_attention(q, st, outs[2], workspace=ws)
        rq.cross_attention(few, st, outs[3], workspace=ws)
        rq.prefix_attention(q1, cache, front, 128, lens1, outs[4], max_len=192, workspace=ws)

    def change(seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        for t in (x, y, q, few, q1, kv, pool):
            t.copy_(torch.randn(t.shape, generator=g, device="cuda").to(t.dtype))
        lens.copy_(torch.tensor([1500 - 7 * seed, 300 * seed], dtype=torch.int32))
        lens1.copy_(torch.tensor([128 + seed, 192, 130, 0], dtype=torch.int32))
    return run, change, outs


def test_captured_and_replayed():
    rng = np.random.default_rng(60)
    run, change, outs = _program(rng)
    run()
    torch.cuda.synchronize()
    graph, other = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    with torch.cuda.graph(other):       # two graphs on one workspace, one after the other
        run()
    for seed in range(1, 5):
        change(seed)
        (graph if seed % 2 else other).replay()
        got = [o.clone() for o in outs]
        torch.cuda.synchronize()
        for o in outs:
            o.fill_(3.0)
        run()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(got, outs)):
            assert same_bits(a, b), (seed, i)


def test_two_programs_on_two_streams():
    programs = [_program(np.random.default_rng(61 + i)) for i in range(2)]
    want = []
    for run, _, outs in programs:
        run()
        torch.cuda.synchronize()
        want.append([o.clone() for o in outs])
        for o in outs:
            o.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in programs]
    for _ in range(3):
        for s, (run, _, _) in zip(streams, programs):
            with torch.cuda.stream(s):
                run()
    torch.cuda.synchronize()
    for w, (_, _, outs) in zip(want, programs):
        for a, b in zip(w, outs):
            assert same_bits(a, b)


# ------------------------------------------------------------------ far offsets

def test_offsets_past_32_bits():
    rng = np.random.default_rng(70)
    # states whose tokens lie 2 MB apart: the last are 6 GB behind the first
    S, hkv, D, ld = 3000, 2, 64, 1 << 20
    memory = torch.empty(3 << 30, dtype=torch.bfloat16, device="cuda")
    pool = memory[:S * ld].view(S, ld)
    kv, kvn = rand(rng, (1, S, 2, hkv, D), "bf16")
    pool[:, :2 * hkv * D] = kv.view(S, -1)
    far = pool[:, :2 * hkv * D].view(1, S, 2, hkv, D)
    for Tq in (2, 200):
        q, _ = rand(rng, (1, Tq, 4, D), "bf16", 1.5)
        a, la = run_cross(q, kv[:, :, 0], kv[:, :, 1], None, None, None, None)
        b, lb = run_cross(q, far[:, :, 0], far[:, :, 1], None, None, None, None)
        assert same_bits(a, b) and same_bits(la, lb)
    # sequences and rows more than 4 GB apart
    x, _ = rand(rng, (3, 1024), "bf16")
    rows = memory.view(3, 1 << 30)
    rows[:, :1024] = x
    pre = rq.Norm(1024, "rms")
    z = torch.empty_like(x)
    rq.block_norm(x, z, pre)
    rq.block_norm(rows[:, :1024], rows[:, 2048:3072], pre)
    assert same_bits(rows[:, 2048:3072], z)
    rows[:2, :1000 * hkv * D] = kv[0, :1000, 0].reshape(1, -1)
    two = rows[:2, :1000 * hkv * D].view(2, 1000, hkv, D)
    q, _ = rand(rng, (2, 150, 4, D), "bf16")
    near = kv[:, :1000, 0].expand(2, 1000, hkv, D)
    a, _ = run_cross(q, two, two, None, None, None, None)
    b, _ = run_cross(q, near, near, None, None, None, None)
    assert same_bits(a, b)
    del memory, pool, rows, far, two
    # pages past 4 GB of a cache
    pages = 70000
    big = torch.empty(pages, hkv, 256, D, dtype=torch.bfloat16, device="cuda")
    small, _ = rand(rng, (12, hkv, 256, D), "bf16")
    at = torch.tensor([69999, 3, 69990, 65000, 7, 50000, 60001, 68000, 1, 69000, 40000, 66000], device="cuda")
    big[at] = small
    table = torch.arange(4, 12, dtype=torch.int32, device="cuda").reshape(2, 4)
    lens = torch.tensor([1500, 1100], dtype=torch.int32, device="cuda")
    q, _ = rand(rng, (2, 4 * D), "bf16")
    near = rq.KVCache(small, small, torch.cat([torch.zeros(2, 4, dtype=torch.int32, device="cuda"), table], 1).contiguous())
    away = rq.KVCache(big, big, at[near.table.long()].to(torch.int32))
    front = torch.arange(4, dtype=torch.int32, device="cuda")
    a, la = run_prefix(q, near, front, 1000, lens, 1500, 4)
    b, lb = run_prefix(q, away, at[:4].to(torch.int32), 1000, lens, 1500, 4)
    assert same_bits(a, b) and same_bits(la, lb)


def test_buffers_of_another_place_are_refused():
    rng = np.random.default_rng(80)
    run, _, _ = _program(rng)
    x = rand(rng, (4, 64), "bf16")[0]
    with pytest.raises(ValueError):
        rq.block_norm(x, x.cpu(), rq.Norm(64))
    with pytest.raises(ValueError):
        rq.block_norm(x, torch.empty_like(x), rq.Norm(64, weight=torch.ones(64)))
    kv = rand(rng, (1, 8, 2, 1, 64), "bf16")[0]
    st = rq.States(kv[:, :, 0].cpu(), kv[:, :, 1].cpu())
    q = rand(rng, (1, 2, 1, 64), "bf16")[0]
    with pytest.raises(ValueError):
        rq.cross_attention(q, st, torch.empty_like(q))
    with pytest.raises(ValueError):
        rq.cross_attention(q, rq.States(kv[:, :, 0], kv[:, :, 1]), torch.empty_like(q), workspace=torch.empty(64, dtype=torch.uint8))
