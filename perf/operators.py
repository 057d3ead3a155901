"""The attention-side operators of a transformer block around the rotated
low-bit linears, as cases to time and to compare:

  qknorm  RMS norm of every query and key head with the position rotation in
          the same pass; optionally stores the keys and values in a paged cache
  attend  attention of one new token per sequence over a paged cache
  evict   shrinks every sequence's cache to a budget by accumulated weight

`run` computes them in plain 32-bit torch operations, or with the package's
kernels where `own` is true.
"""
import math

import torch

own = False

EPS = 1e-6
DEVICE = "cuda"


def _case(op, name, **kw):
    return dict(op=op, name=name, **kw)


def listed():
    return [
        # one new token of one sequence: the per-layer latency of single-stream generation
        _case("qknorm", "qknorm_step", T=1, hq=32, hkv=8, D=128, rot=128, inter=False, dtype="bf16", cache="bf16", page=64),
        # a decode batch that writes an int8 cache
        _case("qknorm", "qknorm_step_int8", T=61, hq=32, hkv=8, D=128, rot=128, inter=False, dtype="bf16", cache="int8", page=32),
        # a prompt of odd length in fp32 with partial rotation (half of each head), stored in a cache
        _case("qknorm", "qknorm_prompt_f32", T=1999, hq=16, hkv=4, D=64, rot=32, inter=False, dtype="f32", cache="bf16", page=16),
        # every token of a video diffusion transformer step (1536 features, 12 heads), no cache
        _case("qknorm", "qknorm_video", T=32760, hq=12, hkv=12, D=128, rot=128, inter=True, dtype="bf16", cache="none", page=16),
        # one sequence, short context, heads without sharing
        _case("attend", "attend_short", B=1, L=333, hq=12, hkv=12, D=128, dtype="bf16", cache="bf16", page=16, ragged=False, track=False, mask=False),
        # one sequence, long context: few rows, all the work along the cache
        _case("attend", "attend_long", B=1, L=131071, hq=32, hkv=8, D=128, dtype="bf16", cache="bf16", page=64, ragged=False, track=False, mask=False),
        # a serving batch of uneven lengths, with the weights that eviction needs
        _case("attend", "attend_batch", B=64, L=8190, hq=32, hkv=8, D=128, dtype="bf16", cache="bf16", page=32, ragged=True, track=True, mask=False),
        # the same kind of batch on an int8 cache
        _case("attend", "attend_int8", B=48, L=8190, hq=32, hkv=8, D=128, dtype="bf16", cache="int8", page=64, ragged=True, track=False, mask=False),
        # fp32 queries, small heads, a mask that leaves holes and one empty sequence
        _case("attend", "attend_mask_f32", B=9, L=2047, hq=16, hkv=4, D=64, dtype="f32", cache="bf16", page=16, ragged=True, track=True, mask=True),
        # one sequence that went a little over its budget
        _case("evict", "evict_step", B=1, L=2080, keep=2048, recent=256, sink=4, hkv=8, D=128, cache="bf16", page=16, ragged=False),
        # long prompts of a batch cut down to their budget
        _case("evict", "evict_prompt", B=16, L=32749, keep=4096, recent=1024, sink=4, hkv=8, D=128, cache="bf16", page=64, ragged=True),
        # a batch on an int8 cache in steady state
        _case("evict", "evict_int8", B=32, L=4352, keep=4096, recent=512, sink=0, hkv=8, D=128, cache="int8", page=32, ragged=False),
    ]


def _log(rng, lo, hi):
    """A whole number, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["qknorm", "attend", "evict"])
    page = rng.choice([16, 32, 64, 128])
    hq, hkv = rng.choice([(12, 12), (32, 8), (16, 4), (16, 2), (8, 1), (20, 4), (28, 4), (32, 1)])
    D = rng.choice([64, 80, 96, 128, 128, 128, 256])
    if op == "qknorm":
        top = 32760 * 24 * 128 // ((hq + 2 * hkv) * D) // 2
        return dict(op=op, T=_log(rng, 1, top), hq=hq, hkv=hkv, D=D, rot=rng.choice([D, D, D // 2 // 8 * 8]),
                    inter=rng.random() < 0.5, dtype=rng.choice(["bf16", "bf16", "f32"]),
                    cache=rng.choice(["none", "bf16", "int8"]), page=page)
    cache = rng.choice(["bf16", "bf16", "int8"])
    if op == "attend":
        B = _log(rng, 1, 128)
        top = min(131072, 64 * 4000 * 8 * 128 // (B * hkv * D))
        return dict(op=op, B=B, L=_log(rng, 1, max(2, top)), hq=hq, hkv=hkv, D=D, dtype=rng.choice(["bf16", "bf16", "f32"]),
                    cache=cache, page=page, ragged=rng.random() < 0.6, track=rng.random() < 0.5, mask=rng.random() < 0.25)
    B = _log(rng, 1, 32)
    L = _log(rng, 64, min(32768, 16 * 16000 * 8 * 128 // (B * hkv * D)))
    keep = max(1, int(L * rng.uniform(0.1, 0.98)))
    return dict(op=op, B=B, L=L, keep=keep, recent=int(keep * rng.uniform(0, 0.6)), sink=rng.choice([0, 0, 4]) if keep > 16 else 0,
                hkv=hkv, D=D, cache=cache, page=page, ragged=rng.random() < 0.5)


# ---------------------------------------------------------------- inputs

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _lens(case, gen):
    """Lengths of the sequences: all L, or spread below it with the longest L and, from three on, an empty one."""
    B, L = case["B"], case["L"]
    lens = torch.full((B,), L, dtype=torch.int32, device=DEVICE)
    if case["ragged"]:
        lens = (torch.rand(B, generator=gen, device=DEVICE) * L).to(torch.int32) + 1
        lens.clamp_(max=L)
        lens[0] = L
        if B > 2:
            lens[1] = 0
    return lens


def _pages(B, L, page, gen):
    """A page table [B][pages a sequence] of distinct pages in random order, and the number of pages."""
    per = -(-L // page)
    return torch.randperm(B * per, generator=gen, device=DEVICE).to(torch.int32).reshape(B, per).contiguous(), B * per


def _fill_cache(st, pages, hkv, page, D, kind, gen):
    shape = (pages, hkv, page, D)
    if kind == "int8":
        for n in ("k", "v"):
            st[n] = torch.randint(-127, 128, shape, generator=gen, device=DEVICE, dtype=torch.int8)
            # code times scale of about unit variance
            st[n + "_scale"] = (torch.rand(shape[:3], generator=gen, device=DEVICE) + 0.5) / 73.0
    else:
        for n in ("k", "v"):
            st[n] = torch.randn(shape, generator=gen, device=DEVICE, dtype=torch.bfloat16)


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(int(seed) * 7919 + 13)
    st = dict(case=dict(case))
    hkv, D, page = case["hkv"], case["D"], case["page"]
    if case["op"] == "qknorm":
        T, hq, rot = case["T"], case["hq"], case["rot"]
        dt = _TYPES[case["dtype"]]
        st["qkv"] = torch.randn(T, (hq + 2 * hkv) * D, generator=gen, device=DEVICE, dtype=dt)
        st["qw"] = 1 + 0.2 * torch.randn(D, generator=gen, device=DEVICE)
        st["kw"] = 1 + 0.2 * torch.randn(D, generator=gen, device=DEVICE)
        rows = 40960
        ang = torch.arange(rows, device=DEVICE, dtype=torch.float64)[:, None] * (
            1e4 ** (-torch.arange(0, rot, 2, device=DEVICE, dtype=torch.float64) / rot))[None]
        st["cos"], st["sin"] = ang.cos().float(), ang.sin().float()
        st["q_out"] = torch.zeros(T, hq * D, device=DEVICE, dtype=dt)
        st["k_out"] = st["positions"] = st["seq"] = st["place"] = None
        if case["cache"] == "none":
            st["k_out"] = torch.zeros(T, hkv * D, device=DEVICE, dtype=dt)
        else:
            # short calls are steps of T sequences, long ones the prompt of one
            step = T <= 256
            B, L = (T, 4 * page) if step else (1, T)
            ar = torch.arange(T, device=DEVICE, dtype=torch.int32)
            st["seq"] = ar if step else torch.zeros_like(ar)
            st["place"] = torch.randint(0, L, (T,), generator=gen, device=DEVICE, dtype=torch.int32) if step else ar
            st["positions"] = torch.randint(0, rows, (T,), generator=gen, device=DEVICE, dtype=torch.int32) if step else ar
            st["table"], pages = _pages(B, L, page, gen)
            shape = (pages, hkv, page, D)
            kind = torch.int8 if case["cache"] == "int8" else torch.bfloat16
            for n in ("k", "v"):
                st[n] = torch.zeros(shape, device=DEVICE, dtype=kind)
                if case["cache"] == "int8":
                    st[n + "_scale"] = torch.zeros(shape[:3], device=DEVICE)
    elif case["op"] == "attend":
        B, L, hq = case["B"], case["L"], case["hq"]
        st["lens"] = _lens(case, gen)
        st["table"], pages = _pages(B, L, page, gen)
        _fill_cache(st, pages, hkv, page, D, case["cache"], gen)
        # scores of a few units: some tokens matter much more than others
        st["q"] = (2 * torch.randn(B, hq * D, generator=gen, device=DEVICE)).to(_TYPES[case["dtype"]])
        st["out"] = torch.zeros_like(st["q"])
        st["lse"] = torch.zeros(B, hq, device=DEVICE)
        st["mask"] = None
        if case["mask"]:
            st["mask"] = (torch.rand(B, L, generator=gen, device=DEVICE) < 0.7).to(torch.uint8)
            st["mask"][B - 1] = 0
        if case["track"]:
            slots = st["table"].shape[1] * page
            st["weight"] = torch.rand(B, hkv, slots, generator=gen, device=DEVICE)
            st["weight_out"] = st["weight"].clone()
    else:
        B, L, keep = case["B"], case["L"], case["keep"]
        st["lens"] = _lens(case, gen)
        st["lens_out"] = torch.zeros_like(st["lens"])
        st["table"], pages = _pages(B, L, page, gen)
        _fill_cache(st, pages, hkv, page, D, case["cache"], gen)
        slots = st["table"].shape[1] * page
        # a few heavy tokens, many light ones, some that nothing ever looked at
        w = torch.exp(2 * torch.randn(B, hkv, slots, generator=gen, device=DEVICE))
        st["weight"] = torch.where(torch.rand(w.shape, generator=gen, device=DEVICE) < 0.05, torch.zeros_like(w), w)
        # what an earlier eviction left below the budget is in no order; what came since is
        pos = torch.arange(slots, device=DEVICE, dtype=torch.int32) + keep
        pos = pos.expand(B, hkv, slots).contiguous()
        pos[..., :keep] = torch.rand(B, hkv, 2 * keep, generator=gen, device=DEVICE).argsort(-1)[..., :keep].to(torch.int32)
        st["pos"] = pos
        st["weight_out"], st["pos_out"] = torch.zeros_like(st["weight"]), torch.zeros_like(pos)
    if own:   # the handles and the scratch that a program keeps beside its buffers
        from rotated_w4a4_quantized_amd import rq
        st["cache"] = rq.KVCache(st["k"], st["v"], st["table"], k_scale=st.get("k_scale"), v_scale=st.get("v_scale"),
                                 weight=st.get("weight"), pos=st.get("pos")) if "k" in st else None
        if case["op"] == "qknorm":
            st["norm"] = rq.QKNorm(case["hq"], hkv, D, st["qw"], st["kw"], st["cos"], st["sin"], eps=EPS, interleaved=case["inter"])
        elif case["op"] == "attend":
            n = rq.paged_attention_workspace_bytes(st["cache"], case["hq"], case["L"], track=case["track"])
            st["workspace"] = torch.empty(max(n, 16), dtype=torch.uint8, device=DEVICE)
        else:
            n = rq.cache_evict_workspace_bytes(st["cache"], case["keep"], case["L"])
            st["workspace"] = torch.empty(max(n, 16), dtype=torch.uint8, device=DEVICE)
    return st


# ---------------------------------------------------------------- one pass

def run(st):
    op = st["case"]["op"]
    if op == "qknorm":
        return (_qknorm_own if own else _qknorm_plain)(st)
    if op == "attend":
        return (_attend_own if own else _attend_plain)(st)
    return (_evict_own if own else _evict_plain)(st)


def _norm_rope(x, w, cos, sin, rot, inter):
    """x [T][heads][D] fp32, cos and sin [T][1][rot / 2]."""
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w
    if inter:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
    else:
        a, b = y[..., :rot // 2], y[..., rot // 2:rot]
    z = y.clone()
    if inter:
        z[..., 0:rot:2], z[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
    else:
        z[..., :rot // 2], z[..., rot // 2:rot] = a * cos - b * sin, b * cos + a * sin
    return z


def _int8(x):
    """Codes and scales of [...][D] fp32 by the symmetric 8-bit rule."""
    amax = x.abs().amax(-1)
    inv = torch.where(amax > 0, 127.0 / amax, torch.zeros_like(amax))
    return torch.round(x * inv[..., None]).clamp(-127, 127).to(torch.int8), amax / 127.0


def _stored(st):
    """What the cache now holds for the tokens of this call. int8: the values that codes and scales stand for."""
    if st["case"]["cache"] == "none":
        return {"k": st["k_out"]}
    if st["case"]["cache"] == "bf16":
        return {"k": st["k"], "v": st["v"]}
    return {n: (st[n].float() * st[n + "_scale"][..., None]).to(torch.bfloat16) for n in ("k", "v")}


def _qknorm_plain(st):
    c = st["case"]
    T, hq, hkv, D, rot, page = c["T"], c["hq"], c["hkv"], c["D"], c["rot"], c["page"]
    x = st["qkv"].float().reshape(T, hq + 2 * hkv, D)
    if st["positions"] is None:
        cos, sin = st["cos"][:T, None], st["sin"][:T, None]
    else:
        cos, sin = st["cos"][st["positions"].long()][:, None], st["sin"][st["positions"].long()][:, None]
    q = _norm_rope(x[:, :hq], st["qw"], cos, sin, rot, c["inter"])
    k = _norm_rope(x[:, hq:hq + hkv], st["kw"], cos, sin, rot, c["inter"])
    st["q_out"].copy_(q.reshape(T, hq * D))
    if c["cache"] == "none":
        st["k_out"].copy_(k.reshape(T, hkv * D))
    else:
        place = st["place"].long()
        pg, off = st["table"][st["seq"].long(), place // page].long(), place % page
        for n, y in (("k", k), ("v", x[:, hq + hkv:])):
            if c["cache"] == "int8":
                codes, scale = _int8(y)
                st[n][pg, :, off] = codes
                st[n + "_scale"][pg, :, off] = scale
            else:
                st[n][pg, :, off] = y.to(torch.bfloat16)
    return {"q": st["q_out"], **_stored(st)}


def _qknorm_own(st):
    from rotated_w4a4_quantized_amd import rq
    rq.qk_norm_rope(st["norm"], st["qkv"], st["q_out"], k_out=st["k_out"], positions=st["positions"],
                    cache=st["cache"] if st["case"]["cache"] != "none" else None, seq=st["seq"], place=st["place"])
    return {"q": st["q_out"], **_stored(st)}


def _gathered(st, n):
    """The cache in the order of the tokens: [B][hkv][slots][D] fp32."""
    x = st[n][st["table"].long()].float()                       # [B][pages][hkv][page][D]
    if n + "_scale" in st:
        x = x * st[n + "_scale"][st["table"].long()][..., None]
    B, P, H, S, D = x.shape
    return x.transpose(1, 2).reshape(B, H, P * S, D)


def _attend_plain(st):
    c = st["case"]
    B, L, hq, hkv, D = c["B"], c["L"], c["hq"], c["hkv"], c["D"]
    G = hq // hkv
    k, v = _gathered(st, "k"), _gathered(st, "v")
    slots = k.shape[2]
    keep = torch.arange(slots, device=DEVICE)[None] < st["lens"][:, None]
    if st["mask"] is not None:
        keep[:, :L] &= st["mask"] != 0
    keep = keep[:, None, :, None]
    qt = st["q"].float().reshape(B, hkv, G, D).transpose(2, 3).contiguous()
    s = torch.matmul(k, qt) / math.sqrt(D)                      # [B][hkv][slots][G]
    s = torch.where(keep, s, torch.full_like(s, -math.inf))
    m = s.amax(2, keepdim=True)
    e = torch.where(keep, torch.exp(s - m), torch.zeros_like(s))
    total = e.sum(2, keepdim=True)
    w = torch.where(total > 0, e / total, torch.zeros_like(e))
    out = torch.matmul(w.transpose(2, 3).contiguous(), v)       # [B][hkv][G][D]
    st["out"].copy_(out.reshape(B, hq * D))
    st["lse"].copy_((m + torch.log(total)).reshape(B, hq))
    got = {"out": st["out"], "lse": st["lse"]}
    if c["track"]:
        st["weight_out"].copy_(st["weight"] + w.sum(-1))
        got["weight"] = st["weight_out"]
    return got


def _attend_own(st):
    from rotated_w4a4_quantized_amd import rq
    c = st["case"]
    rq.paged_attention(st["q"], st["cache"], st["lens"], st["out"], lse=st["lse"], mask=st["mask"], max_len=c["L"],
                       track=c["track"], weight_out=st.get("weight_out"), workspace=st["workspace"])
    got = {"out": st["out"], "lse": st["lse"]}
    if c["track"]:
        got["weight"] = st["weight_out"]
    return got


def _evicted(st):
    got = {n: st[n] for n in ("k", "v", "k_scale", "v_scale") if n in st}
    return {"lens": st["lens_out"], "weight": st["weight_out"], "pos": st["pos_out"], **got}


def _evict_plain(st):
    c = st["case"]
    B, keep, hkv, page = c["B"], c["keep"], c["hkv"], c["page"]
    pos, weight, lens = st["pos"], st["weight"], st["lens"][:, None, None]
    slot = torch.arange(pos.shape[2], device=DEVICE).expand(pos.shape)
    real = slot < lens
    newest = torch.where(real, pos, torch.full_like(pos, -1)).amax(-1, keepdim=True)
    held = real & ((pos < c["sink"]) | (pos > newest - c["recent"]))
    key = torch.where(held, torch.full_like(weight, math.inf), torch.where(real, weight, torch.full_like(weight, -1.0)))
    order = key.sort(dim=-1, descending=True, stable=True).indices
    kept = torch.zeros_like(real).scatter(-1, order[..., :keep], True)
    # the n-th free place below the budget takes the n-th survivor above it
    hole = torch.cumsum((~kept[..., :keep]).int(), -1) - 1
    up = kept[..., keep:] & real[..., keep:]
    rank = torch.cumsum(up.int(), -1) - 1
    width = up.shape[-1] + 1
    source = torch.zeros(B, hkv, width, dtype=torch.int64, device=DEVICE)
    source.scatter_(-1, torch.where(up, rank, torch.full_like(rank, width - 1)).long(), slot[..., keep:])
    first = slot[..., :keep]
    come = torch.where(kept[..., :keep], first, source.gather(-1, hole.clamp(min=0, max=width - 1).long()))
    here = first < lens
    come = torch.where(here, come, first)
    st["weight_out"][..., :keep] = torch.where(here, weight.gather(-1, come), st["weight_out"][..., :keep])
    st["pos_out"][..., :keep] = torch.where(here, pos.gather(-1, come), st["pos_out"][..., :keep])
    st["lens_out"].copy_(st["lens"].clamp(max=keep))
    head = torch.arange(hkv, device=DEVICE)[None, :, None]
    row = torch.arange(B, device=DEVICE)[:, None, None]
    table = st["table"].long()
    to_page, from_page = table[row, first // page], table[row, come // page]
    for n in ("k", "v", "k_scale", "v_scale"):
        if n in st:
            st[n][to_page, head, first % page] = st[n][from_page, head, come % page]
    return _evicted(st)


def _evict_own(st):
    from rotated_w4a4_quantized_amd import rq
    c = st["case"]
    rq.cache_evict(st["cache"], st["lens"], c["keep"], recent=c["recent"], sink=c["sink"], lens_out=st["lens_out"],
                   weight_out=st["weight_out"], pos_out=st["pos_out"], max_len=c["L"], workspace=st["workspace"])
    return _evicted(st)


# ---------------------------------------------------------------- the work of one pass

def _mean_len(case):
    """The mean length that _lens() gives."""
    if not case["ragged"]:
        return float(case["L"])
    B, L = case["B"], case["L"]
    return (L + max(0, B - (2 if B > 2 else 1)) * L / 2) / B


def work(case):
    hkv, D = case["hkv"], case["D"]
    size = {"bf16": 2, "f32": 4, "int8": 1, "none": 0}
    if case["op"] == "qknorm":
        T, hq = case["T"], case["hq"]
        b = size[case["dtype"]]
        n = T * D * (hq + hkv) * b * 2 + T * case["rot"] * 4   # heads in and out, the token's cosines and sines
        if case["cache"] != "none":
            cb = size[case["cache"]]
            n += T * D * hkv * (b + 2 * cb - b) + T * 12 + (T * hkv * 8 if cb == 1 else 0)
        return {"bytes": n, "flops": 8.0 * T * D * (hq + hkv)}
    n = _mean_len(case) * case["B"]                             # tokens in the cache
    row = D * size[case["cache"]] + (4 if case["cache"] == "int8" else 0)
    if case["op"] == "attend":
        hq = case["hq"]
        total = n * hkv * row * 2 + 2 * case["B"] * hq * D * size[case["dtype"]] + case["B"] * hq * 4
        if case["track"]:
            total += n * hkv * 8
        if case["mask"]:
            total += n
        return {"bytes": total, "flops": 4.0 * n * hq * D}
    # what lies above the budget and stays: the recent, and a share of the rest
    B, L, keep = case["B"], case["L"], case["keep"]
    over = max(0, L - keep)
    fresh = min(over, case["recent"])
    share = max(0.0, min(1.0, (keep - case["recent"]) / max(1, L - case["recent"])))
    moved = (fresh + share * (over - fresh)) * B * (0.5 if case["ragged"] else 1.0)
    return {"bytes": 8.0 * n * hkv + 8.0 * min(n, keep * B) * hkv + 4 * hkv * moved * row, "flops": 4.0 * n * hkv}


# ---------------------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "qknorm":
        return _qknorm_exact(st)
    if case["op"] == "attend":
        return _attend_exact(st)
    # eviction moves numbers and computes none
    return None


def _qknorm_exact(st):
    c = st["case"]
    T, hq, hkv, D, rot, page = c["T"], c["hq"], c["hkv"], c["D"], c["rot"], c["page"]
    p = torch.arange(T, device=DEVICE) if st["positions"] is None else st["positions"].long()
    turn = torch.complex(st["cos"].double()[p], st["sin"].double()[p])[:, None]

    def head(x, w):
        x = x.double()
        y = x / torch.sqrt(torch.linalg.vector_norm(x, dim=-1, keepdim=True) ** 2 / D + EPS) * w.double()
        part = y[..., :rot]
        if c["inter"]:
            z = torch.view_as_complex(part.reshape(T, -1, rot // 2, 2).contiguous()) * turn
            part = torch.view_as_real(z).reshape(T, -1, rot)
        else:
            z = torch.complex(part[..., :rot // 2].contiguous(), part[..., rot // 2:].contiguous()) * turn
            part = torch.cat([z.real, z.imag], -1)
        return torch.cat([part, y[..., rot:]], -1)

    q, k, v = st["qkv"].split([hq * D, hkv * D, hkv * D], 1)
    got = {"q": head(q.reshape(T, hq, D), st["qw"]).reshape(T, hq * D)}
    k, v = head(k.reshape(T, hkv, D), st["kw"]), v.reshape(T, hkv, D).double()
    if c["cache"] == "none":
        return {**got, "k": k.reshape(T, hkv * D)}
    at = st["table"].long()[st["seq"].long(), st["place"].long() // page] * page + st["place"].long() % page
    for n, y in (("k", k), ("v", v)):
        if c["cache"] == "int8":
            s = y.abs().amax(-1, keepdim=True) / 127
            y = torch.round(torch.where(s > 0, y / s, torch.zeros_like(y))) * s
        flat = torch.zeros(st[n].shape[0] * page, hkv, D, dtype=torch.float64, device=DEVICE)
        flat.index_copy_(0, at, y)
        got[n] = flat.reshape(-1, page, hkv, D).transpose(1, 2).contiguous()
    return got


def _attend_exact(st):
    c = st["case"]
    B, L, hq, hkv, D, page = c["B"], c["L"], c["hq"], c["hkv"], c["D"], c["page"]
    G = hq // hkv
    out = torch.zeros(B, hkv, G, D, dtype=torch.float64, device=DEVICE)
    lse = torch.full((B, hkv, G), -math.inf, dtype=torch.float64, device=DEVICE)
    weight = st["weight"].double() if c["track"] else None
    for b, n in enumerate(st["lens"].tolist()):
        at = torch.arange(n, device=DEVICE)
        if c["mask"]:
            at = at[st["mask"][b, :n] != 0]
        if not at.numel():
            continue
        pg, off = st["table"][b].long()[at // page], at % page
        for h in range(hkv):
            k, v = st["k"][pg, h, off].double(), st["v"][pg, h, off].double()
            if c["cache"] == "int8":
                k, v = k * st["k_scale"][pg, h, off].double()[:, None], v * st["v_scale"][pg, h, off].double()[:, None]
            q = st["q"][b].double().reshape(hkv, G, D)[h]
            s = (q @ k.T.contiguous()) / math.sqrt(D)
            lse[b, h] = torch.logsumexp(s, -1)
            p = torch.softmax(s, -1)
            out[b, h] = p @ v
            if weight is not None:
                weight[b, h].index_add_(0, at, p.sum(0))
    got = {"out": out.reshape(B, hq * D), "lse": lse.reshape(B, hq)}
    if weight is not None:
        got["weight"] = weight
    return got
