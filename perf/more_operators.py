"""More operators around the rotated low-bit linears of a transformer block, as
cases to time and to compare:

  norm    the residual stream between two blocks in one pass: the branch's
          output, normalized or not, gated and added to the scaled stream, and
          the next block's normalized and modulated input
  cross   attention of many queries to states of another length (an encoder's,
          or the block's own tokens without a causal mask)
  prefix  attention of one new token per sequence where the batch shares the
          first part of the cache, read and computed once for all

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
        # one new token of one sequence between two blocks: latency
        _case("norm", "norm_step", T=1, K=4096, post="none", pre="rms", gate=False, mod=False, groups=1, res="bf16", io="bf16"),
        # an image transformer's tokens, two samples, adaptive layer norm with gate, shift and scale a sample
        _case("norm", "norm_image", T=8192, K=1152, post="none", pre="layer", gate=True, mod=True, groups=2, res="bf16", io="bf16"),
        # every token of a video transformer step, the residual stream in fp32
        _case("norm", "norm_video", T=32760, K=1536, post="none", pre="layer", gate=True, mod=True, groups=1, res="f32", io="bf16"),
        # wide rows of odd number with norms before and after the branch, all fp32, uneven groups of tokens
        _case("norm", "norm_wide_f32", T=1999, K=8960, post="rms", pre="rms", gate=True, mod=False, groups=7, res="f32", io="f32"),
        # one token per sequence that looks at its encoder's states: latency
        _case("cross", "cross_step", B=8, Tq=1, S=300, hq=16, hkv=4, D=64, dtype="bf16", ragged=True, mask=False, qrag=False),
        # image tokens that look at a caption's, padded and masked, heads of 72
        _case("cross", "cross_image", B=4, Tq=4096, S=300, hq=16, hkv=16, D=72, dtype="bf16", ragged=True, mask=True, qrag=False),
        # every token of a video transformer step that looks at its caption's
        _case("cross", "cross_video", B=1, Tq=32760, S=512, hq=12, hkv=12, D=128, dtype="bf16", ragged=False, mask=False, qrag=False),
        # a few learned queries over all of a video's tokens: all the work along the states
        _case("cross", "cross_few", B=1, Tq=77, S=32760, hq=12, hkv=12, D=128, dtype="bf16", ragged=False, mask=False, qrag=False),
        # a block's tokens that look at each other: matrix products
        _case("cross", "cross_joint", B=1, Tq=9216, S=9216, hq=12, hkv=12, D=128, dtype="bf16", ragged=False, mask=False, qrag=False),
        # fp32 queries of uneven numbers, shared heads, a sequence without states
        _case("cross", "cross_f32", B=5, Tq=333, S=1999, hq=16, hkv=4, D=64, dtype="f32", ragged=True, mask=True, qrag=True),
        # a serving batch behind one long system prompt
        _case("prefix", "prefix_batch", B=64, P=16384, L=512, hq=32, hkv=8, D=128, dtype="bf16", cache="bf16", page=64, ragged=True),
        # a few sequences behind a short prompt that ends inside a page, int8 cache: latency
        _case("prefix", "prefix_few_int8", B=5, P=1999, L=130, hq=32, hkv=8, D=128, dtype="bf16", cache="int8", page=16, ragged=False),
    ]


def _log(rng, lo, hi):
    """A whole number, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "cross", "prefix"])
    if op == "norm":
        K = rng.choice([_log(rng, 64, 16384) // 8 * 8, rng.choice([1152, 1536, 4096, 8960])])
        T = _log(rng, 1, max(1, 32760 * 1536 // K // 2))
        return dict(op=op, T=T, K=K, post=rng.choice(["none", "none", "rms", "layer"]), pre=rng.choice(["rms", "layer"]),
                    gate=rng.random() < 0.6, mod=rng.random() < 0.6, groups=rng.choice([1, 1, 2, 7, min(T, 64)]),
                    res=rng.choice(["bf16", "f32"]), io=rng.choice(["bf16", "bf16", "f32"]))
    hq, hkv = rng.choice([(12, 12), (16, 16), (32, 8), (16, 4), (16, 2), (8, 1), (20, 4)])
    D = rng.choice([64, 72, 80, 96, 128, 128, 128, 256])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op == "cross":
        most = 9216 * 9216 * 12 * 128 // (hq * D) // 3
        B = _log(rng, 1, 16)
        Tq = _log(rng, 1, 32760 // B)
        S = _log(rng, 1, max(1, min(32768 // B, most // (B * Tq))))
        return dict(op=op, B=B, Tq=Tq, S=S, hq=hq, hkv=hkv, D=D, dtype=dtype, ragged=rng.random() < 0.5,
                    mask=rng.random() < 0.3, qrag=rng.random() < 0.3)
    B = _log(rng, 1, 96)
    top = 64 * 16384 * 32 * 128 // (B * hq * D)
    return dict(op=op, B=B, P=_log(rng, 16, max(16, min(65536, top))), L=_log(rng, 1, max(1, min(1024, 65536 * 8 // (B * hkv)))),
                hq=hq, hkv=hkv, D=D, dtype=dtype, cache=rng.choice(["bf16", "bf16", "int8"]), page=rng.choice([16, 32, 64, 128]),
                ragged=rng.random() < 0.6)


# ---------------------------------------------------------------- inputs

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _uneven(n, most, gen, ragged):
    """Numbers up to `most`: all of them that, or spread below it with the first `most` and, from three on, the second 0."""
    lens = torch.full((n,), most, dtype=torch.int32, device=DEVICE)
    if ragged:
        lens = (torch.rand(n, generator=gen, device=DEVICE) * most).to(torch.int32) + 1
        lens.clamp_(max=most)
        lens[0] = most
        if n > 2:
            lens[1] = 0
    return lens


def _prepare_norm(case, st, gen):
    T, K, groups = case["T"], case["K"], case["groups"]

    def rand(*shape):
        return torch.randn(*shape, generator=gen, device=DEVICE)

    # a stream that has grown over the blocks, a few channels far larger than the others
    x = 3 * rand(T, K)
    x[:, :: max(1, K // 8)] *= 8
    st["x"], st["y"] = x.to(_TYPES[case["res"]]), rand(T, K).to(_TYPES[case["io"]])
    for n, kind in (("post", case["post"]), ("pre", case["pre"])):
        st[n + "_w"] = 1 + 0.2 * rand(K) if kind == "rms" else None
    # one row of modulations a group: [rows][gate, shift, scale]
    table = 0.4 * rand(groups, 3, K)
    st["gate"] = table[:, 0] if case["gate"] else None
    st["shift"], st["scale"] = (table[:, 1], table[:, 2]) if case["mod"] else (None, None)
    # tokens of a group lie together, in even runs where the groups divide them
    per = -(-T // groups)
    st["per"] = per
    st["index"] = None
    if groups > 1 and T % groups:
        cut = torch.rand(groups - 1, generator=gen, device=DEVICE).sort().values * T
        st["index"] = (torch.arange(T, device=DEVICE)[:, None] >= cut[None]).sum(1).to(torch.int32)
    st["h"], st["z"] = torch.zeros_like(st["x"]), torch.zeros_like(st["y"])


def _prepare_cross(case, st, gen):
    B, Tq, S, hq, hkv, D = (case[n] for n in ("B", "Tq", "S", "hq", "hkv", "D"))
    # scores of a few units: some states matter much more than others
    st["q"] = (1.5 * torch.randn(B, Tq, hq, D, generator=gen, device=DEVICE)).to(_TYPES[case["dtype"]])
    # keys and values as one projection writes them
    kv = torch.randn(B, S, 2, hkv, D, generator=gen, device=DEVICE, dtype=torch.bfloat16)
    st["k"], st["v"] = kv[:, :, 0], kv[:, :, 1]
    st["lens"] = _uneven(B, S, gen, True) if case["ragged"] else None
    st["q_lens"] = _uneven(B, Tq, gen, True) if case["qrag"] else None
    st["mask"] = (torch.rand(B, S, generator=gen, device=DEVICE) < 0.8).to(torch.uint8) if case["mask"] else None
    st["out"] = torch.zeros_like(st["q"])
    st["lse"] = torch.zeros(B, Tq, hq, device=DEVICE)


def _prepare_prefix(case, st, gen):
    B, P, L, hq, hkv, D, page = (case[n] for n in ("B", "P", "L", "hq", "hkv", "D", "page"))
    own_lens = _uneven(B, L, gen, case["ragged"])
    st["lens"] = torch.where(own_lens > 0, own_lens + P, own_lens)
    front, per = -(-P // page), -(-(P + L) // page)
    pages = front + B * (per - P // page)
    order = torch.randperm(pages, generator=gen, device=DEVICE).to(torch.int32)
    st["prefix_table"] = order[:front].contiguous()
    # a sequence's row: the pages of the prefix that are full, then its own
    st["table"] = torch.cat([order[:P // page].expand(B, P // page), order[front:].reshape(B, -1)], 1).contiguous()
    shape = (pages, hkv, page, D)
    for n in ("k", "v"):
        if case["cache"] == "int8":
            st[n] = torch.randint(-127, 128, shape, generator=gen, device=DEVICE, dtype=torch.int8)
            # code times scale of about unit variance
            st[n + "_scale"] = (torch.rand(shape[:3], generator=gen, device=DEVICE) + 0.5) / 73.0
        else:
            st[n] = torch.randn(shape, generator=gen, device=DEVICE, dtype=torch.bfloat16)
    st["q"] = (1.5 * torch.randn(B, hq * D, generator=gen, device=DEVICE)).to(_TYPES[case["dtype"]])
    st["out"] = torch.zeros_like(st["q"])
    st["lse"] = torch.zeros(B, hq, device=DEVICE)


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(int(seed) * 7919 + 29)
    st = dict(case=dict(case))
    {"norm": _prepare_norm, "cross": _prepare_cross, "prefix": _prepare_prefix}[case["op"]](case, st, gen)
    if own:   # the handles and the scratch that a program keeps beside its buffers
        from rotated_w4a4_quantized_amd import rq
        if case["op"] == "norm":
            st["post"] = None if case["post"] == "none" else rq.Norm(case["K"], case["post"], weight=st["post_w"], eps=EPS)
            st["pre"] = rq.Norm(case["K"], case["pre"], weight=st["pre_w"], eps=EPS)
            st["mod"] = None
            if case["gate"] or case["mod"]:
                st["mod"] = rq.Modulation(gate=st["gate"], shift=st["shift"], scale=st["scale"], per=st["per"], index=st["index"])
            return st
        if case["op"] == "cross":
            st["states"] = rq.States(st["k"], st["v"], lens=st["lens"], mask=st["mask"])
            n = rq.cross_attention_workspace_bytes(st["states"], case["Tq"], case["hq"], st["q"].dtype)
        else:
            st["cache"] = rq.KVCache(st["k"], st["v"], st["table"], k_scale=st.get("k_scale"), v_scale=st.get("v_scale"))
            n = rq.prefix_attention_workspace_bytes(st["cache"], case["hq"], case["P"], case["P"] + case["L"], st["q"].dtype)
        st["workspace"] = torch.empty(max(n, 16), dtype=torch.uint8, device=DEVICE)
    return st


# ---------------------------------------------------------------- one pass

def run(st):
    op = st["case"]["op"]
    if op == "norm":
        return (_norm_own if own else _norm_plain)(st)
    if op == "cross":
        return (_cross_own if own else _cross_plain)(st)
    return (_prefix_own if own else _prefix_plain)(st)


def _normed(x, kind, weight):
    """Rows of x in fp32, without or with their mean."""
    if kind == "none":
        return x
    if kind == "layer":
        x = x - x.mean(-1, keepdim=True)
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    return y if weight is None else y * weight


def _of_token(st, name):
    """The modulation row of every token."""
    if st["index"] is not None:
        return st[name][st["index"].long()]
    rows = torch.arange(st["case"]["T"], device=DEVICE) // st["per"]
    return st[name][rows]


def _norm_plain(st):
    c = st["case"]
    branch = _normed(st["y"].float(), c["post"], st["post_w"])
    if st["gate"] is not None:
        branch = branch * _of_token(st, "gate")
    h = st["x"].float() + branch
    z = _normed(h, c["pre"], st["pre_w"])
    if st["shift"] is not None:
        z = z * (1 + _of_token(st, "scale")) + _of_token(st, "shift")
    st["h"].copy_(h)
    st["z"].copy_(z)
    return {"h": st["h"], "z": st["z"]}


def _norm_own(st):
    from rotated_w4a4_quantized_amd import rq
    rq.block_norm(st["x"], st["z"], st["pre"], y=st["y"], post=st["post"], h=st["h"], mod=st["mod"])
    return {"h": st["h"], "z": st["z"]}


def _attention(q, k, v, keep):
    """q [..][rows][D], k and v [..][n][D] fp32, keep [..][1][n]: (out, lse)."""
    s = torch.matmul(q, k.transpose(-1, -2).contiguous()) / math.sqrt(q.shape[-1])
    s = torch.where(keep, s, torch.full_like(s, -math.inf))
    m = s.amax(-1, keepdim=True)
    e = torch.where(keep, torch.exp(s - m), torch.zeros_like(s))
    total = e.sum(-1, keepdim=True)
    out = torch.matmul(e, v)
    return torch.where(total > 0, out / total, torch.zeros_like(out)), (m + torch.log(total))[..., 0]


def _cross_plain(st):
    c = st["case"]
    B, Tq, S, hq, hkv, D = (c[n] for n in ("B", "Tq", "S", "hq", "hkv", "D"))
    G = hq // hkv
    keep = torch.ones(B, S, dtype=torch.bool, device=DEVICE)
    if st["lens"] is not None:
        keep &= torch.arange(S, device=DEVICE)[None] < st["lens"][:, None]
    if st["mask"] is not None:
        keep &= st["mask"] != 0
    q = st["q"].float().reshape(B, Tq, hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, hkv, Tq * G, D).contiguous()
    k, v = (st[n].float().transpose(1, 2).contiguous() for n in ("k", "v"))
    out, lse = _attention(q, k, v, keep[:, None, None])
    out = out.reshape(B, hkv, Tq, G, D).permute(0, 2, 1, 3, 4).reshape(B, Tq, hq, D)
    lse = lse.reshape(B, hkv, Tq, G).permute(0, 2, 1, 3).reshape(B, Tq, hq)
    if st["q_lens"] is not None:   # queries behind a sequence's own are left alone
        real = torch.arange(Tq, device=DEVICE)[None] < st["q_lens"][:, None]
        out = torch.where(real[:, :, None, None], out, st["out"].float())
        lse = torch.where(real[:, :, None], lse, st["lse"])
    st["out"].copy_(out)
    st["lse"].copy_(lse)
    return {"out": st["out"], "lse": st["lse"]}


def _cross_own(st):
    from rotated_w4a4_quantized_amd import rq
    rq.cross_attention(st["q"], st["states"], st["out"], lse=st["lse"], q_lens=st["q_lens"], workspace=st["workspace"])
    return {"out": st["out"], "lse": st["lse"]}


def _pages(st, n, table):
    """Slots of the pages in a table [..][pages], in order: [..][hkv][slots][D] fp32."""
    t = table.long()
    x = st[n][t].float()                                       # [..][pages][hkv][page][D]
    if n + "_scale" in st:
        x = x * st[n + "_scale"][t][..., None]
    x = x.transpose(-4, -3)
    return x.reshape(*x.shape[:-3], -1, x.shape[-1]).contiguous()


def _prefix_plain(st):
    c = st["case"]
    B, P, hq, hkv, D, page = (c[n] for n in ("B", "P", "hq", "hkv", "D", "page"))
    G = hq // hkv
    lens = st["lens"].long()
    q = st["q"].float().reshape(B, hkv, G, D)
    # all queries of a head look at the prefix together
    k0, v0 = (_pages(st, n, st["prefix_table"])[:, :P] for n in ("k", "v"))
    together = q.permute(1, 0, 2, 3).reshape(hkv, B * G, D).contiguous()
    s0 = torch.matmul(together, k0.transpose(1, 2).contiguous()) / math.sqrt(D)
    s0 = s0.reshape(hkv, B, G, P).permute(1, 0, 2, 3)
    full = (lens >= P)[:, None, None, None]
    s0 = torch.where(full, s0, torch.full_like(s0, -math.inf))
    # and each at what its own sequence holds behind
    k1, v1 = (_pages(st, n, st["table"][:, P // page:]) for n in ("k", "v"))
    keep = P // page * page + torch.arange(k1.shape[2], device=DEVICE)[None]
    keep = ((keep >= P) & (keep < lens[:, None]))[:, None, None]
    s1 = torch.matmul(q, k1.transpose(2, 3).contiguous()) / math.sqrt(D)
    s1 = torch.where(keep, s1, torch.full_like(s1, -math.inf))
    m = torch.maximum(s0.amax(-1, keepdim=True), s1.amax(-1, keepdim=True))
    e0 = torch.where(full, torch.exp(s0 - m), torch.zeros_like(s0))
    e1 = torch.where(keep, torch.exp(s1 - m), torch.zeros_like(s1))
    total = e0.sum(-1, keepdim=True) + e1.sum(-1, keepdim=True)
    o0 = torch.matmul(e0.permute(1, 0, 2, 3).reshape(hkv, B * G, P).contiguous(), v0.contiguous())
    out = o0.reshape(hkv, B, G, D).permute(1, 0, 2, 3) + torch.matmul(e1, v1)
    out = torch.where(total > 0, out / total, torch.zeros_like(out))
    st["out"].copy_(out.reshape(B, hq * D))
    st["lse"].copy_((m + torch.log(total)).reshape(B, hq))
    return {"out": st["out"], "lse": st["lse"]}


def _prefix_own(st):
    from rotated_w4a4_quantized_amd import rq
    c = st["case"]
    rq.prefix_attention(st["q"], st["cache"], st["prefix_table"], c["P"], st["lens"], st["out"], max_len=c["P"] + c["L"],
                        lse=st["lse"], workspace=st["workspace"])
    return {"out": st["out"], "lse": st["lse"]}


# ---------------------------------------------------------------- the work of one pass

def _mean(n, most, ragged):
    """The mean that _uneven() gives."""
    return (most + max(0, n - (2 if n > 2 else 1)) * most / 2) / n if ragged else float(most)


def work(case):
    size = {"bf16": 2, "f32": 4, "int8": 1}
    if case["op"] == "norm":
        T, K = case["T"], case["K"]
        n = T * K * 2 * (size[case["res"]] + size[case["io"]])
        rows = (1 if case["gate"] else 0) + (2 if case["mod"] else 0)
        return {"bytes": n + 4 * K * rows * min(case["groups"], T), "flops": 12.0 * T * K}
    hq, hkv, D, io = case["hq"], case["hkv"], case["D"], size[case["dtype"]]
    B = case["B"]
    if case["op"] == "cross":
        nq, nk = _mean(B, case["Tq"], case["qrag"]), _mean(B, case["S"], case["ragged"])
        n = B * (nq * hq * (2 * D * io + 4) + nk * hkv * D * 4 + (nk if case["mask"] else 0))
        return {"bytes": n, "flops": 4.0 * B * nq * nk * hq * D}
    row = 2 * (D * size[case["cache"]] + (4 if case["cache"] == "int8" else 0)) * hkv
    mine = B * _mean(B, case["L"], case["ragged"])
    n = (case["P"] + mine) * row + B * hq * (2 * D * io + 4)
    return {"bytes": n, "flops": 4.0 * hq * D * (B * case["P"] + mine)}


# ---------------------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    return {"norm": _norm_exact, "cross": _cross_exact, "prefix": _prefix_exact}[case["op"]](st)


def _norm_exact(st):
    c = st["case"]
    T, K = c["T"], c["K"]
    group = st["index"].long() if st["index"] is not None else torch.div(torch.arange(T, device=DEVICE), st["per"], rounding_mode="floor")

    def unit(x, kind, weight):
        if kind == "none":
            return x
        if kind == "layer":
            var, mean = torch.var_mean(x, dim=-1, keepdim=True, unbiased=False)
            return (x - mean) / torch.sqrt(var + EPS)
        rms = torch.sqrt(torch.linalg.vector_norm(x, dim=-1, keepdim=True) ** 2 / K + EPS)
        return x / rms if weight is None else x / rms * weight.double()

    h, z = (torch.empty(T, K, dtype=torch.float64, device=DEVICE) for _ in range(2))
    for a in range(0, T, 4096):
        t = slice(a, min(a + 4096, T))
        g = group[t]
        branch = unit(st["y"][t].double(), c["post"], st["post_w"])
        h[t] = st["x"][t].double() + (branch if st["gate"] is None else st["gate"].double()[g] * branch)
        z[t] = unit(h[t], c["pre"], st["pre_w"])
        if st["shift"] is not None:
            z[t] += z[t] * st["scale"].double()[g] + st["shift"].double()[g]
    return {"h": h, "z": z}


def _soft(q, k, v):
    """Attention of rows q over k, v, all fp64, a few thousand rows at a time."""
    out, lse = [], []
    for part in q.split(max(1, (1 << 26) // max(1, k.shape[0]))):
        s = part @ k.T.contiguous() * (q.shape[-1] ** -0.5)
        lse.append(torch.logsumexp(s, -1))
        out.append(torch.softmax(s, -1) @ v)
    return torch.cat(out), torch.cat(lse)


def _cross_exact(st):
    c = st["case"]
    B, Tq, S, hq, hkv = (c[n] for n in ("B", "Tq", "S", "hq", "hkv"))
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device=DEVICE)
    lse = torch.zeros(B, Tq, hq, dtype=torch.float64, device=DEVICE)
    for b in range(B):
        n = S if st["lens"] is None else int(st["lens"][b])
        t = Tq if st["q_lens"] is None else int(st["q_lens"][b])
        at = torch.arange(n, device=DEVICE)
        if st["mask"] is not None:
            at = at[st["mask"][b, :n] != 0]
        if not at.numel():
            lse[b, :t] = -math.inf
            continue
        for h in range(hq):
            kv = h // (hq // hkv)
            out[b, :t, h], lse[b, :t, h] = _soft(st["q"][b, :t, h].double(), st["k"][b, at, kv].double(), st["v"][b, at, kv].double())
    return {"out": out, "lse": lse}


def _prefix_exact(st):
    c = st["case"]
    B, P, hq, hkv, D, page = (c[n] for n in ("B", "P", "hq", "hkv", "D", "page"))
    G = hq // hkv
    out = torch.zeros(B, hq, D, dtype=torch.float64, device=DEVICE)
    lse = torch.full((B, hq), -math.inf, dtype=torch.float64, device=DEVICE)
    for b, n in enumerate(st["lens"].tolist()):
        if n < P:
            continue
        j = torch.arange(n, device=DEVICE)
        row = st["table"][b].long()[j // page]
        row[:P] = st["prefix_table"].long()[j[:P] // page]
        k, v = (st[name][row, :, j % page].double() for name in ("k", "v"))     # [n][hkv][D]
        if c["cache"] == "int8":
            k, v = (x * st[name + "_scale"][row, :, j % page].double()[..., None] for x, name in ((k, "k"), (v, "v")))
        q = st["q"][b].double().reshape(hkv, G, D)
        for h in range(hkv):
            out[b, h * G:(h + 1) * G], lse[b, h * G:(h + 1) * G] = _soft(q[h], k[:, h].contiguous(), v[:, h].contiguous())
    return {"out": out.reshape(B, hq * D), "lse": lse}
