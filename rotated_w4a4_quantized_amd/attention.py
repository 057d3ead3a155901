"""The attention half of a transformer block on rotated W4A4 linears.

DecodeAttention, one new token per sequence and step:

    QKV projection (rotate + quantize + W4A4 GEMM)
    head norm, position rotation and store in the paged cache
    attention over the cache, adding up the weights each token receives, or
        behind a prefix that the sequences share
    output projection (rotate + quantize + W4A4 GEMM)
    eviction, whenever the cache is `slack` tokens over its budget

DiffusionAttention, all tokens of a diffusion transformer's samples:

    layer norm, modulated; QKV projection; head norm and position rotation
    attention of a sample's tokens to each other; output projection
    gated into the residual stream, with the next norm in the same pass
    query projection; attention to the caption's states; output projection
    into the residual stream, with the MLP's modulated norm in the same pass

    python -m rotated_w4a4_quantized_amd.attention [--steps N] [--int8] [--prefix N] [--diffusion]

runs one of them on random weights and prints the time of a step.  Marshalling
only: every computation runs in librq.
"""
from __future__ import annotations

import math

import numpy as np

from . import rq


class DecodeLinear:
    """A W4A4 linear layer for up to max_tokens tokens: RPBH rotation, packed
    weights and buffers on the GPU."""

    def __init__(self, W: np.ndarray, max_tokens: int, block=128, seed=0, device="cuda"):
        import torch
        rng = np.random.default_rng(seed)
        N, K = self.shape = W.shape
        rot = rq.Rotation.rpbh(rng.choice([-1, 1], K), rng.permutation(K), block)
        self.q, self.drot = rq.Quant.int4(), rot.to_device(device)
        self.dw = rq.pack_weights(rot, self.q, W).to_device(device)
        ncode, _, _ = rq.activation_bytes(rot, self.q, 1)
        self.codes = torch.empty((max_tokens, ncode), dtype=torch.uint8, device=device)
        self.scale = torch.empty((max_tokens,), dtype=torch.float32, device=device)

    def __call__(self, X, Y, stream=None):
        T, (N, K) = int(X.shape[0]), self.shape
        if X.shape != (T, K) or T > self.scale.shape[0] or Y.shape != (T, N):
            raise ValueError(f"expected at most {self.scale.shape[0]} rows of {K} values in and as many of {N} out, "
                             f"got {tuple(X.shape)} and {tuple(Y.shape)}")
        if not (X.is_contiguous() and Y.is_contiguous()):
            raise ValueError("the rows must be contiguous")
        if X.device != self.scale.device or Y.device != self.scale.device:
            raise ValueError(f"the layer is on {self.scale.device}, its rows on {X.device} and {Y.device}")
        rq.rotate_quant(self.drot, self.q, X, self.codes[:T], self.scale[:T], stream=stream)
        rq.w4a4_linear(self.dw, self.codes[:T], self.scale[:T], Y, stream=stream)


class DecodeAttention:
    """Attention of `batch` sequences that grow by one token a step.

    Wqkv [(q_heads + 2 kv_heads) * head_dim][hidden] and Wo [hidden][q_heads *
    head_dim] fp32.  max_len: tokens a sequence ever has, evicted ones
    included (a step past it is refused).  budget: tokens a sequence keeps
    (None: all of max_len); the cache holds budget + slack (one more than the
    budget at least), and is cut back to the budget when full, keeping the
    newest `recent` and the first `sink` tokens whatever their weight.  Where
    the budget does not hold both, the first tokens take all of it but one
    place, and the newest what is left.  prefix: tokens in front of all
    sequences (counted in max_len, without a budget), which set_prefix()
    computes and stores once; attention reads them once for the batch."""

    def __init__(self, Wqkv, Wo, q_heads, kv_heads, head_dim, batch, max_len, budget=None, slack=64,
                 recent=32, sink=4, page=64, int8=False, rope_base=1e4, device="cuda", prefix=0):
        import torch
        if prefix and budget is not None:
            raise ValueError("a shared prefix is not evicted from: prefix and budget exclude each other")
        if not 0 <= prefix < max_len:
            raise ValueError(f"a prefix of {prefix} tokens leaves none of {max_len} for the sequences")
        if Wqkv.shape[:1] != ((q_heads + 2 * kv_heads) * head_dim,) or Wo.shape[1:] != (q_heads * head_dim,):
            raise ValueError(f"Wqkv {Wqkv.shape} and Wo {Wo.shape} are not of {q_heads} + 2 * {kv_heads} heads of {head_dim}")
        # (protected tokens tie and ties go to the lower slot, so more of them
        # than the budget would push out the newest)
        if budget is not None:
            sink = min(sink, budget - min(recent, 1))
            recent = min(recent, budget - sink)
        self.batch, self.budget, self.recent, self.sink = batch, budget, recent, sink
        room = max_len if budget is None else min(max_len, budget + max(slack, 1))
        bf16, i32 = torch.bfloat16, torch.int32
        self.qkv_proj = DecodeLinear(Wqkv, batch, seed=1, device=device)
        self.out_proj = DecodeLinear(Wo, batch, seed=2, device=device)
        angle = (torch.arange(max_len, device=device, dtype=torch.float64)[:, None] *
                 rope_base ** (-torch.arange(0, head_dim, 2, device=device, dtype=torch.float64) / head_dim))
        ones = torch.ones(head_dim, device=device)
        self.norm = rq.QKNorm(q_heads, kv_heads, head_dim, ones, ones.clone(), angle.cos().float(), angle.sin().float())
        self.track = budget is not None
        self.room = room
        self.prefix, self.ready = prefix, not prefix
        if prefix:
            self._share(batch, kv_heads, head_dim, room, page, int8, device)
        else:
            self.cache = rq.KVCache.alloc(batch, kv_heads, head_dim, room, page=page, int8=int8, track=self.track, device=device)
        new = lambda n, dt: torch.zeros((batch, n), dtype=dt, device=device)  # noqa: E731
        self.qkv, self.q = new((q_heads + 2 * kv_heads) * head_dim, bf16), new(q_heads * head_dim, bf16)
        self.attn, self.y = new(q_heads * head_dim, bf16), new(Wo.shape[0], bf16)
        self.place, self.lens = new(1, i32)[:, 0], new(1, i32)[:, 0]
        self.position = new(1, i32)[:, 0]
        self.length = 0                     # tokens of a sequence in the cache (the same for all)
        self.max_len, self.tokens = max_len, 0   # tokens that went through, evicted ones included
        if prefix:
            n = rq.prefix_attention_workspace_bytes(self.cache, q_heads, prefix, room, bf16)
        else:
            n = rq.paged_attention_workspace_bytes(self.cache, q_heads, room, track=self.track)
        if self.track:
            n = max(n, rq.cache_evict_workspace_bytes(self.cache, budget, room))
        self.workspace = torch.empty((max(n, 16),), dtype=torch.uint8, device=device)

    def _share(self, batch, heads, head_dim, room, page, int8, device):
        """The cache with the prefix's pages in front: those it fills belong to
        all sequences, the one it ends in has a sequence's own beside it."""
        import torch
        front, full, per = -(-self.prefix // page), self.prefix // page, -(-room // page)
        shape = (front + batch * (per - full), heads, page, head_dim)
        new = lambda dt, *s: torch.zeros(*s, dtype=dt, device=device)  # noqa: E731
        k, v = (new(torch.int8 if int8 else torch.bfloat16, *shape) for _ in range(2))
        scales = {n: new(torch.float32, *shape[:3]) for n in ("k_scale", "v_scale")} if int8 else {}
        self.prefix_table = torch.arange(front, dtype=torch.int32, device=device)
        table = torch.empty((batch, per), dtype=torch.int32, device=device)
        table[:, :full] = self.prefix_table[:full]
        table[:, full:] = front + torch.arange(batch * (per - full), dtype=torch.int32, device=device).reshape(batch, -1)
        self.cache = rq.KVCache(k, v, table, **scales)
        self.prefix_cache = rq.KVCache(k, v, self.prefix_table[None].contiguous(), **scales)

    def set_prefix(self, x, stream=None):
        """x [prefix][hidden] bf16: the shared tokens.  Their keys and values go
        to the cache, and the sequences start anew behind them."""
        if not self.prefix:
            raise ValueError("the block was made without a prefix")
        if x.shape[:1] != (self.prefix,):
            raise ValueError(f"expected the {self.prefix} tokens of the prefix, got {tuple(x.shape)}")
        with self._on(stream):
            import torch
            place = torch.arange(self.prefix, dtype=torch.int32, device=self.y.device)
            seq = torch.zeros_like(place)
            for i in range(0, self.prefix, self.batch):
                n = min(self.batch, self.prefix - i)
                at = slice(i, i + n)
                self.qkv_proj(x[at], self.qkv[:n])
                rq.qk_norm_rope(self.norm, self.qkv[:n], self.q[:n], positions=place[at], cache=self.prefix_cache,
                                seq=seq[at], place=place[at])
            for counter in (self.place, self.lens, self.position):
                counter.fill_(self.prefix)
            self.length = self.tokens = self.prefix
            self.ready = True

    def _on(self, stream):
        """The context that makes `stream` current (None: as it is)."""
        import contextlib
        if stream is None:
            return contextlib.nullcontext()
        import torch
        device = self.y.device
        if isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream, device=device) if stream else torch.cuda.default_stream(device)
        return torch.cuda.stream(stream)

    def step(self, x, stream=None):
        """x [batch][hidden] bf16: the new tokens.  Returns y [batch][hidden],
        which the next step overwrites.  Everything runs on `stream` (a torch
        stream or its address; default: torch's current one)."""
        # (the block's own counters are torch operations, which go to the current stream)
        with self._on(stream):
            return self._step(x)

    def _step(self, x):
        if not self.ready:
            raise ValueError("the shared prefix has not been set")
        if self.tokens >= self.max_len:     # (eviction frees slots, but no rows of the rotation's table)
            raise ValueError(f"the block was made for sequences of {self.max_len} tokens")
        if self.length >= self.room:
            raise ValueError(f"the cache holds {self.room} tokens a sequence")
        if x.shape[:1] != (self.batch,):
            raise ValueError(f"expected a token of each of {self.batch} sequences, got {tuple(x.shape)}")
        self.qkv_proj(x, self.qkv)          # (refuses a wrong x before anything has changed)
        self.lens.add_(1)
        self.length += 1
        rq.qk_norm_rope(self.norm, self.qkv, self.q, positions=self.position, cache=self.cache, place=self.place)
        if self.prefix:
            rq.prefix_attention(self.q, self.cache, self.prefix_table, self.prefix, self.lens, self.attn,
                                max_len=self.length, workspace=self.workspace)
        else:
            rq.paged_attention(self.q, self.cache, self.lens, self.attn, max_len=self.length, track=self.track,
                               workspace=self.workspace)
        self.out_proj(self.attn, self.y)
        if self.track and self.length == self.room and self.room > self.budget:
            rq.cache_evict(self.cache, self.lens, self.budget, recent=self.recent, sink=self.sink,
                           max_len=self.length, workspace=self.workspace)
            self.length = self.budget
        self.place.copy_(self.lens)
        self.position.add_(1)
        self.tokens += 1
        return self.y


class DiffusionAttention:
    """Attention of a diffusion transformer's block: `batch` samples of `tokens`
    tokens to each other and to their captions.

    Wqkv [3 heads * head_dim][hidden], Wo [hidden][heads * head_dim] of the
    tokens' attention; Wq [heads * head_dim][hidden], Wkv [2 heads *
    head_dim][caption], Wco [hidden][heads * head_dim] of the captions', fp32.
    states: tokens of a caption, at most."""

    def __init__(self, Wqkv, Wo, Wq, Wkv, Wco, heads, head_dim, batch, tokens, states, rope_base=1e4, device="cuda"):
        import torch
        inner, hidden = heads * head_dim, Wo.shape[0]
        for name, W, shape in (("Wqkv", Wqkv, (3 * inner, hidden)), ("Wo", Wo, (hidden, inner)), ("Wq", Wq, (inner, hidden)),
                               ("Wkv", Wkv, (2 * inner, Wkv.shape[1])), ("Wco", Wco, (hidden, inner))):
            if W.shape != shape:
                raise ValueError(f"{name} {W.shape} is not {shape}")
        self.heads, self.head_dim, self.batch, self.tokens, self.max_states = heads, head_dim, batch, tokens, states
        T = batch * tokens
        linear = lambda W, rows, seed: DecodeLinear(W, rows, block=math.gcd(W.shape[1], 128), seed=seed, device=device)  # noqa: E731
        self.qkv_proj, self.out_proj, self.q_proj, self.caption_out = (linear(W, T, i) for i, W in enumerate((Wqkv, Wo, Wq, Wco), 1))
        self.caption_proj = linear(Wkv, batch * states, 5)
        angle = (torch.arange(tokens, device=device, dtype=torch.float64)[:, None] *
                 rope_base ** (-torch.arange(0, head_dim, 2, device=device, dtype=torch.float64) / head_dim))
        ones = torch.ones(head_dim, device=device)
        self.head_norm = rq.QKNorm(heads, heads, head_dim, ones, ones.clone(), angle.cos().float(), angle.sin().float())
        self.positions = torch.arange(tokens, dtype=torch.int32, device=device).repeat(batch)
        self.layer_norm = rq.Norm(hidden, "layer")
        new = lambda rows, n: torch.zeros((rows, n), dtype=torch.bfloat16, device=device)  # noqa: E731
        self.z, self.y, self.h = new(T, hidden), new(T, hidden), new(T, hidden)
        self.qkv, self.q, self.attn = new(T, 3 * inner), new(T, inner), new(T, inner)
        self.kv = new(batch * states, 2 * inner)
        heads_of = lambda t, n: t.view(batch, n, -1, head_dim)  # noqa: E731
        self.q4, self.attn4 = heads_of(self.q, tokens), heads_of(self.attn, tokens)
        own = heads_of(self.qkv, tokens)
        self.own = rq.States(own[:, :, heads:2 * heads], own[:, :, 2 * heads:])
        self.states = None
        bf16 = torch.bfloat16
        every = rq.States(*heads_of(self.kv, states).split(heads, 2))
        n = max(rq.cross_attention_workspace_bytes(s, tokens, heads, bf16) for s in (self.own, every))
        self.workspace = torch.empty((max(n, 16),), dtype=torch.uint8, device=device)

    def set_caption(self, text, lens=None, mask=None, stream=None):
        """text [batch][n <= states][caption] bf16 with lens int32 [batch] and
        mask [batch][n]: the captions' keys and values, kept for all steps."""
        if text.dim() != 3 or text.shape[0] != self.batch or not 0 < text.shape[1] <= self.max_states:
            raise ValueError(f"expected captions of {self.batch} samples, at most {self.max_states} tokens each, got {tuple(text.shape)}")
        if not text.is_contiguous():
            raise ValueError("the captions must be contiguous")
        n = text.shape[1]
        kv = self.kv[:self.batch * n]
        self.caption_proj(text.view(self.batch * n, -1), kv, stream=stream)
        self.states = rq.States(*kv.view(self.batch, n, -1, self.head_dim).split(self.heads, 2), lens=lens, mask=mask)

    def step(self, x, mod, stream=None):
        """x [batch * tokens][hidden] bf16, the residual stream; mod [batch][5]
        [hidden] fp32: shift, scale and gate of the tokens' attention, shift and
        scale of the MLP's input.  Returns the stream and the MLP's input, which
        the next step overwrites."""
        import torch
        if self.states is None:
            raise ValueError("the captions have not been set")
        if mod.shape != (self.batch, 5, x.shape[-1]):
            raise ValueError(f"expected modulations [{self.batch}][5][{x.shape[-1]}], got {tuple(mod.shape)}")
        if x.shape != self.h.shape:
            raise ValueError(f"expected tokens {tuple(self.h.shape)}, got {tuple(x.shape)}")
        if x.dtype is not self.h.dtype:
            raise TypeError(f"the block's stream is {self.h.dtype}, got {x.dtype}")
        shift, scale, gate, mlp_shift, mlp_scale = mod.unbind(1)
        s = dict(stream=stream)
        rq.block_norm(x, self.z, self.layer_norm, mod=rq.Modulation(shift=shift, scale=scale, per=self.tokens), **s)
        self.qkv_proj(self.z, self.qkv, **s)
        inner = self.heads * self.head_dim
        rq.qk_norm_rope(self.head_norm, self.qkv, self.q, k_out=self.qkv[:, inner:2 * inner], positions=self.positions, **s)
        rq.cross_attention(self.q4, self.own, self.attn4, workspace=self.workspace, **s)
        self.out_proj(self.attn, self.y, **s)
        rq.block_norm(x, self.z, self.layer_norm, y=self.y, h=self.h, mod=rq.Modulation(gate=gate, per=self.tokens), **s)
        self.q_proj(self.z, self.q, **s)
        rq.cross_attention(self.q4, self.states, self.attn4, workspace=self.workspace, **s)
        self.caption_out(self.attn, self.y, **s)
        rq.block_norm(self.h, self.z, self.layer_norm, y=self.y, h=self.h,
                      mod=rq.Modulation(shift=mlp_shift, scale=mlp_scale, per=self.tokens), **s)
        return self.h, self.z


def _time(steps, step):
    import time

    import torch
    step(0)
    torch.cuda.synchronize()
    t = time.perf_counter()
    for i in range(1, steps):
        step(i)
    torch.cuda.synchronize()
    return (time.perf_counter() - t) / max(steps - 1, 1) * 1e6


def _diffusion(steps, batch):
    import torch
    hidden, heads, D, tokens, states, caption = 1152, 16, 72, 4096, 300, 4096
    inner, rng = heads * D, np.random.default_rng(0)
    weights = [(rng.standard_normal(s) * 0.02).astype(np.float32)
               for s in ((3 * inner, hidden), (hidden, inner), (inner, hidden), (2 * inner, caption), (hidden, inner))]
    block = DiffusionAttention(*weights, heads, D, batch, tokens, states)
    block.set_caption(torch.randn(batch, states, caption, device="cuda", dtype=torch.bfloat16),
                      lens=torch.randint(1, states + 1, (batch,), device="cuda", dtype=torch.int32))
    x = torch.randn(batch * tokens, hidden, device="cuda", dtype=torch.bfloat16)
    mod = 0.2 * torch.randn(batch, 5, hidden, device="cuda")
    us = _time(steps, lambda i: block.step(x, mod))
    print(f"{steps} steps of {batch} samples of {tokens} tokens: {us:.1f} us a step, "
          f"stream rms {float(block.h.float().square().mean().sqrt()):.4f}")


def main(argv=None):
    import argparse
    import time

    import torch
    p = argparse.ArgumentParser(description="decode on random weights: time of a step")
    p.add_argument("--steps", type=int, default=300)
    p.add_argument("--batch", type=int, default=16)
    p.add_argument("--budget", type=int, default=128)
    p.add_argument("--int8", action="store_true", help="int8 cache")
    p.add_argument("--prefix", type=int, default=0, help="tokens that the sequences share (no budget then)")
    p.add_argument("--diffusion", action="store_true", help="a diffusion transformer's block instead")
    a = p.parse_args(argv)
    if a.diffusion:
        return _diffusion(a.steps, a.batch)
    hidden, hq, hkv, D = 1536, 12, 4, 128
    rng = np.random.default_rng(0)
    weights = [(rng.standard_normal(s) * 0.02).astype(np.float32) for s in (((hq + 2 * hkv) * D, hidden), (hidden, hq * D))]
    block = DecodeAttention(*weights, hq, hkv, D, a.batch, max_len=a.prefix + a.steps + 1,
                            budget=None if a.prefix else a.budget, int8=a.int8, prefix=a.prefix)
    if a.prefix:
        block.set_prefix(torch.randn(a.prefix, hidden, device="cuda", dtype=torch.bfloat16))
    x = torch.randn(a.steps, a.batch, hidden, device="cuda", dtype=torch.bfloat16)
    torch.cuda.synchronize()
    t = time.perf_counter()
    for i in range(a.steps):
        y = block.step(x[i])
    torch.cuda.synchronize()
    t = time.perf_counter() - t
    print(f"{a.steps} steps of {a.batch} sequences: {t / a.steps * 1e6:.1f} us a step, "
          f"{block.length} tokens of {a.prefix + a.steps} kept, output rms {float(y.float().square().mean().sqrt()):.4f}")


if __name__ == "__main__":
    main()
