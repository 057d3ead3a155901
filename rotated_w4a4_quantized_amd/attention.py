"""The attention half of a decoder block on rotated W4A4 linears, one new token
per sequence and step:

    QKV projection (rotate + quantize + W4A4 GEMM)
    head norm, position rotation and store in the paged cache
    attention over the cache, adding up the weights each token receives
    output projection (rotate + quantize + W4A4 GEMM)
    eviction, whenever the cache is `slack` tokens over its budget

    python -m rotated_w4a4_quantized_amd.attention [--steps N] [--int8]

runs it on random weights and prints the time of a step.  Marshalling only:
every computation runs in librq.
"""
from __future__ import annotations

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
    place, and the newest what is left."""

    def __init__(self, Wqkv, Wo, q_heads, kv_heads, head_dim, batch, max_len, budget=None, slack=64,
                 recent=32, sink=4, page=64, int8=False, rope_base=1e4, device="cuda"):
        import torch
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
        self.cache = rq.KVCache.alloc(batch, kv_heads, head_dim, room, page=page, int8=int8, track=self.track, device=device)
        new = lambda n, dt: torch.zeros((batch, n), dtype=dt, device=device)  # noqa: E731
        self.qkv, self.q = new((q_heads + 2 * kv_heads) * head_dim, bf16), new(q_heads * head_dim, bf16)
        self.attn, self.y = new(q_heads * head_dim, bf16), new(Wo.shape[0], bf16)
        self.place, self.lens = new(1, i32)[:, 0], new(1, i32)[:, 0]
        self.position = new(1, i32)[:, 0]
        self.length = 0                     # tokens of a sequence in the cache (the same for all)
        self.max_len, self.tokens = max_len, 0   # tokens that went through, evicted ones included
        n = rq.paged_attention_workspace_bytes(self.cache, q_heads, room, track=self.track)
        if self.track:
            n = max(n, rq.cache_evict_workspace_bytes(self.cache, budget, room))
        self.workspace = torch.empty((max(n, 16),), dtype=torch.uint8, device=device)

    def step(self, x, stream=None):
        """x [batch][hidden] bf16: the new tokens.  Returns y [batch][hidden],
        which the next step overwrites.  Everything runs on `stream` (a torch
        stream or its address; default: torch's current one)."""
        if stream is None:
            return self._step(x)
        import torch
        # (the block's own counters are torch operations, which go to the current stream)
        device = self.y.device
        if isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream, device=device) if stream else torch.cuda.default_stream(device)
        with torch.cuda.stream(stream):
            return self._step(x)

    def _step(self, x):
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


def main(argv=None):
    import argparse
    import time

    import torch
    p = argparse.ArgumentParser(description="decode on random weights: time of a step")
    p.add_argument("--steps", type=int, default=300)
    p.add_argument("--batch", type=int, default=16)
    p.add_argument("--budget", type=int, default=128)
    p.add_argument("--int8", action="store_true", help="int8 cache")
    a = p.parse_args(argv)
    hidden, hq, hkv, D = 1536, 12, 4, 128
    rng = np.random.default_rng(0)
    weights = [(rng.standard_normal(s) * 0.02).astype(np.float32) for s in (((hq + 2 * hkv) * D, hidden), (hidden, hq * D))]
    block = DecodeAttention(*weights, hq, hkv, D, a.batch, max_len=a.steps + 1, budget=a.budget, int8=a.int8)
    x = torch.randn(a.steps, a.batch, hidden, device="cuda", dtype=torch.bfloat16)
    torch.cuda.synchronize()
    t = time.perf_counter()
    for i in range(a.steps):
        y = block.step(x[i])
    torch.cuda.synchronize()
    t = time.perf_counter() - t
    print(f"{a.steps} steps of {a.batch} sequences: {t / a.steps * 1e6:.1f} us a step, "
          f"{block.length} tokens of {a.steps} kept, output rms {float(y.float().square().mean().sqrt()):.4f}")


if __name__ == "__main__":
    main()
