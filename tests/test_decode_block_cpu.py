"""The decode block's own bookkeeping without a GPU: its buffers lie in host
memory and the library's calls are replaced by records of them."""
import contextlib

import numpy as np
import pytest

from rotated_w4a4_quantized_amd import attention, rq

torch = pytest.importorskip("torch")

HIDDEN, HQ, HKV, D = 128, 4, 2, 32


def block(calls, monkeypatch, **kw):
    """A block whose library calls are appended to `calls` as (name, what
    the call would read of the block's counters)."""
    rng = np.random.default_rng(0)
    weights = [rng.standard_normal(s).astype(np.float32) for s in (((HQ + 2 * HKV) * D, HIDDEN), (HIDDEN, HQ * D))]
    args = dict(batch=2, max_len=40, page=16, device="cpu")
    args.update(kw)
    blk = attention.DecodeAttention(*weights, HQ, HKV, D, **args)

    def record(name, *keys):
        def f(*a, **k):
            calls.append((name, {n: k[n].clone() if torch.is_tensor(k[n]) else k[n] for n in keys if n in k},
                          blk.lens.clone(), k.get("stream")))
        return f

    monkeypatch.setattr(rq, "rotate_quant", record("rotate"))
    monkeypatch.setattr(rq, "w4a4_linear", record("linear"))
    monkeypatch.setattr(rq, "qk_norm_rope", record("norm", "positions", "place"))
    monkeypatch.setattr(rq, "paged_attention", record("attend", "max_len"))

    def evict(cache, lens, keep, **k):
        calls.append(("evict", dict(keep=keep, **{n: k[n] for n in ("recent", "sink", "max_len")}), lens.clone(), k.get("stream")))
        lens.clamp_(max=keep)
    monkeypatch.setattr(rq, "cache_evict", evict)
    return blk


def x(n=2):
    return torch.zeros(n, HIDDEN, dtype=torch.bfloat16)


def test_step_on_a_stream_runs_all_of_it_there(monkeypatch):
    """The library's calls and the block's own torch operations (which go to
    the current stream) are on one stream, the one given."""
    from torch.utils._python_dispatch import TorchDispatchMode
    calls, current, ops = [], [], []
    blk = block(calls, monkeypatch, budget=4, slack=2, recent=1, sink=0)

    @contextlib.contextmanager
    def use(s):
        current.append(s)
        yield
        current.pop()

    class Operations(TorchDispatchMode):
        def __torch_dispatch__(self, func, types, args=(), kwargs=None):
            if func.__name__.split(".")[0] in ("add_", "copy_"):
                ops.append(list(current))
            return func(*args, **(kwargs or {}))

    monkeypatch.setattr(torch.cuda, "stream", use)
    s = object()
    for _ in range(8):
        before = len(calls), len(ops)
        with Operations():
            blk.step(x(), stream=s)
        assert current == []
        assert len(ops) >= before[1] + 3 and all(o == [s] for o in ops[before[1]:])
        assert len(calls) >= before[0] + 6 and all(c[3] in (None, s) for c in calls[before[0]:])
    assert any(c[0] == "evict" for c in calls)


@pytest.mark.parametrize("kw", [dict(), dict(budget=8, slack=4, recent=2, sink=1), dict(budget=60)])
def test_positions_stay_within_the_rotation_table(monkeypatch, kw):
    """Steps up to max_len use rows 0 .. max_len - 1 of the table; the next is
    refused and changes nothing, however often tokens were evicted."""
    calls = []
    blk = block(calls, monkeypatch, max_len=30, **kw)
    for _ in range(30):
        blk.step(x())
    used = [c[1]["positions"].tolist() for c in calls if c[0] == "norm"]
    assert used == [[i, i] for i in range(30)]
    assert blk.norm.c.table_rows == 30
    state = blk.length, blk.lens.tolist(), blk.place.tolist(), blk.position.tolist(), len(calls)
    for _ in range(2):
        with pytest.raises(ValueError):
            blk.step(x())
    assert state == (blk.length, blk.lens.tolist(), blk.place.tolist(), blk.position.tolist(), len(calls))


@pytest.mark.parametrize("budget,slack,recent,sink", [
    (16, 64, 32, 4), (16, 8, 16, 4), (8, 4, 2, 8), (8, 4, 0, 20), (1, 3, 5, 5), (2, 1, 1, 1), (20, 6, 12, 8), (24, 8, 4, 2)])
def test_the_newest_and_the_first_tokens_survive(monkeypatch, budget, slack, recent, sink):
    """What the block asks of the eviction keeps both groups (the plain
    eviction's result, random weights)."""
    from tests import _attention as A
    calls = []
    steps = 90
    blk = block(calls, monkeypatch, max_len=steps, budget=budget, slack=slack, recent=recent, sink=sink)
    rng = np.random.default_rng(budget)
    pos, weight, evictions = [], [], 0
    first = min(sink, budget - min(recent, 1))
    newest = min(recent, budget - first)
    for t in range(steps):
        before = len(calls)
        blk.step(x())
        pos, weight = pos + [t], weight + [float(rng.exponential())]
        for name, k, _, _ in calls[before:]:
            if name != "evict":
                continue
            evictions += 1
            assert k["keep"] == budget and k["max_len"] == len(pos)
            _, come = A.evict_row(np.array(weight, np.float32), np.array(pos), len(pos), k["keep"], k["recent"], k["sink"])
            pos, weight = [pos[j] for j in come], [weight[j] for j in come]
            assert len(pos) == budget
            assert set(range(t - newest + 1, t + 1)) <= set(pos), "the newest stay"
            assert set(range(first)) <= set(pos), "the first stay"
    assert evictions >= 1


@pytest.mark.parametrize("bad", [
    lambda: x(3), lambda: x(1), lambda: x(0), lambda: torch.zeros(2, HIDDEN + 128, dtype=torch.bfloat16),
    lambda: torch.zeros(2, HIDDEN - 1, dtype=torch.bfloat16), lambda: torch.zeros(2 * HIDDEN, dtype=torch.bfloat16),
    lambda: torch.zeros(2, 1, HIDDEN, dtype=torch.bfloat16),
    lambda: x().to("meta"), lambda: torch.zeros(HIDDEN, 2, dtype=torch.bfloat16).t(),
    lambda: torch.zeros(2, 2 * HIDDEN, dtype=torch.bfloat16)[:, :HIDDEN]])
def test_step_refuses_tokens_that_do_not_fit_its_buffers(monkeypatch, bad):
    """Before any call of the library, which takes addresses and row counts
    as they are, and before any counter moves."""
    calls = []
    blk = block(calls, monkeypatch)
    blk.step(x())
    blk.step(x().float())
    state = blk.length, blk.tokens, blk.lens.tolist(), blk.place.tolist(), blk.position.tolist(), len(calls)
    with pytest.raises(ValueError):
        blk.step(bad())
    assert state == (blk.length, blk.tokens, blk.lens.tolist(), blk.place.tolist(), blk.position.tolist(), len(calls))


@pytest.mark.parametrize("dtype", [torch.float16, torch.float64])
def test_step_refuses_types_before_counters_move(dtype):
    rng = np.random.default_rng(0)
    blk = attention.DecodeAttention(*[rng.standard_normal(s).astype(np.float32) for s in (((HQ + 2 * HKV) * D, HIDDEN), (HIDDEN, HQ * D))],
                                    HQ, HKV, D, 2, 40, page=16, device="cpu")
    with pytest.raises(KeyError):
        blk.step(x().to(dtype))
    assert (blk.length, blk.tokens, blk.lens.tolist(), blk.place.tolist(), blk.position.tolist()) == (0, 0, [0, 0], [0, 0], [0, 0])


def test_weights_of_another_shape_are_refused(monkeypatch):
    good = np.zeros(((HQ + 2 * HKV) * D, HIDDEN), np.float32), np.zeros((HIDDEN, HQ * D), np.float32)
    for Wqkv, Wo in ((np.zeros(((HQ + 2 * HKV) * D + 8, HIDDEN), np.float32), good[1]),
                     (good[0], np.zeros((HIDDEN, HQ * D + 128), np.float32)), (good[0][:-1], good[1])):
        with pytest.raises(ValueError):
            attention.DecodeAttention(Wqkv, Wo, HQ, HKV, D, 2, 40, page=16, device="cpu")


def test_linear_refuses_rows_that_do_not_fit(monkeypatch):
    calls = []
    monkeypatch.setattr(rq, "rotate_quant", lambda *a, **k: calls.append(a))
    monkeypatch.setattr(rq, "w4a4_linear", lambda *a, **k: calls.append(a))
    layer = attention.DecodeLinear(np.zeros((24, 128), np.float32), 4, device="cpu")
    X, Y = torch.zeros(4, 128), torch.zeros(4, 24)
    layer(X, Y)
    layer(X[:2], Y[:2].bfloat16())
    assert len(calls) == 4
    for a, b in ((torch.zeros(5, 128), torch.zeros(5, 24)), (X, Y[:3]), (X, torch.zeros(4, 25)), (X[:, :64], Y),
                 (X, torch.zeros(24, 4).t()), (X, Y.to("meta"))):
        with pytest.raises(ValueError):
            layer(a, b)
    assert len(calls) == 4


def test_a_budget_without_slack_evicts_every_step(monkeypatch):
    calls = []
    blk = block(calls, monkeypatch, budget=5, slack=0, recent=2, sink=1)
    for t in range(20):
        blk.step(x())
        assert blk.length == min(t + 1, 5) and blk.lens.tolist() == [blk.length] * 2
    assert sum(c[0] == "evict" for c in calls) == 15
