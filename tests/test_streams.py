"""What the wrappers allocate themselves: the workspace lives until the launch,
and memory for a call on another stream belongs to that stream."""
from __future__ import annotations

import ctypes
import weakref

import numpy as np
import pytest
import torch

import oracle.cache as oc
import sparse_attention_top_n1_b200 as li
import synth
from parity import to_device
from synth import segment as sseg
from synth import sfa as ssfa

i32 = torch.int32


# ------------------------------------------------------------------ host

@pytest.mark.parametrize("name", ["reserve", "fork", "free", "compact"])
def test_default_workspace_lives_until_the_launch(name, monkeypatch):
    """The tensor behind the workspace pointer exists when the library is called."""
    pr = li.make_pages_params(num_pages=8, page_size=4, max_pages_per_seq=2, B=3)
    state = (torch.zeros(3, 2, dtype=i32), torch.zeros(3, dtype=i32), torch.zeros(8, dtype=i32))
    rows = torch.zeros(3, dtype=i32)
    made, seen, empty = [], [], torch.empty

    def noted(*a, **k):
        t = empty(*a, **k)
        if t.dtype == torch.uint8:
            made.append(weakref.ref(t))
        return t
    monkeypatch.setattr(torch, "empty", noted)
    monkeypatch.setattr(li, "_launch", lambda *a, **k: seen.append([r() is not None for r in made]))
    {"reserve": lambda: li.pages_reserve(pr, *state, rows), "fork": lambda: li.pages_fork(pr, [], *state, rows, rows),
     "free": lambda: li.pages_free(pr, *state, rows), "compact": lambda: li.pages_compact(pr, [], *state)}[name]()
    assert seen == [[True]]


# ------------------------------------------------------------------ GPU

def _state():
    rng = np.random.default_rng(4)
    B, cols, ps, P = 40, 6, 16, 200
    table, lens, refs = np.full((B, cols), -1, np.int32), np.zeros(B, np.int32), np.zeros(P, np.int32)
    free = list(rng.permutation(P))
    for b in range(0, B, 2):
        lens[b] = rng.integers(1, 70)
        for c in range(-(-int(lens[b]) // ps)):
            table[b, c] = free.pop()
            refs[table[b, c]] = 1
    return table, lens, refs, ps, P


def _pages(name):
    """(call, what the model says)"""
    table, lens, refs, ps, P = _state()
    B, cols = table.shape
    host = torch.randint(-99, 99, (P, ps, 4), generator=torch.Generator().manual_seed(1), dtype=torch.int16)
    model = oc.Pages(table, lens, refs, ps, [host.numpy()])
    pr = li.make_pages_params(num_pages=P, page_size=ps, max_pages_per_seq=cols, B=B)
    d, pool = [torch.from_numpy(t).cuda() for t in (table, lens, refs)], host.cuda()
    a, b = list(range(0, B, 2)), list(range(1, B, 2))
    up = [min(int(n) + 20, cols * ps) for n in lens]
    dev = {k: torch.tensor(v, dtype=i32, device="cuda") for k, v in (("a", a), ("b", b), ("up", up))}
    if name == "reserve":
        model.reserve(up)
        f = lambda **k: li.pages_reserve(pr, *d, dev["up"], **k)  # noqa: E731
    elif name == "fork":
        model.fork(a, b)
        f = lambda **k: li.pages_fork(pr, [pool], *d, dev["a"], dev["b"], **k)  # noqa: E731
    elif name == "free":
        model.free(a[:7])
        f = lambda **k: li.pages_free(pr, *d, dev["a"][:7], **k)  # noqa: E731
    else:
        model.compact()
        f = lambda **k: li.pages_compact(pr, [pool], *d, **k)  # noqa: E731
    want = [torch.tensor(v, dtype=i32) for v in (model.table, model.lens, model.refs)] + [torch.from_numpy(model.pools[0])]
    return lambda **k: [*f(**k), pool], want


def _others(name):
    """(call, what it gives on the current stream)"""
    if name == "indexer":
        p, inp = synth.make_tiny()
        x = to_device(inp, "cuda:0")
        f = lambda **k: list(li.indexer(li.make_params(p), x["query"], x["key"], x["weights"], **k))  # noqa: E731
    elif name == "sparse_attention":
        p, x = ssfa.make_sfa(0, B=2, S1=12, S2=200, q_lens=[12, 7], N1=32, K=96, holes=0.2)
        x = to_device(x, "cuda:0")
        f = lambda **k: list(li.sparse_attention(li.make_sfa_params(p), x["query"], x["key"], x["value"],  # noqa: E731
                                                 x["sparse_indices"], act_seq_q=x.get("act_q"), **k))
    elif name == "rope":
        g = torch.Generator().manual_seed(2)
        q, k_ = (torch.randn(50, n, 128, generator=g).to(torch.bfloat16).cuda() for n in (8, 2))
        pos, fr = torch.arange(50, dtype=i32).cuda(), li.rope_frequencies(64)[0].cuda()
        pr = li.make_rope_params(dtype="bf16", rows=50, N1=8, N2=2, D=128, rot_dim=64, rot_offset=0, pairing="half", inverse=0)
        f = lambda **k: list(li.rope(pr, pos, fr, q, k_, **k))  # noqa: E731
    else:
        p, x = sseg.make_segment(3, q_lens=[40, 3], k_lens=[300, 90], N1=8, N2=2, seg_count=4, seg_size=32)
        x, pr = {k: v.cuda() for k, v in x.items()}, li.make_segment_params(p)
        lens = dict(act_seq_k=x["act_k"])
        fill = torch.zeros(p.B, p.max_segs, p.N2, p.D, device="cuda")
        li.segment_pool(pr, x["key"], pooled=fill, **lens)
        idx = li.segment_select(pr, x["query"], fill, act_seq_q=x["act_q"], **lens)
        segs = [-(-n // 32) for n in (300, 90)]

        def pool(**k):                                            # what lies behind a sequence is undefined
            t = li.segment_pool(pr, x["key"], **lens, **k)
            return [t[0, :segs[0]], t[1, :segs[1]]]
        f = {"segment_pool": pool,
             "segment_select": lambda **k: [li.segment_select(pr, x["query"], fill, act_seq_q=x["act_q"], **lens, **k)],
             "segment_attention": lambda **k: list(li.segment_attention(pr, x["query"], x["key"], x["value"], idx,
                                                                        act_seq_q=x["act_q"], **lens, **k))}[name]
    return f, [t.cpu() for t in f()]


@pytest.mark.gpu
@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("name", ["reserve", "fork", "free", "compact", "indexer", "sparse_attention", "rope", "segment_pool",
                                  "segment_select", "segment_attention"])
def test_calls_on_another_stream_allocate_for_it(name, raw):
    """The call waits on its stream while the current one allocates and writes as
    much as it likes: nothing of the call's is given away meanwhile."""
    f, want = (_pages if name in ("reserve", "fork", "free", "compact") else _others)(name)
    side = torch.cuda.Stream()
    f()                                                           # kernels are loaded (again is the same for all of them)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)
    got = f(stream=side.cuda_stream if raw else side)
    assert not side.query()                                       # still asleep: the call has not run
    junk = [torch.full((n,), 0x7f, dtype=torch.uint8, device="cuda") for n in (256, 1000, 5000, 20000, 1 << 20) for _ in range(40)]
    torch.cuda.synchronize()
    assert all(torch.equal(a.cpu(), b) for a, b in zip(got, want))
    assert all(bool((t == 0x7f).all()) for t in junk)


@pytest.mark.gpu
def test_the_default_stream_by_its_handle():
    """Handle 0 is the legacy default stream, the current one here."""
    f, want = _pages("reserve")
    got = f(stream=0)
    torch.cuda.synchronize()
    assert all(torch.equal(a.cpu(), b) for a, b in zip(got, want))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        got = f(stream=0)
        torch.cuda.synchronize()
    assert all(torch.equal(a.cpu(), b) for a, b in zip(got, want))


@pytest.mark.gpu
def test_handles_of_every_kind():
    f, want = _pages("reserve")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for h in (None, 0, 1, 2, ctypes.c_void_p(0), ctypes.c_void_p(side.cuda_stream), side.cuda_stream, side,
              torch.cuda.default_stream()):
        got = f(stream=h)
        torch.cuda.synchronize()
        assert all(torch.equal(a.cpu(), b) for a, b in zip(got, want))
