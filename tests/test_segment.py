"""Segment-sparse attention: refusals on the host; pool, select and attention
against the 64-bit oracle on the GPU.

Tolerances.  Pool: at most 1024 fp32 sums in at most four chains and a division;
each addition rounds by 2^-24 of a partial sum that is at most the sum of |key|,
so the mean is off by at most (n + 1) * 2^-24 * mean |key|.  Select: whole
numbers, equal (the scores differ by 2^-50 relative; the inputs are random, so
nothing lies that near the border, and exact ties are equal on both sides).
Attention: the weights enter the P.V product rounded to the input type (half a
step u = eps/2 each) and are normalised by the sum of those, which is off by one
such rounding at the most; the output rounds once more: |out - ref| <= 2u max|v|
+ u |ref| plus fp32 terms: the logit is off by at most D * 2^-24 * sum |q k| *
scale, which is below 2^-13 here and enters relative to the weights.  lse has
only the fp32 terms.
"""
from __future__ import annotations

import ctypes

import numpy as np
import pytest
import torch

import oracle.segment as oseg
import sparse_attention_top_n1_b200 as li
from synth import segment as sseg

FAKE = 1 << 20
gpu = pytest.mark.gpu


# ------------------------------------------------------------------ host

def _pr(**kw):
    f = dict(layout_q="BSND", layout_kv="BSND", dtype="bf16", B=2, S1=8, S2=256, N1=8, N2=2, D=128, seg_size=64,
             seg_count=4, init_segs=1, local_segs=1, max_segs=4, sparse_mode=3)
    f.update(kw)
    return li.make_segment_params(**f)


BAD = [
    (dict(dtype="fp32"), "LI_ERR_DTYPE"), (dict(layout_q="PA_BSND"), "LI_ERR_LAYOUT"), (dict(layout_kv="TND"), "LI_ERR_LAYOUT"),
    (dict(B=0), "LI_ERR_SHAPE"), (dict(S1=-1), "LI_ERR_SHAPE"), (dict(S2=-1), "LI_ERR_SHAPE"), (dict(N2=3), "LI_ERR_SHAPE"),
    (dict(N1=0), "LI_ERR_SHAPE"), (dict(N1=1032), "LI_ERR_SHAPE"), (dict(N1=258, N2=2), "LI_ERR_SHAPE"),
    (dict(D=96), "LI_ERR_UNSUPPORTED"), (dict(seg_size=8), "LI_ERR_SHAPE"), (dict(seg_size=40), "LI_ERR_SHAPE"),
    (dict(seg_size=1040), "LI_ERR_SHAPE"), (dict(seg_count=0), "LI_ERR_SHAPE"), (dict(seg_count=1025), "LI_ERR_SHAPE"),
    (dict(init_segs=-1), "LI_ERR_SHAPE"), (dict(init_segs=4), "LI_ERR_SHAPE"), (dict(local_segs=0), "LI_ERR_SHAPE"),
    (dict(sparse_mode=1), "LI_ERR_SHAPE"), (dict(max_segs=0), "LI_ERR_SHAPE"), (dict(max_segs=16385), "LI_ERR_SHAPE"),
    (dict(softmax_scale=-1.0), "LI_ERR_SHAPE"), (dict(softmax_scale=float("nan")), "LI_ERR_SHAPE"),
    (dict(reserved=1), "LI_ERR_SHAPE"), (dict(S1=1 << 29), "LI_ERR_SHAPE"), (dict(S2=1 << 30), "LI_ERR_SHAPE"),
    (dict(layout_kv="PA_BSND", num_blocks=4, block_size=24, max_blocks_per_seq=2), "LI_ERR_SHAPE"),
    (dict(layout_kv="PA_BSND", num_blocks=0, block_size=32, max_blocks_per_seq=2), "LI_ERR_SHAPE"),
    (dict(layout_kv="PA_BSND", num_blocks=4, block_size=32, max_blocks_per_seq=2, kv_block_stride=100), "LI_ERR_SHAPE"),
    (dict(layout_kv="PA_BSND", num_blocks=4, block_size=32, max_blocks_per_seq=2, kv_block_stride=32 * 256 + 4), "LI_ERR_SHAPE"),
]


def _calls(pr):
    L, p = li.lib(), ctypes.byref(pr)
    return {"pool": lambda k=FAKE, o=FAKE, bt=FAKE: L.li_segment_pool(p, k, FAKE, bt, None, o, None, None),
            "select": lambda k=FAKE, o=FAKE, bt=FAKE: L.li_segment_select(p, k, FAKE, FAKE, FAKE, o, None, None),
            "attention": lambda k=FAKE, o=FAKE, bt=FAKE: L.li_segment_attention(p, FAKE, k, FAKE, FAKE, FAKE, FAKE, bt, o,
                                                                               None, None, None)}


@pytest.mark.parametrize("kw,err", BAD)
@pytest.mark.parametrize("name", ["pool", "select", "attention"])
def test_segment_refuses_before_launch(name, kw, err):
    assert li.STATUS_NAMES[_calls(_pr(**kw))[name]()] == err, li.li_last_error()
    assert li.li_last_launch_count() == 0


@pytest.mark.parametrize("name", ["pool", "select", "attention"])
def test_segment_pointer_checks(name):
    call = _calls(_pr())[name]
    st = lambda **kw: li.STATUS_NAMES[call(**kw)]  # noqa: E731
    assert st(k=None) == "LI_ERR_NULL" and st(o=None) == "LI_ERR_NULL"
    assert st(k=FAKE + 8) == "LI_ERR_SHAPE" and st(o=FAKE + 2) == "LI_ERR_SHAPE"
    pa = _calls(_pr(layout_kv="PA_BSND", num_blocks=4, block_size=32, max_blocks_per_seq=2))[name]
    if name != "select":
        assert li.STATUS_NAMES[pa(bt=None)] == "LI_ERR_NULL"
    if name != "pool":
        assert li.STATUS_NAMES[_calls(_pr(S1=0))[name]()] == "LI_OK"
    assert li.li_last_launch_count() == 0


def test_wrapper_refuses_wrong_tensors():
    pr = _pr()
    q, k = torch.zeros(2, 8, 8, 128, dtype=torch.bfloat16), torch.zeros(2, 256, 2, 128, dtype=torch.bfloat16)
    idx, pooled = torch.zeros(16, 2, 4, dtype=torch.int32), torch.zeros(2, 4, 2, 128)
    for bad in (lambda: li.segment_pool(pr, k[:1]), lambda: li.segment_pool(pr, k.float()),
                lambda: li.segment_pool(pr, k, first=torch.zeros(2, dtype=torch.int32)),
                lambda: li.segment_select(pr, q, pooled.double()), lambda: li.segment_select(pr, q, pooled[:, :3]),
                lambda: li.segment_attention(pr, q, k, k, idx.long()), lambda: li.segment_attention(pr, q, k, k[:, ::2], idx),
                lambda: li.segment_attention(pr, q, k, k, idx)):   # the last: host tensors
        with pytest.raises((ValueError, TypeError)):
            bad()


EMPTY = [dict(S1=0), dict(layout_q="TND", layout_kv="TND", T1=0, T2=64), dict(S2=0),
         dict(layout_q="TND", layout_kv="TND", T1=5, T2=0), dict(S1=0, S2=0), dict(layout_q="TND", layout_kv="TND")]


@pytest.mark.parametrize("kw", EMPTY)
def test_empty_tensors_have_no_address(kw):
    pr = _pr(**kw)
    L, p = li.lib(), ctypes.byref(pr)
    rows, keys = (pr.B * pr.S1, pr.B * pr.S2) if pr.layout_q == 0 else (pr.T1, pr.T2)
    if not rows:
        assert li.STATUS_NAMES[L.li_segment_select(p, None, FAKE, FAKE, FAKE, None, None, None)] == "LI_OK"
        k = FAKE if keys else None
        assert li.STATUS_NAMES[L.li_segment_attention(p, None, k, k, None, FAKE, FAKE, None, None, None, None, None)] == "LI_OK"
    if not keys:
        assert li.STATUS_NAMES[L.li_segment_pool(p, None, FAKE, None, None, FAKE, None, None)] == "LI_OK"
        if rows:                                                  # keys are not what is missing
            st = L.li_segment_attention(p, FAKE, None, None, FAKE, FAKE, FAKE, None, None, None, None, None)
            assert li.STATUS_NAMES[st] == "LI_ERR_NULL"
    assert li.li_last_launch_count() == 0


@pytest.mark.parametrize("name", ["key", "value"])
def test_wrapper_refuses_pools_shorter_than_their_stride_says(name):
    pr = _pr(layout_kv="PA_BSND", num_blocks=4, block_size=32, max_blocks_per_seq=2, kv_block_stride=32 * 256 + 8)
    reach = 3 * (32 * 256 + 8) + 32 * 256
    t = {n: torch.zeros(reach, dtype=torch.bfloat16) for n in ("key", "value")}
    q, idx = torch.zeros(2, 8, 8, 128, dtype=torch.bfloat16), torch.zeros(16, 2, 4, dtype=torch.int32)
    for short, match in ((0, "CUDA device"), (1, "%s has %d elements of memory" % (name, reach - 1))):
        t[name] = torch.zeros(24 + reach - short, dtype=torch.bfloat16)[24:]
        calls = [lambda: li.segment_attention(pr, q, t["key"], t["value"], idx)]
        if name == "key":
            calls.append(lambda: li.segment_pool(pr, t["key"]))
        for call in calls:
            with pytest.raises(ValueError, match=match):
                call()


# ------------------------------------------------------------------ GPU

def _dev(x):
    return {k: v.cuda() for k, v in x.items()}


def _args(d, *names):
    m = dict(act_seq_q="act_q", act_seq_k="act_k", block_table="block_table")
    return {n: d.get(m[n]) for n in names}


def _select(p, d, pooled, **kw):
    return li.segment_select(li.make_segment_params(p), d["query"], pooled, **_args(d, "act_seq_q", "act_seq_k"), **kw)


def _attend(p, d, idx, **kw):
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = li.segment_attention(li.make_segment_params(p), d["query"], d["key"], d["value"], idx, status=st,
                                    **_args(d, "act_seq_q", "act_seq_k", "block_table"), **kw)
    return out, lse, int(st.item())


def _compare(p, x, out, lse, idx, flags=0, got_flags=0):
    assert got_flags == flags, hex(got_flags)
    ref, rlse = oseg.attention(p, x, idx)
    u = torch.finfo(out.dtype).eps / 2
    v = x["value"].double()
    vmax = float(v[torch.isfinite(v)].abs().max())
    o, l = out.double().cpu().numpy(), lse.double().cpu().numpy()
    assert np.isfinite(o).all()
    tol = (2 * u + 2.0 ** -13) * vmax + u * np.abs(ref) + 1e-7
    assert np.all(np.abs(o - ref) <= tol), np.max(np.abs(o - ref) / tol)
    none = np.isneginf(rlse)
    assert np.array_equal(none, np.isneginf(l)) and np.all(o[none] == 0)
    assert np.all(np.abs(l[~none] - rlse[~none]) <= 2.0 ** -13 + 2.0 ** -22 * np.abs(rlse[~none]))


CASES = {
    "decode": dict(q_lens=[1] * 5, k_lens=[1, 64, 65, 1000, 517], layout_kv="PA_BSND", block_size=128, N1=64, N2=1),
    "decode_drafts": dict(q_lens=[3, 1, 4], k_lens=[700, 90, 333], layout_kv="PA_BSND", block_size=48, N1=32, N2=2),
    "decode_long": dict(q_lens=[1, 1], k_lens=[9000, 12345], layout_kv="PA_BSND", block_size=64, seg_count=70, N1=16, N2=2),
    "prefill": dict(q_lens=[150], k_lens=[700], seg_size=64, N1=64, N2=2, seg_count=5),
    "prefill_mqa128": dict(q_lens=[60], k_lens=[400], seg_size=32, N1=128, N2=1, seg_count=6),
    "prefill_mha": dict(q_lens=[130, 40], k_lens=[260, 41], N1=4, N2=4, seg_size=16, seg_count=7, dtype="fp16"),
    "tnd": dict(layout_q="TND", layout_kv="TND", q_lens=[70, 0, 1, 33], k_lens=[90, 40, 1, 300], N1=12, N2=2, D=64,
                seg_size=32, seg_count=4, dtype="fp16"),
    "tnd_paged": dict(layout_q="TND", layout_kv="PA_BSND", block_size=16, q_lens=[19, 44], k_lens=[500, 44], N1=14, N2=2,
                      seg_size=48, seg_count=5),
    "pages_end_inside": dict(q_lens=[20, 7], k_lens=[333, 100], layout_kv="PA_BSND", block_size=80, seg_size=112, N1=24,
                             N2=3, D=64, seg_count=3),
    "wide_segments": dict(q_lens=[9], k_lens=[3000], seg_size=1024, seg_count=2, N1=10, N2=2),
    "one_entry": dict(q_lens=[40], k_lens=[200], seg_count=1, init_segs=0, N1=6, N2=1),
    "no_mask": dict(q_lens=[20, 30], k_lens=[300, 77], sparse_mode=0, local_segs=0, init_segs=0, seg_size=16, seg_count=9),
    "no_keys": dict(q_lens=[3, 5], k_lens=[0, 90], layout_kv="PA_BSND", sparse_mode=0, block_size=32),
    "more_rows_than_keys": dict(q_lens=[80], k_lens=[30], seg_size=16, seg_count=2),
    "steep": dict(q_lens=[33], k_lens=[500], softmax_scale=3.0, seg_count=4),
    "odd_group": dict(q_lens=[50], k_lens=[333], N1=21, N2=3, seg_count=3),
    "many_windows": dict(q_lens=[100, 3], k_lens=[11200, 5000], N1=2, N2=2, D=64, seg_size=16, seg_count=40),
    "full_list": dict(q_lens=[2], k_lens=[17000], N1=8, N2=1, seg_size=16, seg_count=1024, layout_kv="PA_BSND", block_size=48),
    "group_of_100": dict(q_lens=[11], k_lens=[333], N1=100, N2=1, seg_count=3, layout_kv="PA_BSND", block_size=256),
}


def _case(name, **more):
    return sseg.make_segment(sorted(CASES).index(name), **dict(CASES[name], **more))


@gpu
@pytest.mark.parametrize("name", sorted(CASES))
def test_pool_select_attention_match_the_oracle(name):
    """The three calls as they are used together, each held to the oracle on the
    GPU's own inputs to it; what lies behind the sequences is NaN."""
    p, x = _case(name, junk=float("nan"))
    d = _dev(x)
    pr = li.make_segment_params(p)
    pooled = torch.full((p.B, p.max_segs, p.N2, p.D), 7.0, device="cuda")
    li.segment_pool(pr, d["key"], pooled=pooled, **_args(d, "act_seq_k", "block_table"))
    host, want = pooled.cpu().double().numpy(), oseg.pool(p, x)
    kabs = x["key"].double().abs()
    bound = (p.seg_size + 1) * 2.0 ** -24 * float(kabs[torch.isfinite(kabs)].max())
    for b in range(p.B):
        for s in range(p.max_segs):
            if (b, s) in want:
                assert np.all(np.abs(host[b, s] - want[b, s]) <= bound)
            else:
                assert np.all(host[b, s] == 7.0)                 # behind the sequence: untouched
    idx = _select(p, d, pooled)
    assert np.array_equal(idx.cpu().numpy(), oseg.select(p, x, pooled))
    out, lse, flags = _attend(p, d, idx)
    assert li.li_last_launch_count() == 1
    _compare(p, x, out, lse, idx.cpu().numpy(), 0, flags)


@gpu
@pytest.mark.parametrize("kw", EMPTY)
def test_calls_without_rows_or_without_keys(kw):
    pr = _pr(**kw)
    tnd = pr.layout_q == 1
    e = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="cuda").normal_()  # noqa: E731
    q = e(pr.T1, 8, 128) if tnd else e(2, pr.S1, 8, 128)
    k = e(pr.T2, 2, 128) if tnd else e(2, pr.S2, 2, 128)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    aq, ak = (i32(pr.T1 // 2, pr.T1), i32(pr.T2 // 2, pr.T2)) if tnd else (None, None)
    pooled = torch.full((2, 4, 2, 128), 7.0, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    li.segment_pool(pr, k, act_seq_k=ak, pooled=pooled, status=st)
    assert bool((pooled == 7.0).all()) == (k.numel() == 0)
    idx = li.segment_select(pr, q, pooled, act_seq_q=aq, act_seq_k=ak, status=st)
    out, lse = li.segment_attention(pr, q, k, k, idx, act_seq_q=aq, act_seq_k=ak, status=st)
    rows = q.numel() // (8 * 128)
    assert idx.shape == (rows, 2, 4) and out.shape == (rows, 8, 128) and lse.shape == (rows, 8)
    assert int(st.item()) == 0
    if not k.numel():
        assert bool((idx == -1).all()) and bool((out == 0).all()) and bool(torch.isneginf(lse).all())


@gpu
def test_pool_refreshes_only_from_first():
    p, x = sseg.make_segment(50, q_lens=[1] * 4, k_lens=[64, 65, 200, 7], layout_kv="PA_BSND", block_size=32, seg_size=64)
    d = _dev(x)
    pooled = torch.full((p.B, p.max_segs, p.N2, p.D), 3.0, device="cuda")
    first = torch.tensor([63, 64, 130, -5], dtype=torch.int32, device="cuda")
    li.segment_pool(li.make_segment_params(p), d["key"], first=first, pooled=pooled, **_args(d, "act_seq_k", "block_table"))
    want, got = oseg.pool(p, x), pooled.cpu().double().numpy()
    for b in range(p.B):
        for s in range(p.max_segs):
            if (b, s) in want and s >= max(0, int(first[b])) // 64:
                assert np.all(np.abs(got[b, s] - want[b, s]) <= 65 * 2.0 ** -24 * 6)
            else:
                assert np.all(got[b, s] == 3.0)


@gpu
@pytest.mark.parametrize("ns,rows", [(9, 40), (1000, 3), (5000, 1), (200, 300)])
def test_select_ties_take_the_lower_segment(ns, rows):
    """Means of a few values, so that most scores are exactly equal; -0 and +0
    tie, NaN counts as -inf."""
    g = torch.Generator().manual_seed(ns)
    p, x = sseg.make_segment(51, q_lens=[rows], k_lens=[ns * 16], sparse_mode=0, local_segs=0, init_segs=0, N1=4, N2=2, D=64,
                             seg_size=16, seg_count=min(ns - 1, 37))
    x["query"] = torch.randint(-1, 2, x["query"].shape, generator=g).to(torch.bfloat16)
    pooled = torch.zeros(1, ns, 2, 64)
    pooled[..., 0] = torch.randint(-1, 2, (1, ns, 2), generator=g).float()
    pooled[0, ns // 3, 0] = float("nan")
    pooled[0, ns // 2, 1, 5] = -0.0
    idx = _select(p, _dev(x), pooled.cuda())
    assert np.array_equal(idx.cpu().numpy(), oseg.select(p, x, pooled))


@gpu
def test_select_separates_scores_that_32_bits_would_not():
    """Scores that differ by 2^-30 relative: the order is that of 64 bits."""
    p, x = sseg.make_segment(52, q_lens=[4], k_lens=[64 * 16], sparse_mode=0, local_segs=0, init_segs=0, N1=2, N2=1, D=64,
                             seg_size=16, seg_count=5)
    x["query"] = torch.ones_like(x["query"])
    pooled = torch.zeros(1, 64, 1, 64)
    pooled[0, :, 0, 0] = 1.0
    order = torch.randperm(64, generator=torch.Generator().manual_seed(3))
    pooled[0, :, 0, 1] = order.float() * 2.0 ** -30
    idx = _select(p, _dev(x), pooled.cuda())
    want = torch.argsort(order, descending=True)[:5].sort()[0].tolist()
    assert idx[0, 0].tolist() == want


@gpu
@pytest.mark.parametrize("rows,ns", [(5, 300), (1, 4000)])
def test_select_ranks_scores_near_the_border_in_64_bits(rows, ns):
    """A dozen scores around the last one chosen differ by 2^-28 of their size,
    less than the fast scores can tell: those chosen are the largest, and of two
    equal ones the lower segment."""
    p, x = sseg.make_segment(57, q_lens=[rows], k_lens=[ns * 16], sparse_mode=0, local_segs=0, init_segs=0, N1=2, N2=1, D=64,
                             seg_size=16, seg_count=20)
    g = torch.Generator().manual_seed(5)
    x["query"] = torch.ones_like(x["query"])
    at = torch.randperm(ns, generator=g)
    pooled = torch.randn(1, ns, 1, 64, generator=g) * 0.01
    pooled[0, at[:14], 0, 0] += 8.0                              # 14 clearly above, 12 at the border for 6 places
    pooled[0, at[14:26], 0] = 0.0
    pooled[0, at[14:26], 0, 0] = 4.0
    step = torch.tensor([0, 5, 3, 3, 9, 1, 7, 7, 2, 8, 4, 6])
    pooled[0, at[14:26], 0, 1] = step.float() * 2.0 ** -26
    idx = _select(p, _dev(x), pooled.cuda())
    assert np.array_equal(idx.cpu().numpy(), oseg.select(p, x, pooled))


@gpu
def test_select_of_zeros_and_of_many_rows():
    """Means or queries of zero: every score is zero and the lowest segments are
    chosen; rows enough for blocks of more than 16."""
    p, x = sseg.make_segment(58, q_lens=[650, 650], k_lens=[3000, 2500], N1=8, N2=8, D=64, seg_size=32, seg_count=12)
    x["query"][0, :40] = 0.0
    g = torch.Generator().manual_seed(6)
    pooled = torch.randn(p.B, p.max_segs, 8, 64, generator=g)
    pooled[1] = 0.0
    idx = _select(p, _dev(x), pooled.cuda())
    assert np.array_equal(idx.cpu().numpy(), oseg.select(p, x, pooled))


@gpu
@pytest.mark.parametrize("value", [float("inf"), float("nan"), 1e38, 1e-30])
def test_select_of_extreme_means(value):
    """Scores that overflow, vanish or are not numbers in 32 bits are still chosen
    as 64 bits choose (NaN counts as -inf)."""
    p, x = sseg.make_segment(59, q_lens=[6], k_lens=[90 * 16], sparse_mode=0, local_segs=0, init_segs=0, N1=4, N2=2, D=64,
                             seg_size=16, seg_count=9)
    g = torch.Generator().manual_seed(7)
    pooled = torch.randn(1, 90, 2, 64, generator=g)
    if value == 1e-30:
        pooled *= value
    else:
        pooled[0, 11, :, 3] = value
        pooled[0, 50, :, 5] = -value
    idx = _select(p, _dev(x), pooled.cuda())
    assert np.array_equal(idx.cpu().numpy(), oseg.select(p, x, pooled))


@gpu
@pytest.mark.parametrize("ns", [12, 90, 700, 1500])
def test_select_ties_nan_with_minus_infinity(ns):
    """Where the choice reaches into scores of -inf, a NaN is one of them: the
    lower segment is taken, whichever it is."""
    p, x = sseg.make_segment(62, q_lens=[3], k_lens=[ns * 16], sparse_mode=0, local_segs=0, init_segs=0, N1=4, N2=2, D=64,
                             seg_size=16, seg_count=9)
    x["query"] = torch.ones_like(x["query"])
    g = torch.Generator().manual_seed(8)
    pooled = torch.randn(1, ns, 2, 64, generator=g)
    pooled[0, :, 0, 3] = -float("inf")
    pooled[0, ::2, 0, 5] = float("nan")                          # head 0: NaN and -inf in turn
    pooled[0, :, 1, 3] = float("nan")
    pooled[0, ::2, 1] = 0.0
    pooled[0, ::2, 1, 3] = -float("inf")                         # head 1: -inf and NaN
    for s in (ns - 3, ns - 6):                                   # and two numbers
        pooled[0, s] = 1.0
    idx = _select(p, _dev(x), pooled.cuda())
    assert np.array_equal(idx.cpu().numpy(), oseg.select(p, x, pooled))


@gpu
@pytest.mark.parametrize("value", [1e38, -1e38, float("inf"), float("nan")])
@pytest.mark.parametrize("ns", [5, 90, 300, 1000, 1500])
def test_select_of_forced_segments_alone(ns, value):
    """init_segs + local_segs = seg_count leaves nothing to choose: scores that
    overflow 32 bits are not chosen, and nothing is written behind the row."""
    p, x = sseg.make_segment(61, q_lens=[3], k_lens=[ns * 16], sparse_mode=0, init_segs=1, local_segs=1, N1=4, N2=2, D=64,
                             seg_size=16, seg_count=2)
    x["query"] = torch.ones_like(x["query"])
    pooled = torch.full((1, ns, 2, 64), value)
    n = p.rows * 2 * 2
    wide = torch.full((n + 4096,), 77, dtype=torch.int32, device="cuda")
    idx = _select(p, _dev(x), pooled.cuda(), out=wide[:n].view(p.rows, 2, 2))
    assert bool((idx == torch.tensor([0, ns - 1], dtype=torch.int32, device="cuda")).all())
    assert bool((wide[n:] == 77).all())


@gpu
def test_select_cuts_at_max_segs_and_flags():
    p, x = sseg.make_segment(53, q_lens=[2], k_lens=[700], seg_size=64, max_segs=6, sparse_mode=0, local_segs=0, seg_count=3)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    d = _dev(x)
    pooled = li.segment_pool(li.make_segment_params(p), d["key"], status=st, **_args(d, "act_seq_k"))
    assert int(st.item()) == li.DEV_BAD_KLEN
    st.zero_()
    idx = _select(p, d, pooled, status=st)
    assert int(st.item()) == li.DEV_BAD_KLEN and int(idx.max()) < 6


def _chosen(p, x, seed, keep=0.5):
    """Random ascending rows of existing segments with holes (-1) among them."""
    rng = np.random.default_rng(seed)
    idx = np.full((p.rows, p.N2, p.seg_count), -1, np.int32)
    for b, (first, _, nq, nk) in enumerate(oseg.batches(p, x)):
        segs = -(-nk // p.seg_size)
        for r in range(first, first + nq):
            for n in range(p.N2):
                m = min(segs, p.seg_count)
                pick = np.sort(rng.permutation(segs)[:m])
                at = np.sort(rng.permutation(p.seg_count)[:m])
                idx[r, n, at] = np.where(rng.random(m) < keep, pick, -1)
    return idx


@gpu
@pytest.mark.parametrize("name", ["decode", "prefill", "prefill_mha", "tnd_paged", "pages_end_inside", "no_mask", "odd_group",
                                  "many_windows", "full_list"])
def test_attention_on_any_choice_of_segments(name):
    """Not only what select gives: rows of a block that share nothing, rows with
    nothing, segments that a row does not see at all, holes."""
    p, x = _case(name)
    idx = _chosen(p, x, 9)
    out, lse, flags = _attend(p, _dev(x), torch.from_numpy(idx).cuda())
    _compare(p, x, out, lse, idx, 0, flags)


@gpu
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("name", ["decode_drafts", "prefill", "tnd", "prefill_mqa128", "pages_end_inside"])
def test_attention_is_blind_to_what_a_row_does_not_take(name, value):
    """A key and a value that only some rows may see, or choose, are NaN or
    infinite: the other rows come out as if they were not there."""
    p, x = _case(name)
    idx = _chosen(p, x, 10, keep=0.7)
    geo = oseg.batches(p, x)
    first, _, nq, nk = geo[0]
    t = max(0, nk - nq // 2 - 1)                                 # seen by the later rows only (mode 3)
    bad = (0, t // p.seg_size)
    clean, _ = oseg.attention(p, x, idx)
    sees = np.zeros((p.rows, p.N2), bool)
    for i in range(nq):
        if oseg.visible(p, i, nq, nk) > t:
            sees[first + i] = (idx[first + i] == bad[1]).any(1)
    assert sees.any() and not sees.all()
    y = {k: v.clone() for k, v in x.items()}
    for k in ("key", "value"):
        if p.layout_kv == "PA_BSND":
            y[k][int(x["block_table"][0, t // p.block_size]), t % p.block_size] = value
        elif p.layout_kv == "BSND":
            y[k][0, t] = value
        else:
            y[k][t] = value
    out, lse, flags = _attend(p, _dev(y), torch.from_numpy(idx).cuda())
    assert flags == 0
    blind = np.repeat(~sees, p.N1 // p.N2, 1)
    u = torch.finfo(out.dtype).eps / 2
    o = out.double().cpu().numpy()
    vmax = float(x["value"].abs().max())
    assert np.all(np.abs(o - clean)[blind] <= (2 * u + 2.0 ** -13) * vmax + u * np.abs(clean[blind]) + 1e-7)
    assert not np.isfinite(o[~blind]).all(-1).any()              # and the rows that do take it show it


@gpu
@pytest.mark.parametrize("name", ["decode", "decode_long", "prefill", "prefill_mha", "tnd", "no_mask", "odd_group"])
def test_attention_of_equal_values_is_that_value(name):
    """Values that are the same for every key of a head come out bit for bit: O is
    divided by the sum of the weights that entered it.  Both sums hold at most 4480
    terms of one sign here.  Products are exact and summed in 280 steps of 16, each
    off by at most 2^-23 of the sum, weights in chains of 8 per tile of 64 and 70
    tiles: less than 2^-14 in all, which is below half a step
    (fp16 2^-12 of a value at the least, bf16 2^-9), so the result rounds to the
    value.  The logits' spread (4 here) leaves a few weights that count, none of
    them 1: the sum before rounding would be off by up to a rounding of those."""
    p, x = _case(name, softmax_scale=4.0 * CASES[name].get("D", 128) ** -0.5)
    v = torch.randn(p.N2, p.D, generator=torch.Generator().manual_seed(1)).to(x["value"].dtype)
    v[:, ::4] = 2.0 - 2.0 * torch.finfo(v.dtype).eps              # nearest below 2 but one: its step is the smallest
    x["value"][:] = v
    idx = _chosen(p, x, 14, keep=0.8)
    _, rlse = oseg.attention(p, x, idx)
    out, lse, flags = _attend(p, _dev(x), torch.from_numpy(idx).cuda())
    want = v.repeat_interleave(p.N1 // p.N2, 0).expand(p.rows, p.N1, p.D).clone()
    want[torch.from_numpy(np.isneginf(rlse))] = 0.0
    assert flags == 0 and torch.equal(out.cpu(), want)


@gpu
def test_attention_skips_and_flags_bad_entries():
    p, x = sseg.make_segment(54, q_lens=[40, 6], k_lens=[400, 100], N1=8, N2=2, seg_count=6, seg_size=64)
    idx = _chosen(p, x, 11, keep=1.0)
    d = _dev(x)
    for change, at in ((lambda v: 7, 0), (lambda v: -2, 0), (lambda v: 2 ** 31 - 1, 5)):
        bad = idx.copy()
        bad[::3, :, at] = change(bad)
        out, lse, flags = _attend(p, d, torch.from_numpy(bad).cuda())
        _compare(p, x, out, lse, np.where((bad < 0) | (bad >= 7), -1, bad), li.DEV_BAD_INDEX, flags)
    twice = np.full_like(idx, -1)
    twice[:, :, :3] = [0, 0, 1]                                  # named twice, and out of order behind it
    twice[:, :, 4] = 0
    out, lse, flags = _attend(p, d, torch.from_numpy(twice).cuda())
    _compare(p, x, out, lse, twice, li.DEV_BAD_INDEX, flags)


@gpu
def test_bad_pages_are_skipped_and_flagged():
    p, x = sseg.make_segment(55, q_lens=[5, 3], k_lens=[200, 150], layout_kv="PA_BSND", block_size=32, seg_size=64,
                             N1=4, N2=1, seg_count=4, sparse_mode=0, local_segs=0, init_segs=0)
    y = {k: v.clone() for k, v in x.items()}
    y["block_table"][1, 1], y["block_table"][1, 4] = -1, p.num_blocks
    d = _dev(y)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    pooled = li.segment_pool(li.make_segment_params(p), d["key"], status=st, **_args(d, "act_seq_k", "block_table"))
    assert int(st.item()) == li.DEV_BAD_BLOCK
    k1 = oseg.keys(p, x, "key", 1, np.arange(32))                # segment 0 of batch 1 without its second page
    assert np.all(np.abs(pooled[1, 0].cpu().double().numpy() - k1.mean(0)) <= 65 * 2.0 ** -24 * 6)
    idx = np.zeros((p.rows, 1, 4), np.int32)
    idx[:] = [0, 1, 2, -1]
    out, lse, flags = _attend(p, d, torch.from_numpy(idx).cuda())
    assert flags == li.DEV_BAD_BLOCK
    ref, rlse = oseg.attention(p, x, idx)
    q = oseg.f64(x["query"]).reshape(p.rows, 4, p.D)
    t = np.concatenate([np.arange(32), np.arange(64, 128), np.arange(160 - 10, 150)]).astype(int)   # pages 1 and 4 left out
    kk, vv = oseg.keys(p, x, "key", 1, t)[:, 0], oseg.keys(p, x, "value", 1, t)[:, 0]
    for r in range(p.rows):
        b = r // p.S1
        if b == 0:
            want = ref[r]
        elif r - p.S1 < 3:
            l = p.scale * (q[r] @ kk.T)
            e = np.exp(l - l.max(1, keepdims=True))
            want = (e / e.sum(1, keepdims=True)) @ vv
        else:
            want = np.zeros((4, p.D))
        assert np.all(np.abs(out[r].double().cpu().numpy() - want) <= (2 ** -7 + 2 ** -13) * 5)


@gpu
def test_attention_gives_the_same_bits_again_and_again():
    """Many launches in a row: no wait runs into its limit, no bit changes."""
    for name in ("tnd", "pages_end_inside", "prefill", "decode"):
        p, x = _case(name)
        d, idx = _dev(x), torch.from_numpy(_chosen(p, x, 12)).cuda()
        first = _attend(p, d, idx)
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        pr = li.make_segment_params(p)
        outs = [li.segment_attention(pr, d["query"], d["key"], d["value"], idx, status=st,
                                     **_args(d, "act_seq_q", "act_seq_k", "block_table")) for _ in range(100)]
        assert first[2] == 0 and int(st.item()) == 0
        assert all(torch.equal(o, first[0]) and torch.equal(l, first[1]) for o, l in outs)


@gpu
def test_pools_with_pages_apart():
    """kv_block_stride that is no multiple of a key row."""
    p, x = sseg.make_segment(60, q_lens=[9, 2], k_lens=[300, 128], layout_kv="PA_BSND", block_size=64, N1=16, N2=2)
    d = _dev(x)
    n, page = p.num_blocks, 64 * 2 * 128
    apart = []
    for name in ("key", "value"):
        wide = torch.full((n, page + 24), float("nan"), dtype=torch.bfloat16, device="cuda")
        wide[:, :page] = d[name].view(n, page)
        apart.append(wide.view(-1)[:n * (page + 24)].as_strided((n, 64, 2, 128), (page + 24, 256, 128, 1)))
    p2 = sseg.SegmentProblem(**{**p.__dict__, "kv_block_stride": page + 24})
    pooled = li.segment_pool(li.make_segment_params(p2), apart[0], **_args(d, "act_seq_k", "block_table"))
    idx = _select(p, d, pooled)
    a = _attend(p2, dict(d, key=apart[0], value=apart[1]), idx)
    b = _attend(p, d, idx)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and a[2] == b[2] == 0


@gpu
def test_key_and_value_pages_interleaved_in_one_pool():
    """kv_block_stride: pool [num_blocks, 2, block_size, N2, D] holds keys and values."""
    p, x = sseg.make_segment(56, q_lens=[9, 2], k_lens=[300, 128], layout_kv="PA_BSND", block_size=64, N1=16, N2=2)
    kv = torch.stack([x["key"], x["value"]], 1).contiguous()
    p2 = sseg.SegmentProblem(**{**p.__dict__, "kv_block_stride": 2 * 64 * 2 * 128})
    d = _dev(x)
    both = kv.cuda()
    k, v = both[:, 0], both[:, 1]
    pooled = li.segment_pool(li.make_segment_params(p2), k, **_args(d, "act_seq_k", "block_table"))
    idx = _select(p, d, pooled)
    dense = li.segment_pool(li.make_segment_params(p), d["key"], **_args(d, "act_seq_k", "block_table"))
    assert np.array_equal(idx.cpu().numpy(), _select(p, d, dense).cpu().numpy())
    a = _attend(p2, dict(d, key=k, value=v), idx)
    b = _attend(p, d, idx)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and a[2] == b[2] == 0


@gpu
def test_same_calls_on_streams_and_in_graphs_give_the_same_bits():
    p, x = _case("prefill")
    d = _dev(x)
    pr = li.make_segment_params(p)
    args = _args(d, "act_seq_k", "block_table")

    def chain(pooled, idx, out, lse):
        li.segment_pool(pr, d["key"], pooled=pooled, **args)
        _select(p, d, pooled, out=idx)
        li.segment_attention(pr, d["query"], d["key"], d["value"], idx, out=out, lse=lse,
                             **_args(d, "act_seq_q", "act_seq_k", "block_table"))

    def buffers():
        return (torch.zeros(p.B, p.max_segs, p.N2, p.D, device="cuda"),
                torch.zeros(p.rows, p.N2, p.seg_count, dtype=torch.int32, device="cuda"),
                torch.zeros(p.rows, p.N1, p.D, dtype=torch.bfloat16, device="cuda"),
                torch.zeros(p.rows, p.N1, device="cuda"))
    a, b, c, e = (buffers() for _ in range(4))
    chain(*a)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(s1):
        chain(*b)
    with torch.cuda.stream(s2):
        chain(*c)
    g1 = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g1):
        chain(*e)
    g1.replay()
    torch.cuda.synchronize()
    for other in (b, c, e):
        assert all(torch.equal(u, v) for u, v in zip(a, other))
    d["query"].neg_()
    g1.replay()
    chain(*a)
    assert all(torch.equal(u, v) for u, v in zip(a, e))


@gpu
def test_a_serving_step_over_a_forked_and_packed_cache():
    """Rotary positions, a paged cache that is reserved, filled, forked, freed and
    packed, then pool, select and attention: a child answers as its parent does,
    and packing changes no bit of any answer."""
    B, ps, cols, N1, N2, D, seg = 6, 32, 16, 16, 2, 128, 64
    P = 80
    g = torch.Generator().manual_seed(77)
    lens = [300, 37, 411, 0, 0, 90]
    pp = li.make_pages_params(num_pages=P, page_size=ps, max_pages_per_seq=cols, B=B)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    state = (torch.full((B, cols), -1, dtype=torch.int32, device="cuda"), i32([0] * B), i32([0] * P))
    ws = li.alloc_pages_workspace(pp)
    state = li.pages_reserve(pp, *state, i32(lens), workspace=ws)
    pools = [torch.full((P, ps, N2, D), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    T = sum(lens)
    pos = torch.cat([torch.arange(n) for n in lens]).to(torch.int32).cuda()
    row = torch.cat([torch.full((n,), b) for b, n in enumerate(lens)]).cuda()
    key, value = (torch.randn(T, N2, D, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    f, m = li.rope_frequencies(64, scaling="yarn", factor=4.0, original_positions=4096)
    rp = lambda rows, n1: li.make_rope_params(dtype="bf16", rows=rows, N1=n1, N2=0, D=D, rot_dim=64, rot_offset=0,  # noqa: E731
                                              pairing="half", inverse=0, mscale=m)
    key, _ = li.rope(rp(T, N2), pos, f.cuda(), key)
    page = state[0][row, pos.long() // ps].long()
    pools[0][page, pos.long() % ps], pools[1][page, pos.long() % ps] = key, value
    # rows 3 and 4 become children of 0 and 2; row 1 ends; the rest is packed
    state = li.pages_fork(pp, pools, *state, i32([0, 2]), i32([3, 4]), workspace=ws)
    state = li.pages_free(pp, *state, i32([1]), workspace=ws)
    sp = li.make_segment_params(layout_q="BSND", layout_kv="PA_BSND", dtype="bf16", B=B, S1=1, N1=N1, N2=N2, D=D,
                                num_blocks=P, block_size=ps, max_blocks_per_seq=cols, seg_size=seg, seg_count=4,
                                init_segs=1, local_segs=1, max_segs=cols * ps // seg, sparse_mode=3)
    q0 = torch.randn(B, N1, D, generator=g).to(torch.bfloat16).cuda()
    q0[3], q0[4] = q0[0], q0[2]
    q, _ = li.rope(rp(B, N1), (state[1] - 1), f.cuda(), q0)

    def answer(state):
        pooled = torch.zeros(B, sp.max_segs, N2, D, device="cuda")
        li.segment_pool(sp, pools[0], act_seq_k=state[1], block_table=state[0], pooled=pooled)
        idx = li.segment_select(sp, q, pooled, act_seq_k=state[1])
        return idx, *li.segment_attention(sp, q, pools[0], pools[1], idx, act_seq_k=state[1], block_table=state[0])
    idx, out, lse = answer(state)
    for child, parent in ((3, 0), (4, 2)):
        assert all(torch.equal(v[child], v[parent]) for v in (idx, out, lse))
    assert bool((out[1] == 0).all()) and bool(torch.isneginf(lse[1]).all()) and bool(torch.isfinite(out).all())
    packed = li.pages_compact(pp, pools, *state, workspace=ws)
    live = int((packed[2] != 0).sum())
    assert bool((packed[2][:live] > 0).all()) and not torch.equal(packed[0], state[0])
    assert all(torch.equal(a, b) for a, b in zip(answer(packed), (idx, out, lse)))
    # against the definition, on the packed cache
    p = sseg.SegmentProblem(layout_kv="PA_BSND", B=B, S1=1, N1=N1, N2=N2, D=D, num_blocks=P, block_size=ps,
                            max_blocks_per_seq=cols, seg_size=seg, seg_count=4, max_segs=sp.max_segs)
    x = dict(query=q.cpu(), key=pools[0].cpu(), value=pools[1].cpu(), act_k=packed[1].cpu(), block_table=packed[0].cpu())
    _compare(p, x, out, lse, idx.cpu().numpy())
    # a child that grows writes into its own page: the parent's answer stays
    grown = li.pages_reserve(pp, *packed, packed[1] + i32([0, 0, 0, 1, 0, 0]), workspace=ws)
    n = int(grown[1][3])
    pools[0][grown[0][3, (n - 1) // ps].long(), (n - 1) % ps] = 100.0
    again = answer((grown[0], packed[1], grown[2]))
    assert torch.equal(again[1][0], out[0]) and torch.equal(again[1][3], out[3])
