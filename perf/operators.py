"""Measured cases of the cache-path operators: rotary positions, the pages of a
key/value cache, and sparse attention over the segments a cheap score selects.

``run`` computes an operator either in its plain form (elementary torch
operations, 32 bits, 64 where 32 lose what matters) or, with ``own`` set,
through the library's entry points.  Sizes follow the library's workloads: 64
query heads of 128, 64 decode rows over lengths 4096..65536 in pages of 128,
30720 packed prefill tokens, 2048 selected keys per row.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}


# ------------------------------------------------------------------ the cases

def _rope(**kw):
    return dict(dict(op="rope", dtype="bf16", rows=64, heads=64, key_heads=1, d=128, rot=64, off=0,
                     pairing="interleaved", scaling="none", factor=1.0, inverse=False, max_pos=65536), **kw)


def _pages(**kw):
    return dict(dict(page=128, pools=2, n2=1, d=128, seqs=64, lo=4096, hi=65536, lens_seed=1), **kw)


def _seg(**kw):
    return dict(dict(dtype="bf16", layout_q="BSND", layout_kv="PA_BSND", B=64, q_lo=1, q_hi=1, k_lo=4096, k_hi=65536,
                     n1=64, n2=1, d=128, seg=64, k=32, init=1, local=2, page=128, mode=3, lens_seed=2), **kw)


def listed():
    return [
        # one decode step of 64 sequences: part of the head, neighbouring pairs, far positions; latency
        _rope(name="rope decode"),
        # a packed prefill of 30720 tokens, whole heads, split halves, stretched positions; bandwidth
        _rope(name="rope prefill", rows=30720, heads=64, key_heads=8, rot=128, pairing="half", scaling="yarn", factor=8.0,
              max_pos=16384),
        # parallel sampling: four children each of 16 prompts share their pages, the open page is copied
        _pages(name="pages fork", op="pages_fork", seqs=80, live=16, n=64, lo=1000, hi=8000),
        # after a wave of requests has ended a third of the pool is moved together
        _pages(name="pages compact", op="pages_compact", seqs=64, n=24, lo=4096, hi=16384),
        # a step that retires 16 requests and admits 16 others
        _pages(name="pages turnover", op="pages_turnover", seqs=64, n=16),
        # a decode step refreshes the open segment's mean of each sequence; latency
        _seg(name="pool decode", op="segment_pool", n2=2, new=1),
        # the means of whole prompts, packed
        _seg(name="pool prefill", op="segment_pool", layout_q="TND", layout_kv="TND", B=4, k_lo=2048, k_hi=16384, n2=4,
             new=0),
        # decode: 64 rows over up to 1024 segments
        _seg(name="select decode", op="segment_select"),
        # a chunk of 8192 new rows chooses among the segments of 32768 keys, 4 key heads
        _seg(name="select prefill", op="segment_select", layout_kv="BSND", B=1, q_lo=8192, q_hi=8192, k_lo=32768,
             k_hi=32768, n2=4),
        # paged decode: each row reads 2048 keys of its sequence
        _seg(name="attention decode", op="segment_attention"),
        # a chunk of 4096 new tokens over 16384 keys in pages, 32 query heads to a key head, 2048 keys a row
        _seg(name="attention prefill", op="segment_attention", B=1, q_lo=4096, q_hi=4096, k_lo=16384, k_hi=16384, n2=2),
        # packed short sequences of odd lengths, half-size heads, 6 query heads to a key head
        _seg(name="attention ragged", op="segment_attention", layout_q="TND", layout_kv="TND", dtype="fp16", B=7, q_lo=1,
             q_hi=400, k_lo=1, k_hi=1500, n1=12, n2=2, d=64, seg=32, k=9, local=1),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["rope", "pages_fork", "pages_compact", "pages_turnover", "segment_pool", "segment_select",
                     "segment_attention", "segment_attention"])
    seed = rng.randrange(1 << 20)
    if op == "rope":
        d = rng.choice([64, 96, 128, 192, 256])
        rot = rng.choice([d, d // 2, 2 * rng.randint(1, d // 2)])
        heads = _log(rng, 1, 128)
        scaling = rng.choice(["none", "linear", "ntk", "yarn"])
        rot = max(rot, 4)
        return _rope(dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]), rows=_log(rng, 1, 250_000_000 // (heads * d * 9)),
                     heads=heads, key_heads=rng.randint(0, min(8, heads)), d=d, rot=rot,
                     off=rng.choice([0, d - rot, rng.randint(0, d - rot)]), pairing=rng.choice(["half", "interleaved"]),
                     scaling=scaling, factor=1.0 if scaling == "none" else rng.uniform(1.5, 40.0),
                     inverse=rng.random() < 0.3, max_pos=_log(rng, 128, 1 << 20))
    if op.startswith("pages"):
        seqs = _log(rng, 2, 128)
        page = rng.choice([16, 32, 48, 64, 128, 256])
        hi = _log(rng, 16, 1_000_000 // seqs)
        live = rng.randint(1, seqs - 1)
        n = {"pages_fork": seqs - live, "pages_compact": rng.randint(1, seqs), "pages_turnover": rng.randint(1, seqs)}[op]
        return _pages(op=op, seqs=seqs, page=page, pools=rng.randint(1, 4), n2=rng.choice([1, 2, 4]),
                      d=rng.choice([64, 128]), lo=rng.randint(0, hi), hi=hi, n=n, lens_seed=seed,
                      **({"live": live} if op == "pages_fork" else {}))
    layout_q = rng.choice(["BSND", "TND"])
    n2 = rng.choice([1, 1, 2, 4, 8])
    c = dict(op=op, dtype=rng.choice(["bf16", "fp16"]), layout_q=layout_q,
             layout_kv=rng.choice([layout_q, "PA_BSND"]), n2=n2, n1=n2 * rng.choice([1, 2, 3, 4, 7, 8, 16, 16, 32]),
             d=rng.choice([64, 128]), seg=rng.choice([16, 32, 48, 64, 64, 128]), page=rng.choice([16, 48, 64, 128, 256]),
             mode=rng.choice([0, 3, 3]), lens_seed=seed, init=rng.randint(0, 2), local=rng.randint(1, 3))
    c["n1"] = min(c["n1"], 128)
    if rng.random() < 0.5:                                   # decode, or a few drafted tokens
        B = _log(rng, 1, 64)
        hi = _log(rng, 1, min(65536, 1_000_000_000 // (B * n2 * c["d"])))
        c.update(B=B, q_lo=1, q_hi=rng.choice([1, 1, 1, 4]), k_lo=rng.randint(1, hi), k_hi=hi)
    else:                                                    # prefill
        B = rng.randint(1, 8)
        q = _log(rng, 2, 4096 // B)
        c.update(B=B, q_lo=rng.randint(1, q), q_hi=q, k_lo=1, k_hi=_log(rng, q, 16384))
    rows = B * c["q_hi"]
    if op == "segment_pool":
        c["new"] = rng.choice([0, 1, 1, 5, 70])
    # at most the work of the largest listed case
    most = min(128, 500_000_000 // (rows * c["n1"] * c["seg"]), 16_000_000 // (rows * n2 * c["seg"]))
    c["k"] = _log(rng, c["init"] + c["local"], max(8, most))
    return _seg(**c)


def _lens(c):
    """Lengths of the case's sequences: the case says them, not the seed."""
    rng = random.Random(c["lens_seed"])
    if c["op"].startswith("pages"):
        return [rng.randint(c["lo"], c["hi"]) for _ in range(c["seqs"])]
    q = [rng.randint(c["q_lo"], c["q_hi"]) for _ in range(c["B"])]
    k = [max(rng.randint(c["k_lo"], c["k_hi"]), n) for n in q]
    return q, k


def _cdiv(a, b):
    return -(-a // b)


# ------------------------------------------------------------------ the inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, shape, dtype, std=1.0):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, std, generator=g)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _frequencies(c):
    """Radians per position of each pair, and what the rotation is multiplied by."""
    rot, base, s = c["rot"], 10000.0, c["factor"]
    p = torch.arange(rot // 2, dtype=torch.float64)
    if c["scaling"] == "ntk":
        base *= s ** (rot / (rot - 2))
    f = base ** (-2.0 * p / rot)
    if c["scaling"] == "linear":
        f = f / s
    if c["scaling"] == "yarn":
        # pairs that turn over 32 times in the first 4096 positions stay, those that turn less than once are stretched
        at = [rot * math.log(4096 / (turns * 2 * math.pi)) / (2 * math.log(base)) for turns in (32.0, 1.0)]
        lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rot - 1)
        keep = 1 - ((p - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        f = f * keep + f / s * (1 - keep)
        return f.cuda(), 0.1 * math.log(s) + 1.0
    return f.cuda(), 1.0


def _prepare_rope(c, g):
    f, m = _frequencies(c)
    dt = DTYPES[c["dtype"]]
    s = dict(positions=torch.randint(0, c["max_pos"], (c["rows"],), device="cuda", dtype=torch.int32, generator=g),
             inv_freq=f, mscale=m, query=_randn(g, (c["rows"], c["heads"], c["d"]), dt), key=None, key_out=None)
    s["out"] = torch.empty_like(s["query"])
    if c["key_heads"]:
        s["key"] = _randn(g, (c["rows"], c["key_heads"], c["d"]), dt)
        s["key_out"] = torch.empty_like(s["key"])
    return s


def _pages_geometry(c):
    """(lengths before, rows acted on, their source rows, lengths after, pages of the pool)"""
    rng = random.Random(c["lens_seed"] + 1)
    lens = _lens(c)
    if c["op"] == "pages_fork":
        new = list(range(c["live"], c["seqs"]))[:c["n"]]
        src = [rng.randrange(c["live"]) for _ in new]
        lens = lens[:c["live"]] + [0] * (c["seqs"] - c["live"])
        spare = len(new) + 3
    else:
        new = rng.sample(range(c["seqs"]), c["n"])
        src = new
        spare = 5
    after = list(lens)
    if c["op"] == "pages_turnover":                     # the retired rows take the lengths of others, newly drawn
        for r in new:
            after[r] = rng.randint(c["lo"], c["hi"])
        spare += sum(_cdiv(after[r], c["page"]) for r in new)
    return lens, new, src, after, sum(_cdiv(n, c["page"]) for n in lens) + spare


def _prepare_pages(c, g):
    lens, new, src, after, pages = _pages_geometry(c)
    need = [_cdiv(n, c["page"]) for n in lens]
    columns = max(1, _cdiv(max(max(after), max(lens)), c["page"]))
    perm = torch.randperm(pages, device="cuda", generator=g).to(torch.int32)
    start = _ints([0] + need).cumsum(0)[:-1]
    at = torch.arange(columns, device="cuda", dtype=torch.int32)
    held = at[None] < _ints(need)[:, None]
    table = torch.where(held, perm[(start[:, None] + at[None]).clamp(max=pages - 1)], -1).to(torch.int32)
    ref = torch.zeros(pages + 1, dtype=torch.int32, device="cuda")
    ref[torch.where(held, table, pages).reshape(-1).long()] = 1
    if c["op"] == "pages_compact":                      # the sequences that ended have left holes
        gone = torch.zeros(c["seqs"], dtype=torch.bool, device="cuda")
        gone[_ints(new).long()] = True
        ref[torch.where(held & gone[:, None], table, pages).reshape(-1).long()] = 0
        table = torch.where(gone[:, None], -1, table).to(torch.int32)
        lens = [0 if i in set(new) else n for i, n in enumerate(lens)]
    s = dict(table=table.contiguous(), lens=_ints(lens), ref=ref[:pages].contiguous(), rows=_ints(new), src=_ints(src),
             after=_ints(after), num_pages=pages, columns=columns)
    s["pools"] = [_randn(g, (pages, c["page"], c["n2"], c["d"]), torch.bfloat16) for _ in range(c["pools"])]
    s["table_out"], s["lens_out"], s["ref_out"] = (torch.empty_like(s[k]) for k in ("table", "lens", "ref"))
    return s


def _smooth_rows(g, n, heads, d, dtype):
    """Query rows of one sequence: neighbours resemble each other, as neighbouring tokens' queries do."""
    knots = _randn(g, (n // 16 + 2, heads, d), torch.float32)
    x = torch.arange(n, device="cuda") / 16.0
    i, w = x.long(), (x % 1.0)[:, None, None]
    base = knots[i] * (1 - w) + knots[i + 1] * w
    return (1.3 * base + 0.5 * _randn(g, (n, heads, d), torch.float32)).to(dtype)


def _prepare_segment(c, g):
    q_lens, k_lens = _lens(c)
    dt = DTYPES[c["dtype"]]
    B, n1, n2, d = c["B"], c["n1"], c["n2"], c["d"]
    s = dict(S1=max(q_lens), S2=max(k_lens), T1=sum(q_lens), T2=sum(k_lens), num_blocks=0, columns=0, block_table=None,
             max_segs=_cdiv(max(k_lens), c["seg"]))
    s["act_q"], s["act_k"] = _ints(q_lens), _ints(k_lens)
    if c["layout_q"] == "TND":
        s["act_q"] = s["act_q"].cumsum(0).to(torch.int32)
    if c["layout_kv"] == "TND":
        s["act_k"] = s["act_k"].cumsum(0).to(torch.int32)
    rows = B * s["S1"] if c["layout_q"] == "BSND" else s["T1"]
    s["nrows"] = rows
    if c["layout_kv"] == "PA_BSND":
        need = [_cdiv(n, c["page"]) for n in k_lens]
        s["num_blocks"], s["columns"] = sum(need) + 2, max(need)
        perm = torch.randperm(s["num_blocks"], device="cuda", generator=g).to(torch.int32)
        start = _ints([0] + need).cumsum(0)[:-1]
        at = torch.arange(s["columns"], device="cuda", dtype=torch.int32)
        s["block_table"] = torch.where(at[None] < _ints(need)[:, None],
                                       perm[(start[:, None] + at[None]).clamp(max=s["num_blocks"] - 1)], -1).to(torch.int32)
        shape = (s["num_blocks"], c["page"], n2, d)
    else:
        shape = (B, s["S2"], n2, d) if c["layout_kv"] == "BSND" else (s["T2"], n2, d)
    if c["op"] != "segment_select":
        s["key"] = _randn(g, shape, dt)
    if c["op"] == "segment_pool":
        s["first"] = _ints([max(0, n - c["new"]) for n in k_lens]) if c["new"] else None
        s["pooled"] = _randn(g, (B, s["max_segs"], n2, d), torch.float32)
        return s
    s["query"] = _smooth_rows(g, rows, n1, d, dt).view((B, s["S1"], n1, d) if c["layout_q"] == "BSND" else (rows, n1, d))
    # segment means of keys that have a direction of their own in each segment, as cached keys do
    s["pooled"] = _randn(g, (B, s["max_segs"], n2, d), torch.float32, 0.5)
    s["seg_idx"] = torch.empty((rows, n2, c["k"]), dtype=torch.int32, device="cuda")
    if c["op"] == "segment_attention":
        s["value"] = _randn(g, shape, dt)
        s["seg_idx"] = _plain_select(c, s).contiguous()
        s["out"] = torch.empty((rows, n1, d), dtype=dt, device="cuda")
        s["lse"] = torch.empty((rows, n1), dtype=torch.float32, device="cuda")
    return s


def prepare(case, seed):
    g = _gen(seed)
    make = _prepare_rope if case["op"] == "rope" else _prepare_pages if case["op"].startswith("pages") else _prepare_segment
    return dict(make(case, g), case=case, plan=None)


# ------------------------------------------------------------------ plain forms

def _plain_rope(c, s):
    a = s["positions"].double()[:, None] * s["inv_freq"][None]            # far positions: 64 bits
    cos, sin = (a.cos() * s["mscale"]).float()[:, None], (a.sin() * s["mscale"]).float()[:, None]
    if c["inverse"]:
        sin = -sin

    def turn(x):
        y, h, o = x.clone(), c["rot"] // 2, c["off"]
        if c["pairing"] == "half":
            i, j = slice(o, o + h), slice(o + h, o + 2 * h)
        else:
            i, j = slice(o, o + 2 * h, 2), slice(o + 1, o + 2 * h, 2)
        u, v = x[..., i].float(), x[..., j].float()
        y[..., i] = (u * cos - v * sin).to(x.dtype)
        y[..., j] = (v * cos + u * sin).to(x.dtype)
        return y

    return [turn(s["query"])] + ([turn(s["key"])] if s["key"] is not None else [])


def _free_first(ref):
    """Page numbers, the free ones first and in order."""
    return torch.argsort((ref != 0).to(torch.int8), stable=True)


def _copy_pages(pools, src, dst):
    return [p.index_copy_(0, dst.long(), p[src.long()]) for p in pools]


def _plain_fork(c, s):
    table, lens, ref, src, rows = s["table"], s["lens"], s["ref"], s["src"].long(), s["rows"].long()
    n, at = lens[src].long(), torch.arange(s["columns"], device="cuda")[None]
    full, part = n // c["page"], n % c["page"] != 0
    new = _free_first(ref)[(part.long().cumsum(0) - 1).clamp(min=0)]
    old = table[src].long().gather(1, full[:, None].clamp(max=s["columns"] - 1))[:, 0].clamp(min=0)
    shared = at < full[:, None]
    mine = torch.where(shared, table[src].long(), -1)
    mine = torch.where((at == full[:, None]) & part[:, None], new[:, None], mine)
    table_out, lens_out = table.clone(), lens.clone()
    table_out[rows], lens_out[rows] = mine.to(torch.int32), n.to(torch.int32)
    more = torch.zeros_like(ref).scatter_add_(0, mine.clamp(min=0).reshape(-1), (mine >= 0).to(torch.int32).reshape(-1))
    _copy_pages(s["pools"], old, torch.where(part, new, old))
    return [table_out, lens_out, ref + more, *s["pools"]]


def _plain_compact(c, s):
    ref, table = s["ref"], s["table"]
    live = ref != 0
    n, page = live.sum(), torch.arange(s["num_pages"], device="cuda")
    hole, mover = ~live & (page < n), live & (page >= n)
    to, frm = hole.nonzero()[:, 0], mover.nonzero()[:, 0]
    where = page.clone()
    where[frm] = to
    table_out = torch.where(table >= 0, where[table.clamp(min=0).long()], -1).to(torch.int32)
    ref_out = torch.zeros_like(ref).scatter_add_(0, where, ref)
    _copy_pages(s["pools"], frm, to)
    return [table_out, s["lens"].clone(), ref_out, *s["pools"]]


def _plain_turnover(c, s):
    table, lens, ref, rows = s["table"], s["lens"], s["ref"], s["rows"].long()
    out = table[rows].long()
    ref = ref - torch.zeros_like(ref).scatter_add_(0, out.clamp(min=0).reshape(-1), (out >= 0).to(torch.int32).reshape(-1))
    table, lens = table.clone(), lens.clone()
    table[rows], lens[rows] = -1, 0
    had, want = (lens.long() + c["page"] - 1) // c["page"], (s["after"].long() + c["page"] - 1) // c["page"]
    more = (want - had).clamp(min=0)
    at = torch.arange(s["columns"], device="cuda")[None]
    fresh = (at >= had[:, None]) & (at < want[:, None])
    rank = (more.cumsum(0) - more)[:, None] + at - had[:, None]
    got = _free_first(ref)[rank.clamp(0, s["num_pages"] - 1)]
    table = torch.where(fresh, got, table.long())
    ref = ref + torch.zeros_like(ref).scatter_add_(0, torch.where(fresh, got, 0).reshape(-1),
                                                   fresh.to(torch.int32).reshape(-1))
    return [table.to(torch.int32), torch.maximum(lens, s["after"]), ref]


def _rows_of(c, s):
    """Batch of each query row and the number of keys that it may see."""
    r = torch.arange(s["nrows"], device="cuda")
    if c["layout_q"] == "BSND":
        b, lens = r // s["S1"], s["act_q"].long()
        i = r - b * s["S1"]
        n = lens[b]
    else:
        b = torch.searchsorted(s["act_q"].long(), r, right=True)
        start = torch.cat([s["act_q"].new_zeros(1), s["act_q"]]).long()
        i, n = r - start[b], start[b + 1] - start[b]
    k = s["act_k"].long()
    if c["layout_kv"] == "TND":
        k = torch.diff(k, prepend=k.new_zeros(1))
    sees = k[b] if c["mode"] == 0 else torch.minimum((i + 1 + k[b] - n).clamp(min=0), k[b])
    return b, torch.where(i < n, sees, 0)


def _key_rows(c, s, b, pos):
    """Rows of the flattened keys that hold the positions `pos` of the sequences `b`."""
    if c["layout_kv"] == "BSND":
        return b * s["S2"] + pos
    if c["layout_kv"] == "TND":
        return torch.cat([s["act_k"].new_zeros(1), s["act_k"]]).long()[b] + pos
    return s["block_table"].long()[b, pos // c["page"]] * c["page"] + pos % c["page"]


def _plain_pool(c, s):
    k = s["act_k"].long()
    if c["layout_kv"] == "TND":
        k = torch.diff(k, prepend=k.new_zeros(1))
    first = (torch.zeros_like(k) if s["first"] is None else s["first"].long()) // c["seg"]
    some = s["max_segs"] if not c["new"] else min(s["max_segs"], _cdiv(c["new"], c["seg"]) + 1)
    seg = first[:, None] + torch.arange(some, device="cuda")[None]                     # [B, some]
    pos = seg[:, :, None] * c["seg"] + torch.arange(c["seg"], device="cuda")           # [B, some, seg]
    there = pos < k[:, None, None]
    b = torch.arange(c["B"], device="cuda")[:, None, None]
    x = s["key"].reshape(-1, c["n2"], c["d"])[_key_rows(c, s, b, torch.where(there, pos, 0))].float()
    x = torch.where(there[..., None, None], x, 0.0).sum(2) / there.sum(2).clamp(min=1)[..., None, None]
    # a segment behind the sequence stays as it was: it is written as the first one again
    ok = there[:, :, 0]
    x = torch.where(ok[..., None, None], x, x[:, :1])
    at = b[:, :, 0] * s["max_segs"] + torch.where(ok, seg, first[:, None])
    s["pooled"].view(-1, c["n2"], c["d"])[at.reshape(-1)] = x.reshape(-1, c["n2"], c["d"])
    return s["pooled"]


def _plain_select(c, s):
    b, sees = _rows_of(c, s)
    n2, d, m = c["n2"], c["d"], s["max_segs"]
    q = s["query"].reshape(s["nrows"], n2, -1, d).double().sum(2)                      # 64 bits: scores next to the border
    if c["layout_q"] == "BSND":
        q = q.view(c["B"], -1, n2, d).permute(0, 2, 1, 3)
        sc = (q @ s["pooled"].double().permute(0, 2, 3, 1)).permute(0, 2, 1, 3).reshape(s["nrows"], n2, m)
    else:
        sc = q.permute(1, 0, 2) @ s["pooled"].double().reshape(-1, n2, d).permute(1, 2, 0)
        sc = sc.view(n2, s["nrows"], c["B"], m).permute(1, 0, 2, 3)[torch.arange(s["nrows"], device="cuda"), :, b]
    at = torch.arange(m, device="cuda")
    ns = ((sees + c["seg"] - 1) // c["seg"])[:, None, None]
    sc = torch.where((at < c["init"]) | (at >= ns - c["local"]), 1e300, sc)
    sc = torch.where(at < ns, sc, -math.inf)
    if m < c["k"]:
        sc = torch.cat([sc, sc.new_full((s["nrows"], n2, c["k"] - m), -math.inf)], 2)
    v, i = sc.sort(dim=2, descending=True, stable=True)
    i = torch.where(v[..., :c["k"]] == -math.inf, 1 << 30, i[..., :c["k"]]).sort(dim=2)[0]
    return torch.where(i == 1 << 30, -1, i).to(torch.int32)


def _plain_attention(c, s):
    b, sees = _rows_of(c, s)
    n2, d = c["n2"], c["d"]
    pos = (s["seg_idx"].long()[..., None] * c["seg"] + torch.arange(c["seg"], device="cuda")).flatten(2)   # [rows, n2, L]
    ok = (s["seg_idx"].long() >= 0).repeat_interleave(c["seg"], 2) & (pos < sees[:, None, None])
    at = _key_rows(c, s, b[:, None, None], torch.where(ok, pos, 0))
    head = torch.arange(n2, device="cuda")[None, :, None]
    k, v = (s[x].reshape(-1, n2, d)[at, head].float() for x in ("key", "value"))
    q = s["query"].reshape(s["nrows"], n2, -1, d).float()
    l = (q @ k.transpose(2, 3)) * d ** -0.5
    l = torch.where(ok[:, :, None], l, -math.inf)
    top = l.max(3, keepdim=True)[0]
    e = torch.exp(l - torch.where(top == -math.inf, 0.0, top))
    z = e.sum(3, keepdim=True)
    out = (e @ v) / torch.where(z == 0, 1.0, z)
    lse = (top + z.log()).reshape(s["nrows"], -1)
    return [out.reshape(s["nrows"], c["n1"], d).to(s["query"].dtype), lse]


PLAIN = {"rope": _plain_rope, "pages_fork": _plain_fork, "pages_compact": _plain_compact, "pages_turnover": _plain_turnover,
         "segment_pool": _plain_pool, "segment_select": _plain_select, "segment_attention": _plain_attention}


# ------------------------------------------------------------------ the library's calls

def _own_plan(c, s):
    """What a program sets up once: the parameters of its calls and their workspace."""
    import sparse_attention_top_n1_b200 as li
    if c["op"] == "rope":
        return li, li.make_rope_params(dtype=c["dtype"], rows=c["rows"], N1=c["heads"], N2=c["key_heads"], D=c["d"],
                                       rot_dim=c["rot"], rot_offset=c["off"], pairing=c["pairing"], inverse=c["inverse"],
                                       mscale=s["mscale"]), None
    if c["op"].startswith("pages"):
        pr = li.make_pages_params(num_pages=s["num_pages"], page_size=c["page"], max_pages_per_seq=s["columns"],
                                  B=c["seqs"])
        return li, pr, li.alloc_pages_workspace(pr, "cuda")
    pr = li.make_segment_params(layout_q=c["layout_q"], layout_kv=c["layout_kv"], dtype=c["dtype"], B=c["B"], S1=s["S1"],
                                S2=s["S2"], T1=s["T1"], T2=s["T2"], N1=c["n1"], N2=c["n2"], D=c["d"],
                                num_blocks=s["num_blocks"], block_size=c["page"], max_blocks_per_seq=s["columns"],
                                seg_size=c["seg"], seg_count=c["k"], init_segs=c["init"], local_segs=c["local"],
                                max_segs=s["max_segs"], sparse_mode=c["mode"])
    return li, pr, None


def _own(c, s):
    if s["plan"] is None:
        s["plan"] = _own_plan(c, s)
    li, pr, ws = s["plan"]
    op = c["op"]
    if op == "rope":
        out, key_out = li.rope(pr, s["positions"], s["inv_freq"], s["query"], s["key"], out=s["out"], key_out=s["key_out"])
        return [out] + ([key_out] if key_out is not None else [])
    if op.startswith("pages"):
        out = (s["table_out"], s["lens_out"], s["ref_out"])
        held = s["table"], s["lens"], s["ref"]
        if op == "pages_fork":
            li.pages_fork(pr, s["pools"], *held, s["src"], s["rows"], out=out, workspace=ws)
            return [*out, *s["pools"]]
        if op == "pages_compact":
            li.pages_compact(pr, s["pools"], *held, out=out, workspace=ws)
            return [*out, *s["pools"]]
        li.pages_free(pr, *held, s["rows"], out=out, workspace=ws)
        li.pages_reserve(pr, *out, s["after"], out=out, workspace=ws)
        return list(out)
    if op == "segment_pool":
        return li.segment_pool(pr, s["key"], act_seq_k=s["act_k"], block_table=s["block_table"], first=s["first"],
                               pooled=s["pooled"])
    if op == "segment_select":
        return li.segment_select(pr, s["query"], s["pooled"], act_seq_q=s["act_q"], act_seq_k=s["act_k"],
                                 out=s["seg_idx"])
    return list(li.segment_attention(pr, s["query"], s["key"], s["value"], s["seg_idx"], act_seq_q=s["act_q"],
                                     act_seq_k=s["act_k"], block_table=s["block_table"], out=s["out"], lse=s["lse"]))


def run(state):
    return (_own if own else PLAIN[state["case"]["op"]])(state["case"], state)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    c = case
    if c["op"] == "rope":
        heads = c["heads"] + c["key_heads"]
        return {"bytes": 2 * c["rows"] * heads * c["d"] * BYTES[c["dtype"]] + 4 * c["rows"] + 4 * c["rot"],
                "flops": 3 * c["rows"] * heads * c["rot"]}
    if c["op"].startswith("pages"):
        lens, new, src, after, pages = _pages_geometry(c)
        columns = max(1, _cdiv(max(max(after), max(lens)), c["page"]))
        tables = 2 * 4 * (c["seqs"] * columns + c["seqs"] + pages)
        one = c["page"] * c["n2"] * c["d"] * 2 * c["pools"]
        if c["op"] == "pages_fork":
            return {"bytes": tables + 2 * one * sum(lens[r] % c["page"] != 0 for r in src), "flops": 0}
        if c["op"] == "pages_compact":
            # pages lie at random: of the gone ones, the share that lies below the new end is filled from above
            gone = sum(_cdiv(lens[r], c["page"]) for r in new) + 5
            return {"bytes": tables + 2 * one * gone * (pages - gone) // pages, "flops": 0}
        return {"bytes": tables, "flops": 0}
    q_lens, k_lens = _lens(c)
    es, n1, n2, d, g = BYTES[c["dtype"]], c["n1"], c["n2"], c["d"], c["seg"]
    if c["op"] == "segment_pool":
        read = wrote = 0
        for n in k_lens:
            first = max(0, n - c["new"]) // g if c["new"] else 0
            read += n - first * g
            wrote += _cdiv(n, g) - first
        return {"bytes": n2 * d * (read * es + wrote * 4), "flops": read * n2 * d}
    rows = sum(q_lens) if c["layout_q"] == "TND" else c["B"] * max(q_lens)
    pairs = keys = segs = scored = 0
    for q, k in zip(q_lens, k_lens):
        mine = 0
        for i in range(q):
            sees = k if c["mode"] == 0 else i + 1 + k - q
            ns = _cdiv(sees, g)
            mine += sees if ns <= c["k"] else c["k"] * g - (ns * g - sees)
            scored += ns if ns > c["k"] else 0
        pairs += mine
        keys += min(k, mine)
        segs += _cdiv(k, g)
    if c["op"] == "segment_select":
        return {"bytes": rows * n1 * d * es + segs * n2 * d * 4 + rows * n2 * c["k"] * 4,
                "flops": 2 * scored * n2 * d + rows * n1 * d}
    return {"bytes": rows * n1 * (2 * d * es + 4) + keys * n2 * 2 * d * es + rows * n2 * c["k"] * 4,
            "flops": 4 * pairs * n1 * d}


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    c = case
    if c["op"].startswith("pages") or c["op"] == "segment_select":
        return None                                    # whole numbers and copies
    s = prepare(c, seed)
    if c["op"] == "rope":
        found = []
        w = torch.polar(torch.full_like(s["inv_freq"], s["mscale"]).expand(c["rows"], -1),
                        s["positions"].double()[:, None] * s["inv_freq"] * (-1 if c["inverse"] else 1))
        for x in (s["query"], s["key"]):
            if x is None:
                continue
            y = x.double()
            part = y[..., c["off"]:c["off"] + c["rot"]]
            if c["pairing"] == "half":
                z = torch.complex(*part.reshape(*part.shape[:2], 2, -1).unbind(2))
            else:
                z = torch.view_as_complex(part.reshape(*part.shape[:2], -1, 2).contiguous())
            z = torch.view_as_real(z * w[:, None])
            turned = z.transpose(2, 3) if c["pairing"] == "half" else z
            found.append(torch.cat([y[..., :c["off"]], turned.reshape(part.shape), y[..., c["off"] + c["rot"]:]], -1))
        return found
    q_lens, k_lens = _lens(c)
    k0, q0 = 0, 0

    def keys_of(x, b, k0):
        x = x.double()
        if c["layout_kv"] == "BSND":
            return x[b, :k_lens[b]]
        if c["layout_kv"] == "TND":
            return x[k0:k0 + k_lens[b]]
        return x[s["block_table"][b, :_cdiv(k_lens[b], c["page"])].long()].flatten(0, 1)[:k_lens[b]]

    if c["op"] == "segment_pool":
        out = s["pooled"].double()
        for b in range(c["B"]):
            n, g = _cdiv(k_lens[b], c["seg"]), c["seg"]
            first = max(0, k_lens[b] - c["new"]) // g if c["new"] else 0
            x = keys_of(s["key"], b, k0)[first * g:]
            sums = torch.zeros(((n - first) * g, *x.shape[1:]), dtype=torch.float64, device="cuda")
            sums[:len(x)] = x
            counts = torch.full((n - first, 1, 1), float(g), dtype=torch.float64, device="cuda")
            counts[-1] = k_lens[b] - (n - 1) * g
            out[b, first:n] = sums.view(n - first, g, *x.shape[1:]).sum(1) / counts
            k0 += k_lens[b]
        return out
    n2, g, d = c["n2"], c["n1"] // c["n2"], c["d"]
    out = torch.zeros((s["nrows"], c["n1"], d), dtype=torch.float64, device="cuda")
    lse = torch.full((s["nrows"], c["n1"]), -math.inf, dtype=torch.float64, device="cuda")
    query = s["query"].reshape(s["nrows"], c["n1"], d)
    for b in range(c["B"]):
        first = b * s["S1"] if c["layout_q"] == "BSND" else q0
        k, v = keys_of(s["key"], b, k0), keys_of(s["value"], b, k0)
        at = torch.arange(k_lens[b], device="cuda")
        for lo in range(0, q_lens[b], 512):
            r = torch.arange(lo, min(lo + 512, q_lens[b]), device="cuda")
            sees = k_lens[b] if c["mode"] == 0 else r[:, None] + 1 + k_lens[b] - q_lens[b]
            for n in range(n2):
                chosen = torch.zeros((len(r), s["max_segs"] + 1), dtype=torch.bool, device="cuda")
                chosen.scatter_(1, s["seg_idx"][first + r, n].long() % (s["max_segs"] + 1), True)
                ok = chosen[:, at // c["seg"]] & (at[None] < sees)
                heads = slice(n * g, (n + 1) * g)
                l = torch.matmul(query[first + r, heads].double(), k[:, n].T) * d ** -0.5
                l = l.masked_fill(~ok[:, None], -math.inf)
                lse[first + r, heads] = torch.logsumexp(l, 2)
                out[first + r, heads] = torch.nan_to_num(torch.softmax(l, 2), nan=0.0) @ v[:, n]
        q0 += q_lens[b]
        k0 += k_lens[b]
    return [out, lse]
