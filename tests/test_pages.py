"""The pages of a cache: refusals on the host, every call against a plain model on the GPU."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest
import torch

import oracle.cache as oc
import sparse_attention_top_n1_b200 as li

FAKE = 1 << 20


# ------------------------------------------------------------------ the model itself

def test_model_on_a_small_case_by_hand():
    m = oc.Pages([[2, 0, -1], [-1] * 3], [5, 0], [1, 0, 1, 0, 0], 4, [np.arange(5)])
    m.fork([0], [1])
    assert m.table == [[2, 0, -1], [2, 1, -1]] and m.lens == [5, 5] and m.refs == [1, 1, 2, 0, 0]
    assert m.pools[0].tolist() == [0, 0, 2, 3, 4] and m.flags == 0
    m.free([0])
    assert m.refs == [0, 1, 1, 0, 0] and m.table[0] == [-1, -1, -1]
    m.compact()
    assert m.table[1] == [0, 1, -1] and m.refs == [1, 1, 0, 0, 0] and m.pools[0].tolist() == [2, 0, 2, 3, 4]
    m.reserve([9, 5])
    assert m.table[0] == [2, 3, 4] and m.lens == [9, 5]
    m.free([1, 1, 7])
    assert m.flags == m.BAD_ROW


# ------------------------------------------------------------------ host

def _pr(**kw):
    return li.make_pages_params(**dict(dict(num_pages=64, page_size=16, max_pages_per_seq=8, B=4), **kw))


def _call(name, pr, pools=None, n_pools=0, n=1, ws=FAKE, wsb=1 << 30, table=FAKE, arg=FAKE, out=FAKE):
    L, p = li.lib(), ctypes.byref(pr)
    st = {"reserve": lambda: L.li_pages_reserve(p, table, FAKE, FAKE, arg, out, FAKE, FAKE, None, ws, wsb, None),
          "fork": lambda: L.li_pages_fork(p, pools, n_pools, table, FAKE, FAKE, arg, arg, n, out, FAKE, FAKE, None, ws, wsb, None),
          "free": lambda: L.li_pages_free(p, table, FAKE, FAKE, arg, n, out, FAKE, FAKE, None, ws, wsb, None),
          "compact": lambda: L.li_pages_compact(p, pools, n_pools, table, FAKE, FAKE, out, FAKE, FAKE, None, ws, wsb, None),
          }[name]()
    assert li.li_last_launch_count() == 0
    return li.STATUS_NAMES[st]


@pytest.mark.parametrize("name", ["reserve", "fork", "free", "compact"])
@pytest.mark.parametrize("kw", [dict(num_pages=0), dict(num_pages=(1 << 26) + 1), dict(page_size=0), dict(B=0),
                                dict(max_pages_per_seq=0), dict(max_pages_per_seq=1 << 28), dict(B=1 << 29),
                                dict(reserved=1)])
def test_pages_refuse_shapes(name, kw):
    assert _call(name, _pr(**kw)) == "LI_ERR_SHAPE"


@pytest.mark.parametrize("name", ["reserve", "fork", "free", "compact"])
def test_pages_refuse_pointers(name):
    assert _call(name, _pr(), table=None) == "LI_ERR_NULL"
    assert _call(name, _pr(), out=None) == "LI_ERR_NULL"
    assert _call(name, _pr(), table=FAKE + 2) == "LI_ERR_SHAPE"
    assert _call(name, _pr(), ws=None) == "LI_ERR_WORKSPACE"
    assert _call(name, _pr(), ws=FAKE + 128) == "LI_ERR_WORKSPACE"
    assert _call(name, _pr(), wsb=li.li_pages_workspace_size(_pr()) - 1) == "LI_ERR_WORKSPACE"
    if name != "compact":
        assert _call(name, _pr(), arg=None) == "LI_ERR_NULL"
    if name in ("fork", "free"):
        assert _call(name, _pr(), n=-1) == "LI_ERR_SHAPE"


@pytest.mark.parametrize("name", ["fork", "compact"])
def test_pages_refuse_pools(name):
    def pool(base=FAKE, nbytes=64, stride=64):
        return (li.PagePool * 1)(li.PagePool(base, nbytes, stride))
    assert _call(name, _pr(), pool(base=None), 1) == "LI_ERR_NULL"
    assert _call(name, _pr(), pool(nbytes=0), 1) == "LI_ERR_SHAPE"
    assert _call(name, _pr(), pool(stride=63), 1) == "LI_ERR_SHAPE"
    assert _call(name, _pr(), None, 1) == "LI_ERR_NULL"
    assert _call(name, _pr(), pool(), -1) == "LI_ERR_SHAPE"
    assert _call(name, _pr(), pool(), 257) == "LI_ERR_SHAPE"


def test_pages_copy_refuses():
    L, pr = li.lib(), _pr()
    pool = (li.PagePool * 1)(li.PagePool(FAKE, 64, 64))
    call = lambda s=FAKE, d=FAKE, n=1, st=None: li.STATUS_NAMES[  # noqa: E731
        L.li_pages_copy(ctypes.byref(pr), pool, 1, s, d, n, st, None)]
    assert call(s=None) == "LI_ERR_NULL" and call(d=None) == "LI_ERR_NULL"
    assert call(n=-1) == "LI_ERR_SHAPE" and call(d=FAKE + 1) == "LI_ERR_SHAPE" and call(st=FAKE + 2) == "LI_ERR_SHAPE"
    assert call(n=0) == "LI_OK" and li.li_last_launch_count() == 0


def test_wrapper_refuses_wrong_state():
    pr = _pr()
    t, n, r = (torch.zeros(s, dtype=torch.int32) for s in ((4, 8), (4,), (64,)))
    ws = torch.empty(li.li_pages_workspace_size(pr), dtype=torch.uint8)
    with pytest.raises(ValueError):
        li.pages_reserve(pr, t[:, :7], n, r, n, workspace=ws)
    with pytest.raises(TypeError):
        li.pages_reserve(pr, t, n.long(), r, n, workspace=ws)
    with pytest.raises(ValueError):
        li.pages_free(pr, t, n, r[:63], n, workspace=ws)
    with pytest.raises(ValueError):
        li.pages_fork(pr, [torch.zeros(63, 16)], t, n, r, n, n, workspace=ws)
    with pytest.raises(ValueError):
        li.page_pools([torch.zeros(64, 16, 4).transpose(1, 2)])


def test_wrapper_refuses_a_workspace_with_gaps():
    """Its size counts elements; the calls write that many bytes in a row."""
    pr = _pr()
    t, n, r = (torch.zeros(s, dtype=torch.int32) for s in ((4, 8), (4,), (64,)))
    ws = torch.empty(2 * li.li_pages_workspace_size(pr), dtype=torch.uint8)
    with pytest.raises(ValueError, match="workspace must be contiguous"):
        li.pages_reserve(pr, t, n, r, n, workspace=ws[::2])
    with pytest.raises(ValueError, match="CUDA device"):
        li.pages_reserve(pr, t, n, r, n, workspace=ws[:len(ws) // 2])


@pytest.mark.parametrize("stride", [0, 1, 8, 63])
def test_pools_of_overlapping_pages_are_refused(stride):
    """Their stride is not that of pages side by side: page n - 1 would be looked
    for behind the tensor."""
    t = torch.zeros(6 * 64, dtype=torch.int16)
    with pytest.raises(ValueError, match="overlap"):
        li.page_pools([t.as_strided((6, 16, 4), (stride, 4, 1))])
    if stride == 0:
        with pytest.raises(ValueError, match="overlap"):
            li.page_pools([t[:64].expand(6, 64)])


def test_descriptors_of_pools():
    t = torch.zeros(6, 3, 64, dtype=torch.int16)
    for pool, want in ((t, (384, 384)), (t[:, 1], (128, 384)), (t[:1, 1], (128, 128)), (t[::2], (384, 768)),
                       (t.view(-1)[:64].expand(1, 64), (128, 128)), (t.view(-1).as_strided((1, 64), (5, 1)), (128, 128))):
        d = li.page_pools([pool])[0]
        assert d.base == pool.data_ptr() and (d.page_bytes, d.page_stride) == want


# ------------------------------------------------------------------ GPU

def _state(g, B, cols, ps, P, fill=0.5, shared=0.0):
    """A random valid state: rows of random lengths over a random choice of pages."""
    rng = np.random.default_rng(g)
    free = list(rng.permutation(P))
    table = np.full((B, cols), -1, np.int32)
    lens, refs = np.zeros(B, np.int32), np.zeros(P, np.int32)
    for b in range(B):
        n = int(rng.integers(0, int(cols * ps * fill) + 1)) if rng.random() < 0.8 else 0
        k = -(-n // ps)
        if k > len(free):
            continue
        row = [free.pop() for _ in range(k)]
        if b and shared and rng.random() < shared:                # a prefix of the row before it
            m = min(k, int(lens[b - 1]) // ps)
            free.extend(row[:m])
            row[:m] = [int(p) for p in table[b - 1, :m]]
        table[b, :k], lens[b] = row, n
        np.add.at(refs, row, 1)
    return table, lens, refs


def _pools(g, P, shapes):
    gen = torch.Generator().manual_seed(g)
    return [torch.randint(-100, 100, (P, *s), generator=gen, dtype=t) for s, t in shapes]


SHAPES = [((16, 2, 8), torch.int16), ((5,), torch.int8), ((3, 7), torch.int32), ((40000,), torch.int8)]


def _check(model, got, pools, status):
    table, lens, refs = (t.cpu().numpy() for t in got)
    assert np.array_equal(table, np.array(model.table, np.int32))
    assert np.array_equal(lens, np.array(model.lens, np.int32))
    assert np.array_equal(refs, np.array(model.refs, np.int32))
    for a, b in zip(pools, model.pools):
        assert np.array_equal(a.cpu().numpy(), b)
    assert int(status.item()) == model.flags, hex(int(status.item()))


SIZES = [  # seed, B, cols, page size, pages
    (0, 4, 5, 16, 32), (1, 1, 1, 1, 1), (2, 37, 9, 48, 300), (3, 130, 33, 64, 5000), (4, 3, 700, 16, 40000), (5, 2000, 3, 128, 3500), (6, 700, 400, 1, 9000),
]


@pytest.mark.gpu
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("op", ["reserve", "fork", "free", "compact"])
@pytest.mark.parametrize("seed,B,cols,ps,P", SIZES)
def test_pages_match_the_model(op, seed, B, cols, ps, P, in_place):
    table, lens, refs = _state(seed, B, cols, ps, P, shared=0.5 if op != "fork" else 0.2)
    shapes = SHAPES if P < 10000 else SHAPES[:2]
    host = _pools(seed, P, shapes)
    model = oc.Pages(table, lens, refs, ps, [p.numpy() for p in host])
    d = [torch.from_numpy(t).cuda() for t in (table, lens, refs)]
    pools = [p.cuda() for p in host]
    pr = li.make_pages_params(num_pages=P, page_size=ps, max_pages_per_seq=cols, B=B)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = tuple(d) if in_place else None
    rng = np.random.default_rng(100 + seed)
    i32 = lambda v: torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")  # noqa: E731
    if op == "reserve":
        new = np.minimum(lens + rng.integers(-3 * ps, 4 * ps, B), cols * ps).clip(0)
        model.reserve(new)
        got = li.pages_reserve(pr, *d, i32(new), out=out, status=status)
    elif op == "fork":
        empty = np.flatnonzero(lens == 0)
        src, dst = rng.integers(0, B, len(empty)), rng.permutation(empty)
        model.fork(src, dst)
        got = li.pages_fork(pr, pools, *d, i32(src), i32(dst), out=out, status=status)
    elif op == "free":
        rows = rng.permutation(B)[:max(1, B // 2)]
        model.free(rows)
        got = li.pages_free(pr, *d, i32(rows), out=out, status=status)
    else:
        model.compact()
        got = li.pages_compact(pr, pools, *d, out=out, status=status)
    assert li.li_last_launch_count() == 2
    _check(model, got, pools, status)
    if in_place:
        assert all(a is b for a, b in zip(got, d))
    else:
        assert all(np.array_equal(a.cpu().numpy(), b) for a, b in zip(d, (table, lens, refs)))


@pytest.mark.gpu
def test_fork_of_whole_pages_beside_open_ones():
    """Children of a row that ends with its last page copy nothing; the free pages,
    page 0 among them, go to the others in order."""
    ps, cols, P, B = 4, 5, 12, 9
    table = np.full((B, cols), -1, np.int32)
    table[0, :3], table[1, :2], table[2, :5] = [7, 3, 9], [5, 2], [11, 10, 8, 6, 4]
    lens = np.array([9, 8, 17, 0, 0, 0, 0, 0, 0], np.int32)      # open, whole, open
    refs = np.zeros(P, np.int32)
    refs[[7, 3, 9, 5, 2, 11, 10, 8, 6, 4]] = 1
    host = _pools(3, P, SHAPES)
    model = oc.Pages(table, lens, refs, ps, [p.numpy() for p in host])
    src, dst = [1, 0, 1, 2, 1], [4, 3, 8, 5, 6]
    model.fork(src, dst)
    assert model.flags == 0 and model.table[3][2] == 0 and model.table[5][4] == 1
    d = [torch.from_numpy(t).cuda() for t in (table, lens, refs)]
    pools = [p.cuda() for p in host]
    pr = li.make_pages_params(num_pages=P, page_size=ps, max_pages_per_seq=cols, B=B)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    got = li.pages_fork(pr, pools, *d, i32(src), i32(dst), status=status)
    _check(model, got, pools, status)


@pytest.mark.gpu
def test_pages_run_out_in_order():
    """Rows are served in order until the pages run out; the rest stay as they were."""
    table = np.full((5, 4), -1, np.int32)
    refs = np.zeros(6, np.int32)
    pr = li.make_pages_params(num_pages=6, page_size=8, max_pages_per_seq=4, B=5)
    model = oc.Pages(table, [0] * 5, refs, 8)
    new = [9, 32, 1, 0, 1]                                        # 2, 4, 1, 0, 1 pages
    model.reserve(new)
    d = [torch.tensor(v, dtype=torch.int32, device="cuda") for v in (table, [0] * 5, refs)]
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = li.pages_reserve(pr, *d, torch.tensor(new, dtype=torch.int32, device="cuda"), status=st)
    _check(model, got, [], st)
    assert int(st.item()) == li.DEV_NO_PAGES and got[1].tolist() == [9, 32, 0, 0, 0]
    st.zero_()
    kids = li.pages_fork(pr, [], *got, *(torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([0, 1], [2, 3])), status=st)
    model.flags = 0
    model.fork([0, 1], [2, 3])                                    # the open page has no place, the full ones are shared
    _check(model, kids, [], st)
    assert int(st.item()) == li.DEV_NO_PAGES and kids[1].tolist() == [9, 32, 0, 32, 0]


@pytest.mark.gpu
@pytest.mark.parametrize("in_place", [False, True])
def test_rows_that_need_no_page_are_served_when_pages_have_run_out(in_place):
    """Behind the first row that no longer fits: a row that grows inside its last
    page and a child of whole pages are served, a row that would fit is not."""
    ps, P = 8, 7
    table = np.array([[0, -1, -1, -1], [1, 2, -1, -1], [3, -1, -1, -1], [4, -1, -1, -1], [-1] * 4, [-1] * 4, [-1] * 4], np.int32)
    lens, refs = np.array([8, 16, 3, 8, 0, 0, 0], np.int32), np.array([1, 1, 1, 1, 1, 0, 0], np.int32)
    pr = li.make_pages_params(num_pages=P, page_size=ps, max_pages_per_seq=4, B=7)
    i32 = lambda v: torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")  # noqa: E731
    for op, a0, a1, want in (("reserve", [9, 32, 7, 9, 0, 1, 0], None, [9, 16, 7, 8, 0, 0, 0]),
                             ("fork", [2, 2, 2, 1], [4, 5, 6, 3], None), ("fork", [1, 2, 0], [4, 5, 6], [8, 16, 3, 8, 16, 3, 8])):
        model = oc.Pages(table, lens, refs, ps)
        d, st = [i32(t) for t in (table, lens, refs)], torch.zeros(1, dtype=torch.int32, device="cuda")
        out = tuple(d) if in_place else None
        if op == "reserve":
            model.reserve(a0)
            got = li.pages_reserve(pr, *d, i32(a0), out=out, status=st)
        else:
            model.fork(a0, a1)
            got = li.pages_fork(pr, [], *d, i32(a0), i32(a1), out=out, status=st)
        _check(model, got, [], st)
        assert want is None or got[1].tolist() == want


@pytest.mark.gpu
@pytest.mark.parametrize("in_place", [False, True])
def test_pages_bad_arguments_are_skipped_and_flagged(in_place):
    ps, P = 4, 12
    table = np.array([[1, 3, 99], [5, -1, -1], [-1] * 3, [-1] * 3, [7, 2, -1]], np.int32)
    lens, refs = np.array([11, 3, 0, 0, 99], np.int32), np.zeros(P, np.int32)
    refs[[1, 3, 5, 7]] = 1                                       # page 2 of the last row is not counted
    pr = li.make_pages_params(num_pages=P, page_size=ps, max_pages_per_seq=3, B=5)
    for op, a0, a1 in (("fork", [0, 9, 1, 1, 0, 2], [2, 3, 1, 2, -4, 3]), ("free", [4, 4, -1, 5, 0], None),
                       ("reserve", [3, 13, -1, 12, 0], None), ("compact", None, None)):
        model = oc.Pages(table, lens, refs, ps)
        d = [torch.from_numpy(t.copy()).cuda() for t in (table, lens, refs)]
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = tuple(d) if in_place else None
        args = [torch.tensor(v, dtype=torch.int32, device="cuda") for v in (a0, a1) if v is not None]
        if op == "fork":
            model.fork(a0, a1)
            got = li.pages_fork(pr, [], *d, *args, out=out, status=st)
        elif op == "free":
            model.free(a0)
            got = li.pages_free(pr, *d, *args, out=out, status=st)
        elif op == "reserve":
            model.reserve(a0)
            got = li.pages_reserve(pr, *d, *args, out=out, status=st)
        else:
            # entries that name a page nobody holds are dropped
            got = li.pages_compact(pr, [], *d, out=out, status=st)
            assert got[0].tolist() == [[1, 3, -1], [0, -1, -1], [-1] * 3, [-1] * 3, [2, -1, -1]]
            assert got[2].tolist() == [1, 1, 1, 1] + [0] * 8 and got[1].tolist() == [11, 3, 0, 0, 12]
            assert int(st.item()) == li.DEV_BAD_BLOCK | li.DEV_BAD_KLEN
            continue
        _check(model, got, [], st)


@pytest.mark.gpu
def test_pages_copy_strided_pools_and_many_of_them():
    P, n = 50, 12
    g = torch.Generator().manual_seed(9)
    wide = torch.randint(-99, 99, (P, 3, 64), generator=g, dtype=torch.int16).cuda()       # key, value, spare interleaved
    pools = [wide[:, 0], wide[:, 1]] + [torch.randint(-9, 9, (P, 33), generator=g, dtype=torch.int8).cuda() for _ in range(128)]
    before = [p.clone() for p in pools]
    perm = torch.randperm(P, generator=g).to(torch.int32)
    src, dst = perm[:n].clone(), perm[n:2 * n].clone()
    src[3], dst[4] = -1, P                                       # skipped
    src[5] = dst[5] = perm[2 * n]                                # onto itself: nothing
    spare = wide[:, 2].clone()
    pr = li.make_pages_params(num_pages=P, page_size=64, max_pages_per_seq=1, B=1)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    li.pages_copy(pr, pools, src.cuda(), dst.cuda(), status=st)
    assert li.li_last_launch_count() == 3 and int(st.item()) == li.DEV_BAD_BLOCK
    for p, b in zip(pools, before):
        want = b.clone()
        for i in range(n):
            if i not in (3, 4):
                want[dst[i]] = b[src[i]]
        assert torch.equal(p, want)
    assert torch.equal(wide[:, 2], spare)


@pytest.mark.gpu
def test_pages_life_of_a_cache_in_a_graph():
    """Rows grow, fork, end and are packed, in place; each step captured once and
    replayed, and the model does the same steps."""
    B, cols, ps, P = 12, 20, 16, 150
    pr = li.make_pages_params(num_pages=P, page_size=ps, max_pages_per_seq=cols, B=B)
    host = _pools(1, P, SHAPES[:2])
    model = oc.Pages(np.full((B, cols), -1), [0] * B, [0] * P, ps, [p.numpy() for p in host])
    pools = [p.cuda() for p in host]
    d = tuple(torch.tensor(v, dtype=torch.int32, device="cuda") for v in (model.table, model.lens, model.refs))
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = li.alloc_pages_workspace(pr)
    new = torch.zeros(B, dtype=torch.int32, device="cuda")
    src, dst, rows = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (3, 3, 4))
    arr = li.page_pools(pools)
    graphs = {}
    for name, f in (("reserve", lambda: li.pages_reserve(pr, *d, new, out=d, workspace=ws, status=st)),
                    ("fork", lambda: li.pages_fork(pr, arr, *d, src, dst, out=d, workspace=ws, status=st)),
                    ("free", lambda: li.pages_free(pr, *d, rows, out=d, workspace=ws, status=st)),
                    ("compact", lambda: li.pages_compact(pr, arr, *d, out=d, workspace=ws, status=st))):
        graphs[name] = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graphs[name]):
            f()
    rng = np.random.default_rng(7)
    for step in range(25):
        want = [n + int(rng.integers(0, 60)) if rng.random() < 0.6 else n for n in model.lens]
        new.copy_(torch.tensor(want, dtype=torch.int32))
        graphs["reserve"].replay()
        model.reserve(want)
        s, t = rng.integers(0, B, 3), rng.integers(0, B, 3)
        src.copy_(torch.from_numpy(s.astype(np.int32)))
        dst.copy_(torch.from_numpy(t.astype(np.int32)))
        graphs["fork"].replay()
        model.fork(s, t)
        r = rng.integers(0, B, 4)
        rows.copy_(torch.from_numpy(r.astype(np.int32)))
        graphs["free"].replay()
        model.free(r)
        if step % 3 == 2:
            graphs["compact"].replay()
            model.compact()
        _check(model, d, pools, st)
    held = [p for row, n in zip(model.table, model.lens) for p in row[:-(-n // ps)]]
    assert np.array_equal(np.bincount(held, minlength=P), model.refs)      # every count is its rows' number
