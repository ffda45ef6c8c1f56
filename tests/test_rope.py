"""Rotary positions: frequencies and refusals on the host, rotations on the GPU.

Tolerance of a rotation: the angle reaches fp32 as f = t - rint(t) in turns,
|f| <= 1/2, rounded by at most 2^-26 turns, so cos and sin are off by at most
2 pi 2^-26 < 2^-23 plus 2 ulp (2^-23) of sincospi, and the mscale factor one
more rounding: 2^-21 covers each factor.  The two products and their sum round
by at most 3 * 2^-24 of |x0| + |x1|, and the result is rounded once to the
output type (half a step: finfo.eps / 2).
"""
from __future__ import annotations

import ctypes
import math
import os
import subprocess

import numpy as np
import pytest
import torch

import oracle.cache as oc
import sparse_attention_top_n1_b200 as li

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 20
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------ host

def test_frequencies_follow_the_formulas():
    p = np.arange(32)
    f, m = li.rope_frequencies(64, 10000.0)
    assert m == 1.0 and np.allclose(f.numpy(), 10000.0 ** (-2 * p / 64), rtol=1e-15)
    f, m = li.rope_frequencies(64, 500000.0, "linear", 4.0)
    assert m == 1.0 and np.allclose(f.numpy(), 500000.0 ** (-2 * p / 64) / 4, rtol=1e-15)
    f, m = li.rope_frequencies(64, 10000.0, "ntk", 8.0)
    assert m == 1.0 and np.allclose(f.numpy(), (10000.0 * 8 ** (64 / 62)) ** (-2 * p / 64), rtol=1e-14)
    f, m = li.rope_frequencies(64, 10000.0, "yarn", 16.0, 4096)
    plain = 10000.0 ** (-2 * p / 64)
    turns = 4096 * plain / (2 * math.pi)                       # within the original positions
    assert np.allclose(f.numpy()[turns > 34], plain[turns > 34], rtol=1e-15)
    assert np.allclose(f.numpy()[turns < 0.7], plain[turns < 0.7] / 16, rtol=1e-15)
    assert np.all(np.diff(f.numpy()) < 0) and np.all(f.numpy() >= plain / 16 * (1 - 1e-15))
    assert abs(m - (0.1 * math.log(16) + 1)) < 1e-6


@pytest.mark.parametrize("rot,positions,fast,slow,base", [
    (64, 4, 32.0, 1.0, 1e4), (2, 6, 32.0, 1.0, 1e4), (64, 1, 0.5, 0.2, 1e4), (64, 100, 40.0, 16.0, 1e4), (128, 7, 32.0, 1.0, 1e4),
    (64, 1 << 20, 32.0, 1.0, 1e4), (4, 2 ** 31 - 1, 32.0, 1.0, 1e4), (2, 1 << 20, 32.0, 1.0, 2.0), (64, 4096, 32.0, 1.0, 2.0),
    (64, 4096, 32.0, 1.0, 10.0)])
def test_yarn_keeps_and_divides_by_the_number_of_turns(rot, positions, fast, slow, base):
    """Pairs that turn beta_fast times and more are kept, those that turn beta_slow
    times and less are divided, the first one among them where positions are few."""
    f = li.rope_frequencies(rot, base, "yarn", 8.0, positions, fast, slow)[0].numpy()
    plain = base ** (-2 * np.arange(rot // 2) / rot)
    turns = positions * plain / (2 * math.pi)
    assert np.allclose(f[turns >= fast], plain[turns >= fast], rtol=1e-15)
    assert np.allclose(f[turns <= slow], plain[turns <= slow] / 8, rtol=1e-15)
    assert np.all(f >= plain / 8 * (1 - 1e-15)) and np.all(f <= plain * (1 + 1e-15))


def test_frequencies_of_one_pair_and_factor_one():
    for s in ("none", "linear"):
        f, m = li.rope_frequencies(2, 10000.0, s, 3.0)
        assert f.tolist() == [1.0 if s == "none" else 1.0 / 3.0]
    assert np.allclose(li.rope_frequencies(64, 1e4, "yarn", 1.0, 4096)[0], li.rope_frequencies(64, 1e4)[0], rtol=1e-15)


@pytest.mark.parametrize("kw,err", [
    (dict(rot_dim=3), "LI_ERR_SHAPE"), (dict(rot_dim=0), "LI_ERR_SHAPE"), (dict(base=1.0), "LI_ERR_SHAPE"),
    (dict(base=float("nan")), "LI_ERR_SHAPE"), (dict(scaling="linear", factor=0.5), "LI_ERR_SHAPE"),
    (dict(scaling="yarn", factor=2.0), "LI_ERR_SHAPE"), (dict(scaling="ntk", factor=2.0, rot_dim=2), "LI_ERR_SHAPE"),
    (dict(scaling="yarn", factor=2.0, original_positions=4096, beta_fast=1.0, beta_slow=2.0), "LI_ERR_SHAPE"),
])
def test_frequencies_refuse(kw, err):
    with pytest.raises(li.LiError, match=err):
        li.rope_frequencies(**dict(dict(rot_dim=64), **kw))


def _pr(**kw):
    return li.make_rope_params(**dict(dict(dtype="bf16", rows=8, N1=4, N2=0, D=128, rot_dim=64, rot_offset=0,
                                           pairing="half", inverse=0), **kw))


BAD = [
    (dict(dtype="e4m3"), "LI_ERR_DTYPE"), (dict(pairing=2), "LI_ERR_LAYOUT"), (dict(inverse=2), "LI_ERR_SHAPE"),
    (dict(rows=-1), "LI_ERR_SHAPE"), (dict(N1=0), "LI_ERR_SHAPE"), (dict(N1=1025), "LI_ERR_SHAPE"),
    (dict(D=1025), "LI_ERR_SHAPE"), (dict(rot_dim=63), "LI_ERR_SHAPE"), (dict(rot_dim=0), "LI_ERR_SHAPE"),
    (dict(rot_dim=130), "LI_ERR_SHAPE"), (dict(rot_offset=65), "LI_ERR_SHAPE"), (dict(rot_offset=-1), "LI_ERR_SHAPE"),
    (dict(mscale=0.0), "LI_ERR_SHAPE"), (dict(mscale=float("nan")), "LI_ERR_SHAPE"), (dict(reserved=1), "LI_ERR_SHAPE"),
    (dict(q_row_stride=511), "LI_ERR_SHAPE"), (dict(q_head_stride=127), "LI_ERR_SHAPE"),
    (dict(q_out_row_stride=-512), "LI_ERR_SHAPE"), (dict(N2=1), "LI_ERR_NULL"),
]


@pytest.mark.parametrize("kw,err", BAD)
def test_rope_refuses_before_launch(kw, err):
    st = li.lib().li_rope(ctypes.byref(_pr(**kw)), FAKE, FAKE, FAKE, None, FAKE + 65536, None, None)
    assert li.STATUS_NAMES[st] == err, li.li_last_error()
    assert li.li_last_launch_count() == 0


def test_rope_pointer_checks():
    def call(pr, pos=FAKE, f=FAKE, q=FAKE, k=None, qo=FAKE + 65536, ko=None):
        return li.STATUS_NAMES[li.lib().li_rope(ctypes.byref(pr), pos, f, q, k, qo, ko, None)]
    assert call(_pr(), pos=None) == "LI_ERR_NULL"
    assert call(_pr(), f=None) == "LI_ERR_NULL"
    assert call(_pr(), q=None) == "LI_ERR_NULL"
    assert call(_pr(), qo=None) == "LI_ERR_NULL"
    assert call(_pr(), k=FAKE) == "LI_ERR_NULL"                # a key with N2 = 0
    assert call(_pr(), q=FAKE + 1) == "LI_ERR_SHAPE"
    assert call(_pr(), f=FAKE + 4) == "LI_ERR_SHAPE"
    assert call(_pr(q_out_row_stride=1024), qo=FAKE) == "LI_ERR_SHAPE"   # in place with other strides
    assert call(_pr(rows=0)) == "LI_OK" and li.li_last_launch_count() == 0


@pytest.mark.parametrize("struct,name", [(li.RopeParams, "li_rope_params"), (li.PagesParams, "li_pages_params"),
                                         (li.PagePool, "li_page_pool"), (li.SegmentParams, "li_segment_params")])
def test_struct_mirrors_match_the_header(tmp_path, struct, name):
    fields = [f for f, _ in struct._fields_]
    src = tmp_path / "probe.c"
    src.write_text("#include <stdio.h>\n#include <stddef.h>\n#include \"li.h\"\nint main(void) {\n"
                   '  printf("%%zu\\n", sizeof(%s));\n' % name +
                   "".join('  printf("%%zu\\n", offsetof(%s, %s));\n' % (name, f) for f in fields) + "  return 0;\n}\n")
    exe = tmp_path / "probe"
    subprocess.check_call(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), "-o", str(exe), str(src)])
    out = [int(v) for v in subprocess.check_output([str(exe)]).split()]
    assert out == [ctypes.sizeof(struct)] + [getattr(struct, f).offset for f in fields]


def test_wrapper_refuses_wrong_tensors():
    pr = _pr(rows=2)
    pos, f = torch.zeros(2, dtype=torch.int32), torch.zeros(32, dtype=torch.float64)
    q = torch.zeros(2, 4, 128, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        li.rope(pr, pos.long(), f, q)
    with pytest.raises(TypeError):
        li.rope(pr, pos, f, q.float())
    with pytest.raises(ValueError):
        li.rope(pr, pos, f[:31], q)
    with pytest.raises(ValueError):
        li.rope(pr, pos, f, q[:, :, ::2])
    with pytest.raises(ValueError):
        li.rope(pr, pos, f, q)                                  # host tensors


def test_rope_of_no_rows_needs_no_tensors():
    """Empty tensors have no address; the parameters are checked all the same."""
    def call(**kw):
        return li.STATUS_NAMES[li.lib().li_rope(ctypes.byref(_pr(rows=0, **kw)), None, None, None, None, None, None, None)]
    assert call() == call(N2=2) == call(q_out_row_stride=1024) == "LI_OK" and li.li_last_launch_count() == 0
    assert call(rot_dim=63) == call(q_row_stride=511) == "LI_ERR_SHAPE"


@pytest.mark.parametrize("field,reach", [
    ("q_row_stride", 7 * 600 + 512), ("q_head_stride", 7 * 1024 + 3 * 130 + 128), ("q_out_row_stride", 7 * 600 + 512),
    ("q_out_head_stride", 7 * 1024 + 3 * 130 + 128), ("k_row_stride", 7 * 600 + 256), ("k_out_row_stride", 7 * 600 + 256),
    ("k_head_stride", 7 * 1024 + 130 + 128), ("k_out_head_stride", 7 * 1024 + 130 + 128)])
def test_wrapper_refuses_strides_that_leave_the_memory(field, reach):
    """A row stride of 600, or heads 130 apart in rows of 1024: the last element
    that the call reaches is the last one of the tensor, or one behind it."""
    row = 600 if "row" in field else 1024
    kw = {field: row if "row" in field else 130, field.replace("head", "row"): row}
    pr = _pr(N2=2, **kw)
    pos, f = torch.zeros(8, dtype=torch.int32), torch.zeros(32, dtype=torch.float64)
    t = {n: torch.zeros(8, h, 128, dtype=torch.bfloat16) for n, h in (("query", 4), ("key", 2), ("out", 4), ("key_out", 2))}
    name = {"q_out": "out", "k_out": "key_out"}.get(field[:5], "query" if field[0] == "q" else "key")
    for short, match in ((0, "CUDA device"), (1, "%s has %d elements of memory" % (name, reach - 1))):
        # a view from element 8 on of a longer tensor: what lies before it does not count
        t[name] = torch.zeros(8 + reach - short, dtype=torch.bfloat16)[8:]
        with pytest.raises(ValueError, match=match):
            li.rope(pr, pos, f, **t)


# ------------------------------------------------------------------ GPU

def _tolerance(x, rot, off, pairing, m, dt):
    """Per element of the rotated part: see the module docstring."""
    h = rot // 2
    y = np.abs(x[..., off:off + rot])
    s = (y[..., :h] + y[..., h:]) if pairing == "half" else (y[..., ::2] + y[..., 1::2])
    s = np.concatenate([s, s], -1) if pairing == "half" else np.repeat(s, 2, -1)
    return m * s * (2.0 ** -21 + 3 * 2.0 ** -24)


def _check(y, ref, x, rot, off, pairing, m, dtype):
    eps = torch.finfo(DT[dtype]).eps / 2
    tiny = torch.finfo(DT[dtype]).smallest_normal * eps          # results below the normal range
    err = np.abs(y - ref)
    part = slice(off, off + rot)
    tol = _tolerance(x, rot, off, pairing, m, dtype)
    tol = tol + eps * (np.abs(ref[..., part]) + tol) + tiny
    assert np.all(err[..., part] <= tol), (err[..., part] - tol).max()
    rest = np.ones(x.shape[-1], bool)
    rest[part] = False
    assert np.array_equal(y[..., rest], x[..., rest])


CASES = [
    # dtype, rows, N1, N2, D, rot, off, pairing, inverse, mscale
    ("bf16", 1, 1, 0, 64, 64, 0, "half", 0, 1.0),
    ("bf16", 64, 64, 1, 128, 64, 0, "interleaved", 0, 1.0),
    ("bf16", 700, 64, 8, 128, 128, 0, "half", 0, 1.0),
    ("bf16", 700, 24, 2, 192, 64, 128, "interleaved", 1, 1.37),
    ("fp16", 333, 7, 3, 96, 32, 32, "half", 1, 0.9),
    ("fp16", 5, 128, 128, 128, 16, 8, "interleaved", 0, 1.0),
    ("fp32", 129, 5, 1, 80, 40, 4, "half", 0, 1.2),
    ("fp32", 257, 3, 0, 100, 36, 64, "interleaved", 0, 1.0),
    ("bf16", 65, 5, 2, 99, 50, 7, "half", 0, 1.0),             # nothing aligned
    ("fp16", 65, 5, 2, 99, 50, 7, "interleaved", 1, 1.0),
    ("bf16", 40, 6, 1, 100, 36, 2, "half", 0, 1.0),            # pairs of two
    ("bf16", 3000, 1, 1, 64, 2, 0, "half", 0, 1.0),
    ("bf16", 2, 1024, 1024, 1024, 1024, 0, "half", 0, 1.0),
    ("fp16", 5000, 2, 0, 256, 252, 4, "interleaved", 0, 1.0),
    ("bf16", 300, 40, 3, 128, 90, 31, "interleaved", 1, 1.1),  # whole heads aligned, the turned part not
    ("fp32", 41, 9, 1, 1024, 1000, 5, "half", 0, 1.0),
    ("fp16", 5000, 1, 1, 64, 30, 1, "half", 0, 1.0),
    ("bf16", 1, 7, 2, 96, 50, 46, "half", 0, 1.0),
    ("bf16", 2500, 3, 0, 8, 2, 5, "half", 0, 1.0),
]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,rows,N1,N2,D,rot,off,pairing,inverse,m", CASES)
def test_rope_matches_64_bits(dtype, rows, N1, N2, D, rot, off, pairing, inverse, m):
    g = torch.Generator().manual_seed(rows + D)
    q = torch.randn(rows, N1, D, generator=g).to(DT[dtype])
    k = torch.randn(rows, N2, D, generator=g).to(DT[dtype])
    pos = torch.randint(-(1 << 20), 1 << 24, (rows,), generator=g, dtype=torch.int32)
    f, _ = li.rope_frequencies(rot)
    pr = li.make_rope_params(dtype=dtype, rows=rows, N1=N1, N2=N2, D=D, rot_dim=rot, rot_offset=off, pairing=pairing,
                             inverse=inverse, mscale=m)
    m32 = float(np.float32(m))
    out, kout = li.rope(pr, pos.cuda(), f.cuda(), q.cuda(), k.cuda() if N2 else None)
    assert li.li_last_launch_count() == 1
    for x, y in ((q, out), (k, kout)):
        if y is None:
            continue
        x64 = x.double().numpy()
        ref = oc.rope(x64, pos.numpy(), f.numpy(), rot, off, pairing, bool(inverse), m32)
        _check(y.double().cpu().numpy(), ref, x64, rot, off, pairing, m32, dtype)


@pytest.mark.gpu
def test_rope_of_an_empty_step():
    e = lambda n: torch.empty(0, n, 128, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    pos, f = torch.empty(0, dtype=torch.int32, device="cuda"), li.rope_frequencies(64)[0].cuda()
    out, kout = li.rope(_pr(rows=0, N2=2), pos, f, e(4), e(2))
    assert out.shape == (0, 4, 128) and kout.shape == (0, 2, 128) and li.li_last_launch_count() == 0
    q = e(4)
    assert li.rope(_pr(rows=0, q_row_stride=1000, q_out_row_stride=1000), pos, f, q, out=q)[0] is q


@pytest.mark.gpu
def test_rope_positions_at_the_ends_of_int32():
    pos = torch.tensor([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 2 ** 24 + 1], dtype=torch.int32)
    f, _ = li.rope_frequencies(64)
    x = torch.randn(6, 2, 64, generator=torch.Generator().manual_seed(1))
    pr = li.make_rope_params(dtype="fp32", rows=6, N1=2, N2=0, D=64, rot_dim=64, rot_offset=0, pairing="half", inverse=0)
    out, _ = li.rope(pr, pos.cuda(), f.cuda(), x.cuda())
    ref = oc.rope(x.double().numpy(), pos.numpy(), f.numpy(), 64, 0, "half")
    assert np.array_equal(out[0].cpu().numpy(), x[0].numpy())     # position 0 turns nothing
    # up to 2^31 / (2 pi) turns: two 64-bit roundings of the product are 2^-24 turns, 2^-21.3 in the angle
    err = np.abs(out.double().cpu().numpy() - ref)
    tol = _tolerance(x.double().numpy(), 64, 0, "half", 1.0, "fp32")
    assert np.all(err <= 2.5 * tol + 2.0 ** -24 * np.abs(ref))


@pytest.mark.gpu
def test_rope_in_place_and_heads_inside_a_projection():
    """Query and key heads of one fused projection [rows, N1+N2+N2, D], turned in place."""
    rows, N1, N2, D = 77, 12, 2, 128
    g = torch.Generator().manual_seed(3)
    qkv = torch.randn(rows, N1 + 2 * N2, D, generator=g).to(torch.bfloat16).cuda()
    before = qkv.clone()
    pos = torch.arange(rows, dtype=torch.int32).cuda() * 1000
    f, _ = li.rope_frequencies(64)
    s = (N1 + 2 * N2) * D
    pr = li.make_rope_params(dtype="bf16", rows=rows, N1=N1, N2=N2, D=D, rot_dim=64, rot_offset=64, pairing="interleaved",
                             inverse=0, q_row_stride=s, k_row_stride=s, q_out_row_stride=s, k_out_row_stride=s)
    q, k = qkv[:, :N1], qkv[:, N1:N1 + N2]
    li.rope(pr, pos, f.cuda(), q, k, out=q, key_out=k)
    dense = li.make_rope_params(dtype="bf16", rows=rows, N1=N1, N2=N2, D=D, rot_dim=64, rot_offset=64,
                                pairing="interleaved", inverse=0)
    qd, kd = li.rope(dense, pos, f.cuda(), before[:, :N1].contiguous(), before[:, N1:N1 + N2].contiguous())
    assert torch.equal(qkv[:, :N1], qd) and torch.equal(qkv[:, N1:N1 + N2], kd)
    assert torch.equal(qkv[:, N1 + N2:], before[:, N1 + N2:])      # the values were not touched


@pytest.mark.gpu
@pytest.mark.parametrize("pairing", ["half", "interleaved"])
def test_rope_inverse_is_the_gradient(pairing):
    """d/dx of sum(rope(x) * c) is the inverse turn of c: against the 64-bit
    formula's differences (the map is linear, so a central difference is exact
    up to rounding)."""
    g = torch.Generator().manual_seed(4)
    rows, N, D, rot = 3, 2, 64, 32
    x, c = torch.randn(rows, N, D, generator=g), torch.randn(rows, N, D, generator=g)
    pos = torch.tensor([5, 70000, 123456], dtype=torch.int32)
    f, m = li.rope_frequencies(rot, scaling="yarn", factor=4.0, original_positions=4096)
    kw = dict(dtype="fp32", rows=rows, N1=N, N2=0, D=D, rot_dim=rot, rot_offset=8, pairing=pairing, mscale=m)
    grad, _ = li.rope(li.make_rope_params(inverse=1, **kw), pos.cuda(), f.cuda(), c.cuda())
    x64, c64 = x.double().numpy(), c.double().numpy()
    h = 0.5
    for at in [(0, 0, 3), (0, 1, 8), (1, 0, 9), (1, 1, 24), (2, 0, 39), (2, 1, 63)]:
        up, down = x64.copy(), x64.copy()
        up[at] += h
        down[at] -= h
        diff = sum((oc.rope(v, pos.numpy(), f.numpy(), rot, 8, pairing, False, m) * c64).sum() * s
                   for v, s in ((up, 1), (down, -1))) / (2 * h)
        assert abs(diff - float(grad[at])) <= 1e-5 * (1 + abs(diff))


@pytest.mark.gpu
def test_rope_graph_stream_and_rows_behind():
    rows, N, D = 50, 8, 128
    g = torch.Generator().manual_seed(5)
    q = torch.randn(rows, N, D, generator=g).to(torch.bfloat16).cuda()
    pos = torch.arange(rows, dtype=torch.int32).cuda()
    f = li.rope_frequencies(128)[0].cuda()
    mk = lambda r: li.make_rope_params(dtype="bf16", rows=r, N1=N, N2=0, D=D, rot_dim=128, rot_offset=0, pairing="half", inverse=0)  # noqa: E731
    want, _ = li.rope(mk(rows), pos, f, q)
    out = torch.full_like(q, 7.0)
    li.li_rope(mk(rows - 3), pos, f, q, None, out, None)
    assert torch.equal(out[:-3], want[:-3]) and bool((out[-3:] == 7).all())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out2 = torch.empty_like(q)
    with torch.cuda.stream(side):
        li.rope(mk(rows), pos, f, q, out=out2)
    side.synchronize()
    assert torch.equal(out2, want)
    graph, out3 = torch.cuda.CUDAGraph(), torch.zeros_like(q)
    with torch.cuda.graph(graph):
        li.rope(mk(rows), pos, f, q, out=out3)
    q.mul_(2)                                                    # replays read the buffers' present contents
    graph.replay()
    assert torch.equal(out3, want * 2)
