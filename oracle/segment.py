"""fp64 CPU oracle of segment-sparse attention (test infrastructure; shares
nothing with the CUDA library): the segments' mean keys, the choice of segments
and the attention over them, from the definitions, one row at a time.

``p`` has the fields of a segment problem (``synth.segment``), ``x`` its input
tensors on the host.
"""
from __future__ import annotations

import numpy as np


def f64(t):
    return t.detach().cpu().double().numpy()


def batches(p, x):
    """Per batch: first query row, allocated rows, query length, key length."""
    out = []
    aq, ak = x.get("act_q"), x.get("act_k")
    q0 = k0 = 0
    for b in range(p.B):
        if p.layout_q == "BSND":
            first, alloc, nq = b * p.S1, p.S1, p.S1 if aq is None else int(aq[b])
        else:
            first, alloc, nq = q0, int(aq[b]) - q0, int(aq[b]) - q0
            q0 = int(aq[b])
        if p.layout_kv == "BSND":
            nk = p.S2 if ak is None else int(ak[b])
        elif p.layout_kv == "TND":
            nk, k0 = int(ak[b]) - k0, int(ak[b])
        else:
            nk = int(ak[b])
        out.append((first, alloc, nq, nk))
    return out


def keys(p, x, name, b, t):
    """Rows [len(t), N2, D] of `name` that hold the keys `t` of batch b."""
    v = x[name]
    if p.layout_kv == "BSND":
        return f64(v[b][t])
    if p.layout_kv == "TND":
        start = int(x["act_k"][b - 1]) if b else 0
        return f64(v[start + t])
    ids = x["block_table"][b].numpy()[t // p.block_size]
    return f64(v[ids.astype(np.int64), t % p.block_size])


def pool(p, x):
    """{(b, s): [N2, D]} of every segment that holds a key."""
    out = {}
    for b, (_, _, _, nk) in enumerate(batches(p, x)):
        for s in range(-(-nk // p.seg_size)):
            t = np.arange(s * p.seg_size, min(nk, (s + 1) * p.seg_size))
            out[b, s] = keys(p, x, "key", b, t).mean(0)
    return out


def visible(p, i, nq, nk):
    return nk if p.sparse_mode == 0 else min(max(i + 1 + nk - nq, 0), nk)


def select(p, x, pooled):
    """seg_idx [rows, N2, seg_count] from pooled [B, max_segs, N2, D]."""
    P = f64(pooled)
    q = f64(x["query"]).reshape(p.rows, p.N2, p.N1 // p.N2, p.D).sum(2)
    out = np.full((p.rows, p.N2, p.seg_count), -1, dtype=np.int32)
    for b, (first, _, nq, nk) in enumerate(batches(p, x)):
        for i in range(nq):
            ns = -(-visible(p, i, nq, nk) // p.seg_size)
            for n in range(p.N2):
                sc = P[b, :ns, n] @ q[first + i, n]
                sc = np.where(np.isnan(sc), -np.inf, sc)
                s = np.arange(ns)
                forced = (s < p.init_segs) | (s >= ns - p.local_segs)
                order = np.lexsort((s, -sc, ~forced))[:p.seg_count]
                out[first + i, n, :len(order)] = np.sort(order)
    return out


def attention(p, x, seg_idx):
    """out [rows, N1, D] and lse [rows, N1] in float64."""
    q = f64(x["query"]).reshape(p.rows, p.N2, p.N1 // p.N2, p.D)
    idx = np.asarray(seg_idx).reshape(p.rows, p.N2, p.seg_count)
    out = np.zeros(q.shape)
    lse = np.full(q.shape[:3], -np.inf)
    for b, (first, _, nq, nk) in enumerate(batches(p, x)):
        for i in range(nq):
            vis = visible(p, i, nq, nk)
            for n in range(p.N2):
                segs, last = [], -1
                for s in idx[first + i, n]:
                    if s > last and s < -(-nk // p.seg_size):
                        segs.append(s)
                        last = s
                t = np.concatenate([np.arange(s * p.seg_size, (s + 1) * p.seg_size) for s in segs] or [np.zeros(0, int)])
                t = t[t < vis].astype(np.int64)
                if not len(t):
                    continue
                l = p.scale * (q[first + i, n] @ keys(p, x, "key", b, t)[:, n].T)
                m = l.max(1, keepdims=True)
                e = np.exp(l - m)
                z = e.sum(1, keepdims=True)
                out[first + i, n] = (e / z) @ keys(p, x, "value", b, t)[:, n]
                lse[first + i, n] = (m + np.log(z))[:, 0]
    return out.reshape(p.rows, p.N1, p.D), lse.reshape(p.rows, p.N1)
