"""Seeded synthetic inputs for segment-sparse attention.

Only draws and lays out tensors: query, key and value rows in the layouts of the
library (BSND, TND, paged), ragged lengths, and the rows that lie behind them
(``junk``: what a padded or recycled buffer may hold there, NaN and infinities
among it).
"""
from __future__ import annotations

import dataclasses
from typing import Optional, Sequence

import torch

from . import DTYPES, _gen


@dataclasses.dataclass
class SegmentProblem:
    """Static description of one segment call (the fields of li_segment_params)."""

    layout_q: str = "BSND"
    layout_kv: str = "BSND"
    dtype: str = "bf16"
    B: int = 1
    S1: int = 0
    S2: int = 0
    T1: int = 0
    T2: int = 0
    N1: int = 16
    N2: int = 2
    D: int = 128
    num_blocks: int = 0
    block_size: int = 0
    max_blocks_per_seq: int = 0
    kv_block_stride: int = 0
    seg_size: int = 64
    seg_count: int = 8
    init_segs: int = 1
    local_segs: int = 1
    max_segs: int = 0
    sparse_mode: int = 3
    softmax_scale: float = 0.0

    @property
    def rows(self) -> int:
        return self.B * self.S1 if self.layout_q == "BSND" else self.T1

    @property
    def scale(self) -> float:
        return self.softmax_scale if self.softmax_scale > 0 else self.D ** -0.5


def make_segment(seed: int, *, q_lens: Sequence[int], k_lens: Sequence[int], junk: Optional[float] = None, spare: int = 2,
                 block_size: int = 64, **kw):
    """A random problem: (SegmentProblem, host tensors).  ``junk``: the value of
    every key and value row behind a sequence's end (and of the spare pages)."""
    g = _gen(seed)
    p = SegmentProblem(B=len(q_lens), **kw)
    x = {}
    dt = DTYPES[p.dtype]

    def randn(*shape):
        return torch.randn(*shape, generator=g, dtype=torch.float32).to(dt)

    i32 = lambda v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    p.max_segs = p.max_segs or max(1, max(-(-n // p.seg_size) for n in k_lens))
    if p.layout_q == "BSND":
        p.S1 = max(q_lens)
        x["query"] = randn(p.B, p.S1, p.N1, p.D)
        x["act_q"] = i32(q_lens)
    else:
        p.T1 = sum(q_lens)
        x["query"] = randn(p.T1, p.N1, p.D)
        x["act_q"] = i32(q_lens).cumsum(0).to(torch.int32)
    if p.layout_kv == "BSND":
        p.S2 = max(k_lens)
        shape = (p.B, p.S2, p.N2, p.D)
        x["act_k"] = i32(k_lens)
    elif p.layout_kv == "TND":
        p.T2 = sum(k_lens)
        shape = (p.T2, p.N2, p.D)
        x["act_k"] = i32(k_lens).cumsum(0).to(torch.int32)
    else:
        p.block_size = block_size
        need = [-(-n // block_size) for n in k_lens]
        p.num_blocks = sum(need) + spare
        p.max_blocks_per_seq = max(1, max(need))
        shape = (p.num_blocks, block_size, p.N2, p.D)
        x["act_k"] = i32(k_lens)
        perm = torch.randperm(p.num_blocks, generator=g).to(torch.int32)
        x["block_table"] = torch.full((p.B, p.max_blocks_per_seq), -1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            x["block_table"][b, :n] = perm[at:at + n]
            at += n
    x["key"], x["value"] = randn(*shape), randn(*shape)
    if junk is not None:
        behind = torch.ones(shape[:-2], dtype=torch.bool)
        for b, n in enumerate(k_lens):
            t = torch.arange(n)
            if p.layout_kv == "BSND":
                behind[b, :n] = False
            elif p.layout_kv == "TND":
                behind[:] = False
            elif n:
                behind[x["block_table"][b][t // block_size].long(), t % block_size] = False
        x["key"][behind] = junk
        x["value"][behind] = junk
    return p, x
