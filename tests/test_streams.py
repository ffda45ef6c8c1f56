"""What the wrappers allocate themselves: the workspace lives until the launch."""
from __future__ import annotations

import weakref

import pytest
import torch

import sparse_attention_top_n1_b200 as li

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
