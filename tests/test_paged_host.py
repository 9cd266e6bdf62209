"""The paged cache's call sequences with the library's calls replaced by records: what they allocate, where, and in what
order, without a GPU."""
import contextlib
import types

import pytest
import torch


@pytest.fixture
def calls(monkeypatch):
    """paged.py with recorded library calls; returns the list of (name, args, kwargs)."""
    import __graft_entry__

    __graft_entry__._load_builder().build()
    from dynamic_draft_tree_gb300 import paged

    log = []
    for name in ("dt_kv_reserve", "dt_kv_release", "dt_commit_kv_paged", "dt_tree_attention", "dt_count_tokens",
                 "dt_logits_process"):
        monkeypatch.setattr(paged, name, lambda *a, _n=name, **k: log.append((_n, a, k)))
    return log


def _cache(**over):
    """A PagedCache without its constructor (no handle, no device)."""
    from dynamic_draft_tree_gb300.paged import PagedCache

    kv = PagedCache.__new__(PagedCache)
    kv.h, kv.B, kv.P, kv.H_q, kv.H_kv, kv.D, kv.packed, kv.shared_len = None, 2, 4, 2, 1, 16, False, 0
    kv.pages = torch.zeros(2, 8, 16, 1, 16)
    kv.tmp = torch.zeros(2, 2, 4, 1, 16)
    kv.seq_len = torch.zeros(2, dtype=torch.int32)
    kv.slots = torch.zeros(2, 5, dtype=torch.int64)
    kv.pool = types.SimpleNamespace(page=16, block_table=torch.full((2, 4), -1, dtype=torch.int32),
                                    n_owned=torch.zeros(2, dtype=torch.int32))
    for k, v in over.items():
        setattr(kv, k, v)
    return kv


def test_prefill_allocates_on_the_stream_it_runs_on(calls, monkeypatch):
    """Slots that came from another stream's memory could still be written by what is queued there."""
    current, made, empty = ["default"], [], torch.empty

    @contextlib.contextmanager
    def stream(s):
        before = current[0]
        current[0] = before if s is None else s
        yield
        current[0] = before

    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch, "empty", lambda *a, **k: made.append(current[0]) or empty(*a, **k))
    kv, i32 = _cache(), torch.zeros(3, dtype=torch.int32)

    class Side:
        cuda_stream = 1

    side = Side()
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda *a: None)
    kv.prefill(torch.zeros(2, 9, 1, 16), i32[:2], i32, stream=side)
    kv.prefill(torch.zeros(2, 9, 1, 16), i32[:2], i32)
    assert made == [side, "default"]
    assert [c[0] for c in calls] == ["dt_kv_reserve", "dt_commit_kv_paged"] * 2
    assert [c[2]["stream"] for c in calls] == [side, side, None, None]
