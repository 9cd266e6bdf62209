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
    kv.h, kv.B, kv.P, kv.H_q, kv.H_kv, kv.D, kv.packed, kv.shared_len, kv.filled = None, 2, 4, 2, 1, 16, False, 0, False
    kv.pages = torch.zeros(2, 8, 16, 1, 16)
    kv.tmp = torch.zeros(2, 2, 4, 1, 16)
    kv.seq_len = torch.zeros(2, dtype=torch.int32)
    kv.slots = torch.zeros(2, 5, dtype=torch.int64)
    kv.committed = torch.zeros(2, dtype=torch.int32)
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


class _Anything:
    """Stands for a handle, device buffers and outputs that only pass through."""

    def __getattr__(self, name):
        return _Anything()


def _runner(monkeypatch, log, policy="eagle", B=2, P=4, packed=False):
    """A RoundRunner without its constructor, whose library calls are records."""
    from dynamic_draft_tree_gb300 import DT_ANCHOR_TAIL, rounds

    for name in [n for n in vars(rounds) if n.startswith("dt_")]:
        monkeypatch.setattr(rounds, name, lambda *a, _n=name, **k: log.append((_n, a, k)))
    r = rounds.RoundRunner.__new__(rounds.RoundRunner)
    for name in ("h", "meta", "selected", "m_dev", "width", "stop", "frontier_token", "params", "prune_out", "ret_token",
                 "ret_parent", "ret_count", "ret_anchor", "accept_len", "accept_path", "bonus", "pos_offset"):
        setattr(r, name, _Anything())
    r.policy, r.B, r.P, r.D, r.D_path, r.k, r.m_cap, r.T, r.R_cap = policy, B, P, 2, 5, 2, 3, 0, 2
    r.packed, r.fused, r.block, r.draw, r.top8 = packed, True, False, False, None
    r.stop = types.SimpleNamespace(zero_=lambda: None)
    r.template, r.graft = types.SimpleNamespace(anchor=DT_ANCHOR_TAIL), {"K_total": 4}
    return r


@pytest.mark.parametrize("policy", ["eagle", "graft"])
def test_a_rounds_positions_start_behind_the_cache(calls, monkeypatch, policy):
    run = _runner(monkeypatch, calls, policy)
    kv = _cache()
    offsets = []
    for cache in (kv, None):
        run.run(None, lambda d, t: None, lambda meta: None, kv=cache)
        offsets += [a[4] for n, a, k in calls if n == "dt_build_tree_meta"]
        calls.clear()
    assert offsets[0] is kv.seq_len and offsets[1] is run.pos_offset


def test_tokens_are_counted_after_their_rows_are_in_the_pages(calls, monkeypatch):
    """The count takes what the commit appended, not what was accepted; without a cache, what was accepted."""
    from dynamic_draft_tree_gb300.paged import TokenState

    run = _runner(monkeypatch, calls)
    run.accept_len = torch.zeros(2, dtype=torch.int32)
    state = TokenState.__new__(TokenState)
    state.h = state.counts = state.repetition = state.frequency = state.presence = None
    state.bias_ids = state.bias_vals = state.allow = None
    kv = _cache(committed=torch.zeros(3, dtype=torch.int32))
    for cache in (kv, None):
        run.run(None, lambda d, t: None, lambda meta: None, kv=cache, tokens=state)
        order = [n for n, a, k in calls if n in ("dt_commit_kv_paged", "dt_count_tokens")]
        count = [(a, k) for n, a, k in calls if n == "dt_count_tokens"][0]
        if cache is None:
            assert order == ["dt_count_tokens"] and count[0][3] is run.accept_len and count[1]["n_extra"] == 1
        else:
            assert order == ["dt_commit_kv_paged", "dt_count_tokens"]
            assert [k for n, a, k in calls if n == "dt_commit_kv_paged"][0]["committed"] is kv.committed
            assert count[0][3].data_ptr() == kv.committed.data_ptr() and count[0][3].numel() == 2
            assert count[1]["n_extra"] == 0
        calls.clear()


@pytest.mark.parametrize("over", [dict(packed=True), dict(P=3), dict(B=1)])
def test_a_cache_of_other_rows_is_refused_before_the_round(calls, monkeypatch, over):
    run = _runner(monkeypatch, calls)
    with pytest.raises(ValueError):
        run.run(None, lambda d, t: None, lambda meta: None, kv=_cache(**over))
    assert calls == []
    run.run(None, lambda d, t: None, lambda meta: None, kv=_cache(P=run.P + 1, B=run.B + 1))  # more room is no fault
    assert "dt_commit_kv_paged" in [c[0] for c in calls]


def test_a_release_keeps_the_shared_prefix(calls):
    keep = torch.tensor([0, 40], dtype=torch.int32)
    _cache().release(keep)
    _cache(shared_len=32).release(keep)
    assert [a[2].tolist() for n, a, k in calls] == [[0, 40], [32, 40]]
    assert calls[0][1][2] is keep and calls[1][1][2].dtype is torch.int32 and keep.tolist() == [0, 40]


def test_a_prefix_has_the_caches_length(calls):
    from dynamic_draft_tree_gb300.paged import PagedCache

    for shared, rows, filled in ((0, 32, False), (32, 31, False), (32, 32, True)):
        with pytest.raises(ValueError):
            _cache(shared_len=shared, filled=filled).prefix(torch.zeros(2, rows, 1, 16))
    for shared in (-16, 24, 80):
        with pytest.raises(ValueError):
            PagedCache(None, 2, 4, 1, 2, 1, 16, n_blocks=8, max_blocks=4, page=16, shared_len=shared, device="cpu")
    assert calls == []
