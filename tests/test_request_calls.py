"""Call sequences of prompts, forks and log probabilities in the paged cache and the rounds, with the library's calls replaced by
records: what they hand over, on which stream, without a GPU."""
import contextlib
import types

import pytest
import torch


@pytest.fixture
def calls(monkeypatch):
    import __graft_entry__

    __graft_entry__._load_builder().build()
    from dynamic_draft_tree_gb300 import paged

    log = []
    for name in [n for n in vars(paged) if n.startswith("dt_")]:
        monkeypatch.setattr(paged, name, lambda *a, _n=name, **k: log.append((_n, a, k)) or f"made by {_n}")
    return log


def _cache(**over):
    from dynamic_draft_tree_gb300.paged import PagedCache

    kv = PagedCache.__new__(PagedCache)
    kv.h, kv.B, kv.P, kv.H_q, kv.H_kv, kv.D, kv.packed, kv.shared_len, kv.filled = None, 2, 4, 2, 1, 16, False, 0, False
    kv.pages = torch.zeros(4, 8, 16, 1, 16)
    kv.seq_len = torch.zeros(2, dtype=torch.int32)
    kv.pool = types.SimpleNamespace(page=16, block_table=torch.full((2, 4), -1, dtype=torch.int32))
    for k, v in over.items():
        setattr(kv, k, v)
    return kv


def test_prompts_read_a_layers_pages(calls, monkeypatch):
    current, made_on = ["default"], []

    @contextlib.contextmanager
    def stream(s):
        before = current[0]
        current[0] = before if s is None else s
        yield
        current[0] = before

    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    from dynamic_draft_tree_gb300 import paged

    monkeypatch.setattr(paged, "dt_prompt_attention_workspace", lambda *a: made_on.append((current[0], a)) or "workspace")
    kv = _cache()
    kv.attend_prompts(1, "q", "k", "v", "off", "out", scale=0.25, stream="side")
    kv.attend_prompts(0, "q", "k", "v", "off", "out")
    assert made_on == [("side", (None, 2, 2, 1, 16))]  # once, in memory of the stream of its first call
    (n0, a0, k0), (n1, a1, k1) = calls
    assert n0 == n1 == "dt_prompt_attention"
    assert a0 == (None, "q", "k", "v", "off", "out", "workspace") == a1
    assert k0["stream"] == "side" and k1["stream"] is None and k0["scale"] == 0.25 and k1["scale"] is None
    for k, layer in ((k0, 1), (k1, 0)):
        assert k["k_pages"].data_ptr() == kv.pages[2 * layer].data_ptr()
        assert k["v_pages"].data_ptr() == kv.pages[2 * layer + 1].data_ptr()
        assert k["block_table"] is kv.pool.block_table and k["seq_len"] is kv.seq_len


def test_a_captured_first_call_is_refused(calls, monkeypatch):
    """The workspace would be the graph's memory."""
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    kv = _cache()
    with pytest.raises(RuntimeError):
        kv.attend_prompts(0, "q", "k", "v", "off", "out")
    assert calls == [] and kv.prompt_workspace is None
    kv.prompt_workspace = "workspace"
    kv.attend_prompts(0, "q", "k", "v", "off", "out")
    assert [c[0] for c in calls] == ["dt_prompt_attention"]


def test_forks_take_the_caches_state(calls):
    refs = torch.zeros(8, dtype=torch.int32)
    kv = _cache(refs=refs, shared_len=32)
    kv.fork("src", "dst", length="len", stream="side")
    kv.fork("src", "dst")
    (n0, a0, k0), (n1, a1, k1) = calls
    assert n0 == n1 == "dt_kv_fork"
    assert a0[1] is kv.pool and a0[2] is refs and a0[3] is kv.pages and a0[4:6] == ("src", "dst") and a0[6] is kv.seq_len
    assert k0 == dict(length="len", shared_len=32, stream="side") and k1 == dict(length=None, shared_len=32, stream=None)


def test_a_cache_with_forks_releases_shared_pages(calls):
    keep = torch.zeros(2, dtype=torch.int32)
    refs = torch.zeros(8, dtype=torch.int32)
    _cache(refs=refs).release(keep)
    _cache().release(keep)
    (n0, a0, _), (n1, a1, _) = calls
    assert n0 == "dt_kv_release_shared" and a0[2] is refs and n1 == "dt_kv_release"


def test_a_cache_without_forks_refuses_them(calls):
    with pytest.raises(ValueError):
        _cache().fork("src", "dst")
    assert calls == []


@pytest.mark.parametrize("packed", [False, True])
def test_a_rounds_log_probabilities_are_of_its_verified_rows(calls, monkeypatch, packed):
    from dynamic_draft_tree_gb300 import DT_ANCHOR_TAIL, rounds
    from dynamic_draft_tree_gb300.paged import TokenLogprobs

    class Anything:
        def __getattr__(self, name):
            return Anything()

    for name in [n for n in vars(rounds) if n.startswith("dt_")]:
        monkeypatch.setattr(rounds, name, lambda *a, _n=name, **k: calls.append((_n, a, k)))
    r = rounds.RoundRunner.__new__(rounds.RoundRunner)
    for name in ("h", "selected", "m_dev", "width", "frontier_token", "params", "prune_out", "ret_token", "ret_parent",
                 "ret_count", "ret_anchor", "pos_offset"):
        setattr(r, name, Anything())
    r.meta = types.SimpleNamespace(tokens="tokens", row_off="row_off", P=7)
    r.accept_len, r.bonus = torch.zeros(2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    r.accept_path = torch.zeros(2, 5, dtype=torch.int32)
    r.policy, r.B, r.P, r.D, r.D_path, r.k, r.m_cap, r.T, r.R_cap = "eagle", 2, 7, 2, 5, 2, 3, 0, 2
    r.packed, r.fused, r.block, r.draw, r.top8 = packed, True, False, False, None
    r.stop = types.SimpleNamespace(zero_=lambda: None)
    r.template, r.graft = types.SimpleNamespace(anchor=DT_ANCHOR_TAIL), {"K_total": 4}
    lp = TokenLogprobs.__new__(TokenLogprobs)
    lp.h, lp.K, lp.workspace = "handle", 0, "workspace"
    lp.logp, lp.entropy, lp.rank, lp.top_ids, lp.top_logp = torch.zeros(2, 5), torch.zeros(2, 5), torch.zeros(2, 5), None, None
    rows = torch.zeros(3)
    r.run(None, lambda d, t: None, lambda meta: rows, logprobs=lp)
    names = [c[0] for c in calls]
    assert names.index("dt_token_logprobs") > max(k for k, n in enumerate(names) if n.startswith("dt_verify"))
    _, a, k = [c for c in calls if c[0] == "dt_token_logprobs"][0]
    assert a[0] == "handle" and a[1] is rows and a[2] is r.accept_len and a[3] is lp.logp and a[4] == "workspace"
    assert k["tokens"] == "tokens" and k["last"] is r.bonus and k["path"] is r.accept_path and k["n_extra"] == 1 and k["P"] == 7
    assert k["row_off"] == ("row_off" if packed else None)
    calls.clear()
    lp.logp = torch.zeros(2, 4)
    with pytest.raises(ValueError):
        lp.round(rows, r.accept_len, r.accept_path, r.bonus, r.meta)
    assert calls == []
