"""Token histories of requests that continue others: TokenState.fork takes them along, as PagedCache.fork does pages and lengths."""
import contextlib

import pytest


def _state(t, counts):
    from dynamic_draft_tree_gb300.paged import TokenState

    s = TokenState.__new__(TokenState)
    s.counts = counts
    return s


def _expect(counts, src, dst):
    B, want, seen = len(counts), [list(r) for r in counts], set()
    for f, (s, d) in enumerate(zip(src, dst)):
        if 0 <= s < B and 0 <= d < B and d not in dst[:f] and s not in dst:
            want[d] = list(counts[s])
    return want


PAIRS = {
    "one": ([0], [3]),
    "samples": ([0, 0, 0, 4], [1, 2, 3, 5]),
    "outside": ([0, 6, -1, 1, 1], [2, 3, 4, 6, -1]),
    "named twice": ([0, 1, 4], [2, 2, 3]),
    "a source that is a destination": ([0, 1, 2], [1, 3, 5]),
    "itself": ([2, 0], [2, 5]),
    "far outside": ([2147483647, 0], [1, -2147483648]),
}


@pytest.mark.parametrize("name", list(PAIRS))
def test_histories_go_along(name, monkeypatch):
    import torch

    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    import __graft_entry__

    __graft_entry__._load_builder().build()
    g = torch.Generator().manual_seed(3)
    counts = torch.randint(-2 ** 31, 2 ** 31 - 1, (6, 50), generator=g).int()
    src, dst = PAIRS[name]
    want = _expect(counts.tolist(), src, dst)
    s = _state(torch, counts.clone())
    s.fork(*(torch.tensor(x, dtype=torch.int32) for x in (src, dst)))
    assert s.counts.tolist() == want


@pytest.mark.gpu
def test_samples_keep_their_prompts_history_in_rounds():
    """Rounds with penalties on samples of a request: their processed rows are the source's, and so are their counts."""
    import torch as t

    if not t.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__

    __graft_entry__.build()
    import dynamic_draft_tree_gb300 as dt
    from dynamic_draft_tree_gb300.paged import PagedCache, TokenState
    from dynamic_draft_tree_gb300.rounds import RoundRunner

    B, V, K, k, D, m = 4, 900, 4, 4, 3, 12
    P, D_path = m + 1, D + 1
    g = t.Generator(device="cuda")
    g.manual_seed(11)
    i32 = lambda v: t.tensor(v, dtype=t.int32, device="cuda")  # noqa: E731
    run = RoundRunner("eagle", B, V, K, k, D, P, D_path, m, dt.DT_F32, T=0)
    h = run.h
    kv = PagedCache(h, B, P, 1, 2, 1, 16, n_blocks=40, max_blocks=8, page=16, D_path=D_path, forks=True)
    full = lambda v: t.full((B,), v, device="cuda")  # noqa: E731
    tokens = TokenState(h, B, repetition=full(1.3), frequency=full(0.2), presence=full(0.4))
    tokens.counts[2] = 5  # what an earlier request left in the place
    rows = t.randn(2, 30, 1, 16, generator=g, device="cuda").bfloat16()
    prompt = t.randint(0, V, (30,), generator=g, dtype=t.int32, device="cuda")
    off, n = i32([0, 20, 30, 30, 30]), i32([20, 10, 0, 0])
    kv.prefill(rows, n, off)
    tokens.prompt(prompt, n, row_off=off)
    kv.fork(i32([0, 0]), i32([2, 3]))
    tokens.fork(i32([0, 0]), i32([2, 3]))
    assert dt.dt_get_status(h) == 0 and bool((tokens.counts[2:] == tokens.counts[0]).all())
    assert bool((tokens.counts[0][prompt[:20].long()] == dt.DT_SEEN_PROMPT).all()) and not t.equal(tokens.counts[0], tokens.counts[1])

    def alike(*shape):  # the same rows for every request
        return t.randn(1, *shape, generator=g, device="cuda").expand(B, *shape).contiguous()

    seen = {}

    def target_rows(meta):
        seen["rows"] = alike(P, V) * 3
        return seen["rows"]

    for rnd in range(3):
        run.run(i32([7, 8, 7, 7]), lambda d, f: alike(1 if d == 1 else k, V), target_rows, rnd=rnd, kv=kv, tokens=tokens)
        assert dt.dt_get_status(h) == 0
        n_pos = int(run.meta.n_pos[0])
        for b in (2, 3):  # a sample does as its source
            assert t.equal(seen["rows"][b, :n_pos], seen["rows"][0, :n_pos])
            assert int(run.accept_len[b]) == int(run.accept_len[0]) and int(run.bonus[b]) == int(run.bonus[0])
            assert t.equal(tokens.counts[b], tokens.counts[0])
        assert not t.equal(seen["rows"][1, :n_pos], seen["rows"][0, :n_pos])
    # a captured call, replayed after the histories changed; another stream
    src, dst = i32([0, 1]), i32([2, 3])
    tokens.fork(src, dst)
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        tokens.fork(src, dst)
    tokens.counts[0] += 1
    tokens.counts[3] = 9
    graph.replay()
    t.cuda.synchronize()
    assert t.equal(tokens.counts[2], tokens.counts[0]) and t.equal(tokens.counts[3], tokens.counts[1])
    side = t.cuda.Stream()
    tokens.counts[3] = 9
    side.wait_stream(t.cuda.current_stream())
    tokens.fork(src, dst, stream=side)
    side.synchronize()
    assert t.equal(tokens.counts[3], tokens.counts[1])
    h.close()
