"""Rounds with a paged cache and processed rows, as a serving loop runs them.

Every round the target's "forward" draws keys, values and queries for the tree's positions, attends layer by layer through
``PagedCache`` and makes its rows from the result; ``RoundRunner`` processes, verifies, counts and commits. A shadow of
the state is kept in plain form (dense keys and values a request, a count table); attention and processed rows are compared
with the definitions in 64 bits, pages, lengths and counts exactly. Tolerances as in the operators' own tests: for bf16 with
u = 2^-8, 2.1 u sum p |v| + u |o| covers the rounded weights, the rounded result and the fp32 sums (under 2^-11 of
sum p |v| here); rows 8 * 2^-24 of the largest intermediate plus half a step.
"""
import math

import pytest

pytestmark = pytest.mark.gpu
SEEN = 0x40000000


@pytest.fixture(scope="module")
def torch():
    import torch as t

    if not t.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__

    __graft_entry__.build()
    return t


@pytest.mark.parametrize("packed,T", [(False, 0), (True, 1)])
def test_rounds_with_pages_and_penalties(torch, packed, T):
    import dynamic_draft_tree_gb300 as dt
    from dynamic_draft_tree_gb300.paged import PagedCache, TokenState
    from dynamic_draft_tree_gb300.rounds import RoundRunner

    B, V, K, k, D, m, layers, H_q, H_kv, Dh, page = 3, 1500, 4, 4, 3, 16, 2, 8, 2, 64, 16
    P, D_path = m + 1, D + 1
    g = torch.Generator(device="cuda")
    g.manual_seed(5 + T)
    i32 = dict(dtype=torch.int32, device="cuda")
    run = RoundRunner("eagle", B, V, K, k, D, P, D_path, m, dt.DT_F32, T=T, packed=packed)
    h = run.h
    kv = PagedCache(h, B, P, layers, H_q, H_kv, Dh, n_blocks=40, max_blocks=12, page=page, D_path=D_path, packed=packed)
    rep = torch.tensor([1.3, 1.0, 0.9], device="cuda")
    freq = torch.tensor([0.2, 0.0, 0.5], device="cuda")
    bias_ids = torch.randint(0, V, (B, 5), generator=g, **i32)
    bias_vals = torch.randn(B, 5, generator=g, device="cuda")
    allow = torch.randint(-2 ** 31, 2 ** 31, (B * P, (V + 31) // 32), generator=g, device="cuda",
                          dtype=torch.int64).to(torch.int32)
    state = TokenState(h, B, repetition=rep, frequency=freq, bias_ids=bias_ids, bias_vals=bias_vals,
                       allow=allow if packed else allow.view(B, P, -1))
    # prompts
    n0 = [37, 0, 16]
    off = [0, 37, 37, 53]
    d_off, d_n0 = torch.tensor(off, **i32), torch.tensor(n0, **i32)
    prompt_kv = torch.randn(2 * layers, 53, H_kv, Dh, generator=g, device="cuda").bfloat16()
    prompt_tok = torch.randint(0, V, (53,), generator=g, **i32)
    kv.prefill(prompt_kv, d_n0, d_off)
    state.prompt(prompt_tok, d_n0, row_off=d_off)
    dense = [prompt_kv[:, off[b]:off[b + 1]] for b in range(B)]
    counts = torch.zeros(B, V, dtype=torch.int64)
    for b in range(B):
        for t in prompt_tok[off[b]:off[b + 1]].tolist():
            counts[b, t] |= SEEN
    roots = torch.randint(0, V, (B,), generator=g, **i32)
    out_w = torch.randn(H_q * Dh, V, generator=g, device="cuda") * 0.3
    seen = {}

    def draft_rows(d, ftok):
        return torch.randn(B, 1 if d == 1 else k, V, generator=g, device="cuda")

    def target_rows(meta):
        shape = (B * P,) if packed else (B, P)
        x = 0.0
        seen["attn"] = []
        for layer in range(layers):
            q = torch.randn(*shape, H_q, Dh, generator=g, device="cuda").bfloat16()
            kv.tmp[2 * layer:2 * layer + 2] = torch.randn(2, *shape, H_kv, Dh, generator=g, device="cuda").bfloat16()
            o = torch.zeros(*shape, H_q, Dh, device="cuda", dtype=torch.bfloat16)
            kv.attend(layer, q, o, meta)
            seen["attn"].append((q, o))
            x = x + o.float()
        rows = x.flatten(-2) @ out_w
        seen["rows"], seen["logits"] = rows.clone(), rows
        return rows

    for rnd in range(4):
        tmp_before = [x.shape[1] for x in dense]
        run.run(roots, draft_rows, target_rows, seed=11, rnd=rnd, kv=kv, tokens=state)
        assert dt.dt_get_status(h) in (0, dt.DT_DEV_BAD_LOGITS)  # a grammar may leave a verified row nothing
        meta = run.meta.numpy()
        acc, path = run.accept_len.tolist(), run.accept_path.tolist()
        flat = lambda x: x if packed else x.flatten(0, 1)  # noqa: E731
        for b in range(B):
            n = int(meta["n_pos"][b])
            r0 = int(meta["row_off"][b]) if packed else b * P
            mask = torch.from_numpy(meta["mask"][b, :n, :n].copy()).cuda().bool()
            L = tmp_before[b]
            for layer, (q, o) in enumerate(seen["attn"]):
                tk, tv = (flat(kv.tmp[2 * layer + j])[r0:r0 + n] for j in (0, 1))
                key = torch.cat([dense[b][2 * layer], tk]).double().repeat_interleave(H_q // H_kv, 1)
                val = torch.cat([dense[b][2 * layer + 1], tv]).double().repeat_interleave(H_q // H_kv, 1)
                ok = torch.cat([torch.ones(n, L, dtype=torch.bool, device="cuda"), mask], 1)
                z = torch.einsum("ihd,jhd->hij", flat(q)[r0:r0 + n].double(), key) * Dh ** -0.5
                p = torch.softmax(z.masked_fill(~ok, -math.inf), -1)
                want = torch.einsum("hij,jhd->ihd", p, val)
                size = torch.einsum("hij,jhd->ihd", p, val.abs())
                got = flat(o)[r0:r0 + n].double()
                assert float(((got - want).abs() - (2.1 * size + want.abs()) * 2.0 ** -8).max()) <= 0
            for i in range(n):
                x = flat(seen["rows"])[r0 + i].double().cpu()
                c = (counts[b] & (SEEN - 1)).clone()
                for j in range(n):
                    if meta["mask"][b, i, j] and meta["tokens"][b, j] >= 0:
                        c[int(meta["tokens"][b, j])] += 1
                known = (c > 0) | (counts[b] >= SEEN)
                r = float(rep[b])
                y = torch.where(known, torch.where(x > 0, x / r, x * r), x) - float(freq[b]) * c
                extra = torch.zeros(V, dtype=torch.float64)
                for t, v in zip(bias_ids[b].tolist(), bias_vals[b].tolist()):
                    y[t] += v
                    extra[t] += abs(v)
                words = allow[r0 + i].cpu()
                v = torch.arange(V)
                can = (words[v >> 5] >> (v & 31)) & 1 == 1
                got = flat(seen["logits"])[r0 + i].double().cpu()
                assert torch.isinf(got[~can]).all() and (got[~can] < 0).all()
                tol = 8 * 2.0 ** -24 * (x.abs() * max(r, 1 / r) + float(freq[b]) * c + extra) + 2.0 ** -24 * y.abs()
                assert float(((got - y).abs() - tol)[can].max()) <= 0
            # commits
            rows = [r0 + p_ for p_ in path[b][:acc[b] + 1]]
            dense[b] = torch.cat([dense[b], kv.tmp[:, rows] if packed else
                                  kv.tmp[:, b, path[b][:acc[b] + 1]]], 1)
            for p_ in path[b][:acc[b] + 1]:
                counts[b, int(meta["tokens"][b, p_])] += 1
        assert kv.seq_len.tolist() == [x.shape[1] for x in dense]
        assert torch.equal(state.counts.cpu().long(), counts)
        for b in range(B):
            n = dense[b].shape[1]
            blocks = kv.pool.block_table[b, :-(-n // page)].long()
            assert (blocks >= 0).all()
            have = kv.pages[:, blocks].flatten(1, 2)[:, :n]
            assert torch.equal(have, dense[b])
        roots = run.bonus.clone()
    # every request ends: all pages come back
    kv.release(torch.zeros(B, **i32))
    assert int(kv.pool.free_count) == 40 and sorted(kv.pool.free_list.tolist()) == list(range(40))
    h.close()


def test_committed_round_in_a_graph(torch):
    """Reserve, commit and count captured once and replayed: lengths, pages and counts advance with every replay."""
    import dynamic_draft_tree_gb300 as dt
    from dynamic_draft_tree_gb300.paged import PagedCache, TokenState

    B, P, V = 2, 5, 64
    i32 = dict(dtype=torch.int32, device="cuda")
    h = dt.Handle(B, V, 1, 1, 1, P)
    kv = PagedCache(h, B, P, 1, 2, 1, 64, n_blocks=12, max_blocks=6, page=8, D_path=4)
    state = TokenState(h, B)
    meta = dt.Meta(B, P, 4)
    meta.tokens.copy_(torch.arange(B * P, **i32).view(B, P))
    acc = torch.tensor([3, 0], **i32)
    path = torch.tensor([[0, 1, 3, 4], [0, -1, -1, -1]], **i32)

    def commit():
        state.commit(acc, path, meta)
        kv.commit(acc, path, meta)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        commit()
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        commit()
    seen = [kv.tmp.clone()]
    for rnd in range(4):
        kv.tmp.copy_(torch.randn_like(kv.tmp))
        seen.append(kv.tmp.clone())
        g.replay()
    torch.cuda.synchronize()
    assert dt.dt_get_status(h) == 0
    assert kv.seq_len.tolist() == [20, 5]
    assert state.counts[0, [0, 1, 3, 4]].tolist() == [5] * 4 and int(state.counts.sum()) == 25
    for b, rows in ((0, [0, 1, 3, 4]), (1, [0])):
        want = torch.cat([x[:, b, rows] for x in seen], 1)
        n = want.shape[1]
        have = kv.pages[:, kv.pool.block_table[b, :-(-n // 8)].long()].flatten(1, 2)[:, :n]
        assert torch.equal(have, want)
    h.close()


def test_prefill_on_another_stream_keeps_its_slots(torch):
    """Memory that the current stream allocates while a prefill waits on another stream is not the prefill's."""
    import dynamic_draft_tree_gb300 as dt
    from dynamic_draft_tree_gb300.paged import PagedCache

    n = 100000
    h = dt.Handle(1, 50, 1, 1, 1, 4)
    kv = PagedCache(h, 1, 4, 1, 1, 1, 16, n_blocks=n // 16 + 1, max_blocks=n // 16 + 1, page=16)
    rows = torch.randn(2, n, 1, 16, device="cuda").bfloat16()
    n_new, off = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([n], [0, n]))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(50_000_000)  # tens of milliseconds
    kv.prefill(rows, n_new, off, stream=side)
    later = [torch.full((n,), -7, dtype=torch.int64, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    assert all(bool((x == -7).all()) for x in later)
    assert dt.dt_get_status(h) == 0 and kv.seq_len.tolist() == [n]
    table = kv.pool.block_table[0, :n // 16].long()
    assert torch.equal(kv.pages[:, table].view(2, -1, 1, 16)[:, :n], rows)
    h.close()


def test_prefill_takes_no_memory_that_another_stream_still_writes(torch):
    """A freed tensor of the current stream, which a delayed kernel there still writes, does not become the slots of a
    prefill on another stream."""
    import dynamic_draft_tree_gb300 as dt
    from dynamic_draft_tree_gb300.paged import PagedCache

    n = 100000
    h = dt.Handle(1, 50, 1, 1, 1, 4)
    kv = PagedCache(h, 1, 4, 1, 1, 1, 16, n_blocks=n // 16 + 1, max_blocks=n // 16 + 1, page=16)
    rows = torch.randn(2, n, 1, 16, device="cuda").bfloat16()
    n_new, off = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([n], [0, n]))
    side = torch.cuda.Stream()
    old = [torch.empty((n,), dtype=torch.int64, device="cuda") for _ in range(4)]
    places = {x.data_ptr() for x in old}
    torch.cuda.synchronize()
    torch.cuda._sleep(50_000_000)  # tens of milliseconds
    for x in old:
        x.fill_(0)  # a slot inside the pages
    x = None
    del old
    again = torch.empty((n,), dtype=torch.int64, device="cuda")
    assert again.data_ptr() in places  # such memory is what an allocation of the current stream gets
    del again
    kv.prefill(rows, n_new, off, stream=side)
    torch.cuda.synchronize()
    assert dt.dt_get_status(h) == 0 and kv.seq_len.tolist() == [n]
    table = kv.pool.block_table[0, :n // 16].long()
    assert torch.equal(kv.pages[:, table].view(2, -1, 1, 16)[:, :n], rows)
    h.close()


@pytest.mark.parametrize("packed", [False, True])
def test_positions_of_a_round_start_behind_the_cache(torch, packed):
    """position_ids = seq_len + depth in every round, captured and replayed too: the root follows the cached tokens."""
    import dynamic_draft_tree_gb300 as dt
    from dynamic_draft_tree_gb300.paged import PagedCache
    from dynamic_draft_tree_gb300.rounds import RoundRunner

    B, V, K, k, D, m = 3, 700, 4, 4, 3, 12
    P, D_path = m + 1, D + 1
    i32 = dict(dtype=torch.int32, device="cuda")
    run = RoundRunner("eagle", B, V, K, k, D, P, D_path, m, dt.DT_F32, packed=packed)
    kv = PagedCache(run.h, B, P, 1, 2, 1, 32, n_blocks=60, max_blocks=12, page=16, D_path=D_path, packed=packed)
    n0 = [33, 0, 16]
    kv.prefill(torch.randn(2, 49, 1, 32, device="cuda").bfloat16(), torch.tensor(n0, **i32),
               torch.tensor([0, 33, 33, 49], **i32))
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    draft = [torch.randn(B, k, V, generator=g, device="cuda") for _ in range(D + 1)]
    rows = torch.randn(*((B * P,) if packed else (B, P)), V, generator=g, device="cuda")
    roots = torch.randint(0, V, (B,), generator=g, **i32)

    def one():
        run.run(roots, lambda d, t: draft[d][:, :1].contiguous() if d == 1 else draft[d], lambda meta: rows, kv=kv)

    def check(before):
        assert dt.dt_get_status(run.h) == 0
        meta = run.meta.numpy()
        for b in range(B):
            n = int(meta["n_pos"][b])
            assert meta["position_ids"][b, :n].tolist() == [before[b] + int(d) for d in meta["depth"][b, :n]]
            assert (meta["position_ids"][b, n:] == -1).all()
        after = kv.seq_len.tolist()
        assert after == [x + a + 1 for x, a in zip(before, run.accept_len.tolist())]
        return after

    before = n0
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        one()
    side.synchronize()
    before = check(before)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        one()
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        before = check(before)
    run.h.close()


@pytest.mark.parametrize("packed", [False, True])
def test_a_request_without_pages_keeps_its_length_and_its_history(torch, packed):
    """One request's commits find no free page: neither its length nor its counts move, the other's both do."""
    import dynamic_draft_tree_gb300 as dt
    from dynamic_draft_tree_gb300.paged import PagedCache, TokenState
    from dynamic_draft_tree_gb300.rounds import RoundRunner

    B, V, K, k, D, m, page = 2, 400, 4, 4, 2, 8, 8
    P, D_path = m + 1, D + 1
    i32 = dict(dtype=torch.int32, device="cuda")
    run = RoundRunner("eagle", B, V, K, k, D, P, D_path, m, dt.DT_F32, packed=packed)
    # request 0 has room in its page for two rounds and more; request 1's page is full, and there is no third one
    kv = PagedCache(run.h, B, P, 1, 2, 1, 32, n_blocks=2, max_blocks=4, page=page, D_path=D_path, packed=packed)
    state = TokenState(run.h, B, repetition=torch.full((B,), 1.2, device="cuda"))
    kv.prefill(torch.randn(2, 9, 1, 32, device="cuda").bfloat16(), torch.tensor([1, 8], **i32), torch.tensor([0, 1, 9], **i32))
    assert kv.seq_len.tolist() == [1, 8] and int(kv.pool.free_count) == 0
    g = torch.Generator(device="cuda")
    g.manual_seed(9)
    roots = torch.tensor([5, 6], **i32)
    want = torch.zeros(B, V, dtype=torch.int64)
    length = 1
    for rnd in range(2):
        run.run(roots, lambda d, t: torch.randn(B, 1 if d == 1 else k, V, generator=g, device="cuda"),
                lambda meta: torch.randn(*((B * P,) if packed else (B, P)), V, generator=g, device="cuda"), rnd=rnd, kv=kv,
                tokens=state)
        assert dt.dt_get_status(run.h) == dt.DT_DEV_KV_FULL
        dt.dt_clear_status(run.h)
        acc, path, tok = int(run.accept_len[0]), run.accept_path[0].tolist(), run.meta.tokens[0].tolist()
        for p in path[:acc + 1]:
            want[0, tok[p]] += 1
        length += acc + 1
        assert kv.seq_len.tolist() == [length, 8] and kv.committed.tolist() == [acc + 1, 0]
        assert torch.equal(state.counts.cpu().long(), want)
    run.h.close()


@pytest.mark.parametrize("B,shared,side", [(3, 32, False), (3, 32, True), (24, 2048, False)])
def test_requests_behind_a_shared_prefix(torch, B, shared, side):
    """The prefix is in the pool once, every request attends to it, it outlives the request in place 0, and a request that
    ends gives back its own pages alone. (24 requests behind 2048 tokens: the prefix as work of its own.)"""
    import types

    import dynamic_draft_tree_gb300 as dt
    from dynamic_draft_tree_gb300.paged import PagedCache

    H_q, H_kv, D, page, P = 8, 2, 64, 16, 3
    ns = shared // page
    r = torch.Generator(device="cuda")
    r.manual_seed(B)
    i32 = dict(dtype=torch.int32, device="cuda")
    h = dt.Handle(B, 2, 1, 1, 1, P)
    n_blocks = ns + 4 * B
    kv = PagedCache(h, B, P, 1, H_q, H_kv, D, n_blocks=n_blocks, max_blocks=ns + 4, page=page, D_path=P, shared_len=shared)
    randn = lambda *s: torch.randn(*s, generator=r, device="cuda").bfloat16()  # noqa: E731
    stream = torch.cuda.Stream() if side else None
    prefix = randn(2, shared, H_kv, D)
    torch.cuda.synchronize()
    kv.prefix(prefix, stream=stream)
    torch.cuda.synchronize()
    assert dt.dt_get_status(h) == 0
    assert kv.seq_len.tolist() == [shared] * B and int(kv.pool.free_count) == n_blocks - ns
    dense = [prefix for _ in range(B)]
    pages_of = lambda x: -(-x.shape[1] // page)  # noqa: E731

    def append(n):
        off = [0]
        for x in n:
            off.append(off[-1] + x)
        rows = randn(2, off[-1], H_kv, D)
        torch.cuda.synchronize()
        kv.prefill(rows, torch.tensor(n, **i32), torch.tensor(off, **i32), stream=stream)
        torch.cuda.synchronize()
        for b in range(B):
            dense[b] = torch.cat([dense[b], rows[:, off[b]:off[b + 1]]], 1)

    def check():
        meta = types.SimpleNamespace(n_pos=torch.full((B,), P, **i32), mask=None, row_off=None)
        q, out = randn(B, P, H_q, D), torch.zeros(B, P, H_q, D, device="cuda").bfloat16()
        kv.tmp.copy_(randn(*kv.tmp.shape))
        kv.attend(0, q, out, meta)
        assert dt.dt_get_status(h) == 0
        assert kv.seq_len.tolist() == [x.shape[1] for x in dense]
        own = sum(pages_of(x) - ns for x in dense)
        assert int(kv.pool.free_count) == n_blocks - ns - own
        used = [kv.pool.block_table[b, ns:pages_of(dense[b])].tolist() for b in range(B)]
        free = kv.pool.free_list[:int(kv.pool.free_count)].tolist()
        assert sorted(sum(used, free) + kv.pool.block_table[B - 1, :ns].tolist()) == list(range(n_blocks))
        for b in range(B):
            k = torch.cat([dense[b][0], kv.tmp[0, b]]).double().repeat_interleave(H_q // H_kv, 1)
            v = torch.cat([dense[b][1], kv.tmp[1, b]]).double().repeat_interleave(H_q // H_kv, 1)
            z = torch.einsum("ihd,jhd->hij", q[b].double(), k) * D ** -0.5
            L = dense[b].shape[1]
            ok = torch.ones(P, L + P, dtype=torch.bool, device="cuda").tril(L)
            p = torch.softmax(z.masked_fill(~ok, -math.inf), -1)
            want, size = torch.einsum("hij,jhd->ihd", p, v), torch.einsum("hij,jhd->ihd", p, v.abs())
            assert float(((out[b].double() - want).abs() - (2.1 * size + want.abs()) * 2.0 ** -8).max()) <= 0

    append([5 + b % 30 for b in range(B)])
    check()
    # the requests in places 0 and 2 end, others go on; new ones take their places
    keep = kv.seq_len.clone()
    keep[0] = keep[2] = 0
    torch.cuda.synchronize()
    kv.release(keep, stream=stream)
    torch.cuda.synchronize()
    kv.seq_len[0] = kv.seq_len[2] = shared
    dense[0] = dense[2] = prefix
    check()
    append([20 if b in (0, 2) else b % 2 for b in range(B)])
    check()
    kv.release(torch.zeros(B, **i32))
    assert int(kv.pool.free_count) == n_blocks - ns and dt.dt_get_status(h) == 0
    h.close()


def test_a_prefix_without_pages_changes_nothing(torch):
    import dynamic_draft_tree_gb300 as dt
    from dynamic_draft_tree_gb300.paged import PagedCache

    h = dt.Handle(2, 2, 1, 1, 1, 1)
    kv = PagedCache(h, 2, 1, 1, 1, 1, 16, n_blocks=2, max_blocks=4, page=8, shared_len=24)
    kv.prefix(torch.ones(2, 24, 1, 16, device="cuda").bfloat16())
    assert dt.dt_get_status(h) == dt.DT_DEV_KV_FULL
    assert kv.seq_len.tolist() == [0, 0] and kv.pool.n_owned.tolist() == [0, 0] and int(kv.pool.free_count) == 2
    assert bool((kv.pool.block_table == -1).all()) and not bool(kv.pages.any())
    h.close()


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("T", [0, 1])
def test_a_round_verifies_the_processed_rows(torch, packed, T):
    """Accepted paths and bonus tokens are those of the oracle on rows processed in 64 bits by the definition. The target's
    favourite among a position's children is one that the grammar forbids for every other row, so that verifying the raw rows
    would go another way (held on the oracle too). With T = 1 requests with a decision closer than 1e-4 are left out: the
    kernel's rows are within 1e-5 of the reference here."""
    import numpy as np

    import dynamic_draft_tree_gb300 as dt
    from dynamic_draft_tree_gb300.paged import TokenState
    from dynamic_draft_tree_gb300.rounds import RoundRunner
    from oracle.verify import verify_greedy, verify_sample

    B, V, K, k, D, m = 8, 1100, 4, 4, 4, 24
    P, D_path, seed, rnd = m + 1, D + 1, 17, 3
    i32 = dict(dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda")
    g.manual_seed(40 + T)
    run = RoundRunner("eagle", B, V, K, k, D, P, D_path, m, dt.DT_F32, T=T, packed=packed)
    rep, freq = torch.rand(B, generator=g, device="cuda") * 0.4 + 1, torch.rand(B, generator=g, device="cuda")
    allow = torch.full((B * P, (V + 31) // 32), -1, **i32)
    state = TokenState(run.h, B, repetition=rep, frequency=freq, allow=allow if packed else allow.view(B, P, -1))
    seen = {}

    def target_rows(meta):
        rows = torch.randn(B * P, V, generator=g, device="cuda")
        mt = meta.numpy()
        for b in range(B):
            r0 = int(mt["row_off"][b]) if packed else b * P
            for i in range(int(mt["n_pos"][b])):
                kids = [j for j in range(1, int(mt["n_pos"][b])) if mt["parents"][b, j] == i]
                for rank, j in enumerate(kids[:2]):
                    t = int(mt["tokens"][b, j])
                    rows[r0 + i, t] = 14.0 - 3.0 * rank
                    if rank == 0 and (b + i) % 2:
                        word = int(allow[r0 + i, t >> 5]) & 0xFFFFFFFF & ~(1 << (t & 31))
                        allow[r0 + i, t >> 5] = word - 2 ** 32 if word >= 2 ** 31 else word
        seen["raw"] = rows.clone()
        return rows if packed else rows.view(B, P, V)

    draft = [torch.randn(B, k, V, generator=g, device="cuda") * 3 for _ in range(D + 1)]
    roots = torch.randint(0, V, (B,), generator=g, **i32)
    run.run(roots, lambda d, t: draft[d][:, :1].contiguous() if d == 1 else draft[d], target_rows, seed=seed, rnd=rnd,
            tokens=state)
    assert dt.dt_get_status(run.h) == 0
    mt = run.meta.numpy()
    raw, words = seen["raw"].double().cpu().numpy(), allow.cpu().numpy()
    v = np.arange(V)
    near = {}

    class Gaps:
        def add(self, kind, gap, scale, b):
            near[b] = min(near.get(b, 1.0), abs(gap))

    def row_at(b, i):
        return (int(mt["row_off"][b]) if packed else b * P) + i

    def processed(b, i):
        x, c = raw[row_at(b, i)], np.zeros(V)
        for j in range(int(mt["n_pos"][b])):
            if mt["mask"][b, i, j]:
                c[mt["tokens"][b, j]] += 1
        r = float(rep[b])
        y = np.where(c > 0, np.where(x > 0, x / r, x * r), x) - float(freq[b]) * c
        can = (words[row_at(b, i)][v >> 5] >> (v & 31)) & 1 == 1
        return np.where(can, y, -np.inf)

    verify = (lambda rows: verify_greedy(mt, rows)) if T == 0 else (lambda rows: verify_sample(mt, rows, seed, rnd, Gaps()))
    want = verify(processed)
    clear = [b for b in range(B) if near.get(b, 1.0) > 1e-4]
    assert len(clear) > B // 2
    got = (run.accept_len.cpu().numpy(), run.accept_path.cpu().numpy(), run.bonus.cpu().numpy())
    for name, a, o in zip(("accept_len", "accept_path", "bonus"), got, want):
        np.testing.assert_array_equal(a[clear], o[clear], err_msg=name)
    other = verify(lambda b, i: raw[row_at(b, i)])
    assert sum(not np.array_equal(want[1][b], other[1][b]) for b in clear) >= 2  # the raw rows go another way
    run.h.close()


def test_one_position_a_request_in_rows_of_any_distance(torch):
    """P = 1: queries, keys and values cut out of one projection, heads before positions, and the last position of padded
    logits are rows as they stand; the dimension of one position has any stride."""
    import dynamic_draft_tree_gb300 as dt

    B, H_q, H_kv, D, page, V = 5, 8, 2, 64, 16, 320
    i32 = dict(dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    h = dt.Handle(B, V, 1, 1, 1, 4)
    ws = dt.dt_tree_attention_workspace(h, B, 1, H_q, H_kv, D)
    kp, vp = randn(2 * B, page, H_kv, D), randn(2 * B, page, H_kv, D)
    table = torch.arange(2 * B, **i32).view(B, 2)
    lens, one = torch.tensor([0, 1, 17, 30, 32], **i32), torch.ones(B, **i32)
    fused = randn(B, (H_q + 2 * H_kv) * D)
    q, k, v = (x.view(B, 1, -1, D) for x in fused.split([H_q * D, H_kv * D, H_kv * D], 1))
    assert q.stride(0) != q.stride(1)
    heads_first = torch.zeros(B, H_q, 1, D, device="cuda").bfloat16()

    def attend(q, k, v, out):
        dt.dt_tree_attention(h, q, k, v, kp, vp, table, lens, one, out, ws)
        return out

    want = attend(*(x.contiguous().clone() for x in (q, k, v)), torch.zeros(B, 1, H_q, D, device="cuda").bfloat16())
    assert torch.equal(attend(q, k, v, heads_first.transpose(1, 2)), want)
    wide = randn(B, 3, H_q, D)
    before = wide.clone()
    assert torch.equal(attend(q, k, v, wide[:, 1:2]), want)
    before[:, 1:2] = want
    assert torch.equal(wide, before)
    # rows of logits
    logits = torch.randn(B, 4, V, generator=g, device="cuda").bfloat16()
    rep = torch.full((B,), 1.5, device="cuda")
    tokens = logits[:, -1].argmax(1, keepdim=True).to(torch.int32)
    flat = torch.zeros(B, 1, V, device="cuda").bfloat16()
    dt.dt_logits_process(h, logits[:, -1:].clone(), flat, one, tokens=tokens, repetition=rep)
    assert not torch.equal(flat, logits[:, -1:])
    before = logits.clone()
    dt.dt_logits_process(h, logits[:, -1:], logits[:, -1:], one, tokens=tokens, repetition=rep)
    before[:, -1:] = flat
    assert torch.equal(logits, before)
    # rows of keys and values
    tmp = randn(2, B, 3, H_kv, D)
    slots = torch.arange(3, 3 + 7 * B, 7, dtype=torch.int64, device="cuda").view(B, 1)
    caches = [torch.zeros(2, 3, page, H_kv, D, device="cuda").bfloat16() for _ in range(2)]
    for x, cache in zip((tmp[:, :, 1:2], tmp[:, :, 1:2].clone()), caches):
        dt.dt_commit_kv_paged(h, x, cache, slots, one, lens, torch.zeros(B, **i32))
    rows = caches[0].flatten(1, 2)[:, slots.view(-1)]
    assert torch.equal(rows, tmp[:, :, 1]) and torch.equal(*caches)
    # more positions are still held against their distance
    with pytest.raises(ValueError):
        dt.dt_logits_process(h, logits[:, 1:3], logits[:, 1:3], one)
    with pytest.raises(ValueError):
        dt.dt_commit_kv_paged(h, tmp[:, :, :2], caches[0], slots, one, lens, torch.zeros(B, **i32))
    assert dt.dt_get_status(h) == 0
    h.close()
