"""A request's life around the rounds: prompts in chunks, samples that continue one prompt, answers with log probabilities.

The prompts' attention runs layer by layer before its rows are appended, in two chunks; then requests are forked, drawn rounds are
verified with a paged cache on all of them, and some end. A shadow holds every request's keys and values densely. Attention is
compared with the definition in 64 bits with the operators' tolerance (u = 2^-8 of bf16: 2.1 u sum p |v| + u |o| covers
rounded weights, the rounded result and fp32 sums, under 2^-11 of sum p |v| here); log probabilities with log_softmax in
64 bits: fp32 logits below 64 in absolute value have sums off by less than 2^-24 (0.7 (60 + 93) + 49) < 2^-16.6, so
2^-16 + 2^-23 |logp|; what is owned, lengths and copied rows exactly.
"""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    import torch as t

    if not t.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__

    __graft_entry__.build()
    return t


def _attention(t, q, key, val, ok, got):
    """q [n][H][D] against key, val [L][H_kv][D] where ok [n][L]; got within the tolerance."""
    G = q.shape[1] // key.shape[1]
    key, val = (x.double().repeat_interleave(G, 1) for x in (key, val))
    z = t.einsum("ihd,jhd->hij", q.double(), key) * q.shape[2] ** -0.5
    p = t.softmax(z.masked_fill(~ok, float("-inf")), -1)
    want, size = t.einsum("hij,jhd->ihd", p, val), t.einsum("hij,jhd->ihd", p, val.abs())
    assert float(((got.double() - want).abs() - (2.1 * size + want.abs()) * 2.0 ** -8).max()) <= 0


@pytest.mark.parametrize("packed,shared", [(False, 0), (True, 32)])
def test_prompts_samples_and_answers(torch, packed, shared):
    import dynamic_draft_tree_gb300 as dt
    from dynamic_draft_tree_gb300.paged import PagedCache, TokenLogprobs
    from dynamic_draft_tree_gb300.rounds import RoundRunner

    t = torch
    B, V, K, k, D, m, layers, H_q, H_kv, Dh, page = 6, 1500, 4, 4, 3, 16, 2, 8, 2, 64, 16
    P, D_path = m + 1, D + 1
    g = t.Generator(device="cuda")
    g.manual_seed(17 + shared)
    i32 = lambda v: t.tensor(v, dtype=t.int32, device="cuda")
    randn = lambda *s: t.randn(*s, generator=g, device="cuda").bfloat16()
    run = RoundRunner("eagle", B, V, K, k, D, P, D_path, m, dt.DT_F32, T=0, packed=packed)
    h = run.h
    kv = PagedCache(h, B, P, layers, H_q, H_kv, Dh, n_blocks=80, max_blocks=16, page=page, D_path=D_path, packed=packed,
                    shared_len=shared, forks=True)
    answers = TokenLogprobs(h, B, D_path, K=3)
    dense = [t.zeros(2 * layers, 0, H_kv, Dh, device="cuda", dtype=t.bfloat16) for _ in range(B)]
    if shared:
        x = randn(2 * layers, shared, H_kv, Dh)
        kv.prefix(x)
        dense = [x for _ in range(B)]
    # prompts of requests 0 and 1 in two chunks (the others have no rows)
    for chunk in ([70, 9, 0, 0, 0, 0], [1, 30, 0, 0, 0, 0]):
        off = [0]
        for n in chunk:
            off.append(off[-1] + n)
        rows = randn(2 * layers, off[-1], H_kv, Dh)
        for layer in range(layers):
            q, out = randn(off[-1], H_q, Dh), t.zeros(off[-1], H_q, Dh, device="cuda", dtype=t.bfloat16)
            kv.attend_prompts(layer, q, rows[2 * layer], rows[2 * layer + 1], i32(off), out)
            for b in range(2):
                r, L, n = slice(off[b], off[b + 1]), dense[b].shape[1], chunk[b]
                ok = t.arange(L + n, device="cuda")[None, :] <= L + t.arange(n, device="cuda")[:, None]
                _attention(t, q[r], t.cat([dense[b][2 * layer], rows[2 * layer, r]]),
                           t.cat([dense[b][2 * layer + 1], rows[2 * layer + 1, r]]), ok, out[r])
        kv.prefill(rows, i32(chunk), i32(off))
        dense = [t.cat([dense[b], rows[:, off[b]:off[b + 1]]], 1) for b in range(B)]
    assert kv.seq_len.tolist() == [shared + 71, shared + 39] + [shared] * 4
    # samples: two of request 0, one of request 1 behind its first 20 tokens; place 5 stays idle
    kv.fork(i32([0, 0, 1]), i32([2, 4, 3]), i32([shared + 71, shared + 71, shared + 20]))
    dense[2], dense[4], dense[3] = dense[0], dense[0], dense[1][:, :shared + 20]
    assert dt.dt_get_status(h) == 0
    out_w = t.randn(H_q * Dh, V, generator=g, device="cuda") * 0.3
    seen = {}

    def draft_rows(d, ftok):
        return t.randn(B, 1 if d == 1 else k, V, generator=g, device="cuda")

    def target_rows(meta):
        shape = (B * P,) if packed else (B, P)
        x, seen["attn"] = 0.0, []
        for layer in range(layers):
            q, o = randn(*shape, H_q, Dh), t.zeros(*shape, H_q, Dh, device="cuda", dtype=t.bfloat16)
            kv.tmp[2 * layer:2 * layer + 2] = randn(2, *shape, H_kv, Dh)
            kv.attend(layer, q, o, meta)
            seen["attn"].append((q, o))
            x = x + o.float()
        seen["rows"] = x.flatten(-2) @ out_w
        return seen["rows"]

    flat = lambda x: x if packed else x.flatten(0, 1)  # noqa: E731
    for rnd in range(3):
        run.run(t.randint(0, V, (B,), generator=g, dtype=t.int32, device="cuda"), draft_rows, target_rows, seed=3, rnd=rnd, kv=kv,
                logprobs=answers)
        assert dt.dt_get_status(h) == 0
        meta, acc, path, bonus = run.meta.numpy(), run.accept_len.tolist(), run.accept_path.tolist(), run.bonus.tolist()
        for b in range(B):
            n = int(meta["n_pos"][b])
            r0 = int(meta["row_off"][b]) if packed else b * P
            ok = t.cat([t.ones(n, dense[b].shape[1], dtype=t.bool, device="cuda"),
                        t.from_numpy(meta["mask"][b, :n, :n].copy()).cuda().bool()], 1)
            for layer, (q, o) in enumerate(seen["attn"]):
                tk, tv = (flat(kv.tmp[2 * layer + j])[r0:r0 + n] for j in (0, 1))
                _attention(t, flat(q)[r0:r0 + n], t.cat([dense[b][2 * layer], tk]), t.cat([dense[b][2 * layer + 1], tv]), ok,
                           flat(o)[r0:r0 + n])
            pos = path[b][:acc[b] + 1]
            for j, p in enumerate(pos):
                x = flat(seen["rows"])[r0 + p].double()
                assert float(x.abs().max()) < 64
                z = t.log_softmax(x, 0)
                tok = int(meta["tokens"][b, pos[j + 1]]) if j + 1 < len(pos) else bonus[b]
                assert abs(float(answers.logp[b, j]) - float(z[tok])) <= 2.0 ** -16 + 2.0 ** -23 * abs(float(z[tok]))
                order = t.sort(x, descending=True, stable=True).indices
                assert int(answers.rank[b, j]) == int((order == tok).nonzero())
                assert answers.top_ids[b, j].tolist() == order[:3].tolist()
            dense[b] = t.cat([dense[b], t.stack([flat(kv.tmp[x])[[r0 + p for p in pos]] for x in range(2 * layers)])], 1)
            assert int(kv.seq_len[b]) == dense[b].shape[1]
        if rnd == 1:  # the first sample ends, and the idle place goes; the prompt is sampled once more
            keep = kv.seq_len.clone()
            keep[2] = keep[5] = shared
            kv.release(keep)
            kv.seq_len[2] = kv.seq_len[5] = shared
            kv.fork(i32([0]), i32([5]))
            dense[2], dense[5] = dense[2][:, :shared], dense[0]
    # every request's pages hold its rows
    table = kv.pool.block_table
    for b in range(B):
        L = dense[b].shape[1]
        at = t.arange(L, device="cuda")
        got = kv.pages[:, table[b, (at // page).long()].long(), at % page]
        assert t.equal(got, dense[b])
    # all end: nothing is lost, nothing is counted
    kv.release(t.zeros(B, dtype=t.int32, device="cuda"))
    assert int(kv.pool.free_count) == 80 - shared // page and not kv.refs.any() and dt.dt_get_status(h) == 0
    h.close()


def test_a_cache_without_forks_refuses_them(torch):
    import dynamic_draft_tree_gb300 as dt
    from dynamic_draft_tree_gb300.paged import PagedCache

    h = dt.Handle(2, 2, 1, 1, 1, 4)
    kv = PagedCache(h, 2, 4, 1, 2, 1, 16, n_blocks=8, max_blocks=4)
    one = torch.zeros(1, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        kv.fork(one, one + 1)
    h.close()
