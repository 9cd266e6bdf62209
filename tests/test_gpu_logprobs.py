"""dt_token_logprobs against the definition in 64 bits, through the Python binding.

Tolerance: an exponent x log2 e - m log2 e is an fp32 multiply-add with a rounded second term, off by at most
2^-24 (|d| + 1.45 |m|) (d the exponent, m the row's largest logit in absolute value; weights with |d| > 60 add less than
2^-40 of the sum for 2^20 tokens), which changes a weight by ln 2 times that; ex2 is off by 2^-22, and a sum of 32 terms a thread, five
and three levels of trees and the scaling between them by at most 45 roundings: together a factor within
1 +- u, u = 2^-24 (0.7 (60 + 1.45 |m|) + 4 + 45) of S. log S is then off by u (and 2^-22 for the fp32 logarithm of the mantissa), logp
by that and its own rounding 2^-24 |logp|. The entropy's second sum has weights off by u and factors d off by
2^-24 (|d| + 1.45 |m|): u (1 + 2 H) + 2^-24 (60 + 1.45 |m|) covers both, with u for log S. Whole numbers are equal.
"""
import math

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


class Problem:
    def __init__(self, t, form, used, V, K, dtype="bf16", packed=False, n=None, seed=0, P=None, ld=None, spread=3.0, ties=False,
                 masked=0.0, S=None):
        g = t.Generator(device="cuda")
        g.manual_seed(seed * 7919 + V + K + sum(used))
        self.t, self.form, self.used, self.V, self.K, self.packed = t, form, list(used), V, K, packed
        B, P = len(used), P or max(used)
        self.B, self.P = B, P
        self.off = [0]
        for u in used:
            self.off.append(self.off[-1] + u)
        rows = self.off[-1] + 3 if packed else B * P
        dt_ = {"bf16": t.bfloat16, "fp32": t.float32}[dtype]
        ld = ld or V
        buf = t.full((rows * ld,), float("nan"), dtype=dt_, device="cuda")  # rows that are not read may hold anything
        self.rows = buf.view(rows, ld)[:, :V]
        self.base = [self.off[b] if packed else b * P for b in range(B)]
        for b in range(B):
            x = t.randn(used[b], V, generator=g, device="cuda") * spread
            if ties:
                x = (x * 2).round() / 2
            if masked:
                x.masked_fill_(t.rand(used[b], V, generator=g, device="cuda") < masked, -math.inf)
            self.rows[self.base[b]:self.base[b] + used[b]] = x.to(dt_)
        self.logits = self.rows if packed else self.rows.as_strided((B, P, V), (P * ld, ld, 1))
        self.row_off = t.tensor(self.off, dtype=t.int32, device="cuda") if packed else None
        r = lambda *s: t.randint(0, V, s, generator=g, device="cuda", dtype=t.int32)
        self.n = list(n) if n is not None else list(used)
        self.path = None
        if form == "path":
            S = S or max(self.n)
            self.path = t.full((B, S), -1, dtype=t.int32, device="cuda")
            for b in range(B):
                p = [0] + sorted(t.randperm(used[b] - 1, generator=g, device="cuda")[:self.n[b] - 1].add(1).tolist()) if used[b] > 1 else [0]
                self.path[b, :self.n[b]] = t.tensor(p[:self.n[b]], dtype=t.int32)
            self.tokens, out = r(B, P), (B, S)
        else:
            out = (rows,) if packed else (B, P)
            self.tokens = r(*out)
        self.shift = 0 if form == "labels" else 1
        self.last = r(B) if self.shift else None
        self.n_extra = 1 if form == "path" else 0
        self.n_new = t.tensor([k - self.n_extra for k in self.n], dtype=t.int32, device="cuda")
        f = lambda *s: t.full(s, 7.0, device="cuda")
        i = lambda *s: t.full(s, 7, dtype=t.int32, device="cuda")
        self.logp, self.entropy, self.rank = f(*out), f(*out), i(*out)
        self.top_ids, self.top_logp = (i(*out, K), f(*out, K)) if K else (None, None)
        self.outs = out

    def handle(self, dt):
        h = dt.Handle(self.B, self.V, 1, 1, 1, 1, dt.DT_BF16 if self.rows.dtype is self.t.bfloat16 else dt.DT_F32)
        return h, dt.dt_token_logprobs_workspace(h, self.logp.numel(), self.K)

    def call(self, dt, h, ws, **kw):
        a = dict(tokens=self.tokens, last=self.last, shift=self.shift, n_extra=self.n_extra, path=self.path, row_off=self.row_off,
                 entropy=self.entropy, rank=self.rank, top_ids=self.top_ids, top_logp=self.top_logp)
        a.update(kw)
        dt.dt_token_logprobs(h, self.logits, self.n_new, self.logp, ws, **a)

    def entries(self):
        """(output index, row, token) of every entry."""
        tok = self.tokens.reshape(-1).tolist()
        for b in range(self.B):
            pos = self.path[b, :self.n[b]].tolist() if self.path is not None else list(range(self.n[b]))
            for j, p in enumerate(pos):
                if j + self.shift < len(pos):
                    q = pos[j + self.shift]
                    t = tok[b * self.P + q] if self.path is not None else tok[self.base[b] + q]
                else:
                    t = int(self.last[b])
                o = b * self.path.shape[1] + j if self.path is not None else self.base[b] + j
                yield o, self.base[b] + p, t

    def check(self):
        t, K = self.t, self.K
        logp, ent, rank = self.logp.reshape(-1), self.entropy.reshape(-1), self.rank.reshape(-1)
        seen = set()
        ids = self.top_ids.reshape(-1, K) if K else None
        alt = self.top_logp.reshape(-1, K) if K else None
        for o, row, tok in self.entries():
            seen.add(o)
            x = self.rows[row].double()
            z = t.log_softmax(x, 0)
            m = float(x.max().abs())
            u = 2.0 ** -24 * (0.7 * (60 + 1.45 * m) + 49)
            want = float(z[tok])
            got = float(logp[o])
            if want == -math.inf:
                assert got == -math.inf
            else:
                assert abs(got - want) <= u + 2.0 ** -22 + 2.0 ** -24 * abs(want), (o, got, want)
            H = float(-t.special.xlogy(z.exp(), z.exp()).sum())
            tol = u * (2 + 2 * H) + 2.0 ** -22 + 2.0 ** -24 * (60 + 1.45 * m) + 2.0 ** -24 * H
            assert abs(float(ent[o]) - H) <= tol, (o, float(ent[o]), H, tol)
            v = t.arange(self.V, device="cuda")
            assert int(rank[o]) == int(((x > x[tok]) | ((x == x[tok]) & (v < tok))).sum())
            if K:
                order = t.sort(x, descending=True, stable=True)
                some = order.values[:K] > -math.inf
                assert t.equal(ids[o].long(), t.where(some, order.indices[:K], -1)), o
                w = t.where(some, z[order.indices[:K]], -math.inf)
                d = t.where(some, (alt[o].double() - w).abs() - 2.0 ** -24 * w.abs(), 0.0)
                assert float(d.max()) <= u + 2.0 ** -22 and bool((alt[o][~some] == -math.inf).all())
        rest = [k for k in range(logp.numel()) if k not in seen]
        for x in (logp, ent, rank) + ((ids, alt) if K else ()):
            assert bool((x[rest] == 7).all()), "an output of no entry was written"


CASES = {
    "one row": dict(form="path", used=[1], V=32000, K=0),
    "a round": dict(form="path", used=[61, 17, 40, 1], n=[9, 3, 1, 1], V=1000, K=5),
    "a round, packed": dict(form="path", used=[61, 17, 40, 1], n=[9, 3, 1, 1], V=1000, K=5, packed=True),
    "a round, wide paths": dict(form="path", used=[30, 7], n=[4, 7], V=2000, K=1, S=17),
    "prompts": dict(form="next", used=[5, 1, 30], V=5000, K=1, packed=True),
    "prompts, padded": dict(form="next", used=[5, 1, 30], V=5000, K=3),
    "no entries": dict(form="next", used=[5, 4, 30], n=[5, 0, 3], V=5000, K=3, packed=True),
    "labels": dict(form="labels", used=[3, 9], V=700, K=20, dtype="fp32"),
    "labels, packed": dict(form="labels", used=[3, 9], V=700, K=20, dtype="fp32", packed=True),
    "two tokens": dict(form="labels", used=[4], V=2, K=2),
    "fewer than a warp": dict(form="labels", used=[4], V=33, K=32, dtype="fp32"),
    "piece borders": dict(form="labels", used=[3], V=8192, K=7),
    "piece borders, one more": dict(form="labels", used=[9], V=8193, K=7),
    "piece borders, one less, fp32": dict(form="labels", used=[5], V=8191, K=7, dtype="fp32"),
    "odd vocabulary": dict(form="next", used=[9, 8], V=50257, K=20, packed=True),
    "odd vocabulary, fp32": dict(form="next", used=[5, 4], V=128255, K=20, dtype="fp32"),
    "rows further apart": dict(form="next", used=[5, 4], V=1001, K=4, ld=1013),
    "large vocabulary": dict(form="next", used=[3], V=152064, K=32, packed=True),
    "more pieces than lanes": dict(form="labels", used=[3], V=300001, K=32),
    "ties": dict(form="labels", used=[6], V=40000, K=20, ties=True, spread=0.7),
    "all equal": dict(form="labels", used=[3], V=20000, K=20, spread=0.0),
    "grammar": dict(form="labels", used=[6], V=30000, K=20, masked=0.9),
    "grammar that allows a few": dict(form="labels", used=[6], V=30000, K=20, masked=0.9997),
    "one likely token": dict(form="labels", used=[4], V=30000, K=3, spread=60.0, dtype="fp32"),
    "large logits": dict(form="labels", used=[4], V=3000, K=3, spread=3000.0, dtype="fp32"),
    "many requests": dict(form="next", used=[1 + i % 4 for i in range(300)], V=130, K=2, packed=True),
}


@pytest.mark.parametrize("name", list(CASES))
def test_logprobs_match_the_definition(torch, name):
    import dynamic_draft_tree_gb300 as dt

    pr = Problem(torch, **CASES[name])
    h, ws = pr.handle(dt)
    ws.fill_(0xFF)  # the workspace needs no initial value
    pr.call(dt, h, ws)
    assert dt.dt_get_status(h) == 0
    pr.check()
    first = [x.clone() for x in (pr.logp, pr.entropy, pr.rank)]
    pr.call(dt, h, ws)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, (pr.logp, pr.entropy, pr.rank)))
    h.close()


def test_parts_may_be_left_out(torch):
    import dynamic_draft_tree_gb300 as dt

    pr = Problem(torch, form="next", used=[7, 3], V=3000, K=4, packed=True)
    h, ws = pr.handle(dt)
    pr.call(dt, h, ws)
    full = [x.clone() for x in (pr.logp, pr.entropy, pr.rank, pr.top_ids, pr.top_logp)]
    for x in (pr.logp, pr.entropy, pr.rank, pr.top_ids, pr.top_logp):
        x.fill_(7)
    pr.call(dt, h, ws, rank=None, top_ids=None, top_logp=None)
    dt.dt_token_logprobs(h, pr.logits, pr.n_new, None, ws, row_off=pr.row_off, top_ids=pr.top_ids, top_logp=pr.top_logp)
    torch.cuda.synchronize()
    assert (pr.rank == 7).all()
    for k, x in ((0, pr.logp), (1, pr.entropy), (3, pr.top_ids), (4, pr.top_logp)):
        assert torch.equal(x, full[k])
    # no last token: the last entries have none
    pr.call(dt, h, ws, last=None)
    assert dt.dt_get_status(h) == 0
    ends = [pr.base[b] + pr.n[b] - 1 for b in range(pr.B)]
    assert torch.isnan(pr.logp[ends]).all() and (pr.rank[ends] == -1).all()
    keep = [k for k in range(pr.off[-1]) if k not in ends]
    assert torch.equal(pr.logp[keep], full[0][keep]) and torch.equal(pr.entropy[:pr.off[-1]], full[1][:pr.off[-1]])
    h.close()


@pytest.mark.parametrize("bad", ["nan", "inf", "none"])
def test_bad_rows_are_reported(torch, bad):
    import dynamic_draft_tree_gb300 as dt

    pr = Problem(torch, form="labels", used=[5], V=20000, K=4)
    h, ws = pr.handle(dt)
    if bad == "none":
        pr.rows[2] = -math.inf
    else:
        pr.rows[2, 17000] = float(bad)
    pr.call(dt, h, ws)
    assert dt.dt_get_status(h) == dt.DT_DEV_BAD_LOGITS
    logp, ent, rank = (x.view(-1) for x in (pr.logp, pr.entropy, pr.rank))
    assert math.isnan(logp[2]) and math.isnan(ent[2]) and rank[2] == -1 and (pr.top_ids[0, 2] == -1).all()
    assert (pr.top_logp[0, 2] == -math.inf).all()
    ok = [0, 1, 3, 4]
    assert torch.isfinite(logp[ok]).all() and (rank[ok] >= 0).all()
    h.close()


def test_bad_tokens_and_positions_are_reported(torch):
    import dynamic_draft_tree_gb300 as dt

    pr = Problem(torch, form="path", used=[9, 5], n=[4, 3], V=3000, K=2)
    h, ws = pr.handle(dt)

    def status():
        for x in (pr.logp, pr.entropy, pr.rank):
            x.fill_(7)
        pr.call(dt, h, ws)
        bits = dt.dt_get_status(h)
        dt.dt_clear_status(h)
        return bits

    assert status() == 0
    at = int(pr.path[0, 1])
    keep = int(pr.tokens[0, at])
    for token in (3000, -2):
        pr.tokens[0, at] = token
        assert status() == dt.DT_DEV_BAD_TOKEN
        assert math.isnan(pr.logp[0, 0]) and pr.rank[0, 0] == -1 and math.isfinite(pr.entropy[0, 0])
    pr.tokens[0, at] = -1  # no token: no error
    assert status() == 0 and math.isnan(pr.logp[0, 0])
    pr.tokens[0, at] = keep
    for pos in (9, -1, 1 << 30):
        was = int(pr.path[1, 2])
        pr.path[1, 2] = pos
        assert status() == dt.DT_DEV_BAD_TREE
        assert pr.logp[1, 2] == 7 and math.isfinite(pr.logp[1, 0])
        pr.path[1, 2] = was
    pr.n_new[1] = 4  # five entries, four places
    assert status() == dt.DT_DEV_BAD_TREE and (pr.logp[1] == 7).all()
    pr.n_new[1] = -5
    assert status() == dt.DT_DEV_BAD_TREE
    h.close()


def test_captured_graph_and_other_stream(torch):
    import dynamic_draft_tree_gb300 as dt

    pr = Problem(torch, form="path", used=[20, 9], n=[6, 2], V=9000, K=5, packed=True)
    h, ws = pr.handle(dt)
    pr.call(dt, h, ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pr.call(dt, h, ws)
    other = Problem(torch, form="path", used=[14, 15], n=[3, 6], V=9000, K=5, packed=True, seed=3, P=20)
    for name in ("rows", "row_off", "path", "tokens", "last", "n_new"):
        getattr(pr, name).copy_(getattr(other, name))
    for x in (pr.logp, pr.entropy, pr.rank, pr.top_ids, pr.top_logp):
        x.fill_(7)
    g.replay()
    torch.cuda.synchronize()
    pr.off, pr.base, pr.n, pr.used = other.off, other.base, other.n, other.used
    pr.check()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for x in (pr.logp, pr.entropy, pr.rank, pr.top_ids, pr.top_logp):
        x.record_stream(side)
    before = pr.logp.clone()
    with torch.cuda.stream(side):
        pr.logp.fill_(7)
    pr.call(dt, h, ws, stream=side)
    side.synchronize()
    assert torch.equal(before, pr.logp)
    h.close()


def test_refusals(torch):
    import dynamic_draft_tree_gb300 as dt

    pr = Problem(torch, form="path", used=[9, 5], n=[4, 3], V=3000, K=2)
    h, ws = pr.handle(dt)
    for bad in (dict(tokens=pr.tokens.long()), dict(tokens=pr.tokens[:, :4]), dict(path=pr.path[0]), dict(last=pr.last[:1]),
                dict(rank=pr.logp), dict(top_ids=pr.top_ids[..., :1]), dict(top_logp=None), dict(entropy=pr.entropy[:1]),
                dict(row_off=torch.zeros(3, dtype=torch.int32, device="cuda")), dict(tokens=pr.tokens.cpu())):
        with pytest.raises(ValueError):
            pr.call(dt, h, ws, **bad)
    for bad in (dict(shift=2), dict(n_extra=-1), dict(tokens=None, last=None)):
        with pytest.raises(dt.DtError) as e:
            pr.call(dt, h, ws, **bad)
        assert e.value.code == dt.DT_ERR_ARG
    with pytest.raises(dt.DtError):
        pr.call(dt, h, ws[:256])
    with pytest.raises(dt.DtError):
        dt.dt_token_logprobs_workspace(h, 10, 33)
    with pytest.raises(dt.DtError):
        dt.dt_token_logprobs_workspace(h, 0, 1)
    torch.cuda.synchronize()
    assert (pr.logp == 7).all() and dt.dt_get_status(h) == 0
    h.close()
