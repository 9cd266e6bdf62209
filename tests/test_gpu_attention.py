"""dt_tree_attention against the definition in 64 bits, through the Python binding.

Tolerance, per output element: with p the exact weights (sum 1), A = sum_j p_j |v_j| and u half a step of the
type (bf16 2^-8, fp16 2^-11): the weights are rounded to the type before the second product (u A), the result
once (u |o|); the scores are fp32 sums of D products, off by at most d = (D + 8) 2^-24 max_j scale sum |q k|,
which changes weights by a factor within 1 +- 2 d (and the normaliser likewise), and 2^-18 covers exp2 and the
fp32 sums over up to 2^13 keys: (4 d + 2^-18) A. fp16 weights below the smallest normal number are off by at most
2^-25 of a weight that is at least 2^6 for the largest: 2^-31 sum_j |v_j|.
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


def _up(a, b):
    return -(-a // b)


class Problem:
    """A random paged attention problem; everything that must not be read into a result holds NaN."""

    def __init__(self, t, B, P, H_kv, G, D, page, lens, n_pos=None, shared=0, packed=False, tree=True, dtype="bf16",
                 seed=0, heads_first=False, max_blocks=None, q_scale=2.0, spare=3):
        g = t.Generator(device="cuda")
        g.manual_seed(seed * 1000003 + B * 7919 + P * 31 + D + sum(lens))
        dt_ = {"bf16": t.bfloat16, "fp16": t.float16}[dtype]
        self.t, self.B, self.P, self.G, self.page, self.shared, self.lens, self.D = t, B, P, G, page, shared, lens, D
        self.n = list(n_pos) if n_pos is not None else [P] * B
        ns = shared // page
        need = [_up(x, page) - ns for x in lens]
        self.max_blocks = max_blocks or max(1, max(_up(x, page) for x in lens))
        n_blocks = ns + sum(need) + spare
        perm = t.randperm(n_blocks, generator=g, device="cuda").tolist()
        table, at = [], ns
        for b in range(B):
            table.append(perm[:ns] + perm[at:at + need[b]] + [-1] * (self.max_blocks - ns - need[b]))
            at += need[b]
        for b in range(1, B):  # only the first request's entries of shared pages are read
            table[b][:ns] = [-1 - b] * ns
        self.table = t.tensor(table, dtype=t.int32, device="cuda")
        table = [table[0][:ns] + row[ns:] for row in table]
        nan = float("nan")
        shape = (n_blocks, H_kv, page, D) if heads_first else (n_blocks, page, H_kv, D)
        pages = [t.full(shape, nan, dtype=dt_, device="cuda") for _ in range(2)]
        self.kp, self.vp = (x.transpose(1, 2) if heads_first else x for x in pages)
        self.off = [0]
        for k in self.n:
            self.off.append(self.off[-1] + k)
        rows = self.off[-1] + 5 if packed else B * P
        self.base = [self.off[b] if packed else b * P for b in range(B)]
        H = H_kv * G
        self.q = (t.randn(rows, H, D, generator=g, device="cuda") * q_scale).to(dt_)
        self.kn, self.vn = (t.full((rows, H_kv, D), nan, dtype=dt_, device="cuda") for _ in range(2))
        self.out = t.full((rows, H, D), 7.0, dtype=dt_, device="cuda")
        self.k, self.v = [], []
        for b in range(B):
            for kind, pg, new in ((self.k, self.kp, self.kn), (self.v, self.vp, self.vn)):
                x = t.randn(lens[b] + self.n[b], H_kv, D, generator=g, device="cuda").to(dt_)
                if shared and b:
                    x[:shared] = kind[0][:shared]
                for e in range(_up(lens[b], page)):
                    m = min(page, lens[b] - e * page)
                    pg[table[b][e], :m] = x[e * page:e * page + m]
                new[self.base[b]:self.base[b] + self.n[b]] = x[lens[b]:]
                kind.append(x)
        self.mask = None
        if tree:
            self.mask = t.zeros(B, P, P, dtype=t.uint8, device="cuda")
            import random
            r = random.Random(seed + P)
            m = [[[0] * P for _ in range(P)] for _ in range(B)]
            for b in range(B):
                for i in range(self.n[b]):
                    if i:
                        p = r.randint(max(0, i - 6), i - 1)
                        m[b][i] = list(m[b][p])
                    m[b][i][i] = 1
            self.mask = t.tensor(m, dtype=t.uint8, device="cuda")
        self.row_off = t.tensor(self.off, dtype=t.int32, device="cuda") if packed else None
        self.seq_len = t.tensor(lens, dtype=t.int32, device="cuda")
        self.n_pos = t.tensor(self.n, dtype=t.int32, device="cuda")
        self.packed, self.scale = packed, D ** -0.5

    def views(self):
        if self.packed:
            return self.q, self.kn, self.vn, self.out
        return tuple(x.view(self.B, self.P, *x.shape[1:]) for x in (self.q, self.kn, self.vn, self.out))

    def call(self, dt, h, ws, stream=None):
        q, kn, vn, out = self.views()
        dt.dt_tree_attention(h, q, kn, vn, self.kp, self.vp, self.table, self.seq_len, self.n_pos, out, ws,
                             mask=self.mask, row_off=self.row_off, P=self.P, shared_len=self.shared,
                             scale=self.scale, stream=stream)

    def handle(self, dt):
        h = dt.Handle(self.B, 2, 1, 1, 1, self.P)
        H = self.q.shape[1]
        return h, dt.dt_tree_attention_workspace(h, self.B, self.P, H, H // self.G, self.D, shared=self.shared > 0)

    def reference(self):
        """(out, tolerance) in 64 bits; rows of no position keep what they had (tolerance 0)."""
        t = self.t
        out, tol = self.out.double().clone(), t.zeros(self.out.shape, dtype=t.float64, device="cuda")
        u = t.finfo(self.q.dtype).eps / 2
        for b in range(self.B):
            L, n, r0 = self.lens[b], self.n[b], self.base[b]
            ok = t.ones(n, L + n, dtype=t.bool, device="cuda")
            ok[:, L:] = self.mask[b, :n, :n].bool() if self.mask is not None else ok[:, L:].tril()
            some = ok.any(1, keepdim=True)
            for x in range(self.q.shape[1]):
                q = self.q[r0:r0 + n, x].double()
                k, v = self.k[b][:, x // self.G].double(), self.v[b][:, x // self.G].double()
                z = (q @ k.T * self.scale).masked_fill(~ok, -math.inf)
                p = t.softmax(t.where(some, z, 0.0), 1) * some
                # a weight of zero leaves a value out, whatever it holds
                o = t.where(ok[:, :, None], p[:, :, None] * v[None], 0.0).sum(1)
                a = t.where(ok[:, :, None], p[:, :, None] * v[None].abs(), 0.0).sum(1)
                d = (self.D + 8) * 2.0 ** -24 * (t.where(ok, q.abs() @ k.abs().T, 0.0) * self.scale).amax(1, keepdim=True)
                out[r0:r0 + n, x] = o
                tol[r0:r0 + n, x] = (u + 4 * d + 2.0 ** -18) * a * 1.01 + u * o.abs() + \
                    2.0 ** -31 * t.where(ok[:, :, None], v[None].abs(), 0.0).sum(1)
        return out, tol


def _check(pr, got):
    t = pr.t
    want, tol = pr.reference()
    got = got.double()
    assert t.equal(t.isnan(got), t.isnan(want)), "NaN in other places"
    inf = t.isinf(want)
    assert t.equal(got[inf], want[inf])
    fine = t.isfinite(want)
    off = ((got - want).abs() - tol)[fine]
    assert off.numel() == 0 or float(off.max()) <= 0.0, f"beyond the tolerance by {float(off.max()):.3g}"


CASES = {
    "one token": dict(B=1, P=1, H_kv=2, G=4, D=128, page=16, lens=[37], tree=False),
    "one token, empty cache": dict(B=2, P=1, H_kv=1, G=1, D=64, page=16, lens=[0, 1], tree=False),
    "tile borders": dict(B=6, P=1, H_kv=2, G=2, D=128, page=16, lens=[127, 128, 129, 255, 256, 257], tree=False),
    "page 8": dict(B=3, P=2, H_kv=2, G=3, D=64, page=8, lens=[7, 8, 200], tree=False),
    "page 256": dict(B=2, P=5, H_kv=1, G=8, D=128, page=256, lens=[255, 700]),
    "page 128": dict(B=2, P=5, H_kv=2, G=2, D=128, page=128, lens=[128, 515], dtype="fp16"),
    "tree behind the last tokens": dict(B=7, P=9, H_kv=2, G=2, D=128, page=8, lens=[1, 8, 9, 111, 112, 113, 239]),
    "tree behind the last tokens, boxes that do not fit": dict(B=5, P=61, H_kv=1, G=4, D=64, page=16,
                                                               lens=[63, 64, 65, 48, 193], n_pos=[61, 61, 3, 61, 64 - 3]),
    "chain behind the last tokens": dict(B=6, P=30, H_kv=1, G=2, D=64, page=32, lens=[1, 31, 33, 95, 96, 97], tree=False,
                                         n_pos=[30, 1, 17, 30, 30, 30], dtype="fp16"),
    "tree behind the last tokens, shared": dict(B=4, P=9, H_kv=2, G=2, D=64, page=16, lens=[50, 49, 100, 48], shared=48),
    "pr1 tree": dict(B=1, P=17, H_kv=8, G=4, D=128, page=16, lens=[515]),
    "cast tree packed": dict(B=4, P=61, H_kv=2, G=4, D=128, page=64, lens=[1000, 3, 0, 64], n_pos=[61, 17, 40, 1],
                             packed=True),
    "padded ragged": dict(B=3, P=33, H_kv=3, G=5, D=80, page=32, lens=[100, 0, 77], n_pos=[33, 5, 20], dtype="fp16"),
    "no positions": dict(B=3, P=9, H_kv=2, G=2, D=128, page=16, lens=[40, 50, 60], n_pos=[4, 0, 9], packed=True),
    "group of 7": dict(B=2, P=19, H_kv=2, G=7, D=96, page=16, lens=[300, 31]),
    "group of 128": dict(B=1, P=3, H_kv=1, G=128, D=64, page=16, lens=[90]),
    "more than 256 rows": dict(B=2, P=85, H_kv=2, G=4, D=128, page=16, lens=[513, 20], n_pos=[85, 70]),
    "more than 128 positions": dict(B=2, P=300, H_kv=1, G=2, D=64, page=32, lens=[65, 200], n_pos=[300, 131]),
    "heads of their own": dict(B=3, P=40, H_kv=5, G=1, D=64, page=16, lens=[70, 0, 300], n_pos=[40, 13, 33]),
    "heads of their own, shared": dict(B=9, P=40, H_kv=3, G=1, D=128, page=16, lens=[260 + i for i in range(9)],
                                       shared=256, packed=True, n_pos=[40, 1, 7, 40, 22, 40, 3, 39, 40]),
    "512 positions": dict(B=1, P=512, H_kv=1, G=1, D=128, page=64, lens=[130], tree=False),
    "head size 8": dict(B=2, P=3, H_kv=2, G=2, D=8, page=16, lens=[50, 5]),
    "head size 72": dict(B=2, P=3, H_kv=2, G=2, D=72, page=16, lens=[50, 5], dtype="fp16"),
    "head size 120": dict(B=2, P=3, H_kv=1, G=2, D=120, page=16, lens=[500, 5]),
    "heads first": dict(B=2, P=7, H_kv=4, G=2, D=128, page=32, lens=[190, 33], heads_first=True),
    "long": dict(B=2, P=3, H_kv=1, G=4, D=128, page=64, lens=[8191, 5000]),
    "many requests": dict(B=67, P=2, H_kv=1, G=2, D=64, page=16, lens=[(7 * i) % 150 for i in range(67)]),
    "more requests than threads": dict(B=801, P=2, H_kv=1, G=2, D=64, page=16, lens=[(11 * i) % 97 for i in range(801)],
                                       n_pos=[1 + i % 2 for i in range(801)], packed=True),
    "more requests than threads, shared": dict(B=500, P=1, H_kv=2, G=1, D=64, page=16, tree=False,
                                               lens=[64 + i % 40 for i in range(500)], shared=64),
    "shared": dict(B=5, P=21, H_kv=2, G=4, D=128, page=32, lens=[256, 257, 300, 400, 256], shared=256, packed=True,
                   n_pos=[21, 3, 10, 21, 1]),
    "shared, odd pages": dict(B=4, P=9, H_kv=2, G=5, D=80, page=16, lens=[48, 49, 200, 112], shared=48, dtype="fp16"),
    "shared, one token": dict(B=40, P=1, H_kv=2, G=4, D=128, page=64, lens=[640 + i for i in range(40)], shared=640,
                              tree=False),
    "shared long": dict(B=9, P=33, H_kv=1, G=4, D=64, page=16, lens=[2048 + 9 * i for i in range(9)], shared=2048),
    "shared, read with the own tokens": dict(B=3, P=5, H_kv=2, G=4, D=128, page=16, lens=[64, 100, 64], shared=64),
    "shared, many rows": dict(B=48, P=9, H_kv=4, G=3, D=64, page=32, lens=[1024 + 5 * i for i in range(48)], shared=1024,
                              n_pos=[1 + i % 9 for i in range(48)], packed=True),
    "shared, long and few": dict(B=4, P=1, H_kv=1, G=8, D=128, page=64, lens=[8192, 8200, 8300, 8192], shared=8192,
                                 tree=False),
    "weak scores": dict(B=2, P=9, H_kv=2, G=2, D=128, page=16, lens=[900, 30], q_scale=0.01),
    "sharp scores": dict(B=2, P=9, H_kv=2, G=2, D=128, page=16, lens=[900, 30], q_scale=40.0),
}


@pytest.mark.parametrize("name", list(CASES))
def test_attention_matches_definition(torch, name):
    import dynamic_draft_tree_gb300 as dt

    pr = Problem(torch, **CASES[name])
    h, ws = pr.handle(dt)
    ws.fill_(0xFF)  # the workspace needs no initial value
    pr.call(dt, h, ws)
    assert dt.dt_get_status(h) == 0
    first = pr.out.clone()
    want_out = torch.full_like(first, 7.0)
    pr.out.copy_(want_out)
    _check(pr, first)
    pr.call(dt, h, ws)  # again on the used workspace: the same bits
    torch.cuda.synchronize()
    assert torch.equal(first, pr.out)
    h.close()


def test_rows_whose_mask_leaves_nothing(torch):
    import dynamic_draft_tree_gb300 as dt

    pr = Problem(torch, B=3, P=12, H_kv=2, G=4, D=128, page=16, lens=[0, 40, 0], n_pos=[12, 12, 5])
    pr.mask[:, 1::3] = 0
    h, ws = pr.handle(dt)
    pr.call(dt, h, ws)
    assert dt.dt_get_status(h) == 0
    got = pr.out.clone()
    pr.out.fill_(7.0)
    _check(pr, got)
    assert (got[1] == 0).all() and (got[4] == 0).all()  # positions 1 and 4 of the request without a cache
    h.close()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("shared", [0, 32])
def test_values_of_masked_positions_do_not_reach_other_rows(torch, bad, shared):
    """One branch's keys and values overflow: only the rows that attend to it show it."""
    import dynamic_draft_tree_gb300 as dt

    pr = Problem(torch, B=2, P=20, H_kv=2, G=4, D=64, page=16, lens=[40, 33], shared=shared)
    m = pr.mask[0]
    j = next(c for c in range(19, 0, -1) if 1 < int(m[:, c].sum()) < 12)  # a position with a few descendants
    row = pr.base[0] + j
    pr.vn[row, :, 5] = bad
    pr.v[0][pr.lens[0] + j, :, 5] = bad
    pr.kn[pr.base[0] + 19] = bad if int(m[:, 19].sum()) == 1 else pr.kn[pr.base[0] + 19]
    pr.k[0][pr.lens[0] + 19] = pr.kn[pr.base[0] + 19]
    h, ws = pr.handle(dt)
    pr.call(dt, h, ws)
    got = pr.out.clone()
    pr.out.fill_(7.0)
    sees = m[:, j].bool()
    clean = ~sees & ~m[:, 19].bool()
    o = got.view(2, 20, *got.shape[1:])[0]
    assert torch.isfinite(o[clean]).all()
    assert not torch.isfinite(o[sees][..., 5]).any()
    want, tol = pr.reference()
    d = (got.double() - want).abs() - tol
    keep = clean[:, None, None] & torch.ones_like(o, dtype=torch.bool)
    assert float(d.view(2, 20, *got.shape[1:])[0][keep].max()) <= 0
    only = sees & ~m[:, 19].bool()  # these rows' other elements are numbers as before
    rest = d.view(2, 20, *got.shape[1:])[0][only]
    assert float(torch.cat([rest[..., :5], rest[..., 6:]], -1).max()) <= 0
    h.close()


def test_strided_inputs_and_other_stream(torch):
    """q, k and v as slices of one projection, the output inside a wider buffer, on a side stream."""
    import dynamic_draft_tree_gb300 as dt

    pr = Problem(torch, B=3, P=13, H_kv=2, G=4, D=64, page=16, lens=[70, 5, 129], n_pos=[13, 4, 9], packed=True)
    rows, H, D = pr.q.shape
    wide = torch.zeros(rows, H + 4, D + 8, dtype=pr.q.dtype, device="cuda")
    fused = wide[:, :, :D]
    fused[:, :H], fused[:, H:H + 2], fused[:, H + 2:] = pr.q, pr.kn, pr.vn
    out = torch.full((rows, 2 * H, D), 7.0, dtype=pr.q.dtype, device="cuda")[:, ::2]
    h, ws = pr.handle(dt)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    dt.dt_tree_attention(h, fused[:, :H], fused[:, H:H + 2], fused[:, H + 2:], pr.kp, pr.vp, pr.table, pr.seq_len,
                         pr.n_pos, out, ws, mask=pr.mask, row_off=pr.row_off, scale=pr.scale, stream=side)
    side.synchronize()
    _check(pr, out)
    pr.call(dt, h, ws)
    torch.cuda.synchronize()
    assert torch.equal(out, pr.out)
    h.close()


def test_captured_graph_follows_the_lengths(torch):
    """A captured call replayed after the lengths, the tables and the contents changed."""
    import dynamic_draft_tree_gb300 as dt

    kw = dict(B=4, P=15, H_kv=2, G=4, D=128, page=16, packed=False, max_blocks=64)
    pr = Problem(torch, lens=[30, 600, 2, 0], spare=60, **kw)
    h, ws = pr.handle(dt)
    pr.call(dt, h, ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pr.call(dt, h, ws)
    other = Problem(torch, lens=[1000, 3, 77, 0], n_pos=[15, 1, 7, 15], seed=9, **kw)
    for name in ("table", "seq_len", "n_pos", "mask", "q", "kn", "vn"):
        getattr(pr, name).copy_(getattr(other, name))
    m = other.kp.shape[0]  # fewer pages than the captured buffers have
    pr.kp[:m].copy_(other.kp)
    pr.vp[:m].copy_(other.vp)
    pr.out.fill_(7.0)
    g.replay()
    torch.cuda.synchronize()
    _check(other, pr.out)
    h.close()


def test_bad_tables_are_reported(torch):
    """A block id outside the pages and a length past the table set the status; nothing outside is read."""
    import dynamic_draft_tree_gb300 as dt

    pr = Problem(torch, B=2, P=3, H_kv=1, G=2, D=64, page=16, lens=[40, 40])
    h, ws = pr.handle(dt)
    pr.table[1, 1] = pr.kp.shape[0]
    pr.call(dt, h, ws)
    assert dt.dt_get_status(h) & dt.DT_DEV_BAD_PAGE
    dt.dt_clear_status(h)
    pr.table[1, 1] = 0
    pr.seq_len[1] = 49  # three blocks in the table
    pr.call(dt, h, ws)
    assert dt.dt_get_status(h) & dt.DT_DEV_BAD_PAGE
    h.close()


def test_idle_places_need_no_shared_prefix(torch):
    """A place without positions and tokens among requests behind a shared prefix is no error; one with positions is."""
    import dynamic_draft_tree_gb300 as dt

    for shared in (64, 4096):
        pr = Problem(torch, B=6, P=5, H_kv=8, G=4, D=64, page=16, lens=[shared + 9 * b for b in range(6)],
                     n_pos=[5, 0, 3, 5, 0, 1], shared=shared)
        h, ws = pr.handle(dt)
        pr.seq_len[1] = 0
        pr.seq_len[4] = 0
        pr.call(dt, h, ws)
        assert dt.dt_get_status(h) == 0
        got = pr.out.clone()
        pr.out.fill_(7.0)
        _check(pr, got)
        pr.seq_len[5] = shared - 1
        pr.call(dt, h, ws)
        assert dt.dt_get_status(h) == dt.DT_DEV_BAD_PAGE
        h.close()


@pytest.mark.parametrize("shared", [0, 2048])
def test_rows_past_a_packed_batchs_end(torch, shared):
    """A request whose rows do not end within the packed batch (row_off[B]) sets the status and writes nothing; the
    others keep their results. Behind a prefix read once for all rows, such rows are no item's."""
    import dynamic_draft_tree_gb300 as dt

    B = 32 if shared else 3
    pr = Problem(torch, B=B, P=17, H_kv=8, G=4, D=64, page=16, lens=[shared + 5 + b for b in range(B)], packed=True,
                 shared=shared)
    h, ws = pr.handle(dt)
    pr.row_off[B] = pr.off[B] - 1
    pr.call(dt, h, ws)
    assert dt.dt_get_status(h) == dt.DT_DEV_BAD_PAGE
    dt.dt_clear_status(h)
    got = pr.out.clone()
    assert bool((got[pr.off[B - 1]:] == 7.0).all())
    pr.out.fill_(7.0)
    want, tol = pr.reference()
    n = pr.off[B - 1]
    assert bool(((got[:n].double() - want[:n]).abs() <= tol[:n]).all())
    # a first row far behind the batch, within the buffers
    far = 40 * n
    big = [torch.zeros(far + 17, *x.shape[1:], dtype=x.dtype, device="cuda") for x in (pr.q, pr.kn, pr.vn, pr.out)]
    pr.q, pr.kn, pr.vn, pr.out = big
    pr.row_off[B] = pr.off[B]
    pr.row_off[B - 1] = far
    pr.call(dt, h, ws)
    assert dt.dt_get_status(h) == dt.DT_DEV_BAD_PAGE
    assert bool((pr.out[n:] == 0.0).all())
    h.close()


def test_waits_that_run_out_are_reported(torch):
    """With DT_FLAG_TEST_TIMEOUT no wait is taken: the call ends, says so, and the context stays usable."""
    import dynamic_draft_tree_gb300 as dt

    for case in ("cast tree packed", "one token", "shared"):
        pr = Problem(torch, **CASES[case])
        h = dt.Handle(pr.B, 2, 1, 1, 1, pr.P, flags=dt.DT_FLAG_TEST_TIMEOUT)
        _, ws = pr.handle(dt)
        ws.zero_()
        pr.call(dt, h, ws)
        assert dt.dt_get_status(h) & dt.DT_DEV_TIMEOUT
        h.close()
        h, ws = pr.handle(dt)
        pr.out.fill_(7.0)
        pr.call(dt, h, ws)
        assert dt.dt_get_status(h) == 0
        got = pr.out.clone()
        pr.out.fill_(7.0)
        _check(pr, got)
        h.close()


def test_refusals(torch):
    import dynamic_draft_tree_gb300 as dt

    pr = Problem(torch, B=2, P=4, H_kv=2, G=2, D=64, page=16, lens=[20, 30])
    h, ws = pr.handle(dt)
    q, kn, vn, out = pr.views()
    args = dict(h=h, q=q, k_new=kn, v_new=vn, k_pages=pr.kp, v_pages=pr.vp, block_table=pr.table, seq_len=pr.seq_len,
                n_pos=pr.n_pos, out=out, workspace=ws, mask=pr.mask)

    def no(error, **over):
        with pytest.raises(error):
            dt.dt_tree_attention(**dict(args, **over))

    no(ValueError, q=q.float())
    no(ValueError, k_new=kn.half())
    no(ValueError, seq_len=pr.seq_len.long())
    no(ValueError, mask=pr.mask[:, :3])
    no(ValueError, out=out[:1])
    no(ValueError, q=q.cpu())
    no(ValueError, n_pos=pr.n_pos[:1].expand(3))
    no(dt.DtError, workspace=ws[:128])
    no(dt.DtError, workspace=ws[16:])
    no(dt.DtError, shared_len=8)
    no(dt.DtError, scale=float("nan"))
    no(dt.DtError, scale=-1.0)
    no(dt.DtError, k_pages=pr.kp[:, :12], v_pages=pr.vp[:, :12])
    big = dt.Handle(1, 2, 1, 1, 1, 4)
    no(dt.DtError, h=big)  # B > B_max
    odd = torch.zeros(2 * 4 * 4 * 68, dtype=q.dtype, device="cuda")
    no(dt.DtError, q=odd.view(2, 4, 4, 68)[..., :64])  # a head stride of 68 elements
    dt.dt_tree_attention(**args)
    assert dt.dt_get_status(h) == 0
    h.close()


def test_clear_status_takes_back_arrivals(torch):
    """A handle with arrivals left at its split items, as after a call that gave up, is fit again after dt_clear_status."""
    import dynamic_draft_tree_gb300 as dt

    pr = Problem(torch, B=2, P=2, H_kv=2, G=4, D=64, page=16, lens=[6000, 2500])
    _, ws = pr.handle(dt)
    h = dt.Handle(pr.B, 2, 1, 1, 1, pr.P, flags=dt.DT_FLAG_TEST_ARRIVED)
    dt.dt_clear_status(h)
    pr.out.fill_(7.0)
    want, tol = pr.reference()
    for _ in range(3):
        ws.fill_(255)  # parts that are read before they are written are no numbers
        pr.out.fill_(7.0)
        pr.call(dt, h, ws)
        assert dt.dt_get_status(h) == 0
        assert bool(((pr.out.double() - want).abs() <= tol).all())
    h.close()


def test_workspace_goes_by_the_cuts(torch):
    """Without a shared prefix a CTA's run cuts two items at most: a larger batch needs no more room for parts, and what it
    has is enough, to the byte, for batches whose items are many and long."""
    import dynamic_draft_tree_gb300 as dt

    h = dt.Handle(1024, 2, 1, 1, 1, 64)
    need = {B: dt.dt_tree_attention_workspace(h, B, 61, 32, 8, 64).numel() for B in (64, 256, 1024)}
    assert need[1024] - need[64] <= 2 * 4 * (1024 - 64) + 512 and need[256] <= need[1024]
    small = dt.dt_tree_attention_workspace(h, 1, 61, 32, 8, 64).numel()  # eight items: one slot each and one a CTA
    assert small < need[64]
    h.close()
    r = __import__("random").Random(4)
    for B, P, G, page in ((64, 40, 4, 32), (40, 9, 3, 16), (300, 1, 4, 16)):
        pr = Problem(torch, B=B, P=P, H_kv=8, G=G, D=64, page=page, lens=[r.randint(0, 700) for _ in range(B)], packed=True,
                     n_pos=[r.randint(0, P) for _ in range(B)])
        h, ws = pr.handle(dt)
        room = torch.full((ws.numel() + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
        want, tol = pr.reference()
        pr.call(dt, h, room[:ws.numel()])
        assert dt.dt_get_status(h) == 0
        assert bool(((pr.out.double() - want).abs() <= tol).all())
        assert bool((room[ws.numel():] == 0xA5).all())
        h.close()


def test_results_repeat_exactly(torch):
    """The cuts follow from the lengths and parts are joined in a fixed order: two calls give the same bits."""
    import dynamic_draft_tree_gb300 as dt

    for case in (dict(B=2, P=2, H_kv=2, G=4, D=64, page=16, lens=[6000, 2500]),  # joined by the CTA that comes last
                 dict(B=5, P=40, H_kv=3, G=5, D=80, page=32, lens=[3000, 1, 0, 777, 1500]),  # by the second launch
                 dict(B=32, P=17, H_kv=8, G=4, D=64, page=16, lens=[2048 + 9 * b for b in range(32)], shared=2048)):
        pr = Problem(torch, **case)
        h, ws = pr.handle(dt)
        pr.call(dt, h, ws)
        first = pr.out.clone()
        for _ in range(4):
            pr.out.fill_(7.0)
            ws.fill_(255)
            pr.call(dt, h, ws)
            assert torch.equal(pr.out.view(torch.int16), first.view(torch.int16))
        assert dt.dt_get_status(h) == 0
        h.close()
