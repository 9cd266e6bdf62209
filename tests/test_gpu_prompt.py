"""dt_prompt_attention against the definition in 64 bits, through the Python binding.

Tolerance, per output element: with p the exact weights (sum 1), A = sum_j p_j |v_j| and u half a step of the
type (bf16 2^-8, fp16 2^-11): the weights are rounded to the type before the second product (u A), the result
once (u |o|); the scores are fp32 sums of D products, off by at most d = (D + 8) 2^-24 max_j scale sum |q k|,
which changes weights by a factor within 1 +- 2 d (and the normaliser likewise), and 2^-18 covers exp2 and the
fp32 sums over up to 2^14 keys: (4 d + 2^-18) A. fp16 weights below the smallest normal number are off by at most
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
    """Packed prompts behind cached tokens; everything that must not be read into a result holds NaN."""

    def __init__(self, t, n, H_kv, G, D, lens=None, page=16, dtype="bf16", seed=0, heads_first=False, max_blocks=None,
                 q_scale=2.0, spare=3, room=5, lead=0):
        g = t.Generator(device="cuda")
        g.manual_seed(seed * 1000003 + len(n) * 7919 + D + sum(n) + sum(lens or [0]))
        dt_ = {"bf16": t.bfloat16, "fp16": t.float16}[dtype]
        self.t, self.n, self.G, self.D, self.page, self.B = t, list(n), G, D, page, len(n)
        self.cached = lens is not None
        self.lens = list(lens) if lens is not None else [0] * len(n)
        self.off = [lead]
        for k in n:
            self.off.append(self.off[-1] + k)
        rows, H, nan = self.off[-1] + room, H_kv * G, float("nan")
        self.q = t.full((rows, H, D), nan, dtype=dt_, device="cuda")
        self.q[lead:self.off[-1]] = (t.randn(sum(n), H, D, generator=g, device="cuda") * q_scale).to(dt_)
        self.kn, self.vn = (t.full((rows, H_kv, D), nan, dtype=dt_, device="cuda") for _ in range(2))
        self.out = t.full((rows, H, D), 7.0, dtype=dt_, device="cuda")
        self.row_off = t.tensor(self.off, dtype=t.int32, device="cuda")
        need = [_up(x, page) for x in self.lens]
        self.max_blocks = max_blocks or max(1, max(need))
        n_blocks = sum(need) + spare
        perm = t.randperm(n_blocks, generator=g, device="cuda").tolist()
        shape = (n_blocks, H_kv, page, D) if heads_first else (n_blocks, page, H_kv, D)
        pages = [t.full(shape, nan, dtype=dt_, device="cuda") for _ in range(2)]
        self.kp, self.vp = (x.transpose(1, 2) if heads_first else x for x in pages)
        table, at, self.k, self.v = [], 0, [], []
        for b in range(self.B):
            row = perm[at:at + need[b]]
            at += need[b]
            table.append(row + [-1] * (self.max_blocks - need[b]))
            for kind, pg, new in ((self.k, self.kp, self.kn), (self.v, self.vp, self.vn)):
                x = t.randn(self.lens[b] + n[b], H_kv, D, generator=g, device="cuda").to(dt_)
                for e in range(need[b]):
                    m = min(page, self.lens[b] - e * page)
                    pg[row[e], :m] = x[e * page:e * page + m]
                new[self.off[b]:self.off[b + 1]] = x[self.lens[b]:]
                kind.append(x)
        self.table = t.tensor(table, dtype=t.int32, device="cuda")
        self.seq_len = t.tensor(self.lens, dtype=t.int32, device="cuda")
        self.scale = D ** -0.5

    def handle(self, dt, **kw):
        h = dt.Handle(self.B, 2, 1, 1, 1, 1, **kw)
        H = self.q.shape[1]
        return h, dt.dt_prompt_attention_workspace(h, self.B, H, H // self.G, self.D)

    def call(self, dt, h, ws, **kw):
        if self.cached:
            kw = dict(k_pages=self.kp, v_pages=self.vp, block_table=self.table, seq_len=self.seq_len, **kw)
        dt.dt_prompt_attention(h, self.q, self.kn, self.vn, self.row_off, self.out, ws, scale=self.scale, **kw)

    def reference(self, rows=256):
        """(out, tolerance) in 64 bits; rows of no request keep what they had (tolerance 0)."""
        t = self.t
        out, tol = self.out.double().clone(), t.zeros(self.out.shape, dtype=t.float64, device="cuda")
        u = t.finfo(self.q.dtype).eps / 2
        for b in range(self.B):
            L, n, r0 = self.lens[b], self.n[b], self.off[b]
            for x in range(self.q.shape[1]):
                for i0 in range(0, n, rows):
                    i1 = min(n, i0 + rows)
                    k, v = self.k[b][:L + i1, x // self.G].double(), self.v[b][:L + i1, x // self.G].double()
                    q = self.q[r0 + i0:r0 + i1, x].double()
                    ok = t.arange(L + i1, device="cuda")[None, :] <= L + t.arange(i0, i1, device="cuda")[:, None]
                    z = t.where(ok, q @ k.T * self.scale, -math.inf)
                    p = t.softmax(z, 1)
                    fine = t.isfinite(v)
                    vz = t.where(fine, v, 0.0)
                    o, a = p @ vz, p @ vz.abs()
                    if not bool(fine.all()):  # a weight of zero leaves a value out, whatever it holds
                        for j in (~fine).any(1).nonzero()[:, 0].tolist():
                            o = o + t.where(ok[:, j, None] & ~fine[j][None], p[:, j, None] * v[j][None], 0.0)
                    d = (self.D + 8) * 2.0 ** -24 * (t.where(ok, q.abs() @ k.abs().T, 0.0) * self.scale).amax(1, keepdim=True)
                    out[r0 + i0:r0 + i1, x] = o
                    tol[r0 + i0:r0 + i1, x] = (u + 4 * d + 2.0 ** -18) * a * 1.01 + u * o.abs() + \
                        2.0 ** -31 * (ok.double() @ vz.abs())
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
    "one token": dict(n=[1], H_kv=2, G=4, D=128),
    "one token, one cached": dict(n=[1, 1], H_kv=1, G=1, D=64, lens=[0, 1]),
    "short": dict(n=[17], H_kv=8, G=4, D=128),
    "a tile": dict(n=[128], H_kv=2, G=2, D=128),
    "tile borders": dict(n=[127, 128, 129, 255, 256, 257], H_kv=2, G=4, D=64),
    "item borders": dict(n=[63, 64, 65, 31, 32, 33], H_kv=1, G=4, D=128),
    "no rows": dict(n=[0, 5, 0, 0, 70, 0], H_kv=2, G=2, D=64, lens=[3, 0, 100, 0, 20, 0]),
    "rows in front": dict(n=[40, 9], H_kv=2, G=2, D=128, lead=3),
    "no room behind": dict(n=[40, 9], H_kv=2, G=2, D=128, room=0),
    "cached": dict(n=[100, 30, 1], H_kv=2, G=4, D=128, lens=[300, 128, 127]),
    "cached, tile borders": dict(n=[5] * 6, H_kv=1, G=2, D=128, lens=[127, 128, 129, 255, 256, 257], page=8),
    "page 256": dict(n=[40, 200], H_kv=1, G=8, D=128, lens=[255, 700], page=256),
    "page 128": dict(n=[40, 200], H_kv=2, G=2, D=128, lens=[128, 515], page=128, dtype="fp16"),
    "heads first": dict(n=[77, 12], H_kv=4, G=2, D=128, lens=[190, 33], page=32, heads_first=True),
    "odd heads": dict(n=[100, 1, 333], H_kv=3, G=5, D=80, lens=[77, 5, 0], page=32, dtype="fp16"),
    "group of 7": dict(n=[190, 31], H_kv=2, G=7, D=96, lens=[300, 31]),
    "group of 128": dict(n=[9, 3], H_kv=1, G=128, D=64, lens=[90, 0]),
    "group of 65": dict(n=[9, 3], H_kv=1, G=65, D=64),
    "heads of their own": dict(n=[400, 13, 300], H_kv=5, G=1, D=64, lens=[70, 0, 300]),
    "heads of their own, 128": dict(n=[513, 130], H_kv=2, G=1, D=128),
    "head size 8": dict(n=[150, 3], H_kv=2, G=2, D=8, lens=[50, 5]),
    "head size 72": dict(n=[150, 3], H_kv=2, G=2, D=72, lens=[50, 5], dtype="fp16"),
    "head size 120": dict(n=[150, 3], H_kv=1, G=2, D=120, lens=[500, 5]),
    "long": dict(n=[3000], H_kv=2, G=4, D=128),
    "long, fp16": dict(n=[2049, 100], H_kv=1, G=8, D=128, dtype="fp16"),
    "a chunk behind a long cache": dict(n=[64, 1], H_kv=2, G=4, D=128, lens=[9000, 5000], page=64),
    "one token behind a long cache": dict(n=[1], H_kv=1, G=8, D=128, lens=[12345], page=64),
    "many requests": dict(n=[1 + (5 * i) % 40 for i in range(67)], H_kv=1, G=2, D=64, lens=[(7 * i) % 150 for i in range(67)]),
    "more requests than threads": dict(n=[i % 3 for i in range(801)], H_kv=1, G=2, D=64, lens=[(11 * i) % 97 for i in range(801)]),
    "weak scores": dict(n=[300], H_kv=2, G=2, D=128, q_scale=0.01),
    "sharp scores": dict(n=[300], H_kv=2, G=2, D=128, q_scale=40.0),
}


@pytest.mark.parametrize("name", list(CASES))
def test_prompt_attention_matches_definition(torch, name):
    import dynamic_draft_tree_gb300 as dt

    pr = Problem(torch, **CASES[name])
    h, ws = pr.handle(dt)
    ws.fill_(0xFF)  # the workspace needs no initial value
    pr.call(dt, h, ws)
    assert dt.dt_get_status(h) == 0
    first = pr.out.clone()
    pr.out.fill_(7.0)
    _check(pr, first)
    pr.call(dt, h, ws)  # again on the used workspace: the same bits
    torch.cuda.synchronize()
    assert torch.equal(first, pr.out)
    h.close()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("G", [1, 4])
def test_later_positions_do_not_reach_earlier_rows(torch, bad, G):
    """A position whose keys and values overflow shows in its own row and later ones alone, element by element."""
    import dynamic_draft_tree_gb300 as dt

    for at in (0, 5, 40, 63, 64, 127, 128, 199):
        pr = Problem(torch, n=[200, 30], H_kv=2, G=G, D=64, lens=[40, 33], seed=at)
        pr.vn[pr.off[0] + at, :, 5] = bad
        pr.v[0][40 + at, :, 5] = bad
        h, ws = pr.handle(dt)
        pr.call(dt, h, ws)
        got = pr.out.clone()
        pr.out.fill_(7.0)
        _check(pr, got)
        assert torch.isfinite(got[:at]).all() and not torch.isfinite(got[at:200, :, 5]).any()
        h.close()


def test_a_key_that_is_no_number(torch):
    """NaN in a key makes NaN of the rows that attend to it, and of no other."""
    import dynamic_draft_tree_gb300 as dt

    pr = Problem(torch, n=[200, 30], H_kv=1, G=2, D=128)
    pr.kn[70] = float("nan")
    h, ws = pr.handle(dt)
    pr.call(dt, h, ws)
    torch.cuda.synchronize()
    assert torch.isfinite(pr.out[:70]).all() and torch.isnan(pr.out[70:200]).all() and torch.isfinite(pr.out[200:230]).all()
    h.close()


def test_strided_inputs_and_other_stream(torch):
    """q, k and v as slices of one projection, the output inside a wider buffer, on a side stream."""
    import dynamic_draft_tree_gb300 as dt

    pr = Problem(torch, n=[150, 4, 90], H_kv=2, G=4, D=64, lens=[70, 5, 129])
    rows, H, D = pr.q.shape
    wide = torch.zeros(rows, H + 4, D + 8, dtype=pr.q.dtype, device="cuda")
    fused = wide[:, :, :D]
    fused[:, :H], fused[:, H:H + 2], fused[:, H + 2:] = pr.q, pr.kn, pr.vn
    out = torch.full((rows, 2 * H, D), 7.0, dtype=pr.q.dtype, device="cuda")[:, ::2]
    h, ws = pr.handle(dt)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    dt.dt_prompt_attention(h, fused[:, :H], fused[:, H:H + 2], fused[:, H + 2:], pr.row_off, out, ws, k_pages=pr.kp,
                           v_pages=pr.vp, block_table=pr.table, seq_len=pr.seq_len, stream=side)
    side.synchronize()
    _check(pr, out)
    pr.call(dt, h, ws)
    torch.cuda.synchronize()
    assert torch.equal(out, pr.out)
    h.close()


def test_captured_graph_follows_the_lengths(torch):
    """A captured call replayed after the offsets, lengths, tables and contents changed."""
    import dynamic_draft_tree_gb300 as dt

    kw = dict(H_kv=2, G=4, D=128, max_blocks=64)
    pr = Problem(torch, n=[300, 1, 20, 79], lens=[30, 600, 2, 0], spare=60, **kw)
    h, ws = pr.handle(dt)
    pr.call(dt, h, ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pr.call(dt, h, ws)
    other = Problem(torch, n=[7, 350, 0, 43], lens=[1000, 3, 77, 0], seed=9, **kw)
    for name in ("table", "seq_len", "row_off", "q", "kn", "vn"):
        getattr(pr, name).copy_(getattr(other, name))
    m = other.kp.shape[0]  # fewer pages than the captured buffers have
    pr.kp[:m].copy_(other.kp)
    pr.vp[:m].copy_(other.vp)
    pr.out.fill_(7.0)
    g.replay()
    torch.cuda.synchronize()
    _check(other, pr.out)
    h.close()


def test_two_graphs_share_a_workspace(torch):
    """Captured calls of other shapes on one workspace, replayed in turn."""
    import dynamic_draft_tree_gb300 as dt

    a = Problem(torch, n=[900, 30], H_kv=2, G=4, D=128)
    b = Problem(torch, n=[10, 400], H_kv=1, G=8, D=128, lens=[2000, 5])
    h, ws = a.handle(dt)
    graphs, first = [], []
    for pr in (a, b):
        pr.call(dt, h, ws)
        torch.cuda.synchronize()
        first.append(pr.out.clone())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            pr.call(dt, h, ws)
        graphs.append(g)
    for _ in range(3):
        for g, pr, want in zip(graphs, (a, b), first):
            pr.out.fill_(7.0)
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(pr.out, want)
    h.close()


def test_bad_tables_and_offsets_are_reported(torch):
    """A block id outside the pages, a length past the table and offsets past the rows set the status; nothing outside is
    read or written."""
    import dynamic_draft_tree_gb300 as dt

    pr = Problem(torch, n=[3, 40], H_kv=1, G=2, D=64, lens=[40, 40])
    h, ws = pr.handle(dt)

    def status():
        pr.call(dt, h, ws)
        bits = dt.dt_get_status(h)
        dt.dt_clear_status(h)
        return bits

    assert status() == 0
    pr.table[1, 1] = pr.kp.shape[0]
    assert status() & dt.DT_DEV_BAD_PAGE
    pr.table[1, 1] = 0
    pr.seq_len[1] = 49  # three blocks in the table
    assert status() & dt.DT_DEV_BAD_PAGE
    pr.seq_len[1] = -1
    assert status() & dt.DT_DEV_BAD_PAGE
    pr.seq_len[1] = 40
    for off in ([0, 3, pr.q.shape[0] + 1], [0, 9, 3], [-2, 3, 9]):
        pr.row_off.copy_(torch.tensor(off, dtype=torch.int32))
        pr.out.fill_(7.0)
        assert status() & dt.DT_DEV_BAD_PAGE
    h.close()


def test_a_wait_that_runs_out_is_reported(torch):
    import dynamic_draft_tree_gb300 as dt

    pr = Problem(torch, n=[300, 100], H_kv=2, G=4, D=128, lens=[500, 0])
    h, ws = pr.handle(dt, flags=dt.DT_FLAG_TEST_TIMEOUT)
    ws.zero_()
    pr.call(dt, h, ws)
    assert dt.dt_get_status(h) & dt.DT_DEV_TIMEOUT
    h.close()
    h, ws = pr.handle(dt)  # the device is fit for the next call
    pr.call(dt, h, ws)
    assert dt.dt_get_status(h) == 0
    got = pr.out.clone()
    pr.out.fill_(7.0)
    _check(pr, got)
    h.close()


def test_refusals(torch):
    import dynamic_draft_tree_gb300 as dt

    pr = Problem(torch, n=[20, 9], H_kv=2, G=2, D=64, lens=[40, 33])
    h, ws = pr.handle(dt)
    pages = dict(k_pages=pr.kp, v_pages=pr.vp, block_table=pr.table, seq_len=pr.seq_len)

    def call(q=pr.q, k=pr.kn, v=pr.vn, off=pr.row_off, out=pr.out, w=ws, **kw):
        dt.dt_prompt_attention(h, q, k, v, off, out, w, **kw)

    for bad in (dict(q=pr.q.float()), dict(q=pr.q[0]), dict(k=pr.kn[:-1]), dict(v=pr.vn[:, :1]), dict(out=pr.out[:-1]),
                dict(out=pr.out.half()), dict(off=pr.row_off.long()), dict(off=pr.row_off[:1]), dict(off=pr.row_off.cpu()),
                dict(w=ws.int()), dict(q=pr.q.cpu()), dict(k_pages=pr.kp), dict(seq_len=pr.seq_len),
                dict(pages, block_table=pr.table[:1]), dict(pages, seq_len=pr.seq_len[:1]), dict(pages, v_pages=pr.vp[:, :8]),
                dict(pages, k_pages=pr.kp[..., ::2], v_pages=pr.vp[..., ::2]), dict(pages, k_pages=pr.kp.half()),
                dict(q=pr.q.transpose(1, 2).contiguous().transpose(1, 2))):
        with pytest.raises(ValueError):
            call(**bad)
    for bad in (dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(w=ws[:1000]), dict(w=ws[1:]),
                dict(q=pr.q[:, :3], out=pr.out[:, :3]),  # three heads of two key heads
                dict(k=pr.kn[..., :60], v=pr.vn[..., :60], q=pr.q[..., :60], out=pr.out[..., :60]),
                dict(pages, k_pages=pr.kp[:, :12], v_pages=pr.vp[:, :12])):
        with pytest.raises(dt.DtError) as e:
            call(**bad)
        assert e.value.code == dt.DT_ERR_ARG
    with pytest.raises(dt.DtError):
        call(off=torch.zeros(4, dtype=torch.int32, device="cuda"))  # three requests, B_max is two
    with pytest.raises(dt.DtError):
        dt.dt_prompt_attention_workspace(h, 2, 4, 2, 136)
    torch.cuda.synchronize()
    assert (pr.out == 7.0).all() and dt.dt_get_status(h) == 0
    h.close()
