"""dt_logits_process and dt_count_tokens against the definition in 64 bits.

Tolerance: every step of an element (division or product, frequency product, two differences, the biases' sum and its
addition) rounds once in fp32, each by at most 2^-24 of a value no larger than M = |x| max(r, 1/r) + f c + p + sum |bias|;
with n biases on a token at most (6 + n) 2^-24 M. The result rounds once to the row's type: u |y|, bf16 2^-8, fp32 2^-24.
"""
import math
import random

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


class Problem:
    def __init__(self, t, B, P, V, dtype, packed=False, n_pos=None, n_bias=0, tree=True, ld=None, parts="cthrfpa",
                 seed=0):
        r = random.Random(seed + 77 * V + P)
        g = t.Generator(device="cuda")
        g.manual_seed(seed + V)
        td = {"bf16": t.bfloat16, "fp32": t.float32}[dtype]
        self.t, self.B, self.P, self.V, self.packed = t, B, P, V, packed
        self.n = n_pos or [P] * B
        off = [0]
        for k in self.n:
            off.append(off[-1] + k)
        self.base = off[:-1] if packed else [b * P for b in range(B)]
        rows = off[-1] + 2 if packed else B * P
        i32 = dict(dtype=t.int32, device="cuda")
        self.row_off = t.tensor(off, **i32) if packed else None
        self.n_pos = t.tensor(self.n, **i32)
        self.buf = (t.randn(rows, ld or V, generator=g, device="cuda") * 4).to(td)
        self.x = self.buf[:, :V]
        m = [[[0] * P for _ in range(P)] for _ in range(B)]
        for b in range(B):
            for i in range(self.n[b]):
                if i:
                    m[b][i] = list(m[b][r.randint(max(0, i - 5), i - 1)])
                m[b][i][i] = 1
        self.mask = t.tensor(m, dtype=t.uint8, device="cuda") if tree else None
        few = [r.randrange(V) for _ in range(max(1, P // 3))]  # tokens repeat within a path
        tok = [[r.choice(few) if r.random() < 0.6 else r.randrange(V) for _ in range(P)] for _ in range(B)]
        for b in range(B):
            tok[b][-1] = -1
        self.tokens = t.tensor(tok, **i32) if "t" in parts else None
        self.counts = None
        if "c" in parts:
            self.counts = t.randint(0, 4, (B, V), generator=g, device="cuda", dtype=t.int32) * \
                (t.rand(B, V, generator=g, device="cuda") < 0.2)
            self.counts |= (t.rand(B, V, generator=g, device="cuda") < 0.1).to(t.int32) * SEEN
        u = lambda lo, hi: t.rand(B, generator=g, device="cuda") * (hi - lo) + lo  # noqa: E731
        self.rep = u(0.7, 1.6) if "r" in parts else None
        self.freq = u(-0.5, 1.0) if "f" in parts else None
        self.pres = u(-0.5, 1.0) if "p" in parts else None
        self.bias_ids = self.bias_vals = None
        if n_bias:
            ids = [[r.choice([r.randrange(V), r.randrange(min(V, 40)), -1]) for _ in range(n_bias)] for _ in range(B)]
            self.bias_ids = t.tensor(ids, **i32)
            self.bias_vals = t.randn(B, n_bias, generator=g, device="cuda") * 6
        self.allow = None
        if "a" in parts:
            w = (V + 31) // 32
            self.allow = t.randint(-2 ** 31, 2 ** 31, (rows, w), generator=g, device="cuda", dtype=t.int64).to(t.int32)
            self.allow[rows // 2] = 0  # a row that may say nothing

    def view(self, x):
        return x if self.packed else x.view(self.B, self.P, x.shape[-1]) if x.is_contiguous() else \
            x.unflatten(0, (self.B, self.P))

    def call(self, dt, h, out, logits=None):
        dt.dt_logits_process(h, self.view(self.x if logits is None else logits), self.view(out), self.n_pos,
                             tokens=self.tokens, mask=self.mask, row_off=self.row_off, counts=self.counts,
                             repetition=self.rep, frequency=self.freq, presence=self.pres, bias_ids=self.bias_ids,
                             bias_vals=self.bias_vals, allow=self.allow, P=self.P)

    def reference(self, out):
        t, V = self.t, self.V
        want, tol = out.double().clone(), t.zeros(out.shape, dtype=t.float64, device="cuda")
        u = t.finfo(out.dtype).eps / 2
        for b in range(self.B):
            one = t.ones((), dtype=t.float64, device="cuda")
            r = self.rep[b].double() if self.rep is not None else one
            f = self.freq[b].double() if self.freq is not None else 0 * one
            p = self.pres[b].double() if self.pres is not None else 0 * one
            bias, size, count = (t.zeros(V, dtype=t.float64, device="cuda") for _ in range(3))
            if self.bias_ids is not None:
                for k, v in zip(self.bias_ids[b].tolist(), self.bias_vals[b].tolist()):
                    if k >= 0:
                        bias[k] += v
                        size[k] += abs(v)
                        count[k] += 1
            for i in range(self.n[b]):
                x = self.x[self.base[b] + i].double()
                c = t.zeros(V, dtype=t.float64, device="cuda")
                seen = t.zeros(V, dtype=t.bool, device="cuda")
                if self.counts is not None:
                    c += (self.counts[b] & (SEEN - 1)).double()
                    seen |= self.counts[b] >= SEEN
                if self.tokens is not None:
                    for j in range(self.n[b]):
                        tok = int(self.tokens[b, j])
                        if tok >= 0 and (int(self.mask[b, i, j]) if self.mask is not None else j <= i):
                            c[tok] += 1
                seen |= c > 0
                y = t.where(seen, t.where(x > 0, x / r, x * r), x) - f * c - p * (c > 0) + bias
                big = x.abs() * max(float(r), 1 / float(r)) + f.abs() * c + p.abs() + size
                ok = t.ones(V, dtype=t.bool, device="cuda")
                if self.allow is not None:
                    w = self.allow[self.base[b] + i]
                    v = t.arange(V, device="cuda")
                    ok = (w[v >> 5] >> (v & 31)) & 1 == 1
                want[self.base[b] + i] = t.where(ok, y, -math.inf)
                tol[self.base[b] + i] = t.where(ok, (6 + count) * 2.0 ** -24 * big + u * y.abs(), 0.0) * 1.01
        return want, tol


def _compare(t, got, want, tol):
    got = got.double()
    assert t.equal(t.isnan(got), t.isnan(want))
    special = ~t.isfinite(want) & ~t.isnan(want)
    assert t.equal(got[special], want[special])
    fine = t.isfinite(want)
    assert t.isfinite(got[fine]).all()
    off = ((got - want).abs() - tol)[fine]
    assert off.numel() == 0 or float(off.max()) <= 0, float(off.max())


CASES = {
    "one row": dict(B=1, P=1, V=32000, dtype="bf16"),
    "two tokens": dict(B=2, P=2, V=2, dtype="fp32", n_bias=3),
    "tiny vocabulary": dict(B=2, P=40, V=33, dtype="bf16", n_bias=9),
    "odd vocabulary": dict(B=3, P=17, V=4099, dtype="bf16", n_bias=20),
    "odd vocabulary fp32": dict(B=2, P=18, V=4099, dtype="fp32", n_bias=20, packed=True, n_pos=[18, 3]),
    "packed": dict(B=4, P=33, V=8200, dtype="bf16", packed=True, n_pos=[33, 1, 0, 20], n_bias=5),
    "padded ragged": dict(B=3, P=19, V=6001, dtype="fp32", n_pos=[7, 19, 16]),
    "wide rows": dict(B=2, P=5, V=3000, dtype="bf16", ld=3008, n_bias=2),
    "unaligned rows": dict(B=2, P=5, V=3000, dtype="bf16", ld=3001, n_bias=2),
    "chain": dict(B=2, P=70, V=2500, dtype="fp32", tree=False),
    "512 positions": dict(B=1, P=512, V=2100, dtype="bf16", tree=False),
    "history only": dict(B=2, P=4, V=5000, dtype="bf16", parts="crfp"),
    "path only": dict(B=2, P=20, V=5000, dtype="fp32", parts="trfp"),
    "repetition only": dict(B=2, P=20, V=5000, dtype="fp32", parts="ctr"),
    "grammar only": dict(B=2, P=20, V=5000, dtype="bf16", parts="a"),
    "bias only": dict(B=2, P=3, V=5000, dtype="fp32", parts="", n_bias=70),
    "nothing": dict(B=2, P=3, V=5000, dtype="bf16", parts=""),
    "many biases": dict(B=2, P=2, V=9000, dtype="fp32", n_bias=4096),
}


@pytest.mark.parametrize("name", list(CASES))
def test_matches_definition(torch, name):
    import dynamic_draft_tree_gb300 as dt

    pr = Problem(torch, **CASES[name])
    h = dt.Handle(pr.B, pr.V, 1, 1, 1, pr.P, dt.DT_BF16 if CASES[name]["dtype"] == "bf16" else dt.DT_F32)
    out = torch.full_like(pr.x, 7.0)
    want, tol = pr.reference(out)
    pr.call(dt, h, out)
    assert dt.dt_get_status(h) == 0
    _compare(torch, out, want, tol)
    # in place, in the rows' own buffer: the same bits; what lies between rows stays
    buf, x = pr.buf.clone(), pr.x
    inner = buf[:, :pr.V]
    keep = buf[:, pr.V:].clone()
    pr.x = inner
    pr.call(dt, h, inner)
    torch.cuda.synchronize()
    for b in range(pr.B):
        rows = slice(pr.base[b], pr.base[b] + pr.n[b])
        assert torch.equal(inner[rows], out[rows])
        if not pr.packed:
            rest = slice(pr.base[b] + pr.n[b], pr.base[b] + pr.P)
            assert torch.equal(inner[rest], x[rest])
    assert torch.equal(buf[:, pr.V:], keep)
    h.close()


# dtype, V, elements between rows and in front of the first one: logits, output (None: in place)
ALIGNMENTS = [("bf16", 4099, (4099, 0), (4099, 0)), ("bf16", 4099, (4101, 3), (4101, 3)), ("bf16", 1021, (1030, 5), (1046, 13)),
              ("bf16", 2052, (2052, 1), None), ("bf16", 2048, (2048, 7), (2048, 7)), ("bf16", 1024, (1025, 2), (1024, 2)),
              ("bf16", 3, (3, 0), (3, 0)), ("bf16", 7, (11, 4), None), ("fp32", 4099, (4099, 0), (4099, 0)),
              ("fp32", 2047, (2050, 1), (2054, 5)), ("fp32", 3000, (3001, 3), None), ("fp32", 1024, (1024, 2), (1024, 2)),
              ("fp32", 2, (2, 0), (2, 0)), ("fp32", 513, (513, 1), (516, 0)), ("bf16", 1021, (1030, 0), (1046, 0)),
              ("bf16", 7, (11, 0), None), ("bf16", 2052, (2052, 0), (2052, 0)), ("fp32", 2047, (2050, 0), (2054, 0)),
              ("fp32", 3000, (3001, 0), None)]


@pytest.mark.parametrize("dtype,V,src,dst", ALIGNMENTS)
@pytest.mark.parametrize("P,packed", [(19, True), (85, False), (85, True)])
def test_alignments(torch, dtype, V, src, dst, P, packed):
    """Rows that start anywhere: the definition's values, and nothing but the rows' tokens is written."""
    import dynamic_draft_tree_gb300 as dt

    n_pos = [P, 7, 1]
    pr = Problem(torch, B=3, P=P, V=V, dtype=dtype, packed=packed, n_pos=n_pos, n_bias=9, seed=4)
    rows = pr.x.shape[0]
    h = dt.Handle(3, V, 1, 1, 1, P, dt.DT_BF16 if dtype == "bf16" else dt.DT_F32)

    def place(ld, at, fill):
        flat = torch.full((at + rows * ld + 9,), fill, dtype=pr.x.dtype, device="cuda")
        return flat, flat[at:at + rows * ld].view(rows, ld)[:, :V]

    x_flat, x = place(*src, 5.0)
    x.copy_(pr.x)
    pr.x = x
    out_flat, out = place(*(dst or src), 7.0)
    want, tol = pr.reference(out if dst else x.clone())
    if dst is None:
        out_flat, out = x_flat, x
    before = out_flat.clone()
    pr.call(dt, h, out, logits=x)
    assert dt.dt_get_status(h) == 0
    used = torch.zeros(rows, dtype=torch.bool, device="cuda")
    for b in range(3):
        used[pr.base[b]:pr.base[b] + n_pos[b]] = True
    _compare(torch, out[used], want[used], tol[used])
    out[used] = 0
    ld, at = dst or src
    before[at:at + rows * ld].view(rows, ld)[:, :V][used] = 0
    assert torch.equal(out_flat, before)
    h.close()


def test_special_values(torch):
    """-inf, +inf, NaN and zeros in the rows; a forbidden token is -inf whatever it held."""
    import dynamic_draft_tree_gb300 as dt

    pr = Problem(torch, B=1, P=2, V=3000, dtype="fp32", n_bias=4)
    for k, v in enumerate((math.inf, -math.inf, math.nan, 0.0, -0.0, 3e38, -3e38)):
        pr.buf[:, k::97] = v
    pr.allow[1] = -1
    h = dt.Handle(1, 3000, 1, 1, 1, 2, dt.DT_F32)
    out = torch.zeros_like(pr.x)
    pr.call(dt, h, out)
    want, tol = pr.reference(out)
    # products past the largest fp32 number are infinite there, and finite in 64 bits
    top = torch.finfo(torch.float32).max
    want = torch.where(want.abs() > top, want.sign() * math.inf, want)
    _compare(torch, out, want, tol)
    h.close()


def test_bad_ids_are_reported_and_skipped(torch):
    import dynamic_draft_tree_gb300 as dt

    pr = Problem(torch, B=1, P=3, V=300, dtype="fp32", n_bias=3, parts="ctrfp")
    h = dt.Handle(1, 300, 1, 1, 1, 3, dt.DT_F32)
    good, bad = torch.zeros_like(pr.x), torch.zeros_like(pr.x)
    pr.tokens[0, 1] = -1
    pr.bias_ids[0, 1] = -1
    pr.call(dt, h, good)
    assert dt.dt_get_status(h) == 0
    for token, bias in ((300, -1), (-1, 300), (-2, -1), (-1, -2)):
        pr.tokens[0, 1], pr.bias_ids[0, 1] = token, bias
        pr.call(dt, h, bad)
        assert dt.dt_get_status(h) == dt.DT_DEV_BAD_TOKEN
        dt.dt_clear_status(h)
        assert torch.equal(good, bad)
    h.close()


def test_count_tokens(torch):
    import dynamic_draft_tree_gb300 as dt

    B, V, P, D = 5, 101, 40, 9
    r = random.Random(3)
    i32 = dict(dtype=torch.int32, device="cuda")
    h = dt.Handle(B, V, 1, 1, 1, P)
    counts = torch.zeros(B, V, **i32)
    want = [[0] * V for _ in range(B)]
    tok = [[r.randrange(V) for _ in range(P)] for _ in range(B)]
    n = [P, 0, 7, 1, 39]
    dt.dt_count_tokens(h, counts, torch.tensor(tok, **i32), torch.tensor(n, **i32), prompt=True)
    for b in range(B):
        for t_ in tok[b][:n[b]]:
            want[b][t_] |= SEEN
    assert counts.tolist() == want
    acc = [8, 0, 3, 5, 1]
    path = [[r.randrange(P) for _ in range(D)] for _ in range(B)]
    path[0][1:4] = [path[0][0]] * 3  # the same position several times
    dt.dt_count_tokens(h, counts, torch.tensor(tok, **i32), torch.tensor(acc, **i32), path=torch.tensor(path, **i32),
                       n_extra=1)
    for b in range(B):
        for j in range(acc[b] + 1):
            want[b][tok[b][path[b][j]]] += 1
    assert counts.tolist() == want
    flat = [r.randrange(V) for _ in range(3000)]
    off = [0, 1000, 1000, 1001, 2500, 3000]
    dt.dt_count_tokens(h, counts, torch.tensor(flat, **i32), torch.tensor([1000, 0, 1, 1499, 500], **i32),
                       row_off=torch.tensor(off, **i32))
    for b, k in enumerate((1000, 0, 1, 1499, 500)):
        for t_ in flat[off[b]:off[b] + k]:
            want[b][t_] += 1
    assert counts.tolist() == want and dt.dt_get_status(h) == 0
    before = counts.clone()
    dt.dt_count_tokens(h, counts, torch.full((B, P), V, **i32), torch.ones(B, **i32))
    assert dt.dt_get_status(h) == dt.DT_DEV_BAD_TOKEN
    dt.dt_clear_status(h)
    dt.dt_count_tokens(h, counts, torch.tensor(tok, **i32), torch.full((B,), P + 1, **i32))
    assert dt.dt_get_status(h) == dt.DT_DEV_BAD_TREE
    assert torch.equal(before, counts)
    dt.dt_clear_status(h)
    # packed rows: a path out of the request's rows, rows that do not end in the buffer
    two, one = torch.tensor([0, 3, 5], **i32), torch.ones(2, **i32)
    few = torch.tensor([1, 2, 3, 4, 5], **i32)
    for path, off in (([[3], [0]], two), ([[-1], [0]], two), ([[0], [2]], torch.tensor([0, 3, 6], **i32)),
                      ([[0], [0]], torch.tensor([0, 1 << 30, (1 << 30) + 2], **i32)),
                      ([[0], [0]], torch.tensor([-3, 0, 2], **i32)),
                      ([[0], [0]], torch.tensor([0, 3, 2], **i32))):
        counts.zero_()
        dt.dt_count_tokens(h, counts, few, one, path=torch.tensor(path, **i32), row_off=off, P=3)
        assert dt.dt_get_status(h) == dt.DT_DEV_BAD_TREE
        dt.dt_clear_status(h)
        assert int(counts.sum()) == 1
    counts.zero_()
    dt.dt_count_tokens(h, counts, few, torch.tensor([3, 3], **i32), row_off=torch.tensor([0, 3, 6], **i32))
    assert dt.dt_get_status(h) == dt.DT_DEV_BAD_TREE
    assert int(counts.sum()) == 5  # the sixth lies past the buffer
    h.close()


def test_refusals(torch):
    import dynamic_draft_tree_gb300 as dt

    pr = Problem(torch, B=2, P=4, V=500, dtype="bf16", n_bias=3)
    h = dt.Handle(2, 500, 1, 1, 1, 4, dt.DT_BF16)
    out = torch.zeros_like(pr.x)
    good = dict(h=h, logits=pr.view(pr.x), out=pr.view(out), n_pos=pr.n_pos, tokens=pr.tokens, mask=pr.mask,
                counts=pr.counts, repetition=pr.rep, bias_ids=pr.bias_ids, bias_vals=pr.bias_vals, allow=pr.allow)

    def no(error, **over):
        with pytest.raises(error):
            dt.dt_logits_process(**dict(good, **over))

    no(ValueError, logits=pr.view(pr.x).float())
    no(ValueError, out=pr.view(out)[:1])
    no(ValueError, counts=pr.counts[:, :400])
    no(ValueError, bias_vals=None)
    no(ValueError, bias_vals=pr.bias_vals[:, :2])
    no(ValueError, allow=pr.allow[:, :15].contiguous())
    no(ValueError, repetition=pr.rep[:1])
    no(ValueError, mask=pr.mask.int())
    no(ValueError, tokens=pr.tokens.cpu())
    wide = torch.zeros(8, 504, dtype=torch.bfloat16, device="cuda")
    flat = wide.view(-1)[:8 * 500].view(2, 4, 500)
    no(dt.DtError, logits=pr.view(wide[:, :500]), out=flat)  # in place with another row distance
    no(dt.DtError, bias_ids=pr.bias_ids.repeat(1, 2000), bias_vals=pr.bias_vals.repeat(1, 2000))
    no(dt.DtError, h=dt.Handle(1, 500, 1, 1, 1, 4, dt.DT_BF16))
    dt.dt_logits_process(**good)
    assert dt.dt_get_status(h) == 0
    h.close()
