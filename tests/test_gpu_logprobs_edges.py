"""dt_token_logprobs where its sums leave the ordinary: rows of masked values that are finite, differences past fp32, many equal
logits, requests outside the rows, offsets past 31 bits, two calls at once.

Tolerance: where every logit's distance from the largest is 0 or more than 1000, weights are 0 or within ex2's 2^-22 of 1 (their
exponent is 0, or the rounding of the reference, which is taken back), and S is a whole number times that, off by the roundings of
its sums: 32 terms a thread, five and three levels of trees, and what brings pieces together, at most 49 of 2^-24. The logarithm
adds 2^-22, and the rounding of the result half a step. The entropy has the same S in both of its terms, twice. Elsewhere an
exponent is a distance that is rounded twice (subtraction and product, or multiply-add and the reference's own rounding, which is
taken back).
"""
import math

import pytest

pytestmark = pytest.mark.gpu

LOG = 2.0 ** -22
SUM = 2.0 ** -22 + 49 * 2.0 ** -24


@pytest.fixture(scope="module")
def torch():
    import torch as t

    if not t.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__

    __graft_entry__.build()
    return t


def _labels(t, dt, x, tokens, K=3, ws_entries=None):
    """One request whose rows are x [n][V], labels tokens [n]: (status, logp, entropy, rank, ids, top_logp)."""
    n, V = x.shape
    h = dt.Handle(1, V, 1, 1, 1, 1, dt.DT_BF16 if x.dtype is t.bfloat16 else dt.DT_F32)
    ws = dt.dt_token_logprobs_workspace(h, ws_entries or n, K)
    out = [t.full((n,), 7.0, device="cuda"), t.full((n,), 7.0, device="cuda"), t.full((n,), 7, dtype=t.int32, device="cuda"),
           t.full((n, K), 7, dtype=t.int32, device="cuda"), t.full((n, K), 7.0, device="cuda")]
    dt.dt_token_logprobs(h, x, t.tensor([n], dtype=t.int32, device="cuda"), out[0], ws, tokens=tokens, shift=0,
                         row_off=t.tensor([0, n], dtype=t.int32, device="cuda"), entropy=out[1], rank=out[2], top_ids=out[3],
                         top_logp=out[4])
    status = dt.dt_get_status(h)
    h.close()
    return [status] + out


def _near(got, want, more=0.0):
    """Within the errors of the sum and the logarithm and the rounding; values past fp32 are infinite."""
    if abs(want) > 3.4028235e38:
        assert got == math.copysign(math.inf, want)
    else:
        assert abs(got - want) <= SUM + LOG + 2.0 ** -24 * abs(want) + more, (got, want)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("value", [0.0, 100.0, -300.0, -1e4, 1e9, -1e9, -1e30, -1e38, -2e38, -2.5e38, "lowest", "highest"])
def test_rows_of_one_value(torch, dtype, value):
    """log V, whatever the value."""
    import dynamic_draft_tree_gb300 as dt

    t, V = torch, 20001
    ty = {"bf16": t.bfloat16, "fp32": t.float32}[dtype]
    v = {"lowest": t.finfo(ty).min, "highest": t.finfo(ty).max}.get(value, value)
    x = t.full((2, V), v, dtype=ty, device="cuda")
    status, logp, ent, rank, ids, top = _labels(t, dt, x, t.tensor([17, V - 1], dtype=t.int32, device="cuda"))
    assert status == 0
    for k in range(2):
        _near(float(logp[k]), -math.log(V))
        _near(float(ent[k]), math.log(V), SUM)
    assert rank.tolist() == [17, V - 1] and ids.tolist() == [[0, 1, 2]] * 2
    for y in top.view(-1).tolist():
        _near(y, -math.log(V))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("fill", [-1e4, -1e9, -1e30, -1e38, -2e38, "lowest"])
def test_masked_by_a_finite_value(torch, dtype, fill):
    """Rows in which a few tokens are allowed, whole pieces not: at the first, a middle and the last token, or one alone."""
    import dynamic_draft_tree_gb300 as dt

    t, V = torch, 50001
    ty = {"bf16": t.bfloat16, "fp32": t.float32}[dtype]
    f = t.finfo(ty).min if fill == "lowest" else fill
    x = t.full((3, V), f, dtype=ty, device="cuda")
    x[0, 0] = x[0, 30000] = x[0, V - 1] = 2.5
    x[1, 29999] = -7.0
    x[2, V - 2] = 3.0
    f = float(x[0, 1])
    tok = t.tensor([30000, 29999, 5], dtype=t.int32, device="cuda")
    status, logp, ent, rank, ids, top = _labels(t, dt, x, tok)
    assert status == 0
    _near(float(logp[0]), -math.log(3))
    _near(float(ent[0]), math.log(3), SUM)
    _near(float(logp[1]), 0.0)
    _near(float(ent[1]), 0.0)
    _near(float(logp[2]), f - 3.0)
    assert rank.tolist() == [1, 0, 6]
    assert ids.tolist() == [[0, 30000, V - 1], [29999, 0, 1], [V - 2, 0, 1]]
    _near(float(top[1, 1]), f + 7.0)


def test_differences_past_fp32(torch):
    import dynamic_draft_tree_gb300 as dt

    t, V = torch, 9000
    x = t.full((3, V), -3.3e38, device="cuda")
    x[0, 8000] = 3.3e38
    x[1, :4000] = -math.inf
    x[1, 4500] = -1e37
    x[2, 100], x[2, 8500] = 3e38, 3.2e38  # the second one in another piece than the first
    tok = t.tensor([8000, 5000, 100], dtype=t.int32, device="cuda")
    status, logp, ent, rank, ids, top = _labels(t, dt, x, tok)
    assert status == 0
    z = t.log_softmax(x.double(), 1)
    for k in range(3):
        _near(float(logp[k]), float(z[k, int(tok[k])]))
        _near(float(ent[k]), 0.0)
    assert rank.tolist() == [0, 1 + 500 + 499, 1] and ids[:, 0].tolist() == [8000, 4500, 8500]
    assert ids[0].tolist() == [8000, 0, 1] and top[0, 1] == -math.inf


@pytest.mark.parametrize("shift", [3000.0, -3000.0, 70000.0])
def test_logits_far_from_zero(torch, shift):
    """fp32 rows around a value that is not near zero: distances from the largest count, not the value."""
    import dynamic_draft_tree_gb300 as dt

    t, V = torch, 33000
    g = t.Generator(device="cuda")
    g.manual_seed(3)
    x = (t.randn(3, V, generator=g, device="cuda") * 3 + shift).float()
    tok = t.randint(0, V, (3,), generator=g, device="cuda", dtype=t.int32)
    status, logp, ent, rank, ids, top = _labels(t, dt, x, tok, K=20)
    assert status == 0
    z = t.log_softmax(x.double(), 1)
    # distances below 60 (others add less than 2^-40): subtraction, product and ex2 change a weight by 2^-24 (3 * 60 * 0.7 + 4) at
    # most, sums by 49 roundings
    u = 2.0 ** -24 * (126 + 4 + 49)
    order = t.sort(x, dim=1, descending=True, stable=True)
    for k in range(3):
        _near(float(logp[k]), float(z[k, int(tok[k])]), u)
        H = float(-(z[k].exp() * z[k]).sum())
        assert abs(float(ent[k]) - H) <= u * (2 + 2 * H) + LOG + 2.0 ** -24 * (180 + H)
    assert t.equal(ids.long(), order.indices[:, :20])


@pytest.mark.parametrize("V,K", [(4096, 20), (5000, 32), (20000, 32), (1024, 1), (40, 32), (31, 31), (1100001, 5)])
@pytest.mark.parametrize("spread", [0.0, 0.3, 5.0])
def test_alternatives_of_few_and_of_many_steps(torch, V, K, spread):
    """As few steps as alternatives, and more steps than are ranked at once; with many equal logits too."""
    import dynamic_draft_tree_gb300 as dt

    t = torch
    g = t.Generator(device="cuda")
    g.manual_seed(V + K)
    x = (t.randn(3, V, generator=g, device="cuda") * spread).to(t.bfloat16)
    x[2, : V // 2] = -math.inf
    tok = t.zeros(3, dtype=t.int32, device="cuda")
    status, logp, ent, rank, ids, top = _labels(t, dt, x, tok, K=K)
    assert status == 0
    order = t.sort(x.float(), dim=1, descending=True, stable=True)
    some = order.values[:, :K] > -math.inf
    assert t.equal(ids.long(), t.where(some, order.indices[:, :K], -1))
    z = t.log_softmax(x.double(), 1)
    want = t.where(some, z.gather(1, order.indices[:, :K]), -math.inf)
    assert bool((top[~some] == -math.inf).all())
    u = 2.0 ** -24 * (0.7 * (60 + 1.45 * 64) + 49)
    assert float(((top.double() - want).abs()[some] - 2.0 ** -24 * want.abs()[some]).max()) <= u + LOG


def test_a_workspace_serves_fewer_entries(torch):
    """Fewer entries have more pieces: from 1 to 300 entries on the workspace for 300."""
    import dynamic_draft_tree_gb300 as dt

    t, V = torch, 128256
    h = dt.Handle(1, V, 1, 1, 1, 1, dt.DT_BF16)
    ws = dt.dt_token_logprobs_workspace(h, 300, 4)
    sizes = [dt.dt_token_logprobs_workspace(h, n, 4).numel() for n in range(1, 301)]
    assert sizes == sorted(sizes) and sizes[-1] == ws.numel()
    g = t.Generator(device="cuda")
    g.manual_seed(1)
    x = t.randn(300, V, generator=g, device="cuda").to(t.bfloat16)
    tok = t.randint(0, V, (300,), generator=g, device="cuda", dtype=t.int32)
    want = t.log_softmax(x.float(), 1).gather(1, tok.long()[:, None])[:, 0]
    ids, top = t.zeros(300, 4, dtype=t.int32, device="cuda"), t.zeros(300, 4, device="cuda")
    for n in (1, 38, 39, 76, 77, 78, 116, 155, 194, 299, 300):
        logp = t.zeros(n, device="cuda")
        dt.dt_token_logprobs(h, x[:n], t.tensor([n], dtype=t.int32, device="cuda"), logp, ws, tokens=tok[:n], shift=0,
                             row_off=t.tensor([0, n], dtype=t.int32, device="cuda"), top_ids=ids[:n], top_logp=top[:n])
        assert dt.dt_get_status(h) == 0
        assert float((logp - want[:n]).abs().max()) < 1e-4  # whole rows were summed
        assert t.equal(ids[:n, 0].long(), x[:n].float().argmax(1))
    h.close()


@pytest.mark.parametrize("B", [3, 40])
def test_requests_outside_the_rows_are_reported(torch, B):
    """Packed requests that no row belongs to, or whose rows pass the buffer."""
    import dynamic_draft_tree_gb300 as dt

    t, V, n = torch, 3000, 10
    h = dt.Handle(B, V, 1, 1, 1, 1, dt.DT_BF16)
    ws = dt.dt_token_logprobs_workspace(h, n, 0)
    x = t.zeros(n, V, dtype=t.bfloat16, device="cuda")

    def status(off, new):
        logp = t.full((n,), 7.0, device="cuda")
        off, new = off + [off[-1]] * (B + 1 - len(off)), new + [0] * (B - len(new))
        i32 = lambda v: t.tensor(v, dtype=t.int32, device="cuda")
        dt.dt_token_logprobs(h, x, i32(new), logp, ws, tokens=t.zeros(n, dtype=t.int32, device="cuda"), shift=0, row_off=i32(off))
        bits = dt.dt_get_status(h)
        dt.dt_clear_status(h)
        return bits, [k for k in range(n) if float(logp[k]) != 7.0]

    assert status([0, 4, 4, 10], [4, 0, 6]) == (0, list(range(10)))
    assert status([0, 4, 4, 10], [4, 1, 6]) == (dt.DT_DEV_BAD_TREE, [0, 1, 2, 3] + list(range(4, 10)))  # no rows, one entry
    assert status([0, 4, 4, 10], [4, -1, 6]) == (dt.DT_DEV_BAD_TREE, list(range(10)))
    assert status([0, 4, 10, 13], [4, 6, 3]) == (dt.DT_DEV_BAD_TREE, list(range(10)))  # past the rows
    assert status([0, 4, 8, 13], [4, 4, 2]) == (0, list(range(10)))                    # its entries are not
    assert status([0, 4, 8, 13], [4, 4, 3]) == (dt.DT_DEV_BAD_TREE, list(range(10)))
    assert status([-2, 4, 8, 10], [2, 4, 2])[0] == dt.DT_DEV_BAD_TREE
    h.close()


def test_vocabularies_past_the_counting_of_places_are_refused(torch):
    import dynamic_draft_tree_gb300 as dt

    for V, ok in ((2 ** 31 - 2 ** 16, True), (2 ** 31 - 2 ** 16 + 1, False), (2 ** 31 - 1, False)):
        h = dt.Handle(1, V, 1, 1, 1, 1)
        if ok:
            dt.dt_token_logprobs_workspace(h, 1)
        else:
            with pytest.raises(dt.DtError) as e:
                dt.dt_token_logprobs_workspace(h, 1)
            assert e.value.code == dt.DT_ERR_ARG
        h.close()


def test_offsets_past_31_bits(torch):
    """Rows 2^30 elements apart."""
    import dynamic_draft_tree_gb300 as dt

    t, V, ld = torch, 5000, 1 << 30
    buf = t.empty(2 * ld + V, dtype=t.bfloat16, device="cuda")
    x = buf.as_strided((3, V), (ld, 1))
    g = t.Generator(device="cuda")
    g.manual_seed(4)
    y = t.randn(3, V, generator=g, device="cuda").to(t.bfloat16)
    x.copy_(y)
    tok = t.tensor([1, 4000, 4999], dtype=t.int32, device="cuda")
    a, b = _labels(t, dt, x, tok), _labels(t, dt, y, tok)
    assert a[0] == 0 and all(t.equal(p, q) for p, q in zip(a[1:], b[1:]))


def test_two_calls_at_once(torch):
    """Two streams, a handle for both, a workspace each."""
    import dynamic_draft_tree_gb300 as dt

    t, V, n = torch, 64000, 200
    h = dt.Handle(1, V, 1, 1, 1, 1, dt.DT_F32)
    g = t.Generator(device="cuda")
    g.manual_seed(5)
    xs = [t.randn(n, V, generator=g, device="cuda") for _ in range(2)]
    tok = t.randint(0, V, (n,), generator=g, device="cuda", dtype=t.int32)
    count, off = t.tensor([n], dtype=t.int32, device="cuda"), t.tensor([0, n], dtype=t.int32, device="cuda")
    ws = [dt.dt_token_logprobs_workspace(h, n, 8) for _ in range(2)]
    outs = [[t.zeros(n, device="cuda"), t.zeros(n, 8, dtype=t.int32, device="cuda"), t.zeros(n, 8, device="cuda")] for _ in range(4)]

    def call(k, o, stream=None):
        dt.dt_token_logprobs(h, xs[k], count, o[0], ws[k], tokens=tok, shift=0, row_off=off, top_ids=o[1], top_logp=o[2], stream=stream)

    call(0, outs[0])
    call(1, outs[1])
    streams = [t.cuda.Stream(), t.cuda.Stream()]
    t.cuda.synchronize()
    for _ in range(20):
        call(0, outs[2], streams[0])
        call(1, outs[3], streams[1])
    t.cuda.synchronize()
    assert dt.dt_get_status(h) == 0
    for a, b in ((0, 2), (1, 3)):
        assert all(t.equal(p, q) for p, q in zip(outs[a], outs[b]))
    h.close()
