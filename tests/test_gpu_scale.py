"""Attention whose scores are far apart: scales up to 1e30, in prompts and in trees.

q and k are small whole numbers, so that a score without its scale is a whole number below 2^24 and exact in fp32 in any order of
summation, as is its distance z from the row's largest. What the kernels may add then does not grow with the scores: the
factor scale log2 e is rounded twice, the product once, so that an exponent z scale log2 e is off by 3 2^-24 of itself; weights
with exponents beyond 64 add less than 2^-40 of a sum of up to 2^13 of them, and the others are off by a factor within
1 +- 2^-15 (0.7 * 64 * 3 * 2^-24 = 2^-17, exp2 2^-22, sums of 2^13 terms in fp32 2^-18 at most as in the ordinary case). Parts with references
below 2^8 in log2 units may differ by two roundings of those, 2^-15, in their exponents. Together 2^-13 of
A = sum p |v|; beside it the weights' rounding to the type u A, the result's u |o|, and what is lost of
fp16 weights below the smallest normal number, 2^-31 sum |v|.
"""
import math

import pytest

import test_gpu_attention as tree
import test_gpu_prompt as prompt
from test_gpu_prompt import torch  # noqa: F401 (the fixture)

pytestmark = pytest.mark.gpu

SCALES = [1e-30, 1e-3, 1.0, 30.0, 1e3, 1e6, 1e7, 1e8, 1e10, 1e20, 1e30]


def _whole(t, x, g, most):
    fine = t.isfinite(x)
    w = t.randint(-most, most + 1, x.shape, generator=g, device="cuda").to(x.dtype)
    x.copy_(t.where(fine, w, x))


def _rows(t, q, k, v, ok, scale):
    """(out, tolerance) of rows q [n][D] against k, v [L][D] where ok [n][L], in 64 bits."""
    u = t.finfo(q.dtype).eps / 2
    z = (q.double() @ k.double().T).masked_fill(~ok, -math.inf)
    d = (z - z.amax(1, keepdim=True)) * scale  # whole numbers are subtracted first: exact whatever the scale
    p = t.softmax(d, 1)
    o, a = p @ v.double(), p @ v.double().abs()
    return o, (u + 2.0 ** -13) * a + u * o.abs() + 2.0 ** -31 * (ok.double() @ v.double().abs())


def _fits(t, got, want, tol, what):
    got = got.double()
    assert bool(t.isfinite(got).all()), f"{what}: not a number, or infinite"
    assert float(((got - want).abs() - tol).max()) <= 0.0, (what, float(((got - want).abs() - tol).max()))


PROMPTS = {
    "short": dict(n=[93, 1, 40], H_kv=2, G=4, D=128),
    "cut and joined": dict(n=[1500], H_kv=1, G=4, D=64),
    "behind cached tokens": dict(n=[130, 1], H_kv=1, G=8, D=128, lens=[1700, 2300], page=64),
    "odd heads": dict(n=[100, 1, 233], H_kv=2, G=5, D=80, lens=[77, 5, 0], page=32),
}


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("name", list(PROMPTS))
def test_prompts_of_any_scale(torch, name, dtype):  # noqa: F811
    import dynamic_draft_tree_gb300 as dt

    t = torch
    pr = prompt.Problem(t, dtype=dtype, **PROMPTS[name])
    g = t.Generator(device="cuda")
    g.manual_seed(5)
    _whole(t, pr.q, g, 3)
    for b in range(pr.B):  # keys again, dense, in the pages and in the rows
        _whole(t, pr.k[b], g, 3)
        pr.kn[pr.off[b]:pr.off[b + 1]] = pr.k[b][pr.lens[b]:]
        for e in range(-(-pr.lens[b] // pr.page)):
            m = min(pr.page, pr.lens[b] - e * pr.page)
            pr.kp[pr.table[b, e], :m] = pr.k[b][e * pr.page:e * pr.page + m]
    h, ws = pr.handle(dt)
    for scale in SCALES:
        pr.scale = scale
        pr.out.fill_(7.0)
        pr.call(dt, h, ws)
        assert dt.dt_get_status(h) == 0
        for b in range(pr.B):
            L, n, r0 = pr.lens[b], pr.n[b], pr.off[b]
            ok = t.arange(L + n, device="cuda")[None, :] <= L + t.arange(n, device="cuda")[:, None]
            for x in range(pr.q.shape[1]):
                want, tol = _rows(t, pr.q[r0:r0 + n, x], pr.k[b][:, x // pr.G], pr.v[b][:, x // pr.G], ok, scale)
                _fits(t, pr.out[r0:r0 + n, x], want, tol, (scale, b, x))
    h.close()


TREES = {
    "one token": dict(B=2, P=1, H_kv=1, G=4, D=128, page=16, lens=[37, 2000], tree=False),
    "trees": dict(B=3, P=33, H_kv=2, G=4, D=64, page=32, lens=[100, 0, 777], n_pos=[33, 5, 20], packed=True),
    "many rows": dict(B=1, P=140, H_kv=1, G=2, D=128, page=16, lens=[1300]),
    "shared": dict(B=5, P=21, H_kv=2, G=4, D=128, page=32, lens=[2048 + 9 * i for i in range(5)], shared=2048),
}


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("name", list(TREES))
def test_trees_of_any_scale(torch, name, dtype):  # noqa: F811
    import dynamic_draft_tree_gb300 as dt

    t = torch
    pr = tree.Problem(t, dtype=dtype, **TREES[name])
    g = t.Generator(device="cuda")
    g.manual_seed(5)
    _whole(t, pr.q, g, 3)
    shared = pr.shared // pr.page
    for b in range(pr.B):
        _whole(t, pr.k[b], g, 3)
        if b:
            pr.k[b][:pr.shared] = pr.k[0][:pr.shared]
        pr.kn[pr.base[b]:pr.base[b] + pr.n[b]] = pr.k[b][pr.lens[b]:]
        for e in range(shared if b else 0, -(-pr.lens[b] // pr.page)):
            m = min(pr.page, pr.lens[b] - e * pr.page)
            pr.kp[pr.table[b, e], :m] = pr.k[b][e * pr.page:e * pr.page + m]
    h, ws = pr.handle(dt)
    for scale in SCALES:
        pr.scale = scale
        pr.out.fill_(7.0)
        pr.call(dt, h, ws)
        assert dt.dt_get_status(h) == 0
        for b in range(pr.B):
            L, n, r0 = pr.lens[b], pr.n[b], pr.base[b]
            ok = t.ones(n, L + n, dtype=t.bool, device="cuda")
            ok[:, L:] = pr.mask[b, :n, :n].bool() if pr.mask is not None else ok[:, L:].tril()
            for x in range(pr.q.shape[1]):
                want, tol = _rows(t, pr.q[r0:r0 + n, x], pr.k[b][:, x // pr.G], pr.v[b][:, x // pr.G], ok, scale)
                _fits(t, pr.out[r0:r0 + n, x], want, tol, (scale, b, x))
    h.close()


@pytest.mark.parametrize("dtype,size", [("bf16", 1e3), ("bf16", 1e18), ("fp16", 3e2), ("fp16", 2e4)])
@pytest.mark.parametrize("kind", ["prompt", "cut prompt", "tree"])
def test_large_queries_and_keys(torch, kind, dtype, size):  # noqa: F811
    """The scores themselves are large, up to 2^127. Rows are convex combinations of values; where the largest score is ahead of the
    others by more than fp32 sums are off by, on both sides, and a weight below 2^-64, a row is that token's value. (In fp16 some
    queries and keys of the largest size are infinite: rows whose definition is no number are left out.)"""
    import dynamic_draft_tree_gb300 as dt

    t = torch
    pr = tree.Problem(t, B=2, P=9, H_kv=2, G=2, D=128, page=16, lens=[900, 30], dtype=dtype) if kind == "tree" else \
        prompt.Problem(t, n=[200, 40] if kind == "prompt" else [1400], H_kv=1, G=4, D=64, dtype=dtype)
    pr.q *= size / 2
    for x in (pr.kn, pr.kp):
        x *= size
    pr.k = [x * size for x in pr.k]
    h, ws = pr.handle(dt)
    pr.call(dt, h, ws)
    assert dt.dt_get_status(h) == 0
    u, sure = t.finfo(pr.q.dtype).eps / 2, 0
    for b in range(pr.B):
        L, n = pr.lens[b], pr.n[b]
        r0 = pr.base[b] if kind == "tree" else pr.off[b]
        ok = t.ones(n, L + n, dtype=t.bool, device="cuda")
        ok[:, L:] = pr.mask[b, :n, :n].bool() if kind == "tree" else ok[:, L:].tril()
        for x in range(pr.q.shape[1]):
            q, k, v = (y.double() for y in (pr.q[r0:r0 + n, x], pr.k[b][:, x // pr.G], pr.v[b][:, x // pr.G]))
            got = pr.out[r0:r0 + n, x].double()
            z = (q @ k.T).masked_fill(~ok, -math.inf)
            some = ~(t.isnan(z) | (z == math.inf)).any(1)
            assert bool(t.isfinite(got[some]).all())
            most = t.where(ok[:, :, None], v.abs()[None], 0.0).amax((1, 2))
            assert bool((got.abs().amax(1) <= most * (1 + 3 * u))[some].all())
            two = z.topk(min(2, z.shape[1]), 1)
            off = (pr.D + 8) * 2.0 ** -24 * t.where(ok, q.abs() @ k.abs().T, 0.0).amax(1)
            clear = two.values[:, 0] - two.values[:, -1] > 2 * off + 64 / pr.scale if z.shape[1] > 1 else ok[:, 0]
            clear &= some
            sure += int(clear.sum())
            want = v[two.indices[:, 0]]
            assert bool(((got - want).abs()[clear] <= 2.0 ** -12 * most[clear, None] + u * want.abs()[clear]).all())
    # (an infinite element in 900 keys of 128, one in a thousand beyond 3.3 deviations, leaves no row sure)
    assert sure > 20 or (kind == "tree" and size == 2e4)
    h.close()
