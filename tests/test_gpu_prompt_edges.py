"""dt_prompt_attention and forks at the edges: offsets past 31 bits, two calls at once, idle places, a cache that is used on another
stream than its own."""
import pytest

from test_gpu_prompt import Problem, _check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    import torch as t

    if not t.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__

    __graft_entry__.build()
    return t


def test_offsets_past_31_bits(torch):
    """Pages and rows so far apart that elements lie past 2^31 (and bytes past 2^32)."""
    import dynamic_draft_tree_gb300 as dt

    t = torch
    pr = Problem(t, n=[40, 3], H_kv=2, G=2, D=64, lens=[70, 33], page=16)
    h, ws = pr.handle(dt)
    pr.call(dt, h, ws)
    near = pr.out.clone()
    blocks, rows = pr.kp.shape[0], pr.q.shape[0]
    k_block, q_row = 1 << 28, 1 << 26
    buf = t.zeros(max(blocks << 28, rows << 26) + (1 << 24), dtype=t.bfloat16, device="cuda")
    assert (blocks - 1) * k_block > 1 << 31 and (rows - 1) * q_row > 1 << 31

    def far(x, step, at):
        y = buf[at:].as_strided(x.shape, (step,) + x.stride()[1:])
        y.copy_(x)
        return y

    pr.kp, pr.vp = far(pr.kp, k_block, 0), far(pr.vp, k_block, 1 << 16)
    pr.q, pr.kn, pr.vn = far(pr.q, q_row, 1 << 17), far(pr.kn, q_row, 1 << 18), far(pr.vn, q_row, 1 << 19)
    pr.out = far(t.full_like(near, 7.0), q_row, 1 << 20)
    pr.call(dt, h, ws)
    assert dt.dt_get_status(h) == 0
    assert t.equal(near, pr.out)
    h.close()


@pytest.mark.parametrize("G,D,dtype", [(4, 128, "bf16"), (1, 64, "fp16"), (5, 80, "bf16")])
def test_values_that_are_no_numbers_in_cut_items(torch, G, D, dtype):
    """Infinities and NaN in the values of a prompt that several CTAs work on, at the borders of tiles and items: they show in the
    rows that attend to them, in their elements alone."""
    import dynamic_draft_tree_gb300 as dt

    pr = Problem(torch, n=[2500, 20], H_kv=2, G=G, D=D, lens=[300, 3000], seed=G, dtype=dtype)
    for k, (at, x) in enumerate(((0, float("inf")), (127, float("nan")), (128, float("-inf")), (1000, float("inf")),
                                 (1919, float("nan")), (2047, float("-inf")), (2499, float("nan")))):
        d = (11 * k + 3) % D
        pr.vn[at, :, d] = x
        pr.v[0][300 + at, :, d] = x
    h, ws = pr.handle(dt)
    pr.call(dt, h, ws)
    assert dt.dt_get_status(h) == 0
    got = pr.out.clone()
    pr.out.fill_(7.0)
    _check(pr, got)
    h.close()


def test_two_calls_at_once(torch):
    """Two streams, one handle, a workspace each: cut items of both."""
    import dynamic_draft_tree_gb300 as dt

    t = torch
    prs = [Problem(t, n=[700, 30, 1], H_kv=4, G=2, D=128, lens=[500, 3, 900], seed=k) for k in range(2)]
    h, ws0 = prs[0].handle(dt)
    wss = [ws0, t.empty_like(ws0)]
    want = []
    for pr, ws in zip(prs, wss):
        pr.call(dt, h, ws)
        want.append(pr.out.clone())
        pr.out.fill_(7.0)
    t.cuda.synchronize()
    streams = [t.cuda.Stream(), t.cuda.Stream()]
    for _ in range(20):
        for pr, ws, s in zip(prs, wss, streams):
            pr.call(dt, h, ws, stream=s)
    t.cuda.synchronize()
    assert dt.dt_get_status(h) == 0
    for pr, w in zip(prs, want):
        assert t.equal(pr.out, w)
    h.close()


def test_all_places_idle(torch):
    """Lengths without rows: nothing is read or written."""
    import dynamic_draft_tree_gb300 as dt

    pr = Problem(torch, n=[0, 0, 0], H_kv=2, G=2, D=64, lens=[30, 0, 7])
    h, ws = pr.handle(dt)
    ws.fill_(0xFF)
    for _ in range(3):
        pr.call(dt, h, ws)
    assert dt.dt_get_status(h) == 0 and bool((pr.out == 7.0).all())
    h.close()


@pytest.mark.parametrize("G", [1, 4, 128])
def test_one_position_a_request(torch, G):
    """The decode form: single tokens behind caches of every length around the tiles' borders, in one batch with a prompt."""
    import dynamic_draft_tree_gb300 as dt

    lens = [0, 1, 63, 64, 65, 127, 128, 129, 1000, 2500]
    pr = Problem(torch, n=[1] * len(lens) + [130], H_kv=1, G=G, D=64, lens=lens + [77], page=64, seed=G)
    h, ws = pr.handle(dt)
    pr.call(dt, h, ws)
    assert dt.dt_get_status(h) == 0
    got = pr.out.clone()
    pr.out.fill_(7.0)
    _check(pr, got)
    h.close()


def test_pages_larger_than_the_rows_before(torch):
    """More cached tokens than whole items allow: the items are cut and joined; fewer: they are not. Both agree with the definition
    at the rule's border."""
    import dynamic_draft_tree_gb300 as dt

    for blocks in (3, 4, 5, 6):  # 256 tokens each; with the rows' tile 7, 9, 11 and 13 tiles
        pr = Problem(torch, n=[100], H_kv=2, G=4, D=128, lens=[256 * blocks - 5], page=256, seed=blocks)
        h, ws = pr.handle(dt)
        pr.call(dt, h, ws)
        assert dt.dt_get_status(h) == 0
        got = pr.out.clone()
        pr.out.fill_(7.0)
        _check(pr, got)
        h.close()


def test_forks_past_31_bits(torch):
    """Pages 2^29 elements apart: the last tokens of a fork are copied there."""
    import dynamic_draft_tree_gb300 as dt

    t, page, H, D, blocks = torch, 16, 2, 64, 5
    block, plane = 1 << 29, 1 << 23
    buf = t.zeros((blocks - 1) * block + 2 * plane, dtype=t.bfloat16, device="cuda")
    cache = buf.as_strided((2, blocks, page, H, D), (plane, block, H * D, D, 1))
    h = dt.Handle(3, 2, 1, 1, 1, 1)
    pool = dt.BlockPool.empty(3, 2, blocks, page)
    refs, seq_len = t.zeros(blocks, dtype=t.int32, device="cuda"), t.zeros(3, dtype=t.int32, device="cuda")
    i32 = lambda v: t.tensor(v, dtype=t.int32, device="cuda")
    rows = t.randn(2, 23, H, D, device="cuda").to(t.bfloat16)
    n_new, off = i32([23, 0, 0]), i32([0, 23, 23, 23])
    slots = t.empty(23, dtype=t.int64, device="cuda")
    dt.dt_kv_reserve(h, pool, seq_len, n_new, slots, slot_off=off)
    dt.dt_commit_kv_paged(h, rows, cache, slots, n_new, seq_len, seq_len, row_off=off, slot_off=off)
    dt.dt_kv_fork(h, pool, refs, cache, i32([0, 0]), i32([2, 1]), seq_len, length=i32([23, 21]))
    assert dt.dt_get_status(h) == 0 and seq_len.tolist() == [23, 21, 23]
    table = pool.block_table.tolist()
    assert table[0][0] == table[1][0] == table[2][0] and len({r[1] for r in table}) == 3
    assert refs[table[0][0]] == 2
    for b, n in ((1, 5), (2, 7)):
        assert t.equal(cache[:, table[b][1], :n], rows[:, 16:16 + n])
        assert bool((cache[:, table[b][1], n:] == 0).all())
    h.close()


def test_a_cache_on_another_stream(torch):
    """Prompts, a fork and a release of a cache, all on a stream that is not the current one."""
    import dynamic_draft_tree_gb300 as dt
    from dynamic_draft_tree_gb300.paged import PagedCache

    t = torch
    h = dt.Handle(4, 32, 4, 4, 2, 8)
    results = []
    for stream in (None, t.cuda.Stream()):
        g = t.Generator(device="cuda")
        g.manual_seed(9)
        kv = PagedCache(h, 4, 8, 1, 4, 2, 64, n_blocks=20, max_blocks=5, forks=True)
        off, n = t.tensor([0, 37, 37, 60, 60], dtype=t.int32, device="cuda"), t.tensor([37, 0, 23, 0], dtype=t.int32, device="cuda")
        q, out = t.randn(60, 4, 64, generator=g, device="cuda").to(t.bfloat16), t.zeros(60, 4, 64, dtype=t.bfloat16, device="cuda")
        rows = t.randn(2, 60, 2, 64, generator=g, device="cuda").to(t.bfloat16)
        src, dst = t.tensor([0, 2], dtype=t.int32, device="cuda"), t.tensor([1, 3], dtype=t.int32, device="cuda")
        keep = t.tensor([37, 37, 0, 23], dtype=t.int32, device="cuda")
        t.cuda.synchronize()
        kv.attend_prompts(0, q, rows[0], rows[1], off, out, stream=stream)
        kv.prefill(rows, n, off, stream=stream)
        kv.fork(src, dst, stream=stream)
        kv.release(keep, stream=stream)
        t.cuda.synchronize()
        assert dt.dt_get_status(h) == 0
        results.append([out, kv.seq_len, kv.refs, kv.pool.block_table, kv.pool.n_owned, kv.pool.free_count])
    assert all(t.equal(a, b) for a, b in zip(*results))
    assert float(results[0][0].abs().max()) > 0
    h.close()
