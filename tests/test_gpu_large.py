"""Offsets past 32 bits: pages, slots and rows beyond 2^31 elements, and calls of two streams at once."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    import torch as t

    if not t.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__

    __graft_entry__.build()
    yield t
    t.cuda.empty_cache()


def test_attention_over_the_end_of_a_large_cache(torch):
    """Keys and values of 2.4e9 elements each (4.8 GB); the tokens lie in the last blocks, against a small cache."""
    import dynamic_draft_tree_gb300 as dt

    B, P, H_kv, G, D, page, n_blocks = 2, 5, 8, 4, 128, 16, 147000
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    h = dt.Handle(B, 2, 1, 1, 1, P)
    ws = dt.dt_tree_attention_workspace(h, B, P, H_kv * G, H_kv, D)
    lens = torch.tensor([100, 250], dtype=torch.int32, device="cuda")
    need = 7 + 16
    small = [torch.randn(need, page, H_kv, D, generator=g, device="cuda").bfloat16() for _ in range(2)]
    large = [torch.empty(n_blocks, page, H_kv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    for s, big in zip(small, large):
        big[-need:] = s
    table = torch.full((B, 16), -1, dtype=torch.int32, device="cuda")
    table[0, :7] = torch.arange(7)
    table[1, :16] = torch.arange(7, 23)
    q = torch.randn(B, P, H_kv * G, D, generator=g, device="cuda").bfloat16()
    kn, vn = (torch.randn(B, P, H_kv, D, generator=g, device="cuda").bfloat16() for _ in range(2))
    n = torch.full((B,), P, dtype=torch.int32, device="cuda")
    out = [torch.empty_like(q) for _ in range(2)]
    high = torch.where(table >= 0, table + (n_blocks - need), -1).to(torch.int32)
    dt.dt_tree_attention(h, q, kn, vn, *small, table, lens, n, out[0], ws)
    dt.dt_tree_attention(h, q, kn, vn, *large, high, lens, n, out[1], ws)
    assert dt.dt_get_status(h) == 0
    assert torch.equal(*out) and torch.isfinite(out[0]).all() and out[0].abs().sum() > 0
    h.close()


def test_slots_past_32_bits(torch):
    """2^31 + 512 slots of 16 bytes (34 GB): reserved from the highest blocks, committed and read back."""
    import dynamic_draft_tree_gb300 as dt

    page, n_blocks, B = 256, 2 ** 23 + 2, 2
    i32 = dict(dtype=torch.int32, device="cuda")
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("less than 60 GB free")
    free = torch.zeros(n_blocks, **i32)
    free[:3] = torch.tensor([n_blocks - 1, n_blocks - 2, n_blocks - 3])
    pool = dt.BlockPool(torch.full((B, 4), -1, **i32), torch.zeros(B, **i32), free, torch.tensor([3], **i32), page)
    h = dt.Handle(B, 2, 1, 1, 1, 1)
    n = torch.tensor([300, 20], **i32)
    slots = torch.zeros(B, 300, dtype=torch.int64, device="cuda")
    seq = torch.zeros(B, **i32)
    dt.dt_kv_reserve(h, pool, seq, n, slots)
    want = torch.full((B, 300), -1, dtype=torch.int64)
    j = torch.arange(300)
    want[0] = torch.where(j < 256, (n_blocks - 3) * page + j, (n_blocks - 2) * page + j - 256)
    want[1, :20] = (n_blocks - 1) * page + j[:20]
    assert torch.equal(slots.cpu(), want) and int(want.max()) > 2 ** 31
    cache = torch.empty(1, n_blocks, page, 1, 8, dtype=torch.bfloat16, device="cuda")
    tmp = torch.randn(1, B, 300, 1, 8, device="cuda").bfloat16()
    dt.dt_commit_kv_paged(h, tmp, cache, slots, n, seq, seq)
    assert dt.dt_get_status(h) == 0 and seq.tolist() == [300, 20]
    flat = cache.view(-1, 8)
    for b, k in ((0, 300), (1, 20)):
        assert torch.equal(flat[slots[b, :k]], tmp[0, b, :k, 0])
    h.close()


def test_rows_past_32_bits(torch):
    """40 x 512 rows of 128256 (2.6e9 elements, 5.3 GB), processed in place; the last request is looked at."""
    import dynamic_draft_tree_gb300 as dt

    B, P, V = 40, 512, 128256
    h = dt.Handle(B, V, 1, 1, 1, P)
    n = torch.zeros(B, dtype=torch.int32, device="cuda")
    n[-1] = P
    x = torch.empty(B, P, V, dtype=torch.bfloat16, device="cuda")
    x[-1] = torch.randn(P, V, device="cuda")
    before = x[-1, -3:].float()
    counts = torch.zeros(B, V, dtype=torch.int32, device="cuda")
    counts[-1, ::7] = 1
    two = torch.full((B,), 2.0, device="cuda")
    dt.dt_logits_process(h, x, x, n, counts=counts, repetition=two)
    assert dt.dt_get_status(h) == 0
    want = before.clone()
    want[:, ::7] = torch.where(before[:, ::7] > 0, before[:, ::7] / 2, before[:, ::7] * 2)
    assert torch.equal(x[-1, -3:].float(), want)  # halving and doubling are exact
    h.close()


def test_two_streams_with_a_handle_and_workspace_each(torch):
    """Attention, pages and rows of two handles interleaved on two streams give what they give alone."""
    import dynamic_draft_tree_gb300 as dt
    from test_gpu_attention import CASES, Problem

    probs = [Problem(torch, **CASES[k]) for k in ("cast tree packed", "long")]
    made = [p.handle(dt) for p in probs]
    alone = []
    for p, (h, ws) in zip(probs, made):
        p.call(dt, h, ws)
        torch.cuda.synchronize()
        alone.append(p.out.clone())
        p.out.fill_(7.0)
    streams = [torch.cuda.Stream() for _ in probs]
    torch.cuda.synchronize()
    for _ in range(20):
        for p, (h, ws), s in zip(probs, made, streams):
            p.call(dt, h, ws, stream=s)
    torch.cuda.synchronize()
    for p, (h, ws), want in zip(probs, made, alone):
        assert dt.dt_get_status(h) == 0
        assert torch.equal(p.out, want)
        h.close()
