"""Pages: reservation and slot maps, release, commit, against plain Python on the same inputs (exact)."""
import random

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


class Plain:
    """The pool in plain Python: one request after another."""

    def __init__(self, B, max_blocks, n_blocks, page):
        self.page, self.max_blocks = page, max_blocks
        self.table = [[-1] * max_blocks for _ in range(B)]
        self.free = list(range(n_blocks - 1, -1, -1))
        self.n = [0] * B

    def reserve(self, lens, n_new, room):
        """Slots of every request, None for one that is not served."""
        got, lacked, have = [], 0, len(self.free)
        for b, (x, k) in enumerate(zip(lens, n_new)):
            want = _up(x + k, self.page)
            if want > self.max_blocks or k > room[b]:
                got.append(None)
                continue
            need = max(0, want - self.n[b])
            lacked += need
            if need and lacked > have:
                got.append(None)
                continue
            for e in range(need):
                self.table[b][self.n[b]] = self.free.pop()
                self.n[b] += 1
            got.append([self.table[b][(x + j) // self.page] * self.page + (x + j) % self.page for j in range(k)])
        return got

    def release(self, keep):
        back = []
        for b, x in enumerate(keep):
            m = min(self.n[b], _up(x, self.page))
            back += self.table[b][m:self.n[b]]
            self.table[b][m:] = [-1] * (self.max_blocks - m)
            self.n[b] = m
        self.free += back[::-1]


def _same(t, pool, plain):
    assert pool.block_table.tolist() == plain.table
    assert pool.n_owned.tolist() == plain.n
    k = int(pool.free_count)
    assert pool.free_list[:k].tolist() == plain.free


@pytest.mark.parametrize("B,page,top,n_blocks", [(1, 16, 40, 20), (7, 8, 30, 60), (8, 16, 17, 500), (64, 16, 300, 900),
                                                 (300, 32, 9, 1000), (3, 256, 5000, 200), (1100, 8, 3, 3000)])
@pytest.mark.parametrize("packed", [False, True])
def test_reserve_and_release_match_plain(torch, B, page, top, n_blocks, packed):
    """Several rounds of growing, rolling back and ending requests, with a pool that runs short."""
    import dynamic_draft_tree_gb300 as dt

    r = random.Random(B * 1000 + page)
    h = dt.Handle(B, 2, 1, 1, 1, 1)
    mb = _up(4 * top, page) + 1
    pool, plain = dt.BlockPool.empty(B, mb, n_blocks, page), Plain(B, mb, n_blocks, page)
    lens = [0] * B
    i32 = dict(dtype=torch.int32, device="cuda")
    for rnd in range(6):
        n = [r.choice([0, 1, r.randint(0, top)]) for _ in range(B)]
        extra = rnd % 2
        k = [x + extra for x in n]
        room = [top + 1] * B
        off = [0]
        for x in k:
            off.append(off[-1] + x)
        d_len = torch.tensor(lens, **i32)
        if packed:
            room = k
            slots = torch.full((off[-1] + 3,), -9, dtype=torch.int64, device="cuda")
            dt.dt_kv_reserve(h, pool, d_len, torch.tensor(n, **i32), slots, n_extra=extra,
                             slot_off=torch.tensor(off, **i32), S=top + 1)
        else:
            slots = torch.full((B, top + 1), -9, dtype=torch.int64, device="cuda")
            dt.dt_kv_reserve(h, pool, d_len, torch.tensor(n, **i32), slots, n_extra=extra)
        status = dt.dt_get_status(h)
        dt.dt_clear_status(h)
        want = plain.reserve(lens, k, room)
        assert bool(status & dt.DT_DEV_KV_FULL) == any(w is None for w in want)
        assert status & ~dt.DT_DEV_KV_FULL == 0
        got = slots.tolist()
        for b in range(B):
            mine = got[off[b]:off[b + 1]] if packed else got[b]
            w = want[b] if want[b] is not None else []
            assert mine == w + [-1] * (len(mine) - len(w)), b
        if packed:
            assert got[off[-1]:] == [-9] * 3
        _same(torch, pool, plain)
        for b in range(B):  # served requests commit some of their tokens, the rest is rolled back
            if want[b] is not None:
                lens[b] += r.randint(0, k[b])
            if r.random() < 0.2:
                lens[b] = 0
        dt.dt_kv_release(h, pool, torch.tensor(lens, **i32))
        plain.release(lens)
        _same(torch, pool, plain)
    assert dt.dt_get_status(h) == 0
    h.close()


def test_reserving_twice_takes_nothing_more(torch):
    import dynamic_draft_tree_gb300 as dt

    h = dt.Handle(2, 2, 1, 1, 1, 1)
    pool = dt.BlockPool.empty(2, 8, 10, 16)
    i32 = dict(dtype=torch.int32, device="cuda")
    lens, n = torch.tensor([0, 0], **i32), torch.tensor([20, 16], **i32)
    a, b = (torch.zeros(2, 20, dtype=torch.int64, device="cuda") for _ in range(2))
    dt.dt_kv_reserve(h, pool, lens, n, a)
    dt.dt_kv_reserve(h, pool, lens, n, b)
    assert torch.equal(a, b) and int(pool.free_count) == 7
    assert a[0].tolist() == list(range(0, 20)) and a[1].tolist() == list(range(32, 48)) + [-1] * 4
    h.close()


def test_corrupt_state_is_reported(torch):
    import dynamic_draft_tree_gb300 as dt

    h = dt.Handle(3, 2, 1, 1, 1, 1)
    i32 = dict(dtype=torch.int32, device="cuda")
    one = torch.tensor([1, 1, 1], **i32)
    for what in range(4):
        pool = dt.BlockPool.empty(3, 4, 6, 16)
        lens, off = torch.zeros(3, **i32), torch.tensor([0, 1, 2, 3], **i32)
        if what == 0:
            lens[1] = -1
        elif what == 1:
            pool.n_owned[1] = 5
        elif what == 2:
            pool.free_list[4] = 6  # request 1's block
        else:
            off[2:] = torch.tensor([9, 10], **i32)
        slots = torch.full((3,), -9, dtype=torch.int64, device="cuda")
        dt.dt_kv_reserve(h, pool, lens, one, slots, slot_off=off, S=4)
        assert dt.dt_get_status(h) == dt.DT_DEV_BAD_PAGE
        dt.dt_clear_status(h)
        got = slots.tolist()
        assert got[0] == 0 and got[1] == (-9 if what == 3 else -1)
    h.close()


@pytest.mark.parametrize("planes,H,D,page,heads_first,dtype", [(2, 1, 64, 16, False, "bfloat16"),
                                                               (5, 3, 80, 8, True, "float16"),
                                                               (64, 8, 128, 64, False, "bfloat16"),
                                                               (3, 5, 96, 32, True, "float32"),
                                                               (1, 1, 16, 256, False, "uint8")])
@pytest.mark.parametrize("packed", [False, True])
def test_commit_into_pages(torch, planes, H, D, page, heads_first, dtype, packed):
    import dynamic_draft_tree_gb300 as dt

    B, P, S = 5, 23, 9
    r = random.Random(planes * 100 + D)
    h = dt.Handle(B, 2, 1, 1, 1, P)
    n = [9, 0, 1, 5, 8]
    start = [r.randint(0, 40) for _ in range(B)]
    pool = dt.BlockPool.empty(B, 16, 60, page)
    i32 = dict(dtype=torch.int32, device="cuda")
    acc = torch.tensor([x - 1 for x in n], **i32)
    seq = torch.tensor(start, **i32)
    slots = torch.zeros(B, S, dtype=torch.int64, device="cuda")
    dt.dt_kv_reserve(h, pool, seq, acc, slots, n_extra=1)
    path = torch.tensor([sorted(r.sample(range(P), S)) for _ in range(B)], **i32)
    off = [0, 23, 40, 41, 64, 87] if packed else [b * P for b in range(B + 1)]
    path[2, 0] = 0
    td = getattr(torch, dtype)
    raw = torch.randint(0, 256, (planes, off[-1] if packed else B * P, H, D * (td.itemsize)), device="cuda",
                        dtype=torch.uint8)
    tmp = raw.view(td) if td.itemsize > 1 else raw
    shape = (planes, 60, H, page, D) if heads_first else (planes, 60, page, H, D)
    pages = torch.zeros(shape, dtype=td, device="cuda")
    cache = pages.transpose(2, 3) if heads_first else pages
    want = cache.clone()
    for b in range(B):
        for j in range(n[b]):
            s = int(slots[b, j])
            want[:, s // page, s % page] = tmp[:, off[b] + int(path[b, j])]
    out = torch.zeros(B, **i32)
    if packed:
        dt.dt_commit_kv_paged(h, tmp, cache, slots, acc, seq, out, path=path, row_off=torch.tensor(off, **i32),
                              n_extra=1, P=P)
    else:
        dt.dt_commit_kv_paged(h, tmp.view(planes, B, P, H, D), cache, slots, acc, seq, out, path=path, n_extra=1)
    assert dt.dt_get_status(h) == 0
    assert out.tolist() == [x + k for x, k in zip(start, n)]
    assert torch.equal(cache.contiguous().view(torch.uint8), want.contiguous().view(torch.uint8))
    dt.dt_commit_kv_paged(h, tmp if packed else tmp.view(planes, B, P, H, D), cache, slots, acc, seq, seq, path=path,
                          row_off=torch.tensor(off, **i32) if packed else None, n_extra=1,
                          P=P if packed else None)  # lengths in place
    assert torch.equal(seq, out)
    h.close()


def test_commit_of_prompts(torch):
    """Packed prompts and packed slots, no path; a request without pages commits nothing."""
    import dynamic_draft_tree_gb300 as dt

    B, page = 4, 16
    n = [300, 1, 0, 129]
    off = [0, 300, 301, 301, 430]
    i32 = dict(dtype=torch.int32, device="cuda")
    d_off, d_n, seq = torch.tensor(off, **i32), torch.tensor(n, **i32), torch.zeros(B, **i32)
    h = dt.Handle(B, 2, 1, 1, 1, 1)
    pool = dt.BlockPool.empty(B, 32, 22, page)  # 19 + 1 blocks; the last prompt's nine are not there
    slots = torch.full((430,), -9, dtype=torch.int64, device="cuda")
    dt.dt_kv_reserve(h, pool, seq, d_n, slots, slot_off=d_off)
    tmp = torch.randn(3, 430, 2, 64, device="cuda", dtype=torch.bfloat16)
    cache = torch.zeros(3, 22, page, 2, 64, device="cuda", dtype=torch.bfloat16)
    dt.dt_commit_kv_paged(h, tmp, cache, slots, d_n, seq, seq, row_off=d_off, slot_off=d_off)
    assert dt.dt_get_status(h) == dt.DT_DEV_KV_FULL
    assert seq.tolist() == [300, 1, 0, 0]
    flat = cache.view(3, 22 * page, 2, 64)
    assert torch.equal(flat[:, :300], tmp[:, :300]) and torch.equal(flat[:, 304], tmp[:, 300])
    assert not flat[:, 305:].any() and not flat[:, 300:304].any()
    h.close()


def test_commit_reports_bad_slots_and_rows(torch):
    import dynamic_draft_tree_gb300 as dt

    h = dt.Handle(1, 2, 1, 1, 1, 1)
    i32 = dict(dtype=torch.int32, device="cuda")
    tmp = torch.ones(1, 1, 4, 1, 64, device="cuda", dtype=torch.bfloat16)
    for slot, path, bit in ((64, 0, dt.DT_DEV_BAD_PAGE), (5, 4, dt.DT_DEV_BAD_TREE), (5, -1, dt.DT_DEV_BAD_TREE)):
        cache = torch.zeros(1, 4, 16, 1, 64, device="cuda", dtype=torch.bfloat16)
        seq = torch.zeros(1, **i32)
        dt.dt_commit_kv_paged(h, tmp, cache, torch.tensor([[slot]], device="cuda"), torch.tensor([1], **i32), seq, seq,
                              path=torch.tensor([[path]], **i32))
        assert dt.dt_get_status(h) == bit
        assert not cache.any()
        dt.dt_clear_status(h)
    h.close()


def test_refusals(torch):
    import dynamic_draft_tree_gb300 as dt

    h = dt.Handle(2, 2, 1, 1, 1, 1)
    i32 = dict(dtype=torch.int32, device="cuda")
    pool = dt.BlockPool.empty(2, 4, 6, 16)
    two, slots = torch.ones(2, **i32), torch.zeros(2, 4, dtype=torch.int64, device="cuda")

    def no(error, f, *a, **k):
        with pytest.raises(error):
            f(*a, **k)

    no(ValueError, dt.dt_kv_reserve, h, pool, two, torch.ones(3, **i32), slots)
    no(ValueError, dt.dt_kv_reserve, h, pool, two, two, slots.int())
    no(ValueError, dt.dt_kv_reserve, h, pool, two[:1], two, slots)
    no(ValueError, dt.dt_kv_reserve, h, pool, two, two, slots.view(-1))
    no(dt.DtError, dt.dt_kv_reserve, h, pool, two, two, slots, n_extra=-1)
    no(dt.DtError, dt.dt_kv_reserve, dt.Handle(1, 2, 1, 1, 1, 1), pool, two, two, slots)
    no(dt.DtError, dt.dt_kv_release, h, dt.BlockPool.empty(2, 4, 6, 24), two)
    no(ValueError, dt.BlockPool, torch.zeros(2, 4, **i32).t(), two, two, two, 16)
    no(ValueError, dt.dt_kv_release, h, pool, two.cpu())
    tmp = torch.zeros(2, 2, 3, 1, 64, device="cuda", dtype=torch.bfloat16)
    cache = torch.zeros(2, 6, 16, 1, 64, device="cuda", dtype=torch.bfloat16)
    good = dict(h=h, tmp=tmp, cache=cache, slots=slots, n_new=two, seq_len=two, len_out=two)
    for over in (dict(cache=cache[:, :, :, :, :32]), dict(cache=cache[0]), dict(cache=cache.half()),
                 dict(tmp=tmp[:, :, ::2]), dict(len_out=two.long()), dict(slots=slots[:1])):
        no(ValueError, dt.dt_commit_kv_paged, **dict(good, **over))
    no(dt.DtError, dt.dt_commit_kv_paged, **dict(good, cache=cache[:, :, :12]))
    no(dt.DtError, dt.dt_commit_kv_paged, **dict(good, tmp=tmp[..., :4], cache=cache[..., :4]))
    dt.dt_commit_kv_paged(**good)
    h.close()


def test_commit_says_what_it_appended(torch):
    """committed: the tokens of served requests; 0 where slots are missing, the path is too short, n is 0 or negative."""
    import dynamic_draft_tree_gb300 as dt

    B, S, page = 5, 4, 8
    i32 = dict(dtype=torch.int32, device="cuda")
    h = dt.Handle(B, 2, 1, 1, 1, 8)
    slots = torch.arange(B * S, dtype=torch.int64, device="cuda").view(B, S)
    slots[1, 2:] = -1
    acc, seq = torch.tensor([3, 2, 4, -1, -5], **i32), torch.tensor([4, 5, 6, 7, 8], **i32)
    path = torch.arange(S, **i32).expand(B, S).contiguous()
    tmp = torch.randn(2, B, 8, 1, 16, device="cuda").bfloat16()
    cache = torch.zeros(2, 3, page, 1, 16, device="cuda").bfloat16()
    done, out = torch.full((B + 1,), -7, **i32), torch.zeros(B, **i32)
    dt.dt_commit_kv_paged(h, tmp, cache, slots, acc, seq, out, path=path, n_extra=1, committed=done)
    assert done.tolist() == [4, 0, 0, 0, 0, -7] and out.tolist() == [8, 5, 6, 7, 8]
    assert dt.dt_get_status(h) == dt.DT_DEV_KV_FULL | dt.DT_DEV_BAD_PAGE
    with pytest.raises(ValueError):
        dt.dt_commit_kv_paged(h, tmp, cache, slots, acc, seq, out, path=path, n_extra=1, committed=done[:B - 1])
    with pytest.raises(ValueError):
        dt.dt_commit_kv_paged(h, tmp, cache, slots, acc, seq, out, path=path, n_extra=1, committed=done.long())
    h.close()
