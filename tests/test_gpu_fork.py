"""Requests that continue others: shared pages, the copied last one, and their release, against plain Python (exact)."""
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
    """The pool and its pages' contents in plain Python: rows[block][offset] = a number, one for all planes."""

    def __init__(self, B, max_blocks, n_blocks, page, shared=0):
        self.page, self.max_blocks, self.shared = page, max_blocks, shared // page
        self.table = [[-1] * max_blocks for _ in range(B)]
        self.free = list(range(n_blocks - 1, -1, -1))
        self.n, self.len, self.refs = [0] * B, [0] * B, [0] * n_blocks
        self.rows = [[0] * page for _ in range(n_blocks)]

    def append(self, b, values):
        for v in values:
            if self.len[b] == self.n[b] * self.page:
                self.table[b][self.n[b]] = self.free.pop()
                self.n[b] += 1
            self.rows[self.table[b][self.len[b] // self.page]][self.len[b] % self.page] = v
            self.len[b] += 1

    def fork(self, src, dst, length=None):
        """Bits that the status gets."""
        status, full = 0, False
        have = list(self.len)
        todo = []
        for f, (s, d) in enumerate(zip(src, dst)):
            ok = 0 <= s < len(self.n) and 0 <= d < len(self.n) and s != d and d not in dst[:f] and s not in dst
            n = (have[s] if length is None else length[f]) if ok else 0
            if not ok or not self.shared * self.page <= n <= have[s] or _up(n, self.page) > self.n[s] or self.n[d] != self.shared:
                status |= 64
                continue
            tail = n % self.page
            if tail and (full or not self.free):
                full = True
                status |= 32
                continue
            block = self.free.pop() if tail else None
            todo.append((s, d, n, tail, block))
        for s, d, n, tail, block in todo:
            for e in range(self.shared, n // self.page):
                self.table[d][e] = self.table[s][e]
                self.refs[self.table[s][e]] += 1
            if tail:
                self.table[d][n // self.page] = block
                self.rows[block][:tail] = self.rows[self.table[s][n // self.page]][:tail]
            self.n[d], self.len[d] = _up(n, self.page), n
        return status

    def release(self, keep):
        gave, order = {}, []
        for b, k in enumerate(keep):
            m = min(self.n[b], _up(k, self.page))
            for e in range(m, self.n[b]):
                x = self.table[b][e]
                gave[x] = gave.get(x, 0) + 1
                order.append((b, e, x))
                self.table[b][e] = -1
            self.n[b] = m
        back = []
        for i, (b, e, x) in enumerate(order):
            if any(y == x for _, _, y in order[i + 1:]):
                continue
            if gave[x] > self.refs[x]:
                back.append(x)
                self.refs[x] = 0
            else:
                self.refs[x] -= gave[x]
        self.free += back[::-1]

    def whole(self):
        """Every block is free or owned, as often as it is counted."""
        own = {}
        for b, row in enumerate(self.table):
            for x in row[:self.n[b]]:
                own[x] = own.get(x, 0) + 1
        prefix = set(self.table[0][:self.shared])
        assert sorted(list(own) + self.free) == list(range(len(self.refs)))
        assert all(k == self.refs[x] + 1 for x, k in own.items() if x not in prefix)


class Device:
    def __init__(self, t, dt, plain, planes=3, H=2, D=16, heads_first=False, dtype=None, B_max=None):
        B, n_blocks = len(plain.n), len(plain.refs)
        self.t, self.dt, self.p = t, dt, plain
        self.pool = dt.BlockPool.empty(B, plain.max_blocks, n_blocks, plain.page)
        self.refs = t.zeros(n_blocks, dtype=t.int32, device="cuda")
        self.seq_len = t.zeros(B, dtype=t.int32, device="cuda")
        dtype = dtype or t.bfloat16
        shape = (planes, n_blocks, H, plain.page, D) if heads_first else (planes, n_blocks, plain.page, H, D)
        cache = t.zeros(shape, dtype=dtype, device="cuda")
        self.cache = cache.transpose(2, 3) if heads_first else cache
        self.h = dt.Handle(B_max or B, 2, 1, 1, 1, 1)
        # a plane's and an element's own share of a row's number
        self.own = (t.arange(planes, device="cuda").view(-1, 1, 1) * 7 + t.arange(H * D, device="cuda").view(1, H, D)).to(t.float32)

    def i32(self, v):
        return self.t.tensor(v, dtype=self.t.int32, device="cuda")

    def rows(self, values):
        """[planes][n][H][D]"""
        v = self.t.tensor(values, dtype=self.t.float32, device="cuda")
        return (v.view(1, -1, 1, 1) + self.own.unsqueeze(1)).to(self.cache.dtype)

    def append(self, values):
        """values[b]: numbers of the rows that request b gets."""
        off = [0]
        for v in values:
            off.append(off[-1] + len(v))
        if off[-1] == 0:
            return
        n_new, row_off = self.i32([len(v) for v in values]), self.i32(off)
        slots = self.t.empty(off[-1], dtype=self.t.int64, device="cuda")
        self.dt.dt_kv_reserve(self.h, self.pool, self.seq_len, n_new, slots, slot_off=row_off)
        self.dt.dt_commit_kv_paged(self.h, self.rows([x for v in values for x in v]), self.cache, slots, n_new, self.seq_len,
                                   self.seq_len, row_off=row_off, slot_off=row_off)

    def fork(self, src, dst, length=None, shared=0):
        self.dt.dt_kv_fork(self.h, self.pool, self.refs, self.cache, self.i32(src), self.i32(dst), self.seq_len,
                           length=None if length is None else self.i32(length), shared_len=shared)

    def release(self, keep):
        self.dt.dt_kv_release_shared(self.h, self.pool, self.refs, self.i32(keep))

    def check(self, contents=True):
        p = self.p
        assert self.pool.n_owned.tolist() == p.n and self.pool.block_table.tolist() == p.table
        k = int(self.pool.free_count)
        assert k == len(p.free) and self.pool.free_list[:k].tolist() == p.free
        assert self.refs.tolist() == p.refs
        if contents:
            want = self.rows([x for r in p.rows for x in r]).view(self.cache.shape[0], len(p.rows), p.page, *self.cache.shape[3:])
            used = self.t.tensor([[x != 0 for x in r] for r in p.rows], device="cuda")
            assert self.t.equal(self.cache[:, used], want[:, used])


def _pair(torch, B, max_blocks, n_blocks, page, shared=0, **kw):
    import dynamic_draft_tree_gb300 as dt

    p = Plain(B, max_blocks, n_blocks, page, shared)
    return dt, p, Device(torch, dt, p, **kw)


@pytest.mark.parametrize("seed", range(12))
def test_forks_and_releases_of_a_serving_loop(torch, seed):
    """Requests grow, fork, end and begin again in random order; after every call the pool, the counts, the lengths and
    every row that a request owns are those of the plain pool."""
    rng = random.Random(seed)
    B, page = rng.choice([5, 9, 70]), rng.choice([8, 16, 64])
    dt, p, d = _pair(torch, B, 12, B * 5, page, planes=rng.choice([1, 4]), H=rng.choice([1, 3]), D=rng.choice([8, 24]),
                     heads_first=rng.random() < 0.5)
    counter, expect = 1, 0
    for _ in range(25):
        act = rng.choice(["append", "fork", "fork", "release"])
        if act == "append":
            new = [[] for _ in range(B)]
            left = len(p.free)
            for b in range(B):
                k = rng.choice([0, 0, 1, page - 1, page, page + 3])
                need = _up(p.len[b] + k, page) - p.n[b]
                if k and _up(p.len[b] + k, page) <= p.max_blocks and need <= left:
                    left -= max(0, need)
                    new[b] = [1 + (counter + j) % 120 for j in range(k)]
                    counter += k
            d.append(new)
            for b in range(B):
                p.append(b, new[b])
        elif act == "fork":
            empty = [b for b in range(B) if p.n[b] == 0]
            full = [b for b in range(B) if p.len[b] > 0]
            if not empty or not full:
                continue
            dst = rng.sample(empty, rng.randint(1, len(empty)))
            src = [rng.choice(full) for _ in dst]
            length = [rng.randint(0, p.len[s]) for s in src] if rng.random() < 0.5 else None
            d.fork(src, dst, length)
            expect |= p.fork(src, dst, length)
        else:
            keep = [p.len[b] if rng.random() < 0.6 else 0 for b in range(B)]
            d.release(keep)
            p.release(keep)
            for b in range(B):
                if keep[b] == 0:
                    p.len[b] = 0
            d.seq_len.copy_(d.i32(p.len))
        p.whole()
        d.check()
        assert d.seq_len.tolist() == p.len
    assert dt.dt_get_status(d.h) == expect
    d.h.close()


def test_forks_that_are_refused(torch):
    dt, p, d = _pair(torch, 8, 4, 12, 8)
    values = [[1 + j for j in range(19)], [40 + j for j in range(8)]] + [[] for _ in range(6)]
    d.append(values)
    for b, v in enumerate(values):
        p.append(b, v)

    def fork(src, dst, length=None):
        d.fork(src, dst, length)
        want = p.fork(src, dst, length)
        d.check()
        assert d.seq_len.tolist() == p.len
        got = dt.dt_get_status(d.h)
        dt.dt_clear_status(d.h)
        assert got == want
        return got

    assert fork([0], [1]) == 64          # owns pages
    assert fork([0], [0]) == 64          # itself
    assert fork([0, 9, -1], [-1, 2, 2]) == 64
    assert fork([0], [2], [20]) == 64    # more than there is
    assert fork([0], [2], [-1]) == 64
    assert fork([0, 1], [2, 2]) == 64    # the second one of the same place
    assert fork([2, 0], [3, 2]) == 64    # a source that is a destination, a destination that owns pages
    assert fork([0, 1, 0, 0, 0, 0, 0], [3, 4, 5, 6, 7, 3, 0]) == 64
    p.release([19, 8] + [0] * 6)
    d.release([19, 8] + [0] * 6)
    for b in range(2, 8):
        p.len[b] = 0
    d.seq_len.copy_(d.i32(p.len))
    d.check()
    d.append([[], []] + [[], [9] * 30] + [[]] * 4)  # four blocks of the eight that are left
    p.append(3, [9] * 30)
    d.append([[], [], [], [], [8] * 17] + [[]] * 3)
    p.append(4, [8] * 17)
    d.check()
    assert fork([0, 1, 0, 4], [2, 5, 6, 7]) == 32  # one page left: the first one's; the second one needs none
    assert p.n[2] == 3 and p.n[5] == 1 and p.n[6] == 0 and p.n[7] == 0
    assert fork([0, 0], [6, 7], [16, 3]) == 32
    d.h.close()


@pytest.mark.parametrize("n_blocks, bits", [(500, 64), (300, 96)])
def test_more_forks_than_threads(torch, n_blocks, bits):
    """600 samples of three prompts in one call (about 400 of them need a page), some refused, pages for all or for most."""
    dt, p, d = _pair(torch, 700, 3, n_blocks, 8, planes=1, H=1, D=8)
    values = [[1 + j for j in range(19)], [30 + j for j in range(16)], [60 + j for j in range(5)]] + [[]] * 697
    d.append(values)
    for b in range(3):
        p.append(b, values[b])
    rng = random.Random(5)
    dst = rng.sample(range(3, 700), 600)
    src = [rng.randrange(3) for _ in dst]
    dst[100], dst[300], src[400] = dst[50], 1, dst[10]
    d.fork(src, dst)
    want = p.fork(src, dst)
    d.check()
    assert d.seq_len.tolist() == p.len and dt.dt_get_status(d.h) == want == bits
    keep = [0 if rng.random() < 0.7 else p.len[b] for b in range(700)]
    d.release(keep)
    p.release(keep)
    p.whole()
    d.check()
    keep = [0] * 700
    d.release(keep)
    p.release(keep)
    d.check()
    assert len(p.free) == n_blocks and not any(p.refs)
    d.h.close()


def test_a_release_undoes_a_fork(torch):
    """Ending the samples leaves the free list in the order it had, so that the next ones take the same pages."""
    dt, p, d = _pair(torch, 9, 6, 60, 16)
    values = [[1 + j for j in range(50)]] + [[]] * 8
    d.append(values)
    p.append(0, values[0])
    before = d.pool.free_list[:int(d.pool.free_count)].tolist()
    for _ in range(3):
        d.fork([0] * 8, list(range(1, 9)))
        d.release([50] + [0] * 8)
        assert d.pool.free_list[:int(d.pool.free_count)].tolist() == before and not d.refs.any()
    assert dt.dt_get_status(d.h) == 0
    d.h.close()


def test_keeping_part_of_a_shared_page_is_reported(torch):
    dt, p, d = _pair(torch, 3, 6, 20, 16)
    values = [[1 + j for j in range(50)], [], []]
    d.append(values)
    p.append(0, values[0])
    d.fork([0], [1])
    p.fork([0], [1])
    d.release([50, 32, 0])  # whole pages: its own to go on behind
    p.release([50, 32, 0])
    d.check()
    assert dt.dt_get_status(d.h) == 0
    d.release([50, 20, 0])  # the second page is request 0's too
    p.release([50, 20, 0])
    d.check()
    assert dt.dt_get_status(d.h) == dt.DT_DEV_BAD_PAGE
    dt.dt_clear_status(d.h)
    d.release([0, 20, 0])  # now it is its own
    p.release([0, 20, 0])
    d.check()
    assert dt.dt_get_status(d.h) == 0
    d.h.close()


def test_a_shared_prefix_is_counted_nowhere(torch):
    """Forks behind a prefix that every place owns: the destination keeps it, and gives it back to nobody."""
    dt, p, d = _pair(torch, 5, 6, 30, 8, shared=16)
    d.append([[1 + j for j in range(16)], [], [], [], []])
    p.append(0, [1 + j for j in range(16)])
    for b in range(1, 5):
        p.table[b][:2], p.n[b], p.len[b] = p.table[0][:2], 2, 16
    d.pool.block_table[1:, :2] = d.pool.block_table[:1, :2]
    d.pool.n_owned[1:] = 2
    d.seq_len[1:] = 16
    d.append([[], [50 + j for j in range(13)], [], [], []])
    p.append(1, [50 + j for j in range(13)])
    for src, dst, length in (([1, 0], [2, 3], None), ([1, 1], [4, 3], [24, 15])):
        d.fork(src, dst, length, shared=16)
        p.fork(src, dst, length)
        d.check()
        assert d.seq_len.tolist() == p.len
    assert dt.dt_get_status(d.h) == dt.DT_DEV_BAD_PAGE  # 15 tokens end inside the prefix
    keep = [16, 16, 16, 16, p.len[4]]
    d.release(keep)
    p.release(keep)
    d.check()
    d.h.close()


def test_corrupt_tables_are_reported(torch):
    dt, p, d = _pair(torch, 4, 4, 16, 8)
    d.append([[1 + j for j in range(20)], [], [], []])
    keep = d.cache.clone()
    d.pool.block_table[0, 2] = 16
    d.fork([0], [1])
    assert dt.dt_get_status(d.h) & dt.DT_DEV_BAD_PAGE and d.t.equal(keep, d.cache)
    dt.dt_clear_status(d.h)
    d.pool.block_table[0, 0] = -5
    d.release([0, 0, 0, 0])
    assert dt.dt_get_status(d.h) & dt.DT_DEV_BAD_PAGE
    dt.dt_clear_status(d.h)
    d.pool.n_owned[2] = 5
    d.release([0, 0, 0, 0])
    assert dt.dt_get_status(d.h) & dt.DT_DEV_BAD_PAGE
    d.pool.n_owned[2] = 0
    dt.dt_clear_status(d.h)
    d.release([0, 0, 0, -1])
    assert dt.dt_get_status(d.h) & dt.DT_DEV_BAD_PAGE
    d.h.close()


def test_captured_forks_follow_the_arrays(torch):
    dt, p, d = _pair(torch, 6, 6, 40, 8)
    values = [[1 + j for j in range(21)], [50 + j for j in range(30)]] + [[]] * 4
    d.append(values)
    for b in range(2):
        p.append(b, values[b])
    src, dst, keep = d.i32([0, 0]), d.i32([2, 3]), d.i32([21, 30, 0, 0, 0, 0])

    def step():
        d.dt.dt_kv_release_shared(d.h, d.pool, d.refs, keep)
        d.dt.dt_kv_fork(d.h, d.pool, d.refs, d.cache, src, dst, d.seq_len)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            step()
    torch.cuda.synchronize()
    p.fork([0, 0], [2, 3])
    d.check()
    src.copy_(d.i32([1, 0]))
    dst.copy_(d.i32([5, 4]))
    g.replay()
    torch.cuda.synchronize()
    p.release([21, 30, 0, 0, 0, 0])
    p.len[2] = p.len[3] = 0
    p.fork([1, 0], [5, 4])
    d.check()
    assert dt.dt_get_status(d.h) == 0
    d.h.close()


def test_refusals(torch):
    dt, p, d = _pair(torch, 4, 4, 16, 8)
    one = d.i32([0])
    for bad in (dict(refs=d.refs[:4]), dict(refs=d.refs.long()), dict(cache=d.cache[0]), dict(cache=d.cache[:, :8]),
                dict(cache=d.cache[..., ::2]), dict(dst=d.i32([])), dict(seq_len=d.seq_len[:2]), dict(length=one.float())):
        a = dict(refs=d.refs, cache=d.cache, src=one, dst=d.i32([1]), seq_len=d.seq_len, length=None)
        a.update(bad)
        with pytest.raises(ValueError):
            dt.dt_kv_fork(d.h, d.pool, a["refs"], a["cache"], a["src"], a["dst"], a["seq_len"], length=a["length"])
    for kw in (dict(shared_len=5), dict(shared_len=-8), dict(shared_len=40)):
        with pytest.raises(dt.DtError) as e:
            dt.dt_kv_fork(d.h, d.pool, d.refs, d.cache, one, d.i32([1]), d.seq_len, **kw)
        assert e.value.code == dt.DT_ERR_ARG
    with pytest.raises(dt.DtError):
        dt.dt_kv_fork(d.h, d.pool, d.refs, d.cache, d.i32([0] * 5), d.i32([1] * 5), d.seq_len)  # more than B_max
    with pytest.raises(dt.DtError):
        dt.dt_kv_fork(d.h, d.pool, d.refs, d.cache[..., :4], one, d.i32([1]), d.seq_len)  # rows of 8 bytes
    with pytest.raises(ValueError):
        dt.dt_kv_release_shared(d.h, d.pool, d.refs, d.i32([0] * 5))
    torch.cuda.synchronize()
    assert dt.dt_get_status(d.h) == 0
    d.h.close()
