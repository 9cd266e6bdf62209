"""Forks and shared releases over tables of every size: those that one CTA releases, those that three launches do with the last CTA
changing the counts, and those with a launch for them; against plain Python (exact)."""
import random

import pytest

from test_gpu_fork import _pair, _up

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    import torch as t

    if not t.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__

    __graft_entry__.build()
    return t


@pytest.mark.parametrize("B,max_blocks", [(1, 1024), (17, 60), (18, 60), (64, 40), (65, 40), (300, 7)])
def test_tables_of_every_size(torch, B, max_blocks):
    rng, page = random.Random(B), 8
    dt, p, d = _pair(torch, B, max_blocks, 6 * max_blocks + B, page, planes=2, H=1, D=8)
    first = [rng.randint(page * max_blocks // 2, page * max_blocks - 2) if b < 3 else 0 for b in range(B)]
    values = [[1 + (b * 31 + j) % 120 for j in range(n)] for b, n in enumerate(first)]
    d.append(values)
    for b, v in enumerate(values):
        p.append(b, v)
    for turn in range(4):
        empty = [b for b in range(B) if p.n[b] == 0]
        full = [b for b in range(B) if p.len[b] > 0]
        dst = rng.sample(empty, min(len(empty), 1 + len(empty) * turn // 3))
        if dst and full:
            src = [rng.choice(full) for _ in dst]
            length = [rng.randint(0, p.len[s]) for s in src] if turn % 2 else None
            d.fork(src, dst, length)
            assert p.fork(src, dst, length) in (0, 32)
        d.check()
        assert d.seq_len.tolist() == p.len
        keep = [p.len[b] if rng.random() < 0.5 else 0 for b in range(B)]
        if turn == 3:
            keep = [0] * B
        d.release(keep)
        p.release(keep)
        p.whole()
        d.check()
        for b in range(B):
            p.len[b] = p.len[b] if keep[b] else 0
        d.seq_len.copy_(d.i32(p.len))
    assert not any(p.refs) and len(p.free) == 6 * max_blocks + B
    assert dt.dt_get_status(d.h) & ~32 == 0
    d.h.close()


def test_a_destination_that_is_a_source(torch):
    """A chain in one call: the fork of the place that another fork fills is refused, the other one is served."""
    dt, p, d = _pair(torch, 4, 4, 12, 8)
    d.append([[1 + j for j in range(11)], [], [], []])
    p.append(0, [1 + j for j in range(11)])
    d.fork([1, 0], [2, 1])
    assert p.fork([1, 0], [2, 1]) == 64 and dt.dt_get_status(d.h) == 64
    d.check()
    assert d.seq_len.tolist() == p.len == [11, 11, 0, 0]
    d.h.close()


def test_forks_of_nothing(torch):
    """A length of zero takes no page and owns none."""
    dt, p, d = _pair(torch, 3, 4, 4, 8)
    d.append([[5] * 9, [], []])
    p.append(0, [5] * 9)
    d.fork([0, 0], [1, 2], [0, 8])
    assert p.fork([0, 0], [1, 2], [0, 8]) == 0 and dt.dt_get_status(d.h) == 0
    d.check()
    assert d.seq_len.tolist() == [9, 0, 8]
    d.h.close()
