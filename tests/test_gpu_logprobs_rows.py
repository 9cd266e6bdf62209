"""dt_token_logprobs along paths through packed rows: an entry's row is one of its own request's, whatever the path says."""
import math

import pytest

from test_gpu_logprobs import Problem, torch  # noqa: F401 (the fixture)

pytestmark = pytest.mark.gpu


def _run(pr, dt, h, ws):
    for x in (pr.logp, pr.entropy, pr.rank, pr.top_ids, pr.top_logp):
        x.fill_(7)
    pr.call(dt, h, ws)
    bits = dt.dt_get_status(h)
    dt.dt_clear_status(h)
    return bits


def _untouched(pr, b, j):
    return all(bool((x[b, j] == 7).all()) for x in (pr.logp, pr.entropy, pr.rank, pr.top_ids, pr.top_logp))


def test_positions_outside_the_requests_rows_are_reported(torch):  # noqa: F811
    """Positions below P whose row would be another request's, or lies behind all of them."""
    import dynamic_draft_tree_gb300 as dt

    pr = Problem(torch, form="path", used=[9, 5], n=[4, 3], V=3000, K=2, packed=True, P=14)
    h, ws = pr.handle(dt)
    assert _run(pr, dt, h, ws) == 0
    pr.check()
    fine = [x.clone() for x in (pr.logp, pr.entropy, pr.rank)]
    for b, j, first in ((0, 2, 9), (1, 1, 5)):
        was = int(pr.path[b, j])
        for pos in (first, first + 1, 13, 14, -1):
            pr.path[b, j] = pos
            assert _run(pr, dt, h, ws) == dt.DT_DEV_BAD_TREE, (b, pos)
            assert _untouched(pr, b, j)
            # the entry in front of it has a row, but no token
            assert math.isnan(pr.logp[b, j - 1]) and pr.rank[b, j - 1] == -1 and pr.entropy[b, j - 1] == fine[1][b, j - 1]
            for o in range(2):
                for k in range(pr.n[o]):
                    if o != b or k not in (j - 1, j):
                        assert all(x[o, k] == y[o, k] for x, y in zip((pr.logp, pr.entropy, pr.rank), fine))
        pr.path[b, j] = was
    assert _run(pr, dt, h, ws) == 0
    pr.check()
    h.close()


@pytest.mark.parametrize("V", [700, 40000])
def test_counts_and_offsets_that_do_not_fit_the_rows_are_reported(torch, V):  # noqa: F811
    import dynamic_draft_tree_gb300 as dt

    pr = Problem(torch, form="path", used=[9, 5, 3], n=[4, 3, 1], V=V, K=2, packed=True, S=12)
    h, ws = pr.handle(dt)
    assert _run(pr, dt, h, ws) == 0
    pr.path[1, :6] = torch.tensor([0, 1, 2, 3, 4, 4], dtype=torch.int32)
    pr.n_new[1] = 5  # six entries, five rows, twelve places
    assert _run(pr, dt, h, ws) == dt.DT_DEV_BAD_TREE and _untouched(pr, 1, slice(None))
    pr.n_new[1] = 4  # all of its rows
    assert _run(pr, dt, h, ws) == 0 and not bool((pr.logp[1, :5] == 7).any())
    # request 1's rows end before they begin; request 2 has rows
    pr.row_off.copy_(torch.tensor([0, 9, 4, 17], dtype=torch.int32))
    assert _run(pr, dt, h, ws) == dt.DT_DEV_BAD_TREE and _untouched(pr, 1, slice(None))
    assert bool(torch.isfinite(pr.entropy[0, :4]).all()) and math.isfinite(pr.entropy[2, 0]) and pr.entropy[2, 0] != 7
    h.close()


def test_a_path_longer_than_its_tree_is_reported(torch):  # noqa: F811
    """More entries than the tree has positions, in padded rows."""
    import dynamic_draft_tree_gb300 as dt

    pr = Problem(torch, form="path", used=[4, 4], n=[3, 2], V=900, K=1, S=9)
    h, ws = pr.handle(dt)
    pr.path[0, :5] = torch.tensor([0, 1, 2, 3, 3], dtype=torch.int32)
    pr.n_new[0] = 4
    assert _run(pr, dt, h, ws) == dt.DT_DEV_BAD_TREE and _untouched(pr, 0, slice(None))
    assert bool(torch.isfinite(pr.logp[1, :2]).all())
    h.close()
