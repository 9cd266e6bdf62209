"""dt_token_logprobs within a bound that goes by the distances of a row's logits, not by the logits (tests/test_logprob_bounds.py)."""
import math

import pytest

from test_gpu_logprobs import torch  # noqa: F401 (the fixture)
from test_gpu_logprobs_edges import _labels
from test_logprob_bounds import H, bounds

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("V", [33, 1000, 9001, 152064])
@pytest.mark.parametrize("spread,offset", [(0.0, 0.0), (0.5, 0.0), (3.0, 0.0), (60.0, 0.0), (3000.0, 0.0), (3.0, 300.0), (3.0, -5000.0), (30.0, 1e6)])
def test_errors_go_by_distances(torch, spread, offset, V, dtype):  # noqa: F811
    import dynamic_draft_tree_gb300 as dt

    t = torch
    g = t.Generator(device="cuda")
    g.manual_seed(V + int(spread) + int(offset))
    n, K = 6, 5
    x = (t.randn(n, V, generator=g, device="cuda") * spread + offset).to(t.bfloat16 if dtype == "bf16" else t.float32)
    x[n - 1, ::3] = -math.inf
    tokens = t.randint(0, V, (n,), generator=g, device="cuda", dtype=t.int32)
    tokens[:2] = x[:2].argmax(1).int()
    status, logp, ent, rank, ids, alt = _labels(t, dt, x, tokens, K)
    assert status == 0
    for r in range(n):
        row = x[r].double().cpu().numpy()
        log_s, want, tol, tol_h = bounds(row)
        m = row.max()

        def near(got, xt):
            w = xt - m - log_s
            assert got == w if w == -math.inf else abs(got - w) <= tol + H * abs(w), (r, got, w, tol)

        near(float(logp[r]), row[int(tokens[r])])
        assert abs(float(ent[r]) - want) <= tol_h, (r, float(ent[r]), want, tol_h)
        for k in range(K):
            near(float(alt[r, k]), row[int(ids[r, k])])
