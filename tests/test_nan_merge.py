"""Merging shares of which one is NaN (a NaN score in it): the row is NaN, and no share that counts
as empty."""
import numpy as np
import pytest
import torch

import oracle
from tests.helpers import require_gpu

NAN, INF = float("nan"), float("inf")
LSE = [[NAN, NAN, -INF, 1.0, NAN], [-INF, 2.0, -INF, -INF, NAN]]
BAD = np.array([True, True, False, False, True])


def test_the_oracle_merges_them_so():
    o = np.random.default_rng(0).normal(size=(2, 5, 128))
    ro, rl = oracle.merge_lse(o, LSE)
    assert np.array_equal(np.isnan(ro).all(-1), BAD) and np.array_equal(np.isnan(rl), BAD)
    assert rl[2] == -INF and (ro[2] == 0).all()
    assert rl[3] == 1.0 and np.array_equal(ro[3], o[0, 3])


@pytest.mark.gpu
def test_merge_keeps_a_nan_share():
    pq = require_gpu()
    o = torch.randn((2, 5, 128), device="cuda")
    out = torch.empty((5, 128), dtype=torch.float16, device="cuda")
    merged = torch.empty(5, device="cuda")
    pq.lse_merge(o, torch.tensor(LSE, device="cuda"), out, merged)
    assert np.array_equal(torch.isnan(out).all(-1).cpu().numpy(), BAD)
    assert np.array_equal(torch.isnan(merged).cpu().numpy(), BAD)
    assert (out[2] == 0).all() and merged[2] == -INF
    assert torch.equal(out[3], o[0, 3].half()) and merged[3] == 1.0
