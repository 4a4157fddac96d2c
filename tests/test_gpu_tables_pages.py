"""truncate_block_tables meets page ids that no pool has: pushed as the table has them,
and reported by the call that pushes them."""
import numpy as np
import pytest
import torch

from oracle import tables as T
from tests.helpers import require_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("in_place", [False, True])
def test_pages_below_zero_are_reported(in_place):
    pq = require_gpu()
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")     # noqa: E731
    B, W = 1500, 4
    rng = np.random.default_rng(2)
    lens = rng.integers(0, 16 * W, B, endpoint=True)
    keep = np.maximum(lens - rng.integers(0, 40, B), 0)
    good = np.arange(B * W).reshape(B, W).astype(np.int32)
    first, last = -(-keep // 16), -(-lens // 16)
    s = int(np.flatnonzero(last > first)[-1])
    kept = int(np.flatnonzero(keep > 0)[0])
    for where, bad, told in [(None, 0, 0), ((s, first[s]), -1, 16), ((s, last[s] - 1), -2 ** 31, 16),
                             ((s, first[s]), 2 ** 31 - 1, 0),      # the pool's size is not known
                             ((kept, 0), -1, 0)]:                  # not pushed
        table = good.copy()
        if where:
            table[where] = bad
        stack = np.full(B * W + 3, 7, np.int32)
        sl, fc, fp, status = dev(lens.tolist()), dev([3]), dev(stack.tolist()), dev([0])
        slo, fco = (sl, fc) if in_place else (torch.empty_like(sl), torch.empty_like(fc))
        pq.truncate_block_tables(sl, dev(keep.tolist()), dev(table.tolist()), fp, fc, slo, fco,
                                 status=status)
        want = T.truncate(lens, keep, table, stack, 3)
        assert int(status.item()) == want[3] == told, where
        assert np.array_equal(fp.cpu().numpy(), want[2]) and int(fco.item()) == want[1]
        assert np.array_equal(slo.cpu().numpy(), want[0])
