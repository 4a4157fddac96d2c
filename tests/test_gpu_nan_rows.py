"""A NaN among the scores that a row sees makes the row NaN, whatever the length, the split and
the merge: zeros, or a share that counts as empty, would hide it.  The other rows keep their
values."""
import numpy as np
import pytest
import torch

import workloads as W
from tests.helpers import assert_close, require_gpu
from tests.int4_case import F, Pool, allowance, assert_within, slots, tables

pytestmark = pytest.mark.gpu
FORMATS = [W.FP16, W.FP8_E4M3, W.INT8, W.INT8_ROW, F]
LENS = [20, 128, 900, 3000]        # one tile, one CTA's share, several


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


class Step:
    """Requests of LENS in a pool of any format, and a batch's queries."""

    def __init__(self, fmt, q_len, hq, hkv, lens=LENS):
        pq = require_gpu()
        self.pq, self.fmt, self.q_len, self.lens = pq, fmt, q_len, lens
        rng = np.random.default_rng(q_len)
        bt, n = tables(rng, lens)
        self.bt = torch.from_numpy(bt).cuda()
        self.pages = pq.new_pages(n, hkv, fmt, fill=0)
        self.scale = torch.full((1,), 0.03, device="cuda")
        gen = torch.Generator(device="cuda").manual_seed(q_len)
        at = np.concatenate([slots(bt, s, 0, L) for s, L in enumerate(lens)])
        k, v = (torch.randn((len(at), hkv, 128), generator=gen, device="cuda").half() for _ in "kv")
        pq.kv_append_quant(k, v, torch.from_numpy(at).cuda(), fmt, self.scale, self.scale, self.pages)
        self.q = torch.randn((len(lens) * q_len, hq, 128), generator=gen, device="cuda").half()

    def args(self, q):
        return q, self.pages, self.bt, _i32(self.lens)

    def plain(self, q, **kw):
        out = torch.full_like(q, 7.0)
        self.pq.paged_attention(*self.args(q), self.q_len, self.fmt, self.scale, self.scale, out, **kw)
        return out

    def noalloc(self, q):
        out = torch.full_like(q, 7.0)
        self.pq.paged_attention_noalloc(*self.args(q), self.q_len, self.fmt, self.scale, self.scale,
                                        out)
        return out

    def shared(self, q):
        out = torch.full_like(q, 7.0)
        self.pq.paged_attention_shared_prefix(
            *self.args(q), _i32([0, 1, len(self.lens)]), _i32([16, 0]), self.q_len, self.fmt,
            self.scale, self.scale, out)
        return out

    def partial(self, q, **kw):
        o = torch.full(q.shape, 7.0, device="cuda")
        lse = torch.full(q.shape[:2], 7.0, device="cuda")
        self.pq.paged_attention_partial(*self.args(q), _i32(self.lens) - self.q_len, self.q_len,
                                        self.fmt, self.scale, self.scale, o, lse, **kw)
        return o, lse


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("q_len,hq,hkv", [(1, 8, 2), (5, 8, 2), (3, 14, 2), (8, 8, 2)])
def test_a_nan_in_a_query_stays_in_its_row(fmt, q_len, hq, hkv):
    c = Step(fmt, q_len, hq, hkv)
    q = c.q.clone()
    bad = torch.zeros(q.shape[:2], dtype=torch.bool, device="cuda")
    for s in range(len(LENS)):
        row, head = s * q_len + s % q_len, (3 * s + 1) % hq
        q[row, head, 17 * s] = float("nan") if s % 2 else float("inf")
        bad[row, head] = True
    calls = [(c.plain, {}), (c.plain, {"num_splits": 1}), (c.plain, {"num_splits": 3}),
             (c.plain, {"window": 50}), (c.plain, {"window": 50, "num_splits": 2}),
             (c.noalloc, {}), (c.shared, {})]
    for call, kw in calls:
        want, got = call(c.q, **kw), call(q, **kw)
        what = "%s %s" % (call.__name__, kw)
        nan = torch.isnan(got).all(-1)
        # (an infinity in a query gives +-inf scores: NaN unless all of them are -inf)
        assert nan[bad].all(), what
        assert torch.equal(nan, bad) and torch.isfinite(got[~bad]).all(), what
        assert_close(got[~bad], want[~bad].double().cpu().numpy(), what)
    for kw in ({}, {"num_splits": 1}, {"num_splits": 3}):
        want, got = c.partial(c.q, **kw), c.partial(q, **kw)
        for w, g in zip(want, got):
            nan = torch.isnan(g) if g.dim() == 2 else torch.isnan(g).all(-1)
            assert torch.equal(nan, bad), "partial %s" % kw
            assert_close(g[~bad].half(), w[~bad].double().cpu().numpy(), "partial %s" % kw)
        merged, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
        c.pq.lse_merge(got[0][None].contiguous(), got[1][None].contiguous(), merged, lse)
        assert torch.equal(torch.isnan(merged).all(-1), bad) and torch.equal(torch.isnan(lse), bad)


@pytest.mark.parametrize("L", [7, 100, 128, 200, 5000])
@pytest.mark.parametrize("kw", [{}, {"num_splits": 1}, {"num_splits": 2}])
def test_a_nan_scale_of_a_key_at_4_bits(L, kw):
    """In contexts of one tile, of one share and of several: the rows that see the key are NaN,
    those before it are not touched, and a share's LSE says so too."""
    pq = require_gpu()
    p = Pool(31, [L], 1)
    tile = p.pages.reshape(len(p.pages), 1, 2, 1152)
    page, r = p.bt[0, (L - 2) // 16], (L - 2) % 16
    tile[page, 0, 0, 1024 + 2 * r:1026 + 2 * r] = [0, 0x7E]
    q = p.q(32, 5, 4)                                      # positions L - 5 .. L - 1
    dev = [torch.from_numpy(np.ascontiguousarray(x)).cuda() for x in (q, p.pages, p.bt)]
    out = torch.empty(q.shape, dtype=torch.float16, device="cuda")
    pq.paged_attention(*dev, _i32([L]), 5, "int4_group", None, None, out, **kw)
    assert torch.isnan(out[3:]).all()
    ref, bound = allowance(q[:3], p.pages, p.bt, [L - 2], 3)
    assert_within(out[:3], ref, bound)
    o, lse = torch.empty(q.shape, device="cuda"), torch.empty(q.shape[:2], device="cuda")
    pq.paged_attention_partial(*dev, _i32([L]), _i32([L - 5]), 5, "int4_group", None, None, o, lse,
                               **kw)
    assert torch.isnan(o[3:]).all() and torch.isnan(lse[3:]).all()
    assert torch.isfinite(o[:3]).all() and torch.isfinite(lse[:3]).all()
