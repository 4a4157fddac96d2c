"""Scores of great size, up to 2^25: fp32 steps there are several units of the exponent, so a
softmax is one over the keys with the largest score, and its references must not carry a
probability out of fp16's range, or under it."""
import numpy as np
import pytest
import torch

import workloads as W
from tests.helpers import require_gpu
from tests.int4_case import F, slots, tables

pytestmark = pytest.mark.gpu
FORMATS = [W.FP16, W.FP8_E4M3, W.INT8, W.INT8_ROW, F]
LENS = [20, 700, 2500]


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("q_len", [1, 5])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("size", [2.0 ** 8, 2.0 ** 14])
def test_the_keys_with_the_largest_score_have_the_row(fmt, q_len, sign, size):
    """Every dim of a key is the same, so that keys of one size have one score in every format, and
    a row's result is the mean of the best keys' V: off by half a step of fp16 of each of the
    probabilities, their products with INT8_ROW's scales, kv_read's INT8_ROW values and the result."""
    pq, H, hq = require_gpu(), 1, 4
    rng = np.random.default_rng(q_len)
    bt, n = tables(rng, LENS)
    total = sum(LENS)
    step = rng.choice([28.0, 56.0, 112.0], total)
    ends = np.cumsum(LENS)
    step[[3, 11, 20 + 5, 20 + 130, 20 + 640, 720 + 100, 720 + 2000]] = 224.0
    if sign < 0:
        step = step[::-1].copy()
    k = np.repeat(np.repeat(step[:, None, None], H, 1), 128, 2).astype(np.float16)
    v = np.repeat(rng.choice([-2.0, -1.0, 1.0, 2.0], (total, H, 1)), 128, 2).astype(np.float16)
    pages = pq.new_pages(n, H, fmt, fill=0)
    one = torch.ones(1, device="cuda")
    two = torch.full((1,), 2.0, device="cuda")
    at = np.concatenate([slots(bt, s, 0, L) for s, L in enumerate(LENS)])
    dev = [torch.from_numpy(x).cuda() for x in (k, v, at)]
    pq.kv_append_quant(*dev, fmt, two, one, pages)
    ko, vo = (torch.empty(k.shape, dtype=torch.float16, device="cuda") for _ in "kv")
    btd = torch.from_numpy(bt).cuda()
    pq.kv_read(pages, btd, None, _i32(np.concatenate([[0], ends])), fmt, two, one, ko, vo)
    K, V = ko.double().cpu().numpy()[:, 0], vo.double().cpu().numpy()[:, 0]
    q = np.full((len(LENS) * q_len, hq, 128), sign * size, np.float16)
    ref = np.zeros(q.shape)
    for s, (a, b) in enumerate(zip(np.concatenate([[0], ends]), ends)):
        for i in range(q_len):
            x = (K[a:b - q_len + i + 1] * sign * size).sum(-1) / np.sqrt(128.0)
            p = np.exp(x - x.max())
            ref[s * q_len + i] = (p / p.sum()) @ V[a:b - q_len + i + 1]
    qd, lens = torch.from_numpy(q).cuda(), _i32(LENS)
    for call, kw in ((pq.paged_attention, {}), (pq.paged_attention, {"num_splits": 1}),
                     (pq.paged_attention, {"num_splits": 3}), (pq.paged_attention_shared_prefix, {})):
        out = torch.full_like(qd, float("nan"))
        groups = [_i32([0, 1, 2, 3]), _i32([0, 640, 2400])] if "shared" in call.__name__ else []
        call(qd, pages, btd, lens, *groups, q_len, fmt, two, one, out, **kw)
        g = out.double().cpu().numpy()
        what = "%s %s" % (call.__name__, kw)
        assert np.isfinite(g).all(), what
        assert (np.abs(g - ref) <= 2.0 * (4 * 2.0 ** -11 + 2500 * 2.0 ** -25)).all(), what
