"""Shares that end inside a page, whose queries lie at or behind their end: keys behind the end
(rejected draft tokens, another request's, or bytes that nothing wrote) are never seen, in any
format and with any split, for any q_pos."""
import numpy as np
import pytest
import torch

import oracle
import workloads as W
from tests.helpers import require_gpu
from tests.int4_case import F, Pool, assert_within, slots, tables

pytestmark = pytest.mark.gpu
FORMATS = [W.FP16, W.FP8_E4M3, W.INT8, W.INT8_ROW, F]
LENS = [5, 24, 130, 399]
BEHIND = 9                      # tokens written behind each share's end


def _dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


@pytest.fixture(scope="module", params=FORMATS)
def pool(request):
    pq, fmt, H = require_gpu(), request.param, 2
    rng = np.random.default_rng(5)
    bt, n = tables(rng, [L + BEHIND for L in LENS])
    at = np.concatenate([slots(bt, s, 0, L + BEHIND) for s, L in enumerate(LENS)])
    k, v = (rng.normal(size=(len(at), H, 128)).astype(np.float16) for _ in "kv")
    end = np.cumsum([L + BEHIND for L in LENS])
    for e in end:
        v[e - BEHIND:e] = 8                       # seen, they would move every output
    scale = np.full(1, 8 / 127, np.float32) if fmt == W.INT8 else np.full(1, 0.03, np.float32)
    pages = pq.new_pages(n, H, fmt, fill=0xFF if fmt == F else 0)
    pq.kv_append_quant(_dev(k), _dev(v), _dev(at), fmt, _dev(scale), _dev(scale), pages)
    ref = oracle.new_pool(n, H, 128, fmt, fill=0xFF if fmt == F else 0)
    if fmt == W.INT8_ROW:
        z = oracle.new_scale_pool(n, H)
        ref, ks, vs = oracle.kv_append_quant(k, v, at, fmt, z, z, ref)
    else:
        ref, ks, vs = oracle.kv_append_quant(k, v, at, fmt, scale, scale, ref), scale, scale
    return pq, fmt, H, bt, pages, _dev(scale), ref, ks, vs


@pytest.mark.parametrize("q_len,G", [(1, 4), (3, 1), (4, 4), (5, 5), (8, 4)])
@pytest.mark.parametrize("num_splits", [0, 1, 3])
def test_keys_behind_a_share_are_not_seen(pool, q_len, G, num_splits):
    """Off by at most, with M = max |V| of the tokens seen (below 8): every probability's half
    step in fp16, 2^-11 M; scores in fp32, whose errors move a probability by less than 2^-13 of
    itself; and half a step of 2^-24 for those under 2^-14 of the reference, n 2^-25 M, of
    INT8_ROW for those whose product with the row's scale (above 1 / 64: N(0, 1) rows have values
    above 2 in 128) is."""
    pq, fmt, H, bt, pages, scale, ref, ks, vs = pool
    q = np.random.default_rng(q_len).normal(size=(len(LENS) * q_len, H * G, 128)).astype(np.float16)
    M = 5.5
    for pos in ([L - 1 for L in LENS], [L + 3 for L in LENS],
                [2 ** 31 - 1, 2 ** 31 - 3, 10 ** 9, 16 * 30], [-1, 12, 2 ** 31 - 1, -2 ** 31]):
        ro, rl = oracle.paged_attention_partial(q, ref, bt, LENS, pos, q_len, fmt, ks, vs)
        o = torch.full(q.shape, float("nan"), device="cuda")
        lse = torch.full(q.shape[:2], float("nan"), device="cuda")
        pq.paged_attention_partial(_dev(q), pages, _dev(bt), _i32(LENS), _i32(pos), q_len, fmt,
                                   scale, scale, o, lse, num_splits=num_splits)
        bound = np.full(q.shape, M * (2.0 ** -11 + 2.0 ** -13 + 64 * 400 * 2.0 ** -25))
        assert_within(o, ro, bound, "q_pos %s" % pos)
        got = lse.cpu().numpy()
        assert np.array_equal(np.isneginf(got), np.isneginf(rl)) and not np.isnan(got).any()
        seen = np.isfinite(rl)
        assert (np.abs(got[seen] - rl[seen]) <= 2.0 ** -12).all()


@pytest.mark.parametrize("num_splits", [0, 1, 2])
def test_unwritten_bytes_behind_a_share_at_4_bits(num_splits):
    """They are NaN scales here."""
    pq = require_gpu()
    p = Pool(8, [5, 200, 131], 2)
    q_len = 4
    q = p.q(9, q_len, 8)
    pos = [5, 10 ** 9, 2 ** 31 - 1]
    M = max(np.abs(oracle.gather_kv(p.pages, p.bt[s], L, h, F, None, None)[1]).max()
            for s, L in enumerate(p.lens) for h in range(2))
    ro, rl = oracle.paged_attention_partial(q, p.pages, p.bt, p.lens, pos, q_len, F, None, None)
    o = torch.full(q.shape, float("nan"), device="cuda")
    lse = torch.full(q.shape[:2], float("nan"), device="cuda")
    pq.paged_attention_partial(_dev(q), _dev(p.pages), _dev(p.bt), _i32(p.lens), _i32(pos), q_len,
                               "int4_group", None, None, o, lse, num_splits=num_splits)
    assert_within(o, ro, np.full(q.shape, M * (2.0 ** -11 + 2.0 ** -13 + 200 * 2.0 ** -25)))
    assert (np.abs(lse.cpu().numpy() - rl) <= 2.0 ** -12).all()
