"""Every way through attention over a 4-bit pool (balanced, fixed splits, windows, shares): page
ids outside the pool, and every element of every sequence within its own bound."""
import numpy as np
import pytest
import torch

import oracle
from tests.helpers import require_gpu
from tests.int4_case import F, Pool, allowance, assert_within

pytestmark = pytest.mark.gpu


def _dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def _attend(p, bt, q, q_len, status=None, **kw):
    out = torch.full(q.shape, float("nan"), dtype=torch.float16, device="cuda")
    require_gpu().paged_attention(_dev(q), _dev(p.pages), _dev(bt), _i32(p.lens), q_len,
                                  "int4_group", None, None, out, status=status, **kw)
    return out


def _partial(pages, bt, lens, pos, q, q_len, status=None, **kw):
    o = torch.full(q.shape, float("nan"), device="cuda")
    lse = torch.full(q.shape[:2], float("nan"), device="cuda")
    require_gpu().paged_attention_partial(_dev(q), _dev(pages), _dev(bt), _i32(lens), _i32(pos), q_len,
                                          "int4_group", None, None, o, lse, status=status, **kw)
    return o, lse.cpu().numpy()


def share_allowance(q, pool, bt, lens, pos, q_len):
    """(reference, bound) of a share's rows, float64: query i of sequence s sees its keys
    j <= pos[s] + i.

    With A = sum_j p_j |V_j|, a row is off by
      2^-11 A             every probability rounded to fp16,
      n 2^-25 max |V|     those under 2^-14 of the reference (the sum is at least 1),
      2 e A               scores: an fp32 sum of 128 exact products is off by at most
                          e = 127 2^-24 max_j sum_d |q_d K_jd| / sqrt(128), in any order; a
                          probability and the sum that divides it by e each,
      2^-18 A             2^x, the sums over the keys (some 20 steps in a row) and the quotient."""
    hkv = pool.shape[1]
    G = q.shape[1] // hkv
    ref, bound = np.zeros(q.shape), np.zeros(q.shape)
    for s, L in enumerate(lens):
        for h in range(hkv if L else 0):
            K, V = oracle.gather_kv(pool, bt[s], L, h, F, None, None)
            at = np.s_[s * q_len:(s + 1) * q_len, h * G:(h + 1) * G]
            z = np.einsum("igd,nd->ign", q[at].astype(np.float64), K) / np.sqrt(128.0)
            sees = np.arange(L)[None] <= pos[s] + np.arange(q_len)[:, None]
            z = np.where(sees[:, None], z, -np.inf)
            p = np.exp(z - z.max(-1, keepdims=True, initial=-1e30))
            p = p / np.maximum(p.sum(-1, keepdims=True), 1e-300)
            ref[at] = p @ V
            size = np.einsum("igd,nd->ign", np.abs(q[at]).astype(np.float64), np.abs(K))
            e = 127 * 2.0 ** -24 / np.sqrt(128.0) * (size * sees[:, None]).max(-1, initial=0)
            bound[at] = p @ np.abs(V) * (2.0 ** -11 + 2.0 ** -18 + 2 * e[..., None]) \
                + L * 2.0 ** -25 * np.abs(V).max(initial=0)
    return ref, bound


@pytest.mark.parametrize("bad", [-1, -2 ** 31, 10 ** 6, 2 ** 31 - 1, "n"])
@pytest.mark.parametrize("q_len", [1, 5, 8])
def test_page_ids_outside_the_pool_read_zeros(q_len, bad):
    """(test_gpu_int4.py has the balanced call.)"""
    pq = require_gpu()
    p = Pool(6, [300, 40], 2, slack=0)
    n = len(p.pages)
    bt, zero = p.bt.copy(), p.bt.copy()
    bt[0, [1, 17]], bt[1, 0] = (n if bad == "n" else bad,) * 2
    zero[0, [1, 17]], zero[1, 0] = n, n
    pool = np.concatenate([p.pages, np.zeros_like(p.pages[:1])])
    q = p.q(5, q_len, 8)
    st = _i32([0])
    for kw in ({"num_splits": 1}, {"num_splits": 3}, {"window": 100}, {"window": 60, "num_splits": 1},
               {"window": 100, "num_splits": 2}):
        ref, bound = allowance(q, pool, zero, p.lens, q_len, window=kw.get("window", 0))
        assert_within(_attend(p, bt, q, q_len, status=st, **kw), ref, bound, "%s" % kw)
        assert pq.status_bits(st) == ["block-table page id out of range"]
        st.zero_()
    pos = [L - q_len for L in p.lens]
    ref, bound = share_allowance(q, pool, zero, p.lens, pos, q_len)
    for splits in (0, 1, 3):
        o, lse = _partial(p.pages, bt, p.lens, pos, q, q_len, status=st, num_splits=splits)
        assert_within(o, ref, bound, "share, %d splits" % splits)
        assert np.isfinite(lse).all()
        assert pq.status_bits(st) == ["block-table page id out of range"]
        st.zero_()


@pytest.mark.parametrize("hq,hkv,q_len", [(16, 16, 1), (24, 8, 5), (32, 4, 4)])
def test_every_element_of_many_short_segments(hq, hkv, q_len):
    """Some 30 segments a CTA, of one to three tiles: a key left out, or one too many, moves an
    output by far more than its bound, which is that of its own row's values."""
    rng = np.random.default_rng(hq)
    lens = rng.integers(q_len, 300, 4500 // hkv)
    p = Pool(1, lens.tolist(), hkv)
    q = p.q(2, q_len, hq)
    ref, bound = share_allowance(q, p.pages, p.bt, lens, lens - q_len, q_len)
    bound += np.maximum(np.abs(ref) * 2.0 ** -11, 2.0 ** -25)              # (fp16 results)
    for kw in ({}, {"num_splits": 1}, {"num_splits": 2}):
        assert_within(_attend(p, p.bt, q, q_len, **kw), ref, bound, "%s" % kw)


@pytest.mark.parametrize("num_splits", [0, 1, 3])
@pytest.mark.parametrize("q_len", [1, 5])
def test_every_element_of_shares(q_len, num_splits):
    p = Pool(21, [40, 333, 1600, 129], 2)
    q = p.q(3, q_len, 8)
    for lo, hi in ((0, 2), (2, 9), (2, 200)):
        n = [min(L, 16 * hi) - min(L, 16 * lo) for L in p.lens]
        bt = np.full((4, max(1, min(hi, p.bt.shape[1]) - lo)), -1, np.int32)
        for s in range(4):
            row = p.bt[s, lo:hi]
            bt[s, :len(row)] = row
        pos = [L - q_len - 16 * lo for L in p.lens]
        ref, bound = share_allowance(q, p.pages, bt, n, pos, q_len)
        o, lse = _partial(p.pages, bt, n, pos, q, q_len, num_splits=num_splits)
        assert_within(o, ref, bound, "share from page %d" % lo)
        rl = oracle.paged_attention_partial(q, p.pages, bt, n, pos, q_len, F, None, None)[1]
        assert np.array_equal(np.isneginf(lse), np.isneginf(rl))
        seen = np.isfinite(rl)
        assert (np.abs(lse[seen] - rl[seen]) <= 2.0 ** -12).all()
