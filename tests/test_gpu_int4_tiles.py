"""The tcgen05 kernel of 4-bit pools where its tiles, fragments and references can go wrong:
many short segments a CTA, the largest batch, scores that rise from tile to tile, rows
that see nothing, other lengths than the tables hold."""
import ctypes
import time

import numpy as np
import pytest
import torch

import oracle
import workloads as W
from tests.helpers import Case, require_gpu
from tests.int4_case import F, Pool, allowance, assert_within, slots
from tests.test_gpu_wait_timeout import _run_test_mode

pytestmark = pytest.mark.gpu


def _dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def _attend(pages, bt, lens, q, q_len, status=None, **kw):
    pq = require_gpu()
    out = torch.full(q.shape, float("nan"), dtype=torch.float16, device="cuda")
    pq.paged_attention(_dev(q), pages, bt, _i32(lens), q_len, "int4_group", None, None, out,
                       status=status, **kw)
    return out


@pytest.mark.parametrize("hq,hkv,q_len", [(16, 16, 1), (24, 8, 5), (32, 4, 4)])
def test_many_fragments_a_cta(hq, hkv, q_len):
    """Some 30 segments a CTA, of one to three tiles."""
    rng = np.random.default_rng(hq)
    lens = rng.integers(q_len, 300, 4500 // hkv)
    p = Pool(1, lens.tolist(), hkv)
    q = p.q(2, q_len, hq)
    out = _attend(_dev(p.pages), _dev(p.bt), lens, q, q_len)
    # every 17th sequence against the oracle, all of them against fixed splits
    for s in range(0, len(lens), 17):
        ref, bound = allowance(q[s * q_len:(s + 1) * q_len], p.pages, p.bt[s:s + 1], lens[s:s + 1],
                               q_len)
        assert_within(out[s * q_len:(s + 1) * q_len], ref, bound, "sequence %d" % s)
    other = _attend(_dev(p.pages), _dev(p.bt), lens, q, q_len, num_splits=1)
    # Either is off by at most what allowance() counts with A <= M = max |V| (a stored value is at
    # most 1 + 2^-8 of the largest given one), and half an fp16 step of a value <= M, so the two
    # are within twice that of each other.  (0.06, which stood here, is less than one step, 2^-4,
    # of the fp16 outputs between 64 and 128 that this pool has.)
    M = 1.01 * float(np.abs(p.v.astype(np.float64)).max())
    assert (out.float() - other.float()).abs().max() <= \
        2 * M * (2 * 2.0 ** -11 + 2.0 ** -13 + max(lens) * 2.0 ** -25)


def test_the_largest_batch():
    """2048 sequences: the tables' part of shared memory leaves the fewest stages."""
    rng = np.random.default_rng(3)
    lens = rng.integers(1, 90, 2048)
    lens[1000] = 3000
    p = Pool(4, lens.tolist(), 1)
    q = p.q(5, 1, 4)
    out = _attend(_dev(p.pages), _dev(p.bt), lens, q, 1)
    for s in list(range(0, 2048, 101)) + [1000]:
        ref, bound = allowance(q[s:s + 1], p.pages, p.bt[s:s + 1], lens[s:s + 1], 1)
        assert_within(out[s:s + 1], ref, bound, "sequence %d" % s)
    win = _attend(_dev(p.pages), _dev(p.bt), lens, q, 1, window=40)
    for s in (7, 1000):
        ref, bound = allowance(q[s:s + 1], p.pages, p.bt[s:s + 1], lens[s:s + 1], 1, window=40)
        assert_within(win[s:s + 1], ref, bound, "sequence %d in a window" % s)


@pytest.mark.parametrize("q_len", [1, 5, 8])
def test_scores_that_rise_and_fall(q_len):
    """K along one direction, its length rising over the tiles (each raises every row's
    reference), then falling to nothing, then one key far above all."""
    L = 1500
    p = Pool(6, [L], 2)
    t = np.arange(L)
    size = np.where(t < 1000, t / 100.0, 0.01)
    size[1400] = 14.0
    k = np.repeat(size[:, None, None], 128, -1) * np.ones((1, 2, 1))
    v = p.v
    pool = oracle.kv_append_quant(k.astype(np.float16), v, slots(p.bt, 0, 0, L), F, None, None,
                                  p.pages)
    q = np.abs(p.q(7, q_len, 8)) * 0.3
    q[:, ::2] *= -1
    q = q.astype(np.float16)
    ref, bound = allowance(q, pool, p.bt, [L], q_len)
    # scores reach 14 * 0.3 * 128 / sqrt(128): fp32 is off by 2^-24 of 128 times as much
    bound = bound + 128 * 2.0 ** -24 * 90 * np.abs(v.astype(np.float64)).max()
    for kw in ({}, {"num_splits": 1}):
        assert_within(_attend(_dev(pool), _dev(p.bt), [L], q, q_len, **kw), ref, bound)


def test_partial_rows_that_see_nothing_and_far_positions():
    pq = require_gpu()
    p = Pool(8, [400, 200, 131], 2)
    q_len, hq = 4, 8
    q = p.q(9, q_len, hq)
    # before every key; some rows among the first keys; far behind (a share that ends inside
    # a page: the keys behind its end stay out)
    for pos in ([-5, -2, 10 ** 9], [-2 ** 31, 150, 2 ** 31 - 1], [130, -1, 127]):
        o = torch.full(q.shape, float("nan"), device="cuda")
        lse = torch.full(q.shape[:2], float("nan"), device="cuda")
        pq.paged_attention_partial(_dev(q), _dev(p.pages), _dev(p.bt), _i32(p.lens), _i32(pos), q_len,
                                   "int4_group", None, None, o, lse)
        ro, rl = oracle.paged_attention_partial(q, p.pages, p.bt, p.lens, pos, q_len, F, None, None)
        M = max(np.abs(oracle.gather_kv(p.pages, p.bt[s], L, h, F, None, None)[1]).max()
                for s, L in enumerate(p.lens) for h in range(2))
        assert_within(o, ro, np.full(q.shape, M * (2.0 ** -11 + 2.0 ** -13 + 400 * 2.0 ** -25)))
        got = lse.cpu().numpy()
        assert np.array_equal(np.isinf(got), np.isinf(rl)) and not np.isnan(got).any()
        seen = np.isfinite(rl)
        assert (np.abs(got[seen] - rl[seen]) <= 2.0 ** -12).all()


def test_lengths_outside_their_rows_are_clamped_and_reported():
    pq = require_gpu()
    p = Pool(10, [64, 64], 1)
    q = p.q(11, 5, 4)
    st = _i32([0])
    out = _attend(_dev(p.pages), _dev(p.bt), [3, 1000], q, 5, status=st)
    assert pq.status_bits(st) == ["seq_len out of range"]
    ref, bound = allowance(q, p.pages, p.bt, [5, 64], 5)
    assert_within(out, ref, bound)


def test_one_key_with_nan_reaches_only_those_who_see_it():
    """A NaN scale in a token's K: rows before it are not touched."""
    p = Pool(12, [200], 1)
    tile = p.pages.reshape(len(p.pages), 1, 2, 1152)
    page, r = p.bt[0, 198 // 16], 198 % 16
    tile[page, 0, 0, 1024 + 2 * r:1026 + 2 * r] = [0, 0x7E]
    q = p.q(13, 5, 4)                                      # positions 195 .. 199
    out = _attend(_dev(p.pages), _dev(p.bt), [200], q, 5).float().cpu().numpy()
    assert np.isnan(out[3:]).all()
    with np.errstate(invalid="ignore"):
        ref, bound = allowance(q[:3], p.pages, p.bt, [198], 3)
    assert_within(out[:3], ref, bound)


def test_the_same_call_gives_the_same_bits():
    p = Pool(14, [900, 4000, 33], 4)
    q = p.q(15, 5, 16)
    pages, bt = _dev(p.pages), _dev(p.bt)
    first = _attend(pages, bt, p.lens, q, 5)
    for _ in range(5):
        assert torch.equal(first, _attend(pages, bt, p.lens, q, 5))


@pytest.mark.parametrize("skip_block,skip_tile", [(0, 0), (0, 1), (97, 0)])
def test_a_wait_that_runs_out_reports_timeout_and_returns(skip_block, skip_tile):
    pq = require_gpu()
    w = W.Workload("int4_wait", 3, [20000, 9000, 700], 32, 8, 5, F, pool_slack=0.1)
    c = Case(w, with_oracle=False)
    ws = torch.zeros(pq.workspace_size(3, 5, 32, 8, 0), dtype=torch.uint8, device="cuda")
    status = _i32([0])
    out = torch.full_like(c.q, float("nan"))
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    assert _run_test_mode(pq, c, out, ws, status, 0, skip_block, skip_tile) == 0
    torch.cuda.synchronize()
    assert time.perf_counter() - t0 < 5.0
    assert pq.status_bits(status) == ["pipeline wait timed out"]
    # the context is usable, and the same kernel with nothing skipped gives the call's result
    ws.zero_()
    status.zero_()
    assert _run_test_mode(pq, c, out, ws, status, 0, 0, 1 << 30) == 0
    good = c.attention()
    assert int(status.item()) == 0
    assert torch.equal(out, good)
    assert _run_test_mode(pq, c, out, ws, status, 3, 0, 0) == -2       # balanced calls alone


@pytest.mark.parametrize("q_len,window", [(1, 40), (5, 300)])
def test_fixed_splits_in_a_window(q_len, window):
    p = Pool(20, [8, 40, 333, 1000], 2)
    q = p.q(2, q_len, 8)
    ref, bound = allowance(q, p.pages, p.bt, p.lens, q_len, window=window)
    for splits in (1, 4):
        assert_within(_attend(_dev(p.pages), _dev(p.bt), p.lens, q, q_len, window=window,
                              num_splits=splits), ref, bound, "%d splits" % splits)


@pytest.mark.parametrize("q_len", [1, 5])
def test_fixed_splits_of_shares(q_len):
    """Two shares (the first ends on a page's border), each in fixed splits, against its own
    softmax: off by at most what allowance() counts with A <= M = max |V|."""
    pq = require_gpu()
    p = Pool(21, [40, 333, 1600], 2)
    q = p.q(3, q_len, 8)
    M = max(np.abs(oracle.gather_kv(p.pages, p.bt[s], L, h, F, None, None)[1]).max()
            for s, L in enumerate(p.lens) for h in range(2))
    for lo, hi in ((0, 2), (2, 200)):
        n = [min(L, 16 * hi) - min(L, 16 * lo) for L in p.lens]
        bt = np.full((3, max(1, min(hi, p.bt.shape[1]) - lo)), -1, np.int32)
        for s in range(3):
            row = p.bt[s, lo:hi]
            bt[s, :len(row)] = row
        pos = [L - q_len - 16 * lo for L in p.lens]
        ro, rl = oracle.paged_attention_partial(q, p.pages, bt, n, pos, q_len, F, None, None)
        for splits in (1, 3):
            o = torch.full(q.shape, float("nan"), device="cuda")
            lse = torch.full(q.shape[:2], float("nan"), device="cuda")
            pq.paged_attention_partial(_dev(q), _dev(p.pages), _dev(bt), _i32(n), _i32(pos), q_len,
                                       "int4_group", None, None, o, lse, num_splits=splits)
            assert_within(o, ro, np.full(q.shape, M * (2.0 ** -11 + 2.0 ** -13 + 1600 * 2.0 ** -25)),
                          "share %d, %d splits" % (lo, splits))
            assert np.array_equal(np.isinf(lse.cpu().numpy()), np.isinf(rl))


def test_two_streams_at_once():
    """Calls on two streams, a workspace each, do not meet."""
    pq = require_gpu()
    cases = []
    for seed, lens, q_len in ((22, [3000, 70, 900], 5), (23, [5000, 16], 1)):
        p = Pool(seed, lens, 8)
        q = p.q(1, q_len, 32)
        cases.append((q_len, _dev(q), _dev(p.pages), _dev(p.bt), _i32(p.lens), pq.Workspace(),
                      torch.cuda.Stream(), _attend(_dev(p.pages), _dev(p.bt), p.lens, q, q_len)))
    torch.cuda.synchronize()
    outs = [[torch.full_like(c[1], float("nan")) for _ in range(20)] for c in cases]
    torch.cuda.synchronize()
    for k in range(20):
        for (q_len, q, pages, bt, lens, ws, st, _), o in zip(cases, outs):
            pq.paged_attention(q, pages, bt, lens, q_len, "int4_group", None, None, o[k], stream=st,
                               workspace=ws)
    torch.cuda.synchronize()
    for c, o in zip(cases, outs):
        for x in o:
            assert torch.equal(x, c[-1])


def test_two_graphs_that_share_a_workspace():
    """Replayed in turn on one stream, neither finds what the other left: other
    batch sizes, heads and merges."""
    pq = require_gpu()
    ws, made = pq.Workspace(), []
    for seed, lens, q_len, hq, hkv in ((24, [3000, 70, 900], 5, 24, 8), (25, [9000], 1, 16, 2),
                                       (26, [100] * 40, 1, 8, 8)):
        p = Pool(seed, lens, hkv)
        q = p.q(1, q_len, hq)
        args = (_dev(q), _dev(p.pages), _dev(p.bt), _i32(p.lens), q_len, "int4_group", None, None)
        made.append((args, torch.empty_like(args[0]), _attend(args[1], args[2], p.lens, q, q_len)))
        pq.paged_attention(*args, made[-1][1], workspace=ws)
    graphs = []
    for args, out, _ in made:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            pq.paged_attention(*args, out, workspace=ws)
        graphs.append(g)
    for _ in range(3):
        for g, (_, out, want) in zip(graphs, made):
            out.fill_(float("nan"))
            g.replay()
            assert torch.equal(out, want)
