"""4-bit pools on the GPU against the oracle: what is written bit for bit, attention
within a bound that is derived in tests/int4_case.py."""
import numpy as np
import pytest
import torch

import oracle
import workloads as W
from tests.helpers import require_gpu
from tests.int4_case import F, Pool, allowance, assert_within, rows, slots, tables

pytestmark = pytest.mark.gpu


def _dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def _status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def _append(k, v, at, num_pages, H, fill=0x5A, stride=None):
    pq = require_gpu()
    kd, vd = _dev(k), _dev(v)
    if stride:                                    # column slices of a wider buffer
        big = torch.full((len(k), stride), float("nan"), dtype=torch.float16, device="cuda")
        kd = big[:, 128:128 + H * 128].copy_(kd.reshape(len(k), -1)).view(len(k), H, 128)
    pages = pq.new_pages(num_pages, H, "int4_group", fill=fill)
    assert pages.shape == (num_pages, H, 2, 16, 72) and pages.dtype == torch.uint8
    st = _status()
    pq.kv_append_quant(kd, vd, _dev(np.asarray(at, np.int64)), "int4_group", None, None, pages,
                       status=st)
    assert int(st.item()) == 0
    ref = oracle.kv_append_quant(k, v, at, F, None, None,
                                 oracle.new_pool(num_pages, H, 128, F, fill=fill))
    assert np.array_equal(pages.cpu().numpy(), ref)


def test_append_every_fp16_value():
    """All values, mixed so that each meets largest values of many sizes."""
    rng = np.random.default_rng(0)
    x = np.arange(65536, dtype=np.uint32).astype(np.uint16).view(np.float16)
    x = np.concatenate([x, rng.permutation(x), np.sort(x)]).reshape(-1, 1, 128)
    at = rng.permutation(len(x) + 40)[:len(x)]
    _append(x, x[::-1].copy(), at, (len(x) + 40) // 16 + 1, 1)


def test_append_ties_and_every_scale():
    """For scales of every mantissa: (c + 1/2) s for all codes c, and the fp16 neighbours."""
    mant = (1 + np.arange(128) / 128)[:, None]
    c = np.concatenate([np.arange(-7, 7) + 0.5, [7.0]])
    k = []
    for e in (-24, -20, -17, -14, -3, 0, 5, 11):
        s = mant * 2.0 ** e
        x = (c * s).astype(np.float16)
        for step in (-1, 0, 1):
            bits = x.view(np.int16) + step * (x != 0)
            g = np.zeros((128, 32), np.float16)
            g[:, :15] = np.where(c == 7, x, bits.astype(np.int16).view(np.float16))
            g[:, 15:30] = -g[:, :15]
            k.append(g)
    k = np.concatenate(k).reshape(-1, 1, 128)
    _append(k, np.roll(k, 5, axis=2), np.arange(len(k))[::-1].copy(), len(k) // 16 + 1, 1)


@pytest.mark.parametrize("T,H", [(1, 1), (7, 3), (33, 8), (2500, 2)])
def test_append_odd_sizes_strided_and_skipped(T, H):
    rng = np.random.default_rng(T)
    k, v = rows(rng, T, H), rows(rng, T, H)
    if T > 4:
        k[0, 0, :40], v[1], k[2, 0, 9], v[3, -1, 64] = np.nan, 0, np.inf, -np.inf
    at = rng.permutation(T + 9)[:T].astype(np.int64)
    at[::5] = -1
    _append(k, v, at, (T + 9) // 16 + 1, H, stride=(H + 2) * 128)


def test_append_beyond_the_pool_and_past_4_gib():
    pq = require_gpu()
    rng = np.random.default_rng(1)
    n = (1 << 32) // 2304 + 40                              # one kv-head: pages past 4 GiB
    pages = torch.zeros((n, 1, 2, 16, 72), dtype=torch.uint8, device="cuda")
    k, v = rows(rng, 5, 1), rows(rng, 5, 1)
    at = np.array([16 * (n - 1) + 3, 16 * n, -5, 16 * (n - 1) + 4, 16 * n + 1000])
    st = _status()
    pq.kv_append_quant(_dev(k), _dev(v), _dev(at), "int4_group", None, None, pages, status=st)
    assert pq.status_bits(st) == ["slot beyond the pool"]
    ref = oracle.kv_append_quant(k[[0, 3]], v[[0, 3]], [3, 4], F, None, None,
                                 oracle.new_pool(1, 1, 128, F))
    assert np.array_equal(pages[-1:].cpu().numpy(), ref)
    assert int(pages[:-1].max()) == 0
    # and read there: attention and kv_read
    bt = torch.tensor([[n - 1]], dtype=torch.int32, device="cuda")
    ref = oracle.kv_append_quant(rows(rng, 16, 1), rows(rng, 16, 1), np.arange(16), F, None, None, ref)
    pages[-1:] = _dev(ref)
    q = rng.normal(size=(1, 4, 128)).astype(np.float16)
    out = torch.empty((1, 4, 128), dtype=torch.float16, device="cuda")
    lens = torch.tensor([16], dtype=torch.int32, device="cuda")
    pq.paged_attention(_dev(q), pages, bt, lens, 1, "int4_group", None, None, out)
    want, bound = allowance(q, ref, np.zeros((1, 1), int), [16], 1)
    assert_within(out, want, bound)
    ko, vo = (torch.empty((16, 1, 128), dtype=torch.float16, device="cuda") for _ in "kv")
    pq.kv_read(pages, bt, None, torch.tensor([0, 16], dtype=torch.int32, device="cuda"), "int4_group",
               None, None, ko, vo)
    K, V = oracle.kv_read(ref, np.zeros((1, 1), int), None, [0, 16], F, None, None)
    assert np.array_equal(ko.cpu().numpy(), K) and np.array_equal(vo.cpu().numpy(), V)


def _attend(p, q, q_len, **kw):
    pq = require_gpu()
    out = torch.full(q.shape, float("nan"), dtype=torch.float16, device="cuda")
    st = _status()
    pq.paged_attention(_dev(q), _dev(p.pages), _dev(p.bt),
                       torch.tensor(p.lens, dtype=torch.int32, device="cuda"), q_len,
                       "int4_group", None, None, out, status=st, **kw)
    assert int(st.item()) == 0, pq.status_bits(st)
    return out


LENS = [8, 9, 15, 16, 17, 31, 130, 700, 2049]


@pytest.mark.parametrize("hq,hkv,q_len", [(8, 1, 1), (32, 8, 1), (5, 5, 1), (6, 2, 3), (24, 8, 5),
                                          (32, 8, 5), (32, 8, 8), (64, 8, 4), (32, 1, 1)])
def test_attention_of_ragged_lengths(hq, hkv, q_len):
    p = Pool(hq + q_len, [max(L, q_len) for L in LENS] + [q_len], hkv)
    q = p.q(1, q_len, hq)
    ref, bound = allowance(q, p.pages, p.bt, p.lens, q_len)
    for kw in ({}, {"num_splits": 1}, {"num_splits": 3}, {"max_seq_len": 2100}):
        assert_within(_attend(p, q, q_len, **kw), ref, bound, "%s" % kw)


@pytest.mark.parametrize("q_len", [1, 5, 8])
@pytest.mark.parametrize("window", [1, 16, 100, 5000])
def test_attention_in_a_window(q_len, window):
    p = Pool(3, [8, 40, 333, 1000], 2)
    q = p.q(2, q_len, 8)
    ref, bound = allowance(q, p.pages, p.bt, p.lens, q_len, window=window)
    assert_within(_attend(p, q, q_len, window=window), ref, bound)


@pytest.mark.parametrize("q_len", [1, 5])
def test_partial_shares_merge(q_len):
    """Shares of the keys (one of them empty), each against the oracle, then merged.

    A share's softmax is its own: its A is at most max |V| = M.  Its lse is off by less than
    2^-13 (its probabilities', which l sums in fp32) and as much for the logarithm; weights
    that are off by 2^-12 of themselves, and their sum, move the merged row by 2^-11 M."""
    pq = require_gpu()
    p = Pool(4, [40, 333, 1600], 2)
    q = p.q(3, q_len, 8)
    whole, bound = allowance(q, p.pages, p.bt, p.lens, q_len)
    M = max(np.abs(oracle.gather_kv(p.pages, p.bt[s], L, h, F, None, None)[1]).max()
            for s, L in enumerate(p.lens) for h in range(2))
    os_, lses = [], []
    for lo, hi in ((0, 2), (2, 2), (2, 30), (30, 200)):          # pages
        n = [min(L, 16 * hi) - min(L, 16 * lo) for L in p.lens]
        bt = np.full((3, max(1, hi - lo)), -1, np.int32)
        for s in range(3):
            row = p.bt[s, lo:hi]
            bt[s, :len(row)] = row
        pos = [L - q_len - 16 * lo for L in p.lens]
        o = torch.full(q.shape, float("nan"), device="cuda")
        lse = torch.full(q.shape[:2], float("nan"), device="cuda")
        pq.paged_attention_partial(_dev(q), _dev(p.pages), _dev(bt),
                                   torch.tensor(n, dtype=torch.int32, device="cuda"),
                                   torch.tensor(pos, dtype=torch.int32, device="cuda"), q_len,
                                   "int4_group", None, None, o, lse)
        ro, rl = oracle.paged_attention_partial(q, p.pages, bt, n, pos, q_len, F, None, None)
        assert_within(o, ro, np.full(q.shape, M * (2.0 ** -11 + 2.0 ** -13 + 1600 * 2.0 ** -25)),
                      "share %d" % lo)
        got = lse.cpu().numpy()
        assert np.array_equal(np.isinf(got), np.isinf(rl))
        seen = np.isfinite(rl)
        assert (np.abs(got - rl)[seen] <= 2.0 ** -12).all()
        os_.append(o)
        lses.append(lse)
    out = torch.empty(q.shape, dtype=torch.float16, device="cuda")
    pq.lse_merge(torch.stack(os_), torch.stack(lses), out)
    assert_within(out, whole, bound + 2.0 ** -11 * M)


def test_stale_bytes_behind_the_end_do_not_matter():
    """Bytes that no token wrote are 0xFF: NaN scales."""
    p = Pool(5, [5, 17, 47], 2, fill=0xFF)
    assert np.isnan(p.pages.reshape(-1, 2, 2, 1152)[..., 1024:].copy().view(np.float16)).any()
    for q_len in (1, 5):
        q = p.q(4, q_len, 8)
        ref, bound = allowance(q, p.pages, p.bt, p.lens, q_len)
        assert_within(_attend(p, q, q_len), ref, bound)


@pytest.mark.parametrize("bad", [-1, -7, 10 ** 6, "n"])
def test_a_page_id_outside_the_pool_reads_zeros(bad):
    pq = require_gpu()
    p = Pool(6, [300, 40], 2, slack=0)
    n = len(p.pages)
    bt = p.bt.copy()
    bt[0, [1, 18]] = n if bad == "n" else bad
    zero = p.bt.copy()
    zero[0, [1, 18]] = n
    pool = np.concatenate([p.pages, np.zeros_like(p.pages[:1])])
    for q_len in (1, 5):
        q = p.q(5, q_len, 8)
        ref, bound = allowance(q, pool, zero, p.lens, q_len)
        out = torch.empty(q.shape, dtype=torch.float16, device="cuda")
        st = _status()
        pq.paged_attention(_dev(q), _dev(p.pages), _dev(bt),
                           torch.tensor(p.lens, dtype=torch.int32, device="cuda"), q_len,
                           "int4_group", None, None, out, status=st)
        assert pq.status_bits(st) == ["block-table page id out of range"]
        assert_within(out, ref, bound)


def test_large_values_saturate_and_small_ones_stay():
    """Scales at both ends: V at +-19040 and at the smallest fp16 values."""
    rng = np.random.default_rng(8)
    p = Pool(9, [64], 1)
    for mult in (19040.0 / 7, 2.0 ** -22):
        v = (rng.integers(-7, 8, (64, 1, 128)) * mult).astype(np.float16)
        v[:, :, ::32] = np.float16(7 * mult)
        k = np.full((64, 1, 128), np.float16(0.125))
        pool = oracle.kv_append_quant(k, v, slots(p.bt, 0, 0, 64), F, None, None, p.pages)
        p2 = p
        p2.pages = pool
        q = p.q(6, 1, 4)
        ref, bound = allowance(q, pool, p.bt, p.lens, 1)
        out = _attend(p2, q, 1)
        assert_within(out, ref, bound, "values of %g" % mult)


def test_noalloc_other_streams_and_a_graph():
    pq = require_gpu()
    p = Pool(10, [100, 900], 8)
    for q_len in (1, 5):
        q = p.q(7, q_len, 32)
        ref, bound = allowance(q, p.pages, p.bt, p.lens, q_len)
        qd, pages, bt = _dev(q), _dev(p.pages), _dev(p.bt)
        lens = torch.tensor(p.lens, dtype=torch.int32, device="cuda")
        out = torch.empty_like(qd)
        pq.paged_attention_noalloc(qd, pages, bt, lens, q_len, "int4_group", None, None, out)
        assert_within(out, ref, bound, "noalloc")
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        ws = pq.Workspace()
        out2 = torch.empty_like(qd)
        pq.paged_attention(qd, pages, bt, lens, q_len, "int4_group", None, None, out2, stream=st,
                           workspace=ws)
        st.synchronize()
        assert torch.equal(out, out2)
        g = torch.cuda.CUDAGraph()
        out3 = torch.empty_like(qd)
        with torch.cuda.graph(g):
            pq.paged_attention(qd, pages, bt, lens, q_len, "int4_group", None, None, out3,
                               workspace=ws)
        for _ in range(3):
            out3.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, out3)


def test_a_run_of_a_serving_step():
    """Block tables grown, the new tokens written, verified, the rejected ones given back,
    and the context read out again."""
    pq = require_gpu()
    rng = np.random.default_rng(11)
    B, H, hq, n_pages, q_len = 3, 2, 8, 40, 5
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")     # noqa: E731
    bt = torch.full((B, 12), -1, dtype=torch.int32, device="cuda")
    free = _dev(rng.permutation(n_pages).astype(np.int32))
    count, lens = i32([n_pages]), i32([0] * B)
    pages = pq.new_pages(n_pages, H, "int4_group", fill=0xFF)
    pool = oracle.new_pool(n_pages, H, 128, F, fill=0xFF)
    host = np.zeros(B, int)
    ks, vs = [[] for _ in range(B)], [[] for _ in range(B)]
    for step, new in enumerate([[30, 5, 17], [5] * 3, [5] * 3]):
        T = sum(new)
        at = torch.empty(T, dtype=torch.int64, device="cuda")
        off = torch.empty(B + 1, dtype=torch.int32, device="cuda")
        pq.extend_block_tables(lens, i32(new), bt, free, count, n_pages, lens, count, at,
                               token_offsets=off)
        k, v = rows(rng, T, H), rows(rng, T, H)
        pq.kv_append_quant(_dev(k), _dev(v), at, "int4_group", None, None, pages)
        pool = oracle.kv_append_quant(k, v, at.cpu().numpy(), F, None, None, pool)
        # the step's own tokens read back at their positions
        ko, vo = (torch.empty((T, H, 128), dtype=torch.float16, device="cuda") for _ in "kv")
        pq.kv_read(pages, bt, _dev(host.astype(np.int32)), off, "int4_group", None, None, ko, vo)
        s = oracle.int4_group_scale(k)
        assert np.array_equal(ko.cpu().numpy(), oracle.int4_decode(oracle.int4_encode(k, s), s))
        host = host + new
        if step:
            q = rng.normal(size=(B * q_len, hq, 128)).astype(np.float16)
            out = torch.empty(q.shape, dtype=torch.float16, device="cuda")
            pq.paged_attention(_dev(q), pages, bt, lens, q_len, "int4_group", None, None, out)
            ref, bound = allowance(q, pool, bt.cpu().numpy(), host, q_len)
            assert_within(out, ref, bound, "step %d" % step)
            keep = host - rng.integers(0, 4, B)
            pq.truncate_block_tables(lens, _dev(keep.astype(np.int32)), bt, free, count, lens, count)
            host = keep
    assert np.array_equal(pages.cpu().numpy(), pool)
    off = np.concatenate([[0], np.cumsum(host)])
    ko, vo = (torch.empty((int(off[-1]), H, 128), dtype=torch.float16, device="cuda") for _ in "kv")
    pq.kv_read(pages, bt, None, _dev(off.astype(np.int32)), "int4_group", None, None, ko, vo)
    K, V = oracle.kv_read(pool, bt.cpu().numpy(), None, off, F, None, None)
    assert np.array_equal(ko.cpu().numpy(), K) and np.array_equal(vo.cpu().numpy(), V)


def test_refusals():
    pq = require_gpu()
    pages = pq.new_pages(4, 2, "int4_group", fill=0)
    q = torch.zeros((1, 8, 128), dtype=torch.float16, device="cuda")
    bt = torch.zeros((1, 4), dtype=torch.int32, device="cuda")
    lens = torch.ones(1, dtype=torch.int32, device="cuda")
    eight = pq.new_pages(4, 2, "int8", fill=0)
    with pytest.raises(ValueError, match="16, 72"):
        pq.paged_attention(q, eight, bt, lens, 1, "int4_group", None, None, torch.empty_like(q))
    with pytest.raises(ValueError, match="16, 128"):
        pq.paged_attention(q, pages, bt, lens, 1, "int8_row", None, None, torch.empty_like(q))
    with pytest.raises(ValueError, match="pages must be"):
        pq.kv_append_quant(q[:, :2], q[:, :2], lens.long(), "int4_group", None, None, eight)
    with pytest.raises(KeyError):
        pq.new_pages(4, 2, "int4")
