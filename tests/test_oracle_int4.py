"""Pins of the oracle's 4-bit format, each apart from the oracle's own code."""
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

import oracle
import workloads as W
from tests.int4_case import F, Pool, rows, slots, tables


def _scale_by_hand(amax):
    """min(fp16(bf16(fp32(amax / 7))), 2720), through torch's casts."""
    q = torch.tensor(np.float32(float(amax)) / np.float32(7.0))
    return min(float(q.bfloat16().half()), 2720.0)


def test_scale_of_every_largest_value():
    x = np.arange(0, 0x7C00, dtype=np.uint16).view(np.float16)       # every finite |x|
    group = np.zeros((len(x), 128), np.float16)
    group[:, 0] = x
    group[:, 33] = -x
    s = oracle.int4_group_scale(group)
    want = np.array([_scale_by_hand(a) for a in x])
    assert np.array_equal(s[:, 0], want) and np.array_equal(s[:, 1], want)
    assert (s[:, 2:] == 0).all()
    # 8 significant bits: every code * scale is an fp16 value
    for c in range(8):
        assert np.array_equal((c * want).astype(np.float16).astype(np.float64), c * want)
    assert np.array_equal((24 * want).astype(np.float16).astype(np.float64), 24 * want)


def test_codes_against_exact_rationals():
    rng = np.random.default_rng(0)
    halves = rng.integers(-14, 15, (40, 128)) / 2
    halves[:, ::32] = 7                                              # a scale of 1: ties
    x = np.concatenate([rows(rng, 40, 1).reshape(40, 128), halves.astype(np.float16)])
    s = oracle.int4_group_scale(x)
    c = oracle.int4_encode(x, s)
    ties = 0
    for i in range(len(x)):
        for d in range(128):
            f = Fraction(float(x[i, d])) / Fraction(float(s[i, d // 32]))
            want = max(-7, min(7, round(f)))                         # Python: half to even
            ties += f.denominator == 2
            assert c[i, d] == want, (i, d)
    assert ties > 100


def test_edges():
    x = np.zeros((5, 128), np.float16)
    x[1, 0], x[1, 1], x[1, 2] = np.inf, -np.inf, 100
    x[2, 5], x[2, 6] = np.nan, -3
    x[3, 40] = 60000
    x[4, 100] = 2.0 ** -24
    s = oracle.int4_group_scale(x)
    c = oracle.int4_encode(x, s)
    assert (s[0] == 0).all() and (c[0] == 0).all()
    assert s[1, 0] == 2720 and list(c[1, :3]) == [7, -7, 0]
    assert c[2, 5] == 0 and c[2, 6] == -7
    assert s[3, 1] == 2720 and c[3, 40] == 7
    assert s[4, 3] == 0 and (c[4] == 0).all()                        # amax / 7 rounds to 0


def test_tile_against_the_header_bit_by_bit():
    rng = np.random.default_rng(1)
    codes = rng.integers(-7, 8, (2, 16, 128)).astype(np.int8)
    scale = rng.integers(1, 100, (2, 16, 4)) / 16.0
    tile = oracle.int4_tile(codes, scale)
    assert tile.shape == (2, 1152) and tile.dtype == np.uint8
    for n in range(2):
        for r in range(16):
            for d in range(128):
                g, w, f, e = d // 32, d % 32 // 8, d % 8 // 2, d % 2
                i = r // 2
                chunk = (4 * (r % 2) + g) ^ (0, 5, 2, 7)[i % 4]
                at = 128 * i + 16 * chunk + 4 * w + 2 * e
                half = int(tile[n, at]) + 256 * int(tile[n, at + 1])
                place = ((6, 7, 8, 9), (2, 3, 4, 5), (10, 11, 12, 13), (14, 15, 0, 1))[f]
                got = sum(((half >> b) & 1) << k for k, b in enumerate(place))
                assert got == codes[n, r, d] + 8
            for g in range(4):
                raw = tile[n, 1024 + 2 * (16 * g + r):][:2].copy().view(np.float16)[0]
                assert raw == scale[n, r, g]
    c, s = oracle.int4_untile(tile)
    assert np.array_equal(c, codes) and np.array_equal(s, scale)


def test_append_and_read_back():
    rng = np.random.default_rng(2)
    lens = [37, 1, 16, 50]
    p = Pool(3, lens, 2)
    at = 0
    for s, L in enumerate(lens):
        for h in range(2):
            K, V = oracle.gather_kv(p.pages, p.bt[s], L, h, F, None, None)
            for x, got in ((p.k, K), (p.v, V)):
                x = x[at:at + L, h]
                sc = oracle.int4_group_scale(x)
                err = np.abs(got - x.astype(np.float64)).reshape(L, 4, 32)
                # half a step, and the scale's own rounding (2^-9) times up to 7 steps
                assert (err <= sc[..., None] * (0.5 + 7 * 2.0 ** -8)).all()
        at += L
    # bytes that no token wrote are as they were
    before = oracle.new_pool(4, 1, 128, F, fill=0xA5)
    k = rows(rng, 1, 1)
    after = oracle.kv_append_quant(k, k, [21], F, None, None, before)
    assert (after[[0, 2, 3]] == 0xA5).all()
    assert (after != before).any(-1).sum() <= 2 * (16 + 4)
    assert oracle.kv_append_quant(k, k, [-1], F, None, None, before).tobytes() == before.tobytes()


def test_attention_against_a_loop():
    p = Pool(5, [19, 33], 2)
    q = p.q(6, 3, 4)
    got = oracle.paged_attention(q, p.pages, p.bt, p.lens, 3, F, None, None, window=7)
    for s, L in enumerate(p.lens):
        for i in range(3):
            for hq in range(4):
                K, V = oracle.gather_kv(p.pages, p.bt[s], L, hq // 2, F, None, None)
                last = L - 3 + i
                keys = range(max(0, last - 6), last + 1)
                w = [math.exp(float(np.dot(q[s * 3 + i, hq].astype(np.float64), K[j])) / 128 ** 0.5)
                     for j in keys]
                want = sum(wi * V[j] for wi, j in zip(w, keys)) / sum(w)
                assert np.allclose(got[s * 3 + i, hq], want, rtol=1e-12, atol=1e-12)


@pytest.mark.parametrize("fmt", [W.FP16, W.FP8_E4M3, W.INT8, F])
def test_kv_read_is_the_gather(fmt):
    rng = np.random.default_rng(7)
    lens, first, n = [20, 40, 5], [3, 17, 0], [17, 9, 0]
    bt, pages_n = tables(rng, lens)
    pool = oracle.new_pool(pages_n, 2, 128, fmt)
    sc = np.full(2, 0.5, np.float32)
    at = np.concatenate([slots(bt, s, 0, L) for s, L in enumerate(lens)])
    k, v = rows(rng, len(at), 2, False), rows(rng, len(at), 2, False)
    pool = oracle.kv_append_quant(k, v, at, fmt, sc, sc, pool)
    off = np.concatenate([[0], np.cumsum(n)])
    K, V = oracle.kv_read(pool, bt, first, off, fmt, sc, sc)
    assert K.shape == (26, 2, 128)
    for s in range(3):
        a = sum(lens[:s]) + first[s]
        for x, got in ((k, K), (v, V)):
            err = np.abs(got[off[s]:off[s + 1]] - x[a:a + n[s]].astype(np.float64))
            assert err.max(initial=0) <= {0: 0.0, 1: 0.25, 2: 0.25, F: 0.6}[fmt]
