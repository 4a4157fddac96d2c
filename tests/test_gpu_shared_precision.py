"""Small probabilities of a shared prefix are rounded like paged_attention's: to fp16
with the largest score's probability at 1 or above, so a step of at most 2^-24 of it."""
import numpy as np
import pytest
import torch

import oracle
import workloads as W
from tests.helpers import require_gpu
from tests.shared_case import SharedCase

pytestmark = pytest.mark.gpu

FORMATS = [W.FP16, W.FP8_E4M3, W.INT8, W.INT8_ROW]


@pytest.mark.parametrize("fmt", FORMATS)
def test_a_flat_tail_under_one_large_score(fmt):
    """Key 0 has the largest score and V = 0; every other key has score 0 and the same V.
    Enough rows that a CTA holds a row tile's whole prefix.  The gap is chosen so that a
    tail probability (INT8_ROW: its product with V's row scale) is 2^-22.2 of the
    largest: 2^-25 is the most that rounding one may lose, so the outputs keep their
    first digit.  With the largest at 2^-3 each would be under 2^-25, and lost.

    An output is S w / (1 + S w), S = sum of V over the tail, w = 2^-gap.  Allowed: half a
    step, 2^-25 of the largest, per key, times its V (INT8_ROW: code); 2^-11 of the output
    for its rounding and as much again for what fp32 leaves (scores of 22 in log2, off by
    128 * 2^-23 of them at most: 2^-12 of w)."""
    pq = require_gpu()
    B, q_len, hq, hkv, prefix = 160, 8, 32, 8, 2048
    own = q_len + 3
    shared, per = prefix // 16, 1
    N = shared + B * per
    v_row = 2.0 ** -13 if fmt == W.INT8_ROW else 1.0
    gap = 22.2 + np.log2(v_row)
    kappa = gap / (np.log2(np.e) * 128 / 128 ** 0.5)       # of every value of K's row 0
    one = lambda x: torch.full((1,), float(x), device="cuda")     # noqa: E731
    ks = vs = None
    pages = pq.new_pages(N, hkv, fmt, "cuda", fill=0)
    if fmt == W.FP16:
        kappa, kc, vc, unit = float(np.float16(kappa)), float(np.float16(kappa)), 1.0, 1.0
    elif fmt == W.FP8_E4M3:
        kappa, kc, vc, unit = float(np.float32(kappa)), 0x38, 0x38, 1.0       # codes of 1.0
        ks, vs = one(kappa), one(1.0)
    elif fmt == W.INT8:
        kappa, kc, vc, unit = 127 * float(np.float32(kappa / 127)), 127, 127, 1.0
        ks, vs = one(np.float32(kappa / 127)), one(1 / 127)
    else:
        kappa, kc, vc, unit = 127 * float(np.float16(kappa / 127)), 127, 127, 127.0
        rs = pq.row_scales(pages)
        rs[:, :, 0] = float(np.float16(kappa / 127))
        rs[:, :, 1] = v_row
    pages[:, :, 1] = vc
    pages[0, :, 0, 0] = kc                                  # page 0 is the prefix's first
    pages[0, :, 1, 0] = 0
    bt = torch.empty((B, shared + per), dtype=torch.int32, device="cuda")
    bt[:, :shared] = torch.arange(shared, device="cuda")
    bt[:, shared] = shared + torch.arange(B, device="cuda")
    lens = torch.full((B,), prefix + own, dtype=torch.int32, device="cuda")
    q = torch.ones((B * q_len, hq, 128), dtype=torch.float16, device="cuda")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")   # noqa: E731
    out = pq.paged_attention_shared_prefix(q, pages, bt, lens, i32([0, B]), i32([prefix]), q_len,
                                           fmt, ks, vs, torch.full_like(q, float("nan")))
    w = 2.0 ** -(kappa * np.log2(np.e) * 128 / 128 ** 0.5)
    v = 127 * v_row if fmt == W.INT8_ROW else 127 * float(np.float32(1 / 127)) if fmt == W.INT8 else 1.0
    n = prefix + own - q_len + torch.arange(q_len, device="cuda", dtype=torch.float64)   # tail keys
    want = (n * v * w / (1 + n * w)).repeat(B)[:, None, None]
    allowed = (n * unit * 2.0 ** -25 / (1 + n * w)).repeat(B)[:, None, None] + want * 2.0 ** -10
    worst = ((out.double() - want).abs() / allowed).max().item()
    assert worst <= 1.0, "%.3g of the error allowed" % worst


@pytest.mark.parametrize("v_amp", [1.0, 0.01, 0.001])
@pytest.mark.parametrize("fmt", [W.FP16, W.INT8_ROW])
def test_errors_of_small_values(fmt, v_amp):
    """Values of any size (INT8_ROW: any row scale) over several thousand keys.  What is
    rounded to fp16 -- the probability, INT8_ROW's times V's scale -- is off by half a
    step at most, evenly spread and independent from key to key: a variance of step^2 / 12,
    with a step of 2^-10 of the value, 2^-24 at least, in units of the largest score's
    probability.  Their sum, and the output's own rounding, give the rms error of an
    output; twice that is allowed."""
    require_gpu()
    c = SharedCase([(9000, [5, 9, 20, 1])], 16, 2, 1, fmt, seed=51, outliers=False, v_amp=v_amp)
    got = c.run().double().cpu().numpy()
    err2 = expected2 = 0.0
    for s, L in enumerate(c.lens):
        for h in range(2):
            row = fmt == W.INT8_ROW
            K, V = oracle.gather_kv(c.pool, c.bt[s], int(L), h, fmt, c.pool_ks if row else 1.0,
                                    c.pool_vs if row else 1.0)
            j = np.arange(L)
            scale = c.pool_vs[c.bt[s][j // 16], h, j % 16].astype(np.float64) if row else 1.0
            x = c.q[s, h * 8:(h + 1) * 8].astype(np.float64)
            z = x @ K.T / np.sqrt(128)
            p = np.exp(z - z.max(1, keepdims=True))
            l = p.sum(1, keepdims=True)
            o = p @ V / l
            step = np.maximum(2.0 ** -10 * p * scale, 2.0 ** -24) / scale
            ulp = np.maximum(2.0 ** -10 * np.abs(o), 2.0 ** -24)
            err2 += ((got[s, h * 8:(h + 1) * 8] - o) ** 2).sum()
            expected2 += (step ** 2 @ V ** 2 / l ** 2 + ulp ** 2).sum() / 12
    ratio = (err2 / expected2) ** 0.5
    assert ratio <= 2.0, "%.3g times the expected rms error" % ratio


def test_a_maximum_that_climbs_among_large_scores():
    """Scores of 2^21 (log2 units; 127 of the 128 products are large), where fp32 holds
    quarters: the second half of the prefix lies 15.94 above the first, so that whether a
    row's probabilities still fit fp16 hangs on how its exponents are rounded.  Every
    output is the second half's V, 1, up to a weight of 2^-15 and fp16's rounding."""
    pq = require_gpu()
    B, q_len, hq, hkv, prefix, own = 160, 8, 32, 8, 2048, 11
    shared = prefix // 16
    # raw scores: 124 * 362 * 367 + 2 r + 100 + (0 or 125), all whole and under 2^24
    pages = pq.new_pages(shared + B, hkv, W.FP16, "cuda", fill=0)
    k = pages[:, :, 0]
    k[..., :124] = 367.0
    k[..., 124] = 2.0                                       # varies with the query row
    k[..., 125] = 1.0
    k[:shared // 2, ..., 126] = 0.0
    k[shared // 2:, ..., 126] = 125.0
    pages[shared // 2:, :, 1] = 1.0
    q = torch.zeros((B * q_len, hq, 128), dtype=torch.float16, device="cuda")
    q[..., :124] = 362.0
    q[..., 124] = torch.arange(B * q_len * hq, device="cuda").view(B * q_len, hq) % 997
    q[..., 125] = 100.0
    q[..., 126] = 1.0
    raw = 124 * 362 * 367 + 2 * 996 + 100 + 125
    assert raw < 2 ** 24 and raw * np.log2(np.e) / 128 ** 0.5 > 2 ** 21
    bt = torch.empty((B, shared + 1), dtype=torch.int32, device="cuda")
    bt[:, :shared] = torch.arange(shared, device="cuda")
    bt[:, shared] = shared + torch.arange(B, device="cuda")
    lens = torch.full((B,), prefix + own, dtype=torch.int32, device="cuda")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")   # noqa: E731
    out = pq.paged_attention_shared_prefix(q, pages, bt, lens, i32([0, B]), i32([prefix]), q_len,
                                           W.FP16, None, None, torch.full_like(q, float("nan")))
    worst = (out.float() - 1).abs().max().item()
    assert worst <= 2.0 ** -15 + 2.0 ** -11, worst
