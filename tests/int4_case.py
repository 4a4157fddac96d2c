"""Set-up shared by the tests of 4-bit pools: inputs, and how far attention may be off."""
from __future__ import annotations

import numpy as np
import torch

import oracle
import workloads as W

F = W.INT4_GROUP


def rows(rng, n, heads, outliers=True):
    """fp16 [n, heads, 128]: N(0, 1), about 1% twenty times as large."""
    x = rng.normal(size=(n, heads, 128))
    if outliers:
        x = np.where(rng.random(x.shape) < 0.01, 20 * x, x)
    return x.astype(np.float16)


def tables(rng, lens, slack=3):
    """Block table of requests of these lengths on shuffled pages (-1 behind each), and
    the number of pages."""
    need = [-(-L // 16) for L in lens]
    perm = rng.permutation(sum(need) + slack).astype(np.int32)
    bt = np.full((len(lens), max(need + [1])), -1, np.int32)
    at = 0
    for s, n in enumerate(need):
        bt[s, :n] = perm[at:at + n]
        at += n
    return bt, len(perm)


def slots(bt, s, a, b):
    t = np.arange(a, b)
    return bt[s, t // 16].astype(np.int64) * 16 + t % 16


class Pool:
    """Requests of these lengths in a 4-bit pool (uint8 [pages, H, 2, 16, 72], numpy),
    encoded by the oracle; bytes that no token wrote are `fill`."""

    def __init__(self, seed, lens, hkv, fill=0xFF, slack=3):
        rng = np.random.default_rng(seed)
        self.lens, self.hkv = list(lens), hkv
        self.bt, n = tables(rng, lens, slack)
        self.pages = oracle.new_pool(n, hkv, 128, F, fill=fill)
        at = np.concatenate([slots(self.bt, s, 0, L) for s, L in enumerate(lens)])
        self.k, self.v = rows(rng, len(at), hkv), rows(rng, len(at), hkv)
        self.pages = oracle.kv_append_quant(self.k, self.v, at, F, None, None, self.pages)

    def q(self, seed, q_len, hq):
        rng = np.random.default_rng(seed)
        return rng.normal(size=(len(self.lens) * q_len, hq, 128)).astype(np.float16)


def allowance(q, pool, block_table, lens, q_len, window=0, out16=True):
    """(reference, bound) of the attention rows, float64.

    With p_j the softmax of a row and A = sum_j p_j |V_j|, the kernel's sum is off by
      2^-11 A              every probability rounded to fp16 (half a step),
      n 2^-25 max |V|      those under 2^-14 of the row's reference: half a step of 2^-24,
                           and the sum that divides is at least 1,
      2^-13 A              scores in fp32: off by 128 * 2^-24 of sum_d |q_d K_d| / sqrt(128)
                           (at most 40 here: N(0, 1) queries, keys with outliers of 20), so
                           probabilities by less than 2^-13 of themselves; exp2's 2^-22 and
                           the fp32 sums lie far below,
    and the fp16 result by half a step more, 2^-11 of it (2^-25 at least)."""
    hkv = pool.shape[1]
    G = q.shape[1] // hkv
    ref = np.zeros(q.shape, np.float64)
    bound = np.zeros(q.shape, np.float64)
    for s, L in enumerate(lens):
        for h in range(hkv):
            K, V = oracle.gather_kv(pool, block_table[s], L, h, F, None, None)
            x = q[s * q_len:(s + 1) * q_len, h * G:(h + 1) * G].astype(np.float64)
            z = np.einsum("igd,nd->ign", x, K) / np.sqrt(128.0)
            pos, last = np.arange(L), L - q_len + np.arange(q_len)
            sees = pos[None] <= last[:, None]
            if window:
                sees &= pos[None] > last[:, None] - window
            z = np.where(sees[:, None], z, -np.inf)
            p = np.exp(z - z.max(-1, keepdims=True))
            p /= p.sum(-1, keepdims=True)
            o, A = p @ V, p @ np.abs(V)
            at = np.s_[s * q_len:(s + 1) * q_len, h * G:(h + 1) * G]
            ref[at] = o
            bound[at] = A * (2.0 ** -11 + 2.0 ** -13) + L * 2.0 ** -25 * np.abs(V).max(initial=0)
    if out16:
        bound += np.maximum(np.abs(ref) * 2.0 ** -11, 2.0 ** -25)
    return ref, bound


def assert_within(got, ref, bound, what=""):
    g = got.double().cpu().numpy() if isinstance(got, torch.Tensor) else np.asarray(got)
    assert np.isfinite(g).all(), "%s: not finite" % what
    over = np.abs(g - ref) - bound
    i = int(np.argmax(over))
    assert over.max() <= 0, "%s: %.4g where %.4g was due, %.3g allowed (element %d)" % (
        what, g.flat[i], ref.flat[i], bound.flat[i], i)
