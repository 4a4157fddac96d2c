"""Batches whose sequences share prefixes, built by the oracle's encoder and
uploaded, with the float64 attention and the error a kernel may make."""
from __future__ import annotations

import numpy as np
import torch

import oracle
import workloads as W
from tests.helpers import require_gpu

PAGE, DIM = 16, 128
NAN_FILL = {W.FP16: 0x7E00, W.FP8_E4M3: 0x7F, W.INT8: 0x7F, W.INT8_ROW: 0x7F}


class SharedCase:
    """groups: [(prefix_len, [private tokens of each sequence])].  Only whole
    pages of a prefix are shared; what no sequence holds is NaN."""

    def __init__(self, groups, hq, hkv, q_len, fmt, seed=0, per_head=False, outliers=True,
                 v_amp=1.0):
        rng = np.random.default_rng(seed)
        self.q_len, self.fmt, self.hq, self.hkv = q_len, fmt, hq, hkv
        self.prefix = np.array([g[0] for g in groups], np.int32)
        self.offsets = np.concatenate([[0], np.cumsum([len(g[1]) for g in groups])]).astype(np.int32)
        lens = np.array([g[0] + n for g in groups for n in g[1]], np.int32)
        self.lens = lens
        B = len(lens)
        shared = [g[0] // PAGE for g in groups]
        need = sum(s for s, g in zip(shared, groups) if g[1])
        need += sum(-(-(g[0] + n) // PAGE) - s for s, g in zip(shared, groups) for n in g[1])
        N = need + 3
        perm = rng.permutation(N).astype(np.int32)
        width = int(-(-lens.max() // PAGE)) + 1
        bt = np.full((B, width), -1, np.int32)
        pool = oracle.new_pool(N, hkv, DIM, fmt, fill=NAN_FILL[fmt])
        amax = 90.0
        if fmt == W.FP8_E4M3:
            nk = hkv if per_head else 1
            ks = (np.linspace(0.9, 1.0, nk) * amax / 448).astype(np.float32)
            vs = (np.linspace(1.0, 0.8, nk) * amax / 448).astype(np.float32)
        elif fmt == W.INT8:
            nk = hkv if per_head else 1
            ks = (np.linspace(0.9, 1.0, nk) * amax / 127).astype(np.float32)
            vs = (np.linspace(1.0, 0.8, nk) * amax / 127).astype(np.float32)
        else:
            ks = vs = np.ones(1, np.float32)
        self.ks, self.vs = ks, vs
        if fmt == W.INT8_ROW:
            ks, vs = oracle.new_scale_pool(N, hkv), oracle.new_scale_pool(N, hkv)
            ks[:] = vs[:] = np.nan

        def write(slots):
            nonlocal pool, ks, vs
            x = rng.standard_normal((2, len(slots), hkv, DIM))
            if outliers:
                x *= 1 + 19.0 * (rng.random(x.shape) < 0.01)
            x[1] *= v_amp
            r = oracle.kv_append_quant(x[0].astype(np.float16), x[1].astype(np.float16),
                                       np.asarray(slots), fmt, ks, vs, pool)
            if fmt == W.INT8_ROW:
                pool, ks, vs = r
            else:
                pool = r

        at, s = 0, 0
        slots = []
        for (plen, privs), sh in zip(groups, shared):
            if not privs:
                continue
            mine = perm[at:at + sh]
            at += sh
            slots += [int(p) * PAGE + i for p in mine for i in range(PAGE)]
            for n in privs:
                own = -(-(plen + n) // PAGE) - sh
                bt[s, :sh] = mine
                bt[s, sh:sh + own] = perm[at:at + own]
                at += own
                slots += [int(bt[s, j // PAGE]) * PAGE + j % PAGE for j in range(sh * PAGE, plen + n)]
                s += 1
        write(slots)
        self.bt, self.pool, self.pool_ks, self.pool_vs = bt, pool, ks, vs
        self.q = rng.standard_normal((B * q_len, hq, DIM)).astype(np.float16)

    # -- the GPU's copies
    def upload(self):
        pq = require_gpu()
        N = self.pool.shape[0]
        pages = pq.new_pages(N, self.hkv, self.fmt, "cuda")
        flat = torch.from_numpy(self.pool.view(np.int16) if self.fmt == W.FP16 else self.pool)
        (pages.view(torch.int16) if self.fmt == W.FP16 else pages).copy_(flat)
        if self.fmt == W.INT8_ROW:
            rs = np.stack([self.pool_ks, self.pool_vs], 2).astype(np.float16)   # [N, H, 2, 16]
            pq.row_scales(pages).copy_(torch.from_numpy(rs.reshape(N, self.hkv, 2, 2, 8)))
        dev = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()        # noqa: E731
        self.g = dict(q=dev(self.q), pages=pages, block_table=dev(self.bt), seq_lens=dev(self.lens),
                      group_offsets=dev(self.offsets), prefix_lens=dev(self.prefix),
                      q_len=self.q_len, kv_dtype=self.fmt, k_scale=dev(self.ks),
                      v_scale=dev(self.vs))
        return self.g

    def run(self, **kw):
        pq = require_gpu()
        if not hasattr(self, "g"):
            self.upload()
        args = {**self.g, **kw}
        if "out" not in args:
            args["out"] = torch.full_like(args["q"], float("nan"))
        return pq.paged_attention_shared_prefix(**args)

    # -- the definition in float64, and the error bound of each output
    def expected(self, lens=None, seqs=None, heads=None):
        """(out, tol): float64 attention of every sequence over its own keys,
        and the error the kernel's roundings may leave:
          probabilities rounded to fp16.  With p = 1 for the largest score, what is
          rounded is at least 2^-3 p (the reference of the exponentials is at most 3
          above the largest score seen, in log2), so that half a step is 2^-11 p, or
          2^-25 / 2^-3 = 2^-22 among the subnormals: sum max(2^-11 p, 2^-22) |v| / l,
          where l = sum p >= 1;
          INT8_ROW: the product p * scale is rounded instead of p, with codes of up
          to 127: a subnormal one is off by 127 * 2^-25 / 2^-3 = 127 * 2^-22;
          scores summed in fp32 over 128 products, each sum off by at most
          2^-23 of the products' magnitudes: a relative error d of each
          probability, 2 d A in the quotient, with A = sum p |v| / l;
          sums over the keys and merges in fp32: 2^-18 A;
          the output rounded to fp16: 2^-11 |out|."""
        lens = self.lens if lens is None else lens
        H, G, q_len = self.hkv, self.hq // self.hkv, self.q_len
        out = np.full(self.q.shape, np.nan)
        tol = np.full(self.q.shape, np.nan)
        for s in (range(len(lens)) if seqs is None else seqs):
            L = int(lens[s])
            for h in (range(H) if heads is None else heads):
                if self.fmt == W.INT8_ROW:
                    a, b, unit = self.pool_ks, self.pool_vs, 127.0
                else:
                    a, b = (x[h] if x.size > 1 else x[0] for x in (self.ks, self.vs))
                    unit = 0.0
                K, V = oracle.gather_kv(self.pool, self.bt[s], L, h, self.fmt, a, b)
                x = self.q[s * q_len:(s + 1) * q_len, h * G:(h + 1) * G].astype(np.float64)
                x = x.reshape(q_len * G, DIM)
                z = x @ K.T / np.sqrt(DIM)
                d = 128 * 2.0 ** -23 * (np.abs(x) @ np.abs(K).T).max(1) / np.sqrt(DIM)
                last = L - q_len + np.repeat(np.arange(q_len), G)
                z = np.where(np.arange(L)[None] <= last[:, None], z, -np.inf)
                p = np.exp(z - z.max(1, keepdims=True))
                l = p.sum(1, keepdims=True)
                o, A = p @ V / l, p @ np.abs(V) / l
                t = ((2.0 ** -18 + 2 * d[:, None]) * A + 2.0 ** -11 * np.abs(o)
                     + np.maximum(2.0 ** -11 * p, 2.0 ** -22) @ np.abs(V) / l
                     + 2.0 ** -22 * unit * L / l + 2.0 ** -25)
                rows = slice(s * q_len, (s + 1) * q_len)
                out[rows, h * G:(h + 1) * G] = o.reshape(q_len, G, DIM)
                tol[rows, h * G:(h + 1) * G] = t.reshape(q_len, G, DIM)
        return out, tol

    def check(self, got, what="", **kw):
        want, tol = self.expected(**kw)
        g = got.float().cpu().numpy().astype(np.float64)
        sel = ~np.isnan(want)
        assert np.isfinite(g[sel]).all(), what + ": non-finite output"
        err = np.abs(g - want)[sel]
        worst = (err / tol[sel]).max()
        assert worst <= 1.0, "%s: %.3g of the error allowed" % (what, worst)
        return worst
