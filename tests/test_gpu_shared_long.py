"""Shared prefixes at the sizes they are for -- many row tiles, many key tiles, several
CTAs a row tile -- against the float64 definition of every output, with a bound tight
enough to see one key tile missing, counted twice or read from the wrong place."""
import numpy as np
import pytest
import torch

import workloads as W
from tests.helpers import require_gpu

pytestmark = pytest.mark.gpu

HQ, HKV, G = 32, 8, 4
FORMATS = [W.FP16, W.FP8_E4M3, W.INT8, W.INT8_ROW]
BATCHES = [([(64, 20000)], 5), ([(250, 12000)], 1), ([(24, 40000)], 8),
           ([(70, 30000), (9, 8000), (1, 5000), (40, 17001)], 1)]


def _values(pages, fmt, scale, row):
    """float64 [..., 128] of the pages' codes (row: their rows' scales)."""
    if fmt == W.FP16:
        return pages.double()
    if fmt == W.FP8_E4M3:
        return pages.view(torch.float8_e4m3fn).double() * scale
    x = pages.view(torch.int8).double()
    return x * (scale if row is None else row.double()[..., None])


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("groups,q_len", BATCHES)
def test_every_output_of_a_long_shared_prefix(fmt, groups, q_len):
    """Allowed, with p = exp(score - largest), l = sum p, A = sum p |V| / l:
      2^-11 A + 2^-25 sum |V| / l   each probability rounded to fp16, half a step of it or
                of 2^-24 (INT8_ROW: p times the row scale is rounded, so |code| for |V|);
      2 d A     scores summed in fp32 over 128 products, d = 128 * 2^-23 of the
                products' magnitudes at most;
      2^-18 A   sums over keys, exponentials and merges in fp32;
      2^-11 |out| + 2^-25   the output's rounding."""
    pq = require_gpu()
    gen = torch.Generator(device="cuda").manual_seed(len(groups) * 100 + q_len)
    offsets = np.concatenate([[0], np.cumsum([n for n, _ in groups])])
    B, room = int(offsets[-1]), 3                        # private pages of a sequence
    shared = [p // 16 for _, p in groups]
    width = max(shared) + room
    N = sum(shared) + B * room
    pages = pq.new_pages(N, HKV, fmt, "cuda")
    x = torch.randn(pages.shape, generator=gen, device="cuda")
    x *= 1 + 4 * (torch.rand(pages.shape, generator=gen, device="cuda") < 0.01)
    ks = vs = rows = None
    k, v = 1.0, 1.0
    if fmt == W.FP16:
        pages.copy_(x)
    elif fmt == W.FP8_E4M3:
        k, v = 1 / 16, 1 / 32
        pages.copy_((x * 16).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8))
    else:
        k, v = 0.25, 0.125
        pages.copy_((x * 5).round().clamp(-127, 127).to(torch.int8).view(torch.uint8))
        if fmt == W.INT8_ROW:
            rows = pq.row_scales(pages)
            rows.copy_(0.2 * (1 + torch.rand(rows.shape, generator=gen, device="cuda")))
            rows = rows.reshape(N, HKV, 2, 16)
    del x
    if fmt in (W.FP8_E4M3, W.INT8):
        ks, vs = (torch.full((1,), s, device="cuda") for s in (k, v))
    perm = torch.randperm(N, generator=gen, device="cuda").int()
    bt = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    lens = torch.empty(B, dtype=torch.int32, device="cuda")
    at = 0
    for g, (n, prefix) in enumerate(groups):
        mine = slice(int(offsets[g]), int(offsets[g + 1]))
        bt[mine, :shared[g]] = perm[at:at + shared[g]]
        at += shared[g]
        bt[mine, shared[g]:shared[g] + room] = perm[at:at + n * room].view(n, room)
        at += n * room
        lens[mine] = prefix + torch.randint(q_len, 30, (n,), generator=gen, device="cuda").int()
    q = torch.randn((B * q_len, HQ, 128), generator=gen, device="cuda").half()
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")   # noqa: E731
    got = pq.paged_attention_shared_prefix(
        q, pages, bt, lens, i32(offsets.tolist()), i32([p for _, p in groups]), q_len, fmt, ks, vs,
        torch.full_like(q, float("nan"))).view(B, q_len, HKV, G, 128)

    for g, (n, prefix) in enumerate(groups):
        mine = slice(int(offsets[g]), int(offsets[g + 1]))
        pre = bt[int(offsets[g]), :shared[g]].long()
        own = bt[mine, shared[g]:shared[g] + room].long()             # [n, room]
        pos = shared[g] * 16 + torch.arange(room * 16, device="cuda")
        last = lens[mine].long()[:, None] - q_len + torch.arange(q_len, device="cuda")
        hidden = (pos > last[..., None]).repeat_interleave(G, 1)       # [n, q_len * G, keys]
        for h in range(HKV):
            def part(ids, kv, scale):
                r = None if rows is None else rows[ids, h, kv]
                y = _values(pages[ids, h, kv], fmt, scale, r)
                c = y if r is None else y / r.double()[..., None]      # what p (p r) multiplies
                return y.flatten(-3, -2), c.flatten(-3, -2)
            X = q.view(B, q_len, HKV, G, 128)[mine, :, h].double().reshape(n, q_len * G, 128)
            flat = X.reshape(-1, 128)
            (Kp, _), (Vp, cp) = part(pre, 0, k), part(pre, 1, v)
            (Ko, _), (Vo, co) = part(own, 0, k), part(own, 1, v)
            zp = (flat @ Kp.T).view(n, q_len * G, -1) / 128 ** 0.5
            zo = (X @ Ko.transpose(1, 2) / 128 ** 0.5).masked_fill(hidden, -np.inf)
            size = torch.maximum((flat.abs() @ Kp.abs().T).amax(-1).view(n, q_len * G),
                                 (X.abs() @ Ko.abs().transpose(1, 2)).amax(-1)) / 128 ** 0.5
            top = torch.maximum(zp.amax(-1), zo.amax(-1))[..., None]
            p, po = torch.exp(zp - top), torch.exp(zo - top)
            l = (p.sum(-1) + po.sum(-1))[..., None]
            pf = p.view(n * q_len * G, -1)
            num = (pf @ Vp).view(X.shape) + po @ Vo
            out = num / l
            A = ((pf @ Vp.abs()).view(X.shape) + po @ Vo.abs()) / l
            many = (cp.abs().sum(0) + co.abs().sum(1)[:, None]) / l
            tol = ((2.0 ** -11 + 2.0 ** -18 + 256 * 2.0 ** -23 * size[..., None]) * A
                   + 2.0 ** -25 * many + 2.0 ** -11 * out.abs() + 2.0 ** -25)
            y = got[mine, :, h].double().reshape(X.shape)
            worst = ((y - out).abs() / tol).amax()
            assert worst <= 1.0, "group %d head %d: %.3g of the error allowed" % (g, h, worst)
            # what the bound sees: in the definition's own sums, a key tile left out, counted
            # twice, or with the V of the one before it would be beyond it for every sequence
            # of a few
            if h == 0:
                few = [0, n // 2, n - 1]
                for t in (0, shared[g] // 16 * 128, shared[g] * 16 - 128):
                    w = p[few, :, t:t + 128].cpu()
                    mass, value = w.sum(-1, keepdim=True), w @ Vp[t:t + 128].cpu()
                    other = w @ Vp[t - 128:t].cpu() if t else w @ Vp[t + 128:t + 256].cpu()
                    N_, l_, t_ = num[few].cpu(), l[few].cpu(), tol[few].cpu()
                    for wrong in ((N_ - value) / (l_ - mass), (N_ + value) / (l_ + mass),
                                  (N_ - value + other) / l_):
                        seen = ((wrong - N_ / l_).abs() / t_).amax((1, 2))
                        assert (seen > 1.0).all(), "the bound hides a key tile at %d" % t
