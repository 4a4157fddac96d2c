"""kv_read of every format against the oracle.

FP16 and 4-bit values are exact.  An 8-bit value is a code (8 bits at most) times an fp32
scale, rounded to fp32 and then to fp16: off by half a step of fp16, 2^-11 of the value,
and 2^-24 of it before, and by 2^-25 where fp16 is subnormal."""
import numpy as np
import pytest
import torch

import oracle
import workloads as W
from tests.helpers import require_gpu
from tests.int4_case import F, rows, slots, tables

pytestmark = pytest.mark.gpu
FORMATS = [W.FP16, W.FP8_E4M3, W.INT8, W.INT8_ROW, F]


def _dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


class Filled:
    """A pool filled on the GPU by kv_append_quant (which other tests hold to the oracle)
    and the same in the oracle."""

    def __init__(self, fmt, seed, lens, H, per_head=True, slack=2):
        pq = require_gpu()
        rng = np.random.default_rng(seed)
        self.fmt, self.H, self.lens = fmt, H, lens
        self.bt, n = tables(rng, lens, slack)
        at = np.concatenate([slots(self.bt, s, 0, L) for s, L in enumerate(lens)] + [[]])
        at = at.astype(np.int64)
        k, v = rows(rng, len(at), H), rows(rng, len(at), H)
        sc = (0.05 + 0.3 * rng.random(H if per_head else 1)).astype(np.float32)
        self.ks, self.vs = sc, sc[::-1].copy()
        self.pages = pq.new_pages(n, H, fmt, fill=0)
        pq.kv_append_quant(_dev(k), _dev(v), _dev(at), fmt, _dev(self.ks), _dev(self.vs), self.pages)
        pool = oracle.new_pool(n, H, 128, fmt)
        if fmt == W.INT8_ROW:
            z = oracle.new_scale_pool(n, H)
            self.pool, self.oks, self.ovs = oracle.kv_append_quant(k, v, at, fmt, z, z, pool)
        else:
            self.pool = oracle.kv_append_quant(k, v, at, fmt, self.ks, self.vs, pool)
            self.oks, self.ovs = self.ks, self.vs

    def read(self, first, n, T=None, bt=None, status=None, k=None, v=None, **kw):
        pq = require_gpu()
        off = np.concatenate([[0], np.cumsum(n)]).astype(int)
        T = off[-1] if T is None else T
        if k is None:
            k, v = (torch.full((T, self.H, 128), 77.0, dtype=torch.float16, device="cuda")
                    for _ in "kv")
        pq.kv_read(self.pages, _dev(self.bt if bt is None else bt), None if first is None else
                   _i32(first), _i32(off), self.fmt, _dev(self.ks), _dev(self.vs), k, v,
                   status=status, **kw)
        return off, k, v

    def check(self, off, first, k, v, bt=None, pool=None):
        K, V = oracle.kv_read(self.pool if pool is None else pool, self.bt if bt is None else bt,
                              first, off, self.fmt, self.oks, self.ovs)
        for got, ref in ((k, K), (v, V)):
            g = got[:off[-1]].cpu().numpy().astype(np.float64)
            slack = 0 if self.fmt in (W.FP16, F) else 1
            bound = slack * (np.abs(ref) * (2.0 ** -11 + 2.0 ** -23) + 2.0 ** -25)
            assert (np.abs(g - ref) <= bound).all()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("H", [1, 3, 8])
def test_ragged_requests(fmt, H):
    lens = [1, 15, 16, 17, 100, 0, 333]
    c = Filled(fmt, H, lens, H, per_head=H > 1)
    c.check(*_of(c, None, lens))
    first = [0, 14, 16, 3, 37, 0, 16]
    n = [1, 1, 0, 14, 63, 0, 300]
    c.check(*_of(c, first, n))


def _of(c, first, n):
    off, k, v = c.read(first, n)
    return off, first, k, v


@pytest.mark.parametrize("fmt", FORMATS)
def test_rows_behind_the_last_and_strided_rows_stay(fmt):
    c = Filled(fmt, 5, [40, 9], 2)
    big = torch.full((60, 5 * 256), 77.0, dtype=torch.float16, device="cuda")
    k = big[:, 256:512].view(60, 2, 128)
    v = big[:, 768:1024].view(60, 2, 128)
    off, k, v = c.read([2, 0], [30, 9], k=k, v=v)
    c.check(off, [2, 0], k, v)
    assert (big[39:] == 77).all()
    assert (big[:, :256] == 77).all() and (big[:, 512:768] == 77).all() and (big[:, 1024:] == 77).all()


@pytest.mark.parametrize("fmt", FORMATS)
def test_pages_outside_the_pool_read_zeros(fmt):
    pq = require_gpu()
    c = Filled(fmt, 6, [50, 20], 2, slack=0)
    bt = c.bt.copy()
    bt[0, 1], bt[1, 0] = -1, len(c.pool)
    st = _i32([0])
    off, k, v = c.read(None, [50, 20], bt=bt, status=st)
    assert pq.status_bits(st) == ["block-table page id out of range"]
    zeros = np.zeros(70, bool)
    zeros[16:32] = zeros[50:66] = True
    _, k0, v0 = c.read(None, [50, 20])
    for got, ref in ((k, k0), (v, v0)):
        assert (got[torch.from_numpy(zeros).cuda()] == 0).all()
        assert torch.equal(got[torch.from_numpy(~zeros).cuda()], ref[torch.from_numpy(~zeros).cuda()])


def test_positions_outside_the_row_are_left():
    pq = require_gpu()
    c = Filled(F, 7, [32, 32], 2)
    st = _i32([0])
    off, k, v = c.read([-3, 28], [5, 9], status=st)
    assert pq.status_bits(st) == ["seq_len out of range"]
    assert (k[:3] == 77).all() and (v[9:] == 77).all()
    _, k0, v0 = c.read([0, 28], [2, 4])
    assert torch.equal(k[3:9], k0) and torch.equal(v[3:9], v0)


@pytest.mark.parametrize("off,bits", [([0, 5, 3], True), ([2, 5, 8], True), ([0, 5, 900], True),
                                      ([0, 0, 0], False), ([0, -4, 8], True)])
def test_offsets_that_fall_or_end_outside_are_reported(off, bits):
    pq = require_gpu()
    c = Filled(F, 8, [32, 32], 2)
    big = torch.full((30, 2, 128), 77.0, dtype=torch.float16, device="cuda")
    k, v = big[10:18], torch.full_like(big[10:18], 77.0)
    st = _i32([0])
    pq.kv_read(c.pages, _dev(c.bt), None, _i32(off), F, None, None, k, v, status=st)
    assert pq.status_bits(st) == (["seq_len out of range"] if bits else [])
    assert (big[:10] == 77).all() and (big[18:] == 77).all()


@pytest.mark.parametrize("fmt", [W.FP8_E4M3, W.INT8])
def test_a_bad_scale_leaves_its_rows(fmt):
    pq = require_gpu()
    c = Filled(fmt, 9, [20], 3)
    c.vs = np.array([0.1, np.nan, 0.2], np.float32)
    st = _i32([0])
    _, k, v = c.read(None, [20], status=st)
    assert pq.status_bits(st) == ["bad scale"]
    assert (v[:, 1] == 77).all() and not (v[:, 2] == 77).all() and not (k == 77).any()


def test_many_requests_a_graph_and_another_stream():
    rng = np.random.default_rng(10)
    lens = rng.integers(0, 40, 2048).tolist()
    c = Filled(F, 11, lens, 2)
    off, k, v = c.read(None, lens)
    c.check(off, None, k, v)
    bt, o = _dev(c.bt), _i32(off)
    pq = require_gpu()
    g = torch.cuda.CUDAGraph()
    k2, v2 = torch.zeros_like(k), torch.zeros_like(v)
    with torch.cuda.graph(g):
        pq.kv_read(c.pages, bt, None, o, F, None, None, k2, v2)
    for _ in range(2):
        k2.zero_()
        g.replay()
        assert torch.equal(k, k2) and torch.equal(v, v2)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    k2.zero_()
    torch.cuda.synchronize()
    pq.kv_read(c.pages, bt, None, o, F, None, None, k2, v2, stream=st)
    st.synchronize()
    assert torch.equal(k, k2)


def test_no_requests_and_no_tokens():
    pq = require_gpu()
    pages = pq.new_pages(2, 1, "int4_group", fill=0)
    none = torch.empty((0, 1, 128), dtype=torch.float16, device="cuda")
    pq.kv_read(pages, torch.empty((0, 4), dtype=torch.int32, device="cuda"), None, _i32([0]),
               "int4_group", None, None, none, none)
    pq.kv_read(pages, _i32([[0]]), _i32([0]), _i32([0, 0]), "int4_group", None, None, none, none)


def test_refusals():
    pq = require_gpu()
    c = Filled(W.INT8, 12, [20], 2)
    k = torch.empty((20, 2, 128), dtype=torch.float16, device="cuda")
    good = dict(pages=c.pages, block_table=_dev(c.bt), first_pos=_i32([0]),
                token_offsets=_i32([0, 20]), kv_dtype="int8", k_scale=_dev(c.ks),
                v_scale=_dev(c.vs), k=k, v=k.clone())
    pq.kv_read(**good)
    wide = torch.empty((20, 2 * 128 + 8), dtype=torch.float16, device="cuda")
    for name, bad in [("block_table", _dev(c.bt).long()), ("block_table", _i32([0])),
                      ("first_pos", _i32([0, 0])), ("token_offsets", _i32([0])),
                      ("k", k.float()), ("k", k[:, :1]), ("v", k[:10]), ("k", k.cpu()),
                      ("v", k.transpose(1, 2).contiguous().transpose(1, 2)),
                      ("k", wide[:, :256].view(20, 2, 128)), ("k", wide[:, 8:].view(20, 2, 128)),
                      ("k_scale", _dev(c.ks).double()), ("v_scale", _dev(c.vs)[:1]),
                      ("pages", c.pages[..., :72]), ("status", torch.zeros(1, device="cuda"))]:
        with pytest.raises(ValueError):
            pq.kv_read(**dict(good, **{name: bad}))
    with pytest.raises(ValueError):
        pq.kv_read(**dict(good, block_table=torch.zeros((2049, 1), dtype=torch.int32, device="cuda"),
                          first_pos=None,
                          token_offsets=torch.zeros(2050, dtype=torch.int32, device="cuda")))
