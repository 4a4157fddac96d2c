"""Every wait of the shared-prefix kernels is bounded: a copy that is never issued ends
in PQKV_DEV_TIMEOUT, not in a hang, whichever warps meet it first, and the next call
is right.  No GPU fault is involved: the testing entry point leaves one copy out and
its waits give up after about 1 ms."""
import ctypes
import time

import pytest
import torch

import workloads as W
from tests.helpers import require_gpu
from tests.shared_case import SharedCase

pytestmark = pytest.mark.gpu

K, V, PRIVATE, NONE = 0, 1, 2, 3
DEV_TIMEOUT = 8


def _call(c, out, ws, status, block, part, tile, fmt=None):
    pq = require_gpu()
    fn = pq.load_library().pqkv_testing_shared_prefix_wait_timeout
    i32, i64, vp, sz = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t
    fn.restype = ctypes.c_int
    fn.argtypes = [vp, vp, vp, i64, vp, i32, vp, i32, vp, vp, i32, i32, i32, i32, i32, i32, i32,
                   vp, vp, i32, i32, i32, vp, sz, vp, vp, i32, i32, i32]
    g = c.g
    return fn(g["q"].data_ptr(), out.data_ptr(), g["pages"].data_ptr(), g["pages"].shape[0],
              g["block_table"].data_ptr(), g["block_table"].shape[1], g["seq_lens"].data_ptr(),
              len(c.lens), g["group_offsets"].data_ptr(), g["prefix_lens"].data_ptr(),
              len(c.prefix), c.q_len, c.hq, c.hkv, 128, 16, c.fmt if fmt is None else fmt,
              g["k_scale"].data_ptr(), g["v_scale"].data_ptr(), 0, 0, 0, ws.data_ptr(),
              ws.numel(), status.data_ptr(), torch.cuda.current_stream().cuda_stream, block, part,
              tile)


@pytest.fixture(scope="module", params=[(W.FP8_E4M3, 13), (W.FP8_E4M3, 4), (W.FP16, 13),
                                        (W.FP16, 4)],
                ids=lambda p: "%s-%d" % ("fp16" if p[0] == W.FP16 else "e4m3", p[1]))
def case(request):
    """13 sequences of 20 rows a head: a tile of 256 rows and a small one.  4: only a
    small one, whose streams take the key tiles in turn.  Every CTA has several key
    tiles, every warp several private pages."""
    pq = require_gpu()
    fmt, n = request.param
    c = SharedCase([(22000 if n > 4 else 40000, [1600] * n)], 8, 2, 5, fmt, seed=n)
    c.upload()
    need = pq.shared_prefix_workspace_size(n, 1, 5, 8, 2)
    c.ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    c.good = c.run(workspace=c.ws).clone()
    c.check(c.good, seqs=[0, n - 1], heads=[1])
    return c


@pytest.mark.parametrize("block,part,tile", [
    (0, K, 0), (0, V, 0), (0, K, 1), (0, V, 1), (77, K, 2), (77, V, 2), (151, K, 1), (151, V, 1),
    (0, PRIVATE, 0), (100, PRIVATE, 0)])
def test_a_copy_that_never_comes_is_reported_and_the_call_returns(case, block, part, tile):
    pq = require_gpu()
    c = case
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.empty_like(c.good)
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    assert _call(c, out, c.ws, status, block, part, tile) == 0
    torch.cuda.synchronize()                     # returns: no hang, no CUDA error
    assert time.perf_counter() - t0 < 1.0
    assert int(status.item()) == DEV_TIMEOUT
    status.zero_()
    assert torch.equal(c.run(workspace=c.ws, status=status), c.good)
    assert int(status.item()) == 0


def test_nothing_left_out_is_the_normal_call(case):
    c = case
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for block, part, tile in [(0, NONE, 0), (0, K, 1 << 30), (1 << 30, PRIVATE, 0)]:
        out = torch.empty_like(c.good)
        assert _call(c, out, c.ws, status, block, part, tile) == 0
        assert torch.equal(out, c.good)
    assert int(status.item()) == 0


def test_other_formats_are_refused(case):
    c = case
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.empty_like(c.good)
    assert _call(c, out, c.ws, status, 0, K, 0, fmt=W.INT8) == -2
