"""Append, attention and kv_read over a 4-bit pool where nothing has gone before: the process's
first calls inside a stream capture, without a workspace, and first ones from several threads."""
import subprocess
import sys

import pytest

from tests.helpers import require_gpu

pytestmark = pytest.mark.gpu

SETUP = """
import threading
import numpy as np
import torch
import oracle
import paged_quantized_kv_append_gb300 as pq
from tests.int4_case import F, Pool, allowance, assert_within, rows, slots
dev = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()
i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
p = Pool(1, [3000, 70, 900], 2)
k, v = rows(np.random.default_rng(2), 5, 2), rows(np.random.default_rng(3), 5, 2)
at = slots(p.bt, 1, 65, 70)
pool = oracle.kv_append_quant(k, v, at, F, None, None, p.pages)
kd, vd, atd, bt, lens = dev(k), dev(v), dev(at), dev(p.bt), i32(p.lens)
off = i32([0, 40, 75])
class Run:
    def __init__(self, q_len, hq):
        self.q_len, self.qh, self.pages = q_len, p.q(q_len, q_len, hq), dev(p.pages)
        self.q = dev(self.qh)
        self.outs = [torch.full_like(self.q, float("nan")) for _ in range(3)]
        self.read = [torch.full((75, 2, 128), float("nan"), device="cuda").half() for _ in "kv"]
    def calls(self):
        pq.kv_append_quant(kd, vd, atd, "int4_group", None, None, self.pages)
        for o, kw in zip(self.outs, ({}, {"window": 300}, {"num_splits": 3})):
            pq.paged_attention(self.q, self.pages, bt, lens, self.q_len, "int4_group", None, None, o, **kw)
        pq.kv_read(self.pages, bt[:2], None, off, "int4_group", None, None, *self.read)
    def check(self):
        assert np.array_equal(self.pages.cpu().numpy(), pool)
        for o, w in zip(self.outs, (0, 300, 0)):
            ref, bound = allowance(self.qh, pool, p.bt, p.lens, self.q_len, window=w)
            assert_within(o, ref, bound)
        K, V = oracle.kv_read(pool, p.bt, None, [0, 40, 75], F, None, None)
        assert np.array_equal(self.read[0].cpu().numpy(), K) and np.array_equal(self.read[1].cpu().numpy(), V)
runs = [Run(1, 8), Run(3, 8), Run(5, 8), Run(8, 8)]
torch.cuda.synchronize()
"""
CAPTURED = SETUP + """
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    for r in runs:
        r.calls()
for _ in range(2):
    for r in runs:
        [o.fill_(float("nan")) for o in r.outs]
    graph.replay()
    torch.cuda.synchronize()
    [r.check() for r in runs]
"""
THREADS = SETUP + """
streams = [torch.cuda.Stream() for _ in runs]
start = threading.Barrier(len(runs))
failed = []
def work(k):
    try:
        start.wait()
        with torch.cuda.stream(streams[k]):
            for _ in range(20):
                runs[k].calls()
    except BaseException as e:
        failed.append(e)
threads = [threading.Thread(target=work, args=(k,)) for k in range(len(runs))]
[t.start() for t in threads]
[t.join() for t in threads]
assert not failed, failed
torch.cuda.synchronize()
[r.check() for r in runs]
"""


@pytest.mark.parametrize("program", [CAPTURED, THREADS], ids=["captured", "threads"])
def test_first_calls(program):
    require_gpu()
    r = subprocess.run([sys.executable, "-c", program], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-3000:]
