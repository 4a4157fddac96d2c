"""Calls of the serving-step operators where nothing has gone before: the process's
first one inside a stream capture, and first ones from several host threads at once."""
import subprocess
import sys

import pytest

from tests.helpers import require_gpu

pytestmark = pytest.mark.gpu

SETUP = """
import threading
import torch
import workloads as W
import paged_quantized_kv_append_gb300 as pq
from tests.shared_case import SharedCase
cases = [SharedCase([(600, [30] * 9), (0, [20])], 8, 2, 5, f, seed=f) for f in
         (W.FP16, W.FP8_E4M3, W.INT8, W.INT8_ROW)]
outs = [torch.full_like(c.upload()["q"], float("nan")) for c in cases]
i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
sl, fc, fp, bt = i32([0] * 7), i32([40]), i32(list(range(40))), i32([[-1] * 4] * 7)
new, keep = i32([33] * 7), i32([1] * 7)
slots = torch.empty(300, dtype=torch.int64, device="cuda")
def tables():
    pq.extend_block_tables(sl, new, bt, fp, fc, 40, sl, fc, slots)
    pq.truncate_block_tables(sl, keep, bt, fp, fc, sl, fc)
def check():
    torch.cuda.synchronize()
    for c, o in zip(cases, outs):
        c.check(o)
    assert sl.tolist() == [1] * 7 and int(fc.item()) == 33
torch.cuda.synchronize()
"""
CAPTURED = SETUP + """
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    for c, o in zip(cases, outs):
        c.run(out=o)
    tables()
graph.replay()
check()
"""
THREADS = SETUP + """
streams = [torch.cuda.Stream() for _ in range(5)]
start = threading.Barrier(5)
failed = []
def work(k):
    try:
        start.wait()
        with torch.cuda.stream(streams[k]):
            if k == 4:
                tables()
            else:
                for _ in range(20):
                    cases[k].run(out=outs[k])
    except BaseException as e:
        failed.append(e)
threads = [threading.Thread(target=work, args=(k,)) for k in range(5)]
[t.start() for t in threads]
[t.join() for t in threads]
assert not failed, failed
check()
"""


@pytest.mark.parametrize("program", [CAPTURED, THREADS], ids=["captured", "threads"])
def test_first_calls(program):
    require_gpu()
    r = subprocess.run([sys.executable, "-c", program], capture_output=True, text=True, timeout=240)
    assert r.returncode == 0, r.stderr[-3000:]
