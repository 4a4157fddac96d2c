"""Workspaces on the streams that use them: zeroed in the call's own order, kept while an earlier
call or graph may use them, one per stream where the caller gave none."""
import contextlib

import pytest
import torch

import paged_quantized_kv_append_gb300 as pq
from tests.helpers import require_gpu
from tests.int4_case import Pool


def test_a_buffer_is_made_on_the_calls_stream(monkeypatch):
    """(On the host: the contexts that a call on a stream enters.)"""
    inside, made = [], []

    @contextlib.contextmanager
    def on(stream):
        inside.append(stream)
        yield
        inside.pop()

    zeros = torch.zeros
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch, "zeros", lambda *a, **k: (made.append(list(inside)), zeros(*a, **k))[1])
    ws, st = pq.Workspace("cpu"), object()
    ws.get(9000, 256, stream=st)
    ws.get(9000, 256, stream=object())                # there: nothing is made
    ws.get(64 << 20, 256, stream=st)                  # grown
    ws.get(9000, 1 << 20, stream=st)                  # more counters than room for them
    assert made == [[st]] * 3 and not inside


def test_a_buffer_that_is_too_small_is_kept():
    """Kernels in flight and captured graphs still write there."""
    ws, seen = pq.Workspace("cpu"), []
    for nbytes, counters in ((9000, 256), (3 << 20, 256), (40 << 20, 256), (9000, 1 << 20)):
        part = ws.get(nbytes, counters)
        seen.append(ws.buf)
        assert not part.any()
        part.fill_(1)
    assert len({b.data_ptr() for b in seen}) == len(seen) == len(ws._old) + 1
    assert all(a is b for a, b in zip(ws._old, seen))
    assert sum(b.numel() for b in ws._old) <= ws.buf.numel()
    assert ws.get(9000, 256).data_ptr() - ws.buf.data_ptr() == ws.head - 256


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Call:
    """A verify over a 4-bit pool whose segments are split over several CTAs."""

    def __init__(self, seed, lens, q_len=5, hq=32, hkv=8):
        p = Pool(seed, lens, hkv)
        dev = [torch.from_numpy(x).cuda() for x in (p.q(1, q_len, hq), p.pages, p.bt)]
        self.args = (*dev, _i32(p.lens), q_len, "int4_group", None, None)
        self.want = self(workspace=pq.Workspace())
        torch.cuda.synchronize()

    def __call__(self, **kw):
        out = torch.full_like(self.args[0], float("nan"))
        return pq.paged_attention(*self.args, out, **kw)

    def into(self, out, **kw):
        return pq.paged_attention(*self.args, out, **kw)


def _dirty(nbytes):
    """Freed memory of the current stream that is not zero."""
    x = [torch.full((nbytes,), 255, dtype=torch.uint8, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    del x


@pytest.mark.gpu
def test_first_and_growing_calls_on_a_side_stream():
    """The default stream is busy, and the memory that it would zero is not zero."""
    require_gpu()
    small, large = Call(1, [3000, 70, 900]), Call(2, [700] * 64)
    outs = [torch.empty_like(c.args[0]) for c in (small, large, small)]
    for _ in range(3):
        st, ws = torch.cuda.Stream(), pq.Workspace()
        for size in (1 << 20, 64 << 20):
            _dirty(size)
            with torch.cuda.stream(st):
                _dirty(size)
        for o in outs:
            o.fill_(float("nan"))
        torch.cuda.synchronize()
        torch.cuda._sleep(20_000_000)
        for c, o in zip((small, large, small), outs):
            c.into(o, stream=st, workspace=ws)
        assert len(ws._old) == 1
        torch.cuda.synchronize()
        for c, o in zip((small, large, small), outs):
            assert torch.equal(o, c.want)


@pytest.mark.gpu
def test_streams_without_a_workspace_do_not_meet():
    require_gpu()
    cases = [Call(3, [3000, 70, 900]), Call(4, [5000, 16]), Call(5, [900] * 8)]
    streams = [torch.cuda.Stream() for _ in cases]
    outs = [[torch.full_like(c.args[0], float("nan")) for _ in range(20)] for c in cases]
    torch.cuda.synchronize()
    for k in range(20):
        for c, st, o in zip(cases, streams, outs):
            if k % 2:
                c.into(o[k], stream=st)
            else:
                with torch.cuda.stream(st):
                    c.into(o[k])
    torch.cuda.synchronize()
    for c, o in zip(cases, outs):
        assert all(torch.equal(x, c.want) for x in o)


def _captured(call, **kw):
    out = torch.empty_like(call.args[0])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call.into(out, **kw)
        torch.empty(1 << 22, dtype=torch.uint8, device="cuda").fill_(255)   # of the graph's memory
    return g, out


@pytest.mark.gpu
def test_graphs_without_a_workspace_replay_side_by_side():
    """Captured on one stream, replayed on two at once, beside an eager call."""
    require_gpu()
    a, b, c = Call(6, [3000, 70, 900]), Call(7, [5000, 16]), Call(8, [900] * 8)
    graphs = [_captured(x) for x in (a, b)]
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(10):
        for _, out in graphs:
            out.fill_(float("nan"))
        torch.cuda.synchronize()
        for _ in range(5):
            for (g, _), st in zip(graphs, streams):
                with torch.cuda.stream(st):
                    g.replay()
            got = c()
        torch.cuda.synchronize()
        assert torch.equal(got, c.want)
        for (_, out), x in zip(graphs, (a, b)):
            assert torch.equal(out, x.want)


@pytest.mark.gpu
def test_a_workspace_that_is_first_used_in_a_capture():
    """Another graph and eager calls use it before that graph is replayed; and it grows after a
    graph has captured a smaller buffer."""
    require_gpu()
    a, b, large = Call(9, [3000, 70, 900]), Call(10, [5000, 16]), Call(11, [700] * 64)
    _dirty(1 << 20)
    ws = pq.Workspace()
    first = _captured(a, workspace=ws)
    assert torch.equal(b(workspace=ws), b.want)
    second = _captured(b, workspace=ws)
    assert torch.equal(large(workspace=ws), large.want) and len(ws._old) == 1
    _dirty(ws._old[0].numel())
    for _ in range(3):
        for (g, out), x in zip((second, first), (b, a)):
            out.fill_(float("nan"))
            g.replay()
            assert torch.equal(out, x.want)
        assert torch.equal(a(workspace=ws), a.want)


@pytest.mark.gpu
def test_a_call_on_a_given_stream_that_is_captured():
    """Begun and ended on that stream, which is not the current one when the call is made; the
    current stream stays what it was."""
    require_gpu()
    a, other = Call(12, [3000, 70, 900]), torch.cuda.Stream()
    out, st, g = torch.empty_like(a.args[0]), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    a.into(out, stream=st)                       # st has an eager workspace of its own
    torch.cuda.synchronize()
    before = set(pq._default_ws)
    with torch.cuda.stream(st):
        g.capture_begin()
    try:
        with torch.cuda.stream(other):
            a.into(out, stream=st)
            assert torch.cuda.current_stream() == other
    finally:
        with torch.cuda.stream(st):
            g.capture_end()
    assert set(pq._default_ws) == before
    for _ in range(3):
        out.fill_(float("nan"))
        torch.cuda.synchronize()
        g.replay()
        eager = [a(stream=st) for _ in range(3)]
        torch.cuda.synchronize()
        assert torch.equal(out, a.want) and all(torch.equal(x, a.want) for x in eager)
