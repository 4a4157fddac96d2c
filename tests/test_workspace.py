"""One Workspace for calls of different sizes: merge counters of one call must not lie
where another call has left partial results."""
import pytest
import torch

import paged_quantized_kv_append_gb300 as pq
import workloads as W
from tests.helpers import require_gpu


def test_the_counters_of_every_call_end_at_the_same_byte():
    ws = pq.Workspace("cpu")
    assert ws.get(0, 4) is None
    ends = set()
    for counters in (4, 4 * 8 * 8, 4 * 64 * 8, 4 * 2048 * 8, 256):
        rounded = -(-counters // 256) * 256
        part = ws.get(rounded + 5000, counters)
        assert part.numel() >= rounded + 5000 and part.data_ptr() % 256 == ws.buf.data_ptr() % 256
        ends.add(part.data_ptr() - ws.buf.data_ptr() + rounded)
    assert len(ends) == 1
    part = ws.get(9 << 20, 4 * 2048 * 256)                 # more counters than room for them
    assert part.numel() >= 9 << 20 and not part.any()


def test_a_call_like_an_earlier_one_makes_no_new_view():
    """(The attention calls' own path: a slice a call is a microsecond of the host's.)"""
    ws = pq.Workspace("cpu")
    a, b = ws.get(9000, 4), ws.get(9000, 4 * 64 * 8)
    assert ws.get(9000, 4) is a and ws.get(5000, 250) is a and ws.get(9000, 4 * 64 * 8) is b
    grown = ws.get(8 << 20, 4)                              # a new buffer: no view of the old one
    assert grown.numel() >= 8 << 20 and grown.data_ptr() == ws.buf.data_ptr() + ws.head - 256
    assert ws.get(9000, 4 * 64 * 8).data_ptr() == ws.buf.data_ptr() + ws.head - 2048


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", [W.FP16, W.FP8_E4M3])
def test_batches_of_many_sizes_through_one_workspace(fmt):
    require_gpu()
    gen = torch.Generator(device="cuda").manual_seed(5)
    shared = pq.Workspace("cuda")
    scale = torch.ones(1, device="cuda")
    for B, hkv, L in [(4, 2, 900), (40, 8, 700), (2, 1, 5000), (120, 8, 300), (1, 8, 9000), (64, 4, 500)]:
        width = -(-L // 16)
        pages = pq.new_pages(B * width, hkv, fmt, "cuda")
        x = torch.randn(pages.shape, generator=gen, device="cuda")
        pages.copy_(x if fmt == W.FP16 else x.to(torch.float8_e4m3fn).view(torch.uint8))
        bt = torch.randperm(B * width, generator=gen, device="cuda").int().view(B, width)
        lens = torch.full((B,), L, dtype=torch.int32, device="cuda")
        q = torch.randn((B, 4 * hkv, 128), generator=gen, device="cuda").half()
        args = (q, pages, bt, lens, 1, fmt, scale, scale)
        want = pq.paged_attention(*args, torch.empty_like(q), workspace=pq.Workspace("cuda"))
        for _ in range(2):
            got = pq.paged_attention(*args, torch.full_like(q, float("nan")), workspace=shared)
            assert torch.equal(got, want), (B, hkv, L)


@pytest.mark.gpu
def test_shared_prefix_attention_takes_a_workspace_like_the_other_calls():
    """One Workspace for both attention calls in turn, whose merge counters the shared
    call leaves alone; anything that is no workspace is refused as a ValueError."""
    require_gpu()
    from tests.shared_case import SharedCase
    ws = pq.Workspace("cuda")
    c = SharedCase([(300, [20, 9, 33]), (0, [40])], 16, 4, 2, W.FP8_E4M3, seed=3)
    g = c.upload()
    args = [g[k] for k in ("q", "pages", "block_table", "seq_lens", "q_len", "kv_dtype", "k_scale",
                           "v_scale")]
    want, plain = c.run().clone(), pq.paged_attention(*args, torch.empty_like(g["q"]))
    for _ in range(3):
        assert torch.equal(c.run(workspace=ws), want)
        got = pq.paged_attention(*args, torch.full_like(g["q"], float("nan")), workspace=ws)
        assert torch.equal(got, plain)
    need = pq.shared_prefix_workspace_size(4, 2, 2, 16, 4)
    whole = torch.empty(2 * need, dtype=torch.uint8, device="cuda")
    assert torch.equal(c.run(workspace=whole), want)
    for bad in (17, "ws", [whole], whole.cpu(), whole[::2], whole.data_ptr()):
        with pytest.raises(ValueError, match="workspace"):
            c.run(workspace=bad)
    with pytest.raises(ValueError, match="size"):            # sizes the call refuses
        c.run(q=g["q"].repeat(1, 3, 1).contiguous(), out=torch.empty_like(g["q"]).repeat(1, 3, 1),
              q_len=2, workspace=pq.Workspace("cuda"), group_offsets=torch.zeros(
                  3000, dtype=torch.int32, device="cuda"),
              prefix_lens=torch.zeros(2999, dtype=torch.int32, device="cuda"))
