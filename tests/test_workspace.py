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
