"""The serving-step calls refuse tensors of the wrong number of dimensions, none
included, as they refuse other shapes: with a ValueError that names the tensor."""
import pytest
import torch

import workloads as W
from tests.helpers import require_gpu
from tests.shared_case import SharedCase

pytestmark = pytest.mark.gpu


def test_tensors_of_other_dimensions_are_refused():
    pq = require_gpu()
    z = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")   # noqa: E731
    slots = torch.zeros(6, dtype=torch.int64, device="cuda")
    grow = dict(seq_lens=z(2), new_tokens=z(2), block_table=z(2, 4), free_pages=z(9),
                free_count=z(1), num_pages=9, seq_lens_out=z(2), free_count_out=z(1),
                slot_mapping=slots)
    cut = {k: grow[k] for k in ("seq_lens", "block_table", "free_pages", "free_count",
                                "seq_lens_out", "free_count_out")}
    cut["keep_lens"] = z(2)
    c = SharedCase([(100, [6, 7])], 8, 2, 1, W.FP8_E4M3)
    share = {**c.upload(), "out": torch.empty_like(c.g["q"])}
    for call, ok in ((pq.extend_block_tables, grow), (pq.truncate_block_tables, cut),
                     (pq.paged_attention_shared_prefix, share)):
        call(**ok)
        for name, x in ok.items():
            if not isinstance(x, torch.Tensor) or "scale" in name:
                continue
            for bad in (x.reshape(-1)[0], x[None], x.reshape(-1)[None, None, None]):
                with pytest.raises(ValueError, match=name):
                    call(**{**ok, name: bad})


@pytest.mark.parametrize("fmt", [W.FP8_E4M3, W.INT8])
def test_strided_vectors_are_refused(fmt):
    """The kernels read vectors densely: one with a stride was read in the wrong places."""
    pq = require_gpu()
    c = SharedCase([(100, [6, 7, 9])], 8, 2, 1, fmt, per_head=True)
    g = c.upload()
    strided = lambda x: torch.stack([x, x], 1)[:, 0]              # noqa: E731
    out, part = torch.empty_like(g["q"]), torch.empty(g["q"].shape, device="cuda")
    lse = torch.empty(g["q"].shape[:2], device="cuda")
    base = dict(q=g["q"], pages=g["pages"], block_table=g["block_table"], seq_lens=g["seq_lens"],
                q_len=1, kv_dtype=fmt, k_scale=g["k_scale"], v_scale=g["v_scale"])
    kv = torch.zeros((5, 2, 128), dtype=torch.float16, device="cuda")
    slots = torch.full((5,), -1, dtype=torch.int64, device="cuda")
    calls = [
        (pq.paged_attention, {**base, "out": out}, ("seq_lens", "k_scale", "v_scale")),
        (pq.paged_attention_noalloc, {**base, "out": out}, ("seq_lens", "k_scale", "v_scale")),
        (pq.paged_attention_partial, {**base, "q_pos": g["seq_lens"] - 1, "out_o": part,
                                      "out_lse": lse}, ("seq_lens", "q_pos", "k_scale", "v_scale")),
        (pq.paged_attention_shared_prefix, {**g, "out": out},
         ("seq_lens", "prefix_lens", "group_offsets", "k_scale", "v_scale")),
        (pq.kv_append_quant, dict(k=kv, v=kv, slot_mapping=slots, kv_dtype=fmt, pages=g["pages"],
                                  k_scale=g["k_scale"], v_scale=g["v_scale"]),
         ("slot_mapping", "k_scale", "v_scale")),
        (pq.lse_merge, dict(parts_o=part[None], parts_lse=lse[None], out=out,
                            out_lse=lse.reshape(-1)), ("out_lse",))]
    for call, ok, names in calls:
        call(**ok)
        for name in names:
            bad = strided(ok[name])
            if bad.numel() < 2:
                continue                                          # one element has no stride
            with pytest.raises(ValueError):
                call(**{**ok, name: bad})
