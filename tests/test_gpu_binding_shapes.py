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
