"""What the attention calls take as a workspace: a Workspace or a contiguous tensor on the pool's
GPU.  A strided or expanded one has fewer bytes of its own than elements, and the kernels would
write its neighbours'."""
import pytest
import torch

import workloads as W
from tests.helpers import Case, require_gpu

pytestmark = pytest.mark.gpu


def test_no_workspaces_are_refused():
    pq = require_gpu()
    c = Case(W.workload("e4m3_verify_131k", scale=0.01), with_oracle=False)
    w = c.w
    need = pq.workspace_size(w.num_seqs, w.q_len, w.num_q_heads, w.num_kv_heads)
    whole = torch.zeros(need + (1 << 20), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(c.q)
    o, lse = torch.empty(c.q.shape, device="cuda"), torch.empty(c.q.shape[:2], device="cuda")
    pos = (c.seq_lens - w.q_len).int()

    def plain(ws):
        return pq.paged_attention(c.q, c.pages, c.bt, c.seq_lens, w.q_len, w.kv_dtype, c.ks, c.vs,
                                  out, workspace=ws)

    def partial(ws):
        return pq.paged_attention_partial(c.q, c.pages, c.bt, c.seq_lens, pos, w.q_len, w.kv_dtype,
                                          c.ks, c.vs, o, lse, workspace=ws)

    for call in (plain, partial):
        for bad in (17, "ws", [whole], whole.cpu(), whole.data_ptr(), whole[::2],
                    torch.zeros(1, dtype=torch.uint8, device="cuda").expand(len(whole))):
            with pytest.raises(ValueError, match="workspace must be"):
                call(bad)
        with pytest.raises(pq.PqkvError, match="workspace"):
            call(whole[:4096])             # (workspace_size is that of the largest grid)
    # none was launched: the workspace is as it was, and serves
    assert not whole.any()
    assert torch.equal(plain(whole[:need]), c.attention())
