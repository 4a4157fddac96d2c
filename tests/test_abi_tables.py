"""pqkv_extend_block_tables and pqkv_truncate_block_tables reject bad arguments
on the host, without a GPU."""
import pytest
import torch

import paged_quantized_kv_append_gb300 as pq
from paged_quantized_kv_append_gb300 import build as pqbuild

OK, EINVAL, EUNSUPPORTED, ERANGE, EWORKSPACE, ECUDA = 0, -1, -2, -3, -4, -5
P = 1 << 12


@pytest.fixture(scope="module")
def lib():
    pqbuild.build()
    return pq.load_library()


def _extend(lib, **kw):
    a = dict(sl=P, new=P, B=4, bt=P, W=8, fp=P, fc=P, cap=100, npages=50, ps=16, slo=P, fco=P,
             slots=P, pos=P, T=20, off=P, st=None)
    a.update(kw)
    return lib.pqkv_extend_block_tables(a["sl"], a["new"], a["B"], a["bt"], a["W"], a["fp"],
                                        a["fc"], a["cap"], a["npages"], a["ps"], a["slo"],
                                        a["fco"], a["slots"], a["pos"], a["T"], a["off"], a["st"],
                                        None)


def _truncate(lib, **kw):
    a = dict(sl=P, keep=P, own=P, B=4, bt=P, W=8, fp=P, fc=P, cap=100, ps=16, slo=P, fco=P,
             st=None)
    a.update(kw)
    return lib.pqkv_truncate_block_tables(a["sl"], a["keep"], a["own"], a["B"], a["bt"], a["W"],
                                          a["fp"], a["fc"], a["cap"], a["ps"], a["slo"], a["fco"],
                                          a["st"], None)


@pytest.mark.parametrize("call", [_extend, _truncate])
def test_shared_refusals(lib, call):
    assert call(lib) == ECUDA                             # valid, but no GPU here
    assert call(lib, B=-1) == EINVAL
    assert call(lib, B=2049) == ERANGE
    assert call(lib, W=0) == EINVAL
    assert call(lib, W=32770) == ERANGE                   # beyond 524288 tokens
    assert call(lib, W=32769) == ECUDA
    assert call(lib, ps=32) == EUNSUPPORTED
    assert call(lib, cap=-1) == EINVAL
    assert call(lib, cap=0, fp=None) == ECUDA             # an empty stack is allowed
    for name in ("sl", "bt", "fp", "fc", "slo", "fco"):
        assert call(lib, **{name: None}) == EINVAL, name
        assert call(lib, **{name: P + 2}) == EINVAL, name
    assert call(lib, st=P + 1) == EINVAL
    assert call(lib, B=0, sl=None, bt=None, slo=None) == ECUDA


def test_extend_refusals(lib):
    assert _extend(lib, new=None) == EINVAL
    assert _extend(lib, slots=None) == EINVAL
    assert _extend(lib, slots=P + 4) == EINVAL            # 8-byte entries
    assert _extend(lib, pos=P + 1) == EINVAL
    assert _extend(lib, off=P + 1) == EINVAL
    assert _extend(lib, pos=None, off=None) == ECUDA
    assert _extend(lib, T=0, slots=None) == ECUDA
    assert _extend(lib, T=-1) == EINVAL
    assert _extend(lib, npages=-1) == EINVAL
    assert _extend(lib, npages=1 << 31) == EINVAL


def test_truncate_refusals(lib):
    assert _truncate(lib, keep=None) == EINVAL
    assert _truncate(lib, own=None) == ECUDA
    assert _truncate(lib, own=P + 2) == EINVAL


def test_the_binding_refuses_host_tensors():
    z = lambda *s: torch.zeros(s, dtype=torch.int32)      # noqa: E731
    with pytest.raises(ValueError, match="CUDA"):
        pq.extend_block_tables(z(2), z(2), z(2, 4), z(9), z(1), 9, z(2), z(1),
                               torch.zeros(5, dtype=torch.int64))
    with pytest.raises(ValueError, match="CUDA"):
        pq.truncate_block_tables(z(2), z(2), z(2, 4), z(9), z(1), z(2), z(1))
