"""pqkv_paged_attention_shared_prefix rejects bad arguments on the host."""
import pytest

import paged_quantized_kv_append_gb300 as pq
from paged_quantized_kv_append_gb300 import build as pqbuild

OK, EINVAL, EUNSUPPORTED, ERANGE, EWORKSPACE, ECUDA = 0, -1, -2, -3, -4, -5
P = 1 << 12


@pytest.fixture(scope="module")
def lib():
    pqbuild.build()
    return pq.load_library()


def _call(lib, **kw):
    a = dict(q=P, out=P, pages=P, npages=100, bt=P, W=8, sl=P, B=2, go=P, pl=P, M=1, qlen=5, hq=32,
             hkv=8, D=128, ps=16, dt=1, ks=P, vs=P, sph=0, msl=0, mpl=0, ws=P, wsb=1 << 40, st=None)
    a.update(kw)
    return lib.pqkv_paged_attention_shared_prefix(
        a["q"], a["out"], a["pages"], a["npages"], a["bt"], a["W"], a["sl"], a["B"], a["go"],
        a["pl"], a["M"], a["qlen"], a["hq"], a["hkv"], a["D"], a["ps"], a["dt"], a["ks"], a["vs"],
        a["sph"], a["msl"], a["mpl"], a["ws"], a["wsb"], a["st"], None)


def test_refusals(lib):
    assert _call(lib) == ECUDA                            # valid, but no GPU here
    assert _call(lib, B=0) == OK
    assert _call(lib, B=-1) == EINVAL
    assert _call(lib, B=3000) == ERANGE
    assert _call(lib, D=64) == EUNSUPPORTED
    assert _call(lib, ps=32) == EUNSUPPORTED
    assert _call(lib, hq=30) == EINVAL
    assert _call(lib, qlen=9) == ERANGE
    assert _call(lib, qlen=0) == EINVAL
    assert _call(lib, hq=36, hkv=4, qlen=4) == EUNSUPPORTED   # 36 rows > 32
    assert _call(lib, dt=4) == EINVAL
    assert _call(lib, ks=None) == EINVAL
    assert _call(lib, dt=0, ks=None, vs=None) == ECUDA
    assert _call(lib, dt=3, ks=None, vs=None) == ECUDA
    assert _call(lib, npages=0) == EINVAL
    assert _call(lib, npages=1 << 31) == EINVAL
    assert _call(lib, W=0) == EINVAL
    assert _call(lib, W=32770) == ERANGE
    assert _call(lib, M=0) == EINVAL
    assert _call(lib, M=2049) == ERANGE
    assert _call(lib, msl=-1) == EINVAL
    assert _call(lib, mpl=-1) == EINVAL
    for name, step in [("q", 8), ("out", 8), ("pages", 8), ("bt", 2), ("sl", 2), ("go", 2), ("pl", 2)]:
        assert _call(lib, **{name: None}) == EINVAL, name
        assert _call(lib, **{name: P + step}) == EINVAL, name


def test_workspace(lib):
    need = pq.shared_prefix_workspace_size(2, 1, 5, 32, 8)
    assert need > 0
    assert _call(lib, ws=None) == EWORKSPACE
    assert _call(lib, ws=P + 128) == EWORKSPACE
    assert _call(lib, wsb=need - 1) == EWORKSPACE
    assert _call(lib, wsb=need) == ECUDA
    size = pq.shared_prefix_workspace_size
    assert size(0, 1, 5, 32, 8) == size(2, 0, 5, 32, 8) == size(2, 2049, 5, 32, 8) == 0
    assert size(2, 1, 9, 32, 8) == size(2, 1, 5, 30, 8) == size(3000, 1, 1, 32, 8) == 0
    assert size(2048, 2048, 8, 32, 8) > size(2048, 1, 8, 32, 8) >= size(64, 1, 8, 32, 8)
