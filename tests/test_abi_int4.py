"""The 4-bit format and kv_read at the C entries, without a GPU."""
import re

import pytest

import paged_quantized_kv_append_gb300 as pq
import workloads as W
from tests.test_abi import (ECUDA, EINVAL, ERANGE, EUNSUPPORTED, OK, _append, _attn, _attn_window,
                            _header_text, lib)  # noqa: F401
from tests.test_abi_shared_prefix import _call as _shared

F = 5


def test_header_binding_and_workloads_agree():
    assert re.search(r"\bPQKV_KV_INT4_GROUP = 5\b", _header_text())
    assert pq.INT4_GROUP == W.INT4_GROUP == pq.KV_DTYPES["int4_group"] == F
    w = W.Workload("x", 1, [10], 8, 2, 1, F)
    assert w.kv_bytes() == 10 * 2 * 144


def test_format_numbers(lib):  # noqa: F811
    for dt in (4, 6, -1):
        assert _append(lib, dt=dt) == EINVAL and _attn(lib, dt=dt) == EINVAL
        assert _read(lib, dt=dt) == EINVAL
    # valid, but no GPU here; no scales needed
    assert _append(lib, dt=F, kscale=None, vscale=None) == ECUDA
    assert _attn(lib, dt=F, kscale=None, vscale=None) == ECUDA
    assert _attn_window(lib, 16, dt=F, kscale=None, vscale=None) == ECUDA
    assert _shared(lib, dt=F, ks=None, vs=None) == ECUDA
    assert _shared(lib, dt=6) == _shared(lib, dt=F, npages=0) == EINVAL
    assert _shared(lib, dt=F, ps=32) == EUNSUPPORTED


def _read(lib, **kw):  # noqa: F811
    a = dict(pages=1 << 12, n=10, bt=1 << 12, mpps=8, first=1 << 12, off=1 << 12, B=2, T=20, H=8,
             D=128, P=16, dt=1, ks=1 << 12, vs=1 << 12, sph=0, k=1 << 12, kst=1024, v=1 << 12,
             vst=1024, status=None)
    a.update(kw)
    return lib.pqkv_kv_read(a["pages"], a["n"], a["bt"], a["mpps"], a["first"], a["off"], a["B"],
                            a["T"], a["H"], a["D"], a["P"], a["dt"], a["ks"], a["vs"], a["sph"],
                            a["k"], a["kst"], a["v"], a["vst"], a["status"], None)


@pytest.mark.parametrize("kw,want", [
    ({}, ECUDA), ({"first": None}, ECUDA), ({"dt": F, "ks": None, "vs": None}, ECUDA),
    ({"dt": 3, "ks": None, "vs": None}, ECUDA), ({"B": 0}, OK), ({"T": 0}, OK),
    ({"B": -1}, EINVAL), ({"T": -1}, EINVAL), ({"B": 2049}, ERANGE), ({"D": 64}, EUNSUPPORTED),
    ({"P": 32}, EUNSUPPORTED), ({"H": 0}, EINVAL), ({"ks": None}, EINVAL), ({"pages": None}, EINVAL),
    ({"bt": None}, EINVAL), ({"off": None}, EINVAL), ({"k": None}, EINVAL), ({"v": None}, EINVAL),
    ({"n": 0}, EINVAL), ({"mpps": 0}, EINVAL), ({"mpps": 40000}, ERANGE), ({"kst": 1008}, EINVAL),
    ({"vst": 1032}, EINVAL), ({"k": (1 << 12) + 16}, EINVAL), ({"pages": (1 << 12) + 8}, EINVAL),
    ({"first": (1 << 12) + 2}, EINVAL), ({"status": (1 << 12) + 2}, EINVAL)])
def test_kv_read_validation(lib, kw, want):  # noqa: F811
    assert _read(lib, **kw) == want
