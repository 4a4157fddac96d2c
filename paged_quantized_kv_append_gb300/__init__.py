"""Paged quantized-KV append and paged decode / verify attention on GB300.

A thin ctypes binding of libpqkv.so (include/pqkv.h): it checks tensor
dtypes and shapes, passes device pointers and the current CUDA stream, and
raises on a non-zero return code.  Every step of the computation runs in the
library's CUDA kernels; there is no fallback path.

    kv_append_quant(k, v, slot_mapping, kv_dtype, k_scale, v_scale, pages)
    paged_attention(q, pages, block_table, seq_lens, q_len, kv_dtype,
                    k_scale, v_scale, out)

Pool layout: ``pages`` is [num_pages, num_kv_heads, 2, 16, 128] -- for each
page and kv-head a 16-token K tile followed by a V tile -- of uint8 codes
(E4M3 / INT8) or float16 values.  A 4-bit pool ("int4_group") is uint8
[num_pages, num_kv_heads, 2, 16, 72]: 64 bytes of codes and 8 of scales a row.

    kv_read(pages, block_table, first_pos, token_offsets, kv_dtype, k_scale, v_scale, k, v)
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import os
import threading

import torch

FP16 = 0
FP8_E4M3 = 1
INT8 = 2
INT8_ROW = 3          # int8 with a scale per (token, kv-head) row, computed at append time
INT4_GROUP = 5        # 4-bit codes with a scale per group of 32 values, computed at append time
KV_DTYPES = {"fp16": FP16, "fp8_e4m3": FP8_E4M3, "int8": INT8, "int8_row": INT8_ROW,
             "int4_group": INT4_GROUP}
_SCALED = (FP8_E4M3, INT8)   # formats that take k_scale / v_scale arguments

HEAD_DIM = 128
PAGE_SIZE = 16
INT4_ROW_BYTES = 72   # of a row's codes and scales in a 4-bit pool

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libpqkv.so")

_status_names = {1: "slot beyond the pool", 2: "seq_len out of range", 4: "bad scale",
                 8: "pipeline wait timed out", 16: "block-table page id out of range"}


class PqkvError(RuntimeError):
    pass


_lib = None
_lib_lock = threading.Lock()


def load_library(path: str | None = None):
    """Load libpqkv.so (built in-tree by ``python -m paged_quantized_kv_append_gb300.build``)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lib_lock:
        if _lib is not None:
            return _lib
        path = path or LIB_PATH
        if not os.path.exists(path):
            raise PqkvError("libpqkv.so is not built (expected at %s); run "
                            "`python -m paged_quantized_kv_append_gb300.build`" % path)
        lib = ctypes.CDLL(path)
        c_i32, c_i64, c_vp, c_sz = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t
        lib.pqkv_kv_append_quant.restype = ctypes.c_int
        lib.pqkv_kv_append_quant.argtypes = [c_vp, c_i64, c_vp, c_i64, c_vp, c_i32, c_i32, c_i32,
                                             c_i32, c_vp, c_vp, c_i32, c_vp, c_i64, c_i32, c_vp,
                                             c_vp]
        lib.pqkv_kv_read.restype = ctypes.c_int
        lib.pqkv_kv_read.argtypes = [c_vp, c_i64, c_vp, c_i32, c_vp, c_vp, c_i32, c_i32, c_i32,
                                     c_i32, c_i32, c_i32, c_vp, c_vp, c_i32, c_vp, c_i64, c_vp,
                                     c_i64, c_vp, c_vp]
        lib.pqkv_paged_attention_workspace_size.restype = c_sz
        lib.pqkv_paged_attention_workspace_size.argtypes = [c_i32] * 6
        lib.pqkv_paged_attention.restype = ctypes.c_int
        lib.pqkv_paged_attention.argtypes = [c_vp, c_vp, c_vp, c_i64, c_vp, c_i32, c_vp, c_i32,
                                             c_i32, c_i32, c_i32, c_i32, c_i32, c_i32, c_vp, c_vp,
                                             c_i32, c_i32, c_i32, c_vp, c_sz, c_vp, c_vp]
        lib.pqkv_paged_attention_window.restype = ctypes.c_int
        lib.pqkv_paged_attention_window.argtypes = [c_vp, c_vp, c_vp, c_i64, c_vp, c_i32, c_vp,
                                                    c_i32, c_i32, c_i32, c_i32, c_i32, c_i32,
                                                    c_i32, c_vp, c_vp, c_i32, c_i32, c_i32, c_i32,
                                                    c_vp, c_sz, c_vp, c_vp]
        lib.pqkv_paged_attention_noalloc.restype = ctypes.c_int
        lib.pqkv_paged_attention_noalloc.argtypes = [c_vp, c_vp, c_vp, c_i64, c_vp, c_i32, c_vp,
                                                     c_i32, c_i32, c_i32, c_i32, c_i32, c_i32,
                                                     c_i32, c_vp, c_vp, c_i32, c_i32, c_i32, c_vp,
                                                     c_vp]
        lib.pqkv_paged_attention_partial.restype = ctypes.c_int
        lib.pqkv_paged_attention_partial.argtypes = [c_vp, c_vp, c_i64, c_vp, c_i32, c_vp, c_vp,
                                                     c_i32, c_i32, c_i32, c_i32, c_i32, c_i32,
                                                     c_i32, c_vp, c_vp, c_i32, c_i32, c_i32, c_vp,
                                                     c_vp, c_vp, c_sz, c_vp, c_vp]
        lib.pqkv_lse_merge.restype = ctypes.c_int
        lib.pqkv_lse_merge.argtypes = [c_vp, c_vp, c_i32, c_i64, c_i32, c_vp, c_vp, c_vp]
        lib.pqkv_paged_attention_shared_prefix_workspace_size.restype = c_sz
        lib.pqkv_paged_attention_shared_prefix_workspace_size.argtypes = [c_i32] * 6
        lib.pqkv_paged_attention_shared_prefix.restype = ctypes.c_int
        lib.pqkv_paged_attention_shared_prefix.argtypes = [
            c_vp, c_vp, c_vp, c_i64, c_vp, c_i32, c_vp, c_i32, c_vp, c_vp, c_i32, c_i32, c_i32,
            c_i32, c_i32, c_i32, c_i32, c_vp, c_vp, c_i32, c_i32, c_i32, c_vp, c_sz, c_vp, c_vp]
        lib.pqkv_extend_block_tables.restype = ctypes.c_int
        lib.pqkv_extend_block_tables.argtypes = [c_vp, c_vp, c_i32, c_vp, c_i32, c_vp, c_vp, c_i32,
                                                 c_i64, c_i32, c_vp, c_vp, c_vp, c_vp, c_i32, c_vp,
                                                 c_vp, c_vp]
        lib.pqkv_truncate_block_tables.restype = ctypes.c_int
        lib.pqkv_truncate_block_tables.argtypes = [c_vp, c_vp, c_vp, c_i32, c_vp, c_i32, c_vp,
                                                   c_vp, c_i32, c_i32, c_vp, c_vp, c_vp, c_vp]
        lib.pqkv_status_string.restype = ctypes.c_char_p
        lib.pqkv_status_string.argtypes = [ctypes.c_int]
        lib.pqkv_version.restype = ctypes.c_char_p
        lib.pqkv_version.argtypes = []
        _lib = lib
        return lib


def _check(rc: int, what: str):
    if rc != 0:
        msg = load_library().pqkv_status_string(rc).decode()
        if rc in (-1, -2, -3):
            raise ValueError("%s: %s (code %d)" % (what, msg, rc))
        raise PqkvError("%s: %s (code %d)" % (what, msg, rc))


def _stream(t: torch.Tensor, stream):
    if stream is None:
        stream = torch.cuda.current_stream(t.device)
    return ctypes.c_void_p(stream.cuda_stream)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def _on_device(dev, **tensors):
    """Every tensor the kernels read or write must live on the pool's GPU: a
    host or other-device pointer would be dereferenced on the device."""
    for name, x in tensors.items():
        if x is not None and (not x.is_cuda or x.device != dev):
            raise ValueError("%s must be a CUDA tensor on %s, got %s" % (name, dev, x.device))


def _check_status(status, dev):
    if status is not None:
        _on_device(dev, status=status)
        if status.dtype != torch.int32 or status.numel() < 1:
            raise ValueError("status must be an int32 CUDA tensor of at least one element")


def _dtype_id(kv_dtype) -> int:
    if isinstance(kv_dtype, str):
        return KV_DTYPES[kv_dtype]
    return int(kv_dtype)


def _row_scale_bytes(num_pages, num_kv_heads):
    return num_pages * num_kv_heads * 2 * PAGE_SIZE * 2          # fp16 scales


def _row_elems(kd):
    return INT4_ROW_BYTES if kd == INT4_GROUP else HEAD_DIM


def new_pages(num_pages: int, num_kv_heads: int, kv_dtype, device="cuda", fill=None):
    """Allocate a pool [num_pages, num_kv_heads, 2, 16, 128] for ``kv_dtype``.

    An INT8_ROW pool is the code tensor followed, in the same allocation, by
    its row-scale area (zeroed); ``row_scales(pages)`` views that area.  An
    INT4_GROUP pool's rows are 72 bytes, scales among them: [..., 16, 72].
    """
    kd = _dtype_id(kv_dtype)
    dt = torch.float16 if kd == FP16 else torch.uint8
    shape = (num_pages, num_kv_heads, 2, PAGE_SIZE, _row_elems(kd))
    if kd == INT8_ROW:
        codes = num_pages * num_kv_heads * 2 * PAGE_SIZE * HEAD_DIM
        buf = torch.zeros(codes + _row_scale_bytes(num_pages, num_kv_heads), dtype=torch.uint8,
                          device=device)
        if fill is not None:
            buf[:codes].fill_(fill)
        return buf[:codes].view(shape)
    if fill is None:
        return torch.empty(shape, dtype=dt, device=device)
    return torch.full(shape, fill, dtype=dt, device=device)


def row_scales(pages: torch.Tensor) -> torch.Tensor:
    """float16 view [num_pages, Hkv, 2, 2, 8] of an INT8_ROW pool's row scales:
    ``[p, h, kv, r // 8, r % 8]`` is the scale of row r (slot 16 p + r) of K
    (kv 0) or V (kv 1).  The area stores them as [p][h][r % 8][kv][r // 8];
    ``.reshape(n, Hkv, 2, 16)`` gives a row-ordered copy."""
    _check_pages(pages, INT8_ROW)
    n, H = pages.shape[0], pages.shape[1]
    codes = pages.numel()
    whole = torch.empty(0, dtype=torch.uint8, device=pages.device)
    whole.set_(pages.untyped_storage(), pages.storage_offset(),
               (codes + _row_scale_bytes(n, H),))
    return _row_scale_view(whole[codes:], n, H)


def _row_scale_view(area: torch.Tensor, num_pages: int, num_kv_heads: int) -> torch.Tensor:
    """[p, h, kv, r // 8, r % 8] view of a scale area (uint8 bytes) stored as
    fp16 [p][h][i][4] = (K row i, K row i+8, V row i, V row i+8)."""
    return area.view(torch.float16).view(num_pages, num_kv_heads, 8, 2, 2).permute(0, 1, 3, 4, 2)


def _check_pages(pages, kd):
    want = torch.float16 if kd == FP16 else torch.uint8
    n, shape = _row_elems(kd), pages.shape
    if pages.dtype is not want or len(shape) != 5 or shape[2] != 2 or shape[3] != PAGE_SIZE \
            or shape[4] != n:
        raise ValueError("pages must be %s [num_pages, Hkv, 2, 16, %d], got %s %s"
                         % (want, n, pages.dtype, tuple(pages.shape)))
    if not pages.is_contiguous() or not pages.is_cuda:
        raise ValueError("pages must be a contiguous CUDA tensor")
    if kd == INT8_ROW:
        room = pages.untyped_storage().nbytes() - pages.storage_offset()
        if room < pages.numel() + _row_scale_bytes(pages.shape[0], pages.shape[1]):
            raise ValueError("an int8_row pool needs its row-scale area after the codes "
                             "(allocate it with new_pages)")


def _check_scale(x, H, name):
    if x.dtype != torch.float32 or not x.is_cuda or x.numel() not in (1, H) \
            or not x.is_contiguous():
        raise ValueError("%s must be a contiguous float32 CUDA tensor of 1 or num_kv_heads elements"
                         % name)
    return 1 if (x.numel() == H and H > 1) else 0


def kv_append_quant(k, v, slot_mapping, kv_dtype, k_scale, v_scale, pages, status=None,
                    stream=None):
    """Quantize k, v ([T, Hkv, 128] fp16, token rows may be strided) into their
    ``slot_mapping`` slots (int64 [T], negative = skip) of ``pages``."""
    kd = _dtype_id(kv_dtype)
    _check_pages(pages, kd)
    N, H = pages.shape[:2]
    idx, shape = pages.get_device(), k.shape
    ks, vs, scaled, sph = k.stride(), v.stride(), kd in _SCALED, 0
    # (one expression for what the checks below say one by one: the host's time is the
    # call's where tokens are few)
    if scaled or not (
            k.dtype is torch.float16 and v.dtype is torch.float16 and len(shape) == 3
            and shape[1] == H and shape[2] == HEAD_DIM and v.shape == shape
            and ks[1] == HEAD_DIM and ks[2] == 1 and vs[1] == HEAD_DIM and vs[2] == 1
            and slot_mapping.dtype is torch.int64 and slot_mapping.shape == shape[:1]
            and slot_mapping.is_contiguous() and k.get_device() == idx
            and v.get_device() == idx and slot_mapping.get_device() == idx):
        sph = _check_tokens(k, v, slot_mapping, kd, k_scale, v_scale, pages, H)
    if status is not None:
        _check_status(status, pages.device)
    rc = _call_on(
        idx, stream, load_library().pqkv_kv_append_quant, k.data_ptr(), ks[0], v.data_ptr(), vs[0],
        slot_mapping.data_ptr(), shape[0], H, HEAD_DIM, kd,
        k_scale.data_ptr() if scaled else None, v_scale.data_ptr() if scaled else None, sph,
        pages.data_ptr(), N, PAGE_SIZE, None if status is None else status.data_ptr())
    if rc:
        _check(rc, "kv_append_quant")
    return pages


def _check_tokens(k, v, slot_mapping, kd, k_scale, v_scale, pages, H):
    """kv_append_quant's arguments; returns its scale_per_head."""
    for name, x in (("k", k), ("v", v)):
        if x.dtype != torch.float16 or x.dim() != 3 or x.shape[1:] != (H, HEAD_DIM):
            raise ValueError("%s must be fp16 [T, %d, 128], got %s %s" % (name, H, x.dtype, tuple(x.shape)))
        if x.stride(2) != 1 or x.stride(1) != HEAD_DIM or not x.is_cuda:
            raise ValueError("%s: heads and dims must be contiguous on the GPU" % name)
    T = k.shape[0]
    if v.shape[0] != T or slot_mapping.dtype != torch.int64 or slot_mapping.shape != (T,) \
            or not slot_mapping.is_contiguous():
        raise ValueError("v / slot_mapping (contiguous int64) do not match k's token count")
    sph = 0
    if kd in _SCALED:
        sph = _check_scale(k_scale, H, "k_scale")
        if _check_scale(v_scale, H, "v_scale") != sph:
            raise ValueError("k_scale and v_scale must have the same shape")
    dev = pages.device
    _on_device(dev, k=k, v=v, slot_mapping=slot_mapping, k_scale=k_scale if kd in _SCALED else None,
               v_scale=v_scale if kd in _SCALED else None)
    return sph


def kv_read(pages, block_table, first_pos, token_offsets, kv_dtype, k_scale, v_scale, k, v,
            status=None, stream=None):
    """The inverse of kv_append_quant for whole requests: rows
    ``token_offsets[s]`` .. ``token_offsets[s + 1] - 1`` (int32 [B + 1], from 0)
    of ``k`` and ``v`` ([T, Hkv, 128] fp16, token rows may be strided) receive the
    values of request s's tokens from position ``first_pos[s]`` on (int32 [B];
    None: 0), found through ``block_table`` (int32 [B, max_pages_per_seq]).  Rows
    behind the last request's are left as they are.  Returns (k, v)."""
    kd = _dtype_id(kv_dtype)
    _check_pages(pages, kd)
    idx, (N, H) = pages.get_device(), pages.shape[:2]
    table, T = block_table.shape, _size(k)
    B, W = table if len(table) == 2 else (-1, -1)
    if block_table.dtype is not torch.int32 or B < 0 or not block_table.is_contiguous() \
            or block_table.get_device() != idx:
        _refuse("block_table", block_table, torch.int32, (B, W), idx)
    if token_offsets.dtype is not torch.int32 or token_offsets.shape != (B + 1,) \
            or not token_offsets.is_contiguous() or token_offsets.get_device() != idx:
        _refuse("token_offsets", token_offsets, torch.int32, (B + 1,), idx)
    if first_pos is not None and (
            first_pos.dtype is not torch.int32 or first_pos.shape != (B,)
            or not first_pos.is_contiguous() or first_pos.get_device() != idx):
        _refuse("first_pos", first_pos, torch.int32, (B,), idx)
    shape, step = (T, H, HEAD_DIM), []
    for name, x in (("k", k), ("v", v)):
        st = x.stride()
        if x.dtype is not torch.float16 or x.shape != shape or x.get_device() != idx \
                or st[2] != 1 or (H > 1 and st[1] != HEAD_DIM):
            raise ValueError("%s must be fp16 [T, %d, 128] on cuda:%d with contiguous heads and "
                             "dims, got %s %s (strides %s) on %s" % (
                                 name, H, idx, x.dtype, list(x.shape), list(st), x.device))
        step.append(st[0])
    sph, ks, vs = 0, None, None
    if kd in _SCALED:
        sph = _check_scale(k_scale, H, "k_scale")
        if _check_scale(v_scale, H, "v_scale") != sph:
            raise ValueError("k_scale and v_scale must have the same shape")
        if k_scale.get_device() != idx or v_scale.get_device() != idx:
            raise ValueError("k_scale and v_scale must be on cuda:%d" % idx)
        ks, vs = k_scale.data_ptr(), v_scale.data_ptr()
    if status is not None:
        _check_status(status, pages.device)
    rc = _call_on(
        idx, stream, load_library().pqkv_kv_read, pages.data_ptr(), N, block_table.data_ptr(), W,
        None if first_pos is None else first_pos.data_ptr(), token_offsets.data_ptr(), B, T, H,
        HEAD_DIM, PAGE_SIZE, kd, ks, vs, sph, k.data_ptr(), step[0], v.data_ptr(), step[1],
        None if status is None else status.data_ptr())
    if rc:
        _check(rc, "kv_read")
    return k, v


@functools.lru_cache(maxsize=256)
def workspace_size(num_seqs, q_len, num_q_heads, num_kv_heads, num_splits=0) -> int:
    return int(load_library().pqkv_paged_attention_workspace_size(
        num_seqs, q_len, num_q_heads, num_kv_heads, HEAD_DIM, num_splits))


class Workspace:
    """Zero-initialised device scratch for paged_attention, grown on demand.

    The kernels leave the merge counters at a call's start zeroed again after
    every call, so one workspace serves any number of calls, and graphs that captured calls,
    which run one after another; calls that may overlap on the GPU need one each.  How
    many counters there are depends on the call's num_seqs and num_kv_heads; the
    counters of every call end at the same byte, ``head``, so that none has its
    counters where another has had its partial results.

    A buffer is allocated and zeroed on the stream of the call that needs it.  One that
    has become too small is kept, for the kernels and graphs that still use it, and the next
    is at least twice as large, so that all of the old ones together are smaller."""

    def __init__(self, device="cuda"):
        self.device = torch.device(device)
        self.head = 1 << 18
        self.buf = None
        self._parts = {}
        self._old = []
        self._lock = threading.Lock()

    def get(self, nbytes: int, counter_bytes: int = 0, stream=None):
        """``nbytes`` of scratch, the first ``counter_bytes`` of them counters, for a call on
        ``stream`` (None: the device's current one)."""
        if nbytes == 0:
            return None
        counters = -(-counter_bytes // 256) * 256
        part = self._parts.get(counters)     # (a slice costs a call more than a microsecond)
        if part is not None and part.numel() >= nbytes:
            return part
        with self._lock:
            head, buf = self.head, self.buf
            while head < counters:
                head, buf = 2 * head, None
            need = head - counters + nbytes
            if buf is None or buf.numel() < need:
                if self.device.type == "cuda" and _capturing(self.device.index, stream):
                    return _captured_scratch(self.device, nbytes, counters, stream)
                if self.buf is not None:
                    self._old.append(self.buf)
                    need = max(need, 2 * self.buf.numel())
                with _stream_of(self.device, stream):
                    buf = torch.zeros(max(need, 1 << 20), dtype=torch.uint8, device=self.device)
                self.head, self.buf, self._parts = head, buf, {}
            part = self._parts[counters] = buf[head - counters:]
            return part


def _stream_of(device, stream):
    """The context in which tensors are made on ``stream`` (None: the device's current one)."""
    if stream is not None:
        return torch.cuda.stream(stream)
    return torch.cuda.device(device) if device.type == "cuda" else contextlib.nullcontext()


def _capturing(idx, stream):
    """Whether ``stream`` (None: the current one of cuda:idx) is being captured.  (torch asks the
    current stream alone; its context managers would cost a call 8 microseconds.)"""
    dev = torch._C._cuda_getDevice()
    if stream is None:
        if idx is None or idx == dev:
            return torch._C._cuda_isCurrentStreamCapturing()
        with torch.cuda.device(idx):
            return torch._C._cuda_isCurrentStreamCapturing()
    if stream.device_index != dev:
        with torch.cuda.stream(stream):
            return torch._C._cuda_isCurrentStreamCapturing()
    was = torch._C._cuda_getCurrentStream(dev)
    if was[0] == stream.stream_id:
        return torch._C._cuda_isCurrentStreamCapturing()
    set_stream = torch._C._cuda_setStream
    try:
        set_stream(stream_id=stream.stream_id, device_index=dev, device_type=stream.device_type)
        return torch._C._cuda_isCurrentStreamCapturing()
    finally:
        set_stream(stream_id=was[0], device_index=was[1], device_type=was[2])


def _captured_scratch(device, nbytes, counters, stream):
    """Scratch of one captured call: memory of its graph, whose counters every replay zeroes.
    (What is allocated and zeroed under a capture is neither there nor zero for another graph or
    for an eager call.)"""
    with _stream_of(device, stream):
        buf = torch.empty(nbytes, dtype=torch.uint8, device=device)
        buf[:counters].zero_()
    return buf


def _what(x):
    if not isinstance(x, torch.Tensor):
        return type(x).__name__
    return "%s of strides %s on %s" % (list(x.shape), list(x.stride()), x.device)


def _scratch(workspace, idx, stream, need, counter_bytes=0):
    """Address and bytes of a call's workspace on cuda:idx: a Workspace's part, or a tensor."""
    if isinstance(workspace, Workspace):
        workspace = workspace.get(need, counter_bytes, stream)
        if workspace is None:
            return None, 0
    if not isinstance(workspace, torch.Tensor) or workspace.get_device() != idx \
            or not workspace.is_contiguous():
        raise ValueError("workspace must be a Workspace or a contiguous CUDA tensor on cuda:%d, "
                         "got %s" % (idx, _what(workspace)))
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


_default_ws = {}


def _default_scratch(idx, stream, need, counter_bytes):
    """_scratch of a call that was given no workspace: one per stream, whose calls run one after
    another; a captured call's own, as its graph may be replayed beside any other."""
    if not need:
        return None, 0
    if _capturing(idx, stream):
        part = _captured_scratch(torch.device("cuda", idx), need, -(-counter_bytes // 256) * 256,
                                 stream)
    else:
        raw = torch._C._cuda_getCurrentRawStream(idx) if stream is None else stream.cuda_stream
        ws = _default_ws.get((idx, raw))
        if ws is None:
            ws = _default_ws.setdefault((idx, raw), Workspace(torch.device("cuda", idx)))
        part = ws.get(need, counter_bytes, stream)
    return part.data_ptr(), part.numel()


def paged_attention(q, pages, block_table, seq_lens, q_len, kv_dtype, k_scale, v_scale, out,
                    num_splits=0, max_seq_len=0, workspace=None, status=None, stream=None,
                    window=0):
    """Decode (q_len 1) or verify (q_len > 1) attention over the paged pool.

    q, out: fp16 [num_seqs * q_len, Hq, 128]; block_table: int32
    [num_seqs, max_pages_per_seq]; seq_lens: int32 [num_seqs] (cached tokens,
    the q_len new ones included).  num_splits 0 balances key pages over the
    GPU; k >= 1 cuts each (sequence, kv-head) into k partitions.  window > 0:
    query position p sees only keys p - window + 1 .. p (sliding window).

    workspace: a Workspace, or a zeroed tensor of workspace_size() bytes, that no other call
    uses at the same time.  None: one that is kept for the stream, or, in a capture by
    torch.cuda.graph, memory of that graph; under another kind of capture, and where calls go on
    after a reported timeout (which leaves the workspace to be zeroed), give one.
    """
    kd = _dtype_id(kv_dtype)
    _check_pages(pages, kd)
    N, H = pages.shape[:2]
    idx, rows, table, B = pages.get_device(), q.shape, block_table.shape, seq_lens.shape[0]
    scaled, sph = kd in _SCALED, 0
    # (one expression, as in kv_append_quant)
    if scaled or not (
            q.dtype is torch.float16 and out.dtype is torch.float16 and len(rows) == 3
            and rows[2] == HEAD_DIM and out.shape == rows and rows[0] == B * q_len
            and q.is_contiguous() and out.is_contiguous() and seq_lens.dtype is torch.int32
            and seq_lens.dim() == 1 and seq_lens.is_contiguous()
            and block_table.dtype is torch.int32 and len(table) == 2 and table[0] == B
            and block_table.is_contiguous() and q.get_device() == idx and out.get_device() == idx
            and seq_lens.get_device() == idx and block_table.get_device() == idx):
        sph = _check_attention(q, pages, block_table, seq_lens, q_len, kd, k_scale, v_scale, out,
                               H, B)
    Hq = rows[1]
    if status is not None:
        _check_status(status, pages.device)
    if window < 0:
        raise ValueError("window must be >= 0")
    need = workspace_size(B, q_len, Hq, H, num_splits)
    if workspace is None:
        ws, ws_bytes = _default_scratch(idx, stream, need, 4 * B * H)
    else:
        ws, ws_bytes = _scratch(workspace, idx, stream, need, 4 * B * H)
    lib = load_library()
    args = [q.data_ptr(), out.data_ptr(), pages.data_ptr(), N, block_table.data_ptr(),
            table[1], seq_lens.data_ptr(), B, q_len, Hq, H, HEAD_DIM, PAGE_SIZE, kd,
            k_scale.data_ptr() if scaled else None, v_scale.data_ptr() if scaled else None, sph,
            num_splits, max_seq_len]
    fn = lib.pqkv_paged_attention
    if window > 0:
        fn = lib.pqkv_paged_attention_window
        args.append(window)
    rc = _call_on(idx, stream, fn, *args, ws, ws_bytes, None if status is None else status.data_ptr())
    if rc:
        _check(rc, "paged_attention")
    return out


def _check_attention(q, pages, block_table, seq_lens, q_len, kd, k_scale, v_scale, out, H, B):
    """paged_attention's arguments; returns its scale_per_head."""
    if q.dtype != torch.float16 or q.dim() != 3 or q.shape[2] != HEAD_DIM or not q.is_contiguous():
        raise ValueError("q must be contiguous fp16 [num_seqs*q_len, Hq, 128]")
    if out.shape != q.shape or out.dtype != torch.float16 or not out.is_contiguous():
        raise ValueError("out must be contiguous fp16 shaped like q")
    if seq_lens.dtype != torch.int32 or seq_lens.dim() != 1 or not seq_lens.is_contiguous():
        raise ValueError("seq_lens must be contiguous int32 [num_seqs]")
    if block_table.dtype != torch.int32 or block_table.dim() != 2 or block_table.shape[0] != B \
            or not block_table.is_contiguous():
        raise ValueError("block_table must be contiguous int32 [num_seqs, max_pages_per_seq]")
    if q.shape[0] != B * q_len:
        raise ValueError("q has %d rows, expected num_seqs*q_len = %d" % (q.shape[0], B * q_len))
    sph = 0
    if kd in _SCALED:
        sph = _check_scale(k_scale, H, "k_scale")
        if _check_scale(v_scale, H, "v_scale") != sph:
            raise ValueError("k_scale and v_scale must have the same shape")
    _on_device(pages.device, q=q, out=out, block_table=block_table, seq_lens=seq_lens,
               k_scale=k_scale if kd in _SCALED else None,
               v_scale=v_scale if kd in _SCALED else None)
    return sph


def paged_attention_partial(q, pages, block_table, seq_lens, q_pos, q_len, kv_dtype, k_scale,
                            v_scale, out_o, out_lse, num_splits=0, max_seq_len=0, workspace=None,
                            status=None, stream=None):
    """One rank's share of a decode-context-parallel split: attention over the
    keys held here (``seq_lens`` of them per sequence, possibly 0), query i of
    sequence s seeing local keys j <= q_pos[s] + i.  Writes O / l into
    ``out_o`` (fp32, shaped like q) and the natural-log LSE into ``out_lse``
    (fp32 [num_seqs * q_len, Hq]); merge the ranks' results with lse_merge."""
    kd = _dtype_id(kv_dtype)
    _check_pages(pages, kd)
    H = pages.shape[1]
    if q.dtype != torch.float16 or q.dim() != 3 or q.shape[2] != HEAD_DIM or not q.is_contiguous():
        raise ValueError("q must be contiguous fp16 [num_seqs*q_len, Hq, 128]")
    if out_o.shape != q.shape or out_o.dtype != torch.float32 or not out_o.is_contiguous():
        raise ValueError("out_o must be contiguous fp32 shaped like q")
    if out_lse.shape != q.shape[:2] or out_lse.dtype != torch.float32 or not out_lse.is_contiguous():
        raise ValueError("out_lse must be contiguous fp32 [num_seqs*q_len, Hq]")
    B = seq_lens.shape[0]
    for name, x in (("seq_lens", seq_lens), ("q_pos", q_pos)):
        if x.dtype != torch.int32 or x.shape != (B,) or not x.is_contiguous():
            raise ValueError("%s must be contiguous int32 [num_seqs]" % name)
    if block_table.dtype != torch.int32 or block_table.dim() != 2 or block_table.shape[0] != B \
            or not block_table.is_contiguous():
        raise ValueError("block_table must be contiguous int32 [num_seqs, max_pages_per_seq]")
    if q.shape[0] != B * q_len:
        raise ValueError("q has %d rows, expected num_seqs*q_len = %d" % (q.shape[0], B * q_len))
    Hq = q.shape[1]
    sph = 0
    if kd in _SCALED:
        sph = _check_scale(k_scale, H, "k_scale")
        if _check_scale(v_scale, H, "v_scale") != sph:
            raise ValueError("k_scale and v_scale must have the same shape")
    dev = pages.device
    _on_device(dev, q=q, out_o=out_o, out_lse=out_lse, block_table=block_table,
               seq_lens=seq_lens, q_pos=q_pos, k_scale=k_scale if kd in _SCALED else None,
               v_scale=v_scale if kd in _SCALED else None)
    _check_status(status, dev)
    need = workspace_size(B, q_len, Hq, H, num_splits)
    if workspace is None:
        ws, ws_bytes = _default_scratch(dev.index, stream, need, 4 * B * H)
    else:
        ws, ws_bytes = _scratch(workspace, dev.index, stream, need, 4 * B * H)
    lib = load_library()
    with torch.cuda.device(dev):
        rc = lib.pqkv_paged_attention_partial(
            _ptr(q), _ptr(pages), pages.shape[0], _ptr(block_table), block_table.shape[1],
            _ptr(seq_lens), _ptr(q_pos), B, q_len, Hq, H, HEAD_DIM, PAGE_SIZE, kd,
            _ptr(k_scale if kd in _SCALED else None), _ptr(v_scale if kd in _SCALED else None),
            sph, num_splits, max_seq_len, _ptr(out_o), _ptr(out_lse), ws, ws_bytes,
            _ptr(status), _stream(q, stream))
    _check(rc, "paged_attention_partial")
    return out_o, out_lse


def lse_merge(parts_o, parts_lse, out, out_lse=None, stream=None):
    """Combine partial results: parts_o fp32 [P, rows..., 128], parts_lse fp32
    [P, rows...] -> out fp16 [rows..., 128] (and the merged LSE if given)."""
    P = parts_o.shape[0]
    rows = parts_lse[0].numel()
    if parts_o.dtype != torch.float32 or not parts_o.is_contiguous() or \
            parts_o.numel() != P * rows * HEAD_DIM:
        raise ValueError("parts_o must be contiguous fp32 [P, rows..., 128]")
    if parts_lse.dtype != torch.float32 or not parts_lse.is_contiguous() or parts_lse.shape[0] != P:
        raise ValueError("parts_lse must be contiguous fp32 [P, rows...]")
    if out.dtype != torch.float16 or not out.is_contiguous() or out.numel() != rows * HEAD_DIM:
        raise ValueError("out must be contiguous fp16 with rows * 128 elements")
    if out_lse is not None and (out_lse.dtype != torch.float32 or out_lse.numel() != rows
                                or not out_lse.is_contiguous()):
        raise ValueError("out_lse must be contiguous fp32 with one value per row")
    dev = out.device
    _on_device(dev, parts_o=parts_o, parts_lse=parts_lse, out=out, out_lse=out_lse)
    lib = load_library()
    with torch.cuda.device(dev):
        rc = lib.pqkv_lse_merge(_ptr(parts_o), _ptr(parts_lse), P, rows, HEAD_DIM, _ptr(out),
                                _ptr(out_lse), _stream(out, stream))
    _check(rc, "lse_merge")
    return out


@functools.lru_cache(maxsize=256)
def shared_prefix_workspace_size(num_seqs, num_groups, q_len, num_q_heads, num_kv_heads) -> int:
    """Bytes of workspace of paged_attention_shared_prefix (0: sizes it refuses)."""
    return int(load_library().pqkv_paged_attention_shared_prefix_workspace_size(
        num_seqs, num_groups, q_len, num_q_heads, num_kv_heads, HEAD_DIM))


def _refuse(name, x, dtype, shape, idx):
    raise ValueError("%s must be a contiguous %s tensor of shape %s on cuda:%d, got %s %s on %s%s" % (
        name, dtype, list(shape), idx, x.dtype, list(x.shape), x.device,
        "" if x.is_contiguous() else ", not contiguous"))


def _check_ints(idx, dtype, named):
    """Every (name, tensor, shape) a contiguous tensor of this dtype on cuda:idx."""
    for name, x, shape in named:
        if (x.dtype is not dtype or x.shape != shape or not x.is_contiguous()
                or x.get_device() != idx):
            _refuse(name, x, dtype, shape, idx)


def _size(x, axis=0):
    """An axis' size, -1 (no tensor's) where there is no such axis."""
    return x.shape[axis] if x.dim() > axis else -1


def _cuda_index(name, x):
    """The device index of a CUDA tensor (the host's cost per call counts: a
    step's bookkeeping is a few microseconds of GPU time)."""
    idx = x.get_device()
    if idx < 0:
        raise ValueError("%s must be a CUDA tensor, got %s" % (name, x.device))
    return idx


def _call_on(idx, stream, fn, *args):
    """fn(*args, stream) with device idx current."""
    if stream is None:
        raw = torch._C._cuda_getCurrentRawStream(idx)
    else:
        raw = stream.cuda_stream
    if torch._C._cuda_getDevice() == idx:
        return fn(*args, raw)
    with torch.cuda.device(idx):
        return fn(*args, raw)


def paged_attention_shared_prefix(q, pages, block_table, seq_lens, group_offsets, prefix_lens,
                                  q_len, kv_dtype, k_scale, v_scale, out, max_seq_len=0,
                                  max_prefix_len=0, workspace=None, status=None, stream=None):
    """paged_attention of a batch whose sequences share prefixes, each prefix's
    keys read once per 256 query rows (of a kv-head) of the sequences that share
    it.  Decode gains over paged_attention from some 64K tokens saved on
    (sequences times prefix), verification much earlier: include/pqkv.h.

    Sequences ``group_offsets[g]`` .. ``group_offsets[g + 1] - 1`` (int32
    [num_groups + 1]) start with the same ``prefix_lens[g]`` tokens (int32
    [num_groups]) in the same pool pages: their ``block_table`` rows agree over
    the whole pages of that length.  Everything else, and the result, as in
    paged_attention.  ``max_seq_len`` / ``max_prefix_len`` are upper bounds of
    the lengths (0: unknown) that size the launches.  The default
    workspace is taken from the caching allocator for the call; a Workspace, or
    a tensor of shared_prefix_workspace_size() bytes, may be given instead."""
    kd = _dtype_id(kv_dtype)
    _check_pages(pages, kd)
    idx = pages.get_device()
    N, H = pages.shape[0], pages.shape[1]
    B, M, W, Hq = _size(seq_lens), _size(prefix_lens), _size(block_table, 1), _size(q, 1)
    _check_ints(idx, torch.int32, (("seq_lens", seq_lens, (B,)), ("block_table", block_table, (B, W)),
                                   ("prefix_lens", prefix_lens, (M,)),
                                   ("group_offsets", group_offsets, (M + 1,))))
    rows = (B * q_len, Hq, HEAD_DIM)
    _check_ints(idx, torch.float16, (("q", q, rows), ("out", out, rows)))
    sph, ks, vs = 0, None, None
    if kd in _SCALED:
        sph = _check_scale(k_scale, H, "k_scale")
        if _check_scale(v_scale, H, "v_scale") != sph:
            raise ValueError("k_scale and v_scale must have the same shape")
        if k_scale.get_device() != idx or v_scale.get_device() != idx:
            raise ValueError("k_scale and v_scale must be on cuda:%d" % idx)
        ks, vs = k_scale.data_ptr(), v_scale.data_ptr()
    if status is not None:
        _check_status(status, pages.device)
    ws = workspace
    if ws is None:
        need = shared_prefix_workspace_size(B, M, q_len, Hq, H)
        if stream is None:
            ws = torch.empty(need, dtype=torch.uint8, device=pages.device)
        else:                            # owned by the stream it is used on
            with torch.cuda.stream(stream):
                ws = torch.empty(need, dtype=torch.uint8, device=pages.device)
    at, ws_bytes = _scratch(ws, idx, stream, shared_prefix_workspace_size(B, M, q_len, Hq, H))
    rc = _call_on(
        idx, stream, load_library().pqkv_paged_attention_shared_prefix, q.data_ptr(),
        out.data_ptr(), pages.data_ptr(), N, block_table.data_ptr(), W, seq_lens.data_ptr(), B,
        group_offsets.data_ptr(), prefix_lens.data_ptr(), M, q_len, Hq, H, HEAD_DIM, PAGE_SIZE, kd,
        ks, vs, sph, max_seq_len, max_prefix_len, at, ws_bytes,
        None if status is None else status.data_ptr())
    if rc:
        _check(rc, "paged_attention_shared_prefix")
    return out


def extend_block_tables(seq_lens, new_tokens, block_table, free_pages, free_count, num_pages,
                        seq_lens_out, free_count_out, slot_mapping, positions=None,
                        token_offsets=None, status=None, stream=None):
    """Grow every request by ``new_tokens[s]`` tokens (int32 [B]): take pages
    from the top of the stack ``free_pages[:free_count]``, write them into
    ``block_table`` (int32 [B, max_pages_per_seq]), and fill ``slot_mapping``
    (int64 [T]: the tokens of request 0, then of request 1, ..., then -1) for
    kv_append_quant, with each token's position in its request and each
    request's first token if asked for.  ``num_pages`` is the pool's size.

    A request that finds no pages, or whose tokens fit neither its row nor
    ``slot_mapping``, keeps its length, and its tokens get slot -1 (reported in
    ``status``).  ``seq_lens_out`` / ``free_count_out`` may be the inputs
    themselves.  Returns slot_mapping."""
    idx = _cuda_index("block_table", block_table)
    B, W = _size(seq_lens), _size(block_table, 1)
    T, cap = _size(slot_mapping), _size(free_pages)
    row, one = (B,), (1,)
    _check_ints(idx, torch.int32, (
        ("seq_lens", seq_lens, row), ("block_table", block_table, (B, W)),
        ("new_tokens", new_tokens, row), ("free_pages", free_pages, (cap,)),
        ("free_count", free_count, one), ("seq_lens_out", seq_lens_out, row),
        ("free_count_out", free_count_out, one)))
    _check_ints(idx, torch.int64, (("slot_mapping", slot_mapping, (T,)),))
    pos = off = None
    if positions is not None:
        _check_ints(idx, torch.int32, (("positions", positions, (T,)),))
        pos = positions.data_ptr()
    if token_offsets is not None:
        _check_ints(idx, torch.int32, (("token_offsets", token_offsets, (B + 1,)),))
        off = token_offsets.data_ptr()
    if status is not None:
        _check_status(status, block_table.device)
    rc = _call_on(
        idx, stream, load_library().pqkv_extend_block_tables, seq_lens.data_ptr(),
        new_tokens.data_ptr(), B, block_table.data_ptr(), W, free_pages.data_ptr(),
        free_count.data_ptr(), cap, num_pages, PAGE_SIZE, seq_lens_out.data_ptr(),
        free_count_out.data_ptr(), slot_mapping.data_ptr(), pos, T, off,
        None if status is None else status.data_ptr())
    if rc:
        _check(rc, "extend_block_tables")
    return slot_mapping


def truncate_block_tables(seq_lens, keep_lens, block_table, free_pages, free_count, seq_lens_out,
                          free_count_out, owned_pages=None, status=None, stream=None):
    """Shorten every request to its first ``keep_lens[s]`` tokens and push the
    pages it no longer needs on the stack ``free_pages`` (from entry
    ``free_count`` on): rejected draft tokens, or ended requests (keep 0).
    Pages before ``owned_pages[s]`` (int32 [B], default all 0) belong to
    another request -- a shared prefix -- and stay.  The block table is not
    changed.  ``seq_lens_out`` / ``free_count_out`` may be the inputs
    themselves.  Returns seq_lens_out."""
    idx = _cuda_index("block_table", block_table)
    B, W, cap = _size(seq_lens), _size(block_table, 1), _size(free_pages)
    row, one = (B,), (1,)
    _check_ints(idx, torch.int32, (
        ("seq_lens", seq_lens, row), ("block_table", block_table, (B, W)),
        ("keep_lens", keep_lens, row), ("free_pages", free_pages, (cap,)),
        ("free_count", free_count, one), ("seq_lens_out", seq_lens_out, row),
        ("free_count_out", free_count_out, one)))
    owned = None
    if owned_pages is not None:
        _check_ints(idx, torch.int32, (("owned_pages", owned_pages, row),))
        owned = owned_pages.data_ptr()
    if status is not None:
        _check_status(status, block_table.device)
    rc = _call_on(
        idx, stream, load_library().pqkv_truncate_block_tables, seq_lens.data_ptr(),
        keep_lens.data_ptr(), owned, B, block_table.data_ptr(), W, free_pages.data_ptr(),
        free_count.data_ptr(), cap, PAGE_SIZE, seq_lens_out.data_ptr(), free_count_out.data_ptr(),
        None if status is None else status.data_ptr())
    if rc:
        _check(rc, "truncate_block_tables")
    return seq_lens_out


NOALLOC_SCRATCH_BYTES = 16 << 20


def paged_attention_noalloc(q, pages, block_table, seq_lens, q_len, kv_dtype, k_scale, v_scale,
                            out, num_splits=0, max_seq_len=0, status=None, stream=None):
    """paged_attention for callers that cannot allocate device memory: the
    library uses its own fixed 16 MiB scratch area instead of a workspace.

    The first call on a device must come before any stream capture; calls on
    one device share the scratch area and must not overlap on the GPU.
    Raises ValueError when the launch this call makes needs more scratch than
    the area holds (include/pqkv.h states the sizes).
    """
    kd = _dtype_id(kv_dtype)
    _check_pages(pages, kd)
    H = pages.shape[1]
    if q.dtype != torch.float16 or q.dim() != 3 or q.shape[2] != HEAD_DIM or not q.is_contiguous():
        raise ValueError("q must be contiguous fp16 [num_seqs*q_len, Hq, 128]")
    if out.shape != q.shape or out.dtype != torch.float16 or not out.is_contiguous():
        raise ValueError("out must be contiguous fp16 shaped like q")
    B = seq_lens.shape[0]
    if seq_lens.dtype != torch.int32 or seq_lens.dim() != 1 or not seq_lens.is_contiguous():
        raise ValueError("seq_lens must be contiguous int32 [num_seqs]")
    if block_table.dtype != torch.int32 or block_table.dim() != 2 or block_table.shape[0] != B \
            or not block_table.is_contiguous():
        raise ValueError("block_table must be contiguous int32 [num_seqs, max_pages_per_seq]")
    if q.shape[0] != B * q_len:
        raise ValueError("q has %d rows, expected num_seqs*q_len = %d" % (q.shape[0], B * q_len))
    sph = 0
    if kd in _SCALED:
        sph = _check_scale(k_scale, H, "k_scale")
        if _check_scale(v_scale, H, "v_scale") != sph:
            raise ValueError("k_scale and v_scale must have the same shape")
    dev = pages.device
    _on_device(dev, q=q, out=out, block_table=block_table, seq_lens=seq_lens,
               k_scale=k_scale if kd in _SCALED else None,
               v_scale=v_scale if kd in _SCALED else None)
    _check_status(status, dev)
    lib = load_library()
    with torch.cuda.device(dev):
        rc = lib.pqkv_paged_attention_noalloc(
            _ptr(q), _ptr(out), _ptr(pages), pages.shape[0], _ptr(block_table),
            block_table.shape[1], _ptr(seq_lens), B, q_len, q.shape[1], H, HEAD_DIM, PAGE_SIZE,
            kd, _ptr(k_scale if kd in _SCALED else None),
            _ptr(v_scale if kd in _SCALED else None), sph, num_splits, max_seq_len, _ptr(status),
            _stream(q, stream))
    _check(rc, "paged_attention_noalloc")
    return out


def status_bits(status: torch.Tensor):
    """Names of the device status bits set in an int32 status tensor (syncs)."""
    v = int(status.item())
    return [name for bit, name in _status_names.items() if v & bit]


def version() -> str:
    return load_library().pqkv_version().decode()
