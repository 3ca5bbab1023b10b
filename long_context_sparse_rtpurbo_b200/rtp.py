"""Thin Python binding of librtp's C ABI (include/rtp.h).

The functions keep the C names and only marshal arguments: torch tensors become device
pointers, the current CUDA stream becomes the stream argument. Every step of the decode path
runs in librtp's kernels; there is no CPU fallback, and a missing library raises.
"""
from __future__ import annotations

import ctypes

import numpy as np
import torch

from . import _lib
from ._lib import (RTP_KV_BF16, RTP_KV_E4M3, RTP_OK, RTP_PAGED_CTRL_BYTES, RtpCache,  # noqa: F401
                   RtpLayerDesc, RtpPagedCache, RtpPagePool)


class RtpError(RuntimeError):
    def __init__(self, fn: str, code: int):
        super().__init__(f"{fn} failed: {code} ({rtp_status_str(code)})")
        self.code = code


def _ptr(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, torch.Tensor):
        if t.numel() and not t.is_contiguous():
            raise ValueError("tensors passed to librtp must be contiguous")
        return t.data_ptr() if t.numel() else None
    return int(t)


def _stream(stream) -> int | None:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _check(fn: str, rc: int):
    if rc != RTP_OK:
        raise RtpError(fn, rc)
    return rc


def rtp_status_str(code: int) -> str:
    return _lib.load().rtp_status_str(code).decode()


def rtp_build_slot_map(ret_mask) -> tuple[np.ndarray, int, int]:
    """Host retrieval mask [Hkv] -> (slot_of_kv int32 [Hkv], n_ret, n_loc)."""
    m = np.ascontiguousarray(np.asarray(ret_mask, dtype=np.uint8))
    slots = np.zeros(m.shape[0], dtype=np.int32)
    nr, nl = ctypes.c_int32(), ctypes.c_int32()
    _check("rtp_build_slot_map", _lib.load().rtp_build_slot_map(
        m.ctypes.data, m.shape[0], slots.ctypes.data, ctypes.byref(nr), ctypes.byref(nl)))
    return slots, nr.value, nl.value


class LayerDesc:
    """Owns the host slot array that an RtpLayerDesc points to."""

    def __init__(self, B, Hq, Hkv, sinks, window, max_seq_len, slot_of_kv, rope_base=1e6,
                 head_dim=128, idx_dim=16):
        self.slots = np.ascontiguousarray(np.asarray(slot_of_kv, dtype=np.int32))
        self.c = RtpLayerDesc(B, Hq, Hkv, head_dim, idx_dim, sinks, window, 0, float(rope_base),
                              int(max_seq_len),
                              self.slots.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)))
        self.addr = ctypes.addressof(self.c)
        self.n_ret = int((self.slots >= 0).sum())
        self.n_loc = int((self.slots < 0).sum())

    @property
    def ref(self):
        return ctypes.byref(self.c)


def make_cache(k_ret, v_ret, idx, k_loc, v_loc, seq_off, seq_cap, T_total) -> RtpCache:
    return RtpCache(_ptr(k_ret), _ptr(v_ret), _ptr(idx), _ptr(k_loc), _ptr(v_loc), _ptr(seq_off),
                    _ptr(seq_cap), int(T_total))


def rtp_workspace_bytes(desc: LayerDesc) -> int:
    return int(_lib.load().rtp_workspace_bytes(desc.ref))


def rtp_workspace_init(ws: torch.Tensor, stream=None):
    _check("rtp_workspace_init",
           _lib.load().rtp_workspace_init(_ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))


def rtp_append_kv(desc: LayerDesc, cache: RtpCache, k_pre, v, w_kidx, start_pos, n_new_b, n_new,
                  ws=None, stream=None):
    return _check("rtp_append_kv", _lib.load().rtp_append_kv(
        desc.ref, ctypes.byref(cache), _ptr(k_pre), _ptr(v), _ptr(w_kidx), _ptr(start_pos),
        _ptr(n_new_b), int(n_new), _ptr(ws), _stream(stream)))


def rtp_decode_step(desc: LayerDesc, cache: RtpCache, q_pre, w_qidx, seq_lens, p, out, sel_counts,
                    sel_idx=None, sel_stride=0, ws=None, ws_bytes=None, stream=None):
    if ws_bytes is None:
        ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    return _check("rtp_decode_step", _lib.load().rtp_decode_step(
        desc.ref, ctypes.byref(cache), _ptr(q_pre), _ptr(w_qidx), _ptr(seq_lens), float(p),
        _ptr(out), _ptr(sel_counts), _ptr(sel_idx), int(sel_stride), _ptr(ws), int(ws_bytes),
        _stream(stream)))


def rtp_decode_step_append(desc: LayerDesc, cache: RtpCache, k_new, v_new, w_kidx, q_pre, w_qidx,
                           seq_lens, p, out, sel_counts, sel_idx=None, sel_stride=0, ws=None,
                           ws_bytes=None, stream=None):
    """rtp_append_kv of the decode token and rtp_decode_step in one launch (see include/rtp.h)."""
    if ws_bytes is None:
        ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    return _check("rtp_decode_step_append", _lib.load().rtp_decode_step_append(
        desc.ref, ctypes.byref(cache), _ptr(k_new), _ptr(v_new), _ptr(w_kidx), _ptr(q_pre),
        _ptr(w_qidx), _ptr(seq_lens), float(p), _ptr(out), _ptr(sel_counts), _ptr(sel_idx),
        int(sel_stride), _ptr(ws), int(ws_bytes), _stream(stream)))


def rtp_decode_step_topk(desc: LayerDesc, cache: RtpCache, q_pre, w_qidx, seq_lens, k, out,
                         sel_counts, sel_idx=None, sel_stride=0, ws=None, ws_bytes=None,
                         stream=None):
    """Decode step with the fixed-budget top-k selector (see include/rtp.h)."""
    if ws_bytes is None:
        ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    return _check("rtp_decode_step_topk", _lib.load().rtp_decode_step_topk(
        desc.ref, ctypes.byref(cache), _ptr(q_pre), _ptr(w_qidx), _ptr(seq_lens), int(k),
        _ptr(out), _ptr(sel_counts), _ptr(sel_idx), int(sel_stride), _ptr(ws), int(ws_bytes),
        _stream(stream)))


def rtp_prefill_workspace_bytes(desc: LayerDesc, n_max: int) -> int:
    return int(_lib.load().rtp_prefill_workspace_bytes(desc.ref, int(n_max)))


def rtp_prefill(desc: LayerDesc, q_pre, k_pre, v, n_b, n_max, out, ws=None, ws_bytes=None,
                stream=None):
    """Causal prefill attention of one layer over a prompt (see include/rtp.h)."""
    if ws_bytes is None:
        ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    return _check("rtp_prefill", _lib.load().rtp_prefill(
        desc.ref, _ptr(q_pre), _ptr(k_pre), _ptr(v), _ptr(n_b), int(n_max), _ptr(out), _ptr(ws),
        int(ws_bytes), _stream(stream)))


# ------------------------------------------------------------------------------- paged caches
# The calls below check type, size, contiguity and device of every tensor (csrc/binding.cpp): a
# paged call is cheap enough to be made with the wrong one of many buffers. All tensors must be on
# the current device.

def _arg(t: torch.Tensor, what: str, dtype, n: int, dev: int, optional=False) -> int | None:
    if t is None and optional:
        return None
    if t.dtype is not dtype or t.numel() != n or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{what}: a contiguous {dtype} tensor of {n} elements on cuda:{dev} is "
                         f"wanted, got {tuple(t.shape)} {t.dtype} on {t.device}")
    return t.data_ptr()


def _stream_arg(stream) -> int | None:
    return stream if stream is None else getattr(stream, "cuda_stream", stream)


class PagedCache:
    """A paged cache of one layer (see make_paged_cache): owns the tensors that its struct points
    to."""

    def __init__(self, k, v, block_table, k_scale=None, v_scale=None):
        if k.dim() != 4 or k.shape[3] != 128 or k.shape != v.shape or k.stride() != v.stride():
            raise ValueError("k and v: [n_pages][Hkv][page_size][128] tensors of equal strides")
        n_pages, Hkv, page, _ = k.shape
        block = Hkv * page
        if k.stride()[1:] != (page * 128, 128, 1) or (
                n_pages > 1 and (k.stride(0) % 128 or k.stride(0) < block * 128)):
            raise ValueError("the rows of a page must be dense, and pages a whole number of rows "
                             "apart that do not overlap")
        e4m3 = k.dtype in (torch.uint8, torch.float8_e4m3fn)
        if v.dtype is not k.dtype or not (e4m3 or k.dtype is torch.bfloat16):
            raise ValueError("k and v are both bfloat16, or both e4m3 (float8_e4m3fn or uint8)")
        dev = k.get_device()
        if e4m3 != (k_scale is not None) or e4m3 != (v_scale is not None):
            raise ValueError("k_scale and v_scale go with an e4m3 cache, and only with one")
        if v.get_device() != dev:
            raise ValueError("k and v are on different devices")
        n = n_pages * block
        if block_table.dim() != 2:
            raise ValueError("block_table: [B][entries]")
        self.B, self.table_stride = block_table.shape
        self.Hkv, self.page_size, self.n_pages, self.device_index = Hkv, page, n_pages, dev
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.block_table = block_table
        self.c = RtpPagedCache(
            RTP_KV_E4M3 if e4m3 else RTP_KV_BF16, page, n_pages, self.table_stride, k.data_ptr(),
            v.data_ptr(), _arg(k_scale, "k_scale", torch.float32, n, dev, True),
            _arg(v_scale, "v_scale", torch.float32, n, dev, True),
            k.stride(0) // 128 if n_pages > 1 else 0,
            _arg(block_table, "block_table", torch.int32, self.B * self.table_stride, dev))
        self.addr = ctypes.addressof(self.c)


def make_paged_cache(k, v, block_table, k_scale=None, v_scale=None) -> PagedCache:
    """The paged cache of one layer. k, v: [n_pages][Hkv][page_size][128] in bf16, or e4m3 with
    k_scale and v_scale (float [n_pages][Hkv][page_size]); the page axis may have a stride (K and
    V interleaved in one allocation). block_table: int32 [B][entries]."""
    return PagedCache(k, v, block_table, k_scale, v_scale)


class PagePoolRef:
    """The rtp_page_pool of a batch: owns the tensors that it points to."""

    def __init__(self, free_pages, block_table, page_size):
        if block_table.dim() != 2:
            raise ValueError("block_table: [B][entries]")
        self.B, self.table_stride = block_table.shape
        self.n_pages, self.device_index = free_pages.numel(), free_pages.get_device()
        self.free_pages, self.block_table = free_pages, block_table
        dev = self.device_index
        self.c = RtpPagePool(
            self.B, int(page_size), self.n_pages, self.table_stride,
            _arg(free_pages, "free_pages", torch.int32, self.n_pages, dev),
            _arg(block_table, "block_table", torch.int32, self.B * self.table_stride, dev))
        self.addr = ctypes.addressof(self.c)


def make_page_pool(free_pages, block_table, page_size) -> PagePoolRef:
    """free_pages: int32 [n_pages], the ring of free page ids; block_table: int32 [B][entries]."""
    return PagePoolRef(free_pages, block_table, page_size)


def rtp_paged_workspace_bytes(desc: LayerDesc) -> int:
    return int(_lib.load().rtp_paged_workspace_bytes(desc.ref))


def rtp_paged_workspace_init(ws: torch.Tensor, stream=None):
    """Once after allocating a workspace of the paged calls (256-byte aligned)."""
    if ws.get_device() < 0 or ws.get_device() != torch.cuda.current_device():
        raise ValueError(f"workspace: a tensor on the current device is wanted, got one on {ws.device}")
    return _check("rtp_paged_workspace_init", _lib.load().rtp_paged_workspace_init(
        _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))


def rtp_paged_reserve(pool: PagePoolRef, lens, new_lens, counters, lens_out, counters_out, slot_map,
                      n_new, ws, stream=None):
    """Block tables and slot maps for new lengths (see include/rtp.h). lens, new_lens, lens_out:
    int32 [B]; counters, counters_out: int64 [2]; slot_map: int32 [B][n_new]."""
    return _check("rtp_paged_reserve", (_lib._native or _lib.native()).reserve(
        pool.addr, pool.B, pool.device_index, lens, new_lens, counters, lens_out, counters_out,
        slot_map, n_new, None, ws, _stream_arg(stream)))


def rtp_paged_reserve_step(pool: PagePoolRef, lens, new_lens, counters, lens_out, counters_out,
                           slot_map, n_new, step_lens, ws, stream=None):
    """rtp_paged_reserve that also writes the decode step's lengths (see include/rtp.h): step_lens,
    int32 [B], 0 for the sequences that did not grow."""
    return _check("rtp_paged_reserve_step", (_lib._native or _lib.native()).reserve(
        pool.addr, pool.B, pool.device_index, lens, new_lens, counters, lens_out, counters_out,
        slot_map, n_new, step_lens, ws, _stream_arg(stream)))


def _paged_fits(desc: LayerDesc, cache: PagedCache):
    """The description's struct, if it goes with the cache."""
    c = desc.c
    if cache.Hkv != c.Hkv or cache.B != c.B:
        raise ValueError(f"a cache of {cache.Hkv} KV heads and {cache.B} sequences does not go with "
                         f"a description of {c.Hkv} and {c.B}")
    return c


def rtp_paged_append_kv(desc: LayerDesc, cache: PagedCache, k_pre, v, start_pos, slot_map, n_new,
                        ws=None, stream=None):
    """New tokens to their slots (see include/rtp.h). k_pre, v: bf16 [B][n_new][Hkv][128];
    start_pos: int32 [B]; slot_map: int32 [B][n_new]."""
    _paged_fits(desc, cache)
    return _check("rtp_paged_append_kv", (_lib._native or _lib.native()).append_kv(
        desc.addr, cache.addr, cache.B, cache.Hkv, cache.device_index, k_pre, v, start_pos, slot_map,
        n_new, ws, _stream_arg(stream)))


def rtp_paged_decode_step(desc: LayerDesc, cache: PagedCache, q_pre, seq_lens, out, lse=None, ws=None,
                          stream=None):
    """Decode step of one layer over a paged cache (see include/rtp.h). q_pre, out: bf16
    [B][Hq][128]; seq_lens: int32 [B]; lse: float [B][Hq] or None."""
    c = _paged_fits(desc, cache)
    return _check("rtp_paged_decode_step", (_lib._native or _lib.native()).decode_step(
        desc.addr, cache.addr, cache.B, c.Hq, cache.Hkv, cache.device_index, None, None, q_pre,
        seq_lens, out, lse, ws, _stream_arg(stream)))


def rtp_paged_decode_step_append(desc: LayerDesc, cache: PagedCache, k_new, v_new, q_pre, seq_lens,
                                 out, lse=None, ws=None, stream=None):
    """The decode token's append and the decode step in one launch (see include/rtp.h). k_new,
    v_new: bf16 [B][Hkv][128]; the others as rtp_paged_decode_step."""
    c = _paged_fits(desc, cache)
    if k_new is None or v_new is None:
        raise ValueError("k_new and v_new: tensors are wanted")
    return _check("rtp_paged_decode_step_append", (_lib._native or _lib.native()).decode_step(
        desc.addr, cache.addr, cache.B, c.Hq, cache.Hkv, cache.device_index, k_new, v_new, q_pre,
        seq_lens, out, lse, ws, _stream_arg(stream)))


def rtp_decode_step_static(desc: LayerDesc, cache: RtpCache, q_pre, w_qidx, seq_lens, p, out,
                           sel_counts, stream=None):
    """rtp_decode_step on the library's own fixed scratch (no workspace argument): for callers
    that cannot allocate device memory. See include/rtp.h for its limits and sharing rules."""
    return _check("rtp_decode_step_static", _lib.load().rtp_decode_step_static(
        desc.ref, ctypes.byref(cache), _ptr(q_pre), _ptr(w_qidx), _ptr(seq_lens), float(p),
        _ptr(out), _ptr(sel_counts), _stream(stream)))


def rtp_read_device_status(ws, stream=None) -> int:
    return int(_lib.load().rtp_read_device_status(_ptr(ws), _stream(stream)))


def rtp_last_launch_count() -> int:
    return int(_lib.load().rtp_last_launch_count())


def rtp_debug_set_wait_limit(cycles: int):
    """Test hook: limit (SM cycles) of every device-side wait of later decode launches;
    0 restores the default (about one second)."""
    return _check("rtp_debug_set_wait_limit", _lib.load().rtp_debug_set_wait_limit(int(cycles)))


def rtp_debug_fail_next_call(status: int):
    """Test hook: the next append / decode entry-point call returns ``status`` (a negative
    RTP_E* code) without enqueueing anything; 0 cancels."""
    return _check("rtp_debug_fail_next_call", _lib.load().rtp_debug_fail_next_call(int(status)))
