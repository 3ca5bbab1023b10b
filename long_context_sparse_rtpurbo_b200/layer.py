"""A decode layer's device memory (caches, workspace) allocated with PyTorch, driving librtp
through the C ABI: DecodeLayer over contiguous caches, PageTable and PagedLayer over paged ones.
Allocation and stream plumbing only; no arithmetic of the method."""
from __future__ import annotations

import numpy as np
import torch

from . import rtp


def _workspace(n, device):
    """n bytes at a 256-byte boundary."""
    buf = torch.empty(n + 256, dtype=torch.uint8, device=device)
    off = (-buf.data_ptr()) % 256
    return buf[off:off + n]


def _prefill_scratch(layer, n_max, device, stream):
    """layer.pf_ws, large enough for prompts of n_max tokens: allocated on first use, grown with the
    prompt, always for the stream that the call runs on (a block of another stream's may still be
    written by what that stream has queued). A captured graph holds the address of its scratch, so
    that one stays allocated with the layer (pf_held) when a longer prompt gets another."""
    need = rtp.rtp_prefill_workspace_bytes(layer.desc, n_max)
    if need == 0:
        raise ValueError("librtp rejected the prompt length")
    used = torch.cuda.current_stream(device) if stream is None else stream
    if not hasattr(used, "cuda_stream"):                  # an address; 0 is the default stream's
        used = (torch.cuda.ExternalStream(int(used), device=device) if int(used)
                else torch.cuda.default_stream(device))
    with torch.cuda.stream(used):
        if layer.pf_ws is None or layer.pf_ws.numel() < need:
            layer.pf_ws = _workspace(need, device)
        if torch.cuda.is_current_stream_capturing() and not any(x is layer.pf_ws for x in layer.pf_held):
            layer.pf_held.append(layer.pf_ws)
    # a later, longer prompt lets go of this buffer: not before this call's stream is done
    layer.pf_ws.record_stream(used)
    return layer.pf_ws


class DecodeLayer:
    def __init__(self, B, Hq, Hkv, sinks, window, max_seq_len, ret_mask, seq_caps,
                 device="cuda", rope_base=1e6):
        slots, n_ret, n_loc = rtp.rtp_build_slot_map(ret_mask)
        self.B, self.Hq, self.Hkv = B, Hq, Hkv
        self.sinks, self.window = sinks, window
        self.n_ret, self.n_loc = n_ret, n_loc
        self.slots = slots
        self.desc = rtp.LayerDesc(B, Hq, Hkv, sinks, window, max_seq_len, slots, rope_base)
        caps = np.asarray(seq_caps, dtype=np.int64)
        offs = np.concatenate([[0], np.cumsum(caps)[:-1]]).astype(np.int64)
        self.seq_caps_host, self.seq_offs_host = caps, offs
        self.T_total = int(caps.sum())
        bf = torch.bfloat16
        ring = sinks + window
        self.k_ret = torch.empty((n_ret, self.T_total, 128), dtype=bf, device=device)
        self.v_ret = torch.empty((n_ret, self.T_total, 128), dtype=bf, device=device)
        self.idx = torch.empty((n_ret, self.T_total, 16), dtype=bf, device=device)
        self.k_loc = torch.empty((n_loc, B, ring, 128), dtype=bf, device=device)
        self.v_loc = torch.empty((n_loc, B, ring, 128), dtype=bf, device=device)
        self.seq_off = torch.tensor(offs, dtype=torch.int64, device=device)
        self.seq_cap = torch.tensor(caps.astype(np.int32), dtype=torch.int32, device=device)
        self.cache = rtp.make_cache(self.k_ret, self.v_ret, self.idx, self.k_loc, self.v_loc,
                                    self.seq_off, self.seq_cap, self.T_total)
        self.ws_bytes = rtp.rtp_workspace_bytes(self.desc)
        if self.ws_bytes == 0:
            raise ValueError("librtp rejected the layer description")
        self.ws = torch.empty(self.ws_bytes + 256, dtype=torch.uint8, device=device)
        off = (-self.ws.data_ptr()) % 256
        self.ws = self.ws[off:off + self.ws_bytes]
        rtp.rtp_workspace_init(self.ws)
        self.zeros = torch.zeros(B, dtype=torch.int32, device=device)   # start of a prompt
        self.pf_ws, self.pf_held = None, []

    def append(self, k_pre, v, w_kidx, start_pos, n_new_b=None, stream=None):
        """k_pre, v: bf16 [B][n_new][Hkv][128]."""
        return rtp.rtp_append_kv(self.desc, self.cache, k_pre, v, w_kidx, start_pos, n_new_b,
                                 k_pre.shape[1], self.ws, stream)

    def decode(self, q_pre, w_qidx, seq_lens, p, out, sel_counts, sel_idx=None, stream=None):
        stride = 0 if sel_idx is None else sel_idx.shape[-1]
        return rtp.rtp_decode_step(self.desc, self.cache, q_pre, w_qidx, seq_lens, p, out,
                                   sel_counts, sel_idx, stride, self.ws, self.ws_bytes, stream)

    def decode_topk(self, q_pre, w_qidx, seq_lens, k, out, sel_counts, sel_idx=None, stream=None):
        """Decode step with the fixed-budget top-k selector."""
        stride = 0 if sel_idx is None else sel_idx.shape[-1]
        return rtp.rtp_decode_step_topk(self.desc, self.cache, q_pre, w_qidx, seq_lens, k, out,
                                        sel_counts, sel_idx, stride, self.ws, self.ws_bytes,
                                        stream)

    def decode_append(self, k_new, v_new, w_kidx, q_pre, w_qidx, seq_lens, p, out, sel_counts,
                      sel_idx=None, stream=None):
        """Append of the decode token (k_new, v_new: bf16 [B][Hkv][128] at seq_lens - 1) and
        the decode step in one launch."""
        stride = 0 if sel_idx is None else sel_idx.shape[-1]
        return rtp.rtp_decode_step_append(self.desc, self.cache, k_new, v_new, w_kidx, q_pre,
                                          w_qidx, seq_lens, p, out, sel_counts, sel_idx, stride,
                                          self.ws, self.ws_bytes, stream)

    def prefill(self, q_pre, k_pre, v, w_kidx, n_b, out, stream=None):
        """Prompt of n_b[b] tokens at positions 0..n_b[b]-1 (q_pre: bf16 [B][n_max][Hq][128];
        k_pre, v: bf16 [B][n_max][Hkv][128]; n_b: device int32 [B]): appends its K/V and index
        keys to the caches, then writes the causal prefill attention to out
        ([B][n_max][Hq][128]). The prefill scratch is allocated on first use and grown with
        the prompt."""
        n_max = q_pre.shape[1]
        rtp.rtp_append_kv(self.desc, self.cache, k_pre, v, w_kidx, self.zeros, n_b, n_max, self.ws,
                          stream)
        ws = _prefill_scratch(self, n_max, q_pre.device, stream)
        return rtp.rtp_prefill(self.desc, q_pre, k_pre, v, n_b, n_max, out, ws, ws.numel(), stream)

    def status(self, stream=None) -> int:
        return rtp.rtp_read_device_status(self.ws, stream)


class PageTable:
    """The pages of a batch of B sequences, shared by the layers of a model: lengths, block
    table and ring of free pages, all on the GPU. A sequence holds at most max_seq_len tokens, in pages
    of its own: references are not counted, so block_table never has a page twice (a shared prefix
    goes into another table, see include/rtp.h)."""

    def __init__(self, B, n_pages, page_size, max_seq_len, device="cuda"):
        i32 = dict(dtype=torch.int32, device=device)
        self.B, self.n_pages, self.page_size = B, n_pages, page_size
        self.lens = torch.zeros(B, **i32)
        self.step_lens = torch.zeros(B, **i32)
        self.block_table = torch.zeros((B, max(1, -(-max_seq_len // page_size))), **i32)
        self.free_pages = torch.arange(n_pages, **i32)
        self.counters = torch.tensor([0, n_pages], dtype=torch.int64, device=device)
        self.pool = rtp.make_page_pool(self.free_pages, self.block_table, page_size)
        self.ws = _workspace(rtp.RTP_PAGED_CTRL_BYTES, device)
        rtp.rtp_paged_workspace_init(self.ws)

    def reserve(self, new_lens, slot_map=None, stream=None):
        """Takes or returns pages so that sequence b holds new_lens[b] tokens (int32 [B]; 0 ends
        it) and writes the slots of its new tokens to slot_map (int32 [B][n_new]). Updates lens
        in place: a sequence that the free pages do not suffice for keeps its length. step_lens
        then holds the lengths of the sequences that grew and 0 for the others: the seq_lens of
        the decode step over the new tokens. Further wishes start from lens, not from earlier ones:
        a sequence that was refused would otherwise grow over positions that nothing wrote."""
        n_new = 0 if slot_map is None else slot_map.shape[1]
        return rtp.rtp_paged_reserve_step(self.pool, self.lens, new_lens, self.counters, self.lens,
                                          self.counters, slot_map, n_new, self.step_lens, self.ws,
                                          stream)

    def status(self, stream=None) -> int:
        return rtp.rtp_read_device_status(self.ws, stream)


class PagedLayer:
    """One layer's K/V pages over a PageTable. kv_dtype: torch.bfloat16, or torch.float8_e4m3fn
    with a scale per row."""

    def __init__(self, table: PageTable, Hq, Hkv, sinks, window, max_seq_len, ret_mask,
                 kv_dtype=torch.bfloat16, rope_base=1e6):
        device = table.block_table.device
        self.table, self.B, self.Hq, self.Hkv = table, table.B, Hq, Hkv
        slots, self.n_ret, self.n_loc = rtp.rtp_build_slot_map(ret_mask)
        self.desc = rtp.LayerDesc(table.B, Hq, Hkv, sinks, window, max_seq_len, slots, rope_base)
        shape = (table.n_pages, Hkv, table.page_size, 128)
        self.k = torch.empty(shape, dtype=kv_dtype, device=device)
        self.v = torch.empty(shape, dtype=kv_dtype, device=device)
        self.k_scale = self.v_scale = None
        if kv_dtype is not torch.bfloat16:
            self.k_scale = torch.empty(shape[:3], dtype=torch.float32, device=device)
            self.v_scale = torch.empty(shape[:3], dtype=torch.float32, device=device)
        self.cache = rtp.make_paged_cache(self.k, self.v, table.block_table, self.k_scale,
                                          self.v_scale)
        n = rtp.rtp_paged_workspace_bytes(self.desc)
        if n == 0:
            raise ValueError("librtp rejected the layer description")
        self.ws = _workspace(n, device)
        rtp.rtp_paged_workspace_init(self.ws)
        self.zeros = torch.zeros(table.B, dtype=torch.int32, device=device)
        self.pf_ws, self.pf_held = None, []

    def append(self, k_pre, v, start_pos, slot_map, stream=None):
        """k_pre, v: bf16 [B][n_new][Hkv][128]; start_pos: int32 [B], the lengths before the
        reservation that filled slot_map (int32 [B][n_new])."""
        return rtp.rtp_paged_append_kv(self.desc, self.cache, k_pre, v, start_pos, slot_map,
                                       k_pre.shape[1], self.ws, stream)

    def decode(self, q_pre, seq_lens, out, lse=None, stream=None):
        """Decode step at position seq_lens - 1, whose token the pages hold (0: an idle place)."""
        return rtp.rtp_paged_decode_step(self.desc, self.cache, q_pre, seq_lens, out, lse, self.ws,
                                         stream)

    def decode_append(self, k_new, v_new, q_pre, seq_lens, out, lse=None, stream=None):
        """Append of the decode token (k_new, v_new: bf16 [B][Hkv][128] at seq_lens - 1, whose
        page is reserved) and the decode step in one launch. After a reservation seq_lens is the
        table's step_lens: under its lens, a sequence that got no page would have its last row
        overwritten."""
        return rtp.rtp_paged_decode_step_append(self.desc, self.cache, k_new, v_new, q_pre,
                                                seq_lens, out, lse, self.ws, stream)

    def prefill(self, q_pre, k_pre, v, n_b, slot_map, out, stream=None):
        """Prompts of n_b[b] tokens at positions 0..n_b[b]-1 of sequences that were just reserved
        with slot_map (int32 [B][n_max]): appends their K/V to the pages, then writes the causal
        prefill attention to out, as DecodeLayer.prefill. The prefill attends to the bf16 keys
        and values of the prompt, whatever the cache holds."""
        n_max = q_pre.shape[1]
        rtp.rtp_paged_append_kv(self.desc, self.cache, k_pre, v, self.zeros, slot_map, n_max,
                                self.ws, stream)
        ws = _prefill_scratch(self, n_max, q_pre.device, stream)
        return rtp.rtp_prefill(self.desc, q_pre, k_pre, v, n_b, n_max, out, ws, ws.numel(), stream)

    def status(self, stream=None) -> int:
        return rtp.rtp_read_device_status(self.ws, stream)
