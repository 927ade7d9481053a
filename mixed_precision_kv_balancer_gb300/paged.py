"""Device-resident paged cache of many sequences, all layers in one pool.

The buffers are torch tensors; every operation on them is one of the library's C ABI calls:

  prompt  reserve -> append (every layer) -> mikv_window_attention; a later chunk attends to
          what gather reads back
  decode  reserve (one token each) -> append (every layer) -> attend (every layer)
  mixed   chunks of prompts beside single tokens, as packed rows: reserve -> rows -> in every layer put, then
          attend_rows; or, where each row reads a part of its sequence alone, renew, pick and attend_blocks
  fork    sequences that share a prefix; compact: eviction to the positions mikv_select keeps;
          free: a finished sequence

Tables, lengths and reference counts live on the device, so no call synchronises and a whole
step can be captured into a CUDA graph.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch

from . import _lib

TYPES = {"fp16": _lib.MIKV_PAGES_FP16, "bf16": _lib.MIKV_PAGES_BF16, "int8": _lib.MIKV_PAGES_INT8}


class PagedCache:
    """Pool [layers][n_pages][Hkv][page_size][D], table [max_seqs][max_pages], lens, refs."""

    def __init__(self, layers, n_pages, page_size, Hkv, D, max_seqs, max_pages, type="fp16", device="cuda"):
        dev = torch.device(device)
        shape = (layers, n_pages, Hkv, page_size, D)
        dtype = {"fp16": torch.float16, "bf16": torch.bfloat16, "int8": torch.uint8}[type]
        k, v = torch.zeros(shape, dtype=dtype, device=dev), torch.zeros(shape, dtype=dtype, device=dev)
        k_meta = v_meta = None
        if type == "int8":
            k_meta = torch.zeros(*shape[:4], D // 64, 2, dtype=torch.float16, device=dev)
            v_meta = torch.zeros_like(k_meta)
        self._hold(k, v, k_meta, v_meta, torch.full((max_seqs, max_pages), -1, dtype=torch.int32, device=dev),
                   torch.zeros(max_seqs, dtype=torch.int32, device=dev),
                   torch.zeros(n_pages, dtype=torch.int32, device=dev), type)

    @classmethod
    def over(cls, k, v, table, lens, refs, type="fp16", k_meta=None, v_meta=None):
        """A cache over buffers that exist already (shapes as in the class)."""
        self = cls.__new__(cls)
        self._hold(k, v, k_meta, v_meta, table, lens, refs, type)
        return self

    def _hold(self, k, v, k_meta, v_meta, table, lens, refs, type):
        dtype = {"fp16": torch.float16, "bf16": torch.bfloat16, "int8": torch.uint8}[type]
        layers, n_pages, Hkv, ps, D = k.shape
        max_seqs, max_pages = table.shape
        self.device, self.index = k.device, k.get_device()
        if not k.is_cuda:
            raise ValueError("a paged cache lives on a CUDA device")
        need = lambda t, name, dt, shape: _lib._need(t, name, dt, shape, self.index)
        s = _lib.mikv_pages()
        s.layers, s.n_pages, s.page_size, s.Hkv, s.D, s.type = layers, n_pages, ps, Hkv, D, TYPES[type]
        s.max_seqs, s.max_pages = max_seqs, max_pages
        s.k, s.v = need(k, "k", dtype, k.shape), need(v, "v", dtype, k.shape)
        if type == "int8":
            meta = (layers, n_pages, Hkv, ps, D // 64, 2)
            s.k_meta, s.v_meta = need(k_meta, "k_meta", torch.float16, meta), need(v_meta, "v_meta", torch.float16, meta)
        s.table = need(table, "table", torch.int32, table.shape)
        s.lens, s.refs = need(lens, "lens", torch.int32, (max_seqs,)), need(refs, "refs", torch.int32, (n_pages,))
        self.k, self.v, self.k_meta, self.v_meta = k, v, k_meta, v_meta
        self.table, self.lens, self.refs, self.type = table, lens, refs, type
        self.struct, self.ref = s, ctypes.byref(s)

    # --- workspaces a program keeps --------------------------------------------------
    def page_workspace(self, n):
        """For reserve, fork and compact of up to n requests."""
        return self._bytes(_lib.load().mikv_page_workspace_bytes(self.ref, n))

    def attention_workspace(self, n, Hq, window=0, sinks=0):
        """For attend of n sequences; one for window 0 serves every window."""
        return self._bytes(_lib.load().mikv_paged_attention_workspace_bytes(self.ref, n, Hq, window, sinks))

    def chunk_workspace(self, n, rows, Hq):
        """For attend_rows of n requests with `rows` rows."""
        return self._bytes(_lib.load().mikv_chunk_attention_workspace_bytes(self.ref, n, rows, Hq))

    def block_workspace(self, rows, Hq, keep):
        """For pick and for attend_blocks, one behind the other."""
        lib, rows = _lib.load(), -(-rows // max(1, len(self._row_parts(rows))))
        return self._bytes(max(lib.mikv_block_select_workspace_bytes(self.ref, rows, Hq),
                               lib.mikv_block_attention_workspace_bytes(self.ref, rows, Hq, keep)))

    def bounds_buffers(self):
        """(bounds, scales) of all pages' keys, for renew and pick."""
        layers, n_pages, Hkv, _, D = self.k.shape
        return (torch.zeros(layers, n_pages, Hkv, 2, D, dtype=torch.int8, device=self.device),
                torch.zeros(layers, n_pages, Hkv, dtype=torch.float32, device=self.device))

    def _bytes(self, nbytes):
        if nbytes == 0:
            raise ValueError("the library has no workspace size for these dimensions")
        return torch.empty(nbytes, dtype=torch.uint8, device=self.device)

    def _ints(self, n):
        return torch.empty(n, dtype=torch.int32, device=self.device)

    # --- the calls, with outputs made where none is given -----------------------------
    def reserve(self, add, seqs=None, start=None, ws=None):
        """Room for add [n] more tokens; returns each sequence's first new slot (-1: refused)."""
        start = self._ints(add.shape[0]) if start is None else start
        _lib.mikv_page_reserve(self, seqs, add, start, ws=ws)
        return start

    def fork(self, parent, child, ok=None, ws=None):
        ok = self._ints(parent.shape[0]) if ok is None else ok
        _lib.mikv_page_fork(self, parent, child, ok, ws=ws)
        return ok

    def free(self, seqs, ok=None):
        ok = self._ints(seqs.shape[0]) if ok is None else ok
        _lib.mikv_page_free(self, seqs, ok)
        return ok

    def copy(self, src, dst, ok=None):
        ok = self._ints(src.shape[0]) if ok is None else ok
        _lib.mikv_page_copy(self, src, dst, ok)
        return ok

    def compact(self, keep_pos, keep_n, seqs=None, ok=None, ws=None):
        ok = self._ints(keep_n.shape[0]) if ok is None else ok
        _lib.mikv_page_compact(self, seqs, keep_pos, keep_n, ok, ws=ws)
        return ok

    def append(self, layer, k, v, seqs=None, start=None, counts=None):
        _lib.mikv_paged_append(self, layer, k, v, seqs=seqs, start=start, counts=counts)

    def gather(self, layer, k_out, v_out, seqs=None):
        _lib.mikv_paged_gather(self, layer, k_out, v_out, seqs=seqs)
        return k_out, v_out

    def attend(self, layer, q, window=0, sinks=0, seqs=None, out=None, lse=None, ws=None):
        """q [n][Hq][D] against each sequence's slots; returns out [n][Hq][D] and lse fp32 [n][Hq]."""
        out = torch.empty_like(q) if out is None else out
        lse = torch.empty(q.shape[:2], dtype=torch.float32, device=self.device) if lse is None else lse
        _lib.mikv_paged_attention(q, self, layer, window, sinks, out, lse, seqs=seqs, ws=ws)
        return out, lse

    # --- packed batches ----------------------------------------------------------------
    def rows(self, counts, rows, seqs=None, start=None):
        """BatchRows of requests with counts [n] rows each, in arrays of `rows` rows."""
        b = BatchRows(self._ints(counts.shape[0] + 1), *torch.empty(3, rows, dtype=torch.int32, device=self.device), seqs, start)
        _lib.mikv_batch_rows(self, counts, b.row_start, b.seq, b.pos, b.slot, seqs=seqs, start=start)
        return b

    def put(self, layer, k, v, batch):
        """Rows k, v [rows][Hkv][D] of a batch into their slots."""
        _lib.mikv_slot_append(self, layer, k, v, batch.slot)

    def renew(self, layer, batch, bounds):
        """bounds: (bounds, scales) of the pages that the batch's rows lie on, done anew."""
        _lib.mikv_page_bounds(self, layer, batch.seq, batch.pos, *bounds)

    def attend_rows(self, layer, q, batch, window=0, sinks=0, out=None, lse=None, ws=None):
        """Rows q [rows][Hq][D] of a batch against their sequences; returns out and lse fp32 [rows][Hq].  Rows
        of no request are left as they were (outputs made here: 0).  Softmax weights are rounded once to 16 bits; attend and
        attend_blocks keep two parts of each."""
        out = torch.zeros(q.shape, dtype=q.dtype, device=self.device) if out is None else out
        lse = torch.zeros(q.shape[:2], dtype=torch.float32, device=self.device) if lse is None else lse
        _lib.mikv_chunk_attention(q, self, layer, batch.row_start, window, sinks, out, lse, seqs=batch.seqs, start=batch.start, ws=ws)
        return out, lse

    def pick(self, layer, q, bounds, keep, first=0, recent=1, batch=None, sel=None, n_sel=None, ws=None):
        """The `keep` blocks that each row of q [rows][Hq][D] reads (batch None: row r is sequence r's last token):
        sel int32 [rows][Hkv][keep] and n_sel int32 [rows][Hkv]."""
        rows, Hkv = q.shape[0], self.k.shape[2]
        sel = torch.empty(rows, Hkv, keep, dtype=torch.int32, device=self.device) if sel is None else sel
        n_sel = torch.empty(rows, Hkv, dtype=torch.int32, device=self.device) if n_sel is None else n_sel
        for seq, pos, q, sl, ns in self._in_parts(batch, q, sel, n_sel):
            _lib.mikv_block_select(q, self, layer, *bounds, first, recent, sl, ns, row_seq=seq, row_pos=pos, ws=ws)
        return sel, n_sel

    def attend_blocks(self, layer, q, sel, n_sel, batch=None, out=None, lse=None, ws=None):
        """Rows q [rows][Hq][D] against their picked blocks; returns out and lse fp32 [rows][Hq].  (Rows whose number times the
        key heads is above 65535 go in several calls, as those of pick do.)"""
        out = torch.empty_like(q) if out is None else out
        lse = torch.empty(q.shape[:2], dtype=torch.float32, device=self.device) if lse is None else lse
        for seq, pos, q, sl, ns, o, l in self._in_parts(batch, q, sel, n_sel, out, lse):
            _lib.mikv_block_attention(q, self, layer, sl, ns, o, l, row_seq=seq, row_pos=pos, ws=ws)
        return out, lse

    def _row_parts(self, rows):
        """Bounds of the equal parts in which the calls over picked blocks take rows: 65535 (row, key head) pairs at most."""
        n = -(-rows // max(1, 65535 // self.k.shape[2]))
        return [(rows * i // n, rows * (i + 1) // n) for i in range(n)]

    def _in_parts(self, batch, *tensors):
        """(sequences, positions, *tensors) of each part of the rows."""
        rows = tensors[0].shape[0]
        tensors = (None, None, *tensors) if batch is None else (batch.seq, batch.pos, *tensors)
        parts = self._row_parts(rows)
        if len(parts) < 2:
            return [tensors]
        if any(t is not None and t.shape[0] != rows for t in tensors):
            raise ValueError(f"expected tensors of {rows} rows, got {[None if t is None else t.shape[0] for t in tensors]}")
        if batch is None:   # row r is sequence r
            tensors = (torch.arange(rows, dtype=torch.int32, device=self.device), *tensors[1:])
        return [tuple(None if t is None else t[a:b] for t in tensors) for a, b in parts]


class BatchRows(NamedTuple):
    """Rows of a packed batch: row_start int32 [n + 1]; each row's sequence, position and slot int32 [rows]; and
    the requests' sequences and first slots that they were made from."""
    row_start: torch.Tensor
    seq: torch.Tensor
    pos: torch.Tensor
    slot: torch.Tensor
    seqs: torch.Tensor | None
    start: torch.Tensor | None
