"""Tiered page store of the hierarchical KV cache, through the C ABI (hkv_store_*).

The memories of the store are allocated here (plumbing): the host tier in
page-locked host memory mapped into the device address space, the HBM slot pool
and the residency state with torch.  Every decision and copy runs in the library's
kernels; this class only marshals arguments.
"""
from __future__ import annotations

import ctypes

import torch

from . import (Quant, StoreDesc, _check, _p, _refuse, _stream, hkv_attn_quant, hkv_gather_quant, hkv_page_summary,
               hkv_quant_page_size, hkv_store_write_quant, load_library)


class MappedHostMemory:
    """Page-locked host memory mapped into the device address space
    (cudaHostAlloc with the mapped and portable flags), freed by close()."""

    def __init__(self, nbytes: int):
        from cuda.bindings import runtime as rt
        self._rt = rt
        err, ptr = rt.cudaHostAlloc(nbytes, rt.cudaHostAllocMapped | rt.cudaHostAllocPortable)
        if err != rt.cudaError_t.cudaSuccess:
            raise RuntimeError(f"cudaHostAlloc({nbytes}): {err}")
        self.host_ptr = int(ptr)
        err, dptr = rt.cudaHostGetDevicePointer(self.host_ptr, 0)
        if err != rt.cudaError_t.cudaSuccess:
            rt.cudaFreeHost(self.host_ptr)
            raise RuntimeError(f"cudaHostGetDevicePointer: {err}")
        self.dev_ptr = int(dptr)
        self.nbytes = nbytes

    def close(self):
        if self.host_ptr:
            self._rt.cudaFreeHost(self.host_ptr)
            self.host_ptr = 0


class PageStore:
    """NP pages of [P_tok, H, d] bf16 K and V on the host tier, S of them in HBM slots."""

    def __init__(self, NP: int, S: int, P_tok: int, H: int, d: int, host=None, stream=None):
        """host: optional (K, V) objects with a `dev_ptr` attribute that already hold
        the host tier (e.g. pages written by the caller); else it is allocated here."""
        self.NP, self.S, self.P_tok, self.H, self.d = NP, S, P_tok, H, d
        page_bytes = P_tok * H * d * 2
        self._own = host is None
        self.host = host if host is not None else (MappedHostMemory(NP * page_bytes), MappedHostMemory(NP * page_bytes))
        self.slot_k = torch.empty(S, P_tok, H, d, dtype=torch.bfloat16, device="cuda")
        self.slot_v = torch.empty(S, P_tok, H, d, dtype=torch.bfloat16, device="cuda")
        lib = load_library()
        self.state = torch.zeros(lib.hkv_store_state_size(NP, S), dtype=torch.uint8, device="cuda")
        self.desc = StoreDesc(NP, S, P_tok, H, d, self.host[0].dev_ptr, self.host[1].dev_ptr,
                              self.slot_k.data_ptr(), self.slot_v.data_ptr(), self.state.data_ptr())
        _check(lib.hkv_store_init(ctypes.byref(self.desc), _stream(stream)), "hkv_store_init")
        tk, tv = ctypes.c_void_p(), ctypes.c_void_p()
        _check(lib.hkv_store_tables(ctypes.byref(self.desc), ctypes.byref(tk), ctypes.byref(tv)), "hkv_store_tables")
        self.table_k, self.table_v = tk.value, tv.value

    def check_open(self, call):
        """Refuse what would launch kernels over the host tier of a closed store."""
        if self.host is None:
            _refuse(f"{type(self).__name__}.{call}", "the store is closed: its host tier is gone")

    def page_tables(self):
        """(K, V) device page tables as int64 tensor views (for hkv_gather).  Not to be read once the store is closed."""
        self.check_open("page_tables")
        n = self.NP
        off_k = self.table_k - self.state.data_ptr()
        off_v = self.table_v - self.state.data_ptr()
        return (self.state[off_k:off_k + 8 * n].view(torch.int64), self.state[off_v:off_v + 8 * n].view(torch.int64))

    def seal(self, page: int, K_rows, V_rows, kbar_out, ws, stream=None):
        self.check_open("seal")
        _check(load_library().hkv_store_seal(ctypes.byref(self.desc), page, _p(K_rows), _p(V_rows), _p(kbar_out),
                                             _p(ws), ws.numel(), _stream(stream)), "hkv_store_seal")

    def fetch(self, sel, ws, stream=None):
        self.check_open("fetch")
        _check(load_library().hkv_store_fetch(ctypes.byref(self.desc), _p(sel), sel.numel(), _p(ws), ws.numel(),
                                              _stream(stream)), "hkv_store_fetch")

    def prefetch(self, scores, protect, m: int, ws, stream=None):
        self.check_open("prefetch")
        n = 0 if protect is None else protect.numel()
        _check(load_library().hkv_store_prefetch(ctypes.byref(self.desc), _p(scores), _p(protect), n, m, _p(ws),
                                                 ws.numel(), _stream(stream)), "hkv_store_prefetch")

    def residency(self, stream=None):
        """(slot_of_page [NP], page_of_slot [S]) as device int32 tensors."""
        sp = torch.empty(self.NP, dtype=torch.int32, device="cuda")
        ps = torch.empty(self.S, dtype=torch.int32, device="cuda")
        _check(load_library().hkv_store_residency(ctypes.byref(self.desc), _p(sp), _p(ps), _stream(stream)),
               "hkv_store_residency")
        return sp, ps

    def close(self):
        """Free the host tier where the store owns it (after the kernels that may be reading it); once."""
        if self.host is not None and self._own:
            torch.cuda.synchronize(self.slot_k.device)
            for h in self.host:
                h.close()
        self.host = None


class QuantPageStore(PageStore):
    """A page store whose pages are quantised: half or a quarter of the host tier, of the HBM slots and of the host link's
    traffic of bf16 pages.  The residency calls (fetch, prefetch, residency) are PageStore's: to them a page is a block of
    bytes, passed as page_bytes / 1024 rows of 4 x 128 bf16 elements.  Rows are written to the host tier and to the slots of
    pages that are resident: a page may be fetched before all its rows are written."""

    def __init__(self, quant: Quant, NP: int, S: int, P_tok: int, H: int, d: int, host=None, stream=None):
        self.quant, self.rows, self.heads, self.head_dim = quant, P_tok, H, d
        self.page_bytes, self.scale_offset = hkv_quant_page_size(quant, P_tok, H, d)
        super().__init__(NP, S, self.page_bytes // 1024, 4, 128, host, stream)
        self.P_tok, self.H, self.d = P_tok, H, d  # of the pages; `desc` has the block's

    def write(self, K, V, first_row: int, ws, first_row_dev=None, rope=None, pos=None, stream=None):
        """Append rows K, V [T, H, d] at history row first_row (+ first_row_dev), in stream order with the store's other
        calls: hkv_quant_rows into the host tier, and into the slots of resident pages."""
        self.check_open("write")
        if K.get_device() != self.slot_k.get_device():
            _refuse("QuantPageStore.write", f"K is on {K.device}, the store on {self.slot_k.device}")
        hkv_store_write_quant(self.desc, self.quant, K, V, self.rows, first_row, ws, first_row_dev, rope, pos, stream)

    def seal(self, page: int, K_rows, V_rows, kbar_out, ws, rope=None, pos=None, stream=None):
        """Write the rows of page `page` and its summary kbar_out (the mean of K_rows, bf16, before any rotation)."""
        if K_rows.shape != (self.rows, self.heads, self.head_dim) or K_rows.dtype != torch.bfloat16 or not K_rows.is_contiguous():
            _refuse("QuantPageStore.seal", f"K_rows is {list(K_rows.shape)} {K_rows.dtype}: a contiguous bfloat16 "
                                           f"[{self.rows}, {self.heads}, {self.head_dim}] wanted")
        if not 0 <= page < self.NP:
            _refuse("QuantPageStore.seal", f"page {page} outside [0, {self.NP})")
        self.write(K_rows, V_rows, page * self.rows, ws, rope=rope, pos=pos, stream=stream)
        hkv_page_summary(K_rows, kbar_out, ws, stream)

    def gather(self, sel, Kc, Vc, ws, kbar128=None, rope=None, pos=None, stream=None):
        """hkv_gather_quant of the pages `sel` (int32 device tensor), from their slots or the host tier."""
        self.check_open("gather")
        hkv_gather_quant(self.quant, *self.page_tables(), sel, sel.numel(), self.rows, self.heads, self.head_dim, Kc, Vc, ws,
                         kbar128, rope, pos, stream)

    def attend(self, Q, sel, out, lse, ws, n_rows=None, scale=0.0, stream=None):
        """hkv_attn_quant of a few queries over the pages `sel`."""
        self.check_open("attend")
        hkv_attn_quant(self.quant, Q, *self.page_tables(), sel, sel.numel(), self.rows, self.heads, out, lse, ws, n_rows, scale,
                       stream)
