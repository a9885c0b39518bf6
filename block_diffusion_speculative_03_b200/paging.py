"""A paged key/value pool over the C ABI (include/dflash_paged.h).

:class:`PagePool` owns the device memory of a pool: pages of `page_size` positions of every
layer's keys and values, handed out to sequences through tables on the device.  Its methods
carry the C calls' meaning; they check shapes, types and devices, pass pointers and the
current CUDA stream of the pool's device, and never synchronise (except :meth:`status`).
The pool's memory belongs to the stream it was made on: before a pool that was used on another
one is dropped, that stream's work has to be done (or waited for).

    pool = drafter.new_pool(n_pages=4096, page_size=64, max_seqs=64, max_len=32768)
    pool.reserve(grow)                          # room for the rows about to be written
    for layer in range(n_layers):
        pool.write(layer, k, v)                 # one new row per sequence (or ragged rows)
        o = pool.attention(layer, q)            # over [0, len] of every sequence
    pool.advance()                              # the rows now belong to the context
    pool.fork(src, dst)                         # dst shares src's pages until it writes
    pool.store(cache); pool.load(cache)         # draft cache <-> pages
"""
from __future__ import annotations

from typing import Optional

import torch

from . import dflash as D
from .drafter import _DT, _aligned_empty

# The current stream of a device as a cudaStream_t; the private call takes a tenth of the time
# of building a Stream object, which a call on a few microseconds of work notices.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = torch.cuda.current_device


class PagePool:
    """Pages of a key/value cache, [n_pages][n_layers][2 (K, V)][n_kv_heads][page_size][head_dim]."""

    def __init__(self, n_layers: int, n_q_heads: int, n_kv_heads: int, head_dim: int, dtype: str, *, n_pages: int,
                 page_size: int, max_seqs: int, max_len: int, device="cuda"):
        self.device = torch.device(device)
        if self.device.type != "cuda":
            raise ValueError("a pool lives on a CUDA device, not on %s" % self.device)
        if self.device.index is None:
            self.device = torch.device("cuda", torch.cuda.current_device())
        dt, self.torch_dtype = _DT[dtype]
        c = D.dflash_pool_config(n_layers=n_layers, n_q_heads=n_q_heads, n_kv_heads=n_kv_heads, head_dim=head_dim,
                                 dtype=dt, n_pages=n_pages, page_size=page_size, max_seqs=max_seqs, max_len=max_len)
        self.cfg = c
        self.n_layers, self.n_q_heads, self.n_kv_heads, self.head_dim = n_layers, n_q_heads, n_kv_heads, head_dim
        self.n_pages, self.page_size, self.max_seqs, self.max_len = n_pages, page_size, max_seqs, max_len
        self.handle = None
        self.nbytes = D.dflash_pool_bytes(c)
        self._index = self.device.index
        with torch.cuda.device(self.device):
            self._buf, self.ptr = _aligned_empty(self.nbytes, self.device)
            self.handle = D.dflash_pool_init(c, self.ptr, self.nbytes, _raw_stream(self._index))
        self._lib = D.lib()
        info = D.dflash_pool_get_info(self.handle)
        self.max_pages = info.max_pages
        base = self._buf.data_ptr()

        def i32(addr, n):
            return self._buf[addr - base:addr - base + 4 * n].view(torch.int32)

        #: Views of the pool's device state: positions, page ids (-1: none) and holders per page.
        self.len = i32(info.len, max_seqs)
        self.table = i32(info.table, max_seqs * info.max_pages).view(max_seqs, info.max_pages)
        self.refs = i32(info.refs, n_pages)
        self._slab_at = info.slab - base

    # -- helpers -----------------------------------------------------------------
    def _run(self, fn, *args) -> None:
        """fn(handle, *args, stream) with the pool's device current."""
        index = self._index
        if _current_device() == index:
            st = fn(self.handle, *args, _raw_stream(index))
        else:
            with torch.cuda.device(index):
                st = fn(self.handle, *args, _raw_stream(index))
        if st:
            raise D.DflashError(st, fn.__name__)

    def _ids(self, t: Optional[torch.Tensor], what: str, n: Optional[int] = None) -> Optional[int]:
        """The address of an int32 list on the pool's device (None stays None)."""
        if t is None:
            return None
        if t.dtype is not torch.int32 or t.get_device() != self._index or not t.is_contiguous():
            raise ValueError("%s: a contiguous int32 tensor on %s is wanted" % (what, self.device))
        if n is not None and t.numel() != n:
            raise ValueError("%s has %d entries, not %d" % (what, t.numel(), n))
        return t.data_ptr()

    def _rows(self, t: torch.Tensor, heads: int, what: str) -> int:
        """Row stride in elements of a [rows, heads, head_dim] tensor whose rows are contiguous."""
        if t.dtype is not self.torch_dtype or t.get_device() != self._index:
            raise ValueError("%s: a %s tensor on %s is wanted" % (what, self.torch_dtype, self.device))
        shape = t.shape
        if len(shape) != 3 or shape[1] != heads or shape[2] != self.head_dim:
            raise ValueError("%s: shape [rows, %d, %d] is wanted, not %s" % (what, heads, self.head_dim, tuple(shape)))
        width = heads * self.head_dim
        if t.is_contiguous():
            return width
        stride = t.stride()
        if stride[2] != 1 or (heads > 1 and stride[1] != self.head_dim):
            raise ValueError("%s: the rows have to be contiguous" % what)
        return stride[0] if shape[0] > 1 else width

    # -- state -------------------------------------------------------------------
    def slab(self) -> torch.Tensor:
        """The pages as a tensor view [n_pages, n_layers, 2, n_kv_heads, page_size, head_dim]."""
        es = 2 if self.torch_dtype == torch.bfloat16 else 4
        n = self.n_pages * self.n_layers * 2 * self.n_kv_heads * self.page_size * self.head_dim
        return self._buf[self._slab_at:self._slab_at + n * es].view(self.torch_dtype).view(
            self.n_pages, self.n_layers, 2, self.n_kv_heads, self.page_size, self.head_dim)

    def status(self) -> int:
        """Synchronise, then return and clear the pool's sticky device error."""
        with torch.cuda.device(self._index):
            return D.dflash_pool_status(self.handle, _raw_stream(self._index))

    def launch_count(self) -> int:
        return D.dflash_pool_launch_count(self.handle)

    def set_tables(self, lens: torch.Tensor, table: torch.Tensor) -> None:
        """Replace every length and table (counts are taken from them); see dflash_pool_set_tables."""
        a = self._ids(lens, "lens", self.max_seqs)
        b = self._ids(table, "table", self.max_seqs * self.max_pages)
        self._run(self._lib.dflash_pool_set_tables, a, b)

    # -- pages -------------------------------------------------------------------
    def reserve(self, grow: torch.Tensor, seqs: Optional[torch.Tensor] = None) -> None:
        """Make the positions [len, len + grow[i]) of each sequence writable (copy on write)."""
        n = grow.numel()
        a, g = self._ids(seqs, "seqs", n), self._ids(grow, "grow")
        self._run(self._lib.dflash_pages_reserve, a, g, n)

    def fork(self, src: torch.Tensor, dst: torch.Tensor, deep: bool = False) -> None:
        """dst[i] shares src[i]'s pages (deep: gets copies of them).  A pair with a -1 is padding."""
        n = src.numel()
        a, b = self._ids(src, "src"), self._ids(dst, "dst", n)
        self._run(self._lib.dflash_pages_fork, a, b, n, 1 if deep else 0)

    def free(self, seqs: Optional[torch.Tensor] = None, keep: Optional[torch.Tensor] = None) -> None:
        """Cut each sequence back to keep[i] positions (None: to nothing) and give its pages back."""
        n = seqs.numel() if seqs is not None else keep.numel() if keep is not None else self.max_seqs
        a, k = self._ids(seqs, "seqs"), self._ids(keep, "keep", n)
        self._run(self._lib.dflash_pages_free, a, k, n)

    def compact(self, used: Optional[torch.Tensor] = None) -> torch.Tensor:
        """Move the pages in use to 0..used-1; returns `used` (int32[1] on the device)."""
        if used is None:
            used = torch.empty(1, dtype=torch.int32, device=self.device)
        u = self._ids(used, "used", 1)
        self._run(self._lib.dflash_pages_compact, u)
        return used

    def write(self, layer: int, k: torch.Tensor, v: torch.Tensor, seqs: Optional[torch.Tensor] = None,
              row_start: Optional[torch.Tensor] = None, row_count: Optional[torch.Tensor] = None,
              max_rows: Optional[int] = None) -> None:
        """Write rows of one layer ([rows, n_kv_heads, head_dim]) at len, len + 1, ... of each sequence."""
        sk, sv = self._rows(k, self.n_kv_heads, "k"), self._rows(v, self.n_kv_heads, "v")
        rows = k.shape[0]
        if v.shape[0] != rows or sk != sv:
            raise ValueError("k and v: the same rows and the same row stride are wanted")
        n = self._entries(seqs, row_start, row_count, rows)
        a, s, c = self._ids(seqs, "seqs", n), self._ids(row_start, "row_start", n), self._ids(row_count, "row_count", n)
        if rows == 0:
            return
        self._run(self._lib.dflash_pages_write, a, n, layer, k.data_ptr(), v.data_ptr(), sk, s, c, rows,
                  rows if max_rows is None else max_rows)

    def advance(self, row_count: Optional[torch.Tensor] = None, seqs: Optional[torch.Tensor] = None) -> None:
        """len += row_count[i] (None: 1) for each sequence."""
        n = row_count.numel() if row_count is not None else seqs.numel() if seqs is not None else self.max_seqs
        a, c = self._ids(seqs, "seqs", n), self._ids(row_count, "row_count")
        self._run(self._lib.dflash_pages_advance, a, c, n)

    def store(self, cache, seqs: Optional[torch.Tensor] = None, reqs: Optional[torch.Tensor] = None) -> None:
        """Append to each sequence the positions that its request of the draft cache has more."""
        n = self._pairs(cache, seqs, reqs)
        a, b = self._ids(seqs, "seqs", n), self._ids(reqs, "reqs", n)
        self._run(self._lib.dflash_pages_store, a, cache.handle, b, n)

    def load(self, cache, seqs: Optional[torch.Tensor] = None, reqs: Optional[torch.Tensor] = None) -> None:
        """Append to each request of the draft cache the positions that its sequence has more."""
        n = self._pairs(cache, seqs, reqs)
        a, b = self._ids(seqs, "seqs", n), self._ids(reqs, "reqs", n)
        self._run(self._lib.dflash_pages_load, a, cache.handle, b, n)

    def _pairs(self, cache, seqs, reqs) -> int:
        if cache.drafter.device != self.device:
            raise ValueError("the cache is on %s, the pool on %s" % (cache.drafter.device, self.device))
        return seqs.numel() if seqs is not None else reqs.numel() if reqs is not None else min(cache.batch,
                                                                                             self.max_seqs)

    @staticmethod
    def _entries(seqs, row_start, row_count, rows: int) -> int:
        if (row_start is None) != (row_count is None):
            raise ValueError("row_start and row_count go together")
        if row_count is not None:
            return row_count.numel()
        if seqs is not None and seqs.numel() > rows:
            raise ValueError("%d sequences, %d rows" % (seqs.numel(), rows))
        return rows if seqs is None else seqs.numel()

    # -- attention ---------------------------------------------------------------
    def attention(self, layer: int, q: torch.Tensor, out: Optional[torch.Tensor] = None,
                  seqs: Optional[torch.Tensor] = None, row_start: Optional[torch.Tensor] = None,
                  row_count: Optional[torch.Tensor] = None, max_rows: Optional[int] = None, causal: bool = True,
                  window: int = 0, sinks: int = 0) -> torch.Tensor:
        """Attention of the new rows q [rows, n_q_heads, head_dim] at the positions len, len + 1, ...
        of each sequence over its pages (dflash_paged_attention).  Without row_start / row_count
        row i is the one new token of entry i.  max_rows: a host bound of row_count (default: all
        rows); a near one saves launches of empty work."""
        stride = self._rows(q, self.n_q_heads, "q")
        rows = q.shape[0]
        if out is None:
            out = torch.empty_like(q, memory_format=torch.contiguous_format)
        elif out.dtype is not q.dtype or out.shape != q.shape or not out.is_contiguous() or \
                out.get_device() != self._index:
            raise ValueError("out: a contiguous tensor like q is wanted")
        if seqs is None and row_count is None and row_start is None:
            n, a, s, c = rows, None, None, None
        else:
            n = self._entries(seqs, row_start, row_count, rows)
            a, s = self._ids(seqs, "seqs", n), self._ids(row_start, "row_start", n)
            c = self._ids(row_count, "row_count", n)
        if rows:
            self._run(self._lib.dflash_paged_attention, a, n, layer, q.data_ptr(), stride, s, c, rows,
                      rows if max_rows is None else max_rows, 1 if causal else 0, window, sinks, out.data_ptr())
        return out

    def __del__(self):
        try:
            if getattr(self, "handle", None):
                D.dflash_pool_release(self.handle)
                self.handle = None
        except Exception:
            pass
