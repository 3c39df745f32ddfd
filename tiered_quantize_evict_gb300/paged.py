"""The paged cache (``qe_pages_*`` in ``include/qe.h``): torch tensors in, library calls out.

``PagePool`` wraps the pool's key and value tensors, ``PageTable`` the sequences' page table, lengths
and reference counts, ``Rope`` the rotary positions of several axes.  A serving step:

    pool.resize(seqs, rows, new_len)                      # pages for the new tokens
    for layer in range(n_layers):
        q = pool.append(layer, k, v, q_start, seqs, rows=rows, q=q, rope=rope, positions=positions)
        o = pool.attend(layer, q, q_start, seqs, rows=rows, max_q_len=longest)   # (the longest chunk, or 0 if it is not known)

and ``pool.gather(layer, seqs, 0, n)`` gives keys and values in the layout ``QECache.qe_append`` takes: of a bf16 pool, for
rows that all have n tokens (shorter ones are filled up with zeros), and for a cache with ``rope_theta`` 0 (``append`` stores rotated keys).
Nothing here carries a gradient: tensors are read and written by address, whatever autograd would record.

Work runs on the current stream of the pool's device; nothing waits for the GPU except ``check``.
A pool keeps a scratch buffer for each stream it is used on; a call that is captured into a graph
takes its own from the graph's memory, so neither streams nor graphs share any.
"""
from __future__ import annotations

import ctypes
import math
import struct
import threading
from typing import Optional, Sequence

import torch

from . import QE_ERR_DEVICE, QE_ERR_INVALID_ARG, QEError, load_library

QE_PAGES_ERR_PAGE, QE_PAGES_ERR_ROW, QE_PAGES_ERR_NO_PAGES, QE_PAGES_ERR_TIMEOUT = 1, 2, 4, 8

_P, _I, _L = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong
_I32, _DENSE = torch.int32, torch.contiguous_format
_DTYPES = {torch.bfloat16: 0, torch.float16: 1}


class _Pages(ctypes.Structure):
    _fields_ = [("k", _P), ("v", _P), ("dtype", _I), ("device", _I), ("n_layers", _I), ("n_pages", _I), ("n_kv_heads", _I),
                ("page_size", _I), ("head_dim", _I), ("layer_stride", _L), ("page_stride", _L), ("head_stride", _L),
                ("token_stride", _L), ("err", _P)]


class _Table(ctypes.Structure):
    _fields_ = [("table", _P), ("kv_len", _P), ("refs", _P), ("row_stride", _L), ("n_rows", _I), ("max_pages", _I)]


class _Rope(ctypes.Structure):
    _fields_ = [("rot_dim", _I), ("halves", _I), ("n_axes", _I), ("axis", ctypes.c_byte * 64), ("inv_freq", ctypes.c_double * 64)]


# qe_chunks, qe_pages_append_args and qe_pages_attend_args, packed call by call (native sizes and alignment; a ctypes
# structure costs three times as much to fill)
_CHUNKS = struct.Struct("@PPii0P")
_APPEND = struct.Struct("@PPqqqqPPqqqqiPPq0P")
_ATTEND = struct.Struct("@PPPqqqqiiif0P")

try:   # the raw handle without a Stream object around it
    _raw_stream = torch._C._cuda_getCurrentRawStream
except AttributeError:
    def _raw_stream(index):
        return torch.cuda.current_stream(index).cuda_stream
_get_device, _capturing = torch.cuda.current_device, torch.cuda.is_current_stream_capturing


def _bad(msg: str) -> QEError:
    return QEError(QE_ERR_INVALID_ARG, msg)


def _ints(name: str, t: torch.Tensor, index: int) -> int:
    """Checks an int32 index tensor (1-d, contiguous, on the device of that index); its length."""
    if t.dtype is not _I32 or t.get_device() != index or t.dim() != 1 or not t.is_contiguous():
        raise _bad(f"{name} must be a contiguous 1-d int32 tensor on cuda:{index}")
    return t.shape[0]


class Rope:
    """Rotary positions: channel pair i turns by positions[axis[i]] * inv_freq[i].

    theta: inv_freq[i] = theta ** (-2 i / rot_dim), unless inv_freq (rot_dim / 2 numbers) is given.
    sections: pairs of each axis, in order (their sum is rot_dim / 2); or axis: the axis of every pair.
    halves: pairs are channels (i, i + rot_dim / 2) instead of (2i, 2i + 1).
    """

    def __init__(self, head_dim: int, theta: float = 10000.0, *, rot_dim: Optional[int] = None,
                 sections: Optional[Sequence[int]] = None, axis: Optional[Sequence[int]] = None,
                 inv_freq: Optional[Sequence[float]] = None, halves: bool = False):
        rot = head_dim if rot_dim is None else int(rot_dim)
        if head_dim not in (64, 128) or rot < 0 or rot > head_dim or rot % 2:
            raise _bad("head_dim must be 64 or 128 and rot_dim even, 0 .. head_dim")
        n = rot // 2
        if sections is not None and axis is not None:
            raise _bad("give sections or axis, not both")
        if sections is not None:
            axis = [a for a, c in enumerate(sections) for _ in range(int(c))]
        axis = [0] * n if axis is None else [int(a) for a in axis]
        if inv_freq is None:
            if not (theta > 0):
                raise _bad("theta must be positive")
            inv_freq = [float(theta) ** (-2.0 * i / rot) for i in range(n)]
        inv_freq = [float(f) for f in inv_freq]
        if len(axis) != n or len(inv_freq) != n:
            raise _bad(f"{n} channel pairs, {len(axis)} axes, {len(inv_freq)} frequencies")
        self.n_axes = max(len(sections) if sections is not None else 1, max(axis, default=0) + 1)
        if min(axis, default=0) < 0 or not 1 <= self.n_axes <= 8:
            raise _bad("axes are 0 .. 7")
        self._s = _Rope(rot, 1 if halves else 0, self.n_axes, (ctypes.c_byte * 64)(*axis), (ctypes.c_double * 64)(*inv_freq))
        self._addr = ctypes.addressof(self._s)


class PageTable:
    """Sequences: table [n_rows][max_pages], kv_len [n_rows], refs [n_pages] (int32; refs where pages are managed)."""

    def __init__(self, table: torch.Tensor, kv_len: torch.Tensor, refs: Optional[torch.Tensor] = None):
        dev = table.get_device()
        if table.dtype is not _I32 or table.dim() != 2 or (table.shape[1] > 1 and table.stride(1) != 1):
            raise _bad("table must be a 2-d int32 tensor with contiguous rows")
        if _ints("kv_len", kv_len, dev) != table.shape[0]:
            raise _bad("kv_len must have one entry per row of table")
        if refs is not None:
            _ints("refs", refs, dev)
        self.table, self.kv_len, self.refs = table, kv_len, refs
        self._index, self._n_refs = dev, refs.shape[0] if refs is not None else -1
        self._shape = tuple(table.shape)
        self._s = _Table(table.data_ptr(), kv_len.data_ptr(), refs.data_ptr() if refs is not None else None, table.stride(0),
                         table.shape[0], table.shape[1])
        self._ref = ctypes.byref(self._s)

    @classmethod
    def empty(cls, n_rows: int, max_pages: int, n_pages: int, device="cuda") -> "PageTable":
        """Rows without tokens over a pool of free pages."""
        return cls(torch.full((n_rows, max_pages), -1, dtype=_I32, device=device),
                   torch.zeros(n_rows, dtype=_I32, device=device), torch.zeros(n_pages, dtype=_I32, device=device))


class PagePool:
    """Pages of keys and values: k, v [n_layers, n_pages, n_kv_heads, page_size, head_dim], bf16 or fp16, with the
    same strides (any, the channels contiguous)."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor):
        if not k.is_cuda or k.device != v.device or k.dtype != v.dtype or k.dtype not in _DTYPES:
            raise _bad("k and v must be bf16 or fp16 CUDA tensors of one type and device")
        if k.dim() != 5 or k.shape != v.shape or k.stride() != v.stride() or k.stride(4) != 1:
            raise _bad("k and v must be [n_layers, n_pages, n_kv_heads, page_size, head_dim] with equal strides, channels contiguous")
        self._lib = load_library()
        self.k, self.v, self.device, self.dtype = k, v, k.device, k.dtype
        self.n_layers, self.n_pages, self.n_kv_heads, self.page_size, self.head_dim = k.shape
        self.err = torch.zeros(1, dtype=_I32, device=k.device)
        st = k.stride()
        self._s = _Pages(k.data_ptr(), v.data_ptr(), _DTYPES[k.dtype], k.device.index, *k.shape, st[0], st[1], st[2], st[3],
                         self.err.data_ptr())
        self._ref = ctypes.byref(self._s)
        self._index, self._scale = k.device.index, 1.0 / math.sqrt(k.shape[4])
        self._bytes = {}       # workspace sizes by table shape and entries
        self._kept = {}        # scratch by stream
        self._lock = threading.Lock()

    def _check(self, st: int):
        if st:
            raise QEError(st, self._lib.qe_last_error(None).decode())

    def _need(self, seqs: PageTable, n: int) -> int:
        """Bytes of workspace of attend (n < 0) or of managing n entries, with tables of this shape."""
        key = (seqs._shape, n)
        need = self._bytes.get(key)
        if need is None:
            b = ctypes.c_size_t()
            if n < 0:
                self._check(self._lib.qe_pages_attend_workspace(self._ref, seqs._ref, ctypes.byref(b)))
            else:
                self._check(self._lib.qe_pages_manage_workspace(self._ref, seqs._ref, n, ctypes.byref(b)))
            need = self._bytes[key] = b.value
        return need

    def _scratch(self, need: int, stream: int) -> torch.Tensor:
        """need bytes for work on this stream (held under the lock until the call is enqueued)."""
        if _get_device() != self._index or _capturing():
            return torch.empty(need, dtype=torch.uint8, device=self.device)
        buf = self._kept.get(stream)
        if buf is None or buf.shape[0] < need:
            buf = self._kept[stream] = torch.empty(need, dtype=torch.uint8, device=self.device)
        return buf

    def check(self):
        """Waits for the current stream and raises if a call met a bad page, row or length, or ran out of pages;
        clears the record."""
        bits = int(self.err.item())
        if bits:
            self.err.zero_()
            names = [n for b, n in ((QE_PAGES_ERR_PAGE, "a page index or reference count out of range"),
                                    (QE_PAGES_ERR_ROW, "a row, length or q_start out of range, or a row named twice"),
                                    (QE_PAGES_ERR_NO_PAGES, "not enough free pages (nothing was changed)"),
                                    (QE_PAGES_ERR_TIMEOUT, "a bounded device wait expired")) if bits & b]
            raise QEError(QE_ERR_DEVICE, "; ".join(names))

    def _seqs(self, seqs: PageTable):
        if seqs._index != self._index:
            raise _bad(f"the page table is on {seqs.table.device}, the pool on {self.device}")
        return seqs._ref

    def _layer(self, layer):
        # (here, not in the call: ctypes cuts a number to a C int)
        if not 0 <= layer < self.n_layers:
            raise _bad(f"layer {layer} out of range")
        return layer

    def _chunks(self, q_start, rows, total):
        n = _ints("q_start", q_start, self._index) - 1
        if rows is None:
            return _CHUNKS.pack(q_start.data_ptr(), 0, n, total)
        if _ints("rows", rows, self._index) != n:
            raise _bad("q_start must have one entry more than rows")
        return _CHUNKS.pack(q_start.data_ptr(), rows.data_ptr(), n, total)

    def _tokens(self, name, t, total, heads):
        """Checks a [total][heads][head_dim] tensor of the pool's type; its strides."""
        if t.dtype is not self.dtype or t.get_device() != self._index or t.shape != (total, heads, self.head_dim):
            raise _bad(f"{name} must be a {self.dtype} tensor [{total}, {heads}, {self.head_dim}] on {self.device}")
        st = t.stride()
        if st[2] != 1 and total > 0:   # (numpy's empty arrays have strides of 0)
            raise _bad(f"{name} must have contiguous channels")
        return st

    # ---------------------------------------------------------------- the path
    def append(self, layer: int, k: torch.Tensor, v: torch.Tensor, q_start: torch.Tensor, seqs: PageTable, *,
               rows: Optional[torch.Tensor] = None, q: Optional[torch.Tensor] = None, rope: Optional[Rope] = None,
               positions: Optional[torch.Tensor] = None, q_out: Optional[torch.Tensor] = None) -> Optional[torch.Tensor]:
        """qe_pages_append: rotate q and k, write k and v to their pages; returns the rotated q (q_out, or a new tensor).

        k, v [total][n_kv_heads][head_dim], q [total][n_q_heads][head_dim]; q_start int32 [n + 1]; positions int32
        [n_axes][total] (or [total] for one axis), default the cache positions."""
        total = k.shape[0] if k.dim() else 0
        ks = self._tokens("k", k, total, self.n_kv_heads)
        vs = self._tokens("v", v, total, self.n_kv_heads)
        hq = qp = op = pp = pst = 0
        qs = os = (0, 0)
        if q is not None:
            hq = q.shape[1] if q.dim() == 3 else 0
            qs = self._tokens("q", q, total, hq)
            if q_out is None:
                q_out = torch.empty_like(q, memory_format=_DENSE)
                os = (hq * self.head_dim, self.head_dim)
            else:
                os = self._tokens("q_out", q_out, total, hq)
            qp, op = q.data_ptr(), q_out.data_ptr()
        elif q_out is not None:
            raise _bad("q_out without q")
        if positions is not None:
            if rope is None:
                raise _bad("positions without rope")
            ps = positions.stride()
            if positions.dtype is not _I32 or positions.get_device() != self._index or \
                    positions.shape != ((rope.n_axes, total) if len(ps) == 2 or rope.n_axes > 1 else (total,)) or ps[-1] != 1 and total > 1:
                raise _bad(f"positions must be int32 [{rope.n_axes}, {total}] on {self.device}, tokens contiguous")
            pp, pst = positions.data_ptr(), ps[0]
        st = self._lib.qe_pages_append(
            self._ref, self._layer(layer), self._seqs(seqs), self._chunks(q_start, rows, total),
            _APPEND.pack(k.data_ptr(), v.data_ptr(), ks[0], ks[1], vs[0], vs[1], qp, op, qs[0], qs[1], os[0], os[1], hq,
                         rope._addr if rope is not None else 0, pp, pst), _raw_stream(self._index))
        if st:
            self._check(st)
        return q_out

    def attend(self, layer: int, q: torch.Tensor, q_start: torch.Tensor, seqs: PageTable, *, rows: Optional[torch.Tensor] = None,
               scale: Optional[float] = None, causal: bool = True, max_q_len: int = 0, out: Optional[torch.Tensor] = None,
               return_lse: bool = False):
        """qe_pages_attend: q [total][n_q_heads][head_dim] over the rows' cached tokens; returns out, or (out, lse
        [total][n_q_heads] float32) with return_lse.  scale defaults to head_dim ** -0.5."""
        total, hq = q.shape[:2] if q.dim() == 3 else (0, 0)
        qs = self._tokens("q", q, total, hq)
        if out is None:
            out = torch.empty_like(q, memory_format=_DENSE)
            os = (hq * self.head_dim, self.head_dim)
        else:
            os = self._tokens("out", out, total, hq)
        lse = torch.empty(total, hq, dtype=torch.float32, device=self.device) if return_lse else None
        ref, c = self._seqs(seqs), self._chunks(q_start, rows, total)
        if not 0 <= max_q_len < 2 ** 31:
            raise _bad(f"max_q_len {max_q_len} out of range")
        a = _ATTEND.pack(q.data_ptr(), out.data_ptr(), lse.data_ptr() if return_lse else 0, qs[0], qs[1], os[0], os[1], hq,
                         1 if causal else 0, max_q_len, self._scale if scale is None else scale)
        need, stream, layer = self._need(seqs, -1), _raw_stream(self._index), self._layer(layer)
        if need:
            with self._lock:
                ws = self._scratch(need, stream)
                st = self._lib.qe_pages_attend(self._ref, layer, ref, c, a, ws.data_ptr(), need, stream)
        else:
            st = self._lib.qe_pages_attend(self._ref, layer, ref, c, a, None, 0, stream)
        if st:
            self._check(st)
        return (out, lse) if return_lse else out

    # ---------------------------------------------------------------- managing pages
    def _refs(self, seqs):
        if seqs._n_refs != self.n_pages:
            raise _bad("the page table needs refs with one entry per page of the pool")
        return self._seqs(seqs)

    def _manage(self, fn, seqs, a, b, names):
        ref = self._refs(seqs)
        n = _ints(names[0], a, self._index)
        if b is not None and _ints(names[1], b, self._index) != n:
            raise _bad(f"{names[0]} and {names[1]} must have one entry each")
        need, stream = self._need(seqs, n), _raw_stream(self._index)
        with self._lock:
            ws = self._scratch(need, stream)
            st = fn(self._ref, ref, a.data_ptr(), b.data_ptr() if b is not None else None, n, ws.data_ptr(), need, stream)
        if st:
            self._check(st)

    def resize(self, seqs: PageTable, rows: torch.Tensor, new_len: torch.Tensor):
        """qe_pages_resize: row rows[i] gets length new_len[i]; pages are taken or given back."""
        self._manage(self._lib.qe_pages_resize, seqs, rows, new_len, ("rows", "new_len"))

    def free(self, seqs: PageTable, rows: torch.Tensor):
        """Free whole rows: qe_pages_resize to length 0."""
        self._manage(self._lib.qe_pages_resize, seqs, rows, None, ("rows", "new_len"))

    def fork(self, seqs: PageTable, src: torch.Tensor, dst: torch.Tensor):
        """qe_pages_fork: empty row dst[i] becomes a copy of row src[i], sharing its full pages."""
        self._manage(self._lib.qe_pages_fork, seqs, src, dst, ("src", "dst"))

    def compact(self, seqs: PageTable, *, table_out: Optional[torch.Tensor] = None, refs_out: Optional[torch.Tensor] = None,
                n_live: Optional[torch.Tensor] = None):
        """qe_pages_compact: live pages move to the front of the pool; in place unless table_out / refs_out are given."""
        ref = self._refs(seqs)
        if table_out is not None and (table_out.dtype is not _I32 or table_out.get_device() != self._index or
                                      table_out.shape != seqs.table.shape or table_out.stride() != seqs.table.stride()):
            raise _bad("table_out must be like the page table")
        if refs_out is not None and _ints("refs_out", refs_out, self._index) != self.n_pages:
            raise _bad("refs_out must have one entry per page")
        if n_live is not None and _ints("n_live", n_live, self._index) != 1:
            raise _bad("n_live must have one entry")
        need, stream = self._need(seqs, 0), _raw_stream(self._index)
        with self._lock:
            ws = self._scratch(need, stream)
            st = self._lib.qe_pages_compact(self._ref, ref, *(t.data_ptr() if t is not None else None for t in (table_out, refs_out, n_live)),
                                            ws.data_ptr(), need, stream)
        if st:
            self._check(st)

    def copy(self, src: torch.Tensor, dst: torch.Tensor):
        """qe_pages_copy: page src[i] to page dst[i], all layers."""
        n = _ints("src", src, self._index)
        if _ints("dst", dst, self._index) != n:
            raise _bad("src and dst must have one entry each")
        self._check(self._lib.qe_pages_copy(self._ref, src.data_ptr(), dst.data_ptr(), n, _raw_stream(self._index)))

    def gather(self, layer: int, seqs: PageTable, start: int, n_tokens: int, *, rows: Optional[torch.Tensor] = None,
               out: Optional[Sequence[torch.Tensor]] = None):
        """qe_pages_gather: (k, v), each [n_rows][n_kv_heads][n_tokens][head_dim], the layout ``QECache.qe_append`` takes (bf16
        rows of one length); zeros behind a row's length."""
        n = seqs._shape[0] if rows is None else _ints("rows", rows, self._index)
        if start < 0 or n_tokens < 0 or start + n_tokens > 2 ** 31 - 257:
            raise _bad("start and n_tokens must be >= 0, start + n_tokens below 2^31 - 256")
        shape = (n, self.n_kv_heads, n_tokens, self.head_dim)
        if out is None:
            k = torch.empty(shape, dtype=self.dtype, device=self.device)
            v = torch.empty_like(k)
        else:
            k, v = out
            for t in (k, v):
                if t.dtype is not self.dtype or t.get_device() != self._index or t.shape != shape or not t.is_contiguous():
                    raise _bad(f"out must be two contiguous {self.dtype} tensors {list(shape)} on {self.device}")
        st = self._lib.qe_pages_gather(self._ref, self._layer(layer), self._seqs(seqs), rows.data_ptr() if rows is not None else None, n, start,
                                       n_tokens, k.data_ptr(), v.data_ptr(), _raw_stream(self._index))
        if st:
            self._check(st)
        return k, v
