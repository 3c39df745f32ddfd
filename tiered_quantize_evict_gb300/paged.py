"""The paged cache (``qe_pages_*`` in ``include/qe.h``): torch tensors in, library calls out.

``PagePool`` wraps the pool's key and value tensors, ``PageTable`` the sequences' page table, lengths
and reference counts, ``Rope`` the rotary positions of several axes.  A serving step:

    pool.resize(seqs, rows, new_len)                      # pages for the new tokens
    for layer in range(n_layers):
        q = pool.append(layer, k, v, q_start, seqs, rows=rows, q=q, rope=rope, positions=positions)
        o = pool.attend(layer, q, q_start, seqs, rows=rows)

and ``pool.gather(layer, seqs, 0, n)`` gives keys and values as ``QECache.qe_append`` takes them.

Work runs on the current stream of the pool's device; nothing waits for the GPU except ``check``.
Scratch comes from torch's allocator, call by call, so calls on several streams and captured
graphs never share it.
"""
from __future__ import annotations

import ctypes
import math
from typing import Optional, Sequence

import torch

from . import QE_ERR_DEVICE, QE_ERR_INVALID_ARG, QEError, load_library

QE_PAGES_ERR_PAGE, QE_PAGES_ERR_ROW, QE_PAGES_ERR_NO_PAGES, QE_PAGES_ERR_TIMEOUT = 1, 2, 4, 8

_P, _I, _L = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong
_I32 = torch.int32
_DTYPES = {torch.bfloat16: 0, torch.float16: 1}


class _Pages(ctypes.Structure):
    _fields_ = [("k", _P), ("v", _P), ("dtype", _I), ("device", _I), ("n_layers", _I), ("n_pages", _I), ("n_kv_heads", _I),
                ("page_size", _I), ("head_dim", _I), ("layer_stride", _L), ("page_stride", _L), ("head_stride", _L),
                ("token_stride", _L), ("err", _P)]


class _Table(ctypes.Structure):
    _fields_ = [("table", _P), ("kv_len", _P), ("refs", _P), ("row_stride", _L), ("n_rows", _I), ("max_pages", _I)]


class _Rope(ctypes.Structure):
    _fields_ = [("rot_dim", _I), ("halves", _I), ("n_axes", _I), ("axis", ctypes.c_byte * 64), ("inv_freq", ctypes.c_double * 64)]


class _Chunks(ctypes.Structure):
    _fields_ = [("q_start", _P), ("rows", _P), ("n_seqs", _I), ("total_q", _I)]


class _AppendArgs(ctypes.Structure):
    _fields_ = [("k", _P), ("v", _P), ("k_token_stride", _L), ("k_head_stride", _L), ("v_token_stride", _L),
                ("v_head_stride", _L), ("q", _P), ("q_out", _P), ("q_token_stride", _L), ("q_head_stride", _L),
                ("q_out_token_stride", _L), ("q_out_head_stride", _L), ("n_q_heads", _I), ("rope", _P), ("positions", _P),
                ("pos_stride", _L)]


class _AttendArgs(ctypes.Structure):
    _fields_ = [("q", _P), ("out", _P), ("lse", _P), ("q_token_stride", _L), ("q_head_stride", _L), ("out_token_stride", _L),
                ("out_head_stride", _L), ("n_q_heads", _I), ("causal", _I), ("max_q_len", _I), ("scale", ctypes.c_float)]


def _bad(msg: str) -> QEError:
    return QEError(QE_ERR_INVALID_ARG, msg)


def _ints(name: str, t: torch.Tensor, device, dims: int = 1):
    """Checks an int32 index tensor: device, type, contiguous."""
    if t.dtype is not _I32 or t.device != device or t.dim() != dims or not t.is_contiguous():
        raise _bad(f"{name} must be a contiguous {dims}-d int32 tensor on {device}")


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
        dev = table.device
        if table.dtype is not _I32 or table.dim() != 2 or (table.shape[1] > 1 and table.stride(1) != 1):
            raise _bad("table must be a 2-d int32 tensor with contiguous rows")
        _ints("kv_len", kv_len, dev)
        if kv_len.shape[0] != table.shape[0]:
            raise _bad("kv_len must have one entry per row of table")
        if refs is not None:
            _ints("refs", refs, dev)
        self.table, self.kv_len, self.refs = table, kv_len, refs
        self.device = dev
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
        n = ctypes.c_size_t()
        self._check(self._lib.qe_pages_attend_workspace(self._ref, ctypes.byref(n)))
        self._attend_bytes = n.value

    def _check(self, st: int):
        if st:
            raise QEError(st, self._lib.qe_last_error(None).decode())

    def _stream(self) -> int:
        return torch.cuda.current_stream(self.device).cuda_stream

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

    def _seqs(self, seqs: PageTable, refs: bool = False):
        if seqs.device != self.device:
            raise _bad(f"the page table is on {seqs.device}, the pool on {self.device}")
        if refs and (seqs.refs is None or seqs.refs.shape[0] != self.n_pages):
            raise _bad("the page table needs refs with one entry per page of the pool")
        return seqs._ref

    def _chunks(self, q_start, rows, total):
        _ints("q_start", q_start, self.device)
        n = q_start.shape[0] - 1
        if rows is not None:
            _ints("rows", rows, self.device)
            if rows.shape[0] != n:
                raise _bad("q_start must have one entry more than rows")
        return _Chunks(q_start.data_ptr(), rows.data_ptr() if rows is not None else None, n, total)

    def _tokens(self, name, t, total, heads):
        """Checks a [total][heads][head_dim] tensor of the pool's type."""
        if t.dtype is not self.dtype or t.device != self.device or t.dim() != 3 or t.shape[0] != total or t.shape[2] != self.head_dim \
                or (heads and t.shape[1] != heads) or t.stride(2) != 1:
            raise _bad(f"{name} must be a {self.dtype} tensor [{total}, {heads or 'heads'}, {self.head_dim}] on {self.device}, channels contiguous")

    # ---------------------------------------------------------------- the path
    def append(self, layer: int, k: torch.Tensor, v: torch.Tensor, q_start: torch.Tensor, seqs: PageTable, *,
               rows: Optional[torch.Tensor] = None, q: Optional[torch.Tensor] = None, rope: Optional[Rope] = None,
               positions: Optional[torch.Tensor] = None, q_out: Optional[torch.Tensor] = None) -> Optional[torch.Tensor]:
        """qe_pages_append: rotate q and k, write k and v to their pages; returns the rotated q (q_out, or a new tensor).

        k, v [total][n_kv_heads][head_dim], q [total][n_q_heads][head_dim]; q_start int32 [n + 1]; positions int32
        [n_axes][total] (or [total] for one axis), default the cache positions."""
        total = k.shape[0]
        self._tokens("k", k, total, self.n_kv_heads)
        self._tokens("v", v, total, self.n_kv_heads)
        hq, qp, op, qs, os = 0, None, None, (0, 0), (0, 0)
        if q is not None:
            self._tokens("q", q, total, 0)
            hq = q.shape[1]
            if q_out is None:
                q_out = torch.empty(total, hq, self.head_dim, dtype=self.dtype, device=self.device)
            else:
                self._tokens("q_out", q_out, total, hq)
            qp, op, qs, os = q.data_ptr(), q_out.data_ptr(), q.stride(), q_out.stride()
        elif q_out is not None:
            raise _bad("q_out without q")
        pp, pst = None, 0
        if positions is not None:
            if rope is None:
                raise _bad("positions without rope")
            if positions.dtype is not _I32 or positions.device != self.device or positions.shape[-1] != total or \
                    positions.stride(-1) != 1 and total > 1 or positions.dim() > 2 or \
                    (positions.shape[0] if positions.dim() == 2 else 1) != rope.n_axes:
                raise _bad(f"positions must be int32 [{rope.n_axes}, {total}] on {self.device}, tokens contiguous")
            pp, pst = positions.data_ptr(), positions.stride(0) if positions.dim() == 2 else 0
        c = self._chunks(q_start, rows, total)
        ks, vs = k.stride(), v.stride()
        a = _AppendArgs(k.data_ptr(), v.data_ptr(), ks[0], ks[1], vs[0], vs[1], qp, op, qs[0], qs[1], os[0], os[1], hq,
                        rope._addr if rope is not None else None, pp, pst)
        self._check(self._lib.qe_pages_append(self._ref, layer, self._seqs(seqs), ctypes.byref(c), ctypes.byref(a), self._stream()))
        return q_out

    def attend(self, layer: int, q: torch.Tensor, q_start: torch.Tensor, seqs: PageTable, *, rows: Optional[torch.Tensor] = None,
               scale: Optional[float] = None, causal: bool = True, max_q_len: int = 0, out: Optional[torch.Tensor] = None,
               return_lse: bool = False):
        """qe_pages_attend: q [total][n_q_heads][head_dim] over the rows' cached tokens; returns out, or (out, lse
        [total][n_q_heads] float32) with return_lse.  scale defaults to head_dim ** -0.5."""
        total, hq = q.shape[0], q.shape[1]
        self._tokens("q", q, total, 0)
        if out is None:
            out = torch.empty(total, hq, self.head_dim, dtype=self.dtype, device=self.device)
        else:
            self._tokens("out", out, total, hq)
        lse = torch.empty(total, hq, dtype=torch.float32, device=self.device) if return_lse else None
        ws = torch.empty(self._attend_bytes, dtype=torch.uint8, device=self.device)
        c = self._chunks(q_start, rows, total)
        qs, os = q.stride(), out.stride()
        a = _AttendArgs(q.data_ptr(), out.data_ptr(), lse.data_ptr() if return_lse else None, qs[0], qs[1], os[0], os[1], hq,
                        1 if causal else 0, max_q_len, 1.0 / math.sqrt(self.head_dim) if scale is None else scale)
        self._check(self._lib.qe_pages_attend(self._ref, layer, self._seqs(seqs), ctypes.byref(c), ctypes.byref(a), ws.data_ptr(),
                                              self._attend_bytes, self._stream()))
        return (out, lse) if return_lse else out

    # ---------------------------------------------------------------- managing pages
    def _workspace(self, ref, n):
        b = ctypes.c_size_t()
        self._check(self._lib.qe_pages_manage_workspace(self._ref, ref, n, ctypes.byref(b)))
        return torch.empty(b.value, dtype=torch.uint8, device=self.device), b.value

    def _manage(self, fn, seqs, a, b, names):
        ref = self._seqs(seqs, refs=True)
        _ints(names[0], a, self.device)
        _ints(names[1], b, self.device)
        if a.shape[0] != b.shape[0]:
            raise _bad(f"{names[0]} and {names[1]} must have one entry each")
        ws, nb = self._workspace(ref, a.shape[0])
        self._check(fn(self._ref, ref, a.data_ptr(), b.data_ptr(), a.shape[0], ws.data_ptr(), nb, self._stream()))

    def resize(self, seqs: PageTable, rows: torch.Tensor, new_len: torch.Tensor):
        """qe_pages_resize: row rows[i] gets length new_len[i]; pages are taken or given back."""
        self._manage(self._lib.qe_pages_resize, seqs, rows, new_len, ("rows", "new_len"))

    def free(self, seqs: PageTable, rows: torch.Tensor):
        """Free whole rows: qe_pages_resize to length 0."""
        self.resize(seqs, rows, torch.zeros_like(rows))

    def fork(self, seqs: PageTable, src: torch.Tensor, dst: torch.Tensor):
        """qe_pages_fork: empty row dst[i] becomes a copy of row src[i], sharing its full pages."""
        self._manage(self._lib.qe_pages_fork, seqs, src, dst, ("src", "dst"))

    def compact(self, seqs: PageTable, *, table_out: Optional[torch.Tensor] = None, refs_out: Optional[torch.Tensor] = None,
                n_live: Optional[torch.Tensor] = None):
        """qe_pages_compact: live pages move to the front of the pool; in place unless table_out / refs_out are given."""
        ref = self._seqs(seqs, refs=True)
        if table_out is not None and (table_out.dtype is not _I32 or table_out.device != self.device or
                                      table_out.shape != seqs.table.shape or table_out.stride() != seqs.table.stride()):
            raise _bad("table_out must be like the page table")
        if refs_out is not None:
            _ints("refs_out", refs_out, self.device)
            if refs_out.shape[0] != self.n_pages:
                raise _bad("refs_out must have one entry per page")
        if n_live is not None:
            _ints("n_live", n_live, self.device)
            if n_live.shape[0] != 1:
                raise _bad("n_live must have one entry")
        ws, nb = self._workspace(ref, 0)
        self._check(self._lib.qe_pages_compact(self._ref, ref, *(t.data_ptr() if t is not None else None
                                                                for t in (table_out, refs_out, n_live)), ws.data_ptr(), nb, self._stream()))

    def copy(self, src: torch.Tensor, dst: torch.Tensor):
        """qe_pages_copy: page src[i] to page dst[i], all layers."""
        _ints("src", src, self.device)
        _ints("dst", dst, self.device)
        if src.shape[0] != dst.shape[0]:
            raise _bad("src and dst must have one entry each")
        self._check(self._lib.qe_pages_copy(self._ref, src.data_ptr(), dst.data_ptr(), src.shape[0], self._stream()))

    def gather(self, layer: int, seqs: PageTable, start: int, n_tokens: int, *, rows: Optional[torch.Tensor] = None,
               out: Optional[Sequence[torch.Tensor]] = None):
        """qe_pages_gather: (k, v), each [n_rows][n_kv_heads][n_tokens][head_dim], the layout ``QECache.qe_append`` takes."""
        n = seqs.table.shape[0]
        if rows is not None:
            _ints("rows", rows, self.device)
            n = rows.shape[0]
        shape = (n, self.n_kv_heads, max(0, n_tokens), self.head_dim)
        if out is None:
            out = [torch.empty(shape, dtype=self.dtype, device=self.device) for _ in range(2)]
        for t in out:
            if t.dtype is not self.dtype or t.device != self.device or tuple(t.shape) != shape or not t.is_contiguous():
                raise _bad(f"out must be two contiguous {self.dtype} tensors {list(shape)} on {self.device}")
        self._check(self._lib.qe_pages_gather(self._ref, layer, self._seqs(seqs), rows.data_ptr() if rows is not None else None, n, start,
                                              n_tokens, out[0].data_ptr(), out[1].data_ptr(), self._stream()))
        return out[0], out[1]
