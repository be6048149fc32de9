"""Dense attention over a paged cache: binding of ``dhs_page_*`` and
``dhs_prompt_attend`` (see include/dhs.h for what each call computes).

Tensors are checked for type, shape, layout and device and passed on; nothing
is copied, cast or allocated by a call.  A call runs on the tensors' device and
on ``stream`` (default: torch's current stream there); as with every call of the
library its tensors must stay alive until the stream has passed it.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

PAGE_BF16, PAGE_INT8, PAGE_E4M3 = 0, 1, 2
_KIND = {torch.bfloat16: PAGE_BF16, torch.int8: PAGE_INT8, torch.float8_e4m3fn: PAGE_E4M3}
_DTYPE = {v: k for k, v in _KIND.items()}
_CHECK = {1: "a length or offset outside its range", 2: "a page outside the cache",
          4: "a bounded wait that ran out"}
_SITE = {1: "dhs_page_write", 2: "dhs_page_read", 3: "dhs_page_attend", 4: "dhs_prompt_attend"}


_Strides4, _Strides6 = ctypes.c_int64 * 4, ctypes.c_int64 * 6


class Pages(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("n_pages", ctypes.c_int64),
                ("page_rows", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("kind", ctypes.c_int32)]


# A decode step makes several calls of a few microseconds each, so what a call does on
# the host counts: the current stream's handle and device without torch's wrappers, no
# array of strides for contiguous rows, no context where the device is the current one
# (7.9 -> 6.4 us for a write from Python, of which the launch is 2).
try:
    from torch._C import _cuda_getCurrentRawStream as _current_stream
    from torch._C import _cuda_getDevice as _current_device
except ImportError:
    _current_device = torch.cuda.current_device

    def _current_stream(index):
        return torch.cuda.current_stream(index).cuda_stream

_BF16, _I32, _F32 = torch.bfloat16, torch.int32, torch.float32


def _lib():
    from . import load
    return load()


def _raise(code, what):
    from . import DhsError
    raise DhsError(code, what)


def _bad(name, t, dtype, shape, index):
    """The complaint about a tensor that is not a contiguous ``dtype`` of ``shape``
    (None: any) on CUDA device ``index``."""
    raise ValueError("%s: contiguous %s%s on cuda:%s expected, not %s %s %s on %s" % (
        name, dtype, "" if shape is None else " %s" % (tuple(shape),), index,
        "contiguous" if t.is_contiguous() else "strided", t.dtype, tuple(t.shape), t.device))


def _plain(t, name, dtype, shape, index):
    if not (t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.get_device() == index):
        _bad(name, t, dtype, shape, index)
    return t.data_ptr()


def _table(t, n, index):
    if not (t.dtype is _I32 and t.dim() == 2 and t.shape[0] == n and t.is_contiguous()
            and t.get_device() == index):
        _bad("page_table", t, _I32, (n, "width"), index)
    return t.data_ptr()


def _rows(t, name, index):
    """Tokens, heads, elements, token and head stride of a packed bf16 tensor."""
    if not (t.dtype is _BF16 and t.dim() == 3 and t.get_device() == index):
        raise ValueError("%s: bf16 [tokens, heads, dim] on cuda:%s expected, not %s %s on %s"
                         % (name, index, t.dtype, tuple(t.shape), t.device))
    n, h, d = t.shape
    st, sh, sd = t.stride()
    if sd != 1 and d > 1 and n and h:
        raise ValueError("%s: the elements of a head must be contiguous" % name)
    # a stride that no second token or head uses may be anything
    return n, h, d, (st if n > 1 else h * d), (sh if h > 1 else d)


def _space(t, index):
    if t is None:
        return None, 0
    if not (t.is_contiguous() and t.get_device() == index):
        raise ValueError("workspace: contiguous, on cuda:%s expected" % index)
    return t.data_ptr(), t.numel() * t.element_size()


def _on(index):
    """The context in which a call runs on device ``index``."""
    if index < 0:
        raise ValueError("CUDA tensors expected")
    return torch.cuda.device(index)


def _raw(stream, index):
    if stream is None:
        return _current_stream(index)
    return stream if isinstance(stream, int) else stream.cuda_stream


def check_errors(errors=None, stream=None):
    """Waits for ``stream``, raises DhsError (code 5) if a call recorded a bad
    page, length or offset in ``errors`` (int32[2]), and clears the record.
    Without ``errors``: what :func:`prompt_attend` calls without a record of their own
    found on the current device."""
    if errors is None:
        found = (ctypes.c_int32 * 2)()
        rc = _lib().dhs_prompt_errors(found, _raw(stream, _current_device()))
        if rc:
            _raise(rc, "dhs_prompt_errors")
        return _found(*found)
    with _on(errors.get_device()):
        s = torch.cuda.current_stream() if stream is None else stream
        if isinstance(s, int):
            s = torch.cuda.ExternalStream(s)
        with torch.cuda.stream(s):
            code, site = errors.tolist()
            if code:
                errors.zero_()
    _found(code, site)


def _found(code, site):
    if code:
        _raise(5, "%s: %s" % (_SITE.get(site, "?"), _CHECK.get(code, "check %d" % code)))


class PageCache:
    """A paged cache over caller-owned tensors: ``k`` and ``v`` [n_pages, kv_heads,
    page_rows, head_dim] of bfloat16, int8 or float8_e4m3fn and, for the 8-bit
    kinds, fp32 ``k_scale`` and ``v_scale`` [n_pages, kv_heads, page_rows].

    ``errors`` (int32[2] on the device) collects what the kernels' checks find;
    :meth:`check` raises it.
    """

    def __init__(self, k, v, k_scale=None, v_scale=None, errors=None):
        if k.dtype not in _KIND:
            raise ValueError("a cache of %s is not supported" % k.dtype)
        if k.dim() != 4:
            raise ValueError("k: [n_pages, kv_heads, page_rows, head_dim] expected, not %s"
                             % (tuple(k.shape),))
        self.device, self._index = k.device, k.get_device()
        _on(self._index)
        self.kind = _KIND[k.dtype]
        self.n_pages, self.kv_heads, self.page_rows, self.head_dim = k.shape
        if (self.kind == PAGE_BF16) != (k_scale is None and v_scale is None):
            raise ValueError("an 8-bit cache needs scales, a bf16 cache has none")
        ptr = [_plain(t, name, k.dtype, k.shape, self._index) for t, name in ((k, "k"), (v, "v"))]
        ptr += [None if t is None else _plain(t, name, _F32, k.shape[:3], self._index)
                for t, name in ((k_scale, "k_scale"), (v_scale, "v_scale"))]
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.errors = torch.zeros(2, dtype=_I32, device=self.device) if errors is None else errors
        self._err = _plain(self.errors, "errors", _I32, (2,), self._index)
        self._desc = Pages(*ptr, self.n_pages, self.page_rows, self.kv_heads, self.head_dim, self.kind)
        self._ref = ctypes.byref(self._desc)
        self._lib = _lib()

    @classmethod
    def empty(cls, n_pages: int, page_rows: int, kv_heads: int, head_dim: int,
              kind: int = PAGE_BF16, device="cuda"):
        """A cache of zeros in new tensors."""
        shape = (n_pages, kv_heads, page_rows, head_dim)
        k, v = (torch.zeros(shape, dtype=torch.uint8, device=device).view(_DTYPE[kind])
                if kind != PAGE_BF16 else torch.zeros(shape, dtype=torch.bfloat16, device=device)
                for _ in range(2))
        ks, vs = ((torch.zeros(shape[:3], dtype=torch.float32, device=device) for _ in range(2))
                  if kind != PAGE_BF16 else (None, None))
        return cls(k, v, ks, vs)

    def nbytes(self) -> int:
        return sum(t.numel() * t.element_size()
                   for t in (self.k, self.v, self.k_scale, self.v_scale) if t is not None)

    def _copy(self, fn, what, k, v, cu, seq_lens, page_table, stream):
        ix = self._index
        if _current_device() != ix:
            with _on(ix):
                return self._copy(fn, what, k, v, cu, seq_lens, page_table, stream)
        tok, h, d, kt, kh = _rows(k, "k", ix)
        tv, hv, dv, vt, vh = _rows(v, "v", ix)
        if (tv, hv, dv) != (tok, h, d) or h != self.kv_heads or d != self.head_dim:
            raise ValueError("k and v: [tokens, %d, %d] expected, not %s and %s" % (
                self.kv_heads, self.head_dim, tuple(k.shape), tuple(v.shape)))
        n = seq_lens.shape[0]
        strides = None if kt == vt == h * d and kh == vh == d else _Strides4(kt, kh, vt, vh)
        rc = fn(self._ref, k.data_ptr(), v.data_ptr(), strides, tok,
                _plain(cu, "cu", _I32, (n + 1,), ix),
                _plain(seq_lens, "seq_lens", _I32, (n,), ix), _table(page_table, n, ix),
                page_table.shape[1], n, self._err, _raw(stream, ix))
        if rc:
            _raise(rc, what)

    def write(self, k, v, cu, seq_lens, page_table, stream=None):
        """Store packed tokens' rows (dhs_page_write)."""
        self._copy(self._lib.dhs_page_write, "dhs_page_write", k, v, cu, seq_lens, page_table, stream)

    def read(self, k_out, v_out, cu, seq_lens, page_table, stream=None):
        """Cached rows of packed tokens, as bf16 (dhs_page_read)."""
        self._copy(self._lib.dhs_page_read, "dhs_page_read", k_out, v_out, cu, seq_lens, page_table,
                   stream)

    def attend_workspace(self, n_seqs: int, q_len: int, q_heads: int):
        """A new workspace for :meth:`attend` calls of these sizes.  Calls that may
        overlap on the GPU (other streams, other graphs) each need their own."""
        with _on(self._index):
            nbytes = self._lib.dhs_page_attend_workspace(self._ref, n_seqs, q_len, q_heads)
        if nbytes < 0:
            raise ValueError("attend does not serve n_seqs=%d, q_len=%d, q_heads=%d"
                             % (n_seqs, q_len, q_heads))
        return torch.empty(max(16, nbytes), dtype=torch.uint8, device=self.device)

    def attend(self, q, seq_lens, page_table, out, workspace, lse=None, q_lens=None,
               scale: float = 0.0, stream=None):
        """Attention of the newest tokens over the cache (dhs_page_attend):
        ``q`` and ``out`` [n_seqs, q_len, q_heads, head_dim]."""
        ix, shape = self._index, q.shape
        if _current_device() != ix:
            with _on(ix):
                return self.attend(q, seq_lens, page_table, out, workspace, lse, q_lens, scale, stream)
        if len(shape) != 4 or shape[3] != self.head_dim:
            raise ValueError("q: [n_seqs, q_len, q_heads, %d] expected, not %s"
                             % (self.head_dim, tuple(shape)))
        n, qn, hq, _ = shape
        space, nbytes = _space(workspace, ix)
        rc = self._lib.dhs_page_attend(
            self._ref, _plain(q, "q", _BF16, shape, ix),
            None if q_lens is None else _plain(q_lens, "q_lens", _I32, (n,), ix),
            _plain(seq_lens, "seq_lens", _I32, (n,), ix), _table(page_table, n, ix),
            page_table.shape[1], n, qn, hq, scale, _plain(out, "out", _BF16, shape, ix),
            None if lse is None else _plain(lse, "lse", _F32, (n, qn, hq), ix), space, nbytes,
            self._err, _raw(stream, ix))
        if rc:
            _raise(rc, "dhs_page_attend")

    def check(self, stream=None):
        """Raises DhsError if a call on this cache found a bad page or length."""
        check_errors(self.errors, stream)


def prompt_workspace(q, k, n_seqs: int) -> Optional[torch.Tensor]:
    """A new workspace for :func:`prompt_attend` of tensors of these shapes, or
    None where the call needs none."""
    with _on(q.get_device()):
        nbytes = _lib().dhs_prompt_attend_workspace(q.shape[0], k.shape[0], n_seqs, q.shape[1],
                                                    k.shape[1], q.shape[2])
    if nbytes < 0:
        raise ValueError("prompt_attend does not serve q %s, k %s" % (tuple(q.shape), tuple(k.shape)))
    return torch.empty(nbytes, dtype=torch.uint8, device=q.device) if nbytes else None


def prompt_attend(q, k, v, cu_q, cu_k, out, lse=None, workspace=None, scale: float = 0.0,
                  errors=None, stream=None):
    """Causal attention of packed sequences (dhs_prompt_attend): ``q`` [n_q, q_heads,
    head_dim], ``k`` and ``v`` [n_k, kv_heads, head_dim], ``out`` like ``q``.  Bad offsets
    are recorded in ``errors`` (int32[2] on the device) and raised by
    ``check_errors(errors)``; without it in the device's own record, by ``check_errors()``."""
    ix = q.get_device()
    if ix < 0 or _current_device() != ix:
        with _on(ix):
            return prompt_attend(q, k, v, cu_q, cu_k, out, lse, workspace, scale, errors, stream)
    nq, hq, d, qt, qh = _rows(q, "q", ix)
    nk, hkv, dk, kt, kh = _rows(k, "k", ix)
    nv, hv, dv, vt, vh = _rows(v, "v", ix)
    if (nv, hv, dv) != (nk, hkv, dk) or dk != d:
        raise ValueError("k and v: [tokens, kv_heads, %d] expected, not %s and %s"
                         % (d, tuple(k.shape), tuple(v.shape)))
    n = cu_q.shape[0] - 1
    if n < 0:
        raise ValueError("cu_q: [n_seqs + 1] expected")
    space, nbytes = _space(workspace, ix)
    strides = (None if kt == vt == hkv * d and qt == hq * d and qh == kh == vh == d
               else _Strides6(qt, qh, kt, kh, vt, vh))
    rc = _lib().dhs_prompt_attend(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), strides, nq, nk,
        _plain(cu_q, "cu_q", _I32, (n + 1,), ix), _plain(cu_k, "cu_k", _I32, (n + 1,), ix), n, hq,
        hkv, d, scale, _plain(out, "out", _BF16, q.shape, ix),
        None if lse is None else _plain(lse, "lse", _F32, (nq, hq), ix), space, nbytes,
        None if errors is None else _plain(errors, "errors", _I32, (2,), ix), _raw(stream, ix))
    if rc:
        _raise(rc, "dhs_prompt_attend")
