"""Dense attention over a paged cache: binding of ``dhs_page_*`` and
``dhs_prompt_attend`` (see include/dhs.h for what each call computes).

Tensors are checked for type, shape, layout and device and passed on; nothing
is copied, cast or allocated by a call.  A call runs on the tensors' device and
on ``stream`` (default: torch's current stream there); as with every call of the
library its tensors must stay alive until the stream has passed it.
"""
from __future__ import annotations

import ctypes
from contextlib import nullcontext
from typing import Optional

import torch

PAGE_BF16, PAGE_INT8, PAGE_E4M3 = 0, 1, 2
_KIND = {torch.bfloat16: PAGE_BF16, torch.int8: PAGE_INT8, torch.float8_e4m3fn: PAGE_E4M3}
_DTYPE = {v: k for k, v in _KIND.items()}
_CHECK = {1: "a length or offset outside its range", 2: "a page outside the cache",
          4: "a bounded wait that ran out"}
_SITE = {1: "dhs_page_write", 2: "dhs_page_read", 3: "dhs_page_attend", 4: "dhs_prompt_attend"}


class Pages(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("n_pages", ctypes.c_int64),
                ("page_rows", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("kind", ctypes.c_int32)]


def _lib():
    from . import load
    return load()


def _raise(code, what):
    from . import DhsError
    raise DhsError(code, what)


def _need(ok, what):
    if not ok:
        raise ValueError(what)


def _rows(t, name, heads, dim, device):
    """Token and head stride of a packed bf16 tensor [tokens, heads, dim]."""
    _need(t.dtype is torch.bfloat16 and t.dim() == 3, "%s: bf16 [tokens, heads, dim] expected" % name)
    _need(t.device == device, "%s is on %s, not on %s" % (name, t.device, device))
    n, h, d = t.shape
    _need((heads is None or h == heads) and (dim is None or d == dim),
          "%s has %d heads of %d elements" % (name, h, d))
    st, sh, sd = t.stride()
    _need(sd == 1 or t.numel() == 0, "%s: the elements of a head must be contiguous" % name)
    # a stride that no second token or head uses may be anything
    return (st if n > 1 else h * d), (sh if h > 1 else d)


def _ints(t, name, shape, device):
    _need(t.dtype is torch.int32 and t.is_contiguous(), "%s: contiguous int32 expected" % name)
    _need(t.device == device, "%s is on %s, not on %s" % (name, t.device, device))
    _need(shape is None or tuple(t.shape) == shape, "%s has shape %s, not %s"
          % (name, tuple(t.shape), shape))
    return t.data_ptr()


def _plain(t, name, dtype, shape, device):
    _need(t.dtype is dtype and t.is_contiguous() and tuple(t.shape) == shape,
          "%s: contiguous %s %s expected" % (name, dtype, shape))
    _need(t.device == device, "%s is on %s, not on %s" % (name, t.device, device))
    return t.data_ptr()


def _space(t, device):
    if t is None:
        return None, 0
    _need(t.is_contiguous() and t.device == device, "workspace: contiguous, on %s expected" % device)
    return t.data_ptr(), t.numel() * t.element_size()


def _on(device):
    _need(device.type == "cuda", "CUDA tensors expected, not %s" % device)
    return nullcontext() if torch.cuda.current_device() == device.index else torch.cuda.device(device)


def _raw(stream, device):
    if stream is None:
        return torch.cuda.current_stream(device).cuda_stream
    return stream if isinstance(stream, int) else stream.cuda_stream


def check_errors(errors, stream=None):
    """Waits for ``stream``, raises DhsError (code 5) if a call recorded a bad
    page, length or offset in ``errors`` (int32[2]), and clears the record."""
    with _on(errors.device):
        s = torch.cuda.current_stream() if stream is None else stream
        if isinstance(s, int):
            s = torch.cuda.ExternalStream(s)
        with torch.cuda.stream(s):
            code, site = errors.tolist()
            if code:
                errors.zero_()
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
        _need(k.dtype in _KIND, "a cache of %s is not supported" % k.dtype)
        _need(k.dim() == 4 and k.is_contiguous() and v.is_contiguous() and v.shape == k.shape
              and v.dtype is k.dtype, "k and v: contiguous, of one shape and type expected")
        self.device = k.device
        _on(self.device)
        _need(v.device == self.device, "k and v are on different devices")
        self.kind = _KIND[k.dtype]
        self.n_pages, self.kv_heads, self.page_rows, self.head_dim = k.shape
        if self.kind == PAGE_BF16:
            _need(k_scale is None and v_scale is None, "a bf16 cache has no scales")
        else:
            _need(k_scale is not None and v_scale is not None, "an 8-bit cache needs scales")
            for t, name in ((k_scale, "k_scale"), (v_scale, "v_scale")):
                _plain(t, name, torch.float32, tuple(k.shape[:3]), self.device)
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.errors = torch.zeros(2, dtype=torch.int32, device=self.device) if errors is None else errors
        self._err = _plain(self.errors, "errors", torch.int32, (2,), self.device)
        ptr = lambda t: None if t is None else t.data_ptr()  # noqa: E731
        self._desc = Pages(ptr(k), ptr(v), ptr(k_scale), ptr(v_scale), self.n_pages,
                           self.page_rows, self.kv_heads, self.head_dim, self.kind)
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
        dev = self.device
        strides = (ctypes.c_int64 * 4)(*_rows(k, "k", self.kv_heads, self.head_dim, dev),
                                       *_rows(v, "v", self.kv_heads, self.head_dim, dev))
        n, tok = seq_lens.shape[0], k.shape[0]
        _need(v.shape[0] == tok, "k has %d tokens, v %d" % (tok, v.shape[0]))
        _need(page_table.dim() == 2 and page_table.shape[0] == n, "page_table: [%d, width] expected" % n)
        with _on(dev):
            rc = fn(self._ref, k.data_ptr(), v.data_ptr(), strides, tok,
                    _ints(cu, "cu", (n + 1,), dev), _ints(seq_lens, "seq_lens", (n,), dev),
                    _ints(page_table, "page_table", None, dev), page_table.shape[1], n, self._err,
                    _raw(stream, dev))
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
        with _on(self.device):
            nbytes = self._lib.dhs_page_attend_workspace(self._ref, n_seqs, q_len, q_heads)
        _need(nbytes >= 0, "attend does not serve n_seqs=%d, q_len=%d, q_heads=%d"
              % (n_seqs, q_len, q_heads))
        return torch.zeros(max(16, nbytes), dtype=torch.uint8, device=self.device)

    def attend(self, q, seq_lens, page_table, out, workspace, lse=None, q_lens=None,
               scale: float = 0.0, stream=None):
        """Attention of the newest tokens over the cache (dhs_page_attend):
        ``q`` and ``out`` [n_seqs, q_len, q_heads, head_dim]."""
        dev = self.device
        n, qn, hq, d = q.shape
        _need(d == self.head_dim, "q has %d elements a head, the cache %d" % (d, self.head_dim))
        _need(page_table.dim() == 2 and page_table.shape[0] == n, "page_table: [%d, width] expected" % n)
        space, nbytes = _space(workspace, dev)
        with _on(dev):
            rc = self._lib.dhs_page_attend(
                self._ref, _plain(q, "q", torch.bfloat16, (n, qn, hq, d), dev),
                None if q_lens is None else _ints(q_lens, "q_lens", (n,), dev),
                _ints(seq_lens, "seq_lens", (n,), dev),
                _ints(page_table, "page_table", None, dev), page_table.shape[1], n, qn, hq, scale,
                _plain(out, "out", torch.bfloat16, (n, qn, hq, d), dev),
                None if lse is None else _plain(lse, "lse", torch.float32, (n, qn, hq), dev),
                space, nbytes, self._err, _raw(stream, dev))
        if rc:
            _raise(rc, "dhs_page_attend")

    def check(self, stream=None):
        """Raises DhsError if a call on this cache found a bad page or length."""
        check_errors(self.errors, stream)


def prompt_workspace(q, k, n_seqs: int) -> Optional[torch.Tensor]:
    """A new workspace for :func:`prompt_attend` of tensors of these shapes, or
    None where the call needs none."""
    with _on(q.device):
        nbytes = _lib().dhs_prompt_attend_workspace(q.shape[0], k.shape[0], n_seqs, q.shape[1],
                                                    k.shape[1], q.shape[2])
    _need(nbytes >= 0, "prompt_attend does not serve q %s, k %s" % (tuple(q.shape), tuple(k.shape)))
    return torch.zeros(nbytes, dtype=torch.uint8, device=q.device) if nbytes else None


def prompt_attend(q, k, v, cu_q, cu_k, out, lse=None, workspace=None, scale: float = 0.0,
                  errors=None, stream=None):
    """Causal attention of packed sequences (dhs_prompt_attend): ``q`` [n_q, q_heads,
    head_dim], ``k`` and ``v`` [n_k, kv_heads, head_dim], ``out`` like ``q``."""
    dev = q.device
    strides = (ctypes.c_int64 * 6)(*_rows(q, "q", None, None, dev),
                                   *_rows(k, "k", None, q.shape[2], dev),
                                   *_rows(v, "v", k.shape[1], q.shape[2], dev))
    nq, hq, d = q.shape
    nk, hkv = k.shape[:2]
    n = cu_q.shape[0] - 1
    _need(n >= 0, "cu_q: [n_seqs + 1] expected")
    _need(v.shape[0] == nk, "k has %d tokens, v %d" % (nk, v.shape[0]))
    space, nbytes = _space(workspace, dev)
    with _on(dev):
        rc = _lib().dhs_prompt_attend(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), strides, nq, nk,
            _ints(cu_q, "cu_q", (n + 1,), dev), _ints(cu_k, "cu_k", (n + 1,), dev), n, hq, hkv, d,
            scale, _plain(out, "out", torch.bfloat16, (nq, hq, d), dev),
            None if lse is None else _plain(lse, "lse", torch.float32, (nq, hq), dev), space, nbytes,
            None if errors is None else _plain(errors, "errors", torch.int32, (2,), dev),
            _raw(stream, dev))
    if rc:
        _raise(rc, "dhs_prompt_attend")
