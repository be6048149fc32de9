"""Dense attention over a paged cache: binding of ``dhs_page_*``, ``dhs_rotate`` and
``dhs_prompt_attend`` (see include/dhs.h for what each call computes).

Tensors are checked for type, shape, layout and device and passed on; nothing
is copied, cast or allocated by a call.  A call runs on the tensors' device and
on ``stream`` (default: torch's current stream there); as with every call of the
library its tensors must stay alive until the stream has passed it.
"""
from __future__ import annotations

import ctypes
import struct
from typing import Optional

import torch

PAGE_BF16, PAGE_INT8, PAGE_E4M3 = 0, 1, 2
_KIND = {torch.bfloat16: PAGE_BF16, torch.int8: PAGE_INT8, torch.float8_e4m3fn: PAGE_E4M3}
_DTYPE = {v: k for k, v in _KIND.items()}
_CHECK = {1: "a length or offset outside its range", 2: "a page outside the cache",
          4: "a bounded wait that ran out"}
_SITE = {1: "dhs_page_write", 2: "dhs_page_read", 3: "dhs_page_attend", 4: "dhs_prompt_attend",
         5: "dhs_page_append", 6: "dhs_page_chunk"}
ROTATE_HALVES, ROTATE_NEIGHBOURS = 0, 1

_Strides2, _Strides4, _Strides6 = ctypes.c_int64 * 2, ctypes.c_int64 * 4, ctypes.c_int64 * 6


class Pages(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("n_pages", ctypes.c_int64),
                ("page_rows", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("kind", ctypes.c_int32)]


class _Turns(ctypes.Structure):
    _fields_ = [("turns", ctypes.c_void_p), ("n_pairs", ctypes.c_int32), ("pairing", ctypes.c_int32),
                ("amplitude", ctypes.c_float)]


class _Heads(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("out", ctypes.c_void_p), ("norm", ctypes.c_void_p)] + [
        (n, ctypes.c_int64) for n in ("x_token", "x_head", "out_token", "out_head")] + [
        ("heads", ctypes.c_int32)]


_HEADS = struct.Struct("=QQQqqqqi4x")  # its bytes, which cost a third of its object
assert _HEADS.size == ctypes.sizeof(_Heads)


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


_loaded = None


def _lib():
    global _loaded
    if _loaded is None:
        from . import load
        _loaded = load()
    return _loaded


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


def _strides(name, t, index):
    """Shape of a packed bf16 tensor, and its token's and head's stride; like _rows, sooner for
    the usual one."""
    shape = t.shape
    if t.dtype is _BF16 and len(shape) == 3 and t.get_device() == index and t.is_contiguous():
        d = shape[2]
        return shape, shape[1] * d, d
    return (shape, *_rows(t, name, index)[3:])


def _heads(name, x, out, norm, index):
    """The shape of a tensor's heads, [tokens, heads, head_dim], and a dhs_heads: they and where
    they go."""
    shape, xt, xh = _strides(name, x, index)
    at = ot = oh = weights = 0
    if out is x:
        at, ot, oh = x.data_ptr(), xt, xh
    elif out is not None:
        to, ot, oh = _strides(name + "_out", out, index)
        if to != shape:
            raise ValueError("%s_out: %s expected, not %s" % (name, tuple(shape), tuple(to)))
        at = out.data_ptr()
    if norm is not None:
        weights = _plain(norm, name + "_norm", _F32, shape[2:], index)
    return shape, _HEADS.pack(x.data_ptr(), at, weights, xt, xh, ot, oh, shape[1])


def _turns(rotation, index):
    if rotation is None:
        return None
    if rotation._index != index:
        raise ValueError("rotation: on cuda:%s expected, not cuda:%s" % (index, rotation._index))
    return rotation._ref


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


class Rotation:
    """A position rotation for :func:`rotate` and :meth:`PageCache.append`, laid out once.

    ``freqs``: the angle that pair i of a head's row turns by per position, in radians (numbers,
    or an array or tensor on any device, fp64: what has fewer bits is taken as it is, and far
    positions turn by as many times its error); a multiple of 4 of them, at most half a head's
    elements, the rest of which stay as they are.  ``pairing``: ``ROTATE_HALVES`` for pairs (i, i + len(freqs)),
    ``ROTATE_NEIGHBOURS`` for (2 i, 2 i + 1).  ``amplitude`` multiplies sines and cosines.
    """

    def __init__(self, freqs, pairing: int = ROTATE_HALVES, amplitude: float = 1.0, device=None):
        # (a list of numbers would become 32 bits by itself)
        host = torch.as_tensor(freqs, dtype=torch.float64).detach()
        if device is None:
            device = host.device if host.is_cuda else "cuda"
        host = host.cpu().contiguous()
        if host.dim() != 1 or pairing not in (ROTATE_HALVES, ROTATE_NEIGHBOURS):
            raise ValueError("freqs: [n_pairs], pairing: ROTATE_HALVES or ROTATE_NEIGHBOURS expected")
        turns = torch.empty(host.shape, dtype=torch.int64)
        rc = _lib().dhs_rotation_turns(host.data_ptr(), host.numel(), turns.data_ptr())
        if rc:
            _raise(rc, "dhs_rotation_turns")
        self.turns, self.pairing, self.amplitude = turns.to(device), pairing, amplitude
        self._index = self.turns.get_device()
        with _on(self._index):
            torch.cuda.current_stream().synchronize()  # (calls on any stream may follow)
        self._desc = _Turns(self.turns.data_ptr(), host.numel(), pairing, amplitude)
        self._ref = ctypes.byref(self._desc)


def rotate(q, k, positions, rotation, q_out, k_out, q_norm=None, k_norm=None, eps: float = 1e-6,
           stream=None):
    """Norm and rotation of every head (dhs_rotate): ``q`` and ``k`` [tokens, heads, head_dim]
    bf16 into ``q_out`` and ``k_out`` (which may be ``q`` and ``k``); ``k`` and ``k_out`` or ``q``
    and ``q_out`` may be None.  ``positions`` int32 [tokens]; ``q_norm`` and ``k_norm`` fp32
    [head_dim] or None; ``rotation`` a :class:`Rotation` or None."""
    some = k if q is None else q
    if some is None:
        raise ValueError("q or k expected")
    ix = some.get_device()
    if ix < 0 or _current_device() != ix:
        with _on(ix):
            return rotate(q, k, positions, rotation, q_out, k_out, q_norm, k_norm, eps, stream)
    hq = hk = None
    if q is not None:
        (n, _, d), hq = _heads("q", q, q_out, q_norm, ix)
    if k is not None:
        (nk, _, dk), hk = _heads("k", k, k_out, k_norm, ix)
        if hq is None:
            n, d = nk, dk
        elif nk != n or dk != d:
            raise ValueError("k: [%d, kv_heads, %d] expected, not %s" % (n, d, tuple(k.shape)))
    rc = _lib().dhs_rotate(_turns(rotation, ix), hq, hk, eps, d, n,
                           None if positions is None else _plain(positions, "positions", _I32, (n,), ix),
                           _raw(stream, ix))
    if rc:
        _raise(rc, "dhs_rotate")


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

    def append(self, q, k, v, cu, seq_lens, page_table, q_out, rotation=None, q_norm=None,
               k_norm=None, eps: float = 1e-6, positions=None, k_out=None, stream=None):
        """Norm and rotation of packed tokens' queries and keys, the queries into ``q_out``, keys
        and values into the pages (dhs_page_append).  ``q`` and ``q_out`` may be None; ``k_out``
        takes the keys in bf16 as well; ``positions`` int32 [tokens] to rotate by instead of
        the tokens' own.  The norms and ``rotation`` as in :func:`rotate`."""
        ix = self._index
        if _current_device() != ix:
            with _on(ix):
                return self.append(q, k, v, cu, seq_lens, page_table, q_out, rotation, q_norm, k_norm,
                                   eps, positions, k_out, stream)
        ks, hk = _heads("k", k, k_out, k_norm, ix)
        vs, vt, vh = _strides("v", v, ix)
        tok, h, d = ks
        if d != self.head_dim or h != self.kv_heads or vs != ks:
            raise ValueError("k and v: [tokens, %d, %d] expected, not %s and %s" % (
                self.kv_heads, self.head_dim, tuple(k.shape), tuple(v.shape)))
        hq = None
        if q is not None:
            (nq, _, dq), hq = _heads("q", q, q_out, q_norm, ix)
            if nq != tok or dq != d:
                raise ValueError("q: [%d, q_heads, %d] expected, not %s" % (tok, d, tuple(q.shape)))
        n = seq_lens.shape[0]
        rc = self._lib.dhs_page_append(
            self._ref, _turns(rotation, ix), hq, hk, v.data_ptr(),
            None if vt == h * d and vh == d else _Strides2(vt, vh), eps, tok,
            None if positions is None else _plain(positions, "positions", _I32, (tok,), ix),
            _plain(cu, "cu", _I32, (n + 1,), ix), _plain(seq_lens, "seq_lens", _I32, (n,), ix),
            _table(page_table, n, ix), page_table.shape[1], n, self._err, _raw(stream, ix))
        if rc:
            _raise(rc, "dhs_page_append")

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
               scale: float = 0.0, stream=None, window: int = 0, sinks: int = 0):
        """Attention of the newest tokens over the cache (dhs_page_attend):
        ``q`` and ``out`` [n_seqs, q_len, q_heads, head_dim].  With a ``window`` a token sees
        that many positions up to its own, and the first ``sinks`` ones
        (dhs_page_attend_window)."""
        ix, shape = self._index, q.shape
        if _current_device() != ix:
            with _on(ix):
                return self.attend(q, seq_lens, page_table, out, workspace, lse, q_lens, scale, stream,
                                   window, sinks)
        if len(shape) != 4 or shape[3] != self.head_dim:
            raise ValueError("q: [n_seqs, q_len, q_heads, %d] expected, not %s"
                             % (self.head_dim, tuple(shape)))
        n, qn, hq, _ = shape
        space, nbytes = _space(workspace, ix)
        if window or sinks:
            fn, what, extra = self._lib.dhs_page_attend_window, "dhs_page_attend_window", (window, sinks)
        else:
            fn, what, extra = self._lib.dhs_page_attend, "dhs_page_attend", ()
        rc = fn(
            self._ref, _plain(q, "q", _BF16, shape, ix),
            None if q_lens is None else _plain(q_lens, "q_lens", _I32, (n,), ix),
            _plain(seq_lens, "seq_lens", _I32, (n,), ix), _table(page_table, n, ix),
            page_table.shape[1], n, qn, hq, *extra, scale, _plain(out, "out", _BF16, shape, ix),
            None if lse is None else _plain(lse, "lse", _F32, (n, qn, hq), ix), space, nbytes,
            self._err, _raw(stream, ix))
        if rc:
            _raise(rc, what)

    def chunk_workspace(self, n_tokens: int, n_seqs: int, q_heads: int):
        """A new workspace for :meth:`attend_chunk` calls of these sizes.  Calls that may
        overlap on the GPU (other streams, other graphs) each need their own."""
        with _on(self._index):
            nbytes = self._lib.dhs_page_chunk_workspace(self._ref, n_tokens, n_seqs, q_heads)
        if nbytes < 0:
            raise ValueError("attend_chunk does not serve n_tokens=%d, n_seqs=%d, q_heads=%d"
                             % (n_tokens, n_seqs, q_heads))
        return torch.empty(max(16, nbytes), dtype=torch.uint8, device=self.device)

    def attend_chunk(self, q, cu, seq_lens, page_table, out, workspace, lse=None, window: int = 0,
                     sinks: int = 0, scale: float = 0.0, stream=None):
        """Attention of packed new tokens over the cache (dhs_page_chunk): ``q`` and ``out``
        [tokens, q_heads, head_dim].  With a ``window`` a token sees that many positions up to
        its own, and the first ``sinks`` ones."""
        ix = self._index
        if _current_device() != ix:
            with _on(ix):
                return self.attend_chunk(q, cu, seq_lens, page_table, out, workspace, lse, window,
                                         sinks, scale, stream)
        shape, qt, qh = _strides("q", q, ix)
        tok, hq, d = shape
        if d != self.head_dim:
            raise ValueError("q: [tokens, q_heads, %d] expected, not %s" % (self.head_dim, tuple(q.shape)))
        n = seq_lens.shape[0]
        space, nbytes = _space(workspace, ix)
        rc = self._lib.dhs_page_chunk(
            self._ref, q.data_ptr(), None if qt == hq * d and qh == d else _Strides2(qt, qh), tok,
            _plain(cu, "cu", _I32, (n + 1,), ix), _plain(seq_lens, "seq_lens", _I32, (n,), ix),
            _table(page_table, n, ix), page_table.shape[1], n, hq, window, sinks, scale,
            _plain(out, "out", _BF16, shape, ix),
            None if lse is None else _plain(lse, "lse", _F32, (tok, hq), ix), space, nbytes,
            self._err, _raw(stream, ix))
        if rc:
            _raise(rc, "dhs_page_chunk")

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
