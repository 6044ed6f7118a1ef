"""Binding of the paged 8-bit cache (include/tkv.h): position encoding of queries and
keys, append and attention.  Argument marshalling only, as in tkv.py; the calls run on
the current stream of the tensors' device."""
from __future__ import annotations

import ctypes
from struct import Struct, error as StructError

import torch

from . import tkv
from .tkv import TKV_ERR_CUDA, TKV_ERR_INVALID, TkvError, _check, lib

CODES = {"int8": (0, torch.int8), "e4m3": (1, torch.float8_e4m3fn)}
DTYPES = {torch.bfloat16: 0, torch.float16: 1}


class TkvPagedConfig(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "Hkv", "G", "D", "page", "pages", "max_pages", "code", "dtype")]


class TkvRopeArgs(ctypes.Structure):
    _fields_ = [("inv_freq", ctypes.c_void_p), ("rot", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p), ("eps", ctypes.c_float)]


# The argument structs of include/tkv.h, native layout; row arrays are (address, token
# stride, head stride).
_NORM_ROPE_ARGS = Struct("@PqqPqqPqqPqqPPiiiii4x")
_APPEND_ARGS = Struct("@PqqPqqPqqPqqPPPPii")
_ATTENTION_ARGS = Struct("@PqqPqqPPPiiif")
_NO_ROWS = (0, 0, 0)
_CONTIGUOUS = torch.contiguous_format

# torch.cuda.current_device and .current_stream(i).cuda_stream without their objects, which would
# take 2 of a call's 8 us; the public ones where a torch has no such names.
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", lambda i: torch.cuda.current_stream(i).cuda_stream)


def _bad(msg: str):
    raise TkvError(TKV_ERR_INVALID, msg)


def _run(index: int, fn, *args):
    """Call the library with device `index` current."""
    if index == _current_device():
        status = fn(*args)
    else:
        with torch.cuda.device(index):
            status = fn(*args)
    if status:
        _check(status)


def _pack(struct: Struct, *values) -> bytes:
    try:
        return struct.pack(*values)
    except StructError as e:
        _bad(f"argument out of range or not a number: {e}")


def _rows(t: torch.Tensor, heads: int, dim: int, dtype, index: int, name: str):
    """(address, token stride, head stride) of a [T, heads, dim] tensor."""
    shape = t.shape
    if len(shape) == 3 and shape[1] == heads and shape[2] == dim and t.dtype is dtype and t.get_device() == index:
        st = t.stride()
        if st[2] == 1:
            return t.data_ptr(), st[0], st[1]
        _bad(f"{name} must have a contiguous head dim")
    _bad(f"{name} must be {dtype} [T, {heads}, {dim}] on cuda:{index}, got {t.dtype} {tuple(shape)} on {t.device}")


def _ints(t: torch.Tensor, shape, index: int, name: str) -> int:
    if t.dtype is torch.int32 and t.shape == shape and t.get_device() == index and t.is_contiguous():
        return t.data_ptr()
    _bad(f"{name} must be contiguous int32 {tuple(shape)} on cuda:{index}, got {t.dtype} {tuple(t.shape)} on {t.device}")


def _output(out, like: torch.Tensor, stream, name: str):
    """(out, its address and strides): a new contiguous tensor of the rows' shape, or `out`."""
    if out is None:
        out = (torch.empty_like(like, memory_format=_CONTIGUOUS) if stream is None else
               tkv._empty(like.shape, like.dtype, like.device, stream))
        _, heads, dim = like.shape
        return out, (out.data_ptr(), heads * dim, dim)
    if out.shape != like.shape:
        _bad(f"{name} must be {tuple(like.shape)}, got {tuple(out.shape)}")
    return out, _rows(out, *like.shape[1:], like.dtype, like.get_device(), name)


class TkvRope:
    """How queries and keys are encoded: a norm of each head (weights [D], or None for
    none) and the rotation of the first 2 * len(inv_freq) elements by position * inv_freq
    (fp32, or None for none), as split halves or interleaved pairs."""

    def __init__(self, inv_freq=None, interleaved: bool = False, q_weight=None, k_weight=None, eps: float = 1e-6):
        if (q_weight is None) != (k_weight is None):
            _bad("q_weight and k_weight: both or none")
        self.inv_freq, self.q_weight, self.k_weight = inv_freq, q_weight, k_weight
        self.interleaved, self.eps = bool(interleaved), float(eps)
        for t, name in ((inv_freq, "inv_freq"), (q_weight, "q_weight"), (k_weight, "k_weight")):
            if t is not None and (not t.is_cuda or t.dim() != 1 or not t.is_contiguous()):
                _bad(f"{name} must be a contiguous CUDA vector")
        if inv_freq is not None and inv_freq.dtype is not torch.float32:
            _bad(f"inv_freq must be torch.float32, got {inv_freq.dtype}")
        if q_weight is not None and (q_weight.shape != k_weight.shape or q_weight.dtype is not k_weight.dtype
                                     or q_weight.dtype not in DTYPES):
            _bad("q_weight and k_weight must be bf16 or fp16 vectors of the same size and type")
        self._args = TkvRopeArgs(inv_freq.data_ptr() if inv_freq is not None else None,
                                 2 * inv_freq.numel() if inv_freq is not None else 0, int(self.interleaved),
                                 q_weight.data_ptr() if q_weight is not None else None,
                                 k_weight.data_ptr() if k_weight is not None else None, self.eps)
        self._ptr = ctypes.addressof(self._args)
        devices = {t.device for t in (inv_freq, q_weight, k_weight) if t is not None}
        if len(devices) > 1:
            _bad("inv_freq and the weights must be on one device")
        # what a call has to match (None: anything)
        self.index = devices.pop().index if devices else None
        self.dtype = q_weight.dtype if q_weight is not None else None
        self.dim = q_weight.numel() if q_weight is not None else None

    def _match(self, dtype, dim, index) -> int:
        if self.index is not None and self.index != index:
            _bad(f"the encoding is on cuda:{self.index}, the rows on cuda:{index}")
        if self.dtype is not None and (self.dtype is not dtype or self.dim != dim):
            _bad(f"the norm's weights are {self.dtype} [{self.dim}], the rows {dtype} [{dim}]")
        return self._ptr


def tkv_qk_norm_rope(q: torch.Tensor, k: torch.Tensor, pos: torch.Tensor, rope: TkvRope, q_out=None, k_out=None,
                     stream=None):
    """Norm and rotation of q [T, Hq, D] and k [T, Hkv, D] (bf16 or fp16, any token and head
    strides that are multiples of 4) at positions pos [T] int32; returns (q', k').  The outputs
    may be the inputs."""
    q_shape, k_shape, dtype, index = q.shape, k.shape, q.dtype, q.get_device()
    if len(q_shape) != 3 or len(k_shape) != 3 or index < 0:
        _bad("q and k must be CUDA tensors [T, heads, D]")
    T, Hq, D = q_shape
    Hkv = k_shape[1]
    if dtype not in DTYPES:
        _bad(f"q must be bf16 or fp16, got {dtype}")
    if k_shape[0] != T:
        _bad("q and k must have the same number of tokens")
    qr, kr = _rows(q, Hq, D, dtype, index, "q"), _rows(k, Hkv, D, dtype, index, "k")
    p, r = _ints(pos, (T,), index, "pos"), rope._match(dtype, D, index)
    q_out, qo = _output(q_out, q, stream, "q_out")
    k_out, ko = _output(k_out, k, stream, "k_out")
    args = _pack(_NORM_ROPE_ARGS, *qr, *kr, *qo, *ko, p, r, T, Hq, Hkv, D, DTYPES[dtype])
    _run(index, lib().tkv_qk_norm_rope, args, _current_stream(index) if stream is None else stream.cuda_stream)
    return q_out, k_out


class TkvPagedCache:
    """One layer's paged 8-bit cache: pools of pages with a scale for each (page, kv head),
    the append that fills them and the attention over them.  `pools` gives existing
    (k_pool, v_pool, k_scale, v_scale) tensors, else they are made, zeroed.  `share` is a cache
    whose workspace (up to 43 MB) this one uses too: the layers of a model, say, whose calls
    follow one another on one stream."""

    def __init__(self, B, Hkv, G, D, page, pages, max_pages, code="e4m3", dtype=torch.bfloat16, pools=None,
                 device="cuda", share: TkvPagedCache | None = None):
        if code not in CODES:
            _bad(f"code must be one of {sorted(CODES)}")
        if dtype not in DTYPES:
            _bad(f"dtype must be bf16 or fp16, got {dtype}")
        self.cfg = TkvPagedConfig(B, Hkv, G, D, page, pages, max_pages, CODES[code][0], DTYPES[dtype])
        nbytes = lib().tkv_paged_workspace_bytes(ctypes.byref(self.cfg))
        if nbytes == 0:
            raise TkvError(TKV_ERR_INVALID, lib().tkv_last_error_string().decode())
        self.B, self.Hkv, self.G, self.D, self.page, self.pages, self.max_pages = B, Hkv, G, D, page, pages, max_pages
        self.code, self.dtype = code, dtype
        shape = (pages, Hkv, page, D)
        made = pools is None
        if made:
            device = torch.device(device)
            pools = (*(torch.zeros(shape, dtype=torch.uint8, device=device).view(CODES[code][1]) for _ in range(2)),
                     *(torch.zeros(shape[:2], dtype=torch.float32, device=device) for _ in range(2)))
        self.k_pool, self.v_pool, self.k_scale, self.v_scale = pools
        self.device, self.index = self.k_pool.device, self.k_pool.get_device()
        for t, want, sh, name in ((self.k_pool, CODES[code][1], shape, "k_pool"),
                                  (self.v_pool, CODES[code][1], shape, "v_pool"),
                                  (self.k_scale, torch.float32, shape[:2], "k_scale"),
                                  (self.v_scale, torch.float32, shape[:2], "v_scale")):
            if not t.is_cuda or t.device != self.device or t.dtype is not want or t.shape != sh or not t.is_contiguous():
                _bad(f"{name} must be a contiguous {want} CUDA tensor {sh} on the pools' device")
        if share is None:
            self.workspace = torch.empty(nbytes + 256, dtype=torch.uint8, device=self.device)
        else:
            if share.device != self.device or share.workspace.numel() < nbytes + 256:
                _bad("the shared workspace is on another device or too small")
            self.workspace = share.workspace
        base = self.workspace.data_ptr()
        h = ctypes.c_void_p()
        _check(lib().tkv_paged_create(ctypes.byref(self.cfg), self.k_pool.data_ptr(), self.v_pool.data_ptr(),
                                      self.k_scale.data_ptr(), self.v_scale.data_ptr(), base + (-base) % 256, nbytes,
                                      ctypes.byref(h)))
        self._table_shape, self._len_shape, self._cu_shape = (B, max_pages), (B,), (B + 1,)
        self._append, self._attention, self._destroy = (lib().tkv_paged_append, lib().tkv_paged_attention,
                                                        lib().tkv_paged_destroy)
        self._h = h.value
        if share is None:
            self.reset()
        if share is None or made:
            torch.cuda.current_stream(self.device).synchronize()    # ready for any stream

    def __del__(self):
        h, self._h = getattr(self, "_h", None), None
        if h is not None:
            self._destroy(h)

    def _lengths(self, block_table, kv_len, cu, T):
        i = self.index
        if cu is None and T != self.B:
            _bad(f"without cu there is one row for each of the {self.B} sequences, got {T}")
        return (_ints(block_table, self._table_shape, i, "block_table"), _ints(kv_len, self._len_shape, i, "kv_len"),
                0 if cu is None else _ints(cu, self._cu_shape, i, "cu"))

    def append(self, k: torch.Tensor, v: torch.Tensor, block_table: torch.Tensor, kv_len: torch.Tensor, cu=None,
               max_new: int = 1, rope: TkvRope | None = None, q=None, q_out=None, stream=None):
        """Append k, v [T, Hkv, D]: rows cu[b] .. cu[b+1] (without cu: row b) are the last tokens
        of sequence b, which has kv_len[b] tokens with them.  Keys are encoded by `rope` at their
        index in the sequence; with q [T, Hkv*G, D] the same launch encodes the step's queries,
        which are returned.  max_new bounds a sequence's new tokens."""
        D, index = self.D, self.index
        kr, vr = _rows(k, self.Hkv, D, self.dtype, index, "k"), _rows(v, self.Hkv, D, self.dtype, index, "v")
        T = k.shape[0]
        if v.shape[0] != T:
            _bad("k and v must have the same number of tokens")
        r = 0 if rope is None else rope._match(self.dtype, D, index)
        lengths = self._lengths(block_table, kv_len, cu, T)
        qr = qo = _NO_ROWS
        if q is not None:
            qr = _rows(q, self.Hkv * self.G, D, self.dtype, index, "q")
            if q.shape[0] != T:
                _bad("q and k must have the same number of tokens")
            q_out, qo = _output(q_out, q, stream, "q_out")
        elif q_out is not None:
            _bad("q_out without q")
        _run(index, self._append, self._h, _pack(_APPEND_ARGS, *kr, *vr, *qr, *qo, *lengths, r, T, max_new),
             _current_stream(index) if stream is None else stream.cuda_stream)
        return q_out

    def attention(self, q: torch.Tensor, block_table: torch.Tensor, kv_len: torch.Tensor, softmax_scale: float,
                  cu=None, max_q: int = 1, window: int = 0, out=None, stream=None) -> torch.Tensor:
        """Causal attention of q [T, Hkv*G, D]: rows cu[b] .. cu[b+1] (without cu: row b) are the
        last tokens of sequence b of kv_len[b].  window > 0: each sees the last `window` keys.
        max_q bounds a sequence's rows.  Rows that belong to no sequence are left as they were
        (in an output that is made here: undefined)."""
        index = self.index
        qr = _rows(q, self.Hkv * self.G, self.D, self.dtype, index, "q")
        T = q.shape[0]
        lengths = self._lengths(block_table, kv_len, cu, T)
        out, o = _output(out, q, stream, "out")
        _run(index, self._attention, self._h, _pack(_ATTENTION_ARGS, *qr, *o, *lengths, T, max_q, window, softmax_scale),
             _current_stream(index) if stream is None else stream.cuda_stream)
        return out

    def reset(self, stream=None):
        """Clear the workspace (the pools stay as they are)."""
        _run(self.index, lib().tkv_paged_reset, self._h,
             _current_stream(self.index) if stream is None else stream.cuda_stream)

    def poll_error(self, stream=None) -> int:
        """Synchronise and return (and clear) the first device-side status."""
        with torch.cuda.device(self.device):
            st = lib().tkv_paged_poll_error(self._h, _current_stream(self.index) if stream is None else stream.cuda_stream)
        if st == TKV_ERR_CUDA:
            _check(st)
        return st

    def launch_count(self) -> int:
        return lib().tkv_paged_launch_count(self._h)


def tkv_paged_append(cache: TkvPagedCache, k, v, block_table, kv_len, **kw):
    return cache.append(k, v, block_table, kv_len, **kw)


def tkv_paged_attention(cache: TkvPagedCache, q, block_table, kv_len, softmax_scale, **kw):
    return cache.attention(q, block_table, kv_len, softmax_scale, **kw)
