"""Binding of the calls over whole key ranges of the paged K/V cache: rotary
append, window attention (decode and prefill) and shared-prefix decode.

Each C entry point has a function of its name, which checks its arguments and
marshals them, and a class that holds what a serving loop keeps between calls
(the cache description, the output buffers and the workspace).  A class takes
the cache's tensors when it is made and keeps them: their contents may change; a
tensor put in the place of one later is not seen.  Its outputs are its own
buffers, overwritten by its next call.  Work goes to `stream`, by default the
current stream of the tensors' device; a handle may be made on one stream and
called on others, one call at a time, and dropped while its last call still runs
(on a torch.cuda.ExternalStream only after that: torch cannot order memory behind
such a stream's work safely).
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import _lib
from .api import QSACache, _check, _need

_Q_DTYPES = {torch.float32: _lib.QSA_F32, torch.bfloat16: _lib.QSA_BF16}
_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3}


class _Caches:
    """What every call takes from the caches, found once: the C struct (and a
    reference to it), the device index, the query type, the head shape and the
    requests that the block table has rows for (B: those of a call or handle)."""
    __slots__ = ("struct", "ref", "index", "dtype", "qd", "Hkv", "D", "device", "rows", "tensors")

    def __init__(self, cache: QSACache, B: int = 0):
        if cache.block_table.dim() != 2:
            raise ValueError("block_table must be [requests, pages]")
        self.rows = cache.block_table.shape[0]
        self.holds(B)
        k, at = cache.k_cache, cache.k_cache.get_device()
        if k.dtype == torch.float8_e4m3fn:
            for t, name in ((cache.k_scale, "k_scale"), (cache.v_scale, "v_scale")):
                if t is None or t.dtype is not torch.float32 or t.shape != (k.shape[0], k.shape[2]):
                    raise ValueError(f"{name} of an 8-bit cache must be float32 [{k.shape[0]}, {k.shape[2]}]")
        for t in (cache.v_cache, cache.block_table, cache.k_scale, cache.v_scale):
            if t is not None and t.get_device() != at:
                raise ValueError("the cache's tensors are on different devices")
        self.struct = cache.struct()
        # the struct holds their addresses: they live as long as it does
        self.tensors = (cache.k_cache, cache.v_cache, cache.block_table, cache.k_scale, cache.v_scale)
        self.ref = ctypes.byref(self.struct)
        self.device = cache.k_cache.device
        self.index = cache.k_cache.get_device()
        self.dtype = torch.float32 if cache.k_cache.dtype == torch.float32 else torch.bfloat16
        self.qd = _Q_DTYPES[self.dtype]
        _, _, self.Hkv, self.D = cache.k_cache.shape

    def holds(self, B: int) -> None:
        if B > self.rows:
            raise ValueError(f"block_table has {self.rows} rows for {B} requests")


class _Buffers:
    """A handle's own tensors and the streams that have used them: made on the
    current stream, usable on any."""
    __slots__ = ("tensors", "seen")

    def __init__(self, c: _Caches, *tensors: torch.Tensor | None):
        self.tensors = [t for t in tensors if t is not None]
        made = torch.cuda.current_stream(c.device)
        self.seen = {made.cuda_stream}
        # what fills them, and what their memory was used for before on this stream,
        # ends before another stream may write them (a capture has its own memory)
        if not torch.cuda.is_current_stream_capturing():
            made.synchronize()

    def used_on(self, stream: torch.cuda.Stream) -> None:
        """Keeps their memory, once they are dropped, until `stream` is done."""
        self.seen.add(stream.cuda_stream)
        if not isinstance(stream, torch.cuda.ExternalStream):  # (may be gone by then)
            for t in self.tensors:
                t.record_stream(stream)


def _call(fn, name: str, index: int, args: tuple, stream, buffers: _Buffers | None = None) -> None:
    """fn(*args, stream) with the caches' device as the current one."""
    if torch.cuda.current_device() != index:
        with torch.cuda.device(index):
            return _call(fn, name, index, args, stream, buffers)
    handle = stream.cuda_stream if stream is not None else torch._C._cuda_getCurrentRawStream(index)
    if buffers is not None and handle not in buffers.seen:
        buffers.used_on(stream if stream is not None else torch.cuda.current_stream(index))
    status = fn(*args, handle)
    if status:
        _check(status, name)


def _ints(t: torch.Tensor, n: int, name: str, index: int) -> int:
    if t.dtype is not torch.int32 or t.shape != (n,) or t.get_device() != index or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor of {n} entries on the cache's device")
    return t.data_ptr()


def _dense(t: torch.Tensor, dtype: torch.dtype, shape: tuple, name: str, index: int) -> int:
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape or t.get_device() != index or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous tensor of shape {list(shape)} on the cache's device")
    return t.data_ptr()


def _bytes(workspace: torch.Tensor | None, index: int) -> tuple[int | None, int]:
    if workspace is None:
        return None, 0
    if workspace.get_device() != index or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the cache's device")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _int32(v, name: str) -> int:
    v = int(v)
    if not -(1 << 31) <= v < 1 << 31:
        raise ValueError(f"{name} does not fit 32 bits")
    return v


def _sizes(*v) -> tuple[int, ...]:
    return tuple(_int32(x, "a size") for x in v)


def _workspace(nbytes: int, device) -> torch.Tensor | None:
    return torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes else None


def _outputs(c: _Caches, shape, o: torch.Tensor, lse: torch.Tensor) -> tuple[int, int]:
    return (_dense(o, c.dtype, shape, "o", c.index),
            _dense(lse, torch.float32, shape[:-1], "lse", c.index))


def _heads(q: torch.Tensor, c: _Caches) -> None:
    if q.shape[-1] != c.D:
        raise ValueError("q and the cache have different head dims")


# ------------------------------------------------------------------- rope --
def qsa_rope_freqs(rotary_dim: int, theta: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                   original_max_position: int = 0, beta_fast: float = 32.0,
                   beta_slow: float = 1.0) -> tuple[list[int], list[float], float]:
    """(freqs, inv_freq, mscale): the rotated pairs' turns per token in units
    of 2^-64, their radians per token, and the factor on the rotated dims."""
    if scaling not in _SCALINGS:
        raise ValueError(f"scaling must be one of {sorted(_SCALINGS)}")
    rotary_dim = _int32(rotary_dim, "rotary_dim")
    original_max_position = _int32(original_max_position, "original_max_position")
    n = min(max(rotary_dim, 0), 128) // 2  # (above 128: refused)
    fr, inv, m = (ctypes.c_uint64 * max(n, 1))(), (ctypes.c_double * max(n, 1))(), ctypes.c_float()
    _check(_lib.load().qsa_rope_freqs(rotary_dim, float(theta), _SCALINGS[scaling], float(factor),
                                      original_max_position, float(beta_fast), float(beta_slow),
                                      ctypes.addressof(inv), ctypes.addressof(fr), ctypes.byref(m)),
           "qsa_rope_freqs")
    return list(fr[:n]), list(inv[:n]), m.value


def _rows(t: torch.Tensor, dtype, heads: int, D: int, n: int, name: str, index: int) -> tuple[int, int]:
    """(pointer, row stride) of t [n, heads, D] whose rows are dense."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != (n, heads, D) or t.get_device() != index:
        raise ValueError(f"{name} must be [{n}, {heads}, {D}] on the cache's device")
    s = t.stride()
    if (s[2] != 1 or (heads > 1 and s[1] != D)) and n > 0:
        raise ValueError(f"the heads of a row of {name} must be dense")
    return t.data_ptr(), s[0] if n > 1 else heads * D


def _rope_append(c: _Caches, fn, freqs, rotary_dim, layout, mscale, pos0, cu_new, q, k, v, q_out, stream,
                 buffers=None):
    n, Hq, _ = q.shape
    B, dt, ix, D = pos0.shape[0], c.dtype, c.index, c.D
    c.holds(B)
    qp, qs = _rows(q, dt, Hq, D, n, "q", ix)
    kp, ks = _rows(k, dt, c.Hkv, D, n, "k", ix)
    vp, vs = _rows(v, dt, c.Hkv, D, n, "v", ix)
    _call(fn, "qsa_rope_append", ix,
          (c.ref, B, n, _ints(pos0, B, "pos0", ix), _ints(cu_new, B + 1, "cu_new", ix), qp, qs, kp, ks, vp, vs,
           c.qd, Hq, freqs, rotary_dim, layout, mscale, _dense(q_out, dt, (n, Hq, D), "q_out", ix)), stream, buffers)


def qsa_rope_append(cache: QSACache, pos0: torch.Tensor, cu_new: torch.Tensor, q: torch.Tensor,
                    k: torch.Tensor, v: torch.Tensor, freqs: torch.Tensor, rotary_dim: int,
                    interleaved: bool, mscale: float, q_out: torch.Tensor, stream=None) -> None:
    """Rotates q [N, Hq, D] into q_out and k [N, Hkv, D] into the cache's
    pages, and copies v there.  `freqs`: int64 [rotary_dim / 2] on the cache's
    device, the bits of qsa_rope_freqs.  q, k, v may be strided over tokens
    (parts of one fused projection)."""
    rotary_dim = _int32(rotary_dim, "rotary_dim")
    c = _Caches(cache)
    _need(freqs, torch.int64, "freqs")
    if freqs.shape != (max(rotary_dim, 0) // 2,) or freqs.get_device() != c.index or not freqs.is_contiguous():
        raise ValueError("freqs must hold rotary_dim / 2 entries on the cache's device")
    _rope_append(c, _lib.load().qsa_rope_append, freqs.data_ptr() if rotary_dim else None, rotary_dim,
                 int(bool(interleaved)), float(mscale), pos0, cu_new, q, k, v, q_out, stream)


class QSARopeAppend:
    """qsa_rope_append with the frequencies of one model's layers."""

    def __init__(self, cache: QSACache, Hq: int, rotary_dim: int | None = None, theta: float = 10000.0,
                 interleaved: bool = False, scaling: str = "none", factor: float = 1.0,
                 original_max_position: int = 0, beta_fast: float = 32.0, beta_slow: float = 1.0):
        D = cache.k_cache.shape[-1]
        self.cache, self.Hq, self.interleaved = cache, Hq, bool(interleaved)
        self.rotary_dim = D if rotary_dim is None else int(rotary_dim)
        if not 0 <= self.rotary_dim <= D:
            raise ValueError("rotary_dim must be at most the head dim")
        turns, self.inv_freq, self.mscale = qsa_rope_freqs(self.rotary_dim, theta, scaling, factor,
                                                           original_max_position, beta_fast, beta_slow)
        self.freqs = torch.tensor([f - (1 << 64) if f >> 63 else f for f in turns], dtype=torch.int64,
                                  device=cache.k_cache.device)
        self._c, self._fn = _Caches(cache), _lib.load().qsa_rope_append
        self._buffers = _Buffers(self._c, self.freqs)

    def __call__(self, pos0, cu_new, q, k, v, q_out=None, stream=None) -> torch.Tensor:
        if q.dim() != 3 or q.shape[1] != self.Hq:
            raise ValueError(f"q must be [N, {self.Hq}, D]")
        if q_out is None:
            with torch.cuda.stream(stream):  # its memory belongs to the stream that writes it
                q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        _rope_append(self._c, self._fn, self.freqs.data_ptr() if self.rotary_dim else None, self.rotary_dim,
                     int(self.interleaved), self.mscale, pos0, cu_new, q, k, v, q_out, stream, self._buffers)
        return q_out


# ----------------------------------------------------------------- window --
def qsa_window_decode_workspace_bytes(cache: QSACache, B: int, T: int, Hq: int, window: int, sinks: int) -> int:
    return int(_lib.load().qsa_window_decode_workspace_bytes(ctypes.byref(cache.struct()),
                                                             *_sizes(B, T, Hq, window, sinks)))


def qsa_window_decode(cache: QSACache, q: torch.Tensor, ctx_lens: torch.Tensor, window: int, sinks: int,
                      sm_scale: float, o: torch.Tensor, lse: torch.Tensor, workspace: torch.Tensor | None,
                      stream=None) -> None:
    """Decode attention of q [B, T, Hq, D] over each request's last `window`
    keys and first `sinks` keys.  o: q's type and shape, lse float32."""
    B, T, Hq, _ = shape = q.shape
    c = _Caches(cache, B)
    _heads(q, c)
    ix = c.index
    _call(_lib.load().qsa_window_decode, "qsa_window_decode", ix,
          (c.ref, B, T, Hq, _dense(q, c.dtype, shape, "q", ix), c.qd, _ints(ctx_lens, B, "ctx_lens", ix),
           _int32(window, "window"), _int32(sinks, "sinks"), float(sm_scale), *_outputs(c, shape, o, lse),
           *_bytes(workspace, ix)), stream)


class QSAWindowDecode:
    """qsa_window_decode for batches of B requests with T query tokens."""

    def __init__(self, cache: QSACache, B: int, T: int, Hq: int, window: int, sinks: int = 0,
                 sm_scale: float | None = None):
        self.cache, self.window, self.sinks = cache, _int32(window, "window"), _int32(sinks, "sinks")
        c = self._c = _Caches(cache, B)
        self.sm_scale = 1.0 / math.sqrt(c.D) if sm_scale is None else float(sm_scale)
        self.o = torch.empty((B, T, Hq, c.D), dtype=c.dtype, device=c.device)
        self.lse = torch.empty((B, T, Hq), dtype=torch.float32, device=c.device)
        self.ws = _workspace(qsa_window_decode_workspace_bytes(cache, B, T, Hq, self.window, self.sinks), c.device)
        self._shape, self._fn = self.o.shape, _lib.load().qsa_window_decode
        self._head = (c.ref, B, T, Hq)
        self._tail = (self.window, self.sinks, self.sm_scale, *_outputs(c, self._shape, self.o, self.lse),
                      *_bytes(self.ws, c.index))
        self._buffers = _Buffers(c, self.o, self.lse, self.ws)

    def __call__(self, q, ctx_lens, stream=None) -> tuple[torch.Tensor, torch.Tensor]:
        c = self._c
        _call(self._fn, "qsa_window_decode", c.index,
              (*self._head, _dense(q, c.dtype, self._shape, "q", c.index), c.qd,
               _ints(ctx_lens, self._shape[0], "ctx_lens", c.index), *self._tail), stream, self._buffers)
        return self.o, self.lse


def qsa_window_prefill_workspace_bytes(cache: QSACache, B: int, n_tokens: int, max_q_per_req: int, Hq: int,
                                       window: int, sinks: int) -> int:
    return int(_lib.load().qsa_window_prefill_workspace_bytes(ctypes.byref(cache.struct()),
                                                              *_sizes(B, n_tokens, max_q_per_req, Hq, window, sinks)))


def qsa_window_prefill(cache: QSACache, cu_q: torch.Tensor, ctx_lens: torch.Tensor, max_q_per_req: int,
                       q: torch.Tensor, window: int, sinks: int, sm_scale: float, o: torch.Tensor,
                       lse: torch.Tensor, workspace: torch.Tensor | None, stream=None) -> None:
    """Window attention of a prefill chunk: rows cu_q[r] .. cu_q[r+1]-1 of q
    [N, Hq, D] are the newest tokens of request r."""
    n, Hq, _ = shape = q.shape
    B = ctx_lens.shape[0]
    c = _Caches(cache, B)
    _heads(q, c)
    ix = c.index
    _call(_lib.load().qsa_window_prefill, "qsa_window_prefill", ix,
          (c.ref, B, n, _int32(max_q_per_req, "max_q_per_req"), _ints(cu_q, B + 1, "cu_q", ix),
           _ints(ctx_lens, B, "ctx_lens", ix), _dense(q, c.dtype, shape, "q", ix), c.qd, Hq, _int32(window, "window"),
           _int32(sinks, "sinks"), float(sm_scale), *_outputs(c, shape, o, lse), *_bytes(workspace, ix)), stream)


class QSAWindowPrefill:
    """qsa_window_prefill for chunks of n_tokens rows over B requests."""

    def __init__(self, cache: QSACache, B: int, n_tokens: int, max_q_per_req: int, Hq: int, window: int,
                 sinks: int = 0, sm_scale: float | None = None):
        self.cache, self.window, self.sinks = cache, _int32(window, "window"), _int32(sinks, "sinks")
        self.B, self.max_q = B, _int32(max_q_per_req, "max_q_per_req")
        c = self._c = _Caches(cache, B)
        self.sm_scale = 1.0 / math.sqrt(c.D) if sm_scale is None else float(sm_scale)
        self.o = torch.zeros((n_tokens, Hq, c.D), dtype=c.dtype, device=c.device)
        self.lse = torch.full((n_tokens, Hq), -math.inf, dtype=torch.float32, device=c.device)
        self.ws = _workspace(qsa_window_prefill_workspace_bytes(cache, B, n_tokens, self.max_q, Hq, self.window,
                                                                self.sinks), c.device)
        self._shape, self._fn = self.o.shape, _lib.load().qsa_window_prefill
        self._head = (c.ref, B, n_tokens, self.max_q)
        self._tail = (c.qd, Hq, self.window, self.sinks, self.sm_scale,
                      *_outputs(c, self._shape, self.o, self.lse), *_bytes(self.ws, c.index))
        self._buffers = _Buffers(c, self.o, self.lse, self.ws)

    def __call__(self, q, cu_q, ctx_lens, stream=None) -> tuple[torch.Tensor, torch.Tensor]:
        c = self._c
        _call(self._fn, "qsa_window_prefill", c.index,
              (*self._head, _ints(cu_q, self.B + 1, "cu_q", c.index), _ints(ctx_lens, self.B, "ctx_lens", c.index),
               _dense(q, c.dtype, self._shape, "q", c.index), *self._tail), stream, self._buffers)
        return self.o, self.lse


# ----------------------------------------------------------------- prefix --
def qsa_prefix_decode_workspace_bytes(cache: QSACache, B: int, T: int, Hq: int, n_groups: int, max_group: int,
                                      max_prefix: int, max_tail: int) -> int:
    return int(_lib.load().qsa_prefix_decode_workspace_bytes(ctypes.byref(cache.struct()),
                                                             *_sizes(B, T, Hq, n_groups, max_group, max_prefix,
                                                                     max_tail)))


def qsa_prefix_decode(cache: QSACache, q: torch.Tensor, ctx_lens: torch.Tensor, cu_group: torch.Tensor,
                      prefix_lens: torch.Tensor, max_group: int, max_prefix: int, max_tail: int, sm_scale: float,
                      o: torch.Tensor, lse: torch.Tensor, workspace: torch.Tensor, stream=None) -> None:
    """Decode attention of q [B, T, Hq, D] where the requests of a group share
    their first prefix_lens[g] keys."""
    B, T, Hq, _ = shape = q.shape
    c = _Caches(cache, B)
    _heads(q, c)
    n, ix = prefix_lens.shape[0], c.index
    _call(_lib.load().qsa_prefix_decode, "qsa_prefix_decode", ix,
          (c.ref, B, T, Hq, _dense(q, c.dtype, shape, "q", ix), c.qd, _ints(ctx_lens, B, "ctx_lens", ix), n,
           _ints(cu_group, n + 1, "cu_group", ix), _ints(prefix_lens, n, "prefix_lens", ix),
           *(_int32(v, "a bound") for v in (max_group, max_prefix, max_tail)), float(sm_scale),
           *_outputs(c, shape, o, lse), *_bytes(workspace, ix)), stream)


class QSAPrefixDecode:
    """qsa_prefix_decode for batches of B requests in n_groups groups."""

    def __init__(self, cache: QSACache, B: int, T: int, Hq: int, n_groups: int, max_group: int, max_prefix: int,
                 max_tail: int, sm_scale: float | None = None):
        self.cache, self.n_groups = cache, n_groups
        self.bounds = tuple(_int32(v, "a bound") for v in (max_group, max_prefix, max_tail))
        c = self._c = _Caches(cache, B)
        self.sm_scale = 1.0 / math.sqrt(c.D) if sm_scale is None else float(sm_scale)
        self.o = torch.empty((B, T, Hq, c.D), dtype=c.dtype, device=c.device)
        self.lse = torch.empty((B, T, Hq), dtype=torch.float32, device=c.device)
        self.ws = _workspace(qsa_prefix_decode_workspace_bytes(cache, B, T, Hq, n_groups, *self.bounds), c.device)
        self._shape, self._fn = self.o.shape, _lib.load().qsa_prefix_decode
        self._head = (c.ref, B, T, Hq)
        self._tail = (*self.bounds, self.sm_scale, *_outputs(c, self._shape, self.o, self.lse),
                      *_bytes(self.ws, c.index))
        self._buffers = _Buffers(c, self.o, self.lse, self.ws)

    def __call__(self, q, ctx_lens, cu_group, prefix_lens, stream=None) -> tuple[torch.Tensor, torch.Tensor]:
        c, n = self._c, self.n_groups
        _call(self._fn, "qsa_prefix_decode", c.index,
              (*self._head, _dense(q, c.dtype, self._shape, "q", c.index), c.qd,
               _ints(ctx_lens, self._shape[0], "ctx_lens", c.index), n,
               _ints(cu_group, n + 1, "cu_group", c.index), _ints(prefix_lens, n, "prefix_lens", c.index),
               *self._tail), stream, self._buffers)
        return self.o, self.lse
