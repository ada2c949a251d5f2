"""Binding of the calls over whole key ranges of the paged K/V cache: rotary
append, window attention (decode and prefill) and shared-prefix decode.

Each C entry point has a function of its name, which checks its arguments and
marshals them, and a class that holds what a serving loop keeps between calls
(the cache description, the output buffers and the workspace).  A class takes
the cache's tensors when it is made: their contents may change, the tensors
may not be replaced.  Its outputs are its own buffers, overwritten by its next
call.  Work goes to `stream`, by default the current stream of the tensors'
device.
"""
from __future__ import annotations

import contextlib
import ctypes
import math

import torch

from . import _lib
from .api import _KV_DTYPES, QSACache, _check, _need, new_workspace

_Q_DTYPES = {torch.float32: _lib.QSA_F32, torch.bfloat16: _lib.QSA_BF16}
_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3}
_HERE = contextlib.nullcontext()


def _device(index: int):
    """The caches' device as the current one, for the launch."""
    return _HERE if torch.cuda.current_device() == index else torch.cuda.device(index)


def _stream(stream, index: int) -> int:
    return stream.cuda_stream if stream is not None else torch.cuda.current_stream(index).cuda_stream


def _query_type(cache: QSACache) -> torch.dtype:
    if cache.k_cache.dtype not in _KV_DTYPES:
        raise TypeError("k_cache must be float32, bfloat16 or float8_e4m3fn")
    return torch.float32 if cache.k_cache.dtype == torch.float32 else torch.bfloat16


def _ints(t: torch.Tensor, n: int, name: str, device: torch.device) -> int:
    if t.dtype != torch.int32 or t.shape != (n,) or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor of {n} entries on the cache's device")
    return t.data_ptr()


def _dense(t: torch.Tensor, dtype: torch.dtype, shape: tuple, name: str, device: torch.device) -> int:
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous tensor of shape {list(shape)} on the cache's device")
    return t.data_ptr()


def _bytes(workspace: torch.Tensor | None, device: torch.device) -> tuple[int | None, int]:
    if workspace is None:
        return None, 0
    if workspace.device != device or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the cache's device")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _workspace(nbytes: int, device) -> torch.Tensor | None:
    return new_workspace(nbytes, device) if nbytes else None


# ------------------------------------------------------------------- rope --
def qsa_rope_freqs(rotary_dim: int, theta: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                   original_max_position: int = 0, beta_fast: float = 32.0,
                   beta_slow: float = 1.0) -> tuple[list[int], list[float], float]:
    """(freqs, inv_freq, mscale): the rotated pairs' turns per token in units
    of 2^-64, their radians per token, and the factor on the rotated dims."""
    if scaling not in _SCALINGS:
        raise ValueError(f"scaling must be one of {sorted(_SCALINGS)}")
    n = max(int(rotary_dim), 0) // 2
    fr, inv, m = (ctypes.c_uint64 * max(n, 1))(), (ctypes.c_double * max(n, 1))(), ctypes.c_float()
    _check(_lib.load().qsa_rope_freqs(int(rotary_dim), float(theta), _SCALINGS[scaling], float(factor),
                                      int(original_max_position), float(beta_fast), float(beta_slow),
                                      ctypes.addressof(inv), ctypes.addressof(fr), ctypes.byref(m)),
           "qsa_rope_freqs")
    return list(fr[:n]), list(inv[:n]), m.value


def _rows(t: torch.Tensor, dtype, heads: int, D: int, n: int, name: str, device) -> tuple[int, int]:
    """(pointer, row stride) of t [n, heads, D] whose rows are dense."""
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != (n, heads, D) or t.device != device:
        raise ValueError(f"{name} must be [{n}, {heads}, {D}] on the cache's device")
    s = t.stride()
    if (s[2] != 1 or (heads > 1 and s[1] != D)) and n > 0:
        raise ValueError(f"the heads of a row of {name} must be dense")
    return t.data_ptr(), s[0] if n > 1 else heads * D


def _rope_append(ref, cache, freqs, rotary_dim, interleaved, mscale, pos0, cu_new, q, k, v, q_out, stream):
    kc = cache.k_cache
    dev, (_, _, Hkv, D) = kc.device, kc.shape
    dt = _query_type(cache)
    n, Hq = q.shape[0], q.shape[1]
    B = pos0.shape[0]
    qp, qs = _rows(q, dt, Hq, D, n, "q", dev)
    kp, ks = _rows(k, dt, Hkv, D, n, "k", dev)
    vp, vs = _rows(v, dt, Hkv, D, n, "v", dev)
    op = _dense(q_out, dt, (n, Hq, D), "q_out", dev)
    args = (ref, B, n, _ints(pos0, B, "pos0", dev), _ints(cu_new, B + 1, "cu_new", dev), qp, qs, kp, ks, vp, vs,
            _Q_DTYPES[dt], Hq, freqs.data_ptr() if rotary_dim else None, rotary_dim, 1 if interleaved else 0,
            mscale, op)
    with _device(dev.index):
        _check(_lib.load().qsa_rope_append(*args, _stream(stream, dev.index)), "qsa_rope_append")


def qsa_rope_append(cache: QSACache, pos0: torch.Tensor, cu_new: torch.Tensor, q: torch.Tensor,
                    k: torch.Tensor, v: torch.Tensor, freqs: torch.Tensor, rotary_dim: int,
                    interleaved: bool, mscale: float, q_out: torch.Tensor, stream=None) -> None:
    """Rotates q [N, Hq, D] into q_out and k [N, Hkv, D] into the cache's
    pages, and copies v there.  `freqs`: int64 [rotary_dim / 2] on the cache's
    device, the bits of qsa_rope_freqs.  q, k, v may be strided over tokens
    (parts of one fused projection)."""
    rotary_dim = int(rotary_dim)
    _need(freqs, torch.int64, "freqs")
    if freqs.shape != (max(rotary_dim, 0) // 2,) or freqs.device != cache.k_cache.device or not freqs.is_contiguous():
        raise ValueError("freqs must hold rotary_dim / 2 entries on the cache's device")
    s = cache.struct()
    _rope_append(ctypes.byref(s), cache, freqs, rotary_dim, interleaved, float(mscale), pos0, cu_new, q, k, v,
                 q_out, stream)


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
        self._struct = cache.struct()
        self._ref = ctypes.byref(self._struct)

    def __call__(self, pos0, cu_new, q, k, v, q_out=None, stream=None) -> torch.Tensor:
        if q.dim() != 3 or q.shape[1] != self.Hq:
            raise ValueError(f"q must be [N, {self.Hq}, D]")
        if q_out is None:
            q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        _rope_append(self._ref, self.cache, self.freqs, self.rotary_dim, self.interleaved, self.mscale, pos0,
                     cu_new, q, k, v, q_out, stream)
        return q_out


# ----------------------------------------------------------------- window --
def qsa_window_decode_workspace_bytes(cache: QSACache, B: int, T: int, Hq: int, window: int, sinks: int) -> int:
    return int(_lib.load().qsa_window_decode_workspace_bytes(ctypes.byref(cache.struct()), B, T, Hq, window, sinks))


def _window_decode(ref, cache, q, ctx_lens, window, sinks, sm_scale, o, lse, workspace, stream):
    kc = cache.k_cache
    dev, dt = kc.device, _query_type(cache)
    B, T, Hq, D = q.shape
    if D != kc.shape[3]:
        raise ValueError("q and the cache have different head dims")
    wp, wn = _bytes(workspace, dev)
    args = (ref, B, T, Hq, _dense(q, dt, (B, T, Hq, D), "q", dev), _Q_DTYPES[dt],
            _ints(ctx_lens, B, "ctx_lens", dev), window, sinks, sm_scale, _dense(o, dt, (B, T, Hq, D), "o", dev),
            _dense(lse, torch.float32, (B, T, Hq), "lse", dev), wp, wn)
    with _device(dev.index):
        _check(_lib.load().qsa_window_decode(*args, _stream(stream, dev.index)), "qsa_window_decode")


def qsa_window_decode(cache: QSACache, q: torch.Tensor, ctx_lens: torch.Tensor, window: int, sinks: int,
                      sm_scale: float, o: torch.Tensor, lse: torch.Tensor, workspace: torch.Tensor | None,
                      stream=None) -> None:
    """Decode attention of q [B, T, Hq, D] over each request's last `window`
    keys and first `sinks` keys.  o: q's type and shape, lse float32."""
    s = cache.struct()
    _window_decode(ctypes.byref(s), cache, q, ctx_lens, int(window), int(sinks), float(sm_scale), o, lse,
                   workspace, stream)


class QSAWindowDecode:
    """qsa_window_decode for batches of B requests with T query tokens."""

    def __init__(self, cache: QSACache, B: int, T: int, Hq: int, window: int, sinks: int = 0,
                 sm_scale: float | None = None):
        dev, D = cache.k_cache.device, cache.k_cache.shape[-1]
        self.cache, self.window, self.sinks = cache, int(window), int(sinks)
        self.sm_scale = 1.0 / math.sqrt(D) if sm_scale is None else float(sm_scale)
        self._struct = cache.struct()
        self._ref = ctypes.byref(self._struct)
        self.o = torch.empty((B, T, Hq, D), dtype=_query_type(cache), device=dev)
        self.lse = torch.empty((B, T, Hq), dtype=torch.float32, device=dev)
        self.ws = _workspace(qsa_window_decode_workspace_bytes(cache, B, T, Hq, self.window, self.sinks), dev)

    def __call__(self, q, ctx_lens, stream=None) -> tuple[torch.Tensor, torch.Tensor]:
        if q.shape != self.o.shape:
            raise ValueError(f"q must be {list(self.o.shape)}")
        _window_decode(self._ref, self.cache, q, ctx_lens, self.window, self.sinks, self.sm_scale, self.o,
                       self.lse, self.ws, stream)
        return self.o, self.lse


def qsa_window_prefill_workspace_bytes(cache: QSACache, B: int, n_tokens: int, max_q_per_req: int, Hq: int,
                                       window: int, sinks: int) -> int:
    return int(_lib.load().qsa_window_prefill_workspace_bytes(ctypes.byref(cache.struct()), B, n_tokens,
                                                              max_q_per_req, Hq, window, sinks))


def _window_prefill(ref, cache, cu_q, ctx_lens, max_q_per_req, q, window, sinks, sm_scale, o, lse, workspace, stream):
    kc = cache.k_cache
    dev, dt = kc.device, _query_type(cache)
    n, Hq, D = q.shape
    if D != kc.shape[3]:
        raise ValueError("q and the cache have different head dims")
    B = ctx_lens.shape[0]
    wp, wn = _bytes(workspace, dev)
    args = (ref, B, n, max_q_per_req, _ints(cu_q, B + 1, "cu_q", dev), _ints(ctx_lens, B, "ctx_lens", dev),
            _dense(q, dt, (n, Hq, D), "q", dev), _Q_DTYPES[dt], Hq, window, sinks, sm_scale,
            _dense(o, dt, (n, Hq, D), "o", dev), _dense(lse, torch.float32, (n, Hq), "lse", dev), wp, wn)
    with _device(dev.index):
        _check(_lib.load().qsa_window_prefill(*args, _stream(stream, dev.index)), "qsa_window_prefill")


def qsa_window_prefill(cache: QSACache, cu_q: torch.Tensor, ctx_lens: torch.Tensor, max_q_per_req: int,
                       q: torch.Tensor, window: int, sinks: int, sm_scale: float, o: torch.Tensor,
                       lse: torch.Tensor, workspace: torch.Tensor | None, stream=None) -> None:
    """Window attention of a prefill chunk: rows cu_q[r] .. cu_q[r+1]-1 of q
    [N, Hq, D] are the newest tokens of request r."""
    s = cache.struct()
    _window_prefill(ctypes.byref(s), cache, cu_q, ctx_lens, int(max_q_per_req), q, int(window), int(sinks),
                    float(sm_scale), o, lse, workspace, stream)


class QSAWindowPrefill:
    """qsa_window_prefill for chunks of n_tokens rows over B requests."""

    def __init__(self, cache: QSACache, B: int, n_tokens: int, max_q_per_req: int, Hq: int, window: int,
                 sinks: int = 0, sm_scale: float | None = None):
        dev, D = cache.k_cache.device, cache.k_cache.shape[-1]
        self.cache, self.window, self.sinks = cache, int(window), int(sinks)
        self.B, self.max_q = B, int(max_q_per_req)
        self.sm_scale = 1.0 / math.sqrt(D) if sm_scale is None else float(sm_scale)
        self._struct = cache.struct()
        self._ref = ctypes.byref(self._struct)
        self.o = torch.zeros((n_tokens, Hq, D), dtype=_query_type(cache), device=dev)
        self.lse = torch.full((n_tokens, Hq), -math.inf, dtype=torch.float32, device=dev)
        self.ws = _workspace(qsa_window_prefill_workspace_bytes(cache, B, n_tokens, self.max_q, Hq, self.window,
                                                                self.sinks), dev)

    def __call__(self, q, cu_q, ctx_lens, stream=None) -> tuple[torch.Tensor, torch.Tensor]:
        if q.shape != self.o.shape or ctx_lens.shape != (self.B,):
            raise ValueError(f"q must be {list(self.o.shape)} and ctx_lens [{self.B}]")
        _window_prefill(self._ref, self.cache, cu_q, ctx_lens, self.max_q, q, self.window, self.sinks,
                        self.sm_scale, self.o, self.lse, self.ws, stream)
        return self.o, self.lse


# ----------------------------------------------------------------- prefix --
def qsa_prefix_decode_workspace_bytes(cache: QSACache, B: int, T: int, Hq: int, n_groups: int, max_group: int,
                                      max_prefix: int, max_tail: int) -> int:
    return int(_lib.load().qsa_prefix_decode_workspace_bytes(ctypes.byref(cache.struct()), B, T, Hq, n_groups,
                                                             max_group, max_prefix, max_tail))


def _prefix_decode(ref, cache, q, ctx_lens, cu_group, prefix_lens, max_group, max_prefix, max_tail, sm_scale, o,
                   lse, workspace, stream):
    kc = cache.k_cache
    dev, dt = kc.device, _query_type(cache)
    B, T, Hq, D = q.shape
    if D != kc.shape[3]:
        raise ValueError("q and the cache have different head dims")
    n = prefix_lens.shape[0]
    wp, wn = _bytes(workspace, dev)
    args = (ref, B, T, Hq, _dense(q, dt, (B, T, Hq, D), "q", dev), _Q_DTYPES[dt],
            _ints(ctx_lens, B, "ctx_lens", dev), n, _ints(cu_group, n + 1, "cu_group", dev),
            _ints(prefix_lens, n, "prefix_lens", dev), max_group, max_prefix, max_tail, sm_scale,
            _dense(o, dt, (B, T, Hq, D), "o", dev), _dense(lse, torch.float32, (B, T, Hq), "lse", dev), wp, wn)
    with _device(dev.index):
        _check(_lib.load().qsa_prefix_decode(*args, _stream(stream, dev.index)), "qsa_prefix_decode")


def qsa_prefix_decode(cache: QSACache, q: torch.Tensor, ctx_lens: torch.Tensor, cu_group: torch.Tensor,
                      prefix_lens: torch.Tensor, max_group: int, max_prefix: int, max_tail: int, sm_scale: float,
                      o: torch.Tensor, lse: torch.Tensor, workspace: torch.Tensor, stream=None) -> None:
    """Decode attention of q [B, T, Hq, D] where the requests of a group share
    their first prefix_lens[g] keys."""
    s = cache.struct()
    _prefix_decode(ctypes.byref(s), cache, q, ctx_lens, cu_group, prefix_lens, int(max_group), int(max_prefix),
                   int(max_tail), float(sm_scale), o, lse, workspace, stream)


class QSAPrefixDecode:
    """qsa_prefix_decode for batches of B requests in n_groups groups."""

    def __init__(self, cache: QSACache, B: int, T: int, Hq: int, n_groups: int, max_group: int, max_prefix: int,
                 max_tail: int, sm_scale: float | None = None):
        dev, D = cache.k_cache.device, cache.k_cache.shape[-1]
        self.cache, self.n_groups = cache, n_groups
        self.bounds = (int(max_group), int(max_prefix), int(max_tail))
        self.sm_scale = 1.0 / math.sqrt(D) if sm_scale is None else float(sm_scale)
        self._struct = cache.struct()
        self._ref = ctypes.byref(self._struct)
        self.o = torch.empty((B, T, Hq, D), dtype=_query_type(cache), device=dev)
        self.lse = torch.empty((B, T, Hq), dtype=torch.float32, device=dev)
        self.ws = _workspace(qsa_prefix_decode_workspace_bytes(cache, B, T, Hq, n_groups, *self.bounds), dev)

    def __call__(self, q, ctx_lens, cu_group, prefix_lens, stream=None) -> tuple[torch.Tensor, torch.Tensor]:
        if q.shape != self.o.shape or prefix_lens.shape != (self.n_groups,):
            raise ValueError(f"q must be {list(self.o.shape)} and prefix_lens [{self.n_groups}]")
        _prefix_decode(self._ref, self.cache, q, ctx_lens, cu_group, prefix_lens, *self.bounds, self.sm_scale,
                       self.o, self.lse, self.ws, stream)
        return self.o, self.lse
