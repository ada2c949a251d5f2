"""Rotary append, window attention and shared-prefix decode: what the host
checks before anything is launched, the frequencies, and the workspace sizes.
No GPU."""
import ctypes
import math

import pytest
import torch

from sparse_attention_decode_compress_b200 import QSAError, _lib, qsa_rope_freqs

OK, INVALID, UNSUPPORTED = 0, 1, 2
P = 1 << 20  # an aligned address that nothing reads: every call below is refused


def cache(**kw):
    s = _lib.QsaCacheStruct()
    s.num_pages, s.page_size, s.num_kv_heads, s.head_dim, s.idx_dim = 10, 64, 2, 128, 0
    s.kv_dtype, s.ring_rows, s.max_pages_per_req = _lib.QSA_BF16, 0, 4
    s.k_cache = s.v_cache = s.block_table = P
    for k, v in kw.items():
        setattr(s, k, v)
    return ctypes.byref(s)


# ------------------------------------------------------------ frequencies --
def test_frequencies_are_the_formula():
    for R, theta in ((128, 1e6), (64, 1e4), (2, 1e4), (48, 500000.0)):
        turns, inv, m = qsa_rope_freqs(R, theta)
        assert m == 1.0 and len(turns) == len(inv) == R // 2
        for i, (t, f) in enumerate(zip(turns, inv)):
            assert math.isclose(f, theta ** (-2 * i / R), rel_tol=1e-14)
            # float64 division, and the cut to whole units of 2^-64 (a slow
            # pair's fraction has few of them: the error is absolute)
            assert math.isclose(t / 2 ** 64, f / (2 * math.pi), rel_tol=1e-14, abs_tol=2.0 ** -64)


def test_scaled_frequencies():
    R, theta, s = 64, 1e4, 4.0
    plain = qsa_rope_freqs(R, theta)[1]
    _, lin, m = qsa_rope_freqs(R, theta, "linear", s)
    assert m == 1.0 and all(math.isclose(a, b / s, rel_tol=1e-14) for a, b in zip(lin, plain))
    _, ntk, m = qsa_rope_freqs(R, theta, "ntk", s)
    # the fastest pair is unchanged, the slowest is stretched by the factor
    assert m == 1.0 and ntk[0] == 1.0 and math.isclose(ntk[-1], plain[-1] / s, rel_tol=1e-12)
    _, yarn, m = qsa_rope_freqs(R, theta, "yarn", s, 4096)
    assert math.isclose(m, 0.1 * math.log(s) + 1, rel_tol=1e-6)
    for a, b in zip(yarn, plain):
        turns = 4096 * b / (2 * math.pi)
        assert b / s * (1 - 1e-12) <= a <= b * (1 + 1e-12)
        if turns > 64:
            assert a == b
        if turns < 0.5:
            assert math.isclose(a, b / s, rel_tol=1e-14)
    assert all(x >= y for x, y in zip(yarn, yarn[1:]))


def test_whole_turns_fall_away():
    # a position's angle is freqs * position modulo one turn, however far
    turns, inv, _ = qsa_rope_freqs(64, 1e6)
    for t, f in zip(turns, inv):
        for p in (1, 1000, 2 ** 31 - 1):
            want = math.fmod(p * f / (2 * math.pi), 1.0)
            got = (p * t % 2 ** 64) / 2 ** 64
            d = abs(got - want)
            # p units of 2^-64, and float64's rounding of the turns themselves
            assert min(d, 1 - d) < p * 2.0 ** -64 + 2.0 ** -50 * max(1.0, p * f)


@pytest.mark.parametrize("kw", [dict(rotary_dim=3), dict(rotary_dim=-2), dict(rotary_dim=130),
                                dict(rotary_dim=64, theta=1.0), dict(rotary_dim=64, theta=math.nan),
                                dict(rotary_dim=64, theta=math.inf),
                                dict(rotary_dim=64, scaling="linear", factor=0.5),
                                dict(rotary_dim=2, scaling="ntk", factor=2.0),
                                dict(rotary_dim=64, scaling="yarn", factor=2.0),
                                dict(rotary_dim=64, scaling="yarn", factor=2.0, original_max_position=64,
                                     beta_slow=0.0),
                                dict(rotary_dim=64, scaling="yarn", factor=2.0, original_max_position=64,
                                     beta_fast=0.5)])
def test_frequency_refusals(kw):
    with pytest.raises(QSAError):
        qsa_rope_freqs(**kw)


def test_unknown_scaling():
    with pytest.raises(ValueError):
        qsa_rope_freqs(64, scaling="other")


# ---------------------------------------------------------------- refusals --
def rope(c=None, B=2, n=4, pos0=P, cu=P, q=P, qs=2048, k=P, ks=256, v=P, vs=256, dt=_lib.QSA_BF16, Hq=16,
         freqs=P, R=128, layout=0, m=1.0, out=2 * P):
    return _lib.load().qsa_rope_append(c or cache(), B, n, pos0, cu, q, qs, k, ks, v, vs, dt, Hq, freqs, R,
                                       layout, m, out, None)


@pytest.mark.parametrize("kw,want", [
    (dict(B=-1), INVALID), (dict(n=-1), INVALID), (dict(Hq=0), INVALID), (dict(R=3), INVALID),
    (dict(R=130), INVALID), (dict(R=-2), INVALID), (dict(layout=2), INVALID), (dict(m=math.nan), INVALID),
    (dict(pos0=None), INVALID), (dict(cu=None), INVALID), (dict(q=None), INVALID), (dict(k=None), INVALID),
    (dict(v=None), INVALID), (dict(out=None), INVALID), (dict(freqs=None), INVALID),
    (dict(q=P + 1), INVALID), (dict(freqs=P + 4), INVALID), (dict(qs=2047), INVALID), (dict(ks=255), INVALID),
    (dict(vs=0), INVALID), (dict(out=P, qs=4096), INVALID), (dict(dt=_lib.QSA_F32), UNSUPPORTED),
    (dict(c=cache(head_dim=96), R=64), UNSUPPORTED), (dict(c=cache(kv_dtype=7)), UNSUPPORTED),
    (dict(c=cache(kv_dtype=_lib.QSA_F32)), UNSUPPORTED), (dict(c=cache(kv_dtype=_lib.QSA_FP8_E4M3)), INVALID),
    (dict(c=cache(k_cache=None)), INVALID), (dict(c=cache(page_size=6)), INVALID),
    (dict(c=cache(block_table=None)), INVALID), (dict(B=0), OK), (dict(n=0), OK)])
def test_rope_append_refusals(kw, want):
    assert rope(**kw) == want


def window(c=None, B=2, T=1, Hq=16, q=P, dt=_lib.QSA_BF16, ctx=P, W=64, S=4, scale=1.0, o=P, lse=P, ws=P,
           nws=1 << 40):
    return _lib.load().qsa_window_decode(c or cache(), B, T, Hq, q, dt, ctx, W, S, scale, o, lse, ws, nws, None)


def chunk(c=None, B=2, n=8, mq=8, cu=P, ctx=P, q=P, dt=_lib.QSA_BF16, Hq=16, W=64, S=4, scale=1.0, o=P, lse=P,
          ws=P, nws=1 << 40):
    return _lib.load().qsa_window_prefill(c or cache(), B, n, mq, cu, ctx, q, dt, Hq, W, S, scale, o, lse, ws,
                                          nws, None)


def prefix(c=None, B=2, T=1, Hq=16, q=P, dt=_lib.QSA_BF16, ctx=P, ng=1, cu=P, pl=P, mg=2, mp=64, mt=64, scale=1.0,
           o=P, lse=P, ws=P, nws=1 << 40):
    return _lib.load().qsa_prefix_decode(c or cache(), B, T, Hq, q, dt, ctx, ng, cu, pl, mg, mp, mt, scale, o, lse,
                                         ws, nws, None)


COMMON = [(dict(B=-1), INVALID), (dict(Hq=0), INVALID), (dict(Hq=15), INVALID), (dict(scale=0.0), INVALID),
          (dict(scale=math.inf), INVALID), (dict(q=None), INVALID), (dict(q=P + 2), INVALID),
          (dict(ctx=None), INVALID), (dict(o=None), INVALID), (dict(o=P + 8), INVALID), (dict(lse=None), INVALID),
          (dict(dt=_lib.QSA_F32), UNSUPPORTED), (dict(c=cache(kv_dtype=_lib.QSA_F32)), UNSUPPORTED),
          (dict(c=cache(kv_dtype=_lib.QSA_FP8_E4M3)), INVALID), (dict(c=cache(head_dim=32)), UNSUPPORTED),
          (dict(c=cache(v_cache=P + 8)), INVALID), (dict(c=cache(page_size=2)), INVALID),
          (dict(c=cache(max_pages_per_req=0)), INVALID), (dict(B=65536), UNSUPPORTED), (dict(Hq=128), UNSUPPORTED),
          (dict(B=0), OK)]


@pytest.mark.parametrize("kw,want", COMMON + [
    (dict(T=0), INVALID), (dict(T=5), UNSUPPORTED), (dict(T=4, Hq=32), UNSUPPORTED), (dict(W=0), INVALID),
    (dict(S=-1), INVALID), (dict(W=1 << 20, c=cache(max_pages_per_req=400), ws=None), INVALID),
    (dict(W=1 << 20, c=cache(max_pages_per_req=400), nws=100), INVALID),
    (dict(W=1 << 20, c=cache(max_pages_per_req=400), ws=P + 16), INVALID)])
def test_window_decode_refusals(kw, want):
    assert window(**kw) == want


@pytest.mark.parametrize("kw,want", COMMON + [
    (dict(n=-1), INVALID), (dict(mq=-1), INVALID), (dict(W=0), INVALID), (dict(S=-1), INVALID),
    (dict(cu=None), INVALID), (dict(n=0), OK), (dict(mq=0), OK)])
def test_window_prefill_refusals(kw, want):
    assert chunk(**kw) == want


@pytest.mark.parametrize("kw,want", COMMON + [
    (dict(T=0), INVALID), (dict(T=5), UNSUPPORTED), (dict(ng=0), INVALID), (dict(ng=3), INVALID),
    (dict(mg=0), INVALID), (dict(mg=3), INVALID), (dict(mp=-1), INVALID), (dict(mt=-1), INVALID),
    (dict(cu=None), INVALID), (dict(pl=None), INVALID), (dict(ws=None), INVALID), (dict(nws=16), INVALID),
    (dict(ws=P + 16), INVALID)])
def test_prefix_decode_refusals(kw, want):
    assert prefix(**kw) == want


# --------------------------------------------------------------- workspace --
def test_workspace_bytes():
    lib = _lib.load()
    big = cache(max_pages_per_req=4096)
    w = lib.qsa_window_decode_workspace_bytes
    # no key range to split: none needed, and none for malformed arguments
    assert w(big, 300, 1, 16, 16, 0) == 0
    for bad in ((0, 1, 16, 64, 0), (2, 0, 16, 64, 0), (2, 1, 15, 64, 0), (2, 1, 16, 0, 0), (2, 1, 16, 64, -1)):
        assert w(big, *bad) == 0
    # one slot takes D + 1 floats of every (token, head) row
    n = w(big, 1, 1, 16, 1 << 20, 0)
    assert n > 0 and n % 256 == 0
    # a window wider than the block table holds needs no more than the table
    assert w(big, 1, 1, 16, 2 ** 31 - 1, 2 ** 31 - 1) == w(big, 1, 1, 16, 4096 * 64, 0)
    p = lib.qsa_prefix_decode_workspace_bytes
    assert p(big, 32, 1, 16, 1, 32, 4096, 100) >= 2 * 32 * 16 * 129 * 4
    for bad in ((32, 1, 16, 0, 32, 64, 64), (32, 1, 16, 33, 32, 64, 64), (32, 1, 16, 1, 0, 64, 64),
                (32, 1, 16, 1, 33, 64, 64), (32, 1, 16, 1, 32, -1, 64), (32, 1, 16, 1, 32, 64, -1)):
        assert p(big, *bad) == 0
    assert lib.qsa_window_prefill_workspace_bytes(big, 0, 8, 8, 16, 64, 0) == 0


# ----------------------------------------------------------------- binding --
def test_binding_refuses_host_tensors_and_wrong_types():
    from sparse_attention_decode_compress_b200 import QSACache, QSARopeAppend, QSAWindowDecode
    k = torch.zeros((4, 16, 2, 64), dtype=torch.bfloat16)
    c = QSACache.allocate(k, k.clone(), torch.zeros((2, 2), dtype=torch.int32), 32, 2)
    with pytest.raises(ValueError):
        QSAWindowDecode(c, 2, 1, 4, 16)
    with pytest.raises(ValueError):
        QSARopeAppend(c, 4, rotary_dim=66)


@pytest.mark.parametrize("v", [1 << 31, (1 << 32) + 5, -(1 << 31) - 1])
def test_binding_refuses_what_does_not_fit_32_bits(v):
    """(ctypes would keep the low 32 bits without a word)"""
    from sparse_attention_decode_compress_b200 import QSACache, QSAPrefixDecode, QSAWindowDecode, QSAWindowPrefill
    k = torch.zeros((4, 16, 2, 64), dtype=torch.bfloat16)
    c = QSACache.allocate(k, k.clone(), torch.zeros((2, 2), dtype=torch.int32), 32, 2)
    for make in (lambda: QSAWindowDecode(c, 2, 1, 4, v), lambda: QSAWindowDecode(c, 2, 1, 4, 16, v),
                 lambda: QSAWindowPrefill(c, 2, 8, v, 4, 16), lambda: QSAPrefixDecode(c, 2, 1, 4, 1, 1, v, 1)):
        with pytest.raises(ValueError, match="32 bits"):
            make()


def host_cache(rows=2, kv=torch.bfloat16, **kw):
    from sparse_attention_decode_compress_b200 import QSACache
    k = torch.zeros((4, 16, 2, 64)).to(kv)
    c = QSACache.allocate(k, k.clone(), torch.zeros((rows, 2), dtype=torch.int32), 32, rows)
    for name, v in kw.items():
        setattr(c, name, v)
    return c


def all_calls(c, B):
    """Every call of the module on cache c for B requests (host tensors: the
    shapes are looked at before the devices)."""
    import sparse_attention_decode_compress_b200 as qsa
    i32 = lambda n: torch.zeros(n, dtype=torch.int32)
    dt = torch.float32 if c.k_cache.dtype == torch.float32 else torch.bfloat16
    q, o, lse = (torch.zeros(s, dtype=t) for s, t in (((B, 1, 4, 64), dt), ((B, 1, 4, 64), dt),
                                                      ((B, 1, 4), torch.float32)))
    r, ro, rl = q[:, 0], o[:, 0], lse[:, 0]
    return [lambda: qsa.QSAWindowDecode(c, B, 1, 4, 16), lambda: qsa.QSAWindowPrefill(c, B, B, 1, 4, 16),
            lambda: qsa.QSAPrefixDecode(c, B, 1, 4, 1, 1, 16, 16),
            lambda: qsa.qsa_window_decode(c, q, i32(B), 16, 0, 1.0, o, lse, None),
            lambda: qsa.qsa_window_prefill(c, i32(B + 1), i32(B), 1, r, 16, 0, 1.0, ro, rl, None),
            lambda: qsa.qsa_prefix_decode(c, q, i32(B), i32(2), i32(1), 1, 16, 16, 1.0, o, lse, None)]


def test_more_requests_than_the_block_table_has_rows():
    """(the kernels would read behind the table)"""
    for call in all_calls(host_cache(rows=2), 3):
        with pytest.raises(ValueError, match="2 rows for 3 requests"):
            call()
    for call in all_calls(host_cache(block_table=torch.zeros(8, dtype=torch.int32)), 2):
        with pytest.raises(ValueError, match=r"\[requests, pages\]"):
            call()


def test_scales_of_8_bit_caches():
    """(a short or differently typed scale would be read behind its end)"""
    f8, good = torch.float8_e4m3fn, torch.ones(4, 2)
    for bad in (None, good.to(torch.bfloat16), good.double(), torch.ones(8), torch.ones(3, 2), torch.ones(2, 4)):
        for kw in (dict(k_scale=bad, v_scale=good), dict(k_scale=good, v_scale=bad)):
            for call in all_calls(host_cache(kv=f8, **kw), 2):
                with pytest.raises(ValueError, match=r"8-bit cache must be float32 \[4, 2\]"):
                    call()
    # the host caches above are refused for being on the host, and for nothing before
    for call in all_calls(host_cache(kv=f8, k_scale=good, v_scale=good), 2) + all_calls(host_cache(), 2):
        with pytest.raises(ValueError, match="CUDA tensors"):
            call()


@pytest.mark.parametrize("v", [1 << 31, (1 << 32) + 64, -(1 << 31) - 1])
def test_frequencies_and_workspaces_refuse_what_does_not_fit_32_bits(v):
    import sparse_attention_decode_compress_b200 as qsa
    with pytest.raises(ValueError, match="32 bits"):
        qsa_rope_freqs(v)
    with pytest.raises(ValueError, match="32 bits"):
        qsa_rope_freqs(64, scaling="yarn", factor=2.0, original_max_position=v)

    class Described:  # the workspace calls read a cache's geometry alone
        def struct(self):
            return cache()._obj

    for fn, n in ((qsa.qsa_window_decode_workspace_bytes, 5), (qsa.qsa_window_prefill_workspace_bytes, 6),
                  (qsa.qsa_prefix_decode_workspace_bytes, 7)):
        fn(Described(), *[2] * n)
        for i in range(n):
            with pytest.raises(ValueError, match="32 bits"):
                fn(Described(), *[v if j == i else 2 for j in range(n)])


# ------------------------------------------------- layers without an index --
def test_a_cache_without_an_index():
    """What reads neither compressed keys nor the ring needs none of them; what
    does is refused."""
    from sparse_attention_decode_compress_b200 import (QSACache, QSASession, allocate_norm_caches,
                                                       qsa_sparse_prefill)
    k = torch.zeros((4, 16, 2, 64), dtype=torch.bfloat16)
    c = QSACache.allocate(k, k.clone(), torch.zeros((2, 2), dtype=torch.int32), 0, 0)
    assert c.kc is None and c.ring is None
    for call in all_calls(c, 2):  # refused for being on the host alone
        with pytest.raises(ValueError, match="CUDA tensors"):
            call()
    q, i = torch.zeros((2, 4, 64), dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32)
    for call in (lambda: allocate_norm_caches(c, 2),
                 lambda: qsa_sparse_prefill(c, i, i[:2], 1, q[:, 0].to(torch.int8), q[:, 0].to(torch.int8), q, 4, 4, 1.0,
                                            torch.zeros((2, 4), dtype=torch.int32), q.float(), q[..., 0].float(), q)):
        with pytest.raises(ValueError, match="no compressed keys"):
            call()
    half = QSACache(k, k.clone(), None, torch.zeros((2, 4, 32), dtype=torch.int8), c.block_table)
    with pytest.raises(ValueError, match="both or neither"):
        half.struct()
    # the C entries refuse the struct of such a cache
    lib, s = _lib.load(), cache()
    assert lib.qsa_compress_append(s, 2, P, P, P, 1, None) == INVALID
    assert lib.qsa_index_topk(s, 2, P, P, None, 4, 4, P, None, P, 1 << 30, None) == INVALID
    assert lib.qsa_index_topk_noalloc(s, 2, P, P, None, 4, 4, P, None) == INVALID
