"""Rotary append, window attention and shared-prefix decode on the GPU against
their plain float64 forms (tests/attn_oracle.py), at the sizes and masks where
they can go wrong."""
import math

import numpy as np
import pytest
import torch

import attn_oracle as A
from sparse_attention_decode_compress_b200 import (QSAPrefixDecode, QSARopeAppend, QSAWindowDecode,
                                                   QSAWindowPrefill, qsa_get_device_error, qsa_rope_append)

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _cuda_and_cleanup():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    yield
    torch.cuda.synchronize()
    assert qsa_get_device_error() == (0, 0)
    torch.cuda.empty_cache()


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def queries(shape, kv, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(torch.float32 if kv == "f32" else torch.bfloat16)


# ------------------------------------------------------------------ window --
def window_want(kv, q, lens, T, window, sinks):
    """Per request rows; also the keys each request reads."""
    rows, seen = [], {}
    for r, L in enumerate(lens):
        toks = []
        seen[r] = set()
        for t in range(T):
            keys = A.visible(L - T + t, window, sinks)
            seen[r] |= set(keys)
            toks.append(A.attend(q[r, t], kv.values("k", r, keys), kv.values("v", r, keys), kv.D ** -0.5))
        rows.append(A.stack(toks))
    return A.stack(rows), seen


WINDOW = [
    # kv, Hq, Hkv, D, T, page, window, sinks, lens
    ("f32", 8, 1, 64, 1, 16, 100, 4, [1, 2, 99, 100, 101, 104, 105, 400, 0]),
    ("f32", 4, 4, 128, 3, 4, 33, 0, [3, 35, 36, 37, 2, 1, 0, 70]),
    ("bf16", 16, 2, 128, 1, 64, 256, 64, [1, 63, 64, 65, 255, 256, 257, 320, 321, 1000, 0]),
    ("bf16", 16, 2, 128, 4, 64, 130, 5, [4, 5, 134, 135, 700, 3, 0, 64]),
    ("bf16", 12, 4, 64, 2, 20, 47, 1, [2, 47, 48, 49, 333, 61]),
    ("bf16", 8, 8, 128, 1, 16, 1, 0, [1, 2, 17, 300]),
    ("bf16", 8, 8, 64, 1, 12, 1, 3, [1, 2, 3, 4, 5, 300]),
    ("bf16", 32, 4, 128, 4, 128, 500, 101, [4, 100, 101, 102, 600, 601, 605, 1200]),
    ("bf16", 32, 1, 128, 1, 36, 64, 16, [1, 64, 80, 81, 200]),
    ("bf16", 16, 2, 128, 1, 64, 2 ** 31 - 1, 0, [1, 777, 2100]),
    ("bf16", 16, 2, 128, 1, 16, 8, 2 ** 31 - 1, [1, 50, 333]),
    ("e4m3", 32, 4, 128, 1, 64, 200, 16, [1, 16, 199, 200, 201, 216, 217, 1000, 0]),
    ("e4m3", 16, 2, 64, 4, 16, 77, 4, [4, 76, 77, 80, 81, 82, 500]),
    ("e4m3", 12, 4, 128, 2, 8, 50, 0, [2, 3, 50, 51, 52, 53, 210]),
]


@pytest.mark.parametrize("kv,Hq,Hkv,D,T,page,window,sinks,lens", WINDOW)
def test_window_decode(kv, Hq, Hkv, D, T, page, window, sinks, lens):
    c = A.PagedKV(lens, Hkv, D, kv, page, "cuda", seed=page + T)
    q = queries((len(lens), T, Hq, D), kv, 3)
    want, seen = window_want(c, q, lens, T, window, sinks)
    c.poison(seen)   # what no query sees is NaN,
    c.unmap(seen)    # and its pages are gone
    op = QSAWindowDecode(c.cache(), len(lens), T, Hq, window, sinks)
    o, lse = op(q.cuda(), ints(lens))
    A.check(o, lse, want, kv, D, "window")


@pytest.mark.parametrize("kv,page", [("bf16", 64), ("e4m3", 16), ("f32", 16)])
def test_window_decode_long_few_requests(kv, page):
    """One and two requests: the keys are split over many CTAs."""
    for lens, window, sinks in (([9001], 8000, 64), ([5000, 37], 4096, 4)):
        c = A.PagedKV(lens, 2, 128, kv, page, "cuda", seed=11)
        q = queries((len(lens), 1, 16, 128), kv, 4)
        want, seen = window_want(c, q, lens, 1, window, sinks)
        c.poison(seen)
        op = QSAWindowDecode(c.cache(), len(lens), 1, 16, window, sinks)
        o, lse = op(q.cuda(), ints(lens))
        A.check(o, lse, want, kv, 128, "window")


def test_window_decode_sharp_and_flat_logits():
    """Logits in the hundreds, all equal, and falling along the keys (the
    running maximum never moves, or moves at every step)."""
    lens = [700, 700, 700]
    c = A.PagedKV(lens, 2, 128, "bf16", 64, "cuda", seed=21)
    q = queries((3, 1, 16, 128), "bf16", 5)
    q[0] *= 40
    q[1] = 0
    for t in range(700):
        c.k[c.table_host[2, t // 64], t % 64, :, 0] = float(t) / 4
    q[2, ..., 0] = 8
    want, seen = window_want(c, q, lens, 1, 600, 8)
    o, lse = QSAWindowDecode(c.cache(), 3, 1, 16, 600, 8)(q.cuda(), ints(lens))
    A.check(o, lse, want, "bf16", 128, "sharp")


def test_window_decode_masked_rows_need_no_finite_keys():
    """Keys with infinite logits that only some query tokens see."""
    lens = [100]
    c = A.PagedKV(lens, 1, 64, "bf16", 16, "cuda", seed=22)
    q = queries((1, 2, 4, 64), "bf16", 6)
    c.k[c.table_host[0, 99 // 16], 99 % 16] = -3e38  # seen by token 1 only: logits of +-inf
    want, _ = window_want(c, q, lens, 2, 2 ** 31 - 1, 0)
    o, lse = QSAWindowDecode(c.cache(), 1, 2, 4, 2 ** 31 - 1)(q.cuda(), ints(lens))
    first = tuple(x[:, 0] for x in want)
    A.check(o[:, 0], lse[:, 0], first, "bf16", 64, "the token that does not see it")


# ------------------------------------------------------------------- chunk --
def chunk_want(c, q, new, lens, window, sinks):
    rows, seen, at = [], {}, 0
    for r, (m, L) in enumerate(zip(new, lens)):
        seen[r] = set()
        for j in range(m):
            keys = A.visible(L - m + j, window, sinks)
            seen[r] |= set(keys)
            rows.append(A.attend(q[at + j], c.values("k", r, keys), c.values("v", r, keys), c.D ** -0.5))
        at += m
    return A.stack(rows), seen


CHUNK = [
    # kv, Hq, Hkv, D, page, window, sinks, new, lens
    ("f32", 8, 1, 64, 16, 40, 4, [1, 17, 0, 33], [1, 60, 5, 200]),
    ("bf16", 16, 2, 128, 64, 256, 64, [1, 5, 130, 64, 0], [1, 300, 130, 1000, 0]),
    ("bf16", 16, 2, 128, 64, 2 ** 31 - 1, 0, [200, 33], [200, 700]),
    ("bf16", 16, 2, 128, 16, 100, 5, [257, 31], [257, 600]),
    ("bf16", 12, 4, 64, 20, 47, 1, [90, 41, 7], [90, 300, 1001]),
    ("bf16", 8, 8, 128, 16, 1, 0, [150], [170]),
    ("bf16", 32, 1, 64, 36, 64, 16, [45, 3], [45, 500]),
    ("bf16", 8, 8, 64, 128, 300, 130, [300], [700]),
    ("e4m3", 32, 4, 128, 64, 200, 16, [70, 33, 1], [70, 500, 333]),
    ("e4m3", 12, 4, 64, 8, 61, 3, [150, 20], [160, 400]),
    ("e4m3", 16, 2, 128, 20, 128, 0, [129], [640]),
]


@pytest.mark.parametrize("kv,Hq,Hkv,D,page,window,sinks,new,lens", CHUNK)
def test_window_prefill(kv, Hq, Hkv, D, page, window, sinks, new, lens):
    c = A.PagedKV(lens, Hkv, D, kv, page, "cuda", seed=page)
    n = sum(new)
    q = queries((n, Hq, D), kv, 7)
    want, seen = chunk_want(c, q, new, lens, window, sinks)
    c.poison(seen)
    c.unmap(seen)
    pad = 3  # rows behind the last request
    qp = torch.cat([q, queries((pad, Hq, D), kv, 8)]).cuda()
    op = QSAWindowPrefill(c.cache(), len(lens), n + pad, max(new), Hq, window, sinks)
    op.o.fill_(7.0)
    op.lse.fill_(5.0)
    cu = np.concatenate([[0], np.cumsum(new)]).tolist()
    o, lse = op(qp, ints(cu), ints(lens))
    A.check(o[:n], lse[:n], want, kv, D, "chunk")
    assert (o[n:] == 7).all() and (lse[n:] == 5).all(), "rows behind the last request changed"


def test_window_prefill_is_the_decode_of_its_last_token():
    """The chunk's rows and the decode call agree (same numbers to rounding)."""
    lens, new = [500, 300], [20, 20]
    c = A.PagedKV(lens, 2, 128, "bf16", 64, "cuda", seed=31)
    q = queries((40, 16, 128), "bf16", 9)
    cache = c.cache()
    o, lse = QSAWindowPrefill(cache, 2, 40, 20, 16, 128, 4)(q.cuda(), ints([0, 20, 40]), ints(lens))
    qd = torch.stack([q[16:20], q[36:40]]).cuda()
    od, ld = QSAWindowDecode(cache, 2, 4, 16, 128, 4)(qd, ints(lens))
    assert torch.allclose(lse.view(2, 20, 16)[:, 16:], ld, atol=2e-5)
    assert torch.allclose(o.view(2, 20, 16, 128)[:, 16:].float(), od.float(), atol=3e-2)


# ------------------------------------------------------------------ prefix --
def prefix_want(c, q, lens, T):
    rows = []
    for r, L in enumerate(lens):
        toks = []
        for t in range(T):
            keys = A.visible(L - T + t, 2 ** 31 - 1, 0)
            toks.append(A.attend(q[r, t], c.values("k", r, keys), c.values("v", r, keys), c.D ** -0.5))
        rows.append(A.stack(toks))
    return A.stack(rows)


PREFIX = [
    # kv, Hq, Hkv, D, T, page, groups (prefix pages, extra prefix tokens, tails)
    ("f32", 8, 1, 64, 1, 16, [(5, 0, [1, 7, 40]), (0, 0, [9, 3])]),
    ("f32", 4, 4, 128, 2, 4, [(10, 0, [2, 3])]),
    ("bf16", 16, 2, 128, 1, 64, [(8, 0, [1, 2, 63, 64, 65, 500])]),
    ("bf16", 16, 2, 128, 1, 64, [(3, 0, [5] * 40), (1, 0, [9]), (20, 0, [100, 1])]),
    ("bf16", 16, 2, 128, 4, 16, [(7, 0, [4, 5, 90]), (2, 0, [4] * 17)]),
    ("bf16", 12, 4, 64, 2, 20, [(11, 0, [2, 33, 21])]),
    ("bf16", 8, 8, 128, 1, 64, [(6, 0, [3] * 33)]),
    ("bf16", 32, 1, 128, 1, 128, [(4, 0, [17, 200])]),
    ("e4m3", 32, 4, 128, 1, 64, [(9, 0, [1, 65, 130]), (2, 0, [40] * 5)]),
    ("e4m3", 16, 2, 64, 4, 16, [(13, 0, [4, 50]), (0, 0, [6])]),
    ("e4m3", 12, 4, 128, 2, 8, [(30, 0, [2] * 20)]),
]


@pytest.mark.parametrize("kv,Hq,Hkv,D,T,page,groups", PREFIX)
def test_prefix_decode(kv, Hq, Hkv, D, T, page, groups):
    lens, share, cu, pre = [], {}, [0], []
    for pages, extra, tails in groups:
        first = len(lens)
        for i, t in enumerate(tails):
            if i:
                share[len(lens)] = (first, pages)
            lens.append(pages * page + t)
        cu.append(len(lens))
        pre.append(pages * page)
    c = A.PagedKV(lens, Hkv, D, kv, page, "cuda", seed=page + T, share=share)
    q = queries((len(lens), T, Hq, D), kv, 12)
    want = prefix_want(c, q, lens, T)
    c.poison({r: range(L) for r, L in enumerate(lens)})
    op = QSAPrefixDecode(c.cache(), len(lens), T, Hq, len(groups), max_group=max(len(g[2]) for g in groups),
                         max_prefix=max(pre), max_tail=max(max(g[2]) for g in groups))
    o, lse = op(q.cuda(), ints(lens), ints(cu), ints(pre))
    A.check(o, lse, want, kv, D, "prefix")


def test_prefix_decode_unaligned_prefix_ungrouped_and_padding_rows():
    """A prefix that ends inside a page, a prefix longer than a request's
    context, an empty group, requests before and behind all groups, and a
    padding row; the host bounds of the lengths are too small on purpose."""
    page, T, Hq, Hkv, D = 16, 2, 16, 2, 128
    lens = [20, 90, 101, 75, 33, 0]
    c = A.PagedKV(lens, Hkv, D, "bf16", page, "cuda", seed=41, share={2: (1, 5), 3: (1, 4)})
    # requests 1..3 share 77 keys; the page the prefix ends in is a copy
    for r in (2, 3):
        for t in range(64, min(77, lens[r])):
            a, b = (int(c.table_host[x, t // page]) for x in (1, r))
            for kv in (c.k, c.v):
                kv[b, t % page] = kv[a, t % page]
    q = queries((6, T, Hq, D), "bf16", 13)
    want = prefix_want(c, q, lens, T)
    op = QSAPrefixDecode(c.cache(), 6, T, Hq, 2, max_group=3, max_prefix=8, max_tail=1)
    o, lse = op(q.cuda(), ints(lens), ints([1, 4, 4]), ints([77, 50]))
    A.check(o, lse, want, "bf16", D, "prefix")


# -------------------------------------------------------------------- rope --
ROPE = [
    # kv, Hq, Hkv, D, page, R, interleaved, scaling, factor, fused
    ("bf16", 16, 2, 128, 64, 128, False, "none", 1.0, True),
    ("bf16", 16, 2, 128, 64, 64, True, "yarn", 4.0, False),
    ("bf16", 12, 4, 64, 20, 48, False, "linear", 8.0, True),
    ("bf16", 3, 1, 64, 4, 30, True, "ntk", 2.0, True),
    ("bf16", 8, 8, 128, 16, 0, False, "none", 1.0, False),
    ("bf16", 32, 4, 128, 64, 128, True, "none", 1.0, False),
    ("f32", 8, 1, 64, 16, 64, False, "none", 1.0, True),
    ("f32", 8, 8, 128, 16, 80, True, "yarn", 2.5, False),
    ("e4m3", 16, 2, 128, 64, 128, False, "none", 1.0, True),
    ("e4m3", 4, 4, 64, 8, 22, True, "linear", 2.0, False),
]


@pytest.mark.parametrize("kv,Hq,Hkv,D,page,R,interleaved,scaling,factor,fused", ROPE)
@pytest.mark.parametrize("new,pos0", [([1, 1, 1], [0, 5, 130]), ([7, 0, 40, 1], [0, 3, 25, 99]),
                                      ([300] + [1] * 40, [10] + list(range(40)))])
def test_rope_append(kv, Hq, Hkv, D, page, R, interleaved, scaling, factor, fused, new, pos0):
    lens = [p + n for p, n in zip(pos0, new)]
    c = A.PagedKV(lens, Hkv, D, kv, page, "cuda", seed=R + page)
    n, pad = sum(new), 2
    dt = torch.float32 if kv == "f32" else torch.bfloat16
    if fused:
        qkv = queries((n + pad, Hq + 2 * Hkv, D), kv, 14)
        parts = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        dev = qkv.cuda()
        dparts = dev[:, :Hq], dev[:, Hq:Hq + Hkv], dev[:, Hq + Hkv:]
    else:
        parts = [queries((n + pad, h, D), kv, 15 + i) for i, h in enumerate((Hq, Hkv, Hkv))]
        dparts = [x.cuda() for x in parts]
    cache = c.cache()
    op = QSARopeAppend(cache, Hq, R, 10000.0, interleaved, scaling, factor, original_max_position=64)
    q_out = torch.full((n + pad, Hq, D), 9.0, dtype=dt, device="cuda")
    cu = np.concatenate([[0], np.cumsum(new)]).tolist()
    op(ints(pos0), ints(cu), *dparts, q_out)
    got_k, got_v = cache.k_cache.float().double().cpu(), cache.v_cache.float().double().cpu()
    want_k, want_v = c.k.float().double(), c.v.float().double()
    assert (q_out[n:] == 9).all(), "rows behind the last request changed"
    # half a step of the output type, and of the float32 products and angles:
    # 3 roundings of 2^-24 and an angle of 2^-24 half turns, sincospif to 2^-22
    half = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "e4m3": 2.0 ** -4}
    at = 0
    touched = torch.zeros(c.k.shape[:2], dtype=torch.bool)
    for r, m in enumerate(new):
        for j in range(m):
            p = pos0[r] + j
            pg, off = int(c.table_host[r, p // page]), p % page
            touched[pg, off] = True
            for x, got, typ, sc in ((parts[0][at], q_out[at].double().cpu(), "f32" if kv == "f32" else "bf16", None),
                                    (parts[1][at], got_k[pg, off], kv, c.k_scale)):
                y, mag = A.rope_row(x, p, op.inv_freq, op.mscale, R, interleaved)
                if R == 0:
                    mag = y.abs()
                e = mag * 2.0 ** -20
                s = 1.0 if sc is None or typ != "e4m3" else sc[pg].double()[:, None]
                y, e = y / s, e / s
                if typ == "e4m3":
                    y = y.clamp(-448, 448)
                    e = e + 2.0 ** -10  # half the smallest step, and the division
                err = (got - y).abs()
                assert (err <= half[typ] * (y.abs() + e) + e).all(), (r, j, float(err.max()))
            if kv == "e4m3":
                y = (parts[2][at].float() / c.v_scale[pg][:, None]).to(torch.float8_e4m3fn).float().double()
                y = torch.where(y.isnan(), torch.sign(parts[2][at].double()) * 448, y)
            else:
                y = parts[2][at].double()
            assert torch.equal(got_v[pg, off], y)
            at += 1
    assert torch.equal(got_k[~touched], want_k[~touched]) and torch.equal(got_v[~touched], want_v[~touched])


@pytest.mark.parametrize("offset,pad", [(0, 1), (1, 0), (3, 8)])
def test_rope_rows_of_any_alignment(offset, pad):
    """Rows that are not 16 bytes aligned, by their start or their stride, give
    the bits of aligned ones; 1,500 requests, some without a token."""
    Hq, Hkv, D, page = 4, 2, 64, 16
    new = [i % 3 for i in range(1500)]
    pos0 = [(i * 37) % 300 for i in range(1500)]
    n = sum(new)
    c = A.PagedKV([p + 3 for p in pos0], Hkv, D, "bf16", page, "cuda", seed=25)
    width = (Hq + 2 * Hkv) * D
    buf = queries((n * (width + pad) + offset,), "bf16", 26).cuda()
    rows = buf[offset:].view(n, width + pad)[:, :width].unflatten(1, (Hq + 2 * Hkv, D))
    cu = ints(np.concatenate([[0], np.cumsum(new)]).tolist())
    outs = []
    for x in (rows, rows.contiguous()):
        cache = c.cache()
        op = QSARopeAppend(cache, Hq, 32, interleaved=True)
        q = op(ints(pos0), cu, x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:])
        outs.append((q, cache.k_cache, cache.v_cache))
    for a, b in zip(*outs):
        assert torch.equal(a, b)


def test_rope_far_positions_and_in_place():
    """Angles at positions around two billion, and q rotated in place."""
    page, D = 64, 128
    pos = [2 ** 31 - 70, 1048575, 123456789]
    table = torch.full((3, (2 ** 31 - 1) // page + 1), -1, dtype=torch.int32, device="cuda")
    for r, p in enumerate(pos):
        table[r, p // page] = r
    from sparse_attention_decode_compress_b200 import QSACache
    kc, vc = (torch.zeros((3, page, 1, D), device="cuda") for _ in range(2))
    cache = QSACache.allocate(kc, vc, table, 32, 3)
    q, k, v = (queries((3, h, D), "f32", 20 + h).cuda() for h in (2, 1, 1))
    op = QSARopeAppend(cache, 2, theta=1e6)
    keep = q.clone()
    out = op(ints(pos), ints([0, 1, 2, 3]), q, k, v, q)
    assert out is q
    for r, p in enumerate(pos):
        for got, x in ((q[r], keep[r]), (kc[r, p % page], k[r])):
            y, mag = A.rope_row(x.cpu(), p, op.inv_freq, 1.0, D, False)
            # the reference's own angle: p * f in float64, 2^-53 relative, and
            # the frequency's rounding there
            e = mag * (2.0 ** -20 + 2.0 ** -51 * p)
            assert ((got.double().cpu() - y).abs() <= e).all()


# ---------------------------------------------------------------- together --
def test_append_then_attend_then_share():
    """A serving loop: a prompt is appended and attended as a chunk, two
    requests continue behind it token by token, and the shared-prefix decode
    gives what the dense decode of each gives."""
    Hq, Hkv, D, page = 16, 2, 128, 64
    P = 256  # prompt
    c = A.PagedKV([P + 70, P + 70], Hkv, D, "bf16", page, "cuda", seed=51, share={1: (0, P // page)})
    c.k.zero_()
    c.v.zero_()
    cache = c.cache()
    rope = QSARopeAppend(cache, Hq, theta=1e6)
    qkv = queries((P, Hq + 2 * Hkv, D), "bf16", 52).cuda()
    q = rope(ints([0]), ints([0, P]), qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:])
    chunk = QSAWindowPrefill(cache, 1, P, P, Hq, 2 ** 31 - 1)
    o, lse = chunk(q, ints([0, P]), ints([P]))
    c.k, c.v = cache.k_cache.cpu(), cache.v_cache.cpu()
    want, _ = chunk_want(c, q.cpu(), [P], [P], 2 ** 31 - 1, 0)
    A.check(o, lse, want, "bf16", D, "prompt")
    dense = QSAWindowDecode(cache, 2, 1, Hq, 2 ** 31 - 1)
    shared = QSAPrefixDecode(cache, 2, 1, Hq, 1, 2, P, 70)
    for step in range(66):
        qkv = queries((2, Hq + 2 * Hkv, D), "bf16", 100 + step).cuda()
        q = rope(ints([P + step] * 2), ints([0, 1, 2]), qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:])
        q = q.view(2, 1, Hq, D)
        L = ints([P + step + 1] * 2)
        o, lse = shared(q, L, ints([0, 2]), ints([P]))
        o2, lse2 = dense(q, L)
        assert torch.allclose(lse, lse2, atol=2e-5)
        if step in (0, 63, 65):
            c.k, c.v = cache.k_cache.cpu(), cache.v_cache.cpu()
            want = prefix_want(c, q.cpu(), [P + step + 1] * 2, 1)
            A.check(o, lse, want, "bf16", D, "shared")
            A.check(o2, lse2, want, "bf16", D, "dense")


def test_captured_and_replayed_on_another_stream():
    """All calls captured into one graph with device lengths that grow."""
    Hq, Hkv, D, page, B = 16, 2, 128, 64, 3
    lens = [200, 131, 64]
    c = A.PagedKV([n + 8 for n in lens], Hkv, D, "bf16", page, "cuda", seed=61)
    cache = c.cache()
    rope = QSARopeAppend(cache, Hq)
    win = QSAWindowDecode(cache, B, 1, Hq, 100, 4)
    pre = QSAPrefixDecode(cache, B, 1, Hq, 1, 1, 64, 200)
    pos, L = ints(lens), ints([n + 1 for n in lens])
    cu, cug, pl = ints([0, 1, 2, 3]), ints([0, 1]), ints([64])
    qkv = queries((B, Hq + 2 * Hkv, D), "bf16", 62).cuda()
    qr = torch.empty((B, Hq, D), dtype=torch.bfloat16, device="cuda")

    def step(stream=None):
        rope(pos, cu, qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], qr, stream=stream)
        a = win(qr.view(B, 1, Hq, D), L, stream=stream)
        b = pre(qr.view(B, 1, Hq, D), L, cug, pl, stream=stream)
        return a, b

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step(side)
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        out = step()
    for k in range(3):
        qkv.copy_(queries((B, Hq + 2 * Hkv, D), "bf16", 70 + k))
        pos += 1
        L += 1
        g.replay()
        torch.cuda.synchronize()
        c.k, c.v = cache.k_cache.cpu(), cache.v_cache.cpu()
        now = [n + 2 + k for n in lens]
        q = qr.cpu().view(B, 1, Hq, D)
        want, _ = window_want(c, q, now, 1, 100, 4)
        A.check(*out[0], want, "bf16", D, "window")
        A.check(*out[1], prefix_want(c, q, now, 1), "bf16", D, "prefix")


# ------------------------------------------------- recorded on the device --
def test_bad_pages_lengths_and_offsets_are_recorded():
    Hq, Hkv, D, page = 16, 2, 128, 64
    c = A.PagedKV([100, 200], Hkv, D, "bf16", page, "cuda", seed=71)
    q = queries((2, 1, Hq, D), "bf16", 72)
    cache = c.cache()
    dense = 2 ** 31 - 1
    BOUNDS, BAD = 1, 4
    # a length the block table cannot hold
    QSAWindowDecode(cache, 2, 1, Hq, dense)(q.cuda(), ints([100, 100000]))
    assert qsa_get_device_error()[1] & BOUNDS
    # a page that is not there, and one beyond the pool: zeros in its place
    for bad in (-1, 10 ** 6):
        t = cache.block_table.clone()
        cache.block_table[1, 1] = bad
        o, lse = QSAWindowDecode(cache, 2, 1, Hq, dense)(q.cuda(), ints([100, 200]))
        assert qsa_get_device_error()[1] & BOUNDS
        K, V = (c.values(x, 1, range(200)) for x in "kv")
        K[page:2 * page] = V[page:2 * page] = 0
        want, _ = window_want(c, q, [100], 1, dense, 0)
        A.check(o[:1], lse[:1], want, "bf16", D, "the other request")
        part = A.stack([A.stack([A.attend(q[1, 0], K, V, D ** -0.5)])])
        A.check(o[1:], lse[1:], part, "bf16", D, "without the page")
        cache.block_table.copy_(t)
    # offsets that fall, leave the rows, or break the bound
    ch = QSAWindowPrefill(cache, 2, 8, 4, Hq, 64)
    for cu in ([0, 5, 2], [0, 4, 9], [0, 5, 8], [-1, 2, 4]):
        ch(q.view(2, Hq, D).repeat(4, 1, 1).cuda(), ints(cu), ints([100, 200]))
        assert qsa_get_device_error()[1] & BAD
    pr = QSAPrefixDecode(cache, 2, 1, Hq, 1, 1, 64, 200)
    for cu, n in (([0, 2], 64), ([0, 3], 64), ([1, 0], 64), ([0, 1], -5)):
        pr(q.cuda(), ints([100, 200]), ints(cu), ints([n]))
        assert qsa_get_device_error()[1] & BAD
    # a new token without a page: its query is still rotated
    rope = QSARopeAppend(cache, Hq)
    k = queries((2, Hkv, D), "bf16", 73).cuda()
    before = cache.k_cache.clone()
    out = rope(ints([10 ** 5, -1]), ints([0, 1, 2]), q.view(2, Hq, D).cuda(), k, k)
    assert qsa_get_device_error()[1] & BOUNDS
    assert torch.equal(before, cache.k_cache)
    y, mag = A.rope_row(q[0, 0], 10 ** 5, rope.inv_freq, 1.0, D, False)
    assert ((out[0].double().cpu() - y).abs() <= 2.0 ** -8 * y.abs() + 2.0 ** -19 * mag).all()


# ----------------------------------------------- maxima that move, and NaN --
def ramped(kv, Hkv, D, page, lens, jumps, seed):
    """Keys whose first dim jumps at the given positions, so that a row's logits
    leave the weights' range inside a step, between steps and at its quarters."""
    c = A.PagedKV(lens, Hkv, D, kv, page, "cuda", seed=seed)
    for r, L in enumerate(lens):
        for t in range(L):
            level = sum(h for at, h in jumps if t >= at)
            pg, off = int(c.table_host[r, t // page]), t % page
            if kv == "e4m3":  # by the page's scale: the first code is 448 or 0
                c.k[pg, off] = c.k[pg, off].float().clamp(-2, 2).to(torch.float8_e4m3fn)
                c.k_scale[pg] = max(level, 2.0 ** -6) / 448
                c.k[pg, off, :, 0] = torch.tensor(448.0 if level > 0 else 0.0).to(torch.float8_e4m3fn)
            else:
                c.k[pg, off, :, 0] = level
    return c


JUMPS = [[(0, 0.0), (40, 30.0), (70, 25.0), (100, 40.0), (130, 6.0), (250, 90.0)],
         [(0, 1.0), (16, 20.0), (33, 300.0), (64, 12.0), (128, 500.0), (384, 3.0)],
         [(0, 400.0), (1, -400.0), (96, 200.0), (97, -100.0)]]


@pytest.mark.parametrize("kv,page", [("bf16", 64), ("bf16", 20), ("e4m3", 16), ("f32", 16)])
@pytest.mark.parametrize("jumps", JUMPS)
def test_logits_that_jump_along_the_keys(kv, page, jumps):
    Hq, Hkv, D, dense = 8, 2, 128, 2 ** 31 - 1
    lens = [450, 300]
    c = ramped(kv, Hkv, D, page, lens, jumps, seed=81)
    new = [70, 33]
    q = queries((sum(new), Hq, D), kv, 82)
    q[..., 0] = 8.0
    cache = c.cache()
    want, _ = chunk_want(c, q, new, lens, dense, 0)
    o, lse = QSAWindowPrefill(cache, 2, sum(new), max(new), Hq, dense)(q.cuda(), ints([0, 70, 103]), ints(lens))
    A.check(o, lse, want, kv, D, "chunk")
    qd = torch.stack([q[66:70], q[99:103]])
    want, _ = window_want(c, qd, lens, 4, dense, 0)
    o, lse = QSAWindowDecode(cache, 2, 4, Hq, dense)(qd.cuda(), ints(lens))
    A.check(o, lse, want, kv, D, "decode")
    # the prefix of a group of its own, for each
    o, lse = QSAPrefixDecode(cache, 2, 4, Hq, 2, 1, 256, 250)(qd.cuda(), ints(lens), ints([0, 1, 2]), ints([256, 200]))
    A.check(o, lse, want, kv, D, "prefix")


@pytest.mark.parametrize("kv,page", [("bf16", 64), ("e4m3", 16), ("f32", 16)])
def test_a_nan_that_a_query_sees_is_in_its_result_and_nowhere_else(kv, page):
    Hq, Hkv, D = 8, 2, 128
    lens = [200, 200]
    c = A.PagedKV(lens, Hkv, D, kv, page, "cuda", seed=91)
    pg, off = int(c.table_host[1, 150 // page]), 150 % page
    if kv == "e4m3":
        c.k.view(torch.uint8)[pg, off, 1, 5] = 0x7F
    else:
        c.k[pg, off, 1, 5] = float("nan")
    cache = c.cache()
    q = queries((2, 1, Hq, D), kv, 92).cuda()
    clean = [1, 1, 1, 1, 1, 1, 1, 1, 1, 1, 1, 1, 0, 0, 0, 0]  # request 1's heads of kv head 1 see it
    clean = torch.tensor(clean, dtype=torch.bool, device="cuda").view(2, 1, Hq)
    ch = torch.cat([q[:1, 0], q[1:, 0]])
    for o, lse in (QSAWindowDecode(cache, 2, 1, Hq, 100)(q, ints(lens)),
                   QSAPrefixDecode(cache, 2, 1, Hq, 2, 1, 160, 40)(q, ints(lens), ints([0, 1, 2]), ints([160, 128])),
                   QSAWindowPrefill(cache, 2, 2, 1, Hq, 64)(ch, ints([0, 1, 2]), ints(lens))):
        o, lse = o.view(2, 1, Hq, D), lse.view(2, 1, Hq)
        assert torch.equal(torch.isfinite(lse), clean)
        assert torch.equal(torch.isfinite(o).all(-1), clean) and o[~clean].isnan().all() and lse[~clean].isnan().all()
    # out of the window: nothing of it
    o, lse = QSAWindowDecode(cache, 2, 1, Hq, 49)(q, ints(lens))
    assert torch.isfinite(o).all() and torch.isfinite(lse).all()


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_prefix_of_many_rows_per_kv_head_and_ragged_groups(kv):
    """Groups of 1, 70 and 33 requests with two query tokens: partial row tiles
    of 256, and a group without any."""
    page, T, Hq, Hkv, D = 32, 2, 8, 2, 64
    sizes, pages = [1, 70, 0, 33], [3, 11, 2, 7]
    lens, share, cu, pre = [], {}, [0], []
    for n, p in zip(sizes, pages):
        first = len(lens)
        for i in range(n):
            if i:
                share[len(lens)] = (first, p)
            lens.append(p * page + T + (i * 7) % 45)
        cu.append(len(lens))
        pre.append(p * page)
    c = A.PagedKV(lens, Hkv, D, kv, page, "cuda", seed=95, share=share)
    q = queries((len(lens), T, Hq, D), kv, 96)
    op = QSAPrefixDecode(c.cache(), len(lens), T, Hq, 4, 70, max(pre), 47)
    o, lse = op(q.cuda(), ints(lens), ints(cu), ints(pre))
    A.check(o, lse, prefix_want(c, q, lens, T), kv, D, "prefix")


def test_two_streams_with_handles_of_their_own():
    """Calls in flight on two streams at once, each with its own handle."""
    Hq, Hkv, D = 16, 2, 128
    lens = [3000, 2000]
    c = A.PagedKV(lens, Hkv, D, "bf16", 64, "cuda", seed=97)
    cache = c.cache()
    qs = [queries((2, 1, Hq, D), "bf16", 98 + i).cuda() for i in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    ops = [(QSAWindowDecode(cache, 2, 1, Hq, 2 ** 31 - 1), QSAPrefixDecode(cache, 2, 1, Hq, 1, 1, 1500, 1500))
           for _ in range(2)]
    L, cu, pl = ints(lens), ints([0, 1]), ints([1500])
    alone = []
    for q, (w, p) in zip(qs, ops):
        alone.append([t.clone() for t in (*w(q, L), *p(q, L, cu, pl))])
    torch.cuda.synchronize()
    for _ in range(20):
        for q, s, (w, p) in zip(qs, streams, ops):
            w(q, L, stream=s)
            p(q, L, cu, pl, stream=s)
    torch.cuda.synchronize()
    for want, (w, p) in zip(alone, ops):
        for a, b in zip(want, (w.o, w.lse, p.o, p.lse)):
            assert torch.equal(a, b)


# ------------------------------------- contexts shorter than their queries --
@pytest.mark.parametrize("kv", ["f32", "bf16", "e4m3"])
@pytest.mark.parametrize("sinks", [0, 2])
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 3, 3])
def test_contexts_shorter_than_the_query_tokens(kv, sinks, window):
    """Query tokens before position 0 see nothing and take nothing from the
    others, at any window: four decode tokens over 0 to 4 cached ones, and
    chunks longer than their contexts."""
    Hq, Hkv, D, T = 8, 2, 128, 4
    lens = [0, 1, 2, 3, 4, 9]
    c = A.PagedKV(lens, Hkv, D, kv, 16, "cuda", seed=101)
    q = queries((len(lens), T, Hq, D), kv, 102)
    want, seen = window_want(c, q, lens, T, window, sinks)
    c.poison(seen)
    o, lse = QSAWindowDecode(c.cache(), len(lens), T, Hq, window, sinks)(q.cuda(), ints(lens))
    A.check(o, lse, want, kv, D, "decode")
    new, lens = [8, 8, 200, 5], [5, 0, 3, 9]  # 200 tokens: row tiles without a token at position 0 or later
    c = A.PagedKV(lens, Hkv, D, kv, 16, "cuda", seed=103)
    q = queries((sum(new), Hq, D), kv, 104)
    want, seen = chunk_want(c, q, new, lens, window, sinks)
    c.poison(seen)
    cu = np.concatenate([[0], np.cumsum(new)]).tolist()
    o, lse = QSAWindowPrefill(c.cache(), 4, sum(new), max(new), Hq, window, sinks)(q.cuda(), ints(cu), ints(lens))
    A.check(o, lse, want, kv, D, "chunk")


@pytest.mark.parametrize("kv", ["f32", "bf16", "e4m3"])
def test_a_negative_length_is_an_empty_request(kv):
    Hq, Hkv, D, T = 8, 2, 128, 4
    c = A.PagedKV([60, 60, 60], Hkv, D, kv, 16, "cuda", seed=105)
    q = queries((3, T, Hq, D), kv, 106)
    lens, dense = [-1, 60, -2 ** 31], 2 ** 31 - 1
    want, _ = window_want(c, q, [0, 60, 0], T, dense, 0)
    cache = c.cache()
    o, lse = QSAWindowDecode(cache, 3, T, Hq, dense)(q.cuda(), ints(lens))
    A.check(o, lse, want, kv, D, "decode")
    o, lse = QSAPrefixDecode(cache, 3, T, Hq, 3, 1, 32, 32)(q.cuda(), ints(lens), ints([0, 1, 2, 3]), ints([32] * 3))
    A.check(o, lse, want, kv, D, "prefix")
    want, _ = chunk_want(c, q.flatten(0, 1), [T] * 3, [0, 60, 0], dense, 0)
    o, lse = QSAWindowPrefill(cache, 3, 3 * T, T, Hq, dense)(q.flatten(0, 1).cuda(), ints([0, 4, 8, 12]), ints(lens))
    A.check(o, lse, want, kv, D, "chunk")


# ------------------------------------------- refused groups and sequences --
def garbage(op):
    """Finite values in every partial result that a call could take for its own."""
    if op.ws is not None:
        op.ws.view(torch.float32).fill_(7.0)


@pytest.mark.parametrize("kv", ["f32", "bf16", "e4m3"])
@pytest.mark.parametrize("cu,prefix,max_group,bad",
                         [([0, 2], 64, 1, True),      # larger than max_group
                          ([0, 3], 64, 2, True),      # leaves the batch
                          ([-1, 2], 64, 2, True),
                          ([1, 0], 64, 2, True),      # falls: holds nobody
                          ([0, 1], -5, 1, True),      # a negative prefix is none
                          ([0, 2], 64, 2, False)])
def test_a_refused_group_gives_its_tails(kv, cu, prefix, max_group, bad):
    Hq, Hkv, D, page, lens = 16, 2, 128, 64, [100, 200]
    c = A.PagedKV(lens, Hkv, D, kv, page, "cuda", seed=111, share={1: (0, 1)})
    q = queries((2, 1, Hq, D), kv, 112)
    op = QSAPrefixDecode(c.cache(), 2, 1, Hq, 1, max_group, 64, 200)
    rows = []
    for r, L in enumerate(lens):
        lo = max(prefix, 0) if bad and cu[0] <= r < cu[1] else 0
        K, V = (c.values(x, r, range(lo, L)) for x in "kv")
        rows.append(A.stack([A.attend(q[r, 0], K, V, D ** -0.5)]))
    garbage(op)
    o, lse = op(q.cuda(), ints(lens), ints(cu), ints([prefix]))
    A.check(o, lse, A.stack(rows), kv, D, "tails")
    assert qsa_get_device_error()[1] == (4 if bad else 0)


@pytest.mark.parametrize("kv", ["f32", "bf16", "e4m3"])
@pytest.mark.parametrize("window", [40, 2 ** 31 - 1])  # one part a row, and several that are merged
@pytest.mark.parametrize("cu", [[0, 5, 2], [0, 4, 9], [0, 5, 8], [-1, 2, 4], [2, 4, 8], [0, 4, 6], [4, 8, 0]])
def test_rows_of_refused_requests_stay_as_they_were(kv, window, cu):
    Hq, Hkv, D, lens, n, most = 16, 2, 128, [1500, 2000], 8, 4
    c = A.PagedKV(lens, Hkv, D, kv, 64, "cuda", seed=113)
    q = queries((n, Hq, D), kv, 114)
    op = QSAWindowPrefill(c.cache(), 2, n, most, Hq, window)
    assert (op.ws is None) == (window == 40)
    garbage(op)
    op.o.fill_(3.0)
    op.lse.fill_(5.0)
    o, lse = op(q.cuda(), ints(cu), ints(lens))
    live, bad = torch.zeros(n, dtype=torch.bool), False
    for r, L in enumerate(lens):
        a, b = cu[r], cu[r + 1]
        if not (0 <= a <= b <= n and b - a <= most):
            bad = True
            continue
        live[a:b] = True
        rows = []
        for j in range(b - a):
            keys = A.visible(L - (b - a) + j, window, 0)
            rows.append(A.attend(q[a + j], c.values("k", r, keys), c.values("v", r, keys), D ** -0.5))
        if rows:
            A.check(o[a:b], lse[a:b], A.stack(rows), kv, D, "a request beside a refused one")
    assert (o[~live] == 3).all() and (lse[~live] == 5).all(), "rows of no request changed"
    assert qsa_get_device_error()[1] == (4 if bad else 0)


def test_merged_chunks_of_many_requests():
    """More requests than the merge asks in one round, some of them refused."""
    Hq, Hkv, D, B = 2, 1, 64, 70
    lens = [600 + 7 * r for r in range(B)]
    c = A.PagedKV(lens, Hkv, D, "bf16", 64, "cuda", seed=115)
    new = [3 if r % 9 == 4 else r % 3 for r in range(B)]  # at most 2 are taken
    n = sum(new)
    q = queries((n, Hq, D), "bf16", 116)
    op = QSAWindowPrefill(c.cache(), B, n, 2, Hq, 2 ** 31 - 1)
    assert op.ws is not None
    garbage(op)
    op.o.fill_(3.0)
    cu = np.concatenate([[0], np.cumsum(new)]).tolist()
    o, lse = op(q.cuda(), ints(cu), ints(lens))
    assert qsa_get_device_error()[1] == 4
    for r, m in enumerate(new):
        if m > 2:
            assert (o[cu[r]:cu[r + 1]] == 3).all()
        elif m:
            rows = [A.attend(q[cu[r] + j], *(c.values(x, r, range(lens[r] - m + j + 1)) for x in "kv"), D ** -0.5)
                    for j in range(m)]
            A.check(o[cu[r]:cu[r + 1]], lse[cu[r]:cu[r + 1]], A.stack(rows), "bf16", D, f"request {r}")


# ------------------------------------------- small weights of 8-bit caches --
@pytest.mark.parametrize("form", ["window", "chunk", "prefix"])
@pytest.mark.parametrize("nats,scales", [(9.0, 0), (12.0, 0), (15.0, 0), (16.1, 0), (17.0, 0), (18.2, 0), (14.0, 5)])
def test_small_weights_of_an_8_bit_cache(form, nats, scales):
    """One key far above a flat row (logit + nats) with a value of zero: the
    output is the others' values times their small weights.  `scales`: that key's
    page has a V scale 2^scales above the others'.  exp(-18.2) = 2^-26.3 and
    2^-5 exp(-14) = 2^-25.2 are above 2^-27, to which weights keep 2^-8."""
    Hq, Hkv, D, page, L = 16, 2, 128, 64, 3001
    c = A.PagedKV([L], Hkv, D, "e4m3", page, "cuda", seed=121)
    c.k_scale.fill_(2.0 ** -6)
    c.v_scale.fill_(2.0 ** -6)
    c.k.view(torch.uint8).zero_()
    c.v = (c.v.float().clamp(-200, 200).abs() + 16).to(torch.float8_e4m3fn)
    top = 70
    pg = int(c.table_host[0, top // page])
    c.k[pg, top % page, :, 0] = torch.tensor(256.0).to(torch.float8_e4m3fn)  # times the scale: 4
    c.v[pg] = torch.tensor(0.0).to(torch.float8_e4m3fn)
    c.v_scale[pg] *= 2.0 ** scales
    q = torch.zeros((1, 4, Hq, D), dtype=torch.bfloat16)
    q[..., 0] = nats * D ** 0.5 / 4
    dense = 2 ** 31 - 1
    cache = c.cache()
    if form == "window":
        want, _ = window_want(c, q, [L], 4, dense, 0)
        o, lse = QSAWindowDecode(cache, 1, 4, Hq, dense)(q.cuda(), ints([L]))
    elif form == "chunk":
        want, _ = chunk_want(c, q[0], [4], [L], dense, 0)
        o, lse = QSAWindowPrefill(cache, 1, 4, 4, Hq, dense)(q[0].cuda(), ints([0, 4]), ints([L]))
    else:
        want = prefix_want(c, q, [L], 4)
        o, lse = QSAPrefixDecode(cache, 1, 4, Hq, 1, 1, L - 100, 100)(q.cuda(), ints([L]), ints([0, 1]),
                                                                     ints([L - 100]))
    A.check(o, lse, want, "e4m3", D, form)


# ------------------------------------------------- memory on other streams --
def test_a_new_q_out_does_not_take_memory_that_the_current_stream_still_reads():
    """A block freed behind unfinished work of the current stream may be used
    again on that stream alone: the rows that another stream writes come from
    that stream's memory."""
    n, Hq, Hkv, D = 6000, 16, 2, 128  # 24 MB: a block of its own
    c = A.PagedKV([n], Hkv, D, "bf16", 64, "cuda", seed=131)
    op = QSARopeAppend(c.cache(), Hq)
    q, k, v = (queries((n, h, D), "bf16", 132 + h).cuda() for h in (Hq, Hkv, Hkv))
    pos, cu, side = ints([0]), ints([0, n]), torch.cuda.Stream()
    want = op(pos, cu, q, k, v)
    old, copy = torch.ones_like(q), torch.zeros_like(q)
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)  # (clock ticks: some 50 ms)
    copy.copy_(old)
    del old
    got = op(pos, cu, q, k, v, stream=side)
    torch.cuda.synchronize()
    assert (copy == 1).all()
    assert torch.equal(got, want)


def test_a_handle_made_on_one_stream_is_called_on_another():
    """The fills of a handle's outputs may not overtake its first call, though
    the stream that it is made on is late."""
    L, n, Hq, D = 600, 64, 16, 128
    c = A.PagedKV([L], 2, D, "bf16", 64, "cuda", seed=133)
    cache = c.cache()
    q = queries((n, Hq, D), "bf16", 134)
    dq, cu, ctx, side = q.cuda(), ints([0, n]), ints([L]), torch.cuda.Stream()
    QSAWindowPrefill(cache, 1, n, n, Hq, 100)(dq, cu, ctx)  # (a kernel's first launch may wait for the device)
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)
    o, lse = QSAWindowPrefill(cache, 1, n, n, Hq, 100)(dq, cu, ctx, stream=side)
    torch.cuda.synchronize()
    A.check(o, lse, chunk_want(c, q, [n], [L], 100, 0)[0], "bf16", D, "chunk")


def test_a_handle_dropped_while_its_call_runs_keeps_its_memory():
    L, Hq, D = 6000, 16, 128
    c = A.PagedKV([L], 2, D, "bf16", 64, "cuda", seed=135)
    q = queries((1, 1, Hq, D), "bf16", 136)
    dq, ctx, cu, pre, side = q.cuda(), ints([L]), ints([0, 1]), ints([4096]), torch.cuda.Stream()
    op = QSAPrefixDecode(c.cache(), 1, 1, Hq, 1, 1, 4096, 2000)
    n = op.ws.numel()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)
        o, lse = op(dq, ctx, cu, pre)
    del op
    others = [torch.full((n,), 1, dtype=torch.uint8, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    assert all((x == 1).all() for x in others)
    A.check(o, lse, prefix_want(c, q, [L], 1), "bf16", D, "prefix")


@pytest.mark.parametrize("kv", ["f32", "bf16", "e4m3"])
def test_the_tails_see_what_was_written_right_before_the_call(kv):
    """The tails of a shared-prefix decode start beside its prefixes.  Queries,
    lengths, tails and tables that the work right before the call writes give,
    step after step without a pause, the bits of steps with a pause between
    all calls."""
    Hq, Hkv, D, page, B, P, steps = 16, 2, 128, 16, 6, 64, 60
    c = A.PagedKV([P + 80] * B, Hkv, D, kv, page, "cuda", seed=141, share={r: (0, P // page) for r in range(1, B)})
    tables = [torch.from_numpy(c.table_host), torch.from_numpy(c.table_host)]
    own = tables[1][:, P // page:]
    tables[1][:, P // page:] = torch.roll(own, 1, 0)  # the tails' pages change hands every step
    tables = [t.cuda() for t in tables]
    qkv = [queries((B, Hq + 2 * Hkv, D), kv, 150 + i).cuda() for i in range(steps)]
    lens = [ints([P + 1 + (7 * r + i) % 79 for r in range(B)]) for i in range(steps)]
    cu, cug, pl = ints(list(range(B + 1))), ints([0, B]), ints([P])

    def steps_of(pause):
        cache = c.cache()
        rope, op = QSARopeAppend(cache, Hq), QSAPrefixDecode(cache, B, 1, Hq, 1, B, P, 80)
        ctx, pos, outs = ints([0] * B), ints([0] * B), []
        for i in range(steps):
            cache.block_table.copy_(tables[i % 2])
            ctx.copy_(lens[i])
            torch.sub(ctx, 1, out=pos)
            pause()
            x = qkv[i]
            q = rope(pos, cu, x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:])
            pause()
            outs.append([t.clone() for t in op(q.view(B, 1, Hq, D), ctx, cug, pl)])
            pause()
        torch.cuda.synchronize()
        return outs

    for a, b in zip(steps_of(torch.cuda.synchronize), steps_of(lambda: None)):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


# ------------------------------------------------------------- the binding --
def test_no_call_takes_more_requests_than_the_block_table_has_rows():
    c = A.PagedKV([40, 40], 2, 64, "bf16", 16, "cuda", seed=151)
    cache, q = c.cache(), queries((3, 1, 4, 64), "bf16", 152).cuda()
    for make in (lambda: QSAWindowDecode(cache, 3, 1, 4, 16), lambda: QSAWindowPrefill(cache, 3, 3, 1, 4, 16),
                 lambda: QSAPrefixDecode(cache, 3, 1, 4, 1, 1, 16, 16),
                 lambda: QSARopeAppend(cache, 4)(ints([0] * 3), ints([0, 1, 2, 3]), q[:, 0], q[:, 0, :2], q[:, 0, :2])):
        with pytest.raises(ValueError, match="2 rows for 3 requests"):
            make()


def test_a_handle_keeps_the_tensors_it_was_made_with():
    c = A.PagedKV([300, 200], 2, 128, "e4m3", 16, "cuda", seed=153)
    cache = c.cache()
    old = [cache.k_cache, cache.v_cache, cache.block_table, cache.k_scale, cache.v_scale]
    addresses = {t.data_ptr() for t in old}
    op = QSAWindowDecode(cache, 2, 1, 16, 100)
    for name in ("k_cache", "v_cache", "block_table", "k_scale", "v_scale"):
        setattr(cache, name, getattr(cache, name).clone())
    shapes = [(t.shape, t.dtype) for t in old]
    del old, c.dk, c.dv
    new = [torch.zeros(s, dtype=torch.uint8, device="cuda").to(d) for s, d in shapes for _ in range(4)]
    assert not addresses & {t.data_ptr() for t in new}, "memory that the handle reads was given away"
    q = queries((2, 1, 16, 128), "e4m3", 154)
    o, lse = op(q.cuda(), ints([300, 200]))
    A.check(o, lse, window_want(c, q, [300, 200], 1, 100, 0)[0], "e4m3", 128, "window")


@pytest.mark.parametrize("kv", ["f32", "bf16", "e4m3"])
def test_a_layer_without_an_index(kv):
    """Caches without compressed keys and ring give the bits of those with them."""
    from sparse_attention_decode_compress_b200 import QSACache, qsa_compress_append
    Hq, Hkv, D, lens = 16, 2, 128, [300, 200]
    outs = []
    for idx_dim, rows in ((32, 2), (0, 0)):
        c = A.PagedKV(lens, Hkv, D, kv, 16, "cuda", seed=155)
        full = c.cache()
        cache = QSACache.allocate(full.k_cache, full.v_cache, full.block_table, idx_dim, rows,
                                  k_scale=full.k_scale, v_scale=full.v_scale)
        x = queries((2, Hq + 2 * Hkv, D), kv, 156).cuda()
        q = QSARopeAppend(cache, Hq)(ints([n - 1 for n in lens]), ints([0, 1, 2]), x[:, :Hq], x[:, Hq:Hq + Hkv],
                                     x[:, Hq + Hkv:])
        outs.append([q, cache.k_cache, cache.v_cache,
                     *QSAWindowDecode(cache, 2, 1, Hq, 100, 4)(q.unsqueeze(1), ints(lens)),
                     *QSAWindowPrefill(cache, 2, 2, 1, Hq, 100, 4)(q, ints([0, 1, 2]), ints(lens)),
                     *QSAPrefixDecode(cache, 2, 1, Hq, 2, 1, 64, 236)(q.unsqueeze(1), ints(lens), ints([0, 1, 2]),
                                                                      ints([64, 64]))])
    for a, b in zip(*outs):
        assert torch.equal(a.float(), b.float())
    with pytest.raises(RuntimeError):
        qsa_compress_append(cache, ints([0, 0]), ints([0, 1, 2]), torch.zeros((2, 32), dtype=torch.int8, device="cuda"), 1)


@pytest.mark.parametrize("kv", ["f32", "bf16", "e4m3"])
def test_appended_rows_are_what_the_sparse_decode_reads(kv):
    """Prompts and then single tokens, rotated and appended, attended by the
    sparse decode over every block: dense attention of the same rows."""
    from sparse_attention_decode_compress_b200 import (new_workspace, qsa_sparse_decode_merged,
                                                       qsa_sparse_decode_workspace_bytes)
    Hq, Hkv, D, page, B, S = 16, 2, 128, 16, 3, 2
    lens = [70, 33, 101]
    c = A.PagedKV([n + 4 for n in lens], Hkv, D, kv, page, "cuda", seed=161)
    if kv == "e4m3":  # scales that the appended rows fit
        c.k_scale.fill_(2.0 ** -5)
        c.v_scale.fill_(2.0 ** -5)
    c.k.zero_()
    c.v.zero_()
    cache = c.cache()
    rope = QSARopeAppend(cache, Hq, theta=1e6)

    def append(pos, new, seed):
        x = queries((sum(new), Hq + 2 * Hkv, D), kv, seed).cuda()
        cu = np.concatenate([[0], np.cumsum(new)]).tolist()
        return rope(ints(pos), ints(cu), x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:])

    append([0] * B, lens, 162)
    for step in range(3):
        q = append([n + step for n in lens], [1] * B, 163 + step).view(B, 1, Hq, D)
        now = [n + step + 1 for n in lens]
        topk = max(-(-n // 4) for n in now)
        sel = torch.full((B, topk), -1, dtype=torch.int32)
        for r, n in enumerate(now):
            sel[r, :-(-n // 4)] = torch.arange(-(-n // 4))
        f32 = dict(dtype=torch.float32, device="cuda")
        o_part, lse_part = torch.empty((S, B, 1, Hq, D), **f32), torch.empty((S, B, 1, Hq), **f32)
        o, lse = torch.empty((B, 1, Hq, D), **f32), torch.empty((B, 1, Hq), **f32)
        ws = new_workspace(qsa_sparse_decode_workspace_bytes(B, 1, Hq, Hkv, D, topk, S), "cuda")
        qsa_sparse_decode_merged(cache, q, ints(now), sel.cuda(), D ** -0.5, S, o_part, lse_part, o, lse, ws)
        c.k, c.v = cache.k_cache.cpu(), cache.v_cache.cpu()
        A.check(o, lse, prefix_want(c, q.cpu(), now, 1), kv, D, f"step {step}")


# --------------------------------------------------- each weight once rounded --
@pytest.mark.parametrize("kv", ["f32", "bf16", "e4m3"])
def test_weights_are_rounded_once(kv):
    """Rows of a chunk whose windows begin in the first and in the second 32 keys
    of a tile.  The first ones' weights 2^-c, c = 1 - log2(1 + 2^-8 + 2^-11), round
    up to bf16 by nearly 2^-8, and so would their products with another 2^-c, the
    factor of a maximum that is higher by one step: rounded again behind the keys
    that the second ones start with, they would be off by 2^-7.  The two keys of
    the maxima have values of zero, the others 128 values that share the error."""
    D, page, n, window, first = 128, 64, 32, 100, 16
    L = first + n - 1 + window  # token i sees the keys from first + i on
    c = A.PagedKV([L], 1, D, kv, page, "cuda", seed=171)
    if kv == "e4m3":
        c.k_scale.fill_(1.0)
        c.v_scale.fill_(1.0)
    typ = c.k.dtype
    k, v = torch.zeros((L, D)), torch.zeros((L, D))
    k[:, 0] = -8.0
    k[first:31, 0], k[31, 0], k[40, 0] = -1.0, 0.0, 1.0
    v[first:31] = 1 + torch.arange(D) / 128
    for t in range(L):
        pg = int(c.table_host[0, t // page])
        c.k[pg, t % page, 0], c.v[pg, t % page, 0] = k[t].to(typ), v[t].to(typ)
    q = torch.zeros((n, 1, D), dtype=torch.float32 if kv == "f32" else torch.bfloat16)
    q[..., 0] = 1.0
    scale = (1 - math.log2(1 + 2.0 ** -8 + 2.0 ** -11)) * math.log(2)
    keys = [A.visible(L - n + i, window, 0) for i in range(n)]
    want = A.stack([A.attend(q[i], c.values("k", 0, keys[i]), c.values("v", 0, keys[i]), scale) for i in range(n)])
    o, lse = QSAWindowPrefill(c.cache(), 1, n, n, 1, window, sm_scale=scale)(q.cuda(), ints([0, n]), ints([L]))
    A.check(o, lse, want, kv, D, "chunk")
