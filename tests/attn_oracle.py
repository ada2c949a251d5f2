"""Plain float64 forms of the calls over whole key ranges (rotary append,
window attention, shared-prefix decode) and the error bounds their kernels are
held to.  Nothing here is shared with the package."""
from __future__ import annotations

import math

import numpy as np
import torch

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}


class PagedKV:
    """Random K/V in a paged cache, and the same values as float64 rows.

    lens[r] tokens per request on pages of their own; share[r] = (other, n):
    the first n pages are those of request `other`."""

    def __init__(self, lens, Hkv, D, kv="bf16", page=16, device="cpu", seed=0, share=None, spare_pages=3, std=1.0):
        gen = torch.Generator().manual_seed(seed)
        rng = np.random.RandomState(seed)
        self.lens, self.page, self.kv, self.Hkv, self.D = list(lens), page, kv, Hkv, D
        B = len(lens)
        width = max([-(-n // page) for n in lens] + [1])
        need, table = 0, np.full((B, width), -1, dtype=np.int32)
        for r, n in enumerate(lens):
            pages = -(-n // page)
            shared = 0
            if share and r in share:
                other, shared = share[r]
                table[r, :shared] = table[other, :shared]
            table[r, shared:pages] = np.arange(need, need + pages - shared)
            need += pages - shared
        perm = rng.permutation(need + spare_pages)
        table = np.where(table >= 0, perm[np.clip(table, 0, None)], -1).astype(np.int32)
        self.num_pages = need + spare_pages
        self.table_host = table
        shape = (self.num_pages, page, Hkv, D)
        self.k_scale = self.v_scale = None
        made = []
        for i in range(2):
            x = torch.randn(shape, generator=gen) * std
            if kv == "e4m3":
                s = torch.exp2(torch.rand((self.num_pages, Hkv), generator=gen) * 6 - 9)  # 2^-9 .. 2^-3
                made.append(((x / s[:, None, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn), s))
            else:
                made.append((x.to(TYPES[kv]), None))
        (self.k, self.k_scale), (self.v, self.v_scale) = made
        self.device = device

    def values(self, which, r, keys):
        """float64 rows [len(keys), Hkv, D] of request r."""
        keys = torch.as_tensor(keys, dtype=torch.long)
        pages = torch.as_tensor(self.table_host[r].astype(np.int64))[keys // self.page]
        x = getattr(self, which)[pages, keys % self.page].double()
        s = getattr(self, which + "_scale")
        return x if s is None else x * s[pages].double()[..., None]

    def poison(self, seen):
        """NaN in every cache row that no query sees: seen[r] lists the keys
        that some query reads through row r."""
        hit = torch.zeros((self.num_pages, self.page), dtype=torch.bool)
        for r, keys in seen.items():
            keys = torch.as_tensor(sorted(keys), dtype=torch.long)
            if len(keys):
                hit[torch.as_tensor(self.table_host[r].astype(np.int64))[keys // self.page], keys % self.page] = True
        for t in (self.k, self.v):
            if self.kv == "e4m3":
                t.view(torch.uint8)[~hit] = 0x7F
            else:
                t[~hit] = float("nan")

    def unmap(self, seen):
        """-1 in the block table for pages that no query reads."""
        for r in range(len(self.lens)):
            used = {k // self.page for k in seen.get(r, ())}
            for lp in range(self.table_host.shape[1]):
                if lp not in used:
                    self.table_host[r, lp] = -1

    def cache(self):
        from sparse_attention_decode_compress_b200 import QSACache
        dev = self.device
        up = lambda t: None if t is None else t.to(dev)
        self.dk, self.dv = up(self.k), up(self.v)
        return QSACache.allocate(self.dk, self.dv, torch.from_numpy(self.table_host).to(dev), idx_dim=32,
                                 ring_rows=max(1, len(self.lens)), k_scale=up(self.k_scale),
                                 v_scale=up(self.v_scale))


def visible(p, window, sinks):
    """Keys a query at position p sees."""
    if p < 0:
        return []
    lo = max(0, p + 1 - window)
    return list(range(min(sinks, lo))) + list(range(lo, p + 1))


def attend(q, K, V, scale):
    """q [Hq, D], K, V [n, Hkv, D] float64 -> o [Hq, D], lse [Hq], and per head
    A = sum p |v| [Hq, D] and the largest sum of |q_d k_d| * scale [Hq]."""
    Hq, D = q.shape
    n, Hkv, _ = K.shape
    G = Hq // Hkv
    if n == 0:
        z = torch.zeros((Hq, D), dtype=torch.float64)
        return z, torch.full((Hq,), -math.inf, dtype=torch.float64), z, torch.zeros(Hq, dtype=torch.float64)
    qg = q.double().view(Hkv, G, D)
    s = torch.einsum("hgd,nhd->hgn", qg, K) * scale
    e = torch.logsumexp(s, -1)
    p = torch.exp(s - e[..., None])
    o = torch.einsum("hgn,nhd->hgd", p, V)
    A = torch.einsum("hgn,nhd->hgd", p, V.abs())
    mag = torch.einsum("hgd,nhd->hgn", qg.abs(), K.abs()).amax(-1) * scale
    return o.reshape(Hq, D), e.reshape(Hq), A.reshape(Hq, D), mag.reshape(Hq)


def bounds(o, lse, A, mag, kv, D):
    """(bound on |o error|, bound on |lse error|), element by element.

    Logits: a float32 sum of D products, each add off by at most 2^-23 of the
    running magnitude (2^-24 rounded, 2^-23 where an adder cuts): d = D 2^-23
    sum|q k|, and 2^-22 relative for scaling and the base change.  A weight
    exp(s) is then off by a factor within 2 (d + 2^-20) (its own exponential
    and its row's; 2^-20 covers exp2 to 2 units, up to 64 float32 partial
    sums of 2^-24 and the merge's logarithms).  16-bit caches round each
    weight once more to bf16 or finer (2^-8 of it), 8-bit caches also each
    dequantised value (2^-8), and the output itself is rounded to bf16
    (2^-8 of it).
    """
    d = (D * 2.0 ** -23 + 2.0 ** -22) * mag + 2.0 ** -20
    rel = 2 * d
    bo = rel[..., None] * A
    if kv != "f32":
        bo = bo + 2.0 ** -8 * A * (2 if kv == "e4m3" else 1) * (1 + 2.0 ** -7) + 2.0 ** -8 * (o.abs() + bo)
    bl = d + 2.0 ** -22 * torch.where(torch.isinf(lse), torch.zeros_like(lse), lse.abs())
    return bo + 1e-30, bl


def check(got_o, got_lse, want, kv, D, what=""):
    o, lse, A, mag = want
    bo, bl = bounds(o, lse, A, mag, kv, D)
    go, gl = got_o.double().cpu(), got_lse.double().cpu()
    assert torch.isfinite(go).all(), f"{what}: non-finite output"
    none = torch.isinf(lse)
    assert (gl[none] == -math.inf).all() and (go[none] == 0).all(), f"{what}: a row that sees nothing"
    worst = ((go - o).abs() / bo)[~none]
    assert worst.numel() == 0 or worst.max() <= 1, f"{what}: o off by {worst.max():.3f} of its bound"
    worst = ((gl - lse).abs()[~none] / bl[~none])
    assert worst.numel() == 0 or worst.max() <= 1, f"{what}: lse off by {worst.max():.3f} of its bound"


def stack(rows):
    return tuple(torch.stack(x) for x in zip(*rows))


def rope_row(x, p, inv_freq, mscale, R, interleaved):
    """Rotated float64 copy of x [..., D] at position p, and per element the
    sum of the magnitudes of its two products."""
    y, mag = x.double().clone(), x.double().abs().clone()
    for i in range(R // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)
        c, s = math.cos(p * inv_freq[i]) * mscale, math.sin(p * inv_freq[i]) * mscale
        xa, xb = x[..., a].double(), x[..., b].double()
        y[..., a], y[..., b] = xa * c - xb * s, xa * s + xb * c
        mag[..., a] = mag[..., b] = (xa.abs() + xb.abs()) * mscale
    return y, mag
