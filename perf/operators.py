"""What the operators over the paged K/V cache are measured on.

Four calls that write or read the same paged caches as the sparse decode:

* ``rope``     rotary positions on new queries and keys, and the append of the
               new K/V rows to their pages;
* ``window``   decode attention over a sliding window and the first tokens
               (sinks) of each request, 1 to 4 query tokens per request;
* ``chunk``    the same visibility for a prefill chunk of many query tokens;
* ``prefix``   decode attention of a batch whose requests share long prefixes,
               each prefix read once for its whole group.

``run`` computes a case in elementary torch operations, or, with ``own`` set,
through the package.  Outputs: rotated queries and the caches (``rope``),
attention output in the query type and its float32 log-sum-exp (the others).
"""
import math
import random

import numpy as np
import torch

own = False

_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
_ELEM = {"f32": 4, "bf16": 2, "e4m3": 1}


# ------------------------------------------------------------------ cases --
def listed():
    return [
        # a decode step of 128 long requests: one new token each, the QKV
        # projection's output as one fused tensor (latency of a small call)
        dict(name="rope_decode_b128", op="rope", batch=128, new_lo=1, new_hi=1, pos_lo=262143,
             pos_hi=262143, Hq=16, Hkv=2, D=128, kv="bf16", page=64, rotary=128, interleaved=False,
             scaling="none", factor=1.0, fused=True, lens=1),
        # a prefill chunk of four requests at 32k
        dict(name="rope_chunk_4x1024", op="rope", batch=4, new_lo=1024, new_hi=1024, pos_lo=31744,
             pos_hi=31744, Hq=16, Hkv=2, D=128, kv="bf16", page=64, rotary=128, interleaved=False,
             scaling="none", factor=1.0, fused=True, lens=2),
        # whole prompts of odd lengths, half of each head rotated, neighbouring
        # pairs, positions stretched for long contexts
        dict(name="rope_prompts_ragged", op="rope", batch=17, new_lo=301, new_hi=4001, pos_lo=0,
             pos_hi=1000001, Hq=32, Hkv=4, D=128, kv="bf16", page=64, rotary=64, interleaved=True,
             scaling="yarn", factor=4.0, fused=False, lens=3),
        # one float32 request (latency)
        dict(name="window_tiny_f32", op="window", batch=1, T=1, ctx_lo=4096, ctx_hi=4096, Hq=8, Hkv=1,
             D=64, kv="f32", page=16, window=1024, sinks=4, lens=4),
        # serving at 32k contexts
        dict(name="window_b32_32k", op="window", batch=32, T=1, ctx_lo=32768, ctx_hi=32768, Hq=16, Hkv=2,
             D=128, kv="bf16", page=64, window=4096, sinks=64, lens=5),
        # a large mixed batch on an 8-bit cache, contexts from 37 tokens to a million
        dict(name="window_mixed_fp8", op="window", batch=256, T=1, ctx_lo=37, ctx_hi=1048576, Hq=32,
             Hkv=4, D=128, kv="e4m3", page=64, window=4096, sinks=16, lens=6),
        # verification of three draft tokens
        dict(name="window_verify_b64", op="window", batch=64, T=4, ctx_lo=1000, ctx_hi=262144, Hq=16,
             Hkv=2, D=128, kv="bf16", page=64, window=2000, sinks=4, lens=7),
        # a prefill chunk of four requests at 32k
        dict(name="chunk_4x1024", op="chunk", batch=4, new_lo=1024, new_hi=1024, ctx_lo=32768,
             ctx_hi=32768, Hq=16, Hkv=2, D=128, kv="bf16", page=64, window=4096, sinks=64, lens=8),
        # a long prompt's chunk in one request: the largest
        dict(name="chunk_long_8192", op="chunk", batch=1, new_lo=8192, new_hi=8192, ctx_lo=24577,
             ctx_hi=24577, Hq=32, Hkv=4, D=128, kv="bf16", page=64, window=8192, sinks=4, lens=9),
        # a batch behind one 28k prompt
        dict(name="prefix_b32_28k", op="prefix", groups=1, per=32, T=1, prefix_lo=28672,
             prefix_hi=28672, tail_lo=1, tail_hi=4096, Hq=16, Hkv=2, D=128, kv="bf16", page=64, lens=10),
        # 128 requests behind one document of a quarter million tokens
        dict(name="prefix_b128_250k", op="prefix", groups=1, per=128, T=1, prefix_lo=250000,
             prefix_hi=250000, tail_lo=1, tail_hi=8192, Hq=16, Hkv=2, D=128, kv="bf16", page=64, lens=11),
        # eight prompts of different lengths, 8-bit cache, two query tokens
        dict(name="prefix_8x16_fp8", op="prefix", groups=8, per=16, T=2, prefix_lo=3001,
             prefix_hi=16384, tail_lo=2, tail_hi=1025, Hq=32, Hkv=4, D=128, kv="e4m3", page=64, lens=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case of the listed ones' ranges."""
    op = rng.choice(("rope", "window", "window", "chunk", "prefix"))
    Hq, Hkv = rng.choice(((16, 2), (32, 4), (8, 1), (12, 4), (8, 8)))
    c = dict(op=op, Hq=Hq, Hkv=Hkv, D=rng.choice((64, 128, 128)), page=rng.choice((16, 64, 64, 128, 20)),
             lens=rng.randrange(1 << 30))
    if op == "rope":
        c["kv"] = rng.choice(("f32", "bf16", "bf16"))
        c["batch"] = _log(rng, 1, 256)
        most = max(1, 20000 // c["batch"])
        c["new_lo"] = 1
        c["new_hi"] = _log(rng, 1, most)
        c["pos_lo"], c["pos_hi"] = 0, _log(rng, 100, 1000000)
        c["rotary"] = rng.choice((c["D"], c["D"], c["D"] // 2, 32, 48))
        c["interleaved"] = rng.random() < 0.5
        c["scaling"] = rng.choice(("none", "linear", "ntk", "yarn"))
        c["factor"] = 1.0 if c["scaling"] == "none" else rng.choice((2.0, 4.0, 8.0, 2.5))
        c["fused"] = rng.random() < 0.5
        return c
    c["kv"] = rng.choice(("f32", "bf16", "bf16", "e4m3"))
    if op == "window":
        c["T"] = rng.choice((1, 1, 2, 3, 4))
        c["batch"] = _log(rng, 1, 256)
        c["ctx_lo"] = _log(rng, 4, 4000)
        c["ctx_hi"] = _log(rng, c["ctx_lo"], 1000000)
        c["window"], c["sinks"] = _log(rng, 1, 4096), rng.choice((0, 1, 4, 64, 101))
    elif op == "chunk":
        c["batch"] = _log(rng, 1, 16)
        c["new_lo"] = 1
        c["new_hi"] = _log(rng, 2, 4096 // c["batch"])
        c["ctx_lo"] = c["new_hi"]
        c["ctx_hi"] = _log(rng, c["ctx_lo"], 100000)
        c["window"], c["sinks"] = _log(rng, 1, 4096), rng.choice((0, 1, 4, 64, 101))
    else:
        c["T"] = rng.choice((1, 1, 2, 4))
        c["groups"] = _log(rng, 1, 16)
        c["per"] = _log(rng, 1, max(1, 128 // c["groups"]))
        c["prefix_hi"] = _log(rng, 10, 200000 // c["groups"])
        c["prefix_lo"] = max(1, int(c["prefix_hi"] * rng.uniform(0.3, 1)))
        c["tail_lo"] = c["T"]
        c["tail_hi"] = max(c["T"], _log(rng, 4, 4096))
    if c["kv"] == "f32":  # the float32 cache is the small setting
        c["batch"] = min(c.get("batch", 1), 8)
        if op == "chunk":
            c["new_hi"] = min(c["new_hi"], 256)
        if op == "prefix":
            c["per"] = min(c["per"], 8)
    return c


def _spread(rng, lo, hi, n):
    """n whole numbers of [lo, hi], spread over their logarithm where the range is wide."""
    if hi > 10 * max(lo, 1):
        return [min(hi, max(lo, int(math.exp(rng.uniform(math.log(max(lo, 1)), math.log(hi)))))) for _ in range(n)]
    return [rng.randint(lo, hi) for _ in range(n)]


def _lengths(case):
    """The case's lengths on the host, the same for every seed."""
    rng = random.Random(case["lens"])
    op = case["op"]
    if op == "rope":
        return dict(new=_spread(rng, case["new_lo"], case["new_hi"], case["batch"]),
                    pos0=_spread(rng, case["pos_lo"], case["pos_hi"], case["batch"]))
    if op == "window":
        return dict(ctx=[max(case["T"], n) for n in _spread(rng, case["ctx_lo"], case["ctx_hi"], case["batch"])])
    if op == "chunk":
        new = _spread(rng, case["new_lo"], case["new_hi"], case["batch"])
        ctx = _spread(rng, case["ctx_lo"], case["ctx_hi"], case["batch"])
        return dict(new=new, ctx=[max(a, b) for a, b in zip(new, ctx)])
    pre = _spread(rng, case["prefix_lo"], case["prefix_hi"], case["groups"])
    tail = _spread(rng, case["tail_lo"], case["tail_hi"], case["groups"] * case["per"])
    return dict(prefix=pre, ctx=[pre[i // case["per"]] + t for i, t in enumerate(tail)])


# ----------------------------------------------------------------- inputs --
def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _offsets(v):
    return [0] + np.cumsum(v).tolist()


def _table(rows, width, perm):
    """Block table [len(rows), width]: rows[r] lists (first logical page,
    count) runs that get pages of their own from `perm`, the rest is -1."""
    t, at = np.full((len(rows), width), -1, dtype=np.int32), 0
    for r, runs in enumerate(rows):
        for first, count in runs:
            t[r, first:first + count] = perm[at:at + count]
            at += count
    return t, at


def _runs(parts, page):
    """(first, count) runs of the pages under the token ranges `parts`."""
    pages = sorted({p for a, b in parts for p in range(a // page, (b - 1) // page + 1) if b > a})
    runs = []
    for p in pages:
        if runs and runs[-1][0] + runs[-1][1] == p:
            runs[-1][1] += 1
        else:
            runs.append([p, 1])
    return runs


def _pool(case, num_pages, gen):
    """K/V pools of num_pages pages, standard normal, in the cache's type."""
    shape = (num_pages, case["page"], case["Hkv"], case["D"])
    made = []
    for _ in range(2):
        if case["kv"] != "e4m3":
            made.append((torch.randn(shape, generator=gen, device="cuda", dtype=_TYPES[case["kv"]]), None))
            continue
        x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16).float()
        s = x.abs().amax(dim=(1, 3)) / 448.0
        made.append(((x / s[:, None, :, None]).to(torch.float8_e4m3fn), s))
    return made


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    n, op, P = _lengths(case), case["op"], case["page"]
    s = dict(case=case, n=n)
    if op == "rope":
        rows = [_runs([(p, p + m)], P) for p, m in zip(n["pos0"], n["new"])]
    elif op == "window":
        # pages behind the window are not mapped any more
        rows = [_runs([(0, min(case["sinks"], L)), (max(0, L - case["T"] + 1 - case["window"]), L)], P)
                for L in n["ctx"]]
    elif op == "chunk":
        rows = [_runs([(0, min(case["sinks"], L)), (max(0, L - m + 1 - case["window"]), L)], P)
                for m, L in zip(n["new"], n["ctx"])]
    else:
        # whole pages of the prefix are shared; its last tokens sit in each
        # request's own first page
        rows, per = [], case["per"]
        for g, pre in enumerate(n["prefix"]):
            rows.append([(0, pre // P)] if pre // P else [])
        for r, L in enumerate(n["ctx"]):
            first = n["prefix"][r // per] // P
            rows.append([(first, -(-L // P) - first)])
    used = sum(c for r in rows for _, c in r)
    width = max([f + c for r in rows for f, c in r] + [1])
    perm = np.random.RandomState(seed % (1 << 31)).permutation(used)
    table, _ = _table(rows, width, perm)
    if op == "prefix":
        G, per = case["groups"], case["per"]
        own_rows, shared = table[G:], table[:G]
        for g, pre in enumerate(n["prefix"]):
            own_rows[g * per:(g + 1) * per, :pre // P] = shared[g, :pre // P]
        table = own_rows
    (s["k"], s["ks"]), (s["v"], s["vs"]) = _pool(case, used, gen)
    if op == "prefix":
        # the prefix's last, unfilled page is the same in every request of the group
        for g, pre in enumerate(n["prefix"]):
            m = pre % P
            if m:
                own_pages = torch.from_numpy(table[g * per:(g + 1) * per, pre // P].astype(np.int64)).cuda()
                for c, sc in ((s["k"], s["ks"]), (s["v"], s["vs"])):
                    flat = c.view(torch.uint8) if case["kv"] == "e4m3" else c
                    flat[own_pages, :m] = flat[own_pages[0], :m].clone()
                    if sc is not None:
                        sc[own_pages] = sc[own_pages[0]].clone()
    s["table"] = torch.from_numpy(table).cuda()
    qd = torch.float32 if case["kv"] == "f32" else torch.bfloat16
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    if op == "rope":
        N = sum(n["new"])
        s["pos0"], s["cu"] = _ints(n["pos0"]), _ints(_offsets(n["new"]))
        if case["fused"]:
            qkv = torch.randn((N, Hq + 2 * Hkv, D), generator=gen, device="cuda", dtype=qd)
            s["q"], s["k_new"], s["v_new"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        else:
            s["q"], s["k_new"], s["v_new"] = (torch.randn((N, h, D), generator=gen, device="cuda", dtype=qd)
                                              for h in (Hq, Hkv, Hkv))
        s["q_out"] = torch.empty((N, Hq, D), device="cuda", dtype=qd)
    else:
        s["ctx"] = _ints(n["ctx"])
        if op == "chunk":
            s["cu"] = _ints(_offsets(n["new"]))
            shape = (sum(n["new"]), Hq, D)
        else:
            shape = (len(n["ctx"]), case["T"], Hq, D)
        s["q"] = torch.randn(shape, generator=gen, device="cuda", dtype=qd)
        if op == "prefix":
            s["cu"] = _ints([case["per"] * g for g in range(case["groups"] + 1)])
            s["prefix"] = _ints(n["prefix"])
    if own:  # the handle that a serving program makes once for these caches
        import sparse_attention_decode_compress_b200 as qsa
        cache = qsa.QSACache.allocate(s["k"], s["v"], s["table"], idx_dim=32, ring_rows=len(table),
                                      k_scale=s["ks"], v_scale=s["vs"])
        if op == "rope":
            s["handle"] = qsa.QSARopeAppend(cache, Hq, rotary_dim=case["rotary"], theta=1e6,
                                            interleaved=case["interleaved"], scaling=case["scaling"],
                                            factor=case["factor"], original_max_position=32768)
        elif op == "window":
            s["handle"] = qsa.QSAWindowDecode(cache, len(n["ctx"]), case["T"], Hq, case["window"], case["sinks"])
        elif op == "chunk":
            s["handle"] = qsa.QSAWindowPrefill(cache, len(n["ctx"]), shape[0], max(n["new"]), Hq,
                                               case["window"], case["sinks"])
        else:
            s["handle"] = qsa.QSAPrefixDecode(
                cache, len(n["ctx"]), case["T"], Hq, case["groups"], max_group=case["per"],
                max_prefix=max(n["prefix"]),
                max_tail=max(L - n["prefix"][i // case["per"]] for i, L in enumerate(n["ctx"])))
    return s


# ------------------------------------------------------------ plain forms --
def _frequencies(case):
    """Radians per token of each rotated pair (float64) and the factor on cos and sin."""
    R, base, factor = case["rotary"], 1e6, case["factor"]
    i = np.arange(R // 2, dtype=np.float64)
    if case["scaling"] == "ntk":
        base = base * factor ** (R / (R - 2))
    f = base ** (-2.0 * i / R)
    if case["scaling"] == "linear":
        f = f / factor
    if case["scaling"] != "yarn":
        return f, 1.0
    # pairs that turn more than 32 times within the trained length keep their
    # frequency, those below one turn are stretched, a ramp lies between
    at = [R * math.log(32768 / (2 * math.pi * turns)) / (2 * math.log(base)) for turns in (32.0, 1.0)]
    low, high = max(math.floor(at[0]), 0), min(math.ceil(at[1]), R - 1)
    ramp = np.clip((i - low) / max(high - low, 0.001), 0.0, 1.0)
    return f * (1 - ramp) + f / factor * ramp, 0.1 * math.log(factor) + 1.0


def _rotate(x, cos, sin, case):
    R = case["rotary"]
    a, b = (x[..., 0:R:2], x[..., 1:R:2]) if case["interleaved"] else (x[..., :R // 2], x[..., R // 2:R])
    u, w = a * cos - b * sin, a * sin + b * cos
    r = torch.stack((u, w), -1).flatten(-2) if case["interleaved"] else torch.cat((u, w), -1)
    return torch.cat((r, x[..., R:]), -1)


def _plain_rope(s):
    c = s["case"]
    N = s["q"].shape[0]
    cu = s["cu"].long()
    row = torch.searchsorted(cu[1:].contiguous(), torch.arange(N, device="cuda"), right=True)
    pos = s["pos0"].long()[row] + torch.arange(N, device="cuda") - cu[row]
    f, m = _frequencies(c)
    angle = pos.double()[:, None] * torch.from_numpy(f).cuda()
    cos, sin = ((fn(angle) * m).float()[:, None, :] for fn in (torch.cos, torch.sin))
    q = _rotate(s["q"].float(), cos, sin, c).to(s["q"].dtype)
    page, off = s["table"].long()[row, pos // c["page"]], pos % c["page"]
    s["k"][page, off] = _rotate(s["k_new"].float(), cos, sin, c).to(s["k"].dtype)
    s["v"][page, off] = s["v_new"].to(s["v"].dtype)
    return q, s["k"], s["v"]


def _rows(s, table, pos, which):
    """Rows [R, J, Hkv, D] of positions pos [R, J] in float32 (page 0 stands
    in where there is none: those are masked)."""
    c = s["case"]
    at = pos.clamp(min=0)
    page = torch.gather(table.long(), 1, (at // c["page"]).clamp(max=table.shape[1] - 1)).clamp(min=0)
    x = s[which][page, at % c["page"]].float()
    if s[which + "s"] is not None:
        x = x * s[which + "s"][page][..., None]
    return x


def _attend(s, q, pos, seen, table):
    """Unnormalised attention of q [R, n, Hkv, G, D] over positions pos
    [R, J], seen [R, n, J]: maximum, sum and weighted values in float32."""
    x = torch.einsum("rnhgd,rjhd->rhgnj", q, _rows(s, table, pos, "k")) * s["case"]["D"] ** -0.5
    x = x.masked_fill(~seen[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - m.masked_fill(m == -math.inf, 0.0))
    o = torch.einsum("rhgnj,rjhd->rnhgd", p, _rows(s, table, pos, "v"))
    return m[..., 0].permute(0, 3, 1, 2), p.sum(-1).permute(0, 3, 1, 2), o


def _finish(m, l, o, dtype):
    ok = l > 0
    o = torch.where(ok[..., None], o / torch.where(ok, l, 1.0)[..., None], 0.0)
    return o.flatten(2, 3).to(dtype), torch.where(ok, m + torch.log(torch.where(ok, l, 1.0)), -math.inf).flatten(2)


def _heads(q, c):
    return q.float().unflatten(-2, (c["Hkv"], c["Hq"] // c["Hkv"]))


def _windowed(s, q, ctx):
    """q [R, n, Hq, D], the newest n tokens of each request."""
    c, n, W = s["case"], q.shape[1], s["case"]["window"]
    ctx = ctx.long()[:, None]
    p = ctx - n + torch.arange(n, device="cuda")
    sink = torch.arange(c["sinks"], device="cuda").expand(ctx.shape[0], -1)
    near = ctx - n - W + 1 + torch.arange(n + W - 1, device="cuda")
    pos = torch.cat((sink, near), 1)
    seen = pos[:, None, :] <= p[..., None]
    first = torch.arange(pos.shape[1], device="cuda") < c["sinks"]
    seen &= first | ((pos[:, None, :] > p[..., None] - W) & (pos[:, None, :] >= c["sinks"]))
    return _finish(*_attend(s, _heads(q, c), pos, seen, s["table"]), q.dtype)


def _plain_chunk(s):
    cu, ctx = s["cu"].long(), s["ctx"]
    n = max(s["n"]["new"])
    # requests shorter than the longest: their rows end with the newest token
    at = cu[1:, None] - n + torch.arange(n, device="cuda")
    live = at >= cu[:-1, None]
    o, lse = _windowed(s, s["q"][at.clamp(min=0)], ctx)
    return o[live], lse[live]


def _plain_prefix(s):
    c, T = s["case"], s["case"]["T"]
    G, per, Hq, D = c["groups"], c["per"], c["Hq"], c["D"]
    ctx, pre = s["ctx"].long(), s["prefix"].long()
    mine = pre.repeat_interleave(per, output_size=G * per)
    p = ctx[:, None] - T + torch.arange(T, device="cuda")
    pos = torch.arange(max(s["n"]["prefix"]), device="cuda").expand(G, -1)
    seen = (pos < pre[:, None])[:, None, :] & (pos[:, None, :] <= p.view(G, per * T, 1))
    a = _attend(s, _heads(s["q"].view(G, per * T, Hq, D), c), pos, seen, s["table"][::per])
    longest = max(L - s["n"]["prefix"][i // per] for i, L in enumerate(s["n"]["ctx"]))
    pos = mine[:, None] + torch.arange(longest, device="cuda")
    b = _attend(s, _heads(s["q"], c), pos, pos[:, None, :] <= p[..., None], s["table"])
    m0, l0, o0 = (x.reshape(y.shape) for x, y in zip(a, b))
    m1, l1, o1 = b
    m = torch.maximum(m0, m1)
    f0, f1 = (torch.exp(x - m).nan_to_num(0.0) for x in (m0, m1))
    return _finish(m, l0 * f0 + l1 * f1, o0 * f0[..., None] + o1 * f1[..., None], s["q"].dtype)


def run(state):
    s, op = state, state["case"]["op"]
    if own:
        h = s["handle"]
        if op == "rope":
            h(s["pos0"], s["cu"], s["q"], s["k_new"], s["v_new"], s["q_out"])
            return s["q_out"], s["k"], s["v"]
        if op == "window":
            return h(s["q"], s["ctx"])
        if op == "chunk":
            return h(s["q"], s["cu"], s["ctx"])
        return h(s["q"], s["ctx"], s["cu"], s["prefix"])
    if op == "rope":
        return _plain_rope(s)
    if op == "window":
        return _windowed(s, s["q"], s["ctx"])
    return _plain_chunk(s) if op == "chunk" else _plain_prefix(s)


# ------------------------------------------------------------------ costs --
def _visible(n, L, window, sinks):
    """(query, key) pairs of the newest n of L tokens, and the distinct keys they read."""
    p = np.arange(L - n, L, dtype=np.int64)
    lo = np.maximum(0, p + 1 - window)
    pairs = int((p + 1 - lo + np.minimum(lo, sinks)).sum())
    return pairs, int(L - lo[0] + min(lo[0], sinks))


def work(case):
    n, op = _lengths(case), case["op"]
    Hq, Hkv, D, e = case["Hq"], case["Hkv"], case["D"], _ELEM[case["kv"]]
    qe = 4 if case["kv"] == "f32" else 2
    if op == "rope":
        N = sum(n["new"])
        return {"bytes": 2 * N * (Hq + 2 * Hkv) * D * qe + 8 * len(n["new"]),
                "flops": 3 * N * (Hq + Hkv) * case["rotary"]}
    if op == "prefix":
        T, per = case["T"], case["per"]
        keys, pairs, tokens = sum(n["prefix"]), 0, len(n["ctx"]) * T
        for i, L in enumerate(n["ctx"]):
            keys += L - n["prefix"][i // per]
            pairs += _visible(T, L, L, 0)[0]
    else:
        new = n["new"] if op == "chunk" else [case["T"]] * len(n["ctx"])
        both = [_visible(m, L, case["window"], case["sinks"]) for m, L in zip(new, n["ctx"])]
        pairs, keys, tokens = sum(b[0] for b in both), sum(b[1] for b in both), sum(new)
    scales = 8 * Hkv * -(-keys // case["page"]) if case["kv"] == "e4m3" else 0
    return {"bytes": 2 * keys * Hkv * D * e + scales + tokens * Hq * (2 * D * qe + 4) + 4 * -(-keys // case["page"]),
            "flops": 4 * pairs * Hq * D}


# ------------------------------------------------------------------ exact --
def exact(case, seed):
    """The definition in float64, request by request."""
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    n, P, op = s["n"], case["page"], case["op"]
    table = s["table"].cpu().numpy()
    if op == "rope":
        return _exact_rope(case, s, table)
    scale = 1.0 / math.sqrt(case["D"])
    G = case["Hq"] // case["Hkv"]
    outs, lses = [], []
    cu = _offsets(n["new"]) if op == "chunk" else None
    for r, L in enumerate(n["ctx"]):
        q = s["q"][cu[r]:cu[r + 1]] if op == "chunk" else s["q"][r]
        m = q.shape[0]
        W, S = (L, 0) if op == "prefix" else (case["window"], min(case["sinks"], L))
        a = max(0, L - m + 1 - W)
        keys = torch.tensor(sorted(set(range(min(S, a))) | set(range(a, L))), device="cuda")
        page = torch.from_numpy(table[r].astype(np.int64)).cuda()[keys // P]
        kv = []
        for name in ("k", "v"):
            x = s[name][page, keys % P].double()
            kv.append(x if s[name + "s"] is None else x * s[name + "s"][page].double()[..., None])
        o = torch.empty((m, case["Hq"], case["D"]), dtype=torch.float64, device="cuda")
        lse = torch.empty((m, case["Hq"]), dtype=torch.float64, device="cuda")
        for b in range(0, m, 1024):
            p = torch.arange(L - m + b, L - m + min(m, b + 1024), device="cuda")[:, None]
            hide = (keys > p) | ((keys <= p - W) & (keys >= S))
            for h in range(case["Hkv"]):
                for g in range(h * G, (h + 1) * G):
                    x = (q[b:b + 1024, g].double() @ kv[0][:, h].T) * scale
                    x[hide] = -math.inf
                    e = torch.logsumexp(x, 1, keepdim=True)
                    lse[b:b + 1024, g] = e[:, 0]
                    o[b:b + 1024, g] = torch.exp(x - e) @ kv[1][:, h]
        outs.append(o)
        lses.append(lse)
    if op == "chunk":
        return torch.cat(outs), torch.cat(lses)
    return torch.stack(outs), torch.stack(lses)


def _exact_rope(case, s, table):
    n, P, R = s["n"], case["page"], case["rotary"]
    f, m = _frequencies(case)
    pos = np.concatenate([np.arange(p, p + k) for p, k in zip(n["pos0"], n["new"])])
    row = np.repeat(np.arange(len(n["new"])), n["new"])
    z = np.exp(1j * (pos[:, None].astype(np.float64) * f)) * m
    z = torch.from_numpy(z).cuda()[:, None, :]
    first = torch.arange(0, R, 2) if case["interleaved"] else torch.arange(R // 2)
    second = first + (1 if case["interleaved"] else R // 2)

    def turned(x):
        y = x.double().clone()
        w = torch.complex(y[..., first], y[..., second]) * z
        y[..., first], y[..., second] = w.real, w.imag
        return y

    k, v = s["k"].double(), s["v"].double()
    page, off = torch.from_numpy(table[row, pos // P].astype(np.int64)).cuda(), torch.from_numpy(pos % P).cuda()
    k[page, off], v[page, off] = turned(s["k_new"]), s["v_new"].double()
    return turned(s["q"]), k, v
