"""What the cache operators are measured on.

The operators: attention over a paged cache of K and V rows in bf16, with a
sliding window and first tokens that stay visible ("attend"); the same over a
cache held in 4 bits ("attend_q4"); and storing bf16 rows in the 4-bit cache
and reading them back ("store_q4").

With ``own = False`` ``run`` computes each in its plain form (elementary torch
operations in fp32, rounded once at the end); with ``own = True`` it makes the
calls a user makes of ``mrope_qk_norm_b200``.

The 4-bit format: 32 consecutive elements of a head row share one scale, a
bf16 number of 5 significant bits, and an element stands for (code - 8) *
scale, which is a bf16 number exactly.  A head row of K holds element d =
32w + 8c + i (i < 8) in nibble i of the 4-byte word at byte c*(D/8) + 4w; a
head row of V holds element d = 32w + 4g + i (i < 4) in nibble i of the 2-byte
word at byte g*(D/16) + 2w.
"""
from __future__ import annotations

import math
import random

import torch

own = False

_DEV = "cuda"
_EPS_SCALE_BITS = 0x7FFFF  # low fp32 mantissa bits a 5-bit scale leaves empty


# --------------------------------------------------------------------------
# Cases
# --------------------------------------------------------------------------

def _attend(name, op, batch, q_lo, q_hi, len_lo, len_hi, hq, hkv, dim, page, window=0, sink=0,
            spread=1):
    c = {"op": op, "batch": batch, "q_lo": q_lo, "q_hi": q_hi, "len_lo": len_lo,
         "len_hi": len_hi, "hq": hq, "hkv": hkv, "dim": dim, "page": page, "window": window,
         "sink": sink, "spread": spread}
    if name:
        c["name"] = name
    return c


def _store(name, tokens, hkv, dim, page):
    c = {"op": "store_q4", "tokens": tokens, "hkv": hkv, "dim": dim, "page": page}
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one interactive user, a short chat: the launch latency shows
        _attend("decode_single", "attend", 1, 1, 1, 517, 517, 16, 8, 128, 16),
        # a decode step of a server's batch, every length between a greeting and a document
        _attend("decode_ragged", "attend", 32, 1, 1, 64, 8192, 32, 8, 128, 64, spread=2),
        # a decode step of a model with window layers: long caches of which little is read
        _attend("decode_window", "attend", 64, 1, 1, 300, 32768, 16, 8, 64, 32, window=1000,
                sink=4, spread=3),
        # two users with a book each in the cache
        _attend("decode_long", "attend", 2, 1, 1, 90001, 110000, 16, 8, 128, 64, spread=4),
        # a whole prompt at once
        _attend("prefill_prompt", "attend", 1, 8192, 8192, 8192, 8192, 16, 8, 128, 64),
        # a server step that mixes prompts, chunks of prompts and decoding users, window layers
        _attend("prefill_window_mixed", "attend", 12, 1, 4096, 700, 16384, 32, 8, 128, 48,
                window=2048, sink=4, spread=5),
        # the rows of one decode step go into the cache
        _store("store_step", 32, 8, 128, 64),
        # the rows of a prompt go into the cache
        _store("store_prompt", 8192, 8, 128, 64),
        # as decode_single, over the 4-bit cache
        _attend("q4_decode_single", "attend_q4", 1, 1, 1, 1213, 1213, 16, 8, 128, 16),
        # as decode_ragged, with the longer lengths the smaller cache has room for
        _attend("q4_decode_ragged", "attend_q4", 32, 1, 1, 64, 16384, 32, 8, 128, 64, spread=6),
        # as decode_long
        _attend("q4_decode_long", "attend_q4", 2, 1, 1, 120000, 140000, 16, 8, 128, 64,
                spread=7),
        # chunks of prompts whose beginnings are in the 4-bit cache already
        _attend("q4_prefill_chunk", "attend_q4", 4, 300, 512, 2000, 8192, 16, 8, 128, 64,
                window=4000, sink=4, spread=8),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case; the lengths are halved until it costs no more than the largest listed."""
    top = [work(c) for c in listed()]
    most = {k: max(w[k] for w in top) for k in ("bytes", "flops")}
    case = _draw(rng)
    while any(work(case)[k] > most[k] for k in most):
        for k in ("q_lo", "q_hi", "len_lo", "len_hi"):
            case[k] = (case[k] + 1) // 2
    return case


def _draw(rng):
    kind = rng.choice(["decode", "decode", "window", "prefill", "store", "q4", "q4", "q4_prefill"])
    spread = rng.randrange(1, 1 << 30)
    page = rng.choice([16, 32, 48, 64, 128, 256])
    if kind == "store":
        return _store(None, _log_int(rng, 1, 8192), rng.choice([1, 2, 4, 8]),
                      rng.choice([64, 128]), page)
    q4 = kind.startswith("q4")
    op = "attend_q4" if q4 else "attend"
    dim = rng.choice([64, 128]) if q4 else rng.choice([64, 80, 96, 128])
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 2, 3, 4, 8])
    window, sink = 0, 0
    if kind == "window" or rng.random() < 0.3:
        window, sink = _log_int(rng, 16, 8192), rng.choice([0, 1, 4, 17, 128])
    if kind in ("prefill", "q4_prefill"):
        batch = _log_int(rng, 1, 8)
        q_hi = _log_int(rng, 2, 4096 // batch if q4 else 8192 // batch)
        len_hi = max(q_hi, _log_int(rng, 128, 16384 // batch))
        return _attend(None, op, batch, rng.choice([1, q_hi]), q_hi, min(q_hi, len_hi), len_hi,
                       hq if hq <= 16 else 16, hkv, dim, page, window, sink, spread)
    batch = _log_int(rng, 1, 64)
    len_hi = _log_int(rng, 32, min(131072, (1 << 18) // batch))
    q = rng.choice([1, 1, 1, 2, 3, 4])
    return _attend(None, op, batch, q, q, min(len_hi, rng.choice([q, 32, len_hi])), len_hi, hq,
                   hkv, dim, page, window, sink, spread)


def _lengths(case):
    """(new tokens, cached tokens) of every sequence; from the case alone."""
    rng = random.Random(case["spread"])
    n = [_log_int(rng, case["q_lo"], case["q_hi"]) for _ in range(case["batch"])]
    lens = [max(k, _log_int(rng, case["len_lo"], case["len_hi"])) for k in n]
    n[0] = case["q_hi"]
    lens[0] = max(n[0], case["len_hi"])
    return n, lens


# --------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------

def _normal(shape, gen):
    return torch.randn(shape, generator=gen, device=_DEV, dtype=torch.float32).to(torch.bfloat16)


def _quantise(x):
    """Codes (0..15) and scales of x [..., D] in fp32."""
    g = x.float().reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    hi, lo = g.amax(-1), g.amin(-1)
    e = torch.where(-lo >= hi, lo, hi) * -0.125
    bits = e.view(torch.int32)
    s = ((bits + _EPS_SCALE_BITS) & ~_EPS_SCALE_BITS).view(torch.float32)
    c = torch.where(s.unsqueeze(-1) == 0, torch.zeros_like(g), g / s.unsqueeze(-1))
    c = torch.round(c).clamp(-8, 7) + 8
    return c.reshape(x.shape).to(torch.uint8), s.to(torch.bfloat16)


def _pack(c, kind):
    """Codes [..., D] to the bytes [..., D/2] of a K or V head row."""
    D = c.shape[-1]
    lead = c.shape[:-1]
    b = c[..., 0::2] | (c[..., 1::2] << 4)                       # element order
    if kind == "k":
        return b.reshape(*lead, D // 32, 4, 4).transpose(-3, -2).reshape(*lead, D // 2)
    return b.reshape(*lead, D // 32, 8, 2).transpose(-3, -2).reshape(*lead, D // 2)


def _unpack(b, s, kind, dtype=torch.float32):
    """Bytes [..., D/2] and scales [..., D/32] to the values they stand for."""
    lead, half = b.shape[:-1], b.shape[-1]
    G = half // 16
    if kind == "k":
        b = b.reshape(*lead, 4, G, 4).transpose(-3, -2).reshape(*lead, half)
    else:
        b = b.reshape(*lead, 8, G, 2).transpose(-3, -2).reshape(*lead, half)
    c = torch.stack([b & 15, b >> 4], dim=-1).reshape(*lead, G, 32).to(dtype) - 8
    return (c * s.to(dtype).unsqueeze(-1)).reshape(*lead, 2 * half)


def _q4_planes(n_pages, hkv, page, dim, gen):
    """A 4-bit cache [pages, page, heads, .] stored head by head within a page."""
    planes = []
    for kind in ("k", "v"):
        codes = torch.empty((n_pages, hkv, page, dim // 2), dtype=torch.uint8, device=_DEV)
        scales = torch.empty((n_pages, hkv, page, dim // 32), dtype=torch.bfloat16, device=_DEV)
        step = max(1, (1 << 25) // (hkv * page * dim))
        for p in range(0, n_pages, step):
            x = _normal((min(step, n_pages - p), hkv, page, dim), gen)
            c, s = _quantise(x)
            codes[p:p + step] = _pack(c, kind)
            scales[p:p + step] = s
        planes += [codes.transpose(1, 2), scales.transpose(1, 2)]
    return planes


def prepare(case, seed):
    gen = torch.Generator(device=_DEV).manual_seed(seed)
    st = {"case": case}
    if case["op"] == "store_q4":
        T, H, D, page = case["tokens"], case["hkv"], case["dim"], case["page"]
        n_pages = (T + page - 1) // page + 1
        st["k"] = _normal((T, H, D), gen)
        st["v"] = _normal((T, H, D), gen)
        st["planes"] = _q4_planes(n_pages, H, page, D, gen)
        st["rows"] = torch.randperm(n_pages * page, generator=gen, device=_DEV)[:T].contiguous()
        st["all"] = torch.arange(n_pages * page, device=_DEV)
        st["k_out"] = torch.empty((n_pages * page, H, D), dtype=torch.bfloat16, device=_DEV)
        st["v_out"] = torch.empty_like(st["k_out"])
        if own:
            import mrope_qk_norm_b200 as qkr
            st["cache"] = qkr.cache_desc_q4(*st["planes"])
        return st
    n, lens = _lengths(case)
    B, page, D, hq, hkv = case["batch"], case["page"], case["dim"], case["hq"], case["hkv"]
    pages = [(m + page - 1) // page for m in lens]
    n_pages = sum(pages) + 3
    perm = torch.randperm(n_pages, generator=gen, device=_DEV).to(torch.int32)
    table = torch.zeros((B, max(pages)), dtype=torch.int32, device=_DEV)
    at = 0
    for b, m in enumerate(pages):
        table[b, :m] = perm[at:at + m]
        at += m
    T = sum(n)
    cu = [0]
    for k in n:
        cu.append(cu[-1] + k)
    st.update(n=n, lens_host=lens, table=table, max_q=max(n), max_len=max(lens),
              lens=torch.tensor(lens, dtype=torch.int32, device=_DEV),
              cu=torch.tensor(cu, dtype=torch.int32, device=_DEV),
              q=_normal((T, hq, D), gen),
              out=torch.empty((T, hq, D), dtype=torch.bfloat16, device=_DEV))
    if case["op"] == "attend":
        st["planes"] = [_normal((n_pages, page, hkv, D), gen) for _ in range(2)]
    else:
        st["planes"] = _q4_planes(n_pages, hkv, page, D, gen)
    if own:
        import mrope_qk_norm_b200 as qkr
        make = qkr.cache_desc if case["op"] == "attend" else qkr.cache_desc_q4
        st["cache"] = make(*st["planes"])
        st["workspace"] = torch.empty(
            qkr.cache_attention_workspace(st["q"], st["cache"], B, st["max_q"], st["max_len"],
                                          window=case["window"], n_sink=case["sink"]),
            dtype=torch.uint8, device=_DEV)
    return st


# --------------------------------------------------------------------------
# One pass
# --------------------------------------------------------------------------

def run(state):
    case = state["case"]
    if own:
        import mrope_qk_norm_b200 as qkr
        if case["op"] == "store_q4":
            qkr.cache_set_rows_q4(state["k"], state["v"], state["cache"], state["rows"])
            qkr.cache_get_rows_q4(state["cache"], state["all"], state["k_out"], state["v_out"])
            return {"k": state["k_out"], "v": state["v_out"]}
        qkr.cache_attention(state["q"], state["cache"], state["out"], state["table"],
                            state["lens"], state["cu"], state["max_q"], state["max_len"],
                            window=case["window"], n_sink=case["sink"],
                            workspace=state["workspace"])
        return state["out"]
    if case["op"] == "store_q4":
        return _store_plain(state)
    return _attend_plain(state)


def _store_plain(st):
    page = st["case"]["page"]
    out = {}
    for name, (codes, scales) in (("k", st["planes"][0:2]), ("v", st["planes"][2:4])):
        c, s = _quantise(st[name])
        p, r = st["rows"] // page, st["rows"] % page
        codes[p, r] = _pack(c, name)
        scales[p, r] = s
        v = _unpack(codes, scales, name)
        out[name] = v.reshape(-1, *v.shape[2:]).to(torch.bfloat16)
    return out


def _rows_plain(st, b, idx):
    """K and V rows of the tokens idx of sequence b, in fp32 [tokens, heads, D]."""
    page = st["case"]["page"]
    p, r = st["table"][b][idx // page].long(), idx % page
    if st["case"]["op"] == "attend":
        k, v = st["planes"]
        return k[p, r].float(), v[p, r].float()
    kc, ks, vc, vs = st["planes"]
    return _unpack(kc[p, r], ks[p, r], "k"), _unpack(vc[p, r], vs[p, r], "v")


def _attend_plain(st):
    case = st["case"]
    D, hq, hkv = case["dim"], case["hq"], case["hkv"]
    G, window, sink = hq // hkv, case["window"], case["sink"]
    at = 0
    for b, (n, L) in enumerate(zip(st["n"], st["lens_host"])):
        for i0 in range(0, n, 512):
            i1 = min(n, i0 + 512)
            first, last = L - n + i0, L - n + i1 - 1
            lo = max(0, first - window + 1) if window else 0
            idx = torch.arange(lo, last + 1, device=_DEV)
            if min(sink, lo) > 0:
                idx = torch.cat([torch.arange(min(sink, lo), device=_DEV), idx])
            k, v = _rows_plain(st, b, idx)
            q = st["q"][at + i0:at + i1].float().reshape(i1 - i0, hkv, G, D)
            q = q.permute(1, 2, 0, 3).reshape(hkv, G * (i1 - i0), D)
            s = torch.matmul(q, k.permute(1, 2, 0)) * (1.0 / math.sqrt(D))
            pos = torch.arange(first, last + 1, device=_DEV).unsqueeze(1)
            see = idx <= pos
            if window:
                see = see & ((pos - idx < window) | (idx < sink))
            s = s.reshape(hkv, G, i1 - i0, -1).masked_fill(~see, float("-inf"))
            s = torch.exp(s - s.amax(-1, keepdim=True))
            s = s / s.sum(-1, keepdim=True)
            o = torch.matmul(s.reshape(hkv, G * (i1 - i0), -1), v.permute(1, 0, 2))
            o = o.reshape(hkv, G, i1 - i0, D).permute(2, 0, 1, 3).reshape(i1 - i0, hq, D)
            st["out"][at + i0:at + i1] = o.to(torch.bfloat16)
        at += n
    return st["out"]


# --------------------------------------------------------------------------
# Work and the exact results
# --------------------------------------------------------------------------

def work(case):
    if case["op"] == "store_q4":
        T, H, D, page = case["tokens"], case["hkv"], case["dim"], case["page"]
        R = ((T + page - 1) // page + 1) * page
        row = H * (D // 2 + D // 16)
        # rows in, their 4-bit rows out; then every 4-bit row in and its values out
        return {"bytes": 2 * (T * (2 * H * D + row) + R * (row + 2 * H * D)) + 8 * (T + R),
                "flops": 4 * (T + R) * H * D}
    n, lens = _lengths(case)
    D, hq, hkv = case["dim"], case["hq"], case["hkv"]
    row = 2 * D if case["op"] == "attend" else D // 2 + D // 16
    window, sink = case["window"], case["sink"]
    bytes_, pairs = 0, 0
    for k, L in zip(n, lens):
        lo = max(0, L - k - window + 1) if window else 0
        bytes_ += 2 * hkv * row * (L - lo + min(sink, lo)) + 4 * k * hq * D
        for p in range(L - k, L):
            if not window or p < window:
                pairs += p + 1
            else:
                pairs += window + min(sink, p - window + 1)
    return {"bytes": bytes_, "flops": 4 * D * hq * pairs}


def exact(case, seed):
    st = prepare(case, seed)
    page = case["page"]
    if case["op"] == "store_q4":
        out = {}
        for name, (codes, scales) in (("k", st["planes"][0:2]), ("v", st["planes"][2:4])):
            flat = _unpack(codes, scales, name, torch.float64).reshape(-1, case["hkv"], case["dim"])
            x = st[name].double()
            g = x.reshape(*x.shape[:-1], -1, 32)
            big = g.abs().amax(-1, keepdim=True)
            sign = torch.where((g == -big).any(-1, keepdim=True), 1.0, -1.0)
            mant, expo = torch.frexp(big / 8)
            s = sign * torch.ldexp(torch.ceil(mant * 32) / 32, expo)
            c = torch.clamp(torch.round(torch.where(s == 0, 0.0, g / s)), -8, 7)
            flat[st["rows"]] = (c * s).reshape(x.shape)
            out[name] = flat
        return out
    D, G = case["dim"], case["hq"] // case["hkv"]
    res = torch.empty((sum(st["n"]), case["hq"], D), dtype=torch.float64, device=_DEV)
    row = 0
    for b in range(case["batch"]):
        n, L = st["n"][b], st["lens_host"][b]
        j = torch.arange(L, device=_DEV)
        rows = (st["table"][b].long()[j // page], j % page)
        if case["op"] == "attend":
            k, v = (x[rows].double() for x in st["planes"])
        else:
            k = _unpack(st["planes"][0][rows], st["planes"][1][rows], "k", torch.float64)
            v = _unpack(st["planes"][2][rows], st["planes"][3][rows], "v", torch.float64)
        for i in range(0, n, 256):
            pos = torch.arange(L - n + i, L - n + min(n, i + 256), device=_DEV)[:, None]
            hidden = j[None] > pos
            if case["window"]:
                hidden |= (j[None] <= pos - case["window"]) & (j[None] >= case["sink"])
            for h in range(case["hq"]):
                z = st["q"][row + i:row + i + 256][:pos.shape[0], h].double() @ k[:, h // G].T
                z = (z / math.sqrt(D)).masked_fill_(hidden, float("-inf"))
                w = torch.exp(z - torch.logsumexp(z, 1, keepdim=True))
                res[row + i:row + i + pos.shape[0], h] = w @ v[:, h // G]
        row += n
    return res
