"""Inputs and the 64-bit definition for the cache tests.

The definition (``attend64``) is written from the formulas of include/qkr.h and
knows nothing of tiles, splits or lane layouts; it also returns, per output
element, the error the arithmetic of the kernels may make.
"""
from __future__ import annotations

import torch

import mrope_qk_norm_b200 as qkr

HALF_BF16 = 2.0 ** -8     # bf16: half a step, relative
EXP_REL = 2.0 ** -16      # exponentials and fp32 sums of a row, relative
DOT_REL = 2.0 ** -20      # fp32 accumulation of a dot product, relative to its magnitudes

NAN = float("nan")


def quantise64(x):
    """Codes 0..15 and scales of x [..., D] by the definition, in fp64."""
    g = x.double().reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    big = g.abs().amax(-1, keepdim=True)
    neg = (g == -big).any(-1, keepdim=True)
    mant, expo = torch.frexp(big / 8)
    s = torch.ldexp(torch.ceil(mant * 32) / 32, expo).clamp(max=31 * 2.0 ** 120)
    s = torch.where(neg, s, -s)
    c = torch.where(s == 0, torch.zeros_like(g), torch.round(g / torch.where(s == 0, 1.0, s)))
    c = c.clamp(-8, 7) + 8
    return c.reshape(x.shape).to(torch.uint8), s.squeeze(-1)


def pack(codes, is_v):
    """Codes [..., D] into the row layout, element by element from its formula."""
    D = codes.shape[-1]
    out = torch.zeros((*codes.shape[:-1], D // 2), dtype=torch.uint8, device=codes.device)
    for d in range(D):
        w, r = divmod(d, 32)
        if is_v:
            byte = (r // 4) * (D // 16) + 2 * w + (r % 4) // 2
        else:
            byte = (r // 8) * (D // 8) + 4 * w + (r % 8) // 2
        out[..., byte] |= codes[..., d] << (4 * (d % 2))
    return out


def values64(x):
    """What the 4-bit cache stands for after storing x, in fp64."""
    c, s = quantise64(x)
    g = (c.double() - 8).reshape(*x.shape[:-1], -1, 32) * s.unsqueeze(-1)
    return g.reshape(x.shape)


class Batch:
    """A ragged batch over a paged cache in which everything no token sees is
    NaN, infinity or (page ids) out of range."""

    def __init__(self, n, lens, hq, hkv, D, page, window=0, sink=0, fmt="bf16", order="nhd",
                 seed=0, pad=3, scale_v=1.0, poison=True):
        g = torch.Generator().manual_seed(seed)
        dev = "cuda"
        self.n, self.L, self.D, self.page = list(n), list(lens), D, page
        self.hq, self.hkv, self.window, self.sink, self.fmt = hq, hkv, window, sink, fmt
        B = len(n)
        pages = [(m + page - 1) // page for m in lens]
        P = sum(pages) + 2
        perm = torch.randperm(P, generator=g)
        T = sum(n) + pad
        self.T, self.B = T, B
        cu = [0]
        for k in n:
            cu.append(cu[-1] + k)
        table = torch.full((B, max(1, max(pages)) + 1), 2 ** 30, dtype=torch.int32)
        at = 0
        k = torch.randn((P, page, hkv, D), generator=g).to(torch.bfloat16)
        v = (torch.randn((P, page, hkv, D), generator=g) * scale_v).to(torch.bfloat16)
        seen = torch.zeros((P, page), dtype=torch.bool)
        for b, m in enumerate(pages):
            ids = perm[at:at + m]
            at += m
            lo = max(0, lens[b] - n[b] - window + 1) if window else 0
            for j in range(lens[b] if n[b] else 0):
                if j >= lo or j < sink:
                    table[b, j // page] = ids[j // page]
                    seen[ids[j // page], j % page] = True
        if not poison:
            table = table.clamp(max=P - 1)
        self.seen = seen.to(dev)
        # q as a view of a packed buffer, out with a wide token stride
        buf = torch.randn((T, hq + 2, D), generator=g).to(torch.bfloat16)
        if poison:
            buf[sum(n):] = NAN
        self.q = buf.to(dev)[:, 1:1 + hq]
        self.out_buf = torch.full((T, hq * D + 8), 7.0, dtype=torch.bfloat16, device=dev)
        self.out = self.out_buf[:, :hq * D].view(T, hq, D)
        self.lse = torch.full((T, hq), 7.0, dtype=torch.float32, device=dev)
        self.table, self.cu = table.to(dev), torch.tensor(cu, dtype=torch.int32, device=dev)
        self.lens = torch.tensor(lens, dtype=torch.int32, device=dev)
        k, v = k.to(dev), v.to(dev)
        if fmt == "bf16":
            self.k64, self.v64 = k.double(), v.double()
            if poison:
                k[~self.seen] = NAN
                v[~self.seen] = float("inf")
            self.planes = [self._laid(x, order) for x in (k, v)]
            self.cache = qkr.cache_desc(*self.planes)
        else:
            self.k64, self.v64 = values64(k), values64(v)
            planes = []
            for i, x in enumerate((k, v)):
                c, s = quantise64(x)
                s = s.to(torch.bfloat16)
                if poison:
                    s[~self.seen] = NAN
                planes += [self._laid(pack(c, i == 1), order), self._laid(s, order)]
            self.planes = planes
            self.cache = qkr.cache_desc_q4(*planes)

    @staticmethod
    def _laid(x, order):
        if order == "hnd":   # a head's rows of a page side by side
            return x.transpose(1, 2).contiguous().transpose(1, 2)
        return x.contiguous()

    def call(self, scale=None, max_q=None, max_len=None, lse=True, workspace=None, stream=None):
        mq = max(self.n) if max_q is None else max_q
        ml = max(self.L) if max_len is None else max_len
        need = qkr.cache_attention_workspace(self.q, self.cache, self.B, mq, ml, self.window,
                                             self.sink)
        ws = workspace
        if ws is None:
            # whatever the workspace holds before a call means nothing
            ws = torch.full((need,), 0xff, dtype=torch.uint8, device="cuda")
        qkr.cache_attention(self.q, self.cache, self.out, self.table, self.lens, self.cu, mq, ml,
                            scale=scale, window=self.window, n_sink=self.sink,
                            lse=self.lse if lse else None, workspace=ws, stream=stream)
        return ws

    def rows64(self, b):
        j = torch.arange(self.L[b], device="cuda")
        p = self.table[b].long()[j // self.page].clamp(0, self.k64.shape[0] - 1)
        return self.k64[p, j % self.page], self.v64[p, j % self.page]

    def check(self, scale=None):
        """Every output element against the definition."""
        scale = self.D ** -0.5 if scale is None else scale
        G = self.hq // self.hkv
        row = 0
        worst = 0.0
        for b, (n, L) in enumerate(zip(self.n, self.L)):
            if n == 0:
                continue
            k, v = self.rows64(b) if L else (None, None)
            pos = torch.arange(L - n, L, device="cuda")[:, None]
            j = torch.arange(max(L, 1), device="cuda")[None]
            see = (j <= pos) & (j < L)
            if self.window:
                see &= (pos - j < self.window) | (j < self.sink)
            for h in range(self.hq):
                got = self.out[row:row + n, h].double()
                lse = self.lse[row:row + n, h].double()
                if L == 0:
                    assert (got == 0).all() and (lse == -float("inf")).all()
                    continue
                q = self.q[row:row + n, h].double()
                kk, vv = k[:, h // G], v[:, h // G]
                s = (q @ kk.T) * scale
                # magnitudes the fp32 accumulation runs over; the 4-bit form sums
                # 128 + nibble against an offset, 144 steps of the scale at most
                mag = q.abs() @ kk.abs().T
                if self.fmt != "bf16":
                    step = kk.reshape(L, -1, 32).abs().amax(-1, keepdim=True) / 7
                    mag = q.abs() @ (144 * step).expand(-1, -1, 32).reshape(L, -1).T
                s = s.masked_fill(~see, -float("inf"))
                m = s.amax(-1, keepdim=True)
                none = ~see.any(-1)
                w = torch.exp(s - torch.where(none[:, None], torch.zeros_like(m), m))
                l = w.sum(-1, keepdim=True)
                w = w / torch.where(l == 0, torch.ones_like(l), l)
                ref = w @ vv
                size = w @ vv.abs()
                delta = (mag * abs(scale)).masked_fill(~see, 0).amax(-1, keepdim=True) * DOT_REL
                # a weight: rounded to bf16 once, its score off by delta, its
                # exponential and the normalising sum by EXP_REL each
                tol = size * (HALF_BF16 + 2 * delta + 2 * EXP_REL) * 1.01
                tol = tol + ref.abs() * HALF_BF16 + 2.0 ** -133
                err = (got - ref).abs()
                ok = err <= tol
                assert ok.all(), "seq %d head %d: off by %g, allowed %g (%d of %d)" % (
                    b, h, err[~ok].max().item() if torch.isfinite(err[~ok]).any() else NAN,
                    tol[~ok].min().item(), int((~ok).sum()), ok.numel())
                worst = max(worst, (err / tol).max().item())
                ref_lse = torch.where(none, torch.full_like(m[:, 0], -float("inf")),
                                      (m + torch.log(l))[:, 0])
                assert ((lse == ref_lse) | ((lse - ref_lse).abs() <= delta[:, 0] + 2 * EXP_REL +
                                            ref_lse.abs() * 2.0 ** -22)).all(), "lse"
            row += n
        assert (self.out[row:] == 7).all() and (self.lse[row:] == 7).all(), "rows behind the last"
        assert (self.out_buf[:, self.hq * self.D:] == 7).all(), "between the rows of out"
        return worst
