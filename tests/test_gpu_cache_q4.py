"""cache_set_rows_q4 and cache_get_rows_q4: bit for bit against the 64-bit definition."""
import pytest
import torch

import mrope_qk_norm_b200 as qkr
from tests._cache_util import Batch, pack, quantise64, values64

pytestmark = pytest.mark.gpu


def _planes(P, page, H, D, order="nhd", fill=0x5a):
    def plane(last, dtype):
        shape = (P, page, H, last) if order == "nhd" else (P, H, page, last)
        t = torch.empty(shape, dtype=dtype, device="cuda")
        t.view(torch.uint8).fill_(fill)
        return t if order == "nhd" else t.transpose(1, 2)
    return [plane(D // 2, torch.uint8), plane(D // 32, torch.bfloat16),
            plane(D // 2, torch.uint8), plane(D // 32, torch.bfloat16)]


def _bits(t):
    return t.contiguous().view(torch.int16)


@pytest.mark.parametrize("order", ["nhd", "hnd"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T,H,page", [(1, 1, 16), (7, 3, 48), (130, 8, 64), (1000, 2, 16)])
def test_rows_go_in_and_come_back(T, H, D, page, order):
    g = torch.Generator().manual_seed(T + D)
    P = (T + page - 1) // page + 2
    buf = torch.randn((T, 2 * H + 1, D), generator=g).to(torch.bfloat16).cuda()
    k, v = buf[:, :H], buf[:, H + 1:]          # windows of a packed buffer
    rows = torch.randperm(P * page, generator=g)[:T].cuda()
    planes = _planes(P, page, H, D, order)
    before = [p.clone() for p in planes]
    cache = qkr.cache_desc_q4(*planes)
    qkr.cache_set_rows_q4(k, v, cache, rows)
    ko = torch.full((T, H, D), 7.0, dtype=torch.bfloat16, device="cuda")
    vo = torch.full_like(ko, 7.0)
    qkr.cache_get_rows_q4(cache, rows, ko, vo)
    torch.cuda.synchronize()
    p, r = rows // page, rows % page
    for i, (x, o) in enumerate(((k, ko), (v, vo))):
        c, s = quantise64(x)
        assert torch.equal(planes[2 * i][p, r], pack(c, i == 1))
        assert torch.equal(_bits(planes[2 * i + 1][p, r]), _bits(s.to(torch.bfloat16)))
        assert (o.double() == values64(x)).all()     # exact: every value is a bf16 number
        # nothing clipped at the extreme: off by a step of the group at most
        step = s.abs().unsqueeze(-1)
        err = (values64(x) - x.double()).reshape(T, H, -1, 32).abs()
        assert (err <= step).all()
    named = torch.zeros((P, page), dtype=torch.bool, device="cuda")
    named[p, r] = True
    for a, b in zip(planes, before):
        assert torch.equal(a.contiguous().view(torch.uint8).view(P, page, -1)[~named],
                           b.contiguous().view(torch.uint8).view(P, page, -1)[~named])


def test_ties_zeros_and_extremes():
    """Both signs tie (the negative one sets the scale), quotients half way
    between two codes (to even), groups of zeros, the largest and smallest numbers."""
    D = 64
    x = torch.zeros((12, 1, D))
    x[0, 0, 3], x[0, 0, 9] = 4.0, -4.0
    x[1, 0, 3], x[1, 0, 9] = -4.0, 4.0
    x[2, 0, :16] = torch.arange(16) * 0.5 - 4.0          # steps of half a code
    x[2, 0, 32:48] = torch.arange(16) * -0.5 + 4.0
    x[3] = 3.3895e38
    x[4, 0, ::2] = -3.3895e38
    x[5] = 2.0 ** -126
    x[6, 0, 7] = 2.0 ** -133
    x[7, 0, 0] = 1e-30
    x[8, 0, :32] = torch.linspace(-1, 1, 32)
    x[9] = -0.0
    x[10, 0, 40] = 2.0 ** -128
    x[11, 0, 1], x[11, 0, 2] = 1.0, 0.996
    x = x.to(torch.bfloat16).cuda()
    planes = _planes(1, 16, 1, D)
    cache = qkr.cache_desc_q4(*planes)
    rows = torch.arange(12, device="cuda")
    qkr.cache_set_rows_q4(x, x, cache, rows)
    normal = [i for i in range(12) if i not in (5, 6, 10)]
    c, s = quantise64(x)
    assert torch.equal(planes[0][0, :12][normal], pack(c, False)[normal])
    assert torch.equal(planes[2][0, :12][normal], pack(c, True)[normal])
    ko = torch.empty_like(x)
    vo = torch.empty_like(x)
    qkr.cache_get_rows_q4(cache, rows, ko, vo)
    assert torch.equal(ko, vo)
    assert (ko.double()[normal] == values64(x)[normal]).all()
    # groups whose scale is below the normal numbers: within a step of the
    # 2^-130 grid that fp32's bit arithmetic rounds such a scale to
    err = (ko.double() - x.double()).abs()[[5, 6, 10]]
    assert (err <= x.double().abs()[[5, 6, 10]] / 8 + 2.0 ** -126).all()


def test_every_mantissa_against_every_scale():
    """Each of the 16 scale mantissas with every bf16 mantissa at every exponent
    whose quotient can reach half a code, both signs: all quotients and ties there
    are (up to a common power of two)."""
    D, groups = 128, []
    x = torch.tensor([sign * m * 2.0 ** e for e in range(-12, 1) for m in range(128, 256)
                      for sign in (1.0, -1.0)])
    for mant in range(16, 32):
        for extreme in (-8.0 * mant, 8.0 * mant):
            v = x[(x.abs() <= 8 * mant) & (x != -extreme)]
            pad = (-len(v)) % 31
            v = torch.cat([v, torch.zeros(pad)]).view(-1, 31)
            groups.append(torch.cat([torch.full((len(v), 1), extreme), v], 1))
    g = torch.cat(groups)
    g = torch.cat([g, torch.zeros(-len(g) % (D // 32), 32)])
    T = g.numel() // D
    k = g.view(T, 1, D).to(torch.bfloat16).cuda()
    assert (k.float().cpu().view(-1) == g.view(-1)).all()
    page = 64
    planes = _planes((T + page - 1) // page, page, 1, D)
    cache = qkr.cache_desc_q4(*planes)
    rows = torch.arange(T, device="cuda")
    qkr.cache_set_rows_q4(k, k, cache, rows)
    c, sc = quantise64(k)
    assert torch.equal(planes[0].view(-1, 1, D // 2)[:T], pack(c, False))
    assert torch.equal(planes[2].view(-1, 1, D // 2)[:T], pack(c, True))
    assert torch.equal(_bits(planes[1].view(-1, 1, D // 32)[:T]), _bits(sc.to(torch.bfloat16)))


def test_nonfinite_groups_read_back_as_nan():
    x = torch.ones((3, 2, 128), dtype=torch.bfloat16, device="cuda")
    x[0, 0, 40] = float("inf")
    x[1, 1, 127] = float("nan")
    x[2, 0, 0] = float("-inf")
    planes = _planes(1, 16, 2, 128)
    cache = qkr.cache_desc_q4(*planes)
    rows = torch.tensor([4, 0, 15], device="cuda")
    qkr.cache_set_rows_q4(x, x, cache, rows)
    ko, vo = torch.empty_like(x), torch.empty_like(x)
    qkr.cache_get_rows_q4(cache, rows, ko, vo)
    want = torch.zeros((3, 2, 128), dtype=torch.bool, device="cuda")
    want[0, 0, 32:64] = want[1, 1, 96:] = want[2, 0, :32] = True
    for o in (ko, vo):
        assert torch.equal(torch.isnan(o), want)
        # an extreme of 1 asks for a step of 1/8: it comes back as it was
        assert (o[~want] == 1).all()


def test_rows_outside_are_skipped_and_reported():
    k = torch.randn((4, 2, 64), device="cuda").to(torch.bfloat16)
    planes = _planes(2, 16, 2, 64)
    before = [p.clone() for p in planes]
    cache = qkr.cache_desc_q4(*planes)
    rows = torch.tensor([-1, 32, 5, 1 << 40], device="cuda")
    assert qkr.device_status(reset=True) == 0
    qkr.cache_set_rows_q4(k, k, cache, rows)
    assert qkr.device_status(reset=True) == 4
    for a, b in zip(planes, before):
        same = (a.view(torch.uint8) == b.view(torch.uint8)).view(32, -1).all(-1)
        assert same[[i for i in range(32) if i != 5]].all()
    ko, vo = torch.full_like(k, 7.0), torch.full_like(k, 7.0)
    qkr.cache_get_rows_q4(cache, rows, ko, vo)
    assert qkr.device_status(reset=True) == 4
    assert (ko[[0, 1, 3]] == 0).all() and (ko[2].double() == values64(k[2])).all()
    # the same row twice may be read
    qkr.cache_get_rows_q4(cache, torch.tensor([5, 5, 5, 5], device="cuda"), ko, vo)
    assert torch.equal(ko[0], ko[3]) and (vo[1].double() == values64(k[2])).all()
    # nothing to do
    qkr.cache_set_rows_q4(k[:0], k[:0], cache, rows[:0])
    assert qkr.last_launch()["launches"] == 0


@pytest.mark.parametrize("fmt", ["bf16", "q4"])
def test_prompt_then_decode_steps(fmt):
    """The operators as a server runs them: rotate the new rows of a packed QKV
    buffer, store them, attend; a prompt first, then captured single-token
    steps.  Every step against the definition over the rows as stored."""
    torch.manual_seed(1)
    B, hq, hkv, D, page, steps = 2, 4, 2, 64, 16, 4
    prompt = [70, 33]
    pages = 8
    P = B * pages
    order = torch.randperm(P)
    inv = torch.pow(10000.0, -torch.arange(D // 2, device="cuda", dtype=torch.float32) / (D // 2))
    kc = torch.full((P * page, hkv, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    vc = torch.full_like(kc, float("nan"))
    planes = _planes(P, page, hkv, D, "hnd", fill=0xff)
    cache = qkr.cache_desc(kc.view(P, page, hkv, D), vc.view(P, page, hkv, D)) if fmt == "bf16" \
        else qkr.cache_desc_q4(*planes)
    b = Batch(n=prompt, lens=prompt, hq=hq, hkv=hkv, D=D, page=page, fmt=fmt, pad=0, poison=False)
    b.table = order.view(B, pages).to(torch.int32).cuda()
    b.cache = cache
    table = b.table.long()
    max_len = pages * page

    def step(qkv, pos, rows, b):
        q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        qkr.mrope_apply(q, k, q, k, pos, inv, D)
        if fmt == "bf16":
            qkr.rope_set_rows(k, kc, rows, pos, inv, 0)
            qkr.rope_set_rows(v, vc, rows, pos, inv, 0)
        else:
            qkr.cache_set_rows_q4(k, v, cache, rows)
        b.q = q
        return q

    def look(b, n, lens):
        every = torch.arange(P * page, device="cuda")
        if fmt == "bf16":
            k, v = kc, vc
        else:
            k = torch.empty((P * page, hkv, D), dtype=torch.bfloat16, device="cuda")
            v = torch.empty_like(k)
            qkr.cache_get_rows_q4(cache, every, k, v)
        b.k64 = torch.nan_to_num(k.double()).view(P, page, hkv, D)
        b.v64 = torch.nan_to_num(v.double()).view(P, page, hkv, D)
        b.n, b.L = n, lens
        b.check()

    qkv = torch.randn((sum(prompt), hq + 2 * hkv, D), device="cuda").to(torch.bfloat16)
    pos = torch.cat([torch.arange(n) for n in prompt]).to(torch.int32).cuda()
    seq = torch.cat([torch.full((n,), s) for s, n in enumerate(prompt)]).cuda()
    rows = table[seq, pos.long() // page] * page + pos.long() % page
    step(qkv, pos, rows, b)
    b.call(max_len=max_len)
    torch.cuda.synchronize()
    look(b, prompt, prompt)

    d = Batch(n=[1] * B, lens=[1] * B, hq=hq, hkv=hkv, D=D, page=page, fmt=fmt, pad=0,
              poison=False)
    d.table, d.cache = b.table, cache
    qkv1 = torch.zeros((B, hq + 2 * hkv, D), dtype=torch.bfloat16, device="cuda")
    pos1 = torch.zeros(B, dtype=torch.int32, device="cuda")
    rows1 = torch.arange(B, device="cuda") + P * page     # outside: the warm-up stores nothing
    step(qkv1, pos1, rows1, d)
    ws = d.call(max_len=max_len)
    torch.cuda.synchronize()
    assert qkr.device_status(reset=True) == 4
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(qkv1, pos1, rows1, d)
        qkr.cache_attention(d.q, cache, d.out, d.table, d.lens, d.cu, 1, max_len, lse=d.lse,
                            workspace=ws)
    lens = list(prompt)
    for _ in range(steps):
        lens = [m + 1 for m in lens]
        qkv1.copy_(torch.randn((B, hq + 2 * hkv, D)).to(torch.bfloat16))
        p = torch.tensor([m - 1 for m in lens])
        pos1.copy_(p.to(torch.int32))
        rows1.copy_(table.cpu()[torch.arange(B), p // page] * page + p % page)
        d.lens.copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        look(d, [1] * B, lens)
