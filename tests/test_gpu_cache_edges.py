"""The cache operators at the edges of what include/qkr.h allows."""
import ctypes
import math
import random

import pytest
import torch

import mrope_qk_norm_b200 as qkr
from tests._cache_util import Batch, pack, values64

pytestmark = pytest.mark.gpu

FORMATS = ["bf16", "q4"]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("D", [64, 128])
def test_blocks_that_see_nothing(fmt, D):
    """More new tokens than the cache holds, over many 256-row blocks: every row
    before the cache's first token is zero, however often the call is made."""
    b = Batch(n=[3000, 1200, 40], lens=[3, 0, 700], hq=6, hkv=2, D=D, page=16, fmt=fmt, seed=31)
    for _ in range(20):
        b.out_buf.fill_(7.0)
        b.lse.fill_(7.0)
        b.call()
        torch.cuda.synchronize()
        assert (b.out[:2997] == 0).all() and (b.out[3000:4200] == 0).all()
        assert (b.lse[:2997] == -float("inf")).all() and (b.lse[3000:4200] == -float("inf")).all()
    b.check()


def test_most_tiles_a_batch_can_have():
    """70 sequences of the longest length in tiles of 16 keys, more than 2^31 tiles.
    Each sequence's page table names one page throughout, every query is zero and a
    page's values are one power of two a dim, so all sums are exact."""
    B, D, page, L = 70, 8, 65520, 1 << 29
    k = torch.randn((B, page, 1, D), device="cuda").to(torch.bfloat16)
    want = torch.pow(2.0, ((torch.arange(B)[:, None] + torch.arange(D)) % 9 - 4).float())
    want = (want * (1 - 2 * (torch.arange(B) % 2))[:, None]).to(torch.bfloat16).cuda()
    v = want[:, None, None].expand(B, page, 1, D).contiguous()
    cache = qkr.cache_desc(k, v)
    table = torch.arange(B, dtype=torch.int32, device="cuda")[:, None].repeat(1, -(-L // page))
    q = torch.zeros((B, 1, D), dtype=torch.bfloat16, device="cuda")
    out = torch.full_like(q, 7.0)
    lse = torch.full((B, 1), 7.0, device="cuda")
    lens = torch.full((B,), L, dtype=torch.int32, device="cuda")
    cu = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    ws = torch.empty(qkr.cache_attention_workspace(q, cache, B, 1, L), dtype=torch.uint8,
                     device="cuda")
    qkr.cache_attention(q, cache, out, table, lens, cu, 1, L, lse=lse, workspace=ws)
    torch.cuda.synchronize()
    assert torch.equal(out[:, 0], want)
    # a sum of 2^29 ones: ln(2^29) to fp32's accuracy
    assert (lse.double() - 29 * 0.6931471805599453).abs().max() < 20.2 * 2.0 ** -22
    assert qkr.device_status(reset=True) == 0


@pytest.mark.parametrize("order", ["nhd", "hnd"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("n,lens", [([1], [2500]), ([1] * 3, [9000, 5000, 3000])])
def test_pages_outside_the_cache_among_others(order, D, page, n, lens):
    """4-bit rows: every second or third page reads as zeros, so that stages of the
    ring are zeroed and copied into by turns."""
    b = Batch(n=n, lens=lens, hq=4, hkv=2, D=D, page=page, fmt="q4", order=order, seed=32,
              poison=False)
    b.k64 = torch.cat([b.k64, torch.zeros_like(b.k64[:1])])
    b.v64 = torch.cat([b.v64, torch.zeros_like(b.v64[:1])])
    assert qkr.device_status(reset=True) == 0
    b.table[:, ::2] = 2 ** 30       # the definition clamps it to the page of zeros
    b.table[:, 1::3] = 2 ** 30
    for _ in range(3):
        b.out_buf.fill_(7.0)
        b.lse.fill_(7.0)
        b.call()
        torch.cuda.synchronize()
        b.check()
    assert qkr.device_status(reset=True) == 8


def test_long_piece_key_by_key():
    """An infinite value that only the last token of a sequence sees sends a CTA's whole
    piece, some 200,000 keys of 16 rows, through the key-by-key path (some 0.4 s).  The
    next sequence's piece of the same CTA comes out as if nothing had happened, and no
    bounded wait runs out."""
    D, page, L, G, n = 64, 64, 1 << 25, 8, 2
    P = 512                                     # pages in turn, L / (64 P) times over
    g = torch.Generator().manual_seed(33)
    v = torch.randint(-8, 25, (P + 2, page, 1, D), generator=g).to(torch.bfloat16)
    v[P] = v[P - 1]                             # the sequences' last pages, of their own
    v[P + 1] = v[P - 1]
    v[P, page - 1, 0, 3] = float("inf")
    k = torch.randn((P + 2, page, 1, D), generator=g).to(torch.bfloat16)
    cache = qkr.cache_desc(k.cuda(), v.cuda())
    table = (torch.arange(L // page) % P).to(torch.int32).repeat(2, 1)
    table[0, -1], table[1, -1] = P, P + 1
    # zero queries: every weight is one, and the sums are exact but for the joins
    q = torch.zeros((2 * n, G, D), dtype=torch.bfloat16, device="cuda")
    out = torch.full_like(q, 7.0)
    lens = torch.full((2,), L, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, n, 2 * n], dtype=torch.int32, device="cuda")
    ws = torch.empty(qkr.cache_attention_workspace(q, cache, 2, n, L), dtype=torch.uint8,
                     device="cuda")
    assert qkr.device_status(reset=True) == 0
    qkr.cache_attention(q, cache, out, table.cuda(), lens, cu, n, L, workspace=ws)
    torch.cuda.synchronize()
    assert qkr.device_status(reset=True) == 0
    # the CTA in question ends the first sequence and begins the second
    ctas, cost = qkr.last_launch()["grid"], L // 64 + 2
    quota = -(-2 * cost // ctas)
    assert cost % quota > quota // 2 and quota - cost % quota > 16
    total = v[:P].double().sum((0, 1))[0] * (L // (64 * P))
    last = v[P - 1, page - 1, 0].double()
    # half a step of bf16, and a rounding of fp32 for each of at most `ctas` parts joined
    rel = 2.0 ** -8 + 2 * ctas * 2.0 ** -24
    for s in range(2):
        for i in range(n):
            want = (total if i else total - last) / (L - n + 1 + i)
            got = out[s * n + i].double().cpu()
            if s == 0 and i == 1:
                assert torch.isposinf(got[:, 3]).all()
                got[:, 3] = want[3]
            # the numerators' parts are as large as the sum of magnitudes
            size = v[:P].double().abs().mean((0, 1))[0]
            assert ((got - want).abs() <= want.abs() * 2.0 ** -8 + size * (rel - 2.0 ** -8)).all()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("what", ["past", "wholly_past", "negative", "decreasing", "long_empty",
                                  "negative_empty"])
@pytest.mark.parametrize("kernel", ["cluster", "shares", "tiles", "mixed"])
def test_metadata_that_leaves_no_rows_is_reported(kernel, what, fmt):
    """Offsets and lengths outside their bounds raise bit 8 also where clamping leaves
    the sequence no tokens; the others are as they should be."""
    n = [0] + {"cluster": [1, 1], "shares": [1, 2], "tiles": [70, 3], "mixed": [1, 70]}[kernel] + [0, 0]
    lens = [5] + ([9000, 300] if kernel == "shares" else [300, 200]) + [7, 0]
    b = Batch(n=n, lens=lens, hq=24 if kernel == "tiles" else 4, hkv=1, D=64, page=16, fmt=fmt,
              seed=34, poison=False, pad=0)
    most, longest = max(n), max(lens)

    def check():
        b.out_buf.fill_(7.0)
        b.lse.fill_(7.0)
        b.call(max_q=most, max_len=longest)
        torch.cuda.synchronize()
        b.check()
        assert qkr.last_launch()["kernel_name"] == ("attn_tiles" if kernel in ("tiles", "mixed")
                                                    else "attn_rows")
    assert qkr.device_status(reset=True) == 0
    check()
    assert qkr.device_status(reset=True) == 0
    if what == "past":              # a last sequence that begins at T
        b.cu[5] = b.T + 3
    elif what == "wholly_past":
        b.cu[4:] = torch.tensor([b.T + 1, b.T + 3])
    elif what == "negative":        # before the first row
        b.cu[0] = -1
    elif what == "decreasing":
        b.cu[5] = b.T - 1
    elif what == "long_empty":      # no new tokens, and a length past max_len
        b.lens[0] = longest + 1
    else:
        b.lens[4] = -1
    check()
    assert qkr.device_status(reset=True) == 8



@pytest.mark.parametrize("fmt", FORMATS)
def test_a_single_token_may_have_any_token_stride(fmt):
    """The token stride of one token is never used: a row of any wider buffer will do."""
    b = Batch(n=[1], lens=[200], hq=4, hkv=2, D=64, page=16, fmt=fmt, seed=36, pad=0)
    q = torch.zeros(4 * 64 + 3, dtype=torch.bfloat16, device="cuda").as_strided((1, 4, 64), (259, 64, 1))
    q.copy_(b.q)
    assert q.stride(0) % 8
    b.q = q
    b.call()
    torch.cuda.synchronize()
    b.check()



@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("n", [1, 50])
def test_queries_and_result_in_one_buffer(fmt, n):
    """q and out as column windows of one packed buffer share no element."""
    b = Batch(n=[n, 1], lens=[300, 40], hq=4, hkv=2, D=64, page=16, fmt=fmt, seed=37)
    buf = torch.full((b.T, 2 * 4 + 1, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    buf[:, 5:] = b.q
    b.q, b.out = buf[:, 5:], buf[:, :4]
    b.call()
    torch.cuda.synchronize()
    b.check()
    with pytest.raises(qkr.QkrError):
        b.out = buf[:, 2:6]
        b.call()



@pytest.mark.parametrize("D", [64, 128])
def test_rows_come_back_into_one_buffer(D):
    """k_out and v_out as column windows of one packed buffer share no element."""
    T, H, page = 33, 3, 16
    x = torch.randn((2, T, H, D), device="cuda").to(torch.bfloat16)
    planes = [torch.empty((4, page, H, w), dtype=t, device="cuda")
              for w, t in ((D // 2, torch.uint8), (D // 32, torch.bfloat16)) * 2]
    cache = qkr.cache_desc_q4(*planes)
    rows = torch.randperm(4 * page)[:T].cuda()
    qkr.cache_set_rows_q4(x[0], x[1], cache, rows)
    buf = torch.full((T, 2 * H + 1, D), 7.0, dtype=torch.bfloat16, device="cuda")
    qkr.cache_get_rows_q4(cache, rows, buf[:, :H], buf[:, H + 1:])
    assert torch.equal(buf[:, :H].double(), values64(x[0]))
    assert torch.equal(buf[:, H + 1:].double(), values64(x[1]))
    assert (buf[:, H] == 7).all()
    with pytest.raises(qkr.QkrError):
        qkr.cache_get_rows_q4(cache, rows, buf[:, :H], buf[:, 1:H + 1])



@pytest.mark.parametrize("fmt", FORMATS)
def test_last_launch_of_a_mixed_call(fmt):
    """What is recorded is the tiles launch's own, and all launches are counted."""
    b = Batch(n=[1, 90, 2], lens=[40, 300, 50], hq=4, hkv=2, D=64, page=16, fmt=fmt, seed=35)
    b.call()
    torch.cuda.synchronize()
    info = qkr.last_launch()
    assert info["kernel_name"] == "attn_tiles" and info["launches"] >= 2
    assert info["cluster"] == 1



@pytest.mark.parametrize("fmt", FORMATS)
def test_even_shares_cut_a_long_sequence(fmt):
    """The shares computed from the lengths: the long sequence's keys lie in many CTAs."""
    b = Batch(n=[1, 1], lens=[9000, 33], hq=8, hkv=1, D=128, page=64, fmt=fmt, seed=39)
    b.call()
    torch.cuda.synchronize()
    info = qkr.last_launch()
    ctas, tile, piece = info["stages"], 64, (128 if fmt == "bf16" else 512) // 64
    work = sum(piece + -(-m // tile) for m in b.L)
    quota = max(-(-work // ctas), 128 // tile)
    assert info["launches"] == 2 and -(-9000 // tile) > 2 * quota
    b.check()



def test_scales_below_the_normal_numbers():
    """Groups whose scale is subnormal: rounded up to a multiple of 2^-130, bit for bit.
    Every positive and negative extreme below 2^-121, beside other elements of the group."""
    D, page = 128, 64
    top = torch.arange(1, 0x0300, dtype=torch.int16)      # 2^-133 .. 2^-121
    x = torch.zeros((2 * len(top), 32), dtype=torch.int16)
    x[:, 0] = torch.cat([top, top | -0x8000])
    g = torch.Generator().manual_seed(38)
    for i in range(1, 32):          # magnitudes up to the extreme's, either sign
        part = (x[:, 0] & 0x7fff).float() * torch.rand(len(x), generator=g)
        sign = torch.randint(0, 2, (len(x),), generator=g).to(torch.int16) * -0x8000
        x[:, i] = part.to(torch.int16) | sign
    x = torch.cat([x, torch.zeros((-len(x) % 4, 32), dtype=torch.int16)])
    k = x.view(torch.bfloat16).view(-1, 1, D).cuda()
    T = len(k)
    planes = [torch.empty((-(-T // page), page, 1, w), dtype=t, device="cuda")
              for w, t in ((D // 2, torch.uint8), (D // 32, torch.bfloat16)) * 2]
    cache = qkr.cache_desc_q4(*planes)
    rows = torch.arange(T, device="cuda")
    qkr.cache_set_rows_q4(k, k, cache, rows)
    # the definition, with the grid of the subnormal scales
    y = k.cpu().double().view(T, 1, 4, 32)
    big = y.abs().amax(-1, keepdim=True)
    mant, expo = torch.frexp(big / 8)
    s = torch.ldexp(torch.ceil(mant * 32) / 32, expo)
    s = torch.where(big / 8 < 2.0 ** -126, torch.ceil(big / 8 * 2.0 ** 130) * 2.0 ** -130, s)
    s = torch.where((y == -big).any(-1, keepdim=True), s, -s)
    c = torch.round(torch.where(s == 0, 0.0, y / torch.where(s == 0, 1.0, s))).clamp(-8, 7)
    codes = (c + 8).to(torch.uint8).view(T, 1, D).cuda()
    want = (c * s).view(T, 1, D)
    assert torch.equal(planes[0].view(-1, 1, D // 2)[:T], pack(codes, False))
    assert torch.equal(planes[2].view(-1, 1, D // 2)[:T], pack(codes, True))
    for i in (1, 3):
        assert torch.equal(planes[i].view(-1, 1, 4)[:T].double().cpu(), s.squeeze(-1))
    ko, vo = torch.empty_like(k), torch.empty_like(k)
    qkr.cache_get_rows_q4(cache, rows, ko, vo)
    assert torch.equal(ko.double().cpu(), want) and torch.equal(vo.double().cpu(), want)


def _scaled(b, i, f):
    """Multiplies the K (0) or V (1) rows of a batch by a power of two."""
    pl = b.planes[i if b.fmt == "bf16" else 2 * i + 1]
    pl.copy_((pl.double() * f).to(torch.bfloat16))
    if i:
        b.v64 *= f
    else:
        b.k64 *= f


@pytest.mark.parametrize("fmt", FORMATS)
def test_a_scale_of_zero_takes_the_mean_of_any_scores(fmt):
    """Scores of some 2^125 times zero are zero."""
    b = Batch(n=[1, 40], lens=[300, 100], hq=4, hkv=2, D=64, page=16, fmt=fmt, seed=40,
              poison=False)
    _scaled(b, 0, 2.0 ** 60)
    b.q = b.q * 2.0 ** 60
    b.call(scale=0.0)
    torch.cuda.synchronize()
    b.check(scale=0.0)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("D", [64, 128])
def test_largest_values_and_queries(fmt, D):
    """Values just below 2^120 over the number of keys, queries just below 2^114."""
    b = Batch(n=[1, 40, 5], lens=[250, 100, 200], hq=4, hkv=2, D=D, page=16, fmt=fmt, seed=41,
              poison=False)
    _scaled(b, 1, 2.0 ** 107)                       # a few times that: up to 2^110
    assert 2.0 ** 109 < b.v64.abs().max() < 2.0 ** 110
    b.q = b.q * 2.0 ** 111
    assert 2.0 ** 112 < b.q[:46].abs().max() < 2.0 ** 114
    scale = D ** -0.5 * 2.0 ** -111
    b.call(scale=scale)
    torch.cuda.synchronize()
    b.check(scale=scale)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("hq", [4, 8, 16])
@pytest.mark.parametrize("D", [64, 128])
def test_even_shares_for_resident_ctas(fmt, D, hq):
    """The CTAs that share a batch's keys all fit the SMs at once: by shared memory, 3 or 4
    CTAs of up to 8 rows of 64 dims, 2 or 3 otherwise."""
    b = Batch(n=[1] * 4, lens=[5000, 17, 800, 4000], hq=hq, hkv=1, D=D, page=64, fmt=fmt, seed=42)
    b.call()
    torch.cuda.synchronize()
    info = qkr.last_launch()
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    # the ring (K and V of a stage, and scales) and the four warps' outputs in fp32
    keys, row = (64, 2 * D) if fmt == "bf16" else (128, D // 2 + D // 16)
    stages = 4 if D == 64 else (2 if fmt == "bf16" and hq > 8 else 3)
    rows = 8 if hq <= 8 else 16
    smem = stages * 2 * keys * row + 4 * rows * (D + 4) * 4
    assert info["launches"] == 2 and info["grid"] % sms == 0
    assert info["grid"] // sms * (smem + 1024) <= 228 * 1024
    b.check()


@pytest.mark.parametrize("fmt", FORMATS)
def test_most_sequences_of_a_call(fmt):
    """2^16 sequences, most of one key, some without new tokens."""
    B = 1 << 16
    n = [0 if i % 7 == 3 else 1 for i in range(B)]
    cu = torch.tensor([0] + n).cumsum(0).to(torch.int32)
    T, P, page, D = int(cu[-1]), 64, 16, 64
    g = torch.Generator().manual_seed(43)
    k, v = (torch.randn((P, page, 1, D), generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    if fmt == "bf16":
        cache = qkr.cache_desc(k, v)
    else:
        planes = [torch.empty((P, page, 1, w), dtype=t, device="cuda")
                  for w, t in ((D // 2, torch.uint8), (D // 32, torch.bfloat16)) * 2]
        cache = qkr.cache_desc_q4(*planes)
        every = torch.arange(P * page, device="cuda")
        qkr.cache_set_rows_q4(k.view(-1, 1, D), v.view(-1, 1, D), cache, every)
        qkr.cache_get_rows_q4(cache, every, k.view(-1, 1, D), v.view(-1, 1, D))
    table = torch.randint(0, P, (B, 1), generator=g).to(torch.int32)
    lens = torch.ones(B, dtype=torch.int32)
    lens[100], lens[B - 1] = 16, 9
    q = torch.randn((T, 2, D), generator=g).to(torch.bfloat16).cuda()
    out = torch.full_like(q, 7.0)
    ws = torch.empty(qkr.cache_attention_workspace(q, cache, B, 1, 16), dtype=torch.uint8,
                     device="cuda")
    qkr.cache_attention(q, cache, out, table.cuda(), lens.cuda(), cu.cuda(), 1, 16, workspace=ws)
    seq = torch.arange(B)[torch.tensor(n) > 0]
    # one key: its value row, whatever the query
    want = v[table[seq, 0].long().cuda(), 0].expand(-1, 2, -1).clone()
    one = lens[seq].cuda() == 1
    torch.cuda.synchronize()
    assert torch.equal(out[one], want[one])
    for b in (100, B - 1):
        kk, vv = (x[int(table[b, 0]), :int(lens[b]), 0].double() for x in (k, v))
        t = int(cu[b])
        w = torch.softmax(q[t].double() @ kk.T * D ** -0.5, -1)
        # the weights' rounding and the result's, and 2^-10 for all that is fp32
        assert ((out[t].double() - w @ vv).abs() <= (w @ vv.abs()) * (2 * 2.0 ** -8 + 2.0 ** -10)).all()
    assert qkr.device_status(reset=True) == 0


@pytest.mark.parametrize("n", [1, 2])
@pytest.mark.parametrize("D", [64, 128])
def test_zero_codes_under_a_large_weight(D, n):
    """4-bit rows whose scores let one key have nearly all the weight: where its values
    are zero, its offset leaves little in the fp32 sums.

    A code's products run on 16 + nibble, 31 at most, and on -24; each of a tile's two
    sums rounds (or cuts) to fp32, 2^-23 relative to 31 times its keys' weights times
    scales, so all tiles together are off by 2^-22 * 31 times their weighted mean."""
    lens = [max(n, (37 * i) % 400) for i in range(40)]
    b = Batch(n=[n] * 40, lens=lens, hq=8, hkv=2, D=D, page=32, fmt="q4", seed=44, poison=False,
              pad=0)
    b.call(scale=0.5)
    torch.cuda.synchronize()
    for s, L in enumerate(lens):
        k, v = b.rows64(s)
        for h in range(8):
            for i in range(n):
                q = b.q[s * n + i, h].double()
                see = L - n + i + 1
                kk, vv = k[:see, h // 4], v[:see, h // 4]
                z = 0.5 * (kk @ q)
                w = torch.softmax(z, -1)
                # scores: 31 steps of the scale a product, fp32 sums of D of them
                step = kk.reshape(see, -1, 32).abs().amax(-1) / 7
                mag = (q.abs().reshape(-1, 32).sum(-1) * 31 * step).sum(-1).max() * 0.5
                rel = 2.0 ** -8 + 2 * mag * 2.0 ** -20 + 2 * 2.0 ** -16
                tol = 1.01 * rel * (w @ vv.abs()) + (w @ vv).abs() * 2.0 ** -8
                scales = b.planes[3][b.table[s].long()].flatten(0, 1)[:see, h // 4].double().abs()
                tol = tol + 31 * 2.0 ** -22 * (w @ scales).repeat_interleave(32)
                err = (b.out[s * n + i, h].double() - w @ vv).abs()
                assert (err <= tol).all(), (s, h, i, (err / tol).max().item())


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("n", [[2, 1], [300, 0, 5]])
def test_an_empty_cache_needs_no_page_table(fmt, n):
    """max_len 0: nothing is looked up, every row is zero."""
    b = Batch(n=n, lens=[0] * len(n), hq=4, hkv=2, D=64, page=16, fmt=fmt, seed=45)
    b.table = b.table[:, :0]
    b.call()
    torch.cuda.synchronize()
    b.check()
    assert qkr.device_status(reset=True) == 0


@pytest.mark.parametrize("fmt", FORMATS)
def test_a_captured_mixed_step_serves_any_lengths(fmt):
    """One captured call with both kernels and their joins, replayed for other numbers of
    new tokens and lengths, beside eager calls on another stream."""
    most, longest = [130, 130, 60, 8], [2500, 700, 300, 1000]
    b = Batch(n=most, lens=longest, hq=4, hkv=2, D=64, page=16, fmt=fmt, seed=46, poison=False,
              pad=40)
    other = Batch(n=[1, 70], lens=[900, 300], hq=4, hkv=2, D=128, page=32, fmt=fmt, seed=47)
    ws = b.call(max_q=130)
    side_ws = other.call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.call(max_q=130, max_len=2500, workspace=ws)
    side = torch.cuda.Stream()
    for n, lens in (([1, 1, 1, 1], [2400, 5, 300, 999]), ([0, 130, 0, 2], [7, 131, 0, 2]),
                    (most, longest), ([3, 129, 17, 0], [2500, 700, 17, 0]), ([130, 0, 5, 0], [90, 1, 4, 2])):
        b.n, b.L = n, lens
        b.lens.copy_(torch.tensor(lens, dtype=torch.int32))
        b.cu.copy_(torch.tensor([0] + n).cumsum(0).to(torch.int32))
        b.out_buf.fill_(7.0)
        b.lse.fill_(7.0)
        other.out_buf.fill_(7.0)
        other.lse.fill_(7.0)
        torch.cuda.synchronize()
        for _ in range(3):
            graph.replay()
            other.call(stream=side, workspace=side_ws)
        torch.cuda.synchronize()
        b.check()
        other.check()
    assert qkr.device_status(reset=True) == 0


@pytest.mark.parametrize("seed", range(24))
def test_random_calls(seed):
    """Formats, sizes, head layouts, lengths, windows and host bounds drawn together."""
    rng = random.Random(seed)

    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    for it in range(4):
        fmt = FORMATS[it % 2]
        D = rng.choice([64, 128]) if fmt == "q4" else rng.choice([8, 24, 40, 64, 72, 96, 104, 128])
        hkv, G = rng.choice([1, 1, 2, 3, 5]), rng.choice([1, 2, 3, 4, 5, 7, 8, 11, 16, 17, 33])
        B, page = log_int(1, 12), 16 * rng.choice([1, 1, 2, 3, 4, 5, 8, 9, 16])
        top = rng.choice([1, 5, 200, 400])
        n = [rng.choice([0, 1, log_int(1, top)]) for _ in range(B)]
        n[0] = max(n[0], 1)
        lens = [max(k, rng.choice([k, log_int(1, 3000 if B < 4 else 600)])) for k in n]
        if rng.random() < 0.2:
            lens[-1] = n[-1] // 2       # fewer tokens in the cache than new ones
        window, sink = rng.choice([(0, 0), (log_int(1, 700), rng.choice([0, 1, 4, 17, 600]))])
        b = Batch(n=n, lens=lens, hq=hkv * G, hkv=hkv, D=D, page=page, window=window, sink=sink,
                  fmt=fmt, order=rng.choice(["nhd", "hnd"]), seed=seed, pad=rng.choice([0, 3, 20]),
                  poison=rng.random() < 0.8)
        scale = rng.choice([None, 0.0, -0.1])
        b.call(scale=scale, max_q=max(n) + rng.choice([0, 1, 30]),
               max_len=min(b.table.shape[1] * page, max(max(lens), 1) + rng.choice([0, 1, page])))
        torch.cuda.synchronize()
        b.check(scale=scale)
    assert qkr.device_status(reset=True) == 0


def test_more_blocks_than_a_launch_takes_are_refused():
    c = qkr.CacheDesc(format=qkr.CACHE_BF16, page_size=16, n_pages=1, Hkv=256, D=64)
    n = ctypes.c_int64(-1)

    def need(T, B, max_q):
        return qkr.lib().cache_attention_workspace(ctypes.byref(c), T, 256, B, max_q, 64, 0, 0,
                                                   ctypes.byref(n))
    assert need(1 << 16, 1 << 16, 1) == qkr.QKR_ERR_UNSUPPORTED       # 2^24 blocks of few rows
    assert need(1 << 15, (1 << 15) - 1, 1) == qkr.QKR_OK
    assert need(1 << 20, 1 << 15, 1 << 10) == qkr.QKR_ERR_UNSUPPORTED  # and of many
    assert need(1 << 20, 1 << 14, 1 << 10) == qkr.QKR_OK
