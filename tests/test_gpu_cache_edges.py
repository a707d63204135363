"""The cache operators at the edges of what include/qkr.h allows."""
import pytest
import torch

import mrope_qk_norm_b200 as qkr
from tests._cache_util import Batch

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
