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
