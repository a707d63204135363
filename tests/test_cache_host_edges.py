"""What the cache entry points accept and refuse at the edges, on the host."""
import pytest
import torch

import mrope_qk_norm_b200 as qkr
from tests.test_cache_host import BASE, E, U, _attend, _cache, _message, _rows  # noqa: F401

pytestmark = pytest.mark.skipif(torch.cuda.is_available(),
                                reason="an accepted call would launch on the fake addresses")

OK = qkr.QKR_ERR_CUDA       # past validation: fails only for want of a device


def test_the_token_stride_of_one_token_is_not_used():
    for kw in (dict(qts=0), dict(qts=-3), dict(qts=259), dict(qts=1 << 60), dict(ots=0),
               dict(ots=3), dict(ots=1 << 60)):
        assert _attend(T=1, **kw) == OK, _message()
        assert _attend(T=2, **kw) in (E, U)
