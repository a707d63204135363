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


def test_column_windows_of_one_buffer_do_not_overlap():
    Q, O = BASE + (4 << 30), BASE + (5 << 30)
    row, at = 2 * 256, lambda n: Q + 2 * n          # Hq * D = 256 elements a token
    for qts in (512, 768):
        for off in (256, qts - 256, 256 - qts, qts + 256, -256):
            assert _attend(qts=qts, ots=qts, out=at(off)) == OK, _message()
        for off in (0, 8, 248, -8, qts - 248, qts, -248):
            assert _attend(qts=qts, ots=qts, out=at(off)) == U
        assert _attend(qts=qts, ots=qts + 256, out=at(256)) == U       # other strides
    assert _attend(T=1, out=at(256)) == OK and _attend(T=1, out=at(248)) == U
    assert _attend(out=O, lse=Q + row) == U                             # lse in q
    for off in (128, 256):                          # Hkv * D = 128
        assert _rows(get=True, k=Q, v=at(off), kts=384, vts=384) == OK, _message()
    for off in (0, 120, 264, -120):
        assert _rows(get=True, k=Q, v=at(off), kts=384, vts=384) == U
    assert _rows(get=True, k=Q, v=at(128), kts=384, vts=392) == U


def test_a_scale_beyond_the_range_is_refused():
    """scale * log2(e) has to be a finite fp32 number."""
    for x in (2.0 ** 127, -2.0 ** 127, 2.3e38, 1e-45, 0.0):
        assert _attend(scale=x) == OK, _message()
    for x in (2.4e38, -3.4e38):
        assert _attend(scale=x) == E and "scale" in _message()
