"""cache_attention against its definition in 64 bits, bf16 and 4-bit caches.

Every case runs over a cache in which all that no token sees is NaN or infinity
and the page ids of unseen pages are out of range, with rows behind the last
sequence, and compares every element with a bound from the roundings the
kernels make (tests/_cache_util.py).
"""
import math

import pytest
import torch

import mrope_qk_norm_b200 as qkr
from tests._cache_util import Batch

pytestmark = pytest.mark.gpu

FORMATS = ["bf16", "q4"]


def _run(**kw):
    b = Batch(**kw)
    b.call()
    torch.cuda.synchronize()
    b.check()
    return b


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("L", [1, 2, 15, 16, 17, 63, 64, 65, 511, 517, 1500])
def test_one_token_lengths(fmt, L):
    _run(n=[1], lens=[L], hq=4, hkv=2, D=128, page=16, fmt=fmt, seed=L)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("hq,hkv", [(1, 1), (2, 2), (3, 1), (8, 1), (9, 3), (16, 1), (24, 2),
                                    (40, 1)])
def test_head_layouts(fmt, hq, hkv):
    _run(n=[1, 1, 1], lens=[5, 130, 77], hq=hq, hkv=hkv, D=64, page=32, fmt=fmt, seed=hq)


@pytest.mark.parametrize("D", [8, 16, 40, 64, 72, 80, 96, 120, 128])
def test_head_dims(D):
    _run(n=[1, 20], lens=[200, 61], hq=4, hkv=2, D=D, page=48, seed=D)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("order", ["nhd", "hnd"])
@pytest.mark.parametrize("page", [16, 48, 64, 256, 1040])
def test_pages_and_layouts(fmt, order, page):
    _run(n=[1, 2, 33], lens=[300, 47, 450], hq=4, hkv=2, D=128, page=page, fmt=fmt, order=order,
         seed=page)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("window,sink", [(1, 0), (1, 1), (7, 3), (16, 16), (17, 4), (100, 0),
                                         (100, 33), (128, 128), (129, 500), (4000, 4)])
@pytest.mark.parametrize("n", [1, 3, 150])
def test_window_and_sinks(fmt, window, sink, n):
    _run(n=[n, n, 1], lens=[700, n, 333], hq=4, hkv=2, D=64, page=32, window=window, sink=sink,
         fmt=fmt, seed=window + n)


@pytest.mark.parametrize("fmt", FORMATS)
def test_empty_sequences_and_rows(fmt):
    """No new tokens, an empty cache, and more new tokens than the cache holds
    (the first of them see nothing)."""
    _run(n=[0, 3, 0, 5, 1, 0], lens=[40, 0, 0, 2, 9, 7], hq=4, hkv=2, D=64, page=16, fmt=fmt)
    _run(n=[200, 0, 1], lens=[90, 12, 0], hq=6, hkv=2, D=64, page=16, fmt=fmt, window=50, sink=2)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("n", [2, 4, 7, 16, 31, 64, 65, 127, 128, 129, 256, 300])
def test_new_tokens(fmt, n):
    _run(n=[n, 1, n // 2], lens=[n, 200, n // 2 + 333], hq=4, hkv=2, D=128, page=64, fmt=fmt,
         seed=n)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("D", [64, 128])
def test_prompt(fmt, D):
    _run(n=[1100], lens=[1100], hq=4, hkv=2, D=D, page=64, fmt=fmt, seed=3)
    _run(n=[700], lens=[2111], hq=6, hkv=2, D=D, page=128, fmt=fmt, seed=4, window=300, sink=5)


@pytest.mark.parametrize("fmt", FORMATS)
def test_ragged_mixture(fmt):
    """Prompts, chunks, decoding users and empty places in one call."""
    b = _run(n=[1, 300, 0, 1, 17, 2, 129, 1, 1], lens=[900, 300, 50, 1, 517, 2, 700, 65, 1300],
             hq=8, hkv=2, D=128, page=48, fmt=fmt, seed=9)
    b.out_buf.fill_(7.0)
    b.lse.fill_(7.0)
    b.call(max_q=400, max_len=2000 // 48 * 0 + 28 * 48)  # wider host bounds than needed
    torch.cuda.synchronize()
    b.check()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("scale", [0.0, -0.05, 1.0, 0.3])
def test_scales(fmt, scale):
    b = Batch(n=[1, 40], lens=[300, 100], hq=4, hkv=4, D=64, page=16, fmt=fmt, seed=5)
    b.call(scale=scale)
    torch.cuda.synchronize()
    b.check(scale=scale)


@pytest.mark.parametrize("fmt", FORMATS)
def test_growing_maximum(fmt):
    """Scores that rise along the axis move the running maximum again and again."""
    b = Batch(n=[1, 140], lens=[2000, 800], hq=2, hkv=1, D=64, page=16, fmt=fmt, seed=6,
              poison=False)
    for s in range(2):
        j = torch.arange(b.L[s], device="cuda")
        p = b.table[s].long()[j // 16]
        ramp = (1 + j / 100.0).view(-1, 1, 1)
        if fmt == "bf16":
            k = (b.k64[p, j % 16] * ramp).to(torch.bfloat16)
            b.planes[0][p, j % 16] = k
            b.k64[p, j % 16] = k.double()
        else:
            r = torch.pow(2.0, torch.floor(torch.log2(ramp)))
            b.planes[1][p, j % 16] = (b.planes[1][p, j % 16].double() * r).to(torch.bfloat16)
            b.k64[p, j % 16] *= r
    b.call()
    torch.cuda.synchronize()
    b.check()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("n", [4, 200])
def test_nonfinite_value_in_a_key_only_later_tokens_see(fmt, n):
    """An infinite or NaN value row reaches the tokens that see it and no other,
    though they share its tile."""
    b = Batch(n=[n], lens=[n + 30], hq=4, hkv=2, D=64, page=16, fmt=fmt, seed=8, poison=False)
    j = n + 30 - 2          # seen by the last two tokens only
    p = int(b.table[0, j // 16])
    if fmt == "bf16":
        b.planes[1][p, j % 16, 0, 5] = float("inf")
    else:
        b.planes[3][p, j % 16, 0, 1] = float("nan")
    b.call()
    torch.cuda.synchronize()
    out = b.out[:n].clone()
    bad = ~torch.isfinite(out)
    # KV head 0 serves query heads 0 and 1
    want = torch.zeros_like(bad)
    if fmt == "bf16":
        want[n - 2:, :2, 5] = True
    else:
        want[n - 2:, :2, 32:] = True
    assert torch.equal(bad, want)
    b.out[:n][want] = 0
    ref = Batch(n=[n], lens=[n + 30], hq=4, hkv=2, D=64, page=16, fmt=fmt, seed=8, poison=False)
    ref.call()
    torch.cuda.synchronize()
    good = ~want
    tol = 2 ** -7 * ref.out[:n][good].double().abs() + 2 ** -6
    assert ((out[good].double() - ref.out[:n][good].double()).abs() <= tol).all()


@pytest.mark.parametrize("fmt", FORMATS)
def test_split_axis_equals_itself_and_is_deterministic(fmt):
    b = Batch(n=[1, 1], lens=[9000, 33], hq=8, hkv=1, D=128, page=64, fmt=fmt, seed=10)
    b.call()
    torch.cuda.synchronize()
    assert qkr.last_launch()["stages"] > 1
    first, lse = b.out.clone(), b.lse.clone()
    b.check()
    for _ in range(3):
        b.out_buf.fill_(7.0)
        b.call()
        torch.cuda.synchronize()
        assert torch.equal(first.view(torch.int16), b.out.view(torch.int16))
        assert torch.equal(lse, b.lse)


@pytest.mark.parametrize("fmt", FORMATS)
def test_many_sequences(fmt):
    n = [(7 * i) % 3 for i in range(150)]
    lens = [max(1, (37 * i) % 200) for i in range(150)]
    n[0] = 2
    _run(n=n, lens=lens, hq=4, hkv=2, D=64, page=16, fmt=fmt, window=60, sink=2)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("order", ["nhd", "hnd"])
@pytest.mark.parametrize("n,lens", [(1, 300), (2, 9000), (60, 300)])
@pytest.mark.parametrize("bad", [-1, -2, -3, 2 ** 31 - 1, -2 ** 31])
def test_any_page_id_outside_reads_as_zeros(fmt, order, n, lens, bad):
    """Negative ids and ids past the last page, in every kernel and scale layout."""
    b = Batch(n=[n], lens=[lens], hq=4, hkv=2, D=64, page=16, fmt=fmt, order=order, seed=20,
              poison=False)
    b.k64 = torch.cat([b.k64, torch.zeros_like(b.k64[:1])])
    b.v64 = torch.cat([b.v64, torch.zeros_like(b.v64[:1])])
    where = [0, 3, 7, (lens - 1) // 16]
    assert qkr.device_status(reset=True) == 0
    b.table[0, where] = bad
    b.call()
    torch.cuda.synchronize()
    assert qkr.device_status(reset=True) == 8
    b.table[0, where] = 2 ** 30     # the definition clamps it to the page of zeros
    b.check()


@pytest.mark.parametrize("fmt", FORMATS)
def test_bad_metadata_is_clamped_and_reported(fmt):
    """Lengths, offsets and page ids outside their bounds: no access outside the
    buffers, the other sequences as they should be, bit 8 of the status word."""
    b = Batch(n=[1, 1, 1], lens=[100, 100, 100], hq=4, hkv=2, D=64, page=16, fmt=fmt, seed=11)
    assert qkr.device_status(reset=True) == 0
    b.call()
    torch.cuda.synchronize()
    good = b.out[0].clone()
    assert qkr.device_status(reset=True) == 0
    b.table[1, 2] = 10 ** 9
    b.table[1, 3] = -5
    b.lens[2] = 10 ** 6
    b.call(max_len=100)
    torch.cuda.synchronize()
    assert qkr.device_status(reset=True) & 8
    assert torch.equal(b.out[0], good)
    # a page outside the cache reads as rows of zeros
    b.k64 = torch.cat([b.k64, torch.zeros_like(b.k64[:1])])
    b.v64 = torch.cat([b.v64, torch.zeros_like(b.v64[:1])])
    b.table[1, 2:4] = 10 ** 9       # the definition clamps it to the row of zeros
    b.lens[2] = 100
    b.call()
    torch.cuda.synchronize()
    assert qkr.device_status(reset=True) & 8
    b.check()
    b.cu[3] = 10 ** 9
    b.cu[1] = -7
    b.call()
    torch.cuda.synchronize()
    assert qkr.device_status(reset=True) & 8


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("layout", ["padded", "one_tensor", "heads_outermost"])
def test_strides(fmt, layout):
    """Rows, heads and pages padded by odd multiples of the alignment; K and V in
    one tensor; a plane a head."""
    b = Batch(n=[1, 70, 3], lens=[200, 150, 90], hq=6, hkv=3, D=64, page=16, fmt=fmt, seed=17,
              window=100, sink=3)
    planes = []
    for x in b.planes:
        P, ps, H, w = x.shape
        unit = 16 // x.element_size() if w * x.element_size() >= 16 else w
        if layout == "padded":
            hs, rs = w + unit, (w + unit) * H + 3 * unit
            pg = rs * ps + 5 * unit
        elif layout == "one_tensor":
            hs, rs, pg = w, w * H, 2 * w * H * ps
        else:
            rs, pg = w, w * ps
            hs = pg * P + 7 * unit
        size = (P - 1) * pg + (ps - 1) * rs + (H - 1) * hs + w
        buf = torch.empty(size + 64, dtype=x.dtype, device="cuda")
        buf.view(torch.uint8).fill_(0xff)
        y = buf.as_strided(x.shape, (pg, rs, hs, 1))
        y.copy_(x)
        planes.append(y)
    if layout == "one_tensor":
        k, v = (planes[0], planes[1]) if fmt == "bf16" else (planes[0], planes[2])
        P, ps, H, w = k.shape
        both = torch.empty((P, 2, ps, H, w), dtype=k.dtype, device="cuda")
        both[:, 0], both[:, 1] = k, v
        planes[0], planes[1 if fmt == "bf16" else 2] = both[:, 0], both[:, 1]
    b.planes = planes
    b.cache = (qkr.cache_desc if fmt == "bf16" else qkr.cache_desc_q4)(*planes)
    b.call()
    torch.cuda.synchronize()
    b.check()


@pytest.mark.parametrize("fmt", FORMATS)
def test_nonfinite_query_stays_in_its_row(fmt):
    for n in (3, 90):
        b = Batch(n=[n], lens=[n + 40], hq=4, hkv=2, D=64, page=16, fmt=fmt, seed=18, poison=False)
        ref = Batch(n=[n], lens=[n + 40], hq=4, hkv=2, D=64, page=16, fmt=fmt, seed=18,
                    poison=False)
        b.q[1, 2, 7] = float("nan")
        b.call()
        ref.call()
        torch.cuda.synchronize()
        assert torch.isnan(b.out[1, 2]).all()
        b.out[1, 2] = ref.out[1, 2]
        assert torch.equal(b.out[:n].view(torch.int16), ref.out[:n].view(torch.int16))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("n", [1, 40])
def test_huge_values_behind_the_mask(fmt, n):
    """The largest finite numbers in keys a token does not see leave no trace."""
    b = Batch(n=[n], lens=[n + 300], hq=2, hkv=2, D=64, page=16, fmt=fmt, seed=19, poison=False,
              window=40, sink=2)
    plain = Batch(n=[n], lens=[n + 300], hq=2, hkv=2, D=64, page=16, fmt=fmt, seed=19,
                  poison=False, window=40, sink=2)
    for pl in b.planes:
        if pl.dtype == torch.bfloat16:
            pl[~b.seen] = 3.3e38     # rows that no token sees
    b.call()
    plain.call()
    torch.cuda.synchronize()
    assert torch.equal(b.out[:n].view(torch.int16), plain.out[:n].view(torch.int16))


@pytest.mark.parametrize("fmt", FORMATS)
def test_far_rows(fmt):
    """Pages whose rows lie beyond 2^31 bytes (and elements, for bf16)."""
    D, hkv, page = 64, 1, 16
    wide = (1 << 32) + 64
    b = Batch(n=[1, 30], lens=[40, 30], hq=2, hkv=hkv, D=D, page=page, fmt=fmt, seed=12)
    planes = []
    for x in b.planes:
        es = x.element_size()
        gap = wide // 4 // es // 16 * 16      # pages about 1 GiB apart
        buf = torch.empty(gap * (x.shape[0] - 1) + x[0].numel() + 64, dtype=x.dtype, device="cuda")
        y = buf.as_strided(x.shape, (gap, x.shape[2] * x.shape[3], x.shape[3], 1))
        y.copy_(x)
        planes.append(y)
    b.planes = planes
    b.cache = (qkr.cache_desc if fmt == "bf16" else qkr.cache_desc_q4)(*planes)
    b.call()
    torch.cuda.synchronize()
    b.check()


@pytest.mark.parametrize("fmt", FORMATS)
def test_captured_and_replayed_with_growing_lengths(fmt):
    """One captured decode step serves every length up to its bounds; eager
    calls on another stream with their own workspace run beside it."""
    b = Batch(n=[1, 1], lens=[400, 399], hq=4, hkv=2, D=64, page=16, fmt=fmt, seed=13,
              poison=False)
    ws = b.call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qkr.cache_attention(b.q, b.cache, b.out, b.table, b.lens, b.cu, 1, 400, lse=b.lse,
                            workspace=ws)
    other = Batch(n=[1, 1], lens=[300, 20], hq=4, hkv=2, D=64, page=16, fmt=fmt, seed=14)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for a, c in ((1, 0), (16, 399), (333, 17), (400, 399)):
        b.L = [a, c]
        b.lens.copy_(torch.tensor(b.L, dtype=torch.int32))
        b.out_buf.fill_(7.0)
        b.lse.fill_(7.0)
        graph.replay()
        other.call(stream=side, workspace=None)
        torch.cuda.synchronize()
        b.check()
        other.check()


def test_overlap_switch_changes_nothing():
    outs = []
    for on in (True, False):
        qkr.launch_overlap(on)
        try:
            b = Batch(n=[1, 90], lens=[3000, 400], hq=8, hkv=2, D=128, page=64, seed=15)
            b.call()
            b.call()
            torch.cuda.synchronize()
            outs.append(b.out.clone())
        finally:
            qkr.launch_overlap(True)
    assert torch.equal(outs[0].view(torch.int16), outs[1].view(torch.int16))


def test_lse_is_optional_and_joins_two_caches():
    """Attention over a cache equals the lse-weighted sum over its two halves."""
    b = Batch(n=[1], lens=[512], hq=4, hkv=2, D=64, page=16, seed=16, poison=False)
    b.call(lse=False)
    whole = b.out[:1].double().clone()
    assert (b.lse == 7).all()
    parts = []
    table = b.table
    for half in range(2):
        b.table = table[:, 16 * half:16 * half + 17].contiguous()
        b.lens.fill_(256)
        b.call(max_len=256)
        torch.cuda.synchronize()
        parts.append((b.out[:1].double().clone(), b.lse[:1].double().clone()))
    w = torch.softmax(torch.stack([p[1] for p in parts]), 0)
    joined = sum(x.unsqueeze(-1) * p[0] for x, p in zip(w, parts))
    assert (joined - whole).abs().max() < 3 * 2 ** -8 * whole.abs().max()
    assert math.isfinite(float(joined.sum()))


@pytest.mark.parametrize("fmt", FORMATS)
def test_binding_refusals(fmt):
    """What the binding itself refuses, before the library is called."""
    b = Batch(n=[1, 2], lens=[40, 50], hq=4, hkv=2, D=64, page=16, fmt=fmt, seed=21)

    def call(**kw):
        a = dict(q=b.q, cache=b.cache, out=b.out, page_table=b.table, lens=b.lens, cu_q=b.cu,
                 max_q=2, max_len=50)
        a.update(kw)
        qkr.cache_attention(**a)
    call()
    for kw in (dict(q=b.q.float()), dict(q=b.q.cpu()), dict(q=b.q[..., :32]), dict(q=b.q[0]),
               dict(q=b.q.transpose(1, 2)), dict(out=b.out[:1]), dict(out=b.out.float()),
               dict(out=b.out.transpose(0, 1)), dict(page_table=b.table.long()),
               dict(page_table=b.table[:1]), dict(page_table=b.table.t().contiguous().t()),
               dict(lens=b.lens.long()), dict(lens=b.lens[:1]), dict(cu_q=b.cu[:2]),
               dict(cu_q=b.cu.cpu()), dict(max_len=16 * b.table.shape[1] + 1),
               dict(lse=b.lse.half()), dict(lse=b.lse[:, :2])):
        with pytest.raises(ValueError):
            call(**kw)
    with pytest.raises(qkr.QkrError) as e:
        call(window=-1)
    assert e.value.status == qkr.QKR_ERR_INVALID_ARG
    big = Batch(n=[1] * 8, lens=[5000] * 8, hq=4, hkv=2, D=64, page=16, fmt=fmt, seed=22)
    need = qkr.cache_attention_workspace(big.q, big.cache, 8, 1, 5000)
    assert need > 0
    with pytest.raises(qkr.QkrError) as e:
        big.call(workspace=torch.empty(need - 1, dtype=torch.uint8, device="cuda"))
    assert "workspace" in str(e.value)
    planes = b.planes
    make = qkr.cache_desc if fmt == "bf16" else qkr.cache_desc_q4
    for bad in (planes[0][0], planes[0].float(), planes[0].cpu(), planes[0][..., :-8]):
        with pytest.raises(ValueError):
            make(bad, *planes[1:])
