"""The paged cache and its attention against 64-bit restatements."""
import math

import pytest
import torch

from gated_delta_rule_43_gb300 import kda
from tests import paged_util as U
from tests.paged_util import BF, E4M3, F32, Batch

pytestmark = pytest.mark.gpu
DEV = "cuda"
KINDS = [(BF, BF), (BF, E4M3), (F32, F32), (F32, E4M3)]


def bits(t):
    return t.contiguous().view(torch.uint8)


def write_case(lens, before, Hk, D, dtype, cache, ps=16, seed=0, halves=False, fused=True):
    b = Batch(lens, before, Hk, D, dtype, cache, ps, seed, DEV, halves)
    gen = torch.Generator().manual_seed(seed + 100)
    x = torch.randn(b.T, 2 * Hk + 1, D, generator=gen) * torch.exp(3 * torch.randn(b.T, 1, 1, generator=gen))
    x = x.to(dtype).to(DEV)
    k, v = x[:, :Hk], x[:, Hk:2 * Hk]
    if not fused:
        k, v = k.contiguous(), v.contiguous()
    return b, k, v


def expect_write(b, k, v):
    """The pools as they have to be afterwards."""
    out = []
    for x, pages, scales in ((k, b.k_pages, b.k_scales), (v, b.v_pages, b.v_scales)):
        pages, scales = pages.clone(), None if scales is None else scales.clone()
        if scales is None:
            y, s = x.to(pages.dtype), None
        else:
            y, s = U.quantise(x.float())
        for t, n, pos in U.places(b):
            if pos >= 0:
                page, slot = int(b.table[n, pos // b.ps]), pos % b.ps
                pages.view(torch.uint8).reshape(*pages.shape[:3], -1)[page, :, slot] = \
                    y[t].contiguous().view(torch.uint8).reshape(b.Hk, -1)
                if s is not None:
                    scales[page, :, slot] = s[t]
        out.append((pages, scales))
    return out


def check_write(b, k, v, **kw):
    want = expect_write(b, k, v)
    kda.kv_cache_write(k, v, *b.cache, b.cu, **b.scales, check=True, **kw)
    for (pages, scales), p, s in zip(want, (b.k_pages, b.v_pages), (b.k_scales, b.v_scales)):
        assert torch.equal(bits(p), bits(pages))
        if s is not None:
            assert torch.equal(bits(s), bits(scales))


@pytest.mark.parametrize("dtype,cache", KINDS)
@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("Hk,ps", [(1, 16), (3, 32), (8, 64), (17, 128)])
def test_write_and_read(dtype, cache, D, Hk, ps):
    b, k, v = write_case([5, 0, 37, 1, 130], [3, 9, 0, 15, 200], Hk, D, dtype, cache, ps, seed=D + Hk)
    check_write(b, k, v)
    # read back: exactly the stored values, in every type
    pools = [U.values(p, s) for p, s in ((b.k_pages, b.k_scales), (b.v_pages, b.v_scales))]
    for out in {dtype} | ({BF, F32} if cache is E4M3 else set()):
        got = kda.kv_cache_read(*b.cache, b.cu, total_tokens=b.T, dtype=out, **b.scales, check=True)
        for g, pool in zip(got, pools):
            assert g.dtype is out and g.shape == (b.T, Hk, D)
            for t, n, pos in U.places(b):
                assert torch.equal(g[t].double(), pool[int(b.table[n, pos // ps]), :, pos % ps])


@pytest.mark.parametrize("dtype,cache", KINDS)
def test_write_halves_of_one_pool_and_packed_rows(dtype, cache):
    b, k, v = write_case([40, 3], [0, 61], 4, 64, dtype, cache, 32, halves=True, fused=False)
    check_write(b, k, v)


@pytest.mark.parametrize("cache", [BF, E4M3])
def test_write_a_step_with_padding(cache):
    """cu_seqlens None: one token a sequence; one without tokens writes nothing."""
    b, k, v = write_case([1] * 40, [int(7 * i % 90) for i in range(40)], 2, 128, BF, cache, 16)
    b.kv_lens[3] = b.kv_lens[39] = 0
    want = expect_write(b, k, v)
    kda.kv_cache_write(k, v, *b.cache, **b.scales, check=True)
    for (pages, scales), p, s in zip(want, (b.k_pages, b.v_pages), (b.k_scales, b.v_scales)):
        assert torch.equal(bits(p), bits(pages)) and (s is None or torch.equal(bits(s), bits(scales)))
    k2, v2 = kda.kv_cache_read(*b.cache, None, total_tokens=40, **b.scales, check=True)
    assert not k2[3].any() and not v2[39].any()


def test_left_padding_and_rows_behind_the_last():
    """Sequences shorter than their rows: padding is not written, reads as zeros, attends to
    nothing; rows past cu[N] stay as they are."""
    b, k, v = write_case([8, 8, 8], [-3, 0, -8], 2, 64, BF, BF, 16, seed=4)
    check_write(b, k, v)
    b.T += 5                                    # (five more rows behind the last sequence)
    q = b.queries(4)
    o = torch.full((b.T, 4, 64), 7.0, dtype=BF, device=DEV)
    kda.paged_attn_fwd(q, *b.cache, b.cu, o=o, check=True)
    assert (o[24:] == 7).all() and not o[:3].any() and not o[16:24].any()
    U.check_attention(o[:24], b, q[:24])
    rk, rv = (torch.full((b.T, 2, 64), 7.0, dtype=BF, device=DEV) for _ in range(2))
    kda.kv_cache_read(*b.cache, b.cu, total_tokens=b.T, k=rk, v=rv, check=True)
    assert (rk[24:] == 7).all() and not rv[:3].any() and torch.equal(rk[8:16], k[8:16])


def test_values_at_the_edges_of_e4m3():
    """Rows of zeros, one value, borders of the scale, infinities and NaN."""
    top = [0.0, 1.0, 448.0, 449.0, 1.75, 1.7578125, 2.0 ** 127 * 1.75, 2.0 ** 127 * 1.99, 2.0 ** -126,
           2.0 ** -133, 3e38, 1e-30]
    x = torch.zeros(len(top) + 3, 2, 32)
    for i, t in enumerate(top):
        x[i, 0, 5], x[i, 1] = t, torch.linspace(-t, t, 32)
    x[-3, 0, 3], x[-3, 0, 4] = math.inf, 2.0
    x[-2, 1, 3], x[-2, 1, 4] = math.nan, 2.0
    x[-1, 0, :] = -math.inf
    for dtype in (F32, BF):
        b = Batch([len(x)], [0], 1, 32, dtype, E4M3, 16, device=DEV)
        y = x.to(dtype).to(DEV)
        check_write(b, y[:, :1], y[:, 1:])


ATTN = [
    # lens, before, Hk, group, ps
    ([1], [0], 1, 1, 16),
    ([1], [127], 1, 4, 16),
    ([128], [0], 1, 1, 128),
    ([129], [0], 2, 1, 16),
    ([17, 1, 0, 150, 96], [0, 300, 20, 0, 77], 2, 4, 16),
    ([300], [77], 1, 3, 32),
    ([64], [1000], 2, 8, 64),
    ([5, 5], [500, 3], 1, 16, 16),
    ([33], [95], 1, 40, 16),
    ([2, 700], [2000, 13], 3, 2, 128),
    ([3] * 50, [11 * i for i in range(50)], 2, 5, 16),
]


@pytest.mark.parametrize("dtype,cache", KINDS)
@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("case", ATTN, ids=[str(i) for i in range(len(ATTN))])
def test_chunk(dtype, cache, D, case):
    lens, before, Hk, group, ps = case
    b = Batch(lens, before, Hk, D, dtype, cache, ps, seed=sum(lens) + D, device=DEV)
    q = b.queries(Hk * group)
    o = kda.paged_attn_fwd(q, *b.cache, b.cu, **b.scales, check=True)
    assert o.dtype is dtype and o.shape == q.shape
    U.check_attention(o, b, q)


@pytest.mark.parametrize("dtype,cache", KINDS)
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (7, 0), (64, 4), (128, 128), (129, 1), (200, 300),
                                          (1000000, 5), (130, 1000000)])
def test_window_and_sinks(dtype, cache, window, sinks):
    for D, group in ((64, 4), (128, 1)):
        b = Batch([1, 300, 0, 77, 9], [600, 13, 4, 800, 0], 2, D, dtype, cache, 16, seed=window, device=DEV)
        q = b.queries(2 * group)
        o = kda.paged_attn_fwd(q, *b.cache, b.cu, window=window, sinks=sinks, **b.scales, check=True)
        U.check_attention(o, b, q, window=window, sinks=sinks)


DECODE = [
    ([1], 1, 4, 16), ([2000], 8, 4, 16), ([5, 1, 130, 128, 127, 129, 999], 2, 8, 32), ([3] * 70, 1, 1, 16),
    ([700, 20], 1, 16, 64), ([700, 20], 2, 17, 64), ([300], 1, 100, 128), ([64, 6000], 3, 5, 256),
]


@pytest.mark.parametrize("dtype,cache", KINDS)
@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("case", DECODE, ids=[str(i) for i in range(len(DECODE))])
def test_decode(dtype, cache, D, case):
    ctx, Hk, group, ps = case
    b = Batch([1] * len(ctx), [c - 1 for c in ctx], Hk, D, dtype, cache, ps, seed=D, device=DEV)
    q = b.queries(Hk * group)
    o = kda.paged_attn_decode_step(q, *b.cache, **b.scales, check=True)
    U.check_attention(o, b, q)
    # the same through the chunk's entry point
    U.check_attention(kda.paged_attn_fwd(q, *b.cache, b.cu, **b.scales, check=True), b, q)


@pytest.mark.parametrize("dtype,cache", KINDS)
@pytest.mark.parametrize("window,sinks", [(1, 0), (5, 2), (128, 4), (1000, 0), (300, 500)])
def test_decode_window_and_sinks(dtype, cache, window, sinks):
    b = Batch([1] * 5, [0, 3, 700, 1500, 128], 2, 128, dtype, cache, 16, seed=window, device=DEV)
    q = b.queries(8)
    # pages that the window has passed are given back: their entries may be anything
    for n, c in enumerate(b.kv_lens.tolist()):
        lo, s = max(0, c - window) // 16, -(-sinks // 16)
        if lo > s:
            b.table[n, s:lo] = torch.tensor([-1, 1 << 30], dtype=torch.int32).repeat(lo)[:lo - s].to(DEV)
    keep = b.table.clone()
    o = kda.paged_attn_decode_step(q, *b.cache, window=window, sinks=sinks, **b.scales, check=True)
    b.table = keep.clamp(0, b.P - 1)
    U.check_attention(o, b, q, window=window, sinks=sinks)


def test_decode_of_a_padded_batch():
    """Sequences without tokens get zeros, whatever their table says."""
    for cache in (BF, E4M3):
        b = Batch([1] * 6, [40, 0, 900, 0, 2, 17], 2, 128, BF, cache, 16, device=DEV)
        q = b.queries(8)
        b.kv_lens[1] = b.kv_lens[3] = 0
        b.table[1], b.table[3] = -5, 1 << 30
        o = kda.paged_attn_decode_step(q, *b.cache, **b.scales, check=True)
        assert not o[1].any() and not o[3].any()
        U.check_attention(o, b, q)


@pytest.mark.parametrize("dtype,cache", [(BF, BF), (BF, E4M3), (F32, F32)])
def test_scale_strides_and_halves(dtype, cache):
    b = Batch([33, 9], [100, 0], 2, 64, dtype, cache, 32, device=DEV, halves=True)
    q = b.queries(6, sharp=16.0)
    x = torch.empty(b.T, 10, 64, dtype=dtype, device=DEV)
    x[:, 2:8] = q
    o = kda.paged_attn_fwd(x[:, 2:8], *b.cache, b.cu, scale=0.125, **b.scales, check=True)
    U.check_attention(o, b, q, scale=0.125)
    one = q[:1].expand(b.T, 6, 64)                       # one token for all rows
    o = kda.paged_attn_fwd(one, *b.cache, b.cu, scale=0.125, **b.scales, check=True)
    U.check_attention(o, b, one, scale=0.125)


def test_large_scores():
    """Weights that differ by many orders of magnitude, maxima that keep growing along the keys."""
    b = Batch([200], [1500], 1, 128, BF, BF, 64, seed=3, device=DEV)
    grow = torch.linspace(0, 6, 1700).to(DEV)
    for j in range(1700):
        b.k_pages[int(b.table[0, j // 64]), :, j % 64] *= grow[j]
    q = b.queries(4, sharp=6.0)
    want, size = U.attention(b, q)
    o = kda.paged_attn_fwd(q, *b.cache, b.cu, check=True).double()
    # scores of up to 6 * 6 * 5: an exponent of 180 carries 180 * 2^-24 a few times over
    assert ((o - want).abs() <= 2.0 ** -8 * (want.abs() + size) + 1e-4 * size).all()


def test_pools_past_32_bits():
    """Pages whose elements lie beyond 2^31."""
    P, ps, D = 18000, 1024, 128
    pools = [torch.empty(P, 1, ps, D, dtype=BF, device=DEV) for _ in range(2)]
    b = Batch([50], [2000], 1, D, BF, BF, ps, device=DEV)
    far = torch.tensor([[17999, 3, 16500, 0]], dtype=torch.int32, device=DEV)
    for pool, own in zip(pools, (b.k_pages, b.v_pages)):
        for i in range(3):
            pool[int(far[0, i])] = own[int(b.table[0, i])]
    q = b.queries(4)
    U.check_attention(kda.paged_attn_fwd(q, *pools, far, b.kv_lens, b.cu, check=True), b, q)
    one = torch.tensor([0, 1], dtype=torch.int32, device=DEV)
    last = kda.paged_attn_decode_step(q[-1:], *pools, far, b.kv_lens, check=True)
    b2 = b
    b2.cu, b2.T = one, 1
    U.check_attention(last, b2, q[-1:])
    k = torch.randn(1, 1, D, device=DEV).to(BF)
    kda.kv_cache_write(k, -k, *pools, far, b.kv_lens, check=True)
    rk, rv = kda.kv_cache_read(*pools, far, b.kv_lens, None, total_tokens=1, check=True)
    assert torch.equal(rk, k) and torch.equal(rv, -k)
    assert torch.equal(pools[0][16500, 0, 2049 - 2048], k[0, 0])


@pytest.mark.parametrize("cache", [BF, E4M3])
def test_many_sequences_most_without_tokens(cache):
    """Thousands of sequences, few of them with tokens, and long ones among them."""
    lens, before = [0] * 3000, [0] * 3000
    for i, n in enumerate((0, 1, 40, 700, 701, 702, 2047, 2048, 2999)):
        lens[n], before[n] = 1 + 37 * i, 500 * (i % 3)
    b = Batch(lens, before, 2, 64, BF, cache, 16, device=DEV)
    q = b.queries(8)
    o = kda.paged_attn_fwd(q, *b.cache, b.cu, **b.scales, check=True)
    U.check_attention(o, b, q)
    # one token each: those without are padding
    ctx = b.kv_lens.clone()
    b.cu, b.T = torch.arange(3001, dtype=torch.int32, device=DEV), 3000
    one = torch.randn(3000, 8, 64, device=DEV).to(BF)
    got = kda.paged_attn_decode_step(one, *b.cache, **b.scales, check=True)
    live = ctx > 0
    assert not got[~live].any()
    U.check_attention(got, b, one)


@pytest.mark.parametrize("D", [64, 128])
def test_scales_of_others(D):
    """Scales that are no powers of two, some tiny, some large."""
    b = Batch([40, 3], [700, 200], 2, D, BF, E4M3, 32, device=DEV)
    gen = torch.Generator().manual_seed(1)
    for s, spread in ((b.k_scales, 0.3), (b.v_scales, 4.0)):
        s.mul_(torch.exp(spread * torch.randn(s.shape, generator=gen)).to(DEV))
    q = b.queries(8)
    # chunks take keys and values rounded to bf16 once, so that is what they are held against
    k, v = U.values(b.k_pages, b.k_scales), U.values(b.v_pages, b.v_scales)
    rounded = Batch([40, 3], [700, 200], 2, D, BF, BF, 32, device=DEV)
    rounded.k_pages, rounded.v_pages, rounded.table = k.to(BF), v.to(BF), b.table
    U.check_attention(kda.paged_attn_fwd(q, *b.cache, b.cu, **b.scales, check=True), rounded, q)
    b.cu, b.T, one = torch.tensor([0, 1, 2], dtype=torch.int32, device=DEV), 2, q[:2]
    U.check_attention(kda.paged_attn_decode_step(one, *b.cache, **b.scales, check=True), b, one)
    rk, rv = kda.kv_cache_read(*b.cache, b.cu, total_tokens=2, dtype=F32, **b.scales, check=True)
    for t, n, pos in U.places(b):
        page = int(b.table[n, pos // 32])
        assert torch.equal(rk[t].double(), k[page, :, pos % 32].float().double())
        assert torch.equal(rv[t].double(), v[page, :, pos % 32].float().double())


@pytest.mark.parametrize("cache", [BF, E4M3])
def test_what_is_not_finite(cache):
    """A NaN in a query spoils its own row and head; in a key or a value, those who see it."""
    b = Batch([100, 5], [300, 10], 2, 128, BF, cache, 16, device=DEV)
    q = b.queries(8)
    good = kda.paged_attn_fwd(q, *b.cache, b.cu, **b.scales, check=True)
    bad = q.clone()
    bad[7, 3, 5], bad[50, 1, 0] = math.nan, math.inf
    o = kda.paged_attn_fwd(bad, *b.cache, b.cu, **b.scales)
    hurt = torch.zeros(105, 8, dtype=torch.bool, device=DEV)
    hurt[7, 3] = hurt[50, 1] = True
    assert o[hurt].isnan().all() and torch.equal(o[~hurt], good[~hurt])
    two = kda.paged_attn_decode_step(bad[6:8], *b.cache, **b.scales)
    assert two[1, 3].isnan().all() and two[0].isfinite().all() and two[1, 4:].isfinite().all()
    # a value of the last token of sequence 0, head 0: its last row sees it, sequence 1 and head 1 do not
    page = int(b.table[0, 399 // 16])
    b.v_pages.view(torch.uint8)[page, 0, 399 % 16] = 0x7f
    o = kda.paged_attn_fwd(q, *b.cache, b.cu, **b.scales)
    if cache is E4M3:
        assert o[99, :4].isnan().all()
    assert torch.equal(o[100:], good[100:]) and torch.equal(o[:100, 4:], good[:100, 4:])


def code_of(call):
    ws = torch.zeros(1 << 26, dtype=torch.uint8, device=DEV)
    call(ws)
    return kda.query_status(ws)


@pytest.mark.parametrize("cache", [BF, E4M3])
def test_bad_pages_are_reported_and_not_touched(cache):
    b = Batch([40, 30, 1], [100, 60, 500], 2, 128, BF, cache, 16, seed=9, device=DEV)
    q = b.queries(8)
    good = kda.paged_attn_fwd(q, *b.cache, b.cu, **b.scales, check=True)
    b.table[1, 2], b.table[1, 4] = b.P, -1
    o = torch.zeros_like(good)
    code, info = code_of(lambda ws: kda.paged_attn_fwd(q, *b.cache, b.cu, **b.scales, o=o, workspace=ws))
    assert (code, info) == (kda.KDA_ERR_INVALID_ARG, 1)
    assert torch.equal(o[:40], good[:40]) and torch.equal(o[70:], good[70:]) and o.isfinite().all()
    k = torch.randn(b.T, 2, 128, device=DEV).to(BF)
    b.table[1, 3:] = 1 << 20
    want = expect_write(Batch_without(b, 1), k, k)
    code, info = code_of(lambda ws: kda.kv_cache_write(k, k, *b.cache, b.cu, **b.scales, workspace=ws))
    assert (code, info) == (kda.KDA_ERR_INVALID_ARG, 1)
    assert torch.equal(bits(b.k_pages), bits(want[0][0]))
    code, info = code_of(lambda ws: kda.kv_cache_read(*b.cache, b.cu, total_tokens=b.T, **b.scales, workspace=ws))
    assert (code, info) == (kda.KDA_ERR_INVALID_ARG, 1)
    # decode: lens of one token each
    code, info = code_of(lambda ws: kda.paged_attn_decode_step(q[:3], *b.cache, **b.scales, workspace=ws))
    assert (code, info) == (kda.KDA_ERR_INVALID_ARG, 1)


class Batch_without:
    """A batch as places() sees it, less the tokens of one sequence (which keeps its rows)."""

    def __init__(self, b, n):
        self.__dict__.update(b.__dict__)
        self.skip = n
        self.kv_lens = b.kv_lens.clone()
        self.kv_lens[n] = 0                     # all of its positions are below 0


def test_bad_lengths_are_reported():
    b = Batch([20, 10, 5], [0, 40, 7], 2, 64, BF, BF, 16, device=DEV)
    q = b.queries(4)
    good = kda.paged_attn_fwd(q, *b.cache, b.cu, check=True)
    ctx = b.kv_lens.clone()
    for bad in (-1, 100000):
        b.kv_lens[1] = bad
        o = torch.full_like(good, 7.0)
        assert code_of(lambda ws: kda.paged_attn_fwd(q, *b.cache, b.cu, o=o, workspace=ws)) == \
            (kda.KDA_ERR_SEQLENS, 1)
        assert torch.equal(o[:20], good[:20]) and (o[20:30] == 7).all() and torch.equal(o[30:], good[30:])
    b.kv_lens = ctx
    for cu, n in (([0, 20, 15, 35], 1), ([0, 20, 30, 36], 2), ([0, 20, 99, 35], 1), ([-1, 20, 30, 35], 0),
                  ([1, 20, 30, 35], 0)):
        b.cu = torch.tensor(cu, dtype=torch.int32, device=DEV)
        for call in (lambda ws: kda.paged_attn_fwd(q, *b.cache, b.cu, workspace=ws),
                     lambda ws: kda.kv_cache_write(q[:, :2], q[:, 2:], *b.cache, b.cu, workspace=ws),
                     lambda ws: kda.kv_cache_read(*b.cache, b.cu, total_tokens=35, workspace=ws)):
            code, info = code_of(call)
            assert code == kda.KDA_ERR_SEQLENS and info in (n, n + 1)


def test_nothing_to_do():
    b = Batch([0, 0], [5, 0], 2, 64, BF, BF, 16, device=DEV)
    q = b.queries(4)
    assert kda.paged_attn_fwd(q, *b.cache, b.cu, check=True).shape == (0, 4, 64)
    kda.kv_cache_write(q[:, :2], q[:, 2:], *b.cache, b.cu, check=True)
    none = torch.empty(0, 3, dtype=torch.int32, device=DEV)
    no = torch.empty(0, dtype=torch.int32, device=DEV)
    assert kda.paged_attn_decode_step(q, b.k_pages, b.v_pages, none, no, check=True).shape == (0, 4, 64)


def test_outputs_stay_inside_their_bands():
    """Outputs and workspace between sentinels, inputs unchanged."""
    for dtype, cache, D in ((BF, BF, 128), (BF, E4M3, 128), (BF, BF, 64), (F32, F32, 64)):
        b = Batch([1, 150, 31], [3000, 13, 1000], 2, D, dtype, cache, 16, device=DEV)
        q = b.queries(10)
        before = [bits(t).clone() for t in (q, b.k_pages, b.v_pages, b.table)]
        band = torch.full((b.T * 10 * D + 2048,), 7.0, dtype=dtype, device=DEV)
        o = band[1024:-1024].view(b.T, 10, D)
        need = kda._paged_workspace_size(0, 3, b.table.shape[1], b.P, 16, 2, D, kda.KDA_E4M3 if cache is E4M3 else
                                         kda._DT[dtype], b.T, 10, kda._DT[dtype], False)
        ws = torch.full((need + 8192,), 77, dtype=torch.uint8, device=DEV)
        kda.paged_attn_fwd(q, *b.cache, b.cu, **b.scales, o=o, workspace=ws[4096:4096 + need], check=True)
        U.check_attention(o, b, q)
        assert (band[:1024] == 7).all() and (band[-1024:] == 7).all()
        assert (ws[:4096] == 77).all() and (ws[4096 + need:] == 77).all()
        assert all(torch.equal(x, bits(t)) for x, t in zip(before, (q, b.k_pages, b.v_pages, b.table)))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_addresses_of_16_bytes(dtype, D):
    """Inputs and outputs that are aligned to 16 bytes and no more."""
    b = Batch([150, 9], [30, 1000], 2, D, dtype, dtype, 16, device=DEV)
    n = 16 // torch.empty(0, dtype=dtype).element_size()

    def off(t):
        x = torch.empty(t.numel() + n, dtype=t.dtype, device=DEV)[n:].view(t.shape)
        x.copy_(t)
        assert x.data_ptr() % 32 == 16
        return x
    b.k_pages, b.v_pages = off(b.k_pages), off(b.v_pages)
    q = off(b.queries(6))
    o = off(torch.zeros_like(q))
    kda.paged_attn_fwd(q, *b.cache, b.cu, o=o, check=True)
    U.check_attention(o, b, q)
    k, v = off(q[:, :2].contiguous()), off(q[:, 2:4].contiguous())
    kda.kv_cache_write(k, v, *b.cache, b.cu, check=True)
    rk, rv = off(torch.zeros_like(k)), off(torch.zeros_like(v))
    kda.kv_cache_read(*b.cache, b.cu, total_tokens=b.T, k=rk, v=rv, check=True)
    assert torch.equal(rk, k) and torch.equal(rv, v)
    b.cu, b.T = torch.tensor([0, 1, 2], dtype=torch.int32, device=DEV), 2
    kda.paged_attn_decode_step(q[:2], *b.cache, o=o[:2], check=True)
    U.check_attention(o[:2], b, q[:2])


@pytest.mark.parametrize("dtype,cache", [(BF, BF), (BF, E4M3), (F32, F32)])
def test_in_a_graph_on_another_stream(dtype, cache):
    """Write, chunk and decode captured once, replayed with new tokens and lengths."""
    b = Batch([30, 50], [400, 10], 2, 128, dtype, cache, 16, seed=5, device=DEV)
    grown = Batch([30, 50], [400, 10], 2, 128, dtype, cache, 16, seed=6, device=DEV)
    q, q2 = b.queries(8), grown.queries(8, seed=8)
    kv = torch.randn(b.T, 4, 128, device=DEV).to(dtype)
    side = torch.cuda.Stream()
    sizes = dict(workspace=torch.empty(1 << 27, dtype=torch.uint8, device=DEV))

    def step():
        kda.kv_cache_write(kv[:, :2], kv[:, 2:], *b.cache, b.cu, **b.scales)
        chunk = kda.paged_attn_fwd(q, *b.cache, b.cu, **b.scales, **sizes)
        return chunk, kda.paged_attn_decode_step(q[:2], *b.cache, **b.scales, **sizes)
    with torch.cuda.stream(side):
        step()
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            chunk, one = step()
    for name in ("k_pages", "v_pages", "k_scales", "v_scales", "table", "kv_lens"):
        if getattr(b, name) is not None:
            getattr(b, name).copy_(getattr(grown, name))
    q.copy_(q2)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    U.check_attention(chunk, b, q)
    b.cu, b.T = torch.tensor([0, 1, 2], dtype=torch.int32, device=DEV), 2
    U.check_attention(one, b, q[:2])


@pytest.mark.parametrize("cache", [BF, E4M3])
def test_a_serving_loop(cache):
    """A hybrid layer's life: a prompt in two chunks, then single tokens; queries and keys prepared,
    keys and values written, attention over the pages; against attention over all tokens at once."""
    H, Hk, D, ps, total, first, second = 8, 2, 128, 16, 200, 77, 100
    gen = torch.Generator(device=DEV).manual_seed(11)
    x = torch.randn(total, H + 2 * Hk, D, device=DEV, generator=gen).to(BF)
    freq, rs = kda.rope_inv_freq(D, device=DEV)
    pos = torch.arange(total, dtype=torch.int32, device=DEV)
    b = Batch([total], [0], Hk, D, BF, cache, ps, device=DEV)
    for t in (b.k_pages, b.v_pages):
        t.view(torch.uint8).fill_(0x7f)
    out, queries = [], []
    cuts = [0, first, first + second] + list(range(first + second + 1, total + 1))
    for a, e in zip(cuts, cuts[1:]):
        q, k = kda.qk_norm_rope(x[a:e, :H], x[a:e, H:H + Hk], pos[a:e], freq, norm="rms", q_scale=D ** -0.5,
                                rope_scale=rs)
        lens = torch.tensor([e], dtype=torch.int32, device=DEV)
        cu = torch.tensor([0, e - a], dtype=torch.int32, device=DEV)
        kda.kv_cache_write(k, x[a:e, H + Hk:], b.k_pages, b.v_pages, b.table, lens, cu, **b.scales, check=True)
        if e - a > 1:
            out.append(kda.paged_attn_fwd(q, b.k_pages, b.v_pages, b.table, lens, cu, **b.scales, check=True))
        else:
            out.append(kda.paged_attn_decode_step(q, b.k_pages, b.v_pages, b.table, lens, **b.scales, check=True))
        queries.append(q)
    U.check_attention(torch.cat(out), b, torch.cat(queries))


def test_calls_on_two_streams_at_once():
    b = Batch([100, 3], [900, 2500], 2, 128, BF, BF, 16, device=DEV)
    c = Batch([60, 9], [300, 1200], 2, 64, BF, E4M3, 16, device=DEV)
    qb, qc = b.queries(8), c.queries(4)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = []
    for i in range(10):
        for s, x, q in ((streams[0], b, qb), (streams[1], c, qc)):
            got.append(kda.paged_attn_fwd(q, *x.cache, x.cu, **x.scales, stream=s))
    torch.cuda.synchronize()
    U.check_attention(got[0], b, qb)
    U.check_attention(got[1], c, qc)
    for i in range(2, 20):
        assert torch.equal(got[i], got[i % 2])


@pytest.mark.parametrize("decode", [False, True])
@pytest.mark.parametrize("cache", [BF, E4M3])
def test_an_expired_wait_is_reported(cache, decode):
    """A part that leaves out a load waits for 2.2 s and gives up; the next call on the same workspace
    is as ever."""
    b = Batch([1, 1] if decode else [200, 9], [3000, 900], 2, 128, BF, cache, 16, device=DEV)
    q = b.queries(8)
    ws = torch.zeros(1 << 26, dtype=torch.uint8, device=DEV)

    def call():
        if decode:
            return kda.paged_attn_decode_step(q, *b.cache, **b.scales, workspace=ws)
        return kda.paged_attn_fwd(q, *b.cache, b.cu, **b.scales, workspace=ws)
    good = call()
    assert kda.query_status(ws)[0] == kda.KDA_OK
    assert kda.load().kda_test_paged_fault(2) == kda.KDA_OK
    call()
    assert kda.query_status(ws) == (kda.KDA_ERR_TIMEOUT, 2)
    again = call()
    assert kda.query_status(ws)[0] == kda.KDA_OK and torch.equal(again, good)
    U.check_attention(again, b, q)


def spoil(b, seen):
    """Keys, values and scales of the positions that no token sees become NaN; seen(n, ctx) -> bool [ctx]."""
    for n, c in enumerate(b.kv_lens.tolist()):
        j = torch.arange(c)[~seen(n, c)].to(DEV)
        page, slot = b.table[n, j // b.ps].long(), j % b.ps
        for pages, scales in ((b.k_pages, b.k_scales), (b.v_pages, b.v_scales)):
            raw = torch.full((len(j), b.Hk, b.D), math.nan, device=DEV).to(pages.dtype)
            pages.view(torch.uint8)[page, :, slot] = raw.view(torch.uint8)
            if scales is not None:
                scales[page, :, slot] = math.nan


@pytest.mark.parametrize("dtype,cache", KINDS)
@pytest.mark.parametrize("window,sinks", [(1, 0), (5, 2), (100, 4), (250, 200), (128, 130)])
@pytest.mark.parametrize("ps", [16, 256])
def test_what_the_windows_have_passed_may_be_anything(dtype, cache, window, sinks, ps):
    for D, group in ((64, 4), (128, 2)):
        b = Batch([1, 3, 0, 60], [600, 1300, 4, 777], 2, D, dtype, cache, ps, seed=window, device=DEV)
        q = b.queries(2 * group)
        spoil(b, lambda n, c: (torch.arange(c) < sinks) | (torch.arange(c) > c - b.lens[n] - window))
        o = kda.paged_attn_fwd(q, *b.cache, b.cu, window=window, sinks=sinks, **b.scales, check=True)
        U.check_attention(o, b, q, window=window, sinks=sinks)
        b = Batch([1] * 4, [600, 1300, 0, 255], 2, D, dtype, cache, ps, seed=window, device=DEV)
        q = b.queries(2 * group)
        spoil(b, lambda n, c: (torch.arange(c) < sinks) | (torch.arange(c) >= c - window))
        o = kda.paged_attn_decode_step(q, *b.cache, window=window, sinks=sinks, **b.scales, check=True)
        U.check_attention(o, b, q, window=window, sinks=sinks)


@pytest.mark.parametrize("cache", [F32, E4M3])
def test_single_precision_reports_what_does_not_fit(cache):
    b = Batch([1] * 5, [700, 60, 0, 5, 1500], 2, 64, F32, cache, 16, seed=3, device=DEV)
    q = b.queries(8)
    good = kda.paged_attn_decode_step(q, *b.cache, **b.scales, check=True)
    table, lens = b.table.clone(), b.kv_lens.clone()
    b.table[1, 2] = b.P
    o = torch.zeros_like(good)
    call = lambda ws: kda.paged_attn_decode_step(q, *b.cache, **b.scales, o=o, workspace=ws)  # noqa: E731
    assert code_of(call) == (kda.KDA_ERR_INVALID_ARG, 1)
    others = [0, 2, 3, 4]
    assert torch.equal(o[others], good[others]) and o.isfinite().all()
    b.table = table
    for bad in (-3, 1 << 20):
        b.kv_lens[3] = bad
        o.fill_(7.0)
        assert code_of(call) == (kda.KDA_ERR_SEQLENS, 3)
        assert (o[3] == 7).all() and torch.equal(o[[0, 1, 2, 4]], good[[0, 1, 2, 4]])
        b.kv_lens = lens.clone()
    assert code_of(call)[0] == kda.KDA_OK
    assert torch.equal(o, good)
    q[2, 5, 1] = math.nan
    o = kda.paged_attn_decode_step(q, *b.cache, **b.scales)
    hurt = torch.zeros(5, 8, dtype=torch.bool, device=DEV)
    hurt[2, 5] = True
    assert o[hurt].isnan().all() and torch.equal(o[~hurt], good[~hurt])


@pytest.mark.parametrize("dtype,cache", KINDS)
@pytest.mark.parametrize("D", [32, 128])
def test_single_tokens_stay_inside_their_bands(dtype, cache, D):
    b = Batch([1] * 9, [3000, 13, 0, 1000, 128, 127, 1, 40, 2222], 2, D, dtype, cache, 16, device=DEV)
    q = b.queries(10)
    before = [bits(t).clone() for t in (q, b.k_pages, b.v_pages, b.table)]
    band = torch.full((9 * 10 * D + 2048,), 7.0, dtype=dtype, device=DEV)
    o = band[1024:-1024].view(9, 10, D)
    need = kda._paged_workspace_size(0, 9, b.table.shape[1], b.P, 16, 2, D, kda.KDA_E4M3 if cache is E4M3 else
                                     kda._DT[dtype], 9, 10, kda._DT[dtype], True)
    ws = torch.full((need + 8192,), 77, dtype=torch.uint8, device=DEV)
    kda.paged_attn_decode_step(q, *b.cache, **b.scales, o=o, workspace=ws[4096:4096 + need], check=True)
    U.check_attention(o, b, q)
    assert (band[:1024] == 7).all() and (band[-1024:] == 7).all()
    assert (ws[:4096] == 77).all() and (ws[4096 + need:] == 77).all()
    assert all(torch.equal(x, bits(t)) for x, t in zip(before, (q, b.k_pages, b.v_pages, b.table)))


@pytest.mark.parametrize("cache", [F32, E4M3])
def test_single_precision_of_many_sequences(cache):
    """More items than CTAs, most of them short, among them some without tokens; and one long one."""
    before = [(37 * i) % 150 for i in range(700)]
    before[350] = 9000
    b = Batch([1] * 700, before, 1, 32, F32, cache, 16, seed=5, device=DEV)
    b.kv_lens[::7] = 0
    q = b.queries(3)
    o = kda.paged_attn_decode_step(q, *b.cache, **b.scales, check=True)
    assert not o[::7].any()
    U.check_attention(o, b, q)


def test_two_graphs_take_turns():
    """Captured with workspaces of their own making, replayed in any order, on the stream's data of then."""
    b = Batch([1] * 4, [500, 3, 1200, 64], 2, 128, BF, BF, 16, device=DEV)
    c = Batch([30, 1, 200], [100, 900, 0], 2, 64, F32, F32, 32, device=DEV)
    qb, qc = b.queries(8), c.queries(4)
    want = [[], []]
    other = [b.queries(8, seed=9), c.queries(4, seed=9)]
    for x, y in ((qb, qc), other):
        want[0].append(kda.paged_attn_decode_step(x, *b.cache, check=True))
        want[1].append(kda.paged_attn_fwd(y, *c.cache, c.cu, check=True))
    torch.cuda.synchronize()
    graphs, outs = [], []
    for call in (lambda: kda.paged_attn_decode_step(qb, *b.cache), lambda: kda.paged_attn_fwd(qc, *c.cache, c.cu)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(call())
        graphs.append(g)
    for turn in (0, 1, 0):
        if turn:
            qb.copy_(other[0])
            qc.copy_(other[1])
        for i in (1, 0, 0, 1):
            outs[i].fill_(7.0)
            graphs[i].replay()
        assert torch.equal(outs[0], want[0][turn]) and torch.equal(outs[1], want[1][turn])
        if turn:
            qb.copy_(b.queries(8))
            qc.copy_(c.queries(4))
