"""The paged cache and its attention: cases that once went wrong, or that nothing looked at."""
import math

import pytest
import torch

from gated_delta_rule_43_gb300 import kda
from tests import paged_util as U
from tests.paged_util import BF, E4M3, F32

pytestmark = pytest.mark.gpu
DEV = "cuda"
KINDS = [(BF, BF), (BF, E4M3), (F32, F32), (F32, E4M3)]


@pytest.mark.parametrize("cache", [BF, E4M3])
def test_single_tokens_behind_the_longest_context(cache):
    """2^31 - 1024 tokens, every page of them the same one: the answer is that of one page.  A CTA goes through
    110377 tiles, whose pieces' places pass 32 bits when they are multiplied out."""
    ps, Hk, group, D = 1024, 1, 4, 32
    width = (1 << 31) // ps - 1
    b = U.Batch([1, 1], [ps - 1, 299], Hk, D, BF, cache, ps, seed=1, device=DEV)
    q = b.queries(Hk * group)
    table = b.table[:, :1].repeat(1, width).contiguous()
    lens = torch.tensor([width * ps, 300], dtype=torch.int32, device=DEV)
    got = kda.paged_attn_decode_step(q, b.k_pages, b.v_pages, table, lens, **b.scales, check=True).double()
    want, size = U.attention(b, q)
    # A thread adds up to 110377 / 4 pieces of 4 tiles, sums of weights and of values, at 2^-24 of the sum each:
    # 2 * 27595 * 2^-24 = 3.3e-3; beside that the roundings of any call (check_attention).
    slack = 2.0 ** -8 * (want.abs() + size) + 3.4e-3 * size + 1e-30
    assert got.isfinite().all() and ((got - want).abs() <= slack).all()


def bits(t):
    return t.contiguous().view(torch.uint8)


def status_of(call):
    ws = torch.zeros(1 << 26, dtype=torch.uint8, device=DEV)
    call(ws)
    return kda.query_status(ws)


@pytest.mark.parametrize("dtype,cache", KINDS)
def test_a_first_sequence_that_does_not_begin_at_0_is_skipped(dtype, cache):
    b = U.Batch([20, 10, 5], [0, 40, 7], 2, 64, dtype, cache, 16, device=DEV)
    q, bad = b.queries(4), torch.tensor([1, 20, 30, 35], dtype=torch.int32, device=DEV)
    good = kda.paged_attn_fwd(q, *b.cache, b.cu, **b.scales, check=True)
    o = torch.full_like(good, 7.0)
    assert status_of(lambda ws: kda.paged_attn_fwd(q, *b.cache, bad, **b.scales, o=o, workspace=ws)) == \
        (kda.KDA_ERR_SEQLENS, 0)
    assert (o[:20] == 7).all() and torch.equal(o[20:], good[20:])
    want = kda.kv_cache_read(*b.cache, b.cu, total_tokens=35, **b.scales, check=True)
    got = [torch.full_like(t, 7.0) for t in want]
    assert status_of(lambda ws: kda.kv_cache_read(*b.cache, bad, total_tokens=35, **b.scales, k=got[0], v=got[1],
                                                  workspace=ws)) == (kda.KDA_ERR_SEQLENS, 0)
    for g, w in zip(got, want):
        assert (g[:20] == 7).all() and torch.equal(g[20:], w[20:])
    pools = [t for t in (b.k_pages, b.v_pages, b.k_scales, b.v_scales) if t is not None]
    before = [t.clone() for t in pools]
    k, v = q[:, :2], q[:, 2:]
    kda.kv_cache_write(k, v, *b.cache, b.cu, **b.scales, check=True)
    want = [t.clone() for t in pools]
    own = b.table[0, :2].long()
    for t, x, w in zip(pools, before, want):
        t.copy_(x)
        w[own] = x[own]
    assert status_of(lambda ws: kda.kv_cache_write(k, v, *b.cache, bad, **b.scales, workspace=ws)) == \
        (kda.KDA_ERR_SEQLENS, 0)
    assert all(torch.equal(bits(t), bits(w)) for t, w in zip(pools, want))


@pytest.mark.parametrize("dtype,cache", KINDS)
def test_sequences_of_more_tokens_than_there_are_rows(dtype, cache):
    """A cu_seqlens that goes back: sequence 1 does not fit, and 0 and 2 have 40 tokens in 35 rows. Nothing is
    written; with rows enough for 40 both are gone through (rows that both claim have the values of either)."""
    b = U.Batch([20, 10, 20], [0, 40, 30], 2, 64, dtype, cache, 16, device=DEV)
    bad = torch.tensor([0, 20, 15, 35], dtype=torch.int32, device=DEV)
    q = b.queries(4)
    for rows in (35, 50):
        o = torch.full((rows, 4, 64), 7.0, dtype=dtype, device=DEV)
        assert status_of(lambda ws: kda.paged_attn_fwd(q[:rows], *b.cache, bad, **b.scales, o=o, workspace=ws)) == \
            (kda.KDA_ERR_SEQLENS, 1)
        if rows == 35:
            assert (o == 7).all()
            continue
        b.cu, b.T = torch.tensor([0, 20, 20, 50], dtype=torch.int32, device=DEV), 50
        first = kda.paged_attn_fwd(q, b.k_pages, b.v_pages, b.table[:1], b.kv_lens[:1], b.cu[:2], **b.scales, check=True)
        last = kda.paged_attn_fwd(q[15:35], b.k_pages, b.v_pages, b.table[2:].contiguous(), b.kv_lens[2:],
                                  torch.tensor([0, 20], dtype=torch.int32, device=DEV), **b.scales, check=True)
        assert torch.equal(o[:15], first[:15]) and torch.equal(o[20:35], last[5:]) and (o[35:] == 7).all()


@pytest.mark.parametrize("dtype,cache", KINDS)
def test_what_is_not_finite_reaches_those_who_see_it(dtype, cache):
    """A NaN in the key, then in the value, of one position and head: the tokens that see it, and no other head or
    sequence; a key's no token before it either."""
    for name in ("k_pages", "v_pages"):
        b = U.Batch([100, 5], [300, 10], 2, 128, dtype, cache, 16, device=DEV)
        q = b.queries(8)
        good = kda.paged_attn_fwd(q, *b.cache, b.cu, **b.scales, check=True)
        pages = getattr(b, name)
        nan = torch.full((128,), math.nan, device=DEV).to(pages.dtype)
        bits_of = pages.view(torch.uint8)
        bits_of[int(b.table[0, 380 // 16]), 0, 380 % 16] = nan.view(torch.uint8)
        o = kda.paged_attn_fwd(q, *b.cache, b.cu, **b.scales, check=True)
        assert o[80:100, :4].isnan().all()
        assert torch.equal(o[100:], good[100:]) and torch.equal(o[:, 4:], good[:, 4:])
        if name == "k_pages":
            assert torch.equal(o[:80, :4], good[:80, :4])
        one = kda.paged_attn_decode_step(q[98:100], b.k_pages, b.v_pages, b.table[[0, 0]].contiguous(),
                                         torch.tensor([399, 381], dtype=torch.int32, device=DEV), **b.scales, check=True)
        assert one[:, :4].isnan().all() and one[:, 4:].isfinite().all()
        one = kda.paged_attn_decode_step(q[99:100], b.k_pages, b.v_pages, b.table[:1], b.kv_lens[:1], window=19,
                                         **b.scales, check=True)
        assert one.isfinite().all()      # (positions 381 on: the window has passed it)
        one = kda.paged_attn_decode_step(q[79:80], b.k_pages, b.v_pages, b.table[:1],
                                         torch.tensor([380], dtype=torch.int32, device=DEV), **b.scales, check=True)
        assert one.isfinite().all()      # (behind the sequence's end)


@pytest.mark.parametrize("dtype,cache", KINDS)
def test_a_serving_loop_over_pages_of_nan(dtype, cache):
    """A prompt in two chunks, then single tokens, in pages that held NaN: no slot counts before it is written."""
    H, Hk, D, ps, total, first, second = 8, 2, 128, 16, 200, 77, 100
    gen = torch.Generator(device=DEV).manual_seed(12)
    x = torch.randn(total, H + 2 * Hk, D, device=DEV, generator=gen).to(dtype)
    q = x[:, :H] * D ** -0.5
    b = U.Batch([total], [0], Hk, D, dtype, cache, ps, device=DEV)
    for t in (b.k_pages, b.v_pages):
        t.view(torch.uint8).copy_(torch.full(t.shape, math.nan, device=DEV).to(t.dtype).view(torch.uint8))
        assert t.float().isnan().all()
    for t in (b.k_scales, b.v_scales):
        if t is not None:
            t.fill_(math.nan)
    out = []
    cuts = [0, first, first + second] + list(range(first + second + 1, total + 1))
    for a, e in zip(cuts, cuts[1:]):
        lens = torch.tensor([e], dtype=torch.int32, device=DEV)
        cu = torch.tensor([0, e - a], dtype=torch.int32, device=DEV)
        cache = (b.k_pages, b.v_pages, b.table, lens)
        kda.kv_cache_write(x[a:e, H:H + Hk], x[a:e, H + Hk:], *cache, cu, **b.scales, check=True)
        if e - a > 1:
            out.append(kda.paged_attn_fwd(q[a:e], *cache, cu, **b.scales, check=True))
        else:
            out.append(kda.paged_attn_decode_step(q[a:e], *cache, **b.scales, check=True))
    U.check_attention(torch.cat(out), b, q)


@pytest.mark.parametrize("dtype,cache", KINDS)
@pytest.mark.parametrize("D", [32, 64, 128])
def test_a_pool_without_pages(dtype, cache, D):
    """Every page is outside it: what would be there counts as zeros and is reported."""
    pages = torch.empty(0, 2, 16, D, dtype=cache, device=DEV)
    scales = {} if cache is not E4M3 else dict(k_scales=torch.empty(0, 2, 16, device=DEV),
                                               v_scales=torch.empty(0, 2, 16, device=DEV))
    q = torch.randn(40, 6, D, device=DEV).to(dtype)
    cu = torch.tensor([0, 5, 5, 30, 37], dtype=torch.int32, device=DEV)
    table = torch.zeros(4, 3, dtype=torch.int32, device=DEV)
    for lens, code in (([0, 0, 0, 0], (kda.KDA_OK, 0)), ([0, 0, 30, 0], (kda.KDA_ERR_INVALID_ARG, 2)),
                       ([0, 0, 0, 49], (kda.KDA_ERR_SEQLENS, 3))):
        kv_lens = torch.tensor(lens, dtype=torch.int32, device=DEV)
        o = torch.full_like(q, 7.0)
        assert status_of(lambda ws: kda.paged_attn_fwd(q, pages, pages.clone(), table, kv_lens, cu, **scales, o=o,
                                                       workspace=ws)) == code
        skipped = code[0] == kda.KDA_ERR_SEQLENS
        assert not o[:30].any() and (o[37:] == 7).all()
        assert (o[30:37] == 7).all() if skipped else not o[30:37].any()
        k = torch.full((40, 2, D), 7.0, dtype=dtype, device=DEV)
        v = k.clone()
        got = status_of(lambda ws: kda.kv_cache_write(k, v, pages, pages.clone(), table, kv_lens, cu, **scales, workspace=ws))
        assert got == code
        got = status_of(lambda ws: kda.kv_cache_read(pages, pages.clone(), table, kv_lens, cu, total_tokens=40, k=k, v=v,
                                                     **scales, workspace=ws))
        assert got == code and not k[:30].any() and not v[:30].any() and (k[37:] == 7).all()
        one = torch.full((4, 6, D), 7.0, dtype=dtype, device=DEV)
        assert status_of(lambda ws: kda.paged_attn_decode_step(q[:4], pages, pages.clone(), table, kv_lens, **scales, o=one,
                                                               workspace=ws)) == code
        assert not one[:3].any() and ((one[3] == 7).all() if skipped else not one[3].any())


def test_small_weights_beside_a_large_one():
    """One key whose weight is 2^16 to 2^22 times the others' and whose value is zero in half of the channels, where
    the output is the others' sum; from e4m3 pages, where a weight is a sum of two e4m3 (off by 2^-8 of itself, or by
    2^-21 of the largest weight times scale of its 512 keys)."""
    b = U.Batch([1], [1999], 1, 64, BF, E4M3, 16, device=DEV)
    q = torch.zeros(1, 4, 64, dtype=BF, device=DEV)
    q[0, :, 0] = torch.tensor([16.0, 18.0, 20.0, 22.0], device=DEV)
    k = torch.randn(2000, 1, 64, device=DEV) * 0.05
    k[:, 0, 0] = 0
    k[777, 0, 0] = math.log(2.0)
    v = torch.randn(2000, 1, 64, device=DEV)
    v[777, 0, ::2] = 0
    kda.kv_cache_write(k.to(BF), v.to(BF), *b.cache, torch.tensor([0, 2000], dtype=torch.int32, device=DEV),
                       **b.scales, check=True)
    got = kda.paged_attn_decode_step(q, *b.cache, **b.scales, check=True).double()
    want, size = U.attention(b, q)
    page, slot = b.table[0, torch.arange(2000, device=DEV) // 16].long(), torch.arange(2000, device=DEV) % 16
    keys = U.values(b.k_pages, b.k_scales)[page, 0, slot]
    scale, byte = b.v_scales[page, 0, slot].double(), b.v_pages[page, 0, slot].double().abs()
    w = torch.softmax(q[0].double() @ keys.T, -1)                                    # [4, 2000]
    floor = 2.0 ** -21 * (w * scale).amax(-1, keepdim=True) * byte.sum(0)[None]      # [4, 64]
    slack = 2.0 ** -8 * (want.abs() + size) + 2e-5 * size + floor[None] + 1e-30
    assert ((got - want).abs() <= slack).all()


@pytest.mark.parametrize("shift", [-93, 90])
def test_scales_far_from_one(shift):
    """Values whose scales are 2^-101 to 2^-99, and around 2^83, through every call."""
    b = U.Batch([40, 1], [700, 2000], 2, 64, BF, E4M3, 16, device=DEV)
    far = b.v_scales * 2.0 ** shift
    assert 2.0 ** -101 <= far[far.isfinite()].min() and far[far.isfinite()].max() < 2.0 ** 100
    q, back = b.queries(8), 2.0 ** -shift
    scales = dict(k_scales=b.k_scales, v_scales=far)
    U.check_attention(kda.paged_attn_fwd(q, *b.cache, b.cu, **scales, check=True).double() * back, b, q)
    _, v = kda.kv_cache_read(*b.cache, b.cu, total_tokens=41, **b.scales, check=True)
    _, w = kda.kv_cache_read(*b.cache, b.cu, total_tokens=41, **scales, check=True)
    assert torch.equal(v.double(), w.double() * back)
    b.cu, b.T = torch.tensor([0, 1, 2], dtype=torch.int32, device=DEV), 2
    q = q[39:].contiguous()
    U.check_attention(kda.paged_attn_decode_step(q, *b.cache, **scales, check=True).double() * back, b, q)


@pytest.mark.parametrize("dtype,cache", KINDS)
@pytest.mark.parametrize("D", [32, 128])
@pytest.mark.parametrize("window,sinks", [(0, 0), (0, 3), (9, 2)])
def test_padding_at_the_left_in_every_type(dtype, cache, D, window, sinks):
    """Sequences of fewer tokens than rows, some of them across a tile; first tokens without a window count for nothing."""
    lens, before = [8, 300, 40, 1, 150], [-3, -290, -40, 0, -1]
    b = U.Batch(lens, before, 2, D, dtype, cache, 16, seed=D, device=DEV)
    q = b.queries(6)
    o = kda.paged_attn_fwd(q, *b.cache, b.cu, window=window, sinks=sinks, **b.scales, check=True)
    U.check_attention(o, b, q, window=window, sinks=sinks)
    k, v = kda.kv_cache_read(*b.cache, b.cu, total_tokens=b.T, **b.scales, check=True)
    for row, n, pos in U.places(b):
        if pos < 0:
            assert not o[row].any() and not k[row].any() and not v[row].any()


@pytest.mark.parametrize("dtype,cache", KINDS)
def test_windows_and_first_tokens_at_the_end_of_int32(dtype, cache):
    most = (1 << 31) - 1
    b = U.Batch([5, 200, 0, 9], [600, 13, 4, -9], 2, 64, dtype, cache, 16, device=DEV)
    q = b.queries(8)
    one = U.Batch([1] * 4, [600, 13, 0, 130], 2, 64, dtype, cache, 16, device=DEV)
    one.kv_lens[2] = 0
    p = one.queries(8)
    for window, sinks in ((most, most), (most, 0), (1, most)):
        o = kda.paged_attn_fwd(q, *b.cache, b.cu, window=window, sinks=sinks, **b.scales, check=True)
        U.check_attention(o, b, q)
        o = kda.paged_attn_decode_step(p, *one.cache, window=window, sinks=sinks, **one.scales, check=True)
        U.check_attention(o, one, p)


@pytest.mark.parametrize("cache", [BF, E4M3])
def test_more_tiles_than_the_plan_keeps_in_shared_memory(cache):
    """Chunks of 1 to 4 tiles of 256 rows, more than 4096 in all, over fewer and over more than 2048 sequences."""
    for N, most in ((2000, 60), (3000, 30)):
        lens = [1 + (7 * n) % most for n in range(N)]
        assert sum(-(-16 * m // 256) for m in lens) > 4096
        b = U.Batch(lens, [(5 * n) % 40 for n in range(N)], 1, 32, BF, cache, 16, device=DEV)
        q = b.queries(16)
        o = kda.paged_attn_fwd(q, *b.cache, b.cu, **b.scales, check=True)
        U.check_attention(o, b, q)


@pytest.mark.parametrize("cache", [BF, E4M3])
@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("T", [512, 29184])
@pytest.mark.parametrize("grow", [False, True])
def test_chunks_behind_millions_of_tokens(cache, D, T, grow):
    """4 M tokens in two pages, over and over: a sum that is added up block after block must not lose what is
    small beside it (32768 blocks; the tensor cores cut off what does not fit, which took 2.4 % off in one
    sum). With 512 new tokens the SMs share items, with 29184 they have three each. `grow`: the second half's
    first page brings a score that everything before is small beside."""
    H, ps, width = 4, 1024, 4096
    gen = torch.Generator(device=DEV).manual_seed(D)
    k = torch.randn(2, 1, ps, D, device=DEV, generator=gen)
    v = 1.0 + 0.25 * torch.randn(2, 1, ps, D, device=DEV, generator=gen)
    q = torch.randn(T, H, D, device=DEV, generator=gen) * (2.0 * D ** -0.5)
    if grow:
        q.zero_()
        q[:, :, 0] = torch.tensor([3.5, 4.0, 4.5, 5.0], device=DEV)
        k[:, :, :, 0] = 0
        k[1, 0, 5, 0] = 2.25
    scales = {}
    if cache is E4M3:
        scales = dict(k_scales=torch.full((2, 1, ps), 2.0 ** -6, device=DEV), v_scales=torch.full((2, 1, ps), 2.0 ** -6, device=DEV))
        k, v = k * 64, v * 64
    k, v, q = k.to(cache), v.to(cache), q.to(BF)
    half = 3 * width // 4
    table = (torch.arange(width, device=DEV) >= half).to(torch.int32)[None].contiguous()
    lens = torch.tensor([width * ps], dtype=torch.int32, device=DEV)
    cu = torch.tensor([0, T], dtype=torch.int32, device=DEV)
    o = kda.paged_attn_fwd(q, k, v, table, lens, cu, **scales, check=True)
    rows = torch.cat([torch.arange(0, T, max(1, T // 300)), torch.tensor([T - 1])]).to(DEV)
    keys, vals = (U.values(t, scales.get(n)).reshape(2 * ps, D) for t, n in ((k, "k_scales"), (v, "v_scales")))
    # how often a token sees each of the 2048 different keys
    seen = width * ps - T + rows + 1 - half * ps
    times = torch.cat([torch.full((len(rows), ps), float(half), device=DEV, dtype=torch.float64),
                       (seen[:, None] // ps + (torch.arange(ps, device=DEV) < seen[:, None] % ps)).double()], 1)
    w = torch.einsum("thd,jd->thj", q[rows].double(), keys)
    w = times[:, None] * torch.exp(w - w.amax(-1, keepdim=True))
    want = torch.einsum("thj,jd->thd", w / w.sum(-1, keepdim=True), vals)
    size = torch.einsum("thj,jd->thd", w / w.sum(-1, keepdim=True), vals.abs())
    # as check_attention, and the sums' own: 256 blocks of 8 products each, at most 2^-23 of the sum cut off a product,
    # then 128 such sums at 2^-24; a sum of weights of 32768 blocks, 2^-24 of it a block at most.
    slack = 2.0 ** -8 * (want.abs() + size) + (2e-5 + 2048 * 2.0 ** -23 + (128 + 32768) * 2.0 ** -24) * size
    off = (o[rows].double() - want).abs() - slack
    assert o.isfinite().all() and off.max() <= 0, f"{off.max():.3e} over; mean off by {((o[rows].double() - want) / want).mean():.2e}"


def test_an_item_that_takes_longer_than_a_wait():
    """2^28 tokens, one page over and over, and as many items as SMs: 2097152 blocks each, 2.9 s, where a wait ends
    after 2.2. Whoever waits for an item's end has to wait longer."""
    H, D, ps, T, width = 4, 64, 1024, 9728, 1 << 18
    gen = torch.Generator(device=DEV).manual_seed(3)
    k = torch.randn(1, 1, ps, D, device=DEV, generator=gen).to(BF)
    v = (1.0 + 0.25 * torch.randn(1, 1, ps, D, device=DEV, generator=gen)).to(BF)
    q = (torch.randn(T, H, D, device=DEV, generator=gen) * (2.0 * D ** -0.5)).to(BF)
    table = torch.zeros(1, width, dtype=torch.int32, device=DEV)
    lens = torch.tensor([width * ps], dtype=torch.int32, device=DEV)
    cu = torch.tensor([0, T], dtype=torch.int32, device=DEV)
    o = kda.paged_attn_fwd(q, k, v, table, lens, cu, check=True)
    rows = torch.arange(0, T, 31, device=DEV)
    w = torch.softmax(torch.einsum("thd,jd->thj", q[rows].double(), k[0, 0].double()), -1)
    want, size = (torch.einsum("thj,jd->thd", w, x) for x in (v[0, 0].double(), v[0, 0].double().abs()))
    # as check_attention; 256 blocks of 8 products, 2^-23 of the sum each; 8192 such sums, of values and of weights, at 2^-24; a
    # token sees 262134 to 262144 whole pages and part of one more: 1 / 262134 of a weight
    slack = 2.0 ** -8 * (want.abs() + size) + (2e-5 + 2048 * 2.0 ** -23 + 2 * 8448 * 2.0 ** -24 + 4e-6) * size
    assert o.isfinite().all() and ((o[rows].double() - want).abs() <= slack).all()


@pytest.mark.parametrize("decode", [False, True])
def test_an_expired_wait_is_reported_with_a_wide_table(decode):
    """A table with room for 2^25 tokens: single tokens' waits for an item's end have twice the limit, and end as well."""
    b = U.Batch([1, 1] if decode else [200, 9], [3000, 900], 2, 128, BF, BF, 16, device=DEV)
    wide = torch.full((2, 1 << 21), 1 << 30, dtype=torch.int32, device=DEV)
    wide[:, :b.table.shape[1]] = b.table
    q = b.queries(8)
    ws = torch.zeros(1 << 26, dtype=torch.uint8, device=DEV)

    def call():
        if decode:
            return kda.paged_attn_decode_step(q, b.k_pages, b.v_pages, wide, b.kv_lens, workspace=ws)
        return kda.paged_attn_fwd(q, b.k_pages, b.v_pages, wide, b.kv_lens, b.cu, workspace=ws)
    good = call()
    U.check_attention(good, b, q)
    assert kda.load().kda_test_paged_fault(2) == kda.KDA_OK
    call()
    assert kda.query_status(ws) == (kda.KDA_ERR_TIMEOUT, 2)
    assert torch.equal(call(), good) and kda.query_status(ws)[0] == kda.KDA_OK


@pytest.mark.parametrize("cache", [F32, E4M3])
@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("T", [40, 2432])
def test_chunks_in_fp32_behind_a_million_tokens(cache, D, T):
    """8192 keys over and over, with weights of very different sizes: one sum of a million of them leaves out what is
    small beside it (3.7e-4 at most, 9e-5 on average). With 40 new tokens 64 CTAs share the keys, with 2432 few or none do."""
    H, ps, width, pages = 4, 1024, 1024, 8
    gen = torch.Generator(device=DEV).manual_seed(D)
    k = torch.randn(pages, 1, ps, D, device=DEV, generator=gen)
    v = 1.0 + 0.25 * torch.randn(pages, 1, ps, D, device=DEV, generator=gen)
    q = torch.randn(T, H, D, device=DEV, generator=gen) * (2.0 * D ** -0.5)
    scales = {}
    if cache is E4M3:
        scales = dict(k_scales=torch.full((pages, 1, ps), 2.0 ** -6, device=DEV),
                      v_scales=torch.full((pages, 1, ps), 2.0 ** -6, device=DEV))
        k, v = (k * 64).to(cache), (v * 64).to(cache)
    table = (torch.arange(width, device=DEV) % pages).to(torch.int32)[None].contiguous()
    lens = torch.tensor([width * ps], dtype=torch.int32, device=DEV)
    cu = torch.tensor([0, T], dtype=torch.int32, device=DEV)
    o = kda.paged_attn_fwd(q, k, v, table, lens, cu, **scales, check=True)
    rows = torch.arange(0, T, max(1, T // 150), device=DEV)
    keys, vals = (U.values(t, scales.get(n)).reshape(pages * ps, D) for t, n in ((k, "k_scales"), (v, "v_scales")))
    seen = width * ps - T + rows + 1
    times = (seen[:, None] // (pages * ps) + (torch.arange(pages * ps, device=DEV) < seen[:, None] % (pages * ps))).double()
    w = torch.einsum("thd,jd->thj", q[rows].double(), keys)
    w = times[:, None] * torch.exp(w - w.amax(-1, keepdim=True))
    want, size = (torch.einsum("thj,jd->thd", w / w.sum(-1, keepdim=True), x) for x in (vals, vals.abs()))
    # check_attention's 2e-5 of the sum of |w v|: half of it for the exponents, half for sums of 8192 keys, each of
    # which rounds by 2^-25 of the sum so far: sqrt(8192) * 2^-25 = 2.7e-6 where they fall either way
    off = (o[rows].double() - want).abs() - 2e-5 * size
    assert o.isfinite().all() and off.max() <= 0, f"{off.max():.3e} over; mean off by {((o[rows].double() - want) / want).mean():.2e}"


@pytest.mark.parametrize("dtype,cache", KINDS)
@pytest.mark.parametrize("window,sinks", [(0, 0), (70000, 130), (40000, 20000)])
def test_long_items_of_random_pages(dtype, cache, window, sinks):
    """Contexts of 90000 tokens whose pages are all different, items that are not shared between SMs: joined links, through
    a window and first tokens too."""
    H, Hk, D, ps, ctx = 4, 1, 64, 64, 90000
    T = 9728 if dtype is BF else 2432
    gen = torch.Generator(device=DEV).manual_seed(window)
    pages = -(-ctx // ps)
    scales, pools = {}, []
    for name in ("k_scales", "v_scales"):
        x = torch.randn(pages, Hk, ps, D, device=DEV, generator=gen)
        x[-1, :, ctx % ps:] = math.nan
        if cache is E4M3:
            scales[name] = torch.exp2(torch.randint(-8, -4, (pages, Hk, ps), device=DEV, generator=gen).float())
            pools.append((x * 64).to(cache))
        else:
            pools.append(x.to(cache))
    table = torch.randperm(pages, device=DEV, generator=gen).to(torch.int32)
    k, v = (torch.empty_like(x.view(torch.uint8)).index_copy_(0, table.long(), x.view(torch.uint8)).view(cache) for x in pools)
    stored = {n: torch.empty_like(s).index_copy_(0, table.long(), s) for n, s in scales.items()}
    q = (torch.randn(T, H, D, device=DEV, generator=gen) * (2.0 * D ** -0.5)).to(dtype)
    o = kda.paged_attn_fwd(q, k, v, table[None].contiguous(), torch.tensor([ctx], dtype=torch.int32, device=DEV),
                           torch.tensor([0, T], dtype=torch.int32, device=DEV), window=window, sinks=sinks, **stored, check=True)
    rows = torch.cat([torch.arange(0, T, max(1, T // 60)), torch.tensor([T - 1])]).to(DEV)
    keys, vals = (U.values(x, scales.get(n)).reshape(-1, D)[:ctx] for x, n in zip(pools, ("k_scales", "v_scales")))
    pos, j = ctx - T + rows[:, None], torch.arange(ctx, device=DEV)[None]
    see = j <= pos
    if window:
        see &= (j > pos - window) | (j < sinks)
    w = torch.einsum("thd,jd->thj", q[rows].double(), keys).masked_fill(~see[:, None], -math.inf).softmax(-1)
    want, size = (torch.einsum("thj,jd->thd", w, x) for x in (vals, vals.abs()))
    # as check_attention, and for bf16 what a link's products cut off (256 blocks of 8 products, 2^-23 of the sum each)
    slack = 2e-5 * size + 1e-30
    if dtype is BF:
        slack += 2.0 ** -8 * (want.abs() + size) + 2048 * 2.0 ** -23 * size
    assert o.isfinite().all() and ((o[rows].double() - want).abs() <= slack).all()
