"""Refusals of the paged cache and its attention: every one comes back before anything reaches a
device, so they run without a GPU."""
import ctypes
import os
import types

import pytest
import torch

from gated_delta_rule_43_gb300 import kda
from tests import paged_util as U
from tests.test_devices_host import Library, On
from tests.test_la_host import caller

OK, INVALID, UNSUPPORTED = kda.KDA_OK, kda.KDA_ERR_INVALID_ARG, kda.KDA_ERR_UNSUPPORTED
A = 0x100000   # stand-in device addresses, never dereferenced on these paths
SIZES = dict(N=3, width=10, pages=40, ps=16, Hk=2, D=64, dtype=kda.KDA_BF16)
GOOD = dict(cu=A, lens=2 * A, table=3 * A, k=4 * A, v=5 * A, ks=None, vs=None, stride=2 * 16 * 64, ss=0, **SIZES)


@pytest.fixture(scope="module")
def lib():
    from gated_delta_rule_43_gb300 import _build
    if not os.path.exists(kda.LIB_PATH):
        _build.build()
    return kda.load()


def cache(**kw):
    assert set(kw) <= set(GOOD)
    return kda.PagedCache(*{**GOOD, **kw}.values())


BAD_CACHE = [dict(lens=None), dict(table=None), dict(k=None), dict(v=None), dict(lens=2 * A + 2),
             dict(table=3 * A + 1), dict(cu=A + 2), dict(k=4 * A + 8), dict(v=5 * A + 4), dict(v=4 * A),
             dict(stride=2047), dict(stride=2052), dict(stride=0), dict(stride=1 << 60), dict(ks=6 * A),
             dict(vs=6 * A), dict(dtype=kda.KDA_E4M3), dict(dtype=kda.KDA_E4M3, ks=6 * A, vs=7 * A, ss=31),
             dict(dtype=kda.KDA_E4M3, ks=6 * A, vs=6 * A, ss=32),
             dict(dtype=kda.KDA_E4M3, ks=6 * A + 4, vs=7 * A, ss=32), dict(dtype=kda.KDA_E4M3, ks=6 * A, vs=7 * A, ss=33),
             dict(N=-1), dict(width=-1), dict(pages=-1), dict(Hk=0), dict(Hk=-2), dict(width=1 << 27)]
BAD_TYPES = [dict(D=48), dict(D=256), dict(D=0), dict(ps=8), dict(ps=48), dict(ps=2048), dict(ps=0), dict(ps=-16),
             dict(dtype=kda.KDA_F32), dict(dtype=3), dict(dtype=-1)]


@pytest.mark.parametrize("decode", [False, True])
def test_attention(lib, decode):
    size = lib.kda_paged_attn_workspace_size
    cu = None if decode else A
    T = 3 if decode else 50

    def made(**kw):
        return ctypes.byref(cache(**{"cu": cu, **kw}))
    need = size(made(), T, 4, kda.KDA_BF16)
    assert need >= 256
    base = dict(cache=made(), q=8 * A, qs=256, o=9 * A, T=T, H=4, dtype=kda.KDA_BF16, scale=1.0, window=0,
                sinks=0, ws=10 * A, wsb=need, stream=None)
    if decode:
        del base["T"]
    call = caller(lib.kda_paged_attn_decode_step if decode else lib.kda_paged_attn_fwd, **base)
    for kw in BAD_TYPES:
        assert call(cache=made(**kw)) == UNSUPPORTED and size(made(**kw), T, 4, kda.KDA_BF16) == 0, kw
    for kw in BAD_CACHE:
        assert call(cache=made(**kw)) == INVALID, kw
    assert call(cache=None) == call(cache=made(cu=A if decode else None)) == INVALID
    for kw in (dict(H=3), dict(H=0), dict(H=-2), dict(H=1 << 20), dict(q=None), dict(o=None), dict(o=8 * A), dict(q=8 * A + 8),
               dict(o=9 * A + 4), dict(qs=255), dict(qs=258), dict(qs=-256), dict(qs=1 << 61), dict(scale=0.0),
               dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(window=-1),
               dict(sinks=-1), dict(ws=None), dict(ws=10 * A + 64), dict(wsb=need - 1), dict(wsb=0)):
        assert call(**kw) == INVALID, kw
    assert call(dtype=2) == call(dtype=kda.KDA_F32) == UNSUPPORTED
    if not decode:
        for kw in (dict(T=-1), dict(T=1 << 31), dict(T=1 << 30, H=8)):
            assert call(**kw) == INVALID and size(made(), kw["T"], kw.get("H", 4), kda.KDA_BF16) == 0, kw


def test_write_and_read(lib):
    tail = dict(ws=None, wsb=0, stream=None)

    def made(**kw):
        return ctypes.byref(cache(**kw))
    write = caller(lib.kda_kv_cache_write, cache=made(), k=8 * A, v=9 * A, T=50, dtype=kda.KDA_BF16, ks=128, vs=128,
                   **tail)
    read = caller(lib.kda_kv_cache_read, cache=made(), k=8 * A, v=9 * A, T=50, dtype=kda.KDA_BF16, **tail)
    for call in (write, read):
        for kw in BAD_TYPES:
            assert call(cache=made(**kw)) == UNSUPPORTED, kw
        for kw in BAD_CACHE:
            assert call(cache=made(**kw)) == INVALID, kw
        assert call(cache=made(cu=None)) == INVALID          # 50 tokens for three sequences
        for kw in (dict(cache=None), dict(k=None), dict(v=None), dict(k=8 * A + 8), dict(T=-1), dict(T=1 << 31),
                   dict(ws=7 * A + 8, wsb=256), dict(ws=7 * A, wsb=16)):
            assert call(**kw) == INVALID, kw
        assert call(dtype=kda.KDA_E4M3) == call(dtype=kda.KDA_F32) == UNSUPPORTED
        assert call(T=0) == OK and call(cache=made(N=0), T=0) == OK
    for kw in (dict(ks=127), dict(ks=132), dict(vs=64), dict(vs=-128), dict(vs=1 << 61)):
        assert write(**kw) == INVALID, kw
    for kw in (dict(v=8 * A), dict(k=4 * A), dict(v=5 * A), dict(k=5 * A)):
        assert read(**kw) == INVALID, kw


def test_fault_hook(lib):
    assert lib.kda_test_paged_fault(-2) == INVALID
    assert lib.kda_test_paged_fault(3) == lib.kda_test_paged_fault(-1) == OK


def test_binding_refuses_what_does_not_fit(lib):
    b = U.Batch([5, 3], [2, 0], 2, 32, U.F32, U.F32)
    e = U.Batch([5, 3], [2, 0], 2, 32, U.F32, U.E4M3)
    q, k = b.queries(4), torch.zeros(8, 2, 32)
    attn, one, write, read = (kda.paged_attn_fwd, kda.paged_attn_decode_step, kda.kv_cache_write,
                              kda.kv_cache_read)
    with pytest.raises(ValueError, match="CUDA"):
        attn(q, *b.cache, b.cu)
    with pytest.raises(ValueError, match="CUDA"):
        one(q[:2], *b.cache)
    with pytest.raises(ValueError, match="CUDA"):
        write(k, k, *b.cache, b.cu)
    with pytest.raises(ValueError, match="CUDA"):
        read(*b.cache, b.cu, total_tokens=8)
    with pytest.raises(ValueError, match="needs cu_seqlens"):
        attn(q, *b.cache, None)
    with pytest.raises(ValueError, match="8 rows for 2"):
        one(q, *b.cache)
    with pytest.raises(ValueError, match="need cu_seqlens"):
        write(k, k, *b.cache)
    with pytest.raises(ValueError, match="share"):
        attn(q[:, :3], *b.cache, b.cu)
    with pytest.raises(TypeError, match="q has dtype torch.float16"):
        attn(q.half(), *b.cache, b.cu)
    with pytest.raises(TypeError, match="the pages"):
        attn(q.bfloat16(), *b.cache, b.cu)
    with pytest.raises(ValueError, match="q has shape"):
        attn(q[:, :, :16], *b.cache, b.cu)
    with pytest.raises(ValueError, match="packed"):
        attn(q.transpose(1, 2).contiguous().transpose(1, 2), *b.cache, b.cu)
    with pytest.raises(ValueError, match="o has shape"):
        attn(q, *b.cache, b.cu, o=torch.empty(8, 4, 16))
    with pytest.raises(ValueError, match="k_scales"):
        attn(q, *e.cache, e.cu)
    with pytest.raises(ValueError, match="scales go with"):
        attn(q, *b.cache, b.cu, **e.scales)
    with pytest.raises(ValueError, match="v_pages has shape"):
        attn(q, b.k_pages, b.v_pages[:-1], b.table, b.kv_lens, b.cu)
    with pytest.raises(ValueError, match="v_pages has dtype|v_pages"):
        attn(q, b.k_pages, b.v_pages[:, :, :8], b.table, b.kv_lens, b.cu)
    with pytest.raises(TypeError, match="k_pages has dtype"):
        attn(q, b.k_pages.half(), b.v_pages.half(), b.table, b.kv_lens, b.cu)
    with pytest.raises(ValueError, match="inside a page"):
        attn(q, b.k_pages.transpose(1, 2).contiguous().transpose(1, 2), b.v_pages, b.table, b.kv_lens, b.cu)
    with pytest.raises(ValueError, match="same stride"):
        attn(q, torch.zeros(b.P, 2, 2, 16, 32)[:, 0], b.v_pages, b.table, b.kv_lens, b.cu)
    with pytest.raises(ValueError, match=r"\[P, Hk"):
        attn(q, b.k_pages[0], b.v_pages[0], b.table, b.kv_lens, b.cu)
    with pytest.raises(TypeError, match="block_table has dtype"):
        attn(q, b.k_pages, b.v_pages, b.table.long(), b.kv_lens, b.cu)
    with pytest.raises(ValueError, match="kv_lens has shape"):
        attn(q, b.k_pages, b.v_pages, b.table, b.kv_lens[:1], b.cu)
    with pytest.raises(ValueError, match="cu_seqlens has shape"):
        attn(q, b.k_pages, b.v_pages, b.table, b.kv_lens, b.cu[:2])
    with pytest.raises(ValueError, match="contiguous"):
        attn(q, b.k_pages, b.v_pages, b.table.t().contiguous().t(), b.kv_lens, b.cu)
    with pytest.raises(ValueError, match="v has shape"):
        write(k, k[:5], *b.cache, b.cu)
    with pytest.raises(ValueError, match="k has shape"):
        read(*b.cache, b.cu, total_tokens=8, k=torch.empty(7, 2, 32))
    with pytest.raises(TypeError, match="the pages"):
        read(*b.cache, b.cu, total_tokens=8, dtype=torch.bfloat16, k=torch.empty(8, 2, 32, dtype=U.BF))




@pytest.fixture
def fake(monkeypatch):
    library = Library()
    monkeypatch.setattr(kda, "_lib", library)
    monkeypatch.setattr(kda, "_current_device", lambda: 0, raising=False)
    monkeypatch.setattr(kda, "_current_raw_stream", lambda device: 0)
    monkeypatch.setattr(kda, "_raw_alloc", None)
    monkeypatch.setattr(kda, "_new", lambda like, shape, dtype, stream: torch.empty(shape, dtype=dtype))
    kda._paged_workspace_size.cache_clear()
    yield library
    kda._paged_workspace_size.cache_clear()


def every_call(device, stream=None):
    b = U.Batch([5, 3], [2, 0], 2, 32, U.F32, U.E4M3)
    on = [On(t, device) for t in (*b.cache, b.cu, b.queries(4), torch.zeros(8, 2, 32), b.k_scales, b.v_scales,
                                  b.queries(4)[:2])]
    kp, vp, table, lens, cu, q, k, ks, vs, q2 = on
    scales = dict(k_scales=ks, v_scales=vs, stream=stream)
    return [lambda: kda.paged_attn_fwd(q, kp, vp, table, lens, cu, **scales),
            lambda: kda.paged_attn_decode_step(q2, kp, vp, table, lens, **scales),
            lambda: kda.kv_cache_write(k, k, kp, vp, table, lens, cu, **scales),
            lambda: kda.kv_cache_read(kp, vp, table, lens, cu, total_tokens=8, dtype=U.F32, **scales)]


def test_calls_of_another_device_are_refused(fake):
    for call in every_call(0):
        call()
    assert len(fake.launched) == 4
    for call in every_call(1):
        with pytest.raises(ValueError, match="current"):
            call()
    for call in every_call(0, types.SimpleNamespace(device=torch.device("cuda:1"), cuda_stream=0)):
        with pytest.raises(ValueError, match="stream"):
            call()
    assert len(fake.launched) == 4


def test_scales_are_the_least_powers_of_two():
    """The restatement itself, at the borders of a scale."""
    x = torch.tensor([[448.0], [448.5], [449.0], [1.75], [1.76], [0.0], [2.0 ** -120], [3e38]])
    s = U.quantise(x)[1]
    want = [1.0, 2.0, 2.0, 2.0 ** -8, 2.0 ** -7, 1.0, 2.0 ** -100, 2.0 ** 119 if 3e38 <= 448 * 2.0 ** 119 else 2.0 ** 120]
    assert s.tolist()[:7] == want[:7] and s[7] == 2.0 ** 119


@pytest.mark.parametrize("kw", [dict(window=1 << 32), dict(window=(1 << 32) + 5), dict(window=-(1 << 32)),
                                dict(sinks=(1 << 40) + 1)])
def test_binding_refuses_what_int32_cannot_hold(lib, kw):
    b = U.Batch([5, 3], [2, 0], 2, 32, U.F32, U.F32)
    for call in (lambda: kda.paged_attn_fwd(b.queries(4), *b.cache, b.cu, **kw),
                 lambda: kda.paged_attn_decode_step(b.queries(4)[:2], *b.cache, **kw)):
        with pytest.raises(ValueError, match="below 2.31"):
            call()


def test_binding_refuses_pages_without_heads(lib):
    b = U.Batch([5, 3], [2, 0], 2, 32, U.F32, U.F32)
    with pytest.raises(ValueError, match="share 0"):
        kda.paged_attn_fwd(b.queries(4), b.k_pages[:, :0], b.v_pages[:, :0], b.table, b.kv_lens, b.cu)
