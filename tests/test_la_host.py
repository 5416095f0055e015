"""Refusals of the decayed linear attention, the query/key preparation and the state pool:
every one comes back before anything reaches a device, so they run without a GPU."""
import os

import pytest
import torch

from gated_delta_rule_43_gb300 import kda
from tests import la_util as U

OK, INVALID, UNSUPPORTED = kda.KDA_OK, kda.KDA_ERR_INVALID_ARG, kda.KDA_ERR_UNSUPPORTED
A = 0x100000   # stand-in device addresses, never dereferenced on these paths


@pytest.fixture(scope="module")
def lib():
    from gated_delta_rule_43_gb300 import _build
    if not os.path.exists(kda.LIB_PATH):
        _build.build()
    return kda.load()


def caller(fn, **base):
    def call(**kw):
        assert set(kw) <= set(base)
        return fn(*{**base, **kw}.values())
    return call


def test_prefill(lib):
    size = lib.kda_la_chunk_fwd_workspace_size
    need = size(300, 2, 4, 2, 64, 64, kda.KDA_BF16)
    assert need >= 256
    for bad in ((-1, 2, 4, 2, 64, 64, 1), (300, -1, 4, 2, 64, 64, 1), (300, 0, 4, 2, 64, 64, 1),
                (300, 2, 4, 3, 64, 64, 1), (300, 2, 4, 0, 64, 64, 1), (300, 2, 0, 1, 64, 64, 1),
                (300, 2, 4, 2, 48, 64, 1), (300, 2, 4, 2, 64, 256, 1), (300, 2, 4, 2, 64, 64, 2),
                (1 << 31, 2, 4, 2, 64, 64, 1), (1 << 62, 1, 1, 1, 32, 32, 0)):
        assert size(*bad) == 0
    call = caller(lib.kda_la_chunk_fwd, q=A, k=2 * A, v=3 * A, g=4 * A, cu=5 * A, N=2, T=300, H=4,
                  Hk=2, dk=64, dv=64, dtype=kda.KDA_BF16, qs=128, ks=128, vs=256, gpt=1, h0=None,
                  hT=None, o=6 * A, ws=7 * A, wsb=need, stream=None)
    assert call(dk=48) == call(dv=0) == call(dtype=2) == UNSUPPORTED
    for kw in (dict(Hk=3), dict(Hk=0), dict(H=0), dict(N=0), dict(N=-1), dict(T=-1), dict(q=None),
               dict(k=None), dict(v=None), dict(g=None), dict(cu=None), dict(o=None),
               dict(ws=None), dict(wsb=need - 1), dict(ws=7 * A + 64), dict(q=A + 8),
               dict(h0=8 * A + 4), dict(hT=8 * A + 8), dict(g=4 * A + 2), dict(qs=127),
               dict(qs=132), dict(ks=64), dict(vs=0), dict(vs=(1 << 62)), dict(o=A),
               dict(o=3 * A), dict(T=1 << 31)):
        assert call(**kw) == INVALID, kw


def test_prefill_of_more_chunks_than_can_be_counted(lib):
    size = lib.kda_la_chunk_fwd_workspace_size
    assert size(1 << 28, 1 << 22, 100, 100, 32, 32, kda.KDA_F32) > 0
    assert size(1 << 28, 1 << 24, 100, 100, 32, 32, kda.KDA_F32) == 0


def test_decode(lib):
    base = dict(q=A, k=2 * A, v=3 * A, g=4 * A, S=5 * A)
    tail = dict(H=4, Hk=2, dk=64, dv=64, dtype=kda.KDA_F32, qs=128, ks=128, vs=256, gpt=0)
    call = caller(lib.kda_la_decode_step, **base, o=6 * A, N=3, **tail, stream=None)
    pool = caller(lib.kda_la_decode_step_indexed, **base, idx=7 * A, P=9, o=6 * A, N=3, **tail,
                  ws=None, wsb=0, stream=None)
    for f in (call, pool):
        assert f(dk=16) == f(dtype=-1) == UNSUPPORTED
        for kw in (dict(Hk=3), dict(Hk=-1), dict(N=-1), dict(q=None), dict(S=None), dict(o=None),
                   dict(g=None), dict(k=2 * A + 4), dict(S=5 * A + 8), dict(g=4 * A + 1),
                   dict(qs=126), dict(vs=255), dict(ks=-128), dict(o=5 * A), dict(o=A)):
            assert f(**kw) == INVALID, kw
        assert f(N=0) == OK
    assert pool(idx=None) == pool(P=-1) == pool(idx=7 * A + 2) == INVALID
    assert pool(ws=8 * A, wsb=16) == pool(ws=8 * A + 16, wsb=256) == INVALID


def test_qk_norm_rope(lib):
    call = caller(lib.kda_qk_norm_rope, q=A, k=2 * A, qo=3 * A, ko=4 * A, T=5, Hq=4, Hk=2, D=64,
                  dtype=kda.KDA_BF16, qs=256, ks=128, qos=256, kos=128, qw=None, kw=None, norm=1,
                  eps=1e-6, q_scale=1.0, k_scale=1.0, pos=5 * A, freq=6 * A, rot=64, layout=0,
                  rope_scale=1.0, stream=None)
    assert call(D=48) == call(dtype=3) == call(rot=24) == UNSUPPORTED
    for kw in (dict(norm=3), dict(norm=-1), dict(layout=2), dict(rot=80), dict(rot=-16),
               dict(T=-1), dict(T=1 << 31), dict(Hq=0), dict(Hk=-1), dict(eps=-1.0),
               dict(eps=float("nan")), dict(eps=float("inf")), dict(q=None), dict(qo=None),
               dict(k=None), dict(ko=None), dict(pos=None), dict(freq=None), dict(qs=255),
               dict(qos=0), dict(kos=100), dict(ks=-128), dict(q=A + 2), dict(qw=7 * A + 4),
               dict(pos=5 * A + 2), dict(qo=A, qos=512), dict(ko=2 * A, kos=512), dict(qo=2 * A),
               dict(ko=A), dict(ko=3 * A)):
        assert call(**kw) == INVALID, kw
    assert call(T=0) == OK


def test_pool(lib):
    copy = caller(lib.kda_state_pool_copy, pool=A, P=4, elems=64, src=2 * A, dst=3 * A, n=2,
                  ws=None, wsb=0, stream=None)
    for kw in (dict(pool=None), dict(pool=A + 8), dict(P=-1), dict(elems=0), dict(elems=66),
               dict(elems=-4), dict(elems=1 << 60), dict(src=None), dict(dst=None), dict(n=-1),
               dict(n=1 << 25), dict(src=2 * A + 1), dict(ws=4 * A, wsb=8),
               dict(ws=4 * A + 8, wsb=256)):
        assert copy(**kw) == INVALID, kw
    assert copy(n=0) == OK
    need = lib.kda_state_pool_workspace_size(4)
    assert need > 256 and lib.kda_state_pool_workspace_size(-1) == 0
    pack = caller(lib.kda_state_pool_compact, pool=A, P=4, elems=64, live=2 * A, new=3 * A, n=4 * A,
                  ws=5 * A, wsb=need, stream=None)
    for kw in (dict(pool=None), dict(elems=2), dict(live=None), dict(new=None), dict(n=None),
               dict(ws=None), dict(wsb=need - 1), dict(ws=5 * A + 128), dict(new=3 * A + 2)):
        assert pack(**kw) == INVALID, kw


def test_binding_refuses_what_does_not_fit(lib):
    q, k, v, g, cu, h0 = U.make([5, 3], 4, 2, 32, 64, torch.float32)
    f = kda.la_chunk_fwd
    with pytest.raises(ValueError, match="CUDA"):
        f(q, k, v, g, cu, h0)
    with pytest.raises(ValueError, match="k has shape"):
        f(q, k[:7], v, g, cu)
    with pytest.raises(TypeError, match="v has dtype"):
        f(q, k, v.bfloat16(), g, cu)
    with pytest.raises(TypeError, match="q has dtype"):
        f(q.half(), k, v, g, cu)
    with pytest.raises(ValueError, match="share"):
        f(q, k, v[:, :3], g[:, :3], cu)
    with pytest.raises(ValueError, match="packed"):
        f(q.transpose(1, 2).contiguous().transpose(1, 2), k, v, g, cu)
    with pytest.raises(ValueError, match="g has shape"):
        f(q, k, v, g[:, :2], cu)
    with pytest.raises(TypeError, match="g has dtype"):
        f(q, k, v, g.double(), cu)
    with pytest.raises(TypeError, match="cu_seqlens"):
        f(q, k, v, g, cu.long())
    with pytest.raises(ValueError, match="initial_state has shape"):
        f(q, k, v, g, cu, h0[:1])
    with pytest.raises(ValueError, match="o has shape"):
        f(q, k, v, g, cu, o=torch.empty(8, 4, 32))
    with pytest.raises(ValueError, match="state has shape"):
        kda.la_decode_step(q, k, v, g, h0)
    with pytest.raises(ValueError, match="state_pool must be"):
        kda.la_decode_step_indexed(q, k, v, g, h0[0], torch.zeros(8, dtype=torch.int32))
    with pytest.raises(TypeError, match="state_idx has dtype"):
        kda.la_decode_step_indexed(q, k, v, g, h0, torch.zeros(8, dtype=torch.int64))
    pos, freq = torch.zeros(8, dtype=torch.int32), torch.ones(16)
    with pytest.raises(ValueError, match="CUDA"):
        kda.qk_norm_rope(q, k, pos, freq)
    with pytest.raises(ValueError, match="norm"):
        kda.qk_norm_rope(q, k, pos, freq, norm="layer")
    with pytest.raises(ValueError, match="together"):
        kda.qk_norm_rope(q, k, pos, None)
    with pytest.raises(TypeError, match="positions has dtype"):
        kda.qk_norm_rope(q, k, pos.long(), freq)
    with pytest.raises(ValueError, match="q_weight has shape"):
        kda.qk_norm_rope(q, k, pos, freq, q_weight=torch.ones(16))
    with pytest.raises(ValueError, match="need k"):
        kda.qk_norm_rope(q, None, pos, freq, k_weight=torch.ones(32))
    with pytest.raises(TypeError, match="state pool"):
        kda.state_pool_copy(h0.double(), pos, pos)
    with pytest.raises(ValueError, match="dst_idx has shape"):
        kda.state_pool_copy(h0, pos, pos[:3])
    with pytest.raises(TypeError, match="live has dtype"):
        kda.state_pool_compact(h0, torch.ones(2))
    with pytest.raises(ValueError, match="live has shape"):
        kda.state_pool_compact(h0, torch.ones(3, dtype=torch.bool))
    for kw in (dict(scaling="else"), dict(factor=0.5)):
        with pytest.raises(ValueError):
            kda.rope_inv_freq(64, **kw)
    with pytest.raises(ValueError):
        kda.rope_inv_freq(7)
