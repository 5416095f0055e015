"""Query/key preparation and state-pool moves against 64-bit and index-by-index answers."""
import pytest
import torch

from gated_delta_rule_43_gb300 import kda
from tests import la_util as U

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
DEV = "cuda"
# bf16: one rounding to 8 bits, at most 2^-8 of the value; fp32: a norm, a rotation and two
# scales, a few 2^-24 each, and the angle's cosine and sine
TOL = {BF: 2.0 ** -8, F32: 1e-6}


def rates(rot, base=10000.0, **kw):
    return kda.rope_inv_freq(rot, base, **kw)[0]


def run(T, Hq, Hk, D, rot, dtype, norm, layout, positions=None, weights=False, seed=0, eps=1e-6,
        spread=1.0):
    gen = torch.Generator().manual_seed(seed)
    q = (torch.randn(T, Hq, D, generator=gen) * spread).to(dtype)
    k = (torch.randn(T, Hk, D, generator=gen) * spread).to(dtype)
    w = [torch.randn(D, generator=gen) if weights else None for _ in range(2)]
    f = rates(rot) if rot else None
    if rot and positions is None:
        positions = torch.randint(0, 1 << 20, (T,), generator=gen, dtype=torch.int32)
    positions = positions if rot else None
    g = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    qo, ko = kda.qk_norm_rope(q.to(DEV), k.to(DEV), g(positions), g(f), norm=norm, layout=layout,
                              eps=eps, q_weight=g(w[0]), k_weight=g(w[1]), q_scale=0.125,
                              k_scale=-2.0, rope_scale=1.25)
    rq = U.qk_ref(q, positions, f, norm, layout, eps, w[0], 0.125, 1.25)
    rk = U.qk_ref(k, positions, f, norm, layout, eps, w[1], -2.0, 1.25)
    assert qo.dtype == dtype and qo.shape == q.shape and ko.shape == k.shape
    assert U.rel(qo, rq) <= TOL[dtype] and U.rel(ko, rk) <= TOL[dtype]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D,rot", [(32, 0), (32, 16), (32, 32), (64, 48), (64, 64), (128, 16),
                                   (128, 80), (128, 112), (128, 128)])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_sizes(dtype, D, rot, layout):
    run(37, 5, 3, D, rot, dtype, "l2", layout, seed=D + rot)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("norm", ["none", "l2", "rms"])
@pytest.mark.parametrize("weights", [False, True])
def test_norms(dtype, norm, weights):
    run(11, 4, 2, 128, 64, dtype, norm, "half", weights=weights)


@pytest.mark.parametrize("T,Hq,Hk", [(1, 1, 1), (1, 32, 8), (2, 7, 1), (3, 40, 40), (500, 8, 8),
                                     (4001, 2, 1)])
def test_tokens_and_heads(T, Hq, Hk):
    run(T, Hq, Hk, 128, 128, BF, "rms", "interleaved", seed=T)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_long_and_negative_positions_are_exact(layout):
    p = torch.tensor([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 999999937, 1 << 20], dtype=torch.int32)
    # fp64 itself carries an angle of 2^31 to 2^-22 at most: 2.4e-7, inside the tolerance
    run(7, 2, 2, 64, 64, F32, "none", layout, positions=p)


def test_scaled_rates():
    f, s = kda.rope_inv_freq(64, 10000.0, scaling="linear", factor=8.0)
    assert s == 1.0 and U.rel(f, rates(64).double() / 8) < 1e-6
    f, s = kda.rope_inv_freq(64, 10000.0, scaling="base", factor=8.0)
    r = rates(64).double()
    assert f[0] == 1.0 and abs(float(f[-1] / r[-1]) * 8 - 1) < 1e-5
    f, s = kda.rope_inv_freq(64, 10000.0, scaling="parts", factor=8.0, original_length=4096)
    turns = 4096 * r / (2 * torch.pi)
    assert torch.equal(f[turns > 32], rates(64)[turns > 32])
    assert U.rel(f[turns < 1], r[turns < 1] / 8) < 1e-6 and abs(s - 1.2079441541679836) < 1e-12


@pytest.mark.parametrize("dtype", [BF, F32])
def test_zero_and_extreme_rows(dtype):
    x = torch.randn(4, 2, 64)
    x[0] = 0.0
    x[1] *= 1e-15
    x[2] *= 1e15
    x = x.to(dtype)
    y, _ = kda.qk_norm_rope(x.to(DEV), None, None, None, norm="l2", eps=1e-12)
    assert not y[0].any()
    ref = U.qk_ref(x, None, None, "l2", "half", 1e-12, None, 1.0, 1.0)
    for t in range(1, 4):
        assert U.rel(y[t], ref[t]) <= TOL[dtype]


@pytest.mark.parametrize("dtype", [BF, F32])
def test_in_place_on_slices_of_a_fused_projection(dtype):
    T, Hq, Hk, D = 50, 6, 2, 64
    x = torch.randn(T, Hq + 2 * Hk, D).to(dtype)
    pos, f = torch.arange(T, dtype=torch.int32), rates(D)
    y = x.to(DEV)
    q, k = y[:, :Hq], y[:, Hq:Hq + Hk]
    qo, ko = kda.qk_norm_rope(q, k, pos.to(DEV), f.to(DEV), q_out=q, k_out=k)
    assert qo is q and ko is k
    assert U.rel(y[:, :Hq], U.qk_ref(x[:, :Hq], pos, f, "l2", "half", 1e-6, None, 1, 1)) <= TOL[dtype]
    assert U.rel(y[:, Hq:Hq + Hk],
                 U.qk_ref(x[:, Hq:Hq + Hk], pos, f, "l2", "half", 1e-6, None, 1, 1)) <= TOL[dtype]
    assert torch.equal(y[:, Hq + Hk:].cpu(), x[:, Hq + Hk:])
    # written into a wider buffer: what lies between is left alone
    z = torch.full((T + 2, Hq + 3, D), 9.0, dtype=dtype, device=DEV)
    kda.qk_norm_rope(x.to(DEV)[:, :Hq], None, pos.to(DEV), f.to(DEV), q_out=z[1:T + 1, 1:Hq + 1])
    assert torch.equal(z[1:T + 1, 1:Hq + 1], y[:, :Hq])
    assert (z[0] == 9).all() and (z[-1] == 9).all() and (z[:, 0] == 9).all() and (z[:, Hq + 1:] == 9).all()


def test_offsets_past_32_bits():
    T, wide, D = 34000, 1026, 64
    x = torch.zeros(T, wide, D, dtype=BF, device=DEV)
    x[-5:, 1000:1003] = torch.randn(5, 3, D, device=DEV).to(BF)
    y, _ = kda.qk_norm_rope(x[:, 1000:1003], None, None, None, q_out=x[:, 4:7])
    ref = U.qk_ref(x[-5:, 1000:1003].cpu(), None, None, "l2", "half", 1e-6, None, 1, 1)
    assert U.rel(x[-5:, 4:7], ref) <= TOL[BF]


def test_no_tokens():
    q = torch.empty(0, 3, 64, dtype=BF, device=DEV)
    a, b = kda.qk_norm_rope(q, q, None, None)
    assert a.shape == b.shape == (0, 3, 64)


# ----------------------------------------------------------------------------- pool
def idx(*x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("shape", [(9, 4), (9, 3, 32, 32), (9, 2, 128, 128), (9, 1021, 4)])
def test_copy_fork_and_clear(shape):
    pool = torch.randn(*shape, device=DEV)
    want = pool.clone()
    src, dst = [3, 3, -1, 8, 5], [0, 7, 1, 2, 5]
    for a, b in zip(src, dst):
        want[b] = want[a] if a >= 0 else 0.0
    kda.state_pool_copy(pool, idx(*src), idx(*dst), check=True)
    assert torch.equal(pool, want)
    kda.state_pool_copy(pool, idx(), idx(), check=True)
    assert torch.equal(pool, want)


def test_copies_that_break_the_rules_are_left_out():
    pool = torch.randn(8, 64, device=DEV)
    want = pool.clone()
    # 0 -> 1 and 2 -> 1 share a destination; 3 -> 4 writes what 4 -> 5 reads; 6 -> 9 and 9 -> 6
    # leave the pool, -2 is no slot; 4 -> 5 and 0 -> 7 are sound
    with pytest.raises(kda.KdaError) as e:
        kda.state_pool_copy(pool, idx(0, 2, 3, 4, 6, 9, -2, 0), idx(1, 1, 4, 5, 9, 6, 3, 7),
                            check=True)
    want[5], want[7] = want[4], want[0]
    assert e.value.code == kda.KDA_ERR_INVALID_ARG and e.value.info in (0, 1, 2, 4, 5, 6)
    assert torch.equal(pool, want)


def test_many_copies():
    P = 3000
    pool = torch.randn(P, 32, device=DEV)
    want = pool.clone()
    p = torch.randperm(P, device=DEV)
    want[p[:1500]] = want[p[1500:]]
    kda.state_pool_copy(pool, p[1500:].to(torch.int32), p[:1500].to(torch.int32), check=True)
    assert torch.equal(pool, want)


@pytest.mark.parametrize("P", [1, 2, 31, 32, 33, 200, 1024, 1025, 5000])
@pytest.mark.parametrize("kind", ["none", "all", "front", "back", "some"])
def test_compact(P, kind):
    gen = torch.Generator().manual_seed(P)
    live = {"none": torch.zeros(P, dtype=torch.bool), "all": torch.ones(P, dtype=torch.bool),
            "front": torch.arange(P) < P // 2, "back": torch.arange(P) >= P // 2,
            "some": torch.rand(P, generator=gen) < 0.6}[kind]
    pool = torch.randn(P, 2, 8, generator=gen).to(DEV)
    want, on = pool.cpu().clone(), live.tolist()
    n = sum(on)
    index = [i if x else -1 for i, x in enumerate(on)]
    for a, b in zip([i for i in range(n, P) if on[i]], [i for i in range(n) if not on[i]]):
        want[b] = want[a]
        index[a] = b
    new, count = kda.state_pool_compact(pool, live.to(DEV))
    assert count.tolist() == [n] and new.tolist() == index
    assert torch.equal(pool.cpu(), want)


def test_a_serving_loop():
    """Normalise and rotate, prefill, fork the state, decode the forks, drop one, compact."""
    H, D, P = 2, 64, 6
    gen = torch.Generator().manual_seed(1)
    x = torch.randn(40, 3 * H, D, generator=gen)
    g = -torch.rand(40, H, generator=gen) * 0.1
    f, scale = kda.rope_inv_freq(D)
    pos = torch.arange(40, dtype=torch.int32)
    q, k = (U.qk_ref(x[:, i * H:(i + 1) * H], pos, f, "l2", "half", 1e-6, None, 1, 1)
            for i in range(2))
    v = x[:, 2 * H:]
    ro, rS = U.la_ref(q, k, v, g, torch.tensor([0, 40]))
    X, G = x.to(DEV), g.to(DEV)
    Q, K = kda.qk_norm_rope(X[:, :H], X[:, H:2 * H], pos.to(DEV), f.to(DEV))
    V = X[:, 2 * H:]
    pool = torch.zeros(P, H, D, D, device=DEV)
    kda.la_chunk_fwd(Q[:39], K[:39], V[:39], G[:39],
                     torch.tensor([0, 39], dtype=torch.int32, device=DEV), final_state=pool[5:])
    kda.state_pool_copy(pool, idx(5, 5), idx(1, 3))
    o = kda.la_decode_step_indexed(*(t[39:].expand(2, H, D) for t in (Q, K)),
                                   V[39:].expand(2, H, D), G[39:].expand(2, H).contiguous(), pool,
                                   idx(3, 1))
    live = torch.tensor([False, False, False, True, False, True], device=DEV)
    new, n = kda.state_pool_compact(pool, live)
    assert new.tolist() == [-1, -1, -1, 0, -1, 1] and n.tolist() == [2]
    assert U.rel(o[0], ro[39]) <= 2e-5 and torch.equal(o[0], o[1])
    assert U.rel(pool[0], rS[0]) <= 2e-5
