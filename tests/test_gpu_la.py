"""Linear attention with one decay per head (prefill and single tokens) against the
token-by-token recurrence in 64 bits."""
import pytest
import torch

from gated_delta_rule_43_gb300 import kda
from tests import la_util as U

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
DEV = "cuda"


def gpu(*ts):
    return [None if t is None else t.to(DEV) for t in ts]


def check(args, ref_args=None, **kw):
    o, S = kda.la_chunk_fwd(*gpu(*args), check=True, **kw)
    ro, rS = U.la_ref(*(ref_args or args))
    assert U.rel(o, ro) <= U.TOL_O[args[2].dtype]
    assert U.rel(S, rS) <= U.TOL_S
    return o, S


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dk,dv", [(32, 32), (32, 128), (64, 64), (64, 128), (128, 32), (128, 64),
                                   (128, 128)])
def test_head_sizes(dtype, dk, dv):
    check(U.make([130, 1, 0, 67], 4, 2, dk, dv, dtype, seed=dk + dv))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("lens", [[1], [2, 0, 1], [31, 32, 33], [127, 128, 129], [255, 256, 257],
                                  [0, 0, 5, 0], [1] * 40, [640, 3]])
@pytest.mark.parametrize("decay,h0", [("token", True), ("head", False)])
def test_lengths(dtype, lens, decay, h0):
    check(U.make(lens, 2, 2, 128, 128, dtype, seed=len(lens), decay=decay, h0=h0))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("H,Hk", [(1, 1), (3, 1), (6, 3), (8, 2)])
def test_shared_heads(dtype, H, Hk):
    check(U.make([200, 77], H, Hk, 64, 64, dtype, seed=H))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("in_place", [False, True])
def test_long_sequences_in_segments(dtype, in_place):
    """Sequences of many segments beside short ones, the state kept for thousands of steps."""
    args = U.make([3000, 5, 0, 1900], 2, 1, 128, 128, dtype, seed=3, speed=0.01)
    q, k, v, g, cu, h0 = gpu(*args)
    o, S = kda.la_chunk_fwd(q, k, v, g, cu, h0, final_state=h0 if in_place else None, check=True)
    ro, rS = U.la_ref(*args)
    assert U.rel(o, ro) <= U.TOL_O[dtype]
    assert U.rel(S, rS) <= U.TOL_S
    assert (S is h0) == in_place


@pytest.mark.parametrize("lens,H,Hk,dk,dv", [([4153], 16, 4, 128, 128), ([2100, 130, 3000], 14, 7, 64, 128),
                                             ([9300, 0, 700], 16, 2, 32, 32), ([5000, 4100], 24, 8, 32, 64),
                                             ([11000], 13, 13, 64, 32)])
@pytest.mark.parametrize("h0", [True, False])
def test_many_heads_of_many_segments(lens, H, Hk, dk, dv, h0):
    """More than one cut in most heads, and ranges that start behind several of them."""
    check(U.make(lens, H, Hk, dk, dv, BF, seed=H, h0=h0, speed=0.01))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_many_heads_of_many_segments_in_place(dtype):
    args = U.make([2900, 1300], 16, 4, 64, 64, dtype, seed=12, speed=0.01)
    q, k, v, g, cu, h0 = gpu(*args)
    o, S = kda.la_chunk_fwd(q, k, v, g, cu, h0, final_state=h0, check=True)
    ro, rS = U.la_ref(*args)
    assert U.rel(o, ro) <= U.TOL_O[dtype] and U.rel(h0, rS) <= U.TOL_S


@pytest.mark.parametrize("dk", [32, 64, 128])
@pytest.mark.parametrize("h0", [True, False])
def test_single_precision_with_a_range_an_sm(dk, h0):
    check(U.make([2500, 37, 0, 600], 4, 2, dk, 128, F32, seed=dk, h0=h0, speed=0.02))


MANY = [1300, 1500, 1250, 0, 1700, 900, 1600, 1, 1100, 2000, 1290, 1410, 300, 1820]


@pytest.mark.parametrize("H,Hk,dk,dv", [(16, 16, 32, 32), (16, 4, 32, 64), (24, 8, 64, 32), (16, 16, 128, 128)])
@pytest.mark.parametrize("start", ["none", "h0", "in place"])
def test_sequences_cut_once(H, Hk, dk, dv, start):
    """Many sequences, each cut between two ranges at most."""
    lens = MANY if dk < 128 else MANY[:11]
    args = U.make(lens, H, Hk, dk, dv, BF, seed=H + dk, h0=start != "none", speed=0.01)
    q, k, v, g, cu, h0 = gpu(*args)
    for _ in range(3):
        s = None if h0 is None else h0.clone()
        o, S = kda.la_chunk_fwd(q, k, v, g, cu, s, final_state=s if start == "in place" else None, check=True)
    ro, rS = U.la_ref(*args)
    assert U.rel(o, ro) <= U.TOL_O[BF] and U.rel(S, rS) <= U.TOL_S


@pytest.mark.parametrize("dtype", [BF, F32])
def test_no_decay_and_fast_decay(dtype):
    args = list(U.make([300, 260], 3, 3, 64, 128, dtype, seed=5))
    args[3][:, 0] = 0.0          # a plain sum
    args[3][:, 1] *= 30.0        # forgets within a token or two
    args[3][:, 2] = -200.0       # keeps nothing: e^-200 is zero in fp32
    check(args)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_resets(dtype):
    """g = -inf forgets everything before a token."""
    args = list(U.make([400, 150], 2, 2, 128, 64, dtype, seed=6, speed=0.05))
    for t in (0, 1, 127, 128, 200, 201, 399, 400, 533):
        args[3][t] = -float("inf")
    o, S = check(args)
    assert torch.isfinite(o).all() and torch.isfinite(S).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_neighbours_do_not_leak(dtype, bad):
    """Non-finite values in one sequence leave the sequences packed beside it alone."""
    args = list(U.make([70, 90, 45], 2, 1, 128, 128, dtype, seed=7))
    ro, rS = U.la_ref(*args)
    for x in args[:3]:
        x[70:160] = bad
    o, S = kda.la_chunk_fwd(*gpu(*args), check=True)
    keep = torch.ones(205, dtype=torch.bool)
    keep[70:160] = False
    assert U.rel(o[keep], ro[keep]) <= U.TOL_O[dtype]
    assert U.rel(S[[0, 2]], rS[[0, 2]]) <= U.TOL_S


@pytest.mark.parametrize("dtype", [BF, F32])
def test_slices_of_a_fused_projection(dtype):
    q, k, v, g, cu, h0 = U.make([150, 33], 4, 2, 64, 64, dtype, seed=8)
    x = torch.full((183, 8 + 2, 64), float("nan"), dtype=dtype)
    x[:, :2], x[:, 2:4], x[:, 5:9] = q, k, v
    x = x.to(DEV)
    o, S = kda.la_chunk_fwd(x[:, :2], x[:, 2:4], x[:, 5:9], g.to(DEV), cu.to(DEV), h0.to(DEV),
                            check=True)
    ro, rS = U.la_ref(q, k, v, g, cu, h0)
    assert U.rel(o, ro) <= U.TOL_O[dtype] and U.rel(S, rS) <= U.TOL_S


def test_offsets_past_32_bits():
    """Tokens so far apart that element offsets do not fit 32 bits."""
    T, wide = 33000, 65664
    q, k, v, g, cu, h0 = U.make([T - 400, 400], 1, 1, 64, 64, BF, seed=9, decay="head", speed=0.5)
    x = torch.zeros(T, wide // 64, 64, dtype=BF, device=DEV)
    x[:, 100:101], x[:, 500:501], x[:, 1025:1026] = gpu(q, k, v)
    o, S = kda.la_chunk_fwd(x[:, 100:101], x[:, 500:501], x[:, 1025:1026], g.to(DEV), cu.to(DEV),
                            h0.to(DEV), check=True)
    ro, rS = U.la_ref(q[-400:], k[-400:], v[-400:], g, torch.tensor([0, 400]), h0[1:])
    assert U.rel(o[-400:], ro) <= U.TOL_O[BF] and U.rel(S[1:], rS) <= U.TOL_S


def test_no_tokens_and_no_sequences():
    args = gpu(*U.make([0, 0], 2, 2, 64, 64, BF))
    o, S = kda.la_chunk_fwd(*args, check=True)
    assert o.shape[0] == 0 and torch.equal(S, args[5])
    o, S = kda.la_chunk_fwd(*args[:5], None, check=True)
    assert not S.any()
    q, k, v, g, _, _ = args
    o, S = kda.la_chunk_fwd(q, k, v, g, torch.zeros(1, dtype=torch.int32, device=DEV), check=True)
    assert S.shape == (0, 2, 64, 64)


def test_split_calls_and_single_tokens_agree_with_one_call():
    args = U.make([260], 4, 2, 128, 128, F32, seed=10, speed=0.1)
    q, k, v, g, cu, h0 = gpu(*args)
    at = lambda n: torch.tensor([0, n], dtype=torch.int32, device=DEV)  # noqa: E731
    _, S = kda.la_chunk_fwd(q[:200], k[:200], v[:200], g[:200], at(200), h0)
    o2, S = kda.la_chunk_fwd(q[200:250], k[200:250], v[200:250], g[200:250], at(50), S)
    rows = [kda.la_decode_step(q[t:t + 1], k[t:t + 1], v[t:t + 1], g[t:t + 1], S)
            for t in range(250, 260)]
    ro, rS = U.la_ref(*args)
    assert U.rel(torch.cat([o2] + rows), ro[200:]) <= U.TOL_O[F32]
    assert U.rel(S, rS) <= U.TOL_S


def test_captured_in_a_graph():
    args = gpu(*U.make(MANY[:11], 16, 4, 64, 64, BF, seed=21, speed=0.01))
    kda.la_chunk_fwd(*args)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, S = kda.la_chunk_fwd(*args)
        o1 = kda.la_decode_step(*(x[:11].contiguous() for x in args[:4]), S)
    for seed in (22, 23):
        for x, y in zip(args, U.make(MANY[:11], 16, 4, 64, 64, BF, seed=seed, speed=0.01)):
            x.copy_(y)
        graph.replay()
        ro, rS = kda.la_chunk_fwd(*args, check=True)
        r1 = kda.la_decode_step(*(x[:11] for x in args[:4]), rS)
        assert torch.equal(o, ro) and torch.equal(S, rS) and torch.equal(o1, r1)


def test_repeatable_on_another_stream_with_a_reused_workspace():
    args = gpu(*U.make([700, 90, 1], 4, 4, 128, 128, BF, seed=11))
    N, H = 3, 4
    ws = kda.alloc_workspace(kda.load().kda_la_chunk_fwd_workspace_size(791, N, H, 4, 128, 128,
                                                                         kda.KDA_BF16), DEV)
    ws.fill_(0xAB)
    o1, S1 = kda.la_chunk_fwd(*args, workspace=ws, check=True)
    side = torch.cuda.Stream()
    q2 = torch.empty_like(args[0])
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        q2.copy_(args[0])
    o2, S2 = kda.la_chunk_fwd(q2, *args[1:], workspace=ws, stream=side)
    side.synchronize()
    assert torch.equal(o1, o2) and torch.equal(S1, S2)


def test_outputs_stay_inside_their_buffers():
    for dtype in (BF, F32):
        args = gpu(*U.make([130, 1, 0, 64], 3, 3, 64, 128, dtype, seed=12))
        T, N = 195, 4
        ob = torch.full((T + 64, 3, 128), 7.0, dtype=dtype, device=DEV)
        sb = torch.full((N + 2, 3, 64, 128), 7.0, device=DEV)
        need = kda.load().kda_la_chunk_fwd_workspace_size(T, N, 3, 3, 64, 128, kda._DT[dtype])
        wb = torch.full((need + 4096,), 0x5A, dtype=torch.uint8, device=DEV)
        kda.la_chunk_fwd(*args, o=ob[32:32 + T], final_state=sb[1:1 + N],
                         workspace=wb[2048:2048 + need], check=True)
        assert (ob[:32] == 7).all() and (ob[32 + T:] == 7).all()
        assert (sb[0] == 7).all() and (sb[-1] == 7).all()
        assert (wb[:2048] == 0x5A).all() and (wb[2048 + need:] == 0x5A).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_device_found_errors(dtype):
    q, k, v, g, cu, h0 = gpu(*U.make([100, 60], 2, 2, 64, 64, dtype, seed=13))
    g2 = g.clone()
    g2[130, 1] = 0.25
    with pytest.raises(kda.KdaError) as e:
        kda.la_chunk_fwd(q, k, v, g2, cu, h0, check=True)
    assert e.value.code == kda.KDA_ERR_DECAY_RANGE and e.value.info == 130 * 2 + 1
    g2[130, 1] = float("nan")
    with pytest.raises(kda.KdaError) as e:
        kda.la_chunk_fwd(q, k, v, g2, cu, h0, check=True)
    assert e.value.code == kda.KDA_ERR_DECAY_RANGE
    for bad in ([0, 170, 160], [0, 100, 150], [1, 100, 160], [0, -5, 160]):
        with pytest.raises(kda.KdaError) as e:
            kda.la_chunk_fwd(q, k, v, g, torch.tensor(bad, dtype=torch.int32, device=DEV), h0,
                             check=True)
        assert e.value.code == kda.KDA_ERR_SEQLENS
    o, S = kda.la_chunk_fwd(q, k, v, g, cu, h0, check=True)   # the next call is clean
    ro, rS = U.la_ref(*(x.cpu() for x in (q, k, v, g, cu, h0)))
    assert U.rel(o, ro) <= U.TOL_O[dtype]


# ------------------------------------------------------------------- single tokens
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dk,dv", [(32, 32), (32, 128), (64, 32), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("N", [1, 9])
def test_decode(dtype, dk, dv, N):
    q, k, v, g, cu, h0 = U.make([1] * N, 6, 3, dk, dv, dtype, seed=N + dk)
    g[0, 0] = -float("inf")
    ro, rS = U.la_ref(q, k, v, g, cu, h0)
    S = h0.to(DEV)
    o = kda.la_decode_step(*gpu(q, k, v, g), S)
    # one rounding of the stored output; the state is fp32 throughout
    assert U.rel(o, ro) <= (2.0 ** -9 if dtype == BF else 2e-6)
    assert U.rel(S, rS) <= 1e-6


@pytest.mark.parametrize("decay", ["token", "head"])
def test_decode_from_a_pool_and_slices(decay):
    N, H, Hk, D, P = 5, 4, 2, 64, 11
    q, k, v, g, cu, h0 = U.make([1] * N, H, Hk, D, D, BF, seed=20, decay=decay)
    x = torch.zeros(N, H + 2 * Hk, D, dtype=BF, device=DEV)
    x[:, :Hk], x[:, Hk:2 * Hk], x[:, 2 * Hk:] = gpu(q, k, v)
    pool = torch.randn(P, H, D, D, device=DEV)
    before = pool.clone()
    idx = torch.tensor([7, 0, 10, 3, 4], dtype=torch.int32)
    ro, rS = U.la_ref(q, k, v, g, cu, before.cpu()[idx.long()])
    o = kda.la_decode_step_indexed(x[:, :Hk], x[:, Hk:2 * Hk], x[:, 2 * Hk:], g.to(DEV), pool,
                                   idx.to(DEV), check=True)
    assert U.rel(o, ro) <= 2.0 ** -9 and U.rel(pool[idx.long()], rS) <= 1e-6
    rest = [i for i in range(P) if i not in idx.tolist()]
    assert torch.equal(pool[rest], before[rest])


def test_decode_skips_indices_outside_the_pool():
    N, H, D, P = 4, 2, 32, 3
    q, k, v, g, cu, h0 = gpu(*U.make([1] * N, H, H, D, D, F32, seed=21))
    pool = torch.randn(P, H, D, D, device=DEV)
    want = pool.clone()
    idx = torch.tensor([2, -1, 3, 0], dtype=torch.int32, device=DEV)
    o = torch.full((N, H, D), 5.0, device=DEV)
    with pytest.raises(kda.KdaError) as e:
        kda.la_decode_step_indexed(q, k, v, g, pool, idx, o=o, check=True)
    assert e.value.code == kda.KDA_ERR_INVALID_ARG and e.value.info in (1, 2)
    assert (o[1:3] == 5).all() and torch.equal(pool[1], want[1])
    sub = want[[2, 0]]
    o2 = kda.la_decode_step(q[::3].contiguous(), k[::3].contiguous(), v[::3].contiguous(),
                            g[::3].contiguous(), sub)
    assert torch.equal(o[::3], o2) and torch.equal(pool[[2, 0]], sub)
    kda.la_decode_step_indexed(q, k, v, g, pool, idx)   # without a status word: still skipped


def test_decode_in_a_pool_past_32_bits():
    H, D, P = 64, 128, 2200                       # 2.3e9 state values
    pool = torch.zeros(P, H, D, D, device=DEV)
    q, k, v, g, cu, h0 = U.make([1, 1], H, H, D, D, BF, seed=22)
    idx = torch.tensor([P - 1, 0], dtype=torch.int32, device=DEV)
    pool[[P - 1, 0]] = h0.to(DEV)
    o = kda.la_decode_step_indexed(*gpu(q, k, v, g), pool, idx)
    ro, rS = U.la_ref(q, k, v, g, cu, h0)
    assert U.rel(o, ro) <= 2.0 ** -9 and U.rel(pool[[P - 1, 0]], rS) <= 1e-6
    kda.state_pool_copy(pool, torch.tensor([P - 1, -1], dtype=torch.int32, device=DEV),
                        torch.tensor([P - 2, 0], dtype=torch.int32, device=DEV), check=True)
    assert torch.equal(pool[P - 2], pool[P - 1]) and not pool[0].any()


def test_decode_of_no_sequences():
    q, k, v, g, cu, h0 = gpu(*U.make([], 2, 2, 64, 64, BF))
    assert kda.la_decode_step(q, k, v, g, h0).shape == (0, 2, 64)
