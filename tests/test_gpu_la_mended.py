"""Cases of the decayed linear attention and the state pool that were once answered wrongly."""
import time

import pytest
import torch

from gated_delta_rule_43_gb300 import kda
from tests import la_util as U

pytestmark = pytest.mark.gpu
F32, BF = torch.float32, torch.bfloat16
DEV = "cuda"


def gpu(*ts):
    return [None if t is None else t.to(DEV) for t in ts]


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("cu", [[0, 160, 0, 160], [0, 100, 20, 160], [0, 160] * 40])
def test_sequences_that_overlap_are_not_gone_through(dtype, cu):
    """A decreasing cu_seqlens lets the sequences around it overlap: their lengths have no bound
    by the number of tokens, and neither would the work."""
    N = len(cu) - 1
    q, k, v, g, _, h0 = gpu(*U.make([160] + [0] * (N - 1), 2, 2, 64, 64, dtype, seed=3))
    o = torch.full((160, 2, 64), 7.0, dtype=dtype, device=DEV)
    at = torch.tensor(cu, dtype=torch.int32, device=DEV)
    with pytest.raises(kda.KdaError) as e:
        kda.la_chunk_fwd(q, k, v, g, at, h0, o=o, check=True)
    assert e.value.code == kda.KDA_ERR_SEQLENS
    assert (o == 7).all()


@pytest.mark.parametrize("dtype", [F32, BF])
def test_sequences_beside_an_offending_one_are(dtype):
    q, k, v, g, _, h0 = gpu(*U.make([100, 60], 2, 2, 64, 64, dtype, seed=4))
    cu = torch.tensor([0, 100, 90], dtype=torch.int32, device=DEV)
    o = torch.full((160, 2, 64), 7.0, dtype=dtype, device=DEV)
    with pytest.raises(kda.KdaError) as e:
        kda.la_chunk_fwd(q, k, v, g, cu, h0, o=o, check=True)
    assert e.value.code == kda.KDA_ERR_SEQLENS
    ro, _ = U.la_ref(*(x.cpu() for x in (q[:100], k[:100], v[:100], g[:100])),
                     torch.tensor([0, 100]), h0[:1].cpu())
    assert U.rel(o[:100], ro) <= U.TOL_O[dtype] and (o[100:] == 7).all()


def time_of(args, calls=20, turns=20):
    """The least time of a call, in us, of calls replayed from a graph."""
    q, k, v, g, cu, h0 = gpu(*args)
    o, S = torch.empty_like(v), torch.empty_like(h0)
    N, H, dk, dv = h0.shape
    ws = kda.alloc_workspace(kda.load().kda_la_chunk_fwd_workspace_size(
        q.shape[0], N, H, q.shape[1], dk, dv, kda._DT[q.dtype]), DEV)
    call = lambda: kda.la_chunk_fwd(q, k, v, g, cu, h0, o=o, final_state=S, workspace=ws)  # noqa: E731
    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(calls):
            call()
    best = float("inf")
    for _ in range(turns):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        graph.replay()
        b.record()
        torch.cuda.synchronize()
        best = min(best, a.elapsed_time(b) / calls * 1e3)
    return best


def test_column_blocks_where_few_ranges_hold_work():
    """One sequence of 600 tokens and 8 heads has as many ranges as SMs by its size and work for
    72 of them: it takes about as long as one of 575 tokens (one chunk in 18 less, and one piece
    in nine of two chunks instead of three: up to 1.3), not 1.6 times as long."""
    short, longer = (time_of(U.make([n], 8, 8, 128, 128, F32, seed=5)) for n in (575, 600))
    assert longer <= 1.4 * short


def idx(*x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def test_a_fork_may_include_its_own_slot():
    """3 -> 3 does nothing and disturbs nobody who reads slot 3."""
    pool = torch.randn(8, 2, 32, 32, device=DEV)
    want = pool.clone()
    want[5], want[0] = want[3], want[3]
    kda.state_pool_copy(pool, idx(3, 3, 3, 7), idx(3, 5, 0, 7), check=True)
    assert torch.equal(pool, want)
    with pytest.raises(kda.KdaError) as e:   # but 1 -> 3 would write it
        kda.state_pool_copy(pool, idx(3, 1, 4), idx(3, 3, 6), check=True)
    want[6] = want[4]
    assert e.value.code == kda.KDA_ERR_INVALID_ARG and e.value.info in (0, 1)
    assert torch.equal(pool, want)


@pytest.mark.parametrize("n", [2048, 2049, 20000, 100000])
def test_many_copies_with_some_that_break_the_rules(n):
    """Beyond some thousand copies they are checked by marks, with the same answers."""
    P = 2 * n
    gen = torch.Generator().manual_seed(n)
    p = torch.randperm(P, generator=gen).to(torch.int32)
    src, dst = p[:n].clone(), p[n:].clone()
    src[:50] = dst[:50]                      # to themselves
    src[50:60] = dst[:10]                    # ... and read by others
    src[100:200] = -1                        # cleared
    src[200], src[201], dst[202], dst[203] = P, -2, -1, P
    dst[300] = dst[301]                      # one destination twice
    src[400] = dst[401]                      # 401 writes what 400 reads
    bad = {200, 201, 202, 203, 300, 301, 401}
    pool = torch.randn(P, 8, generator=gen)
    want = pool.clone()
    good = torch.ones(n, dtype=torch.bool)
    good[list(bad)] = False
    s, d = src[good].long(), dst[good].long()
    want[d] = torch.where((s >= 0)[:, None], pool[s.clamp_min(0)], torch.zeros(()))
    pool = pool.to(DEV)
    with pytest.raises(kda.KdaError) as e:
        kda.state_pool_copy(pool, src.to(DEV), dst.to(DEV), check=True)
    assert e.value.code == kda.KDA_ERR_INVALID_ARG and e.value.info in bad
    assert torch.equal(pool.cpu(), want)
    pool.copy_(torch.randn(P, 8, generator=gen))
    want = pool.cpu()
    want[d] = torch.where((s >= 0)[:, None], want[s.clamp_min(0)], torch.zeros(()))
    kda.state_pool_copy(pool, src[good].to(DEV), dst[good].to(DEV), check=True)
    assert torch.equal(pool.cpu(), want)


# What a call's waits are for: nothing but its own tiles; states at cuts formed by a first pass, put
# together by the ranges behind or (in place) by a scan; states handed on from SM to SM.
WAITS = {"whole": ([17, 1, 0, 150, 96], 8, 8, 128, False), "cuts": ([4000, 300], 4, 4, 128, False),
         "scan": ([2900, 1300], 16, 4, 64, True),
         "handed": ([1300, 1500, 1250, 0, 1700, 900, 1600, 1, 1100, 2000, 1290], 16, 16, 128, False)}


@pytest.mark.parametrize("case", WAITS)
def test_expired_waits_are_reported_and_the_next_call_is_clean(case):
    """One CTA leaves out its first load of keys: its waits expire, after a second at least, the call
    ends with KDA_ERR_TIMEOUT, and the next one on the same workspace is right."""
    lens, H, Hk, D, in_place = WAITS[case]
    args = U.make(lens, H, Hk, D, D, BF, seed=30, speed=0.01)
    q, k, v, g, cu, h0 = gpu(*args)
    lib = kda.load()
    ws = kda.alloc_workspace(lib.kda_la_chunk_fwd_workspace_size(q.shape[0], len(lens), H, Hk, D, D,
                                                                 kda.KDA_BF16), DEV)

    def call():
        s = h0.clone()
        return kda.la_chunk_fwd(q, k, v, g, cu, s, final_state=s if in_place else None, workspace=ws)
    call()
    torch.cuda.synchronize()
    part = 0
    if case == "handed":   # the range before the first cut whose state is handed on: the plan's cuts
        cuts = ws[256:256 + 48 * 153].view(torch.int32).view(-1, 12)   # stand behind the status word
        handed = cuts[:, 10].nonzero()
        assert len(handed)
        part = int(handed[0]) - 1
    assert lib.kda_test_la_fault(part) == kda.KDA_OK
    t0 = time.perf_counter()
    call()
    code, info = kda.query_status(ws)
    took = time.perf_counter() - t0
    assert code == kda.KDA_ERR_TIMEOUT and 0 <= info < 1024
    assert 1.0 <= took < 20.0
    if case == "handed":   # the wait for what that CTA would have handed on ends before those behind it
        site = int(ws[4:8].view(torch.int32).item())
        assert site == 41 + 13   # (the load warp)
    o, S = call()
    assert kda.query_status(ws) == (kda.KDA_OK, 0)
    ro, rS = U.la_ref(*args)
    assert U.rel(o, ro) <= U.TOL_O[BF] and U.rel(S, rS) <= U.TOL_S


@pytest.mark.parametrize("dtype,chunk", [(BF, 128), (F32, 32)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_value_that_is_not_finite_stays_in_its_chunk_and_head(dtype, chunk, bad):
    """Chunks are products: zeros meet such a value too.  What lies before its chunk, and other heads,
    are right."""
    args = list(U.make([300, 70], 2, 1, 64, 64, dtype, seed=8, speed=0.05))
    ro, rS = U.la_ref(*args)
    args[2][200, 1] = bad
    o, S = kda.la_chunk_fwd(*gpu(*args), check=True)
    first = 200 // chunk * chunk
    assert U.rel(o[:first], ro[:first]) <= U.TOL_O[dtype]
    assert U.rel(o[:, 0], ro[:, 0]) <= U.TOL_O[dtype] and U.rel(S[:, 0], rS[:, 0]) <= U.TOL_S
    assert U.rel(o[300:], ro[300:]) <= U.TOL_O[dtype] and U.rel(S[1], rS[1]) <= U.TOL_S
    assert not torch.isfinite(o[200:300, 1]).any()
