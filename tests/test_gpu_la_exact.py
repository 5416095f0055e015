"""Single-precision prefill of the decayed linear attention held to single precision, with
resets and strong decays at every spacing, against the recurrence in 64 bits.

Bounds, with u = 2^-24.  A term of an output goes through about 200 roundings in a row (a score of
at most 128 products, a decay, 32 values or 128 state rows, the chunks that its state lives
through).  Each is at most u of a partial sum, which the same recurrence over absolute values
bounds; in random directions they come to sqrt(200) u = 14 u.  Every value: within 32 u of that
bound.  A whole tensor: partial sums of random products are as large as their result in the
mean, and a rounding is 0.3 u in the mean, so about sqrt(200) * 0.3 u = 2.5e-7 of the norm; four
times that."""
import pytest
import torch

from gated_delta_rule_43_gb300 import kda
from tests import la_util as U

pytestmark = pytest.mark.gpu
F32, BF = torch.float32, torch.bfloat16
DEV = "cuda"
WHOLE, EACH = 1e-6, 32 * 2.0 ** -24


def check(args, **kw):
    q, k, v, g, cu, h0 = args
    o, S = kda.la_chunk_fwd(*(None if t is None else t.to(DEV) for t in args), check=True, **kw)
    ro, rS = U.la_ref(*args)
    if q.dtype == BF:
        assert U.rel(o, ro) <= U.TOL_O[BF] and U.rel(S, rS) <= U.TOL_S
        return
    ao, aS = U.la_ref(q.abs(), k.abs(), v.abs(), g, cu, None if h0 is None else h0.abs())
    for x, ref, size in ((o, ro, ao), (S, rS, aS)):
        assert U.rel(x, ref) <= WHOLE
        assert bool(((x.cpu().double() - ref).abs() <= EACH * size).all())


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("every", [1, 2, 4, 8, 16])
@pytest.mark.parametrize("value", [-float("inf"), -1e30, -200.0, -60.0])
def test_resets_at_every_spacing(dtype, every, value):
    args = list(U.make([400, 33, 150], 3, 3, 64, 128, dtype, seed=every, speed=0.3))
    for h in range(3):
        args[3][h::every, h] = value
    check(args)


@pytest.mark.parametrize("dk,dv", [(32, 32), (64, 64), (128, 64), (128, 128)])
@pytest.mark.parametrize("lens", [[1], [130, 1, 0, 67], [2500]])
def test_single_precision(dk, dv, lens):
    check(U.make(lens, 4, 2, dk, dv, F32, seed=dk, speed=0.05))


def test_single_precision_of_resets_in_a_long_sequence():
    """Cut over many ranges: the states at the cuts see the resets too."""
    args = list(U.make([3000, 500], 2, 1, 128, 128, F32, seed=2, speed=0.02))
    args[3][::7, 0] = -float("inf")
    args[3][5::300, 1] = -float("inf")
    check(args)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("N", [1023, 1024, 1025, 3000])
def test_more_sequences_than_the_plan_keeps_beside_it(dtype, N):
    """The plan's sums stand in shared memory up to 1024 sequences, behind the workspace's header
    beyond."""
    lens = [(7 * n) % 5 for n in range(N)]
    lens[N // 2], lens[-1] = 700, 130
    check(U.make(lens, 2, 1, 32, 32, dtype, seed=N, speed=0.2))
