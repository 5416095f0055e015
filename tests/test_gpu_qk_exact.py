"""Query/key preparation held to one rounding of the stored type, on tensors that are large
enough for a mean.

bf16 has 8 significant bits: a rounding is off by up to half a unit in the last place, evenly
spread, 2^-9 to 2^-8 of the value by where it lies between powers of two; over many values
1.66e-3 in the mean.  2^-9 = 1.95e-3 leaves room for one rounding and none for a second one
(2.35e-3).  fp32, u = 2^-24: the sum of squares, its root, the factor, weight, two products
and a sum of the rotation, and cosine and sine within 2 units in the last place: ten roundings of
0.3 u in the mean, and u to 2 u of the angle: below 4 u = 2.4e-7; twice that."""
import pytest
import torch

from gated_delta_rule_43_gb300 import kda
from tests import la_util as U

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
DEV = "cuda"
BOUND = {BF: 2.0 ** -9, F32: 8 * 2.0 ** -24}


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("norm", ["none", "l2", "rms"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("D,rot", [(32, 32), (64, 48), (128, 0), (128, 128)])
def test_one_rounding(dtype, norm, layout, D, rot):
    gen = torch.Generator().manual_seed(D + rot)
    T, Hq, Hk = 700, 5, 3
    q, k = (torch.randn(T, h, D, generator=gen).to(dtype) for h in (Hq, Hk))
    qw, kw = (torch.randn(D, generator=gen) for _ in range(2))
    f = kda.rope_inv_freq(rot, 500000.0)[0] if rot else None
    pos = torch.randint(0, 1 << 20, (T,), generator=gen, dtype=torch.int32) if rot else None
    g = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    qo, ko = kda.qk_norm_rope(g(q), g(k), g(pos), g(f), norm=norm, layout=layout, q_weight=g(qw),
                              k_weight=g(kw), q_scale=D ** -0.5, k_scale=1.0, rope_scale=1.1)
    for x, y, w, scale in ((q, qo, qw, D ** -0.5), (k, ko, kw, 1.0)):
        ref = U.qk_ref(x, pos, f, norm, layout, 1e-6, w, scale, 1.1)
        assert U.rel(y, ref) <= BOUND[dtype]
