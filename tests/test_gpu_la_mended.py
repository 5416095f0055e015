"""Cases of the decayed linear attention and the state pool that were once answered wrongly."""
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
