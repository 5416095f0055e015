"""The paged cache and its attention: cases that once went wrong, or that nothing looked at."""
import pytest
import torch

from gated_delta_rule_43_gb300 import kda
from tests import paged_util as U
from tests.paged_util import BF, E4M3

pytestmark = pytest.mark.gpu
DEV = "cuda"


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
