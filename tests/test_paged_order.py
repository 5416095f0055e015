"""What no run of the paged attention can show, read from its source (no GPU)."""
import re

from tests.test_la_order import source, statements


def test_a_wait_on_several_barriers_orders_memory_for_the_whole_warp():
    """Each of the barriers is seen by one lane, and another lane issues the products on what has
    arrived: a vote joins them, which orders no memory, so a barrier of the warp has to stand
    behind it."""
    code = source("kda_paged_tc.cuh")
    start = code.index("bool wait_warp(uint32_t bar0")
    body = statements(code[start:])[0]
    wins = re.findall(r"__all_sync\([^;{]*\)\)\s*(\{[^}]*\}|[^;{}]*;)", body)
    assert len(wins) == 1
    assert [x.strip("{} \n") for x in statements(wins[0].strip("{}\n "))[:2]] == ["__syncwarp();", "return true;"]
