"""How many copies kda_state_pool_copy takes (no GPU: refused before anything is launched)."""
import os

import pytest

from gated_delta_rule_43_gb300 import kda

A = 0x100000   # stand-in device addresses, never dereferenced


@pytest.fixture(scope="module")
def lib():
    from gated_delta_rule_43_gb300 import _build
    if not os.path.exists(kda.LIB_PATH):
        _build.build()
    return kda.load()


def test_many_copies_need_room_to_be_checked_in(lib):
    """Looked through one by one, 2^20 copies are 10^12 pairs: refused without room for marks."""
    P = 1 << 21
    room = lib.kda_state_pool_workspace_size(P)
    assert room >= 256 + 4 * P   # a header and a mark a slot

    def copy(n, ws, bytes_):
        return lib.kda_state_pool_copy(A, P, 64, 2 * A, 3 * A, n, ws, bytes_, None)
    for n in ((1 << 16) + 1, 1 << 20, 1 << 24):
        assert copy(n, None, 0) == copy(n, 4 * A, 256) == copy(n, 4 * A, room - 1) == \
            kda.KDA_ERR_INVALID_ARG
