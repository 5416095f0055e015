"""The refusals of the prefill's test hook (no GPU)."""
import os

import pytest

from gated_delta_rule_43_gb300 import kda


@pytest.fixture(scope="module")
def lib():
    from gated_delta_rule_43_gb300 import _build
    if not os.path.exists(kda.LIB_PATH):
        _build.build()
    return kda.load()


def test_parts_that_are_none(lib):
    assert lib.kda_test_la_fault(-2) == kda.KDA_ERR_INVALID_ARG
    assert lib.kda_test_la_fault(-1) == kda.KDA_OK
