"""Host side of the calls on a paged cache at the edges of what their documentation allows.  CPU only:
no call here reaches a kernel."""
import pytest

import decode_fathom_plan_b200 as fp
from decode_fathom_plan_b200 import build as fbuild


@pytest.fixture(scope="module")
def lib():
    fbuild.build()
    return fp.load_library()


def test_wait_limit_is_kept_and_given_back(lib):
    before = fp.fathom_set_wait_limit(7)
    assert before == 500000000
    assert fp.fathom_set_wait_limit(2 ** 64 - 1) == 7
    assert fp.fathom_set_wait_limit(before) == 2 ** 64 - 1
