"""Calls on a paged cache at the edges of what their documentation allows: padded batch rows before
the others, waits that run out, probabilities far below the largest, sizes past 32 bits."""
import math

import numpy as np
import pytest
import torch

import decode_fathom_plan_b200 as fp
from tests import paged_oracle as po
from tests.test_paged_gpu import BF16, F16, Batch, check, check_rows, few_rows, status

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    fp.load_library()
    torch.cuda.set_device(0)
    fp.fathom_last_device_status()


# ------------------------------------------------- a shared prefix behind padded batch rows
def shared(lens, dtype=BF16, prefix=2048, H=8, G=2, d=64, page=16, seed=50):
    """A batch whose repeated reads of the prefix pass the 8 MB from which one kernel serves them all."""
    assert 4 * d * H * prefix * (len(lens) - 1) >= 8 << 20
    return Batch(lens, prefix, H, G, d, page, dtype, False, seed)


@pytest.mark.parametrize("first", [1, 2, 37])
@pytest.mark.parametrize("entry", [-7, 0, 5, 2 ** 31 - 1])
def test_prefix_of_a_batch_whose_first_rows_are_padded(first, entry):
    """An empty sequence's row of the table holds anything; the prefix is read by another's."""
    b = shared([0] * first + [2100, 0, 2049, 2048])
    b.table_t[:first] = entry
    b.attention()
    assert status() == fp.FATHOM_OK
    assert (b.out[:first] == 0).all() and (b.out[first + 1] == 0).all()
    check_rows(b, {(s, i) for s in (0, first, first + 2, first + 3) for i in (0, 7, 15)})
    one = b.out.clone()
    b.prefix = 0                                    # each sequence reads the prefix for itself
    b.attention()
    assert status() == fp.FATHOM_OK
    check_rows(b, {(s, i) for s in (0, first, first + 2, first + 3) for i in (0, 7, 15)})
    assert (one[:first] == 0).all()


@pytest.mark.parametrize("length", [-1, 5, 10 ** 6])
def test_prefix_is_not_read_by_the_row_of_a_refused_length(length):
    b = shared([2060, 2100, 2049, 2050, 2051])
    b.lens_t[0] = length
    b.table_t[0] = 3
    b.attention()
    assert status() == fp.FATHOM_ERR_INVALID_ARG
    assert (b.out[0] == 0).all()
    check_rows(b, {(s, i) for s in range(1, 5) for i in (0, 9, 15)})


def test_prefix_of_a_batch_of_padded_rows_alone():
    b = shared([2060, 2100, 2049, 2050, 2051])
    b.lens_t.zero_()
    b.table_t.fill_(-9)
    b.attention()
    assert status() == fp.FATHOM_OK                 # no entry of the table was used
    assert (b.out == 0).all()
