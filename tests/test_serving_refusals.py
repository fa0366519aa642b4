"""CPU checks of page planning and row adjustment: calls that the documentation excludes are
refused on the host before any HIP call."""
import ctypes

import pytest

import draft_selection_topk16_amd as df2
from test_steps_host import EINVAL, EUNSUPPORTED, plan, spot


@pytest.fixture(scope="module")
def lib():
    return df2.load()


def test_pools_whose_pages_a_number_of_32_bits_cannot_step_through(lib):
    """Items of pages are counted in steps of a workgroup: from 2^31 - 1024 pages on the next
    step would pass the largest int and go below zero, to places before the table."""
    assert ctypes.c_int32((1 << 31) - 1 - 256 + 1024).value < 0
    for pages in ((1 << 30) + 1, (1 << 31) - 1):
        assert plan(lib, num_pages=pages) == EUNSUPPORTED
        assert "num_pages above 2^30" in lib.dflash2_last_error().decode()


def test_lengths_go_in_place_of_lengths_only(lib):
    """ctx_out may be ctx_len; in place of the advances or the requests it would undo them for
    the next call of a loop."""
    for name, at in (("advance", spot(5)), ("n_new", spot(6))):
        assert plan(lib, ctx_out=at) == EINVAL
        assert "ctx_out must not overlap " + name in lib.dflash2_last_error().decode()
    # nor where the advances are given as the lengths too
    assert plan(lib, ctx_out=spot(4), advance=spot(4)) == EINVAL
    assert "ctx_out must not overlap advance" in lib.dflash2_last_error().decode()
