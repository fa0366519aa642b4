"""CPU checks of page planning and row adjustment: calls that the documentation excludes are
refused on the host before any HIP call."""
import ctypes

import pytest

import draft_selection_topk16_amd as df2
from test_steps_host import EINVAL, EUNSUPPORTED, OK, adjust, plan, spot


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


SPOTS = dict(history=1, history_len=2, path=3, bias_token=4, bias=5, mask=6, prompt_len=7, repetition=8, frequency=9, presence=10)


@pytest.mark.parametrize("name", sorted(SPOTS))
def test_rows_must_not_be_written_over_what_is_read(lib, name):
    """Two sequences of three rows of 100 bf16: 200 bytes each, 600 a sequence.  Lists that a
    row of out begins or ends in, or that lie in a row."""
    for at in (spot(64), spot(64) + 1196, spot(64) + 700, spot(64) - 4):
        assert adjust(lib, **{"prompt_len": spot(7), "repetition": spot(8), "frequency": spot(9), "presence": spot(10), name: at}) == EINVAL
        said = lib.dflash2_last_error().decode()
        assert said == "out must not overlap " + name, said
    # and in place
    assert adjust(lib, out=spot(0), **{"prompt_len": spot(7), name: spot(0) + 400}) == EINVAL
    assert "out must not overlap " + name in lib.dflash2_last_error().decode()


def test_lists_may_lie_between_rows(lib):
    """Rows of 100 bf16 that are 256 bytes apart, sequences 1024: penalties of two sequences
    (8 bytes) in every place of four bytes, in a call in place that has nothing else to do."""
    kw = dict(out=spot(0), row_stride=128, out_row_stride=128, seq_stride=512, out_seq_stride=512, history=None, path=None, M=0, mask=None)
    for at in range(-16, 2048, 4):
        hit = any(at < b * 1024 + t * 256 + 200 and at + 8 > b * 1024 + t * 256 for b in range(2) for t in range(3))
        assert adjust(lib, repetition=spot(0) + at, **kw) == (EINVAL if hit else OK), at


def test_tokens_beyond_what_a_count_holds(lib):
    far = dict(B=1, R=1 << 28, V=1, row_stride=1, out_row_stride=1, history_stride=1 << 28, out=1 << 61, M=0, mask=None)
    assert adjust(lib, L=(1 << 28) + 1, **far) == EUNSUPPORTED
    assert "together" in lib.dflash2_last_error().decode()
