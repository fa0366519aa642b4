"""CPU checks of page planning and row adjustment: refusals on the host before any
HIP call, shapes in the binding, and the plain forms the GPU tests use."""
import ctypes

import pytest
import torch

import draft_selection_topk16_amd as df2
from draft_selection_topk16_amd.binding import Adjust, PagePool
from steps_ref import adjust_ref, pages_ref

OK, EINVAL, EUNSUPPORTED = 0, 1, 2
FAKE = 0x10000      # never dereferenced


@pytest.fixture(scope="module")
def lib():
    return df2.load()


def spot(i):
    return FAKE + i * 0x10000


def plan(lib, ctx=spot(4), advance=spot(5), n_new=spot(6), ctx_out=spot(7), start=spot(8), slots=spot(9), positions=spot(10), none=False, **kw):
    d = dict(block_table=spot(0), held=spot(1), free_list=spot(2), free_count=spot(3), table_stride=8, B=4, N=30, page_size=16,
             num_pages=50, table_width=8)
    d.update(kw)
    p = PagePool(*[d[n] for n, _ in PagePool._fields_])
    return lib.dflash2_plan_pages(None if none else ctypes.byref(p), ctx, advance, n_new, ctx_out, start, slots, positions, None)


def test_pages_refusals(lib):
    assert plan(lib, none=True) == EINVAL
    for kw, status, msg in ((dict(B=-1), EINVAL, "B and N"), (dict(N=-1), EINVAL, "B and N"), (dict(B=(1 << 20) + 1), EUNSUPPORTED, "B above"),
                            (dict(N=(1 << 30) + 1), EUNSUPPORTED, "N above"), (dict(page_size=0), EUNSUPPORTED, "page_size"),
                            (dict(page_size=24), EUNSUPPORTED, "page_size"), (dict(page_size=1 << 17), EUNSUPPORTED, "page_size"),
                            (dict(num_pages=0), EINVAL, "num_pages"), (dict(table_width=0), EINVAL, "table_width"),
                            (dict(table_stride=7), EINVAL, "table_width"), (dict(table_width=1 << 27, table_stride=1 << 27), EUNSUPPORTED, "2^30"),
                            (dict(block_table=None), EINVAL, "NULL"), (dict(free_count=None), EINVAL, "NULL"), (dict(ctx=None), EINVAL, "NULL"),
                            (dict(n_new=None), EINVAL, "NULL"), (dict(ctx_out=None), EINVAL, "NULL"), (dict(start=None), EINVAL, "NULL"),
                            (dict(held=spot(1) + 2), EINVAL, "misaligned"), (dict(slots=spot(9) + 4), EINVAL, "misaligned"),
                            (dict(n_new=spot(6) + 1), EINVAL, "misaligned"), (dict(start=spot(7) + 12), EINVAL, "overlap"),
                            (dict(ctx_out=spot(4) + 4), EINVAL, "overlap"), (dict(positions=spot(9) + 200), EINVAL, "overlap"),
                            (dict(free_list=spot(0) + 100), EINVAL, "overlap"), (dict(advance=spot(1)), EINVAL, "overlap")):
        assert plan(lib, **kw) == status, kw
        assert msg in lib.dflash2_last_error().decode(), kw
    assert plan(lib, B=0, block_table=None) == OK


def adjust(lib, logits=spot(0), out=spot(64), none=False, **kw):
    d = dict(B=2, R=3, V=100, L=10, M=2, dtype=1, seq_stride=300, row_stride=100, out_seq_stride=300, out_row_stride=100, history=spot(1),
             history_stride=10, history_len=spot(2), prompt_len=None, path=spot(3), repetition=None, frequency=None, presence=None,
             bias_token=spot(4), bias=spot(5), mask=spot(6), mask_seq_stride=12, mask_row_stride=4)
    d.update(kw)
    a = Adjust(*[d[n] for n, _ in Adjust._fields_])
    return lib.dflash2_adjust_logits(None if none else ctypes.byref(a), logits, out, None)


def test_adjust_refusals(lib):
    assert adjust(lib, none=True) == EINVAL
    for kw, status, msg in ((dict(dtype=3), EINVAL, "dtype"), (dict(B=-1), EINVAL, "B and R"), (dict(R=-1), EINVAL, "B and R"),
                            (dict(V=0), EINVAL, "V < 1"), (dict(V=(1 << 29) + 1), EUNSUPPORTED, "V above"), (dict(L=-1), EINVAL, "L and M"),
                            (dict(M=-1), EINVAL, "L and M"), (dict(L=1 << 29), EUNSUPPORTED, "L must"), (dict(logits=None), EINVAL, "NULL"),
                            (dict(out=None), EINVAL, "NULL"), (dict(out=spot(64) + 1), EINVAL, "misaligned"),
                            (dict(dtype=0, logits=spot(0) + 2), EINVAL, "misaligned"), (dict(history_len=None), EINVAL, "history_len"),
                            (dict(history_stride=9), EINVAL, "history_stride"), (dict(bias=None), EINVAL, "bias"),
                            (dict(path=spot(3) + 2), EINVAL, "aligned"), (dict(mask=spot(6) + 1), EINVAL, "aligned"),
                            (dict(row_stride=99), EINVAL, "row strides"), (dict(out_row_stride=64), EINVAL, "row strides"),
                            (dict(seq_stride=299), EINVAL, "sequence strides"), (dict(out_seq_stride=0), EINVAL, "sequence strides"),
                            (dict(out=spot(0) + 64), EINVAL, "overlap"), (dict(out=spot(0), out_seq_stride=400), EINVAL, "overlap"),
                            (dict(mask_row_stride=3), EINVAL, "mask strides"), (dict(mask_seq_stride=3), EINVAL, "mask strides"),
                            (dict(B=1 << 27, R=1 << 20, V=1, row_stride=1, out_row_stride=1, seq_stride=1 << 20, out_seq_stride=1 << 20,
                                  out=1 << 62), EUNSUPPORTED, "too large")):
        assert adjust(lib, **kw) == status, kw
        assert msg in lib.dflash2_last_error().decode(), kw
    assert adjust(lib, B=0, logits=None) == OK and adjust(lib, R=0, logits=None) == OK
    # in place and nothing to do
    assert adjust(lib, out=spot(0), history=None, path=None, M=0, mask=None) == OK


def test_binding_refuses_bad_shapes():
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    good = dict(block_table=i(3, 8), held=i(3), free_list=i(20), free_count=i(1), ctx_len=i(3), n_new=i(3), page_size=16, rows=10)
    with pytest.raises(ValueError, match="GPU tensor"):
        df2.plan_pages(**good)
    x = torch.zeros((2, 3, 50))
    for kw, msg in ((dict(history=i(2, 5)), "come together"), (dict(prompt_len=i(2)), "without history"), (dict(bias=torch.zeros((2, 4))), "come together")):
        with pytest.raises(ValueError, match="GPU tensor|" + msg):
            df2.adjust_logits(x, **kw)
    with pytest.raises(ValueError, match="logits must"):
        df2.adjust_logits(x[0])
    with pytest.raises(TypeError):
        df2.adjust_logits(x.half())
    with pytest.raises(ValueError, match="shape and dtype"):
        df2.adjust_logits(x, out=x[:, :2])
    with pytest.raises(ValueError, match="GPU tensor"):
        df2.adjust_logits(x)


def test_plain_forms():
    """By hand: pages given back and taken, and a row with every step."""
    got, flags = pages_ref([[4, 9], [2, -1]], [2, 1], [7, -1, -1, -1], 1, [20, 10], [3, 8], 16, 12, [-10, 2])
    assert flags == 0 and got["table"] == [[4, -1], [2, 9]] and got["count"] == [1] and got["free"][:2] == [7, 9]
    assert got["start"] == [0, 3, 11] and got["slots"] == [74, 75, 76, 44, 45, 46, 47, 9 * 16, 145, 146, 147, -1] and got["ctx"] == [10, 12]
    x = torch.tensor([[[2.0, -2.0, 1.0, 0.5], [2.0, -2.0, 1.0, 0.5]]])
    y, _ = adjust_ref(x, torch.tensor([[0, 0, 1]]), torch.tensor([3]), torch.tensor([1]), torch.tensor([[2]]), torch.tensor([2.0]),
                      torch.tensor([0.25]), torch.tensor([0.5]), torch.tensor([[3, 3]]), torch.tensor([[9.0, 1.0]]), torch.tensor([[[0b1101], [-1]]]))
    assert y[0, 0].tolist() == [1.0 - 0.75, -float("inf"), 1.0, 1.5]
    assert y[0, 1].tolist() == [0.25, -4.75, 0.5 - 0.75, 1.5]
