"""GPU tests of page planning and row adjustment beyond their ordinary calls: page counts
that are wrong, many rows with drafts before them."""
import pytest
import torch

import draft_selection_topk16_amd as df2
from gpu_util import say
from test_gpu_steps import check_rows, i32, on_gpu, rows_case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    df2.load()
    df2.device_error()
    yield
    torch.cuda.synchronize()


def test_pages_given_back_beyond_the_list_are_dropped():
    """A page held twice: the list takes what it has places for, the flag says so, and what lies
    behind the list stays."""
    say("pages dropped")
    for B in (2, 300, 1500):
        table = torch.arange(2 * B, dtype=torch.int32, device="cuda").view(B, 2)
        store = torch.full((2 * B,), -9, dtype=torch.int32, device="cuda")
        free, count, held = store[:B + 1], i32([2]), torch.full((B,), 2, dtype=torch.int32, device="cuda")
        gone = torch.full((B,), -1, dtype=torch.int32, device="cuda")
        start, _, _, _ = df2.plan_pages(table, held, free, count, torch.zeros_like(gone), gone, 16, 8)
        assert df2.device_error() == 8 and count.item() == B + 1 and start.tolist() == [0] * (B + 1)
        assert free.tolist() == [-9, -9] + list(range(B - 1)) and bool((store[B + 1:] == -9).all())
        assert bool((table == -1).all()) and bool((held == 0).all())


@pytest.mark.parametrize("place", [False, True])
def test_rows_lists_and_masks_in_one_region_a_sequence(place):
    """Histories behind each sequence's rows and masks behind each row of them: none of it
    overlaps, and what lies between the rows stays."""
    say("adjust regions", place)
    x, c = rows_case(71, torch.float32, 3, 4, 1003, 70, 6, "half")
    d, words = on_gpu(c), (1003 + 31) // 32
    region = torch.zeros((3, 4 * 1100 + 80), dtype=torch.int32, device="cuda")
    rows = region[:, :4400].unflatten(1, (4, 1100))
    mask, history = rows[:, :, 1040:1040 + words], region[:, 4400:4470]
    mask.copy_(d["mask"])
    history.copy_(d["history"])
    view = rows.view(torch.float32)[:, :, :1003]
    src = x.cuda()
    if place:
        view.copy_(src)
    got = df2.adjust_logits(view if place else src, **dict(d, history=history, mask=mask), out=view)
    check_rows(x, c, got)
    assert torch.equal(mask, d["mask"]) and torch.equal(history, d["history"])
    assert bool((rows[:, :, 1003:1040] == 0).all()) and bool((rows[:, :, 1040 + words:] == 0).all())


@pytest.mark.parametrize("R,V", [(37, 70001), (300, 4099), (700, 40)])
@pytest.mark.parametrize("place", [False, True])
def test_drafts_before_and_between_the_rows_of_a_workgroup(R, V, place):
    """Many rows are divided over workgroups: a draft counts from the row behind it on, in its
    own workgroup and in those of later rows, as often as it was drafted."""
    say("adjust many rows", R, V, place)
    x, c = rows_case(81 + R, torch.bfloat16, 1, R, V, 9, 4, "half")
    c["path"] = (c["path"].long() % max(V // 50, 7)).int()              # the same few words again and again
    d = x.cuda()
    check_rows(x, c, df2.adjust_logits(d, **on_gpu(c), out=d if place else None))
