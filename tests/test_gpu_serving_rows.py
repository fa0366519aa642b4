"""GPU tests of page planning and row adjustment beyond their ordinary calls: page counts
that are wrong, many rows with drafts before them."""
import pytest
import torch

import draft_selection_topk16_amd as df2
from gpu_util import say
from test_gpu_steps import i32

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
