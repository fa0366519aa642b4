"""GPU tests of how the target's side is called: flags raised beside a running
query of them, prepared calls dropped while they run on another stream."""
import pytest
import torch

import draft_selection_topk16_amd as df2
from gpu_util import say
from target_ref import paged_case

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    df2.load()
    df2.device_error()
    yield
    torch.cuda.synchronize()


def test_flags_raised_during_a_query_are_reported_later():
    """A call on another stream raises bit 3 while the flags are read: each is seen,
    in that query or in a later one."""
    say("flags beside a query")
    c = paged_case(80, BF, 64, 2, 1, 16, [2], [20], device="cuda")
    bad = c["table"].clone()
    bad[0, 1] = -1
    k = torch.zeros((2, 1, 64), dtype=BF, device="cuda")
    call = df2.PreparedAppend(k, k, c["k_cache"], c["v_cache"], bad, c["ctx"], c["start"])
    # a bit that stays raised makes the query clear something every time
    other = df2.PreparedVerify(torch.zeros((1, 2, 8), device="cuda"), torch.full((1, 1), 9, dtype=torch.int32, device="cuda"),
                               None, None, None, temperature=0.0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    lost = 0
    for i in range(400):
        other()
        with torch.cuda.stream(side):
            torch.cuda._sleep(1 + 1500 * (i % 32))
            call()
        flags = df2.device_error()
        assert flags & 32 and not flags & ~40
        side.synchronize()
        lost += not (flags | df2.device_error()) & 8
    assert lost == 0
