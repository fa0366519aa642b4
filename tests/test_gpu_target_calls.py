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


@pytest.mark.parametrize("keep_out", [True, False])
def test_memory_of_a_dropped_call_stays_while_it_runs(keep_out):
    """A prepared call made on one stream, called on another behind a long wait and
    dropped: what it uses is not handed out again before it has run."""
    say("dropped call")
    c = paged_case(81, BF, 128, 8, 2, 16, [8, 8], [2500, 900])
    args = (c["q"], c["k_cache"], c["v_cache"], c["table"], c["ctx"], c["start"])
    want = df2.paged_attention(*args)
    torch.cuda.synchronize()
    call = df2.PreparedAttention(*args)
    sizes = {t.data_ptr(): t.numel() * t.element_size() for t in (call._keep[-1], call._out)}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(60_000_000)
        out = call()
        if not keep_out:
            got = out.clone()
            del out
    del call
    taken = [torch.empty((n,), dtype=torch.uint8, device="cuda").fill_(255) for n in sizes.values() for _ in range(4)]
    busy = not side.query()
    assert not (busy and {t.data_ptr() for t in taken} & set(sizes))
    side.synchronize()
    assert torch.equal(out if keep_out else got, want)


def test_prepared_calls_on_streams_of_a_graph():
    """Captured on the capture's own stream, replayed, and called eagerly on a third."""
    say("prepared call on graph streams")
    c = paged_case(82, BF, 64, 4, 2, 16, [4, 2], [700, 90])
    args = (c["q"], c["k_cache"], c["v_cache"], c["table"], c["ctx"], c["start"])
    call = df2.PreparedAttention(*args)
    want = call().clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    side = torch.cuda.Stream()
    for _ in range(3):
        call._out.zero_()
        graph.replay()
        assert torch.equal(call._out, want)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            call._out.zero_()
            assert torch.equal(call(), want)
        torch.cuda.current_stream().wait_stream(side)
    assert df2.device_error() == 0
