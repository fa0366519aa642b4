"""GPU test of the sampling select with its draft distributions in every launch
plan."""
import pytest
import torch

import draft_selection_topk16_amd as df2
from draft_selection_topk16_amd import synth
from gpu_util import say, to_device

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("launches", [1, 2, 3, 4])
@pytest.mark.parametrize("name", ["tiny_f32", "qwen3_4b_b1", "t27b_b8"])
def test_rows_in_every_launch_plan(name, launches):
    """Path, q, score, candidates and rows are the same bits as in the automatic plan;
    the drawn entries are q; and a captured call gives them on every replay."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    say("sample rows", name, launches)
    wl = synth.WORKLOADS[name]
    t = to_device(synth.make_inputs(wl))
    u = df2.philox_uniforms(5, 2, wl.B * wl.P).view(wl.B, wl.P)
    args = (t["logits"], t["hidden"], t["A"], t["Bt"], t["W"], t["prev"], wl.K, u)
    want = df2.select_sample(*args, temperature=0.8, rows=True)
    side = torch.cuda.Stream()
    with df2.plan(launches=launches):
        got = df2.select_sample(*args, temperature=0.8, rows=True)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        hit = got[3] == got[0][..., None]
        assert bool((hit.sum(-1) == 1).all()) and torch.equal((got[4] * hit).sum(-1), got[1])
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            call = df2.PreparedSelect(*args[:7], walk="sample", u=u, temperature=0.8, rows=True)
            call()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                call()
        for _ in range(3):
            with torch.cuda.stream(side):
                for x in (call.out_path, call.out_q, call.out_score, call.out_cand, call.out_rows):
                    x.zero_()
                graph.replay()
            side.synchronize()
            assert all(torch.equal(a, b) for a, b in zip((call.out_path, call.out_q, call.out_score, call.out_cand,
                                                          call.out_rows), want))
    assert df2.device_error() == 0
