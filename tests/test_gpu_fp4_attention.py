"""GPU tests of attention over a 4-bit paged cache against the fp64 form over the
values that it holds, with the bounds derived in target_ref."""
import pytest
import torch

import draft_selection_topk16_amd as df2
from fp4_ref import fp4_case, held
from gpu_util import say
from target_ref import attention_ref
from test_gpu_target import ATTENTION

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


def attend(c, **kw):
    return df2.paged_attention_fp4(c["q"], c["k_cache"], c["v_cache"], c["table"], c["ctx"], c["start"], **kw)


def check(c, out, causal=True, window=0, scale=None):
    """Against fp64 with attention_ref's bound, and what fp32 cannot hold on top of it: a
    weight p = exp(s - max) below 2^-126 may count as 0 (the exponential does not
    make denormals), and so may a product p v below that; the largest weight of a row is at
    least 1 and so is the sum that all are divided by, so an output over n keys is off by
    n 2^-126 max(1, |v|) more at most.  (Scores here lie up to hundreds apart, and one key's
    zero is then the whole output.)"""
    D = c["q"].shape[2]
    numbers = dict(c, k_cache=held(c["k_cache"], c["page"], D), v_cache=held(c["v_cache"], c["page"], D))
    ref, bound = attention_ref(numbers, D ** -0.5 if scale is None else scale, causal, window)
    table, most = c["table"].cpu().long(), c["page"] * c["table"].shape[1]
    for b, (s0, s1, ctx) in enumerate(zip(c["start"].tolist(), c["start"].tolist()[1:], c["ctx"].tolist())):
        j = torch.arange(max(0, min(ctx + s1 - s0, most)))
        v = numbers["v_cache"][table[b, j // c["page"]], :, j % c["page"]].abs()
        bound[s0:s1] += len(j) * 2.0 ** -126 * max(1.0, float(v.max()) if len(j) else 0.0)
    got = out.cpu().double()
    owned = ~torch.isnan(ref)
    err = (got - ref).abs()
    assert bool((torch.isfinite(got) | ~owned).all())
    worst = float((err / (bound + 1e-300))[owned].max()) if bool(owned.any()) else 0.0
    assert bool((err <= bound)[owned].all()), "largest error is %.3g of its bound" % worst
    return worst


# the cases of the other cache, on pages of 16 tokens at least
CASES = [c[:5] + (max(c[5], 16),) + c[6:] for c in ATTENTION] + [
    ("rows_of_15", BF, 128, 15, 1, 16, [1, 1], [700, 15], True, 0),
    ("rows_of_16", BF, 64, 32, 2, 64, [1, 1, 0], [700, 64, 9], True, 0),
    ("rows_of_17", BF, 128, 17, 1, 32, [1, 1], [700, 63], True, 0),
    ("rows_of_17_256", BF, 256, 17, 1, 32, [1, 1], [700, 63], True, 0),
    ("rows_of_33", BF, 128, 33, 1, 32, [1], [900], True, 0),
    ("one_key", BF, 128, 8, 8, 16, [1, 1, 1], [0, 0, 0], True, 0),
    ("many_decodes", BF, 128, 32, 8, 16, [1] * 150, [(37 * i) % 1111 for i in range(150)], True, 0),
    ("many_decodes_64_window", BF, 64, 8, 8, 64, [1] * 70, [(137 * i) % 3111 for i in range(70)], True, 300),
    ("decodes_f32_256", F32, 256, 8, 2, 16, [1] * 9, [(537 * i) % 3111 for i in range(9)], True, 0),
    ("long_page", BF, 128, 8, 2, 65536, [3, 1], [70000, 5], True, 0),
]


@pytest.mark.parametrize("case", CASES, ids=[c[0] for c in CASES])
def test_attention_against_fp64(case):
    name, dtype, D, Hq, Hkv, page, new, ctx, causal, window = case
    say("fp4 attention", name)
    c = fp4_case(len(name) * 101 + D, dtype, D, Hq, Hkv, page, new, ctx)
    worst = check(c, attend(c, causal=causal, window=window), causal, window)
    assert df2.device_error() == 0
    say("  worst error / bound %.3f" % worst)


@pytest.mark.parametrize("dtype,D,G", [(BF, 128, 4), (BF, 64, 8), (F32, 128, 2), (BF, 256, 1), (F32, 64, 1), (F32, 256, 3), (BF, 128, 16)])
def test_attention_over_split_keys(dtype, D, G):
    """A long context in few rows is split over workgroups and joined; one sequence of
    the batch is short, and more page ids than a workgroup holds at a time are passed."""
    say("fp4 attention splits", dtype, D, G)
    c = fp4_case(7, dtype, D, 2 * G, 2, 16, [3, 2], [30000 if D < 256 else 17000, 5])
    ws = df2.PreparedAttentionFp4(c["q"], c["k_cache"], c["v_cache"], c["table"], c["ctx"], c["start"])._keep[-1]
    assert ws.numel() > 0
    check(c, attend(c))
    # another plan
    check(c, attend(c, max_len=40))
    assert df2.device_error() == 0


@pytest.mark.parametrize("dtype,D", [(BF, 128), (BF, 64), (F32, 128), (BF, 256)])
def test_scales_far_apart_and_large_scores(dtype, D):
    """Blocks whose scales differ by 2^40 and more, in keys and values, within a position
    and between positions; scores of some hundreds."""
    say("fp4 attention scales", dtype, D)
    for n in (1, 9):
        c = fp4_case(11, dtype, D, 8, 2, 16, [n, n], [300, 41], spread=9.0)
        check(c, attend(c, scale=1e-3), scale=1e-3)
        c = fp4_case(12, dtype, D, 8, 2, 16, [n, n], [300, 41], spread=1.5)
        check(c, attend(c, scale=1.0), scale=1.0)
    # values near the ends of the scales, keys of zeros: sums of up to 2^7 keys' values with
    # weights up to 2^8, before they are divided, are fp32, so a scale of 2^108 is the last
    # whose 6 * 2^(108 + 7 + 8) stays below 2^127
    c = fp4_case(13, dtype, D, 8, 2, 16, [1, 4], [100, 41])
    scales = c["v_cache"][..., 8 * D:]
    scales.copy_(torch.where(torch.arange(scales.shape[-1], device="cuda") % 3 == 0, 7, torch.where(scales == 255, 255, 108 + 127)).to(torch.uint8))
    check(c, attend(c))
    c["k_cache"][..., :8 * D].zero_()
    check(c, attend(c))
    assert df2.device_error() == 0


def test_positions_before_the_first_and_behind_the_table():
    say("fp4 attention positions")
    for n, G in ((6, 2), (70, 4)):
        c = fp4_case(14, BF, 128, 2 * G, 2, 16, [n, 3], [-4, 20])
        out = attend(c, causal=False)
        check(c, out, False)
        assert bool((out[:4] == 0).all())
    c = fp4_case(15, BF, 64, 4, 2, 16, [3, 2], [45, 20])
    want = attend(c)
    far = dict(c, ctx=torch.tensor([(1 << 31) - 1, 20], dtype=torch.int32, device="cuda"))
    assert torch.equal(attend(far), want) and df2.device_error() == 16
    low = dict(c, ctx=torch.tensor([-(1 << 31), 20], dtype=torch.int32, device="cuda"))
    assert torch.equal(attend(low), torch.cat((torch.zeros_like(want[:3]), want[3:]))) and df2.device_error() == 0
    # a page id outside the cache reads page 0, and says so
    bad = c["table"].clone()
    bad[1, 1] = 99
    zero = c["table"].clone()
    zero[1, 1] = 0
    c["k_cache"][0, :, 8 * 64:] = 127
    c["v_cache"][0, :, 8 * 64:] = 127
    assert torch.equal(attend(dict(c, table=bad)), attend(dict(c, table=zero))) and df2.device_error() == 8
    # sequences that overlap: nothing is done
    out = torch.full_like(want, -7.0)
    attend(dict(c, start=torch.tensor([4, 0, 5], dtype=torch.int32, device="cuda")), out=out)
    assert bool((out == -7.0).all()) and df2.device_error() == 16


def test_shared_pages_strided_rows_and_pages_apart():
    """Sequences that share pages, queries and outputs that are parts of wider rows,
    pages with a gap between them."""
    say("fp4 attention strides")
    c = fp4_case(16, BF, 128, 8, 2, 16, [5, 7], [90, 120], pad_rows=3, garbage=False)
    c["table"][1, :4] = c["table"][0, :4]
    want = attend(c, out=torch.full_like(c["q"], -7.0))
    check(c, want)
    wide = torch.zeros((c["N"], 12, 128), dtype=BF, device="cuda")
    wide[:, :8] = c["q"]
    to = torch.full((c["N"], 10, 128), 3.0, dtype=BF, device="cuda")
    size = c["k_cache"].shape[2]
    far = torch.full((c["k_cache"].shape[0], 2, 2 * size + 32), 255, dtype=torch.uint8, device="cuda")
    apart = [far[:, i, :2 * size].unflatten(1, (2, size)) for i in (0, 1)]
    for a, b in zip(apart, (c["k_cache"], c["v_cache"])):
        a.copy_(b)
    out = df2.paged_attention_fp4(wide[:, :8], apart[0], apart[1], c["table"], c["ctx"], c["start"], out=to[:, 1:9])
    assert torch.equal(out[:12], want[:12]) and bool((to[12:] == 3).all()) and bool((to[:, 0] == 3).all()) and bool((to[:, 9] == 3).all())
    assert bool((want[12:] == -7).all()) and df2.device_error() == 0


def test_attention_in_a_graph_with_lengths_that_grow():
    """A captured call takes the lengths, tables and bytes of each replay."""
    say("fp4 attention graph")
    c = fp4_case(17, BF, 128, 8, 2, 16, [2, 3], [600, 90], garbage=False)
    call = df2.PreparedAttentionFp4(c["q"], c["k_cache"], c["v_cache"], c["table"], c["ctx"], c["start"])
    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    side = torch.cuda.Stream()
    for ctx in ([600, 90], [3, 0], [577, 31], [0, 89]):
        c["ctx"].copy_(torch.tensor(ctx, dtype=torch.int32))
        call._out.zero_()
        graph.replay()
        check(c, call._out)
        got = call._out.clone()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            call._out.zero_()
            assert torch.equal(call(), got)
        torch.cuda.current_stream().wait_stream(side)
    assert df2.device_error() == 0
