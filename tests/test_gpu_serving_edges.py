"""GPU tests of the serving operators at the ends of their ranges: caches and rows whose
offsets pass 32 bits, windows across workgroups, scores beyond what fp32 tells apart,
calls that run side by side."""
import pytest
import torch

import draft_selection_topk16_amd as df2
from fp4_ref import appended, fp4_case, held
from gpu_util import say
from steps_ref import adjust_ref
from target_ref import attention_ref, paged_case
from test_gpu_fp4_append import append_case
from test_gpu_fp4_attention import attend, check
from test_gpu_steps import check_rows, on_gpu, rows_case

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


def test_pages_beyond_32_bits():
    """Pages two and more GiB apart: written, attended and unpacked where they are."""
    say("fp4 far pages")
    c = append_case(21, BF, 128, 8, 2, 16, [3, 2], [5, 20], 128, True, pad=0)
    pages, size = c["k_cache"].shape[0], c["k_cache"].shape[2]
    stride = (1 << 31) // 2 + 4096
    store = torch.full((2, pages * stride), 7, dtype=torch.uint8, device="cuda")
    far = []
    for i, name in enumerate(("k_cache", "v_cache")):
        v = store[i].as_strided((pages, 2, size), (stride, size, 1))
        v.copy_(c[name])
        far.append(v)
    assert pages * stride > 1 << 32
    want = appended(c, 128, c["freq"].cpu().numpy(), False)
    q = df2.kv_append_fp4(c["k"], c["v"], far[0], far[1], c["table"], c["ctx"], c["start"], q=c["q"], q_norm=c["q_norm"], k_norm=c["k_norm"],
                          rope_freq=c["freq"])
    for v, (cache, _) in zip(far, want):
        assert (v.cpu().numpy() == cache).all()
    near = [v.contiguous() for v in far]
    out = df2.paged_attention_fp4(q, far[0], far[1], c["table"], c["ctx"], c["start"])
    assert torch.equal(out, df2.paged_attention_fp4(q, near[0], near[1], c["table"], c["ctx"], c["start"]))
    check(dict(c, q=q, k_cache=near[0], v_cache=near[1]), out)
    for a, b in zip(df2.kv_unpack_fp4(far[0], far[1], 128), df2.kv_unpack_fp4(near[0], near[1], 128)):
        assert torch.equal(torch.nan_to_num(a), torch.nan_to_num(b))
    # what lies between the pages is as it was
    assert bool((store[0, 2 * size:stride] == 7).all()) and df2.device_error() == 0


def test_rows_beyond_32_bits():
    say("adjust far rows")
    x, c = rows_case(31, BF, 3, 2, 4099, 60, 5, "half")
    stride = (1 << 30) + 8
    store = torch.zeros((2 * stride * 3,), dtype=BF, device="cuda")
    view = store.as_strided((3, 2, 4099), (2 * stride, stride, 1))
    assert view.stride(0) * 2 > 1 << 32
    view.copy_(x)
    check_rows(x, c, df2.adjust_logits(view, **on_gpu(c)))
    check_rows(x, c, df2.adjust_logits(view, **on_gpu(c), out=view))
    assert bool((store[4099:4099 + 64] == 0).all())


@pytest.mark.parametrize("dtype,D,Hq,n,window", [(BF, 128, 8, 1, 7001), (BF, 128, 8, 8, 7001), (BF, 64, 4, 3, 12345), (F32, 128, 8, 2, 9000),
                                                 (BF, 256, 4, 5, 5003), (BF, 128, 16, 8, 6007), (BF, 128, 8, 8, 20)])
def test_windows_that_begin_inside_a_page(dtype, D, Hq, n, window):
    say("fp4 windows", dtype, D, n, window)
    c = fp4_case(window, dtype, D, Hq, 2, 16, [n, n], [20003, 9])
    check(c, attend(c, window=window), window=window)
    check(c, attend(c, window=window, causal=False), False, window)
    assert df2.device_error() == 0


@pytest.mark.parametrize("n", [1, 8, 16, 70])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_scores_far_beyond_their_differences(dtype, n):
    """Scores of 10^10 and more, where the argument of the exponential is no longer told
    from its rounding: finite outputs within the bound, over either cache."""
    say("large scores", dtype, n)
    c = fp4_case(33 + n, dtype, 64, 8, 2, 16, [n], [200], garbage=False)
    big = dict(c, q=(c["q"].float() * 1e9).to(dtype))
    check(big, attend(big, scale=30.0), scale=30.0)
    d = paged_case(34 + n, dtype, 64, 8, 2, 16, [n], [200])
    d["q"] = (d["q"].float() * 1e9).to(dtype)
    out = df2.paged_attention(d["q"], d["k_cache"], d["v_cache"], d["table"], d["ctx"], d["start"], scale=30.0)
    ref, bound = attention_ref(d, 30.0)
    assert bool(torch.isfinite(out).all()) and bool(((out.cpu().double() - ref).abs() <= bound + 200 * 2.0 ** -126 * 8).all())


def test_calls_side_by_side():
    """Two streams, each with its own cache, workspace and rows, many times over: every
    call's result is that of the call alone."""
    say("serving calls side by side")
    jobs = []
    for seed, n, ctx in ((41, 1, 9000), (42, 8, 3000)):
        c = fp4_case(seed, BF, 128, 8, 2, 16, [n, n], [ctx, 77])
        x, r = rows_case(seed, BF, 4, 8, 20011, 900, 9, "few")
        a = df2.PreparedAttentionFp4(c["q"], c["k_cache"], c["v_cache"], c["table"], c["ctx"], c["start"])
        b = df2.PreparedAdjust(x.cuda(), **on_gpu(r))
        u = df2.PreparedUnpackFp4(c["k_cache"], c["v_cache"], 128)
        jobs.append((a, b, u, [a().clone(), b().clone(), u()[0].clone()], torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for a, b, u, _, side in jobs:
            with torch.cuda.stream(side):
                for call in (a, b, u):
                    call()
    torch.cuda.synchronize()
    for a, b, u, want, _ in jobs:
        assert torch.equal(a._out, want[0]) and torch.equal(b._out, want[1])
        assert torch.equal(torch.nan_to_num(u._out[0]), torch.nan_to_num(want[2]))
    assert df2.device_error() == 0


def test_a_row_at_a_time_and_all_at_once():
    """Rows of one sequence adjusted alone, with the drafts before them as history, are
    those of one call; aligned rows and rows that begin anywhere agree."""
    say("adjust row by row")
    x, c = rows_case(51, F32, 1, 6, 4097, 200, 7, "half")
    d = on_gpu(c)
    want = df2.adjust_logits(x.cuda(), **d)
    wide = torch.zeros((1, 6, 4100), device="cuda")
    wide[:, :, :4097] = x.cuda()
    assert torch.equal(df2.adjust_logits(wide[:, :, :4097], **d), want)
    n = int(c["history_len"][0])
    for t in range(6):
        text = torch.cat((c["history"][:, :n], c["path"][:, :t]), 1).cuda()
        one = df2.adjust_logits(x[:, t:t + 1].cuda(), history=text, history_len=torch.tensor([n + t], dtype=torch.int32, device="cuda"),
                                prompt_len=d["prompt_len"], mask=d["mask"][:, t:t + 1],
                                **{k: d[k] for k in ("repetition", "frequency", "presence", "bias_token", "bias")})
        assert torch.equal(one[:, 0], want[:, t])
    ref, _ = adjust_ref(x, **c)
    assert torch.equal(torch.isinf(want.cpu()), torch.isinf(ref))


def test_values_an_append_makes_are_what_attention_reads():
    """A bf16 cache filled from the unpacked 4-bit one gives the same outputs where both
    kernels round alike, and near ones elsewhere."""
    say("fp4 against bf16 pages")
    c = append_case(61, BF, 128, 8, 2, 16, [1, 1], [600, 33], 128, True, pad=0)
    df2.kv_append_fp4(c["k"], c["v"], c["k_cache"], c["v_cache"], c["table"], c["ctx"], c["start"], k_norm=c["k_norm"], rope_freq=c["freq"])
    k, v = (torch.nan_to_num(t) for t in df2.kv_unpack_fp4(c["k_cache"], c["v_cache"], 128))
    q = c["q"].contiguous()
    a = df2.paged_attention_fp4(q, c["k_cache"], c["v_cache"], c["table"], c["ctx"], c["start"]).float()
    b = df2.paged_attention(q, k, v, c["table"], c["ctx"], c["start"]).float()
    ref, bound = attention_ref(dict(c, q=q, k_cache=held(c["k_cache"], 16, 128), v_cache=held(c["v_cache"], 16, 128)), 128 ** -0.5)
    assert bool(((a - b).abs().cpu() <= 2 * bound).all())
