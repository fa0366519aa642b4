"""GPU tests of what stands between the steps of a serving loop: pages of the next
step, and penalties, biases and masks on rows, against plain forms."""
import random

import pytest
import torch

import draft_selection_topk16_amd as df2
from gpu_util import say
from steps_ref import adjust_ref, pages_ref

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


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def pool(seed, B, page, width, most_ctx, most_new, spare, ends=0.0):
    """A consistent state: pages held cover each context and up to a block more."""
    r = random.Random(seed)
    ctx = [r.randint(0, most_ctx) for _ in range(B)]
    held = [min(width, -(-(c + r.randint(0, 16)) // page)) for c in ctx]
    ids = list(range(sum(held) + spare))
    r.shuffle(ids)
    table, at = [], 0
    for h in held:
        table.append(ids[at:at + h] + [-1] * (width - h))
        at += h
    free = ids[at:] + [-1] * at
    n = [-1 if r.random() < ends else r.randint(0, most_new) for _ in range(B)]
    return dict(table=table, held=held, free=free, count=spare, ctx=ctx, n_new=n, advance=[r.randint(0, 8) for _ in range(B)])


def check_pages(s, page, rows, advance=True, in_place=False, flags=None):
    want, raised = pages_ref(s["table"], s["held"], s["free"], s["count"], s["ctx"], s["n_new"], page, rows,
                             s["advance"] if advance else None)
    t = {k: i32([s[k]] if k == "count" else s[k]) for k in ("table", "held", "free", "count", "ctx", "n_new", "advance")}
    got = df2.plan_pages(t["table"], t["held"], t["free"], t["count"], t["ctx"], t["n_new"], page, rows,
                         advance=t["advance"] if advance else None, ctx_out=t["ctx"] if in_place else None)
    for name, x in zip(("start", "ctx", "slots", "positions"), got):
        assert x.tolist() == want[name], name
    for name in ("table", "held", "free", "count"):
        assert t[name].tolist() == want[name], name
    assert df2.device_error() == raised
    assert flags is None or raised == flags
    return want


PAGES = [
    # name, B, page, width, longest context, most new, spare pages, rows, ended
    ("one", 1, 16, 8, 100, 8, 5, 8, 0.0), ("one_nothing", 1, 16, 8, 0, 0, 1, 0, 0.0), ("four", 4, 16, 40, 600, 8, 9, 32, 0.0),
    ("page_of_one", 5, 1, 400, 300, 9, 60, 45, 0.3), ("all_ended", 9, 16, 40, 600, 8, 3, 16, 1.0),
    ("empty_pool", 30, 16, 40, 600, 30, 1, 900, 0.0), ("few_rows", 30, 16, 40, 600, 30, 99, 100, 0.1),
    ("narrow_table", 30, 16, 12, 190, 40, 99, 1300, 0.1), ("wave", 64, 32, 40, 900, 8, 64, 512, 0.1),
    ("past_a_wave", 65, 32, 40, 900, 8, 64, 512, 0.1), ("workgroup", 256, 16, 40, 600, 5, 256, 1024, 0.2),
    ("past_a_workgroup", 257, 16, 40, 600, 9, 256, 2000, 0.2), ("rows_apart", 40, 16, 300, 2000, 700, 2500, 30000, 0.1),
    ("chunks", 1024, 16, 20, 300, 4, 1100, 4096, 0.1), ("past_a_chunk", 1025, 16, 20, 300, 4, 300, 4096, 0.1),
    ("three_chunks", 2500, 16, 20, 300, 8, 1500, 12000, 0.3), ("three_chunks_apart", 2500, 64, 6, 300, 40, 2500, 60000, 0.1),
    ("four_a_thread", 4096, 16, 20, 300, 4, 4100, 12000, 0.2), ("past_four_a_thread", 4097, 16, 20, 300, 4, 1000, 4096, 0.2),
    ("many_chunks", 9000, 32, 8, 200, 9, 4000, 40000, 0.3),
]


@pytest.mark.parametrize("case", PAGES, ids=[c[0] for c in PAGES])
@pytest.mark.parametrize("advance", [True, False])
def test_pages_against_the_plain_form(case, advance):
    name, B, page, width, ctx, new, spare, rows, ends = case
    say("pages", name, advance)
    check_pages(pool(len(name) * 7 + B, B, page, width, ctx, new, spare, ends), page, rows, advance, in_place=not advance)


def test_pages_flags_and_refused_requests():
    say("pages flags")
    base = dict(table=[[3, 4, -1, -1], [5, -1, -1, -1], [0, 1, 2, 6]], held=[2, 1, 4], free=[7, 8] + [-1] * 7, count=2, ctx=[30, 16, 60],
                advance=[0, 0, 0])
    # served / pool too small for the second / table too narrow for the third / negative sums
    check_pages(dict(base, n_new=[2, 3, 4]), 16, 20, flags=0)
    check_pages(dict(base, n_new=[19, 20, 0]), 16, 60, flags=128)
    check_pages(dict(base, n_new=[1, 1, 5]), 16, 20, flags=16)
    check_pages(dict(base, n_new=[2, 3, 4], advance=[-40, -3, -1]), 16, 20, flags=0)
    check_pages(dict(base, n_new=[2**31 - 1, 3, -5]), 16, 20, flags=16)
    check_pages(dict(base, n_new=[20, 400000, 2**30 - 60], table=[r + [-1] * 4 for r in base["table"]]), 1 << 16, 20, flags=128 | 16)
    # a request with many pages ends, among others that take them up at once
    check_pages(dict(base, n_new=[30, 40, -1]), 16, 80, flags=0)


def test_pages_over_a_captured_graph_of_cycles():
    """The lengths stay on the device: every replay advances them, as eager calls do."""
    say("pages in a graph")
    s = pool(5, 70, 16, 60, 400, 0, 400)
    s["n_new"] = [8] * 70
    keys = ("table", "held", "free", "ctx", "n_new", "advance")
    t = {k: i32(s[k]) for k in keys}
    count = i32([s["count"]])
    call = df2.PreparedPages(t["table"], t["held"], t["free"], count, t["ctx"], t["n_new"], 16, 600, advance=t["advance"], ctx_out=t["ctx"])
    state = dict(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    r = random.Random(1)
    for step in range(12):
        adv = [r.randint(1, 8) for _ in range(70)]
        new = [-1 if r.random() < 0.05 else r.choice([1, 8, 8]) for _ in range(70)]
        t["advance"].copy_(i32(adv))
        t["n_new"].copy_(i32(new))
        if step % 3 == 2:
            call()
        else:
            graph.replay()
        want, _ = pages_ref(state["table"], state["held"], state["free"], state["count"], state["ctx"], new, 16, 600, adv)
        for name, x in zip(("start", "ctx", "slots", "positions"), call._out):
            assert x.tolist() == want[name], (step, name)
        assert t["table"].tolist() == want["table"] and t["held"].tolist() == want["held"] and count.item() == want["count"][0]
        state.update(table=want["table"], held=want["held"], free=want["free"], count=want["count"][0], ctx=want["ctx"])
    df2.device_error()


def rows_case(seed, dtype, B, R, V, L, M, mask, drafts=True, lo=0):
    g = torch.Generator().manual_seed(seed)
    x = (3 * torch.randn((B, R, V), generator=g)).to(dtype)
    length = torch.randint(lo, L + 1, (B,), generator=g).to(torch.int32)
    length[0] = L
    c = dict(history=(torch.rand((B, max(L, 1)), generator=g) ** 4 * V).int().clamp(max=V - 1)[:, :max(L, 1)].contiguous(),
             history_len=length, prompt_len=(torch.rand((B,), generator=g) * (length + 1)).to(torch.int32))
    if L == 0:
        c = {}
    if drafts and R > 1:
        c["path"] = (torch.rand((B, R - 1), generator=g) ** 3 * V).int().clamp(max=V - 1)
        c["path"][0, -1] = c["path"][0, 0]         # drafted twice
    c.update(repetition=0.7 + torch.rand((B,), generator=g), frequency=torch.rand((B,), generator=g) - 0.2,
             presence=torch.rand((B,), generator=g) - 0.2)
    if M:
        c["bias_token"] = torch.randint(0, V, (B, M), generator=g).int()
        c["bias_token"][:, -1] = c["bias_token"][:, 0]        # given twice
        c["bias"] = 5 * torch.randn((B, M), generator=g)
    if mask:
        words = torch.randint(-2**31, 2**31, (3, B, R, (V + 31) // 32), generator=g)
        w = words[0] if mask == "half" else words.amin(0) & words[0] & words[1] & words[2] if mask == "few" else words[0] | words[1] | words[2]
        if mask == "few":
            w = torch.where(torch.rand(w.shape, generator=g) < 0.6, torch.zeros_like(w), w)
        elif mask == "most":
            w = torch.where(torch.rand(w.shape, generator=g) < 0.6, torch.full_like(w, -1), w)
        if mask == "nothing":
            w = torch.zeros_like(w)
        c["mask"] = w.to(torch.int32)
    return x, c


def check_rows(x, c, out):
    ref, bound = adjust_ref(x, **c)
    got = out.cpu().double()
    low = torch.isinf(ref)
    assert torch.equal(got[low], ref[low])
    still = (bound == 0) & ~low
    same = got[still] == ref[still]
    assert bool((same | torch.isnan(ref[still])).all()), "values that nothing happens to changed"
    err = (got - ref).abs()[~low & ~still]
    assert bool((err <= bound[~low & ~still]).all())


def on_gpu(c):
    return {k: v.cuda() for k, v in c.items()}


ROWS = [
    # name, dtype, B, R, V, L, M, mask
    ("one", BF, 1, 1, 1, 3, 1, None), ("tiny", BF, 2, 3, 37, 40, 5, "half"), ("word", F32, 2, 2, 32, 9, 0, "most"),
    ("no_lists", BF, 2, 3, 1000, 0, 0, "few"), ("history", BF, 1, 8, 5000, 333, 0, None), ("one_row", F32, 3, 1, 4099, 50, 7, None),
    ("odd", BF, 3, 5, 8191, 100, 20, "half"), ("odd_f32", F32, 3, 4, 8193, 100, 20, "most"), ("segments", BF, 2, 4, 32003, 700, 50, "few"),
    ("none_allowed", BF, 2, 2, 4097, 30, 3, "nothing"), ("biases", F32, 2, 3, 9000, 0, 5000, None), ("long", BF, 2, 3, 20000, 5000, 3, "most"),
    ("many", BF, 40, 9, 1500, 60, 4, "half"), ("many_f32", F32, 33, 16, 2000, 60, 4, "few"), ("wide", BF, 1, 17, 70001, 1001, 9, "half"),
]


@pytest.mark.parametrize("case", ROWS, ids=[c[0] for c in ROWS])
@pytest.mark.parametrize("place", [False, True])
def test_rows_against_fp64(case, place):
    name, dtype, B, R, V, L, M, mask = case
    say("adjust", name, place)
    x, c = rows_case(len(name) * 31 + V, dtype, B, R, V, L, M, mask)
    d = x.cuda()
    out = df2.adjust_logits(d, **on_gpu(c), out=d if place else None)
    assert (out.data_ptr() == d.data_ptr()) == place
    check_rows(x, c, out)
    if not place:
        assert torch.equal(d.cpu(), x)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("place", [False, True])
def test_rows_with_strides_and_broadcast_masks(dtype, place):
    """Rows of a padded vocabulary that begin anywhere; what lies between them is left
    alone; one mask for all rows of a sequence, and for all sequences."""
    say("adjust strides", dtype, place)
    x, c = rows_case(3, dtype, 3, 4, 1003, 70, 6, "half")
    for off in (0, 1, 3):
        wide = torch.full((3, 5, 1040), 7.0, dtype=dtype, device="cuda")
        view = wide[:, :4, off:off + 1003]
        view.copy_(x)
        for cut in (1, 4):
            m = c["mask"][:1, :1].expand(3, 4, -1) if cut == 1 else c["mask"][:, :1].expand(3, 4, -1)
            d = on_gpu(dict(c, mask=m.contiguous()))
            d["mask"] = (m[:1, :1].cuda().expand(3, 4, -1) if cut == 1 else m[:, :1].cuda().expand(3, 4, -1))
            d["history"] = torch.cat((d["history"], d["history"]), 1)[:, :70]
            keep = wide.clone()
            to = torch.full((3, 4, 1010), 5.0, dtype=dtype, device="cuda")
            got = df2.adjust_logits(view, **d, out=view if place else to[:, :, 2:1005])
            check_rows(x, dict(c, mask=m.contiguous()), got)
            if place:
                rest = wide.clone()
                rest[:, :4, off:off + 1003] = keep[:, :4, off:off + 1003]
                assert torch.equal(rest, keep)
                view.copy_(x)
            else:
                assert torch.equal(wide, keep) and bool((to[:, :, :2] == 5).all()) and bool((to[:, :, 1005:] == 5).all())


def test_rows_of_infinities_nan_and_lists_of_nothing():
    say("adjust odd values")
    x = torch.tensor([[[float("inf"), -float("inf"), float("nan"), -0.0, 0.0, 1.0, -1.0, 3e38]]]).repeat(1, 2, 1)
    for dtype in (BF, F32):
        y = x.to(dtype)
        # nothing happens: bits stay
        got = df2.adjust_logits(y.cuda(), history=i32([[-1, 8, 2**31 - 1, -2**31]]), history_len=i32([4]), path=i32([[-1]]),
                                bias_token=i32([[-1, 9]]), bias=torch.ones((1, 2), device="cuda"))
        view = torch.int16 if dtype == BF else torch.int32
        assert torch.equal(got.cpu().view(view), y.view(view))
        # lengths beyond the array and below zero
        one = dict(repetition=torch.tensor([2.0], device="cuda"), history=i32([[5, 6, 5]]))
        got = df2.adjust_logits(y.cuda(), **one, history_len=i32([99])).float().cpu()
        assert got[0, 0, 5:7].tolist() == [0.5, -2.0] and got[0, 0, 3].item() == 0
        assert torch.equal(df2.adjust_logits(y.cuda(), **one, history_len=i32([-4])).cpu().view(view), y.view(view))
        # penalties of infinities and NaN
        got = df2.adjust_logits(y.cuda(), history=i32([[0, 1, 2, 7]]), history_len=i32([4]), prompt_len=i32([0]),
                                frequency=torch.tensor([0.5], device="cuda"), repetition=torch.tensor([2.0], device="cuda")).float().cpu()
        assert got[0, 0, 0] == float("inf") and got[0, 0, 1] == -float("inf") and torch.isnan(got[0, 0, 2])
        # a forbidden NaN is -inf, and so is a forbidden token with a bias
        got = df2.adjust_logits(y.cuda(), mask=i32([[[0b11100000], [-1]]]), bias_token=i32([[4]]), bias=torch.ones((1, 1), device="cuda"))
        assert got[0, 0, :5].float().cpu().tolist() == [-float("inf")] * 5 and got[0, 1, 4].item() == 1.0


def test_rows_in_a_graph_and_on_another_stream():
    """Replays take what the history, drafts and masks then hold."""
    say("adjust in a graph")
    x, c = rows_case(9, BF, 4, 8, 32003, 400, 9, "half")
    d, x_dev = on_gpu(c), x.cuda()
    call = df2.PreparedAdjust(x_dev, **d)
    want = call().clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    side = torch.cuda.Stream()
    for k in range(4):
        y, e = rows_case(20 + k, BF, 4, 8, 32003, 400, 9, "most" if k % 2 else "few")
        x_dev.copy_(y)
        for name in d:
            d[name].copy_(e[name])
        call._out.zero_()
        graph.replay()
        got = call._out.clone()
        check_rows(y, e, got)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            call._out.zero_()
            assert torch.equal(call(), got)
        torch.cuda.current_stream().wait_stream(side)
    assert not torch.equal(got, want)
    assert df2.device_error() == 0


def test_rows_before_verification():
    """At temperature 0 a forbidden draft is refused and the best allowed token follows."""
    say("adjust then verify")
    x = torch.zeros((1, 3, 200), dtype=BF, device="cuda")
    x[0, 0, 7], x[0, 1, 8], x[0, 1, 9], x[0, 2, 3] = 5, 5, 4, 5
    mask = torch.full((1, 3, 7), -1, dtype=torch.int32, device="cuda")
    mask[0, 1, 0] = ~(1 << 8)
    path = i32([[7, 8]])
    tok, count, _ = df2.verify(df2.adjust_logits(x, mask=mask), path, temperature=0.0)
    assert tok.tolist() == [[7, 9, -1]] and count.tolist() == [2]
    # a draft weighs against itself in the rows behind it
    x[0, 1, 7] = 5.5
    tok, count, _ = df2.verify(df2.adjust_logits(x, path=path, presence=torch.ones((1,), device="cuda"), out=x), path, temperature=0.0)
    assert tok.tolist() == [[7, 8, 3]] and count.tolist() == [3]
