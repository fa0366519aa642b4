"""GPU tests of attention over both paged caches where numbers are out of the ordinary:
queries and blocks of NaN, whatever the launch plan makes of them."""
import pytest
import torch

import draft_selection_topk16_amd as df2
from fp4_ref import fp4_case, held
from gpu_util import say
from target_ref import attention_ref, paged_case

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


def case(fp4, *args):
    c = fp4_case(*args, garbage=False) if fp4 else paged_case(*args)
    return dict(c, fp4=fp4, page=args[5])


def attend(c, **kw):
    f = df2.paged_attention_fp4 if c["fp4"] else df2.paged_attention
    return f(c["q"], c["k_cache"], c["v_cache"], c["table"], c["ctx"], c["start"], **kw)


def expected(c, scale=None):
    """(out, bound) of attention_ref, and what fp32 cannot hold on top of its bound: a weight
    p = exp(s - max) below 2^-126 may count as 0 (the exponential does not make denormals), and
    so may a product p v below that; the sum that all are divided by is at least 1 in units
    of the largest weight, so an output over n keys is off by n 2^-126 max(1, |v|) more at most.
    (Keys of the 4-bit cases differ so much that one key's weight can be nearly all.)"""
    D, page = c["q"].shape[2], c["page"]
    if c["fp4"]:
        c = dict(c, k_cache=held(c["k_cache"], page, D), v_cache=held(c["v_cache"], page, D))
    ref, bound = attention_ref(c, D ** -0.5 if scale is None else scale)
    start, table = c["start"].tolist(), c["table"].cpu().long()
    for b, ctx in enumerate(c["ctx"].tolist()):
        j = torch.arange(ctx + start[b + 1] - start[b])
        v = c["v_cache"].cpu()[table[b, j // page], :, j % page].abs()
        bound[start[b]:start[b + 1]] += len(j) * 2.0 ** -126 * max(1.0, float(v.max()))
    return ref, bound


# one split over workgroups and one that a workgroup has whole; another plan for either
NAN = [(fp4, dtype, D, n) for fp4 in (True, False) for dtype, D, n in
       ((BF, 128, 1), (BF, 128, 8), (BF, 128, 16), (BF, 128, 50), (BF, 64, 1), (BF, 256, 8), (F32, 128, 1), (F32, 64, 16), (F32, 256, 2))]


@pytest.mark.parametrize("fp4,dtype,D,n", NAN)
def test_a_query_of_nan_gives_nan(fp4, dtype, D, n):
    """Heads of a token whose query holds a NaN give NaN, with one element or all of them,
    in a sequence that is split or whole; all other heads are within the usual bound."""
    say("nan queries", fp4, dtype, D, n)
    c = case(fp4, n + D, dtype, D, 8, 2, 16, [n, n], [5000, 5])
    ref, bound = expected(c)
    hit = torch.zeros((2 * n, 8), dtype=torch.bool)
    hit[0, 1] = hit[n, 5] = hit[2 * n - 1, 0] = True
    bad = dict(c, q=c["q"].clone())
    bad["q"][0, 1, 3] = float("nan")
    bad["q"][n, 5] = float("nan")
    bad["q"][2 * n - 1, 0, D - 1] = -float("nan")
    for max_len in (None, 40):
        got = attend(bad, max_len=max_len).cpu().double()
        assert bool(torch.isnan(got[hit]).all())
        err = (got - ref).abs()
        assert bool((err <= bound)[~hit].all())
    assert df2.device_error() == 0


@pytest.mark.parametrize("dtype,D,n", [(BF, 128, 1), (BF, 128, 8), (BF, 64, 16), (F32, 128, 3), (BF, 256, 40)])
def test_a_key_block_of_nan_reaches_the_tokens_that_see_it(dtype, D, n):
    """A block of keys that held an infinity or NaN has scale 255: the query heads of its
    key head that see it give NaN, also where it is all that a workgroup's part has of the
    row's keys; tokens before it, other heads and other sequences do not."""
    say("nan keys", dtype, D, n)
    c = case(True, n + D, dtype, D, 4, 2, 16, [n, n], [5000, 33])
    ref, bound = expected(c)
    table = c["table"].cpu()
    for at in (0, 2500, 5000 + n - 1):
        bad = dict(c, k_cache=c["k_cache"].clone())
        scales = bad["k_cache"][:, :, 16 * D // 2:].unflatten(2, (16, D // 32))
        scales[int(table[0, at // 16]), 1, at % 16, D // 32 - 1] = 255
        hit = torch.zeros((2 * n, 4), dtype=torch.bool)
        hit[max(0, at - 5000):n, 2:] = True
        for max_len in (None, 40):
            got = attend(bad, max_len=max_len).cpu().double()
            assert bool(torch.isnan(got[hit]).all())
            assert bool(((got - ref).abs() <= bound)[~hit].all())
    # the last key of a window of one
    got = attend(bad, window=1).cpu()
    assert bool(torch.isnan(got[n - 1, 2:]).all()) and bool(torch.isfinite(got[n:]).all()) and bool(torch.isfinite(got[:n, :2]).all())
    assert df2.device_error() == 0
