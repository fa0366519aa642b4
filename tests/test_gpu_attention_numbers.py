"""GPU tests of attention over both paged caches where numbers are out of the ordinary:
queries and blocks of NaN, scores beyond what fp32 tells apart, scales far apart, and
sequences of very different lengths in one batch, whatever the launch plan makes of them.

Every comparison here is one that zeros in place of the output would fail (telling)."""
import math

import pytest
import torch

import draft_selection_topk16_amd as df2
from fp4_ref import fp4_case, held
from gpu_util import say
from target_ref import HALF, U, attention_ref, paged_case

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
        if start[b + 1] == start[b]:
            continue
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


def telling(ref, bound):
    """Whether the bound would find an output of zeros wrong, nearly everywhere."""
    return float((ref.abs() > bound).double().mean()) > 0.9


def seen(c, b):
    """Positions of sequence b's keys, and their keys and values [L, Hkv, D] in fp64."""
    D, page = c["q"].shape[2], c["page"]
    k, v = ((held(c[x], page, D) if c["fp4"] else c[x].cpu().double()) for x in ("k_cache", "v_cache"))
    start, ctx, table = c["start"].tolist(), c["ctx"].tolist(), c["table"].cpu().long()
    j = torch.arange(ctx[b] + start[b + 1] - start[b])
    return j, k[table[b, j // page], :, j % page], v[table[b, j // page], :, j % page]


FAR = [(fp4, dtype, D, n) for fp4 in (True, False) for dtype, D, n in
       ((BF, 128, 1), (BF, 128, 8), (BF, 128, 16), (BF, 128, 50), (BF, 64, 8), (BF, 256, 3), (F32, 128, 1), (F32, 64, 16), (F32, 256, 2))]


@pytest.mark.parametrize("fp4,dtype,D,n", FAR)
@pytest.mark.parametrize("e", [31, 60, 100])
def test_scores_beyond_what_fp32_tells_apart(fp4, dtype, D, n, e):
    """Queries of one power of two: every score is one product, exact, and the largest ones are
    apart from all others by far more than they are rounded by, so the output is the mean of
    the values of the keys that share the largest score.  Their weights are 1, exact in either
    type; T of them are added and divided in fp32, (T + 8) u of their mean magnitude, and
    rounded once.  The heads between have ordinary queries and the ordinary bound."""
    say("far scores", fp4, dtype, D, n, e)
    c = case(fp4, n + D + e, dtype, D, 8, 2, 16, [n, n], [3000, 40])
    if not fp4:
        c["k_cache"][..., 0] = (2 * c["k_cache"][..., 0]).round() / 2       # some keys alike
    q = c["q"]
    far = torch.zeros((2 * n, 8))
    far[:, 0::4], far[:, 1::4], far[1::2, 3::4] = 1, -1, 1
    q.copy_(torch.where(far.cuda()[..., None] != 0, 0, q))
    q[..., 0] = torch.where(far.cuda() != 0, far.cuda() * 2.0 ** e, q[..., 0].float()).to(dtype)
    ref, bound = expected(dict(c, q=torch.where(far.cuda()[..., None] != 0, 0, q)))
    h, ties = HALF[dtype], []
    for b in range(2):
        j, k, v = seen(c, b)
        for t in range(n):
            for head in range(8):
                r, sign = b * n + t, float(far[b * n + t, head])
                if sign == 0:
                    continue
                x = torch.where(j <= c["ctx"].tolist()[b] + t, sign * k[:, head // 4, 0], -float("inf"))
                top = v[x == x.max(), head // 4]
                ties.append(len(top))
                ref[r, head] = top.mean(0)
                bound[r, head] = ((len(top) + 8) * U * top.abs().mean(0) + h * top.mean(0).abs()) * (1 + 2 * h)
    assert max(ties) > 1 and telling(ref, bound)
    for max_len in (None, 40):
        got = attend(c, max_len=max_len).cpu().double()
        assert bool(((got - ref).abs() <= bound).all())
    assert df2.device_error() == 0


@pytest.mark.parametrize("fp4,dtype,D,n", FAR)
def test_steps_of_eight_at_scores_of_two_to_the_26th(fp4, dtype, D, n):
    """Scores 2^26 + 8 i, the next numbers that fp32 has there, with a scale whose product
    with log2(e) is 1 in fp32: weights are powers of 2^-8, exact in either type, and their sums
    over L keys are off by (L + 8) u."""
    say("steps of eight", fp4, dtype, D, n)
    c = case(fp4, n + D, dtype, D, 8, 2, 16, [n, n], [2000, 20])
    g = torch.Generator().manual_seed(n)
    codes = torch.tensor([0, 2, 4, 5, 6, 7], dtype=torch.uint8)                # 0, 1, 2, 3, 4, 6
    pick = torch.randint(0, 6, c["k_cache"].shape[:2] + (16,), generator=g)
    # a rare step at the top, so that the maximum moves late too
    pick = torch.where((pick == 5) & (torch.rand(pick.shape, generator=g) < 0.97), 0, pick)
    if fp4:
        c["k_cache"][:, :, 0:16 * D // 2:D // 2] = (2 | codes[pick] << 4).cuda()           # 1, then the step
        c["k_cache"][:, :, 16 * D // 2::D // 32] = 127
    else:
        c["k_cache"][..., 0] = 1
        c["k_cache"][..., 1] = torch.tensor([0.0, 1.0, 2.0, 3.0, 4.0, 6.0])[pick].to(dtype).cuda()
    c["q"].zero_()
    c["q"][..., 0], c["q"][..., 1] = 2.0 ** 26, 8
    scale = float(torch.tensor(math.log(2), dtype=F32))
    assert torch.tensor(scale * math.log2(math.e), dtype=F32).item() == 1.0
    h = HALF[dtype]
    ref, bound = torch.zeros((2, 2 * n, 8, D), dtype=torch.float64)
    for b in range(2):
        j, k, v = seen(c, b)
        assert bool((k[..., 0] == 1).all())
        for t in range(n):
            w = 8 * k[..., 1]
            w = torch.where((j <= c["ctx"].tolist()[b] + t)[:, None], torch.exp2(w - w[:c["ctx"].tolist()[b] + t + 1].amax(0)), 0)
            o, A = ((w[..., None] * x).sum(0) / w.sum(0)[:, None] for x in (v, v.abs()))
            ref[b * n + t] = o.repeat_interleave(4, 0)
            bound[b * n + t] = (((len(j) + 8) * U * A + h * o.abs()) * (1 + 2 * h)).repeat_interleave(4, 0)
    assert telling(ref, bound)
    for max_len in (None, 40):
        got = attend(c, max_len=max_len, scale=scale).cpu().double()
        assert bool(((got - ref).abs() <= bound).all())
    assert df2.device_error() == 0


@pytest.mark.parametrize("dtype,D,n", [(BF, 128, 1), (BF, 64, 8), (BF, 128, 16), (BF, 256, 1), (F32, 128, 1), (F32, 64, 20)])
def test_scales_far_apart_within_a_telling_bound(dtype, D, n):
    """Values whose scales differ by 2^40 and more under moderate keys; then keys as far
    apart in a block where the queries are zero."""
    say("scales far apart", dtype, D, n)
    args = (n + D, dtype, D, 8, 2, 16, [n, n], [900, 41])
    c, apart = (dict(fp4_case(*args, garbage=False, spread=s), fp4=True) for s in (0.0, 9.0))
    far = dict(c, v_cache=apart["v_cache"])
    ref, bound = expected(far)
    assert telling(ref, bound)
    assert bool(((attend(far).cpu().double() - ref).abs() <= bound).all())
    # the last block of each key, codes and scale
    k = c["k_cache"].clone()
    for part, last in ((slice(0, 8 * D), slice(D // 2 - 16, None)), (slice(8 * D, None), slice(D // 32 - 1, None))):
        x, y = (t[:, :, part].unflatten(2, (16, -1))[..., last] for t in (k, apart["k_cache"]))
        x.copy_(y)
    q = c["q"].clone()
    q[..., -32:] = 0
    far = dict(c, k_cache=k, q=q)
    assert float(held(k, 16, D)[..., -32:].abs().max()) > 2.0 ** 30
    ref, bound = expected(far)
    assert telling(ref, bound)
    assert bool(((attend(far).cpu().double() - ref).abs() <= bound).all())
    assert df2.device_error() == 0


@pytest.mark.parametrize("fp4", [True, False])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_single_tokens_beside_a_chunk_and_many_idle_rows(fp4, dtype):
    """Sequences keep the bound whatever else the step holds: single tokens beside a piece of
    a prompt, sequences without tokens, and a step of many more rows than are used, whose
    outputs stay as they are."""
    say("mixed batch", fp4, dtype)
    new = [1, 1, 0, 260, 1, 0] + [1] * 9
    ctx = [900, 3, 50, 70, 1500, 0] + [40 * i for i in range(9)]
    c = case(fp4, 5, dtype, 64, 8, 2, 16, new, ctx)
    ref, bound = expected(c)
    assert telling(ref, bound)
    for idle in (0, 3, 4000):
        wide = dict(c, q=torch.cat((c["q"], torch.full((idle, 8, 64), float("nan"), dtype=dtype, device="cuda"))))
        out = torch.full_like(wide["q"], -7.0)
        for max_len in (None, 40):
            got = attend(wide, max_len=max_len, out=out.clone()).cpu().double()
            assert bool(((got[:len(ref)] - ref).abs() <= bound).all()) and bool((got[len(ref):] == -7.0).all())
    assert df2.device_error() == 0


@pytest.mark.parametrize("dtype,D,n", [(BF, 128, 1), (BF, 128, 8), (BF, 64, 16), (BF, 128, 60), (F32, 128, 1), (F32, 256, 9)])
def test_values_up_to_the_documented_scale(dtype, D, n):
    """Values times 2^87: every product and sum is the same but for its exponent, up to the
    largest values under the largest weights, so the outputs are those times 2^87, bit for bit
    (none is near the other end of the exponents)."""
    say("large values", dtype, D, n)
    c = case(True, n + D, dtype, D, 8, 2, 16, [n, n], [20000, 3])
    scales = c["v_cache"][:, :, 8 * D:]
    scales.fill_(127)
    want = attend(c)
    scales.fill_(127 + 87)
    got = attend(c)
    assert bool(torch.isfinite(got).all()) and float(got.abs().max()) > 2.0 ** 80
    tiny = want.abs() < 2.0 ** -60                      # weights that vanish beside the largest
    assert torch.equal(got[~tiny], (want * 2.0 ** 87)[~tiny]) and float(tiny.double().mean()) < 0.2
    assert df2.device_error() == 0


@pytest.mark.parametrize("dtype", [BF, F32])
def test_unpack_at_the_ends_of_the_scales(dtype):
    """All codes under the smallest and the largest scales: subnormal numbers under 0, exact up
    to the end of the range, infinities beyond it, NaN under 255."""
    say("unpack ends", dtype)
    which = [0, 1, 2, 6, 7, 126, 127, 128, 247, 250, 251, 252, 253, 254, 255, 0]
    cache = torch.zeros((1, 1, 16 * 34), dtype=torch.uint8)
    cache[..., :16 * 32] = (torch.arange(16).repeat(32) * 17).to(torch.uint8)       # both halves of byte i: code i % 16
    cache[..., 16 * 32:] = torch.tensor(which, dtype=torch.uint8).repeat_interleave(2)
    ref = held(cache, 16, 64)
    most = torch.finfo(dtype).max
    ref = torch.where(ref.abs() > most, torch.sign(ref) * float("inf"), ref)
    assert bool(torch.isinf(ref).any()) and bool(((ref != 0) & (ref.abs() < 2.0 ** -126)).any())
    for got in df2.kv_unpack_fp4(cache.cuda(), cache.cuda(), 64, dtype):
        assert torch.equal(torch.nan_to_num(got.cpu().double(), 12345.0, 1e300, -1e300), torch.nan_to_num(ref, 12345.0, 1e300, -1e300))
