"""GPU tests of appending to a 4-bit paged cache and of what it then holds: codes and
scales have to be those of the fp64 form, bit for bit."""
import numpy as np
import pytest
import torch

import draft_selection_topk16_amd as df2
from fp4_ref import MAGNITUDES, appended, fp4_case, held
from gpu_util import say
from test_gpu_append_edges import check_queries

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


def append_case(seed, dtype, D, Hq, Hkv, page, new, ctx, rot, norm, pad=2):
    c = fp4_case(seed, dtype, D, Hq, Hkv, page, new, ctx, pad_rows=pad)
    g = torch.Generator().manual_seed(seed + 1)
    qkv = (3 * torch.randn((c["N"], Hq + 2 * Hkv, D), generator=g)).to(dtype).cuda()
    c.update(q=qkv[:, :Hq], k=qkv[:, Hq:Hq + Hkv], v=qkv[:, Hq + Hkv:])
    w = (1 + 0.3 * torch.randn((2, D), generator=g)).to(dtype).cuda()
    c["q_norm"], c["k_norm"] = (w[0].contiguous(), w[1].contiguous()) if norm else (None, None)
    c["freq"] = df2.rope_freqs(rot, 1e6, "cuda") if rot else None
    return c


def append(c, inter=False, **kw):
    return df2.kv_append_fp4(c["k"], c["v"], c["k_cache"], c["v_cache"], c["table"], c["ctx"], c["start"], q=c["q"], q_norm=c["q_norm"],
                             k_norm=c["k_norm"], rope_freq=c["freq"], interleaved=inter, **kw)


APPEND = [
    # name, dtype, D, Hq, Hkv, page, new, ctx, rot, interleaved, norm
    ("block", BF, 128, 32, 8, 16, [8], [1003], 128, False, True),
    ("ragged", BF, 128, 5, 1, 16, [1, 0, 9, 3], [0, 5, 15, 100000], 128, False, True),
    ("partial", BF, 128, 4, 2, 32, [3, 4], [7, 0], 64, False, True),
    ("interleaved", BF, 64, 4, 4, 64, [5, 2], [3, 9], 64, True, False),
    ("f32", F32, 64, 12, 4, 32, [7, 29], [40001, 0], 32, True, False),
    ("f32_half", F32, 256, 3, 1, 16, [2], [123456], 256, False, True),
    ("no_rotation", BF, 256, 2, 1, 64, [70], [60], 0, False, True),
    ("as_they_are", BF, 64, 2, 1, 16, [3], [14], 0, False, False),
    ("before_the_start", BF, 128, 2, 1, 16, [5], [-2], 128, False, True),
    ("many", BF, 64, 3, 1, 16, [(37 * i) % 113 for i in range(80)], [(91 * i) % 300 for i in range(80)], 64, False, True),
    ("many_f32", F32, 128, 2, 2, 16, [2049, 0, 2048, 7], [5, 0, 1000, 70], 128, True, True),
    ("many_256", BF, 256, 2, 1, 256, [4100], [3], 32, False, True),
]


@pytest.mark.parametrize("case", APPEND, ids=[c[0] for c in APPEND])
def test_append_against_fp64(case):
    name, dtype, D, Hq, Hkv, page, new, ctx, rot, inter, norm = case
    say("fp4 append", name)
    c = append_case(len(name), dtype, D, Hq, Hkv, page, new, ctx, rot, norm)
    q0 = c["q"].clone()
    want = appended(c, D, None if c["freq"] is None else c["freq"].cpu().numpy(), inter)
    out = torch.full((c["N"], Hq, D), -7.0, dtype=dtype, device="cuda")
    append(c, inter, out_q=out)
    assert df2.device_error() == 0
    for key, (cache, sure) in zip(("k_cache", "v_cache"), want):
        got = c[key].cpu().numpy()
        assert sure.all() and (got == cache).all(), (key, int((got != cache).sum()))
    if rot and len(new) < 60 and sum(new) < 200:
        check_queries(c, q0, out, inter)
    elif not rot and not norm:
        assert torch.equal(out[:sum(new)], q0[:sum(new)])
    assert bool((out[sum(new):] == -7.0).all())         # rows that no sequence owns


@pytest.mark.parametrize("dtype", [BF, F32])
def test_borders_scales_and_what_is_not_finite(dtype):
    """Values on and next to the borders of two codes at small, ordinary and large scales,
    zeros of either sign, blocks of nothing, infinities and NaN; keys go through fp64, values
    through fp32."""
    say("fp4 borders", dtype)
    D, rows = 64, []
    step = 2.0 ** -7 if dtype == BF else 2.0 ** -23
    borders = (MAGNITUDES[:-1] + MAGNITUDES[1:]) / 2
    near = np.concatenate([borders, borders * (1 + step), borders * (1 - step / 2), MAGNITUDES, [6.5, 7.0, -0.0]])
    for top in (3.5, 3.5 * (1 + step), 4.0, 6.0, 7.0, 7.0 * (1 - step / 2), 7.0 * (1 + step)):
        for e in (-130, -119, -30, 0, 5, 100, 118, 121):
            x = np.zeros(D)
            x[:len(near)] = near * (1 if e % 2 else -1)
            x[:len(near)] = np.clip(x[:len(near)], -top, top)
            x[31] = top
            x[32:32 + len(near)] = -x[:len(near)]
            x[63] = top
            rows.append(x * 2.0 ** min(e, 124))
    rows += [np.zeros(D), -np.zeros(D)]
    for odd in (np.inf, -np.inf, np.nan):
        x = np.linspace(-3, 3, D)
        x[40] = odd
        rows.append(x)
    x = torch.tensor(np.array(rows)).to(dtype).cuda()[:, None, :]
    n = len(rows)
    table = torch.arange(-(-n // 16), dtype=torch.int32, device="cuda")[None]
    kc, vc = df2.fp4_cache(table.shape[1], 1, 16, D)
    c = dict(k=x, v=x, k_norm=None, k_cache=kc, v_cache=vc, table=table, ctx=torch.zeros(1, dtype=torch.int32, device="cuda"),
             start=torch.tensor([0, n], dtype=torch.int32, device="cuda"), page=16)
    want = appended(c, D, None, False)
    df2.kv_append_fp4(x, x, kc, vc, table, c["ctx"], c["start"])
    for got, (cache, sure) in zip((kc, vc), want):
        same = got.cpu().numpy() == cache
        assert same[sure].all(), np.argwhere(~same & sure)[:5]
    assert df2.device_error() == 0
    for t in (BF, F32):
        k, v = df2.kv_unpack_fp4(kc, vc, D, t)
        for got, cache in ((k, kc), (v, vc)):
            ref = held(cache, 16, D)
            assert torch.equal(torch.nan_to_num(got.cpu().double(), 12345.0), torch.nan_to_num(ref, 12345.0))
    assert bool(torch.isnan(k[-1]).any())


@pytest.mark.parametrize("D,page,Hkv,pages", [(64, 16, 1, 1), (128, 16, 8, 37), (256, 64, 3, 5), (64, 65536, 1, 2), (128, 32, 5, 11)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_unpack_of_every_byte(D, page, Hkv, pages, dtype):
    """All codes under all scales whose values are in range of the type, pages apart."""
    say("fp4 unpack", D, page, dtype)
    g = torch.Generator().manual_seed(D + page)
    size = df2.fp4_page_bytes(page, D)
    wide = torch.randint(0, 256, (2, pages, Hkv * size + 48), generator=g).to(torch.uint8)
    part = wide[:, :, :Hkv * size].unflatten(2, (Hkv, size))
    scales = part[..., page * D // 2:]
    scales.copy_(torch.where(scales == 0, 127, torch.where(scales > 251, 255, scales)))     # 6 * 2^125 is not finite
    dev = wide.cuda()
    view = dev[:, :, :Hkv * size].unflatten(2, (Hkv, size))
    got = df2.kv_unpack_fp4(view[0], view[1], D, dtype)
    for x, cache in zip(got, part):
        ref = held(cache, page, D)
        assert x.dtype == dtype and torch.equal(torch.nan_to_num(x.cpu().double(), 12345.0), torch.nan_to_num(ref, 12345.0))
    assert torch.equal(dev.cpu(), wide)


def test_places_outside_the_table():
    """Tokens before the first place, behind the last or on a bad page are not written;
    flags as for the other append."""
    say("fp4 append flags")
    c = append_case(4, BF, 64, 2, 1, 16, [4, 4], [14, 14], 64, True, pad=0)
    freq = c["freq"].cpu().numpy()
    t = c["table"].clone()
    t[0, 1] = -5
    k0 = c["k_cache"].clone()
    append(dict(c, table=t))
    assert df2.device_error() == 8
    changed = (c["k_cache"] != k0).flatten(1).any(1).nonzero().flatten().tolist()
    assert sorted(changed) == sorted([int(c["table"][0, 0]), int(c["table"][1, 0]), int(c["table"][1, 1])])
    for ctx0 in (29, 1 << 30, (1 << 31) - 1, -3, -(1 << 31)):
        bad = dict(c, ctx=torch.tensor([ctx0, 14], dtype=torch.int32, device="cuda"))
        want = appended(bad, 64, freq, False)
        q0 = c["q"].clone()
        out = append(bad)
        assert df2.device_error() == (16 if ctx0 > 0 else 0)
        check_queries(bad, q0, out)
        for key, (cache, _) in zip(("k_cache", "v_cache"), want):
            assert (c[key].cpu().numpy() == cache).all()


def test_append_in_a_graph_in_place_and_keys_only():
    say("fp4 append in a graph")
    c = append_case(3, BF, 128, 4, 2, 16, [5, 3], [10, 31], 128, True)
    call = df2.PreparedAppendFp4(c["k"], c["v"], c["k_cache"], c["v_cache"], c["table"], c["ctx"], c["start"], q=c["q"], q_norm=c["q_norm"],
                                 k_norm=c["k_norm"], rope_freq=c["freq"])
    before = [c["k_cache"].clone(), c["v_cache"].clone()]
    out = call().clone()
    k1, v1 = c["k_cache"].clone(), c["v_cache"].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    side = torch.cuda.Stream()
    for _ in range(3):
        call._out.zero_()
        for cache, after in ((c["k_cache"], k1), (c["v_cache"], v1)):
            # what the call writes is gone, the rest stays
            cache.copy_(torch.where(after != before[1 if after is v1 else 0], 0, after))
        graph.replay()
        assert torch.equal(call._out[:8], out[:8]) and torch.equal(c["k_cache"], k1) and torch.equal(c["v_cache"], v1)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            call._out.zero_()
            assert torch.equal(call()[:8], out[:8])
        torch.cuda.current_stream().wait_stream(side)
    c["k_cache"][:, :, :16].zero_()
    assert df2.kv_append_fp4(c["k"], c["v"], c["k_cache"], c["v_cache"], c["table"], c["ctx"], c["start"], k_norm=c["k_norm"],
                             rope_freq=c["freq"]) is None
    rows = appended(c, 128, c["freq"].cpu().numpy(), False)
    assert (c["k_cache"].cpu().numpy() == rows[0][0]).all()
    q = c["q"]
    got = append(c, out_q=q)
    assert torch.equal(q[:8], out[:8]) and got.data_ptr() == q.data_ptr() and df2.device_error() == 0


def test_a_cache_does_not_depend_on_the_batch():
    """The same tokens one by one, in one call and among others: the same bytes."""
    say("fp4 append split")
    c = append_case(9, BF, 128, 2, 2, 16, [90], [700], 128, True, pad=0)
    append(c)
    whole = c["k_cache"].clone()
    for n in (1, 7):
        c["k_cache"][:, :, ::3] ^= 77
        d = append_case(9, BF, 128, 2, 2, 16, [90], [700], 128, True, pad=0)
        c["k_cache"].copy_(d["k_cache"])
        for i in range(0, 90, n):
            m = min(n, 90 - i)
            part = dict(c, q=c["q"][i:i + m], k=c["k"][i:i + m], v=c["v"][i:i + m], ctx=c["ctx"] + i,
                        start=torch.tensor([0, m], dtype=torch.int32, device="cuda"))
            append(part)
        assert torch.equal(c["k_cache"], whole)
    assert df2.device_error() == 0
