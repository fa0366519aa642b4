"""GPU tests of the target-side operators (paged append, paged attention, draft
verification) against plain fp64 forms, with the bounds derived in target_ref."""
import numpy as np
import pytest
import torch

import draft_selection_topk16_amd as df2
from draft_selection_topk16_amd import synth
from gpu_util import say, to_device
from target_ref import HALF, U, append_ref, attention_ref, paged_case, verify_ref

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    df2.load()
    df2.device_error()
    yield
    torch.cuda.synchronize()


def attend(c, **kw):
    return df2.paged_attention(c["q"], c["k_cache"], c["v_cache"], c["table"], c["ctx"], c["start"], **kw)


def check_attention(c, out, causal=True, window=0, scale=None):
    D = c["q"].shape[2]
    ref, bound = attention_ref(c, D ** -0.5 if scale is None else scale, causal, window)
    got = out.cpu().double()
    owned = ~torch.isnan(ref)
    err = (got - ref).abs()
    assert bool((torch.isfinite(got) | ~owned).all())
    worst = float((err / (bound + 1e-300))[owned & (bound > 0)].max()) if bool((owned & (bound > 0)).any()) else 0.0
    assert bool((err <= bound)[owned].all()), "largest error is %.3g of its bound" % worst
    return worst


ATTENTION = [
    # name, dtype, D, Hq, Hkv, page, new, ctx, causal, window
    ("one_token", BF, 128, 32, 8, 16, [1], [0], True, 0),
    ("decode", BF, 128, 32, 8, 16, [1, 1, 1], [1003, 5, 128], True, 0),
    ("decode_mha", BF, 64, 3, 3, 1, [1, 1], [77, 300], True, 0),
    ("decode_mqa_g40", BF, 128, 40, 1, 32, [1, 1], [511, 512], True, 0),
    ("block8_g5", BF, 128, 10, 2, 16, [8, 8, 3], [0, 60, 1000], True, 0),
    ("block8_g8", BF, 128, 16, 2, 16, [8, 8], [63, 640], True, 0),
    ("block16_g7", BF, 64, 7, 1, 64, [16, 9], [33, 95], True, 0),
    ("chunk", BF, 128, 4, 1, 16, [150, 0, 97], [201, 9, 0], True, 0),
    ("chunk_many_blocks", BF, 128, 32, 8, 16, [3000, 1111, 2], [40, 300, 7], True, 0),
    ("chunk_many_blocks_window", BF, 64, 32, 8, 16, [4100, 300], [0, 900], True, 500),
    ("chunk_64", BF, 64, 2, 1, 32, [333], [100], True, 0),
    ("chunk_256", BF, 256, 2, 1, 16, [70, 3], [45, 31], True, 0),
    ("decode_256", BF, 256, 8, 2, 64, [1, 2], [200, 77], True, 0),
    ("whole_block", BF, 128, 8, 2, 16, [8, 7, 1], [50, 0, 9], False, 0),
    ("window", BF, 128, 8, 2, 16, [8, 40, 1], [300, 10, 77], True, 33),
    ("window_1", BF, 64, 4, 2, 16, [5, 5], [40, 0], True, 1),
    ("window_whole_block", BF, 128, 4, 1, 16, [8], [100], False, 20),
    ("f32_decode", F32, 128, 8, 2, 16, [1, 1], [333, 2], True, 0),
    ("f32_block", F32, 64, 12, 4, 32, [8, 7, 8], [17, 90, 260], False, 0),
    ("f32_chunk", F32, 64, 2, 1, 16, [140], [50], True, 0),
    ("f32_chunk_128", F32, 128, 4, 2, 8, [60, 33], [0, 70], True, 25),
    ("f32_256", F32, 256, 2, 1, 16, [40, 1], [20, 99], True, 0),
    ("empty_and_late", BF, 128, 4, 1, 16, [0, 4, 0, 1], [10, 0, 0, 65], True, 0),
    ("before_the_start", BF, 128, 4, 1, 16, [6, 2], [-3, -7], True, 0),
    ("big_page", BF, 128, 4, 2, 1024, [9], [1500], True, 0),
    # one tile in all: no workspace
    ("one_tile", BF, 128, 4, 1, 16, [1], [20], True, 0),
    ("one_tile_64", BF, 64, 1, 1, 16, [1], [0], True, 0),
    ("one_tile_f32", F32, 128, 2, 1, 16, [3], [5], False, 0),
    ("one_tile_256", BF, 256, 8, 1, 16, [2], [3], True, 0),
    # short blocks, taken whole
    ("many_short", BF, 128, 32, 8, 16, [1 + i % 3 for i in range(70)], [(37 * i) % 211 for i in range(70)], True, 0),
    ("many_short_64_f32", F32, 64, 16, 8, 16, [4 + i % 5 for i in range(66)], [(37 * i) % 311 for i in range(66)], False, 0),
    ("many_short_256", BF, 256, 16, 4, 16, [i % 4 for i in range(40)], [(91 * i) % 300 for i in range(40)], True, 60),
    ("chunk_from_nothing", BF, 128, 32, 8, 16, [1024], [0], True, 0),
    ("mixed_lengths", BF, 128, 16, 4, 16, [8, 1, 300, 8, 2], [9000, 3, 0, 40, 700], True, 0),
    ("pages_of_one_token", BF, 128, 8, 2, 1, [3, 1], [5003, 2050], True, 0),
    ("pages_of_one_token_f32_window", F32, 64, 4, 4, 1, [2, 1], [3500, 1], True, 2500),
    ("chunk_small_pages", BF, 128, 32, 8, 2, [4100], [300], True, 0),
    # enough tiles for blocks of 256, 128 and 64 rows, not for whole ones
    ("blocks_of_256", BF, 128, 32, 8, 16, [200, 130], [3000, 2500], True, 0),
    ("blocks_of_256_64", BF, 64, 32, 8, 32, [200, 130], [1500, 1900], True, 0),
    ("blocks_of_256_whole_block", BF, 128, 16, 4, 16, [300, 257], [3000, 3050], False, 0),
    ("blocks_of_128", BF, 128, 32, 8, 16, [31, 1, 32], [3300, 2, 3100], True, 0),
    ("blocks_of_128_window", BF, 64, 32, 8, 16, [31, 20, 32], [3300, 40, 3100], True, 900),
    ("blocks_of_128_f32", F32, 128, 16, 8, 16, [64, 40], [1650, 1700], True, 0),
    ("blocks_of_128_f32_64", F32, 64, 16, 8, 16, [64, 40], [1650, 1700], False, 0),
    ("blocks_of_128_256", BF, 256, 16, 8, 16, [64, 40], [1650, 1700], True, 0),
    ("blocks_of_64", BF, 128, 32, 8, 16, [16, 9, 16], [2300, 4, 2200], True, 0),
    ("blocks_of_64_64", BF, 64, 32, 8, 16, [16, 9, 16], [4700, 4, 4500], True, 0),
    ("blocks_of_64_f32", F32, 64, 32, 8, 16, [16, 9, 16], [2300, 4, 2200], True, 700),
]


@pytest.mark.parametrize("case", ATTENTION, ids=[c[0] for c in ATTENTION])
def test_attention_against_fp64(case):
    name, dtype, D, Hq, Hkv, page, new, ctx, causal, window = case
    say("attention", name)
    c = paged_case(len(name) * 101 + D, dtype, D, Hq, Hkv, page, new, ctx, garbage=NAN)
    worst = check_attention(c, attend(c, causal=causal, window=window), causal, window)
    assert df2.device_error() == 0
    say("  worst error / bound %.3f" % worst)


@pytest.mark.parametrize("dtype,D,G", [(BF, 128, 4), (BF, 64, 8), (F32, 128, 2), (BF, 256, 1), (F32, 64, 1), (F32, 256, 3)])
def test_attention_over_split_keys(dtype, D, G):
    """A long context in few rows is split over workgroups and joined; one
    sequence of the batch is short (a single split)."""
    say("attention splits", dtype, D, G)
    c = paged_case(7, dtype, D, 2 * G, 2, 16, [3, 2], [2200, 5], garbage=NAN)
    kw = dict(k_cache=c["k_cache"])
    ws = df2.PreparedAttention(c["q"], kw["k_cache"], c["v_cache"], c["table"], c["ctx"], c["start"])._keep[-1]
    assert ws.numel() > 0
    check_attention(c, attend(c))


def test_attention_split_windows_and_empty_rows():
    say("attention split window")
    c = paged_case(8, BF, 128, 8, 2, 16, [4, 4, 2], [3000, 10, -2], garbage=NAN)
    check_attention(c, attend(c, window=1300), True, 1300)


@pytest.mark.parametrize("max_len", [1, 40, 700, 100000])
def test_attention_does_not_depend_on_the_length_estimate(max_len):
    say("attention max_len", max_len)
    c = paged_case(9, BF, 128, 8, 2, 16, [8, 8], [1500, 30])
    check_attention(c, attend(c, max_len=max_len))


def test_attention_strides_and_padding_rows():
    """Queries and outputs inside wider rows, K and V pages in one tensor, a
    page table inside a wider one; rows behind the last sequence stay."""
    say("attention strides")
    c = paged_case(10, BF, 128, 8, 2, 16, [5, 8], [100, 31], pad_rows=3)
    N = c["N"]
    both = torch.stack((c["k_cache"], c["v_cache"]), 1).contiguous()
    wide_q = torch.full((N, 12, 128), NAN, dtype=BF, device="cuda")
    wide_q[:, 2:10] = c["q"]
    wide_o = torch.full((N, 11, 128), -7.0, dtype=BF, device="cuda")
    wide_t = torch.full((2, c["table"].shape[1] + 5), -1, dtype=torch.int32, device="cuda")
    wide_t[:, :c["table"].shape[1]] = c["table"]
    out = df2.paged_attention(wide_q[:, 2:10], both[:, 0], both[:, 1], wide_t[:, :c["table"].shape[1]], c["ctx"],
                              c["start"], out=wide_o[:, 1:9])
    check_attention(c, out)
    assert df2.device_error() == 0
    rest = wide_o.clone()
    rest[:N - 3, 1:9] = -7.0
    assert bool((rest == -7.0).all())


def test_attention_bad_pages_and_lengths_raise_flags():
    say("attention flags")
    c = paged_case(11, BF, 64, 2, 1, 16, [2, 2], [40, 20])
    good = attend(c)
    t = c["table"].clone()
    t[0, 1] = 10 ** 6
    c2 = dict(c, table=t)
    out = attend(c2)
    assert df2.device_error() == 8
    assert torch.equal(out[2:], good[2:])
    # the same with page 0 named
    t[0, 1] = 0
    assert torch.equal(attend(dict(c, table=t)), out)
    assert df2.device_error() == 0
    # a context beyond the page table: taken to end at its last place
    ctx = c["ctx"].clone()
    ctx[1] = 10 ** 9
    out = attend(dict(c, ctx=ctx))
    assert df2.device_error() == 16
    ctx[1] = c["table"].shape[1] * 16 - 2
    assert torch.equal(attend(dict(c, ctx=ctx)), out)


def test_attention_far_pages():
    """Pages beyond 2^31 elements of the cache."""
    say("attention far pages")
    D, Hkv, page = 128, 2, 64
    num = (1 << 31) // (Hkv * page * D) + 40
    c = paged_case(12, BF, D, 8, Hkv, page, [4], [700])
    small = c["k_cache"].shape[0]
    kc = torch.empty((num, Hkv, page, D), dtype=BF, device="cuda")
    vc = torch.empty((num, Hkv, page, D), dtype=BF, device="cuda")
    kc[num - small:], vc[num - small:] = c["k_cache"], c["v_cache"]
    far = dict(c, k_cache=kc, v_cache=vc, table=c["table"] + (num - small))
    assert torch.equal(attend(far), attend(c))
    # and what append writes there
    k, v = torch.randn((4, Hkv, D), device="cuda").to(BF), torch.randn((4, Hkv, D), device="cuda").to(BF)
    df2.kv_append(k, v, kc, vc, far["table"], c["ctx"], c["start"])
    df2.kv_append(k, v, c["k_cache"], c["v_cache"], c["table"], c["ctx"], c["start"])
    assert torch.equal(kc[num - small:], c["k_cache"]) and torch.equal(vc[num - small:], c["v_cache"])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_attention_shared_pages(dtype):
    """Sequences with a common beginning name the same pages; one is listed twice."""
    say("attention shared pages", dtype)
    c = paged_case(60, dtype, 64, 8, 2, 16, [3, 3, 8], [800, 800, 793])
    c["table"][1, :49] = c["table"][0, :49]
    c["table"][2, :30] = c["table"][0, :30]
    check_attention(c, attend(c))
    twice = dict(c, table=c["table"][[0, 0, 2]].contiguous(), ctx=c["ctx"][[0, 0, 2]].contiguous())
    twice["q"][3:6] = twice["q"][:3]
    out = attend(twice)
    check_attention(twice, out)


def test_attention_many_sequences():
    """More sequences than a wave scans at once, empty ones among them."""
    say("attention many sequences")
    new = [(i * 5) % 4 for i in range(150)]
    ctx = [(i * 37) % 90 for i in range(150)]
    c = paged_case(13, BF, 64, 4, 2, 16, new, ctx, garbage=NAN)
    check_attention(c, attend(c))


def test_attention_extreme_scores():
    """Scores of +-2000 (bf16 keys of 64 times the size): the running maximum
    moves and nothing overflows."""
    say("attention extreme scores")
    c = paged_case(14, F32, 64, 2, 1, 16, [3], [300])
    c["k_cache"].mul_(64.0)
    c["q"].mul_(8.0)
    check_attention(c, attend(c))


APPEND = [
    # name, dtype, D, Hq, Hkv, page, new, ctx, rot, interleaved, norm
    ("block", BF, 128, 32, 8, 16, [8], [1003], 128, False, True),
    ("ragged", BF, 128, 5, 1, 16, [1, 0, 9, 3], [0, 5, 15, 100000], 128, False, True),
    ("partial", BF, 128, 4, 2, 32, [3, 4], [7, 0], 64, False, True),
    ("interleaved", BF, 64, 4, 4, 1, [5, 2], [3, 9], 64, True, False),
    ("f32", F32, 64, 12, 4, 32, [7, 29], [40001, 0], 32, True, False),
    ("f32_half", F32, 256, 3, 1, 16, [2], [123456], 256, False, True),
    ("no_rotation", BF, 256, 2, 1, 64, [70], [60], 0, False, True),
    ("copy", BF, 64, 2, 1, 16, [3], [14], 0, False, False),
    ("before_the_start", BF, 128, 2, 1, 16, [5], [-2], 128, False, True),
    ("many", BF, 64, 3, 1, 16, [(37 * i) % 113 for i in range(80)], [(91 * i) % 300 for i in range(80)], 64, False, True),
    ("many_f32", F32, 128, 2, 2, 8, [2049, 0, 2048, 7], [5, 0, 100000, 70000], 128, True, True),
]


def append_case(seed, dtype, D, Hq, Hkv, page, new, ctx, rot, norm, pad=2):
    c = paged_case(seed, dtype, D, Hq, Hkv, page, new, ctx, pad_rows=pad)
    g = torch.Generator().manual_seed(seed + 1)
    qkv = (3 * torch.randn((c["N"], Hq + 2 * Hkv, D), generator=g)).to(dtype).cuda()
    c.update(q=qkv[:, :Hq], k=qkv[:, Hq:Hq + Hkv], v=qkv[:, Hq + Hkv:])
    w = (1 + 0.3 * torch.randn((2, D), generator=g)).to(dtype).cuda()
    c["q_norm"], c["k_norm"] = (w[0].contiguous(), w[1].contiguous()) if norm else (None, None)
    c["freq"] = df2.rope_freqs(rot, 1e6, "cuda") if rot else None
    return c


def append(c, interleaved, **kw):
    return df2.kv_append(c["k"], c["v"], c["k_cache"], c["v_cache"], c["table"], c["ctx"], c["start"], q=c["q"],
                         q_norm=c["q_norm"], k_norm=c["k_norm"], rope_freq=c["freq"], interleaved=interleaved, **kw)


@pytest.mark.parametrize("case", APPEND, ids=[c[0] for c in APPEND])
def test_append_against_fp64(case):
    """Relative to the largest |y| of a head before the turn: the norm's sum of D
    squares, its root and two products (D / 2 + 6 u), the turn's four (its
    cosine and sine good to 2^-22: half a step of the turn's fraction times
    2 pi, and the function's own), the store h; nothing else changes."""
    name, dtype, D, Hq, Hkv, page, new, ctx, rot, inter, norm = case
    say("append", name)
    c = append_case(len(name), dtype, D, Hq, Hkv, page, new, ctx, rot, norm)
    k0, v0, q0 = c["k_cache"].clone(), c["v_cache"].clone(), c["q"].clone()
    out = torch.full((c["N"], Hq, D), -7.0, dtype=dtype, device="cuda")
    append(c, inter, out_q=out)
    assert df2.device_error() == 0
    h = HALF[dtype]
    slack = (D / 2 + 6) * U + (2 * 2.0 ** -22 + 4 * U if rot else 0.0)
    freq = None if c["freq"] is None else c["freq"].cpu().numpy()
    want_k, want_v = k0.cpu(), v0.cpu()
    seen = torch.zeros(k0.shape[0], page, dtype=torch.bool)
    start, table = c["start"].tolist(), c["table"].cpu()
    got_k, got_q = c["k_cache"].cpu().double(), out.cpu().double()
    for b in range(len(new)):
        for t in range(new[b]):
            r, pos = start[b] + t, ctx[b] + t
            for x, w, got in ((q0[r], c["q_norm"], got_q[r]), (c["k"][r], c["k_norm"], None)):
                y, big = append_ref(x.double().cpu().numpy(), None if w is None else w.double().cpu().numpy(), 1e-6,
                                    freq, pos, inter)
                if got is None:
                    if pos < 0:
                        continue
                    page_id, slot = int(table[b, pos // page]), pos % page
                    seen[page_id, slot] = True
                    got = got_k[page_id, :, slot]
                    want_v[page_id, :, slot] = c["v"][r].cpu()
                err = np.abs(got.numpy() - y)
                assert np.all(err <= (slack * 2 * big + h * np.abs(y)) * (1 + 2 * h)), (name, b, t, err.max())
    assert torch.equal(c["v_cache"].cpu(), want_v)
    keep = ~seen[:, None, :, None].expand(k0.shape)
    assert torch.equal(c["k_cache"].cpu()[keep], want_k[keep])
    assert bool((out[sum(new):] == -7.0).all())         # rows that no sequence owns


def test_nothing_is_done_for_rows_that_no_sequence_owns():
    say("no owned rows")
    c = append_case(5, BF, 128, 4, 2, 16, [0, 0, 0], [10, 0, 31], 128, True, pad=6)
    k0, v0 = c["k_cache"].clone(), c["v_cache"].clone()
    out = torch.full_like(c["q"].contiguous(), -7.0)
    append(c, False, out_q=out)
    assert torch.equal(c["k_cache"], k0) and torch.equal(c["v_cache"], v0) and bool((out == -7.0).all())
    df2.paged_attention(c["q"], c["k_cache"], c["v_cache"], c["table"], c["ctx"], c["start"], out=out)
    assert bool((out == -7.0).all()) and df2.device_error() == 0


def test_append_in_place_and_keys_only():
    say("append in place, keys only")
    c = append_case(3, BF, 128, 4, 2, 16, [5, 3], [10, 31], 128, True)
    k0, v0 = c["k_cache"].clone(), c["v_cache"].clone()
    out = append(c, False)
    k1, v1 = c["k_cache"].clone(), c["v_cache"].clone()
    c["k_cache"].copy_(k0)
    c["v_cache"].copy_(v0)
    assert df2.kv_append(c["k"], c["v"], c["k_cache"], c["v_cache"], c["table"], c["ctx"], c["start"],
                         k_norm=c["k_norm"], rope_freq=c["freq"]) is None
    assert torch.equal(c["k_cache"], k1) and torch.equal(c["v_cache"], v1)
    q = c["q"]
    got = append(c, False, out_q=q)
    assert torch.equal(q[:8], out[:8]) and got.data_ptr() == q.data_ptr()


def test_append_bad_pages_and_lengths():
    say("append flags")
    c = append_case(4, BF, 64, 2, 1, 16, [4, 4], [14, 14], 64, True, pad=0)
    t = c["table"].clone()
    t[0, 1] = -5
    k0 = c["k_cache"].clone()
    df2.kv_append(c["k"], c["v"], c["k_cache"], c["v_cache"], t, c["ctx"], c["start"])
    assert df2.device_error() == 8
    changed = (c["k_cache"] != k0).flatten(1).any(1).nonzero().flatten().tolist()
    assert sorted(changed) == sorted([int(c["table"][0, 0]), int(c["table"][1, 0]), int(c["table"][1, 1])])
    ctx = c["ctx"].clone()
    ctx[0] = 1 << 30
    df2.kv_append(c["k"], c["v"], c["k_cache"], c["v_cache"], c["table"], ctx, c["start"])
    assert df2.device_error() == 16


def verify_case(seed, dtype, B, P, V, K, sharp=2.0, device="cuda"):
    g = torch.Generator().manual_seed(seed)
    step = V // K
    ids = torch.arange(K) * step + torch.randint(0, step, (B, P, K), generator=g)
    ids = ids.gather(-1, torch.rand((B, P, K), generator=g).argsort(-1))
    score = sharp * torch.randn((B, P, K), generator=g)
    target = 1.5 * torch.randn((B, P + 1, V), generator=g)
    lift = np.log(V) + score + 0.7 * torch.randn((B, P, K), generator=g)
    target[:, :P].scatter_(2, ids, lift)
    prob = torch.softmax(score, -1)
    pick = (prob.cumsum(-1) < torch.rand((B, P, 1), generator=g)).sum(-1, keepdim=True).clamp_(max=K - 1)
    pick = torch.where(torch.rand((B, P, 1), generator=g) < 0.5, lift.argmax(-1, keepdim=True), pick)
    u = torch.randint(0, 1 << 24, (B, P + 1), generator=g).float() / (1 << 24)
    path = ids.gather(-1, pick).squeeze(-1).to(torch.int32).contiguous()
    return dict(target=target.to(dtype).to(device), path=path.to(device), cand=ids.to(torch.int32).to(device),
                prob=prob.contiguous().to(device), u=u.to(device))


def check_verify(c, got, temperature=1.0, n_draft=None, kind="logits"):
    """Tokens and counts equal wherever no comparison is nearer than rounding
    allows (acceptance: p is good to 2^-18, a row sum of fp32 exponentials; the
    draw: fp64); p to the same 2^-18."""
    tok, cnt, p, margin = verify_ref(c["target"], c["path"], c["cand"], c["prob"], c["u"], temperature, n_draft, kind)
    gt, gc, gp = (x.cpu().numpy() for x in got)
    clear = margin > 2.0 ** -18
    assert clear.mean() > 0.9
    assert np.array_equal(gt[clear], tok[clear]) and np.array_equal(gc[clear], cnt[clear])
    assert np.all(np.abs(gp - p)[clear] <= 2.0 ** -18 * p[clear])
    return cnt


@pytest.mark.parametrize("dtype,B,P,V,K,tau", [
    (BF, 1, 7, 151936, 16, 1.0), (BF, 3, 7, 32000, 16, 0.6), (F32, 4, 5, 32003, 5, 1.0), (BF, 5, 3, 1001, 1, 1.3),
    (BF, 2, 64, 2049, 64, 1.0), (F32, 7, 1, 64, 64, 1.0), (BF, 40, 7, 9973, 16, 1.0), (F32, 2, 15, 100, 4, 5.0),
    (BF, 300, 2, 517, 8, 1.0), (BF, 2, 2, 1, 1, 1.0), (F32, 2, 2, 3, 3, 0.05),
])
def test_verify_against_fp64(dtype, B, P, V, K, tau):
    say("verify", dtype, B, P, V, K, tau)
    c = verify_case(B * 31 + V, dtype, B, P, V, K)
    got = df2.verify(c["target"], c["path"], c["cand"], c["prob"], c["u"], temperature=tau)
    assert df2.device_error() == 0
    cnt = check_verify(c, got, tau)
    say("  accepted", np.bincount(cnt - 1).tolist())


def test_verify_ragged_and_extreme_uniforms():
    say("verify ragged")
    c = verify_case(5, BF, 12, 7, 4001, 16)
    nd = torch.tensor([0, 1, 7, 9, -3, 3, 7, 7, 7, 7, 7, 7], dtype=torch.int32, device="cuda")
    c["u"][6] = 0.0                     # all accepted, lowest token with weight drawn
    c["u"][7] = 1.0                     # clamped below 1
    c["u"][8] = -5.0
    c["u"][9] = NAN
    c["u"][10, 7] = 1 - 2.0 ** -24
    c["u"][11, 7] = 2.0 ** -24
    got = df2.verify(c["target"], c["path"], c["cand"], c["prob"], c["u"], n_draft=nd)
    check_verify(c, got, 1.0, nd)
    assert got[1].tolist()[:2][0] == 1 and got[1][4] == 1


@pytest.mark.parametrize("dtype", [BF, F32])
def test_verify_probabilities(dtype):
    say("verify probs", dtype)
    c = verify_case(6, F32, 9, 7, 5003, 16)
    c["target"] = torch.softmax(c["target"], -1).to(dtype)
    got = df2.verify(c["target"], c["path"], c["cand"], c["prob"], c["u"], kind="probs")
    check_verify(c, got, 1.0, None, "probs")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V", [2, 1000, 32003])
def test_verify_greedy(dtype, V):
    """Temperature 0, ties among the largest values of coarse rows."""
    say("verify greedy", dtype, V)
    g = torch.Generator().manual_seed(V)
    B, P = 6, 7
    target = torch.randint(-3, 4, (B, P + 1, V), generator=g).float()
    best = (target == target.amax(-1, keepdim=True)).int().argmax(-1)
    path = best[:, :P].to(torch.int32).contiguous()
    for b in range(B):
        if b < P:
            path[b, b] = (path[b, b] + 1) % V
    target = target.to(dtype).cuda()
    tok, cnt, p = df2.verify(target, path.cuda(), temperature=0.0)
    want, wcnt, wp, _ = verify_ref(target, path, None, None, None, 0.0)
    assert np.array_equal(tok.cpu().numpy(), want) and np.array_equal(cnt.cpu().numpy(), wcnt)
    assert np.array_equal(p.cpu().numpy(), wp)


def test_verify_masked_vocabulary_and_rows_without_mass():
    say("verify masked")
    c = verify_case(7, F32, 4, 3, 700, 7)
    dead = torch.ones(700, dtype=torch.bool)
    dead[c["cand"].cpu().long().flatten()] = False
    c["target"][:, :, dead.cuda()] = -float("inf")
    got = df2.verify(c["target"], c["path"], c["cand"], c["prob"], c["u"])
    check_verify(c, got)
    assert df2.device_error() == 0
    c["target"][1] = -float("inf")
    c["target"][2] = torch.finfo(F32).min           # the lowest value everywhere: an even row
    got = df2.verify(c["target"], c["path"], c["cand"], c["prob"], c["u"])
    assert df2.device_error() == 64
    assert got[0][1].tolist() == [0, -1, -1, -1] and int(got[1][1]) == 1 and float(got[2][1, 0]) == 0.0
    even = {k: v[2:3].contiguous() for k, v in c.items()}
    check_verify(even, tuple(x[2:3] for x in got))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("tau", [0.3, 0.45, 0.7, 0.9, 1.0, 1.1, 1.7, 1e-6, 1e30])
def test_verify_masked_vocabulary_at_temperatures(dtype, tau):
    """Rows with -inf logits, whatever the sign of what fp32 leaves of log2(e) over
    the temperature."""
    say("verify masked", dtype, tau)
    c = verify_case(17, F32, 3, 3, 5000, 7)
    dead = torch.rand(5000, generator=torch.Generator().manual_seed(18)) < 0.5
    dead[c["cand"].cpu().long().flatten()] = False
    c["target"][:, :, dead.cuda()] = -float("inf")
    c["target"] = c["target"].to(dtype)
    got = df2.verify(c["target"], c["path"], c["cand"], c["prob"], c["u"], temperature=tau)
    assert df2.device_error() == 0
    assert bool((got[2] >= 0).all()) and not bool(dead[got[0].cpu().long().clamp(min=0)][got[0].cpu() >= 0].any())
    if tau >= 0.3:
        check_verify(c, got, tau)


@pytest.mark.parametrize("dtype,V", [(BF, 9000001), (F32, 4194311), (BF, 4095), (F32, 4097), (BF, 262151)])
def test_verify_draws_at_every_place_of_a_row(dtype, V):
    """Uniforms spread over the row, its ends among them; rows of odd lengths start at
    every alignment."""
    say("verify places", dtype, V)
    B = 2 if V > 1000000 else 9
    c = verify_case(V, dtype, B, 2, V, 4)
    c["u"][:, :2] = 0.0                                  # accepted while p > 0: the draw is from the last row
    c["u"][:, 2] = torch.linspace(0, 1 - 2.0 ** -24, B)
    check_verify(c, df2.verify(c["target"], c["path"], c["cand"], c["prob"], c["u"]))
    c["u"][:, 0] = 1.0                                   # refused mostly: candidates lose weight
    c["prob"].fill_(0.25)
    check_verify(c, df2.verify(c["target"], c["path"], c["cand"], c["prob"], c["u"]))
    assert df2.device_error() == 0


@pytest.mark.parametrize("dtype,B,P,V,K,tau", [
    (BF, 32, 7, 70001, 16, 0.8), (F32, 4300, 3, 1003, 5, 1.2), (BF, 300, 64, 1001, 64, 1.0), (F32, 70, 15, 16384, 3, 1.0),
    (BF, 130, 2, 50000, 8, 2.0), (BF, 8, 7, 262143, 16, 1.0), (BF, 8, 7, 262145, 16, 1.0),
])
def test_verify_many_elements_against_fp64(dtype, B, P, V, K, tau):
    """Sizes on both sides of what takes fp64 sums of every row."""
    say("verify many", dtype, B, P, V, K, tau)
    c = verify_case(B + V, dtype, B, P, V, K)
    nd = torch.randint(0, P + 1, (B,), generator=torch.Generator().manual_seed(B), dtype=torch.int32).cuda()
    got = df2.verify(c["target"], c["path"], c["cand"], c["prob"], c["u"], temperature=tau, n_draft=nd)
    assert df2.device_error() == 0
    check_verify(c, got, tau, nd)


@pytest.mark.parametrize("B", [3, 1200])
@pytest.mark.parametrize("kind,tau", [("logits", 0.45), ("logits", 0.7), ("logits", 1.3), ("probs", 1.0)])
def test_verify_masked_rows_few_and_many(B, kind, tau):
    """Half of the vocabulary without weight, some rows without any."""
    say("verify masked", B, kind, tau)
    V = 5000
    c = verify_case(B, F32, B, 3, V, 7)
    dead = torch.rand((B, 1, V), generator=torch.Generator().manual_seed(B)) < 0.5
    dead.scatter_(2, c["cand"].cpu().long().flatten(1)[:, None], False)
    c["target"] = c["target"].masked_fill(dead.cuda(), -float("inf"))
    if kind == "probs":
        c["target"] = torch.softmax(c["target"], -1)
    args = (c["path"], c["cand"], c["prob"], c["u"])
    check_verify(c, df2.verify(c["target"], *args, temperature=tau, kind=kind), tau, None, kind)
    assert df2.device_error() == 0
    c["target"][1] = 0.0 if kind == "probs" else -float("inf")
    tok, cnt, p = df2.verify(c["target"], *args, temperature=tau, kind=kind)
    assert df2.device_error() == 64
    assert tok[1].tolist() == [0, -1, -1, -1] and int(cnt[1]) == 1 and float(p[1].abs().max()) == 0.0


def test_verify_ids_outside_the_vocabulary():
    say("verify bad ids")
    c = verify_case(8, BF, 3, 4, 1000, 4)
    c["path"][0, 0] = 1000
    c["path"][1, 1] = -1
    got = df2.verify(c["target"], c["path"], c["cand"], c["prob"], c["u"])
    assert df2.device_error() & 32
    assert int(got[1][0]) == 1 and int(got[1][1]) <= 2
    assert bool((got[0][got[0] >= 0] < 1000).all())


def test_verify_keeps_the_target_distribution():
    """40000 sequences of one draft over 6 tokens, tokens drafted from q by the
    test: the first emitted token follows p.  Each count is binomial, so it
    stays within 5 standard deviations (a fair run fails once in 10^5)."""
    say("verify distribution")
    B, V, K = 40000, 6, 3
    g = torch.Generator().manual_seed(9)
    row = torch.tensor([0.3, -1.0, 1.2, 0.1, -0.4, 0.9])
    ids, q = torch.tensor([4, 2, 1]), torch.tensor([0.5, 0.3, 0.2])
    pick = torch.multinomial(q, B, replacement=True, generator=g)
    target = row.repeat(B, 2, 1).cuda()
    u = torch.rand((B, 2), generator=g)
    tok, cnt, p = df2.verify(target, ids[pick].to(torch.int32).view(B, 1).cuda(),
                             ids.to(torch.int32).repeat(B, 1, 1).contiguous().cuda(),
                             q.repeat(B, 1, 1).contiguous().cuda(), u.cuda())
    want = torch.softmax(row.double(), 0).numpy()
    got = torch.bincount(tok[:, 0].cpu().long(), minlength=V).numpy()
    assert np.all(np.abs(got - B * want) <= 5 * np.sqrt(B * want * (1 - want)))


@pytest.mark.parametrize("name,walk_K", [("qwen3_4b_b1", None), ("t27b_b8", 32)])
def test_select_sample_rows(name, walk_K):
    """The rows of the fused select equal the stages' softmax rows, their drawn
    entries the walk's q bit for bit; path, q and score as without rows."""
    say("sample rows", name)
    wl = synth.WORKLOADS[name]
    K = walk_K or wl.K
    t = to_device(synth.make_inputs(wl))
    u = df2.philox_uniforms(3, 1, wl.B * wl.P).view(wl.B, wl.P)
    args = (t["logits"], t["hidden"], t["A"], t["Bt"], t["W"], t["prev"], K, u)
    path, q, score = df2.select_sample(*args, temperature=1.5)
    path2, q2, score2, cand, rows = df2.select_sample(*args, temperature=1.5, rows=True)
    assert torch.equal(path, path2) and torch.equal(q, q2) and torch.equal(score, score2)
    hit = cand == path[..., None]
    assert bool((hit.sum(-1) == 1).all())
    assert torch.equal((rows * hit).sum(-1), q)
    ids, val = df2.topk(t["logits"], K)
    assert torch.equal(ids, cand)
    S = df2.pair_scores(ids, val, df2.project(t["hidden"], t["W"]), t["A"], t["Bt"], t["prev"])
    assert torch.equal(df2.draft_rows(S, ids, path, 1.5), rows)
    prev = torch.cat((torch.zeros_like(hit[:, :1]), hit[:, :-1]), 1)
    prev[:, 0, 0] = True
    s = (S.double() * prev[..., None]).sum(2)
    want = torch.softmax(s / 1.5, -1)
    # exponent (v - m) / tau: two roundings of its size and the exponential's, a sum of K
    slack = 2 * U * (2 * (s.amax(-1) - s.amin(-1)) / 1.5 + K + 6)
    assert bool(((rows.double() - want).abs() <= slack[..., None] * want + 1e-38).all())


def cycle(c, bufs):
    """One draft-verify cycle on the GPU: append, attend, target rows, verify."""
    out_q = df2.kv_append(c["k"], c["v"], c["k_cache"], c["v_cache"], c["table"], c["ctx"], c["start"], q=c["q"],
                          q_norm=c["q_norm"], k_norm=c["k_norm"], rope_freq=c["freq"])
    o = df2.paged_attention(out_q, c["k_cache"], c["v_cache"], c["table"], c["ctx"], c["start"])
    B, R = bufs["path"].shape[0], bufs["path"].shape[1] + 1
    target = (o.reshape(B * R, -1) @ bufs["head"]).view(B, R, -1)
    return (out_q, o, target) + df2.verify(target, bufs["path"], bufs["cand"], bufs["prob"], bufs["u"])


def cycle_case(seed, B=4, P=7, V=2000, K=16):
    # pages for two blocks
    c = append_case(seed, BF, 128, 8, 2, 16, [P + 1] * B, [100 + 61 * b for b in range(B)], 128, True, pad=0)
    c["ctx"] -= P + 1
    g = torch.Generator().manual_seed(seed)
    v = verify_case(seed, BF, B, P, V, K)
    v["head"] = (0.2 * torch.randn((8 * 128, V), generator=g)).to(BF).cuda()
    return c, v


def test_cycle_of_append_attention_and_verify():
    say("cycle")
    c, v = cycle_case(20)
    out_q, o, target, tok, cnt, p = cycle(c, v)
    assert df2.device_error() == 0
    check_attention(dict(c, q=out_q), o)
    check_verify(dict(v, target=target), (tok, cnt, p))
    # the next cycle: the accepted tokens stay, the rest of the block is overwritten
    c["ctx"] += cnt
    out_q, o, target, tok, cnt, p = cycle(c, v)
    check_attention(dict(c, q=out_q), o)


def test_cycle_captured_twice_and_replayed():
    """Two graphs of the cycle, replayed in turn with fresh inputs and eager work
    between the replays; every replay equals the eager run."""
    say("cycle graphs")
    cases = [cycle_case(30), cycle_case(31, B=2, P=3, V=999, K=5)]
    graphs, outs = [], []
    for c, v in cases:
        cycle(c, v)
    torch.cuda.synchronize()
    for c, v in cases:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(cycle(c, v))
        graphs.append(g)
    for rep in range(4):
        for (c, v), g, o in zip(cases, graphs, outs):
            gen = torch.Generator(device="cuda").manual_seed(100 + rep)
            c["q"].copy_(torch.randn(c["q"].shape, generator=gen, device="cuda"))
            c["k"].copy_(torch.randn(c["k"].shape, generator=gen, device="cuda"))
            v["u"].copy_(torch.rand(v["u"].shape, generator=gen, device="cuda"))
            c["ctx"] += 1
            g.replay()
            got = [x.clone() for x in o]
            kc = c["k_cache"].clone()
            want = cycle(c, v)
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want))
            assert torch.equal(kc, c["k_cache"])
            c["ctx"] -= 1
    assert df2.device_error() == 0


def test_calls_on_two_streams():
    """Prepared calls launched on another stream than the tensors were made on,
    two at a time."""
    say("two streams")
    c = [paged_case(40 + i, BF, 128, 8, 2, 16, [8, 8], [2500, 900]) for i in range(2)]
    want = [attend(x) for x in c]
    torch.cuda.synchronize()
    calls = [df2.PreparedAttention(x["q"], x["k_cache"], x["v_cache"], x["table"], x["ctx"], x["start"]) for x in c]
    streams = [torch.cuda.Stream() for _ in c]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(10):
        for s, call in zip(streams, calls):
            with torch.cuda.stream(s):
                out = call()
    torch.cuda.synchronize()
    for call, w in zip(calls, want):
        assert torch.equal(call._out, w)


def test_results_do_not_change_from_run_to_run():
    say("determinism")
    c = paged_case(50, BF, 128, 8, 2, 16, [8, 8], [2500, 900])
    v = verify_case(51, BF, 5, 7, 20000, 16)
    a0 = attend(c)
    v0 = df2.verify(v["target"], v["path"], v["cand"], v["prob"], v["u"])
    for _ in range(5):
        assert torch.equal(attend(c), a0)
        assert all(torch.equal(x, y) for x, y in zip(df2.verify(v["target"], v["path"], v["cand"], v["prob"], v["u"]), v0))
