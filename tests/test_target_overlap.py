"""Outputs of the paged operators that share memory with their inputs are refused
on the host; parts of one wider row are not."""
import ctypes
import random

import pytest
import torch

import draft_selection_topk16_amd as df2
from draft_selection_topk16_amd.binding import PagedKv
from target_ref import paged_case

EINVAL = 1
AT = 1 << 20        # 16-byte aligned, never dereferenced: every call here is refused
BF = torch.bfloat16


def kv(N, Hq=8, Hkv=2, D=64):
    return PagedKv(AT, AT, AT, AT, AT, Hkv * 16 * D, 8, 1, N, Hq, Hkv, D, 16, 10, 8, 1)


def attend(lib, k, q, q_stride, out, out_stride):
    st = lib.dflash2_paged_attention(ctypes.byref(k), q, q_stride, 0.1, 1, 0, 1, out, out_stride, AT << 8, 1 << 40, None)
    return st, lib.dflash2_last_error().decode()


def append(lib, k, q, q_stride, kk, k_stride, v, v_stride, out, out_stride):
    st = lib.dflash2_kv_append(ctypes.byref(k), q, q_stride, kk, k_stride, v, v_stride, None, None, 1e-6, None, 0, 0, out,
                               out_stride, None)
    return st, lib.dflash2_last_error().decode()


def meet(N, a, sa, wa, b, sb, wb):
    """By listing the 16-byte pieces (8 elements) of every row."""
    def pieces(at, s, w):
        return {at // 16 + (i * s + x) // 8 for i in range(N) for x in range(0, w, 8)}
    return bool(pieces(a, sa, wa) & pieces(b, sb, wb))


def test_outputs_over_inputs_are_refused():
    lib, rng, seen = df2.load(), random.Random(4), 0
    for _ in range(4000):
        N = rng.choice([1, 2, 3, 7])
        s = [512 + 8 * rng.choice([0, 0, 8, 16, 64, 100]) for _ in range(2)]
        out = AT + 16 * rng.randint(-N * 80, N * 80)
        if not meet(N, AT, s[0], 512, out, s[1], 512):
            continue        # would be launched
        seen += 1
        st, msg = attend(lib, kv(N), AT, s[0], out, s[1])
        assert st == EINVAL and "overlap" in msg, (N, s, out - AT)
        if out != AT:
            st, msg = append(lib, kv(N), AT, s[0], AT << 4, 128, AT << 5, 128, out, s[1])
            assert st == EINVAL and "overlap" in msg, (N, s, out - AT)
        # the same with keys, or values, of 128 elements
        ks = rng.choice([128, 512, 640])
        if meet(N, AT, ks, 128, out, s[1], 512):
            for kk, v in ((AT, AT << 5), (AT << 5, AT)):
                st, msg = append(lib, kv(N), AT << 4, 512, kk, ks, v, ks, out, s[1])
                assert st == EINVAL and "overlap" in msg, (N, ks, s, out - AT)
    assert seen > 1000


@pytest.mark.gpu
def test_inputs_and_outputs_in_one_row():
    """Queries, keys, values and both outputs side by side in each token's row, and an
    output in other rows of another stride between them."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    c = paged_case(90, BF, 64, 8, 2, 16, [5, 3], [30, 700])
    N = c["N"]
    row = torch.randn((N, 8 + 2 + 2 + 8 + 8, 64), generator=torch.Generator().manual_seed(1)).to(BF).cuda()
    q, k, v, out_q, out = row.split((8, 2, 2, 8, 8), 1)
    args = (c["k_cache"], c["v_cache"], c["table"], c["ctx"], c["start"])
    want_q = df2.kv_append(k, v, *args, q=q, rope_freq=df2.rope_freqs(64, device="cuda"))
    want = df2.paged_attention(want_q, *args)
    df2.kv_append(k, v, *args, q=q, rope_freq=df2.rope_freqs(64, device="cuda"), out_q=out_q)
    df2.paged_attention(out_q, *args, out=out)
    assert torch.equal(out_q, want_q) and torch.equal(out, want)
    with pytest.raises(df2.SelectorError, match="overlap"):
        df2.paged_attention(out, *args, out=out)
    # two rows of one buffer: 1500 elements apart, and their outputs 700 apart between them
    two = dict(c, q=want_q[:2], start=torch.tensor([0, 2, 2], dtype=torch.int32, device="cuda"))
    flat = torch.empty(3000, dtype=BF, device="cuda")
    q2, o2 = flat.as_strided((2, 8, 64), (2400, 64, 1)), flat.as_strided((2, 8, 64), (800, 64, 1), 600)
    q2.copy_(two["q"])
    want = df2.paged_attention(two["q"], *args[:4], two["start"])
    assert torch.equal(df2.paged_attention(q2, *args[:4], two["start"], out=o2), want) and torch.equal(q2, two["q"])
