"""GPU test of how exactly bf16 attention weighs values in blocks of few rows."""
import pytest
import torch

import draft_selection_topk16_amd as df2
from gpu_util import say
from target_ref import HALF, attention_ref, paged_case
from test_gpu_target import attend

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.mark.parametrize("D,Hq,Hkv,page,new,ctx,causal,window", [
    (128, 32, 8, 16, [1], [1003], True, 0), (128, 32, 8, 16, [8, 8, 8], [3, 60, 2000], True, 0), (128, 64, 8, 16, [8, 8], [301, 77], True, 0),
    (64, 12, 4, 32, [7, 8], [2049, 17], False, 0), (64, 32, 8, 16, [16, 9, 16], [4700, 4, 4500], True, 0),
    (256, 8, 2, 16, [1, 8], [900, 30], True, 0), (256, 16, 8, 16, [32, 20], [3000, 40], True, 0), (128, 8, 2, 16, [8, 5], [3000, 40], True, 700),
])
def test_probabilities_of_few_rows_keep_16_bits(D, Hq, Hkv, page, new, ctx, causal, window):
    """The bound of the plain form in fp32 for the same values (its error beside weights
    rounded to bf16 is some 2^-8 / sqrt(keys) of sum p |v| / sum p), plus 2^-16 of that sum
    for the weights (a rounding to 8 bits, and one of what that left) and half a step
    of the output."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    say("attention precision", D, new, ctx)
    c = paged_case(D + new[0], BF, D, Hq, Hkv, page, new, ctx)
    out = attend(c, causal=causal, window=window).cpu().double()
    wide = dict(c, **{n: c[n].float() for n in ("q", "k_cache", "v_cache")})
    want, bound = attention_ref(wide, D ** -0.5, causal, window)
    size, _ = attention_ref(dict(wide, v_cache=wide["v_cache"].abs()), D ** -0.5, causal, window)
    limit = (bound + 2.0 ** -16 * size) * (1 + HALF[BF]) + HALF[BF] * want.abs()
    err = (out - want).abs()
    say("  worst error / bound %.3f" % float((err / limit).max()))
    assert bool((err <= limit).all())
    # and altogether no further off than the rounding of the outputs alone, but for a twentieth
    norm = float((want.to(BF).double() - want).norm())
    assert float((out - want).norm()) <= 1.05 * norm
