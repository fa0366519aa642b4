"""GPU tests of the paged append where a token's position lies outside the page
table: before the first place or behind the last."""
import numpy as np
import pytest
import torch

import draft_selection_topk16_amd as df2
from gpu_util import say
from target_ref import HALF, U, append_ref
from test_gpu_target import append, append_case

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


def check_queries(c, q0, out, inter=False):
    """Every owned query against fp64 at position ctx_len + j, with the bound of
    test_append_against_fp64."""
    dtype, (_, Hq, D) = out.dtype, out.shape
    h, slack = HALF[dtype], (D / 2 + 6) * U + 2 * 2.0 ** -22 + 4 * U
    start, ctx, freq, w = c["start"].tolist(), c["ctx"].tolist(), c["freq"].cpu().numpy(), c["q_norm"]
    for b in range(len(ctx)):
        for t in range(start[b + 1] - start[b]):
            r = start[b] + t
            y, big = append_ref(q0[r].double().cpu().numpy(), None if w is None else w.double().cpu().numpy(), 1e-6, freq,
                                ctx[b] + t, inter)
            err = np.abs(out[r].cpu().double().numpy() - y)
            assert np.all(err <= (slack * 2 * big + h * np.abs(y)) * (1 + 2 * h)), (b, t, err.max())


@pytest.mark.parametrize("dtype,D,ctx", [(BF, 128, [-9, -2, 5]), (F32, 64, [-70, 3, -4]), (F32, 128, [-(1 << 31), 0, -8])])
def test_queries_before_the_first_position(dtype, D, ctx):
    """Queries turn by ctx_len + j also where that is far below 0; nothing is written
    for those tokens."""
    say("append before the start", dtype, D, ctx)
    new = [4, 5, 3]
    c = append_case(D, dtype, D, 4, 2, 16, new, ctx, D, True)
    q0, k0, v0 = c["q"].clone(), c["k_cache"].clone(), c["v_cache"].clone()
    out = append(c, False)
    assert df2.device_error() == 0
    check_queries(c, q0, out)
    pages = {int(c["table"][b, p // 16]) for b in range(3) for p in range(max(ctx[b], 0), max(ctx[b] + new[b], 0))}
    for cache, before in ((c["k_cache"], k0), (c["v_cache"], v0)):
        assert set((cache != before).flatten(1).any(1).nonzero().flatten().tolist()) == pages


@pytest.mark.parametrize("ctx0", [45, 47, 48, 1 << 30, (1 << 31) - 1])
@pytest.mark.parametrize("many", [False, True])
def test_nothing_is_written_behind_the_page_table(ctx0, many):
    """Tokens whose place the page table does not have raise the flag and are not
    written, nor does another of their sequence move; queries turn by ctx_len + j."""
    say("append behind the table", ctx0, many)
    new = [4, 3] + ([4200] if many else [])         # many: several tokens a workgroup
    c = append_case(6, F32, 64, 4, 2, 16, new, [40, 7] + ([0] if many else []), 64, True)
    c["table"] = c["table"][:, :3].contiguous()     # 48 places; the third sequence has 4200 tokens for them
    q0, k0, v0 = c["q"].clone(), c["k_cache"].clone(), c["v_cache"].clone()
    ctx = c["ctx"].clone()
    ctx[0] = ctx0
    bad = dict(c, ctx=ctx)
    out = append(bad, False)
    assert df2.device_error() == 16
    check_queries(dict(bad, start=bad["start"][:3], ctx=ctx[:2]), q0, out)
    # the tokens that have a place, appended alone, leave the same cache
    k1, v1 = c["k_cache"].clone(), c["v_cache"].clone()
    c["k_cache"].copy_(k0)
    c["v_cache"].copy_(v0)
    has = [max(0, min(4, 48 - ctx0)), 3] + ([48] if many else [])
    rows = torch.cat([torch.arange(n) + s for n, s in zip(has, bad["start"].tolist())]).cuda()
    part = dict(bad, q=c["q"][rows], k=c["k"][rows], v=c["v"][rows],
                start=torch.tensor([0] + has).cumsum(0).to(torch.int32).cuda())
    part["ctx"] = torch.where(torch.tensor(has).cuda() > 0, ctx, 0).to(torch.int32)
    append(part, False)
    assert df2.device_error() == 0
    assert torch.equal(c["k_cache"], k1) and torch.equal(c["v_cache"], v1)
