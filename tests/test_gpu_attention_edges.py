"""GPU tests of paged attention at the ends of its ranges: positions before the
first, whole blocks of every head size."""
import pytest
import torch

import draft_selection_topk16_amd as df2
from gpu_util import say
from target_ref import paged_case
from test_gpu_target import attend, check_attention

pytestmark = pytest.mark.gpu

BF, F32, NAN = torch.bfloat16, torch.float32, float("nan")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    df2.load()
    df2.device_error()
    yield
    torch.cuda.synchronize()


BEFORE = [
    # name, dtype, D, Hq, Hkv, page, new, ctx, window
    ("few_rows", BF, 128, 4, 1, 16, [6, 2, 8], [-3, -7, -1], 0),
    ("few_rows_64", BF, 64, 3, 3, 1, [6, 5], [-3, 20], 0),
    ("few_rows_256", BF, 256, 4, 2, 16, [6, 8], [-3, 40], 0),
    ("few_rows_f32", F32, 128, 8, 2, 16, [6, 2], [-3, 9], 0),
    ("window", BF, 128, 8, 2, 16, [9, 8], [-4, -2], 2),
    ("blocks_of_64", BF, 128, 32, 8, 16, [16, 9], [-5, 2300], 0),
    ("blocks_of_128_f32", F32, 64, 16, 8, 16, [64, 40], [-9, -30], 0),
    ("blocks_of_256", BF, 128, 32, 8, 16, [200, 130], [-77, 2500], 0),
    ("blocks_of_256_window", BF, 64, 32, 8, 16, [300, 130], [-77, -129], 20),
    ("many_blocks", BF, 64, 32, 8, 16, [4100, 300], [-100, -299], 0),
    ("split", BF, 128, 8, 2, 16, [5, 3, 4], [-2, 2900, -3], 0),
]


@pytest.mark.parametrize("case", BEFORE, ids=[c[0] for c in BEFORE])
def test_whole_blocks_before_the_first_position(case):
    """A token whose position is negative sees nothing and gets 0, in a whole block too."""
    name, dtype, D, Hq, Hkv, page, new, ctx, window = case
    say("attention whole block before the start", name)
    c = paged_case(len(name) * 7 + D, dtype, D, Hq, Hkv, page, new, ctx, garbage=NAN)
    out = attend(c, causal=False, window=window)
    check_attention(c, out, False, window)
    start = c["start"].tolist()
    for b, at in enumerate(ctx):
        if at < 0:
            assert bool((out[start[b]:start[b] + min(-at, new[b])] == 0).all())
    assert df2.device_error() == 0


@pytest.mark.parametrize("dtype,new,ctx,window", [(BF, [8, 5], [50, 0], 0), (BF, [70, 3], [45, 31], 0), (BF, [9, 8], [400, 7], 33),
                                                  (F32, [8, 40], [99, 3], 0)])
def test_whole_blocks_of_head_size_256(dtype, new, ctx, window):
    say("attention whole block 256", dtype, new)
    c = paged_case(new[0] + ctx[0], dtype, 256, 8, 2, 16, new, ctx, garbage=NAN)
    check_attention(c, attend(c, causal=False, window=window), False, window)
    assert df2.device_error() == 0


def test_slots_without_new_tokens_may_hold_any_length():
    """A captured batch has empty slots whose lengths are stale: nothing is read for
    them and no flag is raised, in the append as in the attention."""
    say("attention empty slots")
    c = paged_case(70, BF, 128, 8, 2, 16, [0, 3, 0, 2, 0], [0, 40, 0, 7, 0], garbage=NAN)
    want = attend(c)
    stale = dict(c, ctx=torch.tensor([1 << 30, 40, -(1 << 31), 7, (1 << 31) - 1], dtype=torch.int32, device="cuda"))
    assert torch.equal(attend(stale), want)
    assert df2.device_error() == 0
    k = torch.randn((5, 2, 128), device="cuda").to(BF)
    df2.kv_append(k, k, c["k_cache"], c["v_cache"], c["table"], stale["ctx"], c["start"])
    assert df2.device_error() == 0


@pytest.mark.parametrize("ctx", [(1 << 31) - 1, 48, -(1 << 31)])
def test_lengths_at_the_ends_of_their_type(ctx):
    """Beyond the page table: as if the last new token had the last place; far below
    0: zeros."""
    say("attention lengths", ctx)
    c = paged_case(71, BF, 64, 4, 2, 16, [3, 2], [45, 20])
    far = dict(c, ctx=torch.tensor([ctx, 20], dtype=torch.int32, device="cuda"))
    out, want = attend(far), attend(c)
    assert df2.device_error() == (16 if ctx > 0 else 0)
    assert torch.equal(out, want if ctx > 0 else torch.cat((torch.zeros_like(want[:3]), want[3:])))


DOWN = [
    # starts, and the sequences with tokens of the same batch in order (None: refused)
    ([0, 8, 0, 8, 0, 8, 13], None), ([13, 0, 2, 4, 6, 8, 10], None), ([0, 2, 4, 6, 8, 7, 9], None),
    ([0, 2, 4, 6, 0, 0, 0], [0, 2, 4, 6, 6, 6, 6]), ([13, 0, 0, 0, 0, 0, 0], [0] * 7), ([0, 2, 4, 6, 8, 13, 12], [0, 2, 4, 6, 8, 13, 13]),
]


@pytest.mark.parametrize("start,same", DOWN)
@pytest.mark.parametrize("B", [6, 150])
def test_descending_token_starts(start, same, B):
    """Overlapping sequences could ask for more work than there are tokens: outputs stay
    and flag bit 4 is raised.  Starts that fall where no tokens follow, as zeros behind
    the last sequence, leave the batch as it is."""
    say("attention descending starts", start, B)
    c = paged_case(72, BF, 128, 8, 2, 16, [2, 2, 2, 2, 2, 3], [500, 3, 0, 70, 9, 40])
    good = attend(c)

    def with_starts(s, more):
        """B sequences: these, and empty ones that begin at `more`."""
        wide = torch.cat((c["table"], c["table"][:1].expand(B - 6, -1)))
        return dict(c, table=wide, ctx=torch.cat((c["ctx"], c["ctx"][:1].expand(B - 6))),
                    start=torch.tensor(s + [more] * (B - 6), dtype=torch.int32, device="cuda"))
    out = torch.full_like(good, -7.0)
    attend(with_starts(start, start[-1]), out=out)
    if same is None:
        assert bool((out == -7.0).all()) and df2.device_error() == 16
        # seen from the next wave of sequences too
        late = with_starts([0] * 7, 0)
        if B > 64:
            late["start"][7:] = torch.tensor([13] * 80 + [3] * (B - 6 - 81) + [5], dtype=torch.int32, device="cuda")
            attend(late, out=out)
            assert bool((out == -7.0).all()) and df2.device_error() == 16
    else:
        want = torch.full_like(good, -7.0)
        attend(with_starts(same, same[-1]), out=want)
        assert torch.equal(out, want) and df2.device_error() == 0
    assert torch.equal(attend(c), good) and df2.device_error() == 0
