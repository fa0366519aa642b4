"""GPU tests of draft verification where a range of the row has nothing left to
draw: its candidates hold all of its weight and lose all of it."""
import numpy as np
import pytest
import torch

import draft_selection_topk16_amd as df2
from gpu_util import say
from target_ref import verify_ref
from test_gpu_target import verify_case

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
LAST = 1 - 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    df2.load()
    df2.device_error()
    yield
    torch.cuda.synchronize()


def one_token_left(seed, dtype, B, V, K, kind):
    """Rows whose weight lies on K tokens close together, of which the draft gives
    each more than the target does, and on one token more, the only one that is left.
    That one stands before, between or behind them, near or far, and weighs as much
    as they do, or 10^-9 or 10^-26 of it."""
    rng = np.random.default_rng(seed)
    x = np.full((B, V), -np.inf)
    cand, left = np.zeros((B, K), np.int64), np.zeros(B, np.int64)
    for b in range(B):
        span = int(rng.choice([K + 1, 100, 400]))
        base = int(rng.integers(0, V - span))
        cand[b] = base + rng.choice(span, K, replace=False)
        far = int(rng.choice([1, 60, 300, 1500, 5000, V]))
        lo, hi = max(0, base - far), min(V, base + span + far)
        spot = np.setdiff1d(np.arange(lo, hi), cand[b])
        left[b] = spot[[0, -1, rng.integers(len(spot))][b % 3]]
        x[b, cand[b]] = 3 * rng.random(K)
        x[b, left[b]] = rng.choice([1.5, -20.0, -60.0])
    if kind == "probs":
        x = np.exp(x - x.max(-1, keepdims=True))
    t = torch.tensor(x).to(dtype)
    w = t.double().numpy()
    w = w if kind == "probs" else np.exp(w - w.max(-1, keepdims=True))
    p = w / w.sum(-1, keepdims=True)
    q = np.take_along_axis(p, cand, -1) * 1.02          # more than p, also rounded to fp32
    u = np.zeros((B, 2))
    u[:, 0] = LAST                                      # 1.02 u p < p is false: refused
    u[:, 1] = np.array([0.0, -1.0, LAST, 0.5, 1.0, 2.0 ** -24])[np.arange(B) % 6]
    return dict(target=torch.stack((t, t), 1).cuda(), path=torch.tensor(cand[:, :1], dtype=torch.int32).cuda(),
                cand=torch.tensor(cand[:, None], dtype=torch.int32).cuda(),
                prob=torch.tensor(q[:, None], dtype=F32).cuda(), u=torch.tensor(u, dtype=F32).cuda(),
                left=left, p=np.take_along_axis(p, left[:, None], -1)[:, 0])


@pytest.mark.parametrize("kind", ["logits", "probs"])
@pytest.mark.parametrize("dtype,B,V,K", [(BF, 96, 20000, 4), (F32, 96, 9999, 3), (BF, 700, 20011, 4), (F32, 700, 20000, 7),
                                         (BF, 90, 100003, 16)])
def test_the_only_token_left_is_drawn(dtype, B, V, K, kind):
    """Both forms, up to 2^24 elements and above.  p within 2^-18 of its value, a row
    sum of fp32 exponentials."""
    say("verify one token left", dtype, B, V, K, kind)
    c = one_token_left(B + V + K, dtype, B, V, K, kind)
    tok, cnt, p = df2.verify(c["target"], c["path"], c["cand"], c["prob"], c["u"], kind=kind)
    assert df2.device_error() == 0
    assert np.array_equal(tok[:, 0].cpu().numpy(), c["left"]) and bool((tok[:, 1] == -1).all()) and bool((cnt == 1).all())
    assert np.all(np.abs(p[:, 0].cpu().double().numpy() - c["p"]) <= 2.0 ** -18 * c["p"])


@pytest.mark.parametrize("B", [5, 900])
def test_no_token_left_raises_the_flag(B):
    """The same rows without that token and each candidate drafted surely: nothing is left."""
    say("verify no token left", B)
    c = one_token_left(B, F32, B, 10000, 4, "logits")
    c["target"].scatter_(2, torch.tensor(c["left"]).view(B, 1, 1).expand(B, 2, 1).cuda(), -float("inf"))
    c["prob"].fill_(1.5)
    tok, cnt, p = df2.verify(c["target"], c["path"], c["cand"], c["prob"], c["u"])
    assert df2.device_error() == 64
    assert bool((tok[:, 0] == 0).all()) and bool((cnt == 1).all()) and float(p.abs().max()) == 0.0


@pytest.mark.parametrize("dtype,B,P,V,K,tau,kind", [(BF, 4, 7, 151936, 16, 1.0, "logits"), (F32, 9, 7, 32003, 5, 0.7, "logits"),
                                                    (F32, 64, 15, 5000, 32, 1.3, "logits"), (BF, 20, 3, 9001, 8, 1.0, "probs")])
def test_few_elements_are_summed_in_64_bits(dtype, B, P, V, K, tau, kind):
    """Up to 2^24 elements p is rounded once, to fp32 (half a step 2^-24; the fp64 weights
    and sums are good to 10^-11), and decisions further apart than that are fp64's."""
    say("verify 64 bits", dtype, B, P, V, K, tau, kind)
    c = verify_case(B + P + V, F32, B, P, V, K)
    c["target"] = (torch.softmax(c["target"], -1) if kind == "probs" else c["target"]).to(dtype)
    args = (c["target"], c["path"], c["cand"], c["prob"], c["u"])
    got = [x.cpu().numpy() for x in df2.verify(*args, temperature=tau, kind=kind)]
    tok, cnt, p, margin = verify_ref(*args, tau, None, kind)
    clear = margin > 2.0 ** -24
    assert clear.mean() > 0.9 and df2.device_error() == 0
    assert np.array_equal(got[0][clear], tok[clear]) and np.array_equal(got[1][clear], cnt[clear])
    assert np.all(np.abs(got[2] - p)[clear] <= 2.0 ** -24 * (1 + 2.0 ** -10) * p[clear])
