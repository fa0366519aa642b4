"""GPU tests of the serving side as it is used: pages planned from the lengths, tokens
appended in 4 bits, their attention, the target's rows adjusted and verified, and what
was accepted into the next step, all of it on the device."""
import random

import pytest
import torch

import draft_selection_topk16_amd as df2
from fp4_ref import appended
from gpu_util import say
from steps_ref import adjust_ref, pages_ref
from target_ref import verify_ref
from test_gpu_fp4_attention import check
from test_gpu_steps import check_rows

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
B, P, V, D, HQ, HKV, PAGE, WIDTH, PAGES = 6, 7, 997, 128, 8, 2, 16, 12, 60


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    df2.load()
    df2.device_error()
    yield
    torch.cuda.synchronize()


class Loop:
    """One step of a serving loop over prepared calls; a captured one replays them all."""

    def __init__(self, seed):
        g = torch.Generator().manual_seed(seed)
        z = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
        n = B * (P + 1)
        self.table, self.held, self.ctx, self.new, self.advance = z(B, WIDTH) - 1, z(B), z(B), z(B), z(B)
        self.free, self.count = torch.randperm(PAGES, generator=g).to(torch.int32).cuda(), z(1) + PAGES
        self.cache = df2.fp4_cache(PAGES, HKV, PAGE, D)
        self.qkv = torch.zeros((n, HQ + 2 * HKV, D), dtype=BF, device="cuda")
        self.q, self.k, self.v = self.qkv[:, :HQ], self.qkv[:, HQ:HQ + HKV], self.qkv[:, HQ + HKV:]
        self.k_norm = (1 + 0.2 * torch.randn((D,), generator=g)).to(BF).cuda()
        self.freq = df2.rope_freqs(D, 1e4, "cuda")
        self.pages = df2.PreparedPages(self.table, self.held, self.free, self.count, self.ctx, self.new, PAGE, n,
                                       advance=self.advance, ctx_out=self.ctx)
        self.start = self.pages._out[0]
        where = (self.table, self.ctx, self.start)
        self.append = df2.PreparedAppendFp4(self.k, self.v, *self.cache, *where, q=self.q, k_norm=self.k_norm, rope_freq=self.freq)
        self.attend = df2.PreparedAttentionFp4(self.append._out, *self.cache, *where)
        # the rest of the target: rows from the attention's output
        self.head = (torch.randn((HQ * D, V), generator=g) / 40).cuda()
        self.rows = torch.zeros((B, P + 1, V), dtype=BF, device="cuda")
        self.history, self.length = z(B, 300), z(B)
        self.path = z(B, P)
        self.mask = torch.full((B, P + 1, (V + 31) // 32), -1, dtype=torch.int32, device="cuda")
        self.pen = dict(repetition=torch.full((B,), 1.2, device="cuda"), frequency=torch.full((B,), 0.1, device="cuda"))
        self.adjust = df2.PreparedAdjust(self.rows, history=self.history, history_len=self.length, path=self.path, mask=self.mask,
                                         out=self.rows, **self.pen)
        self.verify = df2.PreparedVerify(self.rows, self.path, None, None, None, temperature=0.0)

    def step(self):
        self.pages()
        self.append()
        x = self.attend().reshape(B * (P + 1), HQ * D).float() @ self.head
        self.rows.copy_(x.view(B, P + 1, V))
        self.raw = self.rows.clone()
        self.adjust()
        return self.verify()

    def feed(self, r, g, step):
        """A step's new tokens, as a drafter would have them, and which requests end."""
        self.qkv.copy_(torch.randn(self.qkv.shape, generator=g).to(BF))
        ends = [step > 2 and r.random() < 0.1 for _ in range(B)]
        self.new.copy_(torch.tensor([-1 if e else P + 1 for e in ends], dtype=torch.int32))
        self.path.copy_(torch.randint(0, V, (B, P), generator=g).to(torch.int32))
        mask = torch.randint(-2**31, 2**31, self.mask.shape, generator=g).to(torch.int32)
        self.mask.copy_(torch.where(torch.rand((B, 1, 1), generator=g) < 0.5, mask, -1))

    def take(self, tokens, counts):
        """What was accepted joins the histories and the next step's lengths, on the device."""
        at = torch.arange(P + 1, device="cuda")
        new = at < counts[:, None]
        alive = self.new >= 0
        spot = torch.where(new & alive[:, None], self.length[:, None].long() + at, 299)
        keep = self.history[:, 299].clone()
        self.history.scatter_(1, spot, tokens)
        self.history[:, 299] = keep
        self.length.copy_(torch.where(alive, (self.length + counts).clamp(max=290), 0))
        self.advance.copy_(torch.where(alive, counts, 0))


def state(x):
    return [t.clone() for t in (x.table, x.held, x.ctx, x.free, x.count, x.history, x.length, x.advance) + tuple(x.cache)]


def test_cycles_step_by_step_against_plain_forms():
    say("serving cycle")
    x, r, g = Loop(1), random.Random(1), torch.Generator().manual_seed(2)
    accepted = 0
    for step in range(9):
        x.feed(r, g, step)
        if step % 2:
            # drafts that the target agrees with: the step is tried first, on copies
            before = state(x)
            x.pages()
            x.append()
            rows = (x.attend().reshape(B * (P + 1), HQ * D).float() @ x.head).view(B, P + 1, V)
            x.path.copy_(rows[:, :P].argmax(-1))
            for t, old in zip((x.table, x.held, x.ctx, x.free, x.count, x.history, x.length, x.advance) + tuple(x.cache), before):
                t.copy_(old)
        want, _ = pages_ref(x.table.tolist(), x.held.tolist(), x.free.tolist(), x.count.item(), x.ctx.tolist(), x.new.tolist(), PAGE,
                            B * (P + 1), x.advance.tolist())
        x.pages()
        for name, t in zip(("start", "ctx", "slots", "positions"), x.pages._out):
            assert t.tolist() == want[name], (step, name)
        assert x.table.tolist() == want["table"] and x.free.tolist() == want["free"] and x.count.tolist() == want["count"]
        c = dict(q=x.append._out, k=x.k, v=x.v, k_norm=x.k_norm, k_cache=x.cache[0], v_cache=x.cache[1], table=x.table, ctx=x.ctx,
                 start=x.start, N=B * (P + 1), page=PAGE)
        bytes_ = appended(c, D, x.freq.cpu().numpy(), False)
        x.append()
        for got, (ref, _) in zip(x.cache, bytes_):
            assert (got.cpu().numpy() == ref).all()
        out = x.attend()
        check(c, out)
        x.rows.copy_((out.reshape(B * (P + 1), HQ * D).float() @ x.head).view(B, P + 1, V))
        raw = x.rows.clone()
        x.adjust()
        args = dict(history=x.history.cpu(), history_len=x.length.cpu(), path=x.path.cpu(), mask=x.mask.cpu(),
                    **{k: v.cpu() for k, v in x.pen.items()})
        check_rows(raw.cpu(), args, x.rows)
        tok, count, p = x.verify()
        ref = verify_ref(x.rows.cpu().float(), x.path.cpu(), None, None, None, 0.0)
        assert tok.tolist() == ref[0].tolist() and count.tolist() == ref[1].tolist()
        accepted += int((count - 1).sum())
        x.take(tok, count)
        assert df2.device_error() == 0
    assert accepted > 0


def test_cycles_captured_and_replayed_equal_eager_ones():
    say("serving cycle captured")
    runs = []
    for captured in (False, True):
        x, r, g = Loop(3), random.Random(4), torch.Generator().manual_seed(5)
        x.feed(r, g, 0)
        # libraries' first calls stay out of the graph; the state is put back
        before = state(x)
        x.step()
        for t, old in zip((x.table, x.held, x.ctx, x.free, x.count, x.history, x.length, x.advance) + tuple(x.cache), before):
            t.copy_(old)
        torch.cuda.synchronize()
        if captured:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                out = x.step()
        trace = []
        for step in range(8):
            x.feed(r, g, step)
            if captured:
                graph.replay()
            else:
                out = x.step()
            x.take(out[0], out[1])
            trace.append([t.clone() for t in out] + state(x))
        runs.append(trace)
        assert df2.device_error() == 0
    for a, b in zip(*runs):
        for s, t in zip(a, b):
            assert torch.equal(s, t)
