"""The serving side of a draft-verify cycle, case by case: what the target model does with a drafted block.

Three operators, each with its plain form in elementary torch operations:

  append  new tokens' queries and keys normed per head and rotated by their positions, keys and values written
          into a paged cache (`kv_append`)
  attend  attention of each sequence's new tokens over its paged cache (`paged_attention`)
  verify  the drafted tokens accepted or rejected against the target's rows, and the next token drawn, from given
          uniforms (`verify`)

Where `own` is true, `run` calls the package's kernels through their prepared calls, as a serving loop does.
"""
import math

import torch

own = False

# ---------------------------------------------------------------------------------------------------------------------
# Cases.
#
# append, attend: B sequences; sequence b has ctx tokens in the cache (spread evenly from ctx_lo to ctx_hi over the
# batch) and n new ones (n_lo to n_hi); Hq query heads share Hkv key/value heads of size D; pages of `page` tokens.
# verify: B sequences with P drafted positions (n_lo to P of them in use), vocabulary V, K candidates a position.
# ---------------------------------------------------------------------------------------------------------------------


def listed():
    return [
        # one verified token and seven drafted ones of a single user: the smallest append, where launch latency counts
        dict(name="append_block_b1", op="append", dtype="bf16", B=1, n_lo=8, n_hi=8, ctx_lo=1003, ctx_hi=1003, Hq=32, Hkv=8,
             D=128, page=16, rot=128, pairs="half", norm=True),
        # a batch's blocks of odd lengths in full precision, half of each head rotated in neighbouring pairs
        dict(name="append_ragged_f32", op="append", dtype="f32", B=37, n_lo=1, n_hi=29, ctx_lo=0, ctx_hi=40001, Hq=12, Hkv=4,
             D=64, page=32, rot=32, pairs="interleaved", norm=False),
        # prompts on their way into the cache
        dict(name="append_prompt", op="append", dtype="bf16", B=3, n_lo=2047, n_hi=8190, ctx_lo=0, ctx_hi=70000, Hq=32, Hkv=8,
             D=128, page=16, rot=128, pairs="half", norm=True),
        # one token of a single user over a short context: latency
        dict(name="attend_decode_b1", op="attend", dtype="bf16", B=1, n_lo=1, n_hi=1, ctx_lo=1003, ctx_hi=1003, Hq=32, Hkv=8,
             D=128, page=16, causal=True, window=0),
        # a drafter's block in full precision: every position of the block sees all of it
        dict(name="attend_block_f32", op="attend", dtype="f32", B=3, n_lo=7, n_hi=8, ctx_lo=17, ctx_hi=2049, Hq=12, Hkv=4,
             D=64, page=32, causal=False, window=0),
        # verification of drafted blocks at concurrency 32, contexts of mixed lengths
        dict(name="attend_verify_b32", op="attend", dtype="bf16", B=32, n_lo=8, n_hi=8, ctx_lo=301, ctx_hi=12007, Hq=64, Hkv=8,
             D=128, page=16, causal=True, window=0),
        # the same over very long contexts
        dict(name="attend_verify_long", op="attend", dtype="bf16", B=4, n_lo=8, n_hi=8, ctx_lo=65501, ctx_hi=131001, Hq=32, Hkv=8,
             D=128, page=64, causal=True, window=0),
        # a chunk of a long prompt: bound by the matrix cores
        dict(name="attend_prompt", op="attend", dtype="bf16", B=2, n_lo=3501, n_hi=4096, ctx_lo=4000, ctx_hi=4097, Hq=32, Hkv=8,
             D=128, page=16, causal=True, window=0),
        # one drafted block of seven against a 151936-token vocabulary: latency
        dict(name="verify_b1", op="verify", dtype="bf16", B=1, P=7, n_lo=7, V=151936, K=16, temperature=1.0),
        # a small vocabulary of odd size in full precision, sequences with fewer drafted tokens among them
        dict(name="verify_ragged_f32", op="verify", dtype="f32", B=5, P=7, n_lo=0, V=32003, K=5, temperature=0.7),
        # concurrency 32
        dict(name="verify_b32", op="verify", dtype="bf16", B=32, P=7, n_lo=7, V=151936, K=16, temperature=1.0),
        # blocks of 16 at a high concurrency and a large vocabulary
        dict(name="verify_stress", op="verify", dtype="bf16", B=64, P=15, n_lo=15, V=262144, K=32, temperature=0.8),
    ]


def _log(rng, lo, hi):
    """A whole number from lo to hi, spread over its logarithm."""
    return int(min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "verify"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op == "verify":
        V = _log(rng, 1000, 262144)
        P = rng.randint(1, 15)
        rows = max(1, (64 * 16 * 262144) // ((P + 1) * V * (1 if dtype == "bf16" else 2)))
        return dict(op=op, dtype=dtype, B=_log(rng, 1, min(64, rows)), P=P, n_lo=rng.choice([0, P]), V=V,
                    K=rng.choice([1, 4, 16, 32]), temperature=rng.choice([0.0, 0.6, 1.0, 1.3]))
    D = rng.choice([64, 128, 128, 256])
    Hkv = rng.choice([1, 2, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 4, 5, 8])
    page = rng.choice([16, 32, 64])
    c = dict(op=op, dtype=dtype, D=D, Hkv=Hkv, Hq=Hq, page=page)
    if op == "append":
        total = _log(rng, 1, 8192)
        B = _log(rng, 1, min(64, total))
        n = max(1, total // B)
        ctx = _log(rng, 1, 65536)
        rot = rng.choice([D, D // 2])
        return dict(c, B=B, n_lo=rng.randint(1, n), n_hi=n, ctx_lo=rng.randint(0, ctx), ctx_hi=ctx, rot=rot,
                    pairs=rng.choice(["half", "half", "interleaved"]), norm=rng.choice([True, False]))
    n = rng.choice([1, _log(rng, 1, 16), _log(rng, 1, 2048)])
    B = _log(rng, 1, max(1, min(32, 2048 // n)))
    # no more scores, and no more cached values, than the largest listed cases have
    most = min(131072, (2 * 32 * 4096 * 8192 // (4 if dtype == "f32" else 1)) // (B * Hq * n) - n,
               (4 * 131072 * 8 * 128) // (B * Hkv * D * (2 if dtype == "f32" else 1)))
    ctx = _log(rng, 1, max(1, most))
    return dict(c, B=B, n_lo=rng.randint(1, n), n_hi=n, ctx_lo=rng.randint(0, ctx), ctx_hi=ctx, causal=rng.choice([True, True, False]),
                window=rng.choice([0, 0, 0, 100, 1024]))


# ---------------------------------------------------------------------------------------------------------------------
# Inputs.
# ---------------------------------------------------------------------------------------------------------------------
_DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _spread(lo, hi, count):
    """`count` whole numbers from lo to hi in an order that mixes short and long."""
    if count == 1:
        return [hi]
    return [lo + (hi - lo) * ((i * 7) % count if count % 7 else i) // (count - 1) for i in range(count)]


def _lengths(case):
    return _spread(case["n_lo"], case["n_hi"], case["B"]), _spread(case["ctx_lo"], case["ctx_hi"], case["B"])


def _paged(case, g):
    """The cache, its page table and the lengths that the append and attention cases share."""
    dt, dev = _DTYPES[case["dtype"]], "cuda"
    B, Hkv, D, page = case["B"], case["Hkv"], case["D"], case["page"]
    new, ctx = _lengths(case)
    pages = [-(-(c + n) // page) for c, n in zip(ctx, new)]
    width, used = max(pages), sum(pages)
    order = torch.randperm(used + 3, generator=g, device=dev).to(torch.int32)
    table = torch.zeros((B, width), dtype=torch.int32)
    at = torch.tensor([0] + pages).cumsum(0).tolist()
    order = order.cpu()
    for b in range(B):
        table[b, :pages[b]] = order[at[b]:at[b + 1]]
    start = torch.tensor([0] + new).cumsum(0).to(torch.int32)
    cache = [torch.randn((used + 3, Hkv, page, D), generator=g, device=dev, dtype=dt) for _ in range(2)]
    return dict(case=case, k_cache=cache[0], v_cache=cache[1], table=table.to(dev), ctx=torch.tensor(ctx, dtype=torch.int32, device=dev),
                start=start.to(dev), N=sum(new), most_new=max(new), most_len=max(c + n for c, n in zip(ctx, new)))


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 17)
    dt, dev = _DTYPES[case["dtype"]], "cuda"
    if case["op"] == "verify":
        return _prepare_verify(case, g)
    s = _paged(case, g)
    N, Hq, Hkv, D = s["N"], case["Hq"], case["Hkv"], case["D"]
    if case["op"] == "append":
        # the projection's output, queries, keys and values side by side in each token's row
        qkv = 3 * torch.randn((N, Hq + 2 * Hkv, D), generator=g, device=dev, dtype=dt)
        s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        s["q_norm"] = s["k_norm"] = None
        if case["norm"]:
            s["q_norm"] = (1 + 0.2 * torch.randn((D,), generator=g, device=dev)).to(dt)
            s["k_norm"] = (1 + 0.2 * torch.randn((D,), generator=g, device=dev)).to(dt)
        half = case["rot"] // 2
        s["freq"] = 1e6 ** (-torch.arange(half, dtype=torch.float64, device=dev) / half)
        if own:
            import draft_selection_topk16_amd as df2
            s["call"] = df2.PreparedAppend(s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["ctx"], s["start"], q=s["q"],
                                           q_norm=s["q_norm"], k_norm=s["k_norm"], eps=1e-6, rope_freq=s["freq"],
                                           interleaved=case["pairs"] == "interleaved")
        return s
    s["q"] = 2 * torch.randn((N, Hq, D), generator=g, device=dev, dtype=dt)
    if own:
        import draft_selection_topk16_amd as df2
        s["call"] = df2.PreparedAttention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["ctx"], s["start"],
                                          causal=case["causal"], window=case["window"], max_len=s["most_len"])
    return s


def _prepare_verify(case, g):
    dt, dev = _DTYPES[case["dtype"]], "cuda"
    B, P, V, K = case["B"], case["P"], case["V"], case["K"]
    # distinct candidates: one in each of K stretches of the vocabulary, in random order
    step = V // K
    ids = torch.arange(K, device=dev) * step + torch.randint(0, step, (B, P, K), generator=g, device=dev)
    ids = ids.gather(-1, torch.rand((B, P, K), generator=g, device=dev).argsort(-1))
    # the drafter's scores, and a target whose scores of the same tokens are near them, above a broad rest
    score = 2.5 * torch.randn((B, P, K), generator=g, device=dev)
    target = torch.randn((B, P + 1, V), generator=g, device=dev, dtype=torch.float32).mul_(1.5)
    lift = 11.0 + score + 0.6 * torch.randn((B, P, K), generator=g, device=dev)
    target[:, :P].scatter_(2, ids, lift)
    prob = torch.softmax(score, -1)
    pick = (prob.cumsum(-1) < torch.rand((B, P, 1), generator=g, device=dev)).sum(-1, keepdim=True).clamp_(max=K - 1)
    # each position's draft is one of its candidates, or of them the target's best half the time
    best = lift.argmax(-1, keepdim=True)
    pick = torch.where(torch.rand((B, P, 1), generator=g, device=dev) < 0.5, best, pick)
    s = dict(case=case, target=target.to(dt), cand=ids.to(torch.int32), prob=prob.contiguous(),
             path=ids.gather(-1, pick).squeeze(-1).to(torch.int32).contiguous(),
             u=torch.randint(0, 1 << 24, (B, P + 1), generator=g, device=dev).to(torch.float32) / (1 << 24),
             drafted=torch.tensor(_spread(case["n_lo"], P, B), dtype=torch.int32, device=dev))
    if own:
        import draft_selection_topk16_amd as df2
        s["call"] = df2.PreparedVerify(s["target"], s["path"], s["cand"], s["prob"], s["u"], temperature=case["temperature"],
                                       n_draft=s["drafted"])
    return s


# ---------------------------------------------------------------------------------------------------------------------
# The operators.
# ---------------------------------------------------------------------------------------------------------------------
def run(state):
    op = state["case"]["op"]
    if own:
        r = state["call"]()
        return (r, state["k_cache"], state["v_cache"]) if op == "append" else r
    return {"append": _append, "attend": _attend, "verify": _verify}[op](state)


def _places(s):
    """Each new token's sequence and position, and where the cache holds it."""
    start, page = s["start"].long(), s["case"]["page"]
    tok = torch.arange(s["N"], device=start.device)
    seq = torch.searchsorted(start, tok, right=True) - 1
    pos = s["ctx"].long()[seq] + tok - start[seq]
    return seq, pos, s["table"].long()[seq, pos // page], pos % page


def _append(s):
    case = s["case"]
    seq, pos, pages, slots = _places(s)
    half, dt = case["rot"] // 2, s["q"].dtype
    angle = pos.double()[:, None] * s["freq"]          # 64 bits: far positions
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def turned(x, weight):
        x = x.float()
        if weight is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * weight.float()
        r = x[..., :case["rot"]]
        if case["pairs"] == "half":
            a, b = r[..., :half], r[..., half:]
            r = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
        else:
            a, b = r[..., 0::2], r[..., 1::2]
            r = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
        return torch.cat((r, x[..., case["rot"]:]), -1).to(dt)

    s["k_cache"][pages, :, slots] = turned(s["k"], s["k_norm"])
    s["v_cache"][pages, :, slots] = s["v"]
    return turned(s["q"], s["q_norm"]), s["k_cache"], s["v_cache"]


def _attend(s):
    case, B = s["case"], s["case"]["B"]
    Hq, Hkv, D, page = case["Hq"], case["Hkv"], case["D"], case["page"]
    G, n, dev = Hq // Hkv, s["most_new"], s["q"].device
    width = -(-s["most_len"] // page)
    table = s["table"][:, :width].long()
    k = s["k_cache"][table].float().permute(0, 2, 1, 3, 4).reshape(B, Hkv, width * page, D)
    v = s["v_cache"][table].float().permute(0, 2, 1, 3, 4).reshape(B, Hkv, width * page, D)
    seq, pos, _, _ = _places(s)
    row = torch.arange(s["N"], device=dev) - s["start"].long()[seq]
    q = torch.zeros((B, n, Hq, D), device=dev)
    q[seq, row] = s["q"].float()
    q = q.view(B, n, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * n, D)
    w = torch.matmul(q, k.transpose(-1, -2).contiguous()).mul_(1.0 / math.sqrt(D))
    # which keys each new token sees
    key = torch.arange(width * page, device=dev)
    at = s["ctx"].long()[:, None] + torch.arange(n, device=dev)
    end = s["ctx"].long() + s["start"].long().diff()
    hidden = key >= end[:, None, None]
    if case["causal"]:
        hidden = hidden | (key > at[:, :, None])
    if case["window"]:
        hidden = hidden | (key <= at[:, :, None] - case["window"])
    w = w.view(B, Hkv, G, n, -1).masked_fill_(hidden.expand(B, n, -1)[:, None, None], -math.inf)
    top = w.amax(-1, keepdim=True).clamp_(min=torch.finfo(torch.float32).min)
    w = w.sub_(top).exp_()
    total = w.sum(-1, keepdim=True)
    out = torch.matmul(w.view(B, Hkv, G * n, -1), v).view(B, Hkv, G, n, D) / total.clamp(min=1e-30)
    out = out.permute(0, 3, 1, 2, 4).reshape(B, n, Hq, D)
    return out[seq, row].to(s["q"].dtype)


def _verify(s):
    case, x, P = s["case"], s["target"], s["case"]["P"]
    B, V, tau = case["B"], case["V"], case["temperature"]
    dev = x.device
    x = x.float()
    top, first = x.max(-1, keepdim=True)
    at = s["path"].long()[..., None]
    if tau == 0:
        # the lowest token of the largest value
        best = torch.where(x == top, torch.arange(V, device=dev), V).amin(-1)
        yes = best[:, :P] == s["path"]
    else:
        total = ((x - top) / tau).exp_().sum(-1, dtype=torch.float64)
        here = ((x[:, :P].gather(-1, at) - top[:, :P]).double() / tau).exp().squeeze(-1) / total[:, :P]
        q = (s["prob"].double() * (s["cand"] == s["path"][..., None])).sum(-1)
        yes = s["u"][:, :P].double() * q < here
    drafted = s["drafted"].long()
    yes = yes & (torch.arange(P, device=dev) < drafted[:, None])
    taken = yes.long().cumprod(-1).sum(-1)
    rows = torch.arange(B, device=dev)
    place = torch.arange(P + 1, device=dev)
    if tau == 0:
        token, chance = best[rows, taken], torch.ones((B,), device=dev)
        odds = torch.ones((B, P), device=dev)
    else:
        # the last row in 64 bits: running sums next to the given number
        last = ((x[rows, taken] - top[rows, taken]).double() / tau).exp_()
        last = last / last.sum(-1, keepdim=True)
        left = last.clone()
        t = taken.clamp(max=P - 1)
        cut = torch.where((taken < drafted)[:, None], s["prob"][rows, t].double(), 0.0)
        left = left.scatter_add_(-1, s["cand"][rows, t].long(), -cut).clamp_(min=0)
        run_sum = left.cumsum(-1)
        token = (run_sum <= s["u"][:, P:].double() * run_sum[:, -1:]).sum(-1).clamp_(max=V - 1)
        chance, odds = last[rows, token].float(), here.float()
    tokens = torch.cat((s["path"].long(), torch.zeros_like(s["path"][:, :1]).long()), 1)
    odds = torch.cat((odds, torch.zeros_like(odds[:, :1])), 1)
    tokens[rows, taken], odds[rows, taken] = token, chance
    gone = place > taken[:, None]
    return tokens.masked_fill(gone, -1).to(torch.int32), (taken + 1).to(torch.int32), odds.masked_fill(gone, 0.0)


# ---------------------------------------------------------------------------------------------------------------------
# What a pass cannot do without.
# ---------------------------------------------------------------------------------------------------------------------
def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "verify":
        B, P, V, K = case["B"], case["P"], case["V"], case["K"]
        rows = B * (P + 1)
        # every row's values once; candidates, probabilities, drafts, uniforms and outputs beside them
        return {"bytes": rows * V * size + B * P * (8 * K + 4) + 4 * B + rows * 12 + 4 * B, "flops": 4 * rows * V}
    new, ctx = _lengths(case)
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    N = sum(new)
    if case["op"] == "append":
        # queries, keys and values read and written once
        return {"bytes": 2 * N * (Hq + 2 * Hkv) * D * size + 4 * case["rot"], "flops": N * (Hq + Hkv) * D * 8}
    keys, pairs = 0, 0
    for n, c in zip(new, ctx):
        low = max(0, c + 1 - case["window"]) if case["window"] else 0
        keys += c + n - low
        for t in range(n):
            end = c + t + 1 if case["causal"] else c + n
            pairs += end - (max(0, c + t + 1 - case["window"]) if case["window"] else 0)
    return {"bytes": (2 * N * Hq + 2 * keys * Hkv) * D * size, "flops": 4 * pairs * Hq * D}


# ---------------------------------------------------------------------------------------------------------------------
# The definitions in 64 bits, one sequence (and head) at a time.
# ---------------------------------------------------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "attend": _exact_attend, "verify": _exact_verify}[case["op"]](s)


def _exact_append(s):
    case, page, rot = s["case"], s["case"]["page"], s["case"]["rot"]
    i = torch.arange(rot // 2, device="cuda")
    one, two = (i, i + rot // 2) if case["pairs"] == "half" else (2 * i, 2 * i + 1)
    kc, vc, out = s["k_cache"].double(), s["v_cache"].double(), s["q"].double()
    begin, ctx, table = s["start"].tolist(), s["ctx"].tolist(), s["table"].tolist()

    def head(x, weight, turn):
        y = x.double()
        if weight is not None:
            y = y / torch.sqrt(torch.mean(y ** 2, dim=-1, keepdim=True) + 1e-6) * weight.double()
        z = torch.view_as_complex(torch.stack((y[..., one], y[..., two]), -1).contiguous()) * turn
        y = y.clone()
        y[..., one], y[..., two] = z.real, z.imag
        return y

    for b in range(case["B"]):
        rows = slice(begin[b], begin[b + 1])
        p = torch.arange(ctx[b], ctx[b] + begin[b + 1] - begin[b], device="cuda", dtype=torch.float64)
        turn = torch.polar(torch.ones((len(p), rot // 2), dtype=torch.float64, device="cuda"), torch.outer(p, s["freq"]))[:, None, :]
        out[rows] = head(s["q"][rows], s["q_norm"], turn)
        where = torch.tensor(table[b], device="cuda")[p.long() // page]
        kc[where, :, p.long() % page] = head(s["k"][rows], s["k_norm"], turn)
        vc[where, :, p.long() % page] = s["v"][rows].double()
    return out, kc, vc


def _exact_attend(s):
    case, page = s["case"], s["case"]["page"]
    G = case["Hq"] // case["Hkv"]
    out = torch.zeros((s["N"], case["Hq"], case["D"]), dtype=torch.float64, device="cuda")
    begin, ctx = s["start"].tolist(), s["ctx"].tolist()
    for b in range(case["B"]):
        n, c = begin[b + 1] - begin[b], ctx[b]
        if n == 0:
            continue
        ids = s["table"][b, :-(-(c + n) // page)].long()
        j, i = torch.arange(c + n, device="cuda")[None], c + torch.arange(n, device="cuda")[:, None]
        sees = torch.ones((n, c + n), dtype=torch.bool, device="cuda")
        if case["causal"]:
            sees &= j <= i
        if case["window"]:
            sees &= i - j < case["window"]
        for h in range(case["Hkv"]):
            k = s["k_cache"][ids, h].reshape(-1, case["D"])[:c + n].double()
            v = s["v_cache"][ids, h].reshape(-1, case["D"])[:c + n].double()
            for head in range(h * G, h * G + G):
                a = (s["q"][begin[b]:begin[b + 1], head].double() @ k.T) / math.sqrt(case["D"])
                a = torch.softmax(torch.where(sees, a, -math.inf), -1)
                out[begin[b]:begin[b + 1], head] = a @ v
    return out


def _exact_verify(s):
    case, P, V, tau = s["case"], s["case"]["P"], s["case"]["V"], s["case"]["temperature"]
    tokens = torch.full((case["B"], P + 1), -1, dtype=torch.int32)
    count = torch.zeros((case["B"],), dtype=torch.int32)
    odds = torch.zeros((case["B"], P + 1), dtype=torch.float64)
    path, cand, prob = s["path"].tolist(), s["cand"].tolist(), s["prob"].double().tolist()
    u, drafted = s["u"].double().tolist(), s["drafted"].tolist()
    for b in range(case["B"]):
        x = s["target"][b].double()
        if tau == 0:
            p = torch.zeros_like(x)
            p[torch.arange(P + 1, device="cuda"), torch.argmax((x == x.amax(-1, keepdim=True)).to(torch.int8), -1)] = 1.0
        else:
            p = torch.softmax(x / tau, -1)
        ps = p[torch.arange(P, device="cuda"), s["path"][b].long()].tolist()
        t, rest = 0, None
        while t < drafted[b]:
            q = dict(zip(cand[b][t], prob[b][t]))
            if tau == 0:
                ok = ps[t] == 1.0
            else:
                ok = u[b][t] * q[path[b][t]] < ps[t]
            if not ok:
                rest = q
                break
            tokens[b, t], odds[b, t] = path[b][t], ps[t]
            t += 1
        left = p[t].clone()
        if rest is not None and tau != 0:
            at = torch.tensor(list(rest), device="cuda")
            left[at] = torch.clamp(left[at] - torch.tensor(list(rest.values()), dtype=torch.float64, device="cuda"), min=0.0)
        sums = torch.cumsum(left, 0)
        y = int(torch.searchsorted(sums, (u[b][P] * sums[-1]).reshape(1), right=True))
        y = min(y, V - 1) if tau != 0 else int(torch.argmax(left))
        tokens[b, t], odds[b, t], count[b] = y, float(p[t, y]), t + 1
    return tokens.cuda(), count.cuda(), odds.cuda()
