"""More of the serving side of a draft-verify cycle, case by case.

Operators, each with its plain form in elementary torch operations:

  pages   block tables, token starts and slot maps of the next step made on the GPU from the lengths of the requests
          (`plan_pages`)
  append  new tokens' queries and keys normed per head and rotated by their positions, keys and values written into a
          paged cache that holds them in 4 bits, in blocks of 32 with a power of two as their scale
          (`kv_append_fp4`; what the cache then holds comes from `kv_unpack_fp4`)
  attend  attention of each sequence's new tokens over its 4-bit paged cache (`paged_attention_fp4`)
  adjust  penalties for repeated tokens, biases and grammar masks on the target's rows (`adjust_logits`)

Where `own` is true, `run` calls the package's kernels through their prepared calls, as a serving loop does.
"""
import math

import torch

own = False

# ---------------------------------------------------------------------------------------------------------------------
# Cases.
#
# pages: B requests of which each holds ctx tokens (ctx_lo to ctx_hi), takes 1 to `block` of the last block's tokens
# over and asks for n_lo to n_hi new ones, every `ends`-th is finished (0: none); `spare`: free pages per request.
# append, attend: B sequences; sequence b has ctx tokens in the cache (spread evenly from ctx_lo to ctx_hi over the
# batch) and n new ones (n_lo to n_hi); Hq query heads share Hkv key/value heads of size D; pages of `page` tokens.
# adjust: B sequences with R rows of a vocabulary V, the tokens drafted between them, histories of L_lo to L_hi tokens,
# M biases each; mask: "none", "few" (a grammar that allows few tokens), "most" (one that forbids few) or "mixed".
# ---------------------------------------------------------------------------------------------------------------------


def listed():
    return [
        # a handful of users, a block of eight tokens each: the smallest step, where launch latency counts
        dict(name="pages_b4", op="pages", B=4, page=16, ctx_lo=300, ctx_hi=4003, n_lo=8, n_hi=8, block=8, ends=0, spare=2.0),
        # a large server's step: thousands of requests, blocks and pieces of prompts among them, some of them finished
        dict(name="pages_b3000", op="pages", B=3000, page=16, ctx_lo=0, ctx_hi=8191, n_lo=1, n_hi=61, block=8, ends=17, spare=2.5),
        # a batch's blocks of odd lengths in full precision, half of each head rotated in neighbouring pairs
        dict(name="append_ragged_f32", op="append", dtype="f32", B=37, n_lo=1, n_hi=29, ctx_lo=0, ctx_hi=401, Hq=12, Hkv=4,
             D=64, page=32, rot=32, pairs="interleaved", norm=False),
        # prompts on their way into the cache
        dict(name="append_prompt", op="append", dtype="bf16", B=3, n_lo=2047, n_hi=8190, ctx_lo=0, ctx_hi=1500, Hq=32, Hkv=8,
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
        # single tokens over very long contexts
        dict(name="attend_decode_long", op="attend", dtype="bf16", B=4, n_lo=1, n_hi=1, ctx_lo=65501, ctx_hi=131001, Hq=32, Hkv=8,
             D=128, page=64, causal=True, window=0),
        # a chunk of a long prompt: bound by the matrix cores
        dict(name="attend_prompt", op="attend", dtype="bf16", B=2, n_lo=3501, n_hi=4096, ctx_lo=4000, ctx_hi=4097, Hq=32, Hkv=8,
             D=128, page=16, causal=True, window=0),
        # the rows of one drafted block of seven, a short history: latency
        dict(name="adjust_b1", op="adjust", dtype="bf16", B=1, R=8, V=151936, L_lo=1003, L_hi=1003, M=5, mask="none", place=False),
        # a small vocabulary of odd size in full precision under a grammar
        dict(name="adjust_ragged_f32", op="adjust", dtype="f32", B=5, R=8, V=32003, L_lo=1, L_hi=5001, M=300, mask="most", place=False),
        # concurrency 64 in place, long histories, half of the requests under a grammar that allows few tokens
        dict(name="adjust_b64", op="adjust", dtype="bf16", B=64, R=8, V=151936, L_lo=301, L_hi=12007, M=16, mask="mixed", place=True),
    ]


def _log(rng, lo, hi):
    """A whole number from lo to hi, spread over its logarithm."""
    return int(min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["pages", "append", "attend", "attend", "adjust"])
    if op == "pages":
        B = _log(rng, 1, 3000)
        n, page = _log(rng, 1, max(1, min(2048, 90000 // B))), rng.choice([1, 16, 16, 32, 64])
        return dict(op=op, B=B, page=page, ctx_lo=0, ctx_hi=_log(rng, 1, min(131072, page * 1500000 // B)),
                    n_lo=rng.randint(0, n), n_hi=n, block=rng.choice([1, 8, 16]), ends=rng.choice([0, 3, 17]), spare=rng.choice([0.3, 1.0, 4.0]))
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op == "adjust":
        V = _log(rng, 1000, 262144)
        R = rng.randint(1, 16)
        B = _log(rng, 1, max(1, min(64, (64 * 8 * 151936) // (2 * R * V * (1 if dtype == "bf16" else 2)))))
        L = _log(rng, 1, 16384)
        return dict(op=op, dtype=dtype, B=B, R=R, V=V, L_lo=rng.randint(0, L), L_hi=L, M=rng.choice([0, 5, 300]),
                    mask=rng.choice(["none", "few", "most", "mixed"]), place=rng.choice([True, False]))
    D = rng.choice([64, 128, 128, 256])
    Hkv = rng.choice([1, 2, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 4, 5, 8])
    page = rng.choice([16, 32, 64])
    c = dict(op=op, dtype=dtype, D=D, Hkv=Hkv, Hq=Hq, page=page)
    if op == "append":
        total = _log(rng, 1, 4096)
        B = _log(rng, 1, min(64, total))
        n = max(1, total // B)
        ctx = _log(rng, 1, 16384 // B)
        return dict(c, B=B, n_lo=rng.randint(1, n), n_hi=n, ctx_lo=rng.randint(0, ctx), ctx_hi=ctx, rot=rng.choice([D, D // 2]),
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
# 4-bit values: sign and one of eight magnitudes, two to a byte (the first in the low half), in blocks of 32 elements of
# a head that share a power of two, held as its exponent plus 127.  The power is the smallest, of 2^-120 to 2^120, of
# which the largest magnitude is at most 7; values are rounded to the nearest, ties to the even code.  A page holds, for
# each head, its tokens' codes (D / 2 bytes each), then their scales (D / 32 bytes each).
# ---------------------------------------------------------------------------------------------------------------------
_MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _codes(x):
    """Codes [..., D / 2] and scales [..., D / 32], as bytes, of float64 values [..., D]."""
    y = x.unflatten(-1, (-1, 32))
    m, e = torch.frexp(y.abs().amax(-1))                # m 2^e, 1/2 <= m < 1
    e = torch.where(8 * m <= 7, e - 3, e - 2).clamp(-120, 120)
    y = y * ((1023 - e.long()) << 52).view(torch.float64)[..., None]
    a = y.abs()
    code = torch.zeros_like(a, dtype=torch.uint8)
    for i in range(7):
        border = (_MAGNITUDES[i] + _MAGNITUDES[i + 1]) / 2
        code += (a > border) if i % 2 == 0 else (a >= border)
    code += 8 * torch.signbit(y).to(torch.uint8)
    code = code.flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), (e + 127).to(torch.uint8)


def _values(cache, page, D):
    """The values that pages [pages, Hkv, bytes] of a 4-bit cache stand for: [pages, Hkv, page, D] float32."""
    codes, scales = cache.split((page * D // 2, page * D // 32), -1)
    grid = torch.tensor(_MAGNITUDES + tuple(-x for x in _MAGNITUDES), device=cache.device)
    x = grid[torch.stack((codes & 15, codes >> 4), -1).int()].view(cache.shape[:2] + (page, D // 32, 32))
    power = (scales.int() << 23).view(torch.float32).view(cache.shape[:2] + (page, D // 32, 1))
    return (x * power).flatten(-2)


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
    dev = "cuda"
    B, Hkv, D, page = case["B"], case["Hkv"], case["D"], case["page"]
    new, ctx = _lengths(case)
    pages = [-(-(c + n) // page) for c, n in zip(ctx, new)]
    width, used = max(pages), sum(pages)
    order = torch.randperm(used + 3, generator=g, device=dev).to(torch.int32).cpu()
    table = torch.zeros((B, width), dtype=torch.int32)
    at = torch.tensor([0] + pages).cumsum(0).tolist()
    for b in range(B):
        table[b, :pages[b]] = order[at[b]:at[b + 1]]
    start = torch.tensor([0] + new).cumsum(0).to(torch.int32)
    cache = []
    for _ in range(2):
        # keys and values as a model has them, made 4-bit some pages at a time
        bytes_ = torch.empty((used + 3, Hkv, page * (D // 2 + D // 32)), dtype=torch.uint8, device=dev)
        step = max(1, (1 << 24) // (Hkv * page * D))
        for p in range(0, used + 3, step):
            part = bytes_[p:p + step]
            codes, scales = _codes(torch.randn((len(part), Hkv, page, D), generator=g, device=dev).double())
            part[..., :page * D // 2] = codes.flatten(-2)
            part[..., page * D // 2:] = scales.flatten(-2)
        cache.append(bytes_)
    return dict(case=case, k_cache=cache[0], v_cache=cache[1], table=table.to(dev), ctx=torch.tensor(ctx, dtype=torch.int32, device=dev),
                start=start.to(dev), N=sum(new), most_new=max(new), most_len=max(c + n for c, n in zip(ctx, new)))


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 17)
    if case["op"] == "pages":
        return _prepare_pages(case, g)
    dt, dev = _DTYPES[case["dtype"]], "cuda"
    if case["op"] == "adjust":
        return _prepare_adjust(case, g)
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
            s["call"] = df2.PreparedAppendFp4(s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["ctx"], s["start"], q=s["q"],
                                              q_norm=s["q_norm"], k_norm=s["k_norm"], eps=1e-6, rope_freq=s["freq"],
                                              interleaved=case["pairs"] == "interleaved")
            s["held"] = df2.PreparedUnpackFp4(s["k_cache"], s["v_cache"], D)
        return s
    s["q"] = 2 * torch.randn((N, Hq, D), generator=g, device=dev, dtype=dt)
    if own:
        import draft_selection_topk16_amd as df2
        s["call"] = df2.PreparedAttentionFp4(s["q"], s["k_cache"], s["v_cache"], s["table"], s["ctx"], s["start"],
                                             causal=case["causal"], window=case["window"], max_len=s["most_len"])
    return s


def _prepare_pages(case, g):
    dev, B, page = "cuda", case["B"], case["page"]
    new, ctx = _lengths(case)
    order = torch.randperm(B, generator=g, device=dev)
    ctx = torch.tensor(ctx, device=dev)[order]
    new = torch.tensor(new, device=dev)
    if case["ends"]:
        new = torch.where(torch.arange(B, device=dev) % case["ends"] == case["ends"] - 1, -1, new)
    # each holds the pages of its context and of the last block, of which some tokens were accepted
    taken = torch.randint(1, case["block"] + 1, (B,), generator=g, device=dev)
    held = (ctx + case["block"] + page - 1) // page
    width = (case["ctx_hi"] + case["block"] + max(case["n_hi"], 1) + page - 1) // page
    used = int(held.sum())
    spare = int(case["spare"] * B) + 1
    ids = torch.randperm(used + spare, generator=g, device=dev).to(torch.int32)
    table = torch.full((B, width), -1, dtype=torch.int32, device=dev)
    have = torch.arange(width, device=dev) < held[:, None]
    table[have] = ids[:used]
    free = torch.full((used + spare,), -1, dtype=torch.int32, device=dev)
    free[:spare] = ids[used:]
    s = dict(case=case, table=table, held=held.to(torch.int32), ctx=ctx.to(torch.int32), advance=taken.to(torch.int32),
             new=new.to(torch.int32), free=free, count=torch.tensor([spare], dtype=torch.int32, device=dev),
             rows=int(new.clamp(min=0).sum()) + 5)
    if own:
        import draft_selection_topk16_amd as df2
        s["call"] = df2.PreparedPages(s["table"], s["held"], s["free"], s["count"], s["ctx"], s["new"], page, s["rows"],
                                      advance=s["advance"])
    return s


def _prepare_adjust(case, g):
    dt, dev = _DTYPES[case["dtype"]], "cuda"
    B, R, V, M = case["B"], case["R"], case["V"], case["M"]
    length = torch.tensor(_spread(case["L_lo"], case["L_hi"], B), dtype=torch.int32, device=dev)
    # texts repeat themselves: token ids spread over their logarithm, a few of them often
    most = max(1, case["L_hi"])
    ids = torch.randperm(V, generator=g, device=dev)
    rank = torch.exp(torch.rand((B, most + R - 1), generator=g, device=dev) * math.log(V)).long().clamp(1, V) - 1
    text = ids[rank].to(torch.int32)
    x = torch.randn((B, R, V), generator=g, device=dev).mul_(2.5)
    x.scatter_(2, text[:, None, :min(most, 64)].long().expand(B, R, -1), 9.0)
    s = dict(case=case, logits=x.to(dt), history=text[:, :most].contiguous(), length=length, prompt=(length // 3).contiguous(),
             path=text[:, most:].contiguous() if R > 1 else None,
             repetition=1 + 0.3 * torch.rand((B,), generator=g, device=dev), frequency=0.5 * torch.rand((B,), generator=g, device=dev),
             presence=0.7 * torch.rand((B,), generator=g, device=dev), bias_token=None, bias=None, mask=None)
    if M:
        # distinct tokens: one in each of M stretches of the vocabulary
        s["bias_token"] = (torch.arange(M, device=dev) * (V // M) + torch.randint(0, V // M, (B, M), generator=g, device=dev)).to(torch.int32)
        s["bias"] = 4 * torch.randn((B, M), generator=g, device=dev)
    if case["mask"] != "none":
        words = (V + 31) // 32
        a, b, c = (torch.randint(-2**31, 2**31, (B, R, words), generator=g, device=dev) for _ in range(3))
        few = (a & b & c & torch.where(torch.rand((B, R, words), generator=g, device=dev) < 0.02, -1, 0))
        few[..., 0] |= 1
        most_ = a | b | c | torch.where(torch.rand((B, R, words), generator=g, device=dev) < 0.7, -1, 0)
        if case["mask"] == "mixed":
            most_ = torch.where((torch.arange(B, device=dev) % 2 == 0)[:, None, None], few, -1)
        s["mask"] = (few if case["mask"] == "few" else most_).to(torch.int32)
    if own:
        import draft_selection_topk16_amd as df2
        s["call"] = df2.PreparedAdjust(s["logits"], history=s["history"], history_len=s["length"], prompt_len=s["prompt"], path=s["path"],
                                       repetition=s["repetition"], frequency=s["frequency"], presence=s["presence"],
                                       bias_token=s["bias_token"], bias=s["bias"], mask=s["mask"],
                                       out=s["logits"] if case["place"] else None)
    return s


# ---------------------------------------------------------------------------------------------------------------------
# The operators.
# ---------------------------------------------------------------------------------------------------------------------
def run(state):
    op = state["case"]["op"]
    if own:
        r = state["call"]()
        if op == "pages":
            return r, state["table"], state["held"], state["free"], state["count"]
        return (r, state["held"]()) if op == "append" else r
    return {"pages": _pages, "append": _append, "attend": _attend, "adjust": _adjust}[op](state)


def _pages(s):
    """Pages that a request no longer needs go back to the free list, in the order of the requests; missing ones come
    from its end.  A request is served while the pages and the rows that requests up to it ask for are there."""
    page, rows = s["case"]["page"], s["rows"]
    table, free = s["table"], s["free"]
    B, width = table.shape
    dev = table.device
    new, held, count = s["new"].long(), s["held"].long(), s["count"].long()
    ctx = torch.where(new < 0, 0, s["ctx"].long() + s["advance"].long())
    n = new.clamp(min=0)
    want = (ctx + n + page - 1) // page
    n, want = torch.where(want > width, 0, n), torch.where(want > width, held, want)
    ask = (want - held).clamp(min=0)
    # released pages, in the order of requests and positions
    at = torch.arange(width, device=dev)
    gone = (at >= want[:, None]) & (at < held[:, None])
    back = table[gone]
    free.scatter_(0, count + torch.arange(len(back), device=dev), back)
    count = count + len(back)
    table.masked_fill_(gone, -1)
    served = (ask.cumsum(0) <= count) & (n.cumsum(0) <= rows)
    n, ask = torch.where(served, n, 0), torch.where(served, ask, 0)
    first = ask.cumsum(0) - ask
    fresh = (at >= held[:, None]) & (at < (held + ask)[:, None])
    which = (count - 1 - first)[:, None] - (at - held[:, None])
    table.copy_(torch.where(fresh, free[which.clamp(0, len(free) - 1)], table))
    s["held"].copy_(torch.minimum(held, want) + ask)
    s["count"].copy_(count - ask.sum())
    start = torch.cat((n.new_zeros(1), n.cumsum(0)))
    row = torch.arange(rows, device=dev)
    seq = (torch.searchsorted(start, row, right=True) - 1).clamp(max=B - 1)
    pos = ctx[seq] + row - start[seq]
    used = row < start[-1]
    slot = table.long()[seq, (pos // page).clamp(max=width - 1)] * page + pos % page
    return ((start.to(torch.int32), ctx.to(torch.int32), torch.where(used, slot, -1), torch.where(used, pos, -1).to(torch.int32)),
            table, s["held"], free, s["count"])


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
    half, dt, page, D = case["rot"] // 2, s["q"].dtype, case["page"], case["D"]
    angle = pos.double()[:, None] * s["freq"]          # 64 bits: far positions, and values next to a border of two codes
    cos, sin = angle.cos()[:, None], angle.sin()[:, None]
    eps = float(torch.tensor(1e-6))

    def turned(x, weight):
        x = x.double()
        if weight is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * weight.double()
        r = x[..., :case["rot"]]
        if case["pairs"] == "half":
            a, b = r[..., :half], r[..., half:]
            r = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
        else:
            a, b = r[..., 0::2], r[..., 1::2]
            r = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
        return torch.cat((r, x[..., case["rot"]:]), -1)

    held = []
    for cache, x in ((s["k_cache"], turned(s["k"], s["k_norm"])), (s["v_cache"], s["v"].double())):
        codes, scales = _codes(x)
        cache[..., :page * D // 2].unflatten(-1, (page, -1))[pages, :, slots] = codes
        cache[..., page * D // 2:].unflatten(-1, (page, -1))[pages, :, slots] = scales
        held.append(_values(cache, page, D).to(torch.bfloat16))        # as exact as in 32 bits
    return turned(s["q"], s["q_norm"]).to(dt), tuple(held)


def _attend(s):
    case, B = s["case"], s["case"]["B"]
    Hq, Hkv, D, page = case["Hq"], case["Hkv"], case["D"], case["page"]
    G, n, dev = Hq // Hkv, s["most_new"], s["q"].device
    width = -(-s["most_len"] // page)
    table = s["table"][:, :width].long()
    k, v = (_values(s[c], page, D)[table].permute(0, 2, 1, 3, 4).reshape(B, Hkv, width * page, D) for c in ("k_cache", "v_cache"))
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


def _adjust(s):
    case, x = s["case"], s["logits"]
    B, R, V, dev = case["B"], case["R"], case["V"], x.device
    at = torch.arange(s["history"].shape[1], device=dev)
    there, text = at < s["length"][:, None], s["history"].long()
    seen = torch.zeros((B, V), device=dev).scatter_add_(1, text, there.float())
    times = torch.zeros((B, V), device=dev).scatter_add_(1, text, (there & (at >= s["prompt"][:, None])).float())
    seen, times = seen[:, None].expand(B, R, V), times[:, None]
    if R > 1:
        # tokens drafted before a row count as generated
        first = torch.zeros((B, R, V), device=dev)
        first[:, 1:].scatter_(2, s["path"].long()[:, :, None], 1.0)
        drafted = first.cumsum_(1)
        times, seen = times + drafted, seen + drafted
    per = lambda t: t[:, None, None]  # noqa: E731
    y = x.float()
    y = torch.where(seen > 0, torch.where(y > 0, y / per(s["repetition"]), y * per(s["repetition"])), y)
    y = y - per(s["frequency"]) * times
    y = y - per(s["presence"]) * (times > 0)
    if s["bias"] is not None:
        y = y + torch.zeros((B, V), device=dev).scatter_(1, s["bias_token"].long(), s["bias"])[:, None]
    if s["mask"] is not None:
        bits = (s["mask"][..., None] >> torch.arange(32, device=dev, dtype=torch.int32)) & 1
        y = y.masked_fill_(bits.flatten(-2)[..., :V] == 0, -math.inf)
    return x.copy_(y) if case["place"] else y.to(x.dtype)


# ---------------------------------------------------------------------------------------------------------------------
# What a pass cannot do without.
# ---------------------------------------------------------------------------------------------------------------------
def work(case):
    new, ctx = _lengths(case) if case["op"] != "adjust" else (None, None)
    if case["op"] == "pages":
        B, rows = case["B"], sum(new)
        # lengths, advances, requests and page counts read, starts, lengths and counts written; a slot and a position a
        # row; the pages that hold a request's new tokens read
        return {"bytes": 32 * B + 12 * rows + 4 * sum(n // case["page"] + 1 for n in new), "flops": 8 * B + 8 * rows}
    size = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "adjust":
        B, R, V, M = case["B"], case["R"], case["V"], case["M"]
        lengths = _spread(case["L_lo"], case["L_hi"], B)
        lists = 4 * sum(lengths) + B * (8 * M + 4 * R + 24)
        masks = 0 if case["mask"] == "none" else 4 * B * R * ((V + 31) // 32)
        if not case["place"]:
            return {"bytes": 2 * B * R * V * size + lists + masks, "flops": 6 * B * R * V}
        # in place: the tokens of the history (about half of them distinct) and the biases read and written, the
        # forbidden ones written
        touched = sum(min(L // 2 + 1, V) for L in lengths) + B * M
        gone = {"none": 0.0, "few": 1.0, "most": 0.04, "mixed": 0.5}[case["mask"]] * B * R * V
        return {"bytes": int((2 * touched * R + gone) * size + lists + masks), "flops": 6 * R * touched}
    Hq, Hkv, D, page = case["Hq"], case["Hkv"], case["D"], case["page"]
    N, four = sum(new), D // 2 + D // 32
    if case["op"] == "append":
        # queries, keys and values read, queries and codes written; then all codes read and their values written
        cached = page * sum(-(-(c + n) // page) for c, n in zip(ctx, new))
        return {"bytes": N * ((2 * Hq + 2 * Hkv) * D * size + 2 * Hkv * four) + cached * 2 * Hkv * (four + 2 * D) + 4 * case["rot"],
                "flops": N * (Hq + Hkv) * D * 8}
    keys, pairs = 0, 0
    for n, c in zip(new, ctx):
        low = max(0, c + 1 - case["window"]) if case["window"] else 0
        keys += c + n - low
        for t in range(n):
            end = c + t + 1 if case["causal"] else c + n
            pairs += end - (max(0, c + t + 1 - case["window"]) if case["window"] else 0)
    return {"bytes": 2 * N * Hq * D * size + 2 * keys * Hkv * four, "flops": 4 * pairs * Hq * D}


# ---------------------------------------------------------------------------------------------------------------------
# The definitions in 64 bits, one sequence (and head) at a time.
# ---------------------------------------------------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"pages": _exact_pages, "append": _exact_append, "attend": _exact_attend, "adjust": _exact_adjust}[case["op"]](s)


def _exact_pages(s):
    page, rows = s["case"]["page"], s["rows"]
    table, free = [r[r >= 0].tolist() for r in s["table"].cpu()], s["free"].tolist()
    width, left = s["table"].shape[1], int(s["count"])
    ctx = [c + a if n >= 0 else 0 for c, a, n in zip(s["ctx"].tolist(), s["advance"].tolist(), s["new"].tolist())]
    new = [max(n, 0) for n in s["new"].tolist()]
    need = [-(-(c + n) // page) for c, n in zip(ctx, new)]
    for b, t in enumerate(table):
        while len(t) > need[b]:
            # pages go back from the first that is too many
            free[left] = t.pop(need[b])
            left += 1
    pages_asked = rows_asked = 0
    top, start, slot, pos = left, [0], [], []
    for b, t in enumerate(table):
        n, ask = new[b], max(0, need[b] - len(t))
        if need[b] > width:
            n = ask = 0
        pages_asked += ask
        rows_asked += n
        if pages_asked > top or rows_asked > rows:
            n = ask = 0
        for _ in range(ask):
            left -= 1
            t.append(free[left])
        start.append(start[-1] + n)
        for p in range(ctx[b], ctx[b] + n):
            slot.append(t[p // page] * page + p % page)
            pos.append(p)
    rest = [-1] * (rows - len(slot))
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    return ((i32(start), i32(ctx), torch.tensor(slot + rest, dtype=torch.int64, device="cuda"), i32(pos + rest)),
            i32([t + [-1] * (width - len(t)) for t in table]), i32([len(t) for t in table]), i32(free), i32([left]))


def _nearest(x):
    """What 4 bits hold of float64 rows [..., D], by search over all sixteen values."""
    y = x.unflatten(-1, (-1, 32))
    top = y.abs().amax(-1, keepdim=True)
    scale = torch.full_like(top, 2.0 ** -120)
    while bool((top > 7 * scale).any()):
        scale = torch.where(top > 7 * scale, 2 * scale, scale)
    grid = torch.tensor((0.0, 1.0, 2.0, 4.0, 0.5, 1.5, 3.0, 6.0), dtype=torch.float64, device=x.device)    # even codes first: ties
    off = torch.stack([((y / scale).abs() - v).abs() for v in grid], -1)
    return (torch.sign(y) * grid[off.argmin(-1)] * scale).flatten(-2)


def _held(cache, page, D):
    """The values of a 4-bit cache [pages, Hkv, page, D] in float64, number by number from their bits."""
    half = page * D // 2
    x = torch.empty(cache.shape[:2] + (page * D,), dtype=torch.float64, device=cache.device)
    for part, shift in ((0, 0), (1, 4)):
        c = (cache[..., :half] >> shift) & 15
        e, m = ((c >> 1) & 3).double(), (c & 1).double()
        v = torch.where(e == 0, 0.5 * m, torch.exp2(e - 1) * (1 + 0.5 * m))
        x[..., part::2] = torch.where(c >= 8, -v, v)
    return (x.unflatten(-1, (-1, 32)) * torch.exp2(torch.round(cache[..., half:].double() - 127))[..., None]).flatten(-2).unflatten(-1, (page, D))


def _exact_append(s):
    case, page, rot, D = s["case"], s["case"]["page"], s["case"]["rot"], s["case"]["D"]
    i = torch.arange(rot // 2, device="cuda")
    one, two = (i, i + rot // 2) if case["pairs"] == "half" else (2 * i, 2 * i + 1)
    kc, vc, out = _held(s["k_cache"], page, D), _held(s["v_cache"], page, D), s["q"].double()
    begin, ctx, table = s["start"].tolist(), s["ctx"].tolist(), s["table"].tolist()
    eps = float(torch.tensor(1e-6))

    def head(x, weight, turn):
        y = x.double()
        if weight is not None:
            y = y / torch.sqrt(torch.mean(y ** 2, dim=-1, keepdim=True) + eps) * weight.double()
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
        kc[where, :, p.long() % page] = _nearest(head(s["k"][rows], s["k_norm"], turn))
        vc[where, :, p.long() % page] = _nearest(s["v"][rows].double())
    return out, (kc, vc)


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
        keys, values = _held(s["k_cache"][ids], page, case["D"]), _held(s["v_cache"][ids], page, case["D"])
        j, i = torch.arange(c + n, device="cuda")[None], c + torch.arange(n, device="cuda")[:, None]
        sees = torch.ones((n, c + n), dtype=torch.bool, device="cuda")
        if case["causal"]:
            sees &= j <= i
        if case["window"]:
            sees &= i - j < case["window"]
        for h in range(case["Hkv"]):
            k = keys[:, h].reshape(-1, case["D"])[:c + n]
            v = values[:, h].reshape(-1, case["D"])[:c + n]
            for head in range(h * G, h * G + G):
                a = (s["q"][begin[b]:begin[b + 1], head].double() @ k.T) / math.sqrt(case["D"])
                a = torch.softmax(torch.where(sees, a, -math.inf), -1)
                out[begin[b]:begin[b + 1], head] = a @ v
    return out


def _exact_adjust(s):
    case, R, V = s["case"], s["case"]["R"], s["case"]["V"]
    if case["B"] * R > 600:
        return None
    out = s["logits"].double()
    pen = [s[k].double().tolist() for k in ("repetition", "frequency", "presence")]
    length, prompt = s["length"].tolist(), s["prompt"].tolist()
    for b in range(case["B"]):
        text = s["history"][b, :length[b]].long()
        for t in range(R):
            before = text if t == 0 else torch.cat((text, s["path"][b, :t].long()))
            known = torch.unique(before)
            x = out[b, t]
            x[known] = torch.where(x[known] > 0, x[known] / pen[0][b], x[known] * pen[0][b])
            said, times = torch.unique(before[prompt[b]:], return_counts=True)
            x[said] -= pen[1][b] * times.double() + pen[2][b]
            if s["bias"] is not None:
                x[s["bias_token"][b].long()] += s["bias"][b].double()
            if s["mask"] is not None:
                v = torch.arange(V, device="cuda")
                x[(s["mask"][b, t].long()[v // 32] >> (v % 32)) % 2 == 0] = -math.inf
    return out
