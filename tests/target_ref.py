"""Plain fp64 forms of the target-side operators (CPU, one sequence and head at
a time), the inputs their tests draw, and the error bounds of the kernels.

Bounds.  u = 2^-24 is half a step of fp32 relative to the value, h half a step
of the stored type (bf16 2^-8, fp32 2^-24).  Attention: a score is a sum of D
products, off by at most (D + 1) u sum|q k| scale, and the exponent's argument
is rounded once more, off by u |argument|; so a weight is off by a factor
1 + d with
    d = 2 (D + 2) u smax + 2 u amax + 4 u,
smax the largest scale sum|q k| of the row, amax the largest argument (both
sides of the ratio may move, hence the 2; the exponential itself is good to a
step).  The sums over n keys add n u.  With bf16, weights are rounded to bf16
for the second product: h more.  Everything is relative to A = sum p |v| / sum p,
and the result is rounded once: h |o|.
"""
import numpy as np
import torch

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def paged_case(seed, dtype, D, Hq, Hkv, page, new, ctx, extra_pages=2, pad_rows=0, device="cuda", garbage=0.0):
    """Inputs of one paged batch.  Positions that no new token may see hold
    `garbage` in a fifth of their values (NaN to see that they are unused)."""
    g = torch.Generator().manual_seed(seed)
    B, N = len(new), sum(new) + pad_rows
    pages = [max(1, -(-(max(c, 0) + n) // page)) for c, n in zip(ctx, new)]
    num = sum(pages) + extra_pages
    perm = torch.randperm(num, generator=g).to(torch.int32)
    table = torch.full((B, max(pages)), num - 1, dtype=torch.int32)
    at = 0
    kc = torch.randn((num, Hkv, page, D), generator=g).to(dtype)
    vc = torch.randn((num, Hkv, page, D), generator=g).to(dtype)
    used = torch.zeros((num, page), dtype=torch.bool)
    for b in range(B):
        table[b, :pages[b]] = perm[at:at + pages[b]]
        at += pages[b]
        for p in range(max(0, ctx[b] + new[b])):
            used[table[b, p // page], p % page] = True
    if garbage != 0.0:
        hole = (~used)[:, None, :, None] & (torch.rand(kc.shape, generator=g) < 0.2)
        kc = torch.where(hole, torch.full_like(kc, garbage), kc)
        vc = torch.where(hole, torch.full_like(vc, garbage), vc)
    q = torch.randn((N, Hq, D), generator=g).to(dtype)
    start = torch.tensor([0] + list(new)).cumsum(0).to(torch.int32)
    return dict(q=q.to(device), k_cache=kc.to(device), v_cache=vc.to(device), table=table.to(device),
                ctx=torch.tensor(ctx, dtype=torch.int32, device=device), start=start.to(device), N=N)


def attention_ref(c, scale, causal=True, window=0):
    """(out, bound) in fp64 on the CPU; rows that no sequence owns are NaN in out."""
    q, kc, vc = c["q"].cpu().double(), c["k_cache"].cpu(), c["v_cache"].cpu()
    dtype, (N, Hq, D) = c["q"].dtype, c["q"].shape
    Hkv, page = kc.shape[1], kc.shape[2]
    h, G = HALF[dtype], Hq // kc.shape[1]
    out, bound = torch.full((N, Hq, D), float("nan"), dtype=torch.float64), torch.zeros((N, Hq, D), dtype=torch.float64)
    start, ctx, table = c["start"].tolist(), c["ctx"].tolist(), c["table"].cpu().long()
    for b in range(len(ctx)):
        n, cb = start[b + 1] - start[b], ctx[b]
        L = max(0, cb + n)
        j = torch.arange(L)
        k = kc[table[b, j // page], :, j % page].double()       # [L, Hkv, D]
        v = vc[table[b, j // page], :, j % page].double()
        if n == 0:
            continue
        rows = slice(start[b], start[b] + n)
        pos = cb + torch.arange(n)[:, None]
        see = (j <= pos) if causal else (j < L).expand(n, L)
        if window:
            see = see & (j > pos - window)
        see = see & (pos >= 0)
        some = see.any(-1)
        if L == 0 or not bool(some.any()):
            out[rows] = 0.0
            continue
        for head in range(Hq):
            kk, vv, x = k[:, head // G], v[:, head // G], q[rows, head]
            kk, vv = torch.nan_to_num(kk), torch.nan_to_num(vv)
            s = torch.where(see, x @ kk.T * scale, -float("inf"))
            top = torch.where(some, s.amax(-1), 0.0)[:, None]
            p = torch.exp(s - top)
            total = p.sum(-1, keepdim=True).clamp(min=1e-300)
            o, A = p @ vv / total, p @ vv.abs() / total
            smax = torch.where(see, x.abs() @ kk.abs().T * scale, 0.0).amax(-1, keepdim=True)
            low = torch.where(see, s, float("inf")).amin(-1, keepdim=True)
            amax = torch.where(some[:, None], top - low, 0.0) + torch.where(see, s.abs(), 0.0).amax(-1, keepdim=True)
            d = 2 * (D + 2) * U * smax + 2 * U * amax + 4 * U + see.sum(-1, keepdim=True) * U
            if dtype == torch.bfloat16:
                d = d + h
            out[rows, head] = o
            bound[rows, head] = (d * A + h * o.abs()) * (1 + 2 * h)
    return out, bound


def append_ref(k, weight, eps, freq, pos, interleaved):
    """One token's heads [H, D] normed and rotated in fp64."""
    x = np.asarray(k, dtype=np.float64)
    if weight is not None:
        x = x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps) * np.asarray(weight, dtype=np.float64)
    y = x.copy()
    if freq is not None:
        half = len(freq)
        a = pos * np.asarray(freq, dtype=np.float64)
        i = np.arange(half)
        one, two = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        y[:, one] = x[:, one] * np.cos(a) - x[:, two] * np.sin(a)
        y[:, two] = x[:, two] * np.cos(a) + x[:, one] * np.sin(a)
    return y, np.abs(x).max(axis=-1, keepdims=True)


def verify_ref(target, path, cand, prob, u, temperature, n_draft=None, kind="logits"):
    """(tokens, count, p, margin) in fp64: margin is the smallest distance of any
    compared pair (acceptances relative to p, the draw to the whole sum), under
    which a kernel may decide otherwise."""
    x = target.double().cpu().numpy()
    B, R, V = x.shape
    P = R - 1
    path = path.cpu().numpy()
    tok, cnt, out = np.full((B, R), -1, np.int32), np.zeros(B, np.int32), np.zeros((B, R))
    margin = np.full(B, np.inf)
    nd = np.full(B, P) if n_draft is None else np.clip(n_draft.cpu().numpy(), 0, P)
    if temperature > 0:
        cand, prob, u = cand.cpu().numpy(), prob.double().cpu().numpy(), u.double().cpu().numpy()
        u = np.where(u >= 0, np.minimum(u, 1 - 2.0 ** -24), 0.0)
    for b in range(B):
        def row(t):
            if kind == "probs":
                w = np.maximum(x[b, t], 0.0)
            else:
                w = np.exp((x[b, t] - x[b, t].max()) / temperature)
            return w / w.sum()
        t, cut = 0, None
        while t < nd[b]:
            d = path[b, t]
            if temperature == 0:
                if d != int(np.argmax(x[b, t])):
                    break
                pd = 1.0
            else:
                p = row(t)
                pd = p[d] if 0 <= d < V else 0.0
                q = sum(prob[b, t, k] for k in range(cand.shape[2]) if cand[b, t, k] == d)
                margin[b] = min(margin[b], abs(u[b, t] * q - pd) / max(pd, 1e-300))
                if not u[b, t] * q < pd:
                    cut = t
                    break
            tok[b, t], out[b, t] = d, pd
            t += 1
        cnt[b] = t + 1
        if temperature == 0:
            tok[b, t], out[b, t] = int(np.argmax(x[b, t])), 1.0
            continue
        p = row(t)
        left = p.copy()
        if cut is not None:
            for k in range(cand.shape[2]):
                if 0 <= cand[b, cut, k] < V:
                    left[cand[b, cut, k]] = max(0.0, left[cand[b, cut, k]] - prob[b, cut, k])
        sums = np.cumsum(left)
        goal = u[b, P] * sums[-1]
        y = int(np.searchsorted(sums, goal, side="right"))
        near = np.abs(sums - goal)[left > 0].min() if (left > 0).any() else np.inf
        margin[b] = min(margin[b], near / max(sums[-1], 1e-300) * 1e5)     # the draw is fp64: 10^5 times as sharp
        tok[b, t], out[b, t] = y, p[min(y, V - 1)]
    return tok, cnt, out, margin
