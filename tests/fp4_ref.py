"""The 4-bit paged cache in plain fp64 on the CPU: codes and scales of given numbers,
the numbers that a cache holds, and the inputs its tests draw.

Exact throughout: a scale is a power of two and a code's value has two bits, so the
only rounding is the choice of the code, which the kernels must make the same way.
"""
import numpy as np
import torch

from target_ref import append_ref

MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def quantise(x):
    """(codes [..., D / 2], scales [..., D / 32]) uint8 of float64 numbers [..., D]."""
    y = np.asarray(x, dtype=np.float64)
    y = y.reshape(y.shape[:-1] + (-1, 32))
    top = np.abs(y).max(-1)                             # NaN where a block has one
    bad = ~np.isfinite(top)
    e = np.full(top.shape, -120)
    for k in range(-119, 121):                          # the smallest power of which the largest is at most 7
        e = np.where(np.where(bad, 0, top) > 7 * 2.0 ** (k - 1), k, e)
    a = np.abs(np.where(bad[..., None], 0, y)) / 2.0 ** e[..., None]
    code = np.zeros(a.shape, dtype=np.uint8)
    for i in range(7):
        border = (MAGNITUDES[i] + MAGNITUDES[i + 1]) / 2
        code += ((a > border) | ((a == border) & (i % 2 == 1))).astype(np.uint8)       # ties: the even code
    code |= (np.signbit(y) << 3).astype(np.uint8)
    code = code.reshape(code.shape[:-2] + (-1,))
    return code[..., 0::2] | (code[..., 1::2] << 4), np.where(bad, 255, e + 127).astype(np.uint8), bad


def held(cache, page, D):
    """The numbers [pages, Hkv, page, D] float64 that a 4-bit cache (uint8 tensor) holds."""
    c = cache.cpu().numpy()
    codes, scales = c[..., :page * D // 2], c[..., page * D // 2:].astype(np.float64)
    n = np.stack((codes & 15, codes >> 4), -1).reshape(c.shape[:2] + (page, D // 32, 32))
    x = np.where(n >= 8, -1.0, 1.0) * MAGNITUDES[n & 7]
    with np.errstate(invalid="ignore"):
        x = x * np.where(scales == 255, np.nan, 2.0 ** (scales - 127)).reshape(c.shape[:2] + (page, D // 32, 1))
    return torch.from_numpy(x.reshape(c.shape[:2] + (page, D)))


def put(cache, page, D, page_id, slot, x):
    """Writes numbers [Hkv, D] into one place of a numpy cache; blocks with an infinity or
    NaN get their scale only (their codes say nothing): a mask of the bytes that count."""
    codes, scales, bad = quantise(x)
    cache[page_id, :, slot * D // 2:(slot + 1) * D // 2] = codes
    first = page * D // 2 + slot * (D // 32)
    cache[page_id, :, first:first + D // 32] = scales
    return np.repeat(~bad, 16, axis=-1)


def fp4_case(seed, dtype, D, Hq, Hkv, page, new, ctx, extra_pages=2, pad_rows=0, garbage=True, spread=1.0):
    """Inputs of one paged batch over a 4-bit cache.  With `garbage`, positions that no
    new token may see hold random bytes, NaN scales among them."""
    g = torch.Generator().manual_seed(seed)
    B, N = len(new), sum(new) + pad_rows
    pages = [max(1, -(-(max(c, 0) + n) // page)) for c, n in zip(ctx, new)]
    num = sum(pages) + extra_pages
    perm = torch.randperm(num, generator=g).to(torch.int32)
    table = torch.full((B, max(pages)), num - 1, dtype=torch.int32)
    at = 0
    used = np.zeros((num, page), dtype=bool)
    for b in range(B):
        table[b, :pages[b]] = perm[at:at + pages[b]]
        at += pages[b]
        n = max(0, ctx[b] + new[b])
        p = np.arange(n)
        used[table[b].numpy()[p // page], p % page] = True
    caches = []
    for _ in range(2):
        x = torch.randn((num, Hkv, page, D), generator=g).numpy() * np.exp(spread * torch.randn((num, Hkv, page, D // 32), generator=g).numpy()).repeat(32, -1)
        codes, scales, _ = quantise(x)
        if garbage:
            noise = torch.randint(0, 256, codes.shape, generator=g).numpy().astype(np.uint8)
            codes = np.where(used[:, None, :, None], codes, noise)
            noise = torch.randint(0, 256, scales.shape, generator=g).numpy().astype(np.uint8)
            scales = np.where(used[:, None, :, None], scales, np.where(noise < 90, 255, noise)).astype(np.uint8)
        caches.append(torch.from_numpy(np.concatenate((codes.reshape(num, Hkv, -1), scales.reshape(num, Hkv, -1)), -1)).cuda())
    start = torch.tensor([0] + list(new)).cumsum(0).to(torch.int32)
    q = torch.randn((N, Hq, D), generator=g).to(dtype)
    return dict(q=q.cuda(), k_cache=caches[0], v_cache=caches[1], table=table.cuda(), ctx=torch.tensor(ctx, dtype=torch.int32).cuda(),
                start=start.cuda(), N=N, page=page)


def appended(c, D, freq, inter):
    """The caches (numpy) after the append of c["k"], c["v"], and masks of the bytes that
    are defined."""
    out = []
    start, ctx, table, page = c["start"].tolist(), c["ctx"].tolist(), c["table"].cpu().numpy(), c["page"]
    for name, x, w in (("k_cache", c["k"], c["k_norm"]), ("v_cache", c["v"], None)):
        cache = c[name].cpu().numpy().copy()
        sure = np.ones(cache.shape, dtype=bool)
        for b in range(len(ctx)):
            for t in range(start[b + 1] - start[b]):
                pos = ctx[b] + t
                if pos < 0 or pos >= table.shape[1] * page:
                    continue
                y = x[start[b] + t].double().cpu().numpy()
                if name == "k_cache":
                    y, _ = append_ref(y, None if w is None else w.double().cpu().numpy(), float(np.float32(1e-6)), freq, pos, inter)
                slot = pos % page
                mask = put(cache, page, D, table[b, pos // page], slot, y)
                sure[table[b, pos // page], :, slot * D // 2:(slot + 1) * D // 2] = mask
        out.append((cache, sure))
    return out
