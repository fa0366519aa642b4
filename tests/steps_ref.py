"""Plain forms of the operators between the steps of a serving loop, one request and
row at a time on the CPU, and the error bound of adjusted rows.

Bound of an adjusted value: each of its at most four steps in fp32 rounds once, off by
at most u = 2^-24 of its result; a division by the repetition penalty, the product
frequency * c and the subtractions move values of at most
    S = |x| max(rep, 1 / rep) + frequency c + presence + |bias|
so the sum of all is off by at most 5 u S (one for the product too); the store rounds
once more: half a step h of the type, relative to the result.
"""
import numpy as np
import torch

from target_ref import HALF, U


def pages_ref(table, held, free, count, ctx, n_new, page, rows, advance=None):
    """What plan_pages returns and leaves behind, from lists; flags of the device word."""
    table, held, free = [list(r) for r in table], list(held), list(free)
    B, width, flags = len(table), len(table[0]), 0
    total, want, n = [], [], []
    for b in range(B):
        end = n_new[b] < 0
        total.append(0 if end else max(0, ctx[b] + (advance[b] if advance else 0)))
        n.append(max(n_new[b], 0))
        want.append(0 if end else -(-(total[b] + n[b]) // page))
        if want[b] > width:
            flags |= 16
            n[b], want[b] = 0, held[b]
        for i in range(want[b], held[b]):
            free[count] = table[b][i]
            table[b][i] = -1
            count += 1
        if want[b] < held[b]:
            held[b] = want[b]
    top, pages, asked = count, 0, 0
    start, slots, positions = [0], [], []
    for b in range(B):
        ask = want[b] - held[b]
        pages += ask
        asked += n[b]
        if pages > top or asked > rows:
            if ask or n[b]:
                flags |= 128
            ask = n[b] = 0
        for i in range(held[b], held[b] + ask):
            count -= 1
            table[b][i] = free[count]
        held[b] += ask
        start.append(start[-1] + n[b])
        for p in range(total[b], total[b] + n[b]):
            slots.append(table[b][p // page] * page + p % page)
            positions.append(p)
    idle = [-1] * (rows - len(slots))
    return dict(start=start, ctx=total, slots=slots + idle, positions=positions + idle, table=table, held=held, free=free,
                count=[count]), flags


def adjust_ref(x, history=None, history_len=None, prompt_len=None, path=None, repetition=None, frequency=None,
               presence=None, bias_token=None, bias=None, mask=None):
    """(rows, bound) in fp64; the bound is 0 where nothing happens to a value."""
    h = HALF[x.dtype]
    y = x.double().cpu().numpy().copy()
    B, R, V = y.shape
    bound = np.zeros_like(y)
    lists = [None if t is None else t.cpu().tolist() for t in (history, history_len, prompt_len, path, repetition, frequency,
                                                                presence, bias_token, bias)]
    history, history_len, prompt_len, path, rep, freq, pres, bias_token, bias = lists
    words = None if mask is None else mask.cpu().numpy().astype(np.int64) & 0xFFFFFFFF
    for b in range(B):
        n = 0 if history is None else min(max(history_len[b], 0), len(history[b]))
        for t in range(R):
            seen, often = set(), {}
            for i in range(n):
                v = history[b][i]
                seen.add(v)
                if i >= (prompt_len[b] if prompt_len else 0):
                    often[v] = often.get(v, 0) + 1
            for v in (path[b][:t] if path else []):
                seen.add(v)
                often[v] = often.get(v, 0) + 1
            add = dict(zip(bias_token[b], bias[b])) if bias_token else {}       # a token given twice: the last
            for v in seen | set(add):
                if not 0 <= v < V:
                    continue
                z = y[b, t, v]
                size = abs(z)
                if v in seen:
                    r = rep[b] if rep else 1.0
                    z = z / r if z > 0 else z * r
                    size *= max(r, 1 / r)
                c = often.get(v, 0)
                if c:
                    z -= (freq[b] if freq else 0.0) * c + (pres[b] if pres else 0.0)
                    size += (abs(freq[b]) if freq else 0.0) * c + (abs(pres[b]) if pres else 0.0)
                if v in add:
                    z += add[v]
                    size += abs(add[v])
                y[b, t, v] = z
                with np.errstate(invalid="ignore"):
                    bound[b, t, v] = np.nan_to_num((5 * U * size + h * abs(z)) * (1 + 2 * h), posinf=0.0)
            if words is not None:
                v = np.arange(V)
                gone = (words[b, t][v >> 5] >> (v & 31)) & 1 == 0
                y[b, t, gone], bound[b, t, gone] = -np.inf, 0.0
    return torch.from_numpy(y), torch.from_numpy(bound)
