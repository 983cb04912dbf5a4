"""Float64 oracle of the serving operators: plan, append, paged attention.

Written from the definitions, request by request and row by row, on host
arrays; it shares nothing with the library.
"""

import numpy as np


def plan(ctx, new, table, page, tokens, free, count):
    """What qlora_kv_plan writes, one request after another.  table [B, W] and
    free [P] are not changed; returns a dict of the new arrays."""
    ctx, new = [int(c) for c in ctx], [int(n) for n in new]
    table, pool = np.array(table), [int(x) for x in free[:count]]
    free_out = np.array(free)
    B, width = table.shape
    pages = lambda t: -(-t // page)   # noqa: E731
    for b in range(B):
        if new[b] < 0:
            for i in range(min(pages(max(ctx[b], 0)), width)):
                if 0 <= table[b, i] < len(free_out):     # else: given away, or never a page
                    free_out[len(pool)] = table[b, i]
                    pool.append(int(table[b, i]))
    cu, kv_len = [0], []
    positions, slots = np.full(tokens, -1), np.full(tokens, -1)
    rows, exhausted = 0, False
    for b in range(B):
        n = max(new[b], 0)
        ok = new[b] >= 0 and ctx[b] >= 0 and ctx[b] + n <= width * page and (n == 0 or rows + n <= tokens)
        if ok:
            need = pages(ctx[b] + n) - pages(ctx[b])
            if need and (exhausted or need > len(pool)):
                ok, exhausted = False, True
        if ok:
            for i in range(pages(ctx[b]), pages(ctx[b] + n)):
                table[b, i] = pool.pop()
            for i in range(n):
                x = ctx[b] + i
                positions[rows + i] = x
                if 0 <= table[b, x // page] < len(free_out):     # no slot on an entry that is no page
                    slots[rows + i] = table[b, x // page] * page + x % page
        kv_len.append(ctx[b] + n if ok else 0)
        rows += n
        cu.append(min(rows, tokens))
    return {"block_table": table, "cu_q": np.array(cu), "kv_len": np.array(kv_len), "positions": positions,
            "slots": slots, "free_pages": free_out, "free_count": len(pool)}


def rotate(x, positions, base):
    """x [T, H, D] float64: the pairs (i, i + D/2) turned by position * base^(-2i/D)."""
    D = x.shape[-1]
    out = np.empty_like(x)
    for i in range(D // 2):
        a = positions.astype(np.float64) * float(base) ** (-2.0 * i / D)
        c, s = np.cos(a)[:, None], np.sin(a)[:, None]
        out[..., i] = x[..., i] * c - x[..., i + D // 2] * s
        out[..., i + D // 2] = x[..., i] * s + x[..., i + D // 2] * c
    return out


def attention(q, k, v, first, scale, window=0, sinks=0, present=None):
    """One request: q [n, H, D] at positions first, first + 1, ...; k, v
    [L, Hkv, D]; `present` [L]: positions that exist.  Returns (out, lse,
    sum of p |v|), the last to scale error bounds with."""
    n, H, D = q.shape
    L, Hkv = k.shape[:2]
    out, mag = np.zeros((n, H, D)), np.zeros((n, H, D))
    lse = np.full((n, H), -np.inf)
    at = np.arange(L)
    for i in range(n):
        x = first + i
        seen = at <= x
        if window:
            seen &= (at > x - window) | (at < sinks)
        if present is not None:
            seen &= present
        if not seen.any():
            continue
        for h in range(Hkv):
            g = slice(h * (H // Hkv), (h + 1) * (H // Hkv))
            s = scale * (q[i, g] @ k[seen, h].T)
            top = s.max(1, keepdims=True)
            e = np.exp(s - top)
            z = e.sum(1, keepdims=True)
            out[i, g] = e / z @ v[seen, h]
            mag[i, g] = e / z @ np.abs(v[seen, h])
            lse[i, g] = (top + np.log(z))[:, 0]
    return out, lse, mag
