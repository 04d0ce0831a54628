"""Plain 64-bit forms of the softmax-attention serving calls, on the CPU."""
import math

import torch


def page_plan(new, cached, table, free, ps, cursor, N):
    """Lists in, lists out: (offsets, kv_lens, positions, slots, table, cursor)."""
    table = [list(r) for r in table]
    offsets, kv, positions, slots = [0], [], [], []
    for b, (n, c) in enumerate(zip(new, cached)):
        for page in range(-(-c // ps), -(-(c + n) // ps)):
            table[b][page] = free[cursor]
            cursor += 1
        for t in range(c, c + n):
            positions.append(t)
            slots.append(table[b][t // ps] * ps + t % ps)
        offsets.append(offsets[-1] + n)
        kv.append(c + n)
    positions += [0] * (N - len(positions))
    slots += [-1] * (N - len(slots))
    return offsets, kv, positions, slots, table, cursor


def norm_rope(x, weight, eps, row, style):
    """x [N, heads, D]; row [N, R] cosines then sines (None: no rotation)."""
    y = x.detach().cpu().double().clone()
    if weight is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * weight.detach().cpu().double()
    if row is None:
        return y
    row = row.detach().cpu().double()
    half = row.shape[1] // 2
    for i in range(half):
        a, b = (i, i + half) if style == 0 else (2 * i, 2 * i + 1)
        c, s = row[:, i:i + 1], row[:, half + i:half + i + 1]
        ya, yb = y[:, :, a].clone(), y[:, :, b].clone()
        y[:, :, a], y[:, :, b] = ya * c - yb * s, yb * c + ya * s
    return y


def attention(q, k, v, scale=None):
    """q [n, H, D] the last n of kv keys, k and v [kv, HKV, D].  Returns the output and
    sum_j p_j |v_j|, the scale of its rounding errors; a row without keys gives 0."""
    q, k, v = (x.detach().cpu().double() for x in (q, k, v))
    n, H, D = q.shape
    kv, HKV = k.shape[:2]
    scale = 1 / math.sqrt(D) if scale is None else scale
    out, mag = torch.zeros(n, H, D, dtype=torch.float64), torch.zeros(n, H, D, dtype=torch.float64)
    for h in range(H):
        g = h // (H // HKV)
        x = scale * (q[:, h] @ k[:, g].T)
        for i in range(n):
            seen = kv - n + i + 1
            if seen <= 0:
                continue
            p = torch.softmax(x[i, :seen], -1)
            out[i, h] = p @ v[:seen, g]
            mag[i, h] = p @ v[:seen, g].abs()
    return out, mag


def cached_rows(cache, table_row, kv):
    """The first kv tokens of a sequence from a paged cache [pages, ps, HKV, D]."""
    ps = cache.shape[1]
    rows = [cache[int(table_row[t // ps]), t % ps] if 0 <= int(table_row[t // ps]) < cache.shape[0]
            else torch.zeros_like(cache[0, 0]) for t in range(kv)]
    return torch.stack(rows) if rows else cache.new_zeros((0, *cache.shape[2:]))
