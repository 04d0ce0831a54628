"""Plain 64-bit forms of the calls for 4-bit caches, beams and their pages, on the CPU."""
import math

import numpy as np
import torch

CODES = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def e4m3(byte):
    """What a scale's byte stands for; the bytes of NaN count as 480."""
    if byte & 127 == 127:
        return 480.0
    e, m = byte >> 3 & 15, byte & 7
    v = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
    return -v if byte & 128 else v


SCALES = np.array([e4m3(b) for b in range(256)])


def nearest(grid, x):
    """Index of the grid value nearest to x, of two as near the even index."""
    away = np.abs(np.asarray(grid) - x)
    best = np.flatnonzero(away == away.min())
    return int(next((i for i in best if i % 2 == 0), best[0]))


def f32(x):
    return float(np.float32(x))


def kv4_group(x, ts):
    """16 floats: (codes, scale byte, values held)."""
    amax = max([abs(v) for v in x if v == v], default=0.0)
    s = min(f32(amax / f32(6 * ts)), 448.0)
    byte = nearest(SCALES[:127], s)
    unit = f32(SCALES[byte] * ts)
    r = f32(1 / unit) if unit > 0 else 0.0
    codes = []
    for v in x:
        t = v * r  # (of two 32-bit values: exact here)
        t = float("nan") if t != t else f32(t)
        sign = 0 if t != t else int(math.copysign(1, t) < 0)
        codes.append((7 if t != t else nearest(CODES, min(abs(t), 6.0))) + 8 * sign)
    return codes, byte, [(-1 if c > 7 else 1) * CODES[c & 7] * unit for c in codes]


def kv4_cache(x, ts=None):
    """x [pages, heads, ps, D] of any values: the bytes of a cache that holds about those."""
    pages, heads, ps, D = x.shape
    ts = torch.ones(heads) if ts is None else ts.float().cpu()
    g = x.float().cpu().view(pages, heads, ps, D // 16, 16)
    s8 = (g.abs().amax(-1) / (6 * ts[:, None, None])).clamp_max(448).to(torch.float8_e4m3fn)
    unit = (s8.float() * ts[:, None, None])[..., None]
    t = torch.where(unit > 0, g / unit, 0.0)
    code = (t.abs()[..., None] - torch.tensor(CODES)).abs().argmin(-1) + 8 * (t < 0)
    code = code.flatten(-2).to(torch.uint8)
    return torch.cat([(code[..., 0::2] | code[..., 1::2] << 4).flatten(2), s8.view(torch.uint8).flatten(2)], 2)


def kv4_values(cache, ps, D, ts=None):
    """The values [pages, ps, heads, D] in 64 bits that a cache's bytes stand for."""
    cache = cache.cpu()
    pages, heads, _ = cache.shape
    codes = cache[:, :, :ps * D // 2].reshape(pages, heads, ps, D // 2).long()
    s8 = torch.from_numpy(SCALES)[cache[:, :, ps * D // 2:].reshape(pages, heads, ps, D // 16).long()]
    grid = torch.tensor(CODES + [-c for c in CODES], dtype=torch.float64)
    x = torch.stack([grid[codes & 15], grid[codes >> 4]], -1).flatten(-2)
    x = x * s8.repeat_interleave(16, -1)
    if ts is not None:
        x = x * ts.double().cpu()[:, None, None]
    return x.transpose(1, 2)


def beam_select(logits, scores, n, finished=None, end=-1, keep=False):
    """Lists of (total, parent row, token, finished) for each group."""
    x, s = logits.detach().cpu().double().numpy(), scores.detach().cpu().double().numpy()
    G, K = s.shape
    V = x.shape[1]
    out = []
    for g in range(G):
        total = np.full((K, V), -np.inf)
        for k in range(K):
            base = s[g, k] if s[g, k] == s[g, k] else -np.inf
            if finished is not None and bool(finished[g, k]):
                total[k, end] = base
                continue
            row = np.where(np.isnan(x[g * K + k]), -np.inf, x[g * K + k])
            top = row.max()
            if not np.isfinite(top):
                continue
            with np.errstate(invalid="ignore"):
                total[k] = base + (row - (top + math.log(math.fsum(np.exp(row - top)))))
        flat = total.reshape(-1)
        order = np.argsort(-flat, kind="stable")[:n]
        found = [(flat[i], g * K + int(i) // V, int(i) % V) for i in order]
        if keep:
            place, rest = [None] * K, []
            for f in found:
                k = f[1] - g * K
                if place[k] is None:
                    place[k] = f
                else:
                    rest.append(f)
            rest = iter(rest)
            found = [f if f is not None else next(rest) for f in place]
        out.append([f + (f[2] == end or (finished is not None and bool(finished[g, f[1] - g * K])),) for f in found])
    return out


def page_fork(parents, lens, table, free, cursor, ps):
    """Lists in, (table rows, lens, copies, free, cursor) out."""
    rows = [list(r[:-(-n // ps)]) for r, n in zip(table, lens)]
    new = [list(rows[p]) if p >= 0 else [] for p in parents]
    owner, alone = {}, []
    for i, p in enumerate(parents):
        if p >= 0 and lens[p] % ps:
            if p in owner:
                alone.append(i)
            owner.setdefault(p, i)
    kept = set()
    for i, r in enumerate(new):
        kept |= set(r[:-1] if i in alone else r)
    back = sorted({x for r in rows for x in r} - kept)
    free = list(free)
    cursor -= len(back)
    free[cursor:cursor + len(back)] = back
    copies = []
    for i in alone:
        copies.append((new[i][-1], free[cursor]))
        new[i][-1] = free[cursor]
        cursor += 1
    return new, [lens[p] if p >= 0 else 0 for p in parents], copies, free, cursor


def page_compact(lens, table, ps):
    """(table rows, copies, live pages)."""
    rows = [list(r[:-(-n // ps)]) for r, n in zip(table, lens)]
    live = sorted({x for r in rows for x in r})
    high = [p for p in live if p >= len(live)]
    gaps = [p for p in range(len(live)) if p not in set(live)]
    to = dict(zip(high, gaps))
    return [[to.get(x, x) for x in r] for r in rows], list(zip(high, gaps)), len(live)
