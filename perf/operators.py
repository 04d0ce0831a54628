"""Measured cases of the attention-serving operators.

A stack that interleaves gated-delta layers with softmax-attention layers needs, for the latter, in the order of a
serving step:

  plan    gdn_page_plan         block tables, slots and positions of a step's new tokens, from request lengths
  rope    gdn_qk_norm_rope      per-head RMS norm of q and k, position rotation, keys and values into the paged cache
  varlen  gdn_attention_varlen  causal attention of whole packed prompts with grouped heads
  paged   gdn_attention_paged   attention of new tokens (one, a few drafts, a slice of a prompt) over the paged cache

`run` computes a case's operator with elementary torch operations in 32 bits (`own` false) or with the package's call
(`own` true).
"""
import math

import numpy as np
import torch

own = False

BF16, F32 = "bf16", "f32"


def listed():
    g = dict(H=32, HKV=8, D=128, dtype=BF16)  # 32 value heads of 128 as in the delta layer, four to a key-value head
    return [
        # a decode step's bookkeeping: 64 requests, one token each
        dict(name="plan-decode-64", op="plan", B=64, new=1, cached=8192, ps=64, uneven=False),
        # bookkeeping of a ragged prompt batch (32 x U[1, 8192], about 131072 tokens)
        dict(name="plan-ragged-32", op="plan", B=32, new=8192, cached=0, ps=64, uneven=True),
        # one decode step of 64 requests: latency
        dict(name="rope-decode-64", op="rope", N=64, R=128, style="half", cache=True, ps=64, **g),
        # the prefill batch, 8 x 4096 tokens: bandwidth
        dict(name="rope-prefill-32768", op="rope", N=32768, R=128, style="half", cache=True, ps=64, **g),
        # 32-bit activations, half of each head rotated in neighbouring pairs, odd token count, no cache
        dict(name="rope-f32-4099", op="rope", N=4099, R=64, style="pairs", cache=False, ps=64, H=16, HKV=16, D=128,
             dtype=F32),
        # short prompts that arrive together
        dict(name="varlen-short-32", op="varlen", B=32, L=512, uneven=True, **g),
        # the prefill batch, 8 x 4096 tokens: tensor cores
        dict(name="varlen-prefill-8x4096", op="varlen", B=8, L=4096, uneven=False, **g),
        # ragged prompts, narrow heads, no sharing
        dict(name="varlen-ragged-d64", op="varlen", B=16, L=4096, uneven=True, H=16, HKV=16, D=64, dtype=BF16),
        # 32-bit activations
        dict(name="varlen-f32-4x1000", op="varlen", B=4, L=1000, uneven=False, H=16, HKV=4, D=128, dtype=F32),
        # a decode step of 64 requests with histories of U[1, 8192] tokens
        dict(name="paged-decode-64", op="paged", B=64, q=1, kv=8192, uneven=True, ps=64, **g),
        # one request with a 131072-token history
        dict(name="paged-decode-1x131072", op="paged", B=1, q=1, kv=131072, uneven=False, ps=64, **g),
        # five drafted tokens for each of 16 requests, wide heads, eight to a key-value head
        dict(name="paged-drafts-d256", op="paged", B=16, q=5, kv=4096, uneven=True, ps=64, H=16, HKV=2, D=256,
             dtype=BF16),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _heads(rng):
    D = rng.choice([64, 128, 128, 256])
    H = rng.choice([8, 16, 32])
    return dict(H=H, HKV=H // rng.choice([1, 2, 4, 8]), D=D)


def draw(rng):
    op = rng.choice(["plan", "rope", "varlen", "varlen", "paged", "paged"])
    ps = rng.choice([16, 32, 64, 128])
    if op == "plan":
        B = _log_int(rng, 1, 2048)
        new = rng.choice([1, rng.randint(2, 8), _log_int(rng, 1, max(1, min(8192, 131072 // B)))])
        return dict(op=op, B=B, new=new, cached=rng.choice([0, _log_int(rng, 1, 8192)]), ps=ps,
                    uneven=rng.random() < 0.7)
    h = _heads(rng)
    dtype = F32 if rng.random() < 0.25 else BF16
    if op == "rope":
        width = (h["H"] + 2 * h["HKV"]) * h["D"] * (4 if dtype == F32 else 2)
        N = _log_int(rng, 1, 32768 * 12288 // max(width, 12288))
        return dict(op=op, N=N, R=h["D"] // rng.choice([1, 2, 4]), style=rng.choice(["half", "pairs"]),
                    cache=rng.random() < 0.5, ps=ps, dtype=dtype, **h)
    if op == "varlen":
        B, most = _log_int(rng, 1, 64), 8 * 32 * 4096 * 4096 * 128
        if dtype == F32:
            most //= 64
        L = min(8192, int(math.sqrt(most / (B * h["H"] * max(128, h["D"])))))
        return dict(op=op, B=B, L=_log_int(rng, 16, L), uneven=rng.random() < 0.7, dtype=dtype, **h)
    B = _log_int(rng, 1, 128)
    q = rng.choice([1, 1, rng.randint(2, 8), _log_int(rng, 16, 1024)])
    if dtype == F32:
        q = min(q, 64)
    row = h["HKV"] * h["D"] * 2 * (4 if dtype == F32 else 2)
    most = min(64 * 8192 * 4096 // (B * row), (1 << 31) // (B * h["H"] * q), 131072)
    if q > 8:
        most = min(most, 8 * 32 * 4096 * 4096 // (B * h["H"] * q))
    kv = _log_int(rng, min(16, most), most)
    return dict(op=op, B=B, q=min(q, kv), kv=kv, uneven=rng.random() < 0.7, ps=ps, dtype=dtype, **h)


# ---------------------------------------------------------------- inputs

def _torch_type(case):
    return torch.float32 if case["dtype"] == F32 else torch.bfloat16


def _lengths(rs, B, most, uneven, least=1):
    return rs.randint(least, most + 1, B) if uneven else np.full(B, most)


def _i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()


def _lens_of(case):
    """The host lengths of a case, the same for every seed: (new tokens, tokens already cached) of each request."""
    rs = np.random.RandomState(case["B"])
    if case["op"] == "plan":
        new = _lengths(rs, case["B"], case["new"], case["uneven"])
        return new, rs.randint(0, case["cached"] + 1, case["B"])
    if case["op"] == "varlen":
        return _lengths(rs, case["B"], case["L"], case["uneven"]), np.zeros(case["B"], np.int64)
    kv = _lengths(rs, case["B"], case["kv"], case["uneven"])
    new = np.minimum(case["q"], kv)
    return new, kv - new


def _offsets(lens):
    return np.concatenate([[0], np.cumsum(lens)])


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    rs = np.random.RandomState((seed + 1) % (1 << 31))
    op = case["op"]
    s = dict(case=case)

    def rand(*shape, std=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * std).to(_torch_type(case))

    if op == "plan":
        new, cached = _lens_of(case)
        ps = case["ps"]
        old, tot = -(-cached // ps), -(-(cached + new) // ps)
        M = int(tot.max()) + 3
        pool = rs.permutation(int(tot.sum()) + 64)
        table = np.full((case["B"], M), -1)
        at = np.arange(M)[None, :] < old[:, None]
        table[at] = pool[:at.sum()]
        free = np.concatenate([rs.permutation(len(pool))[:7], pool[at.sum():]])  # the first seven are handed out already
        return dict(s, new=_i32(new), cached=_i32(cached), table=_i32(table), free=_i32(free), cursor=_i32([7]),
                    N=int(new.sum()))
    H, HKV, D = case["H"], case["HKV"], case["D"]
    if op == "rope":
        N, R, ps = case["N"], case["R"], case["ps"]
        P = 8192
        angle = np.arange(P)[:, None] * 10000.0 ** (-np.arange(R // 2) * 2.0 / R)[None, :]
        table = np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)
        pages = N // ps + 3
        return dict(s, qkv=rand(N, (H + 2 * HKV) * D), table=torch.from_numpy(table).cuda(),
                    positions=_i32(rs.randint(0, P, N)), slots=_i32(rs.permutation(pages * ps)[:N]),
                    qw=1 + 0.2 * torch.randn(D, generator=gen, device="cuda"),
                    kw=1 + 0.2 * torch.randn(D, generator=gen, device="cuda"),
                    k_cache=rand(pages, ps, HKV, D), v_cache=rand(pages, ps, HKV, D))
    new, cached = _lens_of(case)
    N = int(new.sum())
    s.update(offsets=_i32(_offsets(new)), lens=[int(x) for x in new], max_q=int(new.max()))
    s["q"] = rand(N, H, D, std=2.0)  # scores of spread 2 with the scale 1 / sqrt(D)
    if op == "varlen":
        # keys from the norm and rotation, values as columns of the projection's rows
        rows = rand(N, (H + 2 * HKV) * D)
        return dict(s, k=rand(N, HKV, D), v=rows[:, (H + HKV) * D:].view(N, HKV, D))
    ps = case["ps"]
    kv = new + cached
    M = -(-case["kv"] // ps)
    used = -(-kv // ps)
    table = np.zeros((case["B"], M))
    at = np.arange(M)[None, :] < used[:, None]
    pages = int(at.sum()) + 5
    table[at] = rs.permutation(pages)[:at.sum()]
    return dict(s, kv_lens=_i32(kv), kv=[int(x) for x in kv], table=_i32(table), k_cache=rand(pages, ps, HKV, D),
                v_cache=rand(pages, ps, HKV, D))


# ---------------------------------------------------------------- the operators

def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import varlen_gated_delta_gb300 as gdn
    case = s["case"]
    op = case["op"]
    if op == "plan":
        offsets, kv_lens, positions, slots, cursor, status = gdn.gdn_page_plan(
            s["new"], s["cached"], s["table"], s["free"], page_size=case["ps"], N=s["N"], cursor=s["cursor"])
        return dict(offsets=offsets, kv_lens=kv_lens, positions=positions, slots=slots, table=s["table"],
                    cursor=cursor, status=status)
    if op == "rope":
        kept = dict(slots=s["slots"], k_cache=s["k_cache"], v_cache=s["v_cache"]) if case["cache"] else {}
        q, k = gdn.gdn_qk_norm_rope(
            s["qkv"], s["table"], s["positions"], H=case["H"], HKV=case["HKV"], D=case["D"], q_weight=s["qw"],
            k_weight=s["kw"], eps=1e-6,
            style=gdn.GDN_ROPE_HALF if case["style"] == "half" else gdn.GDN_ROPE_PAIRS, **kept)
        return dict(q=q, k_cache=s["k_cache"], v_cache=s["v_cache"]) if case["cache"] else dict(q=q, k=k)
    if op == "varlen":
        return gdn.gdn_attention_varlen(s["q"], s["k"], s["v"], s["offsets"])
    return gdn.gdn_attention_paged(s["q"], s["k_cache"], s["v_cache"], s["table"], s["kv_lens"], s["offsets"],
                                   max_q=s["max_q"])


def _run_plain(s):
    return {"plan": _plain_plan, "rope": _plain_rope, "varlen": _plain_varlen, "paged": _plain_paged}[s["case"]["op"]](s)


def _plain_plan(s):
    ps, new, cached, table, free = s["case"]["ps"], s["new"], s["cached"], s["table"], s["free"]
    B, M = table.shape
    ends = torch.cumsum(new, 0, dtype=torch.int32)
    offsets = torch.cat([torch.zeros_like(ends[:1]), ends])
    kv = cached + new
    old, tot = (cached + ps - 1) // ps, (kv + ps - 1) // ps
    need = tot - old
    first = s["cursor"] + torch.cumsum(need, 0, dtype=torch.int32) - need
    col = torch.arange(M, dtype=torch.int32, device="cuda")[None, :]
    fresh = (col >= old[:, None]) & (col < tot[:, None])
    at = (first[:, None] + col - old[:, None]).clamp(0, free.numel() - 1)
    table = torch.where(fresh, free[at], table)
    seq = torch.repeat_interleave(torch.arange(B, device="cuda"), new, output_size=s["N"])
    positions = cached[seq] + torch.arange(s["N"], dtype=torch.int32, device="cuda") - offsets[seq]
    slots = table[seq, positions // ps] * ps + positions % ps
    cursor = s["cursor"] + need.sum(dtype=torch.int32)
    status = torch.where(cursor > free.numel(), 9, 0).to(torch.int32)
    return dict(offsets=offsets, kv_lens=kv, positions=positions, slots=slots, table=table, cursor=cursor,
                status=status)


def _norm_rotate(x, w, cos, sin, style):
    """x [N, heads, D] in 32 bits: RMS norm over D with weight w, then the first R values of each head rotated."""
    x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w
    R = 2 * cos.shape[1]
    a, b = (x[..., :R // 2], x[..., R // 2:R]) if style == "half" else (x[..., 0:R:2], x[..., 1:R:2])
    cos, sin = cos[:, None, :], sin[:, None, :]
    ra, rb = a * cos - b * sin, b * cos + a * sin
    turned = torch.cat([ra, rb], -1) if style == "half" else torch.stack([ra, rb], -1).flatten(-2)
    return torch.cat([turned, x[..., R:]], -1)


def _plain_rope(s):
    c = s["case"]
    H, HKV, D, R, T = c["H"], c["HKV"], c["D"], c["R"], _torch_type(c)
    x = s["qkv"].float().view(-1, H + 2 * HKV, D)
    row = s["table"][s["positions"]]
    cos, sin = row[:, :R // 2], row[:, R // 2:]
    q = _norm_rotate(x[:, :H], s["qw"], cos, sin, c["style"]).to(T)
    k = _norm_rotate(x[:, H:H + HKV], s["kw"], cos, sin, c["style"]).to(T)
    if not c["cache"]:
        return dict(q=q, k=k)
    s["k_cache"].view(-1, HKV, D)[s["slots"]] = k
    s["v_cache"].view(-1, HKV, D)[s["slots"]] = s["qkv"].view(-1, H + 2 * HKV, D)[:, H + HKV:]
    return dict(q=q, k_cache=s["k_cache"], v_cache=s["v_cache"])


def _attend(q, k, v, visible):
    """q [B, Lq, H, D], k and v [B, Lk, HKV, D] in 32 bits, visible [B, Lq, Lk]: softmax attention, heads grouped."""
    B, Lq, H, D = q.shape
    HKV = k.shape[2]
    q = q.view(B, Lq, HKV, H // HKV, D).permute(0, 2, 3, 1, 4).reshape(B, HKV, -1, D)
    x = torch.matmul(q, k.permute(0, 2, 3, 1)).mul_(1.0 / math.sqrt(D)).view(B, HKV, -1, Lq, k.shape[1])
    x.masked_fill_(~visible[:, None, None], -math.inf)
    x = x.sub_(x.amax(-1, keepdim=True).clamp_min(-3e38)).exp_()
    total = x.sum(-1, keepdim=True)
    x = torch.matmul(x.view(B, HKV, -1, k.shape[1]), v.permute(0, 2, 1, 3)).view(B, HKV, -1, Lq, D)
    x = x / total.clamp_min(1e-30)
    return x.permute(0, 3, 1, 2, 4).reshape(B, Lq, H, D)


def _rows(offsets, longest, N):
    """Packed row of each (request, place) of a padded batch, and which places are real."""
    place = torch.arange(longest, device="cuda")[None, :]
    real = place < (offsets[1:] - offsets[:-1])[:, None]
    return (offsets[:-1, None] + place).clamp_max(N - 1), real


def _plain_varlen(s):
    q, k, v = s["q"], s["k"], s["v"]
    rows, real = _rows(s["offsets"], s["max_q"], q.shape[0])
    place = torch.arange(s["max_q"], device="cuda")
    visible = (place[None, :] <= place[:, None])[None] & real[:, None, :]
    return _attend(q.float()[rows], k.float()[rows], v.float()[rows], visible)[real].to(q.dtype)


def _plain_paged(s):
    q, ps, kv = s["q"], s["case"]["ps"], s["kv_lens"]
    rows, real = _rows(s["offsets"], s["max_q"], q.shape[0])
    longest = max(s["kv"])
    place = torch.arange(longest, device="cuda")
    slot = s["table"][:, place // ps].long() * ps + place % ps
    flat = (-1,) + tuple(s["k_cache"].shape[2:])
    k, v = s["k_cache"].view(flat)[slot].float(), s["v_cache"].view(flat)[slot].float()
    new = s["offsets"][1:] - s["offsets"][:-1]
    last = (kv - new)[:, None] + torch.arange(s["max_q"], device="cuda")  # the last key each query sees
    visible = place <= last[:, :, None]
    return _attend(q.float()[rows], k, v, visible)[real].to(q.dtype)


# ---------------------------------------------------------------- work, and the definitions in 64 bits

def work(case):
    op, esz = case["op"], 4 if case.get("dtype") == F32 else 2
    new, cached = _lens_of(case) if op != "rope" else (None, None)
    if op == "plan":
        N, B, ps = int(new.sum()), case["B"], case["ps"]
        fresh = int((-(-(new + cached) // ps) - -(-cached // ps)).sum())
        return dict(bytes=4.0 * (4 * B + 2 * N + 2 * fresh), flops=0.0)
    H, HKV, D = case["H"], case["HKV"], case["D"]
    if op == "rope":
        N, R = case["N"], case["R"]
        moved = (H + 2 * HKV if case["cache"] else H + HKV) * D * esz * 2
        return dict(bytes=float(N * (moved + (8 if case["cache"] else 4)) + min(N, 8192) * R * 4),
                    flops=float(N * (H + HKV) * (4 * D + 3 * R)))
    N, kv = float(new.sum()), float((new + cached).sum())
    pairs = float((new * cached + new * (new + 1) // 2).sum())
    return dict(bytes=(2 * N * H + 2 * kv * HKV) * D * esz, flops=4.0 * pairs * H * D)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "plan":
        return _exact_plan(s)
    if op == "rope":
        return _exact_rope(s)
    H, HKV, D = case["H"], case["HKV"], case["D"]
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    at = 0
    for b, n in enumerate(s["lens"]):
        if op == "varlen":
            kv, k, v = n, s["k"][at:at + n], s["v"][at:at + n]
        else:
            kv = s["kv"][b]
            pages = s["table"][b, :-(-kv // case["ps"])].long()
            k, v = (c[pages].flatten(0, 1)[:kv] for c in (s["k_cache"], s["v_cache"]))
        hidden = torch.ones(n, kv, dtype=torch.bool, device="cuda").triu(kv - n + 1)
        for h in range(H):
            g = h // (H // HKV)
            x = (s["q"][at:at + n, h].double() @ k[:, g].double().T) / math.sqrt(D)
            p = torch.softmax(x.masked_fill(hidden, -math.inf), -1)
            out[at:at + n, h] = p @ v[:, g].double()
        at += n
    return out


def _exact_plan(s):
    ps, new, cached, table, free = s["case"]["ps"], *(s[n].cpu().numpy().astype(np.int64) for n in
                                                      ("new", "cached", "table", "free"))
    at, positions, slots = int(s["cursor"]), [], []
    for b in range(len(new)):
        old, tot = -(-cached[b] // ps), -(-(cached[b] + new[b]) // ps)
        table[b, old:tot] = free[at:at + tot - old]
        at += tot - old
        t = np.arange(cached[b], cached[b] + new[b])
        positions.append(t)
        slots.append(table[b, t // ps] * ps + t % ps)
    i32 = lambda x: np.asarray(x).astype(np.int32)  # noqa: E731
    return dict(offsets=i32(_offsets(new)), kv_lens=i32(cached + new), positions=i32(np.concatenate(positions)),
                slots=i32(np.concatenate(slots)), table=i32(table), cursor=i32([at]), status=i32([0]))


def _exact_rope(s):
    c = s["case"]
    N, H, HKV, D, R = (c[n] for n in ("N", "H", "HKV", "D", "R"))
    x = s["qkv"].double().view(N, H + 2 * HKV, D)
    w = torch.cat([s["qw"].double().expand(H, D), s["kw"].double().expand(HKV, D)])
    y = x[:, :H + HKV]
    y = y / torch.sqrt((y ** 2).sum(-1, keepdim=True) / D + 1e-6) * w
    row = s["table"].double()[s["positions"].long()]
    turn = torch.complex(row[:, :R // 2], row[:, R // 2:])[:, None, :]
    pair = torch.arange(R // 2, device="cuda")
    i, j = (pair, pair + R // 2) if c["style"] == "half" else (2 * pair, 2 * pair + 1)
    z = torch.complex(y[..., i], y[..., j]) * turn
    y = y.clone()
    y[..., i], y[..., j] = z.real, z.imag
    q, k = y[:, :H], y[:, H:]
    if not c["cache"]:
        return dict(q=q, k=k)
    k_cache, v_cache = s["k_cache"].double(), s["v_cache"].double()
    k_cache.view(-1, HKV, D)[s["slots"].long()] = k
    v_cache.view(-1, HKV, D)[s["slots"].long()] = x[:, H + HKV:]
    return dict(q=q, k_cache=k_cache, v_cache=v_cache)
