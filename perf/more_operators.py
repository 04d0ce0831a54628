"""Measured cases of the operators for beam search and 4-bit caches in a serving loop.

A stack that serves gated-delta and softmax-attention layers over a paged cache needs, to hold that cache in 4 bits and
to search with beams:

  write    gdn_kv4_write            keys and values into a paged cache of 4-bit values with a scale to each 16 channels
  kv4      gdn_attention_paged_kv4  attention of new tokens (one, a few drafts, a slice of a prompt) over that cache
  beam     gdn_beam_select          the best continuations of each group of beams, from logits and running scores
  reorder  gdn_state_reorder        recurrent and convolution states follow the chosen beams, in place
  pages    gdn_page_fork, gdn_page_compact, gdn_page_copy
                                    block tables follow the chosen beams: full pages are shared, a last page that is
                                    still written is copied, pages without an owner return; live pages move to the front

`run` computes a case's operator with elementary torch operations (`own` false) or with the package's calls (`own` true).
"""
import math

import numpy as np
import torch

own = False

BF16, F32 = "bf16", "f32"


def listed():
    g = dict(H=32, HKV=8, D=128, dtype=BF16)  # the heads of perf/operators.py: 32 of 128, four to a key-value head
    return [
        # one decode step of 64 requests: latency
        dict(name="write-decode-64", op="write", N=64, HKV=8, D=128, dtype=BF16, ps=64, scaled=False),
        # the prefill batch, 8 x 4096 tokens, with the rounded values that its own attention reads: bandwidth
        dict(name="write-prefill-32768", op="write", N=32768, HKV=8, D=128, dtype=BF16, ps=64, scaled=True),
        # a decode step of 64 requests with histories of U[1, 8192] tokens
        dict(name="kv4-decode-64", op="kv4", B=64, q=1, kv=8192, uneven=True, ps=64, scaled=True, **g),
        # one request with a 131072-token history
        dict(name="kv4-decode-1x131072", op="kv4", B=1, q=1, kv=131072, uneven=False, ps=64, scaled=False, **g),
        # five drafted tokens for each of 16 requests, wide heads, eight to a key-value head
        dict(name="kv4-drafts-d256", op="kv4", B=16, q=5, kv=4096, uneven=True, ps=64, scaled=False, H=16, HKV=2, D=256,
             dtype=BF16),
        # slices of 512 prompt tokens of four requests, the last of 8192
        dict(name="kv4-slices-4x512", op="kv4", B=4, q=512, kv=8192, uneven=False, ps=64, scaled=False, **g),
        # one request with four beams: latency
        dict(name="beam-1x4", op="beam", G=1, K=4, n=4, V=32768, dtype=BF16, done=0.0, keep=False),
        # 64 requests with eight beams over a large vocabulary, some beams at their end: bandwidth
        dict(name="beam-64x8", op="beam", G=64, K=8, n=8, V=131072, dtype=BF16, done=0.1, keep=True),
        # one request's four beams: the states of one layer (32 heads of 128 x 128)
        dict(name="reorder-1x4", op="reorder", G=1, K=4, layers=1, H=32, D=128, W=8192),
        # 32 requests with eight beams: the states of two layers
        dict(name="reorder-32x8", op="reorder", G=32, K=8, layers=2, H=32, D=128, W=8192),
        # tables and pages of 64 requests with four beams follow a selection: bookkeeping and copies of last pages
        dict(name="fork-64x4", op="pages", what="fork", G=64, K=4, kv=4096, shared=0.9, ps=64, spare=0.2, HKV=8, D=128),
        # a pool with two pages of five free: the live ones move to its front
        dict(name="compact-32x4", op="pages", what="compact", G=32, K=4, kv=4096, shared=0.8, ps=64, spare=0.6, HKV=8,
             D=128),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["write", "kv4", "kv4", "kv4", "beam", "beam", "reorder", "pages"])
    ps = rng.choice([16, 32, 48, 64, 128])
    D = rng.choice([64, 80, 96, 128, 128, 256])
    dtype = F32 if rng.random() < 0.25 else BF16
    if op == "write":
        HKV = rng.choice([1, 2, 4, 8, 16])
        N = _log_int(rng, 1, 32768 * 1024 // max(1024, HKV * D * (2 if dtype == F32 else 1)))
        return dict(op=op, N=N, HKV=HKV, D=D, dtype=dtype, ps=ps, scaled=rng.random() < 0.5)
    if op == "kv4":
        H = rng.choice([8, 16, 32])
        HKV = H // rng.choice([1, 2, 4, 8])
        B = _log_int(rng, 1, 128)
        q = rng.choice([1, 1, rng.randint(2, 8), _log_int(rng, 16, 1024)])
        if dtype == F32:
            q = min(q, 64)
        most = min(64 * 8192 * 4096 // (B * HKV * D * 4), (1 << 29) // (B * H * q), 131072)
        if q > 8:
            most = min(most, 4 * 32 * 512 * 8192 * 128 // (B * H * q * D))
        kv = _log_int(rng, min(16, max(1, most)), max(1, most))
        return dict(op=op, B=B, q=min(q, kv), kv=kv, uneven=rng.random() < 0.7, ps=ps, scaled=rng.random() < 0.5, H=H,
                    HKV=HKV, D=D, dtype=dtype)
    if op == "beam":
        K = rng.choice([1, 2, 4, 5, 8, 16])
        V = _log_int(rng, 1000, 200000)
        G = _log_int(rng, 1, max(1, 64 * 8 * 131072 // (K * V * (2 if dtype == F32 else 1))))
        n = rng.choice([K, K, 2 * K])
        return dict(op=op, G=min(G, 256), K=K, n=n, V=V, dtype=dtype, done=rng.choice([0.0, 0.3]) if n == K else 0.0,
                    keep=n == K and rng.random() < 0.5)
    K = rng.choice([2, 3, 4, 8])
    if op == "reorder":
        H, layers = rng.choice([4, 8, 16, 32]), rng.randint(1, 4)
        d = rng.choice([64, 128])
        G = _log_int(rng, 1, max(1, 32 * 8 * 2 * 32 * 128 * 128 // (K * layers * H * d * d)))
        return dict(op=op, G=min(G, 128), K=K, layers=layers, H=H, D=d, W=rng.choice([768, 1000, 4096, 8192]))
    D, HKV = rng.choice([64, 128]), rng.choice([1, 2, 4, 8])
    kv = _log_int(rng, ps, 8192)
    G = _log_int(rng, 1, max(1, min(128, 64 * 4 * 4096 * 8 * 128 // 4 // (K * kv * HKV * D))))
    return dict(op=op, what=rng.choice(["fork", "fork", "compact"]), G=G, K=K, kv=kv, shared=rng.choice([0.3, 0.8, 0.95]),
                ps=ps, spare=rng.choice([0.2, 0.6, 1.5]), HKV=HKV, D=D)


# ---------------------------------------------------------------- inputs

def _torch_type(case):
    return torch.float32 if case["dtype"] == F32 else torch.bfloat16


def _i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()


def _lens_of(case):
    """The host lengths of a kv4 case, the same for every seed: (new tokens, tokens in all) of each request."""
    rs = np.random.RandomState(case["B"])
    kv = rs.randint(1, case["kv"] + 1, case["B"]) if case["uneven"] else np.full(case["B"], case["kv"])
    return np.minimum(case["q"], kv), kv


def _tables_of(case, seed=0):
    """A pages case on the host: (tokens of each row, block table, pages of the pool, live pages in all).  The beams of a
    group have the pages of their prompt in common and the others of their own."""
    rs = np.random.RandomState(case["G"])
    G, K, ps = case["G"], case["K"], case["ps"]
    lens = rs.randint(max(1, case["kv"] // 8), case["kv"] + 1, G)
    common = (lens * case["shared"]).astype(np.int64) // ps
    used = -(-lens // ps)
    live = int((common + K * (used - common)).sum())
    pool = live + int(live * case["spare"]) + 8
    order = np.random.RandomState((seed + 17) % (1 << 31)).permutation(pool)
    table, at = np.full((G * K, -(-case["kv"] // ps) + 1), -1, np.int64), 0
    for g in range(G):
        c, rest = common[g], used[g] - common[g]
        table[g * K:(g + 1) * K, :c] = order[at:at + c]
        at += c
        for k in range(K):
            table[g * K + k, c:used[g]] = order[at:at + rest]
            at += rest
    return np.repeat(lens, K), table, pool, order, live


def _choices(rs, G, K):
    """Parents of each new beam of a step: the better beams have more children."""
    p = 0.6 ** np.arange(K)
    return np.stack([g * K + rs.permutation(K)[rs.choice(K, K, p=p / p.sum())] for g in range(G)])


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    rs = np.random.RandomState((seed + 1) % (1 << 31))
    op = case["op"]
    s = dict(case=case)

    def rand(*shape, std=1.0, dtype=None):
        return (torch.randn(*shape, generator=gen, device="cuda") * std).to(dtype or _torch_type(case))

    def scales(heads):
        if not case["scaled"]:
            return None
        return torch.rand(heads, generator=gen, device="cuda") * 0.1 + 0.01

    if op == "write":
        N, HKV, D, ps = (case[n] for n in ("N", "HKV", "D", "ps"))
        pages = -(-N // ps) + 3
        # keys from the norm and rotation, values as columns of the projection's rows, of smaller size
        rows = rand(N, 3 * HKV * D, std=0.3)
        k_cache, v_cache = (torch.zeros(pages, HKV, ps * D * 9 // 16, dtype=torch.uint8, device="cuda") for _ in "kv")
        return dict(s, k=rand(N, HKV, D), v=rows[:, 2 * HKV * D:].view(N, HKV, D), slots=_i32(rs.permutation(pages * ps)[:N]),
                    k_cache=k_cache, v_cache=v_cache, k_scale=scales(HKV), v_scale=scales(HKV))
    if op == "kv4":
        B, H, HKV, D, ps = (case[n] for n in ("B", "H", "HKV", "D", "ps"))
        new, kv = _lens_of(case)
        used = -(-kv // ps)
        M = -(-case["kv"] // ps)
        table = np.zeros((B, M))
        at = np.arange(M)[None, :] < used[:, None]
        pages = int(at.sum()) + 5
        table[at] = rs.permutation(pages)[:at.sum()]
        ks, vs = scales(HKV), scales(HKV)
        s.update(k_cache=_random_cache(gen, pages, HKV, ps, D, ks), v_cache=_random_cache(gen, pages, HKV, ps, D, vs),
                 k_scale=ks, v_scale=vs)
        return dict(s, q=rand(int(new.sum()), H, D, std=2.0), table=_i32(table), kv_lens=_i32(kv), max_q=int(new.max()),
                    offsets=_i32(np.concatenate([[0], np.cumsum(new)])), kv=[int(x) for x in kv], lens=[int(x) for x in new])
    if op == "beam":
        G, K, V = case["G"], case["K"], case["V"]
        done = torch.from_numpy(rs.rand(G, K) < case["done"]).cuda()
        return dict(s, logits=rand(G * K, V, std=3.0), scores=-5 * torch.rand(G, K, generator=gen, device="cuda"),
                    finished=done if case["done"] > 0 else None)
    if op == "reorder":
        G, K, H, D, W = (case[n] for n in ("G", "K", "H", "D", "W"))
        states = []
        for _ in range(case["layers"]):
            states.append(torch.randn(G * K, H, D, D, generator=gen, device="cuda"))
            states.append(rand(G * K, W, 3, dtype=torch.bfloat16))
        # as gdn_beam_select places them with keep_rows: a beam that goes on keeps its row, the rows of those that end
        # take the others
        chosen = _choices(rs, G, K)
        parents = np.arange(G * K)
        for g in range(G):
            here = np.arange(g * K, (g + 1) * K)
            goes_on = np.isin(here, chosen[g])
            extra = [p for i, p in enumerate(chosen[g]) if p in chosen[g][:i]]
            parents[here[~goes_on]] = extra
        return dict(s, states=states, parents=_i32(parents))
    lens, table, pool, order, live = _tables_of(case, seed)
    k_cache, v_cache = (rand(pool, case["ps"], case["HKV"], case["D"], dtype=torch.bfloat16) for _ in "kv")
    # the pages of the tables are handed out, the others follow in the list
    return dict(s, parents=_i32(_choices(rs, case["G"], case["K"]).reshape(-1)), kv_lens=_i32(lens), table=_i32(table),
                free=_i32(order), cursor=_i32([live]), pool=pool, caches=[k_cache, v_cache])


def _random_cache(gen, pages, HKV, ps, D, scale):
    """A cache of normal values, held in 4 bits."""
    cache = torch.empty(pages, HKV, ps * D * 9 // 16, dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 26) // (HKV * ps * D))
    for i in range(0, pages, step):
        x = torch.randn(min(step, pages - i), HKV, ps, D, generator=gen, device="cuda")
        codes, s8 = _quantise(x, None if scale is None else scale[:, None, None])
        cache[i:i + step] = torch.cat([codes.flatten(2), s8.view(torch.uint8).flatten(2)], 2)
    return cache


# ---------------------------------------------------------------- the operators

def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import varlen_gated_delta_gb300 as gdn
    case = s["case"]
    op = case["op"]
    if op == "write":
        k, v = gdn.gdn_kv4_write(s["k"], s["v"], s["slots"], s["k_cache"], s["v_cache"], k_scale=s["k_scale"],
                                 v_scale=s["v_scale"], values=True)
        return dict(k=k, v=v, k_cache=s["k_cache"], v_cache=s["v_cache"])
    if op == "kv4":
        return gdn.gdn_attention_paged_kv4(s["q"], s["k_cache"], s["v_cache"], s["table"], s["kv_lens"], s["offsets"],
                                           max_q=s["max_q"], k_scale=s["k_scale"], v_scale=s["v_scale"])
    if op == "beam":
        tokens, parents, scores, finished = gdn.gdn_beam_select(
            s["logits"], s["scores"], n=case["n"], finished=s["finished"], end_token=1, keep_rows=case["keep"])
        return dict(tokens=tokens, parents=parents, scores=scores, **({} if finished is None else {"finished": finished}))
    if op == "reorder":
        gdn.gdn_state_reorder(s["states"], s["parents"])
        return list(s["states"])
    if case["what"] == "fork":
        table, kv_lens, copies, cursor, status = gdn.gdn_page_fork(
            s["parents"], s["kv_lens"], s["table"], s["free"], page_size=case["ps"], num_pages=s["pool"], cursor=s["cursor"])
        gdn.gdn_page_copy(s["caches"], copies)
        return dict(table=table, kv_lens=kv_lens, copies=copies, cursor=cursor, status=status, free=s["free"],
                    caches=s["caches"])
    table, copies, free, cursor, status = gdn.gdn_page_compact(s["kv_lens"], s["table"], page_size=case["ps"],
                                                               num_pages=s["pool"])
    gdn.gdn_page_copy(s["caches"], copies)
    return dict(table=table, copies=copies, cursor=cursor, status=status, free=free, caches=s["caches"])


def _run_plain(s):
    return {"write": _plain_write, "kv4": _plain_kv4, "beam": _plain_beam, "reorder": _plain_reorder,
            "pages": _plain_fork if s["case"].get("what") == "fork" else _plain_compact}[s["case"]["op"]](s)


def _quantise(x, scale):
    """x [..., D] in 32 bits: 4-bit codes, two to a byte, and the 8-bit scales of 16 channels each."""
    g = x.unflatten(-1, (-1, 16))
    scale = 1.0 if scale is None else scale
    s8 = (g.abs().amax(-1) / (6.0 * scale)).clamp_max(448.0).to(torch.float8_e4m3fn)
    unit = s8.float() * scale
    t = g * torch.where(unit > 0, 1.0 / unit, 0.0)[..., None]
    a = t.abs()
    # halfway goes to the even code
    code = ((a > 0.25).byte() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)
            + 8 * torch.signbit(t).byte()).flatten(-2)
    return code[..., 0::2] | code[..., 1::2] << 4, s8


_CODES = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _values(codes, s8, scale):
    """What 4-bit codes and scales stand for, in 32 bits."""
    of = torch.tensor(_CODES + [-c for c in _CODES], device=codes.device)
    v = torch.stack([of[(codes & 15).long()], of[(codes >> 4).long()]], -1).flatten(-2)
    unit = s8.float() * (1.0 if scale is None else scale)
    return (v.unflatten(-1, (-1, 16)) * unit[..., None]).flatten(-2)


def _plain_write(s):
    c = s["case"]
    HKV, D, ps, out = c["HKV"], c["D"], c["ps"], {}
    page, place = s["slots"].long() // ps, s["slots"].long() % ps
    for name in "kv":
        scale = s[name + "_scale"]
        scale = None if scale is None else scale[:, None]
        codes, s8 = _quantise(s[name].float(), scale)
        cache = s[name + "_cache"]
        cache[:, :, :ps * D // 2].unflatten(2, (ps, D // 2))[page, :, place] = codes
        cache[:, :, ps * D // 2:].unflatten(2, (ps, D // 16))[page, :, place] = s8.view(torch.uint8)
        out[name], out[name + "_cache"] = _values(codes, s8, scale).to(s[name].dtype), cache
    return out


def _cached(s, name, page):
    """The tokens of these pages [..., ps, HKV, D] in 32 bits."""
    c = s["case"]
    D, ps = c["D"], c["ps"]
    rows = s[name + "_cache"][page]
    codes = rows[..., :ps * D // 2].unflatten(-1, (ps, D // 2))
    s8 = rows[..., ps * D // 2:].unflatten(-1, (ps, D // 16)).contiguous().view(torch.float8_e4m3fn)
    scale = s[name + "_scale"]
    return _values(codes, s8, None if scale is None else scale[:, None, None]).transpose(-3, -2)


def _plain_kv4(s):
    c, q = s["case"], s["q"]
    H, HKV, D = c["H"], c["HKV"], c["D"]
    out = torch.empty_like(q)
    at = 0
    for b, (n, kv) in enumerate(zip(s["lens"], s["kv"])):  # (lengths differ: one request at a time)
        page = s["table"][b, :-(-kv // c["ps"])].long()
        k, v = (_cached(s, name, page).flatten(0, 1)[:kv] for name in "kv")
        x = q[at:at + n].float().view(n, HKV, H // HKV, D).permute(1, 2, 0, 3).reshape(HKV, -1, D)
        x = torch.matmul(x, k.permute(1, 2, 0)).mul_(1.0 / math.sqrt(D)).view(HKV, -1, n, kv)
        if n > 1:
            place = torch.arange(kv, device="cuda")
            x.masked_fill_(place[None, :] > place[kv - n:, None], -math.inf)
        x = x.sub_(x.amax(-1, keepdim=True)).exp_()
        total = x.sum(-1, keepdim=True)
        x = torch.matmul(x.view(HKV, -1, kv), v.transpose(0, 1)).view(HKV, -1, n, D) / total
        out[at:at + n] = x.permute(2, 0, 1, 3).reshape(n, H, D)
        at += n
    return out


def _plain_beam(s):
    c = s["case"]
    G, K, n, V = c["G"], c["K"], c["n"], c["V"]
    x = s["logits"].float() + 0.0  # (no negative zeros)
    # a row's best n: whole numbers in the order of the logits, of equal ones the lowest token first
    bits = x.view(torch.int32)
    order = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long()
    key = (order << 32) + (V - 1 - torch.arange(V, device="cuda"))
    token = V - 1 - (torch.topk(key, min(n, V), -1).values & 0xFFFFFFFF)
    del bits, order, key
    # sums and scores in 64 bits: what is selected hangs on small differences
    top = x.amax(-1, keepdim=True)
    lse = top.double() + (x.double() - top.double()).exp().sum(-1, keepdim=True).log()
    score = s["scores"].double().view(G * K, 1) + (x.gather(1, token).double() - lse)
    if s["finished"] is not None:  # a beam at its end goes on as it is, once
        done = s["finished"].view(G * K, 1)
        first = torch.arange(score.shape[1], device="cuda") == 0
        score = torch.where(done, torch.where(first, s["scores"].double().view(G * K, 1), -math.inf), score)
        token = torch.where(done & first, 1, token)
    score, at = score.view(G, -1).sort(stable=True, dim=-1, descending=True)
    score, at = score[:, :n], at[:, :n]
    beam = at // min(n, V)
    token = token.view(G, -1).gather(1, at)
    if c["keep"]:  # a beam's best child takes its row, the others the rows that are left, in order
        same = beam[:, :, None] == beam[:, None, :]
        best = ~(same.tril(-1)).any(-1)
        taken = torch.zeros(G, K, dtype=torch.bool, device="cuda").scatter(1, torch.where(best, beam, beam[:, :1]), True)
        free = torch.sort((taken.long() * K + torch.arange(K, device="cuda")), -1).values  # rows that are left first
        place = torch.where(best, beam, free.gather(1, ((~best).long().cumsum(-1) - 1).clamp_min(0)))
        back = torch.sort(place, -1).indices
        score, token, beam = (t.gather(1, back) for t in (score, token, beam))
    out = dict(tokens=token.int(), parents=(beam + torch.arange(G, device="cuda")[:, None] * K).int(), scores=score.float())
    if s["finished"] is not None:
        out["finished"] = s["finished"].gather(1, beam) | (token == 1)
    return out


def _plain_reorder(s):
    for t in s["states"]:
        t.copy_(t[s["parents"].long()])
    return list(s["states"])


def _move(caches, src, dst):
    for c in caches:
        c[dst] = c[src]


def _plain_fork(s):
    ps, pool, old, free = s["case"]["ps"], s["pool"], s["table"], s["free"]
    parents = s["parents"].long()
    B, M = old.shape
    col = torch.arange(M, device="cuda")
    row = torch.arange(B, device="cuda")

    def mark(table, used):
        live = torch.zeros(pool + 1, dtype=torch.bool, device="cuda")
        live[torch.where(used, table, pool).long().view(-1)] = True
        return live[:pool]

    before = mark(old, col < ((s["kv_lens"] + ps - 1) // ps)[:, None])
    kv = s["kv_lens"][parents]
    n = (kv + ps - 1) // ps
    table = torch.where(col < n[:, None], old[parents], -1)
    keeper = torch.full((B,), B, device="cuda").scatter_reduce(0, parents, row, "amin")
    copied = (kv % ps != 0) & (keeper[parents] != row)
    after = mark(table, col < (n - copied.int())[:, None])
    back = torch.nonzero(before & ~after).view(-1).int()
    start = s["cursor"] - back.numel()
    free[(start + torch.arange(back.numel(), device="cuda")).long()] = back
    i = torch.nonzero(copied).view(-1)
    dst = free[(start + torch.arange(i.numel(), device="cuda")).long()]
    last = (n[i] - 1).long()
    src = table[i, last]
    table[i, last] = dst
    copies = torch.full((B, 2), -1, dtype=torch.int32, device="cuda")
    copies[:i.numel()] = torch.stack([src, dst], 1)
    _move(s["caches"], src.long(), dst.long())
    return dict(table=table, kv_lens=kv, copies=copies, cursor=start + i.numel(), status=torch.zeros_like(start), free=free,
                caches=s["caches"])


def _plain_compact(s):
    ps, pool, old = s["case"]["ps"], s["pool"], s["table"]
    used = torch.arange(old.shape[1], device="cuda") < ((s["kv_lens"] + ps - 1) // ps)[:, None]
    live = torch.zeros(pool + 1, dtype=torch.bool, device="cuda")
    live[torch.where(used, old, pool).long().view(-1)] = True
    live = live[:pool]
    n = int(live.sum())
    src, dst = torch.nonzero(live[n:]).view(-1) + n, torch.nonzero(~live[:n]).view(-1)
    to = torch.arange(pool, dtype=torch.int32, device="cuda")
    to[src] = dst.int()
    table = torch.where(used, to[old.clamp_min(0).long()], -1)
    copies = torch.full((pool // 2, 2), -1, dtype=torch.int32, device="cuda")
    copies[:src.numel()] = torch.stack([src, dst], 1).int()
    _move(s["caches"], src, dst)
    return dict(table=table, copies=copies, cursor=_i32([n]), status=_i32([0]),
                free=torch.arange(pool, dtype=torch.int32, device="cuda"), caches=s["caches"])


# ---------------------------------------------------------------- work, and the definitions in 64 bits

def work(case):
    op = case["op"]
    if op == "write":
        n, esz = float(case["N"] * case["HKV"] * case["D"]), 4 if case["dtype"] == F32 else 2
        return dict(bytes=2 * n * (2 * esz + 9 / 16) + 4.0 * case["N"], flops=2 * 6 * n)
    if op == "kv4":
        H, HKV, D = case["H"], case["HKV"], case["D"]
        new, kv = _lens_of(case)
        pairs = float((new * (kv - new) + new * (new + 1) // 2).sum())
        return dict(bytes=float(2 * new.sum() * H * D * (4 if case["dtype"] == F32 else 2) + 2 * kv.sum() * HKV * D * 9 / 16),
                    flops=4.0 * pairs * H * D)
    if op == "beam":
        values = float(case["G"] * case["K"] * case["V"]) * (1 - case["done"])  # (a beam at its end reads none)
        return dict(bytes=values * (4 if case["dtype"] == F32 else 2), flops=3 * values)
    # what _choices gives on average: beams of a group that end, and beams with more than one child
    p = 0.6 ** np.arange(case["K"])
    p, K = p / p.sum(), case["K"]
    none, one = ((1 - p) ** K).sum(), (K * p * (1 - p) ** (K - 1)).sum()
    ended, several = float(none), float(K - none - one)
    if op == "reorder":  # one child in the place of each beam that ends
        row = case["layers"] * (case["H"] * case["D"] ** 2 * 4.0 + case["W"] * 3 * 2)
        return dict(bytes=case["G"] * (ended + several) * row, flops=0.0)
    lens, table, pool, _, live = _tables_of(case)
    page, tables = 2 * case["ps"] * case["HKV"] * case["D"] * 2.0, 8.0 * float((-(-lens // case["ps"])).sum())
    if case["what"] == "fork":  # a copy of each last page that is not full, for every child but the first
        return dict(bytes=(ended + several) * page * float((lens[::K] % case["ps"] != 0).sum()) + tables, flops=0.0)
    # a live page lies behind the first `live` ones with the chance of the free part of the pool
    return dict(bytes=2 * live * (pool - live) / pool * page + tables, flops=0.0)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "write":
        # (k and v are what the caches' bytes stand for)
        return dict({name: _exact_write(s[name], s[name + "_scale"]) for name in "kv"}, k_cache=None, v_cache=None)
    if op == "kv4":
        return _exact_kv4(s)
    if op == "beam":
        return _exact_beam(s)
    if op == "reorder":
        return [t[s["parents"].long()].double() for t in s["states"]]
    return (_exact_fork if case["what"] == "fork" else _exact_compact)(s)


def _exact_write(x, scale):
    """The definition rounds three times to 32 bits on its way; each of them here from the 64-bit result."""
    x = x.double()
    N, H, D = x.shape
    ts = torch.ones(H, dtype=torch.float64, device="cuda") if scale is None else scale.double()
    f32 = lambda t: t.float().double()  # noqa: E731
    x = x.view(N, H, D // 16, 16)
    s8 = f32(x.abs().amax(-1) / f32(6 * ts)[:, None]).clamp_max(448).float().to(torch.float8_e4m3fn).double()
    unit = f32(s8 * ts[:, None])
    t = f32(x * f32(1 / unit).nan_to_num(posinf=0.0)[..., None])
    grid = torch.tensor(_CODES, dtype=torch.float64, device="cuda")
    away = (t.abs()[..., None] - grid).abs()
    odd = torch.arange(8, device="cuda") % 2 * 1e-9  # of two as near the even one
    near = grid[(away + odd).argmin(-1)]
    return f32(torch.copysign(near, t) * unit[..., None]).view(N, H, D)


def _exact_kv4(s):
    c = s["case"]
    H, HKV, D, ps = c["H"], c["HKV"], c["D"], c["ps"]
    grid = torch.tensor(_CODES + [-v for v in _CODES], dtype=torch.float64, device="cuda")
    out, at = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda"), 0

    def rows(name, b, h, kv):
        block = s[name + "_cache"][s["table"][b, :-(-kv // ps)].long(), h]
        codes = block[:, :ps * D // 2].reshape(-1, D // 2).long()
        x = torch.empty(codes.shape[0], D, dtype=torch.float64, device="cuda")
        x[:, 0::2], x[:, 1::2] = grid[codes % 16], grid[codes // 16]
        s8 = block[:, ps * D // 2:].reshape(-1, D // 16).contiguous().view(torch.float8_e4m3fn).double()
        ts = 1.0 if s[name + "_scale"] is None else s[name + "_scale"][h].double()
        return (x * s8.repeat_interleave(16, 1) * ts)[:kv]

    for b, (n, kv) in enumerate(zip(s["lens"], s["kv"])):
        hidden = torch.ones(n, kv, dtype=torch.bool, device="cuda").triu(kv - n + 1)
        for g in range(HKV):
            k, v = rows("k", b, g, kv), rows("v", b, g, kv)
            for h in range(g * (H // HKV), (g + 1) * (H // HKV)):
                x = (s["q"][at:at + n, h].double() @ k.T) / math.sqrt(D)
                out[at:at + n, h] = torch.softmax(x.masked_fill(hidden, -math.inf), -1) @ v
        at += n
    return out


def _exact_beam(s):
    c = s["case"]
    G, K, n, V = c["G"], c["K"], c["n"], c["V"]
    out = dict(tokens=np.zeros((G, n), np.int32), parents=np.zeros((G, n), np.int32), scores=np.zeros((G, n)))
    done = None if s["finished"] is None else s["finished"].cpu().numpy()
    finished = np.zeros((G, n), bool)
    scores = s["scores"].double().cpu().numpy()
    for g in range(G):
        lp = torch.log_softmax(s["logits"][g * K:(g + 1) * K].double(), -1)
        # more of a row than can be chosen, with room for equal ones
        best, token = torch.topk(lp, min(V, n + 64), -1)
        best, token = best.cpu().numpy(), token.cpu().numpy()
        found = []
        for k in range(K):
            if done is not None and done[g, k]:
                found.append((-scores[g, k], k, 1))
            else:
                found += [(-(scores[g, k] + b), k, int(t)) for b, t in zip(best[k], token[k])]
        found = sorted(found)[:n]
        if c["keep"]:
            place, first = [None] * K, {}
            for f in found:
                first.setdefault(f[1], f)
            for k, f in first.items():
                place[k] = f
            rest = iter([f for f in found if first[f[1]] is not f])
            found = [f if f is not None else next(rest) for f in place]
        for i, (minus, k, t) in enumerate(found):
            out["tokens"][g, i], out["parents"][g, i], out["scores"][g, i] = t, g * K + k, -minus
            finished[g, i] = t == 1 or (done is not None and done[g, k])
    if done is not None:
        out["finished"] = finished
    return out


def _exact_fork(s):
    ps, pool = s["case"]["ps"], s["pool"]
    old, lens, parents, free = (s[n].cpu().numpy().astype(np.int64) for n in ("table", "kv_lens", "parents", "free"))
    at = int(s["cursor"])
    rows = [list(r[:-(-n // ps)]) for r, n in zip(old, lens)]
    new = [list(rows[p]) for p in parents]
    kept, seen, copied = set(), set(), []
    for i, p in enumerate(parents):
        if lens[p] % ps and p in seen:
            copied.append(i)
        seen.add(p)
        kept.update(new[i])
    back = sorted(set(x for r in rows for x in r) - kept)
    at -= len(back)
    free[at:at + len(back)] = back
    copies = np.full((len(parents), 2), -1)
    for j, i in enumerate(copied):
        copies[j] = new[i][-1], free[at]
        new[i][-1] = free[at]
        at += 1
    table = np.full(old.shape, -1)
    for r, t in zip(new, table):
        t[:len(r)] = r
    return dict(table=table.astype(np.int32), kv_lens=lens[parents].astype(np.int32), copies=copies.astype(np.int32),
                cursor=np.array([at], np.int32), status=np.zeros(1, np.int32), free=free.astype(np.int32),
                caches=_exact_caches(s, copies))


def _exact_caches(s, copies):
    out = [c.clone() for c in s["caches"]]
    for a, b in copies[copies[:, 0] >= 0].tolist():
        for c, d in zip(s["caches"], out):
            d[b] = c[a]
    return out


def _exact_compact(s):
    ps, pool = s["case"]["ps"], s["pool"]
    old, lens = (s[n].cpu().numpy().astype(np.int64) for n in ("table", "kv_lens"))
    live = sorted(set(int(x) for r, n in zip(old, lens) for x in r[:-(-n // ps)]))
    n, have = len(live), set(live)
    pairs = list(zip([p for p in live if p >= n], [p for p in range(n) if p not in have]))
    copies = np.full((pool // 2, 2), -1)
    copies[:len(pairs)] = np.array(pairs, np.int64).reshape(-1, 2)
    to = dict(pairs)
    table = np.full(old.shape, -1)
    for t, r, m in zip(table, old, lens):
        t[:-(-m // ps)] = [to.get(int(x), int(x)) for x in r[:-(-m // ps)]]
    return dict(table=table.astype(np.int32), copies=copies.astype(np.int32), cursor=np.array([n], np.int32),
                status=np.zeros(1, np.int32), free=np.arange(pool).astype(np.int32), caches=_exact_caches(s, copies))
