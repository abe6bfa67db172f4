"""Measured cases of three operators of a serving step over a paged KV cache.

  packed   attention of the new tokens of a batch of requests, as many as each has (a decode step's one token, a
           prompt, a chunk of one), packed one request behind the other (``paged_decode_packed``);
  rope     norms of each head of the queries and keys, the rotation by the tokens' positions, and the keys and
           values written to their cache slots, in one pass (``rope_append``);
  verify   which nodes of a drafted tree the target model's probabilities accept, from given random numbers, and
           the token that follows them (``verify_tree``).

``own = False`` computes them with elementary torch operations, ``own = True`` calls the library.
"""
import math
import random

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------------------------------------
def listed():
    return [
        # one chat request that adds a few tokens to a short context: the latency of one call
        dict(name="packed_one_request", op="packed", B=1, one=0, new_lo=5, new_hi=5, Hq=32, Hkv=8, D=128, bs=16, lo=700, hi=700, kv="bf16"),
        # a long prompt from its first token on
        dict(name="packed_prompt", op="packed", B=1, one=0, new_lo=8192, new_hi=8192, Hq=32, Hkv=8, D=128, bs=16, lo=0, hi=0, kv="bf16"),
        # continuous batching: most requests decode one token, some bring the next chunk of their prompt
        dict(name="packed_mixed", op="packed", B=64, one=56, new_lo=200, new_hi=512, Hq=32, Hkv=8, D=128, bs=16, lo=1000, hi=8000, kv="bf16"),
        # chunks of any length on an E4M3 cache, and few tokens each on an INT8 one
        dict(name="packed_fp8", op="packed", B=16, one=3, new_lo=2, new_hi=700, Hq=32, Hkv=8, D=128, bs=32, lo=100, hi=8000, kv="fp8"),
        dict(name="packed_int8", op="packed", B=24, one=4, new_lo=3, new_hi=40, Hq=32, Hkv=8, D=128, bs=16, lo=77, hi=5001, kv="int8"),
        # a layer of 64-wide heads without head sharing: prompts of odd lengths
        dict(name="packed_d64", op="packed", B=16, one=2, new_lo=33, new_hi=1501, Hq=16, Hkv=16, D=64, bs=16, lo=0, hi=2000, kv="bf16"),
        # the step's tokens of a decode batch, and of a long prompt, with norms of each head
        dict(name="rope_decode", op="rope", N=64, Hq=32, Hkv=8, D=128, R=128, axes=1, pairs="halves", norm=True, bs=16, far=8000, kv="bf16"),
        dict(name="rope_prompt", op="rope", N=8192, Hq=32, Hkv=8, D=128, R=128, axes=1, pairs="halves", norm=True, bs=16, far=130000, kv="bf16"),
        # images and text: three position axes, neighbouring elements in pairs, half of each head turned; E4M3 cache
        dict(name="rope_axes_fp8", op="rope", N=5003, Hq=64, Hkv=8, D=128, R=64, axes=3, pairs="neighbours", norm=False, bs=32, far=4000, kv="fp8"),
        # one request with a small tree
        dict(name="verify_one_request", op="verify", B=1, T=8, V=32000, ragged=False, draft="sampled"),
        # a batch with wide trees over a large vocabulary, nodes drawn from the draft model's probabilities
        dict(name="verify_batch", op="verify", B=64, T=32, V=128256, ragged=False, draft="sampled"),
        # drafts without randomness (the draft's best tokens), an odd vocabulary, requests with fewer nodes among them
        dict(name="verify_best", op="verify", B=48, T=21, V=50257, ragged=True, draft="best"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["packed", "packed", "packed", "packed", "rope", "rope", "verify", "verify"])
    if op == "verify":
        V = _log(rng, 1000, 150000)
        T = _log(rng, 1, 64)
        B = max(1, min(_log(rng, 1, 128), 260_000_000 // (T * V), 8_000_000 // V))
        return dict(op=op, B=B, T=T, V=V, ragged=rng.random() < 0.5, draft=rng.choice(["sampled", "sampled", "best"]))
    kv = rng.choice(["bf16", "bf16", "fp8"])
    D = 64 if kv == "bf16" and rng.random() < 0.35 else 128
    bs, Hkv = rng.choice([16, 32]), rng.choice([1, 2, 4, 8])
    if op == "rope":
        G = rng.choice([1, 2, 3, 4, 8, 16])
        N = min(_log(rng, 1, 20000), max(1, 41_000_000 // ((G + 2) * Hkv * D)))
        axes = rng.choice([1, 1, 2, 3, 4])
        return dict(op=op, N=N, Hq=G * Hkv, Hkv=Hkv, D=D, R=rng.choice([D, D, D // 2, D // 4]), axes=axes, pairs=rng.choice(["halves", "halves", "neighbours"]),
                    norm=rng.random() < 0.6, bs=bs, far=_log(rng, 100, 200000), kv=kv)
    if kv == "fp8" and rng.random() < 0.4:
        kv = "int8"
    G = rng.choice([1, 2, 3, 4, 8, 16])
    new_hi, hi = _log(rng, 1, 6000), _log(rng, 1, 16000)
    new_hi = min(new_hi, max(1, 1_000_000_000 // (Hkv * G * (hi + new_hi))))
    room = min(1_000_000_000 // (Hkv * G * new_hi * (hi + new_hi)), 400_000_000 // (Hkv * D * (hi + new_hi)))
    B = max(1, min(_log(rng, 1, 100), room))
    return dict(op=op, B=B, one=rng.choice([0, B // 2, B - B // 8]), new_lo=rng.randint(1, max(1, new_hi // 4)), new_hi=new_hi, Hq=G * Hkv, Hkv=Hkv, D=D, bs=bs,
                lo=rng.randint(0, hi // 2), hi=hi, kv=kv)


# ------------------------------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------------------------------
def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _cache(g, NB, c):
    """N(0, 1) keys or values in the cache's type, with the page parameters that quantising them takes."""
    x = torch.randn((1, NB, c["Hkv"], c["bs"], c["D"]), generator=g, device=DEV, dtype=torch.bfloat16)
    if c["kv"] == "bf16":
        return x, None
    hi, lo = x.amax(dim=(3, 4)).float(), x.amin(dim=(3, 4)).float()
    if c["kv"] == "fp8":
        s = torch.maximum(hi, -lo) / 448.0
        return (x.float() / s[..., None, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8), s
    s = (hi - lo) / 255.0
    z = torch.round(-128.0 - lo / s).clamp(-128, 127)
    low = torch.where(z == 0, -127.0, -128.0)[..., None, None]
    q = torch.round(x.float() / s[..., None, None]) + z[..., None, None]
    return torch.minimum(torch.maximum(q, low), torch.full_like(q, 127.0)).to(torch.int8), torch.stack([s, z], -1).contiguous()


def prepare(case, seed):
    c = dict(case)
    rng = random.Random("%d %s" % (seed, sorted((k, v) for k, v in c.items() if k != "name")))
    g = torch.Generator(device=DEV).manual_seed(rng.randrange(1 << 60))
    return {"packed": _prepare_packed, "rope": _prepare_rope, "verify": _prepare_verify}[c["op"]](c, rng, g)


def _prepare_packed(c, rng, g):
    B, bs = c["B"], c["bs"]
    # how many rows there are belongs to the case, whose they are to the inputs
    counts = random.Random(str(sorted((k, v) for k, v in c.items() if k != "name")))
    new = [1 if b < c["one"] else counts.randint(c["new_lo"], c["new_hi"]) for b in range(B)]
    rng.shuffle(new)
    lens = [rng.randint(c["lo"], c["hi"]) + n for n in new]
    need = [-(-n // bs) for n in lens]
    NB = sum(need) + 5
    ids = list(range(NB))
    rng.shuffle(ids)
    tables, at = [], 0
    for k in need:
        tables.append(ids[at:at + k] + [-1] * (max(need) - k))
        at += k
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    s = dict(c=c, new=new, lens=lens, starts_host=starts, starts=_ints(starts), ctx=_ints(lens), bt=_ints(tables))
    s["k"], s["ks"] = _cache(g, NB, c)
    s["v"], s["vs"] = _cache(g, NB, c)
    s["q"] = torch.randn((starts[-1], c["Hq"], c["D"]), generator=g, device=DEV, dtype=torch.bfloat16)
    if own:
        import paged_kv_cache_274_gb300 as pkv
        s["call"] = pkv.PreparedDecode(s["q"], s["k"], s["v"], s["bt"], s["ctx"], k_scale=s["ks"], v_scale=s["vs"], query_starts=s["starts"],
                                       max_query_tokens=max(new))
    return s


def _inv_freq(c):
    return [10000.0 ** (-2.0 * i / c["R"]) for i in range(c["R"] // 2)]


def _axes(c):
    """Which axis turns each pair: runs of pairs for the axes in turn."""
    n = c["R"] // 2
    return [i * c["axes"] // n for i in range(n)]


def _prepare_rope(c, rng, g):
    N, Hq, Hkv, D, bs = c["N"], c["Hq"], c["Hkv"], c["D"], c["bs"]
    NB = N // bs + 9
    s = dict(c=c)
    # the rows of the projections, side by side as one product leaves them
    s["qkv"] = torch.randn((N, (Hq + 2 * Hkv) * D), generator=g, device=DEV, dtype=torch.bfloat16)
    rows = s["qkv"].view(N, Hq + 2 * Hkv, D)
    s["q"], s["k"], s["v"] = rows[:, :Hq], rows[:, Hq:Hq + Hkv], rows[:, Hq + Hkv:]
    s["k_cache"], s["ks"] = _cache(g, NB, c)
    s["v_cache"], s["vs"] = _cache(g, NB, c)
    s["pos"] = torch.randint(0, c["far"], (c["axes"], N), generator=g, device=DEV, dtype=torch.int32)
    s["slots"] = torch.randperm(NB * bs, generator=g, device=DEV)[:N].clone()
    s["qw"] = s["kw"] = None
    if c["norm"]:
        s["qw"] = (1 + 0.2 * torch.randn((D,), generator=g, device=DEV)).bfloat16()
        s["kw"] = (1 + 0.2 * torch.randn((D,), generator=g, device=DEV)).bfloat16()
    s["freq"] = torch.tensor(_inv_freq(c), dtype=torch.float64, device=DEV)
    s["axis"] = torch.tensor(_axes(c), device=DEV)
    if own:
        import paged_kv_cache_274_gb300 as pkv
        s["call"] = pkv.PreparedCall(pkv.rope_append, s["q"], s["k"], s["v"], s["pos"], _inv_freq(c), s["slots"], s["k_cache"], s["v_cache"],
                                     k_scale=s["ks"], v_scale=s["vs"], q_weight=s["qw"], k_weight=s["kw"], eps=1e-6, freq_axes=_axes(c),
                                     interleaved=c["pairs"] == "neighbours")
    return s


def _prepare_verify(c, rng, g):
    B, T, V = c["B"], c["T"], c["V"]
    parents = [[-1] + [rng.randint(max(0, t - 8), t - 1) for t in range(1, T)] for _ in range(B)]
    nodes = [rng.randint(max(1, T // 2), T) if c["ragged"] else T for _ in range(B)]
    rank = [[sum(1 for u in range(1, t) if p[u] == p[t]) for t in range(T)] for p in parents]
    # a target of some 20 likely tokens a row, and a draft that is close to it
    logits = torch.randn((B, T, V), generator=g, device=DEV).mul_(3.0)
    s = dict(c=c, parents=_ints(parents), nodes=_ints(nodes))
    s["p"] = torch.softmax(logits, -1)
    logits.add_(torch.randn((B, T, V), generator=g, device=DEV).mul_(0.7))
    sampled = c["draft"] == "sampled"
    s["q"] = torch.softmax(logits, -1) if sampled else None
    if sampled:  # the order of these keys is a draw without replacement
        logits.sub_(torch.empty_like(logits).exponential_(generator=g).clamp_min_(1e-30).log_())
    most = min(V, 1 + max(max(r) for r in rank))
    best = logits.topk(most, -1).indices
    up, place = torch.tensor(parents, device=DEV).clamp_min(0), torch.tensor(rank, device=DEV)
    s["tokens"] = best[torch.arange(B, device=DEV)[:, None], up, place].to(torch.int32)
    s["r"] = torch.rand((B, T), generator=g, device=DEV)
    s["u"] = torch.rand((B,), generator=g, device=DEV)
    if own:
        import paged_kv_cache_274_gb300 as pkv
        s["call"] = pkv.PreparedCall(pkv.verify_tree, s["tokens"], s["parents"], s["p"], s["r"], s["u"], draft_probs=s["q"], node_counts=s["nodes"])
    return s


# ------------------------------------------------------------------------------------------------------------------
# one pass
# ------------------------------------------------------------------------------------------------------------------
def run(s):
    op = s["c"]["op"]
    if op == "rope":
        out = s["call"]() if own else _rope(s)
        e4m3 = s["c"]["kv"] == "fp8"  # the values that the codes stand for
        return [out] + [t.view(torch.float8_e4m3fn) if e4m3 else t for t in (s["k_cache"], s["v_cache"])]
    if own:
        return s["call"]()
    return _packed(s) if op == "packed" else _verify(s)


def _packed(s):
    c = s["c"]
    Hq, Hkv, D, bs = c["Hq"], c["Hkv"], c["D"], c["bs"]
    G = Hq // Hkv
    out = torch.empty_like(s["q"])

    def pages(cache, par, ids):
        x = cache[0][ids]  # [pages, Hkv, bs, D]
        if c["kv"] == "fp8":
            x = x.view(torch.float8_e4m3fn).float() * par[0][ids][..., None, None]
        elif c["kv"] == "int8":
            p = par[0][ids]
            x = (x.float() - p[..., 1, None, None]) * p[..., 0, None, None]
        return x.float().transpose(0, 1).reshape(Hkv, -1, D)

    for b, (m, n) in enumerate(zip(s["new"], s["lens"])):
        ids = s["bt"][b, :-(-n // bs)].long()
        k, v = pages(s["k"], s["ks"], ids)[:, :n], pages(s["v"], s["vs"], ids)[:, :n]
        lo = s["starts_host"][b]
        q = s["q"][lo:lo + m].float().view(m, Hkv, G, D).permute(1, 2, 0, 3).reshape(Hkv, G * m, D)
        row = torch.arange(m, device=DEV).repeat(G)
        hide = torch.arange(n, device=DEV)[None] > (n - m + row)[:, None]
        step = max(1, 500_000_000 // (G * m * n))  # KV heads at a time
        for h in range(0, Hkv, step):
            x = (q[h:h + step] @ k[h:h + step].transpose(1, 2)) * D ** -0.5
            x = x.masked_fill_(hide, -math.inf)
            w = torch.exp(x - x.amax(-1, keepdim=True))
            o = (w @ v[h:h + step]) / w.sum(-1, keepdim=True)
            some = o.shape[0]
            out[lo:lo + m, h * G:(h + some) * G] = o.view(some, G, m, D).permute(2, 0, 1, 3).reshape(m, some * G, D).to(torch.bfloat16)
    return out


def _rope(s):
    c = s["c"]
    N, R, bs = c["N"], c["R"], c["bs"]
    angle = s["pos"].double()[s["axis"]].t() * s["freq"]  # [N, R / 2], in 64 bits: positions are far
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]

    def turn(x, weight):
        x = x.float()
        if weight is not None:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * weight.float()
        y = x.clone()
        if c["pairs"] == "halves":
            a, b = x[..., :R // 2], x[..., R // 2:R]
            y[..., :R // 2], y[..., R // 2:R] = a * cos - b * sin, b * cos + a * sin
        else:
            a, b = x[..., 0:R:2], x[..., 1:R:2]
            y[..., 0:R:2], y[..., 1:R:2] = a * cos - b * sin, b * cos + a * sin
        return y

    blk, off = s["slots"] // bs, s["slots"] % bs
    for cache, par, x in ((s["k_cache"], s["ks"], turn(s["k"], s["kw"])), (s["v_cache"], s["vs"], s["v"].float())):
        if par is not None:
            x = (x / par[0][blk][..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        cache[0, blk, :, off] = x.to(cache.dtype)
    return turn(s["q"], s["qw"]).to(torch.bfloat16)


def _verify(s):
    c = s["c"]
    B, T, V = c["B"], c["T"], c["V"]
    rows = torch.arange(B, device=DEV)
    token, parent = s["tokens"].long(), s["parents"].long()
    zero = torch.zeros((B,), dtype=torch.float64, device=DEV)
    # the node reached, the target's and the draft's weights there that are left, and their sums.  In 64 bits: the
    # sampled token is a border among sums over the vocabulary
    at = torch.zeros((B,), dtype=torch.long, device=DEV)
    P = s["p"][:, 0].double()
    Q = s["q"][:, 0].double() if s["q"] is not None else None
    Z, Y = zero + 1, zero + 1
    idx = torch.full((B, T), -1, dtype=torch.long, device=DEV)
    idx[:, 0] = 0
    count = torch.ones((B,), dtype=torch.long, device=DEV)
    for t in range(1, T):
        x = token[:, t]
        mine = (parent[:, t] == at) & (t < s["nodes"])
        px = P[rows, x]
        qx = Q[rows, x] if Q is not None else zero + 1
        take = mine & (s["r"][:, t].double() * qx * Z < px * Y)
        drop = mine & ~take
        if Q is not None:
            less = (P - (torch.where(Y > 0, Z / Y, zero))[:, None] * Q).clamp_min(0)
        else:
            less = P.clone()
            less[rows, x] = 0
        P = torch.where(take[:, None], s["p"][:, t].double(), torch.where(drop[:, None], less, P))
        Z = torch.where(take, zero + 1, torch.where(drop, P.sum(-1), Z))
        if Q is not None:
            left = Q.clone()
            left[rows, x] = 0
            Q = torch.where(take[:, None], s["q"][:, t].double(), torch.where(drop[:, None], left, Q))
            Y = torch.where(take, zero + 1, torch.where(drop, Q.sum(-1), Y))
        at = torch.where(take, t, at)
        place = count.clamp_max(T - 1)[:, None]
        idx.scatter_(1, place, torch.where(take[:, None], t, idx.gather(1, place)))
        count = count + take
    # nothing is left where the draft has as much everywhere: the target's own weights
    full = s["p"][rows, at].double()
    P = torch.where((P.sum(-1) > 0)[:, None], P, full)
    sums = P.cumsum(-1)
    nxt = (sums <= (s["u"].double() * sums[:, -1])[:, None]).sum(-1)
    last = V - 1 - (P.flip(-1) > 0).to(torch.uint8).argmax(-1)
    return [idx.to(torch.int32), count.to(torch.int32), torch.minimum(nxt, last).to(torch.int32)]


# ------------------------------------------------------------------------------------------------------------------
# what a pass cannot do without
# ------------------------------------------------------------------------------------------------------------------
def work(case):
    c = case
    if c["op"] == "verify":
        # the rows of the last node of each path, where the token is drawn; the nodes
        rows = 2 if c["draft"] == "sampled" else 1
        return {"bytes": 4 * c["B"] * (rows * c["V"] + 5 * c["T"]), "flops": 2 * c["B"] * rows * c["V"]}
    elem = 2 if c["kv"] == "bf16" else 1
    if c["op"] == "rope":
        q, kv = c["N"] * c["Hq"] * c["D"], 2 * c["N"] * c["Hkv"] * c["D"]
        return {"bytes": 4 * q + (2 + elem) * kv + c["N"] * (4 * c["axes"] + 8), "flops": 8 * (q + kv / 2)}
    many, mid = c["B"] - c["one"], (c["new_lo"] + c["new_hi"]) / 2
    start = (c["lo"] + c["hi"]) / 2
    rows = c["one"] + many * mid
    pairs = c["one"] * (start + 1) + many * mid * (start + (mid + 1) / 2)
    tokens = c["B"] * start + rows
    par = {"bf16": 0, "fp8": 4, "int8": 8}[c["kv"]]
    return {"bytes": tokens * (2 * c["Hkv"] * (c["D"] * elem + par / c["bs"]) + 4 / c["bs"]) + 4 * rows * c["Hq"] * c["D"],
            "flops": 4 * c["Hq"] * c["D"] * pairs}


# ------------------------------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ------------------------------------------------------------------------------------------------------------------
def exact(case, seed):
    c = dict(case)
    if c["op"] == "verify":
        return None  # whole numbers only
    s = prepare(case, seed)
    return _exact_rope(c, s) if c["op"] == "rope" else _exact_packed(c, s)


def _values(c, cache, par, ids):
    x = cache[0].index_select(0, ids)
    if c["kv"] == "fp8":
        return x.view(torch.float8_e4m3fn).double() * par[0].index_select(0, ids).double()[:, :, None, None]
    if c["kv"] == "int8":
        p = par[0].index_select(0, ids).double()
        return (x.double() - p[:, :, None, None, 1]) * p[:, :, None, None, 0]
    return x.double()


def _exact_packed(c, s):
    Hq, Hkv, D, bs = c["Hq"], c["Hkv"], c["D"], c["bs"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    table = s["bt"].tolist()
    lo = 0
    for b in range(c["B"]):
        m, n = s["new"][b], s["lens"][b]
        ids = torch.tensor(table[b][:-(-n // bs)], device=DEV)
        k, v = (_values(c, cache, par, ids) for cache, par in ((s["k"], s["ks"]), (s["v"], s["vs"])))
        limit = torch.arange(n - m + 1, n + 1, device=DEV)  # positions that each row sees
        part = max(1, 60_000_000 // n)  # rows at a time
        for h in range(Hq):
            kh, vh = k[:, h // (Hq // Hkv)].reshape(-1, D)[:n], v[:, h // (Hq // Hkv)].reshape(-1, D)[:n]
            for r in range(0, m, part):
                x = s["q"][lo + r:lo + min(m, r + part), h].double() @ kh.t() / math.sqrt(D)
                x.masked_fill_(torch.arange(n, device=DEV) >= limit[r:r + part, None], -math.inf)
                out[lo + r:lo + min(m, r + part), h] = torch.softmax(x, -1) @ vh
        lo += m
    return out


def _exact_rope(c, s):
    N, R, D, bs = c["N"], c["R"], c["D"], c["bs"]
    half = R // 2
    freq = torch.pow(torch.tensor(10000.0, dtype=torch.float64, device=DEV), -torch.arange(half, device=DEV).double() / half)
    which = torch.div(torch.arange(half, device=DEV) * c["axes"], half, rounding_mode="floor")
    turn = torch.polar(torch.ones((N, half), dtype=torch.float64, device=DEV), s["pos"].double().t()[:, which] * freq)[:, None]
    first = torch.arange(half, device=DEV) * (2 if c["pairs"] == "neighbours" else 1)
    second = first + (1 if c["pairs"] == "neighbours" else half)

    def rotate(x, weight):
        x = x.double()
        if weight is not None:
            x = x / (x.pow(2).sum(-1, keepdim=True) / D + 1e-6).sqrt() * weight.double()
        z = torch.complex(x[..., first], x[..., second]) * turn
        return x.index_copy(-1, first, z.real).index_copy(-1, second, z.imag)

    out = [rotate(s["q"], s["qw"])]
    for cache, par, x in ((s["k_cache"], s["ks"], rotate(s["k"], s["kw"])), (s["v_cache"], s["vs"], s["v"].double())):
        new = (cache.view(torch.float8_e4m3fn) if c["kv"] == "fp8" else cache).double()
        blk, off = torch.div(s["slots"], bs, rounding_mode="floor"), s["slots"] % bs
        if par is not None:
            x = _nearest_e4m3(x / par[0].double()[blk][..., None])
        new[0, blk, :, off] = x
        out.append(new)
    return out


def _nearest_e4m3(x):
    """The E4M3 value nearest to x (to even on a tie): steps of 2^(e - 3) from 2^-6 on, of 2^-9 below."""
    e = torch.floor(torch.log2(x.abs().clamp_min(2.0 ** -6)))
    step = torch.exp2(e - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)
