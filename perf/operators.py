"""Measured cases of the operators for speculative decoding with drafted trees.

A serving loop that verifies a tree of drafted tokens per request runs, per step:

  tables   block tables, slot mapping and positions of the step's new tokens, from the requests' lengths and a
           pool of free blocks (``extend_tables``);
  masks    which drafted nodes each node sees, and its position, from the parents (``tree_masks``);
  attend   attention of the nodes over the paged cache, once per layer (``paged_decode_tree``);
  compact  the accepted path's keys and values moved together in every layer's cache (``compact_tokens``).

``own = False`` computes them with elementary torch operations in 32 bits, ``own = True`` calls the library.
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
        # one chat request, a small tree, a short context: the latency of one call
        dict(name="attend_one_request", op="attend", B=1, T=8, Hq=32, Hkv=8, D=128, bs=16, lo=600, hi=600, kv="bf16", ragged=False),
        # a full decode batch of the Llama-3.1-8B-shaped layer, 32 nodes a request
        dict(name="attend_batch_bf16", op="attend", B=64, T=32, Hq=32, Hkv=8, D=128, bs=16, lo=2048, hi=4096, kv="bf16", ragged=False),
        # the same layer on an E4M3 cache with longer contexts; requests with fewer nodes among them
        dict(name="attend_batch_fp8", op="attend", B=64, T=32, Hq=32, Hkv=8, D=128, bs=32, lo=4096, hi=8192, kv="fp8", ragged=True),
        # an INT8 cache, a smaller tree, odd lengths
        dict(name="attend_batch_int8", op="attend", B=48, T=21, Hq=32, Hkv=8, D=128, bs=16, lo=1001, hi=7993, kv="int8", ragged=True),
        # few long documents on a 64/8-headed layer, wide trees
        dict(name="attend_long", op="attend", B=4, T=64, Hq=64, Hkv=8, D=128, bs=16, lo=30000, hi=32768, kv="bf16", ragged=False),
        # a layer of 64-wide heads without head sharing
        dict(name="attend_d64", op="attend", B=32, T=48, Hq=16, Hkv=16, D=64, bs=16, lo=77, hi=2999, kv="bf16", ragged=True),
        # masks of one request, and of a large batch of wide trees
        dict(name="masks_one_request", op="masks", B=1, T=16, ragged=False),
        dict(name="masks_batch", op="masks", B=512, T=64, ragged=True),
        # a decode step's tables (each request adds its nodes; some end), and a step that admits long prompts
        dict(name="tables_decode", op="tables", B=256, MB=512, bs=16, lo=100, hi=4000, new_lo=8, new_hi=32, done=0.1),
        dict(name="tables_prompts", op="tables", B=48, MB=2048, bs=16, lo=0, hi=8000, new_lo=1, new_hi=24000, done=0.05),
        # accepted paths of a batch over a 32-layer bf16 cache, and over an E4M3 cache shared by groups of layers
        dict(name="compact_bf16", op="compact", S=32, B=64, T=32, A=8, Hkv=8, D=128, bs=16, lo=64, hi=256, kv="bf16"),
        dict(name="compact_fp8", op="compact", S=8, B=128, T=48, A=6, Hkv=8, D=128, bs=32, lo=64, hi=512, kv="fp8"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "attend", "masks", "tables", "compact"])
    if op == "masks":
        return dict(op=op, B=_log(rng, 1, 700), T=_log(rng, 1, 128), ragged=rng.random() < 0.5)
    if op == "tables":
        new_hi = _log(rng, 1, 20000)
        B = max(1, min(_log(rng, 1, 1000), 1_000_000 // new_hi))
        bs, hi = rng.choice([16, 32]), _log(rng, 1, 8000)
        return dict(op=op, B=B, MB=-(-(hi + new_hi) // bs) + rng.randint(0, 40), bs=bs, lo=0, hi=hi, new_lo=min(new_hi, rng.randint(0, 2)),
                    new_hi=new_hi, done=rng.choice([0.0, 0.1, 0.5]))
    kv = rng.choice(["bf16", "bf16", "fp8", "int8"])
    D = 64 if kv == "bf16" and rng.random() < 0.35 else 128
    bs, Hkv = rng.choice([16, 32]), rng.choice([1, 2, 4, 8])
    if op == "compact":
        hi = _log(rng, 40, 500)
        S = _log(rng, 1, 32)
        B = max(1, min(_log(rng, 1, 200), 250_000_000 // (S * (hi + 64) * Hkv * D)))
        T = rng.randint(2, 64)
        return dict(op=op, S=S, B=B, T=T, A=rng.randint(1, min(T, 10)), Hkv=Hkv, D=D, bs=bs, lo=max(1, hi // 3), hi=hi, kv=kv)
    G = rng.choice([1, 2, 3, 4, 8, 16])
    T, hi = _log(rng, 1, 128), _log(rng, 20, 24000)
    room = min(400_000_000 // (Hkv * D * (hi + T)), 700_000_000 // (Hkv * G * T * (hi + T)))  # cache elements, scores
    B = max(1, min(_log(rng, 1, 128), room))
    return dict(op=op, B=B, T=T, Hq=G * Hkv, Hkv=Hkv, D=D, bs=bs, lo=max(1, hi // 3), hi=hi, kv=kv, ragged=rng.random() < 0.5)


# ------------------------------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------------------------------
def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _parents(rng, T):
    """A drafted tree in the order its nodes were added: the root, then each node below one of the last eight."""
    return [-1] + [rng.randint(max(0, t - 8), t - 1) for t in range(1, T)]


def _nodes(rng, c):
    return [rng.randint(max(1, c["T"] // 2), c["T"]) if c.get("ragged") else c["T"] for _ in range(c["B"])]


def _paged(rng, lens, c):
    """Random physical blocks for sequences of these lengths: (tables, pool size)."""
    bs = c["bs"]
    need = [-(-n // bs) for n in lens]
    NB = c["B"] * -(-(c["hi"] + c["T"]) // bs) + 5
    ids = list(range(NB))
    rng.shuffle(ids)
    MB = max(1, max(need))
    tables, at = [], 0
    for k in need:
        tables.append(ids[at:at + k] + [-1] * (MB - k))
        at += k
    return _ints(tables), NB


def _cache(g, S, NB, c):
    """N(0, 1) keys or values in the cache's type, with the page parameters that quantising them takes."""
    x = torch.randn((S, NB, c["Hkv"], c["bs"], c["D"]), generator=g, device=DEV, dtype=torch.bfloat16)
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
    s = {"c": c}
    if c["op"] == "tables":
        return _prepare_tables(s, c, rng)
    B, T = c["B"], c["T"]
    parents = [_parents(rng, T) for _ in range(B)]
    s["parents"] = _ints(parents)
    nodes = _nodes(rng, c)
    s["nodes"] = _ints(nodes)
    if c["op"] == "masks":
        s["ctx"] = _ints([rng.randint(1, 8000) + n for n in nodes])
        if own:
            import paged_kv_cache_274_gb300 as pkv
            s["call"] = pkv.PreparedCall(pkv.tree_masks, s["parents"], s["ctx"], s["nodes"])
        return s
    lens = [rng.randint(c["lo"], c["hi"]) + n for n in nodes]
    s["ctx"] = _ints(lens)
    s["bt"], NB = _paged(rng, lens, c)
    S = c.get("S", 1)
    s["k"], s["ks"] = _cache(g, S, NB, c)
    s["v"], s["vs"] = _cache(g, S, NB, c)
    if c["op"] == "compact":
        paths = [_path(rng, p[:n], c["A"]) for p, n in zip(parents, nodes)]
        s["idx"] = _ints([p + [0] * (c["A"] - len(p)) for p in paths])
        s["count"] = _ints([len(p) for p in paths])
        if own:
            import paged_kv_cache_274_gb300 as pkv
            s["call"] = pkv.PreparedCall(pkv.compact_tokens, s["idx"], s["count"], s["ctx"], s["bt"], s["k"], s["v"], T, node_counts=s["nodes"],
                                         k_scale=s["ks"], v_scale=s["vs"])
        return s
    s["q"] = torch.randn((B, T, c["Hq"], c["D"]), generator=g, device=DEV, dtype=torch.bfloat16)
    s["mask"] = _masks(s["parents"], s["nodes"], s["ctx"])[0]
    if own:
        import paged_kv_cache_274_gb300 as pkv
        s["call"] = pkv.PreparedDecode(s["q"], s["k"], s["v"], s["bt"], s["ctx"], k_scale=s["ks"], v_scale=s["vs"], tree_mask=s["mask"],
                                       node_counts=s["nodes"])
    return s


def _path(rng, parents, most):
    """An accepted path, from the root down.  Paths whose moves would write over a row that a second pass reads again
    are left out, so that a pass can be repeated on its own results."""
    for _ in range(16):
        t, path = rng.randrange(len(parents)), []
        while t >= 0:
            path.append(t)
            t = parents[t]
        path = path[::-1][:most]
        if all(t == i or t >= len(path) for i, t in enumerate(path)):
            return path
    return [0]


def _prepare_tables(s, c, rng):
    B, MB, bs = c["B"], c["MB"], c["bs"]
    seq, new = [], []
    left = N = 8 + int(1.05 * (1 - c["done"]) * B * (c["new_lo"] + c["new_hi"]) / 2)  # rows of the step's token buffers
    for _ in range(B):
        n = rng.randint(c["lo"], min(c["hi"], MB * bs))
        seq.append(n)
        new.append(-1 if rng.random() < c["done"] else min(rng.randint(c["new_lo"], c["new_hi"]), MB * bs - n, left))
        left -= max(new[-1], 0)
    held = [-(-n // bs) for n in seq]
    want = sum(max(0, -(-(n + max(a, 0)) // bs) - h) for n, a, h in zip(seq, new, held))
    # the pool has what the step wants and a little more, sometimes a little less: the last requests then wait
    free = min(B * MB - sum(held), max(1, want + rng.randint(-(want // 50), 1 + want // 4)))
    NB = B * MB + 1
    ids = list(range(NB))
    rng.shuffle(ids)
    tables, at = [], 0
    for h in held:
        tables.append(ids[at:at + h] + [-1] * (MB - h))
        at += h
    head = rng.randrange(NB)
    ring = [-1] * NB
    for k, i in enumerate(ids[at:at + free]):
        ring[(head + k) % NB] = i
    s.update(seq=_ints(seq), new=_ints(new), bt=_ints(tables), held=_ints(held), ring=_ints(ring), state=_ints([head, free, 0, 0]))
    s["N"] = N
    if own:
        import paged_kv_cache_274_gb300 as pkv
        s["held2"], s["state2"] = torch.zeros_like(s["held"]), torch.zeros_like(s["state"])
        s["call"] = pkv.PreparedCall(pkv.extend_tables, s["seq"], s["new"], s["bt"], s["held"], s["ring"], s["state"], bs, s["N"],
                                     new_block_counts=s["held2"], new_free_state=s["state2"])
    return s


# ------------------------------------------------------------------------------------------------------------------
# one pass
# ------------------------------------------------------------------------------------------------------------------
def run(s):
    op = s["c"]["op"]
    if op == "attend":
        return s["call"]() if own else _attend(s)
    if op == "masks":
        return s["call"]() if own else _masks(s["parents"], s["nodes"], s["ctx"])
    if op == "compact":
        seq = s["call"]() if own else _compact(s)
        e4m3 = s["c"]["kv"] == "fp8"  # the values that the codes stand for
        return [seq] + [t.view(torch.float8_e4m3fn) if e4m3 else t for t in (s["k"], s["v"])]
    if own:
        ctx, starts, slots, pos = s["call"]()
        return [ctx, starts, slots, pos, s["bt"], s["ring"], s["held2"], s["state2"][:2]]
    return _tables(s)


def _attend(s):
    c = s["c"]
    B, T, Hq, Hkv, D, bs = c["B"], c["T"], c["Hq"], c["Hkv"], c["D"], c["bs"]
    ids = s["bt"].clamp_min(0).long()
    N = ids.shape[1] * bs
    pos = torch.arange(N, device=DEV)
    inside = pos < s["ctx"][:, None]  # [B, N]

    def pages(cache, par):
        x = cache[0][ids]  # [B, MB, Hkv, bs, D]
        if c["kv"] == "fp8":
            x = x.view(torch.float8_e4m3fn).float() * par[0][ids][..., None, None]
        elif c["kv"] == "int8":
            p = par[0][ids]
            x = (x.float() - p[..., 1, None, None]) * p[..., 0, None, None]
        x = x.float().permute(0, 2, 1, 3, 4).reshape(B, Hkv, N, D)
        return torch.where(inside[:, None, :, None], x, 0.0)

    base = (s["ctx"] - s["nodes"])[:, None]
    t = torch.arange(T, device=DEV)
    live = t < s["nodes"][:, None]  # [B, T]
    u = (pos[None] - base).clamp(0, T - 1)  # [B, N] node at a position
    words = s["mask"].gather(2, (u >> 5)[:, None].expand(B, T, N))
    seen = ((words >> (u & 31)[:, None].int()) & 1).bool()
    see = live[:, :, None] & inside[:, None] & ((pos[None] < base)[:, None] | seen)  # [B, T, N]
    q = s["q"].float().view(B, T, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, D)
    x = (q @ pages(s["k"], s["ks"]).transpose(2, 3)) * D ** -0.5
    x = x.view(B, Hkv, Hq // Hkv, T, N)
    see = see[:, None, None]
    x = torch.where(see, x, -math.inf)
    top = x.amax(-1, keepdim=True)
    w = torch.where(see, torch.exp(x - torch.where(top > -math.inf, top, 0.0)), 0.0)
    total = w.sum(-1, keepdim=True)
    o = (w.view(B, Hkv, -1, N) @ pages(s["v"], s["vs"])).view(B, Hkv, Hq // Hkv, T, D)
    o = torch.where(total > 0, o / torch.where(total > 0, total, 1.0), 0.0)
    return o.permute(0, 3, 1, 2, 4).reshape(B, T, Hq, D).to(torch.bfloat16)


def _masks(parents, nodes, ctx):
    """Node t sees itself and what its parent sees: the closure of "is or is below", by squaring."""
    B, T = parents.shape
    t = torch.arange(T, device=DEV)
    live = t < nodes[:, None]
    see = ((t[None, None] == t[None, :, None]) | (t[None, None] == parents[:, :, None])) & live[:, :, None]
    reach = 1
    while reach < T:
        see = (see.float() @ see.float()) > 0
        reach *= 2
    W = -(-T // 32)
    bits = torch.zeros((B, T, W * 32), dtype=torch.int64, device=DEV)
    bits[:, :, :T] = see
    words = (bits.view(B, T, W, 32) << torch.arange(32, device=DEV)).sum(-1).to(torch.int32)
    place = (ctx - nodes)[:, None] + see.sum(-1) - 1
    return words, torch.where(live, place, 0).to(torch.int32)


def _tables(s):
    c = s["c"]
    bs, MB, N = c["bs"], c["MB"], s["N"]
    seq, new, held, ring = s["seq"].long(), s["new"].long(), s["held"].long(), s["ring"]
    head, free = s["state"][0].long(), s["state"][1].long()
    NB = ring.numel()
    done = new == -1
    add = new.clamp_min(0)
    ends = add.cumsum(0)
    need = torch.where(done, 0, ((seq + add + bs - 1) // bs - held).clamp_min(0))
    before = need.cumsum(0) - need
    given = ~done & ((need == 0) | (before + need <= free))
    gone = torch.where(done, held, 0)
    taken = torch.where(given, need, 0).sum()
    # blocks that the requests take, into their rows; blocks of the ended ones, behind the free ones
    j = torch.arange(MB, device=DEV)[None]
    k = j - held[:, None]
    fresh = given[:, None] & (k >= 0) & (k < need[:, None])
    bt = torch.where(fresh, ring[(head + before[:, None] + k.clamp(0, MB)) % NB], s["bt"])
    back = done[:, None] & (j < held[:, None])
    at = torch.where(back, (head + free + (gone.cumsum(0) - gone)[:, None] + j) % NB, NB)
    wide = torch.cat([ring, ring[:1]])
    wide[at] = bt  # the last place takes what is not given back
    ring.copy_(wide[:NB])
    s["bt"].copy_(bt)
    i = torch.arange(N, device=DEV)
    b = torch.searchsorted(ends, i, right=True).clamp_max(c["B"] - 1)
    p = seq[b] + i - (ends - add)[b]
    ok = (i < ends[-1]) & given[b]
    p = torch.where(ok, p, 0)
    slots = torch.where(ok, bt[b, p // bs].long() * bs + p % bs, -1)
    ctx = torch.where(given, seq + add, 0).to(torch.int32)
    starts = torch.cat([ends[:1] * 0, ends]).to(torch.int32)
    counts = torch.where(done, 0, torch.where(given, held + need, held)).to(torch.int32)
    state = torch.stack([(head + taken) % NB, free - taken + gone.sum()]).to(torch.int32)
    return [ctx, starts, slots, p.to(torch.int32), s["bt"], ring, counts, state]


def _compact(s):
    c = s["c"]
    bs, A = c["bs"], c["A"]
    base = (s["ctx"] - s["nodes"]).long()[:, None]
    i = torch.arange(A, device=DEV)[None]
    moved = i < s["count"][:, None]
    src = torch.where(moved, base + s["idx"], 0)  # the others: position 0 onto itself
    dst = torch.where(moved, base + i, 0)
    b = torch.arange(c["B"], device=DEV)[:, None]
    sb, so = s["bt"][b, src // bs].long().flatten(), (src % bs).flatten()
    db, do = s["bt"][b, dst // bs].long().flatten(), (dst % bs).flatten()
    for cache, par in ((s["k"], s["ks"]), (s["v"], s["vs"])):
        row = cache[:, sb, :, so]  # [n, S, Hkv, D]
        if par is not None:
            p, q = par[:, sb].transpose(0, 1), par[:, db].transpose(0, 1)
            if c["kv"] == "fp8":
                x = row.view(torch.float8_e4m3fn).float() * p[..., None] / q[..., None]
                x = x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
                row = torch.where((p == q)[..., None], row, x)
            else:
                x = torch.round((row.float() - p[..., 1:]) * p[..., :1] / q[..., :1]) + q[..., 1:]
                low = torch.where(q[..., 1:] == 0, -127.0, -128.0)
                x = torch.minimum(torch.maximum(x, low), torch.full_like(x, 127.0)).to(torch.int8)
                row = torch.where((p == q).all(-1, keepdim=True), row, x)
        cache[:, db, :, do] = row
    return (base[:, 0] + s["count"]).to(torch.int32)


# ------------------------------------------------------------------------------------------------------------------
# what a pass cannot do without
# ------------------------------------------------------------------------------------------------------------------
def work(case):
    c = case
    B = c["B"]
    if c["op"] == "masks":
        T, W = c["T"], -(-c["T"] // 32)
        return {"bytes": 4 * B * (T + T * W + T + 2), "flops": 0}
    if c["op"] == "tables":
        new = (1 - c["done"]) * B * (c["new_lo"] + c["new_hi"]) / 2
        held = (c["lo"] + c["hi"]) / 2 / c["bs"]
        # per token its slot and position, per block a table entry and a ring entry, per request its lengths and counts
        return {"bytes": 12 * new + 8 * (new / c["bs"] + c["done"] * B * held) + 4 * 7 * B, "flops": 0}
    elem = 2 if c["kv"] == "bf16" else 1
    row = 2 * c["Hkv"] * c["D"] * elem
    if c["op"] == "compact":
        moved = B * min(c["A"], 4)
        return {"bytes": 2 * moved * c["S"] * row + 4 * B * (c["A"] + 4), "flops": 0}
    t = 0.75 * c["T"] if c["ragged"] else c["T"]
    tokens = B * ((c["lo"] + c["hi"]) / 2 + t)
    par = {"bf16": 0, "fp8": 4, "int8": 8}[c["kv"]]
    q = B * c["Hq"] * c["D"]
    return {"bytes": tokens * (row + 2 * c["Hkv"] * par / c["bs"] + 4 / c["bs"]) + 2 * q * (t + c["T"]) + 4 * B * c["T"] * -(-c["T"] // 32),
            "flops": 4 * q * t / B * tokens}


# ------------------------------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ------------------------------------------------------------------------------------------------------------------
def exact(case, seed):
    c = dict(case)
    if c["op"] in ("masks", "tables"):
        return None  # whole numbers only
    s = prepare(case, seed)
    ctx, nodes, table = s["ctx"].tolist(), s["nodes"].tolist(), s["bt"].tolist()
    if c["op"] == "compact":
        return _exact_compact(c, s, ctx, nodes, table)
    B, T, Hq, Hkv, D, bs = c["B"], c["T"], c["Hq"], c["Hkv"], c["D"], c["bs"]
    out = torch.zeros((B, T, Hq, D), dtype=torch.float64, device=DEV)
    mask = s["mask"].tolist()
    for b in range(B):
        n, m = ctx[b], nodes[b]
        ids = torch.tensor(table[b][:-(-n // bs)], device=DEV)
        kv = []
        for cache, par in ((s["k"], s["ks"]), (s["v"], s["vs"])):
            x = cache[0].index_select(0, ids)
            if c["kv"] == "fp8":
                x = x.view(torch.float8_e4m3fn).double() * par[0].index_select(0, ids).double()[:, :, None, None]
            elif c["kv"] == "int8":
                p = par[0].index_select(0, ids).double()
                x = (x.double() - p[:, :, None, None, 1]) * p[:, :, None, None, 0]
            kv.append(x.double().transpose(0, 1).reshape(Hkv, -1, D)[:, :n])
        rows = [[(mask[b][t][x >> 5] >> (x & 31)) & 1 for x in range(m)] for t in range(m)]
        hide = torch.zeros((m, n), dtype=torch.bool, device=DEV)
        hide[:, n - m:] = torch.tensor(rows, device=DEV) == 0
        q = s["q"][b, :m].double().transpose(0, 1).reshape(Hkv, Hq // Hkv, m, D)
        x = torch.einsum("hgtd,hnd->hgtn", q, kv[0]) / math.sqrt(D)
        w = torch.softmax(x.masked_fill(hide, -math.inf), -1)
        out[b, :m] = torch.einsum("hgtn,hnd->hgtd", w, kv[1]).reshape(Hq, m, D).transpose(0, 1)
    return out


def _exact_compact(c, s, ctx, nodes, table):
    bs = c["bs"]
    idx, count = s["idx"].tolist(), s["count"].tolist()
    moves = []
    for b in range(c["B"]):
        for i in range(count[b]):
            p, q = ctx[b] - nodes[b] + idx[b][i], ctx[b] - nodes[b] + i
            if p != q:
                moves.append((table[b][p // bs], p % bs, table[b][q // bs], q % bs))
    if c["kv"] == "int8":
        return [None, None, None]  # the outputs are whole numbers
    out = [None]
    for cache, par in ((s["k"], s["ks"]), (s["v"], s["vs"])):
        codes = cache.view(torch.float8_e4m3fn) if c["kv"] == "fp8" else cache
        new = codes.double()
        if moves:
            sb, so, db, do = (torch.tensor(x, device=DEV) for x in zip(*moves))
            row = new[:, sb, :, so]
            if par is not None:
                ratio = par[:, sb].double() / par[:, db].double()
                row = _nearest_e4m3(row * ratio.transpose(0, 1)[..., None])
            new[:, db, :, do] = row
        out.append(new)
    return out


def _nearest_e4m3(x):
    """The E4M3 value nearest to x (to even on a tie): steps of 2^(e - 3) from 2^-6 on, of 2^-9 below."""
    e = torch.floor(torch.log2(x.abs().clamp_min(2.0 ** -6)))
    step = torch.exp2(e - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)
