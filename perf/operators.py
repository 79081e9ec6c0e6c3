"""Operators next to the H2O step: their plain forms, and the calls a user makes of them.

``tree``        attention of a tree of drafted tokens over the cache, which stays as it is
                (speculative decoding: all drafted nodes are verified in one pass).
``checkpoint``  a step's inputs (chunk and pre-step cache) kept in 8 bits and brought back: what a
                training forward stores per chunk. Held in 8 bits, so the pass returns the values it
                stands for: one save and one restore.
``backward``    gradients of a step's attention at the values an 8-bit checkpoint stands for.
``carry``       the gradient of the cache after a step handed through the eviction to the cache before
                it and to the chunk (training through a run of steps, last chunk first).

``run`` computes the plain form in elementary torch operations, or, where ``own`` is set, calls the
framework. Head counts, sizes and the key distribution follow the repository's synthetic workloads.
"""
import math

import torch

own = False

GROUP = 32  # channels that share one 8-bit scale

_T = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _case(name, op, dtype, B, Hkv, G, d, C, n, T):
    return dict(name=name, op=op, dtype=dtype, B=B, Hkv=Hkv, G=G, d=d, C=C, n=n, T=T)


def listed():
    return [
        # one new token against a full cache: the smallest serving call, latency counts
        _case("tree-t1-c2048", "tree", "bf16", 1, 8, 4, 128, 2048, 2048, 1),
        # a small fp32 cache, partly filled, a short draft
        _case("tree-fp32-t24-c256", "tree", "fp32", 1, 2, 2, 64, 256, 201, 24),
        # a batch of ordinary draft trees of unequal sizes over partly filled caches
        _case("tree-t61-b4-c4096", "tree", "bf16", 4, 8, 4, 128, 4096, 4001, 61),
        # the largest tree over the longest cache
        _case("tree-t256-c16384", "tree", "bf16", 1, 8, 4, 128, 16384, 16384, 256),
        # a small fp32 step's checkpoint
        _case("checkpoint-fp32-t64-c256", "checkpoint", "fp32", 1, 2, 2, 64, 256, 256, 64),
        # one chunk of the 64k prefill layer
        _case("checkpoint-t1024-c2048", "checkpoint", "bf16", 1, 8, 4, 128, 2048, 2048, 1024),
        # a batch of long chunks, the cache not full yet
        _case("checkpoint-b4-t2048-c4096", "checkpoint", "bf16", 4, 8, 4, 128, 4096, 4095, 2048),
        # a small fp32 step
        _case("backward-fp32-t64-c256", "backward", "fp32", 1, 2, 2, 64, 256, 256, 64),
        # odd sizes, many query heads per KV head, a partly filled cache
        _case("backward-t333-c1000-d64", "backward", "bf16", 2, 2, 8, 64, 1000, 777, 333),
        # one chunk of the 64k prefill layer
        _case("backward-t1024-c2048", "backward", "bf16", 1, 8, 4, 128, 2048, 2048, 1024),
        # a small batch, odd sizes, while the cache still fills
        _case("carry-b2-t77-c300", "carry", "fp32", 2, 3, 1, 64, 300, 251, 77),
        # one chunk of the 64k prefill layer
        _case("carry-t1024-c2048", "carry", "bf16", 1, 8, 4, 128, 2048, 2048, 1024),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["tree", "tree", "checkpoint", "backward", "backward", "carry"])
    # fp32 caches are small ones (checking, small models); bf16 is the working type
    small = rng.random() < 0.2
    G = rng.choice([1, 2, 3, 4, 8])
    Hkv = rng.choice([1, 2, 4] if small else [1, 2, 4, 8])
    B = rng.choice([1, 1, 2] if small else [1, 1, 2, 3, 4])
    d = rng.choice([64, 128])
    C = _log(rng, 16, 512) if small else _log(rng, 64, 16384)
    if op == "tree":
        T = _log(rng, 1, 64) if small else _log(rng, 1, 256)
    else:
        T = _log(rng, 1, 128) if small else _log(rng, 16, 2048)
    n = C if rng.random() < 0.5 else rng.randint(0, C)
    c = dict(op=op, dtype="fp32" if small else "bf16", B=B, Hkv=Hkv, G=G, d=d, C=C, n=n, T=T)
    top = max((w for k in listed() if k["op"] == op for w in [work(k)]), key=lambda w: w["bytes"] + w["flops"])
    while work(c)["bytes"] > top["bytes"] or work(c)["flops"] > max(top["flops"], 1):
        if c["B"] > 1:
            c["B"] -= 1
        elif op != "tree" and c["T"] > 100 and c["T"] >= c["C"] // 2:
            c["T"] = c["T"] * 2 // 3
        elif c["C"] > 64:
            c["C"] = c["C"] * 2 // 3
            c["n"] = min(c["n"], c["C"])
        else:
            c["T"] = max(1, c["T"] * 2 // 3)
    return c


def work(case):
    B, Hkv, G, d, C, n, T = (case[k] for k in ("B", "Hkv", "G", "d", "C", "n", "T"))
    e = 4 if case["dtype"] == "fp32" else 2
    Hq = Hkv * G
    q, kv, cache = B * Hq * T * d, 2 * B * Hkv * T * d, 2 * B * Hkv * n * d
    if case["op"] == "tree":
        # every row sees the cache and itself at least
        return {"bytes": e * (2 * q + kv + cache) + 4 * B * T + 4 * B * Hq * T, "flops": 4 * B * Hq * d * T * (n + 1)}
    if case["op"] == "checkpoint":
        vals = q + kv + cache
        held = vals + 4 * (vals // GROUP)  # written once, read once
        return {"bytes": 2 * e * vals + 2 * held, "flops": 0}
    if case["op"] == "backward":
        held = (q + kv + cache) * (1 + 4 / GROUP)
        pairs = B * Hq * (T * n + T * (T + 1) // 2)
        return {"bytes": held + e * (2 * q + kv + 2 * B * Hkv * C * d), "flops": 10 * pairs * d}
    # carry: per step dK, dV, dk, dv in, the next cache's sums in, this cache's sums and the chunk's out
    sums = 4 * 2 * B * Hkv * C * d
    return {"bytes": 4 * B * Hkv * T + e * (2 * B * Hkv * C * d + kv) + 2 * sums + e * kv, "flops": 0}


# ---- inputs ---------------------------------------------------------------------
def _heads(case, gen, dtype):
    """q, k, v of the chunk and K, V of the cache: per KV head a direction that the queries lean to
    and that one key in fifty follows (heavy hitters); empty slots zero."""
    B, Hkv, G, d, C, n, T = (case[k] for k in ("B", "Hkv", "G", "d", "C", "n", "T"))
    dev = "cuda"

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev, dtype=torch.float32)

    m = normal(B, Hkv, 1, d)
    m = m / m.square().sum(-1, keepdim=True).sqrt() * math.sqrt(d)

    def keys(rows):
        heavy = torch.rand((B, Hkv, rows, 1), generator=gen, device=dev) < 0.02
        return normal(B, Hkv, rows, d) + heavy * m

    q = normal(B, Hkv, G, T, d) + 0.5 * m[:, :, None]
    K = torch.zeros((B, Hkv, C, d), device=dev)
    V = torch.zeros((B, Hkv, C, d), device=dev)
    K[:, :, :n] = keys(n)
    V[:, :, :n] = normal(B, Hkv, n, d)
    return [x.to(dtype) for x in (q.reshape(B, Hkv * G, T, d), keys(T), normal(B, Hkv, T, d), K, V)]


def _tree(case, gen):
    """Parents of B drafted trees: every node under one of the nodes before it, mostly a recent one.
    In a batch the later sequences have fewer nodes; the rest of their rows are absent (-2)."""
    B, T = case["B"], case["T"]
    i = torch.arange(T, device="cuda")
    back = (torch.rand((B, T), generator=gen, device="cuda").square() * (i + 1)).floor().long()
    parent = (i - 1 - back).clamp(min=-1)
    nodes = T - torch.arange(B, device="cuda") * (T // 8)
    return torch.where(i < nodes[:, None], parent, -2).to(torch.int32)


def _record(q, k, v, K, V, n):
    """The 8-bit record of a step, as the framework documents its layout: the codes of q, k, v and of
    the n valid slots of K and V, then their scales in the same order."""
    codes, scales = [], []
    for x in (q, k, v, K[:, :, :n], V[:, :, :n]):
        c, s = _quantise(x)
        codes.append(c.reshape(-1).to(torch.int8).view(torch.uint8))
        scales.append(s.reshape(-1).view(torch.uint8))
    return torch.cat(codes + scales)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    B, Hkv, G, d, C, n, T = (case[k] for k in ("B", "Hkv", "G", "d", "C", "n", "T"))
    dtype = _T[case["dtype"]]
    s = dict(case=dict(case), dtype=dtype)
    if case["op"] == "carry":
        def normal(t, *shape):
            return torch.randn(shape, generator=gen, device="cuda").to(t)
        s["dK"], s["dV"] = normal(dtype, B, Hkv, C, d), normal(dtype, B, Hkv, C, d)
        s["dK"][:, :, n:] = 0
        s["dV"][:, :, n:] = 0
        s["dk"], s["dv"] = normal(dtype, B, Hkv, T, d), normal(dtype, B, Hkv, T, d)
        s["gK"], s["gV"] = normal(torch.float32, B, Hkv, C, d), normal(torch.float32, B, Hkv, C, d)
        # while the cache fills, the first tokens take the empty slots; then a token in three takes
        # the slot of an evicted entry; the others are dropped
        slots = torch.full((B, Hkv, T), -1, dtype=torch.int32, device="cuda")
        fill = min(T, C - n)
        slots[:, :, :fill] = torch.arange(n, n + fill, device="cuda", dtype=torch.int32)
        take = min((T - fill) // 3, n)
        if take:
            order = torch.rand((B, Hkv, n), generator=gen, device="cuda").argsort(-1)[..., :take]
            which = torch.rand((B, Hkv, T - fill), generator=gen, device="cuda").argsort(-1)[..., :take]
            slots.scatter_(2, fill + which.sort(-1).values, order.sort(-1).values.to(torch.int32))
        s["slots"] = slots
    else:
        s["q"], s["k"], s["v"], s["K"], s["V"] = _heads(case, gen, dtype)
        if case["op"] == "tree":
            s["parent"] = _tree(case, gen)
        if case["op"] == "backward":
            s["record"] = _record(s["q"], s["k"], s["v"], s["K"], s["V"], n)
            s["dout"] = torch.randn((B, Hkv * G, T, d), generator=gen, device="cuda").to(dtype)
    if own:
        from h2o_kv_cache_step_b200 import H2OCache, H2OCheckpoint
        s["cache"] = H2OCache(B, Hkv * G, Hkv, d, C, dtype, max_T=T)
        if case["op"] in ("tree", "checkpoint"):
            pos = torch.full((B, Hkv, C), -1, dtype=torch.int32, device="cuda")
            pos[:, :, :n] = torch.arange(n, device="cuda", dtype=torch.int32)
            s["cache"].set_state(s["K"], s["V"], torch.ones((B, Hkv, C), device="cuda"), pos, P=n, n=n)
        if case["op"] == "backward":
            s["record"] = H2OCheckpoint(s["record"], B, Hkv * G, Hkv, d, T, n)
    return s


# ---- plain forms ----------------------------------------------------------------
def _visible(parent):
    """[B, T, T]: whether node j is node i or one of its ancestors; and [B, T]: whether i is there."""
    B, T = parent.shape
    i = torch.arange(T, device=parent.device)
    linked = (parent >= 0) & (parent < i)
    up = linked[..., None] & (parent[..., None] == i)
    seen = (up | (i[:, None] == i)).float()
    for _ in range((T - 1).bit_length()):
        seen = (seen @ seen).clamp(max=1)
    broken = (~linked & (parent != -1)).float()
    return seen > 0, (seen @ broken[..., None])[..., 0] == 0


def _attend(q, k, v, mask):
    """softmax(q k^T / sqrt(d)) v under the mask [B, 1, 1, T, keys], and its log-sum-exp."""
    s = (q @ k.transpose(-1, -2)) / math.sqrt(q.shape[-1])
    s = s.masked_fill(~mask, -math.inf)
    top = s.amax(-1, keepdim=True)
    p = (s - top).exp()
    total = p.sum(-1, keepdim=True)
    return (p @ v) / total, (top + total.log())[..., 0]


def _tree_plain(s, t):
    c = s["case"]
    B, Hkv, G, d, n, T = (c[k] for k in ("B", "Hkv", "G", "d", "n", "T"))
    q = s["q"].to(t).reshape(B, Hkv, G, T, d)
    k = torch.cat([s["K"][:, :, :n], s["k"]], 2).to(t)[:, :, None]
    v = torch.cat([s["V"][:, :, :n], s["v"]], 2).to(t)[:, :, None]
    seen, there = _visible(s["parent"])
    mask = torch.cat([seen.new_ones((B, T, n)), seen], 2)[:, None, None]
    out, lse = _attend(q, k, v, mask)
    there = there[:, None, None]
    out = torch.where(there[..., None], out, 0.0)
    lse = torch.where(there, lse, -math.inf)
    return out.reshape(B, Hkv * G, T, d), lse.reshape(B, Hkv * G, T)


def _quantise(x):
    """Codes in -127..127 and one scale for every 32 channels. The quotient is taken in 64 bits, where
    a code next to a border falls on the side that the real quotient does."""
    g = x.double().unflatten(-1, (-1, GROUP))
    top = g.abs().amax(-1, keepdim=True)
    codes = torch.where(top > 0, (127 * g / top).round(), 0.0)
    return codes.flatten(-2), (top[..., 0] / 127).float()


def _values(codes, scales, dtype):
    return (codes.float().unflatten(-1, (-1, GROUP)) * scales[..., None]).flatten(-2).to(dtype)


def _round_trip_plain(s):
    n, dtype = s["case"]["n"], s["dtype"]
    back = []
    for x in (s["q"], s["k"], s["v"], s["K"][:, :, :n], s["V"][:, :, :n]):
        back.append(_values(*_quantise(x), dtype))
    for i in (3, 4):
        full = torch.zeros_like(s["K"])
        full[:, :, :n] = back[i]
        back[i] = full
    return back


def _read(record, case, dtype):
    """q, k, v, K, V (the valid slots) that a record stands for."""
    B, Hkv, G, d, n, T = (case[k] for k in ("B", "Hkv", "G", "d", "n", "T"))
    shapes = [(B, Hkv * G, T), (B, Hkv, T), (B, Hkv, T), (B, Hkv, n), (B, Hkv, n)]
    rows = [math.prod(x) for x in shapes]
    codes = record[: sum(rows) * d].view(torch.int8).split([r * d for r in rows])
    scales = record[sum(rows) * d:].view(torch.float32).split([r * (d // GROUP) for r in rows])
    return [_values(c.view(*x, d), sc.view(*x, d // GROUP), dtype) for c, sc, x in zip(codes, scales, shapes)]


def _backward(q, k, v, K, V, dout, case, t):
    """dq, dK, dV, dk, dv of the step's attention in type t."""
    B, Hkv, G, d, C, n, T = (case[x] for x in ("B", "Hkv", "G", "d", "C", "n", "T"))
    scale = 1 / math.sqrt(d)
    q = q.to(t).reshape(B, Hkv, G * T, d)
    do = dout.to(t).reshape(B, Hkv, G * T, d)
    keys, vals = torch.cat([K, k], 2).to(t), torch.cat([V, v], 2).to(t)
    row = torch.arange(T, device=q.device).repeat(G)
    col = torch.arange(n + T, device=q.device)
    s = (q @ keys.transpose(-1, -2)) * scale
    s = s.masked_fill(col - n > row[:, None], -math.inf)
    p = (s - s.amax(-1, keepdim=True)).exp()
    p = p / p.sum(-1, keepdim=True)
    dp = do @ vals.transpose(-1, -2)
    ds = p * (dp - (p * dp).sum(-1, keepdim=True))
    dq = (ds @ keys) * scale
    dkey = (ds.transpose(-1, -2) @ q) * scale
    dval = p.transpose(-1, -2) @ do
    dK = torch.zeros((B, Hkv, C, d), dtype=t, device=q.device)
    dV = torch.zeros_like(dK)
    dK[:, :, :n] = dkey[:, :, :n]
    dV[:, :, :n] = dval[:, :, :n]
    return dq.reshape(B, Hkv * G, T, d), dK, dV, dkey[:, :, n:], dval[:, :, n:]


def _carry_plain(s, t):
    c = s["case"]
    C, n, T, d = c["C"], c["n"], c["T"], c["d"]
    slot = s["slots"].long()
    placed = slot >= 0
    taken = torch.zeros((*slot.shape[:2], C + 1), dtype=torch.bool, device=slot.device)
    taken.scatter_(2, torch.where(placed, slot, C), True)
    here = torch.arange(C, device=slot.device) < n
    kept = (~taken[..., :C] & here)[..., None]
    at = slot.clamp(min=0)[..., None].expand(-1, -1, -1, d)
    sums, chunk = [], []
    for g, own_cache, own_chunk in ((s["gK"], s["dK"], s["dk"]), (s["gV"], s["dV"], s["dv"])):
        sums.append(torch.where(here[:, None], own_cache.to(t), 0.0) + torch.where(kept, g.to(t), 0.0))
        chunk.append(own_chunk.to(t) + torch.where(placed[..., None], g.to(t).gather(2, at), 0.0))
    return sums + chunk


def run(state):
    op, dtype = state["case"]["op"], state["dtype"]
    if own:
        cache = state["cache"]
        if op == "tree":
            return cache.tree_attend(state["q"], state["k"], state["v"], state["parent"])
        if op == "checkpoint":
            return cache.checkpoint_restore(cache.checkpoint(state["q"], state["k"], state["v"]))
        if op == "backward":
            return cache.checkpoint_backward(state["record"], state["dout"])
        return cache.carry_grad(state["slots"], state["case"]["n"], state["dK"], state["dV"], state["dk"],
                                state["dv"], state["gK"], state["gV"])
    if op == "tree":
        out, lse = _tree_plain(state, torch.float32)
        return out.to(dtype), lse
    if op == "checkpoint":
        return _round_trip_plain(state)
    if op == "backward":
        got = _backward(*_read(state["record"], state["case"], dtype), state["dout"], state["case"], torch.float32)
        return [x.to(dtype) for x in got]
    gK, gV, gk, gv = _carry_plain(state, torch.float32)
    return gK, gV, gk.to(dtype), gv.to(dtype)


# ---- 64 bits --------------------------------------------------------------------
def _exact_tree(s):
    """Row by row of the definition: each node's own list of ancestors, walked on the host."""
    c = s["case"]
    B, Hkv, G, d, n, T = (c[k] for k in ("B", "Hkv", "G", "d", "n", "T"))
    par = s["parent"].tolist()
    see = torch.zeros((B, T, T), dtype=torch.float64)
    for b in range(B):
        for i in range(T):
            j, path = i, []
            while 0 <= j < T:
                path.append(j)
                up = par[b][j]
                j = -2 if up >= j else up
            if j == -1:
                see[b, i, path] = 1.0
    see = see.cuda()
    out = torch.empty((B, Hkv * G, T, d), dtype=torch.float64, device="cuda")
    lse = torch.empty((B, Hkv * G, T), dtype=torch.float64, device="cuda")
    there = see.amax(-1)
    for b in range(B):
        for g in range(Hkv):
            heads = slice(g * G, (g + 1) * G)
            q = s["q"][b, heads].double() / math.sqrt(d)
            a = torch.einsum("htd,jd->htj", q, s["K"][b, g, :n].double())
            e = torch.einsum("htd,jd->htj", q, s["k"][b, g].double())
            top = e.amax(-1)
            if n:
                top = torch.maximum(top, a.amax(-1))
            a, e = (a - top[..., None]).exp(), (e - top[..., None]).exp() * see[b]
            total = a.sum(-1) + e.sum(-1)
            o = torch.einsum("htj,jd->htd", a, s["V"][b, g, :n].double()) + torch.einsum("htj,jd->htd", e, s["v"][b, g].double())
            out[b, heads] = torch.where(there[b, :, None] > 0, o / total[..., None], 0.0)
            lse[b, heads] = torch.where(there[b] > 0, top + total.log(), -math.inf)
    return out, lse


def _exact_round_trip(s):
    n, got = s["case"]["n"], []
    for name in ("q", "k", "v", "K", "V"):
        x = s[name].double()
        y = x.reshape(-1, GROUP)
        step = y.abs().max(dim=1, keepdim=True).values
        y = torch.where(step > 0, torch.round(y * 127 / step) * step / 127, torch.zeros_like(y)).reshape(x.shape)
        if name in ("K", "V"):
            y[:, :, n:] = 0
        got.append(y)
    return got


def _exact_backward(s):
    """Autograd of the attention in 64 bits, one KV head at a time."""
    c = s["case"]
    B, Hkv, G, d, C, n, T = (c[x] for x in ("B", "Hkv", "G", "d", "C", "n", "T"))
    q, k, v, K, V = (x.double() for x in _read(s["record"], c, s["dtype"]))
    do = s["dout"].double()
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    dK = torch.zeros((B, Hkv, C, d), dtype=torch.float64, device="cuda")
    dV = torch.zeros_like(dK)
    hidden = torch.ones((T, T), dtype=torch.bool, device="cuda").triu(1)
    for b in range(B):
        for g in range(Hkv):
            heads = slice(g * G, (g + 1) * G)
            leaves = [x.clone().requires_grad_() for x in (q[b, heads], k[b, g], v[b, g], K[b, g], V[b, g])]
            qh, kh, vh, Kh, Vh = leaves
            z = torch.cat([qh @ Kh.T, (qh @ kh.T).masked_fill(hidden, -math.inf)], -1) / math.sqrt(d)
            w = torch.softmax(z, -1)
            o = w[..., :n] @ Vh + w[..., n:] @ vh
            got = torch.autograd.grad(o, leaves, do[b, heads], allow_unused=True)
            dq[b, heads], dk[b, g], dv[b, g] = got[:3]
            if n:
                dK[b, g, :n], dV[b, g, :n] = got[3:]
    return dq, dK, dV, dk, dv


def _exact_carry(s):
    """Token by token, through an index of every slot's token."""
    c = s["case"]
    C, n, T, d = c["C"], c["n"], c["T"], c["d"]
    slot = s["slots"].reshape(-1, T).long()
    got = [[], []]
    for g, own_cache, own_chunk in ((s["gK"], s["dK"], s["dk"]), (s["gV"], s["dV"], s["dv"])):
        before, chunk = own_cache.double().reshape(-1, C, d).clone(), own_chunk.double().reshape(-1, T, d).clone()
        g = g.double().reshape(-1, C, d)
        for r in range(slot.shape[0]):
            t = (slot[r] >= 0).nonzero()[:, 0]
            chunk[r, t] += g[r, slot[r, t]]
            passed = torch.ones(C, dtype=torch.bool, device="cuda")
            passed[slot[r, t]] = False
            passed[n:] = False
            before[r, passed] += g[r, passed]
            before[r, n:] = 0
        got[0].append(before.reshape(s["dK"].shape))
        got[1].append(chunk.reshape(s["dk"].shape))
    return got[0] + got[1]


def exact(case, seed):
    s = prepare(case, seed)
    return {"tree": _exact_tree, "checkpoint": _exact_round_trip, "backward": _exact_backward, "carry": _exact_carry}[case["op"]](s)
