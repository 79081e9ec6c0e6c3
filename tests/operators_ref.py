"""The operators next to the step in 64 bits, and how far a kernel may be off.

Each function computes its operator from the definition in double precision and
returns, beside the values, the bounds the tests use. They are worst cases over
the roundings a kernel makes (u = half a step of a type):
  logits    a dot product of d products in fp32: (d + 4) u32 |q| |k| / sqrt(d)
            (|.| the rows' norms), doubled, so that the tensor core's own order
            and alignment of the sum are inside it: EPS below; a weight
            p = exp(s - LSE) is then off by a factor of at most 1 + dp with
            dp = 4 EPS + (keys + 32) u32 (its own logit, the maximum and sum of
            the row, the exponential, and the additions)
  weights   fed to the tensor core in bf16: u16 of each, so u16 sum p |v|
  results   rounded once to the element type: u of it.
"""
import math

import torch

U32 = 2.0**-24
U = {torch.float32: U32, torch.bfloat16: 2.0**-8}  # finfo.eps / 2
GROUP = 32


def logits_eps(q, k):
    d = q.shape[-1]
    return float(2 * (d + 4) * U32 * q.norm(dim=-1).max() * k.norm(dim=-1).max() / math.sqrt(d)) if k.numel() else 0.0


def ancestors(parent):
    """[B, T, T] bool: the nodes on the path of node i, itself included; all
    false for an absent node. Walked on the host."""
    B, T = parent.shape
    see = torch.zeros((B, T, T), dtype=torch.bool)
    for b, row in enumerate(parent.tolist()):
        for i in range(T):
            j, path = i, []
            while j >= 0:
                path.append(j)
                up = row[j]
                j = up if -1 <= up < j else -2
            if j == -1:
                see[b, i, path] = True
    return see


def tree(q, k, v, parent, K, V, n, dtype):
    """out, lse, and the bounds of both."""
    B, Hq, T, d = q.shape
    Hkv = k.shape[1]
    G = Hq // Hkv
    see = ancestors(parent).to(q.device)
    q, k, v, K, V = (x.double() for x in (q, k, v, K[:, :, :n], V[:, :, :n]))
    keys, vals = torch.cat([K, k], 2), torch.cat([V, v], 2)
    mask = torch.cat([torch.ones((B, T, n), dtype=torch.bool, device=q.device), see], 2)
    mask &= see.any(-1, keepdim=True)
    s = torch.einsum("bghtd,bgjd->bghtj", q.view(B, Hkv, G, T, d), keys) / math.sqrt(d)
    s = s.masked_fill(~mask[:, None, None], -math.inf)
    lse = torch.logsumexp(s, -1)
    p = torch.where(mask[:, None, None], (s - lse[..., None].nan_to_num(neginf=0.0)).exp(), 0.0)
    out = torch.einsum("bghtj,bgjd->bghtd", p, vals).reshape(B, Hq, T, d)
    size = torch.einsum("bghtj,bgjd->bghtd", p, vals.abs()).reshape(B, Hq, T, d)
    eps = logits_eps(q, keys)
    dp = 4 * eps + (n + T + 32) * U32
    u = U[dtype]
    bound = (dp + (u if dtype == torch.bfloat16 else 0)) * size + u * size + 1e-30
    lse = lse.reshape(B, Hq, T)
    return out, lse, bound, dp + 4 * U32 * (lse.nan_to_num(neginf=0.0).abs() + 1)


def quantise(x):
    """Codes (int8), scales (float32) and the values they stand for."""
    g = x.double().unflatten(-1, (-1, GROUP))
    top = g.abs().amax(-1, keepdim=True)
    bad = ~g.isfinite().all(-1, keepdim=True)
    codes = torch.where((top > 0) & ~bad, (127 * g / top).round(), 0.0).nan_to_num(0.0)
    scale = torch.where(bad, math.nan, top / 127).float()
    values = (codes.float() * scale).flatten(-2).to(x.dtype)
    return codes.flatten(-2).to(torch.int8), scale[..., 0], values


def backward(q, k, v, K, V, dout, n, dtype):
    """(dq, dK, dV, dk, dv) over the n slots and the chunk, and their bounds."""
    B, Hq, T, d = q.shape
    Hkv = k.shape[1]
    G = Hq // Hkv
    q, k, v, K, V, do = (x.double() for x in (q, k, v, K[:, :, :n], V[:, :, :n], dout))
    q, do = q.view(B, Hkv, G, T, d), do.view(B, Hkv, G, T, d)
    keys, vals = torch.cat([K, k], 2), torch.cat([V, v], 2)
    scale = 1 / math.sqrt(d)
    row, col = torch.arange(T, device=q.device)[:, None], torch.arange(n + T, device=q.device) - n
    s = (torch.einsum("bghtd,bgjd->bghtj", q, keys) * scale).masked_fill(col > row, -math.inf)
    p = torch.softmax(s, -1)
    dp = torch.einsum("bghtd,bgjd->bghtj", do, vals)
    D = (p * dp).sum(-1, keepdim=True)
    ds = p * (dp - D)
    grads = (scale * torch.einsum("bghtj,bgjd->bghtd", ds, keys), scale * torch.einsum("bghtj,bghtd->bgjd", ds, q),
             torch.einsum("bghtj,bghtd->bgjd", p, do))
    # |computed ds - ds| <= e: the weight's factor on p |dp| and p |D|, dp's own
    # sum, D's, and bf16 operands
    u = U[dtype]
    half = u if dtype == torch.bfloat16 else 0.0
    fac = 4 * logits_eps(q, keys) + (n + G * T + 32) * U32
    ddp = 2 * (d + 2) * U32 * float(do.norm(dim=-1).max()) * float(vals.norm(dim=-1).max())
    dD = 2 * fac * (p * dp.abs()).sum(-1, keepdim=True) + ddp
    e = 2 * fac * p * (dp.abs() + D.abs()) + p * (ddp + dD) + half * ds.abs()
    bounds = (scale * torch.einsum("bghtj,bgjd->bghtd", e, keys.abs()),
              scale * torch.einsum("bghtj,bghtd->bgjd", e, q.abs()),
              (half + fac) * torch.einsum("bghtj,bghtd->bgjd", p, do.abs()))
    bounds = [x + u * g.abs() + 1e-30 for x, g in zip(bounds, grads)]

    def split(x):
        dq, dkey, dval = x
        return dq.reshape(B, Hq, T, d), dkey[:, :, :n], dval[:, :, :n], dkey[:, :, n:], dval[:, :, n:]

    return split(grads), split(bounds)


def carry(slots, n, own_cache, own_chunk, g):
    """The gradient before the eviction of the slots and of the tokens (one of K
    or V), token by token. g None: no later step."""
    before, chunk = own_cache.double().clone(), own_chunk.double().clone()
    before[:, :, n:] = 0
    if g is not None:
        B, Hkv, T = slots.shape
        passed = torch.ones(before.shape[:3], dtype=torch.bool)
        passed[:, :, n:] = False
        for b, h, t in torch.nonzero((slots >= 0) & (slots < before.shape[2])).tolist():
            s = int(slots[b, h, t])
            chunk[b, h, t] += g[b, h, s].double()
            passed[b, h, s] = False
        before += torch.where(passed[..., None].to(g.device), g.double(), 0.0)
    return before, chunk


def within(name, got, want, bound):
    off = (got.double() - want).abs()
    bad = ~(off <= bound)
    assert not bad.any(), (f"{name}: {int(bad.sum())} of {bad.numel()} values off, worst "
                           f"{float((off / bound).nan_to_num(nan=1e9).max()):.3g} times the bound")
