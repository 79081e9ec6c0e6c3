"""The operators next to the step against their definitions in 64 bits
(operators_ref holds the formulas and derives the tolerances), their edge cases,
streams, graphs and refusals, and a training run through all of them."""
import math

import pytest
import torch

import operators_ref as ref
from h2o_kv_cache_step_b200 import H2OCache, H2OCheckpoint, H2OError, _lib

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")


def heads(dtype, B, Hkv, G, d, C, n, T, seed=0):
    """q, k, v of a chunk and K, V of a cache of C slots, n of them valid; a
    common part in the keys of a head, as trained models have."""
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*s):
        return torch.randn(s, generator=gen, device="cuda")

    lean = normal(B, Hkv, 1, d)
    q = normal(B, Hkv, G, T, d) + 0.5 * lean[:, :, None]
    K, V = normal(B, Hkv, C, d) + lean, normal(B, Hkv, C, d)
    K[:, :, n:] = 0
    V[:, :, n:] = 0
    return [x.to(dtype) for x in (q.reshape(B, Hkv * G, T, d), normal(B, Hkv, T, d) + lean, normal(B, Hkv, T, d), K, V)]


def cache_of(K, V, Hq, n, max_T=None):
    B, Hkv, C, d = K.shape
    c = H2OCache(B, Hq, Hkv, d, C, K.dtype, max_T=max_T)
    pos = torch.full((B, Hkv, C), -1, dtype=torch.int32, device="cuda")
    pos[:, :, :n] = torch.arange(n, dtype=torch.int32, device="cuda")
    c.set_state(K, V, torch.ones((B, Hkv, C), device="cuda"), pos, P=n, n=n)
    return c


def trees(B, T, seed=0, absent=True):
    gen = torch.Generator().manual_seed(seed)
    parent = torch.tensor([[int(torch.randint(-1, i, (1,), generator=gen)) if i else -1 for i in range(T)] for _ in range(B)],
                          dtype=torch.int32)
    if absent:
        parent[-1, T - T // 4:] = -2     # fewer nodes in the last sequence
        if T > 8:
            parent[0, 3], parent[0, 5] = 3, T  # a node above itself, one out of range: absent
    return parent.cuda()


TREES = [
    # dtype, B, Hkv, G, d, C, n, T
    (FP32, 1, 2, 2, 64, 256, 201, 24),
    (FP32, 2, 1, 3, 128, 50, 0, 9),       # an empty cache
    (FP32, 1, 1, 1, 64, 1, 1, 1),         # one slot, one node
    (BF16, 1, 8, 4, 128, 2048, 2048, 1),  # one token
    (BF16, 3, 2, 4, 128, 700, 643, 1),
    (BF16, 2, 2, 1, 64, 64, 64, 1),       # one row to a KV head
    (BF16, 2, 3, 2, 64, 300, 257, 5),     # a few nodes, a page of one slot at the end
    (BF16, 4, 2, 4, 128, 1000, 901, 61),
    (BF16, 1, 2, 3, 64, 129, 128, 43),    # rows 128 and 129 of a group
    (BF16, 1, 1, 8, 128, 128, 127, 16),
    (BF16, 2, 2, 3, 128, 300, 0, 77),     # an empty cache: the tree alone
    (BF16, 1, 2, 4, 64, 4000, 3999, 255),
    (BF16, 1, 2, 8, 128, 5000, 4097, 256),
    (BF16, 2, 1, 1, 128, 40, 33, 256),    # a tree longer than the cache
    # the same kinds with enough work for the tensor cores
    (BF16, 4, 8, 4, 128, 1000, 997, 1),
    (BF16, 8, 8, 2, 64, 700, 641, 3),
    (BF16, 8, 4, 3, 64, 129, 128, 43),
    (BF16, 7, 8, 1, 128, 1500, 1409, 1),
    (BF16, 8, 8, 3, 128, 300, 0, 77),
    (BF16, 16, 4, 1, 128, 40, 33, 256),
    (BF16, 2, 4, 1, 128, 16384, 16383, 5),
    (BF16, 8, 8, 4, 128, 1100, 1097, 1),  # few rows of many sequences
    (BF16, 16, 8, 1, 128, 2100, 2051, 1),
    (BF16, 16, 8, 2, 64, 900, 897, 3),
    (BF16, 1, 8, 4, 128, 9000, 8999, 1),  # one sequence, its keys divided among many CTAs
    (BF16, 14, 8, 4, 128, 2100, 2065, 40),  # more units than a CTA each
    (FP32, 1, 1, 2, 64, 3000, 2990, 1),   # fp32, the keys divided
    (FP32, 1, 2, 4, 128, 900, 899, 2),
]


@pytest.mark.parametrize("dtype,B,Hkv,G,d,C,n,T", TREES)
def test_tree_attention(dtype, B, Hkv, G, d, C, n, T):
    q, k, v, K, V = heads(dtype, B, Hkv, G, d, C, n, T, seed=T)
    parent = trees(B, T, seed=n)
    c = cache_of(K, V, Hkv * G, n)
    before = c.get_state()
    out, lse = c.tree_attend(q, k, v, parent)
    c.sync_check()
    want, wlse, bound, lbound = ref.tree(q, k, v, parent, K, V, n, dtype)
    ref.within("out", out, want, bound)
    there = wlse > -math.inf
    assert torch.equal(there, lse > -math.inf)
    assert not out[~there].any()
    ref.within("lse", lse[there], wlse[there], lbound[there])
    again = c.tree_attend(q, k, v, parent)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    for a, b in zip(before, c.get_state()):
        assert torch.equal(a, b) if torch.is_tensor(a) else a == b


@pytest.mark.parametrize("dtype,B,Hkv,G,d,n,T", [(FP32, 2, 2, 2, 64, 70, 12), (BF16, 2, 2, 4, 128, 700, 3), (BF16, 2, 2, 4, 128, 700, 40),
                                                  (BF16, 2, 2, 2, 64, 130, 200), (BF16, 8, 8, 4, 128, 700, 3)])
def test_tree_keys_that_a_row_does_not_see_leave_it_alone(dtype, B, Hkv, G, d, n, T):
    C = 800
    q, k, v, K, V = heads(dtype, B, Hkv, G, d, C, n, T, seed=5)
    parent = trees(B, T, seed=6)
    clean = cache_of(K, V, Hkv * G, n).tree_attend(q, k, v, parent)
    see = ref.ancestors(parent).cuda()
    K[:, :, n:], V[:, :, n:] = math.nan, math.inf
    for b, node, kv, ww in ((0, T // 2, math.nan, 1.0), (1, T - 1, math.inf, math.nan), (0, T - 1, 0.0, -math.inf),
                          (0, 1, math.nan, 1.0), (1, 2, 0.0, math.nan)):
        k[b, :, node] += kv
        v[b, :, node] *= ww
    hit = torch.zeros((B, T), dtype=torch.bool, device="cuda")
    for b, node in ((0, T // 2), (1, T - 1), (0, T - 1), (0, 1), (1, 2)):
        hit[b] |= see[b, :, node]
    out, lse = cache_of(K, V, Hkv * G, n).tree_attend(q, k, v, parent)
    ok = ~hit[:, None].expand(B, Hkv * G, T)
    assert 0 < int(ok.sum()) < ok.numel()
    assert torch.equal(out[ok], clean[0][ok]) and torch.equal(lse[ok], clean[1][ok])
    assert not out[~ok].isfinite().all(-1).any()


def test_tree_bad_slots_and_queries_are_not_hidden():
    """A NaN in a valid slot reaches every row of its KV head, one in a query its
    own row; an infinite logit is NaN as in the definition."""
    for T in (1, 9, 60):
        q, k, v, K, V = heads(BF16, 1, 2, 4, 128, 512, 512, T, seed=2)
        parent = trees(1, T, absent=False)
        clean = cache_of(K, V, 8, 512).tree_attend(q, k, v, parent)[0]
        for value in (math.nan, math.inf):
            bad = K.clone()
            bad[0, 1, 300, 7] = value
            out, lse = cache_of(bad, V, 8, 512).tree_attend(q, k, v, parent)
            assert torch.equal(out[:, :4], clean[:, :4])
            # an infinite key gives a row +inf or -inf by its query's sign; -inf drops the key
            seen = torch.ones((4, T), dtype=torch.bool, device="cuda") if value != value else q[0, 4:, :, 7] > 0
            assert out[0, 4:][seen].isnan().all() and lse[0, 4:][seen].isnan().all()
            assert out[0, 4:][~seen].isfinite().all()
        qb = q.clone()
        qb[0, 5, T - 1, 3] = math.nan
        out = cache_of(K, V, 8, 512).tree_attend(qb, k, v, parent)[0]
        assert out[0, 5, T - 1].isnan().all()
        out[0, 5, T - 1] = clean[0, 5, T - 1]
        assert torch.equal(out, clean)


@pytest.mark.parametrize("dtype,B", [(FP32, 1), (BF16, 1), (BF16, 16)])
def test_tree_of_one_path_of_256_nodes(dtype, B):
    q, k, v, K, V = heads(dtype, B, 2, 1, 64, 64, 60, 256, seed=4)
    parent = (torch.arange(256, dtype=torch.int32, device="cuda") - 1).expand(B, 256).contiguous()
    parent[-1, 200] = 200                  # the end of the last sequence's path is cut off
    out, lse = cache_of(K, V, 2, 60).tree_attend(q, k, v, parent)
    want, wlse, bound, lbound = ref.tree(q, k, v, parent, K, V, 60, dtype)
    there = wlse > -math.inf
    assert int((~there).sum()) == 2 * 56
    ref.within("out", out, want, bound)
    ref.within("lse", lse[there], wlse[there], lbound[there])
    assert (lse[~there] == -math.inf).all() and not out[~there].any()


@pytest.mark.parametrize("steps", [(0, 20, 21, 60, 61), (0, -90, 15, 200, 199, 500), (300, 0, -300, 310, 400)])
@pytest.mark.parametrize("B,T", [(1, 2), (1, 70), (5, 70)])
def test_tree_scores_that_jump_along_the_cache(steps, B, T):
    """Logits that rise and fall by tens and hundreds of powers of two from one
    128-slot block to the next: the running maximum moves late, at once, or not."""
    G, d, n = 2, 64, 128 * len(steps) - 30
    q, k, v, K, V = heads(BF16, B, 1, G, d, 128 * len(steps), n, T, seed=12)
    q[:, 1, :, 0] *= -1
    q[..., 0] = torch.where(q[..., 0] < 0, -1.0, 1.0)
    for i, s in enumerate(steps):  # s powers of two in the first channel, for the rows with a 1 there
        K[:, :, 128 * i:128 * (i + 1), 0] = s * math.log(2) * math.sqrt(d)
    K[:, :, n:] = 0
    parent = trees(B, T)
    c = cache_of(K, V, G, n)
    out, lse = c.tree_attend(q, k, v, parent)
    want, wlse, bound, lbound = ref.tree(q, k, v, parent, K, V, n, BF16)
    there = wlse > -math.inf
    ref.within("out", out, want, bound)
    ref.within("lse", lse[there], wlse[there], lbound[there])
    assert torch.equal(out, c.tree_attend(q, k, v, parent)[0])


@pytest.mark.parametrize("B,T", [(2, 3), (2, 100), (16, 100)])
def test_tree_with_no_node_in_it(B, T):
    q, k, v, K, V = heads(BF16, B, 2, 2, 64, 256, 200, T)
    parent = torch.full((B, T), -2, dtype=torch.int32, device="cuda")
    parent[0, 1:] = 0                      # under an absent node: absent too
    out, lse = cache_of(K, V, 4, 200).tree_attend(q, k, v, parent)
    assert not out.any() and (lse == -math.inf).all()


@pytest.mark.parametrize("dtype,T", [(FP32, 20), (BF16, 4), (BF16, 130)])
def test_a_chain_is_what_the_step_computes(dtype, T):
    """One path of T nodes: rows as of the step that commits it."""
    q, k, v, K, V = heads(dtype, 2, 2, 4, 128, 384, 380, T, seed=9)
    c = cache_of(K, V, 8, 380)
    parent = (torch.arange(T, dtype=torch.int32, device="cuda") - 1).expand(2, T).contiguous()
    out, lse = c.tree_attend(q, k, v, parent)
    step = c.step(q, k, v)
    _, _, bound, lbound = ref.tree(q, k, v, parent, K, V, 380, dtype)
    extra = 1e-4 if dtype == BF16 else 0.0  # the step's polynomial exponentials: 7.7e-5 each
    ref.within("out", out, step.double(), 2 * bound + 2 * extra * V.abs().max())
    ref.within("lse", lse, c.lse().double(), 2 * lbound + extra)


# ---- checkpoints ------------------------------------------------------------------
RECORDS = [
    # dtype, B, Hkv, G, d, C, n, T
    (FP32, 1, 2, 2, 64, 256, 256, 64),
    (FP32, 2, 1, 1, 128, 9, 0, 1),
    (BF16, 1, 8, 4, 128, 300, 300, 129),
    (BF16, 3, 2, 3, 64, 100, 77, 31),
    (BF16, 1, 1, 1, 64, 1, 1, 1),
]


@pytest.mark.parametrize("dtype,B,Hkv,G,d,C,n,T", RECORDS)
def test_checkpoint_codes_scales_and_values(dtype, B, Hkv, G, d, C, n, T):
    q, k, v, K, V = heads(dtype, B, Hkv, G, d, C, n, T, seed=n + T)
    q[0, 0, 0, :32] = 0                                       # a group of zeros
    k[0, 0, 0, :32] = torch.arange(32, device="cuda") * 0.5   # codes next to and on borders
    k[0, 0, 0, 31] = 127.0
    v[0, 0, 0, 32:64] = 2e-41 * torch.arange(32, device="cuda")  # subnormal
    v[0, 0, 0, :32] = 3e38
    v[0, 0, 0, 1:32:2] = -1.5e38
    q[-1, -1, -1, 40] = math.nan
    q[-1, -1, -1, 1] = math.inf
    c = cache_of(K, V, Hkv * G, n)
    ck = c.checkpoint(q, k, v)
    assert ck.n == n and ck.T == T and ck.nbytes == sum(x.numel() for x in (q, k, v)) * 9 // 8 + 2 * B * Hkv * n * d * 9 // 8
    xs = [q, k, v, K[:, :, :n], V[:, :, :n]]
    want = [ref.quantise(x) for x in xs]
    for name, got, w in zip("qkvKV", ck.codes(), want):
        assert torch.equal(got, w[0]), name
    for name, got, w in zip("qkvKV", ck.scales(), want):
        assert torch.equal(got.nan_to_num(nan=-1), w[1].nan_to_num(nan=-1)), name
    back = c.checkpoint_restore(ck)
    c.sync_check()
    for name, got, w, x in zip("qkvKV", back, want, xs):
        w = w[2]
        if name in "KV":
            assert got.shape[2] == C and not got[:, :, n:].any()
            got = got[:, :, :n]
        assert torch.equal(got.nan_to_num(nan=-1), w.nan_to_num(nan=-1)), name
        assert torch.equal(got.isnan(), w.isnan())


@pytest.mark.parametrize("exponent", [-120, -40, 0, 100])
def test_checkpoint_codes_of_every_bf16_quotient(exponent):
    """Every pair of an 8-bit largest magnitude and an 8-bit value at or below it
    by up to 2^9, the borders k + 1/2 among them."""
    top = torch.arange(128, 256, device="cuda", dtype=torch.float64)
    x = torch.stack([torch.arange(128, 256, device="cuda", dtype=torch.float64) * 2.0**-s for s in range(10)]).reshape(-1)
    x = torch.cat([x, x.new_zeros(-len(x) % 31)]).view(1, -1, 31)
    g = torch.cat([top.view(-1, 1, 1).expand(-1, x.shape[1], 1), x.expand(128, -1, -1)], 2)
    g = torch.where(g > g[..., :1], -g / 2, g) * 2.0**exponent   # nothing above the first
    rows = g.reshape(-1, 32).to(BF16)
    rows = torch.cat([rows, rows.new_zeros((-len(rows) % 4, 32))]).view(1, 1, -1, 128)
    c = H2OCache(1, 1, 1, 128, 4, BF16, max_T=rows.shape[2])
    ck = c.checkpoint(rows, rows, -rows)
    want = ref.quantise(rows)
    for got, sign in zip(ck.codes(), (1, 1, -1)):
        assert torch.equal(got, want[0] * sign)
    assert torch.equal(ck.scales()[0], want[1])


def test_checkpoint_outlives_the_cache_it_was_taken_from():
    q, k, v, K, V = heads(BF16, 1, 2, 2, 64, 64, 64, 16)
    c = cache_of(K, V, 4, 64)
    ck = c.checkpoint(q, k, v)
    first = c.checkpoint_restore(ck)
    c.step(q, k, v)
    c.reset()
    for a, b in zip(first, c.checkpoint_restore(ck)):
        assert torch.equal(a, b)
    other = H2OCache(1, 4, 2, 64, 80, BF16)   # more slots: the record's, then zeros
    K2 = other.checkpoint_restore(ck)[3]
    assert torch.equal(K2[:, :, :64], first[3]) and not K2[:, :, 64:].any()


BACKWARDS = [
    # dtype, B, Hkv, G, d, C, n, T
    (FP32, 1, 2, 2, 64, 256, 256, 64),
    (FP32, 2, 1, 3, 128, 40, 33, 17),
    (FP32, 1, 1, 1, 64, 5, 0, 1),         # a row that sees itself alone: dq and dk are zero
    (BF16, 1, 1, 1, 64, 5, 0, 1),
    (BF16, 1, 2, 2, 128, 40, 0, 130),     # an empty cache
    (BF16, 2, 2, 8, 64, 300, 257, 77),
    (BF16, 2, 3, 3, 128, 200, 127, 129),
    (BF16, 1, 2, 4, 128, 512, 512, 256),
    (BF16, 1, 2, 1, 64, 1000, 999, 1),
    (BF16, 1, 1, 4, 128, 2000, 1921, 300),
    (BF16, 3, 1, 5, 64, 128, 128, 383),
    (BF16, 1, 2, 8, 64, 400, 390, 16),    # eight heads in a query tile
    (BF16, 2, 1, 3, 128, 130, 100, 50),   # heads that end inside a tile
    (BF16, 1, 1, 1, 128, 4000, 3950, 64), # few tiles, many key blocks
    (BF16, 1, 1, 2, 64, 3000, 3000, 200),
    (BF16, 1, 2, 4, 128, 300, 300, 1),
]


@pytest.mark.parametrize("dtype,B,Hkv,G,d,C,n,T", BACKWARDS)
def test_backward_from_a_checkpoint(dtype, B, Hkv, G, d, C, n, T):
    q, k, v, K, V = heads(dtype, B, Hkv, G, d, C, n, T, seed=n + T)
    c = cache_of(K, V, Hkv * G, n)
    ck = c.checkpoint(q, k, v)
    dout = torch.randn(q.shape, generator=torch.Generator(device="cuda").manual_seed(4), device="cuda").to(dtype)
    rest = c.checkpoint_restore(ck)
    c.reset()                              # the cache plays no part
    got = c.checkpoint_backward(ck, dout)
    c.sync_check()
    want, bound = ref.backward(*rest, dout, n, dtype)
    for name, g, w, b in zip(("dq", "dK", "dV", "dk", "dv"), got, want, bound):
        assert g.dtype == dtype
        if name in ("dK", "dV"):
            assert g.shape[2] == C and not g[:, :, n:].any()
            g = g[:, :, :n]
        ref.within(name, g, w, b)
    for a, b in zip(got, c.checkpoint_backward(ck, dout)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("B,Hkv,G,d,n,T", [(2, 2, 3, 64, 130, 50), (1, 8, 4, 128, 2000, 500)])
def test_backward_keeps_a_bad_kv_head_to_itself(B, Hkv, G, d, n, T):
    """NaN and infinities in the record and in dout of one KV head (its heads, its
    last rows and slots, next to the others' in memory) leave the rest bit for bit."""
    q, k, v, K, V = heads(BF16, B, Hkv, G, d, n, n, T, seed=21)
    dout = torch.randn(q.shape, generator=torch.Generator(device="cuda").manual_seed(4), device="cuda").to(BF16)

    def grads(*x):
        c = cache_of(x[3], x[4], Hkv * G, n)
        return c.checkpoint_backward(c.checkpoint(*x[:3]), x[5])

    want = grads(q, k, v, K, V, dout)
    b, g = B - 1, Hkv // 2
    bad = [x.clone() for x in (q, k, v, K, V, dout)]
    for x, h in zip(bad, (g * G + G - 1, g, g, g, g, g * G)):
        x[b, h, -1, 3], x[b, h, 0, 5] = math.nan, math.inf
    got = grads(*bad)
    hit = torch.zeros((B, Hkv), dtype=torch.bool, device="cuda")
    hit[b, g] = True
    for name, x, y in zip(("dq", "dK", "dV", "dk", "dv"), got, want):
        x, y = (t.view(B, Hkv, -1, d) for t in (x, y))
        assert torch.equal(x[~hit], y[~hit]), name
        assert x[hit].isnan().any(), name


def test_backward_of_equal_keys():
    """Every key the same: dq is zero up to the roundings of its operands."""
    q, k, v, K, V = heads(BF16, 1, 1, 2, 64, 256, 256, 128)
    k[:], K[:] = k[:, :, :1], k[:, :, :1]
    c = cache_of(K, V, 2, 256)
    ck = c.checkpoint(q, k, v)
    dout = torch.randn(q.shape, generator=torch.Generator(device="cuda").manual_seed(4), device="cuda").to(BF16)
    want, bound = ref.backward(*c.checkpoint_restore(ck), dout, 256, BF16)
    for name, g, w, b in zip(("dq", "dK", "dV", "dk", "dv"), c.checkpoint_backward(ck, dout), want, bound):
        ref.within(name, g, w, b)


@pytest.mark.parametrize("dtype,B,Hkv,d,C,n,T", [(FP32, 2, 3, 64, 300, 251, 77), (BF16, 1, 2, 128, 33, 33, 100),
                                                  (BF16, 2, 1, 64, 1, 0, 1), (BF16, 1, 2, 128, 500, 499, 1)])
@pytest.mark.parametrize("last", [False, True])
def test_carry(dtype, B, Hkv, d, C, n, T, last):
    gen = torch.Generator(device="cuda").manual_seed(C + T)

    def normal(t, *s):
        return torch.randn(s, generator=gen, device="cuda").to(t)

    dK, dV, dk, dv = [normal(dtype, B, Hkv, x, d) for x in (C, C, T, T)]
    g = [None, None] if last else [normal(FP32, B, Hkv, C, d) for _ in range(2)]
    slots = torch.full((B, Hkv, T), -1, dtype=torch.int32)
    for b in range(B):
        for h in range(Hkv):
            k = min(T, C) // 2 + 1
            at = torch.randperm(T, generator=torch.Generator().manual_seed(b + 7 * h))[:min(k, T)]
            slots[b, h, at] = torch.randperm(C, generator=torch.Generator().manual_seed(b + 9 * h))[:len(at)].int()
            slots[b, h, T // 3] = -5 if h else C + 3  # outside the cache: dropped
    c = H2OCache(B, Hkv, Hkv, d, C, dtype)
    gK, gV, gk, gv = c.carry_grad(slots.cuda(), n, dK, dV, dk, dv, *g)
    c.sync_check()
    # one addition in fp32 and one rounding to the element type: exact ties aside, equal
    for got, tok, own, ch, nxt in ((gK, gk, dK, dk, g[0]), (gV, gv, dV, dv, g[1])):
        before, chunk = ref.carry(slots, n, own, ch, nxt)
        ref.within("cache", got, before, ref.U32 * before.abs())
        ref.within("chunk", tok, chunk, (ref.U[dtype] + 2 * ref.U32) * chunk.abs())


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_offsets_past_32_bits(dtype):
    """K and V of 2^31 values and more, looked at where they end: the last KV head
    of the last sequence, its rows drawn to slots near the cache's end."""
    B, Hkv, d, T, C = 2, 8, 128, 2, 2**20 + 77
    q, k, v, Ke, Ve = heads(dtype, 1, 1, 1, d, C, C, T, seed=5)
    for t in range(T):
        Ke[0, 0, C - 1 - 99 * t] = (20 * q[0, 0, t].float() / q[0, 0, t].float().norm()).to(dtype)

    def last(x, fill=0):  # x as the last head of them all
        whole = torch.full((B, Hkv, *x.shape[2:]), fill, dtype=x.dtype, device="cuda")
        whole[-1, -1] = x[0, 0]
        return whole

    def end(x):
        return x[-1:, -1:].clone()

    c = cache_of(last(Ke), last(Ve), Hkv, C, max_T=8)
    torch.cuda.empty_cache()
    whole = [last(x) for x in (q, k, v)]
    parent = torch.tensor([[-1, -2], [-1, 0]], dtype=torch.int32, device="cuda")
    out, lse = c.tree_attend(*whole, parent)
    c.sync_check()
    want, wlse, bound, lbound = ref.tree(q, k, v, parent[1:], Ke, Ve, C, dtype)
    ref.within("out", end(out), want, bound)
    ref.within("lse", end(lse), wlse, lbound)

    ck = c.checkpoint(*whole)
    rest = c.checkpoint_restore(ck)
    c.sync_check()
    for x, got in zip((q, k, v, Ke, Ve), rest):
        assert torch.equal(ref.quantise(x)[2], end(got)) and not got[0, 0].any()
    rest = [end(x) for x in rest]
    torch.cuda.empty_cache()

    dout = torch.randn(q.shape, generator=torch.Generator(device="cuda").manual_seed(4), device="cuda").to(dtype)
    got = c.checkpoint_backward(ck, last(dout))
    c.sync_check()
    want, bound = ref.backward(*rest, dout, C, dtype)
    for name, g, w, b in zip(("dq", "dK", "dV", "dk", "dv"), got, want, bound):
        assert not g[0, 0].any()
        ref.within(name, end(g), w, b)
    del ck, want, bound, rest
    torch.cuda.empty_cache()

    slots = torch.tensor([[[-1, C - 3]]], dtype=torch.int32, device="cuda")
    nxt = torch.randn(Ke.shape, generator=torch.Generator(device="cuda").manual_seed(6), device="cuda")
    gnext = last(nxt)
    gK, gV, gk, gv = c.carry_grad(last(slots, fill=-1), C, *got[1:], gnext, gnext)
    c.sync_check()
    for g, tok, own, ch in ((gK, gk, got[1], got[3]), (gV, gv, got[2], got[4])):
        before, chunk = ref.carry(slots, C, end(own), end(ch), nxt)
        ref.within("cache", end(g), before, ref.U32 * before.abs())
        ref.within("chunk", end(tok), chunk, (ref.U[dtype] + 2 * ref.U32) * chunk.abs())


# ---- together -----------------------------------------------------------------------
@pytest.mark.parametrize("dtype", [FP32, BF16])
def test_training_run(dtype):
    """Five chunks through checkpoint and step, then backward and carry, last
    chunk first, against autograd in 64 bits through the whole run: the cache's
    contents are replayed with the recorded slots, and every chunk attends to
    the values its record stands for (straight through)."""
    B, Hkv, G, d, C, T, steps = 2, 2, 2, 64, 96, 40, 5
    gen = torch.Generator(device="cuda").manual_seed(8)
    c = H2OCache(B, Hkv * G, Hkv, d, C, dtype)
    chunks, records, slots, ns, douts = [], [], [], [], []
    for _ in range(steps):
        q, k, v = (torch.randn((B, h, T, d), generator=gen, device="cuda").to(dtype) for h in (Hkv * G, Hkv, Hkv))
        records.append(c.checkpoint(q, k, v))
        ns.append(c.counters()[1])
        out = c.step(q, k, v)
        slots.append(c.token_slots())
        douts.append(torch.randn(out.shape, generator=gen, device="cuda").to(dtype))
        chunks.append((q, k, v))
    got, gK, gV = [None] * steps, None, None
    for i in reversed(range(steps)):
        dq, dK, dV, dk, dv = c.checkpoint_backward(records[i], douts[i])
        gK, gV, gk, gv = c.carry_grad(slots[i], ns[i], dK, dV, dk, dv, gK, gV)
        got[i] = (dq, gk, gv)
    c.sync_check()
    assert ns == [0, 40, 80, 96, 96]

    leaves = [[x.double().requires_grad_() for x in ch] for ch in chunks]
    K = torch.zeros((B, Hkv, C, d), dtype=torch.float64, device="cuda")
    V = torch.zeros_like(K)
    total = 0.0
    for i in range(steps):
        n, rest = ns[i], [x.double() for x in c.checkpoint_restore(records[i])]
        q, k, v = leaves[i]
        use = [a + (b - a).detach() for a, b in zip((q, k, v, K, V), rest)]
        s = torch.einsum("bghtd,bgjd->bghtj", use[0].view(B, Hkv, G, T, d), torch.cat([use[3][:, :, :n], use[1]], 2)) / math.sqrt(d)
        s = s.masked_fill(torch.arange(n + T, device="cuda") - n > torch.arange(T, device="cuda")[:, None], -math.inf)
        o = torch.einsum("bghtj,bgjd->bghtd", torch.softmax(s, -1), torch.cat([use[4][:, :, :n], use[2]], 2))
        total = total + (o.reshape(B, Hkv * G, T, d) * douts[i].double()).sum()
        at = slots[i].long()
        put = (at[..., None] == torch.arange(C, device="cuda")).double()       # [B,Hkv,T,C]
        keep = (1 - put.sum(2))[..., None]
        K = K * keep + torch.einsum("bgtc,bgtd->bgcd", put, k)
        V = V * keep + torch.einsum("bgtc,bgtd->bgcd", put, v)
    total.backward()
    # each of the up to 5 terms of a gradient carries the relative roundings of a
    # backward: fp32 sums of a few hundred products (1e-4 of the largest value is
    # far above their worst), bf16 operands and results (3 half steps of the term)
    tol = {FP32: 1e-4, BF16: 3 * 5 * 2.0**-8}[dtype]
    for i in range(steps):
        for name, g, leaf in zip("qkv", got[i], leaves[i]):
            w = leaf.grad
            assert float((g.double() - w).abs().max()) <= tol * float(w.abs().max()), (i, name)


def test_draft_verify_commit():
    """A serving loop: draft a tree, verify it, commit one path with the step;
    the committed rows agree with the tree's."""
    B, Hkv, G, d, C, T = 2, 2, 4, 128, 256, 12
    q, k, v, K, V = heads(BF16, B, Hkv, G, d, C, 256, T, seed=3)
    c = cache_of(K, V, Hkv * G, 256)
    path = [0, 2, 5, 9]
    parent = torch.full((B, T), -1, dtype=torch.int32)
    for a, b in zip(path, path[1:]):
        parent[:, b] = a
    parent[:, 11], parent[:, 7] = 2, 0
    out, _ = c.tree_attend(q, k, v, parent.cuda())
    qc, kc, vc = (x[:, :, path].contiguous() for x in (q, k, v))
    step = c.step(qc, kc, vc)
    chain = (torch.arange(4, dtype=torch.int32, device="cuda") - 1).expand(B, 4).contiguous()
    _, _, bound, _ = ref.tree(qc, kc, vc, chain, K, V, 256, BF16)
    ref.within("committed rows", out[:, :, path], step.double(), 2 * bound + 1e-4 * V.abs().max())
    assert c.counters()[0] == 260


# ---- streams, graphs, refusals --------------------------------------------------------
def calls(dtype=BF16, T=40):
    q, k, v, K, V = heads(dtype, 2, 2, 4, 128, 300, 290, T, seed=1)
    c = cache_of(K, V, 8, 290)
    parent = trees(2, T)
    ck = c.checkpoint(q, k, v)
    dout = torch.randn_like(q)
    dK, dV, dk, dv = [torch.randn_like(x) for x in (K, V, k, v)]
    g = [torch.randn(K.shape, device="cuda") for _ in range(2)]
    slots = torch.full((2, 2, T), -1, dtype=torch.int32, device="cuda")
    slots[:, :, 1] = 7
    return c, {
        "tree": lambda **kw: c.tree_attend(q, k, v, parent, **kw),
        "checkpoint": lambda **kw: (c.checkpoint(q, k, v, **kw).buffer,),
        "restore": lambda **kw: c.checkpoint_restore(ck, **kw),
        "backward": lambda **kw: c.checkpoint_backward(ck, dout, **kw),
        "carry": lambda **kw: c.carry_grad(slots, 290, dK, dV, dk, dv, *g, **kw),
    }


@pytest.mark.parametrize("dtype", [FP32, BF16])
@pytest.mark.parametrize("T", [2, 40])
def test_on_another_stream_and_replayed_from_a_graph(dtype, T):
    c, ops = calls(dtype, T)
    want = {name: op() for name, op in ops.items()}
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for name, op in ops.items():
        got = op(stream=side)
        side.synchronize()
        for a, b in zip(want[name], got):
            assert torch.equal(a, b), name
    for name, op in ops.items():
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = op()
        for _ in range(2):
            for x in got:
                x.zero_()
            graph.replay()
            torch.cuda.synchronize()
            for a, b in zip(want[name], got):
                assert torch.equal(a, b), name
        del graph


def test_a_captured_backward_needs_its_workspace_first():
    q, k, v, K, V = heads(BF16, 1, 2, 2, 64, 64, 64, 32)
    c = cache_of(K, V, 4, 64)
    ck, dout = c.checkpoint(q, k, v), torch.randn_like(q)
    with pytest.raises(H2OError, match="outside a capture"):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            q.add_(0)  # the graph is not empty
            c.checkpoint_backward(ck, dout)
    graph = torch.cuda.CUDAGraph()
    want = c.checkpoint_backward(ck, dout)
    with torch.cuda.graph(graph):
        got = c.checkpoint_backward(ck, dout)
    # a larger call takes a new workspace; the graph keeps the old one
    big = heads(BF16, 1, 2, 2, 64, 64, 64, 200)
    c.checkpoint_backward(c.checkpoint(*big[:3]), torch.randn_like(big[0]))
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [FP32, BF16])
def test_a_captured_tree_needs_its_workspace_first(dtype):
    q, k, v, K, V = heads(dtype, 1, 2, 2, 64, 64, 64, 8)
    c, parent = cache_of(K, V, 4, 64), trees(1, 8)
    with pytest.raises(H2OError, match="outside a capture"):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            q.add_(0)  # the graph is not empty
            c.tree_attend(q, k, v, parent)
    want = c.tree_attend(q, k, v, parent)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = c.tree_attend(q, k, v, parent)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


def test_refusals():
    q, k, v, K, V = heads(BF16, 1, 2, 2, 64, 64, 50, 8)
    c = cache_of(K, V, 4, 50)
    parent = trees(1, 8)
    L, P = _lib.lib(), lambda t: t.data_ptr()
    out, lse = torch.empty_like(q), torch.empty((1, 4, 8), device="cuda")
    assert L.h2o_tree_attend(c.handle, P(q), P(k), P(v), P(parent), P(out), P(lse), 0, None) == _lib.H2O_ERR_ARG
    assert L.h2o_tree_attend(c.handle, P(q), P(k), P(v), P(parent), P(out), P(lse), 257, None) == _lib.H2O_ERR_UNSUPPORTED
    assert L.h2o_tree_attend(c.handle, P(q), P(k), P(v), None, P(out), P(lse), 8, None) == _lib.H2O_ERR_ARG
    assert L.h2o_tree_attend(c.handle, P(q) + 2, P(k), P(v), P(parent), P(out), P(lse), 7, None) == _lib.H2O_ERR_ALIGN
    assert L.h2o_tree_attend(c.handle, P(q), P(k), P(v), P(parent), P(out), P(lse) + 2, 7, None) == _lib.H2O_ERR_ALIGN
    ck = c.checkpoint(q, k, v)
    args = (P(q), P(k), P(v), P(K), P(V), None)
    assert L.h2o_checkpoint_save(c.handle, P(q), P(k), P(v), 8, P(ck.buffer), ck.nbytes - 1, None) == _lib.H2O_ERR_ARG
    assert L.h2o_checkpoint_restore(c.handle, P(ck.buffer), ck.nbytes, 8, 65, *args) == _lib.H2O_ERR_ARG
    assert L.h2o_checkpoint_restore(c.handle, P(ck.buffer), ck.nbytes, 8, -1, *args) == _lib.H2O_ERR_ARG
    assert L.h2o_checkpoint_restore(c.handle, P(ck.buffer), ck.nbytes, 9, 50, *args) == _lib.H2O_ERR_ARG
    assert L.h2o_checkpoint_restore(c.handle, P(ck.buffer), ck.nbytes, 8, 50, *[None] * 6) == _lib.H2O_ERR_ARG
    assert L.h2o_checkpoint_restore(c.handle, P(ck.buffer) + 4, ck.nbytes, 8, 50, *args) == _lib.H2O_ERR_ALIGN
    g = [torch.zeros(K.shape, device="cuda") for _ in range(3)]
    slots = torch.full((1, 2, 8), -1, dtype=torch.int32, device="cuda")
    rest = (P(K), P(V), P(k), P(v))
    assert L.h2o_carry_grad(c.handle, P(slots), 8, 50, *rest, P(g[0]), None, P(g[1]), P(g[2]), P(k), P(v), None) == _lib.H2O_ERR_ARG
    assert L.h2o_carry_grad(c.handle, P(slots), 8, 50, *rest, P(g[0]), P(g[0]), P(g[0]), P(g[2]), P(k), P(v), None) == _lib.H2O_ERR_ARG
    with pytest.raises(ValueError):
        c.tree_attend(q.transpose(2, 3).contiguous().transpose(2, 3), k, v, parent)
    with pytest.raises(ValueError):
        c.tree_attend(q, k, v, parent.long())
    with pytest.raises(ValueError):
        c.checkpoint_backward(ck, torch.zeros((1, 4, 9, 64), dtype=BF16, device="cuda"))
    with pytest.raises(ValueError):
        H2OCheckpoint(ck.buffer[:-1], 1, 4, 2, 64, 8, 50)
    c.set_policy(_lib.H2O_POLICY_INSERT_ALWAYS)
    with pytest.raises(H2OError, match="insert-always"):
        c.tree_attend(q, k, v, parent)
    with pytest.raises(H2OError, match="insert-always"):
        c.checkpoint(q, k, v)
    c.sync_check()


@pytest.mark.parametrize("dtype", [FP32, BF16])
def test_a_failed_allocation_leaves_the_next_step_alone(dtype):
    """A backward whose workspace fits no card (it fails before anything is launched
    or read) and then a step."""
    q, k, v, K, V = heads(dtype, 1, 1, 2, 128, 64, 50, 40)
    c, other = cache_of(K, V, 2, 50), cache_of(K, V, 2, 50)
    p = q.data_ptr()
    rc = _lib.lib().h2o_checkpoint_backward(c.handle, p, 2**62, 2**29, 50, p, p, p, p, p, p, None)
    assert rc == _lib.H2O_ERR_OOM
    assert torch.equal(c.step(q, k, v), other.step(q, k, v))
    ck, dout = c.checkpoint(q, k, v), torch.randn_like(q)
    for a, b in zip(c.checkpoint_backward(ck, dout), other.checkpoint_backward(ck, dout)):
        assert torch.equal(a, b)


def test_checkpoint_codes_of_the_largest_bf16_quotients():
    """As above up to the type's largest value: magnitudes whose reciprocals are subnormal."""
    for exponent in (118, 119, 120):
        test_checkpoint_codes_of_every_bf16_quotient(exponent)


def test_checkpoint_values_over_the_whole_range_of_fp32():
    """Every power of two and the values next to it, the largest finite one among them:
    finite, and off by at most half a code, the scale's rounding and the product's."""
    e = torch.arange(-149, 128, dtype=torch.float64)
    tops = torch.cat([2.0**e, 1.5 * 2.0**e[1:], (2 - 2.0**-23) * 2.0**e[23:]])
    gen = torch.Generator().manual_seed(1)
    x = tops[:, None] * torch.cat([torch.ones(len(tops), 1, dtype=torch.float64),
                                   2 * torch.rand((len(tops), 31), generator=gen, dtype=torch.float64) - 1], 1)
    x = torch.cat([x, -x]).float()
    rows = torch.cat([x, x.new_zeros((-len(x) % 2, 32))]).view(1, 1, -1, 64).cuda()
    c = H2OCache(1, 1, 1, 64, 4, FP32, max_T=rows.shape[2])
    back = c.checkpoint_restore(c.checkpoint(rows, rows, -rows))
    for got, want in zip(back, (rows, rows, -rows)):
        assert got.isfinite().all()
        w = want.double().unflatten(-1, (-1, 32))
        top = w.abs().amax(-1, keepdim=True)
        # a / 254, and twice the roundings (2^-24, or half the smallest step): the scale's,
        # 127 times where it is subnormal, and the product's
        bound = top / 254 + 2 * (2 * ref.U32 * top + 128 * 2.0**-150)
        assert ((got.double().unflatten(-1, (-1, 32)) - w).abs() <= bound).all()


LARGE_BACKWARDS = [
    # dtype, B, Hkv, G, d, C, n, T: grids of several waves on the tensor cores, query tiles that
    # hold the end of one head and the start of another
    (BF16, 1, 8, 4, 128, 2048, 2048, 1024),
    (BF16, 4, 8, 3, 64, 1500, 1409, 333),
    (BF16, 2, 8, 5, 128, 1100, 1037, 260),
    # fp32: two query rows per CTA and one key, then two of both
    (FP32, 2, 2, 2, 64, 70, 61, 77),
    (FP32, 1, 2, 4, 128, 300, 257, 151),
    (FP32, 3, 2, 1, 64, 200, 200, 101),
]


@pytest.mark.parametrize("dtype,B,Hkv,G,d,C,n,T", LARGE_BACKWARDS)
def test_large_backward_from_a_checkpoint(dtype, B, Hkv, G, d, C, n, T):
    """As above, the 64-bit definition one KV head at a time."""
    q, k, v, K, V = heads(dtype, B, Hkv, G, d, C, n, T, seed=n + T)
    c = cache_of(K, V, Hkv * G, n)
    ck = c.checkpoint(q, k, v)
    dout = torch.randn(q.shape, generator=torch.Generator(device="cuda").manual_seed(4), device="cuda").to(dtype)
    rest = c.checkpoint_restore(ck)
    got = c.checkpoint_backward(ck, dout)
    c.sync_check()
    assert not got[1][:, :, n:].any() and not got[2][:, :, n:].any()
    for b in range(B):
        for g in range(Hkv):
            def one(x):
                per = x.shape[1] // Hkv
                return x[b:b + 1, g * per:(g + 1) * per]
            want, bound = ref.backward(*map(one, rest), one(dout), n, dtype)
            for name, x, w, lim in zip(("dq", "dK", "dV", "dk", "dv"), got, want, bound):
                x = one(x)
                ref.within((name, b, g), x[:, :, :n] if name in ("dK", "dV") else x, w, lim)
    for a, b in zip(got, c.checkpoint_backward(ck, dout)):
        assert torch.equal(a, b)


def test_backwards_of_growing_chunks_keep_few_workspaces():
    """Chunks that grow by a little past the context's length: outgrown workspaces stay
    (a graph may hold them), all of them together no more than the one in use."""
    B, Hq, C, d, last = 1, 32, 16, 128, 1280
    c = H2OCache(B, Hq, 1, d, C, FP32, max_T=4)
    flat = [torch.zeros((B, h, last, d), device="cuda") for h in (Hq, 1, 1, Hq, Hq, 1, 1)]
    dK, dV = torch.zeros((B, 1, C, d), device="cuda"), torch.zeros((B, 1, C, d), device="cuda")
    record = torch.zeros(B * (Hq + 2) * last * (d + d // 8), dtype=torch.uint8, device="cuda")
    P = [x.data_ptr() for x in flat]
    torch.cuda.synchronize()
    free = torch.cuda.mem_get_info()[0]
    for T in range(320, last + 1, 16):
        c._check(_lib.lib().h2o_checkpoint_backward(c.handle, record.data_ptr(), record.numel(), T, 0, P[3], P[4],
                                                    dK.data_ptr(), dV.data_ptr(), P[5], P[6], None))
    c.sync_check()
    largest = 4 * B * (Hq + 2) * last * d + 16 * B * Hq * last + (32 << 20)  # the step, its statistics, parts and pages
    # grown to twice its size when outgrown: at most 2 + 1 + 1/2 + ... of the last one needed
    assert free - torch.cuda.mem_get_info()[0] <= 4 * largest


def test_other_threads_run_while_a_call_waits():
    """A context's first call waits for the work before it; Python's other threads do not."""
    import threading
    import time
    q, k, v, K, V = heads(BF16, 1, 2, 2, 64, 64, 64, 8)
    c, parent = cache_of(K, V, 4, 64), trees(1, 8)
    torch.cuda.synchronize()
    ticks, stop = [0], threading.Event()

    def tick():
        while not stop.is_set():
            ticks[0] += 1
            time.sleep(1e-3)

    t = threading.Thread(target=tick)
    t.start()
    try:
        torch.cuda._sleep(int(8e8))  # 0.4 s at 2 GHz
        before, start = ticks[0], time.monotonic()
        c.tree_attend(q, k, v, parent)
        passed, waited = ticks[0] - before, time.monotonic() - start
    finally:
        stop.set()
        t.join()
    assert waited > 0.1 and passed >= 10


def test_two_threads_call_at_once():
    """First calls of one context from two threads on one stream, its workspaces made and
    outgrown meanwhile: what each call computes alone."""
    import threading
    inputs = [heads(BF16, 1, 2, 2, 64, 64, 64, T, seed=T) for T in (8, 40, 100, 200)]
    K, V = inputs[0][3:]
    alone = cache_of(K, V, 4, 64, max_T=8)
    records = [alone.checkpoint(*x[:3]) for x in inputs]
    douts, parents = [torch.randn_like(x[0]) for x in inputs], [trees(1, x[0].shape[2]) for x in inputs]

    def run(c):
        return [(c.checkpoint_backward(r, g), c.tree_attend(*x[:3], p)) for r, g, x, p in zip(records, douts, inputs, parents)]

    want = run(alone)
    for _ in range(5):
        c, got = cache_of(K, V, 4, 64, max_T=8), [None, None]
        go = threading.Barrier(2)

        def work(i):
            go.wait()
            got[i] = run(c)

        threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        c.sync_check()
        for both in got:
            for mine, own in zip(both, want):
                for a, b in zip(mine[0] + mine[1], own[0] + own[1]):
                    assert torch.equal(a, b)


@pytest.mark.parametrize("dtype,B,Hkv,G,d,n,T", [(FP32, 2, 2, 2, 64, 70, 12), (BF16, 2, 2, 4, 128, 700, 3), (BF16, 2, 2, 4, 128, 700, 40),
                                                  (BF16, 2, 2, 2, 64, 130, 200), (BF16, 8, 8, 4, 128, 700, 3), (BF16, 14, 8, 4, 128, 300, 40),
                                                  (BF16, 16, 4, 1, 64, 33, 256), (BF16, 14, 8, 4, 128, 2065, 40),
                                                  (BF16, 1, 8, 4, 128, 8999, 3)])
def test_tree_values_that_are_not_finite_stay_in_their_columns(dtype, B, Hkv, G, d, n, T):
    """A NaN or an infinity in a drafted v is what the definition makes of it, whatever
    the size of the call: in its column of the rows that see the node, and nowhere else."""
    q, k, v, K, V = heads(dtype, B, Hkv, G, d, n, n, T, seed=5)
    parent = trees(B, T, seed=6)
    parent[:, :2] = torch.tensor([-1, 0])
    want, wlse, bound, lbound = ref.tree(q, k, v, parent, K, V, n, dtype)
    clean = cache_of(K, V, Hkv * G, n).tree_attend(q, k, v, parent)
    bad = torch.zeros(v.shape, device="cuda")
    bad[:, :, 0, 3], bad[:, :, 0, 17], bad[:, :, 0, d - 1] = math.nan, math.inf, -math.inf
    bad[:, :, 1, 17], bad[:, :, 1, 40], bad[:, :, T - 1, d // 2] = -math.inf, math.inf, math.inf
    bad[-1, -1, T // 2, 5] = -math.inf
    out, lse = cache_of(K, V, Hkv * G, n).tree_attend(q, k, v + bad.to(dtype), parent)
    see = ref.ancestors(parent).cuda()
    extra = torch.zeros((B, Hkv, T, d), device="cuda")
    for node in range(T):  # every weight is > 0: inf and NaN come through as they are
        extra += torch.where(see[:, None, :, node, None], bad[:, :, None, node], 0.0)
    extra = extra[:, :, None].expand(B, Hkv, G, T, d).reshape(out.shape)
    there = extra.isfinite()
    assert not there.all() and torch.equal(lse, clean[1])
    assert torch.equal(out[~there].float().nan_to_num(nan=7.0), extra[~there].nan_to_num(nan=7.0))
    # the finite columns: without the bad elements, whose own columns are not looked at
    ref.within("out", out[there], want[there], bound[there])


@pytest.mark.parametrize("B,T", [(1, 3), (2, 40), (14, 40), (16, 256)])
def test_tree_values_that_are_not_finite_meet_others(B, T):
    """Infinities of both signs in a slot and a node that share a column, and in rows
    whose scores are NaN, give NaN on either path."""
    q, k, v, K, V = heads(BF16, B, 4, 2, 64, 200, 200, T, seed=5)
    parent = torch.zeros((B, T), dtype=torch.int32, device="cuda")
    parent[:, 0] = -1
    V[:, :, 7, 20] = math.inf
    v[:, :, 0, 20], v[:, :, 0, 21], v[:, :, T - 1, 22] = -math.inf, math.inf, -math.inf
    k[:, 1, 0, 3] = math.nan               # one KV head's rows are NaN
    out, _ = cache_of(K, V, 8, 200).tree_attend(q, k, v, parent)
    assert out[:, 2:4].isnan().all()
    ok = out[:, [0, 1, 4, 5, 6, 7]]
    assert ok[..., 20].isnan().all() and (ok[..., 21] == math.inf).all()
    assert (ok[:, :, T - 1, 22] == -math.inf).all() and ok[:, :, :-1, 22].isfinite().all()
    rest = [c for c in range(64) if c not in (20, 21, 22)]
    assert ok[..., rest].isfinite().all()


@pytest.mark.parametrize("B,Hkv,G,d,C,n,T", [(1, 2, 4, 128, 512, 512, 256), (1, 8, 4, 128, 1024, 1024, 384),
                                             (1, 8, 4, 128, 2048, 2048, 1024), (4, 8, 3, 64, 1500, 1409, 333)])
def test_bf16_gradients_are_rounded_once_whatever_the_size(B, Hkv, G, d, C, n, T):
    """The error of each gradient in 2-norm is that of rounding the 64-bit one to bf16.
    What comes on top is far smaller: a bf16 pair of a weight keeps 2^-16 of it, the fp32
    logits are off by about 2^-20 (a part in 1e-5 of the weights), both added up like
    random steps, against 2^-8 / sqrt(12) to 2^-9 / sqrt(12) of the result; a tenth leaves
    room for terms ten times the result. One bf16 per weight gives 1.2 to 1.7."""
    q, k, v, K, V = heads(BF16, B, Hkv, G, d, C, n, T, seed=n + T)
    c = cache_of(K, V, Hkv * G, n)
    ck = c.checkpoint(q, k, v)
    dout = torch.randn(q.shape, generator=torch.Generator(device="cuda").manual_seed(4), device="cuda").to(BF16)
    rest, got = c.checkpoint_restore(ck), c.checkpoint_backward(ck, dout)
    off, rounding = torch.zeros(5, dtype=torch.float64), torch.zeros(5, dtype=torch.float64)
    for b in range(B):
        for g in range(Hkv):
            def one(x):
                per = x.shape[1] // Hkv
                return x[b:b + 1, g * per:(g + 1) * per]
            want, _ = ref.backward(*map(one, rest), one(dout), n, BF16)
            for i, (x, w) in enumerate(zip(got, want)):
                off[i] += (one(x)[:, :, :w.shape[2]].double() - w).square().sum().cpu()
                rounding[i] += (w.to(BF16).double() - w).square().sum().cpu()
    ratio = (off / rounding).sqrt()
    assert (ratio <= 1.1).all(), ratio
