"""Refusals of the operators next to the step, and the 64-bit backward the GPU
tests compare with against differences (no GPU needed)."""
import ctypes
import math

import pytest
import torch

import operators_ref as ref
from h2o_kv_cache_step_b200 import H2OCache, H2OCheckpoint, _lib


@pytest.fixture(scope="module")
def L():
    from h2o_kv_cache_step_b200 import build
    build.build()
    return _lib.lib()


def test_null_context_is_an_argument_error(L):
    assert L.h2o_tree_attend(None, None, None, None, None, None, None, 4, None) == _lib.H2O_ERR_ARG
    assert L.h2o_checkpoint_bytes(None, 4, 4, ctypes.byref(ctypes.c_size_t())) == _lib.H2O_ERR_ARG
    assert L.h2o_checkpoint_save(None, None, None, None, 4, None, 0, None) == _lib.H2O_ERR_ARG
    assert L.h2o_checkpoint_restore(None, None, 0, 4, 4, None, None, None, None, None, None) == _lib.H2O_ERR_ARG
    assert L.h2o_checkpoint_backward(None, None, 0, 4, 4, None, None, None, None, None, None, None) == _lib.H2O_ERR_ARG
    assert L.h2o_carry_grad(None, None, 4, 4, *[None] * 11) == _lib.H2O_ERR_ARG


def test_constants_match_the_header():
    import os
    import re
    src = open(os.path.join(os.path.dirname(_lib.PKG), "include", "h2o.h")).read()
    assert int(re.search(r"#define H2O_TREE_MAX_T (\d+)", src).group(1)) == _lib.H2O_TREE_MAX_T
    assert int(re.search(r"#define H2O_CKPT_GROUP (\d+)", src).group(1)) == _lib.H2O_CKPT_GROUP


def _closed(B=2, Hq=4, Hkv=2, d=64, C=32, dtype=torch.bfloat16):
    """A cache whose context is gone: its checks come before any call."""
    from h2o_kv_cache_step_b200 import build
    build.build()
    c = H2OCache.__new__(H2OCache)
    c.B, c.Hq, c.Hkv, c.d, c.C, c.dtype, c.device, c._h = B, Hq, Hkv, d, C, dtype, torch.device("cuda", 0), None
    c._ops = c._bind(0)
    return c


def _t(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def test_host_tensors_and_wrong_shapes_are_refused():
    c = _closed()
    tree = _t(2, 5, dtype=torch.int32)
    with pytest.raises(ValueError, match=r"q: need \[B, Hq, T, d\]"):
        c.tree_attend(_t(2, 4, 5), _t(2, 2, 5, 64), _t(2, 2, 5, 64), tree)
    with pytest.raises(ValueError, match="q: need a contiguous BFloat16 tensor of shape .2, 4, 5, 64. on cuda:0, got BFloat16 .* on cpu"):
        c.tree_attend(_t(2, 4, 5, 64), _t(2, 2, 5, 64), _t(2, 2, 5, 64), tree)
    with pytest.raises(TypeError, match="q: need a tensor"):
        c.checkpoint(None, _t(2, 2, 5, 64), _t(2, 2, 5, 64))
    with pytest.raises(ValueError, match=r"token_slots: need \[B, Hkv, T\]"):
        c.carry_grad(tree, 3, *[_t(2, 2, 5, 64)] * 4)
    with pytest.raises(ValueError, match="token_slots: need a contiguous Int"):
        c.carry_grad(_t(2, 2, 5, dtype=torch.int32), 3, *[_t(2, 2, 5, 64)] * 4)
    with pytest.raises(TypeError):
        c.carry_grad(_t(2, 2, 5, dtype=torch.int32), 3.5, *[_t(2, 2, 5, 64)] * 4)
    with pytest.raises(ValueError, match="n: out of range"):
        c.carry_grad(_t(2, 2, 5, dtype=torch.int32), 1 << 40, *[_t(2, 2, 5, 64)] * 4)


def test_a_record_of_another_size_or_place_is_refused():
    rows = 2 * (4 * 5 + 2 * 2 * 5 + 2 * 2 * 3)
    with pytest.raises(ValueError, match="buffer: need"):
        H2OCheckpoint(torch.zeros(rows * (64 + 8), dtype=torch.uint8), 2, 4, 2, 64, 5, 3)
    ck = H2OCheckpoint._of(torch.zeros(rows * 72, dtype=torch.uint8), 2, 4, 2, 64, 5, 3)
    with pytest.raises(ValueError, match="checkpoint: need a contiguous Byte"):
        _closed().checkpoint_restore(ck)
    with pytest.raises(ValueError, match="checkpoint: of"):
        _closed(Hkv=4).checkpoint_restore(ck)


def test_a_record_splits_into_its_sections():
    """codes() and scales() find the five sections where the layout puts them."""
    B, Hq, Hkv, d, T, n = 2, 4, 2, 64, 5, 3
    gen = torch.Generator().manual_seed(1)
    xs = [torch.randn(s, generator=gen) for s in ((B, Hq, T, d), (B, Hkv, T, d), (B, Hkv, T, d), (B, Hkv, n, d), (B, Hkv, n, d))]
    codes, scales, _ = zip(*[ref.quantise(x) for x in xs])
    ck = H2OCheckpoint.__new__(H2OCheckpoint)
    ck.buffer = torch.cat([c.reshape(-1).view(torch.uint8) for c in codes] + [s.reshape(-1).view(torch.uint8) for s in scales])
    ck.shape, ck.T, ck.n = (B, Hq, Hkv, d), T, n
    for a, b in zip(ck.codes(), codes):
        assert torch.equal(a, b)
    for a, b in zip(ck.scales(), scales):
        assert torch.equal(a, b)


def test_reference_backward_against_differences():
    """d/dx of sum(out * dout) by central differences, step 1e-5: off by about
    1e-10 (the third derivative times the step squared) and 1e-16 / 1e-5 of the
    sum's size, far below 1e-6."""
    B, Hkv, G, T, n, d = 1, 2, 2, 5, 4, 32
    gen = torch.Generator().manual_seed(3)
    xs = [torch.randn(s, generator=gen, dtype=torch.float64)
          for s in ((B, Hkv * G, T, d), (B, Hkv, T, d), (B, Hkv, T, d), (B, Hkv, n, d), (B, Hkv, n, d))]
    do = torch.randn((B, Hkv * G, T, d), generator=gen, dtype=torch.float64)

    def loss(q, k, v, K, V):
        s = torch.einsum("bghtd,bgjd->bghtj", q.view(B, Hkv, G, T, d), torch.cat([K, k], 2)) / math.sqrt(d)
        s = s.masked_fill(torch.arange(n + T) - n > torch.arange(T)[:, None], -math.inf)
        o = torch.einsum("bghtj,bgjd->bghtd", torch.softmax(s, -1), torch.cat([V, v], 2))
        return float((o.reshape(B, Hkv * G, T, d) * do).sum())

    dq, dK, dV, dk, dv = ref.backward(*xs, do, n, torch.float32)[0]
    for i, g in enumerate((dq, dk, dv, dK, dV)):
        for _ in range(12):
            at = tuple(int(torch.randint(x, (1,), generator=gen)) for x in g.shape)
            lo, hi = [x.clone() for x in xs], [x.clone() for x in xs]
            lo[i][at] -= 1e-5
            hi[i][at] += 1e-5
            assert abs((loss(*hi) - loss(*lo)) / 2e-5 - float(g[at])) < 1e-6


class _FakeLibrary:
    """Contexts without a device (and without an address: nothing to destroy)."""
    def h2o_create_ex(self, *args):
        return 0


def test_a_cache_needs_the_operators_module_only_for_the_operators(monkeypatch):
    """A library without the torch module beside it still makes caches and steps."""
    from h2o_kv_cache_step_b200 import cache

    def missing():
        raise ImportError("_torch_ops.so is missing")

    monkeypatch.setattr(cache, "lib", _FakeLibrary)
    monkeypatch.setattr(cache, "_ops_type", missing)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    c = H2OCache(2, 4, 2, 64, 32)
    x = _t(2, 4, 5, 64)
    with pytest.raises(ValueError, match="q: need contiguous CUDA"):
        c.step(x, x, x)
    with pytest.raises(ImportError, match="_torch_ops.so is missing"):
        c.tree_attend(x, x, x, x)


def test_a_module_of_another_torch_is_refused(L, monkeypatch):
    from h2o_kv_cache_step_b200 import cache
    cache._ops_type()
    monkeypatch.setattr(torch, "__version__", "1.0.0+cu1")
    with pytest.raises(ImportError, match="built with torch .* this is 1.0.0.*build it with"):
        cache._ops_type()


def test_the_operators_module_is_built_anew_for_another_torch(L, monkeypatch):
    import subprocess

    from h2o_kv_cache_step_b200 import build

    def compiler(cmd, **kw):
        raise RuntimeError("compiled")

    build.build_binding()
    monkeypatch.setattr(subprocess, "run", compiler)
    build.build_binding()  # up to date
    monkeypatch.setattr(torch, "__version__", "1.0.0+cu1")
    with pytest.raises(RuntimeError, match="compiled"):
        build.build_binding()
