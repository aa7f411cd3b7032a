"""The norms on the host: the fp64 oracle against torch's own and finite
differences, and the C ABI's refusals (no kernel is launched)."""

import ctypes
import os

import numpy as np
import pytest
import torch

from oracle import group_norm_swish
from oracle import norm_oracle as oracle
from retnet_retention_amd import binding

A = 1 << 32


def test_head_norm_is_the_retention_epilogue():
    rng = np.random.default_rng(1)
    x, g = rng.standard_normal((2, 3, 5, 2, 8))
    np.testing.assert_allclose(oracle.head_norm(x, None, g, center=True, eps=1e-5), group_norm_swish(x, g, 1e-5),
                               rtol=1e-12)


def test_head_norm_makes_unit_keys():
    x = np.random.default_rng(2).standard_normal((7, 64))
    y = oracle.head_norm(x, np.full(64, 64 ** -0.5), eps=1e-12)
    np.testing.assert_allclose(np.linalg.norm(y, axis=-1), 1.0, rtol=1e-9)


def test_norms_against_torch():
    rng = np.random.default_rng(3)
    x, y = rng.standard_normal((2, 6, 24))
    w = rng.standard_normal(24)
    t = torch.from_numpy
    np.testing.assert_allclose(oracle.residual_norm(x, y, w, skip=1.0)[0],
                               torch.nn.functional.rms_norm(t(x + y), (24,), t(w), 1e-5).numpy(), rtol=1e-12)
    np.testing.assert_allclose(oracle.residual_norm(x, y, w, center=True)[0],
                               torch.nn.functional.layer_norm(t(x + y), (24,), t(w), None, 1e-5).numpy(), rtol=1e-10)


@pytest.mark.parametrize("center", [False, True])
@pytest.mark.parametrize("more", [False, True])
def test_gradients_against_differences(center, more):
    rng = np.random.default_rng(4)
    x, y, gate, dout, dres = rng.standard_normal((5, 3, 10))
    w, post, scale = rng.standard_normal((3, 10))
    if not more:
        post = scale = None

    def check(f, args, grads):
        for name, a in args.items():
            if a is None:
                continue
            for _ in range(8):
                at = tuple(rng.integers(0, m) for m in a.shape)
                old = a[at]
                a[at] = old + 1e-5
                up = f()
                a[at] = old - 1e-5
                down = f()
                a[at] = old
                assert abs((up - down) / 2e-5 - grads["d" + name][0][at]) < 1e-7, name

    r = lambda: oracle.residual_norm(x, y, w, post, scale, 0.8, center)  # noqa: E731
    check(lambda: (dout * r()[0]).sum() + (dres * r()[1]).sum(), dict(x=x, y=y, weight=w, post=post, scale=scale),
          oracle.residual_norm_grad(x, y, w, dout, dres, post, scale, 0.8, center))
    hw, hg = (w, gate) if more else (None, None)
    check(lambda: (dout * oracle.head_norm(x, hw, hg, center)).sum(), dict(x=x, weight=hw, gate=hg),
          oracle.head_norm_grad(x, dout, hw, hg, center))


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(binding.LIB_PATH):
        pytest.skip("libretention.so not built (run __graft_entry__.build())")
    return binding.lib()


def _desc(**kw):
    args = dict(rows=10, width=64, dtype=binding.RET_BF16, center=0, eps=1e-5)
    args.update(kw)
    return binding.NormDesc(**args)


def _hf(L, d, x=A, w=2 * A, g=3 * A, o=4 * A):
    return L.retention_head_norm_fwd(ctypes.byref(d), x, w, g, o, None)


def _hb(L, d, wsb=1 << 30, **kw):
    p = dict(x=A, w=2 * A, g=3 * A, do=4 * A, dx=5 * A, dw=6 * A, dg=7 * A, ws=8 * A)
    p.update(kw)
    return L.retention_head_norm_bwd(ctypes.byref(d), *(p[k] for k in ("x", "w", "g", "do", "dx", "dw", "dg", "ws")), wsb,
                                     None)


def _rf(L, d, skip=1.0, **kw):
    p = dict(x=A, y=2 * A, w=3 * A, post=4 * A, scale=5 * A, out=6 * A, res=7 * A)
    p.update(kw)
    return L.retention_residual_norm_fwd(ctypes.byref(d), skip,
                                         *(p[k] for k in ("x", "y", "w", "post", "scale", "out", "res")), None)


def _rb(L, d, skip=1.0, wsb=1 << 30, **kw):
    names = ("x", "y", "w", "post", "scale", "do", "dr", "dx", "dy", "dw", "dpost", "dscale", "ws")
    p = {n: (i + 1) * A for i, n in enumerate(names)}
    p.update(kw)
    return L.retention_residual_norm_bwd(ctypes.byref(d), skip, *(p[n] for n in names), wsb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), 2), (dict(rows=2**31), 2), (dict(width=0), 2), (dict(width=16385), 2), (dict(dtype=5), 3),
    (dict(eps=0.0), 9), (dict(eps=float("nan")), 9), (dict(eps=float("inf")), 9),
])
def test_descriptor_refusals(L, kw, status):
    d = _desc(**kw)
    assert _hf(L, d) == _hb(L, d) == _rf(L, d) == _rb(L, d) == status
    assert L.retention_head_norm_bwd_workspace_bytes(ctypes.byref(d)) == 0
    assert L.retention_residual_norm_bwd_workspace_bytes(ctypes.byref(d)) == 0


def test_pointer_refusals(L):
    d = _desc()
    assert _hf(L, d, x=None) == 1 and _hf(L, d, o=None) == 1
    assert _hf(L, d, w=2 * A + 4) == 5 and _hf(L, d, o=A) == 8 and _hf(L, d, o=2 * A) == 8
    for k in ("x", "do", "dx", "dw", "dg"):
        assert _hb(L, d, **{k: None}) == 1, k
    assert _hb(L, d, w=None) == 1 and _hb(L, d, g=None) == 1
    assert _hb(L, d, dx=A) == 8 and _hb(L, d, dw=7 * A) == 8 and _hb(L, d, ws=A) == 8 and _hb(L, d, dg=8 * A + 4) == 5
    need = L.retention_head_norm_bwd_workspace_bytes(ctypes.byref(d))
    assert need > 0 and _hb(L, d, wsb=need - 1) == 6 and _hb(L, d, ws=None) == 6
    for k in ("x", "y", "w", "out", "res"):
        assert _rf(L, d, **{k: None}) == 1, k
    assert _rf(L, d, res=2 * A) == 8 and _rf(L, d, res=A + 64) == 8 and _rf(L, d, out=A) == 8
    assert _rf(L, d, skip=float("nan")) == 9 and _rb(L, d, skip=float("inf")) == 9
    for k in ("x", "y", "w", "do", "dx", "dy", "dw", "dpost", "dscale"):
        assert _rb(L, d, **{k: None}) == 1, k
    assert _rb(L, d, post=None) == 1 and _rb(L, d, scale=None) == 1
    assert _rb(L, d, dx=2 * A) == 8 and _rb(L, d, dy=8 * A) == 8 and _rb(L, d, ws=10 * A) == 8
    need = L.retention_residual_norm_bwd_workspace_bytes(ctypes.byref(d))
    assert _rb(L, d, wsb=need - 1) == 6 and _rb(L, d, ws=None) == 6
