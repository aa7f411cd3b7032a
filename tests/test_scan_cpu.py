"""The gated recurrence, the short convolution and the cache of parked states on
the host: the fp64 oracle against differences and other forms of itself, the C
ABI's refusals and sizes, the binding's checks (no kernel is launched)."""

import contextlib
import ctypes
import os

import numpy as np
import pytest
import torch

from oracle import scan_oracle as oracle
from retnet_retention_amd import binding

A = 1 << 32


def make(seed, b, n, w):
    rng = np.random.default_rng(seed)
    r = lambda *s: rng.standard_normal(s)  # noqa: E731
    return dict(x=r(b, n, w), decay=r(b, n, w), gate=r(b, n, w), rate=np.abs(r(w)), state=r(b, w), dout=r(b, n, w),
                d_state=r(b, w)), rng


def differences(f, args, grads, rng, tol=1e-6):
    for name, g in grads.items():
        a = args[name]
        for _ in range(6):
            at = tuple(rng.integers(0, m) for m in a.shape)
            old = a[at]
            a[at] = old + 1e-5
            up = f()
            a[at] = old - 1e-5
            down = f()
            a[at] = old
            assert abs((up - down) / 2e-5 - g[at]) < tol * max(1.0, abs(g[at])), (name, at)


@pytest.mark.parametrize("gates", [False, True])
@pytest.mark.parametrize("normalize", [False, True])
@pytest.mark.parametrize("more", [False, True])
def test_scan_gradients_against_differences(gates, normalize, more):
    y, rng = make(1, 2, 7, 3)
    if not gates:
        y["rate"], y["decay"] = None, -np.abs(y["decay"]) - 0.05
    if not more:
        y["gate"] = y["state"] = y["d_state"] = None

    def loss():
        o, s = oracle.scan(y["x"], y["decay"], y["gate"], y["rate"], normalize, y["state"])
        return (y["dout"] * o).sum() + (0 if y["d_state"] is None else (y["d_state"] * s).sum())

    g = oracle.scan_grad(y["x"], y["decay"], y["dout"], y["gate"], y["rate"], normalize, y["state"], y["d_state"])
    grads = dict(x=g[0], decay=g[1], gate=g[2], rate=g[3], state=g[4])
    differences(loss, y, {k: v for k, v in grads.items() if y[k] is not None}, rng)


def test_scan_forgets_and_carries():
    y, _ = make(2, 1, 9, 4)
    la = -np.abs(y["decay"])
    whole, end = oracle.scan(y["x"], la, state=y["state"])
    first, mid = oracle.scan(y["x"][:, :4], la[:, :4], state=y["state"])
    second, last = oracle.scan(y["x"][:, 4:], la[:, 4:], state=mid)
    np.testing.assert_allclose(np.concatenate([first, second], 1), whole, rtol=1e-12)
    np.testing.assert_allclose(last, end, rtol=1e-12)
    la[:, 0] = -np.inf
    o, _ = oracle.scan(y["x"], la, state=np.full((1, 4), np.nan))
    np.testing.assert_array_equal(o, oracle.scan(y["x"], la)[0])
    # constant factors: a convolution with their powers
    o, _ = oracle.scan(y["x"], np.full_like(la, np.log(0.5)))
    np.testing.assert_allclose(o[:, 3], sum(0.5 ** (3 - t) * y["x"][:, t] for t in range(4)), rtol=1e-12)


@pytest.mark.parametrize("taps", [2, 3, 4])
@pytest.mark.parametrize("swish", [False, True])
@pytest.mark.parametrize("n", [1, 2, 6])
def test_conv_gradients_against_differences(taps, swish, n):
    rng = np.random.default_rng(3)
    r = lambda *s: rng.standard_normal(s)  # noqa: E731
    y = dict(x=r(2, n, 3), weight=r(3, taps), bias=r(3), state=r(2, taps - 1, 3), dout=r(2, n, 3), ds=r(2, taps - 1, 3))

    def loss():
        o, s = oracle.conv(y["x"], y["weight"], y["bias"], swish, y["state"])
        return (y["dout"] * o).sum() + (y["ds"] * s).sum()

    g = oracle.conv_grad(y["x"], y["weight"], y["dout"], y["bias"], swish, y["state"], y["ds"])
    differences(loss, y, dict(zip(("x", "weight", "bias", "state"), g)), rng)


def test_conv_against_torch():
    rng = np.random.default_rng(4)
    x, w = rng.standard_normal((2, 9, 5)), rng.standard_normal((5, 4))
    t = torch.nn.functional.conv1d(torch.from_numpy(x).transpose(1, 2), torch.from_numpy(w)[:, None], padding=3, groups=5)
    np.testing.assert_allclose(oracle.conv(x, w)[0], t[..., :9].transpose(1, 2).numpy(), rtol=1e-10)


def test_park_keeps_a_state_to_half_a_step():
    x = np.random.default_rng(5).standard_normal((3, 200)).astype(np.float32)
    x[1, 64:128] = 0
    x[2, 5] = np.nan
    codes, scales = oracle.park(x)
    back = oracle.resume(codes, scales)
    assert np.isnan(back[2, :64]).all() and (back[1, 64:128] == 0).all()
    step = np.repeat(scales, 64, axis=1)[:, :200]
    ok = np.isfinite(step)
    assert (np.abs(back - x)[ok] <= (0.5 + 2.0 ** -16) * step[ok]).all()
    assert np.abs(codes[:2]).max() == 127


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(binding.LIB_PATH):
        pytest.skip("libretention.so not built (run __graft_entry__.build())")
    return binding.lib()


def _scan(**kw):
    args = dict(batch=2, seqlen=100, width=320, dtype=binding.RET_BF16, normalize=0, reserved=0, x_stride=0,
                decay_stride=0, gate_stride=0)
    args.update(kw)
    return binding.ScanDesc(**args)


def _conv(**kw):
    args = dict(batch=2, seqlen=100, width=320, taps=4, dtype=binding.RET_BF16, swish=1, x_stride=0)
    args.update(kw)
    return binding.ConvDesc(**args)


def _call(f, names, scalars=(), after=()):
    """A call of f with fake addresses by name (each its own), some replaced."""
    def call(d, **kw):
        p = {n: (i + 1) * A for i, n in enumerate(names)}
        tail = {**dict(after), **{k: kw.pop(k) for k in list(kw) if k in dict(after)}}
        mid = {**dict(scalars), **{k: kw.pop(k) for k in list(kw) if k in dict(scalars)}}
        unknown = set(kw) - set(names)
        assert not unknown, unknown
        p.update(kw)
        head = [p["cu"], mid["total"]] if "cu" in p else []
        body = [p[n] for n in names if n != "cu"]
        return f(ctypes.byref(d) if d is not None else None, *head, *body, *tail.values(), None)
    return call


def calls(L):
    big = 1 << 40
    sf = _call(L.retention_scan_fwd, ("cu", "x", "decay", "rate", "gate", "o", "si", "so", "kept", "ws"),
               [("total", 0)], [("wsb", big)])
    sb = _call(L.retention_scan_bwd, ("cu", "x", "decay", "rate", "gate", "dout", "si", "dso", "kept", "dx", "dd", "dr",
                                      "dg", "dsi", "ws"), [("total", 0)], [("wsb", big)])
    ss = _call(L.retention_scan_step, ("x", "decay", "rate", "gate", "o", "state", "slots"), [], [("n", 2)])
    cf = _call(L.retention_conv_fwd, ("cu", "x", "w", "b", "o", "si", "so", "ws"), [("total", 0)], [("wsb", big)])
    cb = _call(L.retention_conv_bwd, ("cu", "x", "w", "b", "dout", "si", "dso", "dx", "dw", "db", "dsi", "ws"),
               [("total", 0)], [("wsb", big)])
    cs = _call(L.retention_conv_step, ("x", "w", "b", "o", "state", "slots"), [], [("n", 2)])
    return sf, sb, ss, cf, cb, cs


@pytest.mark.parametrize("kw,status", [
    (dict(batch=0), 2), (dict(seqlen=0), 2), (dict(width=0), 2), (dict(width=65537), 2), (dict(dtype=3), 3),
    (dict(batch=2**31 - 1, seqlen=2**31 - 1), 2), (dict(x_stride=319), 2), (dict(x_stride=-1), 2),
    (dict(x_stride=2**40), 2), (dict(batch=2**20, seqlen=2047, width=65536), 2),
])
def test_descriptor_refusals(L, kw, status):
    sf, sb, ss, cf, cb, cs = calls(L)
    d, c = _scan(**kw), _conv(**kw)
    assert sf(d, cu=None) == sb(d, cu=None) == ss(d) == status
    assert cf(c, cu=None) == cb(c, cu=None) == cs(c) == status
    r = ctypes.byref
    assert L.retention_scan_workspace_bytes(r(d), 0, 0) == L.retention_scan_kept_bytes(r(d), 0, 0) == 0
    assert L.retention_scan_bwd_workspace_bytes(r(d), 0, 0, 0) == L.retention_conv_bwd_workspace_bytes(r(c), 0, 0) == 0


@pytest.mark.parametrize("kw", [dict(decay_stride=3), dict(gate_stride=319)])
def test_scan_stride_refusals(L, kw):
    sf, sb, ss, *_ = calls(L)
    assert sf(_scan(**kw), cu=None) == sb(_scan(**kw), cu=None) == ss(_scan(**kw)) == 2


@pytest.mark.parametrize("taps", [0, 1, 5, -3])
def test_taps_refusals(L, taps):
    *_, cf, cb, cs = calls(L)
    assert cf(_conv(taps=taps), cu=None) == cb(_conv(taps=taps), cu=None) == cs(_conv(taps=taps, seqlen=1)) == 3


def test_pointer_refusals(L):
    sf, sb, ss, cf, cb, cs = calls(L)
    d, c = _scan(), _conv()
    for k in ("x", "decay", "o"):
        assert sf(d, cu=None, **{k: None}) == 1, k
    for k in ("x", "decay", "dout", "dx", "dd", "dr", "dg", "dsi", "rate", "gate", "si"):
        assert sb(d, cu=None, **{k: None}) == 1, k
    for k in ("x", "w", "o"):
        assert cf(c, cu=None, **{k: None}) == 1, k
    for k in ("x", "w", "dout", "dx", "dw", "db", "dsi", "b", "si"):
        assert cb(c, cu=None, **{k: None}) == 1, k
    for f in (sf, sb, ss, cf, cb, cs):
        kw = {} if f in (ss, cs) else dict(cu=None)
        assert f(None, **kw) == 1
    assert sf(d, cu=None, x=A + 1) == 5 and sf(d, cu=None, o=6 * A + 8) == 5 and sf(d, cu=None, rate=None, decay=2 * A + 2) == 5 and sf(d, cu=A + 2) == 5 and cb(c, cu=None, w=2 * A + 4) == 5
    # written buffers overlap others; a state may be replaced in place exactly
    assert sf(d, cu=None, o=2 * A) == 8 and sf(d, cu=None, so=7 * A + 16, si=7 * A) == 8
    assert sf(d, cu=None, kept=2 * A) == 8 and sf(d, cu=None, ws=2 * A) == 8 and sb(d, cu=None, dx=2 * A) == 8
    assert sb(d, cu=None, dsi=7 * A) == 8 and sb(d, cu=None, kept=15 * A) == 8 and cf(c, cu=None, o=2 * A) == 8
    assert cb(c, cu=None, dsi=6 * A) == 8 and cb(c, cu=None, dx=2 * A) == 8
    for f, desc in ((sf, d), (sb, d), (cb, c)):
        assert f(desc, cu=None, ws=None) == 6 and f(desc, cu=None, wsb=7) == 6
    assert cf(c, total=10, wsb=7) == 6
    # rows that stand apart reach further
    wide = _scan(x_stride=100000)
    assert sf(wide, cu=None, x=A, o=A + 4 * 10**6) == 8


def test_packed_refusals(L):
    sf, sb, _, cf, cb, _ = calls(L)
    for total in (-1, 2**31 - 1, 2**62):
        assert sf(_scan(), total=total) == sb(_scan(), total=total) == 2
        assert cf(_conv(), total=total) == cb(_conv(), total=total) == 2


def test_step_refusals(L):
    _, _, ss, _, _, cs = calls(L)
    for f, mk, names in ((ss, _scan, ("x", "decay", "o", "state")), (cs, _conv, ("x", "w", "o", "state"))):
        assert f(mk()) == 2
        d = mk(seqlen=1)
        for k in names:
            assert f(d, **{k: None}) == 1, k
        assert f(d, n=0) == 2 and f(d, n=2**31) == 2 and f(d, n=3, slots=None) == 2
        assert f(d, state=A) == 8 and f(d, slots=A * 9 + 2) == 5 and f(mk(seqlen=1, batch=65536)) == 2


def test_sizes(L):
    r, up = ctypes.byref, lambda x: (x + 255) // 256 * 256
    d, c = _scan(), _conv()
    assert L.retention_scan_kept_bytes(r(d), 0, 0) % (320 * 4) == 0
    assert L.retention_scan_bwd_workspace_bytes(r(d), 0, 0, 0) >= L.retention_scan_bwd_workspace_bytes(
        r(d), 0, 0, 1) + L.retention_scan_kept_bytes(r(d), 0, 0)
    assert L.retention_conv_workspace_bytes(r(c), 0, 0) == 0 and L.retention_conv_workspace_bytes(r(c), 1, 5) == 256
    # a wide batch of packed tokens grows with the tokens, not with batch times a bound
    assert L.retention_scan_kept_bytes(r(_scan(batch=100)), 1, 1000) <= 110 * 320 * 4


def _cache(**kw):
    args = dict(batch=3, reserved=0, values=1000, num_slots=5, cache_slots=7)
    args.update(kw)
    return binding.StateCacheDesc(**args)


def test_cache_refusals(L):
    def both(d, state=A, codes=2 * A, scales=3 * A, at=4 * A, slots=5 * A):
        r = ctypes.byref(d) if d is not None else None
        w = L.retention_state_cache_write(r, state, codes, scales, at, slots, None)
        assert w == L.retention_state_cache_read(r, codes, scales, state, at, slots, None)
        return w

    for kw in (dict(batch=0), dict(batch=65536), dict(values=0), dict(values=2**34), dict(num_slots=0),
               dict(num_slots=2**31), dict(cache_slots=0), dict(cache_slots=2**40), dict(values=2**33, batch=65535)):
        assert both(_cache(**kw)) == 2, kw
    assert both(None) == 1
    for k in ("state", "codes", "scales", "at"):
        assert both(_cache(), **{k: None}) == 1, k
    assert both(_cache(), slots=None) == 2  # num_slots is not batch
    assert both(_cache(), state=A + 4) == 5 and both(_cache(), codes=2 * A + 8) == 5 and both(_cache(), at=4 * A + 1) == 5
    assert both(_cache(), codes=A) == 8 and both(_cache(), scales=A + 16) == 8


def test_the_bindings_token_strides():
    s = binding._token_stride
    x = torch.zeros(3, 5, 24)
    assert s("x", x) == 24 and s("x", x[..., 8:16]) == 24 and s("x", x[:, 1:2, :8]) == 120 and s("x", x[:1, :, :8]) == 24
    assert s("x", x[0, :, :8]) == 24 and s("x", x[:1, :1, 3:4]) == 1
    for bad in (x[:, :4, :8], x[:, ::2], x.transpose(1, 2), x[..., ::2], x[:, :1, :8].expand(3, 5, 8)):
        with pytest.raises(ValueError):
            s("x", bad)


def test_tensors_on_the_host_are_refused():
    x = torch.zeros(2, 3, 8)
    with pytest.raises(ValueError):
        binding.gated_scan_fwd(x, x)
    with pytest.raises(ValueError):
        binding.short_conv_fwd(x, torch.zeros(8, 4))
    with pytest.raises(ValueError):
        binding.state_cache_write(torch.zeros(2, 64), torch.zeros(2, 64, dtype=torch.int8), torch.zeros(2, 1),
                                  torch.zeros(2, dtype=torch.int32))


@pytest.mark.parametrize("default", [torch.bfloat16, torch.float16, torch.float64, torch.float32])
def test_kept_states_are_fp32_whatever_the_default_type(monkeypatch, default):
    """The library takes no size for them: the buffer has the bytes that it asked for."""
    need, seen = 4 * 640, {}

    class Library:
        def retention_scan_kept_bytes(self, *_):
            return need

        def retention_scan_workspace_bytes(self, *_):
            return 256

        def retention_scan_fwd(self, *args):
            seen["kept"] = args[10]
            return 0

    monkeypatch.setattr(binding, "lib", Library)
    monkeypatch.setattr(binding, "_scan_call", lambda x, *_: (None, x.shape[0], 0, x.shape[2]))
    monkeypatch.setattr(binding, "_current", lambda t: contextlib.nullcontext())
    monkeypatch.setattr(binding, "_stream", lambda t: None)
    x = torch.zeros(2, 300, 64, dtype=torch.float32)
    before = torch.get_default_dtype()
    torch.set_default_dtype(default)
    try:
        _, kept = binding.gated_scan_fwd(x, x, keep=True)
    finally:
        torch.set_default_dtype(before)
    assert kept.data_ptr() == seen["kept"] and kept.dtype == torch.float32 and kept.numel() * kept.element_size() == need
