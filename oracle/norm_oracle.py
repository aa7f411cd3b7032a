"""TEST INFRASTRUCTURE: the norms around a token mixer and their gradients in
plain numpy fp64. Each gradient function also returns the magnitudes of its
terms: where terms cancel, their roundings stay, so an error is measured
against the sum of their absolute values. A normalised value n = (x - mean) r
is off by the roundings of x and of the mean, |x| r + |mean| r, however near
to zero it comes; the same holds for x = skip x + scale z."""

import numpy as np


def _norm(x, center, eps, mag=None):
    """(normalised x, inverse deviation, magnitude of its terms); mag: x's own."""
    m = x.mean(-1, keepdims=True) if center else 0.0
    r = 1.0 / np.sqrt(((x - m) ** 2).mean(-1, keepdims=True) + eps)
    mag = np.abs(x) if mag is None else mag
    return (x - m) * r, r, (mag + (mag.mean(-1, keepdims=True) if center else 0.0)) * r


def _norm_grad(g, gm, n, nm, r, center):
    """(gradient, magnitude of its terms); gm, nm: magnitudes of g and n."""
    a, b = (g * n).mean(-1, keepdims=True), g.mean(-1, keepdims=True) if center else 0.0
    am, bm = (gm * nm).mean(-1, keepdims=True), gm.mean(-1, keepdims=True) if center else 0.0
    return r * (g - b - n * a), r * (gm + bm + nm * am)


def _swish(g):
    s = 1.0 / (1.0 + np.exp(-g))
    return g * s, s + g * s * (1 - s)


def head_norm(x, weight=None, gate=None, center=False, eps=1e-5):
    y = _norm(x, center, eps)[0]
    if weight is not None:
        y = y * weight
    return y * _swish(gate)[0] if gate is not None else y


def head_norm_grad(x, dout, weight=None, gate=None, center=False, eps=1e-5):
    """{name: (gradient, magnitude)} of x, weight, gate."""
    n, r, nm = _norm(x, center, eps)
    w = np.ones(x.shape[-1]) if weight is None else weight
    act, slope = (1.0, 0.0) if gate is None else _swish(gate)
    g = dout * act * w
    out = {"dx": _norm_grad(g, np.abs(g), n, nm, r, center)}
    if weight is not None:
        flat = lambda t: t.reshape(-1, x.shape[-1]).sum(0)  # noqa: E731
        out["dweight"] = flat(dout * act * n), flat(np.abs(dout * act) * nm)
    if gate is not None:
        out["dgate"] = dout * n * w * slope, np.abs(dout * w) * nm
    return out


def residual_norm(x, y, weight, post=None, scale=None, skip=1.0, center=False, eps=1e-5):
    z = y if post is None else _norm(y, center, eps)[0] * post
    h = skip * x + (z if scale is None else scale * z)
    return _norm(h, center, eps)[0] * weight, h


def residual_norm_grad(x, y, weight, dout, dres=None, post=None, scale=None, skip=1.0, center=False, eps=1e-5):
    """{name: (gradient, magnitude)} of x, y, weight, post, scale."""
    w = x.shape[-1]
    s = np.ones(w) if scale is None else scale
    ny, ry, ym = (y, None, np.abs(y)) if post is None else _norm(y, center, eps)
    z, zm = (ny, ym) if post is None else (ny * post, ym * np.abs(post))
    n, r, nm = _norm(skip * x + s * z, center, eps, np.abs(skip * x) + np.abs(s) * zm)
    dh, mag = _norm_grad(dout * weight, np.abs(dout * weight), n, nm, r, center)
    if dres is not None:
        dh, mag = dh + dres, mag + np.abs(dres)
    flat = lambda t: t.reshape(-1, w).sum(0)  # noqa: E731
    out = {"dx": (skip * dh, abs(skip) * mag), "dweight": (flat(dout * n), flat(np.abs(dout) * nm))}
    if scale is not None:
        out["dscale"] = flat(dh * z), flat(mag * zm)
    if post is None:
        out["dy"] = dh * s, mag * np.abs(s)
    else:
        out["dy"] = _norm_grad(dh * s * post, mag * np.abs(s * post), ny, ym, ry, center)
        out["dpost"] = flat(dh * s * ny), flat(mag * np.abs(s) * ym)
    return out
