"""TEST INFRASTRUCTURE: the gated linear recurrence, the short causal convolution
and the cache of parked states in plain numpy fp64, token by token, with the
gradients by the reversed recurrence. Written from the formulas alone;
nothing on the product path imports it.

x, decay, gate: [batch, tokens, width]; rate: [width] or None (then decay holds
log decays); states [batch, width] and [batch, taps - 1, width].
"""

import numpy as np


def sigmoid(x):
    return np.exp(-np.logaddexp(0.0, -x))


def _gates(x, decay, gate, rate, normalize):
    sd = None if rate is None else sigmoid(decay)
    la = decay if rate is None else -rate * sd
    si = np.ones_like(x) if gate is None else sigmoid(gate)
    m = np.sqrt(-np.expm1(2 * la)) if normalize else np.ones_like(x)
    return sd, la, si, m


def scan(x, decay, gate=None, rate=None, normalize=False, state=None):
    """(o, final state)."""
    _, la, si, m = _gates(x, decay, gate, rate, normalize)
    a, u = np.exp(la), m * si * x
    h = np.zeros((x.shape[0], x.shape[2])) if state is None else np.array(state, dtype=np.float64)
    o = np.zeros(x.shape)
    for t in range(x.shape[1]):
        # a factor of 0 forgets whatever was there
        h = np.where(a[:, t] == 0, u[:, t], np.where(a[:, t] == 0, 0.0, a[:, t] * h) + u[:, t])
        o[:, t] = h
    return o, h


def scan_grad(x, decay, dout, gate=None, rate=None, normalize=False, state=None, d_state=None):
    """(dx, ddecay, dgate, drate, dstate) of sum(dout o) + sum(d_state h), None
    where there is no such input (dstate always). Where a log decay is 0 the
    factor sqrt(1 - a^2) counts as having no gradient."""
    sd, la, si, m = _gates(x, decay, gate, rate, normalize)
    a = np.exp(la)
    o, _ = scan(x, decay, gate, rate, normalize, state)
    first = np.zeros_like(o[:, :1]) if state is None else state[:, None]
    before = np.concatenate([first, o[:, :-1]], 1)
    carry = np.zeros_like(first[:, 0]) if d_state is None else np.array(d_state, dtype=np.float64)
    g = np.zeros_like(o)
    for t in reversed(range(x.shape[1])):
        g[:, t] = dout[:, t] + carry
        carry = a[:, t] * g[:, t]
    dla = a * g * before
    if normalize:
        dla -= np.divide(a * a, m, out=np.zeros_like(a), where=m > 0) * g * si * x
    dx, dgate = g * m * si, g * m * x * si * (1 - si)
    if rate is None:
        return dx, dla, None if gate is None else dgate, None, carry
    return dx, -rate * sd * (1 - sd) * dla, None if gate is None else dgate, -(sd * dla).sum((0, 1)), carry


def conv(x, weight, bias=None, swish=False, state=None):
    """(o, final state); weight [width, taps]."""
    b, n, w = x.shape
    taps = weight.shape[1]
    line = np.concatenate([np.zeros((b, taps - 1, w)) if state is None else state, x], 1)
    z = sum(weight[:, j] * line[:, j:j + n] for j in range(taps))
    z = z if bias is None else z + bias
    return (z * sigmoid(z) if swish else z), line[:, n:]


def conv_grad(x, weight, dout, bias=None, swish=False, state=None, d_state=None):
    """(dx, dweight, dbias, dstate) of sum(dout o) + sum(d_state final state)."""
    b, n, w = x.shape
    taps = weight.shape[1]
    z, _ = conv(x, weight, bias, False, state)
    s = sigmoid(z)
    dz = dout * (s + z * s * (1 - s)) if swish else dout
    line = np.concatenate([np.zeros((b, taps - 1, w)) if state is None else state, x], 1)
    dline = np.zeros_like(line)
    if d_state is not None:
        dline[:, n:] += d_state
    dw = np.zeros(weight.shape)
    for j in range(taps):
        dline[:, j:j + n] += weight[:, j] * dz
        dw[:, j] = (dz * line[:, j:j + n]).sum((0, 1))
    return dline[:, taps - 1:], dw, None if bias is None else dz.sum((0, 1)), dline[:, :taps - 1]


def packed(f, lens, rows, others=(), held=()):
    """f on each sequence of packed rows [tokens, width] by itself: `others` are
    passed on as they are, `held` are states with a leading batch axis.
    Returns one list of results per sequence."""
    out, at = [], 0
    for i, n in enumerate(lens):
        part = [None if r is None else r[None, at:at + n] for r in rows]
        out.append(f(*part, *others, *(None if h is None else h[i:i + 1] for h in held)))
        at += n
    return out


def park(x, block=64):
    """(codes, scales) of states [n, values] (fp32 numbers), the scale in fp32."""
    n, values = x.shape
    blocks = -(-values // block)
    y = np.zeros((n, blocks * block))
    y[:, :values] = x
    y = y.reshape(n, blocks, block)
    top = np.abs(y).max(-1)
    scale = (np.where(np.isfinite(top), top, np.nan).astype(np.float32) * np.float32(1 / 127)).astype(np.float32)
    with np.errstate(invalid="ignore", divide="ignore"):
        q = np.where(scale[..., None] > 0, np.rint(y / scale[..., None].astype(np.float64)), 0.0)
    return np.clip(q, -127, 127).reshape(n, -1)[:, :values].astype(np.int8), scale


def resume(codes, scales, block=64):
    n, values = codes.shape
    spread = np.repeat(scales.astype(np.float32), block, axis=1)[:, :values]
    return codes.astype(np.float32) * spread
