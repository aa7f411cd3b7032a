"""TEST INFRASTRUCTURE: the gated delta rule in plain numpy fp64, token by token,
and its gradients by the reversed recurrence. Written from the recurrence
alone; nothing on the product path imports it.

    S' = a_t S_{t-1},  u_t = beta_t (v_t - S'^T k_t),  S_t = S' + k_t u_t^T,
    o_t = scale S_t^T q_t,  a_t = exp(log_decay_t).

q, k: [batch, tokens, k_heads, d]; v: [batch, tokens, heads, d]; log_decay,
beta: [batch, tokens, heads]; states [batch, heads, d, d]. Value head h uses key
head h // (heads / k_heads).
"""

import numpy as np


def _spread(x, heads):
    return np.repeat(x, heads // x.shape[2], axis=2)


def _write(s, k, v, a, beta):
    dec = a[..., None, None] * s
    res = v - np.einsum("bhk,bhkv->bhv", k, dec)
    return dec, res, dec + k[..., :, None] * (beta[..., None] * res)[..., None, :]


def delta(q, k, v, log_decay, beta, scale=1.0, state=None):
    """(o, final state)."""
    b, n, h, d = v.shape
    q, k, a = _spread(q, h), _spread(k, h), np.exp(log_decay)
    s = np.zeros((b, h, d, d)) if state is None else np.array(state, dtype=np.float64)
    o = np.zeros_like(v, dtype=np.float64)
    for t in range(n):
        s = _write(s, k[:, t], v[:, t], a[:, t], beta[:, t])[2]
        o[:, t] = scale * np.einsum("bhk,bhkv->bhv", q[:, t], s)
    return o, s


def delta_grad(q, k, v, log_decay, beta, dout, scale=1.0, state=None, d_state=None):
    """(dq, dk, dv, dlog_decay, dbeta, dstate) of sum(dout o) + sum(d_state S)."""
    b, n, h, d = v.shape
    hk = q.shape[2]
    q, k, a = _spread(q, h), _spread(k, h), np.exp(log_decay)
    s = np.zeros((b, h, d, d)) if state is None else np.array(state, dtype=np.float64)
    kept = []
    for t in range(n):
        kept.append(_write(s, k[:, t], v[:, t], a[:, t], beta[:, t]))
        s = kept[-1][2]
    ds = np.zeros_like(s) if d_state is None else np.array(d_state, dtype=np.float64)
    dq, dk, dv = np.zeros_like(v), np.zeros_like(v), np.zeros_like(v)
    dg, db = np.zeros_like(beta), np.zeros_like(beta)
    for t in reversed(range(n)):
        dec, res, new = kept[t]
        ds = ds + q[:, t][..., :, None] * (scale * dout[:, t])[..., None, :]
        dq[:, t] = scale * np.einsum("bhkv,bhv->bhk", new, dout[:, t])
        u = beta[:, t][..., None] * res
        du = np.einsum("bhk,bhkv->bhv", k[:, t], ds)
        db[:, t] = (du * res).sum(-1)
        dv[:, t] = beta[:, t][..., None] * du
        dk[:, t] = np.einsum("bhkv,bhv->bhk", ds, u) - np.einsum("bhkv,bhv->bhk", dec, dv[:, t])
        ds = ds - k[:, t][..., :, None] * dv[:, t][..., None, :]
        dg[:, t] = (ds * dec).sum((-1, -2))
        ds = a[:, t][..., None, None] * ds
    shared = lambda x: x.reshape(b, n, hk, h // hk, d).sum(3)  # noqa: E731
    return shared(dq), shared(dk), dv, dg, db, ds


def packed(fn, lens, tensors, state=None, d_state=None, **kw):
    """fn (delta or delta_grad) over packed [tokens, ...] tensors, sequence by
    sequence; returns (token outputs packed, stacked states)."""
    outs, states, at = [], [], 0
    for i, n in enumerate(lens):
        sl = [x[at:at + n][None] for x in tensors]
        more = {"state": None if state is None else state[i:i + 1]}
        if fn is delta_grad:
            more["d_state"] = None if d_state is None else d_state[i:i + 1]
        *o, s = fn(*sl, **more, **kw)
        outs.append([x[0] for x in o])
        states.append(s[0])
        at += n
    return [np.concatenate(x) for x in zip(*outs)], np.stack(states)
