"""The gated delta rule on the host: the fp64 oracle against closed forms and
finite differences, and the C ABI's refusals (every call here fails validation,
so no kernel is launched)."""

import ctypes
import os

import numpy as np
import pytest

from oracle import delta_oracle as oracle
from retnet_retention_amd import binding

A = 1 << 32  # fake aligned pointers, never dereferenced


def _inputs(seed, b=2, n=9, hk=1, h=2, d=4):
    rng = np.random.default_rng(seed)
    q, k = rng.standard_normal((2, b, n, hk, d)) / np.sqrt(d)
    v = rng.standard_normal((b, n, h, d))
    return q, k, v, -rng.random((b, n, h)), rng.random((b, n, h)), rng.standard_normal((b, h, d, d)) * 0.3


def test_zero_strength_only_decays():
    q, k, v, g, beta, s0 = _inputs(1)
    o, s = oracle.delta(q, k, v, g, 0 * beta, state=s0)
    a = np.exp(g.cumsum(1))
    np.testing.assert_allclose(s, a[:, -1][..., None, None] * s0, rtol=1e-13)
    np.testing.assert_allclose(o[:, 3], a[:, 3][..., None] * np.einsum("bk,bhkv->bhv", q[:, 3, 0], s0), rtol=1e-12)


def test_full_strength_writes_the_value_along_a_unit_key():
    """beta 1 and |k| = 1: reading along k gives v, whatever the state held."""
    q, k, v, g, beta, s0 = _inputs(2, hk=2)
    k = k / np.linalg.norm(k, axis=-1, keepdims=True)
    o, _ = oracle.delta(k, k, v, g, np.ones_like(beta), state=s0)
    np.testing.assert_allclose(o, v, atol=1e-12)


def test_orthogonal_keys_reduce_to_retention():
    """With keys that never meet, the rule is linear attention with decay."""
    b, n, h, d = 1, 4, 1, 4
    rng = np.random.default_rng(3)
    q, v = rng.standard_normal((2, b, n, h, d))
    k = np.eye(n)[None, :, None, :]
    g = np.full((b, n, h), np.log(0.75))
    o, _ = oracle.delta(q, k, v, g, np.ones((b, n, h)), scale=0.5)
    dist = np.arange(n)[:, None] - np.arange(n)[None]
    w = np.where(dist >= 0, 0.75 ** np.maximum(dist, 0), 0.0) * q[0, :, 0]
    np.testing.assert_allclose(o[0, :, 0], 0.5 * w @ v[0, :, 0], atol=1e-13)


def test_split_sequence_equals_one_run():
    x = _inputs(4, n=11)
    seq, s0 = x[:5], x[5]
    o, s = oracle.delta(*seq, scale=0.7, state=s0)
    o1, mid = oracle.delta(*(t[:, :5] for t in seq), scale=0.7, state=s0)
    o2, end = oracle.delta(*(t[:, 5:] for t in seq), scale=0.7, state=mid)
    np.testing.assert_allclose(np.concatenate([o1, o2], 1), o, atol=1e-13)
    np.testing.assert_allclose(end, s, atol=1e-13)


def test_gradients_against_differences():
    x = _inputs(5, n=6, hk=1, h=2, d=3)
    rng = np.random.default_rng(6)
    dout, dst = rng.standard_normal(x[2].shape), rng.standard_normal(x[5].shape)
    got = oracle.delta_grad(*x[:5], dout, scale=0.9, state=x[5], d_state=dst)

    def loss(args):
        o, s = oracle.delta(*args[:5], scale=0.9, state=args[5])
        return (dout * o).sum() + (dst * s).sum()

    for i, g in enumerate(got):
        for _ in range(12):
            at = tuple(rng.integers(0, m) for m in x[i].shape)
            up, down = [t.copy() for t in x], [t.copy() for t in x]
            up[i][at] += 1e-5
            down[i][at] -= 1e-5
            # central difference: error ~ 1e-10 of the third derivative, rounding ~ 1e-11
            assert abs((loss(up) - loss(down)) / 2e-5 - g[at]) < 1e-7, (i, at)


# --- the C ABI's refusals ---------------------------------------------------
@pytest.fixture(scope="module")
def L():
    if not os.path.exists(binding.LIB_PATH):
        pytest.skip("libretention.so not built (run __graft_entry__.build())")
    return binding.lib()


def _desc(**kw):
    args = dict(batch=2, seqlen=100, k_heads=2, v_heads=4, dk=128, dv=128, dtype=binding.RET_BF16, scale=1.0)
    args.update(kw)
    return binding.DeltaDesc(**args)


def _fwd(L, d, cu=None, total=0, q=A, k=2 * A, v=3 * A, g=4 * A, beta=5 * A, o=6 * A, si=None, so=None, ws=7 * A,
         wsb=1 << 40):
    return L.retention_delta_fwd(ctypes.byref(d), cu, total, q, k, v, g, beta, o, si, so, ws, wsb, None)


def _bwd(L, d, cu=None, total=0, si=None, dso=None, dsi=None, wsb=1 << 40, **kw):
    names = ("q", "k", "v", "g", "beta", "dout")
    outs = ("dq", "dk", "dv", "dg", "dbeta")
    p = {n: (i + 1) * A for i, n in enumerate(names + outs)}
    p.update(kw)
    return L.retention_delta_bwd(ctypes.byref(d), cu, total, *(p[n] for n in names), si, dso, *(p[n] for n in outs),
                                 dsi, p.get("ws", 20 * A), wsb, None)


def _step(L, d, q=A, k=2 * A, v=3 * A, g=4 * A, beta=5 * A, o=6 * A, state=7 * A, slots=None, n=2):
    return L.retention_delta_step(ctypes.byref(d), q, k, v, g, beta, o, state, slots, n, None)


@pytest.mark.parametrize("kw,status", [
    (dict(batch=0), 2), (dict(seqlen=0), 2), (dict(k_heads=0), 2), (dict(v_heads=0), 2), (dict(v_heads=129), 2),
    (dict(k_heads=3), 2), (dict(k_heads=8), 2), (dict(batch=-1), 2), (dict(seqlen=-5), 2),
    (dict(batch=2**31 - 1, seqlen=2**31 - 1), 2), (dict(batch=2**31 - 1, seqlen=1), 2),
    (dict(dk=32, dv=32), 3), (dict(dk=128, dv=64), 3), (dict(dk=512, dv=512), 3), (dict(dtype=2), 3),
    (dict(scale=float("nan")), 9), (dict(scale=float("inf")), 9),
])
def test_descriptor_refusals(L, kw, status):
    d = _desc(**kw)
    assert _fwd(L, d) == status
    assert _bwd(L, d) == status
    assert L.retention_delta_workspace_bytes(ctypes.byref(d), 0, 0) == 0
    assert L.retention_delta_bwd_workspace_bytes(ctypes.byref(d), 0, 0) == 0
    one = _desc(**dict(kw, seqlen=kw.get("seqlen", 1)))
    assert _step(L, one) == status


def test_forward_refusals(L):
    d = _desc()
    assert L.retention_delta_fwd(None, None, 0, *([A] * 9), 1 << 40, None) == 1
    for name in ("q", "k", "v", "g", "beta", "o"):
        assert _fwd(L, d, **{name: None}) == 1, name
    for name in ("q", "k", "v", "o", "si", "so", "ws"):
        assert _fwd(L, d, **{name: 9 * A + 8}) == 5, name
    assert _fwd(L, d, g=9 * A + 2) == 5 and _fwd(L, d, cu=9 * A + 2) == 5
    assert _fwd(L, d, o=A + 256) == 8 and _fwd(L, d, o=4 * A) == 8
    assert _fwd(L, d, so=A) == 8 and _fwd(L, d, si=9 * A, so=9 * A + 256) == 8
    assert _fwd(L, d, ws=A) == 8 and _fwd(L, d, ws=6 * A) == 8
    need = L.retention_delta_workspace_bytes(ctypes.byref(d), 0, 0)
    assert need > 0
    assert _fwd(L, d, wsb=need - 1) == 6 and _fwd(L, d, ws=None) == 6
    # packed: between 0 and batch * seqlen rows
    assert _fwd(L, d, cu=9 * A, total=-1) == 2 and _fwd(L, d, cu=9 * A, total=201) == 2
    assert _fwd(L, d, cu=9 * A, total=200, ws=9 * A) == 8


def test_backward_refusals(L):
    d = _desc()
    for name in ("q", "k", "v", "g", "beta", "dout", "dq", "dk", "dv", "dg", "dbeta"):
        assert _bwd(L, d, **{name: None}) == 1, name
        assert _bwd(L, d, **{name: 30 * A + 2}) == 5, name
    assert _bwd(L, d, si=30 * A) == 1 and _bwd(L, d, dsi=30 * A) == 1
    assert _bwd(L, d, si=30 * A, dsi=30 * A) == 8
    assert _bwd(L, d, dq=A) == 8 and _bwd(L, d, dk=7 * A) == 8 and _bwd(L, d, dbeta=10 * A) == 8
    need = L.retention_delta_bwd_workspace_bytes(ctypes.byref(d), 0, 0)
    assert need > L.retention_delta_workspace_bytes(ctypes.byref(d), 0, 0)
    assert _bwd(L, d, wsb=need - 1) == 6 and _bwd(L, d, ws=None) == 6 and _bwd(L, d, ws=A) == 8


def test_step_refusals(L):
    d = _desc(seqlen=1)
    assert _step(L, _desc(seqlen=2)) == 2
    for name in ("q", "k", "v", "g", "beta", "o", "state"):
        assert _step(L, d, **{name: None}) == 1, name
    assert _step(L, d, state=7 * A + 4) == 5 and _step(L, d, slots=9 * A + 2, n=5) == 5
    assert _step(L, d, state=A) == 8 and _step(L, d, o=7 * A) == 8 and _step(L, d, slots=7 * A, n=5) == 8
    # without slots the pool is the batch; a pool has at least one state
    assert _step(L, d, n=3) == 2 and _step(L, d, slots=9 * A, n=0) == 2 and _step(L, d, slots=9 * A, n=2**31) == 2


def test_packed_workspace_follows_the_tokens(L):
    """Blocks are numbered (row / 64) + sequence, so a ragged batch needs no
    more than its tokens' blocks and one for each sequence."""
    d = _desc(batch=7, seqlen=1000)
    per = L.retention_delta_workspace_bytes(ctypes.byref(_desc(batch=1, seqlen=64)), 0, 0) - 256
    assert L.retention_delta_workspace_bytes(ctypes.byref(d), 1, 640) == 256 + (640 // 64 + 7) * per


def test_block_numbers_of_packed_sequences_never_meet():
    """The numbering of the kernels, over random lengths: block i of sequence
    b is cu[b] // 64 + b + i, below total // 64 + batch; groups of four blocks
    likewise."""
    rng = np.random.default_rng(8)
    for _ in range(300):
        lens = rng.integers(0, 300, rng.integers(1, 9)) * rng.integers(0, 2)
        cu = np.concatenate([[0], np.cumsum(lens)])
        blocks, groups = [], []
        for b, n in enumerate(lens):
            base, nblk = cu[b] // 64 + b, -(-n // 64)
            blocks += [base + i for i in range(nblk)]
            groups += [base // 4 + b + g for g in range(-(-nblk // 4))]
        assert len(set(blocks)) == len(blocks) and len(set(groups)) == len(groups)
        total = cu[-1] // 64 + len(lens)
        assert all(0 <= i < total for i in blocks) and all(0 <= g < total // 4 + len(lens) + 1 for g in groups)


@pytest.mark.parametrize("kw", [dict(batch=2**18, seqlen=1, k_heads=1, v_heads=4),
                                dict(batch=2**20, seqlen=512, k_heads=1, v_heads=1)])
def test_more_threads_than_a_launch_counts(L, kw):
    d = _desc(**kw)
    assert _fwd(L, d) == 2 and _bwd(L, d) == 2
    assert L.retention_delta_workspace_bytes(ctypes.byref(d), 0, 0) == 0
    kw["batch"] -= 1 + kw["batch"] // 2**10
    assert L.retention_delta_workspace_bytes(ctypes.byref(_desc(**kw)), 0, 0) > 0
