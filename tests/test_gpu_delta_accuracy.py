"""How near the gated delta rule's results come to the fp64 oracle's.

Rounded results (o, dq, dk, dv of bf16 tensors) are compared with the oracle's
value rounded once. Before its rounding a value is off by d, at most 8 2^-16 of
a head's norm (six operands that are sums of two bf16 values, each off by 2^-16
or less, and the product of two rests). Two roundings differ only where a border
lies between the values, with a chance of d / ulp, and then by one ulp, which is at
most 2^-7 of the value: the squared difference is d ulp at the mean, so the
norm of all differences is at most sqrt(8 2^-16 2^-7) = 2^-10 of the result's. A
further operand of one bf16 value would add up to 2^-8."""

import numpy as np
import pytest
import torch

import retnet_retention_amd as rr
from oracle import delta_oracle as oracle
from test_gpu_delta import DEV, dev, f64, make

pytestmark = pytest.mark.gpu
ROUNDED_ONCE = 2.0 ** -10
KEYS = ("q", "k", "v", "g", "beta")


def rounded(x):
    return torch.from_numpy(np.ascontiguousarray(x)).bfloat16().double().numpy()


def near_rounded(got, ref, what, axis=-2):
    """Per head: the norm of the difference to the oracle's rounded value."""
    got, ref = (np.moveaxis(x, axis, 0).reshape(x.shape[axis], -1) for x in (f64(got), rounded(ref)))
    err = np.linalg.norm(got - ref, axis=1) / np.linalg.norm(ref, axis=1)
    print(f"  {what}: {err.max():.2e} (bar {ROUNDED_ONCE:.2e})", flush=True)
    assert (err <= ROUNDED_ONCE).all(), f"{what}: {err}"


@pytest.mark.parametrize("b,n,hk,h,d", [(2, 257, 2, 2, 64), (1, 300, 2, 4, 128), (2, 200, 1, 2, 256)])
def test_output_is_at_its_own_rounding(b, n, hk, h, d):
    x = make(31, b, n, hk, h, d, "bf16")
    y = dev(x)
    o = rr.delta_chunkwise_fwd(*(y[k] for k in KEYS), scale=d ** -0.5, state_in=y["s0"])
    ref, _ = oracle.delta(*(f64(x[k]) for k in KEYS), scale=d ** -0.5, state=f64(x["s0"]))
    near_rounded(o, ref, "o")


def test_packed_output_is_at_its_own_rounding():
    lens = [130, 0, 1, 66]
    x = make(32, len(lens), max(lens), 2, 4, 128, "bf16", lens=lens)
    y = dev(x)
    cu = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32, device=DEV)
    o = rr.delta_chunkwise_fwd(*(y[k] for k in KEYS), state_in=y["s0"], cu_seqlens=cu, max_seqlen=max(lens), check=True)
    (ref,), _ = oracle.packed(oracle.delta, lens, [f64(x[k]) for k in KEYS], state=f64(x["s0"]))
    near_rounded(o, ref, "o")


# fp32 results of bf16 tensors. An operand that is the sum of two bf16 values is off
# by the product of two roundings, 2^-9.2 of the value each in the root mean square
# (a rounding is uniform within half a step, at most 2^-8 of the value), so 2^-18.4;
# some ten such operands, independent of each other, lie between a call's inputs
# and a result: 2^-16.7. The bar is three times that.
CARRIED = 2.0 ** -15
# fp32 tensors: a sum of 256 products added one after the other is off by 2^-25.2
# sqrt(256) of its norm; ten of them, 2^-19.5. The bar is twice that.
FP32 = 2.0 ** -18.5


def gates_bar(dtype):
    return CARRIED if dtype == "bf16" else FP32


def grads(x, scale, **more):
    y = dev(x)
    return rr.delta_chunkwise_bwd(*(y[k] for k in KEYS), y["dout"], scale=scale, state_in=y["s0"], d_state_out=y["ds"],
                                  **more)


def reference(x, scale):
    with np.errstate(invalid="ignore"):  # 0 times infinity at a factor of zero
        return oracle.delta_grad(*(f64(x[k]) for k in KEYS), f64(x["dout"]), scale=scale, state=f64(x["s0"]),
                                 d_state=f64(x["ds"]))


def near_norm(got, ref, bar, what):
    """[units, everything else]: the relative norm of each unit."""
    got, ref = f64(got) if isinstance(got, torch.Tensor) else got, np.asarray(ref)
    assert np.isfinite(got).all(), what
    err = np.linalg.norm(got - ref, axis=1) / np.linalg.norm(ref, axis=1)
    print(f"  {what}: {np.array2string(err, precision=2)} (bar {bar:.2e})", flush=True)
    assert (err <= bar).all(), f"{what}: {err}"


def heads_first(t):
    """[batch, tokens, heads] -> [heads, batch * tokens]"""
    t = f64(t) if isinstance(t, torch.Tensor) else np.asarray(t)
    return np.moveaxis(t, -1, 0).reshape(t.shape[-1], -1)


SIZES = [(2, 257, 2, 2, 64), (1, 300, 2, 4, 128), (1, 200, 1, 2, 256)]


@pytest.mark.parametrize("b,n,hk,h,d", SIZES)
def test_gradients_are_at_their_own_rounding(b, n, hk, h, d):
    x = make(33, b, n, hk, h, d, "bf16")
    got, ref = grads(x, d ** -0.5), reference(x, d ** -0.5)
    for name, g, r in zip(("dq", "dk", "dv"), got, ref):
        near_rounded(g, r, name)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("b,n,hk,h,d", SIZES + [(1, 150, 1, 3, 256)])
def test_states_and_gates_by_head(b, n, hk, h, d, dtype):
    x = make(34, b, n, hk, h, d, dtype)
    y = dev(x)
    s = torch.empty_like(y["s0"])
    rr.delta_chunkwise_fwd(*(y[k] for k in KEYS), state_in=y["s0"], state_out=s)
    _, rs = oracle.delta(*(f64(x[k]) for k in KEYS), state=f64(x["s0"]))
    flat = lambda t: (f64(t) if isinstance(t, torch.Tensor) else t).reshape(b * h, -1)  # noqa: E731
    near_norm(flat(s), flat(rs), gates_bar(dtype), "state")
    got, ref = grads(x, 0.25), reference(x, 0.25)
    near_norm(heads_first(got[3]), heads_first(ref[3]), gates_bar(dtype), "dlog_decay")
    near_norm(heads_first(got[4]), heads_first(ref[4]), gates_bar(dtype), "dbeta")
    near_norm(flat(got[5]), flat(ref[5]), gates_bar(dtype), "dstate")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_decay_gradients_of_heads_that_forget(d, dtype):
    """Heads that keep 10^-1 to 10^-8 of the state a token: each head's d log decay
    against that head's own."""
    logs = [-0.3, -3.0, -6.0, -10.0, -14.0, -18.0]
    x = make(35, 1, 150, len(logs), len(logs), d, dtype)
    x["g"] = torch.tensor(logs) * (0.9 + 0.2 * torch.rand(1, 150, len(logs), generator=torch.Generator().manual_seed(1)))
    got, ref = grads(x, d ** -0.5), reference(x, d ** -0.5)
    near_norm(heads_first(got[3]), heads_first(ref[3]), gates_bar(dtype), "dlog_decay")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("at", [33, 64, 100])
def test_decay_gradient_before_loud_gradients(at, dtype):
    """A token that forgets (exp(-12)), and gradients a thousand times larger after it:
    the tokens before it, the token, and those after it, each on their own. The
    token's value is <S', dS'>, a sum of d^2 products that may come out near zero
    by chance: it is off by the roundings of the products, a third of the bar each
    in the root mean square, so by at most the bar (three times that) of the root
    of the sum of their squares."""
    x = make(36, 1, 190, 2, 2, 128, dtype)
    x["g"][0, at] = -12.0
    x["dout"][0, at:] *= 1024
    got, ref = (heads_first(t[3]) for t in (grads(x, 0.1), reference(x, 0.1)))
    for what, part in (("before", slice(0, at)), ("after", slice(at + 1, None))):
        near_norm(got[:, part], ref[:, part], gates_bar(dtype), what)
    head, tail = ({k: f64(t[:, part]) for k, t in x.items() if k not in ("s0", "ds")}
                  for part in (slice(0, at), slice(at, None)))
    _, s = oracle.delta(*(head[k] for k in KEYS), scale=0.1, state=f64(x["s0"]))
    s = s * np.exp(tail["g"][:, 0])[..., None, None]
    tail["g"][:, 0] = 0.0
    ds = oracle.delta_grad(*(tail[k] for k in KEYS), tail["dout"], scale=0.1, state=s, d_state=f64(x["ds"]))[5]
    terms = (s * ds).reshape(2, -1)
    np.testing.assert_allclose(terms.sum(1), ref[:, at], rtol=1e-8)
    err = np.abs(got[:, at] - ref[:, at]) / np.sqrt((terms ** 2).sum(1))
    print(f"  at: {err} (bar {gates_bar(dtype):.2e})", flush=True)
    assert (err <= gates_bar(dtype)).all()


@pytest.mark.parametrize("dtype,hk,h,d", [("bf16", 2, 4, 128), ("f32", 1, 2, 64), ("bf16", 1, 2, 256)])
def test_packed_gradients_by_head(dtype, hk, h, d):
    lens = [130, 0, 1, 66, 64]
    x = make(37, len(lens), max(lens), hk, h, d, dtype, lens=lens)
    cu = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32, device=DEV)
    got = grads(x, 0.25, cu_seqlens=cu, max_seqlen=max(lens), check=True)
    ref, rs = oracle.packed(oracle.delta_grad, lens, [f64(x[k]) for k in (*KEYS, "dout")], state=f64(x["s0"]),
                            d_state=f64(x["ds"]), scale=0.25)
    if dtype == "bf16":
        for name, g, r in zip(("dq", "dk", "dv"), got, ref):
            near_rounded(g, r, name)
    for name, g, r in zip(("dlog_decay", "dbeta"), got[3:5], ref[3:]):
        near_norm(heads_first(g), heads_first(r), gates_bar(dtype), name)
    near_norm(f64(got[5]).reshape(len(lens) * h, -1), rs.reshape(len(lens) * h, -1), gates_bar(dtype), "dstate")


@pytest.mark.parametrize("b,n,hk,h,d", SIZES)
def test_the_backward_takes_three_values_for_its_matrices(b, n, hk, h, d):
    """d beta = dv . V' / beta^2. With the 64 x 64 matrices and what they multiply in
    24 bits, the operands of two bf16 values on its way are the state, its gradient,
    dv and V': sqrt(4) 2^-18.4, and the bar a third more, 2^-17 = 7.6e-6. With two values
    for the matrices too, heads of these sizes were 6.8e-6 to 9.0e-6 off."""
    x = make(38, b, n, hk, h, d, "bf16")
    near_norm(heads_first(grads(x, 0.25)[4]), heads_first(reference(x, 0.25)[4]), 2.0 ** -17, "dbeta")
