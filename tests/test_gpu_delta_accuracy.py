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
