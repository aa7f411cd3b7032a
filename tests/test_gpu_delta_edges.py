"""Calls of the gated delta rule that its documentation allows at its borders:
states that hold no number, large pools, offsets, padding."""

import numpy as np
import pytest
import torch

import retnet_retention_amd as rr
from oracle import delta_oracle as oracle
from test_gpu_delta import DEV, bars, by_head, close, dev, f64, make

pytestmark = pytest.mark.gpu
KEYS = ("q", "k", "v", "g", "beta")


@pytest.mark.parametrize("fill", [float("nan"), float("inf")])
@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 128), ("bf16", 256), ("f32", 64), ("f32", 256)])
def test_a_first_token_that_forgets_clears_any_state(fill, dtype, d):
    """The bits of a call on a state of zeros, forward and backward."""
    x = make(41, 2, 130, 1, 2, d, dtype)
    x["g"][:, 0] = -np.inf
    x["g"][1, 0] = -1000.0  # a factor of 0 as well
    y = dev(x)
    outs = []
    for s0 in (torch.full_like(y["s0"], fill), torch.zeros_like(y["s0"])):
        s = s0.clone()
        o = rr.delta_chunkwise_fwd(*(y[k] for k in KEYS), state_in=s, state_out=s)
        outs.append([o, s, *rr.delta_chunkwise_bwd(*(y[k] for k in KEYS), y["dout"], state_in=s0, d_state_out=y["ds"])])
    for a, b in zip(*outs):
        assert torch.isfinite(a.float()).all() and torch.equal(a, b)
    assert (outs[0][7] == 0).all()  # d state_in


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("f32", 128), ("bf16", 256)])
def test_a_step_that_forgets_clears_its_slot(dtype, d):
    x = make(42, 3, 1, 1, 2, d, dtype)
    x["g"][:2] = -np.inf
    y = dev(x)
    pools = [torch.full((4, 2, d, d), v, device=DEV) for v in (float("nan"), 0.0)]
    for pool in pools:
        pool[2] = y["s0"][2]
    slots = torch.tensor([3, 0, 2], dtype=torch.int32, device=DEV)
    outs = [rr.delta_recurrent_step(*(y[k] for k in KEYS), pool, slots=slots) for pool in pools]
    assert torch.isfinite(outs[0].float()).all() and torch.equal(*outs)
    for slot in (0, 2, 3):
        assert torch.isfinite(pools[0][slot]).all() and torch.equal(pools[0][slot], pools[1][slot])
    assert torch.isnan(pools[0][1]).all()  # nobody's


def test_an_empty_sequence_passes_any_state_on():
    """No token, no reset: the state goes through, NaN and all."""
    x = make(43, 2, 40, 1, 1, 64, "bf16", lens=[0, 40])
    x["g"][0] = -np.inf
    y = dev(x)
    s = y["s0"].clone()
    s[:, 0, 3, 5] = float("nan")
    cu = torch.tensor([0, 0, 40], dtype=torch.int32, device=DEV)
    out = torch.empty_like(s)
    o = rr.delta_chunkwise_fwd(*(y[k] for k in KEYS), state_in=s, state_out=out, cu_seqlens=cu, max_seqlen=40, check=True)
    assert torch.isfinite(o.float()).all() and torch.isfinite(out[1]).all()
    np.testing.assert_array_equal(f64(out[0]), f64(s[0]))
