"""The norms at their borders: rows behind 2^31 elements, in the backward."""

import pytest
import torch

import retnet_retention_amd as rr

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def test_backward_behind_2_31_elements():
    """A row's gradients depend on that row alone: the bits of a call on the last rows."""
    rows, width, tail = 131200, 16384, 64
    assert (rows - tail) * width > 2 ** 31
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GiB of device memory")
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randn(rows, width, generator=g, device=DEV, dtype=torch.bfloat16)
    dout = torch.randn(rows, width, generator=g, device=DEV, dtype=torch.bfloat16)
    w = 1 + 0.1 * torch.randn(width, generator=g, device=DEV)
    last = [t[-tail:].contiguous() for t in (x, dout)]
    dx, dw, dgate = rr.head_norm_bwd(x, dout, w, x)
    d1, _, dg1 = rr.head_norm_bwd(last[0], last[1], w, last[0])
    assert torch.equal(dx[-tail:], d1) and torch.equal(dgate[-tail:], dg1) and torch.isfinite(dw).all()
    del dx, dgate
    dx, dy, dw, dpost, dscale = rr.residual_norm_bwd(x, dout, w, x, dout, post_weight=w, scale=w)
    ref = rr.residual_norm_bwd(last[0], last[1], w, last[0], last[1], post_weight=w, scale=w)
    assert torch.equal(dx[-tail:], ref[0]) and torch.equal(dy[-tail:], ref[1])
    assert all(torch.isfinite(t).all() for t in (dw, dpost, dscale))
    del dx, dy
    torch.cuda.empty_cache()
