"""What the gated recurrence carries across segments and tiles where factors are no ordinary
numbers: the definition's token-by-token recurrence, which the decode step runs, says what a
state that is NaN or infinite, a log decay above 0 or one of NaN leaves behind, and so do the
parts of a sequence that the kernels join. Only a token's own factor of 0 forgets."""

import numpy as np
import pytest
import torch

import retnet_retention_amd as rr
from test_gpu_scan import DEV, dev, f64, fwd_bar, run_scan, scan_inputs

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")
# (sequences, tokens): one workgroup, tiles that hand on, many of them
SHAPES = [(2, 200), (2, 400), (2, 1000)]
LANES = [("bf16", 66), ("bf16", 67), ("f32", 65)]


def steps(x):
    """The whole sequence by decode steps: (outputs, state)."""
    s = torch.zeros(x["x"].shape[0], x["x"].shape[2], device=DEV) if x["s0"] is None else x["s0"].clone()
    cut = lambda t, i: None if t is None else t[:, i:i + 1]  # noqa: E731
    outs = [rr.gated_scan_step(cut(x["x"], i), cut(x["decay"], i), s, cut(x["gate"], i), rate=x["rate"])
            for i in range(x["x"].shape[1])]
    return torch.cat(outs, 1), s


def forward(x):
    s = torch.empty(x["x"].shape[0], x["x"].shape[2], device=DEV)
    return rr.gated_scan_fwd(x["x"], x["decay"], x["gate"], rate=x["rate"], state_in=x["s0"], state_out=s), s


def same_kind(got, ref, what, exact=True):
    """Numbers where the reference has them; NaN where it is NaN and its infinities, but where parts
    of a sum have overflowed by themselves (not exact)."""
    got, ref = got.float(), ref.float()
    assert torch.equal(torch.isfinite(got), torch.isfinite(ref)), what
    if not exact:
        return
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), what
    for v in (INF, -INF):
        assert torch.equal(got == v, ref == v), what


def near_steps(x, n, exact=True):
    """Every element's kind, and each channel's numbers to the error of n tokens on each side (in
    bf16 a rounding of 2^-8 on each side too)."""
    ref, got = steps(x), forward(x)
    for g, r, name in zip(got, ref, ("o", "state")):
        same_kind(g, r, name, exact)
        bar = 2 * fwd_bar(n) + (2.0 ** -7 if g.dtype == torch.bfloat16 else 0)
        ok = torch.isfinite(r.float())
        g, r = (torch.where(ok, t.double(), 0.0) for t in (g, r))
        axes = tuple(range(g.dim() - 1))
        assert ((g - r).norm(dim=axes) <= bar * r.norm(dim=axes)).all(), name
    return got


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype,w", LANES)
@pytest.mark.parametrize("la", [NAN, 80.0, 100.0])
def test_a_reset_forgets_what_any_factor_left(shape, dtype, w, la):
    """A log decay of NaN, or some far above 0, before a token that forgets: in its segment, in
    another one of its tile, in an earlier tile."""
    n = shape[1]
    x = dev(scan_inputs(71, shape, w, dtype, "log", state=shape[0]))
    x["decay"][:, n - 60] = -np.inf
    for c, before in enumerate((1, 3, 20, 100, n - 70)):
        x["decay"][:, n - 60 - before, c::5] = la
        if la > 0:
            x["decay"][:, n - 61 - before, c::5] = la
    o, s = near_steps(x, n, exact=la != la)
    assert torch.isfinite(o[:, n - 60:].float()).all() and torch.isfinite(s).all()
    # nothing of what stood before the reset is left
    cut = {k: t[:, n - 60:].contiguous() if k in ("x", "decay", "gate") else t for k, t in x.items()}
    o1, s1 = forward(dict(cut, s0=torch.zeros_like(x["s0"])))
    bar = 2 * fwd_bar(60) + (2.0 ** -7 if dtype == "bf16" else 0)
    assert (o[:, n - 60:].double() - o1.double()).norm() <= bar * o1.double().norm()
    assert (s.double() - s1.double()).norm() <= 2 * fwd_bar(60) * s1.double().norm()


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype,w", LANES)
@pytest.mark.parametrize("la", [-0.7, -3.0, -7.0, -20.0])
@pytest.mark.parametrize("fill", [NAN, INF, -INF])
def test_only_a_factor_of_zero_forgets(shape, dtype, w, la, fill):
    """Factors whose products are no normal numbers keep a state that is none: from state_in, or
    from a token, to the end of the sequence."""
    x = dev(scan_inputs(72, shape, w, dtype, "log", state=shape[0]))
    x["decay"].fill_(la)
    x["s0"][:, ::3] = fill
    x["x"][:, 90, 1::3] = fill
    o, s = near_steps(x, shape[1])
    assert not torch.isfinite(s[:, 1::3]).any() and not torch.isfinite(s[:, ::3]).any()
    assert torch.isfinite(s[:, 2::3]).all() and torch.isfinite(o[..., 2::3].float()).all()


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype,w", LANES)
@pytest.mark.parametrize("la,size", [(0.5, 0.0), (8.0, 0.0), (None, 1e-30), (-0.5, 1e30), (-6.0, 1e30)])
def test_products_that_leave_the_range(shape, dtype, w, la, size):
    """A state that is 0, tiny or huge under factors whose product over a tile, or a segment, is
    no normal number in 32 bits, while the state itself is one."""
    la = 130.0 / shape[1] if la is None else la  # grows by exp(130) over the sequence
    x = dev(scan_inputs(73, shape, w, dtype, "log", state=shape[0]))
    x["decay"].fill_(la)
    x["decay"][..., ::2] *= 0.9
    x["x"].zero_()
    x["s0"] *= size
    ref, got = steps(x), forward(x)
    # elements next to the smallest normal numbers (a bf16 output's are fp32's) have fewer bits
    for g, r, name in zip(got, ref, ("o", "state")):
        g, r = g.double(), r.double()
        assert torch.isfinite(g).all(), name
        bar = 8 * fwd_bar(shape[1]) + (2.0 ** -7 if name == "o" and dtype == "bf16" else 0)
        assert ((g - r).abs() <= bar * r.abs() + 2.0 ** -126).all(), name


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype,w", LANES)
def test_a_product_that_comes_back(shape, dtype, w):
    """Below the normal numbers inside a tile and up again: the state is a number all the way."""
    x = dev(scan_inputs(78, shape, w, dtype, "log", state=shape[0]))
    x["x"].zero_()
    x["decay"].fill_(0.0)
    x["decay"][:, 1:129], x["decay"][:, 130:199] = -0.8, 0.8
    x["s0"] *= 1e30
    ref, got = steps(x), forward(x)
    for g, r, name in zip(got, ref, ("o", "state")):
        g, r = g.double(), r.double()
        bar = 8 * fwd_bar(shape[1]) + (2.0 ** -7 if name == "o" and dtype == "bf16" else 0)
        assert ((g - r).abs() <= bar * r.abs() + 2.0 ** -126).all(), name


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype,w", LANES)
@pytest.mark.parametrize("la", [-0.7, -7.0])
def test_gradients_that_are_no_numbers_reach_every_token_before(shape, dtype, w, la):
    """Through factors whose products are no normal numbers, from d_state_out or a late dout; a
    factor of 0 lets nothing through, whatever the factors beside it."""
    b, n = shape
    x = dev(scan_inputs(74, shape, w, dtype, "log", state=b))
    x["decay"].fill_(la)
    ref = run_scan(x, False)
    y = dict(x, ds=x["ds"].clone(), dout=x["dout"].clone())
    y["ds"][:, ::4] = NAN
    y["dout"][:, n - 30, 1::4] = INF
    got = run_scan(y, False)
    for k in ("dx", "dgate", "ddecay"):
        assert torch.isnan(got[k][..., ::4].float()).all(), k
        assert not torch.isfinite(got[k][:, :n - 29, 1::4].float()).any(), k
        for c in (2, 3):
            assert torch.equal(got[k][..., c::4], ref[k][..., c::4]), k
    assert torch.isnan(got["dstate"][:, ::4]).all() and not torch.isfinite(got["dstate"][:, 1::4]).any()
    # a token that forgets before them, with a NaN factor behind it in its segment, another one, another tile
    z = dict(y, decay=y["decay"].clone())
    z["decay"][:, 40] = -np.inf
    for c, behind in enumerate((1, 3, 20, 100)):
        z["decay"][:, 40 + behind, c::4] = NAN
    cut = dict(x, decay=x["decay"].clone())
    cut["decay"][:, 40] = -np.inf
    got, ref = run_scan(z, False), run_scan(cut, False)
    for k in ("dx", "dgate", "ddecay"):
        assert torch.equal(got[k][:, :40], ref[k][:, :40]), k
    assert (got["ddecay"][:, 40] == 0).all() and torch.equal(got["dstate"], ref["dstate"])


@pytest.mark.parametrize("dtype,w", LANES)
def test_a_channel_without_numbers_leaves_its_neighbours(dtype, w):
    """Their bits, forward and backward, whatever stands beside them."""
    x = dev(scan_inputs(75, (2, 700), w, dtype, "log", state=2))
    ref = run_scan(x, True)
    y = dict(x, decay=x["decay"].clone(), s0=x["s0"].clone(), ds=x["ds"].clone())
    for c, la in enumerate((NAN, -np.inf, -9.0, -1.0)):
        y["decay"][:, 20 * c:400 + 30 * c, c::6] = la
    y["s0"][:, 2::6], y["ds"][:, 3::6] = INF, NAN
    got = run_scan(y, True)
    for k in got:
        if got[k] is not None:
            for c in (4, 5):
                assert torch.equal(got[k][..., c::6], ref[k][..., c::6]), k


@pytest.mark.parametrize("dtype,w", LANES)
def test_packed_sequences_of_such_factors(dtype, w):
    """Each one gives what it gives alone, gradients too."""
    lens = [300, 0, 70, 600]
    cu = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32, device=DEV)
    x = dev(scan_inputs(76, (sum(lens),), w, dtype, "log", state=4))
    x["decay"][:, ::4] = -1.0
    x["decay"][320, 1::4] = -np.inf
    x["decay"][310, 1::4] = NAN
    x["s0"][:, ::4] = INF
    got = run_scan(x, False, cu_seqlens=cu, check=True)
    for i, (a, b) in enumerate(zip(cu.tolist(), cu.tolist()[1:])):
        if a == b:
            continue
        part = {k: None if t is None else t[i:i + 1].clone() if k in ("s0", "ds") else t[a:b][None].clone()
                for k, t in x.items()}
        one = run_scan(part, False)
        for k in ("o", "dx", "ddecay", "dgate"):
            same_kind(got[k][a:b], one[k][0], k)
            ok = torch.isfinite(one[k][0].float())
            d = torch.where(ok, got[k][a:b].double() - one[k][0].double(), 0.0)
            r = torch.where(ok, one[k][0].double(), 0.0)
            # tiles of other bounds join other parts; bf16 results are rounded on both sides
            bar = 8 * fwd_bar(600) + (2.0 ** -7 if one[k].dtype == torch.bfloat16 else 0)
            assert d.norm() <= bar * r.norm(), k
        for k in ("state", "dstate"):
            same_kind(got[k][i], one[k][0], k)


def test_such_states_are_kept_or_run_again_the_same():
    for dtype, w in LANES:
        x = dev(scan_inputs(77, (2, 700), w, dtype, "log", state=2))
        x["decay"][..., ::3] = -1.5
        x["decay"][:, 300, 1::3] = -np.inf
        x["s0"][:, ::6] = INF
        a, b = run_scan(x, False), run_scan(x, False, keep=False)
        for k in a:
            assert a[k] is None or np.array_equal(f64(a[k]), f64(b[k]), equal_nan=True), k
