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


def free_memory(need):
    """Skips where the card holds less (a smaller device, or a shared one)."""
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < need:
        pytest.skip(f"needs {need >> 30} GiB of device memory")


@pytest.mark.parametrize("slots", [False, True])
def test_states_too_large_for_the_caches(slots):
    """Pools above 512 MiB are streamed past the caches: the bits of smaller calls."""
    b, h, d = 132, 16, 256
    assert b * h * d * d * 4 > 512 << 20
    g = torch.Generator(device=DEV).manual_seed(44)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    q, k, v = (r(b, 1, n, d).bfloat16() / 16 for n in (8, 8, h))
    ld, beta = -torch.rand(b, 1, h, generator=g, device=DEV), torch.rand(b, 1, h, generator=g, device=DEV)
    pool = r(b, h, d, d)
    at = torch.randperm(b, generator=g, device=DEV).to(torch.int32) if slots else None
    want, outs = pool.clone(), []
    for i in range(0, b, 33):
        part = [t[i:i + 33].contiguous() for t in (q, k, v, ld, beta)]
        if slots:
            outs.append(rr.delta_recurrent_step(*part, want, slots=at[i:i + 33].contiguous()))
        else:
            outs.append(rr.delta_recurrent_step(*part, want[i:i + 33]))
    o = rr.delta_recurrent_step(q, k, v, ld, beta, pool, slots=at)
    assert torch.equal(o, torch.cat(outs)) and torch.equal(pool, want)


def test_a_slot_behind_2_31_elements():
    h, d, n = 16, 256, 2060
    assert (n - 2) * h * d * d > 2 ** 31
    free_memory(12 << 30)
    x = make(45, 2, 1, 2, h, d, "bf16")
    y = dev(x)
    pool = torch.zeros(n, h, d, d, device=DEV)
    pool[n - 1], pool[n - 2] = y["s0"][0], y["s0"][1]
    slots = torch.tensor([n - 1, n - 2], dtype=torch.int32, device=DEV)
    o = rr.delta_recurrent_step(*(y[k] for k in KEYS), pool, slots=slots)
    s = y["s0"].clone()
    o1 = rr.delta_recurrent_step(*(y[k] for k in KEYS), s)
    assert torch.equal(o, o1) and torch.equal(pool[n - 1], s[0]) and torch.equal(pool[n - 2], s[1])
    assert (pool[:n - 2] == 0).all()


def test_backward_behind_2_31_elements():
    """The last of two packed sequences starts behind 2^31 elements of v and of its
    gradient (and its states behind 2^33): the bits of that sequence alone."""
    h, d, first, last = 128, 256, 66000, 100
    n = first + last
    assert first * h * d > 2 ** 31
    free_memory(160 << 30)
    g = torch.Generator(device=DEV).manual_seed(46)
    v = torch.randn(n, h, d, generator=g, device=DEV, dtype=torch.bfloat16)
    k = torch.randn(n, 1, d, generator=g, device=DEV, dtype=torch.bfloat16) / 16
    ld, beta = -torch.rand(n, h, generator=g, device=DEV), torch.rand(n, h, generator=g, device=DEV)
    cu = torch.tensor([0, first, n], dtype=torch.int32, device=DEV)
    got = rr.delta_chunkwise_bwd(k, k, v, ld, beta, v, cu_seqlens=cu, max_seqlen=first, check=True)
    tail = [t[first:][None].contiguous() for t in (k, k, v, ld, beta, v)]
    for a, b in zip(got, rr.delta_chunkwise_bwd(*tail)):
        assert torch.equal(a[first:], b[0])
        assert torch.isfinite(a[first - 64:first].float()).all()
    del got
    torch.cuda.empty_cache()


# With one key many times over a written value is beta times what the writes before it
# left, a sum of up to thirty terms of its own size that each carry an error of their
# own: sqrt(30) < 6 times the errors of other inputs.
REPEATED = 6


@pytest.mark.parametrize("d", [128, 256])
def test_strength_extremes_in_bf16(d):
    """beta 0, 1 and 2, one key many times over: values replaced and reflected."""
    from test_gpu_delta_accuracy import CARRIED, ROUNDED_ONCE, near_norm, rounded

    x = make(47, 1, 140, 1, 2, d, "bf16")
    x["beta"][0, 5:30] = 0.0
    x["beta"][0, 30:70] = 1.0
    x["beta"][0, 70:80] = 2.0
    x["k"][0, 32:60] = x["k"][0, 31]
    y, args = dev(x), [f64(x[k]) for k in KEYS]
    s = torch.empty_like(y["s0"])
    o = rr.delta_chunkwise_fwd(*(y[k] for k in KEYS), state_in=y["s0"], state_out=s)
    ro, rs = oracle.delta(*args, state=f64(x["s0"]))
    got = rr.delta_chunkwise_bwd(*(y[k] for k in KEYS), y["dout"], state_in=y["s0"], d_state_out=y["ds"])
    ref = oracle.delta_grad(*args, f64(x["dout"]), state=f64(x["s0"]), d_state=f64(x["ds"]))
    row = lambda t: (f64(t) if isinstance(t, torch.Tensor) else t).reshape(1, -1)  # noqa: E731
    for name, a, r in (("o", o, ro), ("dq", got[0], ref[0]), ("dk", got[1], ref[1]), ("dv", got[2], ref[2])):
        near_norm(row(a), row(rounded(r)), ROUNDED_ONCE * REPEATED ** 0.5, name)
    for name, a, r in (("state", s, rs), ("dlog_decay", got[3], ref[3]), ("dbeta", got[4], ref[4]), ("ds", got[5], ref[5])):
        near_norm(row(a), row(r), CARRIED * REPEATED, name)


@pytest.mark.parametrize("d", [128, 256])
def test_decay_extremes_in_bf16(d):
    """-infinity forgets, 0 keeps, strong decays underflow, all in one block."""
    from test_gpu_delta_accuracy import CARRIED, near_norm, near_rounded

    x = make(48, 1, 150, 1, 2, d, "bf16")
    for at, v in ((10, -np.inf), (70, -1e30), (71, -200.0)):
        x["g"][0, at] = v
    x["g"][0, 20:40] = 0.0
    x["g"][0, 100:103, 0] = -3e4
    y = dev(x)
    s = torch.empty_like(y["s0"])
    o = rr.delta_chunkwise_fwd(*(y[k] for k in KEYS), state_in=y["s0"], state_out=s)
    ro, rs = oracle.delta(*(f64(x[k]) for k in KEYS), state=f64(x["s0"]))
    near_rounded(o, ro, "o")
    got = rr.delta_chunkwise_bwd(*(y[k] for k in KEYS), y["dout"], state_in=y["s0"], d_state_out=y["ds"])
    x["g"] = x["g"].clamp(min=-2000.0)  # a factor of 0 in 64 bits too, and finite
    ref = oracle.delta_grad(*(f64(x[k]) for k in KEYS), f64(x["dout"]), state=f64(x["s0"]), d_state=f64(x["ds"]))
    for name, a, r in zip(("dq", "dk", "dv"), got, ref):
        near_rounded(a, r, name)
    row = lambda t: (f64(t) if isinstance(t, torch.Tensor) else t).reshape(1, -1)  # noqa: E731
    near_norm(row(s), row(rs), CARRIED, "state")
    for name, a, r in zip(("dlog_decay", "dbeta", "dstate"), got[3:], ref[3:]):
        near_norm(row(a), row(r), CARRIED, name)


def workspace(call, fill):
    """A workspace of `call`'s size with every byte `fill` (255: NaN in every type)."""
    need = []
    with pytest.raises(rr.RetentionError):
        call(torch.empty(16, dtype=torch.uint8, device=DEV))
    for size in (1 << i for i in range(16, 36)):
        try:
            call(torch.empty(size, dtype=torch.uint8, device=DEV))
            need.append(size)
            break
        except rr.RetentionError:
            continue
    return torch.full((need[0],), fill, dtype=torch.uint8, device=DEV)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("hk,h,lens", [(2, 2, None), (1, 3, None), (2, 2, [65, 0, 1, 130]), (1, 2, [64, 63])])
def test_nothing_of_the_workspace_is_read_before_it_is_written(dtype, d, hk, h, lens):
    """The same bits whatever the workspace held, call after call, every variant of the kernels."""
    b, n = (len(lens), max(lens)) if lens else (2, 130)
    x = make(49, b, n, hk, h, d, dtype, lens=lens)
    y, more = dev(x), {}
    if lens:
        more = dict(cu_seqlens=torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32, device=DEV), max_seqlen=n)
    s = torch.empty_like(y["s0"])
    fwd = lambda ws: [rr.delta_chunkwise_fwd(*(y[k] for k in KEYS), state_in=y["s0"], state_out=s, workspace=ws,  # noqa: E731
                                             **more), s.clone()]
    bwd = lambda ws: list(rr.delta_chunkwise_bwd(*(y[k] for k in KEYS), y["dout"], state_in=y["s0"],  # noqa: E731
                                                 d_state_out=y["ds"], workspace=ws, **more))
    for call in (fwd, bwd):
        ref = call(workspace(call, 0))
        ws = workspace(call, 255)
        for _ in range(3):
            for a, r in zip(call(ws), ref):
                assert torch.isfinite(a.float()).all() and torch.equal(a, r)


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f32", 64)])
def test_a_loose_bound_on_the_lengths(dtype, d):
    """max_seqlen far above every length: the bits of the tight bound, both directions."""
    lens = [70, 0, 200, 1]
    x = make(50, len(lens), 200, 1, 2, d, dtype, lens=lens)
    y = dev(x)
    cu = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32, device=DEV)
    outs = []
    for bound in (200, 100000):
        s = torch.empty_like(y["s0"])
        o = rr.delta_chunkwise_fwd(*(y[k] for k in KEYS), state_in=y["s0"], state_out=s, cu_seqlens=cu, max_seqlen=bound,
                                   check=True)
        outs.append([o, s, *rr.delta_chunkwise_bwd(*(y[k] for k in KEYS), y["dout"], state_in=y["s0"],
                                                   d_state_out=y["ds"], cu_seqlens=cu, max_seqlen=bound, check=True)])
    assert all(torch.equal(a, b) for a, b in zip(*outs))


def test_the_largest_launch():
    """8191 sequences of one token, 128 heads of 256: just below 2^32 threads."""
    b, h, d = 8191, 128, 256
    assert 8 * b * h * 512 > 2 ** 32 - 2 ** 20
    free_memory(60 << 30)
    g = torch.Generator(device=DEV).manual_seed(51)
    k = torch.randn(b, 1, 1, d, generator=g, device=DEV, dtype=torch.bfloat16) / 16
    v = torch.randn(b, 1, h, d, generator=g, device=DEV, dtype=torch.bfloat16)
    ld, beta = -torch.rand(b, 1, h, generator=g, device=DEV), torch.rand(b, 1, h, generator=g, device=DEV)
    o = rr.delta_chunkwise_fwd(k, k, v, ld, beta)
    for at in (0, 4000, b - 3):
        part = [t[at:at + 3].contiguous() for t in (k, k, v, ld, beta)]
        assert torch.equal(o[at:at + 3], rr.delta_chunkwise_fwd(*part))
    # one token and no state: o = beta (q . k) v
    w = (k.double() ** 2).sum(-1, keepdim=True) * beta[..., None].double()
    err = (o[-64:].double() - w[-64:] * v[-64:].double()).norm() / (w[-64:] * v[-64:].double()).norm()
    assert err < 2.0 ** -8


def test_packed_backward_in_a_graph():
    """Captured on one stream with a workspace that held NaN, replayed on new inputs
    between eager calls."""
    lens = [130, 0, 66]
    x = make(52, len(lens), 130, 1, 2, 64, "bf16", lens=lens)
    y = dev(x)
    more = dict(cu_seqlens=torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32, device=DEV), max_seqlen=130)
    run = lambda ws=None: rr.delta_chunkwise_bwd(*(y[k] for k in KEYS), y["dout"], state_in=y["s0"],  # noqa: E731
                                                 d_state_out=y["ds"], workspace=ws, **more)
    ws = workspace(run, 255)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run(ws)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            outs = run(ws)
    torch.cuda.current_stream().wait_stream(side)
    for seed in range(4):
        for k in ("v", "dout"):
            y[k].copy_(torch.randn(y[k].shape, generator=torch.Generator().manual_seed(seed)))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, run()))
