"""The gated delta rule on the GPU against the fp64 oracle (token by token).

Tolerances, relative Frobenius norms over every (sequence, head):
- bf16 outputs and gradients: each takes its own rounding and that of at most
  three bf16 operands of its two or three terms, each at most eps / 2 = 2^-8 of
  its term; the terms of these inputs do not cancel, so 4 2^-8.
- fp32 results of bf16 tensors: the carried operands are sums of two bf16
  values, off by at most 2^-16, six of them from a block's state to the next
  (the state, T, X, V' twice, the product of two rests): 8 2^-16; the decays'
  gradients are differences of row sums about 8 times their size, 64 2^-16.
- fp32 tensors: sums of d + 2 * 64 products each off by 2^-24, in five
  products: 5 (d + 128) 2^-24; 8 times that for the decays' gradients."""

import numpy as np
import pytest
import torch

import retnet_retention_amd as rr
from oracle import delta_oracle as oracle

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def make(seed, b, n, hk, h, d, dtype, lens=None, decay=0.1, state=True):
    """Inputs on the host: unit keys that share a direction, decays over a
    range of heads; packed [tokens, ...] with `lens`."""
    g = torch.Generator().manual_seed(seed)
    rows = (sum(lens),) if lens is not None else (b, n)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    x = {"q": unit(r(*rows, hk, d) + 0.4 * r(hk, d)).to(DT[dtype]), "k": unit(r(*rows, hk, d) + 0.4 * r(hk, d)).to(DT[dtype]),
         "v": r(*rows, h, d).to(DT[dtype]),
         "g": -decay * torch.nn.functional.softplus(r(*rows, h)), "beta": torch.sigmoid(r(*rows, h)),
         "dout": r(*rows, h, d).to(DT[dtype]),
         "s0": 0.1 * r(b, h, d, d) if state else None, "ds": 0.1 * r(b, h, d, d) if state else None}
    return x


def dev(x):
    return {k: None if t is None else t.to(DEV) for k, t in x.items()}


def f64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def close(got, ref, tol, what, per):
    """Relative norm over the leading `per` axes' units (rows of zeros: absolute)."""
    got, ref = f64(got), np.asarray(ref)
    assert got.shape == ref.shape and np.isfinite(got).all(), what
    g, r = got.reshape(per, -1), ref.reshape(per, -1)
    floor = max(1e-30, 1e-2 * np.sqrt((r ** 2).sum() / per))
    err = np.linalg.norm(g - r, axis=1) / np.maximum(np.linalg.norm(r, axis=1), floor)
    print(f"  {what}: {err.max():.2e} (bar {tol:.2e})", flush=True)
    assert err.max() <= tol, f"{what}: {err.max():.3e} > {tol:.3e}"


def by_head(t):
    """[..., tokens, heads, d] -> [heads, everything else], so a wrong head or sequence shows."""
    t = f64(t) if isinstance(t, torch.Tensor) else np.asarray(t)
    return torch.from_numpy(np.ascontiguousarray(np.moveaxis(t, -2, 0)))


def bars(dtype, d):
    if dtype == "bf16":
        return 4 * 2.0 ** -8, 8 * 2.0 ** -16, 64 * 2.0 ** -16
    e = 5 * (d + 128) * 2.0 ** -24
    return e, e, 8 * e


def forward(x, scale, lens=None, n=None, **kw):
    s_out = None if x["s0"] is None else torch.full_like(x["s0"], float("nan"))
    more = dict(kw)
    if lens is not None:
        cu = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32, device=DEV)
        more.update(cu_seqlens=cu, max_seqlen=n, check=True)
    o = rr.delta_chunkwise_fwd(x["q"], x["k"], x["v"], x["g"], x["beta"], scale=scale, state_in=x["s0"],
                               state_out=s_out, **more)
    torch.cuda.synchronize()
    return o, s_out


SHAPES = [
    # batch, tokens, key heads, heads, d, dtype
    (1, 1, 1, 1, 64, "f32"), (2, 63, 1, 2, 64, "f32"), (1, 64, 2, 2, 128, "f32"), (2, 130, 1, 3, 128, "f32"),
    (1, 200, 2, 2, 256, "f32"), (1, 1, 1, 2, 256, "bf16"), (2, 65, 2, 2, 64, "bf16"), (1, 257, 2, 4, 128, "bf16"),
    (2, 300, 2, 2, 256, "bf16"), (1, 700, 1, 2, 64, "bf16"), (3, 128, 1, 1, 256, "bf16"), (2, 64, 4, 8, 64, "bf16"),
]


@pytest.mark.parametrize("b,n,hk,h,d,dtype", SHAPES)
@pytest.mark.parametrize("state", [False, True])
def test_forward(b, n, hk, h, d, dtype, state):
    x = make(1, b, n, hk, h, d, dtype, state=state)
    o, s = forward(dev(x), d ** -0.5)
    ro, rs = oracle.delta(*(f64(x[k]) for k in ("q", "k", "v", "g", "beta")), scale=d ** -0.5, state=f64(x["s0"]))
    t_out, t_state, _ = bars(dtype, d)
    close(by_head(o), by_head(ro), t_out, "o", h)
    if state:
        close(s, rs, t_state, "state", b * h)


@pytest.mark.parametrize("lens,hk,h,d,dtype", [
    ([0, 70, 0, 1, 200, 0], 1, 2, 64, "bf16"), ([64, 64, 65, 63], 2, 4, 128, "bf16"), ([300, 5], 1, 1, 256, "bf16"),
    ([0, 0], 1, 1, 64, "bf16"), ([33, 0, 129], 2, 2, 128, "f32"),
])
def test_packed(lens, hk, h, d, dtype):
    """Packed sequences, empty ones too, and rows behind the last one left as they were."""
    n = max(max(lens), 1)
    x = make(2, len(lens), n, hk, h, d, dtype, lens=lens)
    pad = {k: (torch.cat([t, torch.full((3, *t.shape[1:]), float("nan"), dtype=t.dtype)]) if k not in ("s0", "ds") else t)
           for k, t in x.items()}
    rows = sum(lens)
    if len(lens) * n < rows + 3:
        pad = x
    y = dev(pad)
    mark = torch.full_like(y["v"], 7.0)
    o, s = forward(y, 0.3, lens=lens, n=n, out=mark)
    (ro,), rs = oracle.packed(oracle.delta, lens, [f64(x[k]) for k in ("q", "k", "v", "g", "beta")], state=f64(x["s0"]),
                              scale=0.3)
    t_out, t_state, _ = bars(dtype, d)
    assert (o[rows:] == 7).all()
    if rows:
        close(by_head(o[:rows]), by_head(ro), t_out, "o", h)
    close(s, rs, t_state, "state", len(lens) * h)
    for i, m in enumerate(lens):
        if m == 0:
            assert torch.equal(s[i], y["s0"][i])


@pytest.mark.parametrize("b,n,hk,h,d,dtype", SHAPES)
@pytest.mark.parametrize("state", [False, True])
def test_backward(b, n, hk, h, d, dtype, state):
    x = make(3, b, n, hk, h, d, dtype, state=state)
    y = dev(x)
    got = rr.delta_chunkwise_bwd(y["q"], y["k"], y["v"], y["g"], y["beta"], y["dout"], scale=0.25, state_in=y["s0"],
                                 d_state_out=y["ds"])
    torch.cuda.synchronize()
    ref = oracle.delta_grad(*(f64(x[k]) for k in ("q", "k", "v", "g", "beta", "dout")), scale=0.25, state=f64(x["s0"]),
                            d_state=f64(x["ds"]))
    t_out, t_state, t_gate = bars(dtype, d)
    for name, g, r, heads in zip(("dq", "dk", "dv"), got, ref, (hk, hk, h)):
        close(by_head(g), by_head(r), t_out, name, heads)
    for name, g, r in zip(("dlog_decay", "dbeta"), got[3:5], ref[3:5]):
        close(g, r, t_gate, name, 1)
    if state:
        close(got[5], ref[5], t_state, "dstate", b * h)
    assert len(got) == (6 if state else 5)


@pytest.mark.parametrize("given", ["state_in", "d_state_out"])
def test_backward_with_one_of_the_states(given):
    x = make(4, 2, 150, 1, 2, 64, "f32")
    y = dev(x)
    s0, ds = (x["s0"], None) if given == "state_in" else (None, x["ds"])
    got = rr.delta_chunkwise_bwd(*(y[k] for k in ("q", "k", "v", "g", "beta", "dout")),
                                 state_in=y["s0"] if s0 is not None else None,
                                 d_state_out=y["ds"] if ds is not None else None)
    ref = oracle.delta_grad(*(f64(x[k]) for k in ("q", "k", "v", "g", "beta", "dout")), state=f64(s0), d_state=f64(ds))
    for i, (g, r) in enumerate(zip(got, ref)):
        close(g, r, bars("f32", 64)[2], str(i), 1)


@pytest.mark.parametrize("lens,hk,h,d,dtype", [([70, 0, 300, 1], 1, 2, 64, "bf16"), ([64, 129], 2, 2, 128, "f32"),
                                               ([40, 280], 1, 2, 256, "bf16")])
def test_packed_backward(lens, hk, h, d, dtype):
    x = make(5, len(lens), max(lens), hk, h, d, dtype, lens=lens)
    y = dev(x)
    cu = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32, device=DEV)
    got = rr.delta_chunkwise_bwd(*(y[k] for k in ("q", "k", "v", "g", "beta", "dout")), state_in=y["s0"],
                                 d_state_out=y["ds"], cu_seqlens=cu, max_seqlen=max(lens), check=True)
    ref, rs = oracle.packed(oracle.delta_grad, lens, [f64(x[k]) for k in ("q", "k", "v", "g", "beta", "dout")],
                            state=f64(x["s0"]), d_state=f64(x["ds"]))
    t_out, t_state, t_gate = bars(dtype, d)
    for name, g, r, t in zip(("dq", "dk", "dv", "dg", "dbeta"), got, ref, (t_out,) * 3 + (t_gate,) * 2):
        close(g, r, t, name, 1)
    close(got[5], rs, t_state, "dstate", len(lens) * h)


@pytest.mark.parametrize("b,hk,h,d,dtype", [(1, 1, 1, 64, "f32"), (3, 2, 4, 128, "bf16"), (5, 2, 2, 256, "bf16"),
                                            (2, 1, 3, 256, "f32")])
def test_step_equals_chunkwise_and_oracle(b, hk, h, d, dtype):
    """Steps one after the other: each output and the final state."""
    n = 5
    x = make(6, b, n, hk, h, d, dtype)
    y = dev(x)
    s = y["s0"].clone()
    outs = [rr.delta_recurrent_step(*(y[k][:, t:t + 1].contiguous() for k in ("q", "k", "v", "g", "beta")), s, scale=0.4)
            for t in range(n)]
    torch.cuda.synchronize()
    ro, rs = oracle.delta(*(f64(x[k]) for k in ("q", "k", "v", "g", "beta")), scale=0.4, state=f64(x["s0"]))
    # one rounding of the output; the state in fp32 throughout, n steps of d-long sums
    close(by_head(torch.cat(outs, 1)), by_head(ro), 2.0 ** -8 if dtype == "bf16" else n * d * 2.0 ** -24, "o", h)
    close(s, rs, n * d * 2.0 ** -24, "state", b * h)
    o2, s2 = forward(y, 0.4)
    close(s2, f64(s), bars(dtype, d)[1], "state against the chunkwise form", b * h)


def test_step_slots():
    """A pool of states: sequences take their slots; a negative slot, one
    outside the pool and one named twice are idle (zero rows, nothing written)."""
    b, h, d, pool = 7, 2, 64, 6
    x = make(7, b, 1, 1, h, d, "bf16", state=False)
    y = dev(x)
    st = torch.randn(pool, h, d, d, generator=torch.Generator().manual_seed(1)).to(DEV)
    before = st.clone()
    slots = torch.tensor([4, -1, 0, 4, 6, 2, -2147483648], dtype=torch.int32, device=DEV)
    o = rr.delta_recurrent_step(y["q"], y["k"], y["v"], y["g"], y["beta"], st, slots=slots)
    live = {0: 4, 2: 0, 5: 2}
    for i in range(b):
        if i in live:
            sl = slice(i, i + 1)
            ro, rs = oracle.delta(*(f64(x[k][sl]) for k in ("q", "k", "v", "g", "beta")),
                                  state=f64(before[live[i]])[None])
            close(o[i], ro[0], 2.0 ** -8, f"o{i}", 1)
            close(st[live[i]], rs[0], d * 2.0 ** -24, f"state{i}", 1)
        else:
            assert (o[i] == 0).all()
    for slot in (1, 3, 5):
        assert torch.equal(st[slot], before[slot])


@pytest.mark.parametrize("d", [64, 256])
def test_decay_extremes(d):
    """-infinity forgets, 0 keeps, a strong decay underflows to nothing, all in one block."""
    x = make(8, 1, 150, 1, 2, d, "f32")
    x["g"][0, 10] = -float("inf")
    x["g"][0, 70] = -1e30
    x["g"][0, 71] = -200.0
    x["g"][0, 20:40] = 0.0
    x["g"][0, 100:103, 0] = -3e4
    y = dev(x)
    o, s = forward(y, 1.0)
    ro, rs = oracle.delta(*(f64(x[k]) for k in ("q", "k", "v", "g", "beta")), state=f64(x["s0"]))
    close(o, ro, bars("f32", d)[0], "o", 1)
    close(s, rs, bars("f32", d)[1], "state", 1)
    got = rr.delta_chunkwise_bwd(*(y[k] for k in ("q", "k", "v", "g", "beta", "dout")), state_in=y["s0"],
                                 d_state_out=y["ds"])
    with np.errstate(invalid="ignore"):
        ref = oracle.delta_grad(*(f64(x[k]) for k in ("q", "k", "v", "g", "beta", "dout")), state=f64(x["s0"]),
                                d_state=f64(x["ds"]))
    for i, (g, r) in enumerate(zip(got, ref)):
        close(g, r, bars("f32", d)[2], str(i), 1)


def test_strength_extremes():
    """beta 0 (padding), 1 and 2, with the same key many times over: values
    replaced and reflected. d beta at beta 0 is a number of its own."""
    x = make(9, 1, 140, 1, 1, 64, "f32")
    x["beta"][0, 5:30] = 0.0
    x["beta"][0, 30:70] = 1.0
    x["beta"][0, 70:80] = 2.0
    x["k"][0, 32:60] = x["k"][0, 31]
    y = dev(x)
    o, s = forward(y, 1.0)
    args = [f64(x[k]) for k in ("q", "k", "v", "g", "beta")]
    ro, rs = oracle.delta(*args, state=f64(x["s0"]))
    close(o, ro, bars("f32", 64)[0], "o", 1)
    close(s, rs, bars("f32", 64)[1], "state", 1)
    got = rr.delta_chunkwise_bwd(*(y[k] for k in ("q", "k", "v", "g", "beta", "dout")), state_in=y["s0"],
                                 d_state_out=y["ds"])
    ref = oracle.delta_grad(*args, f64(x["dout"]), state=f64(x["s0"]), d_state=f64(x["ds"]))
    for i, (g, r) in enumerate(zip(got, ref)):
        close(g, r, bars("f32", 64)[2], str(i), 1)


def test_long_sequence_keeps_its_accuracy():
    """1500 tokens with hardly any decay: states and decay gradients at the same bars."""
    x = make(10, 1, 1500, 1, 1, 64, "bf16", decay=0.002)
    y = dev(x)
    o, s = forward(y, 0.125)
    args = [f64(x[k]) for k in ("q", "k", "v", "g", "beta")]
    ro, rs = oracle.delta(*args, scale=0.125, state=f64(x["s0"]))
    t_out, t_state, t_gate = bars("bf16", 64)
    close(o, ro, t_out, "o", 1)
    close(s, rs, t_state, "state", 1)
    got = rr.delta_chunkwise_bwd(*(y[k] for k in ("q", "k", "v", "g", "beta", "dout")), scale=0.125, state_in=y["s0"],
                                 d_state_out=y["ds"])
    ref = oracle.delta_grad(*args, f64(x["dout"]), scale=0.125, state=f64(x["s0"]), d_state=f64(x["ds"]))
    for name, g, r, t in zip(("dq", "dk", "dv", "dg", "dbeta", "ds"), got, ref, (t_out,) * 3 + (t_gate,) * 2 + (t_state,)):
        close(g, r, t, name, 1)


def test_nan_stays_in_its_sequence_and_goes_forward():
    """NaN in a token: later outputs of its columns are NaN, earlier blocks and other sequences and heads finite."""
    x = make(11, 2, 200, 2, 2, 64, "bf16")
    x["v"][0, 130, 1, 5] = float("nan")
    o, s = forward(dev(x), 1.0)
    o = o.cpu()
    assert torch.isfinite(o[1]).all() and torch.isfinite(o[0, :, 0]).all() and torch.isfinite(o[0, :128]).all()
    assert torch.isnan(o[0, 130:, 1, 5]).all()
    assert torch.isfinite(s[1]).all()


def test_same_bits_and_same_state_buffer():
    """Two runs agree bit for bit; state_out may be state_in."""
    x = dev(make(12, 2, 190, 2, 4, 128, "bf16"))
    o1, s1 = forward(x, 1.0)
    s = x["s0"].clone()
    o2 = rr.delta_chunkwise_fwd(x["q"], x["k"], x["v"], x["g"], x["beta"], state_in=s, state_out=s)
    assert torch.equal(o1, o2) and torch.equal(s1, s)
    a, b = (rr.delta_chunkwise_bwd(*(x[k] for k in ("q", "k", "v", "g", "beta", "dout")), state_in=x["s0"],
                                   d_state_out=x["ds"]) for _ in range(2))
    assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_graphs_and_streams():
    """Forward, backward and step captured and replayed on new inputs, each
    replay against the eager calls; a side stream; two workspaces at once."""
    x = dev(make(13, 1, 150, 1, 2, 64, "bf16"))
    ws_f = torch.empty(1 << 22, dtype=torch.uint8, device=DEV)
    ws_b = torch.empty(1 << 26, dtype=torch.uint8, device=DEV)
    keys = ("q", "k", "v", "g", "beta")
    step = {k: x[k][:, :1].contiguous() for k in keys}

    def run(state, wf=None, wb=None):
        s = torch.empty_like(x["s0"])
        o = rr.delta_chunkwise_fwd(*(x[k] for k in keys), state_in=x["s0"], state_out=s, workspace=wf)
        g = rr.delta_chunkwise_bwd(*(x[k] for k in keys), x["dout"], state_in=x["s0"], d_state_out=x["ds"], workspace=wb)
        state.copy_(s)
        return [o, s, *g, rr.delta_recurrent_step(*(step[k] for k in keys), state)]

    st_g, st_e = torch.empty_like(x["s0"]), torch.empty_like(x["s0"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run(st_g, ws_f, ws_b)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            outs = run(st_g, ws_f, ws_b)
    torch.cuda.current_stream().wait_stream(side)
    for seed in range(3):
        x["v"].copy_(torch.randn(x["v"].shape, generator=torch.Generator().manual_seed(seed)))
        graph.replay()
        torch.cuda.synchronize()
        eager = run(st_e)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, eager)) and torch.equal(st_g, st_e)
    with torch.cuda.stream(side):
        other = run(torch.empty_like(x["s0"]))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(other, eager))


def test_bad_packed_bounds_are_reported_and_stay_inside():
    """Bounds that run backwards, past the rows or past max_seqlen are clamped and told."""
    x = dev(make(14, 3, 100, 1, 1, 64, "bf16", lens=[60, 60, 60]))
    for cu in ([0, 100, 60, 180], [-5, 60, 120, 180], [0, 60, 120, 500], [0, 150, 160, 180]):
        c = torch.tensor(cu, dtype=torch.int32, device=DEV)
        with pytest.raises(rr.RetentionError) as e:
            rr.delta_chunkwise_fwd(*(x[k] for k in ("q", "k", "v", "g", "beta")), cu_seqlens=c, max_seqlen=100,
                                   check=True)
        assert e.value.word == 2
    good = torch.tensor([0, 60, 120, 180], dtype=torch.int32, device=DEV)
    rr.delta_chunkwise_fwd(*(x[k] for k in ("q", "k", "v", "g", "beta")), cu_seqlens=good, max_seqlen=60, check=True)


def test_binding_refusals():
    x = dev(make(15, 1, 70, 1, 2, 64, "bf16"))
    a = [x[k] for k in ("q", "k", "v", "g", "beta")]
    with pytest.raises(ValueError):
        rr.delta_chunkwise_fwd(a[0].transpose(1, 2), *a[1:])
    with pytest.raises(ValueError):
        rr.delta_chunkwise_fwd(a[0], a[1].float(), *a[2:])
    with pytest.raises(ValueError):
        rr.delta_chunkwise_fwd(*a[:3], a[3].bfloat16(), a[4])
    with pytest.raises(ValueError):
        rr.delta_chunkwise_fwd(*a[:3], a[3][:, :, :1].contiguous(), a[4])
    with pytest.raises(ValueError):
        rr.delta_chunkwise_fwd(*a, state_in=x["s0"][0])
    with pytest.raises(ValueError):
        rr.delta_chunkwise_fwd(*(t.cpu() for t in a))
    with pytest.raises(ValueError):
        rr.delta_chunkwise_fwd(*a, max_seqlen=70)
    with pytest.raises(rr.RetentionError):
        rr.delta_chunkwise_fwd(*a, out=a[2])
    with pytest.raises(rr.RetentionError):
        rr.delta_chunkwise_fwd(*a, workspace=torch.empty(64, dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError):
        rr.delta_recurrent_step(*a, x["s0"])
    with pytest.raises(TypeError):
        rr.delta_chunkwise_fwd(*(t.half() if i < 3 else t for i, t in enumerate(a)))


def test_offsets_past_32_bits():
    """The last of two packed sequences starts behind 2^31 elements of v: the
    same bits as that sequence alone."""
    h, d, first, last = 128, 256, 66000, 100
    g = torch.Generator(device=DEV).manual_seed(3)
    n = first + last
    assert first * h * d > 2 ** 31
    v = torch.randn(n, h, d, generator=g, device=DEV, dtype=torch.bfloat16)
    k = torch.randn(n, 1, d, generator=g, device=DEV, dtype=torch.bfloat16) / 16
    ld = -torch.rand(n, h, generator=g, device=DEV)
    beta = torch.rand(n, h, generator=g, device=DEV)
    cu = torch.tensor([0, first, n], dtype=torch.int32, device=DEV)
    s = torch.empty(2, h, d, d, device=DEV)
    o = rr.delta_chunkwise_fwd(k, k, v, ld, beta, state_out=s, cu_seqlens=cu, max_seqlen=first, check=True)
    tail = [t[first:][None].contiguous() for t in (k, k, v, ld, beta)]
    s1 = torch.empty(1, h, d, d, device=DEV)
    o1 = rr.delta_chunkwise_fwd(*tail, state_out=s1)
    assert torch.equal(o[first:], o1[0]) and torch.equal(s[1], s1[0])
    assert torch.isfinite(o[first - 64:first].float()).all()


def test_single_tokens_and_masked_batches():
    """One token a sequence, without and with a state; a batch whose padding
    has beta 0 and no decay leaves each state where its last real token did."""
    x = make(16, 3, 1, 1, 2, 64, "f32")
    y = dev(x)
    got = rr.delta_chunkwise_bwd(*(y[k] for k in ("q", "k", "v", "g", "beta", "dout")))
    assert (got[3] == 0).all()  # a first token's decay acts on nothing
    x = make(17, 2, 130, 1, 2, 64, "f32")
    x["beta"][0, 50:], x["g"][0, 50:] = 0.0, 0.0
    y = dev(x)
    _, s = forward(y, 1.0)
    short = {k: (t[:1, :50].contiguous() if t.dim() > 2 and k not in ("s0", "ds") else t[:1]) for k, t in y.items()}
    _, s50 = forward(short, 1.0)
    # the same products in another order of decays (factors of exactly 1)
    close(s[0], f64(s50[0]), bars("f32", 64)[1], "state", 2)


def test_gradient_of_a_reset_is_zero():
    """A factor that is 0 passes no gradient on, -infinity or not, in a block's
    middle and at its start; the others' gradients are the formula's."""
    x = make(18, 2, 200, 1, 2, 64, "f32")
    at = [0, 33, 64, 150]
    x["g"][:, at[:3]], x["g"][:, at[3]] = -np.inf, -150.0
    y = dev(x)
    names = ("q", "k", "v", "g", "beta", "dout")
    got = rr.delta_chunkwise_bwd(*(y[k] for k in names), state_in=y["s0"], d_state_out=y["ds"])
    assert (got[3][:, at] == 0).all() and torch.isfinite(got[3]).all()
    # the formula's, with a finite log decay whose factor is 0 in 64 bits too
    x["g"][:, at] = -1000.0
    ref = oracle.delta_grad(*(f64(x[k]) for k in names), state=f64(x["s0"]), d_state=f64(x["ds"]))
    assert (ref[3][:, at] == 0).all()
    bar = bars("f32", 64)[2]
    for what, a, r in zip(("dq", "dk", "dv", "dlog_decay", "dbeta", "d_state_in"), got, ref):
        close(a, r, bar, what, 2)


def test_two_streams_at_once():
    """Calls on two streams, each with its own tensors: the bits of calls in turn."""
    sets = [dev(make(20 + i, 2, 300, 2, 4, 128, "bf16")) for i in range(2)]
    names = ("q", "k", "v", "g", "beta")
    w = torch.ones(128, device=DEV)

    def run(y):
        s = y["s0"].clone()
        o = rr.delta_chunkwise_fwd(*(y[k] for k in names), state_in=s, state_out=s)
        n = rr.head_norm_fwd(o, w, y["v"], center=True)
        dx, dw, dg = rr.head_norm_bwd(o, y["dout"], w, y["v"], center=True)
        grads = rr.delta_chunkwise_bwd(*(y[k] for k in names), dx, state_in=y["s0"], d_state_out=y["ds"])
        return (o, s, n, dx, dw, dg, *grads)

    ref = [run(y) for y in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [[], []]
    for _ in range(4):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(run(sets[i]))
    torch.cuda.synchronize()
    for r, runs in zip(ref, got):
        for g in runs:
            assert all(torch.equal(a, b) for a, b in zip(r, g))
