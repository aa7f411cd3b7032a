"""The norms around a token mixer on the GPU against the fp64 oracle, element by
element. A value may be off by its own rounding (bf16 2^-8, fp32 2^-24 of it) and
by the fp32 arithmetic: a row's sums take at most 16 additions in a lane and 10
between lanes, the rest a dozen operations of 1 ulp, so 64 2^-24 of the
magnitude of its terms; weights' gradients add up to 64 rows in turn in a
workgroup, 64 such sums in a strand and 16 strands more: 256 2^-24."""

import numpy as np
import pytest
import torch

import retnet_retention_amd as rr
from oracle import delta_oracle
from oracle import norm_oracle as oracle

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
ROUND = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
WIDTHS = [1, 7, 64, 65, 128, 200, 256, 257, 512, 1000, 1024, 1031, 2048, 2560, 4096, 4100, 8192, 10001, 16384]


def f64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def near(got, ref, mag, own, fp, what):
    got = f64(got)
    assert got.shape == ref.shape and np.isfinite(got).all(), what
    bar = own * np.abs(ref) + fp * 2.0 ** -24 * mag + 1e-37
    worst = float((np.abs(got - ref) / bar).max()) if got.size else 0.0
    print(f"  {what}: {worst:.2f} of the bar", flush=True)
    assert worst <= 1, f"{what}: {worst}"


def make(seed, shape, dtype):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    w = shape[-1]
    t = {k: (r(*shape) * torch.exp(r(*shape[:-1], 1)) + 0.2).to(DT[dtype]) for k in ("x", "y")}
    t |= {k: r(*shape).to(DT[dtype]) for k in ("gate", "dout", "dres")}
    return t | {k: 1 + 0.3 * r(w) for k in ("w", "post", "scale")}


def dev(t):
    return {k: v.to(DEV) for k, v in t.items()}


@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("full", [False, True])
def test_head_norm(width, dtype, full):
    t = make(1, (5, 3, width), dtype)
    d = dev(t)
    n = {k: f64(v) for k, v in t.items()}
    w, g = (("w", "gate") if full else (None, None))
    args, dargs = [n.get(w), n.get(g)], [d.get(w), d.get(g)]
    ref = oracle.head_norm(n["x"], *args, center=full)
    mag = np.abs(ref) + np.abs(n["x"]).max(-1, keepdims=True) / np.abs(n["x"]).std(-1, keepdims=True).clip(1e-2) if full \
        else np.abs(ref)
    near(rr.head_norm_fwd(d["x"], *dargs, center=full), ref, mag, ROUND[dtype], 64, "out")
    got = rr.head_norm_bwd(d["x"], d["dout"], *dargs, center=full)
    grads = oracle.head_norm_grad(n["x"], n["dout"], *args, center=full)
    for name, v in zip(("dx", "dweight", "dgate"), got):
        assert (v is None) == (name not in grads)
        if v is not None:
            ref, m = grads[name]
            near(v, ref, m, 2.0 ** -24 if name == "dweight" else ROUND[dtype], 256, name)


@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("full", [False, True])
def test_residual_norm(width, dtype, full):
    t = make(2, (11, width), dtype)
    d = dev(t)
    n = {k: f64(v) for k, v in t.items()}
    kw = dict(skip=0.75, center=full)
    dk = dict(kw, **({"post_weight": d["post"], "scale": d["scale"]} if full else {}))
    nk = dict(kw, **({"post": n["post"], "scale": n["scale"]} if full else {}))
    ro, rh = oracle.residual_norm(n["x"], n["y"], n["w"], **nk)
    out, res = rr.residual_norm_fwd(d["x"], d["y"], d["w"], **dk)
    spread = 1 + np.abs(rh).max(-1, keepdims=True) / np.maximum(rh.std(-1, keepdims=True), 1e-2)
    near(res, rh, np.abs(n["x"]) + np.abs(rh) + 4, ROUND[dtype], 64, "residual")
    near(out, ro, np.abs(ro) + np.abs(n["w"]) * spread * 4, ROUND[dtype], 64, "out")
    x = d["x"].clone()
    o2, r2 = rr.residual_norm_fwd(x, d["y"], d["w"], residual=x, **dk)
    assert torch.equal(o2, out) and torch.equal(x, res) and r2 is x
    for dres in (None, "dres"):
        got = rr.residual_norm_bwd(d["x"], d["y"], d["w"], d["dout"], d.get(dres), **dk)
        grads = oracle.residual_norm_grad(n["x"], n["y"], n["w"], n["dout"], n.get(dres), **nk)
        for name, v in zip(("dx", "dy", "dweight", "dpost", "dscale"), got):
            assert (v is None) == (name not in grads)
            if v is not None:
                ref, m = grads[name]
                near(v, ref, m, ROUND[dtype] if name in ("dx", "dy") else 2.0 ** -24, 256 * (4 if full else 1), name)


@pytest.mark.parametrize("rows,width,dtype", [(20000, 256, "bf16"), (3001, 4096, "bf16"), (40001, 64, "f32"), (0, 128, "f32"),
                                              (1, 16384, "bf16")])
def test_weight_gradients_over_many_rows(rows, width, dtype):
    t = make(3, (rows, width), dtype)
    d = dev(t)
    n = {k: f64(v) for k, v in t.items()}
    got = rr.residual_norm_bwd(d["x"], d["y"], d["w"], d["dout"], d["dres"], post_weight=d["post"], scale=d["scale"])
    grads = oracle.residual_norm_grad(n["x"], n["y"], n["w"], n["dout"], n["dres"], post=n["post"], scale=n["scale"])
    for name, v in zip(("dx", "dy", "dweight", "dpost", "dscale"), got):
        ref, m = grads[name]
        near(v, ref, m, ROUND[dtype] if name in ("dx", "dy") else 2.0 ** -24, 1024, name)
    again = rr.residual_norm_bwd(d["x"], d["y"], d["w"], d["dout"], d["dres"], post_weight=d["post"], scale=d["scale"])
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    got = rr.head_norm_bwd(d["x"], d["dout"], d["w"], d["gate"], center=True)
    grads = oracle.head_norm_grad(n["x"], n["dout"], n["w"], n["gate"], center=True)
    near(got[1], *grads["dweight"], 2.0 ** -24, 1024, "head dweight")


def test_rows_of_zeros_and_extremes():
    """A row of zeros stays zero (eps), huge rows do not overflow below 2^63, a
    NaN stays in its row and the weights' gradients."""
    x = torch.zeros(4, 256)
    x[1] = 1e18
    x[2, 5] = float("nan")
    x[3] = torch.linspace(-1, 1, 256)
    y = rr.head_norm_fwd(x.to(DEV)).cpu()
    assert (y[0] == 0).all() and torch.isnan(y[2]).all()
    torch.testing.assert_close(y[1], torch.ones(256), rtol=1e-6, atol=0)
    assert torch.isfinite(y[3]).all()
    gate = torch.full((4, 256), -1e30)
    z = rr.head_norm_fwd(x.to(DEV), gate=gate.to(DEV)).cpu()
    assert (z[0] == 0).all() and (z[3] == 0).all()


def test_norm_equals_the_retention_epilogue():
    """Raw retention, then the centred head norm and gate: the fused epilogue's result."""
    g = torch.Generator().manual_seed(4)
    q, k, v, gate = (torch.randn(1, 130, 2, 64, generator=g).to(DEV) / 8 for _ in range(4))
    fused = rr.chunkwise_fwd(q, k, v, gate, chunk=64)
    raw = rr.chunkwise_fwd(q, k, v, chunk=64)
    torch.testing.assert_close(rr.head_norm_fwd(raw, gate=gate, center=True), fused, rtol=1e-4, atol=1e-5)


def test_mixer_block_with_gradients():
    """The operators together as a layer's step uses them: residual join, unit
    keys, delta rule, gated norm, forward and backward by hand against fp64."""
    b, n, h, d = 2, 150, 2, 64
    g = torch.Generator().manual_seed(5)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x, y = r(b, n, h * d), r(b, n, h * d)
    w, w_h, unit = 1 + 0.1 * r(h * d), 1 + 0.1 * r(d), torch.full((d,), d ** -0.5)
    v, gate, dout, dres = r(b, n, h, d), r(b, n, h, d), r(b, n, h, d), r(b, n, h * d)
    ld, beta = -0.1 * torch.rand(b, n, h, generator=g), torch.rand(b, n, h, generator=g)
    t = [a.to(DEV) for a in (x, y, w, w_h, unit, v, gate, dout, dres, ld, beta)]
    X, Y, W, WH, U, V, G, DO, DR, LD, BE = t
    out, res = rr.residual_norm_fwd(X, Y, W)
    heads = out.view(b, n, h, d)
    key = rr.head_norm_fwd(heads, U)
    o = rr.delta_chunkwise_fwd(key, key, V, LD, BE)
    z = rr.head_norm_fwd(o, WH, G)
    do, dwh, dgate = rr.head_norm_bwd(o, DO, WH, G)
    dq, dk, dv, dld, dbe = rr.delta_chunkwise_bwd(key, key, V, LD, BE, do)
    dheads, _, _ = rr.head_norm_bwd(heads, dq + dk, U)
    dx, dy, dw, _, _ = rr.residual_norm_bwd(X, Y, W, dheads.view(b, n, h * d), DR)

    N = {k: f64(a) for k, a in zip("x y w wh u v gate dout dres ld be".split(), t)}
    no, nres = oracle.residual_norm(N["x"], N["y"], N["w"])
    nh = no.reshape(b, n, h, d)
    nk = oracle.head_norm(nh, N["u"])
    nd, _ = delta_oracle.delta(nk, nk, N["v"], N["ld"], N["be"])
    nz = oracle.head_norm(nd, N["wh"], N["gate"])
    gh = oracle.head_norm_grad(nd, N["dout"], N["wh"], N["gate"])
    gd = delta_oracle.delta_grad(nk, nk, N["v"], N["ld"], N["be"], gh["dx"][0])
    gk = oracle.head_norm_grad(nh, gd[0] + gd[1], N["u"])
    gr = oracle.residual_norm_grad(N["x"], N["y"], N["w"], gk["dx"][0].reshape(b, n, h * d), N["dres"])
    # fp32 throughout: four operators each within 1e-5 of their inputs' gradient norms
    for name, a, ref in (("z", z, nz), ("res", res, nres), ("dgate", dgate, gh["dgate"][0]), ("dwh", dwh, gh["dweight"][0]),
                         ("dv", dv, gd[2]), ("dld", dld, gd[3]), ("dbe", dbe, gd[4]), ("dx", dx, gr["dx"][0]),
                         ("dy", dy, gr["dy"][0]), ("dw", dw, gr["dweight"][0])):
        err = np.linalg.norm(f64(a) - ref) / np.linalg.norm(ref)
        print(f"  {name}: {err:.2e}", flush=True)
        assert err <= 4e-5, name


def test_graph_replays():
    t = dev(make(6, (40, 513), "bf16"))
    ws = torch.empty(1 << 20, dtype=torch.uint8, device=DEV)
    run = lambda w=None: [*rr.residual_norm_fwd(t["x"], t["y"], t["w"], post_weight=t["post"]),  # noqa: E731
                          *[g for g in rr.residual_norm_bwd(t["x"], t["y"], t["w"], t["dout"], post_weight=t["post"],
                                                            workspace=w) if g is not None],
                          *[g for g in rr.head_norm_bwd(t["x"], t["dout"], t["w"], t["gate"]) if g is not None]]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run(ws)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            outs = run(ws)
    torch.cuda.current_stream().wait_stream(side)
    for seed in range(3):
        t["x"].copy_(torch.randn(t["x"].shape, generator=torch.Generator().manual_seed(seed)))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, run()))


def test_binding_refusals():
    t = dev(make(7, (4, 64), "bf16"))
    with pytest.raises(ValueError):
        rr.head_norm_fwd(t["x"].t())
    with pytest.raises(ValueError):
        rr.head_norm_fwd(t["x"], t["w"].bfloat16())
    with pytest.raises(ValueError):
        rr.head_norm_fwd(t["x"], None, t["gate"][:2].contiguous())
    with pytest.raises(ValueError):
        rr.residual_norm_fwd(t["x"], t["y"].float(), t["w"])
    with pytest.raises(ValueError):
        rr.residual_norm_fwd(t["x"].cpu(), t["y"], t["w"])
    with pytest.raises(rr.RetentionError):
        rr.residual_norm_fwd(t["x"], t["y"], t["w"], out=t["y"])
    with pytest.raises(rr.RetentionError):
        rr.head_norm_fwd(t["x"], eps=0.0)
    with pytest.raises(TypeError):
        rr.head_norm_fwd(t["x"].half())


def test_offsets_past_32_bits():
    """Rows behind 2^31 elements: the same bits as those rows alone."""
    rows, width = 131200, 16384
    assert (rows - 64) * width > 2 ** 31
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randn(rows, width, generator=g, device=DEV, dtype=torch.bfloat16)
    w = torch.ones(width, device=DEV)
    out, res = rr.residual_norm_fwd(x, x, w)
    o2, r2 = rr.residual_norm_fwd(x[-64:].contiguous(), x[-64:].contiguous(), w)
    assert torch.equal(out[-64:], o2) and torch.equal(res[-64:], r2)
    y = rr.head_norm_fwd(x, w)
    assert torch.equal(y[-64:], rr.head_norm_fwd(x[-64:].contiguous(), w))


def test_more_rows_than_one_line_of_workgroups():
    """2^29 rows of one value take 2^32 lanes: the same bits as those rows alone."""
    rows = 2 ** 29 + 100
    x = torch.randn(rows, 1, generator=torch.Generator(device=DEV).manual_seed(2), device=DEV, dtype=torch.bfloat16)
    y = rr.head_norm_fwd(x)
    for at in (0, 2 ** 26 - 64, 2 ** 29 - 64, rows - 128):
        assert torch.equal(y[at:at + 128], rr.head_norm_fwd(x[at:at + 128].clone())), at
