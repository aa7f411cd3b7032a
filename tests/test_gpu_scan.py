"""The gated linear recurrence and the short convolution on the GPU against the
fp64 oracle (token by token).

Tolerances, relative norms over channels.
- fp32 results of n tokens: a token's factor and its sum are off by 2^-24 of the
  state each, its input by some 2^-20 (sigmoids and root by hardware functions of
  about an ulp, their arguments' rounding), and what earlier tokens left adds up over at
  most n of them: FWD(n) = (2 n + 16) 2^-24. Gradients sum two terms that each take the
  error of a state and of a gradient: GRAD(n) = 4 FWD(n). A rate's gradient sums n terms
  of either sign, sqrt(n) times a single one's size where their errors may add to n times
  it: sqrt(n) GRAD(n) more.
- bf16 results: against the oracle's value rounded once, as two roundings differ only
  where a border lies between the values: sqrt(d 2^-7) for a value off by d before."""

import numpy as np
import pytest
import torch

import retnet_retention_amd as rr
from oracle import scan_oracle as oracle

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def f64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def fwd_bar(n):
    return (2 * n + 16) * 2.0 ** -24


def near(got, ref, bar, what):
    """Relative norm of all, and of each channel against the largest channel's size / 10."""
    assert tuple(got.shape) == tuple(ref.shape), what
    if got.dtype == torch.bfloat16:
        ref, bar = torch.from_numpy(np.ascontiguousarray(ref)).bfloat16().double().numpy(), (bar * 2.0 ** -7) ** 0.5
    got = f64(got)
    assert np.isfinite(got).all(), what
    if not got.size:
        return
    g, r = (np.moveaxis(t, -1, 0).reshape(t.shape[-1], -1) for t in (got, ref))
    err, size = np.linalg.norm(g - r, axis=1), np.linalg.norm(r, axis=1)
    whole = np.linalg.norm(err) / max(np.linalg.norm(size), 1e-30)
    worst = (err / np.maximum(size, 0.1 * size.max() + 1e-30)).max()
    # a channel of a few bf16 values may have all its borders crossed: one rounding of each
    most = max(10 * bar, 2.0 ** -8) if bar > 1e-5 else 10 * bar
    print(f"  {what}: {whole:.2e}, worst channel {worst:.2e} (bar {bar:.2e})", flush=True)
    assert whole <= bar and worst <= most, f"{what}: {whole:.3e}, {worst:.3e} > {bar:.3e}"


def scan_inputs(seed, rows, w, dtype, form, gate=True, state=None, rate=None):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x = {"x": r(*rows, w).to(DT[dtype]), "dout": r(*rows, w).to(DT[dtype]), "rate": None,
         "gate": r(*rows, w).to(DT[dtype]) if gate else None,
         "s0": r(state, w) if state else None, "ds": r(state, w) if state else None}
    rates = torch.exp(-7 + 6.5 * torch.rand(w, generator=g)) if rate is None else torch.full((w,), rate)
    if form == "gates":
        x["rate"], x["decay"] = rates, r(*rows, w).to(DT[dtype])
    else:
        x["decay"] = -rates * torch.nn.functional.softplus(r(*rows, w))
    return x


def dev(x):
    return {k: None if t is None else t.to(DEV) for k, t in x.items()}


def run_scan(y, normalize, keep=True, **kw):
    """Forward and backward: dict of outputs."""
    gates = dict(rate=y["rate"], normalize=normalize, state_in=y["s0"], **kw)
    s = None if y["s0"] is None else torch.full_like(y["s0"], float("nan"))
    o = rr.gated_scan_fwd(y["x"], y["decay"], y["gate"], state_out=s, keep=keep, **gates)
    o, kept = o if keep else (o, None)
    g = rr.gated_scan_bwd(y["x"], y["decay"], y["dout"], y["gate"], d_state_out=y["ds"], kept=kept, **gates)
    out = dict(zip(("dx", "ddecay", "dgate", "drate"), g), o=o)
    if s is not None:
        out.update(state=s, dstate=g[4])
    return out


def scan_reference(x, normalize, lens=None):
    a = {k: f64(t) for k, t in x.items()}
    rest = (a["rate"], normalize)
    if lens is None:
        o, s = oracle.scan(a["x"], a["decay"], a["gate"], *rest, a["s0"])
        g = oracle.scan_grad(a["x"], a["decay"], a["dout"], a["gate"], *rest, a["s0"], a["ds"])
    else:
        fs = oracle.packed(oracle.scan, lens, (a["x"], a["decay"], a["gate"]), rest, (a["s0"],))
        gs = oracle.packed(oracle.scan_grad, lens, (a["x"], a["decay"], a["dout"], a["gate"]), rest, (a["s0"], a["ds"]))
        o, s = np.concatenate([f[0][0] for f in fs]), np.concatenate([f[1] for f in fs])
        join = lambda i: None if gs[0][i] is None else np.concatenate([g[i][0] for g in gs])  # noqa: E731
        g = (join(0), join(1), join(2), None if gs[0][3] is None else sum(g[3] for g in gs),
             np.concatenate([g[4] for g in gs]))
    return dict(o=o, state=s, dx=g[0], ddecay=g[1], dgate=g[2], drate=g[3], dstate=g[4])


def check_scan(got, ref, n, tokens):
    for k in got:
        if got[k] is None:
            assert ref[k] is None, k
            continue
        bar = fwd_bar(n) * (1 if k in ("o", "state") else 4)
        near(got[k], ref[k], bar * (1 + tokens ** 0.5) if k == "drate" else bar, k)


FORMS = [("gates", True, True), ("gates", False, False), ("gates", True, False), ("gates", False, True),
         ("log", False, False), ("log", True, True), ("log", True, False), ("log", False, True)]


@pytest.mark.parametrize("form,gate,normalize", FORMS)
@pytest.mark.parametrize("dtype,w", [("bf16", 130), ("bf16", 67), ("f32", 65)])
def test_scan_forms(form, gate, normalize, dtype, w):
    x = scan_inputs(1, (2, 300), w, dtype, form, gate, state=2)
    check_scan(run_scan(dev(x), normalize), scan_reference(x, normalize), 300, 600)


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 127, 128, 129, 256, 257, 511, 513, 1025, 2500])
@pytest.mark.parametrize("dtype,w,state", [("bf16", 2, None), ("bf16", 1, 3), ("f32", 64, 3)])
def test_scan_lengths(n, dtype, w, state):
    x = scan_inputs(2, (3, n), w, dtype, "gates", state=state)
    check_scan(run_scan(dev(x), True), scan_reference(x, True), n, 3 * n)


@pytest.mark.parametrize("lens", [[5], [0, 0, 3], [130, 0, 1, 66, 128, 0], [1] * 70, [900, 1, 0, 257, 3, 600, 0]])
@pytest.mark.parametrize("dtype,form", [("bf16", "gates"), ("f32", "log")])
def test_scan_packed(lens, dtype, form):
    x = scan_inputs(3, (sum(lens),), 66, dtype, form, state=len(lens))
    cu = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32, device=DEV)
    check_scan(run_scan(dev(x), True, cu_seqlens=cu, check=True), scan_reference(x, True, lens), max(lens), sum(lens))


def test_scan_packed_without_tokens():
    x = dev(scan_inputs(4, (0,), 40, "bf16", "gates", state=3))
    cu = torch.zeros(4, dtype=torch.int32, device=DEV)
    got = run_scan(x, True, cu_seqlens=cu, check=True)
    assert torch.equal(got["state"], x["s0"]) and torch.equal(got["dstate"], x["ds"]) and (got["drate"] == 0).all()


def test_scan_rows_outside_sequences():
    """Left as they were by the forward, gradients of zero; a middle of the tensor, many rows around it."""
    x = dev(scan_inputs(5, (700,), 66, "bf16", "gates", state=2))
    cu = torch.tensor([300, 310, 390], dtype=torch.int32, device=DEV)
    out = torch.full_like(x["x"], 7.0)
    s = torch.empty_like(x["s0"])
    rr.gated_scan_fwd(x["x"], x["decay"], x["gate"], rate=x["rate"], state_in=x["s0"], state_out=s, cu_seqlens=cu, out=out,
                      check=True)
    part = {k: t[300:390].contiguous() if k in ("x", "decay", "gate", "dout") else t for k, t in x.items()}
    got = run_scan(part, False, cu_seqlens=cu - 300)
    assert (out[:300] == 7).all() and (out[390:] == 7).all() and torch.equal(out[300:390], got["o"])
    assert torch.equal(s, got["state"])
    g = rr.gated_scan_bwd(x["x"], x["decay"], x["dout"], x["gate"], rate=x["rate"], state_in=x["s0"], d_state_out=x["ds"],
                          cu_seqlens=cu)
    for t, name in zip(g[:3], ("dx", "ddecay", "dgate")):
        assert (t[:300] == 0).all() and (t[390:] == 0).all() and torch.equal(t[300:390], got[name]), name
    assert torch.equal(g[3], got["drate"]) and torch.equal(g[4], got["dstate"])


@pytest.mark.parametrize("cu", [[0, 500, 90], [-5, 20, 90], [0, 95, 95], [80, 20, 400], [2**31 - 1, 0, -2**31]])
def test_bad_bounds_are_told(cu):
    """Nothing outside the tensors is touched, and the control word tells of them."""
    x = dev(scan_inputs(6, (90,), 66, "bf16", "gates", state=2))
    cu = torch.tensor(cu, dtype=torch.int32, device=DEV)
    guard = torch.full((290, 66), 3.0, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(rr.RetentionError) as e:
        rr.gated_scan_fwd(x["x"], x["decay"], x["gate"], rate=x["rate"], cu_seqlens=cu, out=guard[100:190], check=True)
    assert e.value.word == 2
    assert (guard[:100] == 3).all() and (guard[190:] == 3).all()
    with pytest.raises(rr.RetentionError):
        rr.gated_scan_bwd(x["x"], x["decay"], x["dout"], x["gate"], rate=x["rate"], cu_seqlens=cu, check=True)
    w = torch.ones(66, 4, device=DEV)
    with pytest.raises(rr.RetentionError):
        rr.short_conv_fwd(x["x"], w, cu_seqlens=cu, out=guard[100:190], check=True)
    assert (guard[:100] == 3).all() and (guard[190:] == 3).all()
    with pytest.raises(rr.RetentionError):
        rr.short_conv_bwd(x["x"], w, x["dout"], cu_seqlens=cu, check=True)


@pytest.mark.parametrize("fill", [float("nan"), float("inf")])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_factor_of_zero_forgets(fill, dtype):
    """At a first token and later ones, forward and backward, whatever the state or a token before it was."""
    x = scan_inputs(7, (2, 400), 66, dtype, "log", state=2)
    x["decay"][:, 0] = -np.inf
    x["decay"][:, 200] = -1e30
    a = dev(x)
    b = dict(a, s0=torch.full_like(a["s0"], fill))
    ga, gb = run_scan(a, True), run_scan(b, True)
    for k in ga:
        assert ga[k] is None or torch.equal(ga[k], gb[k]), k
    assert (ga["dstate"] == 0).all() and (ga["ddecay"][:, 0] == 0).all() and (ga["ddecay"][:, 200] == 0).all()
    c = dict(a, x=a["x"].clone())
    c["x"][:, 190] = fill
    gc = run_scan(c, True)
    assert torch.equal(gc["o"][:, :190], ga["o"][:, :190]) and torch.equal(gc["o"][:, 200:], ga["o"][:, 200:])
    assert not torch.isfinite(gc["o"][:, 190:200].float()).any() and torch.equal(gc["state"], ga["state"])
    # loud gradients behind a token that forgets do not reach what stands before it
    d = dict(a, dout=a["dout"].clone())
    d["dout"][:, 300] = fill
    gd = run_scan(d, True)
    assert torch.equal(gd["dx"][:, :200], ga["dx"][:, :200]) and torch.equal(gd["ddecay"][:, :200], ga["ddecay"][:, :200])


@pytest.mark.parametrize("rate", [1e-6, 1e-3, 0.3, 20.0, 300.0])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_scan_rates(rate, dtype):
    """Channels that hardly forget up to those that forget within a token."""
    x = scan_inputs(8, (2, 333), 65, dtype, "gates", state=2, rate=rate)
    check_scan(run_scan(dev(x), True), scan_reference(x, True), 333, 666)


def test_log_decays_of_zero():
    """A factor of 1: nothing forgotten; with normalize nothing written, and finite gradients."""
    x = scan_inputs(9, (1, 200), 66, "f32", "log", state=1)
    x["decay"][:, 50:150] = 0.0
    for normalize in (False, True):
        check_scan(run_scan(dev(x), normalize), scan_reference(x, normalize), 200, 200)


def test_a_token_without_number_stays_in_its_sequence():
    lens = [40, 70, 30]
    x = dev(scan_inputs(10, (sum(lens),), 66, "bf16", "gates", state=3))
    cu = torch.tensor([0, 40, 110, 140], dtype=torch.int32, device=DEV)
    ref = run_scan(x, True, cu_seqlens=cu)
    y = dict(x, x=x["x"].clone())
    y["x"][60] = float("nan")
    got = run_scan(y, True, cu_seqlens=cu)
    for k in ("o", "dx", "ddecay", "dgate"):
        assert torch.equal(got[k][:40], ref[k][:40]) and torch.equal(got[k][110:], ref[k][110:]), k
    assert torch.equal(got["o"][:60], ref["o"][:60]) and torch.isnan(got["o"][60:110].float()).all()
    assert torch.equal(got["state"][[0, 2]], ref["state"][[0, 2]])


def test_scan_keeps_or_runs_again_the_same_bits():
    for dtype, form in (("bf16", "gates"), ("f32", "log")):
        x = dev(scan_inputs(11, (2, 700), 66, dtype, form, state=2))
        a, b = run_scan(x, True), run_scan(x, True, keep=False)
        c = run_scan(x, True)
        for k in a:
            assert a[k] is None or (torch.equal(a[k], b[k]) and torch.equal(a[k], c[k])), k


def test_scan_in_place_state_and_pieces():
    """A sequence in pieces with the state in place is the whole one."""
    x = dev(scan_inputs(12, (2, 900), 130, "f32", "gates", state=2))
    whole = run_scan(x, True)
    s, outs = x["s0"].clone(), []
    for a, b in ((0, 1), (1, 130), (130, 600), (600, 900)):
        cut = {k: x[k][:, a:b].contiguous() for k in ("x", "decay", "gate")}
        outs.append(rr.gated_scan_fwd(cut["x"], cut["decay"], cut["gate"], rate=x["rate"], normalize=True, state_in=s,
                                      state_out=s))
    near(torch.cat(outs, 1), f64(whole["o"]), fwd_bar(900), "o")
    near(s, f64(whole["state"]), fwd_bar(900), "state")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("at", [0, 8, 80])
def test_columns_of_a_wider_projection(dtype, at):
    """x, decay and gate out of one tensor, rows that stand apart: the bits of dense copies."""
    wide = torch.randn(2, 150, 3 * 80 + 5, generator=torch.Generator().manual_seed(13)).to(DT[dtype]).to(DEV)
    parts = [wide[..., a:a + 64] for a in (at, (at + 80) % 240, (at + 160) % 240)]
    rate = torch.full((64,), 0.1, device=DEV)
    a = rr.gated_scan_fwd(*parts[:2], parts[2], rate=rate)
    b = rr.gated_scan_fwd(*(t.contiguous() for t in parts), rate=rate)
    assert torch.equal(a, b)
    for ga, gb in zip(rr.gated_scan_bwd(*parts[:2], a, parts[2], rate=rate),
                      rr.gated_scan_bwd(*(t.contiguous() for t in parts[:2]), a, parts[2].contiguous(), rate=rate)):
        assert torch.equal(ga, gb)
    w = torch.randn(64, 4, device=DEV)
    assert torch.equal(rr.short_conv_fwd(parts[0], w), rr.short_conv_fwd(parts[0].contiguous(), w))
    for ga, gb in zip(rr.short_conv_bwd(parts[0], w, a)[:2], rr.short_conv_bwd(parts[0].contiguous(), w, a)[:2]):
        assert torch.equal(ga, gb)
    s = torch.randn(2, 64, device=DEV)
    t = s.clone()
    one = [p[:, 3:4] for p in parts]
    assert torch.equal(rr.gated_scan_step(one[0], one[1], s, one[2], rate=rate),
                       rr.gated_scan_step(*(p.contiguous() for p in one[:2]), t, one[2].contiguous(), rate=rate))
    assert torch.equal(s, t)


@pytest.mark.parametrize("form,gate,normalize", FORMS)
@pytest.mark.parametrize("dtype,w", [("bf16", 700), ("bf16", 33), ("f32", 65)])
def test_scan_step(form, gate, normalize, dtype, w):
    """Steps of a pool: the oracle's, idle sequences and slots left alone."""
    x = scan_inputs(14, (5, 1), w, dtype, form, gate)
    pool = torch.randn(8, w, generator=torch.Generator().manual_seed(15))
    slots = [6, -1, 2, 6, 8]  # -1 and 8 are outside, the second 6 is taken
    y, p = dev(x), pool.to(DEV)
    o = rr.gated_scan_step(y["x"], y["decay"], p, y["gate"], rate=y["rate"], normalize=normalize,
                           slots=torch.tensor(slots, dtype=torch.int32, device=DEV))
    a = {k: f64(t) for k, t in x.items()}
    for i, slot in ((0, 6), (2, 2)):
        pick = lambda t: None if t is None else t[i:i + 1]  # noqa: E731
        ro, rs = oracle.scan(pick(a["x"]), pick(a["decay"]), pick(a["gate"]), a["rate"], normalize, f64(pool[slot:slot + 1]))
        near(o[i:i + 1], ro, fwd_bar(1), "o")
        near(p[slot:slot + 1], rs, fwd_bar(1), "state")
    assert (o[[1, 3, 4]] == 0).all()
    rest = [i for i in range(8) if i not in (6, 2)]
    assert torch.equal(p.cpu()[rest], pool[rest])


def test_steps_follow_a_prefill():
    """One token after another gives what the sequence gives."""
    x = dev(scan_inputs(16, (2, 40), 66, "f32", "gates", state=2))
    whole = run_scan(x, True)
    s = x["s0"].clone()
    for t in range(40):
        part = [x[k][:, t:t + 1] for k in ("x", "decay", "gate")]
        o = rr.gated_scan_step(part[0], part[1], s, part[2], rate=x["rate"], normalize=True)
        near(o[:, 0], f64(whole["o"][:, t]), fwd_bar(40), f"o {t}")
    near(s, f64(whole["state"]), fwd_bar(40), "state")


def test_a_step_that_forgets_clears_its_slot():
    x = dev(scan_inputs(17, (2, 1), 66, "bf16", "log"))
    x["decay"][0] = -np.inf
    pool = torch.full((2, 66), float("nan"), device=DEV)
    o = rr.gated_scan_step(x["x"], x["decay"], pool, x["gate"])
    assert torch.isfinite(o[0].float()).all() and torch.isfinite(pool[0]).all() and torch.isnan(pool[1]).all()


# ------------------------------------------------------------------ convolution
# fp32 sums of 4 products and a bias, the sigmoid: 16 2^-24 of their terms, which may
# cancel to a tenth of themselves over a channel; bf16: rounded once.
CONV = 160 * 2.0 ** -24


def conv_inputs(seed, rows, w, taps, dtype, bias=True, state=None):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    return {"x": r(*rows, w).to(DT[dtype]), "weight": r(w, taps), "bias": r(w) if bias else None,
            "dout": r(*rows, w).to(DT[dtype]), "s0": r(state, taps - 1, w).to(DT[dtype]) if state else None,
            "ds": r(state, taps - 1, w).to(DT[dtype]) if state else None}


def run_conv(y, swish, **kw):
    s = None if y["s0"] is None else torch.full_like(y["s0"], float("nan"))
    o = rr.short_conv_fwd(y["x"], y["weight"], y["bias"], swish=swish, state_in=y["s0"], state_out=s, **kw)
    g = rr.short_conv_bwd(y["x"], y["weight"], y["dout"], y["bias"], swish=swish, state_in=y["s0"], d_state_out=y["ds"], **kw)
    out = dict(zip(("dx", "dweight", "dbias"), g), o=o)
    if s is not None:
        out.update(state=s, dstate=g[3])
    return out


def check_conv(got, x, swish, lens=None):
    a = {k: f64(t) for k, t in x.items()}
    lens = lens if lens is not None else [None]
    if lens == [None]:
        o, s = oracle.conv(a["x"], a["weight"], a["bias"], swish, a["s0"])
        g = oracle.conv_grad(a["x"], a["weight"], a["dout"], a["bias"], swish, a["s0"], a["ds"])
    else:
        fs, gs, at = [], [], 0
        for i, n in enumerate(lens):
            part = lambda k: a[k][None, at:at + n]  # noqa: E731
            held = lambda k: None if a[k] is None else a[k][i:i + 1]  # noqa: E731
            fs.append(oracle.conv(part("x"), a["weight"], a["bias"], swish, held("s0")))
            gs.append(oracle.conv_grad(part("x"), a["weight"], part("dout"), a["bias"], swish, held("s0"), held("ds")))
            at += n
        o, s = np.concatenate([f[0][0] for f in fs]), np.concatenate([f[1] for f in fs])
        g = (np.concatenate([t[0][0] for t in gs]), sum(t[1] for t in gs),
             None if a["bias"] is None else sum(t[2] for t in gs), np.concatenate([t[3] for t in gs]))
    tokens = int(np.prod(x["x"].shape[:-1]))
    ref = dict(o=o, state=s, dx=g[0], dweight=g[1].T, dbias=g[2], dstate=g[3])
    got = dict(got, dweight=got["dweight"].t())
    for k in got:
        if got[k] is None:
            assert ref[k] is None, k
        else:
            near(got[k], ref[k], CONV * (1 + tokens ** 0.5) if k in ("dweight", "dbias") else CONV, k)


@pytest.mark.parametrize("taps", [2, 3, 4])
@pytest.mark.parametrize("swish,bias", [(True, True), (False, False), (True, False), (False, True)])
@pytest.mark.parametrize("dtype,w", [("bf16", 130), ("bf16", 67), ("f32", 65)])
def test_conv_forms(taps, swish, bias, dtype, w):
    x = conv_inputs(21, (2, 150), w, taps, dtype, bias, state=2)
    check_conv(run_conv(dev(x), swish), x, swish)


@pytest.mark.parametrize("n", [1, 2, 3, 4, 5, 31, 32, 33, 127, 128, 129, 131, 257, 700])
@pytest.mark.parametrize("dtype,w,state", [("bf16", 2, None), ("bf16", 1, 2), ("f32", 64, 2)])
def test_conv_lengths(n, dtype, w, state):
    for taps in (2, 4):
        x = conv_inputs(22, (2, n), w, taps, dtype, state=state)
        check_conv(run_conv(dev(x), True), x, True)


@pytest.mark.parametrize("lens", [[5], [0, 0, 3], [130, 0, 1, 2, 66, 128, 0], [1] * 70, [900, 1, 0, 257, 3, 600, 0]])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_conv_packed(lens, dtype):
    x = conv_inputs(23, (sum(lens),), 66, 4, dtype, state=len(lens))
    cu = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32, device=DEV)
    check_conv(run_conv(dev(x), True, cu_seqlens=cu, check=True), x, True, lens)


def test_conv_rows_outside_sequences():
    x = dev(conv_inputs(24, (700,), 66, 4, "bf16", state=2))
    cu = torch.tensor([300, 310, 390], dtype=torch.int32, device=DEV)
    out = torch.full_like(x["x"], 7.0)
    rr.short_conv_fwd(x["x"], x["weight"], state_in=x["s0"], cu_seqlens=cu, out=out, check=True)
    part = dict(x, x=x["x"][300:390].contiguous(), dout=x["dout"][300:390].contiguous(), bias=None)
    got = run_conv(part, False, cu_seqlens=cu - 300)
    assert (out[:300] == 7).all() and (out[390:] == 7).all() and torch.equal(out[300:390], got["o"])
    g = rr.short_conv_bwd(x["x"], x["weight"], x["dout"], state_in=x["s0"], d_state_out=x["ds"], cu_seqlens=cu)
    assert (g[0][:300] == 0).all() and (g[0][390:] == 0).all() and torch.equal(g[0][300:390], got["dx"])
    near(g[1], f64(got["dweight"]), CONV * 10, "dweight")
    assert torch.equal(g[3], got["dstate"])


@pytest.mark.parametrize("taps", [2, 3, 4])
@pytest.mark.parametrize("dtype,w", [("bf16", 700), ("bf16", 33), ("f32", 65)])
def test_conv_step(taps, dtype, w):
    """Steps of a pool against the oracle; then token by token against the whole."""
    x = conv_inputs(25, (5, 1), w, taps, dtype)
    pool = torch.randn(8, taps - 1, w, generator=torch.Generator().manual_seed(26)).to(DT[dtype])
    y, p = dev(x), pool.to(DEV)
    o = rr.short_conv_step(y["x"], y["weight"], p, y["bias"], swish=True,
                           slots=torch.tensor([6, -1, 2, 6, 8], dtype=torch.int32, device=DEV))
    for i, slot in ((0, 6), (2, 2)):
        ro, rs = oracle.conv(f64(x["x"][i:i + 1]), f64(x["weight"]), f64(x["bias"]), True, f64(pool[slot:slot + 1]))
        near(o[i:i + 1], ro, CONV, "o")
        np.testing.assert_array_equal(f64(p[slot:slot + 1]), rs)
    assert (o[[1, 3, 4]] == 0).all()
    rest = [i for i in range(8) if i not in (6, 2)]
    assert torch.equal(p.cpu()[rest], pool[rest])


def test_conv_state_in_place_and_pieces():
    x = dev(conv_inputs(27, (2, 300), 66, 4, "bf16", state=2))
    whole = run_conv(x, True)
    s, outs = x["s0"].clone(), []
    for a, b in ((0, 1), (1, 3), (3, 130), (130, 300)):
        outs.append(rr.short_conv_fwd(x["x"][:, a:b].contiguous(), x["weight"], x["bias"], swish=True, state_in=s,
                                      state_out=s))
    assert torch.equal(torch.cat(outs, 1), whole["o"]) and torch.equal(s, whole["state"])
    s = x["s0"].clone()
    for t in range(5):
        o = rr.short_conv_step(x["x"][:, t:t + 1], x["weight"], s, x["bias"], swish=True)
        assert torch.equal(o[:, 0], whole["o"][:, t])


# ------------------------------------------------------------- cache of states
@pytest.mark.parametrize("shape", [(2, 64, 64), (3, 7), (1,), (130,), (1000,), (64,)])
def test_cache_is_the_oracles(shape):
    """Codes and scales bit for bit, only the slots that are named; then back."""
    g = torch.Generator().manual_seed(31)
    live = torch.randn(6, *shape, generator=g) * torch.exp(torch.randn(6, *shape, generator=g))
    values = live[0].numel()
    codes = torch.full((9,) + shape, 55, dtype=torch.int8, device=DEV)
    scales = torch.full((9, -(-values // 64)), -1.0, device=DEV)
    at, slots = [4, 8, -1, 4, 9, 0], [5, 0, 1, 2, 3, 6]  # outside: -1, 9, 6; 4 is taken
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    rr.state_cache_write(live.to(DEV), codes, scales, i32(at), slots=i32(slots))
    rc, rs = oracle.park(f64(live).reshape(6, -1))
    for c, s in ((4, 5), (8, 0)):
        np.testing.assert_array_equal(codes[c].cpu().numpy().reshape(-1), rc[s])
        np.testing.assert_array_equal(scales[c].cpu().numpy(), rs[s])
    rest = [0, 1, 2, 3, 5, 6, 7]
    assert (codes[rest] == 55).all() and (scales[rest] == -1).all()
    back = torch.full((7,) + shape, 3.0, device=DEV)
    rr.state_cache_read(codes, scales, back, i32([8, 4, -1, 8, 4, 4]), slots=i32([0, 1, 2, 3, 3, -2]))
    want = oracle.resume(rc, rs)
    for b, s in ((0, 0), (1, 5), (3, 0)):
        np.testing.assert_array_equal(back[b].cpu().numpy().reshape(-1), want[s])
    assert (back[2] == 0).all() and (back[4:] == 3).all()


def test_cache_of_unusual_values():
    x = torch.zeros(1, 64 * 8)
    x[0, 3], x[0, 64 + 3], x[0, 128 + 5] = float("nan"), float("-inf"), 1e-38
    x[0, 192:256] = torch.linspace(-1e-42, 1e-42, 64)
    x[0, 256:320] = torch.arange(64) * 3.0e38 / 64  # passes the largest number: infinities
    x[0, 448:512] = torch.arange(64) / 64 * 3.0e38
    x[0, 320:384] = torch.arange(-32, 32) + 0.5  # halves of a scale that is a power of two
    x[0, 320] = 127.0
    x[0, 384:448] = -0.0
    codes, scales = torch.zeros(1, 512, dtype=torch.int8, device=DEV), torch.zeros(1, 8, device=DEV)
    i32 = torch.zeros(1, dtype=torch.int32, device=DEV)
    rr.state_cache_write(x.to(DEV), codes, scales, i32)
    back = rr.state_cache_read(codes, scales, torch.empty(1, 512, device=DEV), i32).cpu()
    for block in range(8):
        part = slice(64 * block, 64 * block + 64)
        bad = not bool(torch.isfinite(x[0, part]).all())
        assert bad == (block in (0, 1, 4))
        assert bool(torch.isnan(back[0, part]).all()) if bad else bool(torch.isfinite(back[0, part]).all()), block
    rc, rs = oracle.park(f64(x))
    np.testing.assert_array_equal(scales.cpu().numpy(), rs)
    np.testing.assert_array_equal(codes.cpu().numpy()[:, 128:256], rc[:, 128:256])
    np.testing.assert_array_equal(codes.cpu().numpy()[:, 320:], rc[:, 320:])
    assert codes[0, 321:384].cpu().tolist() == [int(np.rint(v)) for v in np.arange(-31, 32) + 0.5]


# --------------------------------------------------------------------- together
def test_a_gated_recurrent_layer():
    """Convolution, recurrence and the gated norm over a prompt, then decode with the
    state parked and resumed on the way: the whole sequence's outputs."""
    b, n, w, d = 2, 200, 256, 64
    g = torch.Generator().manual_seed(41)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    proj, cw = r(b, n, 4 * w).to(DEV), (r(w, 4) / 2).to(DEV)
    rate = torch.exp(-5 + 3 * torch.rand(w, generator=g)).to(DEV)

    def layer(p, conv_state, state):
        x = rr.short_conv_fwd(p[..., :w], cw, swish=True, state_in=conv_state, state_out=conv_state)
        h = rr.gated_scan_fwd(x, p[..., w:2 * w], p[..., 2 * w:3 * w], rate=rate, normalize=True, state_in=state,
                              state_out=state)
        gate = p[..., 3 * w:].reshape(b, -1, w // d, d).contiguous()
        return rr.head_norm_fwd(h.reshape(gate.shape), None, gate, center=True)

    new = lambda: (torch.zeros(b, 3, w, device=DEV), torch.zeros(b, w, device=DEV))  # noqa: E731
    whole = layer(proj, *new())
    conv_state, state = new()
    outs = [layer(proj[:, :150].contiguous(), conv_state, state)]  # a batch of one distance
    near(outs[0].reshape(b, 150, w), f64(whole[:, :150]).reshape(b, 150, w), 64 * fwd_bar(150), "prompt")
    codes, scales = torch.zeros(3, w, dtype=torch.int8, device=DEV), torch.zeros(3, w // 64, device=DEV)
    at = torch.tensor([2, 0], dtype=torch.int32, device=DEV)
    rr.state_cache_write(state, codes, scales, at)
    parked = rr.state_cache_read(codes, scales, torch.empty_like(state), at)
    # half a step of the largest of 64 values
    assert ((parked - state).abs() <= state.abs().reshape(b, -1, 64).amax(-1).repeat_interleave(64, 1) / 253).all()
    for t in range(150, n):
        p = proj[:, t:t + 1]
        x = rr.short_conv_step(p[..., :w], cw, conv_state, swish=True)
        gates = (p[..., w:2 * w], p[..., 2 * w:3 * w])
        h = rr.gated_scan_step(x, gates[0], state, gates[1], rate=rate, normalize=True)
        rr.gated_scan_step(x, gates[0], parked, gates[1], rate=rate, normalize=True)
        gate = p[..., 3 * w:].reshape(b, 1, w // d, d).contiguous()
        o = rr.head_norm_fwd(h.reshape(gate.shape), None, gate, center=True)
        near(o.reshape(b, w), f64(whole[:, t]).reshape(b, w), 64 * fwd_bar(n), f"token {t}")
    # what parking changed fades with the factors
    assert (parked - state).norm() <= 0.01 * state.norm()


def test_a_training_step_of_the_layer():
    """Gradients through recurrence and convolution, chained by hand, against differences of the oracle's loss."""
    b, n, w = 1, 37, 8
    rng = np.random.default_rng(42)
    p = {k: rng.standard_normal(s).astype(np.float32).astype(np.float64) for k, s in
         dict(x=(b, n, w), decay=(b, n, w), gate=(b, n, w), weight=(w, 3), bias=(w,), dout=(b, n, w)).items()}
    p["rate"] = np.abs(rng.standard_normal(w)).astype(np.float32).astype(np.float64) + 0.01

    def loss():
        u, _ = oracle.conv(p["x"], p["weight"], p["bias"], True)
        return (p["dout"] * oracle.scan(u, p["decay"], p["gate"], p["rate"], True)[0]).sum()

    t = {k: torch.from_numpy(v.astype(np.float32)).to(DEV) for k, v in p.items()}
    u = rr.short_conv_fwd(t["x"], t["weight"], t["bias"], swish=True)
    _, kept = rr.gated_scan_fwd(u, t["decay"], t["gate"], rate=t["rate"], normalize=True, keep=True)
    du, ddecay, dgate, drate = rr.gated_scan_bwd(u, t["decay"], t["dout"], t["gate"], rate=t["rate"], normalize=True,
                                                 kept=kept)
    dx, dweight, dbias = rr.short_conv_bwd(t["x"], t["weight"], du, t["bias"], swish=True)
    got = {k: f64(v) for k, v in dict(x=dx, decay=ddecay, gate=dgate, rate=drate, weight=dweight, bias=dbias).items()}
    for k, g in got.items():
        for _ in range(8):
            at = tuple(rng.integers(0, m) for m in g.shape)
            old = p[k][at]
            p[k][at] = old + 1e-5
            up = loss()
            p[k][at] = old - 1e-5
            down = loss()
            p[k][at] = old
            # the difference's own error 1e-7, fp32 gradients to 1e-5 of the tensor's largest
            assert abs((up - down) / 2e-5 - g[at]) <= 1e-6 + 1e-5 * np.abs(g).max(), (k, at)
