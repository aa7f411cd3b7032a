"""Calls of the recurrence, the convolution and the cache of parked states that their
documentation allows at its borders: workspaces that held anything, graphs, streams,
large offsets, many sequences."""

import numpy as np
import pytest
import torch

import retnet_retention_amd as rr
from retnet_retention_amd import binding
from oracle import scan_oracle as oracle
from test_gpu_scan import (CONV, DEV, FORMS, check_conv, check_scan, conv_inputs, dev, f64, fwd_bar, near, run_conv,
                           run_scan, scan_inputs, scan_reference)

pytestmark = pytest.mark.gpu


def i32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def free_memory(need):
    """Skips where the card holds less (a smaller device, or a shared one)."""
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < need:
        pytest.skip(f"needs {need >> 30} GiB of device memory")


def workspace(call, fill):
    """A workspace that `call` accepts with every byte `fill` (255: NaN in every type, a word that looks handed on)."""
    for size in (1 << i for i in range(4, 36)):
        try:
            call(torch.empty(size, dtype=torch.uint8, device=DEV))
            return torch.full((size,), fill, dtype=torch.uint8, device=DEV)
        except rr.RetentionError as e:
            assert e.status == 6
    raise AssertionError("no size was accepted")


def same(a, b):
    return all((x is None and y is None) or torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("dtype,form,w", [("bf16", "gates", 66), ("bf16", "log", 67), ("f32", "gates", 130)])
@pytest.mark.parametrize("n,lens", [(700, None), (200, None), (1, None), (600, [600, 0, 1, 130])])
def test_nothing_of_a_workspace_is_read_before_it_is_written(dtype, form, w, n, lens):
    """The same bits whatever the workspace held, call after call on one workspace."""
    rows, b = ((sum(lens),), len(lens)) if lens else ((2, n), 2)
    x = dev(scan_inputs(51, rows, w, dtype, form, state=b))
    more = dict(rate=x["rate"], normalize=True, state_in=x["s0"])
    if lens:
        more["cu_seqlens"] = i32([0] + list(np.cumsum(lens)))
    s = torch.empty_like(x["s0"])

    def fwd(ws):
        o, kept = rr.gated_scan_fwd(x["x"], x["decay"], x["gate"], state_out=s, keep=True, workspace=ws, **more)
        return [o, s.clone(), kept]

    kept = fwd(None)[2]
    bwd = lambda ws: rr.gated_scan_bwd(x["x"], x["decay"], x["dout"], x["gate"], d_state_out=x["ds"], kept=kept,  # noqa: E731
                                       workspace=ws, **more)
    again = lambda ws: rr.gated_scan_bwd(x["x"], x["decay"], x["dout"], x["gate"], d_state_out=x["ds"], workspace=ws,  # noqa: E731
                                         **more)
    ref = bwd(None)
    for call, want in ((fwd, fwd(None)[:2]), (bwd, ref), (again, ref)):
        for fill in (0, 255, 1):
            ws = workspace(call, fill)
            for _ in range(3):
                assert same(call(ws)[:len(want)], want)
            rr.check_chunkwise(ws)


@pytest.mark.parametrize("lens", [None, [300, 0, 2, 65]])
def test_the_convolutions_workspace(lens):
    rows, b = ((sum(lens),), len(lens)) if lens else ((2, 300), 2)
    x = dev(conv_inputs(52, rows, 66, 4, "bf16", state=b))
    more = dict(cu_seqlens=i32([0] + list(np.cumsum(lens)))) if lens else {}
    ref = rr.short_conv_bwd(x["x"], x["weight"], x["dout"], x["bias"], swish=True, state_in=x["s0"], d_state_out=x["ds"],
                            **more)
    call = lambda ws: rr.short_conv_bwd(x["x"], x["weight"], x["dout"], x["bias"], swish=True, state_in=x["s0"],  # noqa: E731
                                        d_state_out=x["ds"], workspace=ws, **more)
    for fill in (0, 255):
        ws = workspace(call, fill)
        for _ in range(2):
            assert same(call(ws), ref)


@pytest.mark.parametrize("lens", [None, [1300, 0, 66, 257]])
def test_a_layer_in_a_graph(lens):
    """Convolution, recurrence, their gradients and a parked state captured on one stream, with workspaces of its own,
    replayed on new inputs between eager calls."""
    rows, b = ((sum(lens),), len(lens)) if lens else ((2, 1000), 2)
    x = dev(scan_inputs(53, rows, 66, "bf16", "gates", state=b))
    w = torch.randn(66, 4, generator=torch.Generator().manual_seed(54)).to(DEV)
    more = dict(cu_seqlens=i32([0] + list(np.cumsum(lens)))) if lens else {}
    at = i32(list(range(b)))

    def layer():
        codes, scales = torch.empty(b, 66, dtype=torch.int8, device=DEV), torch.empty(b, 2, device=DEV)
        u = rr.short_conv_fwd(x["x"], w, swish=True, **more)
        s = torch.empty_like(x["s0"])
        gates = dict(rate=x["rate"], normalize=True, state_in=x["s0"], **more)
        o, kept = rr.gated_scan_fwd(u, x["decay"], x["gate"], state_out=s, keep=True, **gates)
        g = rr.gated_scan_bwd(u, x["decay"], x["dout"], x["gate"], d_state_out=x["ds"], kept=kept, **gates)
        dx, dw, _ = rr.short_conv_bwd(x["x"], w, g[0], swish=True, **more)
        rr.state_cache_write(s, codes, scales, at)
        back = rr.state_cache_read(codes, scales, torch.empty_like(s), at)
        one = [t.reshape(-1, 66)[:b].reshape(b, 1, 66) for t in (u, x["decay"], x["gate"])]
        step = rr.gated_scan_step(one[0], one[1], back, one[2], rate=x["rate"])
        return [o, s, *g, dx, dw, step, back]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            outs = layer()
    torch.cuda.current_stream().wait_stream(side)
    for seed in range(4):
        for k in ("x", "decay", "gate", "dout", "s0"):
            x[k].copy_(torch.randn(x[k].shape, generator=torch.Generator().manual_seed(seed)))
        graph.replay()
        torch.cuda.synchronize()
        assert same(outs, layer())


def test_two_streams_at_once():
    """Calls with workspaces of their own side by side, on streams that are not the inputs' own."""
    xs = [dev(scan_inputs(55 + i, (2, 3000), 130, "bf16", "gates", state=2)) for i in range(2)]
    refs = [run_scan(x, True) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    for _ in range(5):
        outs = []
        for x, st in zip(xs, streams):
            with torch.cuda.stream(st):
                outs.append(run_scan(x, True))
        torch.cuda.synchronize()
        for got, ref in zip(outs, refs):
            assert all(got[k] is None or torch.equal(got[k], ref[k]) for k in ref)


def test_a_sequence_behind_2_31_elements():
    """The last packed sequence starts behind 2^31 elements of every tensor: the bits of that sequence alone."""
    w, first, last = 4096, 530000, 700
    n = first + last
    assert first * w > 2 ** 31
    free_memory(60 << 30)
    g = torch.Generator(device=DEV).manual_seed(56)
    r = lambda: torch.randn(n, w, generator=g, device=DEV, dtype=torch.bfloat16)  # noqa: E731
    x, decay, gate = r(), r(), r()
    rate, cw = torch.rand(w, generator=g, device=DEV), torch.randn(w, 4, generator=g, device=DEV)
    cu = i32([0, first, n])
    s = torch.empty(2, w, device=DEV)
    o, kept = rr.gated_scan_fwd(x, decay, gate, rate=rate, state_out=s, cu_seqlens=cu, keep=True, check=True)
    tail = [t[first:][None].contiguous() for t in (x, decay, gate)]
    s1 = torch.empty(1, w, device=DEV)
    o1 = rr.gated_scan_fwd(tail[0], tail[1], tail[2], rate=rate, state_out=s1)
    assert torch.equal(o[first:], o1[0]) and torch.equal(s[1], s1[0]) and torch.isfinite(o[first - 300:first].float()).all()
    got = rr.gated_scan_bwd(x, decay, o, gate, rate=rate, cu_seqlens=cu, kept=kept, check=True)
    ref = rr.gated_scan_bwd(tail[0], tail[1], o1, tail[2], rate=rate)
    for a, b in zip(got[:3], ref):
        assert torch.equal(a[first:], b[0]) and torch.isfinite(a[first - 300:first].float()).all()
    del got, kept, decay, gate
    c = rr.short_conv_fwd(x, cw, swish=True, cu_seqlens=cu, check=True)
    assert torch.equal(c[first:], rr.short_conv_fwd(tail[0], cw, swish=True)[0])
    d = rr.short_conv_bwd(x, cw, o, swish=True, cu_seqlens=cu, check=True)[0]
    assert torch.equal(d[first:], rr.short_conv_bwd(tail[0], cw, o1, swish=True)[0][0])
    del x, o, c, d
    torch.cuda.empty_cache()


def test_slots_behind_2_31_elements():
    """Pools of states and of cached codes past 2^31 elements (and 2^33 bytes)."""
    w, n = 4096, 2 ** 31 // 4096 + 40
    free_memory(40 << 30)
    x = dev(scan_inputs(57, (2, 1), w, "bf16", "gates"))
    held = torch.randn(2, w, generator=torch.Generator().manual_seed(58)).to(DEV)
    pool = torch.zeros(n, w, device=DEV)
    pool[n - 1], pool[n - 2] = held[0], held[1]
    o = rr.gated_scan_step(x["x"], x["decay"], pool, x["gate"], rate=x["rate"], slots=i32([n - 1, n - 2]))
    o1 = rr.gated_scan_step(x["x"], x["decay"], held, x["gate"], rate=x["rate"])
    assert torch.equal(o, o1) and torch.equal(pool[n - 1], held[0]) and torch.equal(pool[n - 2], held[1])
    codes, scales = torch.zeros(n, w, dtype=torch.int8, device=DEV), torch.zeros(n, w // 64, device=DEV)
    rr.state_cache_write(pool, codes, scales, i32([n - 1, n - 5]), slots=i32([n - 2, n - 1]))
    rc, rs = oracle.park(f64(held))
    np.testing.assert_array_equal(codes[[n - 1, n - 5]].cpu().numpy(), rc[[1, 0]])
    np.testing.assert_array_equal(scales[[n - 1, n - 5]].cpu().numpy(), rs[[1, 0]])
    rr.state_cache_read(codes, scales, pool, i32([n - 5, -1]), slots=i32([n - 2, n - 3]))
    np.testing.assert_array_equal(pool[n - 2].cpu().numpy(), oracle.resume(rc[:1], rs[:1])[0])
    assert (pool[:n - 2] == 0).all()
    del pool, codes
    torch.cuda.empty_cache()


def test_very_many_sequences():
    """A batch of single tokens, and packed ones, more than a search step's 64 times 64."""
    b, w = 70000, 66
    x = dev(scan_inputs(59, (b, 1), w, "bf16", "gates", state=b))
    whole = run_scan(x, True)
    flat = {k: t.reshape(b, w) if k in ("x", "decay", "gate", "dout") else t for k, t in x.items()}
    cu = torch.arange(b + 1, dtype=torch.int32, device=DEV)
    packed = run_scan(flat, True, cu_seqlens=cu, check=True)
    for k in whole:
        if k != "drate":
            assert torch.equal(packed[k].reshape(whole[k].shape), whole[k]), k
    near(packed["drate"], f64(whole["drate"]), fwd_bar(1) * 4 * (1 + b ** 0.5), "drate")
    for at in (0, 4095, 4096, 65535, b - 1):
        part = {k: t[at:at + 1].clone() if t is not None and k != "rate" else t for k, t in x.items()}  # (aligned)
        one = run_scan(part, True)
        assert torch.equal(one["o"][0], whole["o"][at]) and torch.equal(one["dx"][0], whole["dx"][at])
    y = dev(conv_inputs(60, (b,), w, 4, "bf16", state=b))
    got = run_conv(y, True, cu_seqlens=cu, check=True)
    part = dict(y, **{k: y[k][b - 3:].clone() for k in ("s0", "ds")}, **{k: y[k][b - 3:].reshape(3, 1, w).clone() for k in
                                                                           ("x", "dout")})
    ref = run_conv(part, True)
    assert torch.equal(got["o"][b - 3:], ref["o"][:, 0]) and torch.equal(got["state"][b - 3:], ref["state"])
    assert torch.equal(got["dx"][b - 3:], ref["dx"][:, 0]) and torch.equal(got["dstate"][b - 3:], ref["dstate"])


@pytest.mark.parametrize("w", [1, 2, 63, 64, 65, 127, 129, 2049, 5000, 65536])
def test_widths(w):
    """Each channel by itself: the bits of the same channels alone."""
    x = dev(scan_inputs(61, (1, 600), w, "bf16", "gates", state=1))
    whole = run_scan(x, True)
    for a, b in ((0, min(w, 64)), (max(0, w - 3), w)):
        part = {k: None if t is None else t[..., a:b].clone() for k, t in x.items()}
        got = run_scan(part, True)
        for k in whole:
            assert torch.equal(got[k], whole[k][..., a:b]), k


@pytest.mark.parametrize("lens", [[2000], [257, 1, 0, 700]])
def test_the_longest_chain_is_in_order(lens):
    """Sums over whole sequences: with factors of 1 the state counts its tokens, exactly."""
    n = sum(lens)
    x = torch.ones(n, 66, device=DEV)
    cu = i32([0] + list(np.cumsum(lens)))
    zero = torch.zeros(n, 66, device=DEV)
    s = torch.zeros(len(lens), 66, device=DEV)
    o = rr.gated_scan_fwd(x, zero, state_in=s, state_out=s, cu_seqlens=cu, check=True)
    want = torch.cat([torch.arange(1, k + 1) for k in lens]).float().to(DEV)
    assert torch.equal(o, want[:, None].expand_as(o))
    assert torch.equal(s[:, 0].cpu(), torch.tensor([float(k) for k in lens]))
    dx, dl, _, _ = rr.gated_scan_bwd(x, zero, x, cu_seqlens=cu)
    back = torch.cat([torch.arange(k, 0, -1) for k in lens]).float().to(DEV)
    assert torch.equal(dx, back[:, None].expand_as(dx)) and torch.equal(dl[:, 0], back * (want - 1))


@pytest.mark.parametrize("n", [300, 3000])
def test_a_hundred_thousand_tokens_of_memory(n):
    """A channel that forgets a 10^5th of itself a token keeps its decay rate: n tokens of the same factor."""
    la = torch.full((1, n, 64), -1e-5, device=DEV)
    s = torch.ones(1, 64, device=DEV)
    x = torch.zeros(1, n, 64, dtype=torch.bfloat16, device=DEV)
    rr.gated_scan_fwd(x, la, state_in=s, state_out=s)
    # a factor's rounding is at most 2^-25 of it (values in [1/2, 1)), as is each product's
    assert (np.abs(f64(s) - np.exp(-1e-5 * n)) <= 2 * n * 2.0 ** -25).all()


def test_refused_tensors():
    x = torch.zeros(2, 5, 8, device=DEV)
    rate = torch.ones(8, device=DEV)
    for bad in (lambda: rr.gated_scan_fwd(x, x.bfloat16()), lambda: rr.gated_scan_fwd(x, x[:, :4]),
                lambda: rr.gated_scan_fwd(x, x, rate=rate[:7]), lambda: rr.gated_scan_fwd(x, x, x.bfloat16()),
                lambda: rr.gated_scan_fwd(x, x, out=x.transpose(0, 1)), lambda: rr.gated_scan_fwd(x[0], x[0]),
                lambda: rr.gated_scan_fwd(x, x, state_in=torch.zeros(2, 9, device=DEV)),
                lambda: rr.gated_scan_fwd(x[0], x[0], cu_seqlens=torch.zeros(2, dtype=torch.int64, device=DEV)),
                lambda: rr.gated_scan_bwd(x, x, x, kept=torch.zeros(3, device=DEV)),
                lambda: rr.gated_scan_step(x, x, torch.zeros(2, 8, device=DEV)),
                lambda: rr.gated_scan_step(x[:, :1], x[:, :1], torch.zeros(3, 8, device=DEV)),
                lambda: rr.short_conv_fwd(x, torch.zeros(8, device=DEV)),
                lambda: rr.short_conv_fwd(x, torch.zeros(7, 4, device=DEV)),
                lambda: rr.short_conv_fwd(x, torch.zeros(8, 4, device=DEV), state_in=torch.zeros(2, 4, 8, device=DEV)),
                lambda: rr.short_conv_step(x, torch.zeros(8, 4, device=DEV), torch.zeros(2, 3, 8, device=DEV)),
                lambda: rr.state_cache_write(x, torch.zeros(2, 5, 8, device=DEV), torch.zeros(2, 1, device=DEV), i32([0])),
                lambda: rr.state_cache_read(torch.zeros(2, 5, 8, dtype=torch.int8, device=DEV),
                                            torch.zeros(2, 2, device=DEV), x, i32([0]))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        rr.gated_scan_fwd(x.half(), x)
    for bad, status in ((lambda: rr.gated_scan_fwd(x[:, :0], x[:, :0]), 2), (lambda: rr.gated_scan_fwd(x, x, out=x), 8),
                        (lambda: rr.short_conv_fwd(x, torch.zeros(8, 5, device=DEV)), 3),
                        (lambda: rr.gated_scan_fwd(x, x, workspace=torch.zeros(8, device=DEV)), 6)):
        with pytest.raises(rr.RetentionError) as e:
            bad()
        assert e.value.status == status


def test_convolution_of_one_tensor_with_itself_in_pieces_of_any_size():
    """Prompts cut anywhere, the state handed from piece to piece."""
    x = dev(conv_inputs(62, (1, 120), 66, 4, "f32", state=1))
    whole = run_conv(x, True)
    rng = np.random.default_rng(63)
    for _ in range(5):
        cuts = [0] + sorted(rng.choice(np.arange(1, 120), 6, replace=False).tolist()) + [120]
        s, outs = x["s0"].clone(), []
        for a, b in zip(cuts, cuts[1:]):
            outs.append(rr.short_conv_fwd(x["x"][:, a:b], x["weight"], x["bias"], swish=True, state_in=s, state_out=s))
        near(torch.cat(outs, 1), f64(whole["o"]), CONV, "o")
        assert torch.equal(s, whole["state"])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decays_next_to_nothing(dtype):
    """Gates so far shut, or rates so small, that 1 - a^2 has no normal number: finite gradients, and the formula's where
    they count. A decay that small moves nothing: 2^-63 is the root of the smallest normal number."""
    x = scan_inputs(64, (2, 140), 66, dtype, "gates", state=2)
    x["decay"][:, ::3] = -87.0
    x["decay"][:, 1::3] = -100.0
    x["rate"][:20], x["rate"][20:30], x["rate"][30:35] = 0.01, 0.0, 1e-38
    got, a = run_scan(dev(x), True), {k: f64(t) for k, t in x.items()}
    want = dict(zip(("o", "state"), oracle.scan(a["x"], a["decay"], a["gate"], a["rate"], True, a["s0"])))
    g = oracle.scan_grad(a["x"], a["decay"], a["dout"], a["gate"], a["rate"], True, a["s0"], a["ds"])
    want.update(dict(zip(("dx", "ddecay", "dgate", "drate", "dstate"), g)))
    for k in got:
        assert torch.isfinite(got[k].float()).all(), k
        if k == "drate":  # the root's own share, s_d / m times a gradient, is below 2^-40 of the rest where 1 - a^2 is lost
            continue
        near(got[k], want[k], 4 * fwd_bar(140), k)


@pytest.mark.parametrize("form,gate,normalize", FORMS)
@pytest.mark.parametrize("dtype,w", [("bf16", 130), ("bf16", 67), ("f32", 65)])
def test_forms_of_more_than_one_tile(form, gate, normalize, dtype, w):
    x = scan_inputs(60, (2, 700), w, dtype, form, gate, state=2)
    check_scan(run_scan(dev(x), normalize), scan_reference(x, normalize), 700, 1400)


@pytest.mark.parametrize("b,n,lens", [(1, 512, None), (1, 257, None), (5, 400, None), (260, 260, None),
                                      (3, None, [257, 0, 200]), (4, None, [1, 510, 0, 1]), (2, None, [0, 300]),
                                      (600, None, [1, 0] * 250 + [2] * 100)])
def test_sequences_of_one_workgroup(b, n, lens):
    """Up to 512 tokens: sequences that are one tile where there are few of them, and two where there are many."""
    rows = (sum(lens),) if lens else (b, n)
    x = scan_inputs(61, rows, 66, "bf16", "gates", state=b)
    more = dict(cu_seqlens=i32([0] + list(np.cumsum(lens))), check=True) if lens else {}
    got = run_scan(dev(x), True, **more)
    check_scan(got, scan_reference(x, True, lens), max(lens) if lens else n, int(np.prod(rows)))
    # a state of NaN behind a factor of 0 is forgotten there too
    y = dev(x)
    if lens:
        y["decay"][torch.tensor([t for t, k in zip(np.cumsum([0] + lens[:-1]), lens) if k], device=DEV)] = 88.
    else:
        y["decay"][:, 0] = 88.
    y["rate"] = torch.full_like(y["rate"], 200.)
    y["s0"] = torch.full_like(y["s0"], float("nan"))
    s = y["s0"].clone()
    o = rr.gated_scan_fwd(y["x"], y["decay"], y["gate"], rate=y["rate"], state_in=y["s0"], state_out=s, **more)
    assert torch.isfinite(o.float()).all()
    held = torch.tensor([k > 0 for k in lens], device=DEV) if lens else torch.ones(b, dtype=torch.bool, device=DEV)
    assert torch.isfinite(s[held]).all() and torch.isnan(s[~held]).all()


@pytest.mark.parametrize("stride", [2 ** 20, 2 ** 21, 2 ** 22 - 8])
def test_rows_that_lie_far_apart(stride):
    """300 tokens up to 8 MiB from one another."""
    free_memory(300 * stride * 2 + (2 << 30))
    x = scan_inputs(62, (1, 300), 66, "bf16", "gates", state=1)
    y = dev(x)
    big = torch.empty(300 * stride, dtype=torch.bfloat16, device=DEV)
    y["x"] = big.view(1, 300, stride)[:, :, 7 * 64:7 * 64 + 66].copy_(y["x"])
    assert y["x"].stride(1) == stride
    check_scan(run_scan(y, True), scan_reference(x, True), 300, 300)


def test_rows_of_fp32_that_lie_far_apart():
    """300 tokens 8 MiB apart in fp32."""
    stride = 2 ** 21
    free_memory(300 * stride * 4 + (2 << 30))
    x = scan_inputs(63, (1, 300), 65, "f32", "log", state=1)
    y = dev(x)
    y["decay"] = torch.empty(300 * stride, device=DEV).view(1, 300, stride)[:, :, :65].copy_(y["decay"])
    check_scan(run_scan(y, True), scan_reference(x, True), 300, 300)


def test_a_sequence_that_parks_nothing_takes_no_slot():
    """Idle sequences may name any cache slot: the next one that names it and has a state is parked there."""
    live = torch.randn(3, 130, device=DEV)
    codes, scales = torch.full((2, 130), 55, dtype=torch.int8, device=DEV), torch.full((2, 3), -1.0, device=DEV)
    rr.state_cache_write(live, codes, scales, i32([1, 1, 1, 1, 0]), slots=i32([-1, 3, 2, 0, -5]))
    want = oracle.park(f64(live[2:]))
    np.testing.assert_array_equal(codes[1].cpu().numpy(), want[0][0])
    np.testing.assert_array_equal(scales[1].cpu().numpy(), want[1][0])
    assert (codes[0] == 55).all() and (scales[0] == -1).all()


@pytest.mark.parametrize("dtype,w", [("bf16", 1024), ("bf16", 1155), ("bf16", 1282), ("bf16", 7000), ("f32", 2049)])
@pytest.mark.parametrize("lens", [None, [130, 0, 700, 1]])
def test_widths_of_the_convolution(dtype, w, lens):
    """Each channel by itself, also where a row is more than eight workgroups wide: the formula's values on the first
    channels, the last ones and some between."""
    rows, b = ((sum(lens),), len(lens)) if lens else ((3, 300), 3)
    x = conv_inputs(64, rows, w, 4, dtype, state=b)
    more = dict(cu_seqlens=i32([0] + list(np.cumsum(lens))), check=True) if lens else {}
    got = run_conv(dev(x), True, **more)
    for at in (0, 512, w - 70):
        part = {k: None if t is None else t[at:at + 70] if k in ("weight", "bias") else
                t[..., at:at + 70] for k, t in x.items()}
        cut = {k: None if t is None else t[at:at + 70] if k in ("dweight", "dbias") else
               t[..., at:at + 70] for k, t in got.items()}
        check_conv(cut, part, True, lens)


@pytest.mark.parametrize("dtype,w,columns", [("bf16", 66, False), ("bf16", 67, False), ("bf16", 66, True), ("f32", 65, False)])
@pytest.mark.parametrize("form,gate", [("gates", True), ("log", False)])
@pytest.mark.parametrize("cu", [[300, 310, 390], [1, 1, 1], [0, 699, 699], [700, 700, 700], [17, 40, 683]])
def test_every_row_outside_the_sequences_has_a_gradient_of_zero(monkeypatch, dtype, w, columns, form, gate, cu):
    """Whether lanes take one channel or two, in gradients that held NaN before the call."""
    x = dev(scan_inputs(65, (700,), w, dtype, form, gate, state=2))
    if columns:  # at an odd offset: lanes cannot take pairs
        x["x"] = torch.cat([x["x"][:, :1], x["x"]], 1)[:, 1:]
        assert x["x"].data_ptr() % 4 == 2
    monkeypatch.setattr(binding, "_dense_like", lambda t: torch.full(t.shape, float("nan"), dtype=t.dtype, device=t.device))
    g = rr.gated_scan_bwd(x["x"], x["decay"], x["dout"], x["gate"], rate=x["rate"], state_in=x["s0"], d_state_out=x["ds"],
                          cu_seqlens=i32(cu), check=True)
    assert len(g) == 5 and all(t is None or torch.isfinite(t.float()).all() for t in g)
    for t in g[:3]:
        assert t is None or ((t[:cu[0]] == 0).all() and (t[cu[2]:] == 0).all())


@pytest.mark.parametrize("default", [torch.bfloat16, torch.float64])
def test_training_under_another_default_type(default):
    """The bits of the calls under fp32, from tensors made before."""
    x = dev(scan_inputs(66, (2, 700), 66, "bf16", "gates", state=2))
    want = run_scan(x, True)
    before = torch.get_default_dtype()
    torch.set_default_dtype(default)
    try:
        _, kept = rr.gated_scan_fwd(x["x"], x["decay"], x["gate"], rate=x["rate"], normalize=True, state_in=x["s0"], keep=True)
        got = run_scan(x, True)
    finally:
        torch.set_default_dtype(before)
    assert kept.dtype == torch.float32
    assert all(got[k] is None or (got[k].dtype == want[k].dtype and torch.equal(got[k], want[k])) for k in want)
