"""Cases that measure the gated delta rule (chunkwise forward, its gradients,
the decode step) and the norms around a token mixer (per-head norm with gate,
residual join with the norms before and after a block).

Where `own` is false, run() computes each operator in plain torch operations
in 32 bits (angles of accuracy that 32 bits would lose, the cumulative decays
and the inverse of a block's triangular system, in 64); where it is true,
run() calls the framework.
"""

import math

import torch

own = False

DEV = "cuda" if torch.cuda.is_available() else "cpu"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BLOCK = 64  # tokens of a block in the plain form


# --------------------------------------------------------------------------
# Cases. heads x dim of the bf16 cases are this repository's layers (4, 10 and
# 16 heads of 256), or half as wide heads with two value heads a key head.
# --------------------------------------------------------------------------
def listed():
    return [
        # a short chat turn continued from a cached state: latency counts
        dict(name="delta_fwd_turn", op="delta_fwd", dtype="bf16", batch=1, tokens=257, k_heads=4, heads=4, dim=256,
             state=True, lens=""),
        # prefill of two long prompts on the 7B-class layer
        dict(name="delta_fwd_7b_8k", op="delta_fwd", dtype="bf16", batch=2, tokens=8192, k_heads=16, heads=16,
             dim=256, state=True, lens=""),
        # packed prompts of different lengths, an empty one and a single token among them, shared key heads
        dict(name="delta_fwd_packed", op="delta_fwd", dtype="bf16", batch=9, tokens=4099, k_heads=16, heads=32,
             dim=128, state=True, lens="1900,0,4099,1,640,65,1201,333,2048"),
        # training step of the 3B-class layer: gradients of a 2048-token batch
        dict(name="delta_bwd_3b", op="delta_bwd", dtype="bf16", batch=4, tokens=2048, k_heads=10, heads=10, dim=256,
             state=False, lens=""),
        # training on a long document cut into pieces: state carried in, its gradient carried back
        dict(name="delta_bwd_carried", op="delta_bwd", dtype="bf16", batch=1, tokens=4001, k_heads=8, heads=16,
             dim=128, state=True, lens=""),
        # a small model trained in fp32
        dict(name="delta_bwd_small_f32", op="delta_bwd", dtype="f32", batch=2, tokens=300, k_heads=2, heads=2, dim=64,
             state=True, lens=""),
        # decode: one user, and a full serving batch of the 7B-class layer with idle slots
        dict(name="step_b1", op="step", dtype="bf16", batch=1, slots=1, idle=0, k_heads=16, heads=16, dim=256),
        dict(name="step_b256", op="step", dtype="bf16", batch=256, slots=256, idle=3, k_heads=16, heads=16, dim=256),
        # the gated norm on the output of the 7B-class mixer
        dict(name="head_norm_fwd_7b", op="head_norm_fwd", dtype="bf16", rows=16384, heads=16, dim=256, center=True,
             gate=True, weight=True),
        # and its gradients on the 3B-class layer
        dict(name="head_norm_bwd_3b", op="head_norm_bwd", dtype="bf16", rows=8192, heads=10, dim=256, center=False,
             gate=True, weight=True),
        # residual join at decode: one row a user
        dict(name="residual_fwd_decode", op="residual_fwd", dtype="bf16", rows=64, width=4096, center=False,
             post=True, scale=True),
        # its gradients over a training batch of the 7B-class layer
        dict(name="residual_bwd_7b", op="residual_bwd", dtype="bf16", rows=16384, width=4096, center=False,
             post=True, scale=True),
    ]


def _log(rng, low, high):
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["delta_fwd", "delta_fwd", "delta_bwd", "delta_bwd", "step", "head_norm_fwd", "head_norm_bwd",
                     "residual_fwd", "residual_bwd"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op in ("delta_fwd", "delta_bwd"):
        dim = rng.choice([64, 128, 256])
        k_heads = rng.randint(1, 8)
        heads = k_heads * rng.choice([1, 1, 2, 3])
        tokens = _log(rng, 1, 4096)
        # at most as much as the largest listed case, fp32 a sixteenth of it
        most = 2 * 8192 * 16 * 256 * 256 // (16 if dtype == "f32" else 1) // (6 if op == "delta_bwd" else 1)
        batch = max(1, min(rng.randint(1, 6), most // (tokens * heads * dim * dim)))
        while tokens * batch * heads * dim * dim > most:
            tokens = max(1, tokens // 2)
        lens = ""
        if rng.random() < 0.4:
            lens = [rng.randint(0, tokens) for _ in range(batch)]
            lens[rng.randrange(batch)] = tokens
            lens = ",".join(map(str, lens))
        return dict(op=op, dtype=dtype, batch=batch, tokens=tokens, k_heads=k_heads, heads=heads, dim=dim,
                    state=rng.random() < 0.6, lens=lens)
    if op == "step":
        k_heads = rng.randint(1, 16)
        batch = _log(rng, 1, 160)
        return dict(op=op, dtype=dtype, batch=batch, slots=batch + rng.choice([0, 0, 5]),
                    idle=rng.choice([0, 0, min(batch - 1, 2)]), k_heads=k_heads,
                    heads=k_heads * (rng.choice([1, 2]) if k_heads <= 8 else 1), dim=rng.choice([64, 128, 256]))
    if op.startswith("head_norm"):
        return dict(op=op, dtype=dtype, rows=_log(rng, 1, 8192), heads=rng.randint(1, 16),
                    dim=rng.choice([64, 128, 256]), center=rng.random() < 0.5, gate=rng.random() < 0.7,
                    weight=rng.random() < 0.7)
    return dict(op=op, dtype=dtype, rows=_log(rng, 1, 8192), width=_log(rng, 24, 8192), center=rng.random() < 0.4,
                post=rng.random() < 0.5, scale=rng.random() < 0.5)


def _lens(case):
    return [int(x) for x in case["lens"].split(",")] if case["lens"] else [case["tokens"]] * case["batch"]


def work(case):
    op = case["op"]
    size = 2 if case["dtype"] == "bf16" else 4
    if op.startswith("delta"):
        n, h, hk, d = sum(_lens(case)), case["heads"], case["k_heads"], case["dim"]
        qk, v, gates = n * hk * d * size, n * h * d * size, n * h * 4
        st = case["batch"] * h * d * d * 4
        if op == "delta_fwd":
            # q, k, v, log decay, beta in; o out; the state in and out. Three products of d x d a token and head
            return {"bytes": 2 * qk + 2 * v + 2 * gates + (2 * st if case["state"] else 0),
                    "flops": 6 * n * h * d * d}
        # inputs, dout in; five gradients out; the state, its two gradients. The states are formed again (two
        # products), then twice the forward's three
        return {"bytes": 4 * qk + 3 * v + 4 * gates + (3 * st if case["state"] else 0), "flops": 16 * n * h * d * d}
    if op == "step":
        b, h, hk, d = case["batch"] - case["idle"], case["heads"], case["k_heads"], case["dim"]
        return {"bytes": b * h * d * d * 8 + case["batch"] * (2 * hk + 2 * h) * d * size, "flops": 6 * b * h * d * d}
    if op.startswith("head_norm"):
        n = case["rows"] * case["heads"] * case["dim"]
        if op == "head_norm_fwd":
            return {"bytes": n * size * (3 if case["gate"] else 2), "flops": 12 * n}
        return {"bytes": n * size * (5 if case["gate"] else 3), "flops": 25 * n}
    n = case["rows"] * case["width"]
    if op == "residual_fwd":
        return {"bytes": 4 * n * size, "flops": 12 * n}
    return {"bytes": 6 * n * size, "flops": 30 * n}


# --------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _delta_inputs(case, seed, rows):
    """q, k (unit keys and queries that share a direction, as after an
    activation), v, log decay and beta of `rows` (a shape) tokens."""
    gen, dt = _gen(seed), TYPES[case["dtype"]]
    hk, h, d = case["k_heads"], case["heads"], case["dim"]
    normal = lambda *s: torch.randn(*s, generator=gen, device=DEV)  # noqa: E731
    unit = lambda x: x / x.square().sum(-1, keepdim=True).sqrt()  # noqa: E731
    common = 0.4 * normal(hk, d)
    q = unit(normal(*rows, hk, d) + common).to(dt)
    k = unit(normal(*rows, hk, d) + common).to(dt)
    v = normal(*rows, h, d).to(dt)
    beta = torch.sigmoid(normal(*rows, h))
    # heads that forget within a few tokens up to heads that keep a thousand
    rate = torch.exp(torch.linspace(math.log(0.3), math.log(0.001), h, device=DEV)) if h > 1 else 0.02
    log_decay = -rate * torch.nn.functional.softplus(normal(*rows, h))
    return gen, q, k, v, log_decay, beta


def prepare(case, seed):
    op, s = case["op"], {"case": dict(case)}
    dt = TYPES[case["dtype"]]
    if op.startswith("delta"):
        lens = _lens(case)
        packed = bool(case["lens"])
        rows = (sum(lens),) if packed else (case["batch"], case["tokens"])
        gen, s["q"], s["k"], s["v"], s["log_decay"], s["beta"] = _delta_inputs(case, seed, rows)
        b, h, d = case["batch"], case["heads"], case["dim"]
        s["scale"] = d ** -0.5
        s["state_in"] = 0.1 * torch.randn(b, h, d, d, generator=gen, device=DEV) if case["state"] else None
        if packed:
            ends = torch.tensor([0] + lens).cumsum(0)
            s["cu"], s["max"] = ends.to(torch.int32).to(DEV), max(lens)
            # where each padded place of [batch, max] lies in the packed rows, and the other way round
            t = torch.arange(max(lens))
            s["inside"] = (t[None] < torch.tensor(lens)[:, None]).to(DEV)
            s["from"] = (ends[:-1, None] + t[None]).clamp(max=max(0, sum(lens) - 1)).to(DEV)
            s["to"] = s["inside"].reshape(-1).nonzero().reshape(-1)
        if op == "delta_bwd":
            s["dout"] = torch.randn(s["v"].shape, generator=gen, device=DEV).to(dt)
            s["d_state_out"] = 0.1 * torch.randn(b, h, d, d, generator=gen, device=DEV) if case["state"] else None
    elif op == "step":
        b = case["batch"]
        gen, s["q"], s["k"], s["v"], s["log_decay"], s["beta"] = _delta_inputs(case, seed, (b, 1))
        h, d, n = case["heads"], case["dim"], case["slots"]
        s["scale"] = d ** -0.5
        s["state"] = 0.1 * torch.randn(n, h, d, d, generator=gen, device=DEV)
        s["slots"], s["active"] = None, None
        if n != b or case["idle"]:
            at = torch.randperm(n, generator=gen, device=DEV)[:b].to(torch.int32)
            off = torch.randperm(b, generator=gen, device=DEV)[: case["idle"]]
            at[off] = -1
            s["slots"], s["active"] = at, (at >= 0).nonzero().reshape(-1)
    elif op.startswith("head_norm"):
        gen = _gen(seed)
        shape = (case["rows"], case["heads"], case["dim"])
        normal = lambda *x: torch.randn(*x, generator=gen, device=DEV)  # noqa: E731
        s["x"] = (normal(*shape) * torch.exp(normal(case["rows"], case["heads"], 1)) + 0.2).to(dt)
        s["gate"] = normal(*shape).to(dt) if case["gate"] else None
        s["weight"] = 1 + 0.1 * normal(case["dim"]) if case["weight"] else None
        s["dout"] = normal(*shape).to(dt) if op == "head_norm_bwd" else None
    else:
        gen = _gen(seed)
        shape = (case["rows"], case["width"])
        normal = lambda *x: torch.randn(*x, generator=gen, device=DEV)  # noqa: E731
        s["x"], s["y"] = (2 * normal(*shape)).to(dt), (normal(*shape) + 0.1).to(dt)
        s["weight"] = 1 + 0.1 * normal(case["width"])
        s["post"] = 1 + 0.1 * normal(case["width"]) if case["post"] else None
        s["scale"] = 0.5 + 0.1 * normal(case["width"]) if case["scale"] else None
        s["skip"] = 0.875
        if op == "residual_bwd":
            s["dout"], s["dres"] = normal(*shape).to(dt), normal(*shape).to(dt)
    return s


# --------------------------------------------------------------------------
# Plain forms
# --------------------------------------------------------------------------
def _plain_delta(q, k, v, log_decay, beta, scale, state):
    """[batch, tokens, heads, ...] in 32 bits, blocks of 64 tokens: inside a
    block the writes solve a unit triangular system, the state goes from
    block to block. Returns (o, state)."""
    b, n, hk, d = q.shape
    h = v.shape[2]
    nb = -(-n // BLOCK)
    if h != hk:
        q, k = q.repeat_interleave(h // hk, 2), k.repeat_interleave(h // hk, 2)

    def blocks(x):  # [b, n, h, e] -> [nb, b * h, BLOCK, e], zeros behind the end
        x = torch.cat([x, x.new_zeros(b, nb * BLOCK - n, h, x.shape[-1])], 1)
        return x.reshape(b, nb, BLOCK, h, -1).permute(1, 0, 3, 2, 4).reshape(nb, b * h, BLOCK, -1)

    q, k, v = blocks(q), blocks(k), blocks(v)
    beta = blocks(beta[..., None])
    g = blocks(log_decay[..., None]).double().cumsum(2)
    low = torch.ones(BLOCK, BLOCK, device=q.device, dtype=torch.bool).tril()
    decay = torch.where(low, g - g.transpose(2, 3), -math.inf).exp()
    kt = k.transpose(2, 3)
    a = torch.where(low.tril(-1), beta * decay * torch.matmul(k, kt), 0.0)  # 64 bits, as `decay`
    # (I + A)^-1 = (I - A)(I + A^2)(I + A^4)...: A^64 is zero
    eye = torch.eye(BLOCK, device=q.device, dtype=torch.float64)
    inv, power = eye - a, a
    for _ in range(5):
        power = torch.matmul(power, power)
        inv = torch.matmul(inv, eye + power)
    inv = inv.float()
    p = scale * (torch.matmul(q, kt) * decay.float())
    qe, ke = q * (scale * g.exp()).float(), k * g.exp().float()
    kl = (k * (g[:, :, -1:] - g).exp().float()).transpose(2, 3)
    last = g[:, :, -1:].exp().float()
    if state is None:
        s = q.new_zeros(b * h, d, d)
    else:
        s = state.reshape(b * h, d, d)
    out = []
    for i in range(nb):
        u = torch.matmul(inv[i], beta[i] * (v[i] - torch.matmul(ke[i], s)))
        out.append(torch.matmul(qe[i], s) + torch.matmul(p[i], u))
        s = last[i] * s + torch.matmul(kl[i], u)
    o = torch.stack(out).reshape(nb, b, h, BLOCK, d).permute(1, 0, 3, 2, 4).reshape(b, nb * BLOCK, h, d)
    return o[:, :n], s.reshape(b, h, d, d)


def _padded(s, x):
    """Packed rows as [batch, max, ...], zeros behind each sequence's end."""
    return x[s["from"]] * s["inside"].reshape(s["inside"].shape + (1,) * (x.dim() - 1))


def _plain_delta_of(s, q, k, v, log_decay, beta, state):
    if "cu" not in s:
        return _plain_delta(q, k, v, log_decay, beta, s["scale"], state)
    o, st = _plain_delta(*(_padded(s, x) for x in (q, k, v, log_decay, beta)), s["scale"], state)
    return o.reshape(-1, *o.shape[2:])[s["to"]], st


def _norm(x, center, eps):
    if center:
        x = x - x.mean(-1, keepdim=True)
    return x / (x.square().mean(-1, keepdim=True) + eps).sqrt()


def _plain_head_norm(x, weight, gate, center):
    y = _norm(x, center, 1e-5)
    if weight is not None:
        y = y * weight
    if gate is not None:
        y = y * (gate / (1 + torch.exp(-gate)))
    return y


def _plain_residual(x, y, weight, post, scale, skip, center):
    if post is not None:
        y = _norm(y, center, 1e-5) * post
    if scale is not None:
        y = y * scale
    h = skip * x + y
    return _norm(h, center, 1e-5) * weight, h


def _f(x):
    return None if x is None else x.float()


def _grads(outs, douts, inputs):
    """Gradients of the named inputs (None where there is no input)."""
    given = [x for x in inputs if x is not None]
    pairs = [(o, g) for o, g in zip(outs, douts) if g is not None]
    got = iter(torch.autograd.grad([o for o, _ in pairs], given, [g for _, g in pairs]))
    return [None if x is None else next(got) for x in inputs]


def _leaf(x):
    return None if x is None else x.detach().float().requires_grad_()


def _plain(s):
    op = s["case"]["op"]
    if op == "delta_fwd":
        o, st = _plain_delta_of(s, *(s[x].float() for x in ("q", "k", "v", "log_decay", "beta")), s["state_in"])
        return {"o": o.to(s["v"].dtype), "state": st if s["case"]["state"] else None}
    if op == "delta_bwd":
        leaves = [_leaf(s[x]) for x in ("q", "k", "v", "log_decay", "beta", "state_in")]
        outs = _plain_delta_of(s, *leaves)
        g = _grads(outs, (s["dout"].float(), s["d_state_out"]), leaves)
        dt = s["q"].dtype
        return {"dq": g[0].to(dt), "dk": g[1].to(dt), "dv": g[2].to(dt), "dlog_decay": g[3], "dbeta": g[4],
                "dstate": g[5]}
    if op == "step":
        pool, at = s["state"], s["slots"]
        q, k, v = (s[x][:, 0].float() for x in ("q", "k", "v"))
        a, beta = s["log_decay"][:, 0].exp(), s["beta"][:, 0]
        r = v.shape[1] // q.shape[1]
        q, k = q.repeat_interleave(r, 1), k.repeat_interleave(r, 1)
        if at is not None:
            act = s["active"]
            q, k, v, a, beta = (x[act] for x in (q, k, v, a, beta))
            st = pool[at[act].long()]
        else:
            st = pool
        st = st * a[..., None, None]
        u = beta[..., None] * (v - (st * k[..., None]).sum(2))
        st = st + k[..., None] * u[..., None, :]
        o = s["scale"] * (st * q[..., None]).sum(2)
        if at is not None:
            pool[at[act].long()] = st
            full = s["v"].new_zeros(s["v"].shape)
            full[act, 0] = o.to(full.dtype)
            return {"o": full, "state": pool}
        pool.copy_(st)
        return {"o": o[:, None].to(s["v"].dtype), "state": pool}
    if op == "head_norm_fwd":
        y = _plain_head_norm(s["x"].float(), s["weight"], _f(s["gate"]), s["case"]["center"])
        return {"y": y.to(s["x"].dtype)}
    if op == "head_norm_bwd":
        leaves = [_leaf(s[x]) for x in ("x", "weight", "gate")]
        g = _grads([_plain_head_norm(*leaves, s["case"]["center"])], [s["dout"].float()], leaves)
        return {"dx": g[0].to(s["x"].dtype), "dweight": g[1], "dgate": None if g[2] is None else g[2].to(s["x"].dtype)}
    if op == "residual_fwd":
        y, h = _plain_residual(s["x"].float(), s["y"].float(), s["weight"], s["post"], s["scale"], s["skip"],
                               s["case"]["center"])
        return {"y": y.to(s["x"].dtype), "residual": h.to(s["x"].dtype)}
    leaves = [_leaf(s[x]) for x in ("x", "y", "weight", "post", "scale")]
    outs = _plain_residual(*leaves, s["skip"], s["case"]["center"])
    g = _grads(outs, [s["dout"].float(), s["dres"].float()], leaves)
    dt = s["x"].dtype
    return {"dx": g[0].to(dt), "dy": g[1].to(dt), "dweight": g[2], "dpost": g[3], "dscale": g[4]}


# --------------------------------------------------------------------------
# The framework's calls
# --------------------------------------------------------------------------
def _own(s):
    import retnet_retention_amd as rr

    case = s["case"]
    op = case["op"]
    if op.startswith("delta"):
        args = [s[x] for x in ("q", "k", "v", "log_decay", "beta")]
        more = dict(scale=s["scale"], state_in=s["state_in"])
        if "cu" in s:
            more.update(cu_seqlens=s["cu"], max_seqlen=s["max"])
        if op == "delta_fwd":
            st = torch.empty_like(s["state_in"]) if case["state"] else None
            return {"o": rr.delta_chunkwise_fwd(*args, state_out=st, **more), "state": st}
        g = rr.delta_chunkwise_bwd(*args, s["dout"], d_state_out=s["d_state_out"], **more)
        return {"dq": g[0], "dk": g[1], "dv": g[2], "dlog_decay": g[3], "dbeta": g[4],
                "dstate": g[5] if case["state"] else None}
    if op == "step":
        o = rr.delta_recurrent_step(s["q"], s["k"], s["v"], s["log_decay"], s["beta"], s["state"], scale=s["scale"],
                                    slots=s["slots"])
        return {"o": o, "state": s["state"]}
    if op == "head_norm_fwd":
        return {"y": rr.head_norm_fwd(s["x"], s["weight"], s["gate"], center=case["center"])}
    if op == "head_norm_bwd":
        g = rr.head_norm_bwd(s["x"], s["dout"], s["weight"], s["gate"], center=case["center"])
        return {"dx": g[0], "dweight": g[1], "dgate": g[2]}
    more = dict(post_weight=s["post"], scale=s["scale"], skip=s["skip"], center=case["center"])
    if op == "residual_fwd":
        y, h = rr.residual_norm_fwd(s["x"], s["y"], s["weight"], **more)
        return {"y": y, "residual": h}
    g = rr.residual_norm_bwd(s["x"], s["y"], s["weight"], s["dout"], s["dres"], **more)
    return {"dx": g[0], "dy": g[1], "dweight": g[2], "dpost": g[3], "dscale": g[4]}


def run(state):
    return _own(state) if own else _plain(state)


# --------------------------------------------------------------------------
# From the definitions, in 64 bits: the delta rule token by token (its
# gradients by the reversed recurrence over states formed again from a kept one
# every 64 tokens), the norms' gradients from their formulas.
# --------------------------------------------------------------------------
def _token(st, k, v, a, beta):
    """One token's write: (decayed state, residual v - S'k, new state)."""
    dec = st * a[..., None, None]
    res = v - torch.matmul(k[..., None, :], dec)[..., 0, :]
    return dec, res, dec + k[..., None] * (beta[..., None] * res)[..., None, :]


def _dims(s):
    """The delta inputs in 64 bits, time first, key heads spread over value heads."""
    r = s["case"]["heads"] // s["case"]["k_heads"]
    seqs = []
    for name in ("q", "k", "v", "log_decay", "beta", "dout"):
        if name not in s:
            seqs.append(None)
            continue
        x = s[name].double()
        if "cu" in s:
            x = _padded(s, x)
        if name in ("q", "k"):
            x = x.repeat_interleave(r, 2)
        seqs.append(x.transpose(0, 1).contiguous())
    c = s["case"]
    st = s["state_in"].double() if s["state_in"] is not None else torch.zeros(
        c["batch"], c["heads"], c["dim"], c["dim"], device=DEV, dtype=torch.float64)
    return seqs, st


def _unpad(s, x):
    x = x.transpose(0, 1)
    return x.reshape(-1, *x.shape[2:])[s["to"]] if "cu" in s else x


def _exact_delta(s):
    (q, k, v, ld, beta, dout), st = _dims(s)
    n, a, scale = q.shape[0], ld.exp(), s["scale"]
    o, kept = torch.empty_like(v), []
    for t in range(n):
        if dout is not None and t % 64 == 0:
            kept.append(st)
        st = _token(st, k[t], v[t], a[t], beta[t])[2]
        if dout is None:
            o[t] = scale * torch.matmul(q[t][..., None, :], st)[..., 0, :]
    if dout is None:
        return {"o": _unpad(s, o), "state": st if s["case"]["state"] else None}
    dq, dk, dv, dld, dbeta = (torch.zeros_like(x) for x in (q, k, v, ld, beta))
    ds = s["d_state_out"].double().clone() if s["d_state_out"] is not None else torch.zeros_like(st)
    for b0 in reversed(range(0, n, 64)):
        st, hist = kept[b0 // 64], []
        for t in range(b0, min(n, b0 + 64)):
            hist.append(_token(st, k[t], v[t], a[t], beta[t]))
            st = hist[-1][2]
        for t in reversed(range(b0, min(n, b0 + 64))):
            dec, res, new = hist.pop()
            ds = ds + q[t][..., None] * (scale * dout[t])[..., None, :]
            dq[t] = scale * torch.matmul(new, dout[t][..., None])[..., 0]
            u = beta[t][..., None] * res
            du = torch.matmul(k[t][..., None, :], ds)[..., 0, :]
            dbeta[t] = (du * res).sum(-1)
            dv[t] = beta[t][..., None] * du
            dk[t] = torch.matmul(ds, u[..., None])[..., 0] - torch.matmul(dec, dv[t][..., None])[..., 0]
            ds = ds - k[t][..., None] * dv[t][..., None, :]
            dld[t] = (ds * dec).sum((-1, -2))
            ds = ds * a[t][..., None, None]
    r = s["case"]["heads"] // s["case"]["k_heads"]
    shared = lambda x: x.reshape(*x.shape[:2], -1, r, x.shape[-1]).sum(3)  # noqa: E731
    return {"dq": _unpad(s, shared(dq)), "dk": _unpad(s, shared(dk)), "dv": _unpad(s, dv), "dlog_decay": _unpad(s, dld),
            "dbeta": _unpad(s, dbeta), "dstate": ds if s["case"]["state"] else None}


def _exact_step(s):
    r = s["case"]["heads"] // s["case"]["k_heads"]
    q, k = (s[x][:, 0].double().repeat_interleave(r, 1) for x in ("q", "k"))
    v, a, beta = s["v"][:, 0].double(), s["log_decay"][:, 0].double().exp(), s["beta"][:, 0].double()
    pool = s["state"].double()
    out = torch.zeros_like(v)
    at = range(v.shape[0]) if s["slots"] is None else s["slots"].tolist()
    for i, slot in enumerate(at):
        if slot >= 0:
            pool[slot] = _token(pool[slot], k[i], v[i], a[i], beta[i])[2]
            out[i] = s["scale"] * torch.matmul(q[i][:, None, :], pool[slot])[:, 0, :]
    return {"o": out[:, None], "state": pool}


def _stats(x, center):
    """(normalised x, 1 / its deviation) from the sums of x and x^2."""
    d = x.shape[-1]
    mean = x.sum(-1, keepdim=True) / d if center else torch.zeros_like(x[..., :1])
    rstd = ((x * x).sum(-1, keepdim=True) / d - mean * mean + 1e-5) ** -0.5
    return (x - mean) * rstd, rstd


def _norm_grad(n, rstd, dn, center):
    """d x of n = normalised x, given d n."""
    g = dn - n * (dn * n).mean(-1, keepdim=True)
    return rstd * (g - dn.mean(-1, keepdim=True)) if center else rstd * g


def _exact_head_norm(s):
    x, center = s["x"].double(), s["case"]["center"]
    n, rstd = _stats(x, center)
    w = s["weight"].double() if s["weight"] is not None else torch.ones(x.shape[-1], device=DEV, dtype=torch.float64)
    sig = torch.sigmoid(s["gate"].double()) if s["gate"] is not None else None
    act = s["gate"].double() * sig if sig is not None else torch.ones_like(x)
    if s["dout"] is None:
        return {"y": n * w * act}
    dy = s["dout"].double()
    return {"dx": _norm_grad(n, rstd, dy * act * w, center),
            "dweight": (dy * act * n).sum((0, 1)) if s["weight"] is not None else None,
            "dgate": dy * n * w * (sig + act * (1 - sig)) if sig is not None else None}


def _exact_residual(s):
    x, y, center = s["x"].double(), s["y"].double(), s["case"]["center"]
    one = torch.ones(x.shape[-1], device=DEV, dtype=torch.float64)
    post = s["post"].double() if s["post"] is not None else one
    scale = s["scale"].double() if s["scale"] is not None else one
    w = s["weight"].double()
    ny, ry = _stats(y, center) if s["post"] is not None else (y, None)
    z = ny * post
    h = s["skip"] * x + scale * z
    nh, rh = _stats(h, center)
    if "dout" not in s:
        return {"y": nh * w, "residual": h}
    dout = s["dout"].double()
    dh = s["dres"].double() + _norm_grad(nh, rh, dout * w, center)
    dz = dh * scale
    return {"dx": s["skip"] * dh, "dy": _norm_grad(ny, ry, dz * post, center) if ry is not None else dz,
            "dweight": (dout * nh).sum(0), "dpost": (dz * ny).sum(0) if ry is not None else None,
            "dscale": (dh * z).sum(0) if s["scale"] is not None else None}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op.startswith("delta"):
        return _exact_delta(s)
    return _exact_step(s) if op == "step" else _exact_head_norm(s) if op.startswith("head_norm") else _exact_residual(s)
