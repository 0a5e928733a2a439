"""Cases that time the layer's surrounding operators: the short causal convolution, the selective
state space scan and the group norm with its gate, forward, backward and for single tokens.

``own`` False computes each operator in elementary torch operations in 32 bits, rounded once;
``own`` True calls the framework's kernels on the same inputs."""
import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_EPS = 1e-5


def listed():
    return [
        # one decoded token for each of 64 sequences: launch latency
        dict(name="conv decode 64", op="conv_step", B=64, D=2048, W=4, dtype="bf16"),
        # right-padded prompts of unequal length over a channel count that no vector width divides
        dict(name="conv ragged prompts", op="conv_fwd", B=7, T=1900, D=1923, W=4, dtype="bf16", lens=True, state=True),
        # the training shape of the layer: 8 sequences of 4096 tokens, 16 heads of 128 channels
        dict(name="conv training gradients", op="conv_bwd", B=8, T=4096, D=2048, W=4, dtype="bf16", state=False),
        # one decoded token for each of 256 sequences, 16 heads of 128 channels, 16 states a channel
        dict(name="scan decode 256", op="ssm_step", B=256, D=2048, G=1, N=16, dtype="bf16"),
        # a single long prompt: few channels, so the time axis is all there is to split
        dict(name="scan long prompt", op="ssm_fwd", B=1, T=16384, D=2048, G=1, N=16, dtype="bf16", lens=False,
             state=True, gate=True, softplus=True),
        # the training shape, forward
        dict(name="scan training forward", op="ssm_fwd", B=8, T=4096, D=2048, G=1, N=16, dtype="bf16", lens=False,
             state=False, gate=True, softplus=True),
        # the training shape's gradients
        dict(name="scan training gradients", op="ssm_bwd", B=8, T=2048, D=2048, G=1, N=16, dtype="bf16", state=False,
             gate=True, softplus=True),
        # a small fp32 layer with two groups of B and C, odd sizes and a state carried in and out
        dict(name="scan small gradients", op="ssm_bwd", B=3, T=203, D=142, G=2, N=32, dtype="f32", state=True,
             gate=False, softplus=False),
        # one decoded token for each of 64 sequences, norm over each head, gated
        dict(name="norm decode 64", op="norm_fwd", B=64, L=1, G=16, E=128, dtype="bf16", gate=True, silu=False),
        # every token of the training shape, norm over each head, gated
        dict(name="norm training forward", op="norm_fwd", B=32768, L=1, G=16, E=128, dtype="bf16", gate=True, silu=False),
        dict(name="norm training gradients", op="norm_bwd", B=32768, L=1, G=16, E=128, dtype="bf16", gate=True, silu=False),
        # statistics over a whole sequence, channels last, with the activation, fp32
        dict(name="norm over sequences", op="norm_fwd", B=8, L=4000, G=32, E=30, dtype="f32", gate=False, silu=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["conv_step", "conv_fwd", "conv_bwd", "ssm_step", "ssm_fwd", "ssm_bwd", "norm_fwd", "norm_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    odd = rng.random() < 0.4
    if op.startswith("norm"):
        E = _log(rng, 8, 512)
        E = E | 1 if odd else (E + 7) // 8 * 8
        L = 1 if rng.random() < 0.6 else _log(rng, 2, 4096)
        G = rng.choice([1, 4, 8, 16, 32])
        B = min(_log(rng, 1, 32768), max(1, (1 << 25) // (L * G * E)))
        gate = rng.random() < 0.5
        return dict(op=op, B=B, L=L, G=G, E=E, dtype=dtype, gate=gate, silu=not gate)
    G = rng.choice([1, 1, 2, 4])
    D = _log(rng, 48, 4096)
    D = D | 1 if odd else (D + 7) // 8 * 8
    if op == "conv_step":
        return dict(op=op, B=_log(rng, 1, 1024), D=D, W=rng.choice([2, 3, 4]), dtype=dtype)
    B = _log(rng, 1, 16)
    if op.startswith("conv"):
        T = min(_log(rng, 1, 16384), (1 << 26) // (B * D))
        c = dict(op=op, B=B, T=T, D=D, W=rng.choice([2, 3, 4]), dtype=dtype, state=rng.random() < 0.5)
        return dict(c, lens=rng.random() < 0.5) if op == "conv_fwd" else c
    N = rng.choice([16, 16, 32, 64])
    D = (D + G - 1) // G * G
    if op == "ssm_step":
        return dict(op=op, B=min(_log(rng, 1, 1024), (1 << 25) // (D * N)), D=D, G=G, N=N, dtype=dtype)
    T = max(1, min(_log(rng, 1, 16384), (1 << 28) // (B * D * N)))
    c = dict(op=op, B=B, T=T, D=D, G=G, N=N, dtype=dtype, state=rng.random() < 0.5, gate=rng.random() < 0.6,
             softplus=rng.random() < 0.7)
    return dict(c, lens=rng.random() < 0.4) if op == "ssm_fwd" else c


def prepare(case, seed):
    dt = _TYPES[case["dtype"]]
    rng = torch.Generator(device="cuda")
    rng.manual_seed(int(seed))
    r = lambda *s: torch.randn(*s, generator=rng, device="cuda")  # noqa: E731
    op, B = case["op"], case["B"]
    s = dict(case=dict(case))
    if op.startswith("norm"):
        L, G, E = case["L"], case["G"], case["E"]
        C = G * E
        s["x"] = (r(B, L, C) * 1.5 + 0.3 * r(C)).to(dt)
        s["weight"], s["bias"] = 1 + 0.1 * r(C), 0.1 * r(C)
        s["gate"] = r(B, L, C).to(dt) if case["gate"] else None
        if op == "norm_bwd":
            s["dy"] = r(B, L, C).to(dt)
            x = s["x"].float().reshape(B, L, G, E)
            mean = x.mean((1, 3))
            var = (x - mean[:, None, :, None]).square().mean((1, 3))
            s["stats"] = torch.stack([mean, torch.rsqrt(var + _EPS)], -1).contiguous()
        return s
    D = case["D"]
    if op.startswith("conv"):
        W = case["W"]
        s["w"], s["bias"] = 0.5 * r(D, W), 0.1 * r(D)
        if op == "conv_step":
            s["x"], s["S"] = r(B, D).to(dt), r(B, W - 1, D).to(dt)
            return s
        T = case["T"]
        s["x"] = r(B, T, D).to(dt)
        s["S0"] = r(B, W - 1, D).to(dt) if case["state"] else None
    else:
        G, N = case["G"], case["N"]
        T = case.get("T")
        tok = (B,) if op == "ssm_step" else (B, T)
        s["u"] = r(*tok, D).to(dt)
        if case.get("softplus", True):
            s["dt"], s["dt_bias"] = (0.5 * r(*tok, D)).to(dt), r(D) - 4
        else:
            s["dt"], s["dt_bias"] = torch.exp(0.5 * r(*tok, D) - 4).to(dt), None
        s["Bm"], s["Cm"] = r(*tok, G, N).to(dt), r(*tok, G, N).to(dt)
        s["A"] = -torch.arange(1, N + 1, device="cuda") * torch.exp(0.1 * r(D, N))
        s["D"] = 1 + 0.1 * r(D)
        s["z"] = r(*tok, D).to(dt) if case.get("gate", True) else None
        if op == "ssm_step":
            s["S"] = 0.1 * r(B, D, N)
            return s
        s["S0"] = 0.1 * r(B, D, N) if case["state"] else None
    if case.get("lens"):
        s["lens"] = torch.randint(0, T + 1, (B,), generator=rng, device="cuda", dtype=torch.int32)
    if op.endswith("fwd"):
        s["y"] = torch.zeros(B, T, D, dtype=dt, device="cuda")  # rows past a sequence's length stay as they are
    else:
        s["dy"] = r(B, T, D).to(dt)
        s["dS_T"] = None
        if case["state"]:
            s["dS_T"] = (r(B, case["W"] - 1, D).to(dt) if op == "conv_bwd" else 0.1 * r(B, D, case["N"]))
    return s


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    op, B = case["op"], case["B"]
    if op.startswith("norm"):
        n = B * case["L"] * case["G"] * case["E"]
        streams = (2 if op == "norm_fwd" else 3) + (0 if not case["gate"] else 1 if op == "norm_fwd" else 2)
        return dict(bytes=n * e * streams, flops=n * ((8 if op == "norm_fwd" else 18) + (6 if case["gate"] else 0)))
    D, T = case["D"], case.get("T", 1)
    n = B * T * D
    if op.startswith("conv"):
        W = case["W"]
        if op == "conv_step":
            return dict(bytes=n * e * (2 + 2 * (W - 1)), flops=n * (2 * W + 4))
        return dict(bytes=n * e * (2 if op == "conv_fwd" else 3) + D * W * 4, flops=n * ((2 if op == "conv_fwd" else 6) * W + 8))
    N, gate = case["N"], 1 if case.get("gate", True) else 0
    bc = 2 * B * T * case["G"] * N * e
    if op == "ssm_step":
        return dict(bytes=n * e * (3 + gate) + bc + 2 * B * D * N * 4, flops=n * (7 * N + 16))
    if op == "ssm_fwd":
        return dict(bytes=n * e * (3 + gate) + bc, flops=n * (7 * N + 16))
    return dict(bytes=n * e * (5 + 2 * gate) + 2 * bc, flops=n * (20 * N + 40))


# ---------------------------------------------------------------- the plain form

def _silu(x):
    return x / (1 + torch.exp(-x))


def _dsilu(x):
    p = 1 / (1 + torch.exp(-x))
    return p * (1 + x * (1 - p))


def _softplus(x):
    return torch.clamp(x, min=0) + torch.log1p(torch.exp(-torch.abs(x)))


def _scan(a, b):
    """h[:, t] = a[:, t] h[:, t-1] + b[:, t] from h[:, -1] = 0, by doubling over the time axis."""
    step = 1
    while step < a.shape[1]:
        b = torch.cat([b[:, :step], b[:, step:] + a[:, step:] * b[:, :-step]], 1)
        a = torch.cat([a[:, :step], a[:, step:] * a[:, :-step]], 1)
        step *= 2
    return b


def _padded(s, W):
    x = s["x"].float()
    first = x.new_zeros(x.shape[0], W - 1, x.shape[2]) if s["S0"] is None else s["S0"].float()
    return torch.cat([first, x], 1)


def _taps(full, w, T):
    W = w.shape[1]
    return sum(full[:, j:j + T] * w[:, j] for j in range(W))


def _conv_step(s):
    x = torch.cat([s["S"], s["x"][:, None]], 1)
    pre = (x.float() * s["w"].t()).sum(1) + s["bias"]
    s["S"].copy_(x[:, 1:])
    return _silu(pre).to(x.dtype), s["S"]


def _conv_fwd(s):
    T, W = s["x"].shape[1], s["w"].shape[1]
    full = _padded(s, W)
    y = _silu(_taps(full, s["w"], T) + s["bias"]).to(s["x"].dtype)
    if "lens" not in s:
        return y, full[:, T:].to(y.dtype)
    past = torch.arange(T, device=y.device) >= s["lens"][:, None]
    at = s["lens"].long()[:, None] + torch.arange(W - 1, device=y.device)
    state = full.gather(1, at[:, :, None].expand(-1, -1, full.shape[2]))
    return torch.where(past[:, :, None], s["y"], y), state.to(y.dtype)


def _conv_bwd(s):
    T, W = s["x"].shape[1], s["w"].shape[1]
    full, w, dt = _padded(s, W), s["w"], s["x"].dtype
    dpre = s["dy"].float() * _dsilu(_taps(full, w, T) + s["bias"])
    dw = torch.stack([(dpre * full[:, j:j + T]).sum((0, 1)) for j in range(W)], 1)
    edge = dpre.new_zeros(dpre.shape[0], W - 1, dpre.shape[2])
    wide = torch.cat([edge, dpre, edge], 1)
    dfull = _taps(wide, w.flip(1), T + W - 1)
    if s["dS_T"] is not None:
        dfull[:, T:] += s["dS_T"].float()
    out = dict(dx=dfull[:, W - 1:].to(dt), dw=dw, dbias=dpre.sum((0, 1)))
    if s["S0"] is not None:
        out["dS0"] = dfull[:, :W - 1].to(dt)
    return out


def _delta(s):
    x = s["dt"].float()
    return _softplus(x + s["dt_bias"]) if s["dt_bias"] is not None else x


def _per_channel(m, D):
    """B or C [.., G, N] as [.., D, N]: the group's row for each of its channels."""
    G = m.shape[-2]
    return m.float()[..., :, None, :].expand(*m.shape[:-1], D // G, m.shape[-1]).reshape(*m.shape[:-2], D, m.shape[-1])


def _states(s):
    delta, u = _delta(s), s["u"].float()
    D = u.shape[-1]
    a = torch.exp(delta[..., None] * s["A"])
    b = (delta * u)[..., None] * _per_channel(s["Bm"], D)
    if "lens" in s:
        past = (torch.arange(u.shape[1], device=u.device) >= s["lens"][:, None])[:, :, None, None]
        a, b = torch.where(past, 1.0, a), torch.where(past, 0.0, b)
    if s["S0"] is not None:
        b[:, 0] += a[:, 0] * s["S0"]
    return delta, u, a, _scan(a, b)


def _ssm_fwd(s):
    delta, u, a, h = _states(s)
    y = (h * _per_channel(s["Cm"], u.shape[-1])).sum(-1) + s["D"] * u
    if s["z"] is not None:
        y = y * _silu(s["z"].float())
    y = y.to(s["u"].dtype)
    if "lens" in s:
        past = torch.arange(u.shape[1], device=u.device) >= s["lens"][:, None]
        y = torch.where(past[:, :, None], s["y"], y)
    return y, h[:, -1].clone()


def _ssm_step(s):
    delta, u = _delta(s), s["u"].float()
    D = u.shape[-1]
    h = torch.exp(delta[..., None] * s["A"]) * s["S"] + (delta * u)[..., None] * _per_channel(s["Bm"], D)
    s["S"].copy_(h)
    y = (h * _per_channel(s["Cm"], D)).sum(-1) + s["D"] * u
    return (y * _silu(s["z"].float())).to(s["u"].dtype), s["S"]


def _ssm_bwd(s):
    delta, u, a, h = _states(s)
    B, T, D = u.shape
    G, N = s["Bm"].shape[2:]
    dt, do = s["u"].dtype, s["dy"].float()
    Bd, Cd = _per_channel(s["Bm"], D), _per_channel(s["Cm"], D)
    out = {}
    dy = do
    if s["z"] is not None:
        z = s["z"].float()
        dy = do * _silu(z)
        out["dz"] = (do * ((h * Cd).sum(-1) + s["D"] * u) * _dsilu(z)).to(dt)
    c = Cd * dy[..., None]
    if s["dS_T"] is not None:
        c[:, -1] += s["dS_T"]
    late = torch.cat([a[:, 1:], torch.zeros_like(a[:, :1])], 1)
    g = _scan(late.flip(1), c.flip(1)).flip(1)
    del late, c
    fold = lambda v: v.reshape(B, T, G, D // G, N).sum(3).to(dt)  # noqa: E731
    out["dC"] = fold(h * dy[..., None])
    out["dB"] = fold(g * (delta * u)[..., None])
    gB = (g * Bd).sum(-1)
    ga = g * a
    before = torch.zeros_like(h[:, :1]) if s["S0"] is None else s["S0"][:, None]
    q = ga * torch.cat([before, h[:, :-1]], 1)
    out["dA"] = (q * delta[..., None]).sum((0, 1))
    ddelta = (q * s["A"]).sum(-1) + u * gB
    out["du"] = (delta * gB + s["D"] * dy).to(dt)
    out["dD"] = (dy * u).sum((0, 1))
    if s["dt_bias"] is not None:
        ddelta = ddelta / (1 + torch.exp(-(s["dt"].float() + s["dt_bias"])))
        out["ddt_bias"] = ddelta.sum((0, 1))
    out["ddt"] = ddelta.to(dt)
    if s["S0"] is not None:
        out["dS0"] = ga[:, 0].clone()
    return out


def _norm_fwd(s):
    c = s["case"]
    B, L, G, E = c["B"], c["L"], c["G"], c["E"]
    x = s["x"].float().reshape(B, L, G, E)
    mean = x.mean((1, 3))
    d = x - mean[:, None, :, None]
    rstd = 1 / torch.sqrt(d.square().mean((1, 3)) + _EPS)
    v = (d * rstd[:, None, :, None]).reshape(B, L, G * E) * s["weight"] + s["bias"]
    y = _silu(v) if c["silu"] else v
    if s["gate"] is not None:
        y = y * _silu(s["gate"].float())
    return y.to(s["x"].dtype), torch.stack([mean, rstd], -1)


def _norm_bwd(s):
    c = s["case"]
    B, L, G, E = c["B"], c["L"], c["G"], c["E"]
    dt = s["x"].dtype
    mean, rstd = s["stats"][..., 0][:, None, :, None], s["stats"][..., 1][:, None, :, None]
    xhat = (s["x"].float().reshape(B, L, G, E) - mean) * rstd
    flat = xhat.reshape(B, L, G * E)
    v = flat * s["weight"] + s["bias"]
    dv = s["dy"].float()
    out = {}
    if s["gate"] is not None:
        z = s["gate"].float()
        out["dgate"] = (dv * (_silu(v) if c["silu"] else v) * _dsilu(z)).to(dt)
        dv = dv * _silu(z)
    if c["silu"]:
        dv = dv * _dsilu(v)
    out["dweight"], out["dbias"] = (dv * flat).sum((0, 1)), dv.sum((0, 1))
    gw = (dv * s["weight"]).reshape(B, L, G, E)
    a, b = gw.mean((1, 3), keepdim=True), (gw * xhat).mean((1, 3), keepdim=True)
    out["dx"] = ((gw - a - xhat * b) * rstd).reshape(B, L, G * E).to(dt)
    return out


# ---------------------------------------------------------------- the framework's calls

def _own(s):
    import recurrent_sequence_layers_amd as qd
    op = s["case"]["op"]
    if op == "conv_step":
        return qd.qdelta_conv_step(s["x"], s["w"], s["bias"], s["S"]), s["S"]
    if op == "conv_fwd":
        return qd.qdelta_conv_fwd(s["x"], s["w"], s["bias"], s["S0"], lens=s.get("lens"), y=s["y"])
    if op == "conv_bwd":
        got = qd.qdelta_conv_bwd(s["x"], s["w"], s["bias"], s["S0"], s["dy"], s["dS_T"], want_dS0=s["S0"] is not None)
    elif op == "ssm_step":
        return qd.qdelta_ssm_step(s["u"], s["dt"], s["A"], s["Bm"], s["Cm"], s["D"], s["z"], s["dt_bias"], s["S"]), s["S"]
    elif op == "ssm_fwd":
        return qd.qdelta_ssm_fwd(s["u"], s["dt"], s["A"], s["Bm"], s["Cm"], s["D"], s["z"], s["dt_bias"], s["S0"],
                                 softplus=s["case"]["softplus"], lens=s.get("lens"), o=s["y"])
    elif op == "ssm_bwd":
        got = qd.qdelta_ssm_bwd(s["u"], s["dt"], s["A"], s["Bm"], s["Cm"], s["D"], s["z"], s["dt_bias"], s["S0"],
                                s["dy"], s["dS_T"], softplus=s["case"]["softplus"], want_dS0=s["S0"] is not None)
    elif op == "norm_fwd":
        return qd.qdelta_group_norm_fwd(s["x"], s["case"]["G"], s["weight"], s["bias"], s["gate"], silu=s["case"]["silu"],
                                        eps=_EPS)
    else:
        got = qd.qdelta_group_norm_bwd(s["x"], s["case"]["G"], s["weight"], s["bias"], s["gate"], s["stats"], s["dy"],
                                       silu=s["case"]["silu"])
    return {k: v for k, v in got.items() if v is not None}


def run(state):
    if own:
        return _own(state)
    return dict(conv_step=_conv_step, conv_fwd=_conv_fwd, conv_bwd=_conv_bwd, ssm_step=_ssm_step, ssm_fwd=_ssm_fwd,
                ssm_bwd=_ssm_bwd, norm_fwd=_norm_fwd, norm_bwd=_norm_bwd)[state["case"]["op"]](state)


# ---------------------------------------------------------------- the definition in 64 bits

def _sig64(x):
    return torch.special.expit(x)


def _conv64(s, op):
    w, bias = s["w"].double(), s["bias"].double()
    W = w.shape[1]
    if op == "conv_step":
        rows = torch.cat([s["S"], s["x"][:, None]], 1).double()
        pre = torch.einsum("bjd,dj->bd", rows, w) + bias
        return pre * _sig64(pre), rows[:, 1:]
    x = s["x"].double().transpose(1, 2)
    B, D, T = x.shape
    head = x.new_zeros(B, D, W - 1) if s["S0"] is None else s["S0"].double().transpose(1, 2)
    rows = torch.cat([head, x], 2).requires_grad_(op == "conv_bwd")
    w, bias = w.requires_grad_(op == "conv_bwd"), bias.requires_grad_(op == "conv_bwd")
    windows = rows.unfold(2, W, 1)
    pre = (windows * w[None, :, None, :]).sum(-1) + bias[:, None]
    y = (pre * _sig64(pre)).transpose(1, 2)
    if op == "conv_fwd":
        lens = s["lens"].tolist() if "lens" in s else [T] * B
        y, state = y.clone(), y.new_empty(B, W - 1, D)
        for b, n in enumerate(lens):
            y[b, n:] = s["y"][b, n:].double()
            state[b] = rows[b, :, n:n + W - 1].t()
        return y, state
    total = (y * s["dy"].double()).sum()
    if s["dS_T"] is not None:
        total = total + (rows[:, :, T:].transpose(1, 2) * s["dS_T"].double()).sum()
    drows, dw, dbias = torch.autograd.grad(total, [rows, w, bias])
    out = dict(dx=drows[:, :, W - 1:].transpose(1, 2), dw=dw, dbias=dbias)
    if s["S0"] is not None:
        out["dS0"] = drows[:, :, :W - 1].transpose(1, 2)
    return out


def _ssm64(s, op):
    one = op == "ssm_step"
    v = {k: (t.unsqueeze(1) if one else t).double() for k, t in s.items() if k in ("u", "dt", "Bm", "Cm", "z") and t is not None}
    u, raw, A, skip = v["u"], v["dt"], s["A"].double(), s["D"].double()
    B, T, D = u.shape
    G, N = v["Bm"].shape[2:]
    if s["dt_bias"] is not None:
        raw = raw + s["dt_bias"].double()
        delta = torch.logaddexp(raw, torch.zeros_like(raw))
    else:
        delta = raw
    rows = lambda m, t: m[:, t].repeat_interleave(D // G, 1)  # noqa: E731
    start = s["S"] if one else s["S0"]
    h = torch.zeros(B, D, N, dtype=torch.float64, device=u.device) if start is None else start.double()
    lens = s["lens"].to(u.device)[:, None, None] if "lens" in s else None
    back = op == "ssm_bwd"
    kept = [h] if back else None
    ys = []
    for t in range(T):
        new = torch.exp(A * delta[:, t, :, None]) * h + rows(v["Bm"], t) * (delta[:, t] * u[:, t])[..., None]
        h = new if lens is None else torch.where(lens > t, new, h)
        ys.append((h * rows(v["Cm"], t)).sum(-1))
        if back:
            kept.append(h)
    y = torch.stack(ys, 1) + u * skip
    z = v.get("z")
    if not back:
        o = y if z is None else y * z * _sig64(z)
        if lens is not None:
            o = torch.where(torch.arange(T, device=u.device)[None, :, None] < lens, o, s["y"].double())
        return (o[:, 0], h) if one else (o, h)
    do = s["dy"].double()
    out = {}
    dy = do
    if z is not None:
        p = _sig64(z)
        dy, out["dz"] = do * z * p, do * y * (p + z * p * (1 - p))
    g = torch.zeros_like(h) if s["dS_T"] is None else s["dS_T"].double()
    out.update(du=torch.empty_like(u), ddt=torch.empty_like(u), dB=torch.empty_like(v["Bm"]), dC=torch.empty_like(v["Cm"]),
               dA=torch.zeros_like(A))
    for t in reversed(range(T)):
        per = lambda m: m.reshape(B, G, D // G, N).sum(2)  # noqa: E731
        b = rows(v["Bm"], t)
        g = g + rows(v["Cm"], t) * dy[:, t, :, None]
        out["dC"][:, t] = per(kept[t + 1] * dy[:, t, :, None])
        out["dB"][:, t] = per(g * (delta[:, t] * u[:, t])[..., None])
        along = (g * b).sum(-1)
        g = g * torch.exp(A * delta[:, t, :, None])
        q = g * kept[t]
        out["dA"] += (q * delta[:, t, :, None]).sum(0)
        out["du"][:, t] = delta[:, t] * along + skip * dy[:, t]
        out["ddt"][:, t] = (q * A).sum(-1) + u[:, t] * along
    if s["dt_bias"] is not None:
        out["ddt"] = out["ddt"] * _sig64(raw)
        out["ddt_bias"] = out["ddt"].sum((0, 1))
    out["dD"] = (dy * u).sum((0, 1))
    if s["S0"] is not None:
        out["dS0"] = g
    return out


def _norm64(s, op):
    c = s["case"]
    B, L, G, E = c["B"], c["L"], c["G"], c["E"]
    back = op == "norm_bwd"
    x = s["x"].double().reshape(B, L, G, E).permute(0, 2, 1, 3)
    w, b = (s[k].double().reshape(1, G, 1, E).requires_grad_(back) for k in ("weight", "bias"))
    z = None if s["gate"] is None else s["gate"].double().reshape(B, L, G, E).permute(0, 2, 1, 3).contiguous().requires_grad_(back)
    lay = lambda t: t.permute(0, 2, 1, 3).reshape(B, L, G * E)  # noqa: E731
    if back:
        mean, rstd = (s["stats"][..., k].double()[:, :, None, None] for k in (0, 1))
    else:
        mean = x.mean((2, 3), keepdim=True)
        rstd = (x.var((2, 3), correction=0, keepdim=True) + _EPS).rsqrt()
    hat = ((x - mean) * rstd).requires_grad_(back)
    v = hat * w + b
    y = v * _sig64(v) if c["silu"] else v
    y = y if z is None else y * z * _sig64(z)
    if not back:
        return lay(y), torch.stack([mean[..., 0, 0], rstd[..., 0, 0]], -1)
    total = (lay(y) * s["dy"].double()).sum()
    got = torch.autograd.grad(total, [hat, w, b] + ([] if z is None else [z]))
    dhat = got[0]
    flat = hat.detach()
    m = (2, 3)
    dx = rstd * (dhat - dhat.mean(m, keepdim=True) - flat * (dhat * flat).mean(m, keepdim=True))
    out = dict(dx=lay(dx), dweight=got[1].reshape(-1), dbias=got[2].reshape(-1))
    if z is not None:
        out["dgate"] = lay(got[3])
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    return (_conv64 if op.startswith("conv") else _ssm64 if op.startswith("ssm") else _norm64)(s, op)
