"""Cases that time two operators beside the delta-rule layers: linear attention with a decay for each
head (prompts, single tokens, gradients), and the RMS norms after and before a block joined with its
gate, its scale and the residual sum (forward and gradients).

``own`` False computes each operator in elementary torch operations in 32 bits, rounded once;
``own`` True calls the framework's kernels on the same inputs."""
import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_EPS = 1e-5
_CHUNK = 64


def listed():
    return [
        # one decoded token of one sequence: launch latency
        dict(name="attention decode 1", op="att_step", B=1, H=16, dk=128, dv=128, g="token", dtype="bf16"),
        # one decoded token for each of 256 sequences: the state read and written
        dict(name="attention decode 256", op="att_step", B=256, H=16, dk=128, dv=128, g="head", dtype="bf16"),
        # the training shape of the layer, a decay for each token and head
        dict(name="attention training forward", op="att_fwd", B=8, T=4096, H=16, dk=128, dv=128, g="token", dtype="bf16",
             lens=False, state=False),
        # one long prompt continued from a state, a fixed decay for each head: the time axis is all there is to split
        dict(name="attention long prompt", op="att_fwd", B=1, T=65536, H=16, dk=128, dv=128, g="head", dtype="bf16",
             lens=False, state=True),
        # right-padded prompts of unequal length, keys narrower than values
        dict(name="attention ragged prompts", op="att_fwd", B=7, T=1900, H=12, dk=64, dv=128, g="token", dtype="bf16",
             lens=True, state=True),
        # the training shape's gradients, the decays' among them
        dict(name="attention training gradients", op="att_bwd", B=8, T=4096, H=16, dk=128, dv=128, g="token", dtype="bf16",
             lens=False, state=False),
        # a long sequence's gradients with fixed decays over few heads
        dict(name="attention long gradients", op="att_bwd", B=1, T=16384, H=8, dk=128, dv=128, g="head", dtype="bf16",
             lens=False, state=False),
        # a small fp32 layer at an odd length, a state carried in and out, learned decays
        dict(name="attention small gradients", op="att_bwd", B=3, T=203, H=5, dk=64, dv=64, g="token", dtype="f32",
             lens=False, state=True),
        # one decoded token for each of 64 sequences, sandwich norms around a block
        dict(name="block norm decode 64", op="norm_fwd", B=64, C=2048, dtype="bf16", post=True, gate="none", scale=False,
             pre=True),
        # every token of the training shape: post norm, gate, scale, residual, the next block's norm
        dict(name="block norm training forward", op="norm_fwd", B=32768, C=2048, dtype="bf16", post=True, gate="sigmoid",
             scale=True, pre=True),
        dict(name="block norm training gradients", op="norm_bwd", B=32768, C=2048, dtype="bf16", post=True, gate="sigmoid",
             scale=True, pre=True),
        # the plain residual sum and norm in fp32 over a channel count that no vector width divides
        dict(name="block norm odd gradients", op="norm_bwd", B=5000, C=1923, dtype="f32", post=False, gate="none", scale=True,
             pre=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["att_step", "att_fwd", "att_fwd", "att_bwd", "att_bwd", "norm_fwd", "norm_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op.startswith("norm"):
        C = _log(rng, 64, 8192)
        C = C | 1 if rng.random() < 0.4 else (C + 7) // 8 * 8
        B = max(1, min(_log(rng, 1, 32768), (1 << 25) // C))
        post = rng.random() < 0.7
        return dict(op=op, B=B, C=C, dtype=dtype, post=post, gate=rng.choice(["none", "silu", "sigmoid", "linear"]),
                    scale=rng.random() < 0.5, pre=rng.random() < 0.7)
    H, dk, dv = rng.choice([1, 2, 4, 5, 8, 12, 16, 32]), rng.choice([64, 128, 128]), rng.choice([64, 128, 128])
    c = dict(op=op, H=H, dk=dk, dv=dv, g=rng.choice(["token", "token", "head", "none"]), dtype=dtype)
    if op == "att_step":
        return dict(c, B=max(1, min(_log(rng, 1, 512), 4096 // H)))
    B = _log(rng, 1, 16)
    T = max(1, min(_log(rng, 1, 16384), (1 << (19 if dtype == "bf16" else 17)) // (B * H)))
    return dict(c, B=B, T=T, lens=rng.random() < 0.3, state=rng.random() < 0.5)


def prepare(case, seed):
    dt = _TYPES[case["dtype"]]
    rng = torch.Generator(device="cuda")
    rng.manual_seed(int(seed))
    r = lambda *s: torch.randn(*s, generator=rng, device="cuda")  # noqa: E731
    op, B = case["op"], case["B"]
    s = dict(case=dict(case))
    if op.startswith("norm"):
        C = case["C"]
        s["x"], s["y"] = (r(B, C) * 2).to(dt), r(B, C).to(dt)
        s["post"] = 1 + 0.1 * r(C) if case["post"] else None
        s["gate"] = r(B, C).to(dt) if case["gate"] != "none" else None
        s["scale"] = 0.5 + 0.1 * r(C) if case["scale"] else None
        s["pre"] = 1 + 0.1 * r(C) if case["pre"] else None
        if op == "norm_bwd":
            h, _, stats = _norm_fwd(s)
            s["h"], s["stats"] = h, stats
            s["dh"] = r(B, C).to(dt)
            s["dn"] = r(B, C).to(dt) if case["pre"] else None
            del s["x"]
        return s
    H, dk, dv, T = case["H"], case["dk"], case["dv"], case.get("T")
    tok = (B,) if op == "att_step" else (B, T)
    unit = lambda x: (x / x.norm(dim=-1, keepdim=True)).to(dt)  # noqa: E731
    s["q"], s["k"], s["v"] = unit(r(*tok, H, dk)), unit(r(*tok, H, dk)), r(*tok, H, dv).to(dt)
    s["g"] = None
    if case["g"] == "token":  # most decays near 0.98 a token
        s["g"] = -torch.nn.functional.softplus(r(*tok, H) - 4)
    elif case["g"] == "head":  # horizons from 32 tokens to 2048
        s["g"] = torch.log1p(-torch.exp2(-torch.linspace(5, 11, H, device="cuda") + 0.01 * r(H)))
    if op == "att_step":
        s["S"] = 0.1 * r(B, H, dv, dk)
        return s
    s["S0"] = 0.1 * r(B, H, dv, dk) if case["state"] else None
    s["lens"] = torch.randint(0, T + 1, (B,), generator=rng, device="cuda", dtype=torch.int32) if case["lens"] else None
    if op == "att_fwd":
        s["o"] = torch.zeros(B, T, H, dv, dtype=dt, device="cuda")  # rows past a sequence's length stay as they are
    else:
        s["do"] = r(B, T, H, dv).to(dt)
        s["dS_T"] = 0.1 * r(B, H, dv, dk) if case["state"] else None
    return s


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    op, B = case["op"], case["B"]
    if op.startswith("norm"):
        n, gate, pre = B * case["C"], 0 if case["gate"] == "none" else 1, 1 if case["pre"] else 0
        if op == "norm_fwd":
            return dict(bytes=n * e * (3 + gate + pre), flops=n * (6 + 6 * gate + 5 * pre))
        return dict(bytes=n * e * (4 + 2 * gate + 2 * pre), flops=n * (14 + 10 * gate + 10 * pre))
    H, dk, dv, T = case["H"], case["dk"], case["dv"], case.get("T", 1)
    n, state = B * T * H, 4 * B * H * dk * dv
    gates = 4 * n if case["g"] == "token" else 0
    if op == "att_step":
        return dict(bytes=n * (2 * dk + 2 * dv) * e + gates + 2 * state, flops=n * 5 * dk * dv)
    C = min(T, _CHUNK)
    if op == "att_fwd":
        return dict(bytes=n * (2 * dk + 2 * dv) * e + gates + (2 * state if case["state"] else 0),
                    flops=n * (4 * dk * dv + C * (dk + dv)))
    return dict(bytes=n * (4 * dk + 3 * dv) * e + 2 * gates + (3 * state if case["state"] else 0),
                flops=n * (10 * dk * dv + C * (3 * dk + 2 * dv)))


# ---------------------------------------------------------------- the plain form: linear attention

def _decays(s, T):
    """Log decays [B, H, T] in 64 bits, zero in padding, and the rows that are no padding."""
    q, g = s["q"], s["g"]
    B, H = q.shape[0], q.shape[2]
    if g is None:
        g = q.new_zeros(B, H, T, dtype=torch.float64)
    elif g.dim() == 1:
        g = g.double()[None, :, None].expand(B, H, T)
    else:
        g = g.double().transpose(1, 2)
    if s["lens"] is None:
        return g, None
    live = torch.arange(T, device=q.device) < s["lens"][:, None]
    return torch.where(live[:, None], g, 0.0), live


def _split(t, live):
    """[B, T, H, d] as [B, H, chunks, C, d] in 32 bits, zero in padding."""
    if live is not None:
        t = torch.where(live[:, :, None, None], t, 0.0)
    B, T, H, d = t.shape
    t = torch.nn.functional.pad(t.float().transpose(1, 2), (0, 0, 0, -T % _CHUNK))
    return t.reshape(B, H, -1, _CHUNK, d)


def _join(t, like, live):
    """Back to [B, T, H, d], padding's rows zero."""
    B, T, H = like.shape[:3]
    t = t.reshape(B, H, -1, t.shape[-1])[:, :, :T].transpose(1, 2)
    if live is not None:
        t = torch.where(live[:, :, None, None], t, 0.0)
    return t.to(like.dtype).contiguous()


def _mm(a, b):
    return torch.matmul(a, b.contiguous())


class _Chunks:
    """The decays between the tokens of a chunk, and between chunks."""

    def __init__(self, s):
        T = s["q"].shape[1]
        g, self.live = _decays(s, T)
        g = torch.nn.functional.pad(g, (0, -T % _CHUNK)).reshape(g.shape[0], g.shape[1], -1, _CHUNK)
        G = g.cumsum(-1)
        low = torch.ones(_CHUNK, _CHUNK, dtype=torch.bool, device=g.device).tril()
        self.D = torch.exp(torch.where(low, G[..., :, None] - G[..., None, :], -math.inf)).float()
        self.before = torch.exp(G)[..., None].float()                # from a chunk's start to behind the token
        self.after = torch.exp(G[..., -1:] - G)[..., None].float()   # from behind the token to the chunk's end
        self.all = torch.exp(G[..., -1]).float()
        total = G[..., -1]
        n = total.shape[-1]
        Z = torch.cat([torch.zeros_like(total[..., :1]), total.cumsum(-1)], -1)   # decay before each chunk, and at the end
        m = torch.ones(n + 1, n, dtype=torch.bool, device=g.device).tril(-1)
        self.W = torch.exp(torch.where(m, Z[..., :, None] - Z[..., None, 1:], -math.inf)).float()
        self.Z0 = torch.exp(Z).float()
        m = torch.ones(n + 1, n, dtype=torch.bool, device=g.device).triu()
        self.V = torch.exp(torch.where(m, Z[..., None, :-1] - Z[..., :, None], -math.inf)).float()
        self.Z1 = torch.exp(Z[..., -1:] - Z).float()


def _over(W, U, Z, S):
    """sum_m W[n, m] U[m] + Z[n] S over chunks."""
    B, H, n = U.shape[:3]
    out = torch.matmul(W, U.reshape(B, H, n, -1))
    if S is not None:
        out = out + Z[..., None] * S.reshape(B, H, 1, -1)
    return out.reshape(B, H, n + 1, *U.shape[3:])


def _att_fwd(s):
    c = _Chunks(s)
    q, k, v = (_split(s[n], c.live) for n in ("q", "k", "v"))
    S = _over(c.W, _mm((v * c.after).transpose(-1, -2), k), c.Z0, s["S0"])
    o = _mm(_mm(q, k.transpose(-1, -2)) * c.D, v) + c.before * _mm(q, S[:, :, :-1].transpose(-1, -2))
    o = _join(o, s["v"], c.live)
    return (o, S[:, :, -1].clone()) if s["case"]["state"] else o


def _att_step(s):
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    decay = 1.0 if s["g"] is None else torch.exp(s["g"].expand(q.shape[:2]))[..., None, None]
    S = decay * s["S"] + v[..., :, None] * k[..., None, :]
    o = (S * q[..., None, :]).sum(-1)
    s["S"].copy_(S)
    return o.to(s["q"].dtype), s["S"]


def _att_bwd(s):
    c = _Chunks(s)
    q, k, v, do = (_split(s[n], c.live) for n in ("q", "k", "v", "do"))
    S = _over(c.W, _mm((v * c.after).transpose(-1, -2), k), c.Z0, s["S0"])[:, :, :-1]
    R = _over(c.V, _mm((do * c.before).transpose(-1, -2), q), c.Z1, s["dS_T"])
    first, R = R[:, :, 0], R[:, :, 1:]
    A = _mm(q, k.transpose(-1, -2))
    P, dP = A * c.D, _mm(do, v.transpose(-1, -2)) * c.D
    far_q, far_k = c.before * _mm(do, S), c.after * _mm(v, R)
    out = dict(dq=_join(_mm(dP, k) + far_q, s["q"], c.live),
               dk=_join(_mm(dP.transpose(-1, -2), q) + far_k, s["k"], c.live),
               dv=_join(_mm(P.transpose(-1, -2), do) + c.after * _mm(k, R.transpose(-1, -2)), s["v"], c.live))
    if s["case"]["state"]:
        out["dS0"] = first.clone()
    if s["case"]["g"] == "token":
        M = dP * A
        left = M.cumsum(-1) - M                                  # [s, t]: the pairs of s with a token before t
        low = torch.ones(_CHUNK, _CHUNK, dtype=torch.bool, device=M.device).tril()
        a, b = (far_q * q).sum(-1), (far_k * k).sum(-1)
        dg = (torch.where(low, left, 0.0).sum(-2) + a.flip(-1).cumsum(-1).flip(-1) + (b.cumsum(-1) - b)
              + (c.all * (S * R).sum((-1, -2)))[..., None])
        out["dg"] = _join(dg[..., None], s["g"][..., None], c.live)[..., 0]
    return out


# ---------------------------------------------------------------- the plain form: block norms

def _act(kind, z):
    if kind == "linear":
        return z, torch.ones_like(z)
    p = 1 / (1 + torch.exp(-z))
    if kind == "sigmoid":
        return p, p * (1 - p)
    return z * p, p * (1 + z * (1 - p))


def _norm_fwd(s):
    y, dt = s["y"].float(), s["y"].dtype
    r1 = 1 / torch.sqrt(y.square().mean(-1, keepdim=True) + _EPS)
    f = y if s["post"] is None else y * r1 * s["post"]
    if s["gate"] is not None:
        f = f * _act(s["case"]["gate"], s["gate"].float())[0]
    if s["scale"] is not None:
        f = f * s["scale"]
    h = (s["x"].float() + f).to(dt)
    wide = h.float()                                             # the second norm is of the stream as it is stored
    r2 = 1 / torch.sqrt(wide.square().mean(-1, keepdim=True) + _EPS)
    n = None if s["pre"] is None else (wide * r2 * s["pre"]).to(dt)
    zero = torch.zeros_like(r1)
    stats = torch.cat([zero if s["post"] is None else r1, zero if s["pre"] is None else r2], 1)
    return h, n, stats


def _norm_bwd(s):
    dt, y, t = s["y"].dtype, s["y"].float(), s["dh"].float()
    r1, r2 = s["stats"][:, :1], s["stats"][:, 1:]
    out = {}
    if s["pre"] is not None:
        hat, dn = s["h"].float() * r2, s["dn"].float()
        w = dn * s["pre"]
        t = t + r2 * (w - hat * (w * hat).mean(-1, keepdim=True))
        out["dpre"] = (dn * hat).sum(0)
    out["dx"] = t.to(dt)
    hat = y if s["post"] is None else y * r1
    f = hat if s["post"] is None else hat * s["post"]
    df = t
    if s["gate"] is not None:
        u, du = _act(s["case"]["gate"], s["gate"].float())
        scaled = t if s["scale"] is None else t * s["scale"]
        out["dgate"] = (scaled * f * du).to(dt)
        f, df = f * u, t * u
    if s["scale"] is not None:
        out["dscale"] = (t * f).sum(0)
        df = df * s["scale"]
    if s["post"] is not None:
        out["dpost"] = (df * hat).sum(0)
        w = df * s["post"]
        df = r1 * (w - hat * (w * hat).mean(-1, keepdim=True))
    out["dy"] = df.to(dt)
    return out


# ---------------------------------------------------------------- the framework's calls

def _own(s):
    import recurrent_sequence_layers_amd as qd
    case = s["case"]
    op = case["op"]
    if op == "att_step":
        return qd.qdelta_linattn_step(s["q"], s["k"], s["v"], s["g"], s["S"]), s["S"]
    if op == "att_fwd":
        o, S_T = qd.qdelta_linattn_fwd(s["q"], s["k"], s["v"], s["g"], s["S0"], lens=s["lens"], o=s["o"],
                                       want_state=case["state"])
        return (o, S_T) if case["state"] else o
    if op == "att_bwd":
        got = qd.qdelta_linattn_bwd(s["q"], s["k"], s["v"], s["g"], s["S0"], s["do"], s["dS_T"], want_dS0=case["state"],
                                    want_dg=case["g"] == "token", lens=s["lens"])
    elif op == "norm_fwd":
        return qd.qdelta_block_norm_fwd(s["y"], s["x"], s["post"], s["gate"], s["scale"], s["pre"],
                                        act=case["gate"] if s["gate"] is not None else "silu", eps=_EPS)
    else:
        got = qd.qdelta_block_norm_bwd(s["y"], s["h"], s["post"], s["gate"], s["scale"], s["pre"], s["stats"], s["dh"],
                                       s["dn"], act=case["gate"] if s["gate"] is not None else "silu")
    return {k: v for k, v in got.items() if v is not None}


def run(state):
    if own:
        return _own(state)
    return dict(att_step=_att_step, att_fwd=_att_fwd, att_bwd=_att_bwd, norm_fwd=_norm_fwd,
                norm_bwd=_norm_bwd)[state["case"]["op"]](state)


# ---------------------------------------------------------------- the definition in 64 bits

def _att64(s, op):
    """The recurrence over blocks of 256 tokens, gradients by differentiating it."""
    one, back = op == "att_step", op == "att_bwd"
    at = lambda t: t.double()[:, :, None] if one else t.double().transpose(1, 2).contiguous()  # noqa: E731
    q, k, v = (at(s[n]) for n in ("q", "k", "v"))
    B, H, T, dk = q.shape
    dv = v.shape[-1]
    g = None if s["g"] is None else s["g"].double()
    S = s["S"] if one else s["S0"]
    S = q.new_zeros(B, H, dv, dk) if S is None else S.double()
    leaves = [q, k, v, S] + ([g] if g is not None else [])
    if back:
        leaves = [t.requires_grad_() for t in leaves]
        q, k, v, S = leaves[:4]
        g = leaves[4] if g is not None else None
    first = S
    if g is None:
        per = q.new_zeros(B, H, T)
    elif g.dim() == 1:
        per = g[None, :, None].expand(B, H, T)
    else:
        per = g[:, :, None] if one else g.transpose(1, 2)
    lens = s.get("lens")
    if lens is not None:
        rest = torch.arange(T, device=q.device) >= lens[:, None]
        per = per.masked_fill(rest[:, None], 0.0)
        q, k, v = (t.masked_fill(rest[:, None, :, None], 0.0) for t in (q, k, v))
    outs = []
    for a in range(0, T, 256):
        z = min(a + 256, T)
        run_ = per[:, :, a:z].cumsum(-1)
        ahead = run_[:, :, None, :] - run_[:, :, :, None]            # [key, query]
        kept = torch.triu(torch.ones(z - a, z - a, dtype=torch.bool, device=q.device))
        weight = ahead.masked_fill(~kept, -math.inf).exp()
        near = torch.matmul(k[:, :, a:z], q[:, :, a:z].transpose(-1, -2)) * weight
        o = torch.matmul(v[:, :, a:z].transpose(-1, -2), near)       # [dv, query]
        o = o + torch.matmul(S, q[:, :, a:z].transpose(-1, -2)) * run_.exp()[:, :, None]
        outs.append(o)
        left = (run_[:, :, -1:] - run_).exp()
        S = run_[:, :, -1].exp()[..., None, None] * S + torch.matmul(v[:, :, a:z].transpose(-1, -2) * left[:, :, None], k[:, :, a:z])
    o = torch.cat(outs, -1).permute(0, 3, 1, 2)
    if one:
        return o[:, 0], S
    if not back:
        return (o, S) if s["case"]["state"] else o
    do = s["do"].double()
    if lens is not None:
        do = do.masked_fill(rest[:, :, None, None], 0.0)
    total = (o * do).sum()
    if s["dS_T"] is not None:
        total = total + (S * s["dS_T"].double()).sum()
    want = [leaves[0], leaves[1], leaves[2]]
    names = ["dq", "dk", "dv"]
    if s["case"]["state"]:
        want, names = want + [first], names + ["dS0"]
    if s["case"]["g"] == "token":
        want, names = want + [g], names + ["dg"]
    got = dict(zip(names, torch.autograd.grad(total, want)))
    return {n: t.transpose(1, 2) if n in ("dq", "dk", "dv") else t for n, t in got.items()}


def _norm64(s, op):
    c = s["case"]
    back = op == "norm_bwd"
    w = {n: None if s[n] is None else s[n].double().requires_grad_(back) for n in ("post", "gate", "scale", "pre")}
    y, dt = s["y"].double(), s["y"].dtype
    unit = lambda t: (t.square().sum(-1, keepdim=True) / c["C"] + _EPS).rsqrt()  # noqa: E731
    r1 = s["stats"][:, :1].double() if back else unit(y)
    hat = (y if w["post"] is None else y * r1).detach().requires_grad_(back)
    branch = hat
    if w["post"] is not None:
        branch = branch * w["post"]
    if w["gate"] is not None:
        z = w["gate"]
        branch = branch * (z if c["gate"] == "linear" else z.sigmoid() * (z if c["gate"] == "silu" else 1))
    if w["scale"] is not None:
        branch = branch * w["scale"]
    zero = torch.zeros_like(r1)
    if not back:
        h = s["x"].double() + branch
        stored = h.to(dt).double()
        r2 = unit(stored)
        n = None if w["pre"] is None else stored * r2 * w["pre"]
        return h, n, torch.cat([zero if w["post"] is None else r1, zero if w["pre"] is None else r2], 1)
    out = {}
    toward = lambda d, e, r: r * (d - e * ((d * e).sum(-1, keepdim=True) / c["C"]))  # noqa: E731
    t = s["dh"].double()
    if w["pre"] is not None:
        e = s["h"].double() * s["stats"][:, 1:].double()
        dn = s["dn"].double()
        out["dpre"] = (dn * e).sum(0)
        t = t + toward(dn * s["pre"].double(), e, s["stats"][:, 1:].double())
    out["dx"] = t
    want = [n for n in ("post", "gate", "scale") if w[n] is not None]
    got = torch.autograd.grad((branch * t).sum(), [hat] + [w[n] for n in want])
    out.update({"d" + n: d for n, d in zip(want, got[1:])})
    out["dy"] = got[0] if w["post"] is None else toward(got[0], hat.detach(), r1)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    return (_att64 if op.startswith("att") else _norm64)(s, op)
