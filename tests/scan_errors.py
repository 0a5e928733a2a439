"""The selective scan and its gradients in 64 bits, with a bound on what fp32 arithmetic may be off.

``scan`` walks the tokens once forward and once backward over whole batches of torch float64 tensors.
Beside every quantity it carries, through the same recurrences, a bound on the error of the fp32
walk, in units of 2^-24: what was off before, times the factor that multiplies it, and each new
rounding (1), hardware exponential or reciprocal (one place, 2) times the value it applies to.  A
state forgets its errors as it forgets its values, so the bound does not grow with the number of
tokens.  Products of two errors are left out; ``near`` allows 2 % for them.
"""
import torch

UNIT = 2.0 ** -24


def scan(x, plus=True, lens=None, cut_fwd=0, cut_bwd=0, backward=True):
    """(values, bounds): dicts with o, S_T and, with backward, the gradients that qdelta_ssm_bwd
    names.  x as tests' ssm_inputs gives it, on any device.  lens: tokens a sequence; rows past them
    are zero.  cut_fwd, cut_bwd: tokens a segment where the time axis is cut, 0 where it is not."""
    f = {k: None if v is None else v.double() for k, v in x.items()}
    u, A, dev = f["u"], f["A"], x["u"].device
    B, T, D = u.shape
    G, N = f["Bm"].shape[2:]
    per = D // G
    live = torch.ones(B, T, 1, dtype=torch.float64, device=dev)
    if lens is not None:
        live = (torch.arange(T, device=dev)[None] < lens[:, None]).double()[..., None]
    raw = f["dt"] + (0 if f["dt_bias"] is None else f["dt_bias"])
    if plus:
        delta = torch.clamp(raw, min=0) + torch.log1p(torch.exp(-raw.abs()))
        slope = torch.sigmoid(raw)
        # softplus itself is within 14 units; the sum in its argument is off by one unit of it
        cd = 14 + raw.abs() * slope / delta
    else:
        delta, slope, cd = raw, torch.ones_like(raw), torch.ones_like(raw)
    delta, u = delta * live, u * live
    z = None if f["z"] is None else f["z"] * live
    s = None if z is None else torch.sigmoid(z)
    gate = torch.ones_like(u) if z is None else z * s
    # the sigmoid: its exponent is off by 2 |z|, exponential 2, sum 1, reciprocal 2; two products
    cz = torch.zeros_like(u) if z is None else 2 * z.abs() + 8
    skip = torch.zeros(D, dtype=torch.float64, device=dev) if f["D"] is None else f["D"]
    wide = lambda t, i: t[:, i].repeat_interleave(per, 1)  # noqa: E731  [B, D, N] of a token's B or C
    sums = N + 4                                           # additions over states, waves and D u

    def decay(t):
        e = delta[:, t, :, None] * A
        a = torch.exp(e)
        return a, e.abs() * (cd[:, t, :, None] + 3) + 2

    def boundary(h, cut, t):
        """What a segment's composed effect adds: the factor exp(A sum delta) of its own, one product
        and one sum.  Segment [t - cut, t) for the walk, where the state after it is h."""
        total = delta[:, t:t + cut].sum(1)[..., None] * A
        most = cd.amax() + cut + 3
        return (torch.exp(total) * h).abs() * (total.abs() * most + 4)

    S0 = torch.zeros(B, D, N, dtype=torch.float64, device=dev) if f["S0"] is None else f["S0"]
    val, err = dict(o=torch.zeros_like(u)), dict(o=torch.zeros_like(u))

    def forward(cut):
        h, E, entry = S0, torch.zeros_like(S0), S0
        hs, Es = [h], [E]
        for t in range(T):
            if cut and t and t % cut == 0:
                E = E + boundary(entry, cut, t - cut) + h.abs()
                entry = h
            a, ca = decay(t)
            du = delta[:, t] * u[:, t]
            new = du[..., None] * wide(f["Bm"], t)
            E = a * E + ca * a * h.abs() + (cd[:, t, :, None] + 2) * new.abs()
            h = a * h + new
            E = (E + h.abs()) * live[:, t, :, None] + Es[-1] * (1 - live[:, t, :, None])
            hs.append(h)
            Es.append(E)
        return hs, Es

    def read_out(t, h, E):
        C, d = wide(f["Cm"], t), skip * u[:, t]
        y = (C * h).sum(-1) + d
        return y, (C.abs() * E).sum(-1) + sums * ((C * h).abs().sum(-1) + d.abs())

    hs, Es = forward(cut_fwd)
    for t in range(T):
        y, Ey = read_out(t, hs[t + 1], Es[t + 1])
        val["o"][:, t] = y * gate[:, t] * live[:, t]
        err["o"][:, t] = (gate[:, t].abs() * (Ey + cz[:, t] * y.abs())) * live[:, t]
    val["S_T"], err["S_T"] = hs[T], Es[T]
    if not backward:
        return val, err
    if cut_bwd != cut_fwd:
        del hs, Es
        hs, Es = forward(cut_bwd)
    for k in ("du", "ddt", "dz"):
        val[k], err[k] = torch.zeros_like(u), torch.zeros_like(u)
    for k in ("dB", "dC"):
        val[k], err[k] = torch.zeros_like(f["Bm"]), torch.zeros_like(f["Bm"])
    val["dA"], err["dA"] = torch.zeros_like(A), torch.zeros_like(A)
    for k in ("dD", "ddt_bias"):
        val[k], err[k] = torch.zeros(D, dtype=torch.float64, device=dev), torch.zeros(D, dtype=torch.float64, device=dev)
    segments = -(-T // cut_bwd) if cut_bwd else 1
    over_tokens = 16 + -(-T // 8) + B * segments           # additions of a sum over tokens and sequences
    over_channels = 10 + -(-per // 64)                     # and of one over a group's channels
    fold = lambda m: m.reshape(B, G, per, N).sum(2)  # noqa: E731
    g = torch.zeros_like(S0) if f["dS_T"] is None else f["dS_T"]
    Eg, entry = torch.zeros_like(g), g
    for t in reversed(range(T)):
        if cut_bwd and (t + 1) % cut_bwd == 0 and t + 1 < T:
            Eg = Eg + boundary(entry, cut_bwd, t + 1) + g.abs()
            entry = g
        lt = live[:, t]
        a, ca = decay(t)
        Bt, Ct, h, hp = wide(f["Bm"], t), wide(f["Cm"], t), hs[t + 1], hs[t]
        dt_, ut, cdt = delta[:, t], u[:, t], cd[:, t]
        d_o = f["d_o"][:, t] * lt
        y, Ey = read_out(t, h, Es[t + 1])
        if z is not None:
            st, zt = s[:, t], z[:, t]
            dg = d_o * st * (1 + zt * (1 - st))
            ds = st * (1 - st) * 2 * zt.abs() + 5 * st     # the sigmoid's error
            Edg = d_o.abs() * ((1 + zt.abs()) * ds + 4 * st * (1 + zt.abs() * (1 - st)))
            val["dz"][:, t] = dg * y
            err["dz"][:, t] = dg.abs() * Ey + Edg * y.abs() + 2 * (dg * y).abs()
        dy = d_o * gate[:, t]
        Edy = cz[:, t] * dy.abs()
        gi = g + Ct * dy[..., None]
        Ei = Eg + Ct.abs() * Edy[..., None] + gi.abs()
        du = (dt_ * ut)[..., None]
        terms = gi * du
        val["dB"][:, t] = fold(terms)
        err["dB"][:, t] = fold(Ei * du.abs() + (cdt[..., None] + 2 + over_channels) * terms.abs())
        terms = dy[..., None] * h
        val["dC"][:, t] = fold(terms)
        err["dC"][:, t] = fold(Edy[..., None] * h.abs() + dy.abs()[..., None] * Es[t + 1] + (1 + over_channels) * terms.abs())
        s1, E1 = (gi * Bt).sum(-1), (Ei * Bt.abs() + sums * (gi * Bt).abs()).sum(-1)
        back = a * gi
        Eb = a * Ei + (ca + 1) * back.abs()
        q = back * hp
        Eq = Eb * hp.abs() + back.abs() * Es[t] + q.abs()
        s2, E2 = (A * q).sum(-1), (A.abs() * Eq + (sums + 4) * (A * q).abs()).sum(-1)
        val["dA"] += (dt_[..., None] * q).sum(0)
        err["dA"] += (dt_.abs()[..., None] * (Eq + (cdt[..., None] + over_tokens) * q.abs())).sum(0)
        val["du"][:, t] = dt_ * s1 + skip * dy
        err["du"][:, t] = dt_.abs() * (E1 + (cdt + 2) * s1.abs()) + skip.abs() * (Edy + 2 * dy.abs())
        dd = ut * s1 + s2
        Ed = ut.abs() * (E1 + 2 * s1.abs()) + E2 + 2 * s2.abs()
        sl = slope[:, t] * lt
        val["ddt"][:, t] = dd * sl
        # the slope: e / (1 + e) or 1; its argument's rounding moves it by at most its size times itself
        err["ddt"][:, t] = sl * (Ed + (10 + raw[:, t].abs()) * dd.abs())
        val["dD"] += (dy * ut).sum(0)
        err["dD"] += (Edy * ut.abs() + over_tokens * (dy * ut).abs()).sum(0)
        val["ddt_bias"] += (dd * sl).sum(0)
        err["ddt_bias"] += (err["ddt"][:, t] + over_tokens * (dd * sl).abs()).sum(0)
        Eg = Eb * lt[..., None] + Eg * (1 - lt[..., None])
        g = back * lt[..., None] + g * (1 - lt[..., None])
    val["dS0"], err["dS0"] = g, Eg
    return val, err


def near(got, want, bound, name):
    """|got - want| <= eps_t / 2 |want| + 1.02 bound 2^-24, elementwise.  Values below fp32's normal
    range may be lost, with the sums they are part of: 2^-120."""
    half = torch.finfo(got.dtype).eps / 2
    got = got.double()
    assert got.shape == want.shape, (name, got.shape, want.shape)
    assert bool(torch.isfinite(got).all()), f"{name}: not finite"
    allowed = half * want.abs() + 1.02 * UNIT * bound + 2.0 ** -120
    worst = float(((got - want).abs() / allowed).max())
    print(f"  {name}: {worst:.3f} of the bound", flush=True)
    assert worst <= 1, f"{name}: {worst:.3g} times the bound"
