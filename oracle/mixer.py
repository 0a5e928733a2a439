"""fp64 oracle of the operators around the recurrence: short causal convolution, selective
state space scan, gated group norm, each with its gradients.  TEST INFRASTRUCTURE ONLY (same
import rule as the rest of ``oracle``).

Plain loops over time in numpy, written from the formulas.  Every function also returns, for
each output, a `scale`: the same sums with every term taken by its absolute value, the
quantity that a bound on rounding errors is relative to.
"""
import numpy as np


def f64(a):
    if a is None:
        return None
    if hasattr(a, "detach"):
        a = a.detach().to("cpu").double().numpy()
    return np.asarray(a, dtype=np.float64)


def sigmoid(x):
    return np.where(x >= 0, 1 / (1 + np.exp(-np.abs(x))), np.exp(-np.abs(x)) / (1 + np.exp(-np.abs(x))))


def softplus(x):
    return np.maximum(x, 0) + np.log1p(np.exp(-np.abs(x)))


def silu(x):
    return x * sigmoid(x)


def dsilu(x):
    s = sigmoid(x)
    return s + x * s * (1 - s)


def conv_fwd(x, w, bias=None, S0=None, act=True, lens=None):
    """(y, S_T, scale of the pre-activation).  Rows past a sequence's length are NaN."""
    x, w, bias, S0 = f64(x), f64(w), f64(bias), f64(S0)
    B, T, D = x.shape
    W = w.shape[1]
    full = np.concatenate([np.zeros((B, W - 1, D)) if S0 is None else S0, x], 1)
    y, scale, S_T = np.full((B, T, D), np.nan), np.zeros((B, T, D)), np.zeros((B, W - 1, D))
    for b in range(B):
        n = T if lens is None else int(min(max(int(lens[b]), 0), T))
        for t in range(n):
            terms = full[b, t:t + W] * w.T
            pre = terms.sum(0) + (0 if bias is None else bias)
            scale[b, t] = np.abs(terms).sum(0) + (0 if bias is None else np.abs(bias))
            y[b, t] = silu(pre) if act else pre
        S_T[b] = full[b, n:n + W - 1]
    return y, S_T, scale


def conv_bwd(x, w, bias, S0, dy, dS_T=None, act=True):
    x, w, bias, S0, dy, dS_T = (f64(t) for t in (x, w, bias, S0, dy, dS_T))
    B, T, D = x.shape
    W = w.shape[1]
    full = np.concatenate([np.zeros((B, W - 1, D)) if S0 is None else S0, x], 1)
    dfull, sfull = np.zeros_like(full), np.zeros_like(full)
    dw, sw, db, sb = np.zeros_like(w), np.zeros_like(w), np.zeros(D), np.zeros(D)
    for b in range(B):
        for t in range(T):
            rows = full[b, t:t + W]
            pre = (rows * w.T).sum(0) + (0 if bias is None else bias)
            size = (np.abs(rows) * np.abs(w.T)).sum(0) + (0 if bias is None else np.abs(bias))
            g = dy[b, t] * (dsilu(pre) if act else 1.0)
            # |silu''| <= 1/2: an error in pre, relative to its terms, reaches g through it
            sg = np.abs(dy[b, t]) * ((1.1 + size) if act else 1.0)
            dfull[b, t:t + W] += g * w.T
            sfull[b, t:t + W] += sg * np.abs(w.T)
            dw += (g * rows).T
            sw += (sg * np.abs(rows)).T
            db += g
            sb += sg
    if dS_T is not None:
        dfull[:, T:] += dS_T
        sfull[:, T:] += np.abs(dS_T)
    return (dict(dx=dfull[:, W - 1:], dw=dw, dbias=db, dS0=dfull[:, :W - 1]),
            dict(dx=sfull[:, W - 1:], dw=sw, dbias=sb, dS0=sfull[:, :W - 1]))


def _delta(dt, dt_bias, plus):
    raw = dt + (0 if dt_bias is None else dt_bias)
    return raw, softplus(raw) if plus else raw


def ssm_fwd(u, dt, A, Bm, Cm, D=None, z=None, dt_bias=None, S0=None, plus=True, lens=None):
    """(o, S_T, scale of o, scale of S_T).  Rows past a sequence's length are NaN."""
    u, dt, A, Bm, Cm, D, z, dt_bias, S0 = (f64(t) for t in (u, dt, A, Bm, Cm, D, z, dt_bias, S0))
    B, T, ch = u.shape
    G, N = Bm.shape[2:]
    _, delta = _delta(dt, dt_bias, plus)
    o, so = np.full((B, T, ch), np.nan), np.zeros((B, T, ch))
    S, sS = np.zeros((B, ch, N)), np.zeros((B, ch, N))
    for b in range(B):
        n = T if lens is None else int(min(max(int(lens[b]), 0), T))
        h = np.zeros((ch, N)) if S0 is None else S0[b].copy()
        s = np.abs(h)
        for t in range(n):
            a = np.exp(delta[b, t][:, None] * A)
            Bt, Ct = np.repeat(Bm[b, t], ch // G, 0), np.repeat(Cm[b, t], ch // G, 0)
            du = (delta[b, t] * u[b, t])[:, None]
            h = a * h + du * Bt
            s = a * s + np.abs(du * Bt)
            y, sy = (Ct * h).sum(1), (np.abs(Ct) * s).sum(1)
            if D is not None:
                y, sy = y + D * u[b, t], sy + np.abs(D * u[b, t])
            gate = 1.0 if z is None else silu(z[b, t])
            o[b, t], so[b, t] = y * gate, sy * np.abs(gate)
        S[b], sS[b] = h, s
    return o, S, so, sS


def ssm_bwd(u, dt, A, Bm, Cm, D, z, dt_bias, S0, d_o, dS_T=None, plus=True):
    """(gradients, scales), dicts with du, ddt, dA, dB, dC, dD, dz, ddt_bias, dS0."""
    u, dt, A, Bm, Cm, D, z, dt_bias, S0, d_o, dS_T = (
        f64(t) for t in (u, dt, A, Bm, Cm, D, z, dt_bias, S0, d_o, dS_T))
    B, T, ch = u.shape
    G, N = Bm.shape[2:]
    raw, delta = _delta(dt, dt_bias, plus)
    slope = sigmoid(raw) if plus else np.ones_like(raw)
    skip = np.zeros(ch) if D is None else D
    per = ch // G
    names = dict(du=u.shape, ddt=u.shape, dz=u.shape, dA=A.shape, dB=Bm.shape, dC=Bm.shape, dD=(ch,), ddt_bias=(ch,),
                 dS0=(B, ch, N))
    out = {k: np.zeros(v) for k, v in names.items()}
    mag = {k: np.zeros(v) for k, v in names.items()}
    fold = lambda m: m.reshape(G, per, N).sum(1)  # noqa: E731
    for b in range(B):
        hs, ss = [np.zeros((ch, N)) if S0 is None else S0[b]], []
        ss.append(np.abs(hs[0]))
        for t in range(T):
            a = np.exp(delta[b, t][:, None] * A)
            db = (delta[b, t] * u[b, t])[:, None] * np.repeat(Bm[b, t], per, 0)
            hs.append(a * hs[-1] + db)
            ss.append(a * ss[-1] + np.abs(db))
        g = np.zeros((ch, N)) if dS_T is None else dS_T[b].copy()
        sg = np.abs(g)
        for t in reversed(range(T)):
            a = np.exp(delta[b, t][:, None] * A)
            Bt, Ct = np.repeat(Bm[b, t], per, 0), np.repeat(Cm[b, t], per, 0)
            y, sy = (Ct * hs[t + 1]).sum(1) + skip * u[b, t], (np.abs(Ct) * ss[t + 1]).sum(1) + np.abs(skip * u[b, t])
            dy = d_o[b, t]
            if z is not None:
                out["dz"][b, t] = dy * y * dsilu(z[b, t])
                mag["dz"][b, t] = np.abs(dy) * sy * 1.1
                dy = dy * silu(z[b, t])
            ady = np.abs(dy)
            g, sg = g + Ct * dy[:, None], sg + np.abs(Ct) * ady[:, None]
            du_t = (delta[b, t] * u[b, t])[:, None]
            out["dC"][b, t], mag["dC"][b, t] = fold(dy[:, None] * hs[t + 1]), fold(ady[:, None] * ss[t + 1])
            out["dB"][b, t], mag["dB"][b, t] = fold(g * du_t), fold(sg * np.abs(du_t))
            s1, m1 = (g * Bt).sum(1), (sg * np.abs(Bt)).sum(1)
            g, sg = a * g, a * sg
            q, mq = g * hs[t], sg * ss[t]
            out["dA"] += delta[b, t][:, None] * q
            mag["dA"] += np.abs(delta[b, t])[:, None] * mq
            out["du"][b, t] = delta[b, t] * s1 + skip * dy
            mag["du"][b, t] = np.abs(delta[b, t]) * m1 + np.abs(skip * dy)
            dd, md = (A * q).sum(1) + u[b, t] * s1, (np.abs(A) * mq).sum(1) + np.abs(u[b, t]) * m1
            out["ddt"][b, t], mag["ddt"][b, t] = dd * slope[b, t], md * slope[b, t]
            out["dD"] += dy * u[b, t]
            mag["dD"] += ady * np.abs(u[b, t])
        out["dS0"][b], mag["dS0"][b] = g, sg
    out["ddt_bias"], mag["ddt_bias"] = out["ddt"].sum((0, 1)), mag["ddt"].sum((0, 1))
    return out, mag


def norm_fwd(x, groups, weight=None, bias=None, gate=None, act=False, eps=1e-5):
    """x [N, L, C].  (y, stats [N, G, 2], scale of y)."""
    x, weight, bias, gate = (f64(t) for t in (x, weight, bias, gate))
    n, length, c = x.shape
    e = c // groups
    y, scale, stats = np.zeros_like(x), np.zeros_like(x), np.zeros((n, groups, 2))
    for i in range(n):
        for k in range(groups):
            at = slice(k * e, (k + 1) * e)
            part = x[i, :, at]
            mean = part.mean()
            rstd = 1 / np.sqrt(np.mean((part - mean) ** 2) + eps)
            stats[i, k] = mean, rstd
            hat = (part - mean) * rstd
            w = 1.0 if weight is None else weight[at]
            v = hat * w + (0.0 if bias is None else bias[at])
            size = (np.abs(hat) + (np.abs(part) + np.abs(mean)) * rstd) * np.abs(w) + (0 if bias is None else np.abs(bias[at]))
            f, sf = (silu(v), 1.1 * size) if act else (v, size)
            if gate is not None:
                p = silu(gate[i, :, at])
                f, sf = f * p, sf * np.abs(p)
            y[i, :, at], scale[i, :, at] = f, sf
    return y, stats, scale


def norm_bwd(x, groups, weight, bias, gate, stats, dy, act=False):
    """(gradients, scales), dicts with dx, dweight, dbias, dgate; stats as the kernel is given them."""
    x, weight, bias, gate, stats, dy = (f64(t) for t in (x, weight, bias, gate, stats, dy))
    n, length, c = x.shape
    e = c // groups
    out = dict(dx=np.zeros_like(x), dweight=np.zeros(c), dbias=np.zeros(c), dgate=np.zeros_like(x))
    mag = {k: np.zeros_like(v) for k, v in out.items()}
    for i in range(n):
        for k in range(groups):
            at = slice(k * e, (k + 1) * e)
            mean, rstd = stats[i, k]
            hat = (x[i, :, at] - mean) * rstd
            shat = (np.abs(x[i, :, at]) + abs(mean)) * rstd
            w = np.ones(e) if weight is None else weight[at]
            b = np.zeros(e) if bias is None else bias[at]
            v, sv = hat * w + b, shat * np.abs(w) + np.abs(b)
            g = dy[i, :, at]
            sg = np.abs(g)
            f, sf = (silu(v), 1.1 * sv) if act else (v, sv)
            if gate is not None:
                z = gate[i, :, at]
                out["dgate"][i, :, at], mag["dgate"][i, :, at] = g * f * dsilu(z), sg * sf * 1.1
                g, sg = g * silu(z), sg * np.abs(silu(z))
            if act:
                g, sg = g * dsilu(v), sg * (1.1 + sv)
            out["dbias"][at] += g.sum(0)
            mag["dbias"][at] += sg.sum(0)
            out["dweight"][at] += (g * hat).sum(0)
            mag["dweight"][at] += (sg * shat).sum(0)
            gw, sgw = g * w, sg * np.abs(w)
            out["dx"][i, :, at] = rstd * (gw - gw.mean() - hat * (gw * hat).mean())
            mag["dx"][i, :, at] = rstd * (sgw + sgw.mean() + shat * (sgw * shat).mean())
    return out, mag


def each_sequence(fn, lens, shared, per, *args):
    """fn's (gradients, scales) for a right-padded batch: one sequence at a time without its
    padding, whose rows are zero.  shared: names of the gradients summed over sequences; per:
    indices of the arguments that have a row a sequence and token, or (negative, -1 - index) a
    row a sequence."""
    T = f64(args[per[0]]).shape[1]
    tokens, rows = {p for p in per if p >= 0}, {-1 - p for p in per if p < 0}
    whole = None
    for b, n in enumerate(lens):
        n = int(min(max(int(n), 0), T))
        part = [a if a is None else f64(a)[b:b + 1, :n] if i in tokens else f64(a)[b:b + 1] if i in rows else a
                for i, a in enumerate(args)]
        got = fn(*part)
        if whole is None:
            whole = tuple({k: [] for k in d} for d in got)
        for w, d in zip(whole, got):
            for k, v in d.items():
                if k not in shared and k != "dS0":
                    v = np.concatenate([v, np.zeros((1, T - n) + v.shape[2:])], 1)
                w[k].append(v)
    return tuple({k: sum(v) if k in shared else np.concatenate(v) for k, v in w.items()} for w in whole)
