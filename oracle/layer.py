"""fp64 oracle of linear attention with a decay for each head and of the RMS norms around a block,
each with its gradients.  TEST INFRASTRUCTURE ONLY (same import rule as the rest of ``oracle``).

Plain loops over time in numpy, written from the formulas.  Every function also returns, for each
output, a `scale`: the same sums with every term taken by its absolute value, the quantity that a
bound on rounding errors is relative to.
"""
import numpy as np

from .mixer import f64, sigmoid


def _decays(g, B, T, H):
    if g is None:
        return np.zeros((B, T, H))
    return np.broadcast_to(g, (B, T, H)) if g.ndim == 1 else g


def _len(lens, b, T):
    return T if lens is None else int(min(max(int(lens[b]), 0), T))


def linattn_fwd(q, k, v, g=None, S0=None, lens=None):
    """(o, S_T, scale of o, scale of S_T).  Rows past a sequence's length are NaN."""
    q, k, v, g, S0 = (f64(t) for t in (q, k, v, g, S0))
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    g = _decays(g, B, T, H)
    o, so = np.full((B, T, H, dv), np.nan), np.zeros((B, T, H, dv))
    S_T, sS = np.zeros((B, H, dv, dk)), np.zeros((B, H, dv, dk))
    for b in range(B):
        S = np.zeros((H, dv, dk)) if S0 is None else S0[b].copy()
        s = np.abs(S)
        for t in range(_len(lens, b, T)):
            e = np.exp(g[b, t])[:, None, None]
            w = v[b, t][:, :, None] * k[b, t][:, None, :]
            S, s = e * S + w, e * s + np.abs(w)
            o[b, t] = (S * q[b, t][:, None, :]).sum(-1)
            so[b, t] = (s * np.abs(q[b, t])[:, None, :]).sum(-1)
        S_T[b], sS[b] = S, s
    return o, S_T, so, sS


def linattn_bwd(q, k, v, g, S0, d_o, dS_T=None, lens=None):
    """(gradients, scales), dicts with dq, dk, dv, dg, dS0; padding's rows are zero.  dg's scale for a
    token also holds the terms of all the others of its head: a kernel may add up what reaches a
    token chunk by chunk from either end of the sequence."""
    q, k, v, g, S0, d_o, dS_T = (f64(t) for t in (q, k, v, g, S0, d_o, dS_T))
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    per_head = g is not None and g.ndim == 1
    g = _decays(g, B, T, H)
    names = dict(dq=q.shape, dk=q.shape, dv=v.shape, dg=(B, T, H), dS0=(B, H, dv, dk))
    out, mag = ({n: np.zeros(s) for n, s in names.items()} for _ in range(2))
    for b in range(B):
        n = _len(lens, b, T)
        S = [np.zeros((H, dv, dk)) if S0 is None else S0[b]]
        s = [np.abs(S[0])]
        for t in range(n):
            e = np.exp(g[b, t])[:, None, None]
            w = v[b, t][:, :, None] * k[b, t][:, None, :]
            S.append(e * S[-1] + w)
            s.append(e * s[-1] + np.abs(w))
        R = np.zeros((H, dv, dk)) if dS_T is None else dS_T[b].copy()
        r = np.abs(R)
        all_terms = (s[n] * r).sum((1, 2)) + 0.0
        for t in reversed(range(n)):
            y = d_o[b, t][:, :, None] * q[b, t][:, None, :]
            R, r = R + y, r + np.abs(y)
            out["dq"][b, t] = (S[t + 1] * d_o[b, t][:, :, None]).sum(1)
            mag["dq"][b, t] = (s[t + 1] * np.abs(d_o[b, t])[:, :, None]).sum(1)
            out["dk"][b, t], mag["dk"][b, t] = (R * v[b, t][:, :, None]).sum(1), (r * np.abs(v[b, t])[:, :, None]).sum(1)
            out["dv"][b, t], mag["dv"][b, t] = (R * k[b, t][:, None, :]).sum(2), (r * np.abs(k[b, t])[:, None, :]).sum(2)
            e = np.exp(g[b, t])[:, None, None]
            R, r = e * R, e * r
            out["dg"][b, t], mag["dg"][b, t] = (R * S[t]).sum((1, 2)), (r * s[t]).sum((1, 2))
            all_terms += (mag["dq"][b, t] * np.abs(q[b, t])).sum(-1) + (mag["dk"][b, t] * np.abs(k[b, t])).sum(-1)
        all_terms += (s[0] * r).sum((1, 2))
        mag["dg"][b, :n] += all_terms
        out["dS0"][b], mag["dS0"][b] = R, r
    if per_head:
        out["dg"], mag["dg"] = out["dg"].sum((0, 1)), mag["dg"].sum((0, 1))
    return out, mag


def gate(z, act):
    """The gate's factor and its derivative."""
    if act == "linear":
        return z, np.ones_like(z)
    s = sigmoid(z)
    return (s, s * (1 - s)) if act == "sigmoid" else (z * s, s + z * s * (1 - s))


def block_norm_h(y, x=None, post=None, z=None, scale=None, act="silu", eps=1e-5):
    """(h before it is stored, 1/rms of y, scale of h) for rows y [N, C]."""
    y, x, post, z, scale = (f64(t) for t in (y, x, post, z, scale))
    r = 1 / np.sqrt((y * y).mean(-1, keepdims=True) + eps)
    f = y if post is None else y * r * post
    f = f * (1 if z is None else gate(z, act)[0]) * (1 if scale is None else scale)
    base = 0 if x is None else x
    return base + f, r[:, 0], np.abs(base) + np.abs(f)


def block_norm_n(h, pre, eps=1e-5):
    """(n, 1/rms of h) of h as it is stored."""
    h, pre = f64(h), f64(pre)
    r = 1 / np.sqrt((h * h).mean(-1, keepdims=True) + eps)
    return h * r * pre, r[:, 0]


def block_norm_bwd(y, h, post, z, scale, pre, stats, dh, dn, act="silu"):
    """(gradients, scales), dicts with dx, dy, dgate, dpost, dscale, dpre; h and stats as the kernel is
    given them."""
    y, h, post, z, scale, pre, stats, dh, dn = (f64(t) for t in (y, h, post, z, scale, pre, stats, dh, dn))
    out, mag = {}, {}
    t = np.zeros_like(y) if dh is None else dh
    st = np.abs(t)
    if dn is not None:
        r = stats[:, 1:]
        e, w = h * r, dn * pre
        t = t + r * (w - e * (w * e).mean(-1, keepdims=True))
        st = st + r * (np.abs(w) + np.abs(e) * np.abs(w * e).mean(-1, keepdims=True))
        out["dpre"], mag["dpre"] = (dn * e).sum(0), np.abs(dn * e).sum(0)
    elif pre is not None:
        out["dpre"] = mag["dpre"] = np.zeros(y.shape[1])
    out["dx"], mag["dx"] = t, st
    r = 1.0 if post is None else stats[:, :1]
    hat = y * r
    f = hat if post is None else hat * post
    u, du = (np.ones_like(y), None) if z is None else gate(z, act)
    sc = 1.0 if scale is None else scale
    if z is not None:
        out["dgate"], mag["dgate"] = t * sc * f * du, st * np.abs(sc * f) * (1.1 + np.abs(du))
    if scale is not None:
        out["dscale"], mag["dscale"] = (t * u * f).sum(0), (st * np.abs(u * f)).sum(0)
    df, sdf = t * u * sc, st * np.abs(u * sc)
    if post is not None:
        out["dpost"], mag["dpost"] = (df * hat).sum(0), (sdf * np.abs(hat)).sum(0)
        w, sw = df * post, sdf * np.abs(post)
        df = r * (w - hat * (w * hat).mean(-1, keepdims=True))
        sdf = r * (sw + np.abs(hat) * (sw * np.abs(hat)).mean(-1, keepdims=True))
    out["dy"], mag["dy"] = df, sdf
    return out, mag
