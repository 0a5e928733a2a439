"""Pins of the fp64 oracle of linear attention and of the block norms: closed forms, and every
gradient against central differences of the oracle's own forward.

A central difference with step e has truncation error e^2 / 6 times the third derivative and
rounding error 2^-52 / e times the value: with e = 1e-5 and values and derivatives of order
one to a hundred, both stay under 1e-7; the bar is 1e-6 of the gradient's largest entry."""
import numpy as np
import pytest

import oracle
from oracle import layer

RNG = np.random.default_rng


def differences(f, x, e=1e-5):
    g = np.zeros_like(x)
    flat, out = x.reshape(-1), g.reshape(-1)
    for i in range(flat.size):
        keep = flat[i]
        flat[i] = keep + e
        hi = f()
        flat[i] = keep - e
        lo = f()
        flat[i] = keep
        out[i] = (hi - lo) / (2 * e)
    return g


def agree(got, want, name):
    assert np.abs(got - want).max() <= 1e-6 * max(1.0, np.abs(want).max()), name


def inputs(B, T, H, dk, dv, seed, per_head=False):
    r = RNG(seed)
    x = dict(q=r.normal(size=(B, T, H, dk)), k=r.normal(size=(B, T, H, dk)), v=r.normal(size=(B, T, H, dv)),
             g=-r.random(H) if per_head else -r.random((B, T, H)), S0=r.normal(size=(B, H, dv, dk)))
    return x, r.normal(size=(B, T, H, dv)), r.normal(size=(B, H, dv, dk))


@pytest.mark.parametrize("per_head,lens", [(False, None), (True, None), (False, [2, 0]), (True, [3, 1])])
def test_linattn_gradients(per_head, lens):
    x, do, dS = inputs(2, 4, 2, 3, 2, 1, per_head)

    def f():
        o, S, *_ = layer.linattn_fwd(**x, lens=lens)
        return (np.nan_to_num(o) * do).sum() + (S * dS).sum()
    got, mag = layer.linattn_bwd(**x, d_o=do, dS_T=dS, lens=lens)
    for name in x:
        agree(got["d" + name], differences(f, x[name]), name)
        assert (mag["d" + name] >= np.abs(got["d" + name]) - 1e-12).all()


def test_linattn_is_a_decayed_sum_of_pairs():
    x, *_ = inputs(1, 6, 1, 3, 2, 2)
    o, S, so, _ = layer.linattn_fwd(x["q"], x["k"], x["v"], x["g"])
    G = np.cumsum(x["g"][0, :, 0])
    for t in range(6):
        want = sum(np.exp(G[t] - G[i]) * (x["q"][0, t, 0] @ x["k"][0, i, 0]) * x["v"][0, i, 0] for i in range(t + 1))
        np.testing.assert_allclose(o[0, t, 0], want, rtol=1e-12)
        assert (so[0, t, 0] >= np.abs(want)).all()


def test_linattn_is_the_delta_rule_for_orthonormal_keys():
    """Against the library's own oracle: with beta = 1, lambda = 0 and keys that never meet again the
    erase term is zero, and both recurrences store the same."""
    r = RNG(4)
    T = 5
    k = np.linalg.qr(r.normal(size=(64, 64)))[0][:T].reshape(1, T, 1, 64)
    q, v = r.normal(size=(1, T, 1, 64)), r.normal(size=(1, T, 1, 64))
    alpha = r.random((1, T, 1)) * 0.5 + 0.5
    o, S = oracle.qdelta_fwd(q, k, v, alpha, np.ones((1, T, 1)), None, None)
    got, S_T, *_ = layer.linattn_fwd(q, k, v, np.log(alpha))
    np.testing.assert_allclose(got, o, atol=1e-12)
    np.testing.assert_allclose(S_T, S, atol=1e-12)


def test_linattn_state_joins_two_calls_and_forgets():
    x, *_ = inputs(2, 7, 2, 3, 2, 5)
    o, S, *_ = layer.linattn_fwd(**x)
    cut = lambda a, b: {n: t[:, a:b] if n in "qkvg" else t for n, t in x.items()}  # noqa: E731
    first = layer.linattn_fwd(**cut(0, 3))
    rest = layer.linattn_fwd(**dict(cut(3, 7), S0=first[1]))
    np.testing.assert_allclose(np.concatenate([first[0], rest[0]], 1), o, rtol=1e-13)
    np.testing.assert_allclose(rest[1], S, rtol=1e-13)
    x["g"][:, 4] = -np.inf
    late = layer.linattn_fwd(**x)
    fresh = layer.linattn_fwd(**dict(cut(4, 7), S0=None))
    np.testing.assert_allclose(late[0][:, 4:], fresh[0], rtol=1e-13)


NORMS = [(True, "silu", True, True, True), (True, "sigmoid", False, True, True), (False, "linear", True, False, True),
         (False, None, False, True, True), (True, None, True, False, False), (True, "silu", False, True, False)]


@pytest.mark.parametrize("post,act,scale,x,pre", NORMS)
def test_block_norm_gradients(post, act, scale, x, pre):
    r = RNG(6)
    N, C = 3, 5
    p = dict(y=r.normal(size=(N, C)))
    for name, there, shape in (("x", x, (N, C)), ("post", post, (C,)), ("z", act, (N, C)), ("scale", scale, (C,)), ("pre", pre, (C,))):
        p[name] = r.normal(size=shape) if there else None
    dh, dn = r.normal(size=(N, C)), r.normal(size=(N, C)) if pre else None
    act = act or "silu"

    def forward():
        h, r1, _ = layer.block_norm_h(p["y"], p["x"], p["post"], p["z"], p["scale"], act)
        n, r2 = layer.block_norm_n(h, p["pre"]) if pre else (None, np.zeros(N))
        return h, n, np.stack([r1, r2], 1)

    def f():
        h, n, _ = forward()
        return (h * dh).sum() + (0 if n is None else (n * dn).sum())
    h, _, stats = forward()
    got, mag = layer.block_norm_bwd(p["y"], h, p["post"], p["z"], p["scale"], p["pre"], stats, dh, dn, act)
    for name, key in (("y", "dy"), ("x", "dx"), ("post", "dpost"), ("z", "dgate"), ("scale", "dscale"), ("pre", "dpre")):
        if p[name] is not None:
            agree(got[key], differences(f, p[name]), key)
            assert (mag[key] >= np.abs(got[key]) - 1e-12).all(), key
        elif key != "dx":
            assert key not in got


def test_block_norm_closed_form():
    y = np.full((2, 4), 3.0)
    h, r, _ = layer.block_norm_h(y, None, np.arange(1.0, 5.0), None, None, eps=0.0)
    np.testing.assert_allclose(h, np.tile(np.arange(1.0, 5.0), (2, 1)))
    np.testing.assert_allclose(r, 1 / 3)
    z = np.array([[0.0, 2.0]])
    for act, want in (("linear", z), ("sigmoid", 1 / (1 + np.exp(-z))), ("silu", z / (1 + np.exp(-z)))):
        h, *_ = layer.block_norm_h(np.ones((1, 2)), np.ones((1, 2)), None, z, np.array([2.0, 0.5]), act)
        np.testing.assert_allclose(h, 1 + want * [2.0, 0.5])
