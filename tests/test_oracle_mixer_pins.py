"""Pins of the fp64 oracle of the operators around the recurrence: closed forms, and every
gradient against central differences of the oracle's own forward.

A central difference with step e has truncation error e^2 / 6 times the third derivative and
rounding error 2^-52 / e times the value: with e = 1e-5 and values and derivatives of order
one to a hundred, both stay under 1e-7; the bar is 1e-6 of the gradient's largest entry."""
import numpy as np
import pytest

from oracle import mixer

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


@pytest.mark.parametrize("T,W,act", [(5, 4, True), (1, 3, True), (2, 4, False), (4, 2, True)])
def test_conv_gradients(T, W, act):
    r = RNG(T * 10 + W)
    x, w, b, S0 = r.normal(size=(2, T, 3)), r.normal(size=(3, W)), r.normal(size=3), r.normal(size=(2, W - 1, 3))
    dy, dS = r.normal(size=(2, T, 3)), r.normal(size=(2, W - 1, 3))

    def f():
        y, S, _ = mixer.conv_fwd(x, w, b, S0, act)
        return (y * dy).sum() + (S * dS).sum()
    got, _ = mixer.conv_bwd(x, w, b, S0, dy, dS, act)
    for name, v in (("dx", x), ("dw", w), ("dbias", b), ("dS0", S0)):
        agree(got[name], differences(f, v), name)


def test_conv_state_joins_two_calls():
    r = RNG(3)
    x, w, b = r.normal(size=(2, 7, 3)), r.normal(size=(3, 4)), r.normal(size=3)
    whole, S, _ = mixer.conv_fwd(x, w, b)
    first, S1, _ = mixer.conv_fwd(x[:, :2], w, b)
    rest, S2, _ = mixer.conv_fwd(x[:, 2:], w, b, S1)
    np.testing.assert_allclose(np.concatenate([first, rest], 1), whole, rtol=1e-13)
    np.testing.assert_array_equal(S, S2)


@pytest.mark.parametrize("gate,plus,D,bias", [(True, True, True, True), (False, False, False, False), (True, False, True, True)])
def test_ssm_gradients(gate, plus, D, bias):
    r = RNG(7)
    B, T, ch, G, N = 2, 4, 4, 2, 3
    u, Bm, Cm = r.normal(size=(B, T, ch)), r.normal(size=(B, T, G, N)), r.normal(size=(B, T, G, N))
    dt = r.normal(size=(B, T, ch)) if plus else r.uniform(0.1, 0.5, size=(B, T, ch))
    A = -r.uniform(0.5, 2, size=(ch, N))
    D = r.normal(size=ch) if D else None
    bias = 0.1 * r.uniform(size=ch) if bias else None
    z = r.normal(size=(B, T, ch)) if gate else None
    S0, d_o, dS = r.normal(size=(B, ch, N)), r.normal(size=(B, T, ch)), r.normal(size=(B, ch, N))

    def f():
        o, S, _, _ = mixer.ssm_fwd(u, dt, A, Bm, Cm, D, z, bias, S0, plus)
        return (o * d_o).sum() + (S * dS).sum()
    got, _ = mixer.ssm_bwd(u, dt, A, Bm, Cm, D, z, bias, S0, d_o, dS, plus)
    for name, v in (("du", u), ("ddt", dt), ("dA", A), ("dB", Bm), ("dC", Cm), ("dD", D), ("dz", z), ("ddt_bias", bias),
                    ("dS0", S0)):
        if v is not None:
            agree(got[name], differences(f, v), name)


def test_ssm_closed_form_of_a_constant_input():
    """delta = 1 without softplus, A = log(1/2), u = B = C = 1: h_t = 2 - 2^(1 - t) at t = 1, 2, .."""
    T = 6
    one = np.ones((1, T, 1))
    o, S, _, _ = mixer.ssm_fwd(one, one, np.full((1, 1), np.log(0.5)), np.ones((1, T, 1, 1)), np.ones((1, T, 1, 1)), plus=False)
    np.testing.assert_allclose(o[0, :, 0], 2 - 2.0 ** (1 - np.arange(1, T + 1)), rtol=1e-14)
    np.testing.assert_allclose(S[0, 0, 0], 2 - 2.0 ** (1 - T), rtol=1e-14)


def test_ssm_padding_leaves_the_state_of_the_shorter_prompt():
    r = RNG(11)
    u, dt = r.normal(size=(2, 5, 4)), r.normal(size=(2, 5, 4))
    Bm, Cm, A = r.normal(size=(2, 5, 1, 3)), r.normal(size=(2, 5, 1, 3)), -r.uniform(0.5, 2, size=(4, 3))
    o, S, _, _ = mixer.ssm_fwd(u, dt, A, Bm, Cm, lens=[3, 0])
    short, S1, _, _ = mixer.ssm_fwd(u[:1, :3], dt[:1, :3], A, Bm[:1, :3], Cm[:1, :3])
    np.testing.assert_array_equal(o[0, :3], short[0])
    np.testing.assert_array_equal(S[0], S1[0])
    assert np.isnan(o[0, 3:]).all() and np.isnan(o[1]).all() and (S[1] == 0).all()


@pytest.mark.parametrize("L,gate,act", [(1, True, False), (3, False, True), (2, True, True)])
def test_norm_gradients(L, gate, act):
    r = RNG(L)
    n, G, C, eps = 2, 2, 6, 1e-3
    x, w, b, dy = r.normal(size=(n, L, C)), r.normal(size=C), r.normal(size=C), r.normal(size=(n, L, C))
    z = r.normal(size=(n, L, C)) if gate else None

    def f():
        return (mixer.norm_fwd(x, G, w, b, z, act, eps)[0] * dy).sum()
    _, stats, _ = mixer.norm_fwd(x, G, w, b, z, act, eps)
    got, _ = mixer.norm_bwd(x, G, w, b, z, stats, dy, act)
    for name, v in (("dx", x), ("dweight", w), ("dbias", b), ("dgate", z)):
        if v is not None:
            agree(got[name], differences(f, v), name)


def test_norm_of_a_group_is_standardised():
    r = RNG(5)
    y, stats, _ = mixer.norm_fwd(3 + 2 * r.normal(size=(2, 50, 8)), 4, eps=0.0)
    groups = y.reshape(2, 50, 4, 2)
    np.testing.assert_allclose(groups.mean((1, 3)), 0, atol=1e-13)
    np.testing.assert_allclose(groups.std((1, 3)), 1, rtol=1e-13)
