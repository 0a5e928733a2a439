"""The short causal convolution's kernels against the fp64 oracle."""
import numpy as np
import pytest
import torch

from mixer_cases import DT, dev, gen, randn, within
from oracle import mixer

pytestmark = pytest.mark.gpu

# Roundings on a path: W products and sums, the bias, and silu or its derivative (12).
U_FWD = 2 * 4 + 1 + 12


def make(B, T, D, W, dtype, seed, state=True, bias=True):
    g = gen(seed)
    return (randn(g, B, T, D, dtype=dtype), randn(g, D, W), randn(g, D) if bias else None,
            randn(g, B, W - 1, D, dtype=dtype) if state else None, randn(g, B, T, D, dtype=dtype),
            randn(g, B, W - 1, D, dtype=dtype) if state else None)


CASES = [("bf16", 2, 33, 64, 4, True, True, True), ("bf16", 1, 1, 8, 4, True, True, True),
         ("bf16", 3, 2, 70, 4, True, True, True), ("bf16", 2, 17, 35, 3, False, True, True),
         ("bf16", 1, 130, 1, 2, True, True, False), ("f32", 2, 19, 12, 4, True, True, False),
         ("f32", 1, 3, 5, 3, True, False, True), ("f32", 2, 65, 516, 2, False, False, True),
         ("bf16", 2, 300, 520, 4, False, True, True), ("f32", 5, 7, 33, 4, True, True, True)]


@pytest.mark.parametrize("dtype,B,T,D,W,state,bias,silu", CASES)
def test_forward(qd, dtype, B, T, D, W, state, bias, silu):
    x, w, b, S0, _, _ = make(B, T, D, W, dtype, T + D, state, bias)
    y, S = qd.qdelta_conv_fwd(dev(x), dev(w), dev(b), dev(S0), silu=silu)
    want, S_T, scale = mixer.conv_fwd(x, w, b, S0, silu)
    within(y, want, 1.1 * scale, U_FWD, "y")
    np.testing.assert_array_equal(S.double().cpu().numpy(), S_T)          # a copy of inputs


@pytest.mark.parametrize("dtype,B,T,D,W,state,bias,silu", CASES)
def test_gradients(qd, dtype, B, T, D, W, state, bias, silu):
    x, w, b, S0, dy, dS = make(B, T, D, W, dtype, T + D + 1, state, bias)
    got = qd.qdelta_conv_bwd(dev(x), dev(w), dev(b), dev(S0), dev(dy), dev(dS), silu=silu)
    want, scale = mixer.conv_bwd(x, w, b, S0, dy, dS, silu)
    assert (got["dbias"] is None) == (b is None)
    for k in ("dx", "dw", "dbias", "dS0"):
        if got[k] is not None:
            within(got[k], want[k], scale[k], 2 * U_FWD + (B * T if k in ("dw", "dbias") else 0), k)


def test_gradients_of_many_runs(qd):
    """Enough tokens that a thread's run is at its longest and a block joins several."""
    x, w, b, S0, dy, dS = make(4, 1100, 1024, 4, "bf16", 5)
    got = qd.qdelta_conv_bwd(dev(x), dev(w), dev(b), dev(S0), dev(dy), dev(dS))
    want, scale = mixer.conv_bwd(x, w, b, S0, dy, dS)
    for k in ("dx", "dw", "dbias", "dS0"):
        within(got[k], want[k], scale[k], 2 * U_FWD + (4400 if k in ("dw", "dbias") else 0), k)


@pytest.mark.parametrize("dtype,D", [("bf16", 40), ("f32", 7)])
def test_padded_batch(qd, dtype, D):
    """Rows past a sequence's length stay as they were, and what they hold is not read."""
    B, T, W = 6, 21, 4
    x, w, b, S0, _, _ = make(B, T, D, W, dtype, 9)
    lens = torch.tensor([0, 1, 2, 21, 40, -3], dtype=torch.int32)
    for i, n in enumerate([0, 1, 2, 21, 21, 0]):
        x[i, n:] = float("nan")
    y = torch.full((B, T, D), 7.0, dtype=DT[dtype], device="cuda")
    y, S = qd.qdelta_conv_fwd(dev(x), dev(w), dev(b), dev(S0), lens=dev(lens), y=y)
    want, S_T, scale = mixer.conv_fwd(x, w, b, S0, lens=lens)
    past = np.isnan(want)
    assert (y.double().cpu().numpy()[past] == 7.0).all()
    within(torch.where(torch.from_numpy(past).cuda(), torch.zeros_like(y), y), np.where(past, 0, want), scale, U_FWD, "y")
    np.testing.assert_array_equal(S.double().cpu().numpy(), S_T)


@pytest.mark.parametrize("dtype,D,W", [("bf16", 64, 4), ("bf16", 9, 3), ("f32", 20, 2)])
def test_steps_continue_a_prompt(qd, dtype, D, W):
    """A prompt, then single tokens on its state, against one call over all of it."""
    B, T = 3, 9
    x, w, b, _, _, _ = make(B, T, D, W, dtype, 11, state=False)
    whole, S_end = qd.qdelta_conv_fwd(dev(x), dev(w), dev(b))
    _, S = qd.qdelta_conv_fwd(dev(x[:, :4].contiguous()), dev(w), dev(b))
    for t in range(4, T):
        y = qd.qdelta_conv_step(dev(x[:, t].contiguous()), dev(w), dev(b), S)
        assert torch.equal(y, whole[:, t])
    assert torch.equal(S, S_end)


def test_state_in_place(qd):
    for T in (1, 2, 50):
        x, w, b, S0, _, _ = make(2, T, 48, 4, "bf16", T)
        y0, S1 = qd.qdelta_conv_fwd(dev(x), dev(w), dev(b), dev(S0))
        S = dev(S0).clone()
        y1, _ = qd.qdelta_conv_fwd(dev(x), dev(w), dev(b), S, S_T=S)
        assert torch.equal(S, S1) and torch.equal(y0, y1)


def test_no_tokens(qd):
    x, w, b, S0, dy, dS = make(2, 0, 16, 4, "f32", 1)
    y, S = qd.qdelta_conv_fwd(dev(x), dev(w), dev(b), dev(S0))
    assert y.shape == (2, 0, 16) and torch.equal(S.cpu(), S0)
    _, S = qd.qdelta_conv_fwd(dev(x), dev(w), dev(b))
    assert (S == 0).all()
    got = qd.qdelta_conv_bwd(dev(x), dev(w), dev(b), dev(S0), dev(dy), dev(dS))
    assert (got["dw"] == 0).all() and (got["dbias"] == 0).all() and torch.equal(got["dS0"].cpu(), dS)
    empty = torch.zeros(0, 5, 16, device="cuda")
    assert qd.qdelta_conv_fwd(empty, dev(w))[0].shape == (0, 5, 16)


def test_extreme_values(qd):
    """silu far on either side: no overflow of the exponential reaches the result."""
    x = torch.tensor([-1e4, -200.0, -90.0, 0.0, 90.0, 200.0, 1e4, 3e38]).reshape(1, 1, 8).cuda()
    w = torch.zeros(8, 2)
    w[:, 1] = 1
    y, _ = qd.qdelta_conv_fwd(x, w.cuda())
    want = np.array([0, 0, 0, 0, 90, 200, 1e4, 3e38])
    np.testing.assert_allclose(y.cpu().numpy().reshape(-1), want, rtol=1e-6, atol=1e-30)
    got = qd.qdelta_conv_bwd(x, w.cuda(), None, None, torch.ones_like(x))
    np.testing.assert_allclose(got["dx"].cpu().numpy().reshape(-1), [0, 0, 0, 0.5, 1, 1, 1, 1], rtol=1e-6, atol=1e-30)


def test_refusals(qd):
    x, w, b, S0, _, _ = make(2, 6, 16, 4, "bf16", 2)
    x, w, b, S0 = dev(x), dev(w), dev(b), dev(S0)
    bad = [dict(w=w.bfloat16()), dict(w=w[:, :1].contiguous()), dict(bias=b[:8]), dict(S0=S0.float()), dict(x=x.transpose(1, 2)),
           dict(x=x.half()), dict(lens=torch.zeros(2, dtype=torch.int64, device="cuda")), dict(y=x), dict(stream=3),
           dict(lens=torch.zeros(2, dtype=torch.int32))]
    for kw in bad:
        with pytest.raises(qd.QDeltaError):
            qd.qdelta_conv_fwd(**dict(dict(x=x, w=w, bias=b, S0=S0), **kw))
    with pytest.raises(qd.QDeltaError, match="workspace"):
        qd.qdelta_conv_bwd(x, w, b, S0, x.clone(), workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("dtype,T,D,W", [("bf16", 21, 40, 4), ("f32", 21, 7, 3), ("bf16", 150, 520, 4), ("f32", 1, 8, 2)])
def test_gradients_of_a_padded_batch(qd, dtype, T, D, W):
    """What padding holds is read neither from x nor from dy, and its gradient is zero; dS_T
    belongs to the window at the sequence's end."""
    lens = [0, 1, T // 2, T, T + 19, -3]
    x, w, b, S0, dy, dS = make(6, T, D, W, dtype, 31)
    want, scale = mixer.each_sequence(mixer.conv_bwd, lens, ("dw", "dbias"), (0, -1 - 3, 4, -1 - 5), x, w, b, S0, dy, dS)
    for i, n in enumerate(lens):
        x[i, max(n, 0):], dy[i, max(n, 0):] = float("nan"), float("inf")
    got = qd.qdelta_conv_bwd(dev(x), dev(w), dev(b), dev(S0), dev(dy), dev(dS), lens=dev(torch.tensor(lens, dtype=torch.int32)))
    for k in ("dx", "dw", "dbias", "dS0"):
        within(got[k], want[k], scale[k], 2 * U_FWD + (6 * T if k in ("dw", "dbias") else 0), k)
    full = qd.qdelta_conv_bwd(*[dev(t) for t in make(6, T, D, W, dtype, 31)])
    every = torch.full((6,), T, dtype=torch.int32, device="cuda")
    got = qd.qdelta_conv_bwd(*[dev(t) for t in make(6, T, D, W, dtype, 31)], lens=every)
    assert all(torch.equal(got[k], full[k]) for k in got)
    with pytest.raises(qd.QDeltaError):
        qd.qdelta_conv_bwd(*[dev(t) for t in make(6, T, D, W, dtype, 31)], lens=every.long())
