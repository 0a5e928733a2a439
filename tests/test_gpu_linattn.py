"""Linear attention's kernels against the fp64 oracle."""
import numpy as np
import pytest
import torch

from layer_cases import FWD, call, inputs, near, units
from mixer_cases import DT, dev, gen, randn, within
from oracle import layer

pytestmark = pytest.mark.gpu
BWD = FWD + ("d_o", "dS_T")

# dtype, B, T, H, dk, dv, decay, state, strong decays
CASES = [("bf16", 1, 1, 1, 64, 64, "token", True, False), ("f32", 1, 1, 1, 128, 128, "token", True, False),
         ("bf16", 2, 63, 3, 64, 128, "token", True, False), ("f32", 2, 31, 3, 128, 64, "token", True, False),
         ("bf16", 1, 64, 2, 128, 64, "head", True, False), ("f32", 1, 32, 2, 64, 64, "head", True, False),
         ("bf16", 2, 65, 1, 128, 128, "none", True, False), ("f32", 2, 33, 1, 128, 128, "none", False, False),
         ("bf16", 1, 130, 2, 128, 128, "token", False, True), ("f32", 1, 100, 2, 64, 128, "token", True, True),
         ("bf16", 3, 200, 5, 64, 64, "token", True, False), ("f32", 3, 203, 5, 64, 64, "token", True, False),
         ("bf16", 2, 2, 2, 128, 64, "head", False, False), ("f32", 1, 129, 3, 128, 128, "head", True, False),
         # few heads and many chunks: the time axis is cut, ends inside a chunk and on its border
         ("bf16", 1, 1100, 1, 128, 128, "token", True, False), ("f32", 1, 700, 1, 128, 64, "token", True, False),
         ("bf16", 1, 1024, 2, 64, 128, "head", False, False), ("bf16", 1, 1500, 1, 64, 64, "token", True, True)]


@pytest.mark.parametrize("dtype,B,T,H,dk,dv,decay,state,strong", CASES)
def test_forward(qd, dtype, B, T, H, dk, dv, decay, state, strong):
    x = inputs(B, T, H, dk, dv, dtype, T + H, decay, state, strong)
    o, S = call(qd, "qdelta_linattn_fwd", x, FWD)
    want, S_T, so, sS = layer.linattn_fwd(*[x[n] for n in FWD])
    near(o, want, so, x, "o")
    near(S, S_T, sS, x, "S_T")
    alone, none = call(qd, "qdelta_linattn_fwd", x, FWD, want_state=False)
    assert none is None
    near(alone, want, so, x, "o without the state")


@pytest.mark.parametrize("dtype,B,T,H,dk,dv,decay,state,strong", CASES)
def test_gradients(qd, dtype, B, T, H, dk, dv, decay, state, strong):
    x = inputs(B, T, H, dk, dv, dtype, T + H + 1, decay, state, strong)
    want, scale = layer.linattn_bwd(*[x[n] for n in BWD])
    got = call(qd, "qdelta_linattn_bwd", x, BWD)
    assert (got["dg"] is None) == (decay == "none")
    plain = call(qd, "qdelta_linattn_bwd", x, BWD, want_dg=False)
    bare = call(qd, "qdelta_linattn_bwd", x, BWD, want_dg=False, want_dS0=False)
    assert plain["dg"] is None and bare["dS0"] is None
    for n in ("dq", "dk", "dv", "dS0", "dg"):
        # one number a head or token that sums everything is not as good as random
        single = n == "dg" and got["dg"] is not None and got["dg"].numel() < 64
        for which in (got, plain, bare):
            if which[n] is not None:
                near(which[n], want[n], scale[n], x, n, norm=not single)


@pytest.mark.parametrize("dtype,dk,dv,decay", [("bf16", 64, 128, "token"), ("f32", 128, 64, "token"), ("bf16", 128, 128, "head"),
                                               ("f32", 64, 64, "none"), ("bf16", 64, 64, "none"), ("f32", 128, 128, "head")])
def test_single_token(qd, dtype, dk, dv, decay):
    N, H = 5, 3
    x = inputs(N, 1, H, dk, dv, dtype, 3, decay)
    want, S_T, so, sS = layer.linattn_fwd(*[x[n] for n in FWD])
    S = dev(x["S0"]).clone()
    g = None if x["g"] is None else dev(x["g"] if decay == "head" else x["g"][:, 0])
    o = qd.qdelta_linattn_step(*[dev(x[n][:, 0]).contiguous() for n in ("q", "k", "v")], g, S)
    within(o, want[:, 0], so[:, 0], 64 + dk, "o")          # no rounding inside: every product is in fp32
    within(S, S_T, sS, 16, "S")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_prompt_then_tokens(qd, dtype):
    x = inputs(2, 90, 2, 64, 128, dtype, 8)
    want, S_T, so, sS = layer.linattn_fwd(*[x[n] for n in FWD])
    first = {n: x[n] if n == "S0" else x[n][:, :80].contiguous() for n in FWD}
    _, S = call(qd, "qdelta_linattn_fwd", first, FWD)
    for t in range(80, 90):
        o = qd.qdelta_linattn_step(*[dev(x[n][:, t]).contiguous() for n in ("q", "k", "v", "g")], S)
        near(o, want[:, t], so[:, t], x, f"token {t}", norm=False)
    near(S, S_T, sS, x, "S")


LENS = [("bf16", 64, 64, 130, "token"), ("f32", 64, 128, 70, "head"), ("bf16", 128, 128, 64, "none"), ("bf16", 128, 64, 900, "token"),
        ("f32", 128, 64, 500, "token")]


@pytest.mark.parametrize("dtype,dk,dv,T,decay", LENS)
def test_padded_batches(qd, dtype, dk, dv, T, decay):
    """Padding, here NaN and infinities, is not read; rows of o behind a sequence stay as they were,
    zeros where the binding allocates; gradients there are zero; states belong to the ends."""
    lens = [T, 0, 1, T // 2 + 1, T + 9, -1] if T < 500 else [T // 3]
    B, H = len(lens), 2 if T < 500 else 1
    x = inputs(B, T, H, dk, dv, dtype, 4, decay)
    n_of = [min(max(n, 0), T) for n in lens]
    want, S_T, so, sS = layer.linattn_fwd(*[x[n] for n in FWD], lens=lens)
    grads, scale = layer.linattn_bwd(*[x[n] for n in BWD], lens=lens)
    for b, n in enumerate(n_of):
        for k in ("q", "k", "v", "d_o") + (("g",) if decay == "token" else ()):
            x[k][b, n:] = float("nan") if b % 2 else float("inf")
    at = dev(torch.tensor(lens, dtype=torch.int32))
    o0 = torch.full((B, T, H, dv), 7.0, dtype=DT[dtype], device="cuda")
    o, S = call(qd, "qdelta_linattn_fwd", x, FWD, lens=at, o=o0)
    fresh, _ = call(qd, "qdelta_linattn_fwd", x, FWD, lens=at)
    got = call(qd, "qdelta_linattn_bwd", x, BWD, lens=at)
    for b, n in enumerate(n_of):
        near(o[b, :n], want[b, :n], so[b, :n], x, f"o of {n}", norm=False)
        assert (o[b, n:] == 7).all() and not fresh[b, n:].any() and torch.equal(fresh[b, :n], o[b, :n])
        for k in ("dq", "dk", "dv") + (("dg",) if decay == "token" else ()):
            assert not got[k][b, n:].any(), k
    near(S, S_T, sS, x, "S_T")
    x["g"] = None if decay == "none" else torch.nan_to_num(x["g"], 0.0, 0.0)
    for k, v in got.items():
        if v is not None:
            near(v, grads[k], scale[k], x, k, norm=k != "dg")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [70, 700])
def test_a_decay_of_zero_forgets(qd, dtype, T):
    """g = -inf: nothing from before that token is left, and its gradient is zero; everything is
    finite, tokens before and after it in the same chunk."""
    x = inputs(1, T, 2, 64, 64, dtype, 6)
    for t in (0, 5, 37, T - 2):
        x["g"][:, t] = float("-inf")
    want, S_T, so, sS = layer.linattn_fwd(*[x[n] for n in FWD])
    o, S = call(qd, "qdelta_linattn_fwd", x, FWD)
    near(o, want, so, x, "o")
    near(S, S_T, sS, x, "S_T")
    grads, scale = layer.linattn_bwd(*[x[n] for n in BWD])
    got = call(qd, "qdelta_linattn_bwd", x, BWD)
    for k, v in got.items():
        near(v, grads[k], scale[k], x, k)
    assert (got["dS0"] == 0).all()
    S1 = dev(x["S0"]).clone()
    first = [dev(x[n][:, 0]).contiguous() for n in ("q", "k", "v", "g")]
    qd.qdelta_linattn_step(*first, S1)
    assert torch.equal(S1, first[2].float()[..., :, None] * first[1].float()[..., None, :])


def test_states_through_pieces_whose_decay_is_beyond_fp32(qd):
    """A state of 1e30 that pieces of the time axis multiply by e^-120 in all, no chunk by less than
    e^-60: the product is an ordinary number, though the pieces' factor by itself is below 2^-126."""
    x = inputs(1, 1024, 1, 64, 64, "f32", 7)
    x["g"][:] = -120.0 / 1024
    x["g"][:, ::2] *= 2
    x["g"][:, 1::2] = 0
    x["S0"] *= 1e30
    x["k"] *= 1e-12
    want, S_T, so, sS = layer.linattn_fwd(*[x[n] for n in FWD])
    o, S = call(qd, "qdelta_linattn_fwd", x, FWD)
    assert qd.qdelta_linattn_fwd_workspace_bytes(1, 1024, 1, 64, 64, torch.float32) > 0
    near(S, S_T, sS, x, "S_T")
    assert np.abs(S_T).max() > 1e-25


def test_growing_states(qd):
    """g > 0: a recurrence that doubles every 16 tokens."""
    x = inputs(1, 150, 2, 64, 128, "f32", 9)
    x["g"][:] = np.log(2) / 16
    want, S_T, so, sS = layer.linattn_fwd(*[x[n] for n in FWD])
    o, S = call(qd, "qdelta_linattn_fwd", x, FWD)
    near(o, want, so, x, "o")
    near(S, S_T, sS, x, "S_T")
    grads, scale = layer.linattn_bwd(*[x[n] for n in BWD])
    for k, v in call(qd, "qdelta_linattn_bwd", x, BWD).items():
        near(v, grads[k], scale[k], x, k, norm=k != "dg")


def test_decays_of_every_token_alike(qd):
    """g [H] is g [B, T, H] with the same numbers, and its gradient the sum."""
    x = inputs(2, 140, 3, 64, 64, "bf16", 10, "head")
    wide = dict(x, g=x["g"].expand(2, 140, 3).contiguous())
    a, b = call(qd, "qdelta_linattn_fwd", x, FWD), call(qd, "qdelta_linattn_fwd", wide, FWD)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    a, b = call(qd, "qdelta_linattn_bwd", x, BWD), call(qd, "qdelta_linattn_bwd", wide, BWD)
    assert all(torch.equal(a[n], b[n]) for n in ("dq", "dk", "dv", "dS0"))
    np.testing.assert_allclose(a["dg"].cpu(), b["dg"].double().sum((0, 1)).cpu(), rtol=1e-4)


def test_the_state_may_be_updated_in_place(qd):
    for T in (100, 1200):
        x = inputs(1, T, 2, 128, 64, "bf16", 11)
        want = call(qd, "qdelta_linattn_fwd", x, FWD)
        S = dev(x["S0"]).clone()
        o, S2 = qd.qdelta_linattn_fwd(*[dev(x[n]) for n in FWD[:4]], S, S_T=S)
        assert S2 is S and torch.equal(S, want[1]) and torch.equal(o, want[0])


@pytest.mark.parametrize("B,H,T,lens", [(1, 1, 4000, None), (3, 2, 2000, [2000, 5, 0]), (2, 20, 4000, [64, 4000]), (1, 3, 1200, [1])])
def test_the_state_in_place_over_a_cut_time_axis(qd, B, H, T, lens):
    """The last segment may end, and write S_T, before the first one has read S0."""
    for dtype in ("bf16", "f32"):
        x = inputs(B, T, H, 64, 128, dtype, 17)
        assert qd.qdelta_linattn_fwd_workspace_bytes(B, T, H, 64, 128, DT[dtype]) > 0
        n = None if lens is None else dev(torch.tensor(lens, dtype=torch.int32))
        want = call(qd, "qdelta_linattn_fwd", x, FWD, lens=n)
        a = [dev(x[k]) for k in FWD]
        for _ in range(3):
            S = a[4].clone()
            o, S2 = qd.qdelta_linattn_fwd(*a[:4], S, n, S_T=S)
            assert S2 is S and torch.equal(S, want[1]) and torch.equal(o, want[0])


@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 64), (64, 128), (128, 128)])
@pytest.mark.parametrize("T", [1, 2, 17, 64])
def test_one_chunk_rounds_once(qd, T, dk, dv):
    """Without a state, what one chunk rounds to bf16 inside is a sum of two: 2^-8 of 2^-8 is left of
    each term, beside the rounding of the output."""
    x = inputs(1, T, 1, dk, dv, "bf16", 18, state=False)
    want, S_T, so, sS = layer.linattn_fwd(*[x[n] for n in FWD])
    o, S = call(qd, "qdelta_linattn_fwd", x, FWD)
    near(o, want, so, x, "o", parts=2.0 ** -8)
    near(S, S_T, sS, x, "S_T")
    grads, scale = layer.linattn_bwd(*[x[n] for n in BWD])
    for want_dg in (True, False):
        got = call(qd, "qdelta_linattn_bwd", x, BWD, want_dg=want_dg)
        for n in ("dq", "dk", "dv"):
            near(got[n], grads[n], scale[n], x, n, parts=2.0 ** -8)


@pytest.mark.parametrize("T,lens", [(8192, None), (8200, None), (34000, [33000])])
def test_decays_gradient_over_many_chunks(qd, T, lens):
    """The chain of dg over 256 chunks, 257, and more than 1024 of which the last are padding."""
    x = inputs(1, T, 1, 64, 64, "f32", 19)
    want, scale = layer.linattn_bwd(*[x[n] for n in BWD], lens=lens)
    got = call(qd, "qdelta_linattn_bwd", x, BWD, lens=None if lens is None else dev(torch.tensor(lens, dtype=torch.int32)))
    for n in ("dg", "dq", "dS0"):
        near(got[n], want[n], scale[n], x, n)


def test_decays_gradient_of_many_heads_over_many_chunks(qd):
    """Heads enough to leave the time axis whole, 257 chunks of it; each head has the same inputs, so
    one is checked and the others are it."""
    H, T = 128, 8200
    x = inputs(1, T, 1, 64, 64, "f32", 20)
    want, scale = layer.linattn_bwd(*[x[n] for n in BWD])
    wide = {n: x[n].expand(*[H if (n in ("S0", "dS_T") and i == 1) or (n not in ("S0", "dS_T") and i == 2) else s
                             for i, s in enumerate(x[n].shape)]).contiguous() for n in BWD}
    got = call(qd, "qdelta_linattn_bwd", wide, BWD)
    for n, axis in (("dq", 2), ("dk", 2), ("dv", 2), ("dg", 2), ("dS0", 1)):
        one = got[n].narrow(axis, 0, 1)
        near(one, want[n], scale[n], x, n)
        assert torch.equal(got[n], one.expand_as(got[n])), n


def test_no_tokens_no_sequences(qd):
    x = inputs(2, 0, 3, 64, 128, "bf16", 12)
    o, S = call(qd, "qdelta_linattn_fwd", x, FWD)
    assert o.shape == (2, 0, 3, 128) and torch.equal(S.cpu(), x["S0"])
    _, S = call(qd, "qdelta_linattn_fwd", x, FWD[:4])
    assert not S.any()
    got = call(qd, "qdelta_linattn_bwd", x, BWD)
    assert torch.equal(got["dS0"].cpu(), x["dS_T"]) and got["dg"].shape == (2, 0, 3)
    x = inputs(2, 0, 3, 64, 128, "bf16", 12, "head")
    assert not call(qd, "qdelta_linattn_bwd", x, BWD)["dg"].any()
    x = inputs(0, 5, 3, 64, 64, "f32", 13, "head")
    assert call(qd, "qdelta_linattn_fwd", x, FWD)[0].shape == (0, 5, 3, 64)
    assert not call(qd, "qdelta_linattn_bwd", x, BWD)["dg"].any()
    assert qd.qdelta_linattn_step(*[torch.empty(0, 3, 64, device="cuda")] * 3, None, torch.empty(0, 3, 64, 64, device="cuda")).shape == (0, 3, 64)


def test_the_same_call_twice_gives_the_same_bits(qd):
    x = inputs(2, 300, 3, 128, 128, "bf16", 14)
    a = [dev(x[n]) for n in BWD]
    first, o = qd.qdelta_linattn_bwd(*a), qd.qdelta_linattn_fwd(*a[:5])
    for _ in range(3):
        again, p = qd.qdelta_linattn_bwd(*a), qd.qdelta_linattn_fwd(*a[:5])
        assert all(torch.equal(first[k], again[k]) for k in first) and torch.equal(o[0], p[0]) and torch.equal(o[1], p[1])


def test_gradients_against_differences(qd):
    """fp32, the whole call: (L(x + e d) - L(x - e d)) / 2e along random directions, the losses summed
    in 64 bits.  An output's error is some 2^-22 of its terms, which over a loss of 10^4 outputs that
    are as good as random, divided by 2e = 2e-2, leaves 2^-22 100 / 2e-2 = 1e-3 of an output; the
    third derivative, e^2 / 6 of it, 2e-5 of the rest.  Directions' derivatives are about 100."""
    x = inputs(1, 70, 2, 64, 64, "f32", 15)
    a = {n: dev(x[n]) for n in BWD}
    got = qd.qdelta_linattn_bwd(*[a[n] for n in BWD])

    def loss(b):
        o, S = qd.qdelta_linattn_fwd(*[b[n] for n in FWD])
        return float((o.double() * a["d_o"].double()).sum() + (S.double() * a["dS_T"].double()).sum())
    for n in FWD:
        r = torch.randn(a[n].shape, generator=gen(16)).cuda()
        e = 1e-2
        want = (loss(dict(a, **{n: a[n] + e * r})) - loss(dict(a, **{n: a[n] - e * r}))) / (2 * e)
        have = float((got["d" + n].double() * r.double()).sum())
        print(f"  d{n}: {have:.5f} against {want:.5f}", flush=True)
        assert abs(have - want) <= 2e-3 * abs(want) + 0.1, n


def test_refusals(qd):
    x = {k: dev(v) for k, v in inputs(2, 6, 3, 64, 64, "bf16", 2).items()}
    good = {k: x[k] for k in FWD}
    bad = [dict(k=x["k"].float()), dict(g=x["g"].bfloat16()), dict(g=x["g"][:, :5]), dict(g=x["g"][0, 0, :2].contiguous()),
           dict(q=x["q"].transpose(1, 2)), dict(v=x["v"][:, :4].contiguous()), dict(S0=x["S0"].bfloat16()), dict(S0=x["S0"][:1]),
           dict(k=x["k"].cpu()), dict(lens=torch.zeros(2, device="cuda")), dict(lens=torch.zeros(3, dtype=torch.int32, device="cuda")),
           dict(o=x["q"]), dict(o=x["v"].float()), dict(S_T=x["S0"][:, :2]), dict(q=x["q"][..., :32].contiguous(), k=x["k"][..., :32].contiguous(), S0=None),
           dict(q=x["q"].half(), k=x["k"].half(), v=x["v"].half())]
    for kw in bad:
        with pytest.raises(qd.QDeltaError):
            qd.qdelta_linattn_fwd(**dict(good, **kw))
    with pytest.raises(qd.QDeltaError, match="workspace"):
        qd.qdelta_linattn_bwd(**good, d_o=x["d_o"], workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(qd.QDeltaError):
        qd.qdelta_linattn_bwd(**good, d_o=None)
    with pytest.raises(qd.QDeltaError):
        qd.qdelta_linattn_bwd(**dict(good, g=None), d_o=x["d_o"], out=dict(dq=x["q"]))
    tok = [x[n][:, 0].contiguous() for n in ("q", "k", "v", "g")]
    for S in (x["S0"].bfloat16(), x["S0"][:1], x["S0"].transpose(2, 3)):
        with pytest.raises(qd.QDeltaError):
            qd.qdelta_linattn_step(*tok, S)
