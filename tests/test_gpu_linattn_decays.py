"""The decays' gradient of linear attention where its terms are large, small or forgotten, against the
fp64 oracle."""
import numpy as np
import pytest
import torch

from layer_cases import FWD, call, inputs, near
from mixer_cases import dev
from oracle import layer

pytestmark = pytest.mark.gpu
BWD = FWD + ("d_o", "dS_T")


def finite_and_near(qd, x, lens=None):
    want, scale = layer.linattn_bwd(*[x[n] for n in BWD], lens=lens)
    got = call(qd, "qdelta_linattn_bwd", x, BWD, lens=None if lens is None else dev(torch.tensor(lens, dtype=torch.int32)))
    for n, v in got.items():
        assert bool(v.isfinite().all()), n
        near(v, want[n], scale[n], x, n)
    return got, want


@pytest.mark.parametrize("dtype,T", [("f32", 20), ("f32", 70), ("bf16", 130), ("f32", 700), ("bf16", 1100)])
@pytest.mark.parametrize("size", [1e25, 1e18, 1e-25])
@pytest.mark.parametrize("which", [("S0",), ("d_o", "dS_T"), ("v", "S0")])
def test_terms_whose_squares_leave_fp32(qd, dtype, T, size, which):
    """The terms of dg are linear in the states and their gradients: at 1e25 and 1e-25 they are
    ordinary fp32 numbers, their squares are not.  One chunk, several, and a cut time axis."""
    x = inputs(1, T, 1, 64, 64, dtype, 30)
    for n in which:
        x[n] = x[n] * size
    finite_and_near(qd, x)


def test_terms_whose_squares_leave_fp32_over_many_chunks(qd):
    """257 chunks in one walk, whose chain is a launch of its own."""
    H, T = 128, 8200
    x = inputs(1, T, 1, 64, 64, "f32", 31)
    x["S0"] = x["S0"] * 1e25
    want, scale = layer.linattn_bwd(*[x[n] for n in BWD])
    wide = {n: x[n].repeat_interleave(H, 1 if n in ("S0", "dS_T") else 2) for n in BWD}
    got = call(qd, "qdelta_linattn_bwd", wide, BWD)["dg"]
    one = got[:, :, :1]
    near(one, want["dg"], scale["dg"], x, "dg")
    assert torch.equal(got, one.expand_as(got))


def forget(x, tokens):
    """g = -inf at those tokens, of every head."""
    x["g"][:, list(tokens)] = float("-inf")
    return x


@pytest.mark.parametrize("dtype,T,tokens", [("f32", 32, (0, 1, 15, 16, 31)), ("bf16", 64, (0, 17, 18, 40, 63)), ("bf16", 40, (39,)),
                                            ("f32", 203, (5, 32, 63, 64, 100, 202)), ("bf16", 203, (5, 32, 63, 64, 100, 202)),
                                            ("f32", 700, (0, 128, 129, 400, 699)), ("bf16", 1500, (3, 64, 700, 701, 1499))])
def test_a_forgetting_token_has_no_gradient(qd, dtype, T, tokens):
    """dg_t = e^{g_t} <S_{t-1}, R_t> is zero at g_t = -inf, not what is left of larger numbers."""
    x = forget(inputs(2, T, 2, 64, 128, dtype, 32), tokens)
    got, _ = finite_and_near(qd, x)
    assert not got["dg"][:, list(tokens)].any()


def test_a_forgetting_head_has_no_gradient(qd):
    for dtype, T in (("bf16", 130), ("f32", 700)):
        x = inputs(2, T, 3, 64, 64, dtype, 33, "head")
        x["g"][1] = float("-inf")
        got, want = finite_and_near_but_dg(qd, x)
        assert not got["dg"][1].any() and want["dg"][0] != 0


def finite_and_near_but_dg(qd, x):
    want, scale = layer.linattn_bwd(*[x[n] for n in BWD])
    got = call(qd, "qdelta_linattn_bwd", x, BWD)
    for n in ("dq", "dk", "dv", "dS0"):
        near(got[n], want[n], scale[n], x, n)
    return got, want


def own_scale(x):
    """dg with every term by its absolute value, the token's own terms alone."""
    a = {n: None if x[n] is None else x[n] if n == "g" else x[n].abs() for n in BWD}
    return layer.linattn_bwd(*[a[n] for n in BWD])[0]["dg"]


@pytest.mark.parametrize("dtype,T,dk,dv", [("f32", 32, 64, 64), ("f32", 23, 128, 64), ("bf16", 64, 128, 128), ("bf16", 51, 64, 128), ("bf16", 16, 64, 64)])
@pytest.mark.parametrize("strong", [-20.0, -60.0])
def test_small_gradients_within_a_chunk(qd, dtype, T, dk, dv, strong):
    """A token whose decay is e^-20 among others near one has a dg of e^-20 of theirs, and as exact:
    each product of q and k and of do and v sums d_k and d_v terms, two roundings each; 16 + 48 of a
    block's sums, 8 of scans, 4 of products, 4 of an exponential whose argument, up to m, is off by
    m 2^-24 twice: 2 (d_k + d_v) + 128 + 4 m roundings of the token's own terms."""
    x = inputs(1, T, 2, dk, dv, dtype, 34, state=False)
    x["g"] *= 0.05
    at = sorted({1, T // 3, T // 2, 16 if T > 16 else 5, T - 1})
    x["g"][:, at[1::2]] = strong
    x["g"][:, at[0::2]] = strong / 2
    m = float(x["g"].abs().sum(1).max()) * 1.5
    want, _ = layer.linattn_bwd(*[x[n] for n in BWD])
    got = call(qd, "qdelta_linattn_bwd", x, BWD)["dg"]
    bound = own_scale(x) * (2 * (dk + dv) + 128 + 4 * m) * 2.0 ** -24 + 1e-37
    off = np.abs(got.double().cpu().numpy() - want["dg"]) / bound
    print(f"  dg: {off.max():.3f} of the bound", flush=True)
    assert off.max() <= 1


@pytest.mark.parametrize("dtype,T,at", [("f32", 260, 130), ("f32", 260, 128), ("bf16", 260, 129), ("f32", 1300, 700), ("bf16", 1300, 64), ("bf16", 3000, 1500)])
@pytest.mark.parametrize("which", ["S0", "dS_T"])
def test_nothing_crosses_a_forgetting_token(qd, dtype, T, at, which):
    """Terms of 1e25 on one side of it, of one on the other: each side's dg is right by itself."""
    x = forget(inputs(1, T, 1, 64, 64, dtype, 35), (at,))
    x[which] = x[which] * 1e25
    want, scale = layer.linattn_bwd(*[x[n] for n in BWD])
    got = call(qd, "qdelta_linattn_bwd", x, BWD)["dg"]
    for part in (slice(0, at), slice(at + 1, T)):
        near(got[:, part], want["dg"][:, part], scale["dg"][:, part], x, f"dg of {part}")
    assert not got[:, at].any()


def test_forgetting_tokens_over_many_chunks(qd):
    """The same in walks of 257 chunks: of one side's small terms behind the other's large ones."""
    H, T = 128, 8200
    x = forget(inputs(1, T, 1, 64, 64, "f32", 36), (1000, 1001, 4100, 8199))
    x["S0"], x["dS_T"] = x["S0"] * 1e25, x["dS_T"] * 1e20
    want, scale = layer.linattn_bwd(*[x[n] for n in BWD])
    wide = {n: x[n].repeat_interleave(H, 1 if n in ("S0", "dS_T") else 2) for n in BWD}
    got = call(qd, "qdelta_linattn_bwd", wide, BWD)["dg"]
    one = got[:, :, :1]
    assert torch.equal(got, one.expand_as(got)) and not one[:, [1000, 1001, 4100, 8199]].any()
    for part in (slice(0, 1000), slice(1002, 4100), slice(4101, 8199)):
        near(one[:, part], want["dg"][:, part], scale["dg"][:, part], x, f"dg of {part}")


@pytest.mark.parametrize("H,T", [(128, 8200), (3, 8200), (3, 40)])
def test_one_heads_decays_leave_the_others_alone(qd, H, T):
    """A head that forgets at every token, one that does at some, over 257 chunks in one walk, a cut time
    axis and two chunks: the other heads' gradients are the same bits as without."""
    x = inputs(1, T, 1, 64, 64, "f32", 37)
    a = {n: dev(x[n]).repeat_interleave(H, 1 if n in ("S0", "dS_T") else 2) for n in BWD}
    first = qd.qdelta_linattn_bwd(*[a[n] for n in BWD])
    a["g"][:, :, 0] = float("-inf")
    a["g"][:, ::7, 1] = float("-inf")
    got = qd.qdelta_linattn_bwd(*[a[n] for n in BWD])
    assert not got["dg"][:, :, 0].any() and not got["dg"][:, ::7, 1].any() and bool(got["dg"].isfinite().all())
    for n, v in got.items():
        axis = 1 if n == "dS0" else 2
        assert torch.equal(v.narrow(axis, 2, H - 2), first[n].narrow(axis, 2, H - 2)), n
