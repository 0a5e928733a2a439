"""Linear attention over a cut time axis where the states alone carry the result, and sums of the
decays' gradient, with bounds that zeros and wrong signs do not meet."""
import numpy as np
import pytest
import torch

from layer_cases import FWD, call, inputs, near
from mixer_cases import DT, dev
from oracle import layer

pytestmark = pytest.mark.gpu
BWD = FWD + ("d_o", "dS_T")


def fading(dtype, seed):
    """128 tokens whose decays make e^-100, 2^-144, without one of their chunks falling below e^-50 =
    2^-72, and no other decays.  The time axis is cut in eight segments (bf16: four), one of which has
    all of them."""
    x = inputs(1, 1024, 1, 64, 64, dtype, seed)
    x["g"][:] = 0
    x["g"][:, 256:384] = -100.0 / 128
    return x


def states_alone(got, want, scale, x, name):
    """What is wanted is far above the absolute floors of the comparison, 1e-30 and 1e-37."""
    assert np.linalg.norm(want) > 1e-15 * np.sqrt(want.size)
    near(got, want, scale, x, name)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_state_through_a_segment_whose_decay_is_beyond_fp32(qd, dtype):
    """S0 of 1e38 comes out of it as 1e-6, and nothing is added to it: v is zero."""
    x = fading(dtype, 40)
    x["S0"] = x["S0"].clamp(-3, 3) * 1e38
    x["v"] = torch.zeros_like(x["v"])
    assert qd.qdelta_linattn_fwd_workspace_bytes(1, 1024, 1, 64, 64, DT[dtype]) > 0
    want, S_T, so, sS = layer.linattn_fwd(*[x[n] for n in FWD])
    o, S = call(qd, "qdelta_linattn_fwd", x, FWD)
    states_alone(S, S_T, sS, x, "S_T")
    states_alone(o[:, 400:], want[:, 400:], so[:, 400:], x, "o")
    alone, _ = call(qd, "qdelta_linattn_fwd", x, FWD, want_state=False)
    states_alone(alone[:, 400:], want[:, 400:], so[:, 400:], x, "o without the state")
    x["S0"] = x["S0"] / 2 ** 10
    x["d_o"], x["dS_T"] = x["d_o"] * 2.0 ** -10, None
    grads, scale = layer.linattn_bwd(*[x[n] for n in BWD])
    got = call(qd, "qdelta_linattn_bwd", x, BWD, want_dg=False)
    states_alone(got["dq"][:, 400:], grads["dq"][:, 400:], scale["dq"][:, 400:], x, "dq")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_states_gradient_through_a_segment_whose_decay_is_beyond_fp32(qd, dtype):
    """The same backwards: dS_T of 1e38, d_o zero."""
    x = fading(dtype, 41)
    x["dS_T"] = x["dS_T"].clamp(-3, 3) * 1e38
    x["d_o"] = torch.zeros_like(x["d_o"])
    x["v"], x["k"] = x["v"] / 64, x["k"] / 64
    x["g"] = x["g"].flip(1).contiguous()             # the fading segment is the sixth
    grads, scale = layer.linattn_bwd(*[x[n] for n in BWD])
    for want_dg in (False, True):
        got = call(qd, "qdelta_linattn_bwd", x, BWD, want_dg=want_dg)
        for n in ("dk", "dv"):
            states_alone(got[n][:, :600], grads[n][:, :600], scale[n][:, :600], x, n)
        states_alone(got["dS0"], grads["dS0"], scale["dS0"], x, "dS0")


# dtype, B, T, H, dk, dv, lens: uncut and cut, padded and not
SUMS = [("bf16", 1, 1024, 2, 64, 128, None), ("f32", 1, 129, 3, 128, 128, None), ("bf16", 1, 64, 2, 128, 64, None),
        ("f32", 1, 700, 1, 64, 64, None), ("bf16", 2, 1500, 1, 128, 128, None), ("f32", 4, 70, 2, 64, 128, [70, 0, 1, 36]),
        ("bf16", 4, 130, 2, 64, 64, [130, 0, 1, 66]), ("f32", 2, 900, 1, 64, 64, [300, 900]), ("bf16", 2, 2000, 1, 128, 64, [1111, 600])]


@pytest.mark.parametrize("dtype,B,T,H,dk,dv,lens", SUMS)
@pytest.mark.parametrize("state", [True, False])
def test_the_decays_gradient_and_its_sum_over_tokens(qd, dtype, B, T, H, dk, dv, lens, state):
    """Per token within 2^-14 of the whole in the 2-norm, padding or not.  The sum of n tokens of a
    head is then off by at most sqrt(n) 2^-14 of the head's 2-norm, and by its own roundings: 6 and 4
    steps of a chunk's and of chunks' sums, n / 1024 in a row, of the tokens' sizes."""
    x = inputs(B, T, H, dk, dv, dtype, 42, "head", state)
    wide = dict(x, g=x["g"].expand(B, T, H).contiguous())
    want, scale = layer.linattn_bwd(*[wide[n] for n in BWD], lens=lens)
    at = None if lens is None else dev(torch.tensor(lens, dtype=torch.int32))
    got = call(qd, "qdelta_linattn_bwd", wide, BWD, lens=at)["dg"]
    near(got, want["dg"], scale["dg"], wide, "dg")
    size = np.linalg.norm(want["dg"], axis=(0, 1))
    bound = np.sqrt(B * T) * 2.0 ** -14 * size + (12 + B * T / 1024) * 2.0 ** -24 * np.abs(want["dg"]).sum((0, 1))
    total = want["dg"].sum((0, 1))
    assert (bound < 0.25 * np.abs(total)).any(), (bound, total)      # zeros do not pass
    off = np.abs(call(qd, "qdelta_linattn_bwd", x, BWD, lens=at)["dg"].double().cpu().numpy() - total)
    print(f"  sums: {(off / bound).max():.3f} of the bound", flush=True)
    assert (off <= bound).all()
