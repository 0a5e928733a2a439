"""The batched 64-bit scan that long walks are tested against, itself against the oracle's loops, and
its bounds against a walk in fp32."""
import numpy as np
import pytest
import torch

from mixer_cases import ssm_inputs
from oracle import mixer
from scan_errors import UNIT, scan

FWD = ("u", "dt", "A", "Bm", "Cm", "D", "z", "dt_bias", "S0")


@pytest.mark.parametrize("plus,gate,extras", [(True, True, True), (False, False, False), (True, False, True)])
def test_values_are_the_oracles(plus, gate, extras):
    x = ssm_inputs(3, 11, 10, 2, 16, "f32", 3, True, gate, plus, extras)
    val, _ = scan(x, plus)
    o, S_T, _, _ = mixer.ssm_fwd(*[x[k] for k in FWD], plus=plus)
    want, _ = mixer.ssm_bwd(*[x[k] for k in FWD], x["d_o"], x["dS_T"], plus)
    for k, v in dict(want, o=o, S_T=S_T).items():
        np.testing.assert_allclose(val[k].numpy(), v, rtol=1e-11, atol=1e-13, err_msg=k)


def test_padding_is_left_out():
    x = ssm_inputs(4, 9, 6, 1, 16, "f32", 4)
    lens = [9, 0, 1, 5]
    val, _ = scan(x, lens=torch.tensor(lens))
    order = FWD + ("d_o", "dS_T")
    per = tuple(i if k in ("u", "dt", "Bm", "Cm", "z", "d_o") else -1 - i for i, k in enumerate(order) if k not in ("A", "D", "dt_bias"))
    want, _ = mixer.each_sequence(mixer.ssm_bwd, lens, ("dA", "dD", "ddt_bias"), per, *[x[k] for k in order])
    o, S_T, _, _ = mixer.ssm_fwd(*[x[k] for k in FWD], lens=torch.tensor(lens))
    for k, v in dict(want, o=np.nan_to_num(o), S_T=S_T).items():
        np.testing.assert_allclose(val[k].numpy(), v, rtol=1e-11, atol=1e-13, err_msg=k)


def test_bounds_forget_with_the_states():
    """A thousand tokens allow an error like a hundred's, and one that a plain fp32 walk stays in."""
    x = ssm_inputs(1, 1000, 8, 1, 16, "f32", 5)
    val, err = scan(x, backward=False)
    _, short = scan({k: v[:, :100] if k in ("u", "dt", "Bm", "Cm", "z", "d_o") else v for k, v in x.items()}, backward=False)
    assert float(err["o"].max()) < 3 * float(short["o"].max())
    h = x["S0"].clone()
    for t in range(1000):
        delta = torch.nn.functional.softplus(x["dt"][:, t] + x["dt_bias"])
        h = torch.exp(delta[..., None] * x["A"]) * h + (delta * x["u"][:, t])[..., None] * x["Bm"][:, t]
    assert ((h.double() - val["S_T"]).abs() <= UNIT * err["S_T"]).all()
