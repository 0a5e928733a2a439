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
