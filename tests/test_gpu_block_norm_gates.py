"""The slopes of the block norms' gates where they are small."""
import numpy as np
import pytest
import torch

from mixer_cases import dev, gen, randn

pytestmark = pytest.mark.gpu


def slopes(z, act):
    """The gate's derivative in 64 bits, without 1 - sigmoid(z)."""
    p, q = 1 / (1 + np.exp(-z)), 1 / (1 + np.exp(z))
    return p * q if act == "sigmoid" else p + z * p * q


@pytest.mark.parametrize("C", [70, 513, 8200])
def test_the_sigmoid_gates_gradient_of_large_gates(qd, C):
    """The slope of a sigmoid at z = 20 is e^-20, in fp32 as exact as any number: its exponential's
    argument is off by 2 |z| 2^-24 (the product with log2 e and the constant), and 24 roundings more
    of products, reciprocals and the exponential, two of which are of one unit each."""
    z = torch.linspace(-80, 80, C).view(1, C)
    z = z[:, torch.randperm(C, generator=gen(1))].contiguous()
    y, scale, dh = (randn(gen(s), 1, C) + 3 for s in (2, 3, 4))
    h, _, stats = qd.qdelta_block_norm_fwd(dev(y), None, None, dev(z), dev(scale[0]), act="sigmoid")
    got = qd.qdelta_block_norm_bwd(dev(y), h, None, dev(z), dev(scale[0]), None, stats, dev(dh), act="sigmoid")["dgate"]
    f64 = [t.double().numpy() for t in (y, scale, dh, z)]
    want = f64[0] * f64[1] * f64[2] * slopes(f64[3], "sigmoid")
    bound = (2 * np.abs(f64[3]) + 24) * 2.0 ** -24 * np.abs(want) + 1e-37
    worst = float((np.abs(got.double().cpu().numpy() - want) / bound).max())
    print(f"  dgate: {worst:.3f} of the bound", flush=True)
    assert worst <= 1


def test_slopes_at_the_ends_of_fp32(qd):
    """Gates beyond the exponential's range: a slope of 0, and of 1 for a large SiLU; NaN stays NaN."""
    z = torch.tensor([[-3e38, -1000.0, -90.0, 90.0, 1000.0, 3e38, float("nan"), 0.0]], device="cuda")
    y = torch.ones(1, 8, device="cuda")
    for act, want in (("sigmoid", [0, 0, 0, 0, 0, 0, None, 0.25]), ("silu", [0, 0, 0, 1, 1, 1, None, 0.5])):
        got = qd.qdelta_block_norm_bwd(y, None, None, z, None, None, None, y, act=act)["dgate"].cpu()[0]
        for have, w in zip(got.tolist(), want):
            assert have != have if w is None else abs(have - w) < 1e-6
