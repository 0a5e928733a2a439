"""The group norm's kernels against the fp64 oracle."""
import numpy as np
import pytest
import torch

from mixer_cases import dev, gen, randn, within
from oracle import mixer

pytestmark = pytest.mark.gpu

# dtype, N, L, G, E, weight and bias, gate, silu
CASES = [("bf16", 5, 1, 4, 128, True, True, False), ("f32", 3, 1, 2, 64, True, False, True),
         ("bf16", 7, 1, 3, 1, True, True, False), ("f32", 2, 1, 5, 33, False, True, True),
         ("bf16", 3, 1, 2, 511, True, False, False), ("bf16", 2, 1, 1, 1600, True, True, False),
         ("f32", 3, 1, 2, 2000, True, True, False), ("bf16", 2, 1, 1, 6000, True, False, True),
         ("bf16", 33, 1, 16, 8, True, True, True), ("f32", 2, 1, 1, 9001, True, True, False),
         ("bf16", 2, 9, 4, 16, True, True, False), ("f32", 3, 50, 2, 6, True, False, True),
         ("bf16", 1, 129, 3, 5, False, True, False), ("f32", 2, 300, 32, 30, True, False, True),
         ("f32", 1, 2, 1, 1, True, False, False)]


def make(dtype, N, L, G, E, affine, gate, seed, shift=0.3):
    g = gen(seed)
    C = G * E
    return (randn(g, N, L, C, dtype=dtype) * 1.5 + shift, randn(g, C) if affine else None, randn(g, C) if affine else None,
            randn(g, N, L, C, dtype=dtype) if gate else None, randn(g, N, L, C, dtype=dtype))


def units(L, E):
    """Roundings on a path.  The mean and the square sum add a lane's elements one by one (up to
    64 rows or 8 vectors of 8), then lanes, waves and runs: at most 64 + 16 + 16 + the runs a
    lane joins; the square root, the product with it, weight, bias, silu and gate: 32."""
    return 128 + L * E // 4096 + 32


@pytest.mark.parametrize("dtype,N,L,G,E,affine,gate,silu", CASES)
def test_forward(qd, dtype, N, L, G, E, affine, gate, silu):
    x, w, b, z, _ = make(dtype, N, L, G, E, affine, gate, L + E)
    y, stats = qd.qdelta_group_norm_fwd(dev(x), G, dev(w), dev(b), dev(z), silu=silu)
    want, st, scale = mixer.norm_fwd(x, G, w, b, z, silu)
    within(y, want, scale, units(L, E), "y")
    size = np.abs(x.double().numpy()).reshape(N, L, G, E).mean((1, 3))
    within(stats[..., 0], st[..., 0], size, units(L, E), "mean")
    # 1/std: half the square sum's relative error, whose terms' errors are relative to x itself
    spread = (np.abs(x.double().numpy()).reshape(N, L, G, E).max((1, 3)) * st[..., 1]) ** 2 + 1
    within(stats[..., 1], st[..., 1], st[..., 1] * spread, units(L, E), "1/std")


@pytest.mark.parametrize("dtype,N,L,G,E,affine,gate,silu", CASES)
def test_gradients(qd, dtype, N, L, G, E, affine, gate, silu):
    x, w, b, z, dy = make(dtype, N, L, G, E, affine, gate, L + E + 1)
    _, stats = qd.qdelta_group_norm_fwd(dev(x), G, dev(w), dev(b), dev(z), silu=silu)
    got = qd.qdelta_group_norm_bwd(dev(x), G, dev(w), dev(b), dev(z), stats, dev(dy), silu=silu)
    want, scale = mixer.norm_bwd(x, G, w, b, z, stats, dy, silu)
    for k, dep in (("dweight", w), ("dbias", b), ("dgate", z)):
        assert (got[k] is None) == (dep is None)
    for k, v in got.items():
        if v is not None:
            within(v, want[k], scale[k], 2 * units(L, E) + (N * L if k in ("dweight", "dbias") else 0), k)


def test_gradients_of_many_rows(qd):
    """More units than the persistent grid has slots."""
    x, w, b, z, dy = make("bf16", 9000, 1, 4, 64, True, True, 3)
    _, stats = qd.qdelta_group_norm_fwd(dev(x), 4, dev(w), dev(b), dev(z))
    got = qd.qdelta_group_norm_bwd(dev(x), 4, dev(w), dev(b), dev(z), stats, dev(dy))
    want, scale = mixer.norm_bwd(x, 4, w, b, z, stats, dy)
    for k, v in got.items():
        within(v, want[k], scale[k], 2 * units(1, 64) + 9000, k)


def test_large_outputs_go_around_the_caches(qd):
    """From 64 MiB a tensor on, the second pass stores past the caches."""
    x, w, b, z, dy = make("f32", 1, 4400, 8, 500, True, False, 21)
    assert x.numel() * 4 >= 64 << 20
    y, stats = qd.qdelta_group_norm_fwd(dev(x), 8, dev(w), dev(b), silu=True)
    want, _, scale = mixer.norm_fwd(x, 8, w, b, None, True)
    within(y, want, scale, units(4400, 500), "y")
    got = qd.qdelta_group_norm_bwd(dev(x), 8, dev(w), dev(b), None, stats, dev(dy), silu=True)
    want, scale = mixer.norm_bwd(x, 8, w, b, None, stats, dy, True)
    for k in ("dx", "dweight", "dbias"):
        within(got[k], want[k], scale[k], 2 * units(4400, 500) + (4400 if k != "dx" else 0), k)


@pytest.mark.parametrize("L", [1, 40])
def test_a_mean_far_above_the_spread(qd, L):
    """x = 1000 + N(0, 1) in fp32: the square sum is of centred values, so 1/std keeps the
    accuracy that the inputs have (their own rounding is 2^-24 of 1000, 6e-5 of the spread;
    the mean's, of the order of 2^-24 of 1000 too, enters the variance only squared)."""
    g = gen(4)
    x = 1000 + randn(g, 4, L, 96)
    y, stats = qd.qdelta_group_norm_fwd(dev(x), 3)
    want, st, _ = mixer.norm_fwd(x, 3)
    rel = np.abs(stats[..., 1].double().cpu().numpy() / st[..., 1] - 1).max()
    assert rel <= 64 * 2.0 ** -24, rel
    # y: the mean's error of a few units of 2^-24 * 1000, times 1/std
    assert np.abs(y.double().cpu().numpy() - want).max() <= 16 * 2.0 ** -24 * 1000 * st[..., 1].max()


def test_constant_groups_and_single_elements(qd):
    """No spread: xhat is 0 and y the bias, with 1/std = eps^-1/2."""
    x = torch.full((3, 1, 12), 2.5, device="cuda")
    b = torch.arange(12.0, device="cuda")
    for G in (1, 4, 12):
        y, stats = qd.qdelta_group_norm_fwd(x, G, None, b, eps=1e-4)
        assert torch.equal(y[0, 0], b)
        torch.testing.assert_close(stats[..., 1], torch.full_like(stats[..., 1], 100.0), rtol=1e-6, atol=0)


def test_shapes_without_elements(qd):
    w = torch.ones(8, device="cuda")
    y, _ = qd.qdelta_group_norm_fwd(torch.zeros(0, 3, 8, device="cuda"), 2, w)
    assert y.shape == (0, 3, 8)
    got = qd.qdelta_group_norm_bwd(torch.zeros(0, 3, 8, device="cuda"), 2, w, None, None,
                                   torch.zeros(0, 2, 2, device="cuda"), torch.zeros(0, 3, 8, device="cuda"))
    assert (got["dweight"] == 0).all()


def test_dimensions_between_are_positions(qd):
    x, w, b, _, dy = make("f32", 2, 12, 2, 4, True, False, 6)
    y0, s0 = qd.qdelta_group_norm_fwd(dev(x), 2, dev(w), dev(b))
    y1, s1 = qd.qdelta_group_norm_fwd(dev(x).view(2, 3, 4, 8), 2, dev(w), dev(b))
    assert torch.equal(y0, y1.view(2, 12, 8)) and torch.equal(s0, s1)
    y2, _ = qd.qdelta_group_norm_fwd(dev(x).view(24, 8), 2, dev(w), dev(b))
    want, _, scale = mixer.norm_fwd(x.reshape(24, 1, 8), 2, w, b)
    within(y2[:, None], want, scale, units(1, 4), "y")


def test_refusals(qd):
    x = torch.zeros(4, 2, 16, device="cuda")
    w = torch.ones(16, device="cuda")
    bad = [dict(groups=3), dict(groups=0), dict(weight=w[:8]), dict(weight=w.bfloat16()), dict(gate=x.bfloat16()), dict(gate=x[:2]),
           dict(eps=-1.0), dict(eps=float("nan")), dict(x=x.transpose(0, 1)), dict(x=x.half()), dict(y=x), dict(x=x[0, 0]),
           dict(stats=torch.zeros(4, 2, device="cuda"))]
    for kw in bad:
        with pytest.raises(qd.QDeltaError):
            qd.qdelta_group_norm_fwd(**dict(dict(x=x, groups=2, weight=w), **kw))
    with pytest.raises(qd.QDeltaError, match="stats"):
        qd.qdelta_group_norm_bwd(x, 2, w, None, None, None, x.clone())
    with pytest.raises(qd.QDeltaError, match="workspace"):
        qd.qdelta_group_norm_fwd(x, 2, w, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("shape", [(3, 0, 8), (3, 5, 0)])
def test_groups_without_elements_have_zero_statistics(qd, shape):
    stats = torch.full((3, 2, 2), 7.0, device="cuda")
    x = torch.zeros(shape, device="cuda")
    y, st = qd.qdelta_group_norm_fwd(x, 2, stats=stats)
    assert y.shape == shape and st is stats and not st.any()
    w = torch.ones(shape[-1], device="cuda")
    got = qd.qdelta_group_norm_bwd(x, 2, w, w, None, st, x)
    assert got["dx"].shape == shape and not got["dweight"].any() and not got["dbias"].any()


def test_millions_of_groups_over_rows(qd):
    """More groups than a launch has workgroups of one each: 2^22 + 12, of two rows and four channels."""
    N, L, G, E = (1 << 20) + 3, 2, 4, 4
    x, w, b, _, _ = make("f32", 4, L, G, E, True, False, 17)
    rows = torch.randn(N, L, G * E, generator=torch.Generator(device="cuda").manual_seed(18), device="cuda") * 1.5 + 0.3
    dy = torch.randn(N, L, G * E, generator=torch.Generator(device="cuda").manual_seed(19), device="cuda")
    y, stats = qd.qdelta_group_norm_fwd(rows, G, dev(w), dev(b))
    got = qd.qdelta_group_norm_bwd(rows, G, dev(w), dev(b), None, stats, dy)
    for a in (0, (1 << 18) - 4, (1 << 19) + 1, N - 8):         # groups of the first and of later rounds
        part = slice(a, a + 8)
        want, st, scale = mixer.norm_fwd(rows[part], G, w, b)
        within(y[part], want, scale, units(L, E), f"y {a}")
        grad, size = mixer.norm_bwd(rows[part], G, w, b, None, stats[part], dy[part])
        within(got["dx"][part], grad["dx"], size["dx"], 2 * units(L, E), f"dx {a}")
    hat = (rows - stats[:, None, :, :1].expand(N, L, G, E).reshape(N, L, -1)) * stats[:, None, :, 1:].expand(N, L, G, E).reshape(N, L, -1)
    for k, terms in (("dbias", dy), ("dweight", dy * hat)):
        # a thread adds a sixteenth of the 2^20 rows in four parts, then 16 sums meet
        bound = ((1 << 14) + 64) * 2.0 ** -24 * terms.double().abs().sum((0, 1))
        assert ((got[k].double() - terms.double().sum((0, 1))).abs() <= bound).all(), k


def test_a_million_groups_of_a_sample(qd):
    """More groups than the grid is wide: 2^20 + 5 of one channel and three rows."""
    N, L, G = 2, 3, (1 << 20) + 5
    rand = lambda seed, *s: torch.randn(*s, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")  # noqa: E731
    x, dy, w, b = rand(23, N, L, G) * 1.5 + 0.3, rand(24, N, L, G), rand(25, G), rand(26, G)
    y, stats = qd.qdelta_group_norm_fwd(x, G, w, b)
    got = qd.qdelta_group_norm_bwd(x, G, w, b, None, stats, dy)
    for a in (0, (1 << 19) + 3, G - 8):
        part = slice(a, a + 8)
        xs, dys = x[..., part].contiguous(), dy[..., part].contiguous()
        want, st, scale = mixer.norm_fwd(xs, 8, w[part], b[part])
        # three values may lie close together: their spread's relative error is that of the values over it
        near = np.maximum(1, (np.abs(xs.double().cpu().numpy()).max(1, keepdims=True) * st[:, None, :, 1]) ** 2)
        within(y[..., part], want, scale * near, units(L, 1), f"y {a}")
        grad, size = mixer.norm_bwd(xs, 8, w[part], b[part], None, stats[:, part], dys)
        for k, v in (("dx", got["dx"][..., part]), ("dweight", got["dweight"][part]), ("dbias", got["dbias"][part])):
            within(v, grad[k], size[k], 2 * units(L, 1) + N * L, f"{k} {a}")
