"""Inputs and error bounds shared by the GPU tests of the operators around the recurrence.

An output may be off by the rounding to its type, eps_t / 2 of its value, and by the fp32
roundings on the way.  Those are bounded by (number of roundings on a path from an input to
the output) * 2^-24 * (the sum with every term by its absolute value, the oracle's scale):
every product, sum or library value on the way is off by at most a few units of 2^-24 of its
terms, and errors grow no faster than the terms' sum.  `u` counts 2^-24s.
"""
import numpy as np
import torch

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 2.0 ** -24


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def randn(g, *shape, dtype="f32"):
    return torch.randn(*shape, generator=g).to(DT[dtype])


def dev(t):
    return None if t is None else t.cuda()


def within(got, want, scale, u, name):
    """|got - want| <= eps_t / 2 |want| + u 2^-24 scale, elementwise."""
    half = torch.finfo(got.dtype).eps / 2
    got = got.detach().double().cpu().numpy()
    assert got.shape == want.shape, (name, got.shape, want.shape)
    if got.size == 0:
        return
    assert np.isfinite(got).all(), f"{name}: not finite"
    bound = half * np.abs(want) + u * EPS * scale + 1e-37
    worst = float((np.abs(got - want) / bound).max())
    print(f"  {name}: {worst:.3f} of the bound", flush=True)
    assert worst <= 1, f"{name}: {worst:.3g} times the bound"


def ssm_inputs(B, T, D, G, N, dtype, seed, state=True, gate=True, plus=True, extras=True, big=False):
    """big: dt up to 3, so delta A reaches -30 and most of the state is forgotten at once."""
    g = gen(seed)
    x = dict(u=randn(g, B, T, D, dtype=dtype), Bm=randn(g, B, T, G, N, dtype=dtype), Cm=randn(g, B, T, G, N, dtype=dtype))
    raw = torch.randn(B, T, D, generator=g) * (1.5 if big else 0.7)
    x["dt"] = (raw if plus else torch.nn.functional.softplus(raw - 2)).to(DT[dtype])
    x["A"] = -(0.2 + torch.rand(D, N, generator=g) * (10 if big else 2))
    x["D"] = randn(g, D) if extras else None
    x["dt_bias"] = randn(g, D) - 2 if extras else None
    if not plus and extras:
        x["dt_bias"] = torch.rand(D, generator=g) * 0.1
    x["z"] = randn(g, B, T, D, dtype=dtype) if gate else None
    x["S0"] = randn(g, B, D, N) if state else None
    x["d_o"] = randn(g, B, T, D, dtype=dtype)
    x["dS_T"] = randn(g, B, D, N) if state else None
    return x


def ssm_u(x, plus):
    """Roundings on a path of the scan.  A step: the exponent's product and argument (each 2^-24
    of its size, at most m = max |delta A|, hence 2 m + 3 with the base-2 constant and the
    hardware exp's own unit), the decay's product, delta u B and the sum: 2 m + 8.  softplus,
    silu, their derivatives: 16 together.  Sums over N states, D channels, B T tokens: one a
    term at most."""
    B, T, D = x["u"].shape
    raw = x["dt"].double() + (0 if x["dt_bias"] is None else x["dt_bias"].double())
    delta = torch.nn.functional.softplus(raw) if plus else raw
    m = float((delta.amax() if delta.numel() else torch.tensor(0.)) * x["A"].abs().max())
    return (2 * m + 8) * (T + 1) + x["Bm"].shape[-1] + D + B * T + 32
