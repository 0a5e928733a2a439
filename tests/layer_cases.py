"""Inputs and error bounds shared by the GPU tests of linear attention and the block norms.

Linear attention, elementwise: an output may be off by the rounding to its type, by the bf16
roundings inside (P and the state once each, 2^-8 of the terms they are part of; none in fp32),
and by fp32 roundings, counted as in mixer_cases.  Over a whole output the roundings are
independent: each contributes at most 2^-9 in the 2-norm (a rounding is uniform over the half step
either way, 2^-8 / sqrt(3) at the bottom of a binade and half that at its top, under 2^-8.8 over a
binade; the two inside fall on different parts of the sum), sqrt(2) 2^-8.8 < 2^-8.  In fp32 a
sum of n products in any order is off by under sqrt(n) 2^-24 of its terms in the 2-norm where they
are as good as random: n is under 2^14 here, times a few operators in a row, and the terms' sums are
under eight times the results; 2^-14 covers it with room for a decay's argument (|g| 2^-24 a chunk).
"""
import numpy as np
import torch

from mixer_cases import DT, dev, gen, randn, within

FWD = ("q", "k", "v", "g", "S0")


def inputs(B, T, H, dk, dv, dtype, seed, decay="token", state=True, strong=False):
    """q and k of length about one; decays of 0.98 to 0.4 a token (strong: down to e^-12)."""
    r = gen(seed)
    x = dict(q=(torch.randn(B, T, H, dk, generator=r) / dk ** 0.5).to(DT[dtype]),
             k=(torch.randn(B, T, H, dk, generator=r) / dk ** 0.5).to(DT[dtype]), v=randn(r, B, T, H, dv, dtype=dtype))
    shape = (H,) if decay == "head" else (B, T, H)
    x["g"] = None if decay == "none" else -torch.nn.functional.softplus(torch.randn(*shape, generator=r) * (4 if strong else 1) - (0 if strong else 2))
    x["S0"] = randn(r, B, H, dv, dk) if state else None
    x["d_o"] = randn(r, B, T, H, dv, dtype=dtype)
    x["dS_T"] = randn(r, B, H, dv, dk) if state else None
    return x


def units(x):
    """fp32 roundings on a path: a token's or a chunk's factor and sum, 12 a token; the factor's
    argument, m = max |g|, once a chunk and so at most 64 m a token; sums over both dimensions."""
    B, T, H, dk = x["q"].shape
    m = 0 if x["g"] is None or not x["g"].numel() else float(x["g"][x["g"].isfinite()].abs().max())
    return (12 + 2 * m) * (T + 64) + dk + x["v"].shape[-1]


def near(got, want, scale, x, name, parts=1, norm=True):
    """Within the elementwise bound, and in the 2-norm.  parts: element roundings on the way."""
    u = units(x)
    inside = 0 if got.dtype == torch.float32 else 2.0 ** -8 * parts / 2.0 ** -24
    within(got, want, scale, u + inside, name)
    if norm and got.numel():
        size = np.linalg.norm(want)
        off = np.linalg.norm(got.detach().double().cpu().numpy() - want)
        bar = 2.0 ** -8 if got.dtype != torch.float32 else 2.0 ** -14
        print(f"  {name}: {off / max(size, 1e-300):.2e} in the 2-norm", flush=True)
        assert off <= bar * size + 1e-30, f"{name}: {off / size:.3g}"


def call(qd, fn, x, names, **kw):
    return getattr(qd, fn)(*[dev(x[n]) for n in names], **kw)
