"""The block norms at the ends of their ranges."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_sums_over_rows_of_a_hundred_million_channels(qd):
    """3 C columns of partial sums, 64 a workgroup of 1024: more than 2^32 threads from C = 89.5 million
    on.  One row; the reference in 64 bits on the device.  A row's two sums of C terms are in 1024 parts
    of about 10^5 each, whose fp32 roundings are as good as random and half a unit of 2^-24 each:
    under 2^-24 (sqrt(10^5) + 32) < 2^-15 of the sum in all; the rest, some ten roundings."""
    C = 100_000_001
    g = torch.Generator(device="cuda").manual_seed(1)
    y, dh, post, scale = (torch.randn(C, generator=g, device="cuda") for _ in range(4))
    h, _, stats = qd.qdelta_block_norm_fwd(y[None], None, post, None, scale)
    assert abs(float(stats[0, 0]) - float(1 / (y.double().square().mean() + 1e-5).sqrt())) <= 2.0 ** -14
    got = qd.qdelta_block_norm_bwd(y[None], h, post, None, scale, None, stats, dh[None], want_dx=False)
    hat = y.double() * stats[0, 0].double()
    for name, want in (("dpost", dh.double() * scale * hat), ("dscale", dh.double() * post * hat)):
        off = (got[name].double() - want).abs()
        assert bool((off <= 2.0 ** -20 * want.abs() + 1e-30).all()), name
    w = dh.double() * scale * post
    want = stats[0, 0].double() * (w - hat * (w * hat).mean())
    assert float((got["dy"][0].double() - want).abs().max()) <= 2.0 ** -20 * float(want.abs().max())
