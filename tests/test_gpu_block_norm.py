"""The block norms' kernels against the fp64 oracle."""
import numpy as np
import pytest
import torch

from mixer_cases import DT, dev, gen, randn, within
from oracle import layer

pytestmark = pytest.mark.gpu

# dtype, N, C, post, act (None: no gate), scale, x, pre
CASES = [("bf16", 5, 128, True, "silu", True, True, True), ("f32", 5, 64, True, "sigmoid", True, True, True),
         ("bf16", 3, 1, True, "silu", True, True, True), ("f32", 4, 3, True, "linear", True, True, True),
         ("bf16", 7, 7, True, "sigmoid", False, True, True), ("bf16", 9, 9, False, "linear", True, True, True),
         ("f32", 33, 5, True, None, True, True, False), ("bf16", 70, 100, False, None, False, True, True),
         ("bf16", 3, 511, True, "silu", False, False, False), ("f32", 300, 513, True, None, False, True, True),
         ("bf16", 2, 2048, True, "sigmoid", True, True, True), ("bf16", 3, 2049, True, "silu", True, True, True),
         ("f32", 2, 4100, True, "linear", True, False, True), ("f32", 3, 8191, False, "silu", False, True, True),
         ("bf16", 2, 8192, True, "sigmoid", True, True, True),
         # past a workgroup's registers
         ("bf16", 3, 8200, True, "silu", True, True, True), ("f32", 2, 9001, False, "sigmoid", True, True, True),
         ("bf16", 2, 12001, True, None, False, False, False)]
FLAGS = "dtype,N,C,post,act,scale,x,pre"


def make(dtype, N, C, post, act, scale, x, pre, seed):
    r = gen(seed)
    p = dict(y=randn(r, N, C, dtype=dtype) * 1.5, x=randn(r, N, C, dtype=dtype) if x else None, post=randn(r, C) if post else None,
             gate=randn(r, N, C, dtype=dtype) if act else None, scale=randn(r, C) if scale else None, pre=randn(r, C) if pre else None)
    return p, randn(r, N, C, dtype=dtype), randn(r, N, C, dtype=dtype) if pre else None


def units(C):
    """Roundings on a path: a row's sum of squares, 16 a lane, 6 between lanes, 16 between waves (12 a
    lane more in the looping form's longest rows); half its error in the root, 4; five products and
    the gate's exponential, reciprocal and products, 24."""
    return 80 + C // 1024


@pytest.mark.parametrize(FLAGS, CASES)
def test_forward(qd, dtype, N, C, post, act, scale, x, pre):
    p, *_ = make(dtype, N, C, post, act, scale, x, pre, C)
    h, n, stats = qd.qdelta_block_norm_fwd(*[dev(p[k]) for k in ("y", "x", "post", "gate", "scale", "pre")], act=act or "silu")
    want, r1, size = layer.block_norm_h(p["y"], p["x"], p["post"], p["gate"], p["scale"], act or "silu")
    within(h, want, size, units(C), "h")
    got = stats.cpu()
    if post:
        within(got[:, 0], r1, np.abs(r1), units(C), "1/rms of y")
    assert post or not got[:, 0].any()
    assert (n is None) == (not pre) and (pre or not got[:, 1].any())
    if pre:
        want, r2 = layer.block_norm_n(h, p["pre"])
        within(n, want, np.abs(want), units(C), "n")
        within(got[:, 1], r2, np.abs(r2), units(C), "1/rms of h")


@pytest.mark.parametrize(FLAGS, CASES)
def test_gradients(qd, dtype, N, C, post, act, scale, x, pre):
    p, dh, dn = make(dtype, N, C, post, act, scale, x, pre, C + 1)
    a = {k: dev(v) for k, v in p.items()}
    h, _, stats = qd.qdelta_block_norm_fwd(*[a[k] for k in ("y", "x", "post", "gate", "scale", "pre")], act=act or "silu")
    for d_h, d_n in ((dh, dn), (None, dn), (dh, None)):
        if d_h is None and d_n is None:
            continue
        got = qd.qdelta_block_norm_bwd(a["y"], h, a["post"], a["gate"], a["scale"], a["pre"], stats, dev(d_h), dev(d_n), act=act or "silu")
        want, mag = layer.block_norm_bwd(p["y"], h, p["post"], p["gate"], p["scale"], p["pre"], stats, d_h, d_n, act or "silu")
        for k, dep in (("dgate", "gate"), ("dpost", "post"), ("dscale", "scale"), ("dpre", "pre")):
            assert (got[k] is None) == (p[dep] is None), k
        for k, v in got.items():
            if v is not None:
                # sums over rows: a lane adds its rows one by one, then 64 partial sums, 16 lanes
                within(v, want[k], mag[k], 2 * units(C) + (N + 128 if k in ("dpost", "dscale", "dpre") else 0), k)


def test_many_rows(qd):
    """More rows than the persistent grids have slots, several rows a workgroup."""
    for dtype, N, C in (("bf16", 40000, 64), ("f32", 9000, 260)):
        p, dh, dn = make(dtype, N, C, True, "silu", True, True, True, 3)
        a = {k: dev(v) for k, v in p.items()}
        h, n, stats = qd.qdelta_block_norm_fwd(*[a[k] for k in ("y", "x", "post", "gate", "scale", "pre")])
        want, _, size = layer.block_norm_h(p["y"], p["x"], p["post"], p["gate"], p["scale"])
        within(h, want, size, units(C), "h")
        within(n, *[w for w in (layer.block_norm_n(h, p["pre"])[0],)], np.abs(layer.block_norm_n(h, p["pre"])[0]), units(C), "n")
        got = qd.qdelta_block_norm_bwd(a["y"], h, a["post"], a["gate"], a["scale"], a["pre"], stats, dev(dh), dev(dn))
        want, mag = layer.block_norm_bwd(p["y"], h, p["post"], p["gate"], p["scale"], p["pre"], stats, dh, dn)
        for k, v in got.items():
            within(v, want[k], mag[k], 2 * units(C) + (N if k in ("dpost", "dscale", "dpre") else 0), k)


def test_rows_of_any_shape_and_the_norm_per_head(qd):
    """[.., C]: the gated RMS norm of a layer's output per head is the norm alone with a gate."""
    r = gen(5)
    o, z, w = randn(r, 2, 5, 3, 64, dtype="bf16"), randn(r, 2, 5, 3, 64, dtype="bf16"), randn(r, 64)
    h, n, stats = qd.qdelta_block_norm_fwd(dev(o), post=dev(w), gate=dev(z))
    assert h.shape == o.shape and n is None and stats.shape == (30, 2)
    want, _, size = layer.block_norm_h(o.reshape(30, 64), None, w, z.reshape(30, 64), None)
    within(h.view(30, 64), want, size, units(64), "h")
    one = qd.qdelta_block_norm_fwd(dev(o[0, 0, 0]), post=dev(w), gate=dev(z[0, 0, 0]), want_stats=False)
    assert torch.equal(one[0], h[0, 0, 0]) and one[2] is None


def test_no_rows_no_channels(qd):
    w = torch.ones(8, device="cuda")
    e = torch.empty(0, 8, device="cuda")
    h, n, stats = qd.qdelta_block_norm_fwd(e, e, w, e, w, w)
    assert h.shape == n.shape == (0, 8) and stats.shape == (0, 2)
    got = qd.qdelta_block_norm_bwd(e, h, w, e, w, w, stats, e, e)
    assert all(not got[k].any() and got[k].shape == (8,) for k in ("dpost", "dscale", "dpre")) and got["dy"].shape == (0, 8)
    e = torch.empty(3, 0, device="cuda")
    h, _, stats = qd.qdelta_block_norm_fwd(e, pre=torch.empty(0, device="cuda"))
    assert h.shape == (3, 0) and not stats.any()


def test_zero_rows_stay_finite(qd):
    y = torch.zeros(2, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    h, n, stats = qd.qdelta_block_norm_fwd(y, None, w, None, None, w)
    assert not h.any() and not n.any() and stats.isfinite().all()
    got = qd.qdelta_block_norm_bwd(y, h, w, None, None, w, stats, torch.ones_like(y), torch.ones_like(y))
    assert all(v.isfinite().all() for v in got.values() if v is not None)


def test_gates_of_any_size(qd):
    """Where the sigmoid's exponential overflows or vanishes, the factor is 0 or 1 and its slope 0."""
    z = torch.tensor([[-1e30, -200.0, -100.0, 0.0, 100.0, 200.0, 1e30, 50.0]], device="cuda")
    y = torch.ones(1, 8, device="cuda")
    for act in ("sigmoid", "silu"):
        h, _, stats = qd.qdelta_block_norm_fwd(y, gate=z, act=act)
        want, *_ = layer.block_norm_h(y, None, None, z, None, act)
        np.testing.assert_allclose(h.cpu().numpy(), want, rtol=1e-6, atol=1e-37)
        got = qd.qdelta_block_norm_bwd(y, None, None, z, None, None, None, y, act=act)
        assert got["dgate"].isfinite().all() and float(got["dgate"][0, 0]) == 0


def test_the_same_call_twice_gives_the_same_bits(qd):
    p, dh, dn = make("bf16", 3000, 700, True, "silu", True, True, True, 7)
    a = {k: dev(v) for k, v in p.items()}
    h, _, stats = qd.qdelta_block_norm_fwd(*[a[k] for k in ("y", "x", "post", "gate", "scale", "pre")])
    runs = [qd.qdelta_block_norm_bwd(a["y"], h, a["post"], a["gate"], a["scale"], a["pre"], stats, dev(dh), dev(dn)) for _ in range(3)]
    assert all(torch.equal(runs[0][k], r[k]) for r in runs for k in r)


def test_refusals(qd):
    p, dh, dn = make("bf16", 4, 64, True, "silu", True, True, True, 9)
    a = {k: dev(v) for k, v in p.items()}
    order = ("y", "x", "post", "gate", "scale", "pre")
    for kw in (dict(x=a["x"].float()), dict(gate=a["gate"][:2]), dict(post=a["post"].bfloat16()), dict(pre=a["pre"][:8]),
               dict(scale=a["scale"].cpu()), dict(y=a["y"].t()), dict(act="relu"), dict(eps=-1.0), dict(eps=float("nan")),
               dict(pre=None, n=a["x"]), dict(h=a["y"]), dict(stats=torch.empty(4, 3, device="cuda")), dict(y=a["y"].half())):
        with pytest.raises(qd.QDeltaError):
            qd.qdelta_block_norm_fwd(**dict({k: a[k] for k in order}, **kw))
    h, _, stats = qd.qdelta_block_norm_fwd(*[a[k] for k in order])
    good = dict(y=a["y"], h=h, post=a["post"], gate=a["gate"], scale=a["scale"], pre=a["pre"], stats=stats, dh=dev(dh), dn=dev(dn))
    for kw in (dict(h=None), dict(stats=None), dict(dh=None, dn=None), dict(pre=None), dict(dn=good["dn"].float()), dict(act="tanh"),
               dict(out=dict(dy=a["y"])), dict(workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(qd.QDeltaError):
            qd.qdelta_block_norm_bwd(**dict(good, **kw))
