"""The operators around the recurrence used together: a whole mixer forward and backward, a
prompt followed by single tokens, another stream, captured graphs."""
import numpy as np
import pytest
import torch

import oracle
from mixer_cases import dev, gen, randn
from oracle import mixer

pytestmark = pytest.mark.gpu


def params(D, N, W, seed):
    g = gen(seed)
    return dict(w=randn(g, D, W) * 0.5, b=randn(g, D) * 0.1, A=-(0.2 + torch.rand(D, N, generator=g)), D=randn(g, D),
                dt_bias=randn(g, D) - 2, nw=1 + 0.1 * randn(g, D), nb=0.1 * randn(g, D))


def tokens(B, T, D, G, N, seed):
    g = gen(seed)
    return dict(x=randn(g, B, T, D), dt=randn(g, B, T, D), z=randn(g, B, T, D), Bm=randn(g, B, T, G, N), Cm=randn(g, B, T, G, N))


def forward(qd, p, t, H, stream=None):
    """conv -> scan -> norm per head with the gate: outputs, states and what a backward needs."""
    B, T, D = t["x"].shape
    u, Sc = qd.qdelta_conv_fwd(t["x"], p["w"], p["b"], stream=stream)
    o, Ss = qd.qdelta_ssm_fwd(u, t["dt"], p["A"], t["Bm"], t["Cm"], p["D"], None, p["dt_bias"], stream=stream)
    y, stats = qd.qdelta_group_norm_fwd(o.view(B * T, D), H, p["nw"], p["nb"], t["z"].view(B * T, D), stream=stream)
    return y.view(B, T, D), Sc, Ss, u, o, stats


def reference(p, t, H):
    """The same mixer in torch float64 on the CPU, differentiable."""
    q = {k: v.double() for k, v in p.items()}
    s = {k: v.double() for k, v in t.items()}
    leaves = {**q, **s}
    for v in leaves.values():
        v.requires_grad_()
    B, T, D = t["x"].shape
    W, G, N = p["w"].shape[1], t["Bm"].shape[2], t["Bm"].shape[3]
    full = torch.cat([torch.zeros(B, W - 1, D, dtype=torch.float64), s["x"]], 1)
    u = torch.nn.functional.silu(sum(full[:, j:j + T] * q["w"][:, j] for j in range(W)) + q["b"])
    delta = torch.nn.functional.softplus(s["dt"] + q["dt_bias"])
    h, rows = torch.zeros(B, D, N, dtype=torch.float64), []
    for i in range(T):
        h = torch.exp(delta[:, i, :, None] * q["A"]) * h + (delta * u)[:, i, :, None] * s["Bm"][:, i].repeat_interleave(D // G, 1)
        rows.append((h * s["Cm"][:, i].repeat_interleave(D // G, 1)).sum(-1) + q["D"] * u[:, i])
    o = torch.stack(rows, 1).view(B, T, H, D // H)
    hat = (o - o.mean(-1, keepdim=True)) / torch.sqrt(o.var(-1, correction=0, keepdim=True) + 1e-5)
    y = (hat.view(B, T, D) * q["nw"] + q["nb"]) * torch.nn.functional.silu(s["z"])
    return y, leaves


def close(got, want, name, bar=2e-5):
    """fp32 end to end: a mixer is three operators of some hundred roundings each (2^-24), and the
    norm can enlarge a relative error by the size of its input over its spread, a few here:
    a few hundred units, 2e-5 of the largest value."""
    err = float((got.double().cpu() - want).abs().max() / want.abs().max())
    print(f"  {name}: {err:.2e}", flush=True)
    assert err <= bar, name


def test_mixer_forward_and_backward(qd):
    B, T, D, G, N, H = 2, 37, 96, 2, 16, 4
    p, t = params(D, N, 4, 1), tokens(B, T, D, G, N, 2)
    dy = randn(gen(3), B, T, D)
    ref, leaves = reference(p, t, H)
    (ref * dy.double()).sum().backward()
    P, X = {k: dev(v.detach().float()) for k, v in p.items()}, {k: dev(v.detach().float()) for k, v in t.items()}
    y, _, _, u, o, stats = forward(qd, P, X, H)
    close(y, ref.detach(), "y")
    n = qd.qdelta_group_norm_bwd(o.view(B * T, D), H, P["nw"], P["nb"], X["z"].view(B * T, D), stats, dev(dy).view(B * T, D))
    s = qd.qdelta_ssm_bwd(u, X["dt"], P["A"], X["Bm"], X["Cm"], P["D"], None, P["dt_bias"], None, n["dx"].view(B, T, D))
    c = qd.qdelta_conv_bwd(X["x"], P["w"], P["b"], None, s["du"], want_dS0=False)
    got = dict(x=c["dx"], w=c["dw"], b=c["dbias"], dt=s["ddt"], A=s["dA"], Bm=s["dB"], Cm=s["dC"], D=s["dD"], dt_bias=s["ddt_bias"],
               z=n["dgate"].view(B, T, D), nw=n["dweight"], nb=n["dbias"])
    for k, v in got.items():
        close(v, leaves[k].grad, "d" + k, 1e-4)


def test_prompt_then_tokens(qd):
    """Prefill, then decode token by token through all three, against one call over everything."""
    B, T, D, G, N, H = 3, 24, 64, 1, 16, 2
    p, t = {k: dev(v) for k, v in params(D, N, 4, 5).items()}, {k: dev(v) for k, v in tokens(B, T, D, G, N, 6).items()}
    whole = forward(qd, p, t, H)[0]
    _, Sc, Ss, *_ = forward(qd, p, {k: v[:, :20].contiguous() for k, v in t.items()}, H)
    for i in range(20, T):
        c = {k: v[:, i].contiguous() for k, v in t.items()}
        u = qd.qdelta_conv_step(c["x"], p["w"], p["b"], Sc)
        o = qd.qdelta_ssm_step(u, c["dt"], p["A"], c["Bm"], c["Cm"], p["D"], None, p["dt_bias"], Ss)
        y, _ = qd.qdelta_group_norm_fwd(o, H, p["nw"], p["nb"], c["z"], want_stats=False)
        close(y, whole[:, i].double().cpu(), f"token {i}")


def test_around_the_delta_rule(qd):
    """conv -> Q-Delta (normalising q and k, gates as logits) -> norm per head with the gate."""
    B, T, H, d = 2, 100, 2, 64
    D = H * d
    g = gen(8)
    x = [randn(g, B, T, D, dtype="bf16") for _ in range(3)]
    ws = [(randn(g, D, 4) * 0.5) for _ in range(3)]
    al, be, la = (randn(g, B, T, H) - m for m in (4, 0, 0))
    z, nw = randn(g, B, T, D, dtype="bf16"), 1 + 0.1 * randn(g, D)
    qkv = [qd.qdelta_conv_fwd(dev(a), dev(w), want_state=False)[0].view(B, T, H, d) for a, w in zip(x, ws)]
    o, _ = qd.qdelta_chunk_fwd(*qkv, dev(al), dev(be), dev(la), C=64, raw=True)
    y, _ = qd.qdelta_group_norm_fwd(o.view(B * T, D), H, dev(nw), None, dev(z).view(B * T, D))
    from oracle import prologue
    ref = [mixer.conv_fwd(a, w)[0].reshape(B, T, H, d) for a, w in zip(x, ws)]
    ref = [torch.from_numpy(r).bfloat16().double().numpy() for r in ref]
    qh, kh, a, b, lam = prologue.prologue(ref[0], ref[1], al, be, la)
    ro, _ = oracle.qdelta_fwd(qh, kh, ref[2], a, b, lam, None)
    want, _, _ = mixer.norm_fwd(np.asarray(ro).reshape(B * T, 1, D), H, nw, None, z.reshape(B * T, 1, D))
    # the recurrence in bf16 is held to 2e-2 of its largest value per head; the norm divides by the spread
    spread = np.asarray(ro).reshape(B * T, H, d).std(-1)
    ratio = (np.abs(ro).max() / np.maximum(spread, 1e-6)).reshape(B * T, H, 1).repeat(d, 2).reshape(B * T, D)
    gate = np.abs(mixer.silu(z.double().numpy().reshape(B * T, D)))
    bound = 2e-2 * 3 * ratio * np.abs(nw.double().numpy()) * gate + 2.0 ** -8 * np.abs(want[:, 0]) + 1e-3
    assert (np.abs(y.double().cpu().numpy() - want[:, 0]) <= bound).all()


def test_on_another_stream(qd):
    B, T, D, G, N, H = 2, 700, 64, 1, 16, 2
    p, t = {k: dev(v) for k, v in params(D, N, 4, 5).items()}, {k: dev(v) for k, v in tokens(B, T, D, G, N, 6).items()}
    want = forward(qd, p, t, H)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = forward(qd, p, t, H, stream=s)
    s.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)


def test_captured_and_replayed(qd):
    """Two captured graphs of forward and backward, replayed in turn on new inputs with eager
    work between: every replay gives the eager call's bits."""
    B, T, D, G, N, H = 1, 400, 64, 1, 16, 2
    p = {k: dev(v) for k, v in params(D, N, 4, 5).items()}

    def work(t):
        y, Sc, Ss, u, o, stats = forward(qd, p, t, H)
        n = qd.qdelta_group_norm_bwd(o.view(B * T, D), H, p["nw"], p["nb"], t["z"].view(B * T, D), stats, t["x"].view(B * T, D))
        s = qd.qdelta_ssm_bwd(u, t["dt"], p["A"], t["Bm"], t["Cm"], p["D"], None, p["dt_bias"], None, n["dx"].view(B, T, D))
        c = qd.qdelta_conv_bwd(t["x"], p["w"], p["b"], None, s["du"])
        return [y, Sc, Ss] + [v for r in (n, s, c) for v in r.values() if v is not None]

    graphs = []
    for seed in (1, 2):
        t = {k: dev(v) for k, v in tokens(B, T, D, G, N, seed).items()}
        work(t)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = work(t)
        graphs.append((graph, t, out))
    for step in range(3):
        for k, (graph, t, out) in enumerate(graphs):
            fresh = {n: dev(v) for n, v in tokens(B, T, D, G, N, 10 + 2 * step + k).items()}
            for n in t:
                t[n].copy_(fresh[n])
            graph.replay()
            want = work(fresh)
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, want)), (step, k)


def every_call(qd, seed, workspace=None):
    """Each operator that takes a workspace, on sizes that use all of it; `workspace(bytes)` makes one."""
    ws = workspace or (lambda n: None)
    B, T, D, G, N = 2, 400, 72, 2, 16
    t = {k: dev(v) for k, v in tokens(B, T, D, G, N, seed).items()}
    p = {k: dev(v) for k, v in params(D, N, 4, seed + 1).items()}
    f32 = torch.float32
    o, S = qd.qdelta_ssm_fwd(t["x"], t["dt"], p["A"], t["Bm"], t["Cm"], p["D"], t["z"], p["dt_bias"],
                             workspace=ws(qd.qdelta_ssm_fwd_workspace_bytes(B, T, D, G, N, f32)))
    s = qd.qdelta_ssm_bwd(t["x"], t["dt"], p["A"], t["Bm"], t["Cm"], p["D"], t["z"], p["dt_bias"], None, o,
                          workspace=ws(qd.qdelta_ssm_bwd_workspace_bytes(B, T, D, G, N, f32)))
    c = qd.qdelta_conv_bwd(t["x"], p["w"], p["b"], None, t["z"], workspace=ws(qd.qdelta_conv_bwd_workspace_bytes(B, T, D, 4, f32)))
    y, st = qd.qdelta_group_norm_fwd(t["x"], 4, p["nw"], p["nb"], t["z"],
                                     workspace=ws(qd.qdelta_group_norm_fwd_workspace_bytes(B, T, D, 4, f32)))
    n = qd.qdelta_group_norm_bwd(t["x"], 4, p["nw"], p["nb"], t["z"], st, t["dt"],
                                 workspace=ws(qd.qdelta_group_norm_bwd_workspace_bytes(B, T, D, 4, f32)))
    rows = t["x"].view(B * T, D)
    _, st1 = qd.qdelta_group_norm_fwd(rows, 4, p["nw"], p["nb"])
    r = qd.qdelta_group_norm_bwd(rows, 4, p["nw"], p["nb"], None, st1, t["dt"].view(B * T, D),
                                 workspace=ws(qd.qdelta_group_norm_bwd_workspace_bytes(B * T, 1, D, 4, f32)))
    return [o, S, y, st] + [v for d in (s, c, n, r) for v in d.values() if v is not None]


def test_workspaces_are_not_read_before_they_are_written(qd):
    """Exactly the bytes asked for, filled with NaN, and a guard behind them that stays."""
    guards = []

    def poisoned(n):
        w = torch.full((n // 4 + 64,), float("nan"), device="cuda")
        guards.append(w[n // 4:])
        return w[:n // 4].view(torch.uint8)
    want, got = every_call(qd, 31), every_call(qd, 31, poisoned)
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    assert len(guards) == 6 and all(torch.isnan(g).all() for g in guards)


def test_two_streams_at_once(qd):
    """The same operators on two streams, without an order between them."""
    want = [every_call(qd, s) for s in (41, 43)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(3):
        for k, s in enumerate(streams):
            with torch.cuda.stream(s):
                got.append((k, every_call(qd, 41 + 2 * k)))
    torch.cuda.synchronize()
    for k, g in got:
        for a, b in zip(want[k], g):
            assert torch.equal(a, b)


def test_tensors_of_another_device_are_refused(qd):
    x = torch.zeros(1, 4, 8, device="cuda")
    with pytest.raises(qd.QDeltaError, match="device"):
        qd.qdelta_conv_fwd(x, torch.zeros(8, 4))
    with pytest.raises(qd.QDeltaError, match="device"):
        qd.qdelta_group_norm_fwd(x, 2, torch.ones(8))


# ---------------------------------------------------------------- offsets past 32 bits
LONG_T, LONG_D = 1_050_000, 2048          # 2.15e9 elements a tensor


def wide(seed, *shape):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.bfloat16)


def test_convolution_past_32_bit_offsets(qd):
    """Rows whose element offsets pass 2^31: the last rows against a call on those rows alone."""
    x, w, b = wide(1, 1, LONG_T, LONG_D), dev(randn(gen(2), LONG_D, 4)), dev(randn(gen(3), LONG_D))
    y, S = qd.qdelta_conv_fwd(x, w, b)
    tail = x[:, -50:].contiguous()
    alone, S1 = qd.qdelta_conv_fwd(tail, w, b)
    assert torch.equal(y[:, -47:], alone[:, 3:]) and torch.equal(S, S1)
    got = qd.qdelta_conv_bwd(x, w, b, None, y)
    want = qd.qdelta_conv_bwd(tail, w, b, None, y[:, -50:].contiguous())
    assert torch.equal(got["dx"][:, -47:], want["dx"][:, 3:])


def test_norm_past_32_bit_offsets(qd):
    x, w = wide(4, LONG_T, LONG_D), dev(randn(gen(5), LONG_D))
    y, st = qd.qdelta_group_norm_fwd(x, 16, w, gate=x)
    tail = x[-50:].contiguous()
    alone, st1 = qd.qdelta_group_norm_fwd(tail, 16, w, gate=tail)
    assert torch.equal(y[-50:], alone) and torch.equal(st[-50:], st1)
    got = qd.qdelta_group_norm_bwd(x, 16, w, None, x, st, y)
    want = qd.qdelta_group_norm_bwd(tail, 16, w, None, tail, st1, alone)
    assert torch.equal(got["dx"][-50:], want["dx"]) and torch.equal(got["dgate"][-50:], want["dgate"])


def test_scan_past_32_bit_offsets(qd):
    """The last tokens against a call on them alone from the state before them.  The long call
    cuts its time axis elsewhere, so states differ by fp32 roundings: their errors decay with
    the states, and the outputs may differ by one rounding to bf16, 2^-8 of the value, and by
    2^-14 (2^10 roundings of 2^-24) of the largest."""
    T, D, N, tail = LONG_T, LONG_D, 16, 64
    p = {k: dev(v) for k, v in params(D, N, 4, 7).items()}
    u, Bm, Cm = wide(8, 1, T, D), wide(9, 1, T, 1, N), wide(10, 1, T, 1, N)
    dt, d_o = wide(11, 1, T, D), wide(12, 1, T, D)
    o, S = qd.qdelta_ssm_fwd(u, dt, p["A"], Bm, Cm, p["D"], None, p["dt_bias"])
    cut = lambda t, a, b: t[:, a:b]  # noqa: E731  (contiguous: one sequence)
    _, S1 = qd.qdelta_ssm_fwd(*[cut(t, 0, T - tail) if t.dim() > 2 else t for t in (u, dt, p["A"], Bm, Cm)], p["D"], None,
                              p["dt_bias"])
    last = [cut(t, T - tail, T) if t.dim() > 2 else t for t in (u, dt, p["A"], Bm, Cm)]
    o1, S2 = qd.qdelta_ssm_fwd(*last, p["D"], None, p["dt_bias"], S1)

    def near(a, b, name):
        a, b = a.double(), b.double()
        worst = ((a - b).abs() / (2.0 ** -8 * b.abs() + 2.0 ** -14 * b.abs().max())).max()
        print(f"  {name}: {worst:.3f} of the bound", flush=True)
        assert worst <= 1, name
    near(o[:, -tail:], o1, "o")
    near(S, S2, "S_T")
    got = qd.qdelta_ssm_bwd(u, dt, p["A"], Bm, Cm, p["D"], None, p["dt_bias"], None, d_o, S)
    want = qd.qdelta_ssm_bwd(*last, p["D"], None, p["dt_bias"], S1, d_o[:, -tail:], S)
    for k in ("du", "ddt", "dB", "dC"):
        near(got[k][:, -tail:], want[k], k)


def test_workspaces_that_are_not_device_tensors_are_refused(qd):
    x = torch.randn(2, 6, 16, device="cuda")
    for bad in (torch.empty(1 << 20, dtype=torch.uint8), np.zeros(1 << 20, np.uint8), 1 << 20,
                torch.empty(1 << 20, 2, dtype=torch.uint8, device="cuda")[:, 0]):
        with pytest.raises(qd.QDeltaError, match="workspace"):
            qd.qdelta_conv_bwd(x, torch.randn(16, 4, device="cuda"), None, None, x.clone(), workspace=bad)
        with pytest.raises(qd.QDeltaError, match="workspace"):
            qd.qdelta_group_norm_fwd(x, 2, workspace=bad)


def test_states_of_no_tokens_past_32_bit_offsets(qd):
    """With no tokens the state's gradient is a copy: more elements than a launch has threads."""
    B, D, W = 5_600_000, 256, 4
    dS = torch.empty(B, W - 1, D, device="cuda", dtype=torch.bfloat16).normal_()
    x = torch.empty(B, 0, D, device="cuda", dtype=torch.bfloat16)
    got = qd.qdelta_conv_bwd(x, torch.ones(D, W, device="cuda"), None, None, x, dS)
    assert torch.equal(got["dS0"], dS) and not got["dw"].any()
    del dS, got
    B, D, N = (1 << 22) + 3, 64, 16
    dS = torch.empty(B, D, N, device="cuda").normal_()
    u, Bm = torch.empty(B, 0, D, device="cuda"), torch.empty(B, 0, 1, N, device="cuda")
    got = qd.qdelta_ssm_bwd(u, u, -torch.ones(D, N, device="cuda"), Bm, Bm, None, None, None, None, u, dS)
    assert torch.equal(got["dS0"], dS) and not got["dA"].any()


def test_padded_mixer_forward_and_backward(qd):
    """Convolution, scan and gated norm over a right-padded batch whose padding is NaN up to the
    gate: outputs and every gradient against the sequences one by one, padding's gradients zero."""
    B, T, D, G, N, H, lens = 4, 24, 96, 2, 16, 4, [24, 0, 7, 1]
    p, t = params(D, N, 4, 61), tokens(B, T, D, G, N, 62)
    dy = randn(gen(63), B, T, D)
    sums = {k: torch.zeros(v.shape, dtype=torch.float64) for k, v in {**p, **t}.items()}
    want = torch.zeros(B, T, D, dtype=torch.float64)
    for b, n in enumerate(lens):
        if n:
            y, leaves = reference(p, {k: v[b:b + 1, :n] for k, v in t.items()}, H)
            (y * dy[b:b + 1, :n]).sum().backward()
            want[b, :n] = y.detach()[0]
            for k, v in leaves.items():
                (sums[k][b, :n] if k in t else sums[k]).add_(v.grad[0] if k in t else v.grad)
        dy[b, n:] = 0
        for k in ("x", "dt", "Bm", "Cm"):
            t[k][b, n:] = float("nan")
    P, X, ln = {k: dev(v) for k, v in p.items()}, {k: dev(v) for k, v in t.items()}, torch.tensor(lens, dtype=torch.int32).cuda()
    u, _ = qd.qdelta_conv_fwd(X["x"], P["w"], P["b"], lens=ln)
    o, _ = qd.qdelta_ssm_fwd(u, X["dt"], P["A"], X["Bm"], X["Cm"], P["D"], None, P["dt_bias"], lens=ln)
    rows = (B * T, D)
    y, stats = qd.qdelta_group_norm_fwd(o.view(rows), H, P["nw"], P["nb"], X["z"].view(rows))
    for b, n in enumerate(lens):
        assert not u[b, n:].any() and not o[b, n:].any()
        if n:
            close(y.view(B, T, D)[b, :n], want[b, :n], f"y {b}")
    g = qd.qdelta_group_norm_bwd(o.view(rows), H, P["nw"], P["nb"], X["z"].view(rows), stats, dev(dy).view(rows))
    s = qd.qdelta_ssm_bwd(u, X["dt"], P["A"], X["Bm"], X["Cm"], P["D"], None, P["dt_bias"], None, g["dx"].view(B, T, D), lens=ln)
    c = qd.qdelta_conv_bwd(X["x"], P["w"], P["b"], None, s["du"], lens=ln)
    got = dict(x=c["dx"], w=c["dw"], b=c["dbias"], dt=s["ddt"], A=s["dA"], Bm=s["dB"], Cm=s["dC"], D=s["dD"],
               dt_bias=s["ddt_bias"], z=g["dgate"].view(B, T, D), nw=g["dweight"], nb=g["dbias"])
    for k, v in got.items():
        close(v, sums[k], "d" + k, 1e-4)
        if k in t:
            assert all(not v[b, n:].any() for b, n in enumerate(lens)), k


def test_gradients_into_the_callers_tensors(qd):
    """``out`` supplies any of the results: used and returned, the others new, the same values;
    a tensor of another shape, type or device, or an input's memory, is refused."""
    B, T, D, G, N = 2, 9, 16, 2, 16
    p, t = {k: dev(v) for k, v in params(D, N, 4, 71).items()}, {k: dev(v) for k, v in tokens(B, T, D, G, N, 72).items()}
    dy, S0, C0 = dev(randn(gen(73), B, T, D)), dev(randn(gen(74), B, D, N)), dev(randn(gen(75), B, 3, D))
    _, stats = qd.qdelta_group_norm_fwd(t["x"].view(B * T, D), G, p["nw"], p["nb"], t["z"].view(B * T, D))
    calls = [(lambda **kw: qd.qdelta_conv_bwd(t["x"], p["w"], p["b"], C0, dy, **kw), "dx", "dw", t["x"]),
             (lambda **kw: qd.qdelta_ssm_bwd(t["x"], t["dt"], p["A"], t["Bm"], t["Cm"], p["D"], t["z"], p["dt_bias"], S0, dy, **kw),
              "du", "dS0", t["dt"]),
             (lambda **kw: qd.qdelta_group_norm_bwd(t["x"].view(B * T, D), G, p["nw"], p["nb"], t["z"].view(B * T, D), stats,
                                                    dy.view(B * T, D), **kw), "dx", "dbias", t["z"].view(B * T, D))]
    for call, a, b, taken in calls:
        want = call()
        mine = {k: torch.full_like(want[k], 7.0) for k in (a, b)}
        got = call(out=mine)
        assert got[a] is mine[a] and got[b] is mine[b] and set(got) == set(want)
        for k in want:
            assert torch.equal(got[k], want[k]), k
        for bad in (want[a][:1].contiguous(), want[a].double(), want[a].cpu(), want[a].transpose(0, 1), taken):
            with pytest.raises(qd.QDeltaError):
                call(out={a: bad})


def test_sizes_past_32_bits_are_refused(qd):
    """2^32 + 5 tokens are not the five that their low 32 bits say; nothing of x is read."""
    x = torch.empty(1, (1 << 32) + 5, 1, device="cuda", dtype=torch.bfloat16)
    w, one = torch.ones(1, 4, device="cuda"), torch.ones(1, device="cuda")
    A, Bm = -torch.ones(1, 16, device="cuda"), torch.empty(1, 5, 1, 16, device="cuda", dtype=torch.bfloat16)
    y = torch.zeros_like(x)
    for call in (lambda: qd.qdelta_conv_fwd(x, w, y=y), lambda: qd.qdelta_conv_bwd(x, w, one, None, x, out=dict(dx=y)),
                 lambda: qd.qdelta_conv_step(x[0], w, None, torch.empty(5, 3, 1, device="cuda", dtype=torch.bfloat16)),
                 lambda: qd.qdelta_ssm_fwd(x, x, A, Bm, Bm, o=y), lambda: qd.qdelta_ssm_bwd(x, x, A, Bm, Bm, None, None, None, None, x),
                 lambda: qd.qdelta_group_norm_fwd(x, 1, one, y=y), lambda: qd.qdelta_group_norm_fwd(x.view(1, 3, -1, 1), 1, one),
                 lambda: qd.qdelta_group_norm_bwd(x, 1, one, None, None, torch.ones(1, 1, 2, device="cuda"), x, out=dict(dx=y))):
        with pytest.raises(qd.QDeltaError, match=r"below 2\*\*31"):
            call()
