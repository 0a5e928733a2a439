"""Linear attention and the block norms together, as a layer has them: convolution, attention, the
norm per head with its gate, the norms at the block's end with the residual; forward, backward, a
prompt followed by single tokens, another stream, captured graphs."""
import pytest
import torch

from mixer_cases import dev, gen, randn

pytestmark = pytest.mark.gpu


def params(H, d, seed):
    g = gen(seed)
    D = H * d
    return dict(w=randn(g, D, 4) * 0.5, hw=1 + 0.1 * randn(g, d), post=1 + 0.1 * randn(g, D), scale=0.3 * randn(g, D), pre=1 + 0.1 * randn(g, D))


def tokens(B, T, H, d, seed):
    g = gen(seed)
    D = H * d
    return dict(x=randn(g, B, T, D), q=randn(g, B, T, H, d) / d ** 0.5, k=randn(g, B, T, H, d) / d ** 0.5,
                g=-torch.nn.functional.softplus(randn(g, B, T, H) - 2), z=randn(g, B, T, H, d), z2=randn(g, B, T, D))



def forward(qd, p, t, stream=None):
    """Everything that a backward pass needs: the convolution, attention, norm per head, block end."""
    B, T, H, d = t["q"].shape
    v, Sc = qd.qdelta_conv_fwd(t["x"], p["w"], stream=stream)
    o, S = qd.qdelta_linattn_fwd(t["q"], t["k"], v.view(B, T, H, d), t["g"], stream=stream)
    y, _, hs = qd.qdelta_block_norm_fwd(o, post=p["hw"], gate=t["z"], stream=stream)
    h, n, st = qd.qdelta_block_norm_fwd(y.view(B, T, H * d), t["x"], p["post"], t["z2"], p["scale"], p["pre"], act="sigmoid", stream=stream)
    return dict(v=v, Sc=Sc, o=o, S=S, y=y, hs=hs, h=h, n=n, st=st)


def backward(qd, p, t, f, dh, dn, stream=None):
    B, T, H, d = t["q"].shape
    D = H * d
    e = qd.qdelta_block_norm_bwd(f["y"].view(B, T, D), f["h"], p["post"], t["z2"], p["scale"], p["pre"], f["st"], dh, dn, act="sigmoid",
                                 stream=stream)
    m = qd.qdelta_block_norm_bwd(f["o"], None, p["hw"], t["z"], None, None, f["hs"], e["dy"].view(B, T, H, d), want_dx=False, stream=stream)
    a = qd.qdelta_linattn_bwd(t["q"], t["k"], f["v"].view(B, T, H, d), t["g"], None, m["dy"], want_dS0=False, stream=stream)
    c = qd.qdelta_conv_bwd(t["x"], p["w"], None, None, a["dv"].view(B, T, D), want_dS0=False, stream=stream)
    return dict(x=(e["dx"], c["dx"]), w=c["dw"], q=a["dq"], k=a["dk"], g=a["dg"], z=m["dgate"], hw=m["dpost"], z2=e["dgate"],
                post=e["dpost"], scale=e["dscale"], pre=e["dpre"])


def flat(r):
    return [v for x in r.values() for v in (x if isinstance(x, tuple) else (x,)) if v is not None]


def reference(p, t):
    """The same layer in torch float64 on the CPU, differentiable."""
    q = {k: v.double().cpu().requires_grad_() for k, v in {**p, **t}.items()}
    B, T, H, d = t["q"].shape
    D = H * d
    full = torch.cat([torch.zeros(B, 3, D, dtype=torch.float64), q["x"]], 1)
    v = torch.nn.functional.silu(sum(full[:, j:j + T] * q["w"][:, j] for j in range(4))).view(B, T, H, d)
    S, rows = torch.zeros(B, H, d, d, dtype=torch.float64), []
    for i in range(T):
        S = torch.exp(q["g"][:, i])[..., None, None] * S + v[:, i][..., :, None] * q["k"][:, i][..., None, :]
        rows.append((S * q["q"][:, i][..., None, :]).sum(-1))
    o = torch.stack(rows, 1)
    rms = lambda a: a / torch.sqrt((a * a).mean(-1, keepdim=True) + 1e-5)       # noqa: E731
    y = rms(o) * q["hw"] * torch.nn.functional.silu(q["z"])
    h = q["x"] + q["scale"] * torch.sigmoid(q["z2"]) * rms(y.reshape(B, T, D)) * q["post"]
    return h, rms(h) * q["pre"], q


def close(got, want, name, bar):
    err = float((got.double().cpu() - want).abs().max() / want.abs().max())
    print(f"  {name}: {err:.2e}", flush=True)
    assert err <= bar, name


@pytest.mark.parametrize("B,T,H", [(2, 37, 3), (1, 500, 1)])
def test_layer_forward_and_backward(qd, B, T, H):
    """fp32 end to end: each operator a few hundred roundings of 2^-24 (5e-6 with two norms between,
    which enlarge a relative error by the input's largest value over its size), 2e-5 of the largest
    value; gradients pass through all of them twice, 1e-4."""
    d = 64
    p, t = params(H, d, 1), tokens(B, T, H, d, 2)
    dh, dn = randn(gen(3), B, T, H * d), randn(gen(4), B, T, H * d)
    h, n, leaves = reference(p, t)
    ((h * dh.double()).sum() + (n * dn.double()).sum()).backward()
    P, X = {k: dev(v) for k, v in p.items()}, {k: dev(v) for k, v in t.items()}
    f = forward(qd, P, X)
    close(f["h"], h.detach(), "h", 2e-5)
    close(f["n"], n.detach(), "n", 2e-5)
    got = backward(qd, P, X, f, dev(dh), dev(dn))
    got["x"] = got["x"][0] + got["x"][1]
    for k, v in got.items():
        close(v, leaves[k].grad, "d" + k, 1e-4)


def test_prompt_then_tokens(qd):
    """Prefill, then decode token by token through all of them, against one call over everything."""
    B, T, H, d = 3, 40, 2, 64
    D = H * d
    p, t = {k: dev(v) for k, v in params(H, d, 5).items()}, {k: dev(v) for k, v in tokens(B, T, H, d, 6).items()}
    whole = forward(qd, p, t)
    f = forward(qd, p, {k: v[:, :34].contiguous() for k, v in t.items()})
    for i in range(34, T):
        c = {k: v[:, i].contiguous() for k, v in t.items()}
        v = qd.qdelta_conv_step(c["x"], p["w"], None, f["Sc"])
        o = qd.qdelta_linattn_step(c["q"], c["k"], v.view(B, H, d), c["g"], f["S"])
        y, *_ = qd.qdelta_block_norm_fwd(o, post=p["hw"], gate=c["z"], want_stats=False)
        h, n, _ = qd.qdelta_block_norm_fwd(y.view(B, D), c["x"], p["post"], c["z2"], p["scale"], p["pre"], act="sigmoid", want_stats=False)
        close(h, whole["h"][:, i].double().cpu(), f"h of token {i}", 2e-5)
        close(n, whole["n"][:, i].double().cpu(), f"n of token {i}", 2e-5)
    close(f["S"], whole["S"].double().cpu(), "the state", 2e-5)


def test_on_another_stream(qd):
    B, T, H, d = 1, 700, 2, 64
    p, t = {k: dev(v) for k, v in params(H, d, 5).items()}, {k: dev(v) for k, v in tokens(B, T, H, d, 6).items()}
    f = forward(qd, p, t)
    want = [f, backward(qd, p, t, f, t["x"], t["z2"])]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    f = forward(qd, p, t, s)
    got = [f, backward(qd, p, t, f, t["x"], t["z2"], s)]
    s.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(x, y) for x, y in zip(flat(a), flat(b)))


def test_captured_and_replayed(qd):
    """Two captured graphs of forward, backward and single tokens, replayed in turn on new inputs with
    eager work between: every replay gives the eager call's bits."""
    B, T, H, d = 1, 400, 2, 64
    p = {k: dev(v) for k, v in params(H, d, 5).items()}

    def work(t):
        f = forward(qd, p, t)
        r = backward(qd, p, t, f, t["x"], t["z2"])
        c = {k: t[k][:, -1].contiguous() for k in ("q", "k", "z", "g")}
        S = f["S"].clone()
        return flat(f) + flat(r) + [qd.qdelta_linattn_step(c["q"], c["k"], c["z"], c["g"], S), S]

    graphs = []
    for seed in (1, 2):
        t = {k: dev(v) for k, v in tokens(B, T, H, d, seed).items()}
        work(t)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = work(t)
        graphs.append((graph, t, out))
    for step in range(3):
        for k, (graph, t, out) in enumerate(graphs):
            fresh = {n: dev(v) for n, v in tokens(B, T, H, d, 10 + 2 * step + k).items()}
            for n in t:
                t[n].copy_(fresh[n])
            graph.replay()
            want = work(fresh)
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, want)), (step, k)


def every_call(qd, seed, workspace=None):
    """Each call that takes a workspace, in several of its forms; `workspace(bytes)` makes one."""
    ws = workspace or (lambda n: None)
    r, out = gen(seed), []
    for dtype, B, T, H, dk, dv, decay in (("bf16", 1, 1500, 2, 128, 64, "token"), ("f32", 2, 300, 2, 64, 128, "head"),
                                          ("bf16", 3, 200, 5, 64, 64, "head"), ("f32", 1, 1100, 1, 128, 128, "token"),
                                          ("bf16", 2, 100, 3, 128, 128, "none")):
        q, k = (dev(randn(r, B, T, H, dk, dtype=dtype)) / dk ** 0.5 for _ in range(2))
        v, do = (dev(randn(r, B, T, H, dv, dtype=dtype)) for _ in range(2))
        g = None if decay == "none" else -torch.nn.functional.softplus(dev(randn(r, *((H,) if decay == "head" else (B, T, H)))))
        S0 = dev(randn(r, B, H, dv, dk))
        lens = torch.tensor([T - 70 * b for b in range(B)], dtype=torch.int32, device="cuda")
        for n in (None, lens):
            out += qd.qdelta_linattn_fwd(q, k, v, g, S0, n, workspace=ws(qd.qdelta_linattn_fwd_workspace_bytes(B, T, H, dk, dv, q.dtype)))
            for want in (True, False):
                need = qd.qdelta_linattn_bwd_workspace_bytes(B, T, H, dk, dv, want and g is not None, q.dtype)
                out += flat(qd.qdelta_linattn_bwd(q, k, v, g, S0, do, S0, want_dg=want, lens=n, workspace=ws(need)))
    for N, C in ((3000, 260), (5, 9000), (70, 3)):
        y, x, z, dh, dn = (dev(randn(r, N, C)) for _ in range(5))
        a, b, c = (dev(randn(r, C)) for _ in range(3))
        h, n, st = qd.qdelta_block_norm_fwd(y, x, a, z, b, c)
        out += [h, n, st] + flat(qd.qdelta_block_norm_bwd(y, h, a, z, b, c, st, dh, dn,
                                                          workspace=ws(qd.qdelta_block_norm_bwd_workspace_bytes(N, C, True, y.dtype))))
    return [v for v in out if v is not None]


def test_workspaces_are_not_read_before_they_are_written(qd):
    """Exactly the bytes asked for, filled with NaN, and a guard behind them that stays."""
    guards = []

    def poisoned(n):
        w = torch.full(((n + 3) // 4 + 64,), float("nan"), device="cuda")
        guards.append(w[(n + 3) // 4:])
        return w.view(torch.uint8)[:n]
    want, got = every_call(qd, 31), every_call(qd, 31, poisoned)
    assert len(want) == len(got)
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    assert len(guards) == 33 and all(torch.isnan(g).all() for g in guards)


def test_two_streams_at_once(qd):
    """The same operators on two streams, without an order between them."""
    want = [every_call(qd, s) for s in (41, 43)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(2):
        for k, s in enumerate(streams):
            with torch.cuda.stream(s):
                got.append((k, every_call(qd, 41 + 2 * k)))
    torch.cuda.synchronize()
    for k, g in got:
        for a, b in zip(want[k], g):
            assert torch.equal(a, b)


def test_tensors_of_another_device_are_refused(qd):
    x = torch.zeros(1, 4, 2, 64, device="cuda")
    for call in (lambda: qd.qdelta_linattn_fwd(x, x, x.cpu()), lambda: qd.qdelta_linattn_step(x[0], x[0], x[0], None, torch.zeros(4, 2, 64, 64)),
                 lambda: qd.qdelta_linattn_bwd(x, x, x, torch.zeros(1, 4, 2), None, x), lambda: qd.qdelta_block_norm_fwd(x, x.cpu()),
                 lambda: qd.qdelta_block_norm_bwd(x, None, torch.ones(64), None, None, None, torch.ones(8, 2, device="cuda"), x)):
        with pytest.raises(qd.QDeltaError, match="device"):
            call()


def test_gradients_into_the_callers_tensors(qd):
    B, T, H, d = 2, 70, 2, 64
    p, t = {k: dev(v) for k, v in params(H, d, 71).items()}, {k: dev(v) for k, v in tokens(B, T, H, d, 72).items()}
    f = forward(qd, p, t)
    y, C = f["y"].view(B, T, H * d), H * d
    calls = [(lambda **kw: qd.qdelta_linattn_bwd(t["q"], t["k"], t["z"], t["g"], None, t["z"], **kw), "dq", "dg", t["q"]),
             (lambda **kw: qd.qdelta_block_norm_bwd(y, f["h"], p["post"], t["z2"], p["scale"], p["pre"], f["st"], t["x"], t["z2"], **kw),
              "dy", "dpre", t["x"])]
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


def test_attention_past_32_bit_offsets(qd):
    """Rows whose element offsets pass 2^31, against a call on the last rows that starts from the state
    before them.  What rounds differently between the two is the bf16 copy of P and of the state,
    2^-8 of their terms each and with either sign: 2^-5 of the largest value is far above it."""
    T, H, d, tail = 530_000, 32, 128, 200
    r = torch.Generator(device="cuda")
    r.manual_seed(1)
    wide = lambda: torch.randn(1, T, H, d, generator=r, device="cuda", dtype=torch.bfloat16)        # noqa: E731
    q, k, v, do = (wide() for _ in range(4))
    q.mul_(d ** -0.5), k.mul_(d ** -0.5)
    g = -torch.rand(1, T, H, generator=r, device="cuda")
    assert q.numel() > 2 ** 31
    o, S = qd.qdelta_linattn_fwd(q, k, v, g)
    cut = lambda *x: [a[:, T - tail:].contiguous() for a in x]                                      # noqa: E731
    _, Sm = qd.qdelta_linattn_fwd(*[a[:, T - 2000:T - tail].contiguous() for a in (q, k, v, g)])     # e^-900 behind it
    alone, S1 = qd.qdelta_linattn_fwd(*cut(q, k, v, g), Sm)
    close(S, S1.double().cpu(), "S", 1e-4)
    close(o[:, T - tail:], alone.double().cpu(), "o", 2 ** -5)
    for want_dg in (False, True):
        got = qd.qdelta_linattn_bwd(q, k, v, g, None, do, want_dg=want_dg)
        want = qd.qdelta_linattn_bwd(*cut(q, k, v, g), Sm, cut(do)[0], want_dg=want_dg)
        for n in ("dq", "dk", "dv", "dg")[:3 + want_dg]:
            close(got[n][:, T - tail:], want[n].double().cpu(), n, 2 ** -5)


def test_block_norm_past_32_bit_offsets(qd):
    N, C, tail = 1_050_000, 2048, 50
    r = torch.Generator(device="cuda")
    r.manual_seed(2)
    y, x = (torch.randn(N, C, generator=r, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    w = dev(randn(gen(5), C))
    h, n, st = qd.qdelta_block_norm_fwd(y, x, w, x, w, w)
    h1, n1, st1 = qd.qdelta_block_norm_fwd(y[-tail:], x[-tail:], w, x[-tail:], w, w)
    assert torch.equal(h[-tail:], h1) and torch.equal(n[-tail:], n1) and torch.equal(st[-tail:], st1)
    got = qd.qdelta_block_norm_bwd(y, h, w, x, w, w, st, x, n)
    want = qd.qdelta_block_norm_bwd(y[-tail:], h1, w, x[-tail:], w, w, st1, x[-tail:], n1)
    for k in ("dx", "dy", "dgate"):
        assert torch.equal(got[k][-tail:], want[k]), k


def test_sizes_past_32_bits_are_refused(qd):
    """2^32 + 5 rows are not the five that their low 32 bits say; nothing is read."""
    x = torch.empty((1 << 32) + 5, 1, device="cuda", dtype=torch.bfloat16)
    w, h = torch.ones(1, device="cuda"), torch.empty_like(x)
    for call in (lambda: qd.qdelta_block_norm_fwd(x, post=w, h=h, want_stats=False),
                 lambda: qd.qdelta_block_norm_bwd(x, x, w, None, None, w, torch.ones(5, 2, device="cuda"), x)):
        with pytest.raises(qd.QDeltaError, match=r"below 2\*\*31"):
            call()
