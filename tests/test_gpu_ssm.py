"""The selective scan's kernels against the fp64 oracle."""
import numpy as np
import pytest
import torch

from mixer_cases import DT, dev, ssm_inputs, ssm_u, within
from oracle import mixer

pytestmark = pytest.mark.gpu

FWD = ("u", "dt", "A", "Bm", "Cm", "D", "z", "dt_bias", "S0")
# dtype, B, T, D, G, N, state, gate, softplus, extras (D and dt_bias)
CASES = [("bf16", 2, 40, 64, 1, 16, True, True, True, True), ("bf16", 1, 1, 64, 1, 16, True, True, True, True),
         ("f32", 1, 1, 3, 1, 16, False, False, False, False), ("f32", 2, 7, 70, 2, 16, True, True, True, True),
         ("bf16", 2, 8, 130, 1, 32, False, True, True, True), ("f32", 1, 9, 66, 3, 32, True, False, False, True),
         ("bf16", 1, 23, 100, 4, 64, True, True, True, False), ("f32", 2, 31, 5, 1, 64, False, True, False, False),
         ("f32", 1, 16, 128, 128, 16, True, True, True, True), ("bf16", 3, 15, 65, 1, 16, True, False, True, True)]
# long enough for the time axis to be cut into segments, whole and ragged
LONG = [("f32", 1, 1024, 64, 1, 16, True, True, True, True), ("bf16", 2, 700, 96, 2, 16, True, True, True, True),
        ("f32", 1, 517, 40, 1, 64, False, False, True, True), ("bf16", 1, 333, 33, 1, 32, True, True, True, True)]


def make(case, seed, **kw):
    dtype, B, T, D, G, N, state, gate, plus, extras = case
    return ssm_inputs(B, T, D, G, N, dtype, seed, state, gate, plus, extras, **kw), plus


def run_fwd(qd, x, plus, **kw):
    return qd.qdelta_ssm_fwd(*[dev(x[k]) for k in FWD], softplus=plus, **kw)


@pytest.mark.parametrize("case", CASES + LONG)
def test_forward(qd, case):
    x, plus = make(case, case[2] + case[3])
    o, S = run_fwd(qd, x, plus)
    want, S_T, so, sS = mixer.ssm_fwd(*[x[k] for k in FWD], plus=plus)
    u = ssm_u(x, plus)
    within(o, want, so, u, "o")
    within(S, S_T, sS, u, "S_T")


@pytest.mark.parametrize("case", CASES + LONG)
def test_gradients(qd, case):
    x, plus = make(case, case[2] + case[3] + 1)
    got = qd.qdelta_ssm_bwd(*[dev(x[k]) for k in FWD], dev(x["d_o"]), dev(x["dS_T"]), softplus=plus)
    want, scale = mixer.ssm_bwd(*[x[k] for k in FWD], x["d_o"], x["dS_T"], plus)
    for k, dep in (("dD", "D"), ("dz", "z"), ("ddt_bias", "dt_bias")):
        assert (got[k] is None) == (x[dep] is None)
    for k, v in got.items():
        if v is not None:
            within(v, want[k], scale[k], 2 * ssm_u(x, plus), k)


@pytest.mark.parametrize("case", [CASES[0], CASES[3], CASES[6], LONG[0]])
def test_strong_decay(qd, case):
    """delta A down to tens: decays that underflow, and softplus on both of its branches."""
    x, plus = make(case, 77, big=True)
    o, S = run_fwd(qd, x, plus)
    want, S_T, so, sS = mixer.ssm_fwd(*[x[k] for k in FWD], plus=plus)
    within(o, want, so, ssm_u(x, plus), "o")
    within(S, S_T, sS, ssm_u(x, plus), "S_T")
    got = qd.qdelta_ssm_bwd(*[dev(x[k]) for k in FWD], dev(x["d_o"]), dev(x["dS_T"]), softplus=plus)
    want, scale = mixer.ssm_bwd(*[x[k] for k in FWD], x["d_o"], x["dS_T"], plus)
    for k, v in got.items():
        if v is not None:
            within(v, want[k], scale[k], 2 * ssm_u(x, plus), k)


def test_the_long_cases_are_cut_into_segments(qd):
    rows = lambda B, T, G, N: 2 * B * G * N * ((T + 15) // 16 * 16 + 16) * 4  # noqa: E731  (B and C in fp32)
    for dtype, B, T, D, G, N, *_ in LONG:
        assert qd.qdelta_ssm_fwd_workspace_bytes(B, T, D, G, N, DT[dtype]) > rows(B, T, G, N)
    assert qd.qdelta_ssm_fwd_workspace_bytes(8, 4096, 2048, 1, 16, torch.bfloat16) == rows(8, 4096, 1, 16)


@pytest.mark.parametrize("T", [20, 600])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_padded_prompts(qd, dtype, T):
    """Rows past a prompt's length stay as they were, what they hold is not read, and the
    state is the one after the last token; T = 600 is cut into segments."""
    lens = torch.tensor([T, 0, 1, T // 2 + 1, T + 9, -1], dtype=torch.int32)
    x = ssm_inputs(6, T, 36, 2, 16, dtype, 3)
    ref = mixer.ssm_fwd(*[x[k] for k in FWD], lens=lens)
    for b, n in enumerate([T, 0, 1, T // 2 + 1, T, 0]):
        for k in ("u", "dt", "z", "Bm", "Cm"):
            x[k][b, n:] = float("nan") if b % 2 else float("inf")
    o = torch.full((6, T, 36), 7.0, dtype=DT[dtype], device="cuda")
    o, S = run_fwd(qd, x, True, lens=dev(lens), o=o)
    want, S_T, so, sS = ref
    past = np.isnan(want)
    assert (o.double().cpu().numpy()[past] == 7.0).all()
    u = ssm_u(ssm_inputs(6, T, 36, 2, 16, dtype, 3), True)
    within(torch.where(torch.from_numpy(past).cuda(), torch.zeros_like(o), o), np.where(past, 0, want), so, u, "o")
    within(S, S_T, sS, u, "S_T")


@pytest.mark.parametrize("dtype,D,G,N", [("bf16", 64, 1, 16), ("f32", 35, 5, 32), ("bf16", 9, 1, 64)])
def test_steps_continue_a_prompt(qd, dtype, D, G, N):
    x = ssm_inputs(3, 14, D, G, N, dtype, 21)
    tok = ("u", "dt", "z", "Bm", "Cm")
    cut = lambda k, sl: dev(x[k][:, sl].contiguous()) if k in tok else dev(x[k])  # noqa: E731
    o, S = qd.qdelta_ssm_fwd(*[cut(k, slice(0, 10)) for k in FWD])
    rows = [o]
    for t in range(10, 14):
        rows.append(qd.qdelta_ssm_step(*[cut(k, t) for k in FWD[:-1]], S)[:, None])
    want, S_T, so, sS = mixer.ssm_fwd(*[x[k] for k in FWD])
    within(torch.cat(rows, 1), want, so, ssm_u(x, True), "o")
    within(S, S_T, sS, ssm_u(x, True), "S")


@pytest.mark.parametrize("T", [12, 1024])
def test_state_in_place(qd, T):
    """S_T may be S0, also where the last segment's workgroup ends before the others begin."""
    x = ssm_inputs(1, T, 64, 1, 16, "f32", 4)
    o0, S1 = run_fwd(qd, x, True)
    S = dev(x["S0"]).clone()
    args = [dev(x[k]) for k in FWD[:-1]]
    o1, _ = qd.qdelta_ssm_fwd(*args, S, S_T=S)
    assert torch.equal(o0, o1) and torch.equal(S, S1)


def test_no_tokens(qd):
    x = ssm_inputs(2, 0, 12, 1, 16, "bf16", 5)
    o, S = run_fwd(qd, x, True)
    assert o.shape == (2, 0, 12) and torch.equal(S.cpu(), x["S0"])
    _, S = qd.qdelta_ssm_fwd(*[dev(x[k]) for k in FWD[:5]])
    assert (S == 0).all()
    got = qd.qdelta_ssm_bwd(*[dev(x[k]) for k in FWD], dev(x["d_o"]), dev(x["dS_T"]))
    assert torch.equal(got["dS0"].cpu(), x["dS_T"])
    assert all((got[k] == 0).all() for k in ("dA", "dD", "ddt_bias"))


def test_softplus_over_its_range(qd):
    """One token, N = 16 states of A = 0 and B = C = 1/4: o = delta u, so the output is softplus
    itself.  In units of 2^-24 (half a unit in the last place is at most 1, the hardware's exp,
    log and reciprocal are within one place, 2): e 2 + 1 + 1 (exp2, its first-order factor,
    their product); log 2, its constant 1/2 and product 1; the product with e 1; the reciprocal
    2 and its product 1: 11.5.  Summing 16 terms delta / 16 rounds where 3 delta does, in a
    wave's four terms and in the four waves': 2 more, 13.5, so 14.  The terms' products with
    1/4, twice, are exact while delta / 16 is normal, that is above 2^-122."""
    xs = torch.cat([torch.linspace(-100, 60, 3001), torch.linspace(-20, 25, 2049)])
    D = xs.numel()
    one = torch.ones(1, 1, D, device="cuda")
    q = torch.full((1, 1, 1, 16), 0.25, device="cuda")
    o, _ = qd.qdelta_ssm_fwd(one, dev(xs).reshape(1, 1, D), torch.zeros(D, 16, device="cuda"), q, q)
    want = mixer.softplus(xs.double().numpy())
    got = o.double().cpu().numpy().reshape(-1)
    keep = want > 2.0 ** -122
    rel = np.abs(got - want)[keep] / want[keep]
    print(f"  softplus: {rel.max() / 2 ** -24:.2f} units of 2^-24", flush=True)
    assert rel.max() <= 14 * 2.0 ** -24
    assert (np.abs(got - want)[~keep] <= 2.0 ** -122).all()


def test_the_same_call_twice_gives_the_same_bits(qd):
    x = ssm_inputs(2, 300, 200, 2, 16, "bf16", 8)
    a = [dev(x[k]) for k in FWD] + [dev(x["d_o"]), dev(x["dS_T"])]
    first = qd.qdelta_ssm_bwd(*a)
    for _ in range(3):
        again = qd.qdelta_ssm_bwd(*a)
        assert all(torch.equal(first[k], again[k]) for k in first)


def test_refusals(qd):
    x = {k: dev(v) for k, v in ssm_inputs(2, 6, 16, 2, 16, "bf16", 2).items()}
    good = {k: x[k] for k in FWD}
    bad = [dict(dt=x["dt"].float()), dict(A=x["A"].bfloat16()), dict(A=x["A"][:, :8].contiguous()), dict(Cm=x["Cm"][:, :5]),
           dict(u=x["u"].transpose(1, 2)), dict(D=x["D"][:4]), dict(S0=x["S0"].bfloat16()), dict(z=x["z"].cpu()),
           dict(Bm=x["Bm"][:, :, :, :8].contiguous(), Cm=x["Cm"][:, :, :, :8].contiguous(), A=x["A"][:, :8].contiguous(), S0=None),
           dict(lens=torch.zeros(2, device="cuda")), dict(Bm=x["Bm"].expand(2, 6, 2, 16)[:, :, :1].expand(2, 6, 3, 16)),
           dict(o=x["u"])]
    for kw in bad:
        with pytest.raises(qd.QDeltaError):
            qd.qdelta_ssm_fwd(**dict(good, **kw))
    with pytest.raises(qd.QDeltaError, match="workspace"):
        qd.qdelta_ssm_bwd(**good, d_o=x["d_o"], workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(qd.QDeltaError):
        qd.qdelta_ssm_step(x["u"][:, 0].contiguous(), x["dt"][:, 0].contiguous(), x["A"], x["Bm"][:, 0].contiguous(),
                           x["Cm"][:, 0].contiguous(), None, None, None, x["S0"].bfloat16())


@pytest.mark.parametrize("T", [21, 600])
@pytest.mark.parametrize("N", [16, 64])
def test_decays_without_bound(qd, N, T):
    """A = -inf forgets at once, as -1e30 does to the last bit: tokens past the end, which leave
    the state as it is, must not turn it into NaN.  T = 600 is cut into segments."""
    x = ssm_inputs(3, T, 34, 2, N, "f32", 5)
    lens = dev(torch.tensor([T, T // 2 + 1, 3], dtype=torch.int32))
    x["A"][::3, 1::2] = -1e30
    near = [dev(x[k]) for k in FWD]
    x["A"][::3, 1::2] = float("-inf")
    none = [dev(x[k]) for k in FWD]
    zeros = torch.zeros(3, T, 34, device="cuda")
    for kw in (dict(), dict(lens=lens)):
        got, want = qd.qdelta_ssm_fwd(*none, **kw, o=zeros.clone()), qd.qdelta_ssm_fwd(*near, **kw, o=zeros.clone())
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and got[1].isfinite().all()
    got, want = (qd.qdelta_ssm_bwd(*a, dev(x["d_o"]), dev(x["dS_T"])) for a in (none, near))
    for k in got:
        assert torch.equal(got[k], want[k]) and got[k].isfinite().all(), k
    tok = [t[:, 0].contiguous() if t.dim() > 2 and t.shape[1] == T else t for t in none[:-1]]
    got, want = none[-1].clone(), none[-1].clone()
    o = qd.qdelta_ssm_step(*tok, got)
    tok[2] = near[2]
    assert torch.equal(o, qd.qdelta_ssm_step(*tok, want)) and torch.equal(got, want) and got.isfinite().all()


def test_nothing_carried_through_a_growing_segment(qd):
    """A > 0: a segment's factor overflows where nothing is there to grow."""
    x = ssm_inputs(2, 600, 36, 2, 16, "f32", 6, state=False, plus=False, extras=False)
    x["A"], x["dt"] = torch.full_like(x["A"], 2.0), torch.ones_like(x["dt"])
    x["u"][:, :-5] = 0
    x["d_o"][:, 5:] = 0
    o, S = run_fwd(qd, x, False)
    want, S_T, so, sS = mixer.ssm_fwd(*[x[k] for k in FWD], plus=False)
    within(o, want, so, ssm_u(x, False), "o")
    within(S, S_T, sS, ssm_u(x, False), "S_T")
    got = qd.qdelta_ssm_bwd(*[dev(x[k]) for k in FWD], dev(x["d_o"]), softplus=False)
    want, scale = mixer.ssm_bwd(*[x[k] for k in FWD], x["d_o"], None, False)
    for k, v in got.items():
        if v is not None:
            within(v, want[k], scale[k], 2 * ssm_u(x, False), k)


@pytest.mark.parametrize("dtype,T,D,G,N", [("bf16", 20, 36, 2, 16), ("f32", 20, 36, 2, 16), ("f32", 33, 65, 1, 32),
                                           ("bf16", 17, 40, 1, 64), ("bf16", 600, 36, 2, 16), ("f32", 1, 5, 1, 16)])
def test_gradients_of_a_padded_batch(qd, dtype, T, D, G, N):
    """Padding is not read and its rows' gradients are zero, dB's and dC's too; dS_T belongs to
    the state at the sequence's end.  Segments past an end have no tokens at all."""
    lens = [T, 0, 1, T // 2 + 1, T + 9, -1]
    x = ssm_inputs(6, T, D, G, N, dtype, 41)
    order = FWD + ("d_o", "dS_T")
    per = tuple(i if k in ("u", "dt", "Bm", "Cm", "z", "d_o") else -1 - i for i, k in enumerate(order)
                if k not in ("A", "D", "dt_bias"))
    want, scale = mixer.each_sequence(mixer.ssm_bwd, lens, ("dA", "dD", "ddt_bias"), per, *[x[k] for k in order])
    u = 2 * ssm_u(x, True)
    whole = [dev(x[k]) for k in order]
    for b, n in enumerate(lens):
        for k in ("u", "dt", "z", "Bm", "Cm", "d_o"):
            x[k][b, max(n, 0):] = float("nan") if b % 2 else float("inf")
    got = qd.qdelta_ssm_bwd(*[dev(x[k]) for k in order], lens=dev(torch.tensor(lens, dtype=torch.int32)))
    for k, v in got.items():
        within(v, want[k], scale[k], u, k)
    full = qd.qdelta_ssm_bwd(*whole)
    every = torch.full((6,), T, dtype=torch.int32, device="cuda")
    got = qd.qdelta_ssm_bwd(*whole, lens=every)
    assert all(torch.equal(got[k], full[k]) for k in got)
    with pytest.raises(qd.QDeltaError):
        qd.qdelta_ssm_bwd(*whole, lens=every[:5])


@pytest.mark.parametrize("dtype,B,T,D,G", [("bf16", 8, 530, 2048, 1), ("f32", 12, 545, 1030, 1), ("bf16", 6, 560, 2040, 12)])
def test_long_tiles(qd, dtype, B, T, D, G):
    """Nearly a workgroup for every compute unit and no segments: tiles of 32 tokens, whole and
    ragged, with and without lens, against the same tokens in shorter calls, which take the short
    tiles.  States go over in fp32 and every sum has the same order: the results are the same."""
    x = {k: dev(v) for k, v in ssm_inputs(B, T, D, G, 16, dtype, 51).items()}
    tok = ("u", "dt", "z", "Bm", "Cm")
    need = qd.qdelta_ssm_fwd_workspace_bytes(B, T, D, G, 16, DT[dtype])
    assert need == 2 * B * G * 16 * ((T + 15) // 16 * 16 + 16) * 4          # B and C in fp32 only
    o, S = qd.qdelta_ssm_fwd(*[x[k] for k in FWD])
    lens = torch.arange(B, dtype=torch.int32, device="cuda") * (T // B)
    ol, Sl = qd.qdelta_ssm_fwd(*[x[k] for k in FWD], lens=lens, o=torch.zeros_like(o))
    state, rows = x["S0"], []
    for a in range(0, T, 64):
        part, state = qd.qdelta_ssm_fwd(*[x[k][:, a:a + 64].contiguous() if k in tok else x[k] for k in FWD[:-1]], state)
        rows.append(part)
    assert torch.equal(o, torch.cat(rows, 1)) and torch.equal(S, state)
    for b, n in enumerate(lens.tolist()):
        assert torch.equal(ol[b, :n], o[b, :n]) and not ol[b, n:].any()
    assert torch.equal(Sl[0], x["S0"][0])


@pytest.mark.parametrize("sign", [1, -1])
def test_states_carried_through_segments_by_factors_beyond_fp32(qd, sign):
    """A state of 1e-30 that the first sixteen tokens multiply by e^94 (or one of 1e30 by e^-94): the
    product is an ordinary number, the segment's factor alone is beyond 2^128 (below 2^-126).  The
    gradient that those tokens carry back is scaled alike."""
    small = 10.0 ** (-30 * sign)
    x = ssm_inputs(2, 600, 36, 2, 16, "f32", 9, plus=False, extras=False, gate=False)
    x["A"], x["dt"] = torch.full_like(x["A"], float(sign)), torch.full_like(x["dt"], -sign * 1e-3)
    x["dt"][:, :16] = 94 / 16
    x["S0"] *= small
    x["u"][:, :16] = 0
    x["u"][:, 16:] *= 1e-12
    x["d_o"][:, :16] = 0
    x["d_o"][:, 16:] *= small
    x["dS_T"] *= small
    o, S = run_fwd(qd, x, False)
    want, S_T, so, sS = mixer.ssm_fwd(*[x[k] for k in FWD], plus=False)
    within(o, want, so, ssm_u(x, False), "o")
    within(S, S_T, sS, ssm_u(x, False), "S_T")
    assert np.abs(S_T).min() > (1e5 if sign > 0 else 1e-17)
    got = qd.qdelta_ssm_bwd(*[dev(x[k]) for k in FWD], dev(x["d_o"]), dev(x["dS_T"]), softplus=False)
    want, scale = mixer.ssm_bwd(*[x[k] for k in FWD], x["d_o"], x["dS_T"], False)
    for k, v in got.items():
        if v is not None:
            within(v, want[k], scale[k], 2 * ssm_u(x, False), k)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gradients_without_channels(qd, dtype):
    """dB and dC sum over channels: without any they are zeros, in new tensors and in the caller's."""
    u, Bm = torch.empty(2, 5, 0, dtype=DT[dtype], device="cuda"), torch.ones(2, 5, 3, 16, dtype=DT[dtype], device="cuda")
    A = torch.empty(0, 16, device="cuda")
    mine = {k: torch.full_like(Bm, 7.0) for k in ("dB", "dC")}
    got = qd.qdelta_ssm_bwd(u, u, A, Bm, Bm, None, None, None, None, u, out=mine)
    assert all(got[k] is mine[k] and not got[k].any() for k in mine)
    left = torch.full_like(Bm, float("nan"))           # memory that a new tensor may be given
    del left
    got = qd.qdelta_ssm_bwd(u, u, A, Bm, Bm, None, None, None, None, u)
    assert all(got[k].shape == Bm.shape and not got[k].any() for k in mine)
    assert got["du"].shape == u.shape and got["dA"].shape == A.shape and got["dS0"].shape == (2, 0, 16)
