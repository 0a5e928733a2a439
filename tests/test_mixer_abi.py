"""CPU checks of the C ABI of the operators around the recurrence: every refusal happens on
the host before device work, so no call here reaches a kernel (addresses are never read)."""
import re
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
M = 1 << 20


@pytest.fixture(scope="module")
def lib():
    import recurrent_sequence_layers_amd as qd
    return qd.load_library()


def caller(fn, names, defaults):
    def call(lib, **kw):
        a = dict(defaults, **kw)
        assert set(a) == set(names), set(a) ^ set(names)
        return getattr(lib, fn)(*[a[n] for n in names], None)
    return call


def at(*names):
    return {n: (i + 1) * M for i, n in enumerate(names)}


CONV = ["x", "w", "bias", "S0", "lens", "y", "S_T", "B", "T", "D", "W", "silu", "dtype"]
conv = caller("qdelta_conv_fwd", CONV, dict(at(*CONV[:7]), B=2, T=8, D=64, W=4, silu=1, dtype=1))
CSTEP = ["x", "w", "bias", "S", "y", "N", "D", "W", "silu", "dtype"]
conv_step = caller("qdelta_conv_step", CSTEP, dict(at(*CSTEP[:5]), N=2, D=64, W=4, silu=1, dtype=1))
CBWD = ["x", "w", "bias", "S0", "lens", "dy", "dS_T", "dx", "dw", "dbias", "dS0", "B", "T", "D", "W", "silu", "dtype", "ws", "n"]
conv_bwd = caller("qdelta_conv_bwd", CBWD, dict(at(*CBWD[:4], *CBWD[5:11]), lens=None, B=2, T=8, D=64, W=4, silu=1, dtype=1, ws=64 * M, n=M))
SSM = ["u", "dt", "A", "Bm", "Cm", "D_", "z", "dtb", "S0", "lens", "o", "S_T", "B", "T", "D", "G", "N", "sp", "dtype", "ws", "n"]
ssm = caller("qdelta_ssm_fwd", SSM, dict(at(*SSM[:12]), B=2, T=8, D=64, G=2, N=16, sp=1, dtype=1, ws=64 * M, n=M))
SSTEP = ["u", "dt", "A", "Bm", "Cm", "D_", "z", "dtb", "S", "o", "n_seq", "D", "G", "N", "sp", "dtype"]
ssm_step = caller("qdelta_ssm_step", SSTEP, dict(at(*SSTEP[:10]), n_seq=2, D=64, G=2, N=16, sp=1, dtype=1))
SBWD = ["u", "dt", "A", "Bm", "Cm", "D_", "z", "dtb", "S0", "lens", "d_o", "dS_T", "du", "ddt", "dA", "dB", "dC", "dD", "dz", "ddtb",
        "dS0", "B", "T", "D", "G", "N", "sp", "dtype", "ws", "n"]
ssm_bwd = caller("qdelta_ssm_bwd", SBWD, dict(at(*SBWD[:9], *SBWD[10:21]), lens=None, B=2, T=8, D=64, G=2, N=16, sp=1, dtype=1, ws=64 * M, n=M))
NFWD = ["x", "w", "bias", "gate", "y", "stats", "N", "L", "C", "G", "eps", "silu", "dtype", "ws", "n"]
norm = caller("qdelta_group_norm_fwd", NFWD, dict(at(*NFWD[:6]), N=4, L=1, C=64, G=4, eps=1e-5, silu=0, dtype=1, ws=None, n=0))
NBWD = ["x", "w", "bias", "gate", "stats", "dy", "dx", "dw", "dbias", "dgate", "N", "L", "C", "G", "silu", "dtype", "ws", "n"]
norm_bwd = caller("qdelta_group_norm_bwd", NBWD, dict(at(*NBWD[:10]), N=4, L=1, C=64, G=4, silu=0, dtype=1, ws=64 * M, n=M))


def test_conv_refusals(lib):
    for kw, want in ((dict(B=-1), INVALID), (dict(T=-1), INVALID), (dict(D=-8), INVALID), (dict(W=1), UNSUPPORTED),
                     (dict(W=5), UNSUPPORTED), (dict(dtype=2), UNSUPPORTED), (dict(x=None), INVALID),
                     (dict(w=None), INVALID), (dict(y=None), INVALID), (dict(x=M + 2), INVALID), (dict(S_T=7 * M + 4), INVALID),
                     (dict(y=M), INVALID), (dict(y=M + 128), INVALID), (dict(y=2 * M), INVALID), (dict(S_T=6 * M), INVALID),
                     (dict(S_T=4 * M + 16), INVALID), (dict(T=1 << 30, B=1 << 10), UNSUPPORTED),
                     (dict(B=0), OK), (dict(D=0), OK)):
        assert conv(lib, **kw) == want, kw
    for kw, want in ((dict(N=-1), INVALID), (dict(W=6), UNSUPPORTED), (dict(S=None), INVALID), (dict(S=4 * M + 8), INVALID),
                     (dict(y=4 * M), INVALID), (dict(y=M), INVALID), (dict(N=0), OK)):
        assert conv_step(lib, **kw) == want, kw
    for kw, want in ((dict(W=5), UNSUPPORTED), (dict(dw=None), INVALID), (dict(dx=None), INVALID), (dict(dy=None), INVALID),
                     (dict(ws=None), WORKSPACE), (dict(n=16), WORKSPACE), (dict(ws=64 * M + 4), WORKSPACE), (dict(dx=M), INVALID),
                     (dict(dw=7 * M), INVALID), (dict(lens=7 * M), INVALID), (dict(ws=5 * M), INVALID), (dict(dS0=4 * M), INVALID), (dict(D=0), OK)):
        assert conv_bwd(lib, **kw) == want, kw


def test_ssm_refusals(lib):
    for kw, want in ((dict(B=-1), INVALID), (dict(G=0), INVALID), (dict(G=3), INVALID), (dict(N=8), UNSUPPORTED),
                     (dict(N=24), UNSUPPORTED), (dict(dtype=5), UNSUPPORTED), (dict(A=None), INVALID), (dict(u=None), INVALID),
                     (dict(Cm=None), INVALID), (dict(o=None), INVALID), (dict(A=3 * M + 4), INVALID), (dict(o=M), INVALID),
                     (dict(o=7 * M), INVALID), (dict(S_T=9 * M + 16), INVALID), (dict(S_T=5 * M), INVALID),
                     (dict(D=1 << 28, G=1), UNSUPPORTED), (dict(B=0), OK), (dict(D=0), OK)):
        assert ssm(lib, **kw) == want, kw
    need = lib.qdelta_ssm_fwd_workspace_bytes(1, 4096, 64, 1, 16, 1)
    rows = lambda B, T, G, N: 2 * B * G * N * ((T + 15) // 16 * 16 + 16) * 4  # noqa: E731  (B and C in fp32)
    assert need > rows(1, 4096, 1, 16)                                     # few channels: segments too
    assert lib.qdelta_ssm_fwd_workspace_bytes(8, 4096, 2048, 1, 16, 1) == rows(8, 4096, 1, 16)
    assert lib.qdelta_ssm_fwd_workspace_bytes(8, 0, 2048, 1, 16, 1) == 0
    assert ssm(lib, ws=None) == WORKSPACE and ssm(lib, n=64) == WORKSPACE and ssm(lib, ws=64 * M + 4) == WORKSPACE
    assert ssm(lib, B=1, T=4096, G=1, ws=64 * M, n=need - 1) == WORKSPACE
    assert ssm(lib, B=1, T=4096, G=1, ws=11 * M, n=need) == INVALID        # over o
    for kw, want in ((dict(n_seq=-1), INVALID), (dict(N=20), UNSUPPORTED), (dict(S=None), INVALID), (dict(S=9 * M + 4), INVALID),
                     (dict(o=9 * M), INVALID), (dict(o=8 * M), INVALID), (dict(G=5), INVALID), (dict(n_seq=0), OK)):
        assert ssm_step(lib, **kw) == want, kw
    assert lib.qdelta_ssm_bwd_workspace_bytes(2, 8, 64, 2, 16, 1) <= M
    for kw, want in ((dict(T=-1), INVALID), (dict(N=48), UNSUPPORTED), (dict(dA=None), INVALID), (dict(dB=None), INVALID),
                     (dict(d_o=None), INVALID), (dict(dz=None), INVALID), (dict(z=None), INVALID), (dict(ws=None), WORKSPACE),
                     (dict(n=64), WORKSPACE), (dict(du=M), INVALID), (dict(lens=12 * M), INVALID), (dict(dB=16 * M), INVALID), (dict(ws=10 * M), INVALID),
                     (dict(dS0=9 * M), INVALID), (dict(du=12 * M + 2), INVALID), (dict(D=0), OK)):
        assert ssm_bwd(lib, **kw) == want, kw


def test_norm_refusals(lib):
    for kw, want in ((dict(N=-1), INVALID), (dict(G=0), INVALID), (dict(G=3), INVALID), (dict(dtype=4), UNSUPPORTED),
                     (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID),
                     (dict(x=None), INVALID), (dict(y=None), INVALID), (dict(x=M + 8), INVALID), (dict(y=M), INVALID),
                     (dict(y=4 * M), INVALID), (dict(stats=5 * M), INVALID), (dict(L=100), WORKSPACE), (dict(N=0), OK),
                     (dict(L=0), OK), (dict(C=0), OK)):
        assert norm(lib, **kw) == want, kw
    for kw, want in ((dict(stats=None), INVALID), (dict(dy=None), INVALID), (dict(dx=None), INVALID), (dict(dgate=None), INVALID),
                     (dict(gate=None), INVALID), (dict(ws=None), WORKSPACE), (dict(n=8), WORKSPACE), (dict(dx=M), INVALID),
                     (dict(dw=9 * M), INVALID), (dict(ws=6 * M), INVALID), (dict(C=0), OK)):
        assert norm_bwd(lib, **kw) == want, kw


def test_workspace_queries_refuse_what_the_calls_refuse(lib):
    assert lib.qdelta_conv_bwd_workspace_bytes(2, 8, 64, 5, 1) == 0
    assert lib.qdelta_ssm_fwd_workspace_bytes(1, 4096, 64, 1, 24, 1) == 0
    assert lib.qdelta_ssm_bwd_workspace_bytes(1, 4096, 64, 3, 16, 1) == 0
    assert lib.qdelta_group_norm_fwd_workspace_bytes(4, 10, 64, 3, 1) == 0
    assert lib.qdelta_group_norm_bwd_workspace_bytes(4, 10, 64, 4, 9) == 0
    # the norm of a token's heads keeps its groups in registers; longer groups need the runs' sums
    assert lib.qdelta_group_norm_fwd_workspace_bytes(32768, 1, 2048, 16, 1) == 0
    assert lib.qdelta_group_norm_fwd_workspace_bytes(8, 100, 64, 4, 1) > 0


def test_binding_names_every_entry_point():
    import recurrent_sequence_layers_amd as qd
    text = open(os.path.join(ROOT, "include", "qdelta.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    for name in re.findall(r"\b(qdelta_(?:conv|ssm|group_norm)_[a-z_]+)\s*\(", text):
        assert callable(getattr(qd, name)), name


def test_binding_refuses_host_tensors():
    import torch
    import recurrent_sequence_layers_amd as qd
    x = torch.zeros(1, 2, 8)
    with pytest.raises(qd.QDeltaError, match="device tensor"):
        qd.qdelta_conv_fwd(x, torch.zeros(8, 4))
    with pytest.raises(qd.QDeltaError, match="device tensor"):
        qd.qdelta_ssm_fwd(x, x, torch.zeros(8, 16), torch.zeros(1, 2, 1, 16), torch.zeros(1, 2, 1, 16))
    with pytest.raises(qd.QDeltaError, match="device tensor"):
        qd.qdelta_group_norm_fwd(x, 2)


def test_sizes_past_a_launch_are_refused(lib):
    """One more run of a backward's workgroups, or a group count no power of two divides, and
    the launch has 2^32 threads."""
    big = (1 << 26) - 1
    assert conv_bwd(lib, B=big, T=1, D=256) == UNSUPPORTED and conv(lib, B=big, T=1, D=256) == UNSUPPORTED
    assert lib.qdelta_conv_bwd_workspace_bytes(big, 1, 256, 4, 1) == 0
    odd = (1 << 25) - 1
    assert norm(lib, N=1, C=odd, G=odd) == UNSUPPORTED and norm_bwd(lib, N=1, C=odd, G=odd) == UNSUPPORTED
    assert lib.qdelta_group_norm_bwd_workspace_bytes(1, 1, odd, odd, 1) == 0


def test_the_unsupported_status_names_the_limits(lib):
    text = lib.qdelta_status_string(UNSUPPORTED).decode()
    assert "W in 2..4" in text and "N in {16,32,64}" in text and "2^32" in text


def test_any_number_of_groups_over_rows(lib):
    """What a norm over rows needs is bounded by its rows and channels, not by its groups."""
    n = (1 << 20) + 3
    need = (n * 2 * 16 + n * 4 * 2) * 4                # a run and sample: two sums a channel; two numbers a group
    assert lib.qdelta_group_norm_fwd_workspace_bytes(n, 2, 16, 4, 0) == need
    assert lib.qdelta_group_norm_bwd_workspace_bytes(n, 2, 16, 4, 0) == need
    assert norm(lib, N=n, L=2, C=16, G=4, dtype=0) == WORKSPACE


def test_sizes_past_32_bits_are_refused_by_the_binding():
    """The library takes 32-bit sizes; the low 32 bits of a larger one are another size."""
    import recurrent_sequence_layers_amd as qd
    for T in (1 << 31, (1 << 32) + 16):
        for query, sizes in ((qd.qdelta_conv_bwd_workspace_bytes, (1, T, 1, 4)), (qd.qdelta_ssm_fwd_workspace_bytes, (1, T, 1, 1, 16)),
                             (qd.qdelta_ssm_bwd_workspace_bytes, (1, T, 1, 1, 16)),
                             (qd.qdelta_group_norm_fwd_workspace_bytes, (1, T, 1, 1)),
                             (qd.qdelta_group_norm_bwd_workspace_bytes, (1, T, 1, 1))):
            with pytest.raises(qd.QDeltaError, match="2\\*\\*31"):
                query(*sizes, qd.QD_BF16)


def test_a_stream_of_another_device_is_refused(monkeypatch):
    """Kernels enqueued there would be given addresses of a device that is not theirs."""
    import torch
    import recurrent_sequence_layers_amd as qd

    class Stream:
        def __init__(self, index):
            self.device = torch.device("cuda", index)
    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    for enter in (qd._launch_stream, qd._enter):
        with pytest.raises(qd.QDeltaError, match="stream must be on cuda:0, got one on cuda:1"):
            enter(Stream(1), torch.device("cuda", 0))
    assert qd._launch_stream(mine := Stream(1), torch.device("cuda", 1)) is mine
