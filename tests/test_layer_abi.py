"""CPU checks of the C ABI of linear attention and of the block norms: every refusal happens on the
host before device work, so no call here reaches a kernel (addresses are never read)."""
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
M = 1 << 24


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


FWD = ["q", "k", "v", "g", "S0", "lens", "o", "S_T", "B", "T", "H", "dk", "dv", "per_head", "dtype", "ws", "n"]
fwd = caller("qdelta_linattn_fwd", FWD, dict(at(*FWD[:8]), B=64, T=8, H=4, dk=64, dv=128, per_head=0, dtype=1, ws=None, n=0))
STEP = ["q", "k", "v", "g", "S", "o", "N", "H", "dk", "dv", "per_head", "dtype"]
step = caller("qdelta_linattn_step", STEP, dict(at(*STEP[:6]), N=2, H=4, dk=64, dv=128, per_head=0, dtype=1))
BWD = ["q", "k", "v", "g", "S0", "lens", "d_o", "dS_T", "dq", "dk_", "dv_", "dg", "dS0", "B", "T", "H", "dk", "dv", "per_head",
       "dtype", "ws", "n"]
bwd = caller("qdelta_linattn_bwd", BWD, dict(at(*BWD[:13]), B=64, T=8, H=4, dk=64, dv=128, per_head=0, dtype=1, ws=64 * M, n=M))
NFWD = ["y", "x", "post", "gate", "scale", "pre", "h", "n_", "stats", "N", "C", "eps", "act", "dtype"]
norm = caller("qdelta_block_norm_fwd", NFWD, dict(at(*NFWD[:9]), N=4, C=64, eps=1e-5, act=2, dtype=1))
NBWD = ["y", "h", "post", "gate", "scale", "pre", "stats", "dh", "dn", "dx", "dy", "dgate", "dpost", "dscale", "dpre", "N", "C",
        "act", "dtype", "ws", "n"]
norm_bwd = caller("qdelta_block_norm_bwd", NBWD, dict(at(*NBWD[:15]), N=4, C=64, act=2, dtype=1, ws=64 * M, n=M))


def test_linattn_refusals(lib):
    for kw, want in ((dict(B=-1), INVALID), (dict(T=-1), INVALID), (dict(H=-1), INVALID), (dict(dk=32), UNSUPPORTED),
                     (dict(dv=96), UNSUPPORTED), (dict(dtype=2), UNSUPPORTED), (dict(H=40000, B=1), UNSUPPORTED),
                     (dict(B=1 << 22, H=8), UNSUPPORTED), (dict(T=0x7fffffff), UNSUPPORTED),
                     (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(o=None), INVALID),
                     (dict(q=M + 8), INVALID), (dict(S_T=8 * M + 4), INVALID), (dict(o=M), INVALID), (dict(o=4 * M), INVALID),
                     (dict(S_T=5 * M + 16), INVALID), (dict(S_T=7 * M), INVALID), (dict(lens=7 * M), INVALID),
                     (dict(B=0), OK), (dict(H=0), OK)):
        assert fwd(lib, **kw) == want, kw
    need = lib.qdelta_linattn_fwd_workspace_bytes(1, 4096, 2, 128, 128, 1)
    assert need > 0 and lib.qdelta_linattn_fwd_workspace_bytes(8, 4096, 16, 128, 128, 1) == 0
    assert lib.qdelta_linattn_fwd_workspace_bytes(1, 4096, 2, 96, 128, 1) == 0
    long = dict(B=1, T=4096, H=2, dk=128)
    assert fwd(lib, **long) == WORKSPACE and fwd(lib, **long, ws=64 * M, n=need - 1) == WORKSPACE
    assert fwd(lib, **long, ws=64 * M + 8, n=need) == WORKSPACE and fwd(lib, **long, ws=7 * M, n=need) == INVALID
    for kw, want in ((dict(N=-1), INVALID), (dict(dk=48), UNSUPPORTED), (dict(dtype=3), UNSUPPORTED), (dict(S=None), INVALID),
                     (dict(o=None), INVALID), (dict(S=5 * M + 4), INVALID), (dict(o=5 * M), INVALID), (dict(o=M), INVALID),
                     (dict(g=5 * M), INVALID), (dict(N=1 << 22, H=8), UNSUPPORTED), (dict(N=0), OK)):
        assert step(lib, **kw) == want, kw


def test_linattn_gradient_refusals(lib):
    assert 0 < lib.qdelta_linattn_bwd_workspace_bytes(64, 8, 4, 64, 128, 1, 1) <= M
    assert lib.qdelta_linattn_bwd_workspace_bytes(64, 8, 4, 64, 128, 0, 1) == 0
    assert lib.qdelta_linattn_bwd_workspace_bytes(64, 8, 4, 64, 100, 1, 1) == 0
    for kw, want in ((dict(T=-1), INVALID), (dict(dv=32), UNSUPPORTED), (dict(dtype=7), UNSUPPORTED), (dict(d_o=None), INVALID),
                     (dict(dq=None), INVALID), (dict(dk_=None), INVALID), (dict(dv_=None), INVALID), (dict(g=None), INVALID),
                     (dict(ws=None), WORKSPACE), (dict(n=64), WORKSPACE), (dict(ws=64 * M + 4), WORKSPACE), (dict(dq=M), INVALID),
                     (dict(dg=4 * M), INVALID), (dict(dS0=5 * M), INVALID), (dict(lens=9 * M), INVALID), (dict(ws=7 * M), INVALID),
                     (dict(dv_=11 * M + 2), INVALID), (dict(dS0=8 * M), INVALID), (dict(B=1 << 22, T=64, H=1), UNSUPPORTED), (dict(H=0), OK)):
        assert bwd(lib, **kw) == want, kw


def test_block_norm_refusals(lib):
    for kw, want in ((dict(N=-1), INVALID), (dict(C=-1), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
                     (dict(eps=float("inf")), INVALID), (dict(act=3), INVALID), (dict(act=-1), INVALID), (dict(dtype=2), UNSUPPORTED),
                     (dict(C=1 << 28), UNSUPPORTED), (dict(y=None), INVALID), (dict(h=None), INVALID), (dict(pre=None), INVALID),
                     (dict(n_=None), INVALID), (dict(y=M + 8), INVALID), (dict(h=M), INVALID), (dict(h=2 * M), INVALID),
                     (dict(n_=7 * M), INVALID), (dict(stats=8 * M), INVALID), (dict(h=6 * M), INVALID), (dict(N=0), OK), (dict(C=0), OK)):
        assert norm(lib, **kw) == want, kw
    assert 0 < lib.qdelta_block_norm_bwd_workspace_bytes(4, 64, 1, 1) <= M
    assert lib.qdelta_block_norm_bwd_workspace_bytes(4, 64, 0, 1) == 0 and lib.qdelta_block_norm_bwd_workspace_bytes(4, 64, 1, 9) == 0
    for kw, want in ((dict(N=-1), INVALID), (dict(act=5), INVALID), (dict(dtype=2), UNSUPPORTED), (dict(y=None), INVALID),
                     (dict(dy=None), INVALID), (dict(h=None), INVALID), (dict(stats=None), INVALID), (dict(dgate=None), INVALID),
                     (dict(gate=None), INVALID), (dict(post=None), INVALID), (dict(scale=None), INVALID), (dict(pre=None), INVALID),
                     (dict(dh=None, dn=None), INVALID), (dict(ws=None), WORKSPACE), (dict(n=8), WORKSPACE), (dict(dx=M), INVALID),
                     (dict(dpost=14 * M), INVALID), (dict(ws=8 * M), INVALID), (dict(dy=9 * M), INVALID), (dict(dx=M + 8), INVALID),
                     (dict(C=0), OK)):
        assert norm_bwd(lib, **kw) == want, kw


def test_binding_names_every_entry_point():
    import recurrent_sequence_layers_amd as qd
    text = open(os.path.join(ROOT, "include", "qdelta.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = re.findall(r"\b(qdelta_(?:linattn|block_norm)_[a-z_]+)\s*\(", text)
    assert len(set(names)) == 8
    for name in names:
        assert callable(getattr(qd, name)), name


def test_binding_refuses_host_tensors_and_wrong_names():
    import torch
    import recurrent_sequence_layers_amd as qd
    x = torch.zeros(1, 2, 1, 64)
    with pytest.raises(qd.QDeltaError, match="device tensor"):
        qd.qdelta_linattn_fwd(x, x, x)
    with pytest.raises(qd.QDeltaError, match="device tensor"):
        qd.qdelta_linattn_step(x[0], x[0], x[0], None, torch.zeros(2, 1, 64, 64))
    with pytest.raises(qd.QDeltaError, match="device tensor"):
        qd.qdelta_linattn_bwd(x, x, x, None, None, x)
    with pytest.raises(qd.QDeltaError, match="device tensor"):
        qd.qdelta_block_norm_fwd(x)
    with pytest.raises(qd.QDeltaError, match="device tensor"):
        qd.qdelta_block_norm_bwd(x, x, None, None, None, None, None, x)


def test_sizes_past_32_bits_are_refused_by_the_binding():
    import recurrent_sequence_layers_amd as qd
    for T in (1 << 31, (1 << 32) + 16):
        for query, sizes in ((qd.qdelta_linattn_fwd_workspace_bytes, (1, T, 1, 64, 64)),
                             (qd.qdelta_linattn_bwd_workspace_bytes, (1, T, 1, 64, 64, True)),
                             (qd.qdelta_block_norm_bwd_workspace_bytes, (T, 64, True))):
            with pytest.raises(qd.QDeltaError, match="2\\*\\*31"):
                query(*sizes, qd.QD_BF16)
