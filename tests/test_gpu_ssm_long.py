"""Long walks of the selective scan, forward and gradients, each plan of the time axis on its own:
uncut where the card is full, and segments of many tiles.  Against 64 bits, within bounds that
follow the errors from token to token."""
import pytest
import torch

from mixer_cases import DT, dev, ssm_inputs
from scan_errors import near, scan

pytestmark = pytest.mark.gpu

FWD = ("u", "dt", "A", "Bm", "Cm", "D", "z", "dt_bias", "S0")
# dtype, B, T, D, G, N, tokens a segment forward and backward (0: uncut), lens.  A workgroup is 64 channels
# of a group and a sequence; the gradients are uncut from one workgroup a compute unit (256) on.
CASES = [("bf16", 8, 520, 2048, 1, 16, 0, 0, False), ("bf16", 8, 555, 2048, 1, 16, 0, 0, True),       # 256 workgroups
         ("f32", 9, 545, 1860, 1, 16, 0, 0, False), ("f32", 9, 261, 1857, 1, 32, 0, 0, False),       # 270
         ("bf16", 4, 275, 4130, 2, 64, 0, 0, True), ("bf16", 8, 530, 4104, 1, 16, 0, 0, False),      # 264, 520
         ("f32", 12, 517, 2560, 1, 16, 0, 0, True), ("bf16", 16, 130, 2048, 1, 16, 0, 0, False),     # 480, 512
         ("bf16", 2, 1060, 2048, 1, 32, 144, 272, False), ("f32", 2, 1060, 2046, 1, 32, 144, 272, True),
         ("f32", 3, 900, 1500, 1, 64, 240, 240, False), ("bf16", 1, 2100, 2048, 1, 16, 144, 272, False),
         ("f32", 1, 2100, 2047, 1, 16, 144, 272, True)]


def segments(T, cut):
    return -(-T // cut) if cut else 1


def workspaces(B, T, D, G, N, P_fwd, P_bwd):
    """Bytes of the two workspaces with so many segments."""
    up4 = lambda n: (n + 3) // 4 * 4  # noqa: E731
    rows = 2 * B * G * N * ((T + 15) // 16 * 16 + 16)
    fwd = rows + (B * P_fwd * D * (N + 1) if P_fwd > 1 else 0)
    bwd = rows + (2 * (up4(B * P_bwd * N * D) + up4(B * P_bwd * D)) if P_bwd > 1 else 0)
    bwd += up4(B * -(-T // 8) * N * D) + up4(-(-(D // G) // 64) * B * T * G * 2 * N) + up4(B * P_bwd * D * N) + up4(B * P_bwd * 2 * D)
    return 4 * fwd, 4 * bwd


@pytest.mark.parametrize("case", CASES)
def test_long_walks(qd, case):
    dtype, B, T, D, G, N, cut_fwd, cut_bwd, padded = case
    need = workspaces(B, T, D, G, N, segments(T, cut_fwd), segments(T, cut_bwd))
    assert need == (qd.qdelta_ssm_fwd_workspace_bytes(B, T, D, G, N, DT[dtype]),
                    qd.qdelta_ssm_bwd_workspace_bytes(B, T, D, G, N, DT[dtype])), "another plan than this case is for"
    x = {k: dev(v) for k, v in ssm_inputs(B, T, D, G, N, dtype, T + D).items()}
    lens = (torch.arange(B, device="cuda", dtype=torch.int32) * T // max(B - 1, 1)).flip(0) if padded else None
    if padded and B == 1:
        lens = torch.tensor([T - 300], dtype=torch.int32, device="cuda")
    val, err = scan(x, lens=lens, cut_fwd=cut_fwd, cut_bwd=cut_bwd)
    if padded:                        # what padding holds is not read
        past = torch.arange(T, device="cuda")[None] >= lens[:, None]
        for k in ("u", "dt", "z", "Bm", "Cm", "d_o"):
            x[k][past] = float("nan")
    o, S = qd.qdelta_ssm_fwd(*[x[k] for k in FWD], lens=lens)
    near(o, val["o"], err["o"], "o")
    near(S, val["S_T"], err["S_T"], "S_T")
    got = qd.qdelta_ssm_bwd(*[x[k] for k in FWD], x["d_o"], x["dS_T"], lens=lens)
    for k, v in got.items():
        near(v, val[k], err[k], k)
