"""The workspaces of the training end (CPU): what the head losses' backward holds is one piece of g, the rows and
one dx, the RMSNorm backward a row of partial sums per CTA and no more than it has rows."""
import pytest
import torch

import ternary_weight_matmul_b200 as mmf
from ternary_weight_matmul_b200 import build as mbuild
from test_binding_cpu import fake  # noqa: F401  (fixture)

GIB = 1 << 30


@pytest.fixture(scope="module")
def ws():
    mbuild.build()
    return mmf.lib().mmf_workspace_bytes


@pytest.mark.parametrize("m,d,v", [(16384, 1024, 32000), (16384, 2560, 32000), (65536, 2048, 32000),
                                   (65536, 2560, 32000), (131072, 2560, 32000), (16384, 4096, 128000),
                                   (65536, 2560, 256000)])
@pytest.mark.parametrize("bits", [0, 1, 2, 3])
def test_backward_holds_one_piece_of_g_and_one_dx(ws, m, d, v, bits):
    xf32, tf32 = bits & 1, bits >> 1
    planes = 2 if tf32 else 3 if xf32 else 1
    g = max(512 << 20, m * 4096 * 2 * planes)
    rows = m * d * 2 * ((2 if tf32 else 3) if xf32 else 1) + (m * d * 4 if tf32 else 0)
    table = v * d * 4 if tf32 else 0
    need = ws(mmf.MMF_OP_HEAD_LOSS_BWD, m, d, v, bits)
    assert need <= g + rows + table + 4 * m * d + 64 * m + (1 << 20)
    # a longer vocabulary needs its table's planes and nothing else
    more = ws(mmf.MMF_OP_HEAD_LOSS_BWD, m, d, 4 * v, bits) - need
    assert more <= 3 * table + m * 256 * 2 * planes * 64


def test_backward_stays_below_the_logits(ws):
    for m, d, v in [(16384, 2560, 32000), (65536, 2048, 32000), (65536, 2560, 32000), (131072, 2560, 32000)]:
        assert ws(mmf.MMF_OP_HEAD_LOSS_BWD, m, d, v, 0) < m * v * 2
    assert ws(mmf.MMF_OP_HEAD_LOSS_BWD, 65536, 2560, 32000, 0) < 2 * GIB


def test_norm_backward_holds_no_more_rows_than_it_has(ws, fake):  # noqa: F811
    op = mmf.MMF_OP_RMSNORM_BWD
    for d in (8, 512, 513, 16384, 1 << 24, 1 << 30):
        assert ws(op, 2, d, 0, 0) == (2 * d * 4 + 255) // 256 * 256
        assert ws(op, 1 << 20, d, 0, 0) == (2048 if d <= 512 else 1024) * d * 4
    # a call that asks for no dnorm_w takes no scratch for it
    x = torch.randn(64, 4096)
    mmf.rmsnorm_backward(x, None, x, want_dnorm_w=False)
    assert fake.last("mmf_rmsnorm_backward")[11] == 256
    mmf.rmsnorm_backward(x, None, x)
    assert fake.last("mmf_rmsnorm_backward")[11] == 64 * 4096 * 4


def test_norm_refuses_rows_past_its_index_range():
    L = mmf.lib()
    for d in ((1 << 30) + 1, (1 << 31) - 1):
        assert L.mmf_rmsnorm_fwd(16, 0, 1, d, None, 1e-8, 16, 0, None) == mmf.MMF_ERR_INVALID_ARG
        assert L.mmf_rmsnorm_backward(16, 0, 1, d, None, 1e-8, 16, 0, 16, None, None, 0,
                                      None) == mmf.MMF_ERR_INVALID_ARG
