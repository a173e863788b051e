"""The training end of the tied head on the CPU: what the C entry points and the binding refuse
before anything reaches a GPU, the workspace sizes, and the binding's marshalling against the C
signatures (a recorder stands in for the library, host tensors for device tensors)."""
import pytest
import torch

import ternary_weight_matmul_b200 as mmf
from ternary_weight_matmul_b200 import build as mbuild
from test_binding_cpu import fake  # noqa: F401  (fixture)

INVALID, WORKSPACE, OK = mmf.MMF_ERR_INVALID_ARG, mmf.MMF_ERR_WORKSPACE, mmf.MMF_OK
F32, BF16 = mmf.MMF_F32, mmf.MMF_BF16
BIG = 1 << 40


@pytest.fixture(scope="module")
def L():
    mbuild.build()
    return mmf.lib()


def test_rmsnorm_arguments_on_host(L):
    # mmf_rmsnorm_fwd(x, x_dtype, m, d, norm_w, eps, y, y_dtype, stream)
    f = L.mmf_rmsnorm_fwd
    assert f(16, F32, -1, 8, None, 1e-8, 16, F32, None) == INVALID
    assert f(16, F32, 4, 0, None, 1e-8, 16, F32, None) == INVALID
    assert f(16, 7, 4, 8, None, 1e-8, 16, F32, None) == INVALID
    assert f(16, F32, 4, 8, None, 1e-8, 16, 3, None) == INVALID
    assert f(16, F32, 4, 8, None, -1.0, 16, F32, None) == INVALID
    assert f(16, F32, 4, 8, None, float("nan"), 16, F32, None) == INVALID
    assert f(None, F32, 4, 8, None, 1e-8, 16, F32, None) == INVALID
    assert f(16, F32, 4, 8, None, 1e-8, None, F32, None) == INVALID
    assert f(None, F32, 0, 8, None, 1e-8, None, F32, None) == OK
    # mmf_rmsnorm_backward(x, x_dtype, m, d, norm_w, eps, dy, dy_dtype, dx, dnorm_w, ws, ws_bytes, stream)
    b = L.mmf_rmsnorm_backward
    need = L.mmf_workspace_bytes(mmf.MMF_OP_RMSNORM_BWD, 4, 8, 0, 0)
    assert need >= 8 * 4
    assert b(16, F32, 4, 8, None, 1e-8, None, F32, 16, None, None, 0, None) == INVALID
    assert b(16, F32, 4, 8, None, 1e-8, 16, F32, None, None, None, 0, None) == INVALID
    assert b(16, F32, 4, 8, None, 1e-8, 16, 9, 16, None, None, 0, None) == INVALID
    assert b(16, F32, 4, 8, None, -1e-8, 16, F32, 16, None, None, 0, None) == INVALID
    assert b(16, F32, 4, 8, None, 1e-8, 16, F32, 16, 16, None, 0, None) == WORKSPACE
    assert b(16, F32, 4, 8, None, 1e-8, 16, F32, 16, 16, 256, need - 1, None) == WORKSPACE
    assert b(16, F32, 4, 8, None, 1e-8, 16, F32, 16, 16, 272, need, None) == WORKSPACE  # misaligned
    assert b(None, F32, 0, 8, None, 1e-8, None, F32, None, None, None, 0, None) == OK


SIZES = [(-1, 64, 100), ((1 << 30) + 1, 64, 100), (4, 0, 100), (4, 12, 100), (4, 32776, 100), (4, 64, 0), (4, 64, -5),
         (4, 64, (1 << 30) + 1)]


def test_xent_arguments_on_host(L):
    # mmf_lm_head_xent_fwd(x, x_dtype, m, d, table, table_dtype, vocab, targets, loss, lse, ws, ws_bytes, stream)
    f = L.mmf_lm_head_xent_fwd
    # mmf_lm_head_xent_backward(x, x_dtype, m, d, table, table_dtype, vocab, targets, lse, dloss, dx, dtable,
    #                           ws, ws_bytes, stream)
    b = L.mmf_lm_head_xent_backward
    for m, d, v in SIZES:
        assert f(16, BF16, m, d, 16, BF16, v, 16, 16, 16, 256, BIG, None) == INVALID, (m, d, v)
        assert b(16, BF16, m, d, 16, BF16, v, 16, 16, 16, 16, 16, 256, BIG, None) == INVALID, (m, d, v)
    assert b"head xent" in L.mmf_last_error()
    good = [16, BF16, 4, 64, 16, BF16, 100, 16, 16, 16, 256, BIG, None]
    for i in (0, 4, 7, 8, 9):
        assert f(*[None if j == i else a for j, a in enumerate(good)]) == INVALID, i
    for i, bad in ((0, 24), (4, 20), (1, 2), (5, 5)):
        assert f(*[bad if j == i else a for j, a in enumerate(good)]) == INVALID, i
    need = L.mmf_workspace_bytes(mmf.MMF_OP_HEAD_LOSS, 4, 64, 100, 0)
    assert f(*good[:10], 256, need - 1, None) == WORKSPACE
    assert f(*good[:10], 264, need, None) == WORKSPACE
    assert f(None, BF16, 0, 64, None, BF16, 100, None, None, None, None, 0, None) == OK
    good = [16, BF16, 4, 64, 16, BF16, 100, 16, 16, 16, 16, 16, 256, BIG, None]
    for i in (0, 4, 7, 8, 9):
        assert b(*[None if j == i else a for j, a in enumerate(good)]) == INVALID, i
    for i, bad in ((0, 24), (4, 20), (10, 8), (11, 40), (1, 2), (5, 5)):
        assert b(*[bad if j == i else a for j, a in enumerate(good)]) == INVALID, i
    need = L.mmf_workspace_bytes(mmf.MMF_OP_HEAD_LOSS_BWD, 4, 64, 100, 0)
    assert b(*good[:12], 256, need - 1, None) == WORKSPACE
    # nothing asked for, and no rows without a table gradient: nothing to do
    assert b(16, BF16, 4, 64, 16, BF16, 100, 16, 16, 16, None, None, None, 0, None) == OK
    assert b(None, BF16, 0, 64, None, BF16, 100, None, None, None, None, None, None, 0, None) == OK


def test_distill_arguments_on_host(L):
    # mmf_lm_head_distill_fwd(x, x_dtype, m, d, table, table_dtype, vocab, t_ids, t_logits, t_dtype, top_k,
    #                         temperature, loss, lse, s_top, ws, ws_bytes, stream)
    f = L.mmf_lm_head_distill_fwd
    good = [16, BF16, 4, 64, 16, BF16, 100, 16, 16, F32, 8, 1.0, 16, 16, 16, 256, BIG, None]
    for m, d, v in SIZES:
        assert f(16, BF16, m, d, 16, BF16, v, *good[7:]) == INVALID, (m, d, v)
    for i in (0, 4, 7, 8, 12, 13, 14):
        assert f(*[None if j == i else a for j, a in enumerate(good)]) == INVALID, i
    for i, bad in ((0, 24), (4, 20), (9, 4), (10, 0), (10, 257), (11, 0.0), (11, -1.0), (11, 1e-4), (11, 1e4),
                   (11, float("nan")), (11, float("inf"))):
        assert f(*[bad if j == i else a for j, a in enumerate(good)]) == INVALID, (i, bad)
    assert b"distill" in L.mmf_last_error()
    need = L.mmf_workspace_bytes(mmf.MMF_OP_HEAD_LOSS, 4, 64, 100, 4 * 8)
    assert f(*good[:15], 256, need - 1, None) == WORKSPACE
    # mmf_lm_head_distill_backward(x, x_dtype, m, d, table, table_dtype, vocab, t_ids, t_logits, t_dtype, top_k,
    #                              temperature, lse, s_top, dloss, dx, dtable, ws, ws_bytes, stream)
    b = L.mmf_lm_head_distill_backward
    good = [16, BF16, 4, 64, 16, BF16, 100, 16, 16, F32, 8, 1.0, 16, 16, 16, 16, 16, 256, BIG, None]
    for i in (0, 4, 7, 8, 12, 13, 14):
        assert b(*[None if j == i else a for j, a in enumerate(good)]) == INVALID, i
    for i, bad in ((10, 0), (10, 257), (11, 0.0), (11, float("nan")), (15, 24), (16, 24)):
        assert b(*[bad if j == i else a for j, a in enumerate(good)]) == INVALID, (i, bad)
    need = L.mmf_workspace_bytes(mmf.MMF_OP_HEAD_LOSS_BWD, 4, 64, 100, 4 * 8)
    assert b(*good[:17], 256, need - 1, None) == WORKSPACE
    assert b(*good[:15], None, None, None, 0, None) == OK


def test_workspace_stays_far_below_the_logits(L):
    ws = L.mmf_workspace_bytes
    m, d, v = 16384, 1024, 32000
    fwd, bwd = ws(mmf.MMF_OP_HEAD_LOSS, m, d, v, 0), ws(mmf.MMF_OP_HEAD_LOSS_BWD, m, d, v, 0)
    assert fwd < m * v * 4 // 20                      # the gathered rows and one pair per tile and row
    assert bwd < (1 << 30) and bwd < m * v * 4 // 2   # a piece of g, and dx's float32 partials
    for bits in (1, 2, 3):
        assert ws(mmf.MMF_OP_HEAD_LOSS, m, d, v, bits) > fwd
        assert ws(mmf.MMF_OP_HEAD_LOSS_BWD, m, d, v, bits) > bwd
    assert ws(mmf.MMF_OP_HEAD_LOSS, m, 0, v, 0) == 0 and ws(mmf.MMF_OP_HEAD_LOSS_BWD, m, d, 0, 0) == 0


def _ws_ok(ptr, nbytes, op, *sizes):
    assert ptr is not None and nbytes >= mmf.workspace_bytes(op, *sizes)


def test_norm_marshalling(fake):  # noqa: F811
    x = torch.randn(2, 3, 16, dtype=torch.bfloat16)
    w = torch.ones(16)
    y = mmf.rmsnorm_fwd(x, w, eps=1e-6, y_dtype=torch.float32)
    a = fake.last("mmf_rmsnorm_fwd")
    assert a[:5] == (x.data_ptr(), BF16, 6, 16, w.data_ptr()) and a[5] == 1e-6
    assert a[6] == y.data_ptr() and a[7] == F32 and y.shape == x.shape and y.dtype == torch.float32
    dy = torch.randn(2, 3, 16)
    dx, dw = mmf.rmsnorm_backward(x, None, dy)
    a = fake.last("mmf_rmsnorm_backward")
    assert a[:5] == (x.data_ptr(), BF16, 6, 16, None) and a[5] == 1e-8
    assert a[6:10] == (dy.data_ptr(), F32, dx.data_ptr(), dw.data_ptr())
    assert dx.dtype == torch.bfloat16 and dx.shape == x.shape and tuple(dw.shape) == (16,) and dw.dtype == torch.float32
    _ws_ok(a[10], a[11], mmf.MMF_OP_RMSNORM_BWD, 6, 16, 0, 0)
    assert mmf.rmsnorm_backward(x, None, dy, want_dnorm_w=False)[1] is None
    assert fake.last("mmf_rmsnorm_backward")[9] is None


def test_loss_marshalling(fake):  # noqa: F811
    m, d, v, k = 5, 16, 40, 3
    x, t = torch.randn(m, d), torch.randn(v, d, dtype=torch.bfloat16)
    tg = torch.zeros(m, dtype=torch.int32)
    loss, lse = mmf.lm_head_xent_fwd(x, t, tg)
    a = fake.last("mmf_lm_head_xent_fwd")
    assert a[:7] == (x.data_ptr(), F32, m, d, t.data_ptr(), BF16, v)
    assert a[7:10] == (tg.data_ptr(), loss.data_ptr(), lse.data_ptr())
    _ws_ok(a[10], a[11], mmf.MMF_OP_HEAD_LOSS, m, d, v, 1)
    dl = torch.ones(m)
    dx, dt = mmf.lm_head_xent_backward(x, t, tg, lse, dl)
    a = fake.last("mmf_lm_head_xent_backward")
    assert a[:7] == (x.data_ptr(), F32, m, d, t.data_ptr(), BF16, v)
    assert a[7:12] == (tg.data_ptr(), lse.data_ptr(), dl.data_ptr(), dx.data_ptr(), dt.data_ptr())
    assert dx.dtype == torch.float32 and dt.dtype == torch.bfloat16 and dt.shape == t.shape and dx.shape == x.shape
    _ws_ok(a[12], a[13], mmf.MMF_OP_HEAD_LOSS_BWD, m, d, v, 1)
    dx, dt = mmf.lm_head_xent_backward(x, t, tg, lse, dl, want_dx=False)
    assert dx is None and fake.last("mmf_lm_head_xent_backward")[10] is None
    dx, dt = mmf.lm_head_xent_backward(x, t, tg, lse, dl, want_dtable=False)
    assert dt is None and fake.last("mmf_lm_head_xent_backward")[11] is None

    ids, tl = torch.zeros(m, k, dtype=torch.int32), torch.randn(m, k)
    loss, lse, s = mmf.lm_head_distill_fwd(x, t, ids, tl, temperature=2.0)
    a = fake.last("mmf_lm_head_distill_fwd")
    assert a[:7] == (x.data_ptr(), F32, m, d, t.data_ptr(), BF16, v)
    assert a[7:12] == (ids.data_ptr(), tl.data_ptr(), F32, k, 2.0)
    assert a[12:15] == (loss.data_ptr(), lse.data_ptr(), s.data_ptr()) and tuple(s.shape) == (m, k)
    _ws_ok(a[15], a[16], mmf.MMF_OP_HEAD_LOSS, m, d, v, 1 + 4 * k)
    dx, dt = mmf.lm_head_distill_backward(x, t, ids, tl, lse, s, dl, temperature=2.0)
    a = fake.last("mmf_lm_head_distill_backward")
    assert a[7:12] == (ids.data_ptr(), tl.data_ptr(), F32, k, 2.0)
    assert a[12:17] == (lse.data_ptr(), s.data_ptr(), dl.data_ptr(), dx.data_ptr(), dt.data_ptr())
    _ws_ok(a[17], a[18], mmf.MMF_OP_HEAD_LOSS_BWD, m, d, v, 1 + 4 * k)


def test_wrappers_refuse_mismatched_arguments(fake):  # noqa: F811
    x, t = torch.randn(4, 16), torch.randn(30, 16)
    tg, dl = torch.zeros(4, dtype=torch.int32), torch.ones(4)
    ids, tl, s = torch.zeros(4, 3, dtype=torch.int32), torch.randn(4, 3), torch.zeros(4, 3)
    for match, call in [
        ("norm_w", lambda: mmf.rmsnorm_fwd(x, torch.ones(15))),
        ("norm_w", lambda: mmf.rmsnorm_fwd(x, torch.ones(16, dtype=torch.bfloat16))),
        ("contiguous", lambda: mmf.rmsnorm_fwd(x.T, None)),
        ("one shape", lambda: mmf.rmsnorm_backward(x, None, torch.randn(4, 15))),
        ("x: expected", lambda: mmf.rmsnorm_fwd(torch.randn(4, 0), None)),
        ("x: expected", lambda: mmf.lm_head_xent_fwd(torch.randn(2, 2, 16), t, tg)),
        ("table", lambda: mmf.lm_head_xent_fwd(x, torch.randn(30, 15), tg)),
        ("contiguous", lambda: mmf.lm_head_xent_fwd(x, torch.randn(16, 30).T, tg)),
        ("int32", lambda: mmf.lm_head_xent_fwd(x, t, tg.long())),
        ("targets", lambda: mmf.lm_head_xent_fwd(x, t, tg[:3])),
        ("lse", lambda: mmf.lm_head_xent_backward(x, t, tg, dl[:3], dl)),
        ("dloss", lambda: mmf.lm_head_xent_backward(x, t, tg, dl, dl.double())),
        ("int32", lambda: mmf.lm_head_distill_fwd(x, t, ids.long(), tl)),
        ("one shape", lambda: mmf.lm_head_distill_fwd(x, t, ids, torch.randn(4, 2))),
        ("one shape", lambda: mmf.lm_head_distill_fwd(x, t, ids[:3], tl[:3])),
        ("s_top", lambda: mmf.lm_head_distill_backward(x, t, ids, tl, dl, s[:, :2], dl)),
    ]:
        with pytest.raises(ValueError, match=match):
            call()
    with pytest.raises(TypeError, match="float16"):
        mmf.rmsnorm_fwd(x.half(), None)
    with pytest.raises(TypeError, match="float64"):
        mmf.lm_head_xent_fwd(x.double(), t.double(), tg)
    with pytest.raises(TypeError, match="float16"):
        mmf.lm_head_distill_fwd(x, t, ids, tl.half())
    meta = torch.zeros(4, dtype=torch.int32, device="meta")
    with pytest.raises(ValueError, match="targets: on meta"):
        mmf.lm_head_xent_fwd(x, t, meta)
    assert not [n for n, _ in fake.calls if n not in fake.REAL]


def test_wrappers_refuse_host_tensors():
    x, t = torch.randn(4, 16), torch.randn(30, 16)
    tg, dl = torch.zeros(4, dtype=torch.int32), torch.ones(4)
    ids, tl = torch.zeros(4, 3, dtype=torch.int32), torch.randn(4, 3)
    for call in (lambda: mmf.rmsnorm_fwd(x, None), lambda: mmf.rmsnorm_backward(x, None, x),
                 lambda: mmf.lm_head_xent_fwd(x, t, tg), lambda: mmf.lm_head_xent_backward(x, t, tg, dl, dl),
                 lambda: mmf.lm_head_distill_fwd(x, t, ids, tl)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
