"""Edges of the tied head's losses: waits that run out, and inputs at the ends of the range the entry
points allow. Bounds are derived where they are used; u = 2^-23 is one unit of a float32 sum."""
import math
import time

import pytest
import torch

from test_gpu_head_loss import (BF16, DEV, F32, check_distill, check_norm, check_xent, gen, h, mmf,  # noqa: F401
                                operands, teacher)

pytestmark = pytest.mark.gpu
U = 2.0 ** -23


# The cap is looked at every 16 tries, and a try may sleep for a time the hardware chooses (some microseconds
# here): a wait of tens of microseconds may run out at a cap of one or not, one of a millisecond does. The last
# case's dx tiles sum over 131072 words at once, 80 tiles on 74 pairs that stream 5.4 GB: 0.8 ms at least.
@pytest.mark.parametrize("m,d,v,surely", [(2000, 2048, 32000, False), (60, 4096, 65536, False),
                                          (100, 20480, 131072, True)])
def test_waits_that_run_out_end_in_order(mmf, m, d, v, surely):  # noqa: F811
    x, t, g = operands(71, m, d, v, BF16, BF16)
    targets = torch.randint(0, v, (m,), generator=g, device=DEV).to(torch.int32)
    dloss = torch.randn(m, generator=g, device=DEV)
    loss, lse = mmf.lm_head_xent_fwd(x, t, targets)
    want = mmf.lm_head_xent_backward(x, t, targets, lse, dloss)
    assert mmf.sync_status(DEV) == mmf.MMF_OK
    for _ in range(5):
        mmf.set_wait_limit(1)
        start = time.monotonic()
        try:
            mmf.lm_head_xent_fwd(x, t, targets)
            mmf.lm_head_xent_backward(x, t, targets, lse, dloss)
            status = mmf.sync_status(DEV)
        finally:
            mmf.set_wait_limit(0)
        # ended by copies that landed, not by the 1 s cap of a barrier that nothing completes
        assert time.monotonic() - start < 0.9
        assert status == mmf.MMF_ERR_TIMEOUT or (not surely and status == mmf.MMF_OK)
        again = mmf.lm_head_xent_fwd(x, t, targets)
        got = mmf.lm_head_xent_backward(x, t, targets, again[1], dloss)
        assert torch.equal(again[0], loss) and torch.equal(again[1], lse)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert mmf.sync_status(DEV) == mmf.MMF_OK


def confident(m, d, v, gap, tau=1.0):
    """Rows whose target stands about `gap` above the other words, whose logits are near 17 tau:
    sums of d terms of one sign, which is where an accumulator that cuts bits off drifts. Column 0 of x is
    zero and of the table 8, so that it takes no part in the logits and dx[:, 0] = 8 sum_v g_rv."""
    g = gen(m + v)
    shared = torch.randn(d, generator=g, device=DEV)
    x = (0.7 * shared + 0.7 * torch.randn(m, d, generator=g, device=DEV)).to(BF16)
    x[:, 0] = 0
    targets = torch.randperm(v, generator=g, device=DEV)[:m].to(torch.int32)
    t = (17 * tau / 0.7 / d) * shared + (0.3 * tau / math.sqrt(d)) * torch.randn(v, d, generator=g, device=DEV)
    t[targets.long()] += gap * tau / 0.49 / d * (x.float() - 0.7 * shared)
    t = t.to(BF16)
    t[:, 0] = 8.0
    return x, t, targets, g


def row_errors(x, t, q, tau):
    """float64 p, and bounds on the kernels' relative error of p and absolute error near p = 1 per row: the
    same sums s enter lse and p, whose errors (16 steps of at most u of a piece's sum, added rounding to
    nearest: 32 u max |s| / tau with either sign) cancel in the row's total but not between words; what is
    left on p itself is lse's last bit (half of 2^-23 of 2^floor(log2 |lse|) at most u |lse|), the sum's and
    exponentials' 16 u, and the product with 1 / tau, u |s| / tau."""
    s = x.double() @ t.double().T / tau
    lse = torch.logsumexp(s, 1)
    p = torch.exp(s - lse[:, None])
    words = 64 * U * s.abs().max(1).values
    level = U * (16 + 2 * lse.abs())
    if tau != 1.0:
        level = level + 2 * U * s.abs().max(1).values
    return p, p - q, words, level


@pytest.mark.parametrize("m", [100, 200, 700])
@pytest.mark.parametrize("gap", [13.0, 14.5])
def test_xent_gradient_of_confident_rows(mmf, m, gap):  # noqa: F811
    d, v = 2560, 1000
    x, t, targets, g = confident(m, d, v, gap)
    dloss = 1 + torch.rand(m, generator=g, device=DEV)
    q = torch.zeros(m, v, dtype=torch.float64, device=DEV).scatter_(1, targets.long()[:, None], 1.0)
    p, gv, words, level = row_errors(x, t, q, 1.0)
    assert ((p * q).sum(1) > 0.98).all() and ((p * q).sum(1) < 0.99999).all()
    _, lse = mmf.lm_head_xent_fwd(x, t, targets)
    dx, _ = mmf.lm_head_xent_backward(x, t, targets, lse, dloss)
    c = dloss.double()[:, None]
    T = t.double()
    want = c * (gv @ T)
    # row by row in the 2-norm: g's and dx's roundings to bf16, the words' errors on the off-target part and
    # the level's on all of p; products of V / 16 steps
    size = c * (gv.abs() @ T.norm(dim=1)[:, None])
    tol = (2 * h(BF16) + 3 * words[:, None] + (v / 16 + 64) * U) * size + level[:, None] * c * (p @ T.norm(dim=1)[:, None])
    off = (dx.double() - want).norm(dim=1, keepdim=True)
    assert (off <= tol).all(), float((off / tol).max())
    check_zero_sum(dx, c, p, gv, words, level, m)
    assert mmf.sync_status(DEV) == mmf.MMF_OK


def check_zero_sum(dx, c, p, gv, words, level, m):
    """dx[:, 0] = 8 sum_v g_rv = 0: what is left is each g's rounding (up to 128 rows two bf16 values,
    2^-16 of it, else one, 2^-8), the level's error of p, and 3 V / 16 steps of u of the products' sums."""
    v = p.shape[1]
    planes = 2.0 ** -16 if m <= 128 else 2.0 ** -8
    tol = 8 * c[:, 0] * ((planes + 3 * (v / 16 + 8) * U + 2.0 ** -16) * gv.abs().sum(1) + level * p.sum(1)
                         + words * (1 - p.max(1).values))
    off = dx[:, 0].double().abs()
    assert (off <= tol).all(), float((off / tol).max())
    return tol


def check_one_value_misses(c, gv, tol):
    """The same sums with every g rounded to one bf16 value, in float64: most rows are out of the bound."""
    once = 8 * (c * gv).to(BF16).double().sum(1).abs()
    assert (once > tol).double().mean() > 0.8, float((once / tol).median())


@pytest.mark.parametrize("m", [1, 100, 128, 129])
@pytest.mark.parametrize("tau", [1.0, 2.0])
def test_gradient_rows_sum_to_zero(mmf, m, tau):  # noqa: F811
    """Ordinary rows: g is of order one at the targets and the teacher's entries, whose roundings lead. Up to
    128 rows they are held in two bf16 values, which one value would miss by two orders."""
    d, v, k = 256, 1000, 6
    x, t, g = operands(81 + m, m, d, v, BF16, BF16)
    x[:, 0], t[:, 0] = 0, 8.0
    c = 1 + torch.rand(m, generator=g, device=DEV)
    if tau == 1.0:
        targets = torch.randint(0, v, (m,), generator=g, device=DEV).to(torch.int32)
        q = torch.zeros(m, v, dtype=torch.float64, device=DEV).scatter_(1, targets.long()[:, None], 1.0)
        p, gv, words, level = row_errors(x, t, q, 1.0)
        _, lse = mmf.lm_head_xent_fwd(x, t, targets)
        dx, _ = mmf.lm_head_xent_backward(x, t, targets, lse, c)
        tol = check_zero_sum(dx, c.double()[:, None], p, gv, words, level, m)
        if 1 < m <= 128:
            check_one_value_misses(c.double()[:, None], gv, tol)
    ids = torch.stack([torch.randperm(v, generator=g, device=DEV)[:k] for _ in range(m)]).to(torch.int32)
    logits = 2 * torch.randn(m, k, generator=g, device=DEV)
    w = torch.softmax(logits.double() / tau, 1)
    q = torch.zeros(m, v, dtype=torch.float64, device=DEV).scatter_(1, ids.long(), w)
    p, gv, words, level = row_errors(x, t, q, tau)
    _, lse, s_top = mmf.lm_head_distill_fwd(x, t, ids, logits, temperature=tau)
    dx, _ = mmf.lm_head_distill_backward(x, t, ids, logits, lse, s_top, c, temperature=tau)
    tol = check_zero_sum(dx, c.double()[:, None] / tau, p, gv, words, level + 64 * U, m)
    if 1 < m <= 128:
        check_one_value_misses(c.double()[:, None] / tau, gv, tol)
    assert mmf.sync_status(DEV) == mmf.MMF_OK


@pytest.mark.parametrize("m", [90, 900])
@pytest.mark.parametrize("up", [1e34, 1e36, 1e-34, 1e-36])
def test_float32_ends_of_the_range(mmf, m, up):  # noqa: F811
    """Rows of 1e-36 beside a table of 1e36 and the other way round, logits of order one to ten."""
    x, t, g = operands(91, m, 128, 600, F32, F32)
    x[3] *= 1e-2
    targets = torch.randint(0, 600, (m,), generator=g, device=DEV).to(torch.int32)
    assert float((x @ t.T).abs().max()) > 4
    check_xent(mmf, x * up, t / up, targets, torch.randn(m, generator=g, device=DEV))
    ids, logits, dloss = teacher(92, m, 7, 600, F32)
    check_distill(mmf, x * up, t / up, ids, logits, 2.0, dloss)


@pytest.mark.parametrize("m", [90, 900])
def test_float32_far_magnitudes_of_table_and_dloss(mmf, m):  # noqa: F811
    """dloss takes back what the table is away from one: dx of order one from a table of 1e-36 and dloss of
    1e30, and of 1e36 and 1e-30; c x is what has to stay in range for dtable."""
    x, t, g = operands(93, m, 128, 600, F32, F32)
    targets = torch.randint(0, 600, (m,), generator=g, device=DEV).to(torch.int32)
    dloss = torch.randn(m, generator=g, device=DEV)
    check_xent(mmf, x, t * 1e-36, targets, dloss * 1e30)
    check_xent(mmf, x * 1e-36, t * 1e36, targets, dloss * 1e-30, (True, False))
    # |x| |dloss| is past the range, its share at temperature 1000 is not
    ids, logits, dloss = teacher(94, m, 7, 600, F32)
    check_distill(mmf, x * 1e20, t * 1e-20, ids, logits, 1000.0, (1 + dloss.abs()) * 1e18)


def test_float32_zero_products_of_far_operands(mmf):  # noqa: F811
    """Rows and words of 1e30 that share no column: every logit is zero, as in float32."""
    m, d, v = 40, 64, 300
    x, t, g = operands(95, m, d, v, F32, F32)
    x, t = x * 1e30, t * 1e30
    x[:, 32:], t[:, :32] = 0, 0
    targets = torch.randint(0, v, (m,), generator=g, device=DEV).to(torch.int32)
    check_xent(mmf, x, t, targets, torch.rand(m, generator=g, device=DEV))


def test_few_rows_several_vocabulary_pieces(mmf):  # noqa: F811
    """dx of few rows, which takes the rows as its columns, over two pieces of the vocabulary."""
    m, d, v = 100, 64, 600000
    assert 256 * v * 2 * 2 > 512 << 20
    x, t, g = operands(96, m, d, v, BF16, BF16)
    targets = torch.randint(0, v, (m,), generator=g, device=DEV).to(torch.int32)
    check_xent(mmf, x, t, targets, torch.randn(m, generator=g, device=DEV))


@pytest.mark.parametrize("xt", [F32, BF16])
@pytest.mark.parametrize("d", [1024, 1025, 2817, 9216])
@pytest.mark.parametrize("size,eps", [(1e15, 1e-8), (1e14, 0.0), (1e-15, 0.0), (1e-13, 0.0), (1e-3, 1e-8)])
def test_norm_of_rows_far_from_one(mmf, d, size, eps, xt):  # noqa: F811
    """dy leans towards x, so that the part that the projection takes out is a good share of it; rho^3 alone
    would leave float32's range."""
    g = gen(d)
    n = torch.randn(37, d, generator=g, device=DEV)
    dy = (n + torch.randn(37, d, generator=g, device=DEV)).to(xt)
    check_norm(mmf, (size * n).to(xt), 1 + 0.2 * torch.randn(d, generator=g, device=DEV), dy, eps)


def test_norm_of_few_very_wide_rows(mmf):  # noqa: F811
    """Three rows of five million columns: a thread adds 19532 squares in float32 (half an ulp each at most),
    the block's tree a few more."""
    m, d = 3, 5_000_011
    g = gen(97)
    x, dy = (torch.randn(m, d, generator=g, device=DEV) for _ in range(2))
    w = torch.rand(d, generator=g, device=DEV)
    X, G, W = x.double(), dy.double(), w.double()
    rel = (d / 256 / 2 + 32) * U
    rho = (X.square().mean(1, keepdim=True) + 1e-8) ** -0.5
    y = mmf.rmsnorm_fwd(x, w)
    assert ((y - X * rho * W).abs() <= rel * (X * rho * W).abs() + 1e-37).all()
    torch.cuda.reset_peak_memory_stats()
    start = torch.cuda.memory_allocated()
    dx, dw = mmf.rmsnorm_backward(x, w, dy)
    assert torch.cuda.max_memory_allocated() - start < 10 * m * d * 4
    u = G * W
    mean = (u * X).mean(1, keepdim=True)
    want = rho * u - rho ** 3 * X * mean
    mag = rho * u.abs() + rho ** 3 * X.abs() * (u * X).abs().mean(1, keepdim=True)
    assert ((dx - want).abs() <= 4 * rel * mag).all()
    terms = G * X * rho
    assert ((dw - terms.sum(0)).abs() <= (rel + 8 * U) * terms.abs().sum(0)).all()


def test_offsets_past_32_bits_in_the_table_and_dtable(mmf):  # noqa: F811
    """2.2 M words of 1024: the last words' elements of the table and of dtable lie past 2^31. The call's
    rows have their targets among them, and dtable's last rows are those of a call on the last words alone
    with the same lse (the same tiles' arithmetic)."""
    m, d, v, tail = 200, 1024, 2_200_064, 512
    assert (v - tail) * d > 2 ** 31
    g = gen(98)
    t = torch.empty(v, d, dtype=BF16, device=DEV)
    for r in range(0, v, 1 << 19):
        t[r:r + (1 << 19)] = (torch.randn(min(1 << 19, v - r), d, generator=g, device=DEV) / 32).to(BF16)
    x = torch.randn(m, d, generator=g, device=DEV).to(BF16)
    targets = (v - tail + torch.randint(0, tail, (m,), generator=g, device=DEV)).to(torch.int32)
    loss, lse = mmf.lm_head_xent_fwd(x, t, targets)
    total = torch.zeros(m, dtype=torch.float64, device=DEV)
    for r in range(0, v, 1 << 19):
        total += torch.exp(x.float() @ t[r:r + (1 << 19)].float().T).double().sum(1)   # logits of order one
    last = slice(v - tail, v)
    s_t = (x.double() * t[targets.long()].double()).sum(1)
    assert ((lse - total.log()).abs() <= 1e-4).all()      # the float32 logits' own 1e-5, and v terms in 64 bits
    assert ((loss - (total.log() - s_t)).abs() <= 1e-4).all()
    c = torch.rand(m, generator=g, device=DEV)
    _, dt = mmf.lm_head_xent_backward(x, t, targets, lse, c, want_dx=False)
    small = t[last].contiguous()
    _, dt_tail = mmf.lm_head_xent_backward(x, small, (targets - (v - tail)).to(torch.int32), lse, c, want_dx=False)
    assert dt_tail.any() and torch.equal(dt[last], dt_tail)
    assert mmf.sync_status(DEV) == mmf.MMF_OK


@pytest.mark.parametrize("xt,tt", [(BF16, BF16), (F32, F32)])
def test_offsets_past_32_bits_in_the_rows_with_dtable(mmf, xt, tt):  # noqa: F811
    """2.2 M rows of 1024, all but the first and the last hundred left out: dtable and dx of the few live rows,
    whose elements lie at both ends, are those of a call that has only them."""
    m, d, v, n = 2_200_000, 1024, 300, 100
    x, t, g = operands(99, 2 * n, d, v, xt, tt)
    big = torch.zeros(m, d, dtype=xt, device=DEV)
    big[:n], big[-n:] = x[:n], x[n:]
    targets = torch.randint(0, v, (2 * n,), generator=g, device=DEV).to(torch.int32)
    all_targets = torch.full((m,), -1, dtype=torch.int32, device=DEV)
    all_targets[:n], all_targets[-n:] = targets[:n], targets[n:]
    c = torch.rand(2 * n, generator=g, device=DEV)
    all_c = torch.full((m,), float("nan"), device=DEV)
    all_c[:n], all_c[-n:] = c[:n], c[n:]
    loss, lse = mmf.lm_head_xent_fwd(big, t, all_targets)
    ends = torch.cat([torch.arange(n, device=DEV), torch.arange(m - n, m, device=DEV)])
    want_loss, want_lse = mmf.lm_head_xent_fwd(x, t, targets)
    assert torch.equal(loss[ends], want_loss) and torch.equal(lse[ends], want_lse)
    dx, dt = mmf.lm_head_xent_backward(big, t, all_targets, lse, all_c)
    want_dx, want_dt = mmf.lm_head_xent_backward(x, t, targets, want_lse, c)
    # the small call splits its sums over k differently: float32 partials added in another order
    steps = 64 * U + (2 * h(xt) if xt == BF16 else 0)
    assert ((dx[ends].double() - want_dx.double()).norm() <= steps * want_dx.double().norm())
    assert not dx[n:-n].any()
    assert ((dt.double() - want_dt.double()).norm() <= steps * want_dt.double().norm())
    assert mmf.sync_status(DEV) == mmf.MMF_OK
