"""The training end of the tied head (final RMSNorm, cross entropy and distillation over the
vocabulary, forward and backward) against plain float64 forms of the formulas.

Tolerances, elementwise, from the arithmetic (u = 2^-23 per float32 addition inside the tensor cores,
which may truncate; h(t) = finfo(t).eps / 2 per rounding to t):
  s     a sum of n = d products per plane pair (6 pairs for two float32 operands), terms bounded by
        |x| |T|:                                   e_s = 6 d u (|x| |T|^T)
  lse   a softmax average of the s errors, plus the sums and exponentials: max_v e_s + 64 u (1 + |lse|)
  g     c p with p = exp(s - lse): relative e_s + e_lse + 64 u on p, plus h(bf16) of |g| where g is held
        in bf16 (both operands bf16); the teacher's share q is a float32 softmax: 64 u
  dx    e_g |T| + (6 n + 64) u (|g| |T|), n = vocab terms, plus h(dtype) of |dx|; dtable likewise.
  What is below the smallest normal float32 counts as zero: 2^-126 on p, on g and on every product.
  With a float32 table the operands are pairs of fp16 values under a power of two that brings the
  largest of them to 2^14 at least: 2^-22 relative (three roundings or dropped terms a product, inside
  the n u above) and 2^-25 / 2^14 of the largest absolutely (the last fp16 step is 2^-24): of a row of
  x, of the table, of c x, and of 1 for g / c. A bf16 result takes the leading fp16 values alone: two
  roundings of 2^-11.
These worst cases grow with the number of terms; what the kernels do does not: an accumulator takes 16
steps (of at most u of its sum each) before the pieces are added rounding to nearest. So results are also
held to 16 u of their norm, and gradients, through p's relative error being s's absolute one, to
16 u (1 + max |s| / tau), plus h for each rounding to bf16 (g's and the output's). For a gradient the
norm is the two parts' of g = c p - c q, |(c p) T| + |(c q) T|: the error of p is relative to p, not to
p - q, which vanishes where the student agrees with its target (p = q = 1 at vocab = 1:
g = 0, while p = 1 +- u leaves an error of c u).
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = 2.0 ** -23
TINY = 2.0 ** -126
STEP16 = 2.0 ** -39
F32, BF16 = torch.float32, torch.bfloat16
ORDER6 = 6


@pytest.fixture(scope="module")
def mmf():
    import ternary_weight_matmul_b200 as m
    from ternary_weight_matmul_b200 import build
    build.build()
    m.lib()
    torch.cuda.set_device(0)
    return m


def h(t):
    return torch.finfo(t).eps / 2


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def operands(seed, m, d, v, xt, tt, spread=1.0):
    g = gen(seed)
    x = (spread * torch.randn(m, d, generator=g, device=DEV)).to(xt)
    t = (torch.randn(v, d, generator=g, device=DEV) * 2.0 / math.sqrt(d)).to(tt)
    return x, t, g


def close(got, want, bound, what, norm=None, scale=None):
    got = got.double()
    assert got.shape == want.shape, what
    bad = ~((got - want).abs() <= bound)
    if bad.any():
        i = int(bad.flatten().nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} out, first at {i}: got "
                             f"{float(got.flatten()[i])}, want {float(want.flatten()[i])}, bound "
                             f"{float((bound + 0 * want).flatten()[i])}")
    if norm is not None and want.numel():
        off = float((got - want).norm()), float(want.norm()) if scale is None else scale
        assert off[0] <= norm * off[1] + 1e-30, f"{what}: norm of the error {off[0]:.3e} of {off[1]:.3e}"


class Ref:
    """The losses in float64. q: [m, vocab] teacher weights (one-hot for the cross entropy)."""

    def __init__(self, x, t, q, live, tau=1.0):
        self.x, self.t, self.live, self.tau = x.double(), t.double(), live, tau
        self.x = torch.where(live[:, None], self.x, 0.0)
        self.q = q
        self.s = self.x @ self.t.T
        self.halves = t.dtype == F32
        self.lse = torch.logsumexp(self.s / tau, 1)
        self.e_s = ORDER6 * x.shape[1] * U * (self.x.abs() @ self.t.abs().T) / tau + 4 * U * self.s.abs() / tau
        if self.halves:
            ax, at = self.x.abs(), self.t.abs()
            self.e_s = self.e_s + STEP16 * (ax.sum(1, keepdim=True) * at.max() + ax.max(1, keepdim=True).values
                                            * at.sum(1)[None]) / tau
        self.e_lse = self.e_s.max(1).values + 64 * U * (1 + self.lse.abs())
        self.lse = torch.where(live, self.lse, 0.0)
        self.p = torch.where(live[:, None], torch.exp(self.s / tau - self.lse[:, None]), 0.0)

    def grads(self, dloss, g_type, xt, tt):
        c = torch.where(self.live, dloss.double(), 0.0)[:, None] / self.tau
        g = c * (self.p - self.q)
        e_g = c.abs() * (self.p * (self.e_s + self.e_lse[:, None] + 64 * U) + 64 * U * self.q) + 4 * U * g.abs()
        e_g = e_g + TINY * (1 + c.abs())
        if g_type == BF16:
            e_g = e_g + h(BF16) * (g.abs() + e_g)
        dx, dt = g @ self.t, g.T @ self.x
        self.scale = [float(a.norm() + b.norm()) for a, b in (((c * self.p) @ self.t, (c * self.q) @ self.t),
                                                              ((c * self.p).T @ self.x, (c * self.q).T @ self.x))]
        e_dx = e_g @ self.t.abs() + (6 * g.shape[1] + 64) * U * (g.abs() @ self.t.abs()) + 6 * g.shape[1] * TINY
        e_dt = e_g.T @ self.x.abs() + (6 * g.shape[0] + 64) * U * (g.abs().T @ self.x.abs()) + 6 * g.shape[0] * TINY
        if self.halves:
            e_dx = e_dx + STEP16 * (g.abs().sum(1, keepdim=True) * self.t.abs().max() + c.abs() * self.t.abs().sum(0))
            cx = (c * self.x).abs()
            one = (self.p - self.q).abs()
            e_dt = e_dt + STEP16 * (one.sum(0)[:, None] * cx.max() + cx.sum(0)[None])
            if xt == BF16:
                e_dx = e_dx + 2.0 ** -10 * (g.abs() @ self.t.abs())
        # a bf16 gradient beside float32 rows: products of two bf16 planes, 2^-15 of the terms at most
        if g_type == F32 and tt == BF16:
            e_dt = e_dt + 2.0 ** -14 * (g.abs().T @ self.x.abs())
        return dx, dt, e_dx + h(xt) * (dx.abs() + e_dx), e_dt + h(tt) * (dt.abs() + e_dt)


def gtype(xt, tt):
    """What g is held to: one bf16 value with bf16 operands (finer in calls of few rows, which the bound
    for one value covers)."""
    return BF16 if xt == BF16 and tt == BF16 else F32


def norm_tol(out, g, r):
    """2-norm tolerance: the roundings of g and of the output where they are bf16, of the leading fp16 values
    where those stand alone, and the logits' 16 u."""
    roundings = (out == BF16) + (g == BF16)
    return h(BF16) * roundings + (2.0 ** -10 if r.halves and out == BF16 else 0.0) + 16 * U * (1 + float(r.s.abs().max()) / r.tau)


def check_xent(mmf, x, t, targets, dloss, want=(True, True)):
    m, v = x.shape[0], t.shape[0]
    live = (targets >= 0) & (targets < v)
    q = torch.zeros(m, v, dtype=torch.float64, device=DEV)
    q[live.nonzero()[:, 0], targets[live].long()] = 1.0
    r = Ref(x, t, q, live)
    loss, lse = mmf.lm_head_xent_fwd(x, t, targets)
    at = torch.where(live, targets, 0).long()[:, None]
    s_t = r.s.gather(1, at)[:, 0]
    close(lse, r.lse, torch.where(live, r.e_lse, 0.0), "lse", 16 * U)
    close(loss, torch.where(live, r.lse - s_t, 0.0),
          torch.where(live, r.e_lse + r.e_s.gather(1, at)[:, 0] + 4 * U * (r.lse.abs() + s_t.abs()), 0.0), "loss")
    dx, dt = mmf.lm_head_xent_backward(x, t, targets, lse, dloss, *want)
    assert (dx is not None, dt is not None) == want
    wdx, wdt, bdx, bdt = r.grads(dloss, gtype(x.dtype, t.dtype), x.dtype, t.dtype)
    g = gtype(x.dtype, t.dtype)
    if want[0]:
        assert dx.dtype == x.dtype
        close(dx, wdx, bdx, "dx", norm_tol(x.dtype, g, r), r.scale[0])
        assert not dx[~live].any()
    if want[1]:
        assert dt.dtype == t.dtype
        close(dt, wdt, bdt, "dtable", norm_tol(t.dtype, g, r), r.scale[1])
    assert mmf.sync_status(DEV) == mmf.MMF_OK
    return loss, lse, dx, dt


TYPES = [(BF16, BF16), (F32, F32), (F32, BF16), (BF16, F32)]
IDS = ["bf16", "f32", "f32-bf16", "bf16-f32"]


@pytest.mark.parametrize("xt,tt", TYPES, ids=IDS)
@pytest.mark.parametrize("m,d,v", [(1, 8, 1), (1, 1024, 32000), (2, 64, 2), (31, 72, 257), (128, 128, 256),
                                   (129, 136, 1000), (300, 704, 5003), (513, 256, 255), (200, 72, 257),
                                   (256, 704, 2000), (769, 136, 1000), (1500, 1032, 513)])
def test_xent_shapes_and_types(mmf, m, d, v, xt, tt):
    x, t, g = operands(m * 31 + v, m, d, v, xt, tt)
    targets = torch.randint(0, v, (m,), generator=g, device=DEV).to(torch.int32)
    dloss = torch.randn(m, generator=g, device=DEV)
    check_xent(mmf, x, t, targets, dloss)


@pytest.mark.parametrize("xt,tt,m,v", [(BF16, BF16, 12289, 23001), (F32, F32, 5000, 21007)])
def test_xent_several_vocabulary_pieces(mmf, xt, tt, m, v):
    # g of the whole vocabulary is above the 512 MB a piece aims at
    assert (m + 255) // 256 * 256 * v * (2 if xt == BF16 else 6) > 512 << 20
    x, t, g = operands(7, m, 64, v, xt, tt)
    targets = torch.randint(-200, v, (m,), generator=g, device=DEV).to(torch.int32)
    check_xent(mmf, x, t, targets, torch.randn(m, generator=g, device=DEV))


@pytest.mark.parametrize("xt,tt", TYPES[:2], ids=IDS[:2])
@pytest.mark.parametrize("pattern", ["none", "one", "last", "alternate", "out of range"])
@pytest.mark.parametrize("m", [101, 515, 1030, 5001])
def test_xent_rows_left_out(mmf, m, xt, tt, pattern):
    d, v = 128, 700
    x, t, g = operands(11, m, d, v, xt, tt)
    targets = torch.randint(0, v, (m,), generator=g, device=DEV).to(torch.int32)
    drop = torch.ones(m, dtype=torch.bool, device=DEV)
    if pattern == "one":
        drop[m // 2] = False
    elif pattern == "last":
        drop[-3:] = False
    elif pattern == "alternate":
        drop[1::2] = False
    elif pattern == "out of range":
        drop[:] = False
        targets[5], targets[6], targets[7] = v, -2 ** 31, 2 ** 31 - 1
        drop[5:8] = True
    if pattern != "out of range":
        targets[drop] = -100
    dloss = torch.randn(m, generator=g, device=DEV)
    # what a dropped row holds reaches nothing
    x[drop] = float("nan")
    dloss[drop] = float("inf")
    loss, lse, dx, dt = check_xent(mmf, x, t, targets, dloss)
    for o in (loss, lse):
        assert not o[drop].any() and torch.isfinite(o).all()
    assert torch.isfinite(dx).all() and torch.isfinite(dt).all()
    if pattern == "none":
        assert not dt.any()


def test_xent_one_sided_gradients_and_no_rows(mmf):
    x, t, g = operands(12, 77, 64, 300, BF16, BF16)
    targets = torch.randint(0, 300, (77,), generator=g, device=DEV).to(torch.int32)
    dloss = torch.randn(77, generator=g, device=DEV)
    _, _, dx, dt = check_xent(mmf, x, t, targets, dloss)
    _, _, dx1, _ = check_xent(mmf, x, t, targets, dloss, (True, False))
    _, _, _, dt1 = check_xent(mmf, x, t, targets, dloss, (False, True))
    assert torch.equal(dx, dx1) and torch.equal(dt, dt1)
    e = torch.empty(0, 64, dtype=BF16, device=DEV)
    none = torch.empty(0, dtype=torch.int32, device=DEV)
    loss, lse = mmf.lm_head_xent_fwd(e, t, none)
    assert loss.numel() == 0 and lse.numel() == 0
    dx, dt = mmf.lm_head_xent_backward(e, t, none, lse, loss)
    assert dx.shape == (0, 64) and not dt.any() and dt.shape == t.shape


@pytest.mark.parametrize("m", [130, 800])
def test_xent_large_logits_and_nan_stay_in_their_rows(mmf, m):
    d, v = 64, 400
    x, t, g = operands(13, m, d, v, BF16, BF16, spread=200.0)  # logits of several hundred
    targets = torch.randint(0, v, (m,), generator=g, device=DEV).to(torch.int32)
    check_xent(mmf, x, t, targets, torch.randn(m, generator=g, device=DEV))
    x[17, 3] = float("nan")
    x[40, 5] = float("inf")
    loss, lse = mmf.lm_head_xent_fwd(x, t, targets)
    bad = torch.zeros(m, dtype=torch.bool, device=DEV)
    bad[17] = bad[40] = True
    assert torch.isfinite(loss[~bad]).all() and not torch.isfinite(loss[bad]).any()
    dx, _ = mmf.lm_head_xent_backward(x, t, targets, lse, torch.ones(m, device=DEV), want_dtable=False)
    assert torch.isfinite(dx[~bad]).all() and not torch.isfinite(dx[bad]).all(1).any()
    assert mmf.sync_status(DEV) == mmf.MMF_OK


@pytest.mark.parametrize("m", [90, 900])
@pytest.mark.parametrize("up", [1e18, 1e-18, 1e30, 1e-30])
def test_xent_float32_magnitudes(mmf, m, up):
    """Operands far from one with logits of order one: the fp16 pairs' powers of two at work."""
    x, t, g = operands(14, m, 128, 600, F32, F32)
    x[3] *= 1e-3
    targets = torch.randint(0, 600, (m,), generator=g, device=DEV).to(torch.int32)
    check_xent(mmf, x * up, t / up, targets, torch.randn(m, generator=g, device=DEV))
    check_xent(mmf, x, t, targets, torch.randn(m, generator=g, device=DEV) * up)


def test_offsets_past_32_bits(mmf):
    """2.2 M rows of 1024: the last rows' elements lie past 2^31. Their results equal those of a call that
    has only them (the same tiles' arithmetic; sums of dtable are left to the smaller tests)."""
    m, d, v, tail = 2_200_000, 1024, 257, 512
    assert (m - tail) * d > 2 ** 31
    g = gen(15)
    x = torch.empty(m, d, dtype=BF16, device=DEV)
    x[:-tail] = 0.01
    x[-tail:] = torch.randn(tail, d, generator=g, device=DEV).to(BF16)
    t = (torch.randn(v, d, generator=g, device=DEV) / 16).to(BF16)
    w = torch.rand(d, generator=g, device=DEV)
    targets = torch.randint(0, v, (m,), generator=g, device=DEV).to(torch.int32)
    targets[1::2] = -1                       # every other row is left out
    last = slice(m - tail, m)
    y, y_tail = mmf.rmsnorm_fwd(x, w), mmf.rmsnorm_fwd(x[last].contiguous(), w)
    assert torch.equal(y[last], y_tail)
    loss, lse = mmf.lm_head_xent_fwd(y, t, targets)
    loss_tail, lse_tail = mmf.lm_head_xent_fwd(y_tail, t, targets[last].contiguous())
    assert torch.equal(loss[last], loss_tail) and torch.equal(lse[last], lse_tail)
    one = torch.ones(m, device=DEV)
    dy, _ = mmf.lm_head_xent_backward(y, t, targets, lse, one, want_dtable=False)
    del y
    dy_tail, _ = mmf.lm_head_xent_backward(y_tail, t, targets[last].contiguous(), lse_tail, one[:tail], want_dtable=False)
    assert torch.equal(dy[last], dy_tail)
    dx, _ = mmf.rmsnorm_backward(x, w, dy)
    dx_tail, _ = mmf.rmsnorm_backward(x[last].contiguous(), w, dy_tail)
    assert torch.equal(dx[last], dx_tail)
    assert mmf.sync_status(DEV) == mmf.MMF_OK


def teacher_ref(ids, logits, v, tau):
    """(q [m, k], live [m], q over the vocabulary) in float64."""
    valid = (ids >= 0) & (ids < v) & (logits > -math.inf)
    live = valid.any(1)
    tl = torch.where(valid, logits.double(), -math.inf)
    tl = (tl - torch.where(live, tl.max(1).values, 0.0)[:, None]) / tau
    q = torch.where(live[:, None], torch.softmax(torch.where(live[:, None], tl, 0.0), 1), 0.0)
    q = torch.where(valid, q, 0.0)
    full = torch.zeros(ids.shape[0], v, dtype=torch.float64, device=DEV)
    full.scatter_add_(1, torch.where(valid, ids, 0).long(), q)
    return q, valid, live, full


def check_distill(mmf, x, t, ids, logits, tau, dloss):
    v = t.shape[0]
    q, valid, live, full = teacher_ref(ids, logits, v, tau)
    r = Ref(x, t, full, live, tau)
    loss, lse, s_top = mmf.lm_head_distill_fwd(x, t, ids, logits, temperature=tau)
    at = torch.where(valid, ids, 0).long()
    s = torch.where(valid, r.s.gather(1, at), 0.0)
    e_top = torch.where(valid, r.e_s.gather(1, at) * tau, 0.0)
    close(lse, r.lse, torch.where(live, r.e_lse, 0.0), "lse", 16 * U)
    close(s_top, s, e_top, "s_top", 16 * U)
    logp = s / tau - r.lse[:, None]
    want = (torch.special.xlogy(q, q) - q * logp).sum(1)
    mag = (torch.special.xlogy(q, q).abs() + q * logp.abs()).sum(1)
    e = r.e_lse + (q * e_top / tau).sum(1) + 64 * U * (1 + mag)
    close(loss, torch.where(live, want, 0.0), torch.where(live, e, 0.0), "loss")
    dx, dt = mmf.lm_head_distill_backward(x, t, ids, logits, lse, s_top, dloss, temperature=tau)
    g = gtype(x.dtype, t.dtype)
    wdx, wdt, bdx, bdt = r.grads(dloss, g, x.dtype, t.dtype)
    close(dx, wdx, bdx, "dx", norm_tol(x.dtype, g, r), r.scale[0])
    close(dt, wdt, bdt, "dtable", norm_tol(t.dtype, g, r), r.scale[1])
    assert not dx[~live].any()
    assert mmf.sync_status(DEV) == mmf.MMF_OK
    return loss, lse, s_top, dx, dt


def teacher(seed, m, k, v, dtype):
    g = gen(seed)
    first = torch.randint(0, v, (m, 1), generator=g, device=DEV)
    step = torch.randint(1, max(2, v // k), (m, 1), generator=g, device=DEV)
    ids = ((first + torch.arange(k, device=DEV)[None] * step) % v).to(torch.int32)
    return ids, (4 * torch.randn(m, k, generator=g, device=DEV)).to(dtype), torch.randn(m, generator=g, device=DEV)


@pytest.mark.parametrize("xt,tt", TYPES, ids=IDS)
@pytest.mark.parametrize("m,d,v,k,tau", [(1, 8, 1, 1, 1.0), (1, 1024, 32000, 64, 2.0), (33, 72, 257, 5, 0.5),
                                         (129, 128, 1000, 33, 1.0), (300, 256, 5003, 256, 3.0),
                                         (200, 72, 257, 5, 0.5), (900, 264, 1100, 40, 2.0)])
def test_distill_shapes_and_types(mmf, m, d, v, k, tau, xt, tt):
    x, t, _ = operands(m * 17 + v, m, d, v, xt, tt)
    ids, logits, dloss = teacher(m + k, m, k, v, tt)
    check_distill(mmf, x, t, ids, logits, tau, dloss)


def test_distill_several_vocabulary_pieces(mmf):
    m, v = 12289, 23001
    x, t, _ = operands(21, m, 64, v, BF16, BF16)
    ids, logits, dloss = teacher(22, m, 40, v, BF16)
    check_distill(mmf, x, t, ids, logits, 1.0, dloss)


@pytest.mark.parametrize("lt", [F32, BF16])
@pytest.mark.parametrize("m", [60, 260, 1000])
def test_distill_masked_entries(mmf, m, lt):
    d, v, k = 64, 500, 40
    x, t, _ = operands(23, m, d, v, BF16, BF16)
    ids, logits, dloss = teacher(24, m, k, v, lt)
    low = torch.finfo(lt).min
    ids[0], logits[1] = -1, -math.inf            # no entry left, in two ways
    logits[2] = low                              # every entry at the lowest value: a uniform teacher
    logits[3, :20] = low                         # half of them
    logits[4, 1:] = -math.inf                    # one entry left
    ids[5, 3], ids[6, 7], ids[7, 9] = v, -2 ** 31, 2 ** 31 - 1
    ids[8] = 17                                  # one word in every entry
    ids[9, 10:20] = ids[9, 0]                    # and in some
    logits[ids == -1] = float("nan")             # what an entry that does not count holds
    logits[5, 3] = float("inf")
    x[0], x[1] = float("nan"), float("inf")
    dloss[0] = float("nan")
    logits_ref = torch.where(ids == -1, torch.zeros_like(logits), logits)
    logits_ref[5, 3] = 0.0
    got = mmf.lm_head_distill_fwd(x, t, ids, logits, temperature=0.25)
    ref = mmf.lm_head_distill_fwd(x, t, ids, logits_ref, temperature=0.25)
    assert all(torch.equal(a, b) for a, b in zip(got, ref))
    loss, lse, s_top, dx, dt = check_distill(mmf, x, t, ids, logits_ref, 0.25, dloss)
    for o in (loss, lse, s_top):
        assert not o[:2].any() and torch.isfinite(o).all()
    assert torch.isfinite(dt).all()


# ---------------------------------------------------------------------------------------------
# RMSNorm
# ---------------------------------------------------------------------------------------------
def check_norm(mmf, x, w, dy, eps, y_dtype=None):
    d = x.shape[-1]
    X, G = x.double(), dy.double()
    W = torch.ones(d, dtype=torch.float64, device=DEV) if w is None else w.double()
    y = mmf.rmsnorm_fwd(x, w, eps=eps, y_dtype=y_dtype)
    assert y.dtype == (y_dtype or x.dtype) and y.shape == x.shape
    rho = (X.square().mean(-1, keepdim=True) + eps) ** -0.5
    wy = X * rho * W
    # a float32 sum of d squares (d / 2 + 8 half-ulps relative, halved by the root) and four roundings
    rel = (d / 4 + 16) * U
    close(y, wy, (rel + h(y.dtype)) * wy.abs() + 1e-37, "y")
    dx, dw = mmf.rmsnorm_backward(x, w, dy, eps=eps)
    u = G * W
    mux = (u * X).mean(-1, keepdim=True)
    wdx = rho * u - rho ** 3 * X * mux
    mag = rho * u.abs() + rho ** 3 * X.abs() * (u * X).abs().mean(-1, keepdim=True)
    close(dx, wdx, (3 * rel + h(x.dtype)) * wdx.abs() + 4 * rel * mag + 1e-37, "dx")
    terms = G * X * rho
    wdw, mag = terms.reshape(-1, d).sum(0), terms.abs().reshape(-1, d).sum(0)
    rows = terms.reshape(-1, d).shape[0]
    close(dw, wdw, (rel + (rows + 64) * U) * mag + 1e-37, "dnorm_w")
    dx2, none = mmf.rmsnorm_backward(x, w, dy, eps=eps, want_dnorm_w=False)
    assert none is None and torch.equal(dx, dx2)
    assert mmf.sync_status(DEV) == mmf.MMF_OK


@pytest.mark.parametrize("xt,gt,yt", [(BF16, BF16, BF16), (F32, F32, F32), (BF16, F32, F32), (F32, BF16, BF16)])
@pytest.mark.parametrize("shape", [(1, 1), (3, 7), (1, 8), (2, 5, 64), (1001, 1024), (65, 2560), (7, 704), (9, 4104),
                                   (5, 16384), (3, 16392), (4, 2049)])
def test_norm_shapes_and_types(mmf, shape, xt, gt, yt):
    g = gen(sum(shape))
    x = (3 * torch.randn(*shape, generator=g, device=DEV)).to(xt)
    dy = torch.randn(*shape, generator=g, device=DEV).to(gt)
    w = 1 + 0.2 * torch.randn(shape[-1], generator=g, device=DEV)
    check_norm(mmf, x, w, dy, 1e-8, yt)
    check_norm(mmf, x, None, dy, 1e-2)


# more rows than one turn of all CTAs takes, at every number of rows a turn and on both sides of the widths
# where an odd row moves to the next kernel
@pytest.mark.parametrize("xt,gt", [(BF16, BF16), (F32, F32), (BF16, F32)])
@pytest.mark.parametrize("m,d", [(8005, 200), (5003, 512), (4001, 1024), (2503, 1536), (1501, 2560), (1203, 8192),
                                 (2003, 511), (1999, 513), (2001, 1279), (1501, 1281), (1507, 2303), (1201, 2305),
                                 (1203, 2815), (1205, 2817)])
def test_norm_of_many_turns(mmf, m, d, xt, gt):
    g = gen(m + d)
    x = (torch.randn(m, 1, generator=g, device=DEV).exp() * torch.randn(m, d, generator=g, device=DEV)).to(xt)
    dy = torch.randn(m, d, generator=g, device=DEV).to(gt)
    check_norm(mmf, x, 1 + 0.2 * torch.randn(d, generator=g, device=DEV), dy, 1e-8)


def test_norm_unaligned_rows_zero_rows_and_no_rows(mmf):
    g = gen(3)
    flat = torch.randn(40 * 64 + 1, generator=g, device=DEV)
    x, dy = flat[1:].view(40, 64), torch.randn(40, 64, generator=g, device=DEV)   # 4-byte aligned storage
    check_norm(mmf, x, torch.rand(64, generator=g, device=DEV), dy, 1e-8)
    x = torch.randn(300, 512, generator=g, device=DEV).to(BF16)
    x[5] = 0
    check_norm(mmf, x, None, torch.randn(300, 512, generator=g, device=DEV).to(BF16), 1e-6)
    e = torch.empty(0, 16, device=DEV)
    assert mmf.rmsnorm_fwd(e, None).shape == (0, 16)
    dx, dw = mmf.rmsnorm_backward(e, None, e)
    assert dx.shape == (0, 16) and not dw.any()


# ---------------------------------------------------------------------------------------------
# as they are used
# ---------------------------------------------------------------------------------------------
def test_finite_differences_of_the_mean_loss(mmf):
    """d(mean loss)/d(direction) through norm, cross entropy and distillation against central
    differences of the float32 forward: L(e) - L(-e) over 2 e has the forward's error (2e-6 of losses
    of about 8) over 2 e plus e^2 / 6 of a third derivative of order one."""
    m, d, v, k, e = 64, 128, 900, 16, 0.02
    x, t, g = operands(31, m, d, v, F32, F32)
    w = 1 + 0.1 * torch.randn(d, generator=g, device=DEV)
    targets = torch.randint(0, v, (m,), generator=g, device=DEV).to(torch.int32)
    ids, logits, _ = teacher(32, m, k, v, F32)
    dirs = [torch.randn(a.shape, generator=g, device=DEV) for a in (x, w, t)]
    dirs = [a / a.norm() for a in dirs]

    def total(x, w, t):
        y = mmf.rmsnorm_fwd(x, w)
        return float((mmf.lm_head_xent_fwd(y, t, targets)[0].double().mean()
                      + mmf.lm_head_distill_fwd(y, t, ids, logits, 2.0)[0].double().mean()))

    y = mmf.rmsnorm_fwd(x, w)
    one = torch.full((m,), 1.0 / m, device=DEV)
    _, lse = mmf.lm_head_xent_fwd(y, t, targets)
    dy1, dt1 = mmf.lm_head_xent_backward(y, t, targets, lse, one)
    _, lse, s_top = mmf.lm_head_distill_fwd(y, t, ids, logits, 2.0)
    dy2, dt2 = mmf.lm_head_distill_backward(y, t, ids, logits, lse, s_top, one, 2.0)
    dx, dw = mmf.rmsnorm_backward(x, w, dy1 + dy2)
    for i, grad in enumerate((dx, dw, dt1 + dt2)):
        moved = [[a + s * e * dirs[j] if j == i else a for j, a in enumerate((x, w, t))] for s in (1, -1)]
        diff = (total(*moved[0]) - total(*moved[1])) / (2 * e)
        got = float((grad.double() * dirs[i].double()).sum())
        assert abs(diff - got) <= 16 * U * 16 / e + e * e, (i, diff, got)


def test_run_through_the_model(mmf):
    """Blocks -> final norm -> loss -> gradients back to the blocks' output, as a training step runs
    them, against float64 of the same steps from the same block output."""
    import synth
    shape = synth.BlockShape("t", 256, 704, 1)
    block = mmf.make_block(synth.block_params(3, shape, random_norms=True), DEV)
    g = gen(41)
    v, b, t = 1000, 3, 50
    table = (0.05 * torch.randn(v, 256, generator=g, device=DEV)).to(BF16)
    ids = torch.randint(0, v, (b, t), generator=g, device=DEV).to(torch.int32)
    w = 1 + 0.1 * torch.randn(256, generator=g, device=DEV)
    hidden, _ = mmf.stack_fwd([block], ids, table)
    flat = hidden.reshape(b * t, 256)
    y = mmf.rmsnorm_fwd(flat, w, y_dtype=F32)       # float32 rows: the logits of lm_head_argmax
    targets = torch.full((b, t), -100, dtype=torch.int32, device=DEV)
    targets[:, :-1] = ids[:, 1:]
    targets = targets.reshape(-1)
    n = b * (t - 1)
    loss, lse = mmf.lm_head_xent_fwd(y, table, targets)
    dy, dtable = mmf.lm_head_xent_backward(y, table, targets, lse, torch.full((b * t,), 1.0 / n, device=DEV))
    dx, dw = mmf.rmsnorm_backward(flat, w, dy)
    assert mmf.sync_status(DEV) == mmf.MMF_OK
    X, T, W = (a.double().requires_grad_() for a in (flat, table, w))
    Y = X * (X.square().mean(1, keepdim=True) + 1e-8).rsqrt() * W
    L = torch.nn.functional.cross_entropy(Y @ T.T, targets.long(), ignore_index=-100)
    gx, gt, gw = torch.autograd.grad(L, (X, T, W))
    assert abs(float(loss.double().sum() / n) - L.item()) <= 16 * U * L.item()
    for got, want in ((dx, gx), (dtable, gt), (dw, gw)):
        tol = h(BF16) + 32 * U if got.dtype == BF16 else 32 * U
        assert float((got.double() - want).norm()) <= tol * float(want.norm())
    # the loss and the greedy head see one and the same logits
    top, logits = mmf.lm_head_argmax(flat, w, table, want_logits=True)
    assert torch.allclose(torch.logsumexp(logits.double(), 1)[targets >= 0], lse[targets >= 0].double(), rtol=1e-4)


@pytest.mark.parametrize("m", [70, 700])
def test_repeats_streams_and_graphs(mmf, m):
    d, v, k = 256, 3001, 24
    x, t, g = operands(51, m, d, v, BF16, BF16)
    targets = torch.randint(-300, v, (m,), generator=g, device=DEV).to(torch.int32)
    ids, logits, dloss = teacher(52, m, k, v, BF16)
    w = torch.rand(d, generator=g, device=DEV)

    def step():
        y = mmf.rmsnorm_fwd(x, w)
        loss, lse = mmf.lm_head_xent_fwd(y, t, targets)
        dy, dt = mmf.lm_head_xent_backward(y, t, targets, lse, dloss)
        l2, lse2, s_top = mmf.lm_head_distill_fwd(y, t, ids, logits, 2.0)
        dy2, dt2 = mmf.lm_head_distill_backward(y, t, ids, logits, lse2, s_top, dloss, 2.0)
        dx, dw = mmf.rmsnorm_backward(x, w, dy)
        return loss, lse, dy, dt, l2, lse2, s_top, dy2, dt2, dx, dw

    first = step()
    assert all(torch.equal(a, b) for a, b in zip(first, step()))
    # two streams at once
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = []
    torch.cuda.synchronize()
    for s in streams:
        with torch.cuda.stream(s):
            outs.append([step() for _ in range(3)])
    torch.cuda.synchronize()
    for runs in outs:
        for o in runs:
            assert all(torch.equal(a, b) for a, b in zip(first, o))
    # two captured graphs replayed in turn, with eager calls between, on changed inputs
    graphs = []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            out = step()
        graphs.append((gr, out))
    x.mul_(-0.5)
    want = step()
    for gr, _ in graphs:
        gr.replay()
    eager = step()
    for gr, _ in graphs[::-1]:
        gr.replay()
    torch.cuda.synchronize()
    for _, out in graphs:
        assert all(torch.equal(a, b) for a, b in zip(want, out))
    assert all(torch.equal(a, b) for a, b in zip(want, eager))
    assert mmf.sync_status(DEV) == mmf.MMF_OK


@pytest.mark.parametrize("m", [300, 2000])
def test_waits_that_run_out_are_reported(mmf, m):
    """With the cap at one microsecond the kernels' waits may run out: the call then ends by itself
    and the status says so; with the default cap the same call is right again."""
    d, v = 512, 9000
    x, t, g = operands(61, m, d, v, BF16, BF16)
    targets = torch.randint(0, v, (m,), generator=g, device=DEV).to(torch.int32)
    dloss = torch.randn(m, generator=g, device=DEV)
    want = mmf.lm_head_xent_fwd(x, t, targets)
    grads = mmf.lm_head_xent_backward(x, t, targets, want[1], dloss)
    assert mmf.sync_status(DEV) == mmf.MMF_OK
    mmf.set_wait_limit(1)
    try:
        lse = mmf.lm_head_xent_fwd(x, t, targets)[1]
        mmf.lm_head_xent_backward(x, t, targets, lse, dloss)
        assert mmf.sync_status(DEV) in (mmf.MMF_OK, mmf.MMF_ERR_TIMEOUT)
    finally:
        mmf.set_wait_limit(0)
    again = mmf.lm_head_xent_fwd(x, t, targets)
    assert all(torch.equal(a, b) for a, b in zip(want, again))
    assert all(torch.equal(a, b) for a, b in zip(grads, mmf.lm_head_xent_backward(x, t, targets, again[1], dloss)))
    assert mmf.sync_status(DEV) == mmf.MMF_OK
