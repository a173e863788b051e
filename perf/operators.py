"""The training end of the tied head as measured cases: the final RMSNorm, the softmax cross entropy
over the vocabulary and the distillation from a teacher's top logits, each forward ("fwd") and as a
training step does it, forward then backward ("train").

Sizes are those of the framework's models (hidden 1024 / 2048 / 2560, vocabulary 32000, 8 x 2048
tokens) and generic ragged ones. ``run`` computes the plain form in float32 with elementary torch
operations, or calls the framework when ``own`` is true."""
import math

import torch

own = False

EPS = 1e-8
DEV = "cuda"
_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------
def _norm(name, way, m, d, xt):
    return {"name": name, "op": "norm", "way": way, "m": m, "d": d, "xt": xt}


def _xent(name, way, m, d, v, xt, tt, ignored):
    return {"name": name, "op": "xent", "way": way, "m": m, "d": d, "v": v, "xt": xt, "tt": tt, "ignored": ignored}


def _distill(name, way, m, d, v, xt, tt, k, tau):
    return {"name": name, "op": "distill", "way": way, "m": m, "d": d, "v": v, "xt": xt, "tt": tt, "k": k, "tau": tau}


def listed():
    return [
        # the final norm of one small batch of sequences (2.7B width): a latency-bound call
        _norm("norm fwd 8x2560 bf16", "fwd", 8, 2560, "bf16"),
        # the final norm of one 370M training step, 8 x 2048 tokens
        _norm("norm train 16384x1024 bf16", "train", 16384, 1024, "bf16"),
        # a ragged batch with float32 activations (1.3B width)
        _norm("norm train 5001x2048 f32", "train", 5001, 2048, "f32"),
        # scoring one short prompt: the table streams past a few rows
        _xent("xent fwd 40x1024 bf16", "fwd", 40, 1024, 32000, "bf16", "bf16", 0.0),
        # evaluation of exactly normalised float32 rows against a bf16 table
        _xent("xent fwd 2001x2048 mixed", "fwd", 2001, 2048, 32000, "f32", "bf16", 0.0),
        # one 370M training step, a few padded positions
        _xent("xent train 16384x1024 bf16", "train", 16384, 1024, 32000, "bf16", "bf16", 0.05),
        # one 2.7B fine-tuning step: prompts are masked out of the loss
        _xent("xent train 16384x2560 bf16", "train", 16384, 2560, 32000, "bf16", "bf16", 0.3),
        # float32 training of a small model on a ragged batch with an odd vocabulary
        _xent("xent train 1111x1024 f32", "train", 1111, 1024, 8191, "f32", "f32", 0.1),
        # distillation loss of a validation batch
        _distill("distill fwd 333x2560 bf16", "fwd", 333, 2560, 32000, "bf16", "bf16", 20, 1.0),
        # one 370M distillation step
        _distill("distill train 16384x1024", "train", 16384, 1024, 32000, "bf16", "bf16", 64, 2.0),
        # a ragged 1.3B distillation batch with a long teacher list
        _distill("distill train 4099x2048", "train", 4099, 2048, 32000, "bf16", "bf16", 128, 1.0),
        # float32 distillation of a small model
        _distill("distill train 640x704 f32", "train", 640, 704, 10007, "f32", "f32", 33, 1.5),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("norm", "xent", "xent", "distill", "distill"))
    way = rng.choice(("fwd", "train", "train"))
    d = rng.choice((256, 1024, 2048, 2560, 8 * rng.randint(16, 320)))
    if op == "norm":
        return {"op": op, "way": way, "m": _log(rng, 4, 16384), "d": d + rng.choice((0, 0, 1, 5)),
                "xt": rng.choice(("bf16", "f32"))}
    xt, tt = rng.choice((("bf16", "bf16"), ("bf16", "bf16"), ("bf16", "bf16"), ("f32", "bf16"), ("f32", "f32")))
    m = _log(rng, 1, 16384) if xt == "bf16" else _log(rng, 1, 4096)
    c = {"op": op, "way": way, "m": m, "d": d, "v": rng.choice((32000, rng.randint(1000, 32000))), "xt": xt, "tt": tt}
    if op == "xent":
        c["ignored"] = rng.choice((0.0, 0.05, 0.3, 0.7))
    else:
        c["k"] = _log(rng, 1, 128)
        c["tau"] = rng.choice((0.5, 1.0, 2.0))
    return c


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------
def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    m, d, xt = case["m"], case["d"], _DT[case["xt"]]

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=DEV)

    if case["op"] == "norm":
        # residual-stream rows of different sizes, gains near one, a gradient of a mean loss
        x = (randn(m, d) * (0.5 + 2.0 * torch.rand(m, 1, generator=g, device=DEV))).to(xt)
        return {"case": case, "x": x, "w": 1.0 + 0.1 * randn(d), "dy": (randn(m, d) / 64.0).to(xt)}

    v, k = case["v"], case.get("k", 1)
    table = (0.02 * randn(v, d)).to(_DT[case["tt"]])
    first = torch.randint(0, v, (m,), generator=g, device=DEV)
    # rows that lean towards one word, so that its logit stands out by about 6; unit mean square
    x = randn(m, d) + (6.0 / (0.0004 * d)) * table[first].float()
    x = (x * x.square().mean(1, keepdim=True).rsqrt()).to(xt)
    s = {"case": case, "x": x, "table": table}
    if case["op"] == "xent":
        drop = torch.rand(m, generator=g, device=DEV) < case["ignored"]
        s["targets"] = torch.where(drop, -1, first).to(torch.int32)
        live = (~drop).sum().clamp(min=1)
    else:
        # k distinct words a row, the first the favoured one; teachers that list fewer leave -1
        step = torch.randint(1, max(2, v // k), (m, 1), generator=g, device=DEV)
        ids = (first[:, None] + torch.arange(k, device=DEV)[None] * step) % v
        short = torch.rand(m, k, generator=g, device=DEV) < 0.02
        s["t_ids"] = torch.where(short, -1, ids).to(torch.int32)
        fall = torch.rand(m, k, generator=g, device=DEV).sort(dim=1, descending=True).values
        s["t_logits"] = (4.0 + 8.0 * fall + 0.3 * randn(m, k)).to(xt)
        live = torch.tensor(float(m), device=DEV)
    s["dloss"] = (0.5 + torch.rand(m, generator=g, device=DEV)) / live
    return s


# ---------------------------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------------------------
def _plain_norm(s):
    x, w = s["x"].float(), s["w"]
    rho = (x.square().mean(1, keepdim=True) + EPS).rsqrt()
    y = (x * rho * w).to(s["x"].dtype)
    if s["case"]["way"] == "fwd":
        return [y]
    dy = s["dy"].float()
    u = dy * w
    dx = rho * u - rho * rho * rho * x * (u * x).mean(1, keepdim=True)
    return [y, dx.to(s["x"].dtype), (dy * x * rho).sum(0)]


def _softmax(logits):
    """exp(logits - max), in place, its row sums and the log-sum-exp."""
    top = logits.max(1, keepdim=True).values
    p = logits.sub_(top).exp_()
    total = p.sum(1, keepdim=True)
    return p, total, (top + total.log())[:, 0]


def _plain_xent(s):
    x, t = s["x"].float(), s["table"].float()
    targets = s["targets"].long()
    live = (targets >= 0) & (targets < t.shape[0])
    at = torch.where(live, targets, 0)[:, None]
    logits = x @ t.T
    hit = logits.gather(1, at)[:, 0]
    p, total, lse = _softmax(logits)
    zero = torch.zeros_like(lse)
    loss, lse = torch.where(live, lse - hit, zero), torch.where(live, lse, zero)
    if s["case"]["way"] == "fwd":
        return [loss, lse]
    c = torch.where(live, s["dloss"], zero)[:, None]
    p.mul_(c / total).scatter_add_(1, at, -c)
    return [loss, lse, (p @ t).to(s["x"].dtype), (p.T @ x).to(s["table"].dtype)]


def _plain_distill(s):
    x, t, tau = s["x"].float(), s["table"].float(), s["case"]["tau"]
    ids, tl = s["t_ids"].long(), s["t_logits"].float()
    valid = (ids >= 0) & (ids < t.shape[0]) & (tl > -math.inf)
    live = valid.any(1)
    at = torch.where(valid, ids, 0)
    tl = torch.where(valid, tl, -math.inf)
    top = torch.where(live, tl.max(1).values, 0.0)[:, None]
    e = ((tl - top) / tau).exp()
    norm = torch.where(live, e.sum(1), 1.0)[:, None]
    q = e / norm
    logq = torch.where(q > 0, (tl - top) / tau - norm.log(), 0.0)
    logits = x @ t.T
    hit = logits.gather(1, at)
    p, total, lse = _softmax(logits.div_(tau))
    zero = torch.zeros_like(lse)
    loss = (q * (logq - (hit / tau - lse[:, None]))).sum(1)
    loss, lse = torch.where(live, loss, zero), torch.where(live, lse, zero)
    if s["case"]["way"] == "fwd":
        return [loss, lse]
    c = torch.where(live, s["dloss"], zero)[:, None] / tau
    p.mul_(c / total).scatter_add_(1, at, -c * q)
    return [loss, lse, (p @ t).to(s["x"].dtype), (p.T @ x).to(s["table"].dtype)]


def run(state):
    case = state["case"]
    if own:
        return _own(state)
    if case["op"] == "norm":
        return _plain_norm(state)
    return _plain_xent(state) if case["op"] == "xent" else _plain_distill(state)


def _own(s):
    import ternary_weight_matmul_b200 as mmf

    case = s["case"]
    if case["op"] == "norm":
        y = mmf.rmsnorm_fwd(s["x"], s["w"], eps=EPS)
        if case["way"] == "fwd":
            return [y]
        return [y, *mmf.rmsnorm_backward(s["x"], s["w"], s["dy"], eps=EPS)]
    if case["op"] == "xent":
        loss, lse = mmf.lm_head_xent_fwd(s["x"], s["table"], s["targets"])
        if case["way"] == "fwd":
            return [loss, lse]
        return [loss, lse, *mmf.lm_head_xent_backward(s["x"], s["table"], s["targets"], lse, s["dloss"])]
    tau = case["tau"]
    loss, lse, s_top = mmf.lm_head_distill_fwd(s["x"], s["table"], s["t_ids"], s["t_logits"], temperature=tau)
    if case["way"] == "fwd":
        return [loss, lse]
    return [loss, lse, *mmf.lm_head_distill_backward(s["x"], s["table"], s["t_ids"], s["t_logits"], lse, s_top,
                                                     s["dloss"], temperature=tau)]


# ---------------------------------------------------------------------------------------------
# work and exact values
# ---------------------------------------------------------------------------------------------
def work(case):
    m, d, xb = case["m"], case["d"], 2 if case["xt"] == "bf16" else 4
    train = case["way"] == "train"
    if case["op"] == "norm":
        if not train:
            return {"bytes": 2 * m * d * xb + 4 * d, "flops": 4 * m * d}
        return {"bytes": 4 * m * d * xb + 8 * d, "flops": 15 * m * d}
    v, tb, k = case["v"], 2 if case["tt"] == "bf16" else 4, case.get("k", 0)
    rows = round(m * (1.0 - case.get("ignored", 0.0)))
    read = rows * d * xb + v * d * tb + m * (4 if case["op"] == "xent" else k * (4 + xb)) + 8 * m
    flops = 2 * rows * v * d
    if train:
        return {"bytes": read + m * d * xb + v * d * tb + 4 * m, "flops": 4 * flops}
    return {"bytes": read, "flops": flops}


def exact(case, seed):
    s = prepare(case, seed)
    x = s["x"].double().requires_grad_()
    train = case["way"] == "train"
    if case["op"] == "norm":
        w = s["w"].double().requires_grad_()
        y = x / torch.sqrt(x.pow(2).mean(-1, keepdim=True) + EPS) * w
        if not train:
            return [y.detach()]
        dx, dw = torch.autograd.grad(y, (x, w), s["dy"].double())
        return [y.detach(), dx, dw]
    t = s["table"].double().requires_grad_()
    if case["op"] == "xent":
        logits = x @ t.T
        label = s["targets"].long()
        loss = torch.nn.functional.cross_entropy(logits, label, ignore_index=-1, reduction="none")
        some = label != -1
    else:
        logits = (x @ t.T) / case["tau"]
        teacher = torch.full(logits.shape, -math.inf, dtype=torch.float64, device=DEV)
        rows, cols = (s["t_ids"] >= 0).nonzero(as_tuple=True)
        teacher[rows, s["t_ids"][rows, cols].long()] = s["t_logits"][rows, cols].double() / case["tau"]
        some = (s["t_ids"] >= 0).any(1)
        teacher[~some] = 0.0
        q = torch.softmax(teacher, 1)
        loss = (torch.special.xlogy(q, q) - q * torch.log_softmax(logits, 1)).sum(1)
        loss = torch.where(some, loss, 0.0)
    lse = torch.where(some, torch.logsumexp(logits.detach(), 1), 0.0)
    if not train:
        return [loss.detach(), lse]
    dx, dt = torch.autograd.grad(loss, (x, t), s["dloss"].double())
    return [loss.detach(), lse, dx, dt]
