"""The operators at the end of a training step, case by case: the norm in front
of the vocabulary's projection and the losses behind it, with their gradients.

norm     layer norm with the residual's addition, forward or backward with the
         reduction of the weight's and the bias's gradients
entropy  softmax cross entropy of hidden states over a vocabulary, the logits
         never whole in memory; losses alone, or losses and gradients
distill  the same against a teacher's top logits: a sparse distribution a row

``own`` chooses between this package's kernels and the plain form: elementary
torch operations in 32 bits, rounded once at the end.
"""

import math

import torch

own = False

EPS = 1e-5
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4}


# ---------------------------------------------------------------- the cases

def _norm(name, rows, dim, dtype, grad, residual="none", bias=True):
    return {"name": name, "op": "norm", "rows": rows, "dim": dim, "dtype": dtype, "grad": grad,
            "residual": residual, "bias": bias}


def _entropy(name, rows, dim, vocab, dtype, grad, ignored=0.0, weighted=False):
    return {"name": name, "op": "entropy", "rows": rows, "dim": dim, "vocab": vocab,
            "dtype": dtype, "grad": grad, "ignored": ignored, "weighted": weighted}


def _distill(name, rows, dim, vocab, top, dtype, grad, tau=1.0, ragged=False, weighted=False):
    return {"name": name, "op": "distill", "rows": rows, "dim": dim, "vocab": vocab, "top": top,
            "dtype": dtype, "grad": grad, "tau": tau, "ragged": ragged, "weighted": weighted}


def listed():
    return [
        # the norm of one token of a 768-channel model: a launch and one trip to memory
        _norm("norm_one", 1, 768, "bf16", False),
        # the norm of a training batch, fp32 residual stream
        _norm("norm_batch", 32768, 2560, "bf16", False, "f32"),
        # backward of an odd batch in fp32, odd width, no bias
        _norm("norm_back_odd_f32", 2047, 1001, "f32", True, bias=False),
        # backward of a training batch, gradients of the block and of the residual stream
        _norm("norm_back_batch", 32768, 5120, "bf16", True, "f32"),
        # a few answer tokens of one sample, with gradients: the vocabulary's matrix is read
        # and its gradient written for hardly any rows
        _entropy("entropy_few", 24, 768, 32768, "bf16", True),
        # scoring a document: losses alone, an odd vocabulary
        _entropy("entropy_score", 2000, 1536, 50281, "bf16", False),
        # a small fp32 run, odd sizes, a third of the rows without a target
        _entropy("entropy_odd_f32", 515, 770, 9973, "f32", True, ignored=0.33, weighted=True),
        # a training batch, a quarter of its rows prompts that are not learned
        _entropy("entropy_batch", 8192, 2560, 65536, "bf16", True, ignored=0.25),
        # a few tokens against a teacher's eight best
        _distill("distill_few", 9, 768, 32768, 8, "bf16", True, tau=2.0),
        # how far a student is from its teacher: losses alone
        _distill("distill_score", 1024, 2560, 50304, 32, "bf16", False, tau=1.0, ragged=True),
        # fp32, odd sizes, rows with fewer entries than others and with none
        _distill("distill_odd_f32", 301, 500, 7001, 13, "f32", True, tau=1.7, ragged=True,
                 weighted=True),
        # a training batch against a teacher's 64 best
        _distill("distill_batch", 4096, 2560, 65536, 64, "bf16", True, tau=2.0, ragged=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "entropy", "entropy", "distill"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    grad = rng.random() < 0.7
    while True:
        if op == "norm":
            c = _norm("", _log_int(rng, 1, 32768), _log_int(rng, 8, 8192), dtype, grad,
                      rng.choice(["none", dtype, "f32"]), rng.random() < 0.7)
        else:
            rows, vocab = _log_int(rng, 1, 8192), _log_int(rng, 500, 65536)
            dim = _log_int(rng, 64, 5120)
            if rng.random() < 0.6:
                dim = -(-dim // 64) * 64
            if op == "entropy":
                c = _entropy("", rows, dim, vocab, dtype, grad,
                             rng.choice([0.0, 0.0, rng.uniform(0.0, 0.9)]), rng.random() < 0.3)
            else:
                c = _distill("", rows, dim, vocab, _log_int(rng, 1, 128), dtype, grad,
                             rng.choice([1.0, rng.uniform(0.5, 4.0)]), rng.random() < 0.5,
                             rng.random() < 0.3)
        most = [work(k) for k in listed() if k["op"] == op]
        w = work(c)
        # (products in fp32 cost this card eight times those in bf16)
        cost = w["flops"] * (8 if dtype == "f32" and op != "norm" else 1)
        if w["bytes"] <= max(k["bytes"] for k in most) and cost <= max(k["flops"] for k in most):
            break
    del c["name"]
    return c


def work(case):
    es = BYTES[case["dtype"]]
    if case["op"] == "norm":
        n, d = case["rows"] * case["dim"], case["dim"]
        res = BYTES.get(case["residual"], 0)
        params = d * (8 if case["bias"] else 4)
        if not case["grad"]:
            return {"bytes": n * (2 * es + 2 * res) + 8 * case["rows"] + params, "flops": 8 * n}
        # dy, the normed rows, and with a residual stream its gradient, read; written once for
        # each type that is wanted
        both = 0 if res in (0, es) else res
        rows = es + (res or es) + (res if res else 0) + es + both
        return {"bytes": n * rows + 8 * case["rows"] + d * 4 + params, "flops": 16 * n}
    live = round(case["rows"] * (1 - case.get("ignored", 0.0)))
    d, v = case["dim"], case["vocab"]
    rest = case["rows"] * (8 if case["op"] == "entropy" else 12 * case["top"])
    size = (case["rows"] * d + v * d) * es * (2 if case["grad"] else 1)
    return {"bytes": size + rest + 8 * case["rows"],
            "flops": (6 if case["grad"] else 2) * live * v * d}


# ---------------------------------------------------------------- the inputs

def _randn(g, *shape, dtype=torch.float32, scale=1.0):
    return torch.randn(*shape, generator=g, device="cuda").mul_(scale).to(dtype)


def _rand(g, *shape):
    return torch.rand(*shape, generator=g, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    dt = TYPES[case["dtype"]]
    s = {"op": case["op"], "grad": case["grad"]}
    r, d = case["rows"], case["dim"]
    if case["op"] == "norm":
        s["weight"] = 1 + 0.1 * _randn(g, d)
        s["bias"] = 0.1 * _randn(g, d) if case["bias"] else None
        res = TYPES.get(case["residual"])
        if not case["grad"]:
            s["x"] = _randn(g, r, d, dtype=dt)
            s["residual"] = None if res is None else _randn(g, r, d, dtype=res, scale=2.0)
            return s
        # what the forward pass left: the normed rows and their statistics
        s["dy"] = _randn(g, r, d, dtype=dt)
        s["r"] = (_randn(g, r, d, scale=2.0) + _randn(g, r, 1)).to(res or dt)
        s["dr"] = None if res is None else _randn(g, r, d, dtype=res)
        wide = s["r"].float()
        s["mean"] = wide.mean(1)
        s["rstd"] = torch.rsqrt((wide - s["mean"][:, None]).square().mean(1) + EPS)
        return s
    v = case["vocab"]
    s["weight"] = _randn(g, v, d, dtype=dt, scale=1 / math.sqrt(d))
    x = _randn(g, r, d)
    if case["op"] == "entropy":
        s["targets"] = torch.randint(v, (r,), generator=g, device="cuda")
        first = s["targets"]
    else:
        k = min(case["top"], v)
        gaps = torch.randint(1, v // k + 1, (r, k), generator=g, device="cuda")
        base = torch.randint(v, (r, 1), generator=g, device="cuda")
        s["ids"] = (base + gaps.cumsum(1)) % v
        fall = -torch.log(_rand(g, r, k)).cumsum(1)
        s["teacher"] = (10 - 4 * torch.log1p(fall)).to(dt)
        s["tau"] = case["tau"]
        first = s["ids"][:, 0]
    # rows from undecided to sure of the first target
    x += (2 * math.log(v) * _rand(g, r, 1)) * s["weight"][first].float()
    s["x"] = x.to(dt)
    if case["op"] == "entropy" and case["ignored"]:
        # prompts come in runs: whole stretches of rows have no target
        runs = _rand(g, -(-r // 16))
        cut = torch.quantile(runs, case["ignored"]) if runs.numel() > 1 else runs.new_zeros(())
        s["targets"][(runs < cut).repeat_interleave(16)[:r]] = -100
    if case["op"] == "distill" and case["ragged"]:
        left = torch.randint(0, k + 1, (r, 1), generator=g, device="cuda")
        s["ids"][torch.arange(k, device="cuda") >= left] = -1
    s["row_weight"] = 0.5 * _rand(g, r) / r if case["weighted"] else None
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    if own:
        return _run_own(s)
    if s["op"] == "norm":
        return _plain_norm_back(s) if s["grad"] else _plain_norm(s)
    return _plain_loss(s)


def _run_own(s):
    import mamba_selective_scan_amd as mss
    if s["op"] == "norm":
        if not s["grad"]:
            out = mss.layer_norm_fwd(s["x"], s["weight"], s["bias"], residual=s["residual"], eps=EPS)
            return dict(zip(("y", "mean", "rstd", "r"), out))
        return mss.layer_norm_bwd(s["dy"], s["r"], s["weight"], s["mean"], s["rstd"], dr=s["dr"],
                                  bias=s["bias"] is not None)
    if s["op"] == "entropy":
        if not s["grad"]:
            out = mss.linear_cross_entropy_fwd(s["x"], s["weight"], s["targets"])
        else:
            out = mss.linear_cross_entropy_grad(s["x"], s["weight"], s["targets"], s["row_weight"])
    elif not s["grad"]:
        out = mss.linear_distillation_fwd(s["x"], s["weight"], s["ids"], s["teacher"],
                                          temperature=s["tau"])
    else:
        out = mss.linear_distillation_grad(s["x"], s["weight"], s["ids"], s["teacher"],
                                           s["row_weight"], temperature=s["tau"])
    return dict(zip(("loss", "lse", "dx", "dweight"), out))


def _plain_norm(s):
    x = s["x"].float()
    if s["residual"] is not None:
        x = x + s["residual"].float()
    mean = x.mean(1, keepdim=True)
    mid = x - mean
    rstd = torch.rsqrt(mid.square().mean(1, keepdim=True) + EPS)
    y = mid * rstd * s["weight"]
    if s["bias"] is not None:
        y = y + s["bias"]
    out = {"y": y.to(s["x"].dtype), "mean": mean.squeeze(1), "rstd": rstd.squeeze(1)}
    if s["residual"] is not None:
        out["r"] = x.to(s["residual"].dtype)
    return out


def _plain_norm_back(s):
    dy = s["dy"].float()
    rstd = s["rstd"][:, None]
    h = (s["r"].float() - s["mean"][:, None]) * rstd
    g = dy * s["weight"]
    d = rstd * (g - g.mean(1, keepdim=True) - h * (g * h).mean(1, keepdim=True))
    if s["dr"] is not None:
        d = d + s["dr"].float()
    out = {"x": d.to(s["dy"].dtype), "weight": (dy * h).sum(0)}
    if s["bias"] is not None:
        out["bias"] = dy.sum(0)
    if s["dr"] is not None:
        out["residual"] = d.to(s["dr"].dtype)
    return out


def _plain_loss(s):
    """Targets as a sparse distribution: [rows, entries] of ids and shares."""
    tau = s.get("tau", 1.0)
    x, w = s["x"].float(), s["weight"].float()
    ids = s["targets"][:, None] if s["op"] == "entropy" else s["ids"]
    there = (ids >= 0) & (ids < w.shape[0])
    live = there.any(1)
    at = torch.where(there, ids, torch.zeros_like(ids))
    if s["op"] == "entropy":
        share, known = there.float(), torch.zeros_like(there, dtype=torch.float32)
    else:
        t = (s["teacher"].float() / tau).masked_fill(~there, -math.inf)
        t = t - t.amax(1, keepdim=True).masked_fill(~live[:, None], 0.0)
        total = t.exp().sum(1, keepdim=True).masked_fill(~live[:, None], 1.0)
        share = t.exp() / total
        known = torch.where(there, t - total.log(), torch.zeros_like(t))
    z = torch.matmul(x, w.t())
    if tau != 1.0:
        z.div_(tau)
    top = z.amax(1, keepdim=True)
    picked = z.gather(1, at)
    e = z.sub_(top).exp_()
    total = e.sum(1, keepdim=True)
    lse = top + total.log()
    loss = tau * tau * (share * (known - picked + lse)).sum(1)
    out = {"loss": loss, "lse": lse.squeeze(1).masked_fill(~live, 0.0)}
    if not s["grad"]:
        return out
    if s["row_weight"] is None:
        c = live.float() / live.sum().clamp(min=1)
    else:
        c = s["row_weight"].masked_fill(~live, 0.0)
    g = e.div_(total).scatter_add_(1, at, -share).mul_((c * tau)[:, None])
    out["dx"] = torch.matmul(g, w).to(s["x"].dtype)
    out["dweight"] = torch.matmul(g.t(), x).to(s["weight"].dtype)
    return out


# ---------------------------------------------------------------- 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "norm":
        return _exact_norm_back(s) if s["grad"] else _exact_norm(s)
    return _exact_loss(s)


def _exact_norm(s):
    r = s["x"].double()
    if s["residual"] is not None:
        r = r + s["residual"].double()
    var, mean = torch.var_mean(r, 1, correction=0)
    rstd = 1 / torch.sqrt(var + EPS)
    y = torch.addcmul((s["weight"] * 0 if s["bias"] is None else s["bias"]).double(),
                      (r - mean[:, None]) / torch.sqrt(var + EPS)[:, None], s["weight"].double())
    out = {"y": y, "mean": mean, "rstd": rstd}
    if s["residual"] is not None:
        out["r"] = r
    return out


def _exact_norm_back(s):
    """The gradient of sum(dy * y), with the statistics that the call is given
    taken as the row's own."""
    dim = s["r"].shape[1]
    out = {"x": [], "weight": 0.0, "bias": 0.0}
    for a in range(0, s["r"].shape[0], 4096):
        at = slice(a, a + 4096)
        dy, rstd = s["dy"][at].double(), s["rstd"][at].double()
        h = (s["r"][at].double() - s["mean"][at].double()[:, None]) * rstd[:, None]
        g = dy * s["weight"].double()
        along = (g * h).sum(1) / dim
        d = (g - (g.sum(1) / dim)[:, None] - h * along[:, None]) * rstd[:, None]
        out["x"].append(d if s["dr"] is None else d + s["dr"][at].double())
        out["weight"] = out["weight"] + (dy * h).sum(0)
        out["bias"] = out["bias"] + dy.sum(0)
    out["x"] = torch.cat(out["x"])
    if s["bias"] is None:
        del out["bias"]
    if s["dr"] is not None:
        out["residual"] = out["x"]
    return out


def _exact_loss(s):
    """Blocks of rows; a row's distribution is subtracted entry by entry."""
    rows, vocab = s["x"].shape[0], s["weight"].shape[0]
    w = s["weight"].double()
    tau = s.get("tau", 1.0)
    ids = s["targets"][:, None] if s["op"] == "entropy" else s["ids"]
    there = (ids >= 0) & (ids < vocab)
    live = there.any(1)
    c = live.double() / max(int(live.sum()), 1) if s["row_weight"] is None \
        else s["row_weight"].double() * live
    loss, lse, dx = [], [], []
    dw = torch.zeros_like(w) if s["grad"] else None
    step = max(1, min(rows, (1 << 27) // vocab))
    for a in range(0, rows, step):
        at = slice(a, a + step)
        x, on = s["x"][at].double(), there[at]
        z = torch.matmul(x, w.t()) / tau
        total = torch.logsumexp(z, 1)
        if s["op"] == "entropy":
            t = on.double()
        else:
            t = torch.where(on, s["teacher"][at].double() / tau, torch.tensor(-math.inf, device="cuda").double())
            t = torch.nan_to_num(torch.softmax(t, 1))
        held = torch.take_along_dim(z, ids[at].clamp(0, vocab - 1), 1)
        part = torch.special.xlogy(t, t) - t * (held - total[:, None])
        loss.append(tau * tau * torch.where(on, part, torch.zeros_like(part)).sum(1))
        lse.append(torch.where(live[at], total, torch.zeros_like(total)))
        if not s["grad"]:
            continue
        g = torch.exp(z - total[:, None])
        line = torch.arange(g.shape[0], device="cuda")
        for k in range(ids.shape[1]):
            pick = ids[at][:, k]
            g.index_put_((line[on[:, k]], pick[on[:, k]]), -t[on[:, k], k], accumulate=True)
        g *= (c[at] * tau)[:, None]
        dx.append(torch.matmul(g, w))
        dw += torch.matmul(g.t(), x)
    out = {"loss": torch.cat(loss), "lse": torch.cat(lse)}
    if s["grad"]:
        out["dx"], out["dweight"] = torch.cat(dx), dw
    return out
