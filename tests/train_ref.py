"""The operations around a training step's scans in 64 bits, from their
definitions, with the magnitudes that the error bounds are made of.

A rounding to a type is off by at most half a step, finfo.eps / 2 relative to
the value.  A sum of n terms in fp32, in any order, is off by at most n roundings
of the sum of the terms' magnitudes (the matrix instruction's own additions may
drop bits instead of rounding: twice that).
"""

import torch

U = 2.0 ** -24


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def f64(t):
    return None if t is None else t.detach().double().cpu()


def norm_ref(x, weight, bias, residual, eps):
    """y, mean, rstd, r, and bounds of their errors in fp32 arithmetic."""
    x, weight, bias, residual = map(f64, (x, weight, bias, residual))
    r = x if residual is None else x + residual
    n = r.shape[1]
    mean = r.mean(1)
    mid = r - mean[:, None]
    var = mid.square().mean(1)
    rstd = 1 / torch.sqrt(var + eps)
    h = mid * rstd[:, None]
    y = h * weight + (0 if bias is None else bias)
    # r is rounded to fp32 where it is a sum; a sum takes at most 32 additions a
    # thread and 6 + 16 across threads
    depth = 64
    e_r = (U * r.abs()) if residual is not None else torch.zeros_like(r)
    e_mean = e_r.mean(1) + depth * U * r.abs().mean(1)
    # centred values: r and the mean, whose own rounding is taken out again (what
    # is left of it is a rounding of what was taken out)
    e_mid = e_r + e_r.mean(1)[:, None] + 2 * U * mid.abs() + (depth * U) ** 2 * r.abs().mean(1)[:, None] \
        + 2 * U * depth * U * r.abs().amax(1)[:, None] + depth * U * mid.abs().mean(1)[:, None]
    e_var = (2 * mid.abs() * e_mid + e_mid.square()).mean(1) + depth * U * var
    e_rstd = rstd * (0.5 * e_var / (var + eps) + 8 * U)
    e_h = e_mid * rstd[:, None] + h.abs() * (e_rstd / rstd)[:, None] + 2 * U * h.abs()
    e_y = e_h * weight.abs() + 2 * U * ((h * weight).abs() + y.abs())
    return {"y": (y, e_y), "mean": (mean, e_mean + U * mean.abs()), "rstd": (rstd, e_rstd), "r": (r, e_r)}


def norm_back_ref(dy, r, weight, mean, rstd, dr):
    """dx, dweight, dbias of the given statistics, with bounds."""
    dy, r, weight, mean, rstd, dr = map(f64, (dy, r, weight, mean, rstd, dr))
    h = (r - mean[:, None]) * rstd[:, None]
    g = dy * weight
    n = r.shape[1]
    s1, s2 = g.mean(1), (g * h).mean(1)
    d = rstd[:, None] * (g - s1[:, None] - h * s2[:, None])
    out = d if dr is None else d + dr
    e_h = 3 * U * h.abs()
    depth = 64
    e1 = depth * U * g.abs().mean(1)
    e2 = depth * U * (g * h).abs().mean(1) + (g.abs() * e_h).mean(1)
    e = rstd[:, None] * (4 * U * (g.abs() + s1.abs()[:, None] + (h * s2[:, None]).abs()) + e1[:, None]
                         + h.abs() * e2[:, None] + e_h * s2.abs()[:, None]) + 2 * U * out.abs()
    rows = r.shape[0]
    dw, db = (dy * h).sum(0), dy.sum(0)
    e_dw = (rows + 8) * U * (dy * h).abs().sum(0)
    e_db = (rows + 8) * U * dy.abs().sum(0)
    return {"x": (out, e), "residual": (out, e), "weight": (dw, e_dw), "bias": (db, e_db)}


def shares(ids, teacher, vocab, tau):
    """A row's distribution: where its entries count, and their shares."""
    ids = ids.cpu()
    if ids.dim() == 1:
        ids = ids[:, None]
    on = (ids >= 0) & (ids < vocab)
    if teacher is None:
        return ids, on, on.double()
    t = (f64(teacher) / tau).masked_fill(~on, float("-inf"))
    t = torch.softmax(t, 1).masked_fill(~on, 0.0)
    return ids, on, t.masked_fill(~on.any(1, keepdim=True), 0.0)


def loss_ref(x, weight, ids, teacher=None, row_weight=None, tau=1.0, scale=1.0, dtype=None):
    """loss, lse, dx, dweight with bounds of what the kernels' arithmetic may be
    off by, before the outputs' own rounding.

    The logits' products are exact in fp32 or the sum of six products of planes
    (left out: 3 * 2^-24 of the magnitudes); dz is kept in ``dtype``'s planes: in
    bf16 its log2 is first kept in steps of 2^-10."""
    dtype = dtype or x.dtype
    bf16 = dtype is torch.bfloat16
    rows, vocab, dim = x.shape[0], weight.shape[0], x.shape[1]
    ids, on, t = shares(ids, teacher, vocab, tau)
    live = on.any(1)
    x64, w64 = f64(x).clone(), f64(weight)
    x64[~live] = 0
    z = x64 @ w64.t() * (scale / tau)
    e_z = (x64.abs() @ w64.abs().t()) * abs(scale / tau) * (2 * dim + 12) * U
    lse = torch.logsumexp(z, 1)
    p = torch.exp(z - lse[:, None])
    tiles = (vocab + 63) // 64
    # a tile's sum, the sum over tiles, exponents rounded in fp32 at the logits' size
    e_p = e_z + U * 8 * (z.abs() + lse.abs()[:, None] + 2)
    e_lse = (p * e_p).sum(1) + (256 + tiles) * U + 8 * U * (lse.abs() + 1)
    at = ids.clamp(0, vocab - 1)
    held, e_held = z.gather(1, at), e_p.gather(1, at)
    log_t = torch.where(t > 0, t.clamp(min=1e-300).log(), torch.zeros_like(t))
    part = torch.where(t > 0, t * (log_t - held + lse[:, None]), torch.zeros_like(t))
    loss = tau * tau * part.sum(1)
    e_t = 0.0
    if teacher is not None:
        # a share is e^u over their sum: u, the distance from the row's largest over
        # tau, is off by two roundings of it, and so is every addend of the sum
        u = f64(teacher).masked_fill(~on, float("-inf"))
        u = torch.where(t > 0, (u - u.amax(1, keepdim=True)) / tau, torch.zeros_like(t))
        e_t = 4 * U * (8 + u.abs().amax(1))
    k = ids.shape[1]
    e_loss = tau * tau * ((t * e_held).sum(1) + e_lse + (t * ((log_t - held).abs() + lse.abs()[:, None])).sum(1)
                          * ((k + 8) * U + e_t))
    n = int(live.sum())
    c = (torch.full((rows,), 1.0 / max(n, 1), dtype=torch.float64) if row_weight is None else f64(row_weight).clone())
    c[~live] = 0
    dense = torch.zeros(rows, vocab, dtype=torch.float64)
    dense.scatter_add_(1, at, t)  # (entries that do not count have share 0)
    hit = torch.zeros(rows, vocab, dtype=torch.bool)
    hit.scatter_(1, at, on)
    p = torch.where(live[:, None], p, torch.zeros_like(p))
    f = c[:, None] * (scale * tau)
    dz = f * (p - dense)
    e_soft = p * (e_p + e_lse[:, None] + 8 * U)
    if bf16:
        # the code of a logit, dropped 64 below its tile's largest; then dz
        code = p * 2.0 ** -11 + 2.0 ** -90
        e_dz = torch.where(hit, e_soft + 2 * U, e_soft + code * 1.01)
        e_dz = f.abs() * e_dz + half_step(torch.bfloat16) * 1.01 * dz.abs()
    else:
        e_dz = f.abs() * (e_soft + torch.where(hit, 2.0 * U, 0.0)) + 3 * U * dz.abs()
    if teacher is not None:
        e_dz = e_dz + f.abs() * dense * (e_t if isinstance(e_t, float) else e_t[:, None])
    e_dz = e_dz + 4 * U * dz.abs()
    terms = 2 * U * (6 if not bf16 else 1)
    dx, dw = dz @ w64, dz.t() @ x64
    e_dx = e_dz @ w64.abs() + (vocab + 8) * terms * (dz.abs() @ w64.abs())
    e_dw = e_dz.t() @ x64.abs() + (rows + 8) * terms * (dz.abs().t() @ x64.abs())
    zero = torch.zeros_like(lse)
    return {"loss": (loss, e_loss), "lse": (torch.where(live, lse, zero), e_lse), "dx": (dx, e_dx),
            "dweight": (dw, e_dw)}


def within(name, got, ref, bound, dtype):
    """Every element within its bound and half a step of its type."""
    got = f64(got)
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    limit = bound + half_step(dtype) * (ref.abs() + bound) + torch.finfo(dtype).tiny
    off = (got - ref).abs()
    bad = ~(off <= limit)
    worst = (off / limit).nan_to_num(9e9).max().item() if off.numel() else 0.0
    print(f"[gpu] {name}: worst error is {worst:.3f} of its bound", flush=True)
    assert not bad.any(), (name, int(bad.sum()), worst)
