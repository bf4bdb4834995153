"""Plain 64-bit forms of the head-wise operations, token by token, and the
magnitudes their error bounds are relative to.

``absolute=True`` runs the same sums over absolute values.  An operation that
adds the terms of a sum in any order, each term off by a relative e, is off by
at most e times that sum of absolute values (plus the additions' own rounding,
2^-24 of it for each), however much the terms cancel.
"""

import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}  # half a step, relative


def d(t):
    return None if t is None else t.detach().to("cpu", torch.float64)


def silu(v):
    return v * torch.sigmoid(v)


def spans(cu):
    cu = cu.tolist()
    return list(zip(cu, cu[1:]))


def slots_of(slots, n):
    return list(range(n)) if slots is None else slots.tolist()


def conv_prompts(x, weight, bias, cu, window, slots=None, resume=None, act=True, out=None):
    """(out, window, magnitude of the sums)."""
    x, weight, bias, window = d(x), d(weight), d(bias), d(window).clone()
    out = torch.zeros_like(x) if out is None else d(out).clone()
    mag = torch.zeros_like(out)
    w = weight.shape[1]
    for i, (a, b) in enumerate(spans(cu)):
        s = slots_of(slots, len(cu) - 1)[i]
        if not 0 <= s < window.shape[0]:
            continue
        held = window[s].t()
        if resume is None or not int(resume[i]):
            held = torch.zeros_like(held)
        line = torch.cat([held, x[a:b]])
        v = torch.zeros(b - a, x.shape[1], dtype=torch.float64) + (0 if bias is None else bias)
        m = v.abs()
        for k in range(w):
            v = v + line[k:k + b - a] * weight[:, k]
            m = m + (line[k:k + b - a] * weight[:, k]).abs()
        out[a:b] = silu(v) if act else v
        mag[a:b] = m
        window[s] = line[b - a:].t()
    return out, window, mag


def scan_prompts(x, dt_raw, A_log, B, C, D, z, dt_bias, cu, state, slots=None, resume=None,
                 softplus=True, out=None, absolute=False):
    """(out, state); absolute: (magnitude of out's sums, of the state's)."""
    x, dt_raw, A_log, B, C, D, z, dt_bias = map(d, (x, dt_raw, A_log, B, C, D, z, dt_bias))
    state = d(state).clone()
    heads = x.shape[1]
    per = heads // B.shape[1]
    if absolute:
        x, B, C, state = x.abs(), B.abs(), C.abs(), state.abs()
        D = None if D is None else D.abs()
    out = torch.zeros_like(x) if out is None or absolute else d(out).clone()
    rate = -torch.exp(A_log)
    for i, (a, b) in enumerate(spans(cu)):
        s = slots_of(slots, len(cu) - 1)[i]
        if not 0 <= s < state.shape[0]:
            continue
        h = state[s].clone()
        if resume is None or not int(resume[i]):
            h.zero_()
        for t in range(a, b):
            v = dt_raw[t] + (0 if dt_bias is None else dt_bias)
            delta = torch.nn.functional.softplus(v, threshold=60) if softplus else v
            h = h * torch.exp(delta * rate)[:, None, None]
            push = delta.abs() if absolute else delta
            h = h + (push[:, None] * x[t])[:, :, None] * B[t].repeat_interleave(per, 0)[:, None]
            y = (h * C[t].repeat_interleave(per, 0)[:, None]).sum(2)
            if D is not None:
                y = y + D[:, None] * x[t]
            if z is not None:
                y = y * (silu(z[t]).abs() if absolute else silu(z[t]))
            out[t] = y
        state[s] = h
    return out, state


def step(state, window, xbc, dt_raw, A_log, weight, bias, D, z, dt_bias, groups, slots=None,
         softplus=True, out=None):
    """(out, state, window, magnitude of out, of state): the conv's outputs enter
    the magnitudes by the sums of absolute values they come from."""
    rows = xbc.shape[0]
    heads, headdim, dstate = state.shape[1:]
    cu = torch.arange(rows + 1)
    n = heads * headdim
    resume = torch.ones(rows, dtype=torch.int32)
    u, window, mag = conv_prompts(xbc, weight, bias, cu, window, slots, resume)

    def parts(v):
        return (v[:, :n].unflatten(1, (heads, headdim)),
                v[:, n:n + groups * dstate].unflatten(1, (groups, dstate)),
                v[:, n + groups * dstate:].unflatten(1, (groups, dstate)))

    x, B, C = parts(u)
    y, new = scan_prompts(x, dt_raw, A_log, B, C, D, z, dt_bias, cu, state, slots, resume, softplus,
                          out)
    x, B, C = parts(mag)
    ym, sm = scan_prompts(x, dt_raw, A_log, B, C, D, z, dt_bias, cu, state, slots, resume, softplus,
                          absolute=True)
    return y, new, window, ym, sm


def rms_norm(x, weight, residual=None, eps=1e-5):
    """(y, r)."""
    r = d(x) if residual is None else d(x) + d(residual)
    return r / torch.sqrt((r * r).mean(1, keepdim=True) + eps) * d(weight), r


def within(name, got, ref, bound):
    """|got - ref| <= bound, element by element, with the same NaNs."""
    got, ref, bound = d(got), d(ref), torch.as_tensor(bound, dtype=torch.float64).expand(ref.shape)
    off = (got - ref).abs()
    bad = ~((off <= bound) | (torch.isnan(ref) & torch.isnan(got)))
    worst = float((off / bound.clamp_min(1e-300)).nan_to_num(0).max()) if off.numel() else 0.0
    print(f"[gpu] {name}: worst error {worst:.3f} of its bound", flush=True)
    assert not bad.any(), f"{name}: {int(bad.sum())} values past their bounds, worst {worst:.3g} times"
