"""The head-wise operations: conv and scan over packed prompts, one token a row
through both, and the norm around the projections.

    u = causal_conv1d_prompts(xbc, weight, bias, cu_seqlens=cu, window=windows, slots=slots)
    y = head_scan_prompts(x, dt_raw, A_log, B, C, D, z, dt_bias, cu_seqlens=cu, state=states,
                          slots=slots)
    y = head_scan_step(states, windows, xbc, dt_raw, A_log, weight, bias, D, z, dt_bias,
                       slots=slots)
    q, scale, residual = rms_norm(x, weight, residual=residual, quant="row")

Packed prompts lie one after another along the token axis: prompt i is rows
cu_seqlens[i] .. cu_seqlens[i+1]-1.  ``slots`` (int32, on the device; None means
0, 1, ...) names each prompt's (or row's) entry in the caches; an entry outside
the cache skips the prompt and leaves its rows of ``out`` as they were, as rows
behind the last prompt are.  No two prompts or rows of a call may share a slot.
``resume`` (int32, on the device; None means 0 for all) tells which prompts
start from their cache entries; the others start from zero.

The values of cu_seqlens, slots and resume stay on the device: nothing here
synchronises.  These operations update caches in place and have no gradients.
"""

from __future__ import annotations

import ctypes

import torch

from . import _ACTIVATIONS, _conv_weight, _launch, _lib, _need_gpu, _workspace

_IO = {torch.float32: _lib.MSS_F32, torch.bfloat16: _lib.MSS_BF16}
_QUANT = {None: _lib.MSS_QUANT_NONE, "row": _lib.MSS_QUANT_ROW, "block": _lib.MSS_QUANT_BLOCK}


def _io(t):
    try:
        return _IO[t.dtype]
    except KeyError:
        raise TypeError(f"unsupported dtype {t.dtype}: expected float32 or bfloat16") from None


def _like(t, name, shape, dtype, device):
    """``t`` if it has this shape, dtype and device."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    return t


def _vector(t, name, n, dtype, device):
    """A contiguous vector's address, or None."""
    if t is None:
        return None
    _like(t, name, (n,), dtype, device)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _cache(t, name, inner, dtype, device):
    """A cache [slots, *inner] whose entries are contiguous, at any distance
    from slot to slot: its slot count, address and slot stride."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() != len(inner) + 1 or t.shape[0] < 1:
        raise ValueError(f"{name} must have shape [slots, {', '.join(map(str, inner))}], got "
                         f"{tuple(t.shape)}")
    _like(t, name, (t.shape[0], *inner), dtype, device)
    step = 0 if 0 in inner else 1  # an empty entry has any strides
    for size, stride in zip(reversed(inner), reversed(t.stride()[1:])):
        if size > 1 and step > 0 and stride != step:
            raise ValueError(f"each entry of {name} must be contiguous")
        step *= size
    return t.shape[0], t.data_ptr(), t.stride(0)


def _prompts(a, cu_seqlens, slots, resume, device):
    if not isinstance(cu_seqlens, torch.Tensor) or cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 2:
        raise ValueError("cu_seqlens must be a vector of at least 2 offsets")
    n = cu_seqlens.shape[0] - 1
    a.seqs = n
    a.cu_seqlens = _vector(cu_seqlens, "cu_seqlens", n + 1, torch.int32, device)
    a.slots = _vector(slots, "slots", n, torch.int32, device)
    a.resume = _vector(resume, "resume", n, torch.int32, device)


def _out(out, shape, dtype, device):
    if out is None:
        return torch.empty(shape, dtype=dtype, device=device)
    return _like(out, "out", shape, dtype, device)


def _give_workspace(a, need, workspace, device):
    if workspace is None:
        if need == 0:
            return
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
    a.workspace = _workspace(workspace, device).data_ptr()
    a.workspace_bytes = workspace.numel()


def causal_conv1d_prompts(x, weight, bias=None, *, cu_seqlens, window, slots=None, resume=None,
                          activation="silu", out=None):
    """Causal depthwise conv1d with optional SiLU over packed prompts, ordered
    on torch's current stream.

    x [T, D] (float32 or bfloat16, any strides); weight [D, W] fp32 (or
    [D, 1, W], [D, W, 1]); bias [D] fp32 or None; cu_seqlens [n+1] int32;
    window [slots, D, W-1] (x's dtype, each entry contiguous): the last W-1
    samples of each sequence, read for prompts that resume and left updated.
    Returns out [T, D]; without ``out``, rows of no prompt are undefined.
    """
    _need_gpu(x, "x")
    if x.dim() != 2:
        raise ValueError(f"x must have 2 dimensions, got shape {tuple(x.shape)}")
    dev, (tokens, dim) = x.device, x.shape
    weight = _conv_weight(weight, dim, dev)
    width = weight.shape[1]
    if activation not in _ACTIVATIONS:
        raise ValueError(f"activation must be 'silu' or None, got {activation!r}")
    out = _out(out, x.shape, x.dtype, dev)
    a = _lib.ConvPromptsArgs()
    a.struct_size = ctypes.sizeof(a)
    a.io_dtype = _io(x)
    a.tokens, a.dim, a.width = tokens, dim, width
    a.x, a.x_stride[:] = x.data_ptr(), x.stride()
    a.weight, a.weight_stride[:] = weight.data_ptr(), weight.stride()
    a.bias = _vector(bias, "bias", dim, torch.float32, dev)
    _prompts(a, cu_seqlens, slots, resume, dev)
    a.cache_slots, a.window, a.window_stride = _cache(window, "window", (dim, width - 1), x.dtype,
                                                      dev)
    a.out, a.out_stride[:] = out.data_ptr(), out.stride()
    a.activation = _ACTIVATIONS[activation]
    _launch(_lib.lib().mss_causal_conv1d_prompts, a, dev)
    return out



def head_scan_prompts(x, dt_raw, A_log, B, C, D=None, z=None, dt_bias=None, *, cu_seqlens, state,
                      slots=None, resume=None, delta_softplus=True, out=None, workspace=None):
    """Head-wise selective scan over packed prompts, ordered on torch's current
    stream.

    x, z, out [T, H, P] (float32 or bfloat16, unit stride in P); dt_raw [T, H];
    B, C [T, G, N] (unit stride in N; G divides H and head h reads group
    h // (H / G)); A_log, D, dt_bias [H] fp32; cu_seqlens [n+1] int32; state
    [slots, H, P, N] fp32 (each entry contiguous), read for prompts that resume
    and left updated.  Returns out; without ``out``, rows of no prompt are
    undefined.  ``workspace`` (uint8) may be supplied to avoid its allocation;
    calls that may overlap in time need one each.
    """
    _need_gpu(x, "x")
    if x.dim() != 3:
        raise ValueError(f"x must have 3 dimensions, got shape {tuple(x.shape)}")
    dev, dt, (tokens, heads, headdim) = x.device, x.dtype, x.shape
    if not isinstance(B, torch.Tensor) or B.dim() != 3 or B.shape[0] != tokens:
        raise ValueError(f"B must have shape [{tokens}, groups, dstate]")
    _like(B, "B", B.shape, dt, dev)
    _like(C, "C", B.shape, dt, dev)
    _like(dt_raw, "dt_raw", (tokens, heads), dt, dev)
    groups, dstate = B.shape[1:]
    out = _out(out, x.shape, dt, dev)
    a = _lib.HeadScanArgs()
    a.struct_size = ctypes.sizeof(a)
    a.io_dtype = _io(x)
    a.tokens, a.heads, a.headdim, a.dstate, a.groups = tokens, heads, headdim, dstate, groups
    a.x, a.x_stride[:] = x.data_ptr(), x.stride()
    a.dt_raw, a.dt_stride[:] = dt_raw.data_ptr(), dt_raw.stride()
    a.A_log = _vector(A_log, "A_log", heads, torch.float32, dev)
    a.B, a.B_stride[:] = B.data_ptr(), B.stride()
    a.C, a.C_stride[:] = C.data_ptr(), C.stride()
    a.D = _vector(D, "D", heads, torch.float32, dev)
    if z is not None:
        _like(z, "z", x.shape, dt, dev)
        a.z, a.z_stride[:] = z.data_ptr(), z.stride()
    a.dt_bias = _vector(dt_bias, "dt_bias", heads, torch.float32, dev)
    _prompts(a, cu_seqlens, slots, resume, dev)
    a.cache_slots, a.state, a.state_stride = _cache(state, "state", (heads, headdim, dstate),
                                                    torch.float32, dev)
    a.out, a.out_stride[:] = out.data_ptr(), out.stride()
    a.delta_softplus = 1 if delta_softplus else 0
    lib = _lib.lib()
    st = ctypes.c_int(0)
    need = lib.mss_head_scan_prompts_workspace_size(ctypes.byref(a), ctypes.byref(st))
    _lib.check(st.value)
    _give_workspace(a, need, workspace, dev)
    _launch(lib.mss_head_scan_prompts, a, dev)
    return out


def head_scan_step(state, window, xbc, dt_raw, A_log, weight, bias=None, D=None, z=None,
                   dt_bias=None, *, slots=None, delta_softplus=True, out=None, workspace=None):
    """One token a row: the conv step with SiLU over all channels, then one step
    of the head-wise scan, ordered on torch's current stream.

    state [slots, H, P, N] fp32 and window [slots, C, W-1] (each entry
    contiguous) are updated in place; xbc [rows, C] (float32 or bfloat16) holds
    each row's new samples, x [H, P] first, then B [G, N] and C [G, N], so that
    C = H P + 2 G N; dt_raw [rows, H]; weight [C, W] fp32; bias [C], A_log, D,
    dt_bias [H] fp32; z [rows, H, P] or None.  Returns out [rows, H, P];
    without ``out``, skipped rows are undefined.
    """
    _need_gpu(state, "state")
    _need_gpu(xbc, "xbc")
    if state.dim() != 4 or xbc.dim() != 2:
        raise ValueError("state must be [slots, H, P, N] and xbc [rows, channels]")
    dev, dt, (rows, chans) = state.device, xbc.dtype, xbc.shape
    heads, headdim, dstate = state.shape[1:]
    groups, rest = divmod(chans - heads * headdim, 2 * max(dstate, 1))
    if rest or groups < 1:
        raise ValueError(f"xbc has {chans} channels: expected {heads * headdim} + 2 * groups * "
                         f"{dstate}")
    _like(xbc, "xbc", xbc.shape, dt, dev)
    _like(dt_raw, "dt_raw", (rows, heads), dt, dev)
    weight = _conv_weight(weight, chans, dev)
    width = weight.shape[1]
    out = _out(out, (rows, heads, headdim), dt, dev)
    a = _lib.HeadStepArgs()
    a.struct_size = ctypes.sizeof(a)
    a.io_dtype = _io(xbc)
    a.rows, a.heads, a.headdim, a.dstate, a.groups = rows, heads, headdim, dstate, groups
    a.width = width
    a.cache_slots, a.state, a.state_stride = _cache(state, "state", (heads, headdim, dstate),
                                                    torch.float32, dev)
    slots_w, a.window, a.window_stride = _cache(window, "window", (chans, width - 1), dt, dev)
    if slots_w != a.cache_slots:
        raise ValueError(f"window has {slots_w} slots, state {a.cache_slots}")
    a.xbc, a.xbc_stride[:] = xbc.data_ptr(), xbc.stride()
    a.dt_raw, a.dt_stride[:] = dt_raw.data_ptr(), dt_raw.stride()
    a.A_log = _vector(A_log, "A_log", heads, torch.float32, dev)
    a.weight, a.weight_stride[:] = weight.data_ptr(), weight.stride()
    a.bias = _vector(bias, "bias", chans, torch.float32, dev)
    a.D = _vector(D, "D", heads, torch.float32, dev)
    if z is not None:
        _like(z, "z", (rows, heads, headdim), dt, dev)
        a.z, a.z_stride[:] = z.data_ptr(), z.stride()
    a.dt_bias = _vector(dt_bias, "dt_bias", heads, torch.float32, dev)
    a.slots = _vector(slots, "slots", rows, torch.int32, dev)
    a.out, a.out_stride[:] = out.data_ptr(), out.stride()
    a.delta_softplus = 1 if delta_softplus else 0
    lib = _lib.lib()
    st = ctypes.c_int(0)
    need = lib.mss_head_scan_step_workspace_size(ctypes.byref(a), ctypes.byref(st))
    _lib.check(st.value)
    _give_workspace(a, need, workspace, dev)
    _launch(lib.mss_head_scan_step, a, dev)
    return out


def _rows(t, name, shape, dtype, device):
    _like(t, name, shape, dtype, device)
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must have unit stride in its columns")
    return t.data_ptr(), t.stride(0)


def rms_norm(x, weight, *, residual=None, eps=1e-5, quant=None, out=None, scale=None,
             residual_out=None):
    """Root-mean-square norm over the columns of x [R, D] (float32 or bfloat16),
    after adding ``residual`` [R, D] (float32 or bfloat16, its own dtype),
    ordered on torch's current stream: r = x + residual,
    y = r / sqrt(mean(r^2) + eps) * weight, with weight [D] fp32.

    quant None: returns y in x's dtype.  quant "row": returns (q, scale) with q
    float8_e4m3fn and scale [R, 1] fp32, y = q * scale; quant "block": scale
    [R, D / 128].  With a residual, r in the residual's dtype is returned last;
    ``residual_out`` may be ``residual`` itself, which is then updated in place.
    """
    _need_gpu(x, "x")
    if x.dim() != 2:
        raise ValueError(f"x must have 2 dimensions, got shape {tuple(x.shape)}")
    if quant not in _QUANT:
        raise ValueError(f"quant must be None, 'row' or 'block', got {quant!r}")
    dev, shape = x.device, x.shape
    rows, dim = shape
    a = _lib.NormArgs()
    a.struct_size = ctypes.sizeof(a)
    a.io_dtype = a.residual_dtype = _io(x)
    a.quant = _QUANT[quant]
    a.rows, a.dim, a.eps = rows, dim, eps
    a.x, a.x_stride = _rows(x, "x", shape, x.dtype, dev)
    a.weight = _vector(weight, "weight", dim, torch.float32, dev)
    out = _out(out, shape, x.dtype if quant is None else torch.float8_e4m3fn, dev)
    a.out, a.out_stride = _rows(out, "out", shape, out.dtype, dev)
    left = (out,)
    if quant is not None:
        if quant == "block" and dim % _lib.MSS_SCALE_BLOCK:
            raise ValueError(f"quant 'block' needs a multiple of {_lib.MSS_SCALE_BLOCK} columns, got {dim}")
        want = (rows, 1 if quant == "row" else dim // _lib.MSS_SCALE_BLOCK)
        if scale is None:
            scale = torch.empty(want, dtype=torch.float32, device=dev)
        elif not _like(scale, "scale", want, torch.float32, dev).is_contiguous():
            raise ValueError("scale must be contiguous")
        a.scale = scale.data_ptr()
        left += (scale,)
    elif scale is not None:
        raise ValueError("scale is given without quant")
    if residual is not None:
        a.residual_dtype = _io(residual)
        a.residual, a.residual_stride = _rows(residual, "residual", shape, residual.dtype, dev)
        if residual_out is None:
            residual_out = torch.empty(shape, dtype=residual.dtype, device=dev)
        a.residual_out, a.residual_out_stride = _rows(residual_out, "residual_out", shape,
                                                      residual.dtype, dev)
        left += (residual_out,)
    elif residual_out is not None:
        raise ValueError("residual_out is given without residual")
    _launch(_lib.lib().mss_rms_norm, a, dev)
    return left if len(left) > 1 else out
