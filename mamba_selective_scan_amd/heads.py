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

Calls of no tokens or no rows are fine: they give empty outputs.  The values of
cu_seqlens, slots and resume stay on the device: nothing here synchronises.  These operations update caches in place and have no gradients.
"""

from __future__ import annotations

import ctypes

import torch

from . import _ACTIVATIONS, _conv_weight, _lib, _need_gpu, _workspace

_IO = {torch.float32: _lib.MSS_F32, torch.bfloat16: _lib.MSS_BF16}
_QUANT = {None: _lib.MSS_QUANT_NONE, "row": _lib.MSS_QUANT_ROW, "block": _lib.MSS_QUANT_BLOCK}


_conv_args = _lib.packer(_lib.ConvPromptsArgs)
_scan_args = _lib.packer(_lib.HeadScanArgs)
_step_args = _lib.packer(_lib.HeadStepArgs)
_norm_args = _lib.packer(_lib.NormArgs)
_Tensor = torch.Tensor
_current_device = torch._C._cuda_getDevice
_current_stream = torch._C._cuda_getCurrentRawStream


def _launch(fn, args, device):
    """Call a library entry point on torch's current stream of ``device``, with
    ``device`` current (as the package's own launches, whose stream lookup costs
    more than the rest of a small call)."""
    index = device.index
    if index == _current_device():
        code = fn(ctypes.byref(args), _current_stream(index))
    else:
        with torch.cuda.device(device):
            code = fn(ctypes.byref(args), _current_stream(index))
    if code:
        _lib.check(code)


def _io(t):
    try:
        return _IO[t.dtype]
    except KeyError:
        raise TypeError(f"unsupported dtype {t.dtype}: expected float32 or bfloat16") from None


def _like(t, name, shape, dtype, device):
    """``t`` if it has this shape, dtype and device."""
    if not isinstance(t, _Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    return t


def _gpu(t, name):
    if not isinstance(t, _Tensor) or not t.is_cuda:
        _need_gpu(t, name)  # (raises, saying what it got)
    return t.device


def _weight(weight, dim, device):
    """A conv weight as [dim, W] fp32."""
    if not isinstance(weight, _Tensor):
        raise TypeError("weight must be a torch.Tensor")
    shape = weight.shape
    if len(shape) != 2:
        return _conv_weight(weight, dim, device)
    return _like(weight, "weight", (dim, shape[1]), torch.float32, device)


def _vector(t, name, n, dtype, device):
    """A contiguous vector's address, or 0 for None."""
    if t is None:
        return 0
    _like(t, name, (n,), dtype, device)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _cache(t, name, inner, dtype, device):
    """A cache [slots, *inner] whose entries are contiguous, at any distance
    from slot to slot: its slot count, address and slot stride."""
    if not isinstance(t, _Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    shape = t.shape
    if len(shape) != len(inner) + 1 or shape[0] < 1:
        raise ValueError(f"{name} must have shape [slots, {', '.join(map(str, inner))}], got "
                         f"{tuple(shape)}")
    _like(t, name, (shape[0], *inner), dtype, device)
    if not t.is_contiguous() and not t[0].is_contiguous():
        raise ValueError(f"each entry of {name} must be contiguous")
    return shape[0], t.data_ptr(), t.stride()[0]


def _prompts(cu_seqlens, slots, resume, device):
    """Number of prompts, and the addresses of the three vectors."""
    if not isinstance(cu_seqlens, _Tensor) or cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 2:
        raise ValueError("cu_seqlens must be a vector of at least 2 offsets")
    n = cu_seqlens.shape[0] - 1
    return (n, _vector(cu_seqlens, "cu_seqlens", n + 1, torch.int32, device),
            _vector(slots, "slots", n, torch.int32, device),
            _vector(resume, "resume", n, torch.int32, device))


def _out(out, like, dtype, device):
    """``out`` if it has ``like``'s shape, or a contiguous tensor of it
    (empty_like and empty_strided: half the host time of torch.empty)."""
    if out is None:
        return torch.empty_like(like, dtype=dtype, memory_format=torch.contiguous_format)
    return _like(out, "out", like.shape, dtype, device)


def _optional(t):
    """Address and strides of a 3-d tensor, or zeros for None."""
    return (0, 0, 0, 0) if t is None else (t.data_ptr(), *t.stride())


def _give_workspace(a, need, workspace, device):
    if workspace is None:
        if need == 0:
            return
        workspace = torch.empty_strided((need,), (1,), dtype=torch.uint8, device=device)
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
    dev = _gpu(x, "x")
    if x.dim() != 2:
        raise ValueError(f"x must have 2 dimensions, got shape {tuple(x.shape)}")
    tokens, dim = x.shape
    weight = _weight(weight, dim, dev)
    width = weight.shape[1]
    if activation not in _ACTIVATIONS:
        raise ValueError(f"activation must be 'silu' or None, got {activation!r}")
    out = _out(out, x, x.dtype, dev)
    n, *prompts = _prompts(cu_seqlens, slots, resume, dev)
    cache_slots, *cache = _cache(window, "window", (dim, width - 1), x.dtype, dev)
    a = _conv_args(_io(x), tokens, dim, width, n, cache_slots,
                   x.data_ptr(), *x.stride(), weight.data_ptr(), *weight.stride(),
                   _vector(bias, "bias", dim, torch.float32, dev), *prompts, *cache,
                   out.data_ptr(), *out.stride(), _ACTIVATIONS[activation], 0)
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
    dev = _gpu(x, "x")
    if x.dim() != 3:
        raise ValueError(f"x must have 3 dimensions, got shape {tuple(x.shape)}")
    dt, (tokens, heads, headdim) = x.dtype, x.shape
    if not isinstance(B, _Tensor) or B.dim() != 3 or B.shape[0] != tokens:
        raise ValueError(f"B must have shape [{tokens}, groups, dstate]")
    _like(B, "B", B.shape, dt, dev)
    _like(C, "C", B.shape, dt, dev)
    _like(dt_raw, "dt_raw", (tokens, heads), dt, dev)
    groups, dstate = B.shape[1:]
    out = _out(out, x, dt, dev)
    if z is not None:
        _like(z, "z", x.shape, dt, dev)
    n, *prompts = _prompts(cu_seqlens, slots, resume, dev)
    cache_slots, *cache = _cache(state, "state", (heads, headdim, dstate), torch.float32, dev)
    a = _scan_args(_io(x), tokens, heads, headdim, dstate, groups, n, cache_slots,
                   x.data_ptr(), *x.stride(), dt_raw.data_ptr(), *dt_raw.stride(),
                   _vector(A_log, "A_log", heads, torch.float32, dev),
                   B.data_ptr(), *B.stride(), C.data_ptr(), *C.stride(),
                   _vector(D, "D", heads, torch.float32, dev), *_optional(z),
                   _vector(dt_bias, "dt_bias", heads, torch.float32, dev), *prompts, *cache,
                   out.data_ptr(), *out.stride(), 1 if delta_softplus else 0, 0, 0, 0)
    lib = _lib.lib()
    # (0 for sizes that the launch refuses)
    _give_workspace(a, lib.mss_head_scan_prompts_workspace_size(ctypes.byref(a), None), workspace, dev)
    _launch(lib.mss_head_scan_prompts, a, dev)
    return out


def head_scan_step(state, window, xbc, dt_raw, A_log, weight, bias=None, D=None, z=None,
                   dt_bias=None, *, slots=None, delta_softplus=True, out=None):
    """One token a row: the conv step with SiLU over all channels, then one step
    of the head-wise scan, ordered on torch's current stream.

    state [slots, H, P, N] fp32 and window [slots, C, W-1] (each entry
    contiguous) are updated in place; xbc [rows, C] (float32 or bfloat16) holds
    each row's new samples, x [H, P] first, then B [G, N] and C [G, N], so that
    C = H P + 2 G N; dt_raw [rows, H]; weight [C, W] fp32; bias [C], A_log, D,
    dt_bias [H] fp32; z [rows, H, P] or None.  Returns out [rows, H, P];
    without ``out``, skipped rows are undefined.
    """
    dev = _gpu(state, "state")
    _gpu(xbc, "xbc")
    if state.dim() != 4 or xbc.dim() != 2:
        raise ValueError("state must be [slots, H, P, N] and xbc [rows, channels]")
    dt, (rows, chans) = xbc.dtype, xbc.shape
    heads, headdim, dstate = state.shape[1:]
    groups, rest = divmod(chans - heads * headdim, 2 * max(dstate, 1))
    if rest or groups < 1:
        raise ValueError(f"xbc has {chans} channels: expected {heads * headdim} + 2 * groups * "
                         f"{dstate}")
    _like(xbc, "xbc", xbc.shape, dt, dev)
    _like(dt_raw, "dt_raw", (rows, heads), dt, dev)
    weight = _weight(weight, chans, dev)
    width = weight.shape[1]
    if out is None:
        out = torch.empty_strided((rows, heads, headdim), (heads * headdim, headdim, 1), dtype=dt, device=dev)
    else:
        _like(out, "out", (rows, heads, headdim), dt, dev)
    if z is not None:
        _like(z, "z", (rows, heads, headdim), dt, dev)
    cache_slots, *states = _cache(state, "state", (heads, headdim, dstate), torch.float32, dev)
    window_slots, *windows = _cache(window, "window", (chans, width - 1), dt, dev)
    if window_slots != cache_slots:
        raise ValueError(f"window has {window_slots} slots, state {cache_slots}")
    a = _step_args(_io(xbc), rows, heads, headdim, dstate, groups, width, cache_slots,
                   *states, *windows, xbc.data_ptr(), *xbc.stride(),
                   dt_raw.data_ptr(), *dt_raw.stride(),
                   _vector(A_log, "A_log", heads, torch.float32, dev),
                   weight.data_ptr(), *weight.stride(),
                   _vector(bias, "bias", chans, torch.float32, dev),
                   _vector(D, "D", heads, torch.float32, dev), *_optional(z),
                   _vector(dt_bias, "dt_bias", heads, torch.float32, dev),
                   _vector(slots, "slots", rows, torch.int32, dev),
                   out.data_ptr(), *out.stride(), 1 if delta_softplus else 0, 0)
    if rows:
        _launch(_lib.lib().mss_head_scan_step, a, dev)
    return out


def _rows(t, name, shape, dtype, device):
    """A matrix's address and the distance of its rows."""
    _like(t, name, shape, dtype, device)
    rows, cols = t.stride()
    if cols != 1 and shape[1] > 1:
        raise ValueError(f"{name} must have unit stride in its columns")
    return t.data_ptr(), rows


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
    dev = _gpu(x, "x")
    if x.dim() != 2:
        raise ValueError(f"x must have 2 dimensions, got shape {tuple(x.shape)}")
    if quant not in _QUANT:
        raise ValueError(f"quant must be None, 'row' or 'block', got {quant!r}")
    shape = x.shape
    rows, dim = shape
    out = _out(out, x, x.dtype if quant is None else torch.float8_e4m3fn, dev)
    left, scales, res, res_type = (out,), 0, (0, 0, 0, 0), _io(x)
    if quant is not None:
        if quant == "block" and dim % _lib.MSS_SCALE_BLOCK:
            raise ValueError(f"quant 'block' needs a multiple of {_lib.MSS_SCALE_BLOCK} columns, got {dim}")
        want = (rows, 1 if quant == "row" else dim // _lib.MSS_SCALE_BLOCK)
        if scale is None:
            scale = torch.empty_strided(want, (want[1], 1), dtype=torch.float32, device=dev)
        elif not _like(scale, "scale", want, torch.float32, dev).is_contiguous():
            raise ValueError("scale must be contiguous")
        scales = scale.data_ptr()
        left = (out, scale)
    elif scale is not None:
        raise ValueError("scale is given without quant")
    if residual is not None:
        if not isinstance(residual, _Tensor):
            raise TypeError("residual must be a torch.Tensor")
        res_type = _io(residual)
        res = _rows(residual, "residual", shape, residual.dtype, dev)
        if residual_out is None:
            residual_out = torch.empty_like(residual, memory_format=torch.contiguous_format)
        res += _rows(residual_out, "residual_out", shape, residual.dtype, dev)
        left += (residual_out,)
    elif residual_out is not None:
        raise ValueError("residual_out is given without residual")
    a = _norm_args(_io(x), res_type, _QUANT[quant], rows, dim, *_rows(x, "x", shape, x.dtype, dev),
                   *res[:2], _vector(weight, "weight", dim, torch.float32, dev),
                   *_rows(out, "out", shape, out.dtype, dev), scales, *res[2:], eps, 0)
    if rows:
        _launch(_lib.lib().mss_rms_norm, a, dev)
    return left if len(left) > 1 else out
