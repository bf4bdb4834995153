"""The head-wise operations at their edges: magnitudes, time steps and decays far
from those of a trained layer (what the recurrence gives in 64 bits is what the
chunked form has to give, within the bounds of test_head_ops), calls of no rows,
offsets outside the rules.
"""

import ctypes
import math

import pytest
import torch

import head_ref as ref
from test_head_ops import DT, crowd, gen, ints, mss, randn, scan_check, scan_inputs  # noqa: F401

pytestmark = pytest.mark.gpu

# powers of two a token decays by: 16 tokens of them are at most 2^64 (4), 2^100
# (6, 6.2) and more (6.3, 7)
POWERS = (4.0, 5.0, 6.0, 6.2, 6.3, 7.0)


def fast_decay_inputs(lens, io, headdim, dstate, size, constant):
    """Heads whose every token decays by 2^-POWERS[h], from a zero state, with x,
    B and C of magnitude ``size``: random, or the same everywhere."""
    heads = len(POWERS)
    v, c = scan_inputs(gen(31), lens, heads, headdim, dstate, 1, io)
    v["A_log"] = torch.tensor([math.log(p * math.log(2.0)) for p in POWERS], device="cuda")
    v["dt_raw"].fill_(1.0)
    v["dt_bias"] = v["D"] = None  # (D x would hide the sums over tokens)
    for name in ("x", "B", "C"):
        v[name] = torch.full_like(v[name], size) if constant else v[name] * size
    c["resume"] = None
    return v, c


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("wide", [False, True], ids=["tiles16", "tiles32"])
@pytest.mark.parametrize("size", [1e-9, 1e-5, 1e3, 1e9])
@pytest.mark.parametrize("headdim,dstate", [(8, 8), (32, 128)])
def test_scan_magnitudes_under_fast_decay(mss, headdim, dstate, size, wide, io):  # noqa: F811
    lens = (100, 33)
    for constant in (False, True):
        v, c = fast_decay_inputs(crowd(lens, len(POWERS), headdim, 1) if wide else lens, io, headdim, dstate, size,
                                 constant)
        scan_check(mss, f"scan of {size:g} P={headdim} N={dstate} {io} {constant}", v, c, softplus=False)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_scan_magnitudes_under_fast_decay_cut(mss, io):  # noqa: F811
    """Prompts cut over time, and rows that are no whole vectors."""
    for lens, headdim, dstate in (((700, 5), 32, 64), ((700,), 5, 9)):
        v, c = fast_decay_inputs(lens, io, headdim, dstate, 1e4, False)
        scan_check(mss, f"scan of 1e4 cut P={headdim} {io}", v, c, softplus=False)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_scan_tiny_time_steps_among_fast_decay(mss, io):  # noqa: F811
    """A time step far below the others of its chunk keeps its precision: three
    outputs come from it alone."""
    v, c = fast_decay_inputs((64, 48, 20, 70), io, 16, 16, 1.0, False)
    for at, dt in ((0, 1e-12), (64, 1e-20), (112, 1e-28), (132, 1e-9)):
        v["dt_raw"][at] = dt
        v["x"][at + 1:at + 3] = 0
    scan_check(mss, f"scan of tiny steps {io}", v, c, softplus=False)


@pytest.mark.parametrize("wide", [False, True], ids=["tiles16", "tiles32"])
@pytest.mark.parametrize("lens,heads,headdim,dstate", [((130, 1, 64), 3, 64, 128), ((700, 9), 2, 40, 24),
                                                       ((70,), 3, 33, 20)], ids=str)
def test_scan_bf16_outputs_are_rounded_once(mss, lens, heads, headdim, dstate, wide):  # noqa: F811
    """bf16 outputs are off by their own rounding and 2^-16 of the terms they are a
    sum of, however much those cancel: an operand kept as two bf16 parts is off by
    2^-8 of 2^-8."""
    v, c = scan_inputs(gen(35), crowd(lens, heads, headdim, 1) if wide else lens, heads, headdim, dstate, 1, "bf16")
    args = tuple(v.values())
    want, _ = ref.scan_prompts(*args, c["cu"], c["state"], c["slots"], c["resume"])
    mag, _ = ref.scan_prompts(*args, c["cu"], c["state"], c["slots"], c["resume"], absolute=True)
    got = mss.head_scan_prompts(*args, cu_seqlens=c["cu"], state=c["state"], slots=c["slots"], resume=c["resume"])
    torch.cuda.synchronize()
    k = (2 * max(lens) + dstate + 8) * 2.0 ** -24
    ref.within(f"scan rounded once {lens} {wide}", got, want, (k + 2.0 ** -16) * mag + 2.0 ** -8 * 1.01 * want.abs())


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("lens", [(150, 9), (700, 40)], ids=str)
def test_scan_from_infinite_states(mss, lens, io):  # noqa: F811
    """Infinite and huge entries of a cached state reach the outputs as they are."""
    v, c = scan_inputs(gen(36), lens, 2, 40, 24, 1, io, rates=(-6.0, -5.0))
    c["resume"] = torch.ones(2, dtype=torch.int32, device="cuda")
    c["state"][:, 0, 3, 5] = float("inf")
    c["state"][:, 0, 7, 5] = float("-inf")
    c["state"][:, 1, 9, 2] = 3.4e38
    v["B"].abs_()
    v["C"].fill_(0.5)
    v["x"].abs_()
    state = c["state"].clone()
    want, wstate = ref.scan_prompts(*v.values(), c["cu"], c["state"], c["slots"], c["resume"])
    got = mss.head_scan_prompts(*v.values(), cu_seqlens=c["cu"], state=state, slots=c["slots"], resume=c["resume"])
    torch.cuda.synchronize()
    assert torch.isinf(want).any()
    # (an output past its type's range is an infinity)
    for what, x, y in (("out", ref.d(got), want.to(got.dtype)), ("state", ref.d(state), wstate)):
        for test in (torch.isnan, torch.isposinf, torch.isneginf):
            wrong = int((test(x) != test(y)).sum())
            assert wrong == 0, f"{wrong} values of {what} differ in {test.__name__}"


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("lens,at", [((100,), 37), ((700, 40), 300), ((100,) + (0,) * 600, 37),
                                     ((700, 40) + (0,) * 600, 300)], ids=lambda v: str(v)[:12])
def test_scan_past_an_infinite_time_step(mss, lens, at, io):  # noqa: F811
    """An infinite time step makes the states infinite, not NaN, and tokens before
    it as they are without it."""
    v, c = scan_inputs(gen(32), lens, 2, 40, 24, 1, io)
    c["resume"] = None
    v["D"] = None
    clean = mss.head_scan_prompts(*v.values(), cu_seqlens=c["cu"], state=c["state"].clone(), slots=c["slots"])
    v["dt_raw"][at, 0] = float("inf")
    state = c["state"].clone()
    got = mss.head_scan_prompts(*v.values(), cu_seqlens=c["cu"], state=state, slots=c["slots"])
    want, wstate = ref.scan_prompts(*v.values(), c["cu"], c["state"], c["slots"])
    torch.cuda.synchronize()
    got, state, clean = ref.d(got), ref.d(state), ref.d(clean)
    assert torch.isinf(wstate[int(c["slots"][0]), 0]).all()
    for what, x, y in (("out", got, want), ("state", state, wstate)):
        for test in (torch.isnan, torch.isposinf, torch.isneginf):
            wrong = int((test(x) != test(y)).sum())
            assert wrong == 0, f"{wrong} values of {what} differ in {test.__name__}"
    # the same sums, a chunk's in another order
    ref.within("before", got[:at], clean[:at], 2.0 ** -6 * clean[:at].abs().amax((0, 2), True))


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("lens", [(64, 20), (700,), (64, 20) + (0,) * 600], ids=lambda v: str(v)[:12])
def test_scan_growth_from_nothing(mss, lens, io):  # noqa: F811
    """Negative time steps, whose decays pass the largest fp32 over a chunk, and no
    input but in the last tokens: a zero state stays zero until then."""
    v, c = scan_inputs(gen(33), lens, 2, 40, 24, 1, io)
    c["resume"] = None
    v["A_log"].zero_()
    v["dt_raw"].fill_(-3.0)
    v["dt_bias"] = None
    end = lens[0]
    v["x"][:end - 4] = 0
    scan_check(mss, f"scan of growth {io}", v, c, softplus=False)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_scan_rate_past_fp32(mss, io):  # noqa: F811
    """A decay rate that overflows fp32 leaves each token by itself, as it does in
    the step."""
    v, c = scan_inputs(gen(34), (70, 9), 2, 40, 24, 1, io)
    c["resume"] = None
    v["A_log"] = torch.tensor([100.0, 0.5], device="cuda")
    scan_check(mss, f"scan of a rate past fp32 {io}", v, c)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_no_rows(mss, io):  # noqa: F811
    """A step and a norm of no rows, as a server's empty batch makes them, next to
    a conv and a scan of no tokens: empty outputs, caches as they were."""
    g, dt = gen(26), DT[io]
    state, window = randn(g, 3, 2, 8, 16), randn(g, 3, 48, 3, dtype=dt)
    kept = state.clone(), window.clone()
    v = dict(A_log=randn(g, 2), weight=randn(g, 48, 4), bias=randn(g, 48), D=randn(g, 2))
    y = mss.head_scan_step(state, window, randn(g, 0, 48, dtype=dt), randn(g, 0, 2, dtype=dt), *v.values(),
                           randn(g, 0, 2, 8, dtype=dt), slots=ints())
    assert y.shape == (0, 2, 8) and y.dtype is dt
    assert torch.equal(state, kept[0]) and torch.equal(window, kept[1])
    x, w = randn(g, 0, 256, dtype=dt), randn(g, 256)
    assert mss.rms_norm(x, w).shape == (0, 256)
    for quant, cols in (("row", 1), ("block", 2)):
        q, scale, left = mss.rms_norm(x, w, residual=randn(g, 0, 256), quant=quant)
        assert q.shape == (0, 256) and q.dtype is torch.float8_e4m3fn
        assert scale.shape == (0, cols) and left.shape == (0, 256)
    with pytest.raises(ValueError, match="weight"):
        mss.rms_norm(x, w[:255])
    torch.cuda.synchronize()


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("off", [1024, 1023], ids=["vectors", "elements"])
def test_offsets_outside_the_rules_stay_in_their_buffers(mss, off, io):  # noqa: F811
    """cu_seqlens that runs backwards, starts late or ends past the rows: what lies
    around the outputs, caches and workspace, the entries of no prompt and the
    inputs are as they were."""
    from mamba_selective_scan_amd import _lib
    heads, headdim, dstate, tokens, dim, dt = 2, 64, 64, 1200, 40, DT[io]
    v, c = scan_inputs(gen(37), (400, 300, 500), heads, headdim, dstate, 1, io)
    x, w = randn(gen(38), tokens, dim, dtype=dt), randn(gen(38), dim, 4)
    slots = ints(4, 0, 2)
    a = _lib.HeadScanArgs(struct_size=ctypes.sizeof(_lib.HeadScanArgs), io_dtype=_lib.MSS_F32 if io == "f32" else
                          _lib.MSS_BF16, tokens=tokens, heads=heads, headdim=headdim, dstate=dstate, groups=1, seqs=3,
                          cache_slots=6)
    need = _lib.lib().mss_head_scan_prompts_workspace_size(ctypes.byref(a), None)
    assert need > 0
    kept = [t.clone() for t in (*v.values(), x, w)]

    def between(*shape, dtype):
        """A tensor inside a larger one of sevens."""
        n = math.prod(shape)
        whole = torch.full((n + 2 * off,), 7, dtype=dtype, device="cuda")
        return whole, whole[off:off + n].view(shape)

    for cu in ((0, 1200, 0, 1200), (-7, 700, 300, 5000), (5000, 5000, 5000, 5000), (30, 40, 1100, 1150),
               (1200, 0, 1200, 0), (-(1 << 31), (1 << 31) - 1, -(1 << 31), (1 << 31) - 1)):
        held = [between(tokens, heads, headdim, dtype=dt), between(6, heads, headdim, dstate, dtype=torch.float32),
                between(tokens, dim, dtype=dt), between(6, dim, 3, dtype=dt)]
        work = torch.full((need + 4096,), 7, dtype=torch.uint8, device="cuda")
        out, state, u, window = (inner for _, inner in held)
        mss.head_scan_prompts(*v.values(), cu_seqlens=ints(*cu), state=state, slots=slots, out=out, workspace=work)
        mss.causal_conv1d_prompts(x, w, cu_seqlens=ints(*cu), window=window, slots=slots, out=u)
        torch.cuda.synchronize()
        for whole, _ in held:
            assert (whole[:off] == 7).all() and (whole[-off:] == 7).all(), cu
        assert (work[need:] == 7).all(), cu
        for cache in (state, window):
            assert (cache[1] == 7).all() and (cache[3] == 7).all() and (cache[5] == 7).all(), cu
        assert all(torch.equal(a, b) for a, b in zip(kept, (*v.values(), x, w))), cu


@pytest.mark.parametrize("quant", [None, "row", "block"])
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("dim", [256, 4096, 9088])
def test_norm_of_rows_whose_squares_leave_fp32(mss, dim, io, quant):  # noqa: F811
    """Rows so large that their squares pass fp32, and, without eps, so small that
    they vanish, next to ordinary ones: the norm is what it is for any row."""
    dt, E = DT[io], 2.0 ** -24
    x = randn(gen(39), 6, dim)
    for row, size in enumerate((1e19, 1.0, 1e36, 1e-20, 1e-36)):
        x[row] *= size
    x[5] = 3e38
    x, weight = x.to(dt), randn(gen(40), dim)
    y, _ = ref.rms_norm(x, weight, eps=0.0)
    got = mss.rms_norm(x, weight, eps=0.0, quant=quant)
    torch.cuda.synchronize()
    k = (dim + 8) * E  # the mean square's sum, then a few roundings
    if quant is None:
        ref.within(f"norm {dim} {io}", got, y, (k + ref.HALF[dt] * 1.01) * y.abs())
        return
    q, scale = got
    wide = 128 if quant == "block" else dim
    want = y.unflatten(1, (-1, wide)).abs().amax(2) / 448
    ref.within(f"norm {dim} {io} {quant} scale", scale.reshape(want.shape), want, 2 * (k + 4 * E) * want)
    s = ref.d(scale).reshape(want.shape).repeat_interleave(wide, 1)
    bound = torch.maximum(2.0 ** -4 * y.abs(), 2.0 ** -10 * s) * 1.001
    ref.within(f"norm {dim} {io} {quant} values", ref.d(q.float()) * s, y, bound)
