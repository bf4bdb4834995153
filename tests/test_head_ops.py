"""The head-wise operations on the GPU against their plain 64-bit forms.

Bounds, each relative to the sums of absolute values that a result comes from
(head_ref): an fp32 sum of k terms is off by at most (k + 8) 2^-24 of it, where
the 8 covers the products, softplus, exp and silu of a term (a few 2^-24 each);
a term that is rounded to bf16 once, by 2^-8.  An output rounded to its type is
off by half a step of its own value besides.  Windows are copies and are exact.
"""

import pytest
import torch

import head_ref as ref
from gpu_util import note

pytestmark = pytest.mark.gpu

E = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def mss():
    assert torch.cuda.is_available(), "GPU tests need a visible GPU"
    import mamba_selective_scan_amd as m
    return m


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def offsets(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return torch.tensor(cu, dtype=torch.int32, device="cuda")


def ints(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


# lengths: single tokens, empty prompts, every place around a chunk's border
LENGTHS = [(1,), (0, 1, 0), (3, 0, 2, 1), (63,), (64,), (65, 1), (200, 0, 1, 129, 15)]


# ------------------------------------------------------------------------ conv

def conv_case(mss, lens, dim, io, *, width=4, bias=True, act=True, resume=True, extra=0, layout=None,
              seed=0):
    g = gen(seed)
    dt, n = DT[io], len(lens)
    t = sum(lens) + extra
    if layout == "wide":      # rows of a wider buffer, at an odd column
        x = randn(g, t, dim + 13, dtype=dt)[:, 5:5 + dim]
    elif layout == "strided":  # every other column
        x = randn(g, t, 2 * dim, dtype=dt)[:, ::2]
    elif layout == "tfast":   # channels first
        x = randn(g, dim, t, dtype=dt).t()
    else:
        x = randn(g, t, dim, dtype=dt)
    weight, b = randn(g, dim, width), randn(g, dim) if bias else None
    window = randn(g, n + 3, dim, width - 1, dtype=dt)
    slots = torch.randperm(n + 3, generator=g, device="cuda")[:n].to(torch.int32)
    res = ints(*[i % 2 for i in range(n)]) if resume else None
    cu = offsets(lens)
    out = randn(g, t, dim, dtype=dt)
    want, wwin, mag = ref.conv_prompts(x, weight, b, cu, window, slots, res, act, out)
    got = mss.causal_conv1d_prompts(x, weight, b, cu_seqlens=cu, window=window, slots=slots,
                                    resume=res, activation="silu" if act else None, out=out)
    torch.cuda.synchronize()
    assert got.data_ptr() == out.data_ptr()
    # silu's slope is at most 1.1
    bound = 1.1 * (width + 8) * E * mag + ref.HALF[dt] * want.abs()
    ref.within(f"conv {lens} {dim} {io} {layout}", got, want, bound)
    assert torch.equal(ref.d(window), wwin)
    assert torch.equal(ref.d(got)[sum(lens):], want[sum(lens):])


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("lens", LENGTHS)
def test_conv_lengths(mss, lens, io):
    conv_case(mss, lens, 264, io, extra=3)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("dim", [1, 7, 33, 513, 1001])
def test_conv_odd_dims(mss, dim, io):
    conv_case(mss, (5, 70, 1, 0, 40), dim, io)


@pytest.mark.parametrize("layout", ["wide", "strided", "tfast"])
def test_conv_strides(mss, layout):
    conv_case(mss, (9, 33), 130, "bf16", layout=layout, extra=2)
    conv_case(mss, (9, 33), 130, "f32", layout=layout)


@pytest.mark.parametrize("width", [1, 2, 3])
def test_conv_widths_and_options(mss, width):
    conv_case(mss, (1, 2, 0, 50), 96, "f32", width=width, bias=False, act=False)
    conv_case(mss, (1, 2, 0, 50), 96, "bf16", width=width, resume=False)


def test_conv_many_prompts(mss):
    # more prompts than one count of 64, runs that cross many of them
    lens = tuple((7 * i) % 5 for i in range(300))
    conv_case(mss, lens, 40, "f32")


# ------------------------------------------------------------------------ scan

def scan_inputs(g, lens, heads, headdim, dstate, groups, io, *, gate=True, extra=0, rates=(0.0, 2.7)):
    dt, n = DT[io], len(lens)
    t = sum(lens) + extra
    v = dict(x=randn(g, t, heads, headdim, dtype=dt), dt_raw=randn(g, t, heads, dtype=dt),
             A_log=torch.linspace(rates[0], rates[1], heads, device="cuda"),
             B=randn(g, t, groups, dstate, dtype=dt), C=randn(g, t, groups, dstate, dtype=dt),
             D=randn(g, heads), z=randn(g, t, heads, headdim, dtype=dt) if gate else None,
             dt_bias=randn(g, heads) - 2)
    c = dict(cu=offsets(lens), state=randn(g, n + 2, heads, headdim, dstate),
             slots=torch.randperm(n + 2, generator=g, device="cuda")[:n].to(torch.int32),
             resume=ints(*[(i + 1) % 2 for i in range(n)]))
    return v, c


def scan_check(mss, name, v, c, *, softplus=True, out=None, workspace=None):
    io = v["x"].dtype
    args = (v["x"], v["dt_raw"], v["A_log"], v["B"], v["C"], v["D"], v["z"], v["dt_bias"])
    out = torch.full_like(v["x"], 7.0, memory_format=torch.contiguous_format) if out is None else out
    want, wstate = ref.scan_prompts(*args, c["cu"], c["state"], c["slots"], c["resume"], softplus, out)
    mag, smag = ref.scan_prompts(*args, c["cu"], c["state"], c["slots"], c["resume"], softplus,
                                 absolute=True)
    got = mss.head_scan_prompts(*args, cu_seqlens=c["cu"], state=c["state"], slots=c["slots"],
                                resume=c["resume"], delta_softplus=softplus, out=out,
                                workspace=workspace)
    torch.cuda.synchronize()
    longest = max(b - a for a, b in ref.spans(c["cu"]))
    # a state is a sum over the prompt's tokens, an output one over its states
    # too; a decay's exponent is a sum over the tokens itself
    k = (2 * longest + v["B"].shape[2] + 8) * E
    # bf16 inputs: the two operands of the products that make an output (the
    # decayed weights, the entering state) are rounded to bf16 once
    terms = 2.0 ** -8 if io == torch.bfloat16 else 0.0
    ref.within(f"{name} out", got, want, (k + terms) * mag + ref.HALF[io] * want.abs() * 1.01)
    ref.within(f"{name} state", c["state"], wstate, k * smag)
    end = int(c["cu"][-1])
    assert torch.equal(ref.d(got)[end:], want[end:])
    return got


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("lens", LENGTHS)
def test_scan_lengths(mss, lens, io):
    v, c = scan_inputs(gen(1), lens, 6, 64, 128, 2, io, extra=2)
    scan_check(mss, f"scan {lens} {io}", v, c)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("lens,heads,headdim,dstate", [((1500, 3, 700, 0, 257), 3, 64, 128), ((513,), 2, 33, 20),
                                                       ((2305, 256, 257), 1, 32, 64)])
def test_scan_cut_over_time(mss, lens, heads, headdim, dstate, io):
    """Prompts long enough to run as segments, next to some that are not."""
    v, c = scan_inputs(gen(9), lens, heads, headdim, dstate, 1, io, extra=1, rates=(-2.0, 2.0))
    scan_check(mss, f"scan cut {lens} {io}", v, c)
    c["resume"] = c["slots"] = None
    scan_check(mss, f"scan cut fresh {lens} {io}", v, c)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("lens,at", [((100,), 37), ((700, 40), 300), ((100,) + (0,) * 600, 37),
                                     ((700, 40) + (0,) * 600, 300)], ids=lambda v: str(v)[:12])
def test_scan_is_causal_past_nan_and_infinity(mss, lens, at, io):
    """What follows an infinity or a NaN in x or B is what the recurrence gives;
    what comes before it is as without it."""
    v, c = scan_inputs(gen(10), lens, 2, 40, 24, 1, io)
    c["resume"] = None
    v["D"] = None
    args = lambda: (v["x"], v["dt_raw"], v["A_log"], v["B"], v["C"], v["D"], v["z"], v["dt_bias"])  # noqa: E731
    clean = mss.head_scan_prompts(*args(), cu_seqlens=c["cu"], state=c["state"].clone(), slots=c["slots"])
    for name, index, value in [("x", (at, 1, 3), float("nan")), ("x", (at, 1, 3), float("inf")),
                               ("B", (at, 0, 5), float("-inf")), ("C", (at, 0, 5), float("inf")),
                               ("dt_raw", (at, 0), float("nan"))]:
        kept = v[name].clone()
        v[name][index] = value
        state = c["state"].clone()
        got = mss.head_scan_prompts(*args(), cu_seqlens=c["cu"], state=state, slots=c["slots"])
        want, wstate = ref.scan_prompts(*args(), c["cu"], c["state"], c["slots"])
        torch.cuda.synchronize()
        got, state, clean_ = ref.d(got), ref.d(state), ref.d(clean)
        for what, x, y in (("out", got, want), ("state", state, wstate)):
            for test in (torch.isnan, torch.isinf):
                wrong = int((test(x) != test(y)).sum())
                assert wrong == 0, f"{name} {value}: {wrong} values of {what} differ in {test.__name__}"
        # the same sums, a chunk's in another order
        ref.within(f"{name} {value} before", got[:at], clean_[:at], 2.0 ** -6 * clean_[:at].abs().amax((0, 2), True))
        v[name].copy_(kept)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("heads,headdim,dstate,groups",
                         [(1, 1, 1, 1), (3, 5, 7, 3), (5, 33, 17, 1), (4, 48, 64, 4), (2, 130, 100, 1),
                          (7, 64, 16, 7), (9, 32, 128, 3), (8, 96, 24, 2)])
def test_scan_shapes(mss, heads, headdim, dstate, groups, io):
    v, c = scan_inputs(gen(2), (70, 1, 131), heads, headdim, dstate, groups, io)
    scan_check(mss, f"scan H={heads} P={headdim} N={dstate} G={groups} {io}", v, c)


def crowd(lens, heads, headdim, groups):
    """With so many empty prompts that the call's workgroups, four tiles of 32
    columns each, fill the card: it keeps those tiles, where a small call takes
    tiles of 16."""
    tiles = groups * -(-heads // groups * -(-headdim // 32) // 4)
    return (*lens, *(0,) * (768 // tiles))


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("lens", [(70, 1, 131), (64, 200)], ids=str)
@pytest.mark.parametrize("heads,headdim,dstate,groups",
                         [(4, 48, 64, 4), (7, 64, 16, 7), (9, 32, 128, 3), (8, 96, 24, 2), (6, 64, 128, 2),
                          (3, 40, 32, 1), (5, 8, 8, 1)])
def test_scan_many_prompts(mss, heads, headdim, dstate, groups, lens, io):
    v, c = scan_inputs(gen(22), crowd(lens, heads, headdim, groups), heads, headdim, dstate, groups, io, extra=2)
    scan_check(mss, f"scan crowd H={heads} P={headdim} N={dstate} G={groups} {io}", v, c)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("heads,headdim,dstate,lens", [(3, 64, 128, (1500, 3, 700, 0, 257)), (1, 32, 64, (1025, 321))],
                         ids=str)
def test_scan_many_prompts_cut_over_time(mss, heads, headdim, dstate, lens, io):
    v, c = scan_inputs(gen(23), crowd(lens, heads, headdim, 1), heads, headdim, dstate, 1, io, rates=(-2.0, 2.0))
    scan_check(mss, f"scan crowd cut {io}", v, c)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_scan_many_prompts_fast_decay(mss, io):
    v, c = scan_inputs(gen(24), crowd((150, 64), 6, 32, 1), 6, 32, 32, 1, io, rates=(-12.0, 6.0))
    scan_check(mss, f"scan crowd decays {io}", v, c)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("headdim,dstate", [(8, 8), (16, 16), (24, 40), (72, 128), (80, 64)])
def test_scan_small_tiles(mss, headdim, dstate, io):
    """Columns that end inside a tile of 16, whole and cut over time."""
    v, c = scan_inputs(gen(25), (70, 330, 2), 2, headdim, dstate, 1, io)
    scan_check(mss, f"scan tiles P={headdim} N={dstate} {io}", v, c)
    v, c = scan_inputs(gen(25), (400,), 2, headdim, dstate, 1, io)
    scan_check(mss, f"scan tiles cut P={headdim} N={dstate} {io}", v, c)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_scan_options(mss, io):
    v, c = scan_inputs(gen(3), (90, 20), 4, 64, 64, 1, io, gate=False)
    v["D"] = v["dt_bias"] = None
    scan_check(mss, f"scan bare {io}", v, c)
    v, c = scan_inputs(gen(3), (90, 20), 4, 64, 64, 1, io)
    v["dt_raw"] = v["dt_raw"].abs() * 0.1
    v["dt_bias"] = None
    scan_check(mss, f"scan without softplus {io}", v, c, softplus=False)
    c["slots"] = c["resume"] = None
    scan_check(mss, f"scan default slots {io}", v, c)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_scan_fast_and_slow_decay(mss, io):
    # decays from none at all to below the smallest fp32 within a few tokens
    v, c = scan_inputs(gen(4), (150, 64), 6, 32, 32, 1, io, rates=(-12.0, 6.0))
    scan_check(mss, f"scan decays {io}", v, c)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_scan_views(mss, io):
    """x, B and C as column ranges of one buffer at odd offsets, out and z rows
    of wider buffers, a cache with other layers between its slots."""
    g = gen(5)
    lens, heads, headdim, dstate, groups = (77, 40), 3, 40, 24, 1
    v, c = scan_inputs(g, lens, heads, headdim, dstate, groups, io)
    t, n = sum(lens), heads * headdim
    rows = randn(g, t, 3 + n + 2 * groups * dstate, dtype=DT[io])
    v["x"] = rows[:, 3:3 + n].unflatten(1, (heads, headdim))
    v["B"] = rows[:, 3 + n:3 + n + groups * dstate].unflatten(1, (groups, dstate))
    v["C"] = rows[:, 3 + n + groups * dstate:].unflatten(1, (groups, dstate))
    v["z"] = randn(g, t, heads, headdim + 7, dtype=DT[io])[:, :, 3:3 + headdim]
    v["dt_raw"] = randn(g, heads, t, dtype=DT[io]).t()
    out = randn(g, t, heads, headdim + 1, dtype=DT[io])[:, :, 1:]
    c["state"] = randn(g, 4, 3, heads, headdim, dstate)[:, 1]
    scan_check(mss, f"scan views {io}", v, c, out=out)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_one_token_has_any_row_stride(mss, io):
    """The token stride of a single token means nothing, however large."""
    v, c = scan_inputs(gen(21), (1,), 2, 64, 64, 1, io)
    for name in ("x", "B", "C", "z"):
        shape = v[name].shape
        v[name] = v[name].as_strided(shape, (1 << 24, shape[2], 1))
    scan_check(mss, f"scan one token {io}", v, c)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_caches_at_odd_addresses(mss, io):
    """Entries of an odd number of elements, with others between them: states and
    windows at any element."""
    g = gen(17)
    heads, headdim, dstate, groups = 3, 5, 7, 3
    v, c = scan_inputs(g, (70, 9), heads, headdim, dstate, groups, io)
    c["state"] = randn(g, 4, 3, heads, headdim, dstate)[:, 1]
    scan_check(mss, f"scan odd entries {io}", v, c)
    chans = heads * headdim + 2 * groups * dstate
    state, window = c["state"], randn(g, 4, 3, chans, 3, dtype=DT[io])[:, 1]
    xbc, dt_raw = randn(g, 2, chans, dtype=DT[io]), randn(g, 2, heads, dtype=DT[io])
    weight = randn(g, chans, 4)
    want, ws, ww, mag, smag = ref.step(state, window, xbc, dt_raw, v["A_log"], weight, None, None, None, None,
                                       groups, c["slots"])
    got = mss.head_scan_step(state, window, xbc, dt_raw, v["A_log"], weight, slots=c["slots"])
    k = 1.21 * (2.2 * 12 + dstate + 8) * E
    ref.within(f"step odd entries {io} out", got, want, k * mag + ref.HALF[DT[io]] * want.abs() * 1.01)
    ref.within(f"step odd entries {io} state", state, ws, k * smag)
    assert torch.equal(ref.d(window), ww)


def test_offsets_outside_the_rules(mss):
    """cu_seqlens that runs backwards, starts late or ends past the rows: results
    of no meaning, rows and entries in their places."""
    v, c = scan_inputs(gen(18), (400, 300, 500), 2, 64, 64, 1, "bf16")
    x, w = randn(gen(18), 1200, 40), randn(gen(18), 40, 4)
    for cu in ((0, 1200, 0, 1200), (-7, 700, 300, 5000), (5000, 5000, 5000, 5000), (30, 40, 1100, 1150)):
        out = mss.head_scan_prompts(v["x"], v["dt_raw"], v["A_log"], v["B"], v["C"], cu_seqlens=ints(*cu),
                                    state=c["state"], slots=c["slots"])
        u = mss.causal_conv1d_prompts(x, w, cu_seqlens=ints(*cu), window=randn(gen(18), 5, 40, 3))
        torch.cuda.synchronize()
        assert out.shape == v["x"].shape and u.shape == x.shape


def test_scan_skips_and_keeps(mss):
    """Prompts without an entry leave rows and caches as they were; entries of
    no prompt stay."""
    v, c = scan_inputs(gen(6), (30, 70, 5, 64), 4, 64, 128, 1, "bf16", extra=9)
    c["slots"] = ints(3, -1, 99, 0)
    scan_check(mss, "scan skips", v, c)
    dim = 70
    g = gen(6)
    x, window = randn(g, 178, dim), randn(g, 6, dim, 3)
    w, out = randn(g, dim, 4), randn(g, 178, dim)
    want, wwin, mag = ref.conv_prompts(x, w, None, c["cu"], window, c["slots"], None, True, out)
    mss.causal_conv1d_prompts(x, w, cu_seqlens=c["cu"], window=window, slots=c["slots"], out=out)
    ref.within("conv skips", out, want, 16 * E * mag + E * want.abs())
    assert torch.equal(ref.d(window), wwin)


def test_scan_without_tokens(mss):
    v, c = scan_inputs(gen(7), (0, 0), 2, 32, 16, 1, "f32")
    before = c["state"].clone()
    mss.head_scan_prompts(v["x"], v["dt_raw"], v["A_log"], v["B"], v["C"], cu_seqlens=c["cu"],
                          state=c["state"], slots=c["slots"], resume=c["resume"])
    before[int(c["slots"][1])] = 0
    assert torch.equal(c["state"], before)
    window = randn(gen(7), 4, 8, 3)
    kept = window.clone()
    mss.causal_conv1d_prompts(randn(gen(7), 0, 8), randn(gen(7), 8, 4), cu_seqlens=c["cu"],
                              window=window, slots=c["slots"], resume=c["resume"])
    kept[int(c["slots"][1])] = 0
    assert torch.equal(window, kept)


def test_scan_nan_stays_in_its_prompt(mss):
    """A prompt that holds a NaN or an infinity leaves the others as they are,
    in the same chunk of rows or not, and a fresh prompt ignores a NaN in its
    cache entry."""
    v, c = scan_inputs(gen(8), (20, 50, 3), 3, 64, 64, 1, "bf16")
    c["resume"] = ints(0, 0, 0)
    c["state"].fill_(float("nan"))
    clean = c["state"].nan_to_num(0.0)
    args = lambda: (v["x"], v["dt_raw"], v["A_log"], v["B"], v["C"], v["D"], v["z"], v["dt_bias"])  # noqa: E731
    want = mss.head_scan_prompts(*args(), cu_seqlens=c["cu"], state=clean, slots=c["slots"])
    v["x"][25, 1] = float("nan")
    v["B"][21] = float("inf")
    v["C"][30] = float("inf")
    got = mss.head_scan_prompts(*args(), cu_seqlens=c["cu"], state=c["state"], slots=c["slots"])
    torch.cuda.synchronize()
    for a, b in ((0, 20), (70, 73)):
        assert torch.equal(got[a:b], want[a:b])
    assert not torch.isfinite(got[30]).any()
    for i in (0, 2):
        s = int(c["slots"][i])
        assert torch.equal(c["state"][s], clean[s])


# ------------------------------------------------------------------------ step

def step_case(mss, rows, heads, headdim, dstate, groups, io, *, width=4, gate=True, slots=True,
              softplus=True, bare=False, seed=0):
    g = gen(seed)
    dt = DT[io]
    chans = heads * headdim + 2 * groups * dstate
    total = rows + 2
    state, window = randn(g, total, heads, headdim, dstate), randn(g, total, chans, width - 1, dtype=dt)
    at = torch.randperm(total, generator=g, device="cuda")[:rows].to(torch.int32)
    if rows > 2:
        at[rows // 2] = -1
    v = dict(xbc=randn(g, rows, chans + 5, dtype=dt)[:, 3:3 + chans], dt_raw=randn(g, rows, heads, dtype=dt),
             A_log=torch.linspace(0, 2.7, heads, device="cuda"), weight=randn(g, chans, width),
             bias=None if bare else randn(g, chans), D=None if bare else randn(g, heads),
             z=randn(g, rows, heads, headdim, dtype=dt) if gate else None,
             dt_bias=None if bare else randn(g, heads) - 2)
    at = at if slots else None
    out = randn(g, rows, heads, headdim, dtype=dt)
    want, ws, ww, mag, smag = ref.step(state, window, *v.values(), groups, at, softplus, out)
    got = mss.head_scan_step(state, window, *v.values(), slots=at, delta_softplus=softplus, out=out)
    torch.cuda.synchronize()
    # the conv's sums of `width` terms, silu's slope of at most 1.1 on each of
    # the two factors, and the sum over the states
    k = (2.2 * (width + 8) + dstate + 8) * E
    name = f"step {rows} H={heads} P={headdim} N={dstate} G={groups} {io}"
    ref.within(name + " out", got, want, 1.21 * k * mag + ref.HALF[dt] * want.abs() * 1.01)
    ref.within(name + " state", state, ws, 1.21 * k * smag)
    assert torch.equal(ref.d(window), ww)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("rows,heads,headdim,dstate,groups",
                         [(1, 24, 64, 128, 1), (1, 1, 1, 1, 1), (5, 3, 7, 5, 3), (9, 4, 48, 64, 4),
                          (3, 2, 130, 100, 1), (33, 6, 64, 16, 2), (4, 5, 40, 33, 1), (2, 8, 512, 24, 8)])
def test_step_shapes(mss, rows, heads, headdim, dstate, groups, io):
    step_case(mss, rows, heads, headdim, dstate, groups, io)


@pytest.mark.parametrize("width", [1, 2, 3])
def test_step_options(mss, width):
    step_case(mss, 4, 2, 32, 16, 1, "f32", width=width, gate=False, bare=True)
    step_case(mss, 4, 2, 32, 16, 1, "bf16", width=width, slots=False)
    step_case(mss, 4, 2, 32, 16, 1, "f32", width=width, softplus=False)


# ------------------------------------------------------------------------ norm

def norm_check(name, got, x, weight, residual, quant, res_dtype):
    y, r = ref.rms_norm(x, weight, residual)
    dim = x.shape[1]
    k = (dim + 8) * E  # the mean square's sum, then a few roundings
    if residual is not None:
        left = got[-1]
        m = ref.d(x).abs() + ref.d(residual).abs()
        ref.within(name + " residual", left, r, E * m + ref.HALF[res_dtype] * r.abs() * 1.01)
        got = got[:-1] if quant else got[0]
        # r itself is off by a rounding of the sum
        near = E * m * (ref.d(weight).abs() / torch.sqrt((r * r).mean(1, keepdim=True) + 1e-5))
    else:
        near = 0.0
    if quant is None:
        got = got[0] if isinstance(got, tuple) else got
        ref.within(name, got, y, k * y.abs() + near + ref.HALF[x.dtype] * y.abs() * 1.01)
        return
    q, scale = got
    wide = 128 if quant == "block" else dim
    top = y.unflatten(1, (-1, wide)).abs().amax(2)
    want = torch.where(top / 448 >= 2.0 ** -126, top / 448, torch.ones_like(top))
    ref.within(name + " scale", scale.reshape(want.shape), want, 2 * (k + 4 * E) * want + 1e-30)
    s = ref.d(scale).reshape(want.shape).repeat_interleave(wide, 1)
    # half a step of e4m3 is 2^-4 of the value, at least 2^-10 of the scale
    bound = torch.maximum(2.0 ** -4 * y.abs(), 2.0 ** -10 * s) * 1.001 + near
    ref.within(name + " values", ref.d(q.float()) * s, y, bound)


@pytest.mark.parametrize("quant", [None, "row", "block"])
@pytest.mark.parametrize("io,res", [("bf16", None), ("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"),
                                    ("f32", "bf16"), ("f32", None)])
@pytest.mark.parametrize("rows,dim", [(1, 128), (3, 640), (5, 1024), (2, 1536), (7, 1920), (2, 2176), (3, 5120),
                                      (2, 8192), (2, 8320), (1, 32768)])
def test_norm(mss, rows, dim, io, res, quant):
    g = gen(dim)
    x, weight = randn(g, rows, dim, dtype=DT[io]), randn(g, dim)
    residual = None if res is None else randn(g, rows, dim, dtype=DT[res], scale=3.0)
    got = mss.rms_norm(x, weight, residual=residual, quant=quant)
    torch.cuda.synchronize()
    norm_check(f"norm {rows}x{dim} {io} {res} {quant}", got, x, weight, residual, quant,
               None if res is None else DT[res])


@pytest.mark.parametrize("quant", [None, "row"])
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("dim", [1, 3, 8, 63, 513, 1537, 2049, 6145, 9001])
def test_norm_odd_columns(mss, dim, io, quant):
    g = gen(dim)
    x = randn(g, 6, dim + 3, dtype=DT[io])[:, 1:1 + dim]
    weight, residual = randn(g, dim), randn(g, 6, dim, dtype=DT[io])
    got = mss.rms_norm(x, weight, residual=residual, quant=quant)
    torch.cuda.synchronize()
    norm_check(f"norm odd {dim} {io} {quant}", got, x, weight, residual, quant, DT[io])


@pytest.mark.parametrize("quant", [None, "row", "block"])
def test_norm_zero_rows_and_in_place(mss, quant):
    g = gen(1)
    x, weight = randn(g, 4, 256), randn(g, 256)
    x[1] = 0
    residual = randn(g, 4, 256)
    residual[1] = 0
    want = residual.clone()
    got = mss.rms_norm(x, weight, residual=residual, residual_out=residual, quant=quant)
    assert got[-1].data_ptr() == residual.data_ptr()
    norm_check(f"norm in place {quant}", got, x, weight, want, quant, torch.float32)
    y = got[0].float()
    assert torch.equal(y[1], torch.zeros(256, device="cuda"))
    if quant:
        assert (got[1][1] == 1).all()


@pytest.mark.parametrize("quant", [None, "row", "block"])
def test_norm_nan_and_infinity(mss, quant):
    g = gen(2)
    x, weight = randn(g, 3, 384, dtype=torch.bfloat16), randn(g, 384)
    alone = mss.rms_norm(x, weight, quant=quant)
    x[0, 5], x[2, 7] = float("nan"), float("inf")
    got = mss.rms_norm(x, weight, quant=quant)
    y, other = (got, alone) if quant is None else (got[0].float(), alone[0].float())
    assert torch.isnan(y[0]).all()
    assert torch.isnan(y[2, 7]) and (y[2, :7] == 0).all() and (y[2, 8:] == 0).all()
    assert torch.equal(y[1], other[1])
    if quant:
        assert (got[1][0] == 1).all() and (got[1][2] == 1).all()


# -------------------------------------------------------------- used together

def test_prompts_then_tokens(mss):
    """Two layers' worth of a run as a server makes it: packed prompts through
    norm, conv and scan, then further tokens through norm and step, against the
    plain forms over the whole sequences, fed the same rounded inputs."""
    g = gen(11)
    heads, headdim, dstate, groups, more = 4, 32, 64, 2, 5
    n, chans = heads * headdim, heads * headdim + 2 * groups * dstate
    lens = (70, 1, 0, 33)
    t = sum(lens)
    weight, bias = randn(g, chans, 4), randn(g, chans)
    A_log, D, dt_bias = torch.linspace(0, 2.7, heads, device="cuda"), randn(g, heads), randn(g, heads) - 2
    window = torch.full((6, chans, 3), float("nan"), device="cuda")
    state = torch.full((6, heads, headdim, dstate), float("nan"), device="cuda")
    cu, slots = offsets(lens), ints(4, 0, 2, 1)
    xbc = mss.rms_norm(randn(g, t, chans), randn(g, chans))
    dt_raw, z = randn(g, t, heads), randn(g, t, heads, headdim)
    u = mss.causal_conv1d_prompts(xbc, weight, bias, cu_seqlens=cu, window=window, slots=slots)
    y = mss.head_scan_prompts(u[:, :n].unflatten(1, (heads, headdim)), dt_raw, A_log,
                              u[:, n:n + groups * dstate].unflatten(1, (groups, dstate)),
                              u[:, n + groups * dstate:].unflatten(1, (groups, dstate)), D, z, dt_bias,
                              cu_seqlens=cu, state=state, slots=slots)
    tokens = []
    for _ in range(more):
        xt = mss.rms_norm(randn(g, len(lens), chans), randn(g, chans))
        dtt, zt = randn(g, len(lens), heads), randn(g, len(lens), heads, headdim)
        tokens.append((xt, dtt, zt, mss.head_scan_step(state, window, xt, dtt, A_log, weight, bias, D, zt,
                                                       dt_bias, slots=slots)))
    torch.cuda.synchronize()
    for i, (a, b) in enumerate(ref.spans(cu)):
        x_all = torch.cat([xbc[a:b]] + [v[0][i:i + 1] for v in tokens])
        dt_all = torch.cat([dt_raw[a:b]] + [v[1][i:i + 1] for v in tokens])
        z_all = torch.cat([z[a:b]] + [v[2][i:i + 1] for v in tokens])
        got = torch.cat([y[a:b]] + [v[3][i:i + 1] for v in tokens])
        one = torch.tensor([0, len(x_all)])
        uu, win, um = ref.conv_prompts(x_all, weight, bias, one, torch.zeros(1, chans, 3))
        split = lambda m: (m[:, :n].unflatten(1, (heads, headdim)), dt_all, A_log,  # noqa: E731
                           m[:, n:n + groups * dstate].unflatten(1, (groups, dstate)),
                           m[:, n + groups * dstate:].unflatten(1, (groups, dstate)), D, z_all, dt_bias)
        zero = torch.zeros(1, heads, headdim, dstate)
        want, st = ref.scan_prompts(*split(uu), one, zero)
        mag, smag = ref.scan_prompts(*split(um), one, zero, absolute=True)
        k = 1.21 * (2.2 * 12 + 2 * len(x_all) + dstate + 8) * E
        ref.within(f"run prompt {i} out", got, want, k * mag)
        s = int(slots[i])
        ref.within(f"run prompt {i} state", state[s], st[0], k * smag[0])
        assert torch.equal(ref.d(window[s]), win[0])


def test_captured_run(mss):
    """Conv, scan, norm and step captured into one graph, replayed with eager
    calls between the replays: each replay gives what eager calls give."""
    g = gen(12)
    heads, headdim, dstate, groups = 3, 64, 128, 1
    n, chans = heads * headdim, heads * headdim + 2 * groups * dstate
    lens = (700, 3, 150)
    t = sum(lens)
    p = dict(x=randn(g, t, chans, dtype=torch.bfloat16), weight=randn(g, chans, 4), dt=randn(g, t, heads, dtype=torch.bfloat16),
             A_log=torch.linspace(0, 2.7, heads, device="cuda"), cu=offsets(lens), slots=ints(2, 0, 1),
             resume=ints(1, 1, 1), w=randn(g, n))

    def once(state, window, out):
        u = mss.causal_conv1d_prompts(p["x"], p["weight"], cu_seqlens=p["cu"], window=window,
                                      slots=p["slots"], resume=p["resume"])
        y = mss.head_scan_prompts(u[:, :n].unflatten(1, (heads, headdim)), p["dt"], p["A_log"],
                                  u[:, n:n + dstate].unsqueeze(1), u[:, n + dstate:].unsqueeze(1),
                                  cu_seqlens=p["cu"], state=state, slots=p["slots"], resume=p["resume"])
        q, scale = mss.rms_norm(y.flatten(1), p["w"], quant="row")
        s = mss.head_scan_step(state, window, p["x"][:3], p["dt"][:3], p["A_log"], p["weight"],
                               slots=p["slots"])
        for o, v in zip(out, (y, q.view(torch.uint8), scale, s)):
            o.copy_(v)

    def buffers():
        g2 = gen(13)
        return (randn(g2, 3, heads, headdim, dstate), randn(g2, 3, chans, 3, dtype=torch.bfloat16),
                (torch.zeros(t, heads, headdim, dtype=torch.bfloat16, device="cuda"),
                 torch.zeros(t, n, dtype=torch.uint8, device="cuda"), torch.zeros(t, 1, device="cuda"),
                 torch.zeros(3, heads, headdim, dtype=torch.bfloat16, device="cuda")))

    eager, graphed = buffers(), buffers()
    once(*buffers())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        once(*graphed)
    for i in range(4):
        graph.replay()
        once(*eager)
        torch.cuda.synchronize()
        for a, b in zip((*eager[:2], *eager[2]), (*graphed[:2], *graphed[2])):
            assert torch.equal(a, b), f"replay {i}"
        p["x"].mul_(-0.9)


def test_other_stream(mss):
    g = gen(14)
    v, c = scan_inputs(g, (300, 20), 4, 64, 128, 1, "bf16")
    start = c["state"].clone()
    args = (v["x"], v["dt_raw"], v["A_log"], v["B"], v["C"], v["D"], v["z"], v["dt_bias"])
    want = mss.head_scan_prompts(*args, cu_seqlens=c["cu"], state=c["state"], slots=c["slots"], resume=c["resume"])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = mss.head_scan_prompts(*args, cu_seqlens=c["cu"], state=start, slots=c["slots"], resume=c["resume"])
    side.synchronize()
    assert torch.equal(got, want) and torch.equal(start, c["state"])


def test_far_cache_slots(mss):
    """Cache entries past the 32-bit range of elements and bytes."""
    heads, headdim, dstate, chans = 2, 64, 128, 2 * 64 + 2 * 128
    far = (1 << 31) + 1024
    note("cache entries 8.6 GB apart")
    big = torch.zeros(far + heads * headdim * dstate, device="cuda")
    state = big.as_strided((2, heads, headdim, dstate), (far, headdim * dstate, dstate, 1))
    v, c = scan_inputs(gen(15), (40, 7), heads, headdim, dstate, 1, "f32")
    c["state"], c["slots"] = state, ints(1, 0)
    scan_check(mss, "scan far slots", v, c)
    g = gen(16)
    wide = torch.zeros(far + chans * 3, dtype=torch.bfloat16, device="cuda")
    window = wide.as_strided((2, chans, 3), (far, 3, 1))
    xbc = randn(g, 2, chans, dtype=torch.bfloat16)
    dt_raw, weight = randn(g, 2, heads, dtype=torch.bfloat16), randn(g, chans, 4)
    want, ws, ww, mag, smag = ref.step(state, window, xbc, dt_raw, v["A_log"], weight, None, None, None, None, 1,
                                       c["slots"])
    got = mss.head_scan_step(state, window, xbc, dt_raw, v["A_log"], weight, slots=c["slots"])
    k = 1.21 * (2.2 * 12 + dstate + 8) * E
    ref.within("step far out", got, want, k * mag + 2.0 ** -8 * want.abs() * 1.01)
    ref.within("step far state", state, ws, k * smag)
    assert torch.equal(ref.d(window), ww)
