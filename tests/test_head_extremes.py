"""The head-wise scan at magnitudes, time steps and decays far from those of a
trained layer: what the recurrence gives in 64 bits is what the chunked form has
to give, within the bounds of test_head_ops.
"""

import math

import pytest
import torch

import head_ref as ref
from test_head_ops import crowd, gen, mss, offsets, randn, scan_check, scan_inputs  # noqa: F401

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
