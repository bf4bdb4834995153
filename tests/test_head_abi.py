"""The head-wise operations' C ABI and binding on the host: struct layouts, the
refusals of libmss (made before any HIP call, so fake device addresses do) and
those of the Python binding.
"""

import ctypes

import pytest
import torch

import mamba_selective_scan_amd as mss
from mamba_selective_scan_amd import _lib
from test_abi import HAS_GPU_NODE, _c_layout

no_gpu = pytest.mark.skipif(HAS_GPU_NODE, reason="fake-pointer checks run only where no GPU is present")
BASE = 0x7F0000000000


def fake(i):
    return BASE + i * (1 << 32)


@pytest.mark.parametrize("cls,cname", [(_lib.ConvPromptsArgs, "mss_conv_prompts_args"),
                                       (_lib.HeadScanArgs, "mss_head_scan_args"),
                                       (_lib.HeadStepArgs, "mss_head_step_args"),
                                       (_lib.NormArgs, "mss_norm_args")])
def test_structs_match_c_layout(cls, cname, tmp_path):
    names = [f[0] for f in cls._fields_]
    size, offs = _c_layout(cname, names, tmp_path)
    assert ctypes.sizeof(cls) == size
    assert [getattr(cls, n).offset for n in names] == offs


def put(a, **kw):
    for k, v in kw.items():
        if isinstance(v, tuple):
            getattr(a, k)[:] = v
        else:
            setattr(a, k, v)
    return a


def conv():
    a = _lib.ConvPromptsArgs()
    return put(a, struct_size=ctypes.sizeof(a), io_dtype=1, tokens=100, dim=96, width=4, seqs=3, cache_slots=5,
               x=fake(0), x_stride=(96, 1), weight=fake(1), weight_stride=(4, 1), bias=fake(2),
               cu_seqlens=fake(3), slots=fake(4), resume=fake(5), window=fake(6), window_stride=288,
               out=fake(7), out_stride=(96, 1), activation=1)


def scan():
    a = _lib.HeadScanArgs()
    return put(a, struct_size=ctypes.sizeof(a), io_dtype=1, tokens=100, heads=4, headdim=64, dstate=128, groups=2,
               seqs=3, cache_slots=5, x=fake(0), x_stride=(256, 64, 1), dt_raw=fake(1), dt_stride=(4, 1),
               A_log=fake(2), B=fake(3), B_stride=(256, 128, 1), C=fake(4), C_stride=(256, 128, 1), D=fake(5),
               z=fake(6), z_stride=(256, 64, 1), dt_bias=fake(7), cu_seqlens=fake(8), slots=fake(9),
               resume=fake(10), state=fake(11), state_stride=4 * 64 * 128, out=fake(12),
               out_stride=(256, 64, 1), delta_softplus=1, workspace=fake(13), workspace_bytes=1 << 30)


def step():
    a = _lib.HeadStepArgs()
    return put(a, struct_size=ctypes.sizeof(a), io_dtype=1, rows=3, heads=4, headdim=64, dstate=128, groups=2,
               width=4, cache_slots=5, state=fake(0), state_stride=4 * 64 * 128, window=fake(1),
               window_stride=768 * 3, xbc=fake(2), xbc_stride=(768, 1), dt_raw=fake(3), dt_stride=(4, 1),
               A_log=fake(4), weight=fake(5), weight_stride=(4, 1), bias=fake(6), D=fake(7), z=fake(8),
               z_stride=(256, 64, 1), dt_bias=fake(9), slots=fake(10), out=fake(11), out_stride=(256, 64, 1),
               delta_softplus=1)


def norm():
    a = _lib.NormArgs()
    return put(a, struct_size=ctypes.sizeof(a), io_dtype=1, residual_dtype=0, quant=2, rows=3, dim=256,
               x=fake(0), x_stride=256, residual=fake(1), residual_stride=256, weight=fake(2), out=fake(3),
               out_stride=256, scale=fake(4), residual_out=fake(5), residual_out_stride=256, eps=1e-5)


CALLS = {"conv": (conv, "mss_causal_conv1d_prompts"), "scan": (scan, "mss_head_scan_prompts"),
         "step": (step, "mss_head_scan_step"), "norm": (norm, "mss_rms_norm")}

STRUCT = [dict(struct_size=8), dict(reserved0=1)]
SHAPE = {
    "conv": [dict(tokens=-1), dict(tokens=(1 << 30) + 1), dict(dim=0), dict(width=0), dict(width=5), dict(seqs=0),
             dict(seqs=(1 << 20) + 1), dict(cache_slots=0), dict(tokens=1 << 30, dim=1 << 15, x_stride=(1 << 15, 1))],
    "scan": [dict(tokens=-1), dict(heads=0), dict(headdim=0), dict(groups=0), dict(groups=3), dict(groups=8),
             dict(seqs=0), dict(cache_slots=0), dict(heads=1 << 40), dict(heads=1 << 29), dict(tokens=0, heads=96, seqs=1 << 20, headdim=64)],
    "step": [dict(rows=0), dict(heads=0), dict(headdim=0), dict(groups=3), dict(width=5), dict(cache_slots=0),
             dict(rows=1 << 30), dict(rows=1 << 22)],
    "norm": [dict(rows=0), dict(dim=0), dict(dim=130), dict(dim=32768 + 128), dict(eps=-1.0), dict(eps=float("nan")),
             dict(rows=1 << 26), dict(rows=1 << 24, dim=4096), dict(rows=1 << 22, dim=16384)],
}
NULL = {
    "conv": ["x", "weight", "cu_seqlens", "window", "out"],
    "scan": ["x", "dt_raw", "A_log", "B", "C", "cu_seqlens", "state", "out"],
    "step": ["state", "window", "xbc", "dt_raw", "A_log", "weight", "out"],
    "norm": ["x", "weight", "out", "scale"],
}
STRIDE = {
    "conv": [dict(x_stride=(-96, 1)), dict(out_stride=(0, 1)), dict(out_stride=(95, 1)), dict(window_stride=287),
             dict(weight_stride=(-4, 1))],
    "scan": [dict(x_stride=(256, 64, 2)), dict(out_stride=(256, 63, 1)), dict(z_stride=(256, 1, 64)),
             dict(B_stride=(256, 1, 2)), dict(C_stride=(256, -128, 1)), dict(state_stride=4 * 64 * 128 - 4),
             dict(dt_stride=(-4, 1)), dict(x_stride=((1 << 31) // 260 + 1, 64, 1)),
             dict(B_stride=(1 << 24, 128, 1)), dict(C_stride=(1 << 24, 128, 1)),
             dict(z_stride=(1 << 24, 64, 1)), dict(out_stride=(1 << 24, 64, 1))],
    "step": [dict(xbc_stride=(-1, 1)), dict(out_stride=(255, 64, 1)), dict(state_stride=100),
             dict(window_stride=768), dict(z_stride=(1, -1, 1))],
    "norm": [dict(x_stride=-1), dict(out_stride=255), dict(residual_out_stride=100),
             dict(residual_out=fake(1), residual_out_stride=512)],
}
MISALIGNED = {
    "conv": [("x", 1), ("weight", 2), ("window", 1), ("cu_seqlens", 2), ("slots", 1), ("out", 1)],
    "scan": [("x", 1), ("state", 2), ("cu_seqlens", 2), ("A_log", 2), ("workspace", 16), ("dt_bias", 1)],
    "step": [("state", 1), ("window", 1), ("slots", 2), ("bias", 2), ("xbc", 1)],
    "norm": [("x", 1), ("residual", 2), ("scale", 2), ("weight", 1)],
}
ALIAS = {
    "conv": [("out", 0), ("window", 7), ("out", 4), ("window", 1)],
    "scan": [("out", 0), ("out", 11), ("state", 6), ("out", 3), ("state", 10)],
    "step": [("out", 2), ("out", 0), ("window", 0), ("window", 8), ("state", 5), ("out", 10)],
    "norm": [("out", 0), ("scale", 3), ("residual_out", 0), ("residual_out", 3), ("scale", 1)],
}


def refused(op, expect, **kw):
    make, name = CALLS[op]
    got = getattr(_lib.lib(), name)(ctypes.byref(put(make(), **kw)), None)
    assert got == _lib.STATUS_CODE[expect], (op, kw, _lib.STATUS.get(got, got))


@no_gpu
@pytest.mark.parametrize("op", sorted(CALLS))
def test_refusals(op):
    for kw in STRUCT:
        refused(op, "MSS_ERR_BAD_STRUCT", **kw)
    assert getattr(_lib.lib(), CALLS[op][1])(None, None) == _lib.STATUS_CODE["MSS_ERR_BAD_STRUCT"]
    refused(op, "MSS_ERR_UNSUPPORTED_DTYPE", io_dtype=2)
    for kw in SHAPE[op]:
        refused(op, "MSS_ERR_BAD_SHAPE", **kw)
    for field in NULL[op]:
        refused(op, "MSS_ERR_NULL_POINTER", **{field: None})
    for kw in STRIDE[op]:
        refused(op, "MSS_ERR_BAD_STRIDE", **kw)
    for field, by in MISALIGNED[op]:
        refused(op, "MSS_ERR_MISALIGNED", **{field: getattr(CALLS[op][0](), field) + by})
    for field, where in ALIAS[op]:
        refused(op, "MSS_ERR_ALIASING", **{field: fake(where)})


@no_gpu
def test_other_refusals():
    for n in (0, 129):
        refused("scan", "MSS_ERR_UNSUPPORTED_DSTATE", dstate=n)
        refused("step", "MSS_ERR_UNSUPPORTED_DSTATE", dstate=n)
    refused("conv", "MSS_ERR_BAD_STRUCT", activation=7)
    refused("norm", "MSS_ERR_BAD_STRUCT", quant=3)
    refused("norm", "MSS_ERR_UNSUPPORTED_DTYPE", residual_dtype=5)
    # 600 tokens of 4 heads are cut over time, and need room for the states between
    refused("scan", "MSS_ERR_WORKSPACE_TOO_SMALL", tokens=600, workspace=None)
    refused("scan", "MSS_ERR_WORKSPACE_TOO_SMALL", tokens=600, workspace_bytes=1 << 16)
    refused("scan", "MSS_ERR_ALIASING", tokens=600, workspace=fake(11))
    refused("scan", "MSS_ERR_ALIASING", tokens=600, workspace=fake(12))
    # views between which nothing overlaps but whose ranges interleave are
    # refused as well: the check is on ranges
    refused("norm", "MSS_ERR_ALIASING", out=fake(0) + 512, x_stride=1024, out_stride=2048)


def test_workspace_sizes():
    """From the sizes alone: none for a call of up to five chunks, room for every
    segment's state and decay otherwise."""
    lib, st = _lib.lib(), ctypes.c_int(0)

    def size(**kw):
        return lib.mss_head_scan_prompts_workspace_size(ctypes.byref(put(scan(), **kw)), ctypes.byref(st))

    assert size() == 0 and st.value == 0
    assert size(tokens=320) == 0 and size(tokens=320, seqs=1) == 0
    assert size(tokens=160, io_dtype=0) == 0
    states = 4 * 64 * 128 * 4
    for tokens in (321, 513, 32768, 1 << 20):
        # a cut prompt has segments of at least two chunks, but for its last; of
        # five where the prompts are shorter than that on the average
        for seqs in (1, 3):
            least = 128 if tokens > 320 * seqs else 320
            need = size(tokens=tokens, seqs=seqs)
            assert states <= need <= (2 * tokens // least) * (states + 16) + 256 and st.value == 0
    assert size(dstate=0) == 0 and st.value == _lib.STATUS_CODE["MSS_ERR_UNSUPPORTED_DSTATE"]


class _NoCalls:
    def __getattr__(self, name):
        raise AssertionError(f"libmss.{name} was reached")


def test_host_tensors_are_refused(monkeypatch):
    monkeypatch.setattr(_lib, "lib", lambda *a, **k: _NoCalls())
    x, w = torch.zeros(5, 8), torch.zeros(8, 4)
    cu = torch.tensor([0, 5], dtype=torch.int32)
    with pytest.raises(ValueError, match="on a GPU"):
        mss.causal_conv1d_prompts(x, w, cu_seqlens=cu, window=torch.zeros(1, 8, 3))
    with pytest.raises(ValueError, match="on a GPU"):
        mss.head_scan_prompts(x.view(5, 2, 4), x[:, :2], w[:2, 0], x.view(5, 1, 8), x.view(5, 1, 8),
                              cu_seqlens=cu, state=torch.zeros(1, 2, 4, 8))
    with pytest.raises(ValueError, match="on a GPU"):
        mss.head_scan_step(torch.zeros(5, 2, 4, 8), torch.zeros(5, 24, 3), torch.zeros(5, 24), x[:, :2], w[:2, 0],
                           torch.zeros(24, 4))
    with pytest.raises(ValueError, match="on a GPU"):
        mss.rms_norm(x, w[:, 0])
    with pytest.raises(TypeError, match="torch.Tensor"):
        mss.rms_norm([1.0], w[:, 0])


@pytest.mark.gpu
def test_bad_tensors_are_refused_before_launch(monkeypatch):
    monkeypatch.setattr(_lib, "lib", lambda *a, **k: _NoCalls())
    dev = torch.device("cuda", 0)
    z = lambda *s, dt=torch.float32: torch.zeros(*s, dtype=dt, device=dev)  # noqa: E731
    cu = torch.tensor([0, 5], dtype=torch.int32, device=dev)

    def bad(err, match, fn, *a, **k):
        with pytest.raises(err, match=match):
            fn(*a, **k)

    conv = dict(x=z(5, 8), weight=z(8, 4), cu_seqlens=cu, window=z(1, 8, 3))
    for change, err, match in [
            (dict(x=z(5, 8, 1)), ValueError, "2 dimensions"), (dict(weight=z(7, 4)), ValueError, "weight"),
            (dict(cu_seqlens=cu.long()), TypeError, "cu_seqlens"), (dict(cu_seqlens=cu[:1]), ValueError, "cu_seqlens"),
            (dict(cu_seqlens=cu.cpu()), ValueError, "cu_seqlens"), (dict(window=z(1, 8, 2)), ValueError, "window"),
            (dict(window=z(1, 3, 8).transpose(1, 2)), ValueError, "contiguous"),
            (dict(slots=cu), ValueError, "slots"), (dict(resume=z(1)), TypeError, "resume"),
            (dict(out=z(4, 8)), ValueError, "out"), (dict(activation="gelu"), ValueError, "activation"),
            (dict(x=z(5, 8, dt=torch.float16), window=z(1, 8, 3, dt=torch.float16)), TypeError, "dtype")]:
        bad(err, match, mss.causal_conv1d_prompts, **{**conv, **change})
    scan = dict(x=z(5, 2, 4), dt_raw=z(5, 2), A_log=z(2), B=z(5, 1, 8), C=z(5, 1, 8), cu_seqlens=cu,
                state=z(1, 2, 4, 8))
    for change, err, match in [
            (dict(dt_raw=z(5, 3)), ValueError, "dt_raw"), (dict(C=z(5, 1, 7)), ValueError, "C must"),
            (dict(B=z(4, 1, 8)), ValueError, "B must"), (dict(A_log=z(2, 1)), ValueError, "A_log"),
            (dict(state=z(1, 2, 4, 9)), ValueError, "state"), (dict(z=z(5, 2, 5)), ValueError, "z must"),
            (dict(D=z(2, dt=torch.bfloat16)), TypeError, "D must"),
            (dict(state=z(1, 2, 4, 8, dt=torch.bfloat16)), TypeError, "state")]:
        bad(err, match, mss.head_scan_prompts, **{**scan, **change})
    step = dict(state=z(5, 2, 4, 8), window=z(5, 24, 3), xbc=z(5, 24), dt_raw=z(5, 2), A_log=z(2), weight=z(24, 4))
    for change, err, match in [
            (dict(xbc=z(5, 23)), ValueError, "channels"), (dict(window=z(4, 24, 3)), ValueError, "slots"),
            (dict(bias=z(23)), ValueError, "bias"), (dict(out=z(5, 8)), ValueError, "out"),
            (dict(xbc=z(5, 8)), ValueError, "channels")]:
        bad(err, match, mss.head_scan_step, **{**step, **change})
    norm = dict(x=z(5, 256), weight=z(256))
    for change, err, match in [
            (dict(weight=z(255)), ValueError, "weight"), (dict(quant="col"), ValueError, "quant"),
            (dict(x=z(5, 250), weight=z(250), quant="block"), ValueError, "128"),
            (dict(x=z(256, 5).t()), ValueError, "unit stride"), (dict(scale=z(5)), ValueError, "scale"),
            (dict(quant="row", scale=z(4)), ValueError, "scale"), (dict(residual=z(4, 256)), ValueError, "residual"),
            (dict(residual_out=z(5, 256)), ValueError, "residual_out"),
            (dict(quant="row", out=z(5, 256)), TypeError, "out")]:
        bad(err, match, mss.rms_norm, **{**norm, **change})


def test_workspace_holds_what_prompts_can_be_cut_into():
    """A cut prompt has less than one segment more than its tokens fill: 8 prompts
    in 32768 tokens make at most 40 segments of 1024, one makes at most 40 of 832."""
    lib = _lib.lib()
    for heads, seqs, segments in ((80, 8, 40), (24, 1, 40)):
        a = put(scan(), tokens=32768, heads=heads, groups=1, seqs=seqs)
        need = lib.mss_head_scan_prompts_workspace_size(ctypes.byref(a), None)
        assert 0 < need <= segments * (heads * 64 * 128 * 4 + heads * 4) + 256


def test_workspace_size_of_sizes_that_the_launch_refuses():
    """No size, and the launch's status, where the segments would pass 2^32 threads:
    a binding allocates nothing before the refusal."""
    lib, st = _lib.lib(), ctypes.c_int(0)
    a = put(scan(), tokens=1 << 30, heads=4096, groups=1, x_stride=(1 << 18, 64, 1), z_stride=(1 << 18, 64, 1),
            out_stride=(1 << 18, 64, 1))
    assert lib.mss_head_scan_prompts_workspace_size(ctypes.byref(a), ctypes.byref(st)) == 0
    assert st.value == _lib.STATUS_CODE["MSS_ERR_BAD_SHAPE"]
    assert lib.mss_head_scan_prompts(ctypes.byref(a), None) == st.value
