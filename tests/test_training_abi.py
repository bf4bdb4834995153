"""Layer norm's and the losses' C ABI and binding on the host: struct layouts,
workspace sizes, and the refusals of libmss (made before any HIP call, so fake
device addresses do) and of the Python binding.
"""

import ctypes

import pytest
import torch

import mamba_selective_scan_amd as mss
from mamba_selective_scan_amd import _lib
from test_abi import _c_layout
from test_head_abi import fake, no_gpu, put


@pytest.mark.parametrize("cls,cname", [(_lib.LayerNormArgs, "mss_layer_norm_args"),
                                       (_lib.LayerNormBwdArgs, "mss_layer_norm_bwd_args"),
                                       (_lib.LinearLossArgs, "mss_linear_loss_args")])
def test_structs_match_c_layout(cls, cname, tmp_path):
    names = [f[0] for f in cls._fields_]
    size, offs = _c_layout(cname, names, tmp_path)
    assert ctypes.sizeof(cls) == size
    assert [getattr(cls, n).offset for n in names] == offs


def fwd():
    a = _lib.LayerNormArgs()
    return put(a, struct_size=ctypes.sizeof(a), io_dtype=1, residual_dtype=0, rows=3, dim=256, x=fake(0), x_stride=256,
               residual=fake(1), residual_stride=256, weight=fake(2), bias=fake(3), out=fake(4), out_stride=256,
               mean=fake(5), rstd=fake(6), residual_out=fake(7), residual_out_stride=256, eps=1e-5)


def bwd():
    a = _lib.LayerNormBwdArgs()
    return put(a, struct_size=ctypes.sizeof(a), io_dtype=1, r_dtype=0, rows=3, dim=256, dy=fake(0), dy_stride=256,
               r=fake(1), r_stride=256, dr=fake(2), dr_stride=256, weight=fake(3), mean=fake(4), rstd=fake(5),
               dx=fake(6), dx_stride=256, dresidual=fake(7), dresidual_stride=256, dweight=fake(8), dbias=fake(9),
               workspace=fake(10), workspace_bytes=1 << 20)


def loss():
    a = _lib.LinearLossArgs()
    return put(a, struct_size=ctypes.sizeof(a), io_dtype=1, rows=30, dim=256, vocab=1000, entries=4, x=fake(0),
               x_stride=256, weight=fake(1), weight_stride=256, ids=fake(2), ids_stride=(4, 1), teacher=fake(3),
               teacher_stride=(4, 1), teacher_dtype=0, logit_scale=1.0, temperature=2.0, row_weight=fake(4),
               loss=fake(5), lse=fake(6), total=fake(7), dx=fake(8), dx_stride=256, dweight=fake(9),
               dweight_stride=256, workspace=fake(10), workspace_bytes=1 << 31)


CALLS = {"fwd": (fwd, "mss_layer_norm_fwd"), "bwd": (bwd, "mss_layer_norm_bwd"), "loss": (loss, "mss_linear_loss")}
BAD = [
    ("fwd", dict(struct_size=8), "MSS_ERR_BAD_STRUCT"), ("fwd", dict(reserved0=1), "MSS_ERR_BAD_STRUCT"),
    ("fwd", dict(reserved1=1), "MSS_ERR_BAD_STRUCT"),
    ("fwd", dict(io_dtype=2), "MSS_ERR_UNSUPPORTED_DTYPE"), ("fwd", dict(residual_dtype=-1), "MSS_ERR_UNSUPPORTED_DTYPE"),
    ("fwd", dict(rows=0), "MSS_ERR_BAD_SHAPE"), ("fwd", dict(rows=1 << 31), "MSS_ERR_BAD_SHAPE"),
    ("fwd", dict(rows=(1 << 26) - 3), "MSS_ERR_BAD_SHAPE"),
    ("fwd", dict(dim=0), "MSS_ERR_BAD_SHAPE"), ("fwd", dict(dim=32769), "MSS_ERR_BAD_SHAPE"),
    ("fwd", dict(eps=-1e-5), "MSS_ERR_BAD_SHAPE"), ("fwd", dict(eps=float("nan")), "MSS_ERR_BAD_SHAPE"),
    ("fwd", dict(x=0), "MSS_ERR_NULL_POINTER"), ("fwd", dict(weight=0), "MSS_ERR_NULL_POINTER"),
    ("fwd", dict(out=0), "MSS_ERR_NULL_POINTER"),
    ("fwd", dict(x_stride=-1), "MSS_ERR_BAD_STRIDE"), ("fwd", dict(out_stride=255), "MSS_ERR_BAD_STRIDE"),
    ("fwd", dict(residual_out_stride=255), "MSS_ERR_BAD_STRIDE"),
    ("fwd", dict(residual_out=fake(1), residual_out_stride=257), "MSS_ERR_BAD_STRIDE"),
    ("fwd", dict(x=fake(0) + 1), "MSS_ERR_MISALIGNED"), ("fwd", dict(mean=fake(5) + 2), "MSS_ERR_MISALIGNED"),
    ("fwd", dict(bias=fake(3) + 2), "MSS_ERR_MISALIGNED"),
    ("fwd", dict(out=fake(0)), "MSS_ERR_ALIASING"), ("fwd", dict(rstd=fake(5) + 8), "MSS_ERR_ALIASING"),
    ("fwd", dict(residual_out=fake(1) + 4), "MSS_ERR_ALIASING"), ("fwd", dict(mean=fake(2) + 1020), "MSS_ERR_ALIASING"),
    ("bwd", dict(struct_size=8), "MSS_ERR_BAD_STRUCT"), ("bwd", dict(reserved0=1), "MSS_ERR_BAD_STRUCT"),
    ("bwd", dict(io_dtype=7), "MSS_ERR_UNSUPPORTED_DTYPE"), ("bwd", dict(r_dtype=7), "MSS_ERR_UNSUPPORTED_DTYPE"),
    ("bwd", dict(rows=0), "MSS_ERR_BAD_SHAPE"), ("bwd", dict(dim=32769), "MSS_ERR_BAD_SHAPE"),
    ("bwd", dict(dy=0), "MSS_ERR_NULL_POINTER"), ("bwd", dict(mean=0), "MSS_ERR_NULL_POINTER"),
    ("bwd", dict(dx=0, dresidual=0, dweight=0, dbias=0), "MSS_ERR_NULL_POINTER"),
    ("bwd", dict(dr_stride=-256), "MSS_ERR_BAD_STRIDE"), ("bwd", dict(dx_stride=0), "MSS_ERR_BAD_STRIDE"),
    ("bwd", dict(r=fake(1) + 2), "MSS_ERR_MISALIGNED"), ("bwd", dict(workspace=fake(10) + 16), "MSS_ERR_MISALIGNED"),
    ("bwd", dict(workspace=0), "MSS_ERR_WORKSPACE_TOO_SMALL"), ("bwd", dict(workspace_bytes=99), "MSS_ERR_WORKSPACE_TOO_SMALL"),
    ("bwd", dict(dx=fake(0)), "MSS_ERR_ALIASING"), ("bwd", dict(dresidual=fake(2)), "MSS_ERR_ALIASING"),
    ("bwd", dict(dbias=fake(8) + 512), "MSS_ERR_ALIASING"), ("bwd", dict(workspace=fake(9)), "MSS_ERR_ALIASING"),
    ("loss", dict(struct_size=8), "MSS_ERR_BAD_STRUCT"), ("loss", dict(reserved0=1), "MSS_ERR_BAD_STRUCT"),
    ("loss", dict(io_dtype=3), "MSS_ERR_UNSUPPORTED_DTYPE"), ("loss", dict(teacher_dtype=3), "MSS_ERR_UNSUPPORTED_DTYPE"),
    ("loss", dict(rows=-1), "MSS_ERR_BAD_SHAPE"), ("loss", dict(rows=(1 << 22) + 1), "MSS_ERR_BAD_SHAPE"),
    ("loss", dict(dim=0), "MSS_ERR_BAD_SHAPE"), ("loss", dict(dim=32769), "MSS_ERR_BAD_SHAPE"),
    ("loss", dict(vocab=0), "MSS_ERR_BAD_SHAPE"), ("loss", dict(vocab=(1 << 22) + 1), "MSS_ERR_BAD_SHAPE"),
    ("loss", dict(entries=0), "MSS_ERR_BAD_SHAPE"), ("loss", dict(entries=1025), "MSS_ERR_BAD_SHAPE"),
    ("loss", dict(teacher=0), "MSS_ERR_BAD_SHAPE"), ("loss", dict(teacher=0, entries=1), "MSS_ERR_BAD_SHAPE"),
    ("loss", dict(temperature=0.0), "MSS_ERR_BAD_SHAPE"), ("loss", dict(temperature=float("inf")), "MSS_ERR_BAD_SHAPE"),
    ("loss", dict(logit_scale=float("nan")), "MSS_ERR_BAD_SHAPE"), ("loss", dict(temperature=float("nan")), "MSS_ERR_BAD_SHAPE"),
    ("loss", dict(temperature=1e-39), "MSS_ERR_BAD_SHAPE"), ("loss", dict(temperature=1e20), "MSS_ERR_BAD_SHAPE"),
    ("loss", dict(logit_scale=1e30, temperature=1e-10), "MSS_ERR_BAD_SHAPE"),
    ("loss", dict(logit_scale=1e30, temperature=1e10), "MSS_ERR_BAD_SHAPE"),
    ("loss", dict(vocab=1 << 22, dim=16400), "MSS_ERR_BAD_SHAPE"), ("loss", dict(rows=1 << 22, dim=16400), "MSS_ERR_BAD_SHAPE"),
    ("loss", dict(x=0), "MSS_ERR_NULL_POINTER"), ("loss", dict(weight=0), "MSS_ERR_NULL_POINTER"),
    ("loss", dict(ids=0), "MSS_ERR_NULL_POINTER"), ("loss", dict(loss=0), "MSS_ERR_NULL_POINTER"),
    ("loss", dict(x_stride=-1), "MSS_ERR_BAD_STRIDE"), ("loss", dict(ids_stride=(-4, 1)), "MSS_ERR_BAD_STRIDE"),
    ("loss", dict(dx_stride=255), "MSS_ERR_BAD_STRIDE"), ("loss", dict(dweight_stride=0), "MSS_ERR_BAD_STRIDE"),
    ("loss", dict(ids=fake(2) + 4), "MSS_ERR_MISALIGNED"), ("loss", dict(x=fake(0) + 1), "MSS_ERR_MISALIGNED"),
    ("loss", dict(workspace=fake(10) + 128), "MSS_ERR_MISALIGNED"), ("loss", dict(total=fake(7) + 2), "MSS_ERR_MISALIGNED"),
    ("loss", dict(workspace=0), "MSS_ERR_WORKSPACE_TOO_SMALL"),
    ("loss", dict(workspace_bytes=1000), "MSS_ERR_WORKSPACE_TOO_SMALL"),
    ("loss", dict(dx=fake(0)), "MSS_ERR_ALIASING"), ("loss", dict(dweight=fake(1)), "MSS_ERR_ALIASING"),
    ("loss", dict(lse=fake(5) + 116), "MSS_ERR_ALIASING"), ("loss", dict(workspace=fake(4)), "MSS_ERR_ALIASING"),
    ("loss", dict(total=fake(5)), "MSS_ERR_ALIASING"),
]


@no_gpu
@pytest.mark.parametrize("call,change,want", BAD, ids=[f"{c}-{'-'.join(k)}-{i}" for i, (c, k, _) in enumerate(BAD)])
def test_bad_arguments_are_refused(call, change, want):
    make, name = CALLS[call]
    code = getattr(_lib.lib(), name)(ctypes.byref(put(make(), **change)), None)
    assert _lib.STATUS[code] == want


@no_gpu
def test_null_structs_and_scale():
    lib = _lib.lib()
    for _, name in CALLS.values():
        assert _lib.STATUS[getattr(lib, name)(None, None)] == "MSS_ERR_BAD_STRUCT"
    scale = lambda *a: _lib.STATUS[lib.mss_scale(*a, None)]
    assert scale(fake(0), fake(1), fake(2), 10, 5) == "MSS_ERR_UNSUPPORTED_DTYPE"
    assert scale(fake(0), fake(1), fake(2), -1, 0) == "MSS_ERR_BAD_SHAPE"
    assert scale(fake(0), 0, fake(2), 10, 0) == "MSS_ERR_NULL_POINTER"
    assert scale(0, fake(1), fake(2), 10, 0) == "MSS_ERR_NULL_POINTER"
    assert scale(fake(0) + 2, fake(1), fake(2), 10, 0) == "MSS_ERR_MISALIGNED"
    assert scale(fake(0), fake(1), fake(0) + 4, 10, 0) == "MSS_ERR_ALIASING"
    assert scale(0, fake(1), 0, 0, 0) == "MSS_OK"


def size(call, **change):
    make, name = CALLS[call]
    status = ctypes.c_int(-1)
    n = getattr(_lib.lib(), f"{name}_workspace_size")(ctypes.byref(put(make(), **change)), ctypes.byref(status))
    return n, _lib.STATUS[status.value]


def test_workspace_sizes():
    assert size("bwd") == (3 * 256 * 2 * 4, "MSS_OK") or size("bwd")[0] == 1 * 256 * 2 * 4
    assert size("bwd", dweight=0, dbias=0) == (0, "MSS_OK")
    assert size("bwd", dim=0) == (0, "MSS_ERR_BAD_SHAPE")
    assert size("loss", vocab=0) == (0, "MSS_ERR_BAD_SHAPE")
    n, ok = size("loss")
    assert ok == "MSS_OK" and n > 30 * 1000 * 2
    # without gradients no probabilities are kept
    assert size("loss", dx=0, dweight=0)[0] < n
    # fp32 takes planes of its operands, a few rows of it the matrix as it is
    assert size("loss", rows=65)[0] + 1000 * 256 * 4 < size("loss", rows=65, io_dtype=0)[0]
    assert size("loss", rows=64, io_dtype=0)[0] < 1000 * 256 * 4
    assert size("loss", rows=128, io_dtype=0, dx=0, dweight=0)[0] < 1000 * 256 * 4
    assert size("loss", rows=129, io_dtype=0, dx=0, dweight=0)[0] > 1000 * 256 * 4
    # an unaligned matrix is copied
    assert size("loss", weight=fake(1) + 2)[0] >= n + 1000 * 256 * 2
    # the probabilities of all rows are never there: a piece of them takes 2 GiB
    big = dict(dim=1024, vocab=65536, x_stride=1024, weight_stride=1024, dx_stride=1024, dweight_stride=1024)
    few, many = size("loss", rows=32768, **big)[0], size("loss", rows=262144, **big)[0]
    assert many - few < (262144 - 32768) * (1024 * 2 + 200) + (1 << 30)


# ---------------------------------------------------------------- the binding

def test_host_tensors_are_refused():
    x, w, ids = torch.zeros(4, 8), torch.zeros(8), torch.zeros(4, dtype=torch.int64)
    v = torch.zeros(16, 8)
    top = torch.zeros(4, 2, dtype=torch.int64)
    for call in (lambda: mss.layer_norm_fwd(x, w), lambda: mss.layer_norm(x, w),
                 lambda: mss.layer_norm_bwd(x, x, w, w, w), lambda: mss.linear_cross_entropy_fwd(x, v, ids),
                 lambda: mss.linear_cross_entropy_grad(x, v, ids), lambda: mss.linear_cross_entropy(x, v, ids),
                 lambda: mss.linear_distillation(x, v, top, torch.zeros(4, 2))):
        with pytest.raises(ValueError, match="GPU"):
            call()


class OnGpu(torch.Tensor):
    """A host tensor that says it is on a GPU: the checks that come before the
    library is called."""
    is_cuda = property(lambda self: True)


def on(t):
    return t.as_subclass(OnGpu)


REFUSED = {
    "dims": (lambda t: mss.linear_cross_entropy_fwd(on(torch.zeros(2, 3, 4)), t["w"], t["ids"]), ValueError),
    "weight_dim": (lambda t: mss.linear_cross_entropy_fwd(t["x"], on(torch.zeros(16, 7)), t["ids"]), ValueError),
    "weight_dtype": (lambda t: mss.linear_cross_entropy_fwd(t["x"], t["w"].bfloat16(), t["ids"]), TypeError),
    "weight_columns": (lambda t: mss.linear_cross_entropy_fwd(t["x"], on(torch.zeros(8, 16).t()), t["ids"]), ValueError),
    "half": (lambda t: mss.linear_cross_entropy_fwd(t["x"].half(), t["w"].half(), t["ids"]), TypeError),
    "targets_int32": (lambda t: mss.linear_cross_entropy_fwd(t["x"], t["w"], t["ids"].int()), TypeError),
    "targets_length": (lambda t: mss.linear_cross_entropy_fwd(t["x"], t["w"], t["ids"][:3]), ValueError),
    "row_weight_dtype": (lambda t: mss.linear_cross_entropy_grad(t["x"], t["w"], t["ids"], t["rw"].double()), TypeError),
    "row_weight_stride": (lambda t: mss.linear_cross_entropy_grad(t["x"], t["w"], t["ids"], on(torch.zeros(8))[::2]),
                          ValueError),
    "dx_shape": (lambda t: mss.linear_cross_entropy_grad(t["x"], t["w"], t["ids"], dx=on(torch.zeros(4, 7))), ValueError),
    "dweight_dtype": (lambda t: mss.linear_cross_entropy_grad(t["x"], t["w"], t["ids"], dweight=t["w"].bfloat16()),
                      TypeError),
    "ids_dims": (lambda t: mss.linear_distillation_fwd(t["x"], t["w"], t["ids"], t["teach"]), ValueError),
    "teacher_shape": (lambda t: mss.linear_distillation_fwd(t["x"], t["w"], t["top"], t["teach"][:, :1]), ValueError),
    "teacher_dtype": (lambda t: mss.linear_distillation_fwd(t["x"], t["w"], t["top"], t["teach"].half()), TypeError),
    "teacher_none": (lambda t: mss.linear_distillation_fwd(t["x"], t["w"], t["top"], None), TypeError),
    "norm_dims": (lambda t: mss.layer_norm_fwd(on(torch.zeros(2, 2, 8)), t["nw"]), ValueError),
    "norm_weight": (lambda t: mss.layer_norm_fwd(t["x"], t["nw"][:7]), ValueError),
    "norm_residual": (lambda t: mss.layer_norm_fwd(t["x"], t["nw"], residual=t["x"][:3]), ValueError),
    "norm_residual_out": (lambda t: mss.layer_norm_fwd(t["x"], t["nw"], residual_out=t["x"]), ValueError),
    "norm_columns": (lambda t: mss.layer_norm_fwd(on(torch.zeros(8, 4).t()), t["nw"]), ValueError),
    "norm_bwd_r": (lambda t: mss.layer_norm_bwd(t["x"], t["x"][:3], t["nw"], t["rw"], t["rw"]), ValueError),
    "norm_bwd_mean": (lambda t: mss.layer_norm_bwd(t["x"], t["x"], t["nw"], t["rw"][:3], t["rw"]), ValueError),
    "norm_bwd_none": (lambda t: mss.layer_norm_bwd(t["x"], t["x"], None, t["rw"], t["rw"]), TypeError),
    "norm_bwd_dr": (lambda t: mss.layer_norm_bwd(t["x"], t["x"], t["nw"], t["rw"], t["rw"], dr=t["x"].bfloat16()), TypeError),
    "targets_transposed": (lambda t: mss.linear_cross_entropy(t["x"].view(2, 2, 8), t["w"], t["ids"]), ValueError),
    "row_weight_flat": (lambda t: mss.linear_cross_entropy(t["x"].view(2, 2, 8), t["w"], t["ids"].view(2, 2), t["rw"]),
                        ValueError),
    "ids_flat": (lambda t: mss.linear_distillation(t["x"], t["w"], t["ids"], t["teach"]), ValueError),
    "ids_list": (lambda t: mss.linear_distillation(t["x"], t["w"], [[1, 2]] * 4, t["teach"]), TypeError),
    "teacher_entries": (lambda t: mss.linear_distillation(t["x"], t["w"], t["top"], t["teach"][:, :1]), ValueError),
    "no_rows_dim": (lambda t: mss.linear_cross_entropy(on(torch.zeros(())), t["w"], t["ids"]), ValueError),
    "norm_autograd_residual": (lambda t: mss.layer_norm(t["x"], t["nw"], None, t["x"][:3]), ValueError),
}


@pytest.mark.parametrize("name", REFUSED)
def test_binding_refuses(name, monkeypatch):
    def no_library():
        raise AssertionError("the library was called")

    monkeypatch.setattr(_lib, "lib", no_library)
    t = {"x": on(torch.zeros(4, 8)), "w": on(torch.zeros(16, 8)), "ids": on(torch.zeros(4, dtype=torch.int64)),
         "rw": on(torch.zeros(4)), "top": on(torch.zeros(4, 2, dtype=torch.int64)), "teach": on(torch.zeros(4, 2)),
         "nw": on(torch.zeros(8))}
    call, error = REFUSED[name]
    with pytest.raises(error):
        call(t)
