"""Layer norm and the losses past 32-bit offsets: tensors of more than 2^31
elements or bytes, sampled rows against 64-bit forms on the device."""

import pytest
import torch

import mamba_selective_scan_amd as mss
from train_ref import half_step

gpu = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
DEV = "cuda:0"


def note(msg):
    print(f"[gpu] {msg}", flush=True)


def fill(shape, dtype, seed, scale=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    t = torch.empty(shape, dtype=dtype, device=DEV)
    for part in t.split(max(1, (1 << 28) // shape[1])):
        part.copy_(torch.randn(part.shape, generator=g, device=DEV) * scale)
    return t


def close(name, got, ref, dtype, extra):
    """Within half a step of the type and `extra` of the row's largest value."""
    off = (got.double() - ref).abs()
    limit = half_step(dtype) * ref.abs() * 1.01 + extra * ref.abs().amax(-1, keepdim=True) + 1e-30
    worst = (off / limit).max().item()
    note(f"{name}: {worst:.3f} of the bound")
    assert worst <= 1, name


@gpu
def test_layer_norm_past_2_31_elements():
    rows, dim = 270000, 8192   # 2.2e9 elements, 4.4 GB in bf16
    note(f"layer_norm {rows} x {dim}")
    x = fill((rows, dim), BF16, 1)
    w, b = fill((1, dim), F32, 2)[0], fill((1, dim), F32, 3)[0]
    y, mean, rstd = mss.layer_norm_fwd(x, w, b)
    pick = torch.tensor([0, 1, 65535, 131071, 131072, 262143, 262144, rows - 1], device=DEV)
    r = x[pick].double()
    mid = r - r.mean(1, keepdim=True)
    h = mid / torch.sqrt(mid.square().mean(1, keepdim=True) + 1e-5)
    # (sums of 8192 values in 64 roundings; a row's y is a few times its weights)
    close("y", y[pick], h * w.double() + b.double(), BF16, 64 * 2.0 ** -24)
    g = mss.layer_norm_bwd(y, x, w, mean, rstd)
    dy = y[pick].double()
    gg = dy * w.double()
    d = (gg - gg.mean(1, keepdim=True) - h * (gg * h).mean(1, keepdim=True)) * rstd[pick].double()[:, None]
    close("dx", g["x"][pick], d, BF16, 256 * 2.0 ** -24)
    db = sum(p.double().sum(0) for p in y.split(8192))
    scale = sum(p.double().abs().sum(0) for p in y.split(8192))
    assert ((g["bias"].double() - db).abs() <= (rows / 1024 + 64) * 2.0 ** -24 * scale).all()


@gpu
@pytest.mark.parametrize("dtype,rows,dim,vocab", [(BF16, 150, 4096, 540000), (F32, 70, 2048, 400000)])
def test_losses_past_32_bit_offsets(dtype, rows, dim, vocab):
    """A vocabulary's matrix past 2^32 bytes (fp32: its planes past it), and its gradient."""
    note(f"cross entropy {rows} x {dim} x {vocab} {dtype}")
    w = fill((vocab, dim), dtype, 5, dim ** -0.5)
    x = fill((rows, dim), dtype, 6)
    ids = torch.randint(vocab, (rows,), generator=torch.Generator().manual_seed(1)).to(DEV)
    ids[0], ids[1], ids[2], ids[3] = vocab - 1, 0, -100, vocab // 2
    loss, lse, dx, dw = mss.linear_cross_entropy_grad(x, w, ids)
    live = ids >= 0
    n = int(live.sum())
    z = torch.cat([x.double() @ part.double().t() for part in w.split(1 << 16)], 1)
    want = torch.logsumexp(z, 1)
    held = z.gather(1, ids.clamp(min=0)[:, None])[:, 0]
    zero = torch.zeros_like(want)
    # (logits of 2048 to 4096 products and sums over 4000 to 6000 tiles in fp32)
    assert ((lse.double() - torch.where(live, want, zero)).abs() < 1e-5 * want.abs().max()).all()
    assert ((loss.double() - torch.where(live, want - held, zero)).abs() < 2e-5 * want.abs().max()).all()
    p = torch.exp(z - want[:, None])
    p[torch.arange(rows, device=DEV), ids.clamp(min=0)] -= 1
    p *= (live.double() / n)[:, None]
    ref = sum(p[:, a:a + (1 << 16)] @ w[a:a + (1 << 16)].double() for a in range(0, vocab, 1 << 16))
    loose = 2.0 ** -8 if dtype is BF16 else 1e-5  # (dz in bf16, or the logits' roundings)
    close("dx", dx[live], ref[live], dtype, loose)
    assert not dx[2].any()
    pick = torch.cat([ids[live], torch.tensor([1, 262143, 262144, 399999, vocab - 2], device=DEV)])
    close("dweight", dw[pick], p[:, pick].t() @ x.double(), dtype, loose)
