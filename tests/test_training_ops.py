"""Layer norm and the losses over a vocabulary, with their gradients, against
64-bit forms; refusals of the binding."""

import pytest
import torch

import mamba_selective_scan_amd as mss
from train_ref import f64, loss_ref, norm_back_ref, norm_ref, within

gpu = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
DEV = "cuda:0"


def note(msg):
    print(f"[gpu] {msg}", flush=True)


def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(g, *shape, dtype=F32, scale=1.0):
    return (torch.randn(*shape, generator=g) * scale).to(dtype).to(DEV)


# ---------------------------------------------------------------- layer norm

def check_norm(x, weight, bias, residual, eps=1e-5, **kw):
    was = None if residual is None else residual.clone()
    out = mss.layer_norm_fwd(x, weight, bias, residual=residual, eps=eps, **kw)
    torch.cuda.synchronize()
    ref = norm_ref(x, weight, bias, was, eps)
    for name, got in zip(("y", "mean", "rstd", "r"), out):
        within(name, got, *ref[name], got.dtype)
    return out


@gpu
@pytest.mark.parametrize("rows,dim", [(1, 1), (3, 7), (1, 768), (5, 512), (6, 513), (9, 1001), (4, 1025), (3, 2048),
                                      (2, 2049), (7, 2560), (2, 5120), (3, 8191), (2, 8200), (1, 16384), (2, 20001),
                                      (1, 32768)])
@pytest.mark.parametrize("dtype,res", [(BF16, None), (BF16, F32), (BF16, BF16), (F32, None), (F32, BF16)])
def test_layer_norm_fwd(rows, dim, dtype, res):
    note(f"layer_norm_fwd {rows} x {dim} {dtype} residual {res}")
    g = gen(rows * dim)
    x = randn(g, rows, dim, dtype=dtype) + 0.5
    check_norm(x, 1 + randn(g, dim, scale=0.1), randn(g, dim) if dim % 2 else None,
               None if res is None else randn(g, rows, dim, dtype=res, scale=2.0))


@gpu
def test_layer_norm_fwd_of_strided_rows_and_in_place():
    note("layer_norm_fwd of rows that start anywhere")
    g = gen(3)
    big = randn(g, 11, 301, dtype=BF16)
    res = randn(g, 11, 400)[:, 3:276]
    x, w, b = big[:, 5:278], randn(g, 273), randn(g, 273)
    out = torch.full((11, 300), 7.0, dtype=BF16, device=DEV)
    keep = res.clone()
    y, _, _, r = check_norm(x, w, b, res, out=out[:, 9:282], residual_out=res)
    assert r.data_ptr() == res.data_ptr() and torch.equal(res, x.float() + keep)
    assert (out[:, :9] == 7).all() and (out[:, 282:] == 7).all()
    # one row, and rows that are all the same row
    check_norm(x[:1], w, b, None)
    check_norm(x[:1].expand(6, -1), w, b, None)


@gpu
@pytest.mark.parametrize("scale,offset", [(1e-30, 0.0), (1e25, 0.0), (1.0, 3000.0), (1e-3, 1.0), (0.0, 2.0), (3e37, 0.0)])
def test_layer_norm_fwd_far_from_one(scale, offset):
    note(f"layer_norm_fwd of rows of scale {scale} about {offset}")
    g = gen(4)
    x = randn(g, 5, 600) * scale + offset
    check_norm(x, randn(g, 600), randn(g, 600), None, eps=0.0 if scale == 1e-30 else 1e-5)


@gpu
def test_layer_norm_fwd_keeps_what_is_not_finite_to_its_row():
    note("layer_norm_fwd with an infinity and a NaN")
    g = gen(5)
    x, w = randn(g, 4, 300), randn(g, 300)
    x[1, 7], x[2, 299] = float("inf"), float("nan")
    y, _, rstd = mss.layer_norm_fwd(x, w)
    assert y[1:3].isnan().all() and rstd[1:3].isnan().all()
    ref = norm_ref(x[::3], w, None, None, 1e-5)
    within("y", y[::3], *ref["y"], F32)


def back_case(rows, dim, dtype, r_dtype, with_dr, seed=0):
    g = gen(seed + rows * dim)
    dy = randn(g, rows, dim, dtype=dtype)
    r = randn(g, rows, dim, dtype=r_dtype, scale=2.0) + 0.25
    dr = randn(g, rows, dim, dtype=r_dtype) if with_dr else None
    mean = r.float().mean(1)
    rstd = torch.rsqrt((r.float() - mean[:, None]).square().mean(1) + 1e-5)
    return dy, r, 1 + randn(g, dim, scale=0.1), mean, rstd, dr


def check_back(case, **kw):
    dy, r, w, mean, rstd, dr = case
    got = mss.layer_norm_bwd(dy, r, w, mean, rstd, dr=dr, **kw)
    torch.cuda.synchronize()
    ref = norm_back_ref(*case)
    for name, t in got.items():
        within(name, t, *ref[name], t.dtype)
    return got


@gpu
@pytest.mark.parametrize("rows,dim", [(1, 1), (3, 7), (1, 768), (300, 512), (61, 1001), (13, 1025), (2100, 64),
                                      (1300, 2049), (70, 2560), (20, 5120), (5, 8191), (9, 8200), (3, 16384),
                                      (6, 20001), (2, 32768)])
@pytest.mark.parametrize("dtype,r_dtype,dr", [(BF16, BF16, False), (BF16, F32, True), (BF16, BF16, True),
                                              (F32, F32, False), (F32, BF16, True)])
def test_layer_norm_bwd(rows, dim, dtype, r_dtype, dr):
    note(f"layer_norm_bwd {rows} x {dim} {dtype} {r_dtype} dr {dr}")
    got = check_back(back_case(rows, dim, dtype, r_dtype, dr), bias=dim % 2 == 1)
    assert ("bias" in got) == (dim % 2 == 1)
    assert ("residual" in got) == (dr or r_dtype is not dtype)
    if dr and r_dtype is dtype:
        assert got["residual"] is got["x"]


@gpu
def test_layer_norm_bwd_of_strided_and_repeated_rows():
    note("layer_norm_bwd of strided rows")
    dy, r, w, mean, rstd, dr = back_case(12, 300, BF16, F32, True)
    case = (dy[:, 3:278], r[:, 9:284], w[:275].clone(), mean, rstd, dr[:, 25:])
    check_back(case)
    check_back((dy[:1, 3:278].expand(12, -1), *case[1:]))
    note("layer_norm_bwd without the parameters' sums")
    assert set(check_back(case, params=False)) == {"x", "residual"}


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_layer_norm_bwd_is_the_same_each_time(dtype):
    case = back_case(2500, 1536, dtype, F32, True)
    note("layer_norm_bwd twice")
    a, b = check_back(case), check_back(case)
    assert all(torch.equal(a[k], b[k]) for k in a)


@gpu
def test_layer_norm_of_no_rows():
    note("layer_norm of no rows")
    w = torch.ones(64, device=DEV)
    x = torch.empty(0, 64, device=DEV)
    y, mean, rstd = mss.layer_norm_fwd(x, w)
    assert y.shape == (0, 64) and mean.shape == rstd.shape == (0,)
    g = mss.layer_norm_bwd(x, x, w, mean, rstd)
    assert g["x"].shape == (0, 64) and not g["weight"].any() and not g["bias"].any()


@gpu
@pytest.mark.parametrize("with_res", [False, True])
def test_layer_norm_autograd(with_res):
    note(f"layer_norm autograd, residual {with_res}")
    g = gen(8)
    x = randn(g, 2, 33, 200, dtype=BF16).requires_grad_()
    w, b = (1 + randn(g, 200, scale=0.1)).requires_grad_(), randn(g, 200).requires_grad_()
    res = randn(g, 2, 33, 200).requires_grad_() if with_res else None
    dy, dr = randn(g, 2, 33, 200, dtype=BF16), randn(g, 2, 33, 200)
    if with_res:
        y, r = mss.layer_norm(x, w, b, res)
        grads = torch.autograd.grad((y, r), (x, w, b, res), (dy, dr))
    else:
        y = mss.layer_norm(x, w, b)
        grads = torch.autograd.grad(y, (x, w, b), dy)
        r, dr = x.detach().float(), None
    rows = lambda t: None if t is None else t.detach().reshape(-1, 200)
    wide = f64(rows(r))
    mean = wide.mean(1)
    rstd = 1 / torch.sqrt((wide - mean[:, None]).square().mean(1) + 1e-5)
    ref = norm_back_ref(rows(dy), rows(r), w, mean, rstd, rows(dr))
    for t, name in zip(grads, ("x", "weight", "bias", "residual")):
        bound = ref[name][1] * 1.5 + 3e-6 * ref[name][0].abs()  # (mean and rstd are fp32 there)
        bound = bound + 2.0 ** -20 * rstd.max() * f64(rows(dy)).abs().max() * (66 if name in ("weight", "bias") else 1)
        within(name, rows(t) if t.dim() == 3 else t, ref[name][0], bound, t.dtype)
    # expanded and transposed gradients
    y = mss.layer_norm(x, w, b)
    y.sum().backward()
    assert x.grad.shape == x.shape and x.grad.float().abs().max() < 1


@gpu
def test_layer_norm_gradients_of_leaves_are_their_own():
    note("layer_norm: x and residual of one dtype, gradients added up over two passes")
    g = gen(9)
    leaves = [randn(g, 7, 96).requires_grad_() for _ in range(2)]
    w, b = randn(g, 96).requires_grad_(), randn(g, 96).requires_grad_()
    dy, dr = randn(g, 7, 96), randn(g, 7, 96)

    def once():
        y, r = mss.layer_norm(leaves[0], w, b, leaves[1])
        return torch.autograd.grad((y, r), (*leaves, w, b), (dy, dr))

    want = [2 * t for t in once()]
    for _ in range(2):
        y, r = mss.layer_norm(leaves[0], w, b, leaves[1])
        torch.autograd.backward((y, r), (dy, dr))
    assert leaves[0].grad.data_ptr() != leaves[1].grad.data_ptr()
    assert all(torch.equal(t.grad, q) for t, q in zip((*leaves, w, b), want))
    # x itself as the residual: its gradient is the sum of both
    y, r = mss.layer_norm(leaves[0], w, b, leaves[0])
    both, = torch.autograd.grad((y, r), leaves[0], (dy, dr))
    assert both.shape == (7, 96) and both.isfinite().all()
    # only one of the outputs used, and gradients that are expanded or transposed views
    y, r = mss.layer_norm(leaves[0], w, None, leaves[1])
    one, = torch.autograd.grad(r.sum(), leaves[1])
    assert torch.equal(one, torch.ones_like(one))
    x = randn(g, 96, 7).t().requires_grad_()  # columns not adjacent
    dx, = torch.autograd.grad(mss.layer_norm(x, w, b), x, randn(g, 96, 7).t())
    assert dx.shape == x.shape
    with pytest.raises(RuntimeError):  # (no second derivative)
        dx, = torch.autograd.grad(mss.layer_norm(x, w, b).sum(), x, create_graph=True)
        torch.autograd.grad(dx.sum(), x)


@gpu
def test_layer_norm_outputs_may_change_in_place():
    note("layer_norm: outputs changed in place, one of two outputs used")
    g = gen(10)
    x, res = randn(g, 3, 5, 96, dtype=BF16).requires_grad_(), randn(g, 3, 5, 96).requires_grad_()
    w, b = randn(g, 96).requires_grad_(), randn(g, 96).requires_grad_()
    dy = randn(g, 3, 5, 96, dtype=BF16)
    y, r = mss.layer_norm(x, w, b, res)
    want = torch.autograd.grad((y, r), (x, res, w, b), (dy, torch.zeros_like(r)))
    # y alone: as with a gradient of 0 for r
    y, r = mss.layer_norm(x, w, b, res)
    assert all(torch.equal(p, q) for p, q in zip(torch.autograd.grad(y, (x, res, w, b), dy), want))
    y, r = mss.layer_norm(x, w, b, res)
    y.mul_(2)
    assert all(torch.equal(p, 2 * q) for p, q in zip(torch.autograd.grad(y, (x, res), dy), want))
    y = mss.layer_norm(x, w, b)
    y.add_(1)
    y.backward(dy)
    # r alone: its gradient passes through
    y, r = mss.layer_norm(x, w, b, res)
    dr = randn(g, 3, 5, 96)
    dx, dres, dw = torch.autograd.grad(r, (x, res, w), dr)
    assert torch.equal(dres, dr) and torch.equal(dx, dr.bfloat16()) and not dw.any()
    # r is read by the backward
    y, r = mss.layer_norm(x, w, b, res)
    r.add_(1)
    with pytest.raises(RuntimeError, match="inplace"):
        y.backward(dy)


# ---------------------------------------------------------------- losses

def loss_case(rows, dim, vocab, dtype, seed=0, ignored=0.0, spread=6.0):
    g = gen(seed + rows * dim + vocab)
    w = randn(g, vocab, dim, dtype=dtype, scale=dim ** -0.5)
    x = randn(g, rows, dim)
    ids = torch.randint(vocab, (rows,), generator=g).to(DEV)
    x = (x + spread * torch.rand(rows, 1, generator=g).to(DEV) * w[ids].float()).to(dtype)
    if ignored:
        ids[torch.rand(rows, generator=g).to(DEV) < ignored] = -100
    return x, w, ids


def top_case(rows, vocab, k, seed=0, dtype=F32, ragged=True):
    g = gen(seed + rows + k)
    ids = torch.stack([torch.randperm(vocab, generator=g)[:k] for _ in range(rows)])
    if ragged:
        ids[torch.rand(rows, k, generator=g) < 0.3] = -1
        ids[::5] = vocab + 3
    return ids.to(DEV), randn(g, rows, k, dtype=dtype, scale=3.0)


def check_loss(x, w, ids, teacher=None, row_weight=None, tau=1.0, scale=1.0, **kw):
    if teacher is None:
        fwd = mss.linear_cross_entropy_fwd(x, w, ids, logit_scale=scale)
        got = mss.linear_cross_entropy_grad(x, w, ids, row_weight, logit_scale=scale, **kw)
    else:
        fwd = mss.linear_distillation_fwd(x, w, ids, teacher, temperature=tau, logit_scale=scale)
        got = mss.linear_distillation_grad(x, w, ids, teacher, row_weight, temperature=tau, logit_scale=scale, **kw)
    torch.cuda.synchronize()
    ref = loss_ref(x, w, ids, teacher, row_weight, tau, scale)
    for name, t in zip(("loss", "lse", "dx", "dweight"), got):
        within(name, t, *ref[name], t.dtype)
    for name, t in zip(("loss", "lse"), fwd):
        within(f"{name} alone", t, *ref[name], t.dtype)
    return got


SIZES = [(1, 1, 1), (1, 8, 2), (2, 64, 100), (5, 33, 257), (1, 768, 1000), (17, 100, 63), (64, 64, 256), (65, 72, 300),
         (130, 200, 517), (257, 130, 1025), (300, 320, 777), (513, 96, 2100), (40, 1100, 600)]


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,dim,vocab", SIZES)
def test_cross_entropy(rows, dim, vocab, dtype):
    note(f"cross entropy {rows} x {dim} x {vocab} {dtype}")
    check_loss(*loss_case(rows, dim, vocab, dtype))


@gpu
@pytest.mark.parametrize("rows,dim,vocab", [(1, 20, 31), (3, 1030, 4099), (31, 31, 33), (32, 32, 64), (33, 129, 500),
                                            (64, 260, 1025), (65, 160, 96), (96, 95, 257), (97, 64, 130), (128, 600, 700),
                                            (129, 33, 300), (2, 5, 70000)])
def test_few_rows_of_fp32(rows, dim, vocab):
    """Up to 64 rows (128 without gradients) of fp32 read the matrix as it is: rows of
    it at any distance and any element, all rows, some and none with a target."""
    note(f"few rows of fp32 {rows} x {dim} x {vocab}")
    x, w, ids = loss_case(rows, dim, vocab, F32)
    wide = torch.full((vocab, dim + 5), float("nan"), device=DEV)
    wide[:, 1:dim + 1] = w
    check_loss(x, wide[:, 1:dim + 1], ids, scale=0.7)
    check_loss(x, w, torch.where(torch.arange(rows, device=DEV) % 3 == 1, ids, -100))
    check_loss(x, w, torch.full_like(ids, vocab))
    k = min(5, vocab)
    ids, teacher = top_case(rows, vocab, k)
    if k > 1:
        ids[:, 1] = ids[:, 0]  # (the same id twice)
    check_loss(x, w, ids, teacher, torch.rand(rows, generator=gen(4)).to(DEV), tau=1.3)


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("ignored", [0.4, 0.95, 1.0])
def test_cross_entropy_of_rows_without_a_target(dtype, ignored):
    note(f"cross entropy, {ignored} of the rows without a target, {dtype}")
    x, w, ids = loss_case(301, 136, 900, dtype, ignored=ignored)
    ids[7::50] = w.shape[0]  # (one past the vocabulary does not count either)
    ids[9::70] = 2 ** 40
    ids[11::70] = -2 ** 62
    off = (ids < 0) | (ids >= w.shape[0])
    weight = torch.rand(301, generator=gen(1)).to(DEV)
    x = x.clone()
    x[off] = float("nan")
    x[off.nonzero()[::2, 0]] = float("inf")
    weight[off] = float("nan")
    loss, lse, dx, dw = check_loss(x, w, ids, row_weight=weight)
    assert not loss[off].any() and not lse[off].any() and not dx[off].any()
    loss, lse, dx, dw = check_loss(x, w, ids)
    if ignored == 1.0:
        assert not dw.any()


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_losses_of_strided_inputs_and_outputs(dtype):
    note(f"losses of strided inputs {dtype}")
    g = gen(2)
    x, w, ids = loss_case(90, 200, 400, dtype)
    for xa, wa, d in ((1, 1, 131), (3, 8, 136), (8, 3, 128), (8, 8, 128)):
        dx = torch.full((90, 160), 7.0, dtype=dtype, device=DEV)
        dw = torch.full((400, 160), 7.0, dtype=dtype, device=DEV)
        check_loss(x[:, xa:xa + d], w[:, wa:wa + d], torch.stack([ids, ids + 1], 1)[:, 0],
                   dx=dx[:, 2:2 + d], dweight=dw[:, 5:5 + d])
        assert (dx[:, :2] == 7).all() and (dx[:, 2 + d:] == 7).all()
        assert (dw[:, :5] == 7).all() and (dw[:, 5 + d:] == 7).all()
    # the gaps between a padded matrix's rows are not read into anything
    wide = torch.full((400, 264), float("nan"), dtype=dtype, device=DEV)
    wide[:, :200] = w
    check_loss(x, wide[:, :200], ids)
    # the same hidden state in every row, and every second vocabulary entry
    check_loss(x[:1].expand(90, -1), w[::2], ids // 2)
    tops, teacher = top_case(7, 200, 90)
    check_loss(x, w[:200], tops.t()[:90], teacher.t()[:90], tau=1.5)


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,dim,vocab,k,tau", [(1, 8, 2, 1, 1.0), (9, 64, 300, 8, 2.0), (130, 100, 517, 13, 0.7),
                                                  (61, 72, 700, 300, 3.0), (40, 200, 1500, 64, 1.0),
                                                  (12, 40, 2000, 1024, 2.0)])
def test_distillation(rows, dim, vocab, k, tau, dtype):
    note(f"distillation {rows} x {dim} x {vocab} top {k} at {tau} {dtype}")
    x, w, _ = loss_case(rows, dim, vocab, dtype)
    ids, teacher = top_case(rows, vocab, k, dtype=dtype)
    ids[-1, 0] = 0
    check_loss(x, w, ids, teacher, tau=tau, scale=0.8)
    check_loss(x, w, ids, teacher.float(), torch.rand(rows, generator=gen(1)).to(DEV) - 0.3, tau=tau)


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_distillation_of_masked_and_repeated_entries(dtype):
    note(f"distillation with masked and repeated entries {dtype}")
    x, w, _ = loss_case(40, 96, 300, dtype)
    ids, teacher = top_case(40, 300, 6, ragged=False)
    ids[3] = 5                                   # one id six times
    ids[4, 1] = ids[4, 0]
    teacher[5, 2] = float("-inf")                # an entry without a share
    teacher[6] = torch.finfo(F32).min            # the type's lowest value, alike: equal shares
    teacher[7, 1:] = torch.finfo(F32).min
    ids[8, 3:] = -1
    teacher[8, 3:] = float("nan")                # what does not count may hold anything
    ids[9] = 300
    teacher[9] = float("inf")
    ids[10, 1:] = -7
    check_loss(x, w, ids, teacher, tau=1.0)
    check_loss(x, w, ids, teacher, tau=0.5)


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_sure_and_surprised_rows(dtype):
    note(f"cross entropy of sure rows {dtype}")
    x, w, ids = loss_case(50, 128, 500, dtype, spread=0.0)
    x = (30.0 * w[ids].float() / w[ids].float().norm(dim=1, keepdim=True) ** 2).to(dtype)
    check_loss(x, w, ids)           # probabilities near 1
    check_loss(-x, w, ids)          # and near 0
    check_loss(x * 8, w, (ids + 1) % 500)
    check_loss(x, w, ids, scale=-0.25)
    check_loss(x, w, ids, scale=0.0)


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_what_is_not_finite_reaches_what_the_formula_says(dtype):
    note(f"cross entropy with a NaN row {dtype}")
    x, w, ids = loss_case(70, 64, 300, dtype)
    x[3, 5] = float("nan")
    x[4, 6] = float("inf")
    loss, lse, dx, dw = mss.linear_cross_entropy_grad(x, w, ids)
    assert loss[3:5].isnan().all() and dx[3:5].isnan().all()
    keep = [i for i in range(70) if i not in (3, 4)]
    ref = loss_ref(x[keep], w, ids[keep], row_weight=torch.full((68,), 1 / 70))
    within("loss", loss[keep], *ref["loss"], F32)
    within("dx", dx[keep], *ref["dx"], dtype)
    assert dw.isnan().all()


@gpu
def test_only_the_gradients_that_are_wanted():
    note("losses with one of the two gradients")
    x, w, ids = loss_case(100, 128, 600, BF16)
    full = mss.linear_cross_entropy_grad(x, w, ids)
    xg, wg = x.clone().requires_grad_(), w.clone().requires_grad_()
    mss.linear_cross_entropy(xg, w, ids).backward()
    assert torch.equal(xg.grad, full[2])
    mss.linear_cross_entropy(x, wg, ids).backward()
    assert torch.equal(wg.grad, full[3])
    with torch.no_grad():
        mean = mss.linear_cross_entropy(x, w, ids)
    assert abs(mean.item() - full[0].double().mean().item()) < 1e-6 * abs(mean.item())


@gpu
@pytest.mark.parametrize("op", ["entropy", "distill"])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_losses_autograd(op, dtype):
    note(f"{op} autograd {dtype}")
    x, w, ids = loss_case(6 * 11, 72, 300, dtype, ignored=0.2)
    teacher = None
    if op == "distill":
        ids, teacher = top_case(66, 300, 5)
    x3 = x.view(6, 11, 72).clone().requires_grad_()
    w = w.clone().requires_grad_()
    rows = torch.rand(66, generator=gen(3)).to(DEV)
    for rw in (None, rows):
        rw3 = None if rw is None else rw.view(6, 11)
        if op == "entropy":
            total = mss.linear_cross_entropy(x3, w, ids.view(6, 11), rw3, logit_scale=0.5)
        else:
            total = mss.linear_distillation(x3, w, ids.view(6, 11, 5), teacher.view(6, 11, 5), rw3, temperature=2.0,
                                            logit_scale=0.5)
        dx, dw = torch.autograd.grad(total * 2.0, (x3, w))
        ref = loss_ref(x, w, ids, teacher, rw, 2.0 if op == "distill" else 1.0, 0.5)
        within("dx", dx.view(66, 72), 2 * ref["dx"][0], 2 * ref["dx"][1], dtype)
        within("dweight", dw, 2 * ref["dweight"][0], 2 * ref["dweight"][1], dtype)
        live = ref["lse"][0] != 0
        c = live.double() / live.sum() if rw is None else f64(rw)
        want, off = (c * ref["loss"][0]).sum(), (c * ref["loss"][1]).sum()
        assert abs(total.item() - want.item()) <= off.item() + 4e-7 * abs(want.item())


@gpu
@pytest.mark.parametrize("op", ["entropy", "distill"])
def test_gradients_against_differences(op):
    """Central differences of the kernels' own mean loss along random directions:
    with a step of 2^-6 along directions of unit elements' size 1 / sqrt(n) the
    third derivative leaves less than 2^-12 of |direction| (logits move by less
    than 2^-4), and the fp32 losses' rounding 2^-24 * 8 / 2^-6."""
    note(f"{op}: gradients against differences")
    x, w, ids = loss_case(50, 64, 200, F32)
    if op == "entropy":
        call = lambda a, b: mss.linear_cross_entropy(a, b, ids).double().item()
        g = mss.linear_cross_entropy_grad(x, w, ids)
    else:
        ids, teacher = top_case(50, 200, 7)
        call = lambda a, b: mss.linear_distillation(a, b, ids, teacher, temperature=1.5).double().item()
        g = mss.linear_distillation_grad(x, w, ids, teacher, temperature=1.5)
    step = 2.0 ** -6
    for seed in range(3):
        r = gen(seed)
        for t, grad, put in ((x, g[2], lambda v: (v, w)), (w, g[3], lambda v: (x, v))):
            d = randn(r, *t.shape)
            d /= d.norm()
            slope = (call(*put(t + step * d)) - call(*put(t - step * d))) / (2 * step)
            want = (grad.double() * d.double()).sum().item()
            assert abs(slope - want) < 2.0 ** -12, (seed, slope, want)


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_losses_are_the_same_each_time(dtype):
    note(f"losses twice {dtype}")
    x, w, ids = loss_case(700, 256, 1500, dtype, ignored=0.2)
    a = mss.linear_cross_entropy_grad(x, w, ids)
    b = mss.linear_cross_entropy_grad(x, w, ids)
    assert all(torch.equal(p, q) for p, q in zip(a, b))


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_losses_of_no_rows(dtype):
    note(f"losses of no rows {dtype}")
    x, w, ids = loss_case(4, 64, 300, dtype)
    loss, lse, dx, dw = mss.linear_cross_entropy_grad(x[:0], w, ids[:0])
    assert loss.shape == lse.shape == (0,) and dx.shape == (0, 64) and not dw.any()
    assert mss.linear_cross_entropy(x[:0], w, ids[:0]).item() == 0
    tops, teacher = top_case(4, 300, 3)
    assert not mss.linear_distillation_grad(x[:0], w, tops[:0], teacher[:0])[3].any()
    assert mss.linear_distillation(x[:0].view(2, 0, 64), w, tops[:0].view(2, 0, 3), teacher[:0].view(2, 0, 3)).item() == 0


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,dim,vocab", [(2300, 64, 300), (1500, 72, 120), (3000, 8, 5), (130, 1032, 64), (700, 2051, 90)])
def test_products_cut_along_their_sums(rows, dim, vocab, dtype):
    """Few tiles: dweight's sum over the rows, and dx's over the vocabulary, in parts."""
    note(f"cross entropy of few tiles {rows} x {dim} x {vocab} {dtype}")
    x, w, ids = loss_case(rows, dim, vocab, dtype, ignored=0.3)
    check_loss(x, w, ids, row_weight=torch.rand(rows, generator=gen(2)).to(DEV))


@gpu
def test_the_gradients_of_a_loss_are_taken_once_and_kept():
    note("losses: a second backward pass, a scaled total, a second derivative")
    x, w, ids = loss_case(60, 64, 300, BF16)
    x.requires_grad_()
    total = mss.linear_cross_entropy(x, w, ids)
    a, = torch.autograd.grad(total, x, retain_graph=True)
    b, = torch.autograd.grad(total * 4, x)
    assert torch.equal(a * 4, b)
    assert torch.equal(a, mss.linear_cross_entropy_grad(x.detach(), w, ids)[2])
    wide = x.detach().t().contiguous().t().requires_grad_()  # columns not adjacent
    c, = torch.autograd.grad(mss.linear_cross_entropy(wide, w, ids), wide)
    assert torch.equal(a, c)
    with pytest.raises(RuntimeError):  # (no second derivative)
        d, = torch.autograd.grad(mss.linear_cross_entropy(x, w, ids), x, create_graph=True)
        torch.autograd.grad(d.float().sum(), x)


@gpu
def test_two_losses_at_once_on_two_streams():
    note("losses on two streams")
    cases = [loss_case(400, 256, 5000, BF16, seed=s) for s in (1, 2)]
    want = [mss.linear_cross_entropy_grad(*c) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for turn in range(5):
        got = []
        for c, s in zip(cases, streams):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                got.append(mss.linear_cross_entropy_grad(*c))
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for a, b in zip(got, want) for p, q in zip(a, b))


@gpu
def test_what_lies_around_the_outputs_and_the_workspace():
    """Outputs and a workspace of exactly the size asked for in the middle of larger
    buffers: nothing outside them changes, whatever the workspace held before."""
    note("losses between guards")
    import ctypes
    from mamba_selective_scan_amd import _lib, heads
    for dtype, (rows, dim, vocab) in ((BF16, (150, 136, 777)), (F32, (150, 100, 777)), (BF16, (40, 64, 3001))):
        x, w, ids = loss_case(rows, dim, vocab, dtype, ignored=0.2)
        sizes = []
        real = heads._give_workspace
        want = mss.linear_cross_entropy_grad(x, w, ids)
        import mamba_selective_scan_amd.training as training
        def spy(a, need, workspace, device):
            sizes.append(need)
            return real(a, need, workspace, device)
        training._give_workspace = spy
        try:
            mss.linear_cross_entropy_grad(x, w, ids)
        finally:
            training._give_workspace = real
        need = sizes[0]
        for fill in (0xff, 0x7f, 0):
            big = torch.full((need + 2048,), fill, dtype=torch.uint8, device=DEV)
            dx = torch.full((rows + 4, dim), 3.0, dtype=dtype, device=DEV)
            dw = torch.full((vocab + 4, dim), 3.0, dtype=dtype, device=DEV)
            got = mss.linear_cross_entropy_grad(x, w, ids, dx=dx[2:-2], dweight=dw[2:-2],
                                                workspace=big[1024:1024 + need])
            torch.cuda.synchronize()
            assert all(torch.equal(p, q) for p, q in zip(got, want)), (dtype, fill)
            assert (big[:1024] == fill).all() and (big[1024 + need:] == fill).all()
            for t in (dx, dw):
                assert (t[:2] == 3).all() and (t[-2:] == 3).all()
        with pytest.raises(mss.MssError, match="WORKSPACE"):
            mss.linear_cross_entropy_grad(x, w, ids, workspace=big[:need - 1])


@gpu
def test_rows_in_pieces():
    """More rows than one piece of dz holds: 2^31 bytes over a little more than
    2 * 65536 a row are 16000 rows, so 17000 take two; against one piece of each half."""
    note("cross entropy in two pieces")
    g = gen(11)
    x, w, ids = loss_case(17000, 64, 65536, BF16, ignored=0.05)
    rw = (torch.rand(17000, generator=g) / 17000).to(DEV)
    loss, lse, dx, dw = mss.linear_cross_entropy_grad(x, w, ids, rw)
    halves = [mss.linear_cross_entropy_grad(x[s], w, ids[s], rw[s]) for s in (slice(0, 8500), slice(8500, 17000))]
    assert torch.equal(loss, torch.cat([h[0] for h in halves]))
    assert torch.equal(lse, torch.cat([h[1] for h in halves]))
    # the same sums of the same bf16 values in another order and grouping
    a, b = dx.double(), torch.cat([h[2] for h in halves]).double()
    assert ((a - b).norm() / b.norm()).item() < 2.0 ** -8
    a, b = dw.double(), halves[0][3].double() + halves[1][3].double()
    assert ((a - b).norm() / b.norm()).item() < 2.0 ** -7


@gpu
def test_training_ops_in_a_graph_and_on_another_stream():
    """A captured step (norm, then both losses, with gradients) replayed with new
    inputs between other work gives the eager results."""
    note("norm and losses captured")
    x0, w, ids = loss_case(200, 128, 900, BF16, ignored=0.1)
    tops, teacher = top_case(200, 900, 4)
    nw, nb = torch.ones(128, device=DEV), torch.zeros(128, device=DEV)
    res = randn(gen(1), 200, 128)
    x = x0.clone()

    def step():
        y, mean, rstd, r = mss.layer_norm_fwd(x, nw, nb, residual=res)
        a = mss.linear_cross_entropy_grad(y, w, ids)
        b = mss.linear_distillation_grad(y, w, tops, teacher, temperature=2.0)
        g = mss.layer_norm_bwd(a[2] + b[2], r, nw, mean, rstd)
        return (*a, *b, *g.values())

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        eager = [t.clone() for t in step()]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for turn in range(4):
        x.copy_(x0 * (1.0 + 0.25 * turn))
        graph.replay()
        got = [t.clone() for t in out]
        torch.cuda.synchronize()
        want = step()
        torch.cuda.synchronize()
        note(f"replay {turn}")
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        if turn == 0:
            assert all(torch.equal(a, b) for a, b in zip(got, eager))


@gpu
def test_a_training_step_through_autograd():
    """scan -> norm (with the residual) -> vocabulary loss: gradients of a small
    model against the same model in 64 bits."""
    note("scan, norm and loss through autograd")
    g = gen(21)
    B, D, L, N, V = 2, 48, 40, 16, 130
    mk = lambda *s, k=1.0: randn(g, *s, scale=k)
    u, res = mk(B, D, L).requires_grad_(), mk(B, L, D).requires_grad_()
    dt, bb, cc, a_log = mk(B, D, L, k=0.3), mk(B, N, L), mk(B, N, L), mk(D, N, k=0.2)
    w, b = (1 + mk(D, k=0.1)).requires_grad_(), mk(D, k=0.1).requires_grad_()
    vocab = mk(V, D, k=D ** -0.5).requires_grad_()
    ids = torch.randint(-1, V, (B, L), generator=g).to(DEV)
    y = mss.selective_scan(u, dt, a_log, bb, cc)
    y, r = mss.layer_norm(y.transpose(1, 2), w, b, res)
    total = mss.linear_cross_entropy(y, vocab, ids) + 1e-3 * r.square().mean()
    got = torch.autograd.grad(total, (u, res, w, b, vocab))

    p = [t.detach().double().cpu().requires_grad_() for t in (u, res, w, b, vocab)]
    delta = torch.nn.functional.softplus(f64(dt))
    state, ys = torch.zeros(B, D, N, dtype=torch.float64), []
    for t in range(L):
        state = state * torch.exp(-delta[:, :, t, None] * f64(a_log).exp()) \
            + (delta[:, :, t] * p[0][:, :, t])[..., None] * f64(bb)[:, None, :, t]
        ys.append((state * f64(cc)[:, None, :, t]).sum(2))
    r64 = torch.stack(ys, 1) + p[1]
    y64 = (r64 - r64.mean(2, keepdim=True)) / torch.sqrt(r64.var(2, keepdim=True, correction=0) + 1e-5) * p[2] + p[3]
    logp = torch.log_softmax(y64 @ p[4].t(), 2)
    on = (ids >= 0).cpu()
    picked = logp.gather(2, ids.cpu().clamp(min=0)[..., None]).squeeze(2)
    want_total = -(picked * on).sum() / on.sum() + 1e-3 * r64.square().mean()
    want = torch.autograd.grad(want_total, p)
    assert abs(total.item() - want_total.item()) < 1e-5 * abs(want_total.item())
    for name, a, q in zip(("u", "residual", "weight", "bias", "vocab"), got, want):
        err = (f64(a) - q).norm() / q.norm()
        note(f"{name}: {err:.2e}")
        assert err < 2e-5, name  # (1e2 roundings of fp32 in a row, 6e-8 each)
