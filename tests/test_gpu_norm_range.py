"""dlrm_rmsnorm_fwd where a row's mean square leaves fp32: rows of zeros under
eps = 0, rows whose squares underflow or overflow under an eps as small (and
overflow under an ordinary one), and the backward pass of what the forward
stored for them.

Such a row's squares are those of its values times a power of two, which is
exact: the bounds are those of an ordinary row (40 U for rstd, 44 U and half a
step for y), and half the smallest fp32 step for an rstd that is itself
subnormal: at least 2.9e-39 = 2^-128, so half a step is at most 4 U of it, which
y's 44 U have room for beside the 25 U of its own chain of roundings."""
import pytest
import torch

import block_ref as R
import embedding_bags_dot_b200 as E

pytestmark = pytest.mark.gpu

# every launch shape: a warp a row, a block a row, rows ahead in shared memory, 32 elements a thread
SHAPES = [(5, 64), (600, 96), (5, 1000), (600, 1001), (700, 4096), (5, 20_000), (300, 20_000)]
MOST = torch.finfo(torch.float32).max


def _fwd(x, r, w, eps, q8):
    rows, d = x.shape
    c = lambda t: None if t is None else t.cuda()  # noqa: E731
    y = torch.zeros((rows, d), dtype=torch.float8_e4m3fn if q8 else x.dtype, device="cuda")
    s = torch.full((rows,), -1.0, device="cuda") if q8 else None
    h, rstd = torch.zeros((rows, d), dtype=x.dtype, device="cuda"), torch.full((rows,), -1.0, device="cuda")
    E.dlrm_rmsnorm_fwd(c(x), c(w), y, eps=eps, residual=c(r), h=h, y_scale=s, rstd=rstd)
    return y, s, h, rstd


def _check(x, w, eps, y, s, rstd, dt):
    _, wr, wy = R.rmsnorm(x, None, w, eps)
    zero = (x == 0).all(1) if eps == 0 else torch.zeros(len(x), dtype=torch.bool)
    most = (MOST / wr).clamp(max=1)               # rstd is at most fp32's largest number
    wr, wy = torch.where(zero, 0.0, wr * most), torch.where(zero[:, None], 0.0, wy * most[:, None])
    R.within(rstd, wr, 40 * R.U * wr + R.smallest(torch.float32), "rstd")
    if s is None:
        R.within(y, wy, (R.half_step(R.DT[dt]) + 44 * R.U) * wy.abs() + R.smallest(R.DT[dt]), "y")
    else:
        ws = wy.abs().amax(1) / 448
        # A scale among fp32's subnormals is off by half their step, 2^-150, however exact max|y| is, and max|y| / 448 by
        # 2^-150 / 448 where max|y| is one itself: together below 2^-149. A code is at most 448 of them.
        tiny = 2.0 ** -149
        R.within(s, ws, 48 * R.U * ws + tiny, "scale")
        got = y.float().cpu().double() * s.cpu().double()[:, None]
        # half a step of e4m3 relative to the value, or half of its smallest step 2^-9 in units of the scale
        R.within(got, wy, torch.maximum(2.0 ** -4 * wy.abs(), 2.0 ** -10 * ws[:, None]) + 96 * R.U * wy.abs() + 448 * tiny, "8-bit y")


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("rows,d", SHAPES)
def test_rows_of_zeros_without_eps(dt, q8, rows, d):
    g = torch.Generator().manual_seed(d)
    x = torch.randn((rows, d), generator=g).to(R.DT[dt])
    r = torch.randn((rows, d), generator=g).to(R.DT[dt])
    w = 1 + 0.1 * torch.randn(d, generator=g)
    none = torch.tensor([1, rows - 1])
    x[none] = 0
    y, s, h, rstd = _fwd(x, None, w, 0.0, q8)
    assert bool((y[none].float() == 0).all()) and bool((rstd[none] == 0).all()) and bool((h[none] == 0).all())
    assert s is None or bool((s[none] == 0).all())
    _check(x, w, 0.0, y, s, rstd, dt)
    # a residual that cancels x
    r[none] = x[none] = torch.randn(d, generator=g).to(R.DT[dt])
    r[none] *= -1
    y, s, h, rstd = _fwd(x, r, w, 0.0, q8)
    assert bool((y[none].float() == 0).all()) and bool((rstd[none] == 0).all())
    assert not bool(torch.isnan(y.float()).any())


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("rows,d", SHAPES)
def test_rows_whose_squares_leave_fp32(dt, q8, rows, d):
    g = torch.Generator().manual_seed(d)
    far = [1e-20, 1e-25, 1e-30, 1e-37, 1e18, 1e19, 1e25, 4e37] + ([1e-42] if dt == "f32" else [])
    if rows < 8:
        far = [far[i] for i in (1, 3, 6, 7)]
    x = torch.randn((rows, d), generator=g)
    for i, f in enumerate(far):
        x[1 + i] *= f
    x[0] = x[0] * 1e-3 + 1e-30                   # and rows that do not
    x = x.to(R.DT[dt])
    w = 1 + 0.1 * torch.randn(d, generator=g)
    assert bool(torch.isfinite(x).all())
    for eps in (0.0, 1e-38):
        y, s, _, rstd = _fwd(x, None, w, eps, q8)
        _check(x, w, eps, y, s, rstd, dt)
    # an eps that keeps small rows ordinary: those that overflow have rstd 0 and zeros, the others are exact
    y, s, _, rstd = _fwd(x, None, w, 1e-6, q8)
    over = (x.double().square().sum(1) > MOST)
    assert bool(over.any()) and bool((rstd.cpu()[over] == 0).all()) and bool((y.cpu()[over].float() == 0).all())
    _check(x[~over], w, 1e-6, y.cpu()[~over], None if s is None else s.cpu()[~over], rstd.cpu()[~over], dt)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("rows,d", [(9, 64), (9, 1000), (400, 4096), (9, 20_000)])
def test_gradient_of_such_rows(dt, rows, d):
    g = torch.Generator().manual_seed(d)
    x = torch.randn((rows, d), generator=g)
    x[1], x[2], x[3], x[4] = 0, x[2] * 1e25, x[3] * 1e-15, x[4] * 4e37
    x = x.to(R.DT[dt])
    dy, dh = (torch.randn((rows, d), generator=g).to(R.DT[dt]) for _ in range(2))
    w = 1 + 0.1 * torch.randn(d, generator=g)
    _, _, h, rstd = _fwd(x, None, w, 0.0, False)
    dx, dw = torch.empty_like(h), torch.empty(d, device="cuda")
    ws = E.alloc_workspace(E.dlrm_rmsnorm_bwd_workspace_size(rows, d))
    E.dlrm_rmsnorm_bwd(dy.cuda(), h, rstd, w.cuda(), dx, ws, dw=dw, dh=dh.cuda())
    assert torch.equal(dx[1].cpu(), dh[1])       # a row of zeros without eps passes on what comes by other ways
    wx, ww, mx, mw = R.rmsnorm_grad(dy, h.cpu(), rstd.cpu(), w, dh)
    R.within(dx, wx, R.half_step(R.DT[dt]) * wx.abs() + 60 * R.U * mx + R.smallest(R.DT[dt]), "dx")
    R.within(dw, ww, (rows + 70) * R.U * mw, "dw")
