"""dlrm_rmsnorm_fwd and dlrm_rmsnorm_bwd against 64-bit references: widths of
every launch shape, types, strided and unaligned rows, 8-bit rows, rows of
zeros, infinities and NaN.

Sums: a thread adds at most 32 squares in a chain and 10 shuffle steps follow,
so a mean of squares is good to 45 U, its reciprocal root to 25 U with the
root, the division and the mean's own roundings; 40 U is allowed."""
import pytest
import torch

import block_ref as R
import embedding_bags_dot_b200 as E

pytestmark = pytest.mark.gpu

WIDTHS = [1, 2, 7, 64, 100, 128, 130, 512, 1000, 1024, 2040, 2047, 4096, 4098, 5120, 8193, 16384, 32768]


def _inputs(rows, d, dt, residual, seed=0):
    g = torch.Generator().manual_seed(seed + d)
    x = torch.randn((rows, d), generator=g).to(R.DT[dt])
    r = (2 * torch.randn((rows, d), generator=g)).to(R.DT[dt]) if residual else None
    w = 1 + 0.1 * torch.randn(d, generator=g)
    return x, r, w


def _fwd(x, r, w, y_dt, eps=1e-6, want_h=True):
    rows, d = x.shape
    y = torch.zeros((rows, d), dtype=y_dt, device="cuda")
    h = torch.zeros((rows, d), dtype=x.dtype, device="cuda") if want_h else None
    s = torch.zeros(rows, device="cuda") if y_dt == torch.float8_e4m3fn else None
    rstd = torch.zeros(rows, device="cuda")
    c = lambda t: None if t is None else t.cuda()  # noqa: E731
    E.dlrm_rmsnorm_fwd(c(x), c(w), y, eps=eps, residual=c(r), h=h, y_scale=s, rstd=rstd)
    return y, h, s, rstd


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("d", WIDTHS)
@pytest.mark.parametrize("rows,residual", [(3, True), (700, False)])
def test_norm(dt, d, rows, residual):
    x, r, w = _inputs(rows, d, dt, residual)
    y, h, _, rstd = _fwd(x, r, w, R.DT[dt])
    wh, wr, wy = R.rmsnorm(x, r, w, 1e-6)
    step, tiny = R.half_step(R.DT[dt]), R.smallest(R.DT[dt])
    R.within(rstd, wr, 40 * R.U * wr, "rstd")
    R.within(h, wh, (step + R.U * (1 + step)) * wh.abs() + tiny, "h")
    R.within(y, wy, (step + 44 * R.U) * wy.abs() + tiny, "y")


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("d", WIDTHS)
@pytest.mark.parametrize("rows", [2, 500])
def test_norm_to_8_bits(dt, d, rows):
    x, r, w = _inputs(rows, d, dt, True, seed=5)
    y, _, s, _ = _fwd(x, r, w, torch.float8_e4m3fn)
    _, _, wy = R.rmsnorm(x, r, w, 1e-6)
    ws = wy.abs().amax(1) / 448
    R.within(s, ws, 48 * R.U * ws, "scale")
    got = y.float().cpu().double() * s.cpu().double()[:, None]
    # half a step of e4m3 relative to the value, or half of its smallest step 2^-9 in units of the scale
    bound = torch.maximum(2.0 ** -4 * wy.abs(), 2.0 ** -10 * ws[:, None]) + 96 * R.U * wy.abs()
    R.within(got, wy, bound, "8-bit y")
    assert float(y.float().abs().max()) == 448


def test_8_bit_rows_of_zeros_and_of_the_smallest_values():
    d = 256
    x = torch.zeros((4, d))
    x[1] = 1e-41 * torch.arange(d)            # h * rstd stays tiny under a large eps
    x[2] = 1e-33 * torch.arange(d)
    x[3, 5] = 1.0
    y, _, s, _ = _fwd(x, None, None, torch.float8_e4m3fn, eps=1.0)
    assert float(s[0]) == 0 and bool((y[0].float() == 0).all())
    got = y.float().cpu().double() * s.cpu().double()[:, None]
    _, _, wy = R.rmsnorm(x, None, None, 1.0)
    for i in (1, 2, 3):
        # the scale of row 1 is a subnormal of a few bits: half a quantum of 2^-149 on it, times 448
        tol = 2.0 ** -4 * wy[i].abs() + 2.0 ** -10 * float(s[i]) + 448 * 2.0 ** -150 + 1e-5 * wy[i].abs()
        assert bool(((got[i] - wy[i]).abs() <= tol).all()), i


@pytest.mark.parametrize("d", [64, 1000, 4096])
def test_non_finite_rows_stay_in_their_row(d):
    x, _, w = _inputs(6, d, "f32", False)
    clean_y, _, clean_s, _ = _fwd(x, None, w, torch.float8_e4m3fn)
    x[1, 3], x[3, d - 1], x[4, 0] = float("nan"), float("inf"), -float("inf")
    y, _, s, _ = _fwd(x, None, w, torch.float8_e4m3fn)
    got = y.float() * s[:, None]
    for i in (0, 2, 5):
        assert torch.equal(y[i].view(torch.uint8), clean_y[i].view(torch.uint8)) and s[i] == clean_s[i]
    for i in (1, 3, 4):
        assert bool(torch.isnan(got[i]).all())
    y2, _, _, _ = _fwd(x, None, w, torch.float32)
    assert bool(torch.isfinite(y2[[0, 2, 5]]).all()) and bool(torch.isnan(y2[1]).all())
    assert bool(torch.isnan(y2[3, d - 1])) and bool((y2[3, :3] == 0).all())   # inf * 0; finite / inf


@pytest.mark.parametrize("dt,off", [("bf16", 1), ("bf16", 2), ("f32", 1), ("f16", 4)])
def test_strided_rows_leave_their_neighbours(dt, off):
    rows, d, ld = 40, 96, 131
    base = torch.randn((rows, ld)).to(R.DT[dt])
    out = torch.full((rows, ld), 9.0, dtype=R.DT[dt], device="cuda")
    hb = torch.full((rows, ld), 9.0, dtype=R.DT[dt], device="cuda")
    x = base.cuda()[:, off:off + d]
    E.dlrm_rmsnorm_fwd(x, None, out[:, off:off + d], residual=x, h=hb[:, off:off + d])
    wh, _, wy = R.rmsnorm(base[:, off:off + d], base[:, off:off + d], None, 1e-6)
    step, tiny = R.half_step(R.DT[dt]), R.smallest(R.DT[dt])
    R.within(out[:, off:off + d], wy, (step + 44 * R.U) * wy.abs() + tiny, "y")
    R.within(hb[:, off:off + d], wh, (step + 2 * R.U) * wh.abs() + tiny, "h")
    for b in (out, hb):
        assert bool((b[:, :off] == 9).all()) and bool((b[:, off + d:] == 9).all())


def test_h_in_the_residuals_own_buffer():
    x, r, w = _inputs(300, 1024, "bf16", True)
    y0, h0, _, _ = _fwd(x, r, w, torch.bfloat16)
    res, y = r.cuda(), torch.empty((300, 1024), dtype=torch.bfloat16, device="cuda")
    E.dlrm_rmsnorm_fwd(x.cuda(), w.cuda(), y, residual=res, h=res)
    assert torch.equal(res, h0) and torch.equal(y, y0)


def _bwd(dy, h, rstd, w, dh, with_dw=True):
    rows, d = dy.shape
    c = lambda t: None if t is None else t.cuda()  # noqa: E731
    dx = torch.full((rows, d), float("nan"), dtype=dy.dtype, device="cuda")
    dw = torch.full((d,), float("nan"), device="cuda") if with_dw else None
    ws = E.alloc_workspace(E.dlrm_rmsnorm_bwd_workspace_size(rows, d))
    E.dlrm_rmsnorm_bwd(c(dy), c(h), c(rstd), c(w), dx, ws, dw=dw, dh=c(dh))
    return dx, dw


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("d", WIDTHS)
@pytest.mark.parametrize("rows,with_dh", [(1, False), (37, True), (1500, False)])
def test_norm_gradient(dt, d, rows, with_dh):
    if rows > 1000 and d > 8193:
        rows = 650
    dy, dh, w = _inputs(rows, d, dt, with_dh, seed=9)
    h = (2 * torch.randn((rows, d))).to(R.DT[dt])
    rstd = (h.double().square().mean(1) + 1e-6).rsqrt().float()
    dx, dw = _bwd(dy, h, rstd, w, dh)
    wx, ww, mx, mw = R.rmsnorm_grad(dy, h, rstd, w, dh)
    # the mean of g xh: chains of at most 32 and 10 steps, three roundings per term: 50 U of its magnitudes
    R.within(dx, wx, R.half_step(R.DT[dt]) * wx.abs() + 60 * R.U * mx + R.smallest(R.DT[dt]), "dx")
    # dw: a row's term has three roundings, and at most `rows` + 64 additions follow
    R.within(dw, ww, (rows + 70) * R.U * mw, "dw")


def test_norm_gradient_without_weight_or_rows():
    dy = torch.randn((50, 200))
    h = torch.randn((50, 200))
    rstd = (h.double().square().mean(1)).rsqrt().float()
    dx, dw = _bwd(dy, h, rstd, None, None, with_dw=False)
    wx, _, mx, _ = R.rmsnorm_grad(dy, h, rstd, None, None)
    R.within(dx, wx, 60 * R.U * mx, "dx without w")
    assert dw is None
    dx, dw = _bwd(torch.zeros((0, 200)), torch.zeros((0, 200)), torch.zeros(0), torch.ones(200), None)
    assert dx.numel() == 0 and bool((dw == 0).all())


def test_norm_gradient_agrees_with_differences():
    """Central differences of sum(c * norm(x)) in 64 bits along random directions."""
    rows, d = 5, 48
    g = torch.Generator().manual_seed(2)
    x, c, w = (torch.randn((rows, d), generator=g) for _ in range(3))
    w = w[0]
    rstd = (x.double().square().mean(1) + 1e-5).rsqrt().float()
    dx, dw = _bwd(c, x, rstd, w, None)
    f = lambda xx, ww: float((R.rmsnorm(xx, None, ww, 1e-5)[2] * c.double()).sum())  # noqa: E731
    for k in range(6):
        v, u, t = torch.randn((rows, d), generator=g).double(), torch.randn(d, generator=g).double(), 1e-5
        num = (f(x.double() + t * v, w.double()) - f(x.double() - t * v, w.double())) / (2 * t)
        assert abs(num - float((dx.cpu().double() * v).sum())) <= 1e-5 * float((dx.cpu().double() * v).abs().sum())
        num = (f(x.double(), w.double() + t * u) - f(x.double(), w.double() - t * u)) / (2 * t)
        assert abs(num - float((dw.cpu().double() * u).sum())) <= 1e-5 * float((dw.cpu().double() * u).abs().sum())


def test_norm_gradient_repeats_bit_for_bit():
    dy, dh, w = _inputs(3000, 768, "bf16", True)
    h = torch.randn((3000, 768)).to(torch.bfloat16)
    rstd = (h.double().square().mean(1)).rsqrt().float()
    a, b = _bwd(dy, h, rstd, w, dh), _bwd(dy, h, rstd, w, dh)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
