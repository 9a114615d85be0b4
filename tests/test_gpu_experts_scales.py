"""dlrm_experts_fwd on 8-bit rows whose scales are far apart: the product of a
row's and a weight row's scale leaves fp32, or falls among its subnormals,
while the result does not.

Codes are eighths, so sums are exact; two scalings follow, and one
rounding of the output: well within the 1e-5 of the sum of magnitudes that the
products are held to, beside half the output's smallest step."""
import pytest
import torch

import block_ref as R
import embedding_bags_dot_b200 as E

pytestmark = pytest.mark.gpu

# single-SM tiles of 64 and 128 columns, SM pairs; ragged and odd
SIZES = [([5, 40, 0, 1], 2, 70, 64), ([33, 128, 7], 1, 200, 479), ([4000, 257, 2500], 3, 1024, 479)]


@pytest.mark.parametrize("y_dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("sizes,spare,N,K", SIZES)
def test_scales_far_apart(y_dt, sizes, spare, N, K):
    g = torch.Generator().manual_seed(N)
    M, n_exp = sum(sizes) + spare, len(sizes)
    X = torch.randint(-3, 4, (M, K), generator=g).float() / 8
    W = torch.randint(-3, 4, (n_exp, N, K), generator=g).float() / 8
    X[::5] = 0                                   # sums of exactly zero, under every pair of scales
    pick = lambda values, shape: torch.tensor(values)[torch.randint(0, len(values), shape, generator=g)]  # noqa: E731
    # pairs whose results are ordinary, subnormal, zero, or beyond the largest number
    xs = pick([0.0, 1e-42, 1e-36, 1e-22, 0.01, 1.0, 1e20, 3e37], (M,))
    wsc = pick([1e-42, 1e-38, 1e-5, 1.0, 1e10, 1e36], (n_exp, N))
    offs = torch.tensor([0] + torch.tensor(sizes).cumsum(0).tolist(), dtype=torch.int32)
    ldk, ldn = E.dlrm_ld(K, "e4m3"), E.dlrm_ld(N, y_dt)
    X8, W8 = torch.zeros((M, ldk), dtype=torch.uint8), torch.zeros((n_exp, N, ldk), dtype=torch.uint8)
    X8[:, :K], W8[..., :K] = X.to(torch.float8_e4m3fn).view(torch.uint8), W.to(torch.float8_e4m3fn).view(torch.uint8)
    Y = torch.full((M, ldn), -7.0, dtype=y_dt, device="cuda")[:, :N]
    ws = E.alloc_workspace(E.ERR_RECORD_BYTES)
    E.dlrm_experts_fwd(X8.cuda().view(torch.float8_e4m3fn)[:, :K], W8.cuda().view(torch.float8_e4m3fn)[..., :K], offs.cuda(), Y, ws,
                       x_scale=xs.cuda(), w_scale=wsc.cuda())
    want, mag, owned = R.experts(X, W, offs, None, False, xs, wsc)
    want, mag = want[owned], mag[owned]
    most = float(torch.finfo(y_dt).max)
    sure = (want.abs() / most - 1).abs() > 0.01          # next to the largest number either side of it may come out
    want = torch.where(want.abs() > most, want.sign() * float("inf"), want)
    bound = 1e-5 * mag + R.half_step(y_dt) * want.abs() + R.smallest(y_dt)
    R.within(Y.cpu()[owned][sure], want[sure], bound[sure], "Y")
    assert bool((Y.cpu()[~owned] == -7).all())


def test_scales_that_are_not_numbers():
    """Infinities and NaN among the scales spread as the definition's products do, and to no other row or column."""
    M, N, K = 40, 96, 64
    X, W = torch.ones((M, K)), torch.ones((1, N, K))
    X[3] = 0
    xs, wsc = torch.full((M,), 0.5), torch.full((1, N), 2.0)
    xs[3] = xs[5] = float("inf")
    xs[7] = float("nan")
    wsc[0, 11], wsc[0, 13] = float("inf"), 0.0
    Y = torch.empty((M, N), device="cuda")
    ws = E.alloc_workspace(E.ERR_RECORD_BYTES)
    E.dlrm_experts_fwd(X.cuda().to(torch.float8_e4m3fn), W.cuda().to(torch.float8_e4m3fn), torch.tensor([0, M], dtype=torch.int32).cuda(),
                       Y, ws, x_scale=xs.cuda(), w_scale=wsc.cuda())
    want = (X.double().sum(1) * xs.double())[:, None] * wsc.double()
    R.within(Y, want, 1e-6 * torch.nan_to_num(want, 0, 0, 0).abs(), "Y")
