"""Outputs of the products grouped by expert that are columns of a wider buffer:
what stands between their width and the row pitch stays as it was, whatever
the width (a bulk store clips a tile at 16 bytes, not at an element)."""
import pytest
import torch

import block_ref as R
import embedding_bags_dot_b200 as E

pytestmark = pytest.mark.gpu

BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def _wide(lead, width, dt, extra=16):
    """A view [*lead][width] of a buffer whose other columns hold 5, and that buffer."""
    buf = torch.full((*lead, (width + 15) // 16 * 16 + extra), 5.0, dtype=dt, device="cuda")
    buf[..., :width] = -7
    return buf[..., :width], buf


def _ints(shape, g, dt):
    return torch.randint(-3, 4, shape, generator=g).float().to(dt)


def _rows(t, dt):
    v, _ = _wide(t.shape[:-1], t.shape[-1], torch.uint8 if dt == torch.float8_e4m3fn else dt)
    v.copy_(t.to(dt).view(torch.uint8) if dt == torch.float8_e4m3fn else t)
    return v.view(dt) if dt == torch.float8_e4m3fn else v


# single-SM tiles and pairs; whole groups of 32 rows, and an expert's last ones
SIZES = [[64], [5, 40, 0, 32], [33, 128, 7] * 5, [4000, 257, 2500]]
WIDTHS = [1, 3, 63, 65, 70, 127, 200, 257]


@pytest.mark.parametrize("dt,y_dt", [(BF, BF), (F16, F16), (BF, F32), (torch.float8_e4m3fn, BF), (torch.float8_e4m3fn, F32)])
@pytest.mark.parametrize("sizes", SIZES)
def test_forward_leaves_the_columns_beside_its_own(sizes, dt, y_dt):
    for N in WIDTHS:
        g = torch.Generator().manual_seed(N)
        M, n_exp, K = sum(sizes), len(sizes), 96
        X, W, bias = _ints((M, K), g, F32), _ints((n_exp, N, K), g, F32), _ints((n_exp, N), g, F32)
        offs = torch.tensor([0] + torch.tensor(sizes).cumsum(0).tolist(), dtype=torch.int32)
        Y, buf = _wide((M,), N, y_dt)
        ws, one = E.alloc_workspace(E.ERR_RECORD_BYTES), dt == torch.float8_e4m3fn
        E.dlrm_experts_fwd(_rows(X, dt), _rows(W, dt), offs.cuda(), Y, ws, bias=bias.cuda(),
                           x_scale=torch.ones(M, device="cuda") if one else None,
                           w_scale=torch.ones((n_exp, N), device="cuda") if one else None)
        want = R.experts(X, W, offs, bias, False)[0].to(y_dt)       # small integers: sums are exact
        assert torch.equal(Y.cpu(), want), N
        assert bool((buf[:, N:] == 5).all()), N


@pytest.mark.parametrize("dt,o_dt", [(BF, BF), (F16, F32)])
@pytest.mark.parametrize("relu", [False, True])
@pytest.mark.parametrize("sizes", SIZES)
def test_gradients_leave_the_columns_beside_their_own(sizes, relu, dt, o_dt):
    for N, K in ((40, 1), (33, 65), (300, 70), (7, 127), (130, 257)):
        g = torch.Generator().manual_seed(N)
        M, n_exp = sum(sizes), len(sizes)
        X, W, dY = _ints((M, K), g, F32), _ints((n_exp, N, K), g, F32), _ints((M, N), g, F32)
        Yf = _ints((M, N), g, F32) if relu else None
        offs = torch.tensor([0] + torch.tensor(sizes).cumsum(0).tolist(), dtype=torch.int32)
        (dX, bx), (dW, bw) = _wide((M,), K, o_dt), _wide((n_exp, N), K, o_dt)
        act = E.ACT_RELU if relu else E.ACT_NONE
        ws = E.alloc_workspace(E.dlrm_experts_bwd_workspace_size(n_exp, M, N, K, act))
        E.dlrm_experts_bwd(_rows(dY, dt), _rows(X, dt), _rows(W, dt), offs.cuda(), ws, Y=_rows(Yf, dt) if relu else None, act=act,
                           dX=dX, dW=dW)
        (wX, wW, _), _ = R.experts_grad(dY, X, W, offs, Yf)
        assert torch.equal(dX.cpu(), wX.to(o_dt)) and torch.equal(dW.cpu(), wW.to(o_dt)), (N, K)
        assert bool((bx[:, K:] == 5).all()) and bool((bw[..., K:] == 5).all()), (N, K)
