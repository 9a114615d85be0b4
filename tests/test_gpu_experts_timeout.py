"""Products grouped by expert that give up, as in test_gpu_timeout.py: with
dlrm_set_wait_polls(0) every warp of the tile and of the pair kernel gives up
before its first tile, by the way that a wait which ran out takes. The call
returns, reports DLRM_ERR_TIMEOUT, has freed its tensor memory, and the same
call after the default is restored gives the bits of one that never timed out.
No wait is unbounded, so nothing here can hang or fault the GPU."""
import pytest
import torch

import embedding_bags_dot_b200 as E

pytestmark = pytest.mark.gpu

# tiles of 64 and of 128 columns on one SM, tiles of 256 x 256 on pairs
SIZES = [([5, 40, 0, 1], 70, 64), ([33, 128, 7] * 20, 1200, 479), ([4000, 257, 2500], 1024, 479)]


@pytest.fixture(autouse=True)
def _restore_polls():
    yield
    torch.cuda.synchronize()
    E.dlrm_set_wait_polls(-1)
    torch.cuda.synchronize()


def _protocol(run, ws, outs):
    run()
    assert E.dlrm_check_error(ws)[0] == E.OK
    want = [o.clone() for o in outs]
    E.dlrm_set_wait_polls(0)
    for o in outs:
        o.fill_(float("nan"))
    for _ in range(3):                       # tensor memory that a call kept would stop the next one
        run()
    st = E.dlrm_check_error(ws)              # synchronises: the kernels have finished
    assert st[0] == E.ERR_TIMEOUT and st[1] & 4, st
    E.dlrm_set_wait_polls(-1)
    for o in outs:
        o.fill_(float("nan"))
    run()
    assert E.dlrm_check_error(ws)[0] == E.OK
    assert all(torch.equal(o, w) for o, w in zip(outs, want))


def _case(sizes, N, K):
    g = torch.Generator().manual_seed(N)
    M, n_exp, ld = sum(sizes), len(sizes), E.dlrm_ld(K, "bf16")
    X = torch.randn((M, ld), generator=g).bfloat16().cuda()[:, :K]
    W = torch.randn((n_exp, N, ld), generator=g).bfloat16().cuda()[..., :K]
    offs = torch.tensor([0] + torch.tensor(sizes).cumsum(0).tolist(), dtype=torch.int32).cuda()
    return M, n_exp, X, W, offs


@pytest.mark.parametrize("sizes,N,K", SIZES)
def test_forward_waits_run_out(sizes, N, K):
    M, n_exp, X, W, offs = _case(sizes, N, K)
    Y = torch.empty((M, E.dlrm_ld(N, "bf16")), dtype=torch.bfloat16, device="cuda")[:, :N]
    ws = E.alloc_workspace(E.ERR_RECORD_BYTES)
    _protocol(lambda: E.dlrm_experts_fwd(X, W, offs, Y, ws, act=E.ACT_RELU), ws, [Y])


@pytest.mark.parametrize("sizes,N,K", SIZES[1:])
def test_gradient_waits_run_out(sizes, N, K):
    M, n_exp, X, W, offs = _case(sizes, N, K)
    dY = torch.randn((M, N), device="cuda").bfloat16()
    dX = torch.empty((M, E.dlrm_ld(K, "bf16")), dtype=torch.bfloat16, device="cuda")[:, :K]
    dW = torch.empty((n_exp, N, E.dlrm_ld(K, "f32")), device="cuda")[..., :K]
    ws = E.alloc_workspace(E.dlrm_experts_bwd_workspace_size(n_exp, M, N, K))
    _protocol(lambda: E.dlrm_experts_bwd(dY, X, W, offs, ws, dX=dX, dW=dW), ws, [dX, dW])
