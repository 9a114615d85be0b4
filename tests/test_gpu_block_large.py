"""The token-block operators where element numbers pass 31 and 32 bits: far
rows of large tables, activations and outputs, checked at places drawn over the
whole range and at the far end."""
import pytest
import torch

import block_ref as R
import embedding_bags_dot_b200 as E

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _free_memory():
    yield
    torch.cuda.empty_cache()


def test_lookup_and_gradient_of_a_table_past_32_bits():
    rows, d, n = 1_100_000, 4096, 3000                     # 4.5e9 elements, 9 GB in bf16
    table = torch.empty((rows, d), dtype=torch.bfloat16, device="cuda")
    g = torch.Generator().manual_seed(0)
    idx = torch.randint(0, rows, (n,), generator=g)
    idx[0], idx[1], idx[2] = rows - 1, 0, 2 ** 31 // d
    idx = idx.to(torch.int32).cuda()
    want = torch.randn((n, d), generator=g).to(torch.bfloat16).cuda()
    first = {}
    for i, r in enumerate(idx.tolist()):
        first.setdefault(r, i)
    table[torch.tensor(list(first), device="cuda")] = want[torch.tensor(list(first.values()), device="cuda")]
    out = torch.empty((n, d), dtype=torch.bfloat16, device="cuda")
    ws = E.alloc_workspace(E.dlrm_embed_bwd_workspace_size(rows, d, n))
    E.dlrm_embed_fwd(E.Tables(table, [rows], d), 0, idx, out, ws)
    assert torch.equal(out, table[idx.long()])
    table.fill_(float("nan"))
    E.dlrm_embed_bwd(idx, want, table, ws)                 # every row written, none but these with values
    for r in (0, 1, 2 ** 31 // d, 2 ** 32 // d, rows - 2, rows - 1) + tuple(idx[:50].tolist()):
        hit = (idx == r).nonzero().flatten()
        ref = want[hit].double().sum(0) if len(hit) else torch.zeros(d, dtype=torch.float64, device="cuda")
        R.within(table[r], ref, R.half_step(torch.bfloat16) * ref.abs() + 1e-6, f"row {r}")
    assert not bool(torch.isnan(table.view(-1)[:: 4097]).any()) and not bool(torch.isnan(table[-20000:]).any())


def test_norm_of_rows_past_32_bits():
    rows, d = 1_100_000, 4096
    x = torch.zeros((rows, d), dtype=torch.bfloat16, device="cuda")
    at = torch.tensor([0, 1, 2 ** 31 // d, 2 ** 32 // d, rows - 1], device="cuda")
    x[at] = torch.randn((len(at), d), device="cuda").to(torch.bfloat16)
    y, rstd = torch.empty_like(x), torch.empty(rows, device="cuda")
    E.dlrm_rmsnorm_fwd(x, None, y, rstd=rstd, eps=1e-4)
    _, wr, wy = R.rmsnorm(x[at].cpu(), None, None, 1e-4)
    R.within(y[at], wy, (R.half_step(torch.bfloat16) + 44 * R.U) * wy.abs() + 1e-9, "y")
    R.within(rstd[at], wr, 40 * R.U * wr, "rstd")
    assert abs(float(rstd[5]) - 100.0) < 1e-4 and float(y[-2].float().abs().max()) == 0
    ws = E.alloc_workspace(E.dlrm_rmsnorm_bwd_workspace_size(rows, d))
    dw = torch.empty(d, device="cuda")
    y.fill_(1.0)
    want = (x[at].double() * rstd[at].double()[:, None]).sum(0)
    mag = (x[at].double() * rstd[at].double()[:, None]).abs().sum(0)
    E.dlrm_rmsnorm_bwd(y, x, rstd, None, y, ws, dw=dw)     # dx in dy's own buffer
    R.within(dw, want, 1e-5 * mag + 1e-12, "dw")           # rows of zeros add exact zeros
    assert float(y[-2].float().min()) == float(torch.tensor(100.0).bfloat16()) == float(y[5].float().max())


def test_norm_of_the_most_rows():
    rows = 2 ** 31 - 1
    x = torch.full((rows, 1), 3.0, dtype=torch.bfloat16, device="cuda")
    x[-1], x[2 ** 30] = -3.0, -3.0
    rstd = torch.zeros(rows, device="cuda")
    y = torch.zeros_like(x)
    E.dlrm_rmsnorm_fwd(x, None, y, rstd=rstd, eps=0.0)
    assert float(y[-1]) == -1.0 == float(y[2 ** 30]) and float(y[-2]) == 1.0
    assert int((y == 1.0).sum()) == rows - 2
    third = float(torch.tensor(1.0) / 3.0)
    assert abs(float(rstd.min()) - third) < 1e-7 > abs(float(rstd.max()) - third)
    rstd.fill_(2.0)
    h, dx = torch.zeros_like(x), torch.zeros_like(x)
    ws = E.alloc_workspace(E.dlrm_rmsnorm_bwd_workspace_size(rows, 1))
    E.dlrm_rmsnorm_bwd(y, h, rstd, None, dx, ws)           # h = 0: dx = rstd dy
    assert float(dx[-1]) == -2.0 == float(dx[2 ** 30]) and int((dx == 2.0).sum()) == rows - 2


def test_dropout_past_34_bits():
    n = 2 ** 34 + 4 * 1000 + 3                             # the counter's low half passes 32 bits
    x = torch.ones(n, dtype=torch.bfloat16, device="cuda")  # 34 GB, in place
    rng = torch.tensor([5, 6], dtype=torch.int64, device="cuda")
    E.dlrm_dropout(x, x, 0.5, rng)
    for first in (0, 2 ** 31, 2 ** 32, 2 ** 34 - 2000, n - 4003):
        first -= first % 4
        m = min(4000, n - first)
        kept = torch.from_numpy(R.philox(m, 5, 6, first) >= 2 ** 31)
        assert torch.equal((x[first:first + m] != 0).cpu(), kept), first


def test_experts_of_rows_past_32_bits():
    M, N, K = 2_200_000, 64, 2048                          # 4.5e9 elements of X, 9 GB
    X = torch.zeros((M, K), dtype=torch.bfloat16, device="cuda")
    at = torch.tensor([0, 2 ** 31 // K, 2 ** 32 // K, M - 1], device="cuda")
    g = torch.Generator().manual_seed(3)
    X[at] = torch.randint(-3, 4, (len(at), K), generator=g).to(torch.bfloat16).cuda()
    W = torch.randint(-3, 4, (2, N, K), generator=g).to(torch.bfloat16).cuda()
    offs = torch.tensor([0, 1000, M], dtype=torch.int32, device="cuda")
    Y = torch.full((M, N), float("nan"), device="cuda")
    ws = E.alloc_workspace(E.dlrm_experts_bwd_workspace_size(2, M, N, K))
    E.dlrm_experts_fwd(X, W, offs, Y, ws)
    for i, r in enumerate(at.tolist()):
        assert torch.equal(Y[r].double(), W[0 if r < 1000 else 1].double() @ X[r].double()), r
    assert float(Y.abs().sum(1).count_nonzero()) == len(at)
    dY = torch.zeros((M, N), dtype=torch.bfloat16, device="cuda")
    dY[at] = torch.randint(-3, 4, (len(at), N), generator=g).to(torch.bfloat16).cuda()
    dX = torch.full((M, K), float("nan"), dtype=torch.bfloat16, device="cuda")
    dW, db = torch.empty((2, N, K), device="cuda"), torch.empty((2, N), device="cuda")
    E.dlrm_experts_bwd(dY, X, W, offs, ws, dX=dX, dW=dW, db=db)
    for r in at.tolist():
        e = 0 if r < 1000 else 1
        want = (dY[r].double() @ W[e].double()).to(torch.bfloat16)
        assert torch.equal(dX[r], want), r
    late = at[at >= 1000]
    assert torch.equal(dW[1].double(), dY[late].double().T @ X[late].double())
    assert torch.equal(db[1].double(), dY[late].double().sum(0)) and not bool(torch.isnan(dX[-1000:]).any())
    assert E.dlrm_check_error(ws)[0] == E.OK
