"""The lookup gradient where a device cannot place a cluster of sixteen blocks:
the many-block sort takes the sizes the cluster's would have had, with the
same bits and in the same workspace, eagerly and captured."""
import pytest
import torch

import block_ref as R
import embedding_bags_dot_b200 as E

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _restore():
    yield
    E.dlrm_set_sort_clusters(True)


def _grad(idx, dout, rows, d, ws):
    dt = torch.full((rows, d), float("nan"), device="cuda")
    before = E.dlrm_launch_count()
    E.dlrm_embed_bwd(idx, dout, dt, ws, scale=0.5)
    return dt, E.dlrm_launch_count() - before


@pytest.mark.parametrize("rows", [40, 5000, 1_500_000])
@pytest.mark.parametrize("n", [2049, 8192, 8193, 16_385, 32_769, 65_536])
def test_the_other_sort_gives_the_same_bits(n, rows):
    d = 4
    g = torch.Generator().manual_seed(n)
    idx = torch.randint(0, rows, (n,), generator=g).to(torch.int32)
    idx[:: 3] = rows // 3
    idx[n // 2] = -1
    dout = torch.randn((n, d), generator=g)
    # as small as the query says, in a longer buffer whose rest has to stay
    need = E.dlrm_embed_bwd_workspace_size(rows, d, n)
    buf = torch.full((need + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
    ws = buf[:need]
    ws[:E.ERR_RECORD_BYTES] = 0
    want, launches = _grad(idx.cuda(), dout.cuda(), rows, d, ws)
    assert E.dlrm_check_error(ws) == (E.ERR_INDEX_OOB, 1, 1, 0)
    E.dlrm_set_sort_clusters(False)
    got, others = _grad(idx.cuda(), dout.cuda(), rows, d, ws)
    assert E.dlrm_check_error(ws) == (E.ERR_INDEX_OOB, 1, 1, 0)
    assert others > launches and torch.equal(got, want) and bool((buf[need:] == 0x5A).all())
    ref, mag, count = R.embed_grad(rows, idx, dout, 0.5)
    R.within(got, ref, (R.U * (count + 1)[:, None] * mag + R.smallest(torch.float32)) * (1 + 1e-6), "gradient")


@pytest.mark.parametrize("n", [3000, 50_000])
def test_captured_without_clusters(n):
    rows, d = 700, 8
    g = torch.Generator().manual_seed(n)
    idx = torch.randint(0, rows, (n,), generator=g).to(torch.int32).cuda()
    dout = torch.randint(-8, 9, (n, d), generator=g).float().cuda()
    ws = E.alloc_workspace(E.dlrm_embed_bwd_workspace_size(rows, d, n))
    dt = torch.full((rows, d), float("nan"), device="cuda")
    E.dlrm_set_sort_clusters(False)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        E.dlrm_embed_bwd(idx, dout, dt, ws)
    E.dlrm_set_sort_clusters(True)
    idx.copy_(torch.randint(0, rows, (n,), generator=g))
    graph.replay()
    want = torch.zeros((rows, d), dtype=torch.float64, device="cuda").index_add_(0, idx.long(), dout.double())
    assert torch.equal(dt.double(), want)
