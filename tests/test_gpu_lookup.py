"""dlrm_embed_fwd and dlrm_embed_bwd against plain references: types, widths
with and without whole 16-byte runs, strided and unaligned rows, lengths
from none to past the one-block sort, repeated and out-of-range ids."""
import pytest
import torch

import block_ref as R
import embedding_bags_dot_b200 as E

pytestmark = pytest.mark.gpu


def _table(rows, d, dt, seed=0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn((rows, d), generator=g).to(R.DT[dt])


def _ids(n, rows, seed=1, hot=0.0):
    g = torch.Generator().manual_seed(seed)
    idx = torch.randint(0, rows, (n,), generator=g)
    if hot:
        idx[torch.rand(n, generator=g) < hot] = rows // 3
    return idx.to(torch.int32)


@pytest.mark.parametrize("table,out", [("bf16", "bf16"), ("f16", "f32"), ("f32", "bf16"), ("f32", "f32"), ("f16", "bf16")])
@pytest.mark.parametrize("n,rows,d", [(1, 1, 1), (7, 100, 3), (48, 1000, 128), (3001, 500, 24), (5000, 64, 130),
                                      (9000, 300, 2048), (40_000, 77, 17)])
def test_lookup_rounds_the_scaled_row_once(table, out, n, rows, d):
    t, idx = _table(rows, d, table), _ids(n, rows)
    o = torch.full((n, d), float("nan"), dtype=R.DT[out], device="cuda")
    ws = E.alloc_workspace(E.ERR_RECORD_BYTES)
    E.dlrm_embed_fwd(E.Tables(t.cuda(), [rows], d), 0, idx.cuda(), o, ws, scale=1.7)
    want = (t[idx.long()].float() * torch.tensor(1.7)).to(R.DT[out])
    assert torch.equal(o.cpu(), want)
    assert E.dlrm_check_error(ws)[0] == E.OK


def test_lookup_of_a_later_table_and_strided_output():
    rows, d, n = [10, 33, 5], 20, 100
    t, idx = _table(sum(rows), d, "f32"), _ids(100, 33)
    buf = torch.full((n, 64), -5.0, device="cuda")
    ws = E.alloc_workspace(256)
    E.dlrm_embed_fwd(E.Tables(t.cuda(), rows, d), 1, idx.cuda(), buf[:, 3:3 + d], ws)
    want = torch.full((n, 64), -5.0)
    want[:, 3:3 + d] = t[10 + idx.long()]
    assert torch.equal(buf.cpu(), want)      # and nothing beside the rows is written


def test_lookup_counts_and_zeroes_ids_outside_the_table():
    rows, d = 50, 16
    t = _table(rows, d, "bf16")
    t[7, 3] = float("inf")
    idx = torch.tensor([0, -1, 49, 50, 2 ** 31 - 1, -2 ** 31, 7], dtype=torch.int32)
    o = torch.full((7, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    ws = E.alloc_workspace(256)
    E.dlrm_embed_fwd(E.Tables(t.cuda(), [rows], d), 0, idx.cuda(), o, ws, scale=float("inf"))
    assert E.dlrm_check_error(ws) == (E.ERR_INDEX_OOB, 1, 4, 0)
    assert torch.equal(o.cpu()[[1, 3, 4, 5]], torch.zeros((4, d), dtype=torch.bfloat16))
    assert torch.isinf(o.cpu()[6, 3])


GRADS = [(1, 1, 1), (5, 3, 2), (48, 1000, 128), (300, 7, 24), (4096, 50, 64), (4097, 200_000, 16), (20_000, 1023, 130),
         (30_000, 1024, 8), (9000, 300, 1048), (70_000, 2_000_000, 4)]


@pytest.mark.parametrize("grad,table", [("bf16", "f32"), ("f32", "f32"), ("f16", "f16"), ("f32", "bf16")])
@pytest.mark.parametrize("n,rows,d", GRADS)
def test_gradient_sums_every_occurrence(grad, table, n, rows, d):
    idx = _ids(n, rows, seed=n, hot=0.3)
    g = torch.Generator().manual_seed(d)
    dout = torch.randn((n, d), generator=g).to(R.DT[grad])
    dt = torch.full((rows, d), float("nan"), dtype=R.DT[table], device="cuda")
    ws = E.alloc_workspace(E.dlrm_embed_bwd_workspace_size(rows, d, n))
    E.dlrm_embed_bwd(idx.cuda(), dout.cuda(), dt, ws, scale=0.75)
    want, mag, count = R.embed_grad(rows, idx, dout, 0.75)
    # `count` additions and the scaling in fp32, one rounding of the result
    bound = R.U * (count + 1)[:, None] * mag + R.half_step(R.DT[table]) * want.abs() + R.smallest(R.DT[table])
    R.within(dt, want, bound * (1 + 1e-6), f"gradient {n}x{d} into {rows}")
    assert E.dlrm_check_error(ws)[0] == E.OK


@pytest.mark.parametrize("n", [0, 64, 6000, 100_000])
def test_gradient_of_one_row_and_of_none(n):
    """Every id the same: the run crosses all windows. No ids: all rows are zero."""
    rows, d = 300, 40
    idx = torch.full((n,), 299, dtype=torch.int32)
    dout = torch.ones((n, d))
    dt = torch.full((rows, d), float("nan"), device="cuda")
    ws = E.alloc_workspace(E.dlrm_embed_bwd_workspace_size(rows, d, n))
    E.dlrm_embed_bwd(idx.cuda(), dout.cuda(), dt, ws)
    want = torch.zeros((rows, d))
    want[299] = n        # ones add exactly
    assert torch.equal(dt.cpu(), want)


@pytest.mark.parametrize("n", [50, 5000, 200_000])
def test_gradient_skips_and_counts_ids_outside_the_table(n):
    rows, d = 1000, 8
    idx = _ids(n, rows)
    idx[::5] = torch.tensor([-1, rows, 2 ** 31 - 1], dtype=torch.int32).repeat(n)[: len(idx[::5])]
    dout = torch.randint(-4, 5, (n, d)).float()
    dout[::5] = float("nan")                    # what a skipped id brings must not be read into any sum
    dt = torch.full((rows, d), float("nan"), device="cuda")
    ws = E.alloc_workspace(E.dlrm_embed_bwd_workspace_size(rows, d, n))
    E.dlrm_embed_bwd(idx.cuda(), dout.cuda(), dt, ws)
    want, _, _ = R.embed_grad(rows, idx, torch.nan_to_num(dout), 1.0)
    assert torch.equal(dt.cpu().double(), want)   # small integers add exactly
    assert E.dlrm_check_error(ws) == (E.ERR_INDEX_OOB, 1, len(idx[::5]), 0)


def test_gradient_of_many_blocks_is_exact_and_repeats():
    """Enough ids that each sorting block takes several tiles (more than 296 tiles of 2,048)."""
    n, rows, d = 1_300_000, 30_000, 4
    idx = _ids(n, rows, hot=0.1)
    dout = torch.randint(-8, 9, (n, d)).float()
    ws = E.alloc_workspace(E.dlrm_embed_bwd_workspace_size(rows, d, n))
    outs = []
    for _ in range(2):
        dt = torch.empty((rows, d), device="cuda")
        E.dlrm_embed_bwd(idx.cuda(), dout.cuda(), dt, ws)
        outs.append(dt.cpu())
    assert torch.equal(outs[0].double(), R.embed_grad(rows, idx, dout, 1.0)[0])
    assert torch.equal(outs[0], outs[1])


def test_gradient_of_strided_unaligned_rows():
    n, rows, d = 2000, 90, 33
    buf = torch.randn((n, 50)).to(torch.bfloat16)
    idx = _ids(n, rows)
    dt = torch.empty((rows, d), dtype=torch.float32, device="cuda")
    ws = E.alloc_workspace(E.dlrm_embed_bwd_workspace_size(rows, d, n))
    E.dlrm_embed_bwd(idx.cuda(), buf.cuda()[:, 5:5 + d], dt, ws)
    want, mag, count = R.embed_grad(rows, idx, buf[:, 5:5 + d], 1.0)
    R.within(dt, want, R.U * (count + 1)[:, None] * mag * (1 + 1e-6), "strided gradient")


def test_gradient_is_the_adjoint_of_the_lookup():
    """<lookup(T), G> = <T, gradient(G)> in integers, where both sides are exact."""
    n, rows, d = 3000, 400, 32
    t = torch.randint(-4, 5, (rows, d)).float()
    g = torch.randint(-4, 5, (n, d)).float()
    idx = _ids(n, rows, hot=0.2).cuda()
    out, dt = torch.empty((n, d), device="cuda"), torch.empty((rows, d), device="cuda")
    ws = E.alloc_workspace(E.dlrm_embed_bwd_workspace_size(rows, d, n))
    E.dlrm_embed_fwd(E.Tables(t.cuda(), [rows], d), 0, idx, out, ws, scale=2.0)
    E.dlrm_embed_bwd(idx, g.cuda(), dt, ws, scale=2.0)
    assert float((out.cpu().double() * g).sum()) == float((t.double() * dt.cpu()).sum())


@pytest.mark.parametrize("rows", [40, 5000, 1_500_000])
@pytest.mark.parametrize("n", [2048, 2049, 8192, 8193, 16_384, 16_385, 32_768, 32_769, 65_535, 65_536, 65_537])
def test_gradient_at_the_ends_of_each_sort(n, rows):
    """The one-block, the cluster's and the many-block sort, each of their sizes' ends, one to three digits."""
    d = 3
    idx = _ids(n, rows, seed=n + rows, hot=0.2)
    idx[n // 2] = -1
    g = torch.Generator().manual_seed(n)
    dout = torch.randint(-8, 9, (n, d), generator=g).float()
    ws = E.alloc_workspace(E.dlrm_embed_bwd_workspace_size(rows, d, n))
    dt = torch.full((rows, d), float("nan"), device="cuda")
    E.dlrm_embed_bwd(idx.cuda(), dout.cuda(), dt, ws)
    want = torch.zeros((rows, d), dtype=torch.float64)
    ok = idx >= 0
    want.index_add_(0, idx[ok].long(), dout[ok].double())
    assert torch.equal(dt.cpu().double(), want)             # small integers add exactly
    assert E.dlrm_check_error(ws) == (E.ERR_INDEX_OOB, 1, 1, 0)


@pytest.mark.parametrize("first", [0, 1, 15, 16])
def test_gradient_of_runs_of_every_number_of_windows(first):
    """Ids whose runs cover 1 to 3, 31 to 35 and hundreds of windows of 16, begun at every kind of place."""
    lens = [first] + [1, 15, 16, 17, 33, 31 * 16, 32 * 16 - 1, 32 * 16 + 1, 33 * 16, 33 * 16 + 15, 34 * 16, 35 * 16 + 1, 300 * 16 + 7, 2]
    idx = torch.repeat_interleave(torch.arange(len(lens)), torch.tensor(lens)).to(torch.int32)
    g = torch.Generator().manual_seed(first)
    dout = torch.randint(-8, 9, (len(idx), 8), generator=g).float()
    perm = torch.randperm(len(idx), generator=g)
    ws = E.alloc_workspace(E.dlrm_embed_bwd_workspace_size(len(lens), 8, len(idx)))
    dt = torch.full((len(lens), 8), float("nan"), device="cuda")
    E.dlrm_embed_bwd(idx[perm].cuda(), dout[perm].cuda(), dt, ws)
    assert torch.equal(dt.cpu().double(), torch.zeros((len(lens), 8), dtype=torch.float64).index_add_(0, idx.long(), dout.double()))


@pytest.mark.parametrize("n", [1000, 5000, 40_000, 80_000])
def test_captured_gradient_replays_on_new_ids_beside_another_stream(n):
    rows, d = 3000, 16
    idx = _ids(n, rows, seed=1).cuda()
    dout = torch.randint(-8, 9, (n, d)).float().cuda()
    dt = torch.full((rows, d), float("nan"), device="cuda")
    ws = E.alloc_workspace(E.dlrm_embed_bwd_workspace_size(rows, d, n))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        E.dlrm_embed_bwd(idx, dout, dt, ws)
    idx2, other = _ids(n, rows, seed=2).cuda(), torch.cuda.Stream()
    dt2, ws2 = torch.empty_like(dt), E.alloc_workspace(len(ws))
    want2 = torch.zeros((rows, d), dtype=torch.float64, device="cuda").index_add_(0, idx2.long(), dout.double())
    other.wait_stream(torch.cuda.current_stream())
    for seed in (3, 4):
        idx.copy_(_ids(n, rows, seed=seed, hot=0.4))
        graph.replay()
        E.dlrm_embed_bwd(idx2, dout, dt2, ws2, stream=other)
        want = torch.zeros((rows, d), dtype=torch.float64, device="cuda").index_add_(0, idx.long(), dout.double())
        torch.cuda.synchronize()
        assert torch.equal(dt.double(), want) and torch.equal(dt2.double(), want2)
        dt.fill_(float("nan"))
