"""The token-block operators run together, as a model over sequences of ids
uses them: lookup, dropout, residual norm (bf16 and 8-bit rows), rows gathered
by expert, the experts' layer, their sum back into token order; then the
backward pass down to the table's gradient. Each step is held to the 64-bit
reference on the inputs it was given, by the bounds of its own tests. Also: the
whole run captured into one graph and replayed on new inputs, on a stream of
its own, and next to another run on another stream."""
import pytest
import torch

import block_ref as R
import embedding_bags_dot_b200 as E

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
HALF = R.half_step(BF)
TINY = R.smallest(BF)


class Block:
    """Buffers, workspaces and weights of one run: n tokens of width d, E experts of N outputs."""

    def __init__(self, n=600, rows=5000, d=256, n_exp=6, N=320, p=0.2, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.n, self.rows, self.d, self.n_exp, self.N, self.p = n, rows, d, n_exp, N, p
        self.table = (torch.randn((rows, d), generator=g) * d ** -0.5).to(BF).cuda()
        self.T = E.Tables(self.table, [rows], d)
        self.w = (1 + 0.1 * torch.randn(d, generator=g)).cuda()
        self.W = (torch.randn((n_exp, N, d), generator=g) * d ** -0.5).to(BF).cuda()
        ws = self.W.float().abs().amax(-1) / 448
        self.W8, self.W8s = (self.W.float() / ws[..., None]).to(torch.float8_e4m3fn), ws
        self.bias = (0.1 * torch.randn((n_exp, N), generator=g)).cuda()
        z = lambda *s, dt=BF: torch.zeros(s, dtype=dt, device="cuda")  # noqa: E731
        self.ids, self.perm = z(n, dt=torch.int32), z(n, dt=torch.int32)
        self.offs, self.rng = z(n_exp + 1, dt=torch.int32), z(2, dt=torch.int64)
        self.residual, self.x, self.xd, self.h, self.y = z(n, d), z(n, d), z(n, d), z(n, d), z(n, d)
        self.rstd, self.y8, self.y8s = z(n, dt=torch.float32), z(n, d, dt=torch.float8_e4m3fn), z(n, dt=torch.float32)
        self.Xr, self.out, self.out8, self.dOut = z(n, d), z(n, N), z(n, N), z(n, N)
        self.dXr, self.dW, self.db = z(n, d), z(n_exp, N, d, dt=torch.float32), z(n_exp, N, dt=torch.float32)
        self.dy, self.dh, self.dx, self.dw, self.dxd = z(n, d), z(n, d), z(n, d), z(d, dt=torch.float32), z(n, d)
        self.dtable = z(rows, d, dt=torch.float32)
        self.ws = E.alloc_workspace(max(E.dlrm_embed_bwd_workspace_size(rows, d, n), E.dlrm_embed_bwd_workspace_size(n, d, n),
                                        E.dlrm_rmsnorm_bwd_workspace_size(n, d),
                                        E.dlrm_experts_bwd_workspace_size(n_exp, n, N, d, E.ACT_RELU)))

    def feed(self, seed):
        g = torch.Generator().manual_seed(seed)
        self.ids.copy_(torch.randint(0, self.rows, (self.n,), generator=g))
        self.ids[: self.n // 8] = 3                                  # one frequent id
        expert = torch.randint(0, self.n_exp, (self.n,), generator=g)
        expert[expert == 1] = 0                                      # an expert without rows
        self.perm.copy_(torch.argsort(expert, stable=True))
        self.offs[1:].copy_(torch.bincount(expert, minlength=self.n_exp).cumsum(0))
        self.rng.copy_(torch.tensor([99, seed]))
        self.residual.copy_(torch.randn((self.n, self.d), generator=g))
        self.dOut.copy_(torch.randn((self.n, self.N), generator=g))
        self.dh.copy_(torch.randn((self.n, self.d), generator=g))

    def forward(self):
        E.dlrm_embed_fwd(self.T, 0, self.ids, self.x, self.ws, scale=self.d ** 0.5)
        E.dlrm_dropout(self.x, self.xd, self.p, self.rng)
        E.dlrm_rmsnorm_fwd(self.xd, self.w, self.y, residual=self.residual, h=self.h, rstd=self.rstd)
        E.dlrm_rmsnorm_fwd(self.xd, self.w, self.y8, residual=self.residual, y_scale=self.y8s)
        # rows in expert order: a lookup into the activations
        E.dlrm_embed_fwd(E.Tables(self.y, [self.n], self.d), 0, self.perm, self.Xr, self.ws)
        E.dlrm_experts_fwd(self.Xr, self.W, self.offs, self.out, self.ws, bias=self.bias, act=E.ACT_RELU)

    def forward_8bit(self):
        """The serving form: the norm's 8-bit rows, put in expert order, straight into the 8-bit product."""
        order = self.perm.long()
        E.dlrm_experts_fwd(self.y8.view(torch.uint8)[order].view(torch.float8_e4m3fn), self.W8, self.offs, self.out8, self.ws,
                           bias=self.bias, act=E.ACT_RELU, x_scale=self.y8s[order], w_scale=self.W8s)

    def backward(self):
        E.dlrm_experts_bwd(self.dOut, self.Xr, self.W, self.offs, self.ws, Y=self.out, act=E.ACT_RELU, dX=self.dXr,
                           dW=self.dW, db=self.db)
        # back in token order: the gradient of that lookup
        E.dlrm_embed_bwd(self.perm, self.dXr, self.dy, self.ws)
        E.dlrm_rmsnorm_bwd(self.dy, self.h, self.rstd, self.w, self.dx, self.ws, dw=self.dw, dh=self.dh)
        E.dlrm_dropout(self.dx, self.dxd, self.p, self.rng)
        E.dlrm_embed_bwd(self.ids, self.dxd, self.dtable, self.ws, scale=self.d ** 0.5)

    RESULTS = ("x", "xd", "h", "y", "rstd", "y8s", "Xr", "out", "dXr", "dW", "db", "dy", "dx", "dw", "dxd", "dtable")

    def results(self):
        torch.cuda.synchronize()
        return {k: getattr(self, k).clone() for k in self.RESULTS}


def test_every_step_of_a_run():
    b = Block()
    b.feed(1)
    b.forward()
    b.forward_8bit()
    b.backward()
    assert E.dlrm_check_error(b.ws)[0] == E.OK
    c = {k: getattr(b, k).cpu() for k in b.RESULTS + ("ids", "perm", "offs", "residual", "dOut", "dh", "w", "bias", "W", "table", "out8")}
    scale = b.d ** 0.5
    assert torch.equal(c["x"], (c["table"][c["ids"].long()].float() * scale).to(BF))
    xd, _ = R.dropout(c["x"], None, b.p, 99, 1)
    R.within(c["xd"], xd, (HALF + 4 * R.U) * xd.abs() + TINY, "dropout")
    h, rstd, y = R.rmsnorm(c["xd"], c["residual"], c["w"], 1e-6)
    R.within(c["h"], h, (HALF + 2 * R.U) * h.abs() + TINY, "h")
    R.within(c["rstd"], rstd, 40 * R.U * rstd, "rstd")
    R.within(c["y"], y, (HALF + 44 * R.U) * y.abs() + TINY, "y")
    assert torch.equal(c["Xr"], c["y"][c["perm"].long()])
    out, mag, owned = R.experts(c["Xr"], c["W"], c["offs"], c["bias"], True)
    assert bool(owned.all())
    R.within(c["out"], out, 1e-5 * mag + HALF * out.abs() + TINY, "experts")
    order = c["perm"].long()
    out8, mag8, _ = R.experts(b.y8.cpu().float()[order], b.W8.cpu().float(), c["offs"], c["bias"], True, c["y8s"][order], b.W8s.cpu())
    R.within(c["out8"], out8, 1e-5 * mag8 + HALF * out8.abs() + TINY, "8-bit experts")
    (dX, dW, db), (mX, mW, mb) = R.experts_grad(c["dOut"], c["Xr"], c["W"], c["offs"], c["out"])
    R.within(c["dXr"], dX, 1e-5 * mX + HALF * dX.abs() + TINY, "dXr")
    R.within(c["dW"], dW, 1e-5 * mW, "dW")
    R.within(c["db"], db, 1e-5 * mb, "db")
    assert torch.equal(c["dy"][order], c["dXr"])       # a permutation: each row has one gradient
    dx, dw, mx, mw = R.rmsnorm_grad(c["dy"], c["h"], c["rstd"], c["w"], c["dh"])
    R.within(c["dx"], dx, HALF * dx.abs() + 60 * R.U * mx + TINY, "dx")
    R.within(c["dw"], dw, (b.n + 70) * R.U * mw, "dw")
    dxd, _ = R.dropout(c["dx"], None, b.p, 99, 1)
    R.within(c["dxd"], dxd, (HALF + 4 * R.U) * dxd.abs() + TINY, "dropout's gradient")
    dt, mt, cnt = R.embed_grad(b.rows, c["ids"], c["dxd"], scale)
    R.within(c["dtable"], dt, R.U * (cnt + 2)[:, None] * mt * (1 + 1e-6), "the table's gradient")


def _eager(inputs, **kw):
    b = Block(**kw)
    b.feed(inputs)
    b.forward()
    b.backward()
    return b.results()


def test_a_captured_run_replays_on_new_inputs():
    want = [_eager(s) for s in (1, 2, 3)]
    b = Block()
    b.feed(1)
    b.forward()
    b.backward()           # every kernel has run once before the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.forward()
        b.backward()
    for s in (1, 2, 3):
        b.feed(s)
        graph.replay()
        got = b.results()
        for k, v in want[s - 1].items():
            assert torch.equal(got[k], v), (s, k)
    assert E.dlrm_check_error(b.ws)[0] == E.OK


def test_two_runs_on_two_streams_and_by_the_stream_argument():
    want = _eager(4), _eager(5, n=900, d=192, N=264, seed=1)
    a, b = Block(), Block(n=900, d=192, N=264, seed=1)
    a.feed(4)
    b.feed(5)
    torch.cuda.synchronize()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        with torch.cuda.stream(sa):
            a.forward()
        with torch.cuda.stream(sb):
            b.forward()
        with torch.cuda.stream(sa):
            a.backward()
        with torch.cuda.stream(sb):
            b.backward()
    for blk, w in ((a, want[0]), (b, want[1])):
        got = blk.results()
        for k, v in w.items():
            assert torch.equal(got[k], v), k
    y = torch.empty_like(a.xd)
    with torch.cuda.stream(sa):
        torch.cuda._sleep(20_000_000)                    # the call below has to stay behind this
        a.x.fill_(2.0)
    E.dlrm_dropout(a.x, y, 0.0, a.rng, stream=sa)
    sa.synchronize()
    assert bool((y == 2).all())


def test_single_tokens_match_their_rows_of_a_batch():
    """Row by row through the norm and the experts: a row's result does not depend on the rows around it (the
    norm: bit for bit within its launch shape; the experts: to the sums' bound, since tile widths differ)."""
    b = Block()
    b.feed(6)
    b.forward()
    rows = torch.tensor([0, 7, 300, 599])
    out = torch.empty((1, b.N), dtype=BF, device="cuda")
    offs_all = b.offs.cpu()
    for r in rows.tolist():
        e = int(torch.searchsorted(offs_all[1:].contiguous(), torch.tensor(r, dtype=torch.int32), right=True))
        offs = torch.zeros(b.n_exp + 1, dtype=torch.int32)
        offs[e + 1:] = 1
        E.dlrm_experts_fwd(b.Xr[r:r + 1], b.W, offs.cuda(), out, b.ws, bias=b.bias, act=E.ACT_RELU)
        want, mag, _ = R.experts(b.Xr[r:r + 1].cpu(), b.W.cpu(), offs, b.bias.cpu(), True)
        R.within(out, want, 1e-5 * mag + HALF * want.abs() + TINY, f"row {r}")
        y = torch.empty((1, b.d), dtype=BF, device="cuda")
        E.dlrm_rmsnorm_fwd(b.xd[r:r + 1], b.w, y, residual=b.residual[r:r + 1])
        wy = R.rmsnorm(b.xd[r:r + 1].cpu(), b.residual[r:r + 1].cpu(), b.w.cpu(), 1e-6)[2]
        R.within(y, wy, (HALF + 44 * R.U) * wy.abs() + TINY, f"norm of row {r}")


def test_work_after_the_call_sees_its_outputs():
    """Programmatic dependents keep stream order: torch kernels right behind a call read finished outputs."""
    b = Block()
    b.feed(7)
    want = _eager(7)
    for _ in range(10):
        b.feed(7)
        b.forward()
        copy = b.out.clone()
        b.out.zero_()
        assert torch.equal(copy, want["out"])
