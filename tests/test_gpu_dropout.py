"""dlrm_dropout against Philox4x32-10 on the host: which elements are kept is
held exactly, values to their rounding."""
import pytest
import torch

import block_ref as R
import embedding_bags_dot_b200 as E

pytestmark = pytest.mark.gpu


def _run(x, p, seed, offset, residual=None, y=None):
    y = torch.full_like(x, float("nan")) if y is None else y
    rng = torch.tensor([seed, offset], dtype=torch.int64, device="cuda")
    E.dlrm_dropout(x, y, p, rng, residual=residual)
    return y


def _bound(want, x, p, residual, dtype):
    # x * scale (scale itself rounded), the residual's addition, one rounding to the type
    terms = x.double().abs() / (1 - p) + (0 if residual is None else residual.double().abs())
    return R.half_step(dtype) * want.abs() + 4 * R.U * terms + R.smallest(dtype)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n", [1, 3, 4, 5, 8, 31, 4099, 300_001])
@pytest.mark.parametrize("with_residual", [False, True])
def test_dropout_keeps_what_the_generator_says(dt, n, with_residual):
    g = torch.Generator().manual_seed(n)
    x = torch.randn(n, generator=g).to(R.DT[dt])
    r = torch.randn(n, generator=g).to(R.DT[dt]) if with_residual else None
    seed, offset, p = 0x1234_5678_9ABC_DEF0, 2 ** 40 + 17, 0.3
    y = _run(x.cuda(), p, seed, offset, None if r is None else r.cuda())
    want, kept = R.dropout(x, r, p, seed, offset)
    R.within(y, want, _bound(want, x, p, r, R.DT[dt]), "dropout")
    if not with_residual:
        assert torch.equal((y != 0).cpu(), kept & (x != 0))


@pytest.mark.parametrize("shift", [1, 2, 4])
def test_unaligned_tensors_draw_the_same_words(shift):
    n = 1001
    x = torch.randn(n + shift, device="cuda").to(torch.bfloat16)
    a = _run(x[shift:].clone(), 0.5, 9, 3)
    b = torch.full((n + shift + 8,), 7.0, dtype=torch.bfloat16, device="cuda")
    _run(x[shift:], 0.5, 9, 3, y=b[shift:shift + n])
    assert torch.equal(a, b[shift:shift + n])
    assert bool((b[:shift] == 7).all()) and bool((b[shift + n:] == 7).all())


def test_edges_of_p():
    x = torch.randn(10_000, device="cuda")
    assert torch.equal(_run(x, 0.0, 1, 1), x)
    x[::3] = float("nan")
    x[1::3] = float("inf")
    r = torch.randn(10_000, device="cuda")
    assert torch.equal(_run(x, 1.0, 1, 1, r), r)          # a dropped element is zero whatever it held
    y = _run(x, 0.5, 1, 1)
    _, kept = R.dropout(torch.zeros(10_000), None, 0.5, 1, 1)
    assert bool((y.cpu()[~kept] == 0).all()) and not bool(torch.isfinite(y.cpu()[kept][::3]).all())


def test_backward_is_the_same_call():
    """<dropout(x), g> = <x, dropout(g)>: the mask is drawn again, not stored."""
    n = 50_000
    x, g = torch.randint(-3, 4, (n,)).float().cuda(), torch.randint(-3, 4, (n,)).float().cuda()
    y, dx = _run(x, 0.5, 77, 5), _run(g, 0.5, 77, 5)
    assert float((y * g).sum()) == float((x * dx).sum())


def test_in_place_and_another_offset_in_a_replayed_graph():
    x = torch.randn(4096, device="cuda")
    want = [_run(x, 0.4, 11, k) for k in range(3)]
    rng = torch.tensor([11, 0], dtype=torch.int64, device="cuda")
    src, y = x.clone(), torch.empty_like(x)
    E.dlrm_dropout(src, y, 0.4, rng)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y.copy_(src)
        E.dlrm_dropout(y, y, 0.4, rng)
        rng[1:].add_(1)
    for k in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[k]), k


def test_more_elements_than_one_wave_and_a_fair_share():
    n = 40_000_003
    x = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    y = _run(x, 0.25, 3, 4)
    share = float((y != 0).double().mean())
    assert abs(share - 0.75) < 6 * (0.25 * 0.75 / n) ** 0.5      # six standard deviations
    tail = torch.from_numpy(R.philox(n, 3, 4)[-1000:] >= 2 ** 30)
    assert torch.equal((y[-1000:] != 0).cpu(), tail)
