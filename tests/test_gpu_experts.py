"""dlrm_experts_fwd and dlrm_experts_bwd against 64-bit references: both
tile kernels, types, ragged and empty experts, odd widths, rows that belong to
no expert, bad ranges, infinities and NaN next to an expert's rows.

Bounds: products of 16-bit (and of e4m3) values are exact in fp32, so what is
left is the sums: held, as the library's other tensor-core products are, to
1e-5 of the sum of magnitudes, plus one rounding of the output. Small integers
add exactly and must come out equal."""
import pytest
import torch

import block_ref as R
import embedding_bags_dot_b200 as E

pytestmark = pytest.mark.gpu


def _pitched(t, dt):
    """t on the device in rows that start on 16 bytes, with NaN in the padding."""
    per = 16 // torch.empty(0, dtype=dt).element_size()
    w = t.shape[-1]
    buf = torch.full((*t.shape[:-1], (w + per - 1) // per * per), float("nan"), dtype=torch.float32).to(dt).cuda()
    if dt == torch.float8_e4m3fn:
        buf.view(torch.uint8)[..., :w] = t.to(dt).view(torch.uint8).cuda()
    else:
        buf[..., :w] = t.to(dt)
    return buf[..., :w]


def _offsets(sizes, first=0):
    return torch.tensor([first] + [first + int(s) for s in torch.tensor(sizes).cumsum(0)], dtype=torch.int32)


def _values(kind, shape, g, scale=1.0):
    if kind == "int":
        return torch.randint(-3, 4, shape, generator=g).float()
    return torch.randn(shape, generator=g) * scale


def _case(sizes, spare, N, K, dt, kind, seed=0):
    g = torch.Generator().manual_seed(seed + N + K)
    n_exp, M = len(sizes), sum(sizes) + spare
    X = _values(kind, (M, K), g).to(dt)
    W = _values(kind, (n_exp, N, K), g, K ** -0.5).to(dt)
    bias = _values(kind, (n_exp, N), g)
    return X, W, bias, _offsets(sizes), M


def _forward(X, W, offs, y_dt, bias=None, act=E.ACT_NONE, x_scale=None, w_scale=None, fill=-7.0):
    M, N = X.shape[0], W.shape[1]
    Y = _pitched(torch.full((M, N), fill), y_dt)
    ws = E.alloc_workspace(E.ERR_RECORD_BYTES)
    c = lambda t: None if t is None else t.cuda()  # noqa: E731
    E.dlrm_experts_fwd(_pitched(X, X.dtype), _pitched(W, W.dtype), offs.cuda(), Y, ws, bias=c(bias), act=act,
                       x_scale=c(x_scale), w_scale=c(w_scale))
    return Y, E.dlrm_check_error(ws)


def _check_forward(Y, X, W, offs, bias, relu, y_dt, x_scale=None, w_scale=None, fill=-7.0, exact=False):
    want, mag, owned = R.experts(X, W, offs, bias, relu, x_scale, w_scale)
    got = Y.cpu()
    assert bool((got[~owned] == fill).all()), "rows of no expert were written"
    if exact:
        assert torch.equal(got[owned].double(), want[owned].to(y_dt).double())
    else:
        step = 0 if y_dt == torch.float32 else R.half_step(y_dt)
        R.within(got[owned], want[owned], 1e-5 * mag[owned] + step * want[owned].abs() + R.smallest(y_dt), "Y")


SMALL = [([1], 0, 1, 1), ([1, 0, 2], 3, 8, 16), ([5, 40, 0, 1], 2, 64, 64), ([33, 128, 129, 0, 7], 10, 200, 479),
         ([0, 0, 300], 0, 130, 72), ([31, 32, 33, 64, 65], 0, 1024, 100)]
LARGE = [([4000, 0, 257, 900, 255, 256], 5, 1024, 479), ([20_000], 0, 300, 128), ([1000] * 20, 17, 260, 640)]


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("sizes,spare,N,K", SMALL + LARGE)
def test_small_integers_come_out_exactly(dt, sizes, spare, N, K):
    X, W, bias, offs, _ = _case(sizes, spare, N, K, dt, "int")
    Y, st = _forward(X, W, offs, torch.float32, bias)
    assert st[0] == E.OK
    _check_forward(Y, X, W, offs, bias, False, torch.float32, exact=True)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("sizes,spare,N,K", SMALL + LARGE + [([9, 3], 0, 96, 4096), ([2000, 3000, 4000], 0, 512, 4096)])
def test_forward_with_bias_and_relu(dt, sizes, spare, N, K):
    X, W, bias, offs, _ = _case(sizes, spare, N, K, dt, "randn")
    for y_dt, b, act in ((dt, bias, E.ACT_RELU), (torch.float32, None, E.ACT_NONE)):
        Y, st = _forward(X, W, offs, y_dt, b, act)
        assert st[0] == E.OK
        _check_forward(Y, X, W, offs, b, act == E.ACT_RELU, y_dt)


def _quantized(t):
    s = t.abs().amax(-1) / 448
    return (t / s[..., None]).to(torch.float8_e4m3fn), s


@pytest.mark.parametrize("y_dt", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("sizes,spare,N,K", SMALL + LARGE + [([9, 3], 0, 96, 4096)])
def test_8_bit_operands_with_row_scales(y_dt, sizes, spare, N, K):
    g = torch.Generator().manual_seed(N)
    M = sum(sizes) + spare
    X, xs = _quantized(torch.randn((M, K), generator=g) + 1e-3)
    W, wsc = _quantized(torch.randn((len(sizes), N, K), generator=g) * K ** -0.5 + 1e-4)
    bias = torch.randn((len(sizes), N), generator=g)
    Y, st = _forward(X, W, _offsets(sizes), y_dt, bias, E.ACT_RELU, xs, wsc)
    assert st[0] == E.OK
    _check_forward(Y, X.float(), W.float(), _offsets(sizes), bias, True, y_dt, xs, wsc)


@pytest.mark.parametrize("sizes,spare,N,K", [SMALL[3], LARGE[0]])
def test_rows_do_not_mix(sizes, spare, N, K):
    """NaN in the rows after an expert's last one (the next expert's, and those of none), in another expert's
    weights and in the padding: they stay where they are."""
    X, W, bias, offs, M = _case(sizes, spare, N, K, torch.bfloat16, "randn")
    used = [e for e, s in enumerate(sizes) if s > 3]
    bad = used[1]
    X[int(offs[bad]):int(offs[bad + 1])] = float("nan")
    X[int(offs[-1]):] = float("inf")
    W[bad] = float("nan")
    Y, _ = _forward(X, W, offs, torch.bfloat16, bias)
    got = Y.cpu()
    keep = torch.ones(M, dtype=torch.bool)
    keep[int(offs[bad]):int(offs[bad + 1])] = False
    assert bool(torch.isnan(got[~keep]).all())
    want, mag, owned = R.experts(torch.nan_to_num(X.float(), 0, 0, 0), torch.nan_to_num(W.float()), offs, bias, False)
    keep &= owned
    R.within(got[keep], want[keep], 1e-5 * mag[keep] + R.half_step(torch.bfloat16) * want[keep].abs(), "the others")
    assert bool((got[~owned] == -7).all())


BAD = [[0, 10, 5, 30, 40], [0, 10, 50, 20, 64], [-3, 10, 20, 30, 40], [5, 10, 10, 90, 64], [0, 70, 71, 72, 73],
       [10, 20, 30, 25, 40], [2 ** 31 - 1, -2 ** 31, 0, 64, 64]]


@pytest.mark.parametrize("offsets", BAD)
def test_bad_ranges_are_empty_and_counted(offsets):
    n_exp, M, N, K = 4, 64, 72, 96
    g = torch.Generator().manual_seed(1)
    X, W = _values("int", (M, K), g).bfloat16(), _values("int", (n_exp, N, K), g).bfloat16()
    offs = torch.tensor(offsets, dtype=torch.int32)
    bad = R.ranges(offsets, M)[1]
    assert bad > 0
    Y, st = _forward(X, W, offs, torch.float32)
    assert st == (E.ERR_BAD_OFFSETS, 2, 0, bad)
    _check_forward(Y, X, W, offs, None, False, torch.float32, exact=True)
    dY = _values("int", (M, N), g).bfloat16()
    (dX, dW, db), st = _backward(dY, X, W, offs, None, torch.float32, torch.float32)
    assert st == (E.ERR_BAD_OFFSETS, 2, 0, bad)      # counted once per call
    (wX, wW, wb), _ = R.experts_grad(dY, X, W, offs, None)
    owned = R.experts(X, W, offs, None, False)[2]
    assert torch.equal(dX.cpu()[owned].double(), wX[owned]) and bool((dX.cpu()[~owned] == -7).all())
    assert torch.equal(dW.cpu().double(), wW) and torch.equal(db.cpu().double(), wb)


def _backward(dY, X, W, offs, Y, dx_dt, dw_dt, parts=("dX", "dW", "db")):
    M, (n_exp, N, K) = dY.shape[0], W.shape
    act = E.ACT_NONE if Y is None else E.ACT_RELU
    ws = E.alloc_workspace(E.dlrm_experts_bwd_workspace_size(n_exp, M, N, K, act))
    ws[E.ERR_RECORD_BYTES:] = 0xFF       # what an earlier call left there (NaN in every type)
    out = {"dX": _pitched(torch.full((M, K), -7.0), dx_dt), "dW": _pitched(torch.full((n_exp, N, K), float("nan")), dw_dt),
           "db": torch.full((n_exp, N), float("nan"), device="cuda")}
    E.dlrm_experts_bwd(_pitched(dY, dY.dtype), _pitched(X, X.dtype), _pitched(W, W.dtype), offs.cuda(), ws,
                       Y=None if Y is None else _pitched(Y, Y.dtype), act=act, **{k: out[k] for k in parts})
    return tuple(out[k] for k in parts), E.dlrm_check_error(ws)


GRAD = [([1], 0, 1, 1), ([1, 0, 2], 3, 8, 16), ([33, 128, 129, 0, 7], 10, 200, 479), ([64, 63, 65, 0, 640], 1, 72, 300),
        ([4000, 0, 257, 900, 255, 256], 5, 512, 264), ([1500, 3], 100, 260, 1024)]


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("relu", [False, True])
@pytest.mark.parametrize("sizes,spare,N,K", GRAD)
def test_gradients_of_small_integers_come_out_exactly(dt, relu, sizes, spare, N, K):
    X, W, _, offs, M = _case(sizes, spare, N, K, dt, "int")
    g = torch.Generator().manual_seed(3)
    dY = _values("int", (M, N), g).to(dt)
    Y = _values("int", (M, N), g).to(dt) if relu else None
    (dX, dW, db), st = _backward(dY, X, W, offs, Y, torch.float32, torch.float32)
    assert st[0] == E.OK
    (wX, wW, wb), _ = R.experts_grad(dY, X, W, offs, Y)
    owned = R.experts(X, W, offs, None, False)[2]
    assert torch.equal(dX.cpu()[owned].double(), wX[owned]) and bool((dX.cpu()[~owned] == -7).all())
    assert torch.equal(dW.cpu().double(), wW)
    assert torch.equal(db.cpu().double(), wb)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("sizes,spare,N,K", GRAD + [([3000, 9000], 0, 256, 256)])
def test_gradients(dt, sizes, spare, N, K):
    X, W, bias, offs, M = _case(sizes, spare, N, K, dt, "randn")
    g = torch.Generator().manual_seed(4)
    dY = torch.randn((M, N), generator=g).to(dt)
    Y = torch.randn((M, N), generator=g).clamp(min=0).to(dt)
    owned = R.experts(X, W, offs, None, False)[2]
    (wX, wW, wb), (mX, mW, mb) = R.experts_grad(dY, X, W, offs, Y)
    for o_dt in (dt, torch.float32):
        (dX, dW, db), st = _backward(dY, X, W, offs, Y, o_dt, o_dt)
        assert st[0] == E.OK
        step = 0 if o_dt == torch.float32 else R.half_step(o_dt)
        tiny = R.smallest(o_dt)
        R.within(dX.cpu()[owned], wX[owned], 1e-5 * mX[owned] + step * wX[owned].abs() + tiny, "dX")
        R.within(dW, wW, 1e-5 * mW + step * wW.abs() + tiny, "dW")
        R.within(db, wb, 1e-5 * mb, "db")
    # each output alone is the same
    for k, ref in (("dX", dX), ("dW", dW), ("db", db)):
        (one,), _ = _backward(dY, X, W, offs, Y, torch.float32, torch.float32, parts=(k,))
        assert torch.equal(one, ref), k


@pytest.mark.parametrize("relu", [False, True])
def test_gradients_keep_other_rows_out(relu):
    """Infinities and NaN in rows of no expert, right behind an expert's last row, reach no gradient."""
    X, W, _, offs, M = _case([100, 30, 65], 70, 72, 80, torch.bfloat16, "int")
    dY = _values("int", (M, 72), torch.Generator().manual_seed(5)).bfloat16()
    Y = torch.ones((M, 72), dtype=torch.bfloat16) if relu else None
    clean, _ = _backward(dY, X, W, offs, Y, torch.float32, torch.float32)
    X[195:], dY[195:] = float("nan"), float("inf")
    if relu:
        Y[195:] = float("nan")
    got, _ = _backward(dY, X, W, offs, Y, torch.float32, torch.float32)
    for a, b in zip(got, clean):
        assert torch.equal(a, b)


def test_rows_before_the_first_expert():
    sizes, N, K = [70, 0, 200], 48, 64
    g = torch.Generator().manual_seed(12)
    M = 5 + sum(sizes) + 9
    X, W = _values("int", (M, K), g).bfloat16(), _values("int", (3, N, K), g).bfloat16()
    offs = _offsets(sizes, first=5)
    Y, st = _forward(X, W, offs, torch.float32)
    assert st[0] == E.OK
    _check_forward(Y, X, W, offs, None, False, torch.float32, exact=True)
    dY = _values("int", (M, N), g).bfloat16()
    (dX, dW, db), st = _backward(dY, X, W, offs, None, torch.bfloat16, torch.float32)
    (wX, wW, wb), _ = R.experts_grad(dY, X, W, offs, None)
    assert st[0] == E.OK and torch.equal(dW.cpu().double(), wW) and torch.equal(db.cpu().double(), wb)
    assert torch.equal(dX.cpu()[5:275].double(), wX[5:275].to(torch.bfloat16).double())
    assert bool((dX.cpu()[:5] == -7).all()) and bool((dX.cpu()[275:] == -7).all())


def test_no_rows_at_all():
    X, W = torch.zeros((0, 64), dtype=torch.bfloat16), torch.ones((3, 40, 64), dtype=torch.bfloat16)
    offs = torch.zeros(4, dtype=torch.int32)
    Y, st = _forward(X, W, offs, torch.bfloat16)
    assert Y.shape == (0, 40) and st[0] == E.OK
    (dX, dW, db), st = _backward(torch.zeros((0, 40), dtype=torch.bfloat16), X, W, offs, None, torch.bfloat16, torch.float32)
    assert st[0] == E.OK and bool((dW == 0).all()) and bool((db == 0).all())


def test_many_experts():
    sizes = [(i * 7) % 13 for i in range(256)]
    X, W, bias, offs, M = _case(sizes, 4, 40, 32, torch.bfloat16, "int")
    Y, st = _forward(X, W, offs, torch.float32, bias)
    assert st[0] == E.OK
    _check_forward(Y, X, W, offs, bias, False, torch.float32, exact=True)
    dY = _values("int", (M, 40), torch.Generator().manual_seed(6)).bfloat16()
    (dX, dW, db), _ = _backward(dY, X, W, offs, None, torch.float32, torch.float32)
    (wX, wW, wb), _ = R.experts_grad(dY, X, W, offs, None)
    n = sum(sizes)
    assert torch.equal(dX.cpu()[:n].double(), wX[:n]) and torch.equal(dW.cpu().double(), wW) and torch.equal(db.cpu().double(), wb)


def test_the_same_call_gives_the_same_bits():
    X, W, bias, offs, M = _case([700, 1300, 5], 3, 512, 520, torch.bfloat16, "randn")
    dY = torch.randn((M, 512)).bfloat16()
    a, b = (_forward(X, W, offs, torch.bfloat16, bias)[0] for _ in range(2))
    assert torch.equal(a, b)
    a, b = (_backward(dY, X, W, offs, None, torch.bfloat16, torch.float32)[0] for _ in range(2))
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_gradients_agree_with_differences():
    """The forward of the library itself along random directions, in fp32 outputs of exactly representable steps."""
    X, W, bias, offs, M = _case([20, 0, 45], 0, 24, 40, torch.bfloat16, "int")
    g = torch.Generator().manual_seed(8)
    c = _values("int", (M, 24), g).bfloat16()
    (dX, dW, db), _ = _backward(c, X, W, offs, None, torch.float32, torch.float32)
    f = lambda x, w, b: float((_forward(x, w, offs, torch.float32, b)[0].cpu().double() * c.double()).sum())  # noqa: E731
    base = f(X, W, bias)
    for _ in range(3):
        v, u, t = _values("int", X.shape, g), _values("int", W.shape, g), _values("int", bias.shape, g)
        # linear in each argument, and exact in these integers: the difference is the directional derivative
        assert f((X.float() + v).bfloat16(), W, bias) - base == float((dX.cpu().double() * v).sum())
        assert f(X, (W.float() + u).bfloat16(), bias) - base == float((dW.cpu().double() * u).sum())
        assert f(X, W, bias + t) - base == float((db.cpu().double() * t).sum())
