"""Plain 64-bit references of the token-block operators (lookups and their
gradient, dropout, residual norm, products grouped by expert) and the error
bounds their tests use. U is half a step of fp32 relative to the value, as
torch.finfo(t).eps / 2 is of each output type."""
import numpy as np
import torch

U = torch.finfo(torch.float32).eps / 2
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def smallest(dtype):
    """Half the distance between the type's smallest values (subnormal ones included)."""
    return torch.finfo(dtype).tiny * torch.finfo(dtype).eps / 2


def within(got, want, bound, what):
    """Element by element |got - want| <= bound; NaN and infinities in the same places."""
    got, want, bound = got.double().cpu(), want.double().cpu(), bound.double().cpu()
    fine = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{what}: NaN in other places"
    assert torch.equal(got[~fine & ~torch.isnan(want)], want[~fine & ~torch.isnan(want)]), f"{what}: infinities"
    over = ((got - want).abs() - bound)[fine]
    assert over.numel() == 0 or float(over.max()) <= 0, \
        f"{what}: {int((over > 0).sum())} of {over.numel()} beyond the bound, worst by {float(over.max()):.3g}"


def philox(n, seed, offset, first=0):
    """Words first .. first + n - 1 (first a multiple of 4) of Philox4x32-10 (Salmon, Moraes, Dror and Shaw, 2011):
    counter {i / 4, offset}, key seed."""
    g = (n + 3) // 4
    mask, sh = np.uint64(0xFFFFFFFF), np.uint64(32)
    i = np.arange(g, dtype=np.uint64) + np.uint64(first // 4)
    c = [i & mask, i >> sh, np.full(g, offset & 0xFFFFFFFF, np.uint64), np.full(g, (offset >> 32) & 0xFFFFFFFF, np.uint64)]
    k0, k1 = seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF
    for _ in range(10):
        p0, p1 = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(p1 >> sh) ^ c[1] ^ np.uint64(k0), p1 & mask, (p0 >> sh) ^ c[3] ^ np.uint64(k1), p0 & mask]
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    return np.stack(c, 1).reshape(-1)[:n]


def dropout(x, residual, p, seed, offset):
    kept = torch.from_numpy((philox(x.numel(), seed, offset) >= round(p * 2 ** 32)).reshape(x.shape))
    y = torch.where(kept, x.double() / (1 - p) if p < 1 else 0.0, 0.0)
    return y if residual is None else y + residual.double(), kept


def embed_grad(rows, idx, dout, scale):
    """(gradient, sum of magnitudes, occurrences per row); indices outside the table contribute nothing."""
    idx = idx.long()
    ok = (idx >= 0) & (idx < rows)
    idx, dout = idx[ok], dout.double()[ok]
    z = torch.zeros((rows, dout.shape[1]), dtype=torch.float64)
    return (z.index_add(0, idx, dout * scale), z.index_add(0, idx, dout.abs() * abs(scale)),
            torch.bincount(idx, minlength=rows).double())


def rmsnorm(x, residual, w, eps):
    h = x.double() if residual is None else x.double() + residual.double()
    rstd = (h.square().mean(1) + eps).rsqrt()
    y = h * rstd[:, None]
    return h, rstd, y if w is None else y * w.double()


def rmsnorm_grad(dy, h, rstd, w, dh):
    """(dx, dw, magnitude behind dx, magnitude behind dw)."""
    xh = h.double() * rstd.double()[:, None]
    g = dy.double() if w is None else dy.double() * w.double()
    r = rstd.double()[:, None]
    dx = r * (g - xh * (g * xh).mean(1, keepdim=True))
    mag = r * (g.abs() + xh.abs() * (g * xh).abs().mean(1, keepdim=True))
    if dh is not None:
        dx, mag = dx + dh.double(), mag + dh.double().abs()
    return dx, (dy.double() * xh).sum(0), mag, (dy.double() * xh).abs().sum(0)


def ranges(offsets, M):
    """[begin, end) of every expert; a range that decreases, leaves [0, M] or starts below an earlier offset is
    empty. Also how many are bad."""
    out, most, bad = [], 0, 0
    for e in range(len(offsets) - 1):
        s, t = int(offsets[e]), int(offsets[e + 1])
        ok = s >= most and t >= s and t <= M
        most = max(most, s)
        bad += not ok
        out.append((s, t) if ok else (0, 0))
    return out, bad


def experts(X, W, offsets, bias, relu, x_scale=None, w_scale=None):
    """(Y, sum of magnitudes, rows that belong to an expert)."""
    M, N = X.shape[0], W.shape[1]
    X = X.double() if x_scale is None else X.double() * x_scale.double()[:, None]
    W = W.double() if w_scale is None else W.double() * w_scale.double()[..., None]
    Y, mag, owned = torch.zeros((M, N), dtype=torch.float64), torch.zeros((M, N), dtype=torch.float64), torch.zeros(M, dtype=torch.bool)
    for e, (s, t) in enumerate(ranges(offsets, M)[0]):
        Y[s:t] = X[s:t] @ W[e].T
        mag[s:t] = X[s:t].abs() @ W[e].abs().T
        if bias is not None:
            Y[s:t] += bias[e].double()
            mag[s:t] += bias[e].double().abs()
        owned[s:t] = True
    return (torch.where(Y < 0, 0.0, Y) if relu else Y), mag, owned


def experts_grad(dY, X, W, offsets, Y):
    """dX, dW, db and the sums of magnitudes behind each."""
    M, (E, N, K) = dY.shape[0], W.shape
    dP = dY.double() if Y is None else torch.where(Y.double() > 0, dY.double(), 0.0)
    z = lambda *s: torch.zeros(s, dtype=torch.float64)  # noqa: E731
    dX, dW, db, mX, mW, mb = z(M, K), z(E, N, K), z(E, N), z(M, K), z(E, N, K), z(E, N)
    for e, (s, t) in enumerate(ranges(offsets, M)[0]):
        p, x, w = dP[s:t], X[s:t].double(), W[e].double()
        dX[s:t], mX[s:t] = p @ w, p.abs() @ w.abs()
        dW[e], mW[e] = p.T @ x, p.abs().T @ x.abs()
        db[e], mb[e] = p.sum(0), p.abs().sum(0)
    return (dX, dW, db), (mX, mW, mb)
