"""Host-side checks of the token-block entry points, through the C ABI and
through the bindings (CPU only: every call here is refused, or has nothing to
do, before any kernel is launched). Also the host references' own checks."""
import ctypes as C

import numpy as np
import pytest
import torch

import block_ref as R

FAKE = 1 << 20          # a 16-byte aligned address that no refused call reads


@pytest.fixture(scope="module")
def lib():
    import os

    from embedding_bags_dot_b200 import _abi, build
    if not os.path.exists(_abi.LIB_PATH):
        build.build()
    return _abi.lib()


def _refused(lib, name, good, changes, accepted=()):
    """Every changed argument list gives the status beside it and launches nothing."""
    import embedding_bags_dot_b200 as E
    fn, before = getattr(lib, name), E.dlrm_launch_count()
    for change, status in changes:
        args = dict(good)
        args.update(change)
        assert fn(*args.values()) == status, (name, change)
    for change in accepted:
        args = dict(good)
        args.update(change)
        assert fn(*args.values()) == E.OK, (name, change)
    assert E.dlrm_launch_count() == before


def test_lookup_refusals(lib):
    import embedding_bags_dot_b200 as E
    rows = (C.c_int64 * 3)(10, 20, 30)
    T = lambda **k: C.byref(E._abi.dlrm_tables(*dict(dict(data=FAKE, rows=rows, K=3, d=16, dt=E.F32), **k).values()))  # noqa: E731
    good = dict(T=T(), k=1, n=5, idx=FAKE, scale=1.0, out=FAKE, ld=16, dt=E.F32, ws=FAKE, nws=256, st=None)
    bad = E.ERR_INVALID_ARG
    zero = (C.c_int64 * 3)(10, 0, 30)
    big = (C.c_int64 * 3)(10, 2 ** 31, 30)
    _refused(lib, "dlrm_embed_fwd", good, [
        (dict(T=None), bad), (dict(T=T(data=None)), bad), (dict(T=T(data=FAKE + 8)), bad), (dict(T=T(d=0)), bad),
        (dict(T=T(dt=E.U8ROW)), E.ERR_UNSUPPORTED), (dict(T=T(dt=E.E4M3)), bad), (dict(T=T(dt=9)), bad),
        (dict(T=T(d=65537)), E.ERR_UNSUPPORTED), (dict(T=T(rows=zero)), bad), (dict(T=T(rows=big)), E.ERR_UNSUPPORTED),
        (dict(k=-1), bad), (dict(k=3), bad), (dict(n=-1), bad), (dict(n=2 ** 31), bad), (dict(idx=None), bad),
        (dict(idx=FAKE + 2), bad), (dict(out=None), bad), (dict(out=FAKE + 2), bad), (dict(ld=15), bad),
        (dict(dt=E.E4M3), bad), (dict(dt=E.U8ROW), bad), (dict(ws=None), E.ERR_WORKSPACE),
        (dict(nws=255), E.ERR_WORKSPACE), (dict(ws=FAKE + 8), E.ERR_WORKSPACE)],
        accepted=[dict(n=0), dict(n=0, idx=None, out=None)])


def test_lookup_gradient_refusals(lib):
    import embedding_bags_dot_b200 as E
    need = lib.dlrm_embed_bwd_workspace_size(100, 16, 50)
    assert need >= 256 + 2 * 4 * 50
    good = dict(rows=100, d=16, n=50, idx=FAKE, scale=1.0, dout=FAKE, ld=16, dt=E.BF16, out=FAKE, odt=E.F32, ws=FAKE,
                nws=need, st=None)
    bad = E.ERR_INVALID_ARG
    _refused(lib, "dlrm_embed_bwd", good, [
        (dict(rows=0), bad), (dict(rows=2 ** 31), E.ERR_UNSUPPORTED), (dict(d=0), bad), (dict(d=65537), E.ERR_UNSUPPORTED),
        (dict(n=-1), bad), (dict(n=2 ** 31), bad), (dict(idx=None), bad), (dict(dout=None), bad), (dict(dout=FAKE + 1), bad),
        (dict(ld=15), bad), (dict(dt=E.E4M3), bad), (dict(out=None), bad), (dict(out=FAKE + 2), bad), (dict(odt=7), bad),
        (dict(ws=None), E.ERR_WORKSPACE), (dict(nws=need - 1), E.ERR_WORKSPACE), (dict(ws=FAKE + 8), E.ERR_WORKSPACE)])
    for rows, d, n in ((0, 16, 5), (5, 0, 5), (5, 5, -1), (2 ** 31, 5, 5), (5, 65537, 5)):
        assert E.dlrm_embed_bwd_workspace_size(rows, d, n) == 0


def test_dropout_refusals(lib):
    import embedding_bags_dot_b200 as E
    good = dict(n=100, x=FAKE, res=None, dt=E.F32, p=0.1, rng=FAKE, y=FAKE, st=None)
    bad = E.ERR_INVALID_ARG
    _refused(lib, "dlrm_dropout", good, [
        (dict(n=-1), bad), (dict(x=None), bad), (dict(x=FAKE + 2), bad), (dict(y=None), bad), (dict(y=FAKE + 1), bad),
        (dict(res=FAKE + 2), bad), (dict(rng=None), bad), (dict(rng=FAKE + 4), bad), (dict(dt=E.E4M3), bad), (dict(dt=-1), bad),
        (dict(p=-0.01), bad), (dict(p=1.01), bad), (dict(p=float("nan")), bad)],
        accepted=[dict(n=0), dict(n=0, x=None, y=None, rng=None)])


def test_norm_refusals(lib):
    import embedding_bags_dot_b200 as E
    good = dict(rows=4, d=64, x=FAKE, lx=64, res=FAKE, lr=64, dt=E.BF16, w=FAKE, eps=1e-6, h=FAKE, lh=64, y=FAKE, ly=64,
                ydt=E.BF16, ys=None, rstd=FAKE, st=None)
    bad = E.ERR_INVALID_ARG
    _refused(lib, "dlrm_rmsnorm_fwd", good, [
        (dict(rows=-1), bad), (dict(d=0), bad), (dict(d=32769, lx=40000, lr=40000, lh=40000, ly=40000), E.ERR_UNSUPPORTED),
        (dict(x=None), bad), (dict(lx=63), bad), (dict(x=FAKE + 1), bad), (dict(lr=63), bad), (dict(lh=63), bad), (dict(ly=63), bad),
        (dict(y=None), bad), (dict(dt=E.E4M3), bad), (dict(ydt=E.F32), bad), (dict(ydt=E.E4M3), bad), (dict(ys=FAKE), bad),
        (dict(ydt=E.E4M3, ys=FAKE + 2), bad), (dict(w=FAKE + 2), bad), (dict(rstd=FAKE + 1), bad), (dict(eps=-1.0), bad),
        (dict(eps=float("nan")), bad)], accepted=[dict(rows=0)])
    need = lib.dlrm_rmsnorm_bwd_workspace_size(4, 64)
    assert need >= 256 + 4 * 64 and E.dlrm_rmsnorm_bwd_workspace_size(4, 32769) == 0
    assert E.dlrm_rmsnorm_bwd_workspace_size(-1, 64) == 0 and E.dlrm_rmsnorm_bwd_workspace_size(4, 0) == 0
    good = dict(rows=4, d=64, dy=FAKE, ldy=64, h=FAKE, lh=64, rstd=FAKE, w=None, dh=FAKE, ldh=64, dt=E.F16, dx=FAKE, ldx=64,
                dw=FAKE, ws=FAKE, nws=need, st=None)
    _refused(lib, "dlrm_rmsnorm_bwd", good, [
        (dict(rows=-1), bad), (dict(d=0), bad), (dict(d=32769), E.ERR_UNSUPPORTED), (dict(dy=None), bad), (dict(h=None), bad),
        (dict(rstd=None), bad), (dict(dx=None), bad), (dict(ldy=63), bad), (dict(lh=63), bad), (dict(ldh=63), bad),
        (dict(ldx=63), bad), (dict(dt=E.E4M3), bad), (dict(dw=FAKE + 2), bad), (dict(ws=None), E.ERR_WORKSPACE),
        (dict(nws=need - 1), E.ERR_WORKSPACE), (dict(ws=FAKE + 4), E.ERR_WORKSPACE)])


def test_experts_refusals(lib):
    import embedding_bags_dot_b200 as E
    bad, un, wsp = E.ERR_INVALID_ARG, E.ERR_UNSUPPORTED, E.ERR_WORKSPACE
    good = dict(E=4, M=32, N=24, K=40, offs=FAKE, X=FAKE, ldx=40, xs=None, dt=E.BF16, W=FAKE, ldw=40, wscale=None, bias=FAKE,
                act=E.ACT_RELU, Y=FAKE, ldy=24, ydt=E.BF16, ws=FAKE, nws=256, st=None)
    _refused(lib, "dlrm_experts_fwd", good, [
        (dict(E=0), bad), (dict(E=257), un), (dict(M=-1), bad), (dict(N=0), bad), (dict(K=0), bad), (dict(dt=E.F32), un),
        (dict(dt=E.U8ROW), bad), (dict(ydt=E.F16), un), (dict(ydt=E.E4M3), bad), (dict(act=E.ACT_SIGMOID), bad),
        (dict(offs=None), bad), (dict(offs=FAKE + 2), bad), (dict(X=None), bad), (dict(X=FAKE + 8), bad), (dict(ldx=36), bad),
        (dict(ldx=44), bad), (dict(W=None), bad), (dict(ldw=36), bad), (dict(Y=None), bad), (dict(Y=FAKE + 4), bad),
        (dict(ldy=20), bad), (dict(ldy=28), bad), (dict(bias=FAKE + 1), bad), (dict(xs=FAKE), bad), (dict(wscale=FAKE), bad),
        (dict(dt=E.E4M3, ldx=48, ldw=48), bad), (dict(dt=E.E4M3, ldx=48, ldw=48, xs=FAKE), bad),
        (dict(dt=E.E4M3, ldx=40, ldw=48, xs=FAKE, wscale=FAKE), bad), (dict(ws=None), wsp), (dict(nws=255), wsp),
        (dict(M=2 ** 31 - 1, N=2 ** 20, ldy=2 ** 20), un)], accepted=[dict(M=0)])
    need = lib.dlrm_experts_bwd_workspace_size(4, 32, 24, 40, E.ACT_RELU)
    assert need > lib.dlrm_experts_bwd_workspace_size(4, 32, 24, 40, E.ACT_NONE) > 0
    for args in ((0, 32, 24, 40, 0), (257, 32, 24, 40, 0), (4, -1, 24, 40, 0), (4, 32, 0, 40, 0), (4, 32, 24, 0, 0), (4, 32, 24, 40, 2)):
        assert lib.dlrm_experts_bwd_workspace_size(*args) == 0
    good = dict(E=4, M=32, N=24, K=40, offs=FAKE, dY=FAKE, lddy=24, Y=FAKE, ldy=24, act=E.ACT_RELU, X=FAKE, ldx=40, W=FAKE,
                ldw=40, dt=E.F16, dX=FAKE, lddx=40, dxdt=E.F16, dW=FAKE, lddw=40, dwdt=E.F32, db=FAKE, ws=FAKE, nws=need, st=None)
    _refused(lib, "dlrm_experts_bwd", good, [
        (dict(dt=E.F32), un), (dict(dt=E.E4M3), un), (dict(dt=E.U8ROW), bad), (dict(act=2), bad), (dict(E=257), un),
        (dict(offs=None), bad), (dict(dY=None), bad), (dict(lddy=20), bad), (dict(Y=None), bad), (dict(ldy=28), bad),
        (dict(X=None), bad), (dict(ldx=44), bad), (dict(W=None), bad), (dict(ldw=36), bad), (dict(dX=FAKE + 8), bad),
        (dict(lddx=44), bad), (dict(dxdt=E.BF16), un), (dict(dxdt=E.E4M3), bad), (dict(dwdt=E.BF16), un), (dict(lddw=38), bad),
        (dict(db=FAKE + 2), bad), (dict(ws=None), wsp), (dict(nws=need - 1), wsp), (dict(ws=FAKE + 8), wsp)])


def test_experts_rows_leave_a_tile_below_31_bits(lib):
    import embedding_bags_dot_b200 as E
    for M, ok in ((2 ** 31 - 256, True), (2 ** 31 - 255, False), (2 ** 31 - 1, False)):
        assert (lib.dlrm_experts_bwd_workspace_size(1, M, 8, 8, E.ACT_NONE) > 0) == ok
        if not ok:
            assert lib.dlrm_experts_fwd(1, M, 8, 8, FAKE, FAKE, 8, None, E.BF16, FAKE, 8, None, None, E.ACT_NONE, FAKE, 8,
                                        E.BF16, FAKE, 256, None) == E.ERR_UNSUPPORTED


def _raises(status, call, *args, **kw):
    import embedding_bags_dot_b200 as E
    before = E.dlrm_launch_count()
    with pytest.raises(E.DlrmError) as e:
        call(*args, **kw)
    assert e.value.status == status and E.dlrm_launch_count() == before


def test_bindings_refuse_tensors_that_do_not_fit(lib):
    """Wrong shapes, types and layouts, and host tensors, before the C entry point sees an address."""
    import embedding_bags_dot_b200 as E
    bad = E.ERR_INVALID_ARG
    z = torch.zeros
    bf = torch.bfloat16
    i32, ws = z(8, dtype=torch.int32), z(1 << 16, dtype=torch.uint8)

    class T:        # a table handle whose tensor is on the host
        data, rows, d, K = z((10, 16)), [10], 16, 1
        struct = E._abi.dlrm_tables(FAKE, (C.c_int64 * 1)(10), 1, 16, E.F32)
        ref = classmethod(lambda cls: C.byref(cls.struct))

    out = z((8, 16))
    for idx, o, k in ((i32, out, 0), (i32.long(), out, 0), (i32[::2], out, 0), (i32, out[:7], 0), (i32, z((8, 17)), 0),
                      (i32, z((16, 8)).t(), 0), (i32, out, 1), (i32, out, -1), (i32, z((8, 16), dtype=torch.int32), 0)):
        _raises(bad, E.dlrm_embed_fwd, T, k, idx, o, ws)
    for idx, dout, dt in ((i32, out, z((10, 16))), (i32.long(), out, z((10, 16))), (i32, out[:, :15], z((10, 16))),
                          (i32, out, z((10, 32))[:, :16]), (i32, out, z(160))):
        _raises(bad, E.dlrm_embed_bwd, idx, dout, dt, ws)
    rng = z(2, dtype=torch.int64)
    x = z((4, 6))
    for xx, y, r, res in ((x, x, rng, None), (x, z((4, 5)), rng, None), (x, z((4, 6), dtype=bf), rng, None),
                          (z((4, 12))[:, :6], x, rng, None), (x, x, rng[:1], None), (x, x, rng.int(), None),
                          (x, x, rng, z((6, 4))), (x, x, rng, z((4, 6), dtype=bf)), (x, x, None, None)):
        _raises(bad, E.dlrm_dropout, xx, y, 0.1, r, residual=res)
    w, y8, s = z(6), z((4, 6), dtype=torch.float8_e4m3fn), z(4)
    for kw in (dict(), dict(w=z(5)), dict(w=z(6, dtype=bf)), dict(y=z((4, 7))), dict(y=z((4, 6), dtype=bf)), dict(y=y8),
               dict(y=y8, y_scale=z(3)), dict(y_scale=s), dict(residual=z((4, 6), dtype=bf)), dict(residual=z((3, 6))),
               dict(h=z((4, 6), dtype=bf)), dict(rstd=z(3)), dict(x=z(6)), dict(x=z((6, 4)).t())):
        a = dict(dict(x=x, w=w, y=z((4, 6))), **kw)
        _raises(bad, E.dlrm_rmsnorm_fwd, a.pop("x"), a.pop("w"), a.pop("y"), **a)
    for kw in (dict(), dict(h=z((4, 6), dtype=bf)), dict(rstd=None), dict(rstd=z(3)), dict(dx=z((4, 5))), dict(dw=z(5)),
               dict(dh=z((4, 6), dtype=bf))):
        a = dict(dict(dy=x, h=x, rstd=s, w=w, dx=z((4, 6)), ws=ws), **kw)
        _raises(bad, E.dlrm_rmsnorm_bwd, a.pop("dy"), a.pop("h"), a.pop("rstd"), a.pop("w"), a.pop("dx"), a.pop("ws"), **a)
    X, W, offs, Y = z((8, 16), dtype=bf), z((3, 24, 16), dtype=bf), z(4, dtype=torch.int32), z((8, 24), dtype=bf)
    for kw in (dict(), dict(X=z((8, 15), dtype=bf)), dict(X=z((8, 16), dtype=torch.float16)), dict(W=z((24, 16), dtype=bf)),
               dict(W=z((3, 16, 24), dtype=bf).transpose(1, 2)), dict(W=z((6, 24, 16), dtype=bf)[::2]),
               dict(offs=z(3, dtype=torch.int32)), dict(offs=z(4, dtype=torch.int64)), dict(offs=None),
               dict(Y=z((8, 23), dtype=bf)), dict(Y=z((24, 8), dtype=bf).t()), dict(bias=z((3, 23))), dict(bias=z((3, 24), dtype=bf)),
               dict(x_scale=z(7)), dict(w_scale=z((3, 23)))):
        a = dict(dict(X=X, W=W, offs=offs, Y=Y, ws=ws), **kw)
        _raises(bad, E.dlrm_experts_fwd, a.pop("X"), a.pop("W"), a.pop("offs"), a.pop("Y"), a.pop("ws"), **a)
    dY = z((8, 24), dtype=bf)
    for kw in (dict(), dict(dY=z((8, 24))), dict(act=E.ACT_RELU), dict(Y=z((8, 24)), act=E.ACT_RELU), dict(dX=z((8, 15), dtype=bf)),
               dict(dW=z((3, 24, 15))), dict(db=z((3, 23))), dict(db=z((3, 24), dtype=bf))):
        a = dict(dict(dY=dY, X=X, W=W, offs=offs, ws=ws), **kw)
        _raises(bad, E.dlrm_experts_bwd, a.pop("dY"), a.pop("X"), a.pop("W"), a.pop("offs"), a.pop("ws"), **a)


def test_leading_dimension_of_8_bit_rows(lib):
    import embedding_bags_dot_b200 as E
    assert E.dlrm_ld(479, "e4m3") == 480 and E.dlrm_ld(1, torch.float8_e4m3fn) == 16 and E.dlrm_ld(33, "e4m3") == 48


def test_reference_generator_gives_the_published_words():
    """Known answers of Philox4x32-10 for counters and keys of zeros and of ones (Random123's test vectors)."""
    assert [hex(v) for v in R.philox(4, 0, 0)] == ["0x6627e8d5", "0xe169c58d", "0xbc57ac4c", "0x9b00dbd8"]
    # the all-ones counter cannot be reached by an element number: the rounds alone
    c, k = np.array([0xFFFFFFFF] * 4, np.uint64), [0xFFFFFFFF, 0xFFFFFFFF]
    for _ in range(10):
        p0, p1 = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        sh, m = np.uint64(32), np.uint64(0xFFFFFFFF)
        c = np.array([(p1 >> sh) ^ c[1] ^ np.uint64(k[0]), p1 & m, (p0 >> sh) ^ c[3] ^ np.uint64(k[1]), p0 & m], np.uint64)
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    assert [hex(v) for v in c] == ["0x408f276d", "0x41c83b0e", "0xa20bc7c6", "0x6d5451fd"]


def test_reference_ranges():
    assert R.ranges([0, 3, 3, 8], 8) == ([(0, 3), (3, 3), (3, 8)], 0)
    assert R.ranges([0, 10, 5, 30, 40], 64) == ([(0, 10), (0, 0), (0, 0), (30, 40)], 2)
    assert R.ranges([-1, 2, 9], 8) == ([(0, 0), (0, 0)], 2)
