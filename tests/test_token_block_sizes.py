"""Sizes past 31 bits at the token-block bindings: C takes rows, widths and
expert counts as int, and ctypes would pass the low 32 bits of a longer one (2^32 +
3 rows as 3, and the rest of the output left as it was). CPU only: the device
check is stood in for, and nothing may reach the library."""
import ctypes as C

import pytest
import torch

import embedding_bags_dot_b200 as E
from embedding_bags_dot_b200 import _abi

BIG = 2 ** 32 + 3
bf, f8 = torch.bfloat16, torch.float8_e4m3fn


def _wide(*shape, dtype=torch.float32):
    """A tensor of this shape that takes one element's memory."""
    return torch.zeros((1,) * len(shape), dtype=dtype).expand(*shape)


@pytest.fixture
def calls(monkeypatch):
    """The calls that would have reached the library, with what ctypes makes of their arguments."""
    seen = []
    monkeypatch.setattr(_abi, "_same_device", lambda where, *t: 0)
    monkeypatch.setattr(_abi, "_vector", lambda *a, **k: None)

    def call(where, dev, stream, *args):
        seen.append([t(a).value if t in (C.c_int, C.c_int64) else a for t, a in zip(_abi._SIGS[where][1], args)])
    monkeypatch.setattr(_abi, "_call", call)
    return seen


def _refused(calls, fn, *args, **kw):
    with pytest.raises(E.DlrmError) as e:
        fn(*args, **kw)
    assert e.value.status == E.ERR_UNSUPPORTED and not calls, calls


def test_norm_rows_and_widths(calls):
    x, v, ws = _wide(BIG, 1, dtype=bf), torch.zeros(1), torch.zeros(4096, dtype=torch.uint8)
    _refused(calls, E.dlrm_rmsnorm_fwd, x, None, x)
    _refused(calls, E.dlrm_rmsnorm_bwd, x, x, v, None, x, ws)
    x = _wide(2, BIG, dtype=bf)
    _refused(calls, E.dlrm_rmsnorm_fwd, x, None, x)
    _refused(calls, E.dlrm_rmsnorm_bwd, x, x, v, None, x, ws)


def test_lookup_widths(calls):
    idx, ws = torch.zeros(2, dtype=torch.int32), torch.zeros(4096, dtype=torch.uint8)

    class T:
        data, rows, d, K = _wide(3, BIG), [3], BIG, 1
        struct = _abi.dlrm_tables(16, (C.c_int64 * 1)(3), 1, BIG, E.F32)
        ref = classmethod(lambda cls: C.byref(cls.struct))
    _refused(calls, E.dlrm_embed_fwd, T, 0, idx, _wide(2, BIG), ws)

    class Dense:        # stands for 16 GB: shape and answers of a dense table
        dtype, shape = torch.float32, torch.Size((1, BIG))
        dim = staticmethod(lambda: 2)
        is_contiguous = staticmethod(lambda: True)
        data_ptr = staticmethod(lambda: 16)
        numel = staticmethod(lambda: BIG)
    _refused(calls, E.dlrm_embed_bwd, idx, _wide(2, BIG), Dense, ws)


@pytest.mark.parametrize("n_exp,M,N,K", [(1, BIG, 8, 8), (1, 8, BIG, 8), (1, 8, 8, BIG), (BIG, 8, 8, 8)])
def test_expert_sizes(calls, n_exp, M, N, K):
    X, W, Y, offs = _wide(M, K, dtype=bf), _wide(n_exp, N, K, dtype=bf), _wide(M, N, dtype=bf), torch.zeros(2, dtype=torch.int32)
    ws = torch.zeros(4096, dtype=torch.uint8)
    _refused(calls, E.dlrm_experts_fwd, X, W, offs, Y, ws)
    _refused(calls, E.dlrm_experts_bwd, Y, X, W, offs, ws, dX=X)


def test_workspace_sizes_of_refused_calls_are_zero():
    for fn, good in ((E.dlrm_rmsnorm_bwd_workspace_size, (3, 8)), (E.dlrm_experts_bwd_workspace_size, (1, 8, 8, 8)),
                     (E.dlrm_embed_bwd_workspace_size, (3, 8, 2))):
        assert fn(*good) > 0
        for i in range(len(good)):
            for v in (BIG, 2 ** 31, -BIG):
                assert fn(*good[:i], v, *good[i + 1:]) == 0, (fn.__name__, i, v)


def test_a_gradient_of_too_many_blocks_is_refused_before_its_sort():
    """2^31 - 1 ids of 65,536 columns: more sums than a grid has blocks. Nothing may have been launched by then."""
    n, d, fake = 2 ** 31 - 1, 65_536, 1 << 20
    before = E.dlrm_launch_count()
    status = E.lib().dlrm_embed_bwd(10, d, n, fake, 1.0, fake, d, E.F32, fake, E.F32, fake, 2 ** 62, None)
    assert status == E.ERR_UNSUPPORTED and E.dlrm_launch_count() == before
    assert E.dlrm_embed_bwd_workspace_size(10, d, n) == 0
    # the longest call of each kind that memory can hold is far below
    assert E.dlrm_embed_bwd_workspace_size(10, 16, n) > 0 and E.dlrm_embed_bwd_workspace_size(10, d, 2 ** 20) > 0
