"""Entry points that take no 8-bit floating point rows refuse the type, sizes included (CPU only)."""
import ctypes as C

import torch

import embedding_bags_dot_b200 as E


def test_there_are_no_table_rows_of_8_bit_floats():
    assert E.dlrm_row_bytes(64, "e4m3") == 0 == E.dlrm_row_bytes(64, torch.float8_e4m3fn)
    assert E.dlrm_row_bytes(64, "bf16") == 128 and E.dlrm_row_bytes(64, "f32") == 256 and E.dlrm_row_bytes(64, "u8row") == 80


def test_tables_and_layers_of_8_bit_floats_are_refused():
    rows = (C.c_int64 * 1)(10)
    T = E._abi.dlrm_tables(1 << 20, rows, 1, 64, E.E4M3)
    L = E.lib()
    assert L.dlrm_embbag_fwd(C.byref(T), 1, 1 << 20, 1 << 20, 1, 1 << 20, None, 1 << 20, 4096, None) == E.ERR_INVALID_ARG
    dims = (C.c_int * 2)(16, 16)
    m = E._abi.dlrm_mlp(1, dims, (C.c_void_p * 1)(1 << 20), (C.c_void_p * 1)(1 << 20), E.E4M3)
    assert L.dlrm_mlp_workspace_size(C.byref(m), 8, E.F32) == 0
    m.dt = E.BF16
    assert L.dlrm_mlp_workspace_size(C.byref(m), 8, E.E4M3) == 0
    assert L.dlrm_mlp_workspace_size(C.byref(m), 8, E.F32) > 0
