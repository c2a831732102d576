"""How much scratch the linear calls ask for."""
import pytest
import torch

import fsdp_sharded_state_gb300 as fs


@pytest.mark.parametrize("rows", [1, 2, 4])
def test_workspace_of_a_few_fp32_rows_leaves_the_weight_out(rows):
    # neither forward nor dgrad of one to four fp32 rows splits the weight: room for the terms of
    # both rows' operands (wgrad's), each row padded to 64 elements, each operand to 256 bytes
    n = fs.fsdp_linear_workspace_bytes(rows, 4096, 11008, torch.float32)
    assert 6 * rows * (4096 + 11008) <= n <= 6 * rows * (4096 + 11008) + 2 * 256
    # bf16 dgrad copies an unaligned weight
    assert fs.fsdp_linear_workspace_bytes(rows, 4096, 11008, torch.bfloat16, False) >= 2 * 4096 * 11008


@pytest.mark.parametrize("rows,cols_in,cols_out", [(1 << 30, 1 << 30, 1), (1, (1 << 31) - 2048, (1 << 31) - 2048), (1 << 21, 1, 1 << 20),
                                                   ((1 << 31) - 2048,) * 3])
def test_matrices_past_the_counted_sizes_are_refused(rows, cols_in, cols_out):
    """Matrices of more than 2^40 elements: the bytes of their copies do not fit 64 bits either.
    The calls get no pointers, so that none is launched whatever the answer."""
    L = fs.lib()
    for dtype in (fs.FSDP_F32, fs.FSDP_BF16):
        assert L.fsdp_linear_workspace_bytes(rows, cols_in, cols_out, dtype, 0) == 0
        n = (rows, cols_in, cols_out, dtype)
        assert L.fsdp_linear_forward(*n, None, cols_in, None, cols_in, None, 0, None, None, 0, None, cols_out, None, 0, None, 0, None) == -5
        assert L.fsdp_linear_dgrad(*n, None, cols_out, None, cols_in, 0, None, 0, None, None, 0, None, cols_in, None, 0, None) == -5
        assert L.fsdp_linear_wgrad(*n, None, cols_out, None, cols_in, None, cols_in, None, 0, 0, None, 0, None) == -5
    assert L.fsdp_linear_workspace_bytes(1 << 20, 1 << 20, 1, fs.FSDP_F32, 0) > 0
