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
