"""The block operators among torch's own: memory a refused call may not take, buffers that are written, inputs that
require gradients."""
import pytest
import torch

import quantized_expert_ffn_gemm_b200 as moe

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


def test_numbers_of_experts_out_of_range_take_no_memory():
    idx = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    ws = moe.Workspace(moe.block_workspace_bytes(4, 2, 8))
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    held = torch.cuda.memory_allocated()
    for E in (0, 1, 4097, 1 << 20, (1 << 31) - 1):  # 1: fewer than two slots need
        with pytest.raises(moe.MoeError) as e:
            moe.sort_pairs(idx, E, ws)
        assert e.value.code == moe.MOE_ERR_INVALID_ARG
    assert torch.cuda.max_memory_allocated() == held
    for E in (-1, 1 << 31):
        with pytest.raises(ValueError, match="E"):
            moe.sort_pairs(idx, E, ws)
