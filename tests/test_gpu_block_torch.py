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


@pytest.mark.parametrize("H", [128, 4160])
def test_backward_of_a_gain_that_no_gradient_reaches(H):
    """du None: nothing reaches u. pre_gain's gradient is zero, the others are those of a call without pre_gain."""
    T = 5
    g = torch.Generator().manual_seed(H)
    n = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    r, y, dr, gain, gate = n(T, H), n(T, H), n(T, H), n(H), n(H)
    ry = y.square().mean(1).rsqrt()
    ws = moe.Workspace(moe.block_workspace_bytes(T, H=H))
    args = dict(post_gain=gain, gate=gate, ws=ws)
    want = moe.block_norm_backward(dr, None, r, None, y, ry, **args)
    got = moe.block_norm_backward(dr, None, r, None, y, ry, pre_gain=gain, **args)
    assert want["d_pre_gain"] is None and got["d_pre_gain"].shape == (H,) and bool((got["d_pre_gain"] == 0).all())
    assert all(torch.equal(got[m], want[m]) for m in ("dr", "dy", "d_post_gain", "d_gate"))
    none = moe.block_norm_backward(dr[:0], None, r[:0], None, y[:0], ry[:0], pre_gain=gain, **args)
    assert bool((none["d_pre_gain"] == 0).all())


def test_buffers_that_are_written_count_as_changed():
    """An autograd function that saved r or rows is told that they were written."""
    x = torch.randn(4, 128, device="cuda")
    row_of = torch.arange(8, dtype=torch.int32, device="cuda").view(4, 2)
    rows = torch.zeros(8, 128, device="cuda")
    before = (x._version, rows._version, row_of._version)
    moe.block_norm(x, r_out=x)
    moe.dispatch(x, row_of, None, rows)
    assert (x._version, rows._version, row_of._version) == (before[0] + 1, before[1] + 1, before[2])
    with pytest.raises(moe.MoeError):  # refused: nothing was written
        moe.block_norm(x, r_out=x, eps=-1.0)
    assert x._version == before[0] + 1
    leaf = torch.randn(4, 128, device="cuda", requires_grad=True)
    r = leaf * 1.0
    loss = (r * r).sum()  # saves r
    with torch.no_grad():
        moe.block_norm(r, r_out=r)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    with torch.inference_mode():  # tensors without such a count
        free = torch.randn(4, 128, device="cuda")
        moe.block_norm(free, r_out=free)
    moe.block_norm(free, r_out=free)
