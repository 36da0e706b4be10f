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


def test_backward_through_a_call_says_that_there_is_none():
    """Results of inputs that require gradients are no constants: going back through the call raises, where it would
    otherwise have left their share out. Values, and calls that record nothing, are as they were."""
    T, k, H = 4, 2, 128
    g = torch.Generator().manual_seed(0)
    n = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    r, y, gain, w = n(T, H), n(T, H), n(H), n(T, k)
    row_of = torch.arange(T * k, dtype=torch.int32).view(T, k).cuda()
    rows, s = n(T * k, H), torch.ones(T, device="cuda")
    ws = moe.Workspace(moe.block_workspace_bytes(T, k, 8, H))
    calls = {
        "block_norm": (lambda t: moe.block_norm(t[0], t[1], post_gain=t[2], pre_gain=t[2]), [r, y, gain]),
        "block_norm_backward": (lambda t: list(moe.block_norm_backward(t[0], t[1], r, s, y, s, post_gain=gain, pre_gain=gain,
                                                                       ws=ws).values()), [r, y]),
        "dispatch": (lambda t: [moe.dispatch(t[0], row_of)], [r]),
        "collect": (lambda t: [moe.collect(t[0], row_of, t[1], t[2])], [rows, w, r]),
        "collect_backward": (lambda t: moe.collect_backward(t[0], t[1], row_of, t[2]), [r, rows, w]),
    }
    for name, (call, args) in calls.items():
        want = [t for t in call(args) if t is not None]
        assert not any(t.requires_grad for t in want)
        for i in range(len(args)):
            asked = [t.clone().requires_grad_(j == i) for j, t in enumerate(args)]
            out = [t for t in call(asked) if t is not None]
            assert all(torch.equal(a, b) for a, b in zip(want, out))
            for t in out:
                assert t.requires_grad
                with pytest.raises(RuntimeError, match=name):
                    t.sum().backward()
            assert asked[i].grad is None
            with torch.no_grad():
                assert not any(t.requires_grad for t in call(asked) if t is not None)
    # what is not differentiable by its type stays so
    q = moe.mx4_quantize(r.clone().requires_grad_())
    assert not q.codes.requires_grad and not q.scales.requires_grad


def test_written_buffers_of_calls_that_record():
    x = torch.randn(4, 128, device="cuda")
    row_of = torch.arange(8, dtype=torch.int32, device="cuda").view(4, 2)
    leaf = x.clone().requires_grad_()
    with pytest.raises(RuntimeError, match="leaf"):  # as torch refuses it of its own operators
        moe.block_norm(leaf, r_out=leaf)
    assert torch.equal(leaf, x)
    stream = leaf * 1.0
    want = moe.block_norm(x)
    out = moe.block_norm(stream, r_out=stream)
    assert out[0] is stream and torch.equal(out[1], want[1])
    with pytest.raises(RuntimeError, match="block_norm"):
        stream.sum().backward()
    rows = torch.zeros(8, 128, device="cuda")
    assert moe.dispatch(leaf, row_of, None, rows) is rows and rows.requires_grad
    with pytest.raises(RuntimeError, match="dispatch"):
        rows.sum().backward()


def test_an_autograd_function_over_the_entry_points():
    """How gradients are had: a torch.autograd.Function that calls an operator and its backward entry point."""
    class Norm(torch.autograd.Function):
        @staticmethod
        def forward(ctx, r, y, post, pre):
            r2, u, ry, ru = moe.block_norm(r, y, post_gain=post, pre_gain=pre, u_dtype=F32)
            ctx.save_for_backward(r2, ru, y, ry, post, pre)
            return r2, u

        @staticmethod
        def backward(ctx, dr, du):
            r2, ru, y, ry, post, pre = ctx.saved_tensors
            ws = moe.Workspace(moe.block_workspace_bytes(r2.shape[0], H=r2.shape[1]))
            d = moe.block_norm_backward(dr.contiguous(), du.contiguous(), r2, ru, y, ry, post_gain=post, pre_gain=pre, ws=ws)
            return d["dr"], d["dy"], d["d_post_gain"], d["d_pre_gain"]

    g = torch.Generator().manual_seed(4)
    leaves = [torch.randn(*s, generator=g) for s in ((6, 192), (6, 192), (192,), (192,))]
    here = [t.cuda().requires_grad_() for t in leaves]
    r2, u = Norm.apply(*here)
    (r2.square().sum() + u.sin().sum()).backward()
    there = [t.double().requires_grad_() for t in leaves]
    R, Y, P, Q = there
    rms = lambda v: v / (v.square().mean(1, keepdim=True) + 1e-6).sqrt()  # noqa: E731
    r64 = R + P * rms(Y)
    (r64.square().sum() + (Q * rms(r64)).sin().sum()).backward()
    for a, b in zip(here, there):
        # sums of up to 192 + 6 terms of fp32 values; 2^-24 a step, the terms bounded by the result's own norm
        assert float((a.grad.cpu().double() - b.grad).norm()) <= 1024 * 2.0 ** -24 * float(b.grad.norm())
