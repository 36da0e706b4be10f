"""The norms on batches long enough that a block works on many rows: rows fetched ahead, ring slots filled again and
again, sums over a block's rows, and a last round that only some blocks take. Formulas and bounds as in
test_gpu_block_norm.py: 64 u32 a row's magnitudes, and T u32 more for a sum over T rows.

148 SMs hold 444 blocks of the forward kernel and 296 of the gradient's for rows of up to 2048 values (256 threads, one to
eight rows side by side), 148 of either above that."""
import pytest
import torch

import quantized_expert_ffn_gemm_b200 as moe
from tests.test_gpu_block_norm import BF16, F16, F32, check_forward, dev, inputs, run_backward

pytestmark = pytest.mark.gpu

LONG = [(3001, 2048), (20011, 192), (2000, 1088), (700, 4096), (450, 4160), (310, 8256)]
TYPES = [(F32, F32, F32, "channel"), (F32, F32, BF16, "token"), (BF16, F16, BF16, "channel"), (F16, BF16, F32, "token")]


@pytest.mark.parametrize("r,y,u,gate", TYPES)
@pytest.mark.parametrize("T,H", LONG)
def test_forward_of_many_rows_a_block(T, H, r, y, u, gate):
    d = inputs(T, H, r, y, u, gate)
    c = dev(d)
    args = dict(post_gain=c["post_gain"], gate=c["gate"], res_scale=0.5, pre_gain=c["pre_gain"], u_dtype=u)
    got = moe.block_norm(c["r"], c["y"], **args)
    check_forward(d, 0.5, 1e-6, True, u, got)
    # in place: each row is read before it is written, whatever is fetched ahead
    same = moe.block_norm(c["r"], c["y"], r_out=c["r"], **args)
    assert same[0] is c["r"] and all(torch.equal(a, b) for a, b in zip(got, same))


@pytest.mark.parametrize("r,y,u,gate", TYPES)
@pytest.mark.parametrize("T,H", LONG)
def test_backward_of_many_rows_a_block(T, H, r, y, u, gate):
    c = dev(inputs(T, H, r, y, u, gate))
    got = run_backward(c, 1.5)
    ws = moe.Workspace(moe.block_workspace_bytes(T, H=H))
    ry, ru = ((c[n].float().square().mean(1) + 1e-6).rsqrt() for n in ("y", "r"))
    again = moe.block_norm_backward(c["dr_out"], c["du"], c["r"], ru, c["y"], ry, post_gain=c["post_gain"], gate=c["gate"],
                                    res_scale=1.5, pre_gain=c["pre_gain"], ws=ws)
    assert all(torch.equal(got[n], again[n]) for n in got)
    # dr in dr_out's place
    code = {F32: 0, F16: 1, BF16: 2}
    p = lambda t: t.data_ptr()  # noqa: E731
    place, dy = c["dr_out"].clone(), torch.empty_like(c["y"])
    assert moe.lib().moe_block_norm_backward(
        p(place), p(c["du"]), code[u], p(c["r"]), code[r], p(ru), p(c["y"]), code[y], p(ry), T, H, 1, p(c["post_gain"]),
        p(c["gate"]), moe.GATE_CHANNEL if gate == "channel" else moe.GATE_TOKEN, 1.5, p(c["pre_gain"]), p(place), p(dy),
        None, None, None, p(ws.buf), ws.nbytes, torch.cuda.current_stream().cuda_stream) == 0
    assert torch.equal(place, got["dr"]) and torch.equal(dy, got["dy"])


@pytest.mark.parametrize("T,H", [(3001, 2048), (450, 4160)])
def test_backward_of_many_rows_with_parts_left_out(T, H):
    c = dev(inputs(T, H, BF16, F16, BF16, "token"))
    run_backward(c, 1.0, y=None, post_gain=None, gate=None)
    run_backward(c, 1.0, du=None, pre_gain=None)
    run_backward(c, 1.0, dr_out=None)
    run_backward(c, 1.0, post_norm=False)
