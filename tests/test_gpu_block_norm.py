"""The norms around a block and their gradient against the formulas in fp64 (tests/block_ref.py).

Bounds: the kernels' reductions add 8 values a thread and then at most 10 + 5 levels, so a mean is off by at
most 24 u32 of its magnitudes; elementwise steps add one u32 each. 64 u32 of the magnitudes that a result is
summed from cover them with the statistics' share, and a sum over T rows adds T u32.
"""
import pytest
import torch

import quantized_expert_ffn_gemm_b200 as moe
from tests import block_ref as ref
from tests.block_ref import U32, close, rounded

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
SIZES = [(1, 64), (1, 2048), (3, 192), (7, 256), (9, 320), (5, 576), (33, 1088), (300, 2048), (2, 2112), (5, 4096),
         (3, 4160), (2, 8192), (2, 8256), (1, 16384)]


def inputs(T, H, r=F32, y=F32, u=BF16, gate="channel", seed=0):
    g = torch.Generator().manual_seed(seed + T * 31 + H)
    n = lambda *s, t=F32, m=1.0: (torch.randn(*s, generator=g) * m).to(t)  # noqa: E731
    d = dict(r=n(T, H, t=r, m=2.0), y=n(T, H, t=y, m=0.5), post_gain=1 + n(H, m=0.2), pre_gain=1 + n(H, m=0.2), gate=None,
             dr_out=n(T, H, t=r), du=n(T, H, t=u))
    if gate == "channel":
        d["gate"] = n(H)
    elif gate == "token":
        d["gate"] = n(T, 1)
    return d


def dev(d):
    return {k: None if v is None else v.cuda() for k, v in d.items()}


def f64(t):
    return None if t is None else t.double()


def check_forward(d, res_scale, eps, post_norm, u_type, got):
    r2, u, rstd_y, rstd_u = got
    R, U, RY, RU, mag = ref.block_norm(f64(d["r"]), f64(d.get("y")), f64(d.get("post_gain")), f64(d.get("gate")),
                                       res_scale, f64(d.get("pre_gain")), eps, post_norm)
    close(r2, R, 64 * U32 * mag + rounded(R, r2.dtype), "r'")
    if u is not None:
        assert u.dtype == u_type
        g = 1.0 if d.get("pre_gain") is None else f64(d["pre_gain"]).abs()
        # an error of r' moves u directly and through the mean (at most as much again)
        rel = (mag.norm(dim=1, keepdim=True) / R.norm(dim=1, keepdim=True).clamp(min=1e-300)).clamp(max=1e6)
        close(u, U, 64 * U32 * (g * RU * mag + U.abs() * rel) + rounded(U, u.dtype), "u")
        close(rstd_u, RU[:, 0], 64 * U32 * RU[:, 0] * rel[:, 0], "rstd_u")
    if rstd_y is not None:
        close(rstd_y, RY[:, 0], 24 * U32 * RY[:, 0], "rstd_y")


@pytest.mark.parametrize("T,H", SIZES)
def test_forward(T, H):
    d = inputs(T, H)
    c = dev(d)
    got = moe.block_norm(c["r"], c["y"], post_gain=c["post_gain"], gate=c["gate"], res_scale=0.5, pre_gain=c["pre_gain"])
    check_forward(d, 0.5, 1e-6, True, BF16, got)


@pytest.mark.parametrize("r", [F32, F16, BF16])
@pytest.mark.parametrize("y,u", [(F32, F16), (F16, BF16), (BF16, F32)])
@pytest.mark.parametrize("gate", ["none", "channel", "token"])
def test_forward_types(r, y, u, gate):
    d = inputs(13, 704, r, y, u, gate)
    c = dev(d)
    got = moe.block_norm(c["r"], c["y"], post_gain=c["post_gain"], gate=c["gate"], res_scale=1.25, u_dtype=u, eps=1e-3)
    d["pre_gain"] = None
    check_forward(d, 1.25, 1e-3, True, u, got)


def test_forward_halves_left_out():
    d = inputs(6, 320)
    c = dev(d)
    only_pre = moe.block_norm(c["r"], pre_gain=c["pre_gain"])
    assert only_pre[2] is None and torch.equal(only_pre[0], c["r"])
    check_forward({"r": d["r"], "pre_gain": d["pre_gain"]}, 1.0, 1e-6, True, BF16, only_pre)
    only_post = moe.block_norm(c["r"], c["y"], post_gain=c["post_gain"], gate=c["gate"], pre_norm=False)
    assert only_post[1] is None and only_post[3] is None
    check_forward({**d, "pre_gain": None}, 1.0, 1e-6, True, BF16, only_post)
    no_norm = moe.block_norm(c["r"], c["y"], gate=c["gate"], post_norm=False, res_scale=-2.0)
    assert no_norm[2] is None
    check_forward({**d, "post_gain": None, "pre_gain": None}, -2.0, 1e-6, False, BF16, no_norm)


def test_forward_in_place_and_agreement_with_rmsnorm():
    d = inputs(40, 2048)
    c = dev(d)
    apart = moe.block_norm(c["r"], c["y"], gate=c["gate"])
    r = c["r"].clone()
    same = moe.block_norm(r, c["y"], gate=c["gate"], r_out=r)
    assert same[0] is r and all(torch.equal(a, b) for a, b in zip(apart, same))
    # opening a block alone is the library's RMSNorm (each is within half a bf16 step and a few fp32 ones)
    u = moe.block_norm(c["r"])[1]
    base = moe.rmsnorm_bf16(c["r"])
    assert float((u.double() - base.double()).abs().max()) <= 2 * 2.0 ** -8 * float(base.abs().max())
    assert float((u != base).double().mean()) < 1e-3


def test_rows_of_zeros_infinities_and_nan():
    r = torch.zeros(4, 128)
    y = torch.zeros(4, 128)
    y[1, 5], r[2, 7], y[3, 0] = float("inf"), float("nan"), 1e-30
    got = moe.block_norm(r.cuda(), y.cuda(), eps=1e-6)
    assert bool((got[0][0] == 0).all()) and bool((got[1][0] == 0).all())   # eps keeps an empty row at zero
    assert bool(got[0][1].isnan().any()) and bool(got[1][2].isnan().all())  # inf / inf, NaN through the mean
    close(got[0][3], ref.block_norm(f64(r), f64(y))[0][3], 0 * r[3].double() + 1e-30, "tiny")


def run_backward(c, res_scale, post_norm=True, seed=0, **drop):
    c = {**c, **drop}
    T, H = c["r"].shape
    ws = moe.Workspace(moe.block_workspace_bytes(T, H=H))
    ry = (c["y"].float().square().mean(1) + 1e-6).rsqrt() if c["y"] is not None and post_norm else None
    ru = (c["r"].float().square().mean(1) + 1e-6).rsqrt() if c["du"] is not None else None
    got = moe.block_norm_backward(c["dr_out"], c["du"], c["r"], ru, c["y"], ry, post_gain=c["post_gain"], gate=c["gate"],
                                  res_scale=res_scale, pre_gain=c["pre_gain"], post_norm=post_norm, ws=ws)
    h = {k: None if v is None else v.cpu().double() for k, v in c.items()}
    want, mag = ref.block_norm_grad(h["dr_out"], h["du"], h["r"], None if ru is None else ru.cpu().double(), h["y"],
                                    None if ry is None else ry.cpu().double(), h["post_gain"], h["gate"], res_scale,
                                    h["pre_gain"], post_norm)
    for n, v in got.items():
        if v is None:
            continue
        extra = T if v.dim() == 1 else 0
        close(v, want[n], (128 + extra) * U32 * mag[n] + rounded(want[n], v.dtype), n)
    return got


@pytest.mark.parametrize("T,H", SIZES + [(1000, 64), (700, 2048)])
def test_backward(T, H):
    run_backward(dev(inputs(T, H)), 0.5)


@pytest.mark.parametrize("r", [F32, F16, BF16])
@pytest.mark.parametrize("y,u", [(F32, F16), (F16, BF16), (BF16, F32)])
@pytest.mark.parametrize("gate", ["none", "channel", "token"])
def test_backward_types(r, y, u, gate):
    run_backward(dev(inputs(21, 448, r, y, u, gate)), 1.5)


@pytest.mark.parametrize("y,u", [(F32, F32), (F32, BF16), (BF16, BF16)])
def test_backward_longest_rows(y, u):
    """Rows of up to 256 KB: through shared memory where they fit, else read again from memory."""
    run_backward(dev(inputs(3, 16384, y=y, u=u)), 0.5)
    run_backward(dev(inputs(5, 4160, BF16, y, u, "token")), 1.5)


@pytest.mark.parametrize("H", [192, 4160])
def test_backward_parts_left_out(H):
    c = dev(inputs(11, H, gate="token"))
    got = run_backward(c, 1.0, y=None, post_gain=None, gate=None)
    assert got["dy"] is None and got["d_gate"] is None
    run_backward(c, 1.0, du=None, pre_gain=None)
    run_backward(c, 1.0, dr_out=None)
    run_backward(c, 1.0, post_norm=False)
    run_backward(c, 1.0, post_norm=False, post_gain=None, gate=None)


def test_backward_of_no_tokens_is_zero():
    c = dev(inputs(0, 128))
    ws = moe.Workspace(moe.block_workspace_bytes(1, H=128))
    z = torch.empty(0, device="cuda")
    got = moe.block_norm_backward(c["dr_out"], c["du"], c["r"], z, c["y"], z, post_gain=c["post_gain"], gate=c["gate"],
                                  pre_gain=c["pre_gain"], ws=ws)
    assert all(bool((got[n] == 0).all()) for n in ("d_post_gain", "d_gate", "d_pre_gain"))
    assert moe.block_norm(c["r"], c["y"])[1].shape == (0, 128)


@pytest.mark.parametrize("gate", ["channel", "token"])
def test_gradient_against_differences(gate):
    """The forward formula in fp64, moved along random directions: the slope is the gradient's product."""
    T, H = 6, 192
    d = inputs(T, H, gate=gate, seed=5)
    c = dev(d)
    r2, u, ry, ru = moe.block_norm(c["r"], c["y"], post_gain=c["post_gain"], gate=c["gate"], res_scale=0.75,
                                   pre_gain=c["pre_gain"], u_dtype=F32)
    ws = moe.Workspace(moe.block_workspace_bytes(T, H=H))
    dr_out, du = c["dr_out"], c["du"].float()
    got = moe.block_norm_backward(dr_out, du, r2, ru, c["y"], ry, post_gain=c["post_gain"], gate=c["gate"], res_scale=0.75,
                                  pre_gain=c["pre_gain"], ws=ws)
    h = {k: v.double() for k, v in d.items()}

    def loss(**move):
        x = {k: h[k] + move.get(k, 0) for k in ("r", "y", "post_gain", "gate", "pre_gain")}
        R, U, _, _, _ = ref.block_norm(x["r"], x["y"], x["post_gain"], x["gate"], 0.75, x["pre_gain"])
        return float((R * h["dr_out"]).sum() + (U * du.cpu().double()).sum())

    g = torch.Generator().manual_seed(9)
    for arg, name in (("r", "dr"), ("y", "dy"), ("post_gain", "d_post_gain"), ("gate", "d_gate"),
                      ("pre_gain", "d_pre_gain")):
        way = torch.randn(h[arg].shape, generator=g, dtype=torch.float64)
        step = 1e-5
        slope = (loss(**{arg: step * way}) - loss(**{arg: -step * way})) / (2 * step)
        prod = float((got[name].cpu().double() * way).sum())
        # fp32 gradients: 2^-24 a term with the bounds above; central differences: step^2 and 2^-53 / step
        size = float((got[name].cpu().double() * way).abs().sum()) + abs(slope) + 1.0
        assert abs(slope - prod) <= (300 * U32 + 1e-7) * 4 * size, (arg, slope, prod)


def test_same_result_every_run_on_another_stream_and_in_a_graph():
    c = dev(inputs(500, 1024))
    ws = moe.Workspace(moe.block_workspace_bytes(500, H=1024))

    def step():
        r2, u, ry, ru = moe.block_norm(c["r"], c["y"], post_gain=c["post_gain"], gate=c["gate"], pre_gain=c["pre_gain"])
        g = moe.block_norm_backward(c["dr_out"], u, r2, ru, c["y"], ry, post_gain=c["post_gain"], gate=c["gate"],
                                    pre_gain=c["pre_gain"], ws=ws)
        return [r2, u, ry, ru] + list(g.values())

    first = step()
    assert all(torch.equal(a, b) for a, b in zip(first, step()))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        there = step()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(first, there))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    c["y"].mul_(0.5)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(held, step()))
    assert not torch.equal(held[0], first[0])
