"""MXFP4 rows and their product per expert against fp64 (tests/block_ref.py, which states the bounds).

Codes and scale bytes are equal bit for bit; reading back is exact."""
import ctypes
import math

import pytest
import torch

import quantized_expert_ffn_gemm_b200 as moe
from quantized_expert_ffn_gemm_b200.block import Mx4Mat
from tests import block_ref as ref
from tests.block_ref import close, rounded

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


def check_quantize(x):
    q = moe.mx4_quantize(x.cuda())
    code, byte = ref.mx4_quantize(x.double())
    assert torch.equal(q.scales.cpu(), byte)
    assert torch.equal(q.codes.cpu(), ref.pack(code))
    for t in (F32, BF16):
        got = moe.mx4_dequantize(q, t).cpu().double()
        assert torch.equal(got.nan_to_num(7777.0), ref.mx4_value(code, byte).nan_to_num(7777.0))
    return q


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("T,K", [(1, 64), (3, 2048), (65, 192), (7, 16384), (300, 320)])
def test_quantize(T, K, dtype):
    g = torch.Generator().manual_seed(T + K)
    check_quantize((torch.randn(T, K, generator=g) * torch.exp(2 * torch.randn(T, 1, generator=g))).to(dtype))


def test_quantize_borders():
    """Every border between two codes, one fp32 step to either side of it, both signs, at many scales."""
    mid = torch.tensor([0, 0.25, 0.5, 0.75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 6, 7, 7.999])
    near = torch.cat([mid, torch.nextafter(mid, torch.tensor(100.0)), torch.nextafter(mid, torch.tensor(0.0))])
    near = torch.cat([near, -near])
    blocks = []
    for e in (-127, -126, -100, -20, -1, 0, 1, 30, 100, 124):
        for top in (4.0, 5.0, 7.9999):
            for s in range(0, near.numel(), 31):
                v = torch.zeros(32)
                part = near[s:s + 31]
                v[:part.numel()] = part
                v[31] = top
                blocks.append(torch.ldexp(v.double(), torch.tensor(e)).float())
    n = len(blocks) // 2 * 2
    check_quantize(torch.stack(blocks[:n]).view(-1, 64))


def test_quantize_zeros_subnormals_infinities_and_nan():
    x = torch.zeros(8, 64)
    x[1, 3] = 1e-45
    x[2, :32] = 3e-39
    x[3, 5] = float("inf")
    x[4, 40] = float("nan")
    x[5, 0], x[5, 1] = -0.0, -1e-3
    x[6, 0], x[6, 33] = torch.finfo(F32).max, -torch.finfo(F32).max
    q = check_quantize(x)
    assert q.scales[3].tolist() == [255, 0] and q.scales[4].tolist() == [0, 255]


def test_quantize_to_sorted_rows():
    T, k, E, K = 50, 5, 12, 192
    g = torch.Generator().manual_seed(2)
    idx = torch.rand(T, E, generator=g).topk(k, 1).indices.to(torch.int32)
    idx[::7] = -1
    plan = moe.sort_pairs(idx.cuda(), E, moe.Workspace(moe.block_workspace_bytes(T, k, E)))
    x = torch.randn(T, K, generator=g).to(BF16).cuda()
    whole = moe.mx4_quantize(moe.dispatch(x, plan["row_of"], plan["offsets"]))
    each = moe.mx4_quantize(x, plan["row_of"], plan["offsets"])
    assert torch.equal(whole.codes, each.codes) and torch.equal(whole.scales, each.scales)
    left = moe.mx4_quantize(x, plan["row_of"])
    kept = int(plan["offsets"][-1])
    assert torch.equal(left.codes[:kept], whole.codes[:kept]) and torch.equal(left.scales[:kept], whole.scales[:kept])


def rows_and_weights(sizes, K, N, up, seed=0, spread=0.0):
    g = torch.Generator().manual_seed(seed + K + N + len(sizes))
    R, E = sum(sizes), len(sizes)
    scale = torch.exp(spread * torch.randn(R, 1, generator=g))
    a = moe.mx4_quantize((torch.randn(R, K, generator=g) * scale).to(BF16).cuda())
    w = moe.mx4_quantize((torch.randn(E, N, K, generator=g) * K ** -0.5).cuda())
    u = moe.mx4_quantize((torch.randn(E, N, K, generator=g) * K ** -0.5).cuda()) if up else None
    offsets = torch.tensor([0] + list(torch.tensor(sizes).cumsum(0)), dtype=torch.int32)
    return a, w, u, offsets


def check_product(sizes, K, N, up, dtype, tail=0, **more):
    a, w, u, offsets = rows_and_weights(list(sizes) + ([tail] if tail else []), K, N, up, **more)
    if tail:  # rows behind the last group: the last expert's are cut off
        offsets, w = offsets[:-1].contiguous(), moe.Mx4(w.codes[:-1].contiguous(), w.scales[:-1].contiguous())
        u = None if u is None else moe.Mx4(u.codes[:-1].contiguous(), u.scales[:-1].contiguous())
    ws = moe.Workspace(256)
    got = moe.mx4_product(a, w, offsets.cuda(), up=u, dtype=dtype, ws=ws)
    want, err = ref.mx4_product(ref.mx4_values(a), ref.mx4_values(w), offsets, None if u is None else ref.mx4_values(u))
    close(got, want, err + rounded(want, dtype), "out")
    if tail:
        assert bool((got[-tail:] == 0).all())
    assert moe.read_device_error(ws) == 0
    return got


@pytest.mark.parametrize("up", [False, True])
@pytest.mark.parametrize("K,N", [(64, 64), (192, 64), (256, 128), (320, 192), (512, 320), (2048, 512), (576, 1088)])
def test_product_sizes(K, N, up):
    check_product([3, 0, 130, 1, 17], K, N, up, BF16)


@pytest.mark.parametrize("up", [False, True])
@pytest.mark.parametrize("sizes", [[1], [0, 1], [1, 0, 0], [8, 16, 32, 64], [127, 128, 129], [255, 256, 257], [15, 1, 33, 0, 500], [192, 193, 191],
                                   [97, 96, 95, 1, 0], [385, 577, 15], [300, 0, 0, 0, 10], [80, 81], [176, 1, 353],
                                   [0, 0, 0]])
def test_product_groups(sizes, up):
    if sum(sizes):
        check_product(sizes, 256, 128, up, F16)
    else:
        check_product(sizes, 256, 128, up, F16, tail=5)


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_product_one_group_without_offsets_and_rows_behind(dtype):
    a, w, _, offsets = rows_and_weights([77], 512, 192, False)
    ws = moe.Workspace(256)
    got = moe.mx4_product(a, w, dtype=dtype, ws=ws)
    assert torch.equal(got, moe.mx4_product(a, w, offsets.cuda(), dtype=dtype, ws=ws))
    check_product([40, 0, 9], 512, 192, True, dtype, tail=23)
    check_product([200], 512, 192, False, dtype, tail=150)


def test_product_wide_ranges_of_scales():
    check_product([90, 40], 1024, 128, False, BF16, spread=3.0)


def test_product_long_rows_and_many_experts():
    check_product([2, 5], 16384, 64, False, BF16)
    check_product([1, 0, 0, 2] * 150, 128, 64, True, F16)
    check_product([0, 1] * 2048, 64, 64, False, F16)


def test_product_of_a_nan_block_is_nan_in_its_rows_alone():
    K, N = 256, 128
    g = torch.Generator().manual_seed(0)
    x = torch.randn(40, K, generator=g)
    x[17, 99] = float("inf")
    a, w = moe.mx4_quantize(x.cuda()), moe.mx4_quantize(torch.randn(1, N, K, generator=g).cuda())
    out = moe.mx4_product(a, w, dtype=BF16, ws=moe.Workspace(256))
    assert bool(out[17].isnan().all()) and bool(out[:17].isfinite().all()) and bool(out[18:].isfinite().all())


def test_product_single_tokens_equal_their_batch():
    """Each row's sum runs over K alone, so a row of a large group and the same row alone are bit-identical."""
    a, w, u, _ = rows_and_weights([260], 512, 256, True)
    ws = moe.Workspace(256)
    whole = moe.mx4_product(a, w, up=u, ws=ws)
    for i in (0, 100, 259):
        one = moe.Mx4(a.codes[i:i + 1].clone(), a.scales[i:i + 1].clone())
        assert torch.equal(moe.mx4_product(one, w, up=u, ws=ws)[0], whole[i])


def test_product_on_a_stream_and_in_a_graph():
    a, w, u, offsets = rows_and_weights([33, 0, 150, 4], 512, 256, True)
    off, ws = offsets.cuda(), moe.Workspace(256)
    first = moe.mx4_product(a, w, off, up=u, ws=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        there = moe.mx4_product(a, w, off, up=u, ws=ws)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(first, there)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = moe.mx4_product(a, w, off, up=u, ws=ws)
    off.copy_(torch.tensor([0, 10, 100, 120, 187], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(held, moe.mx4_product(a, w, off, up=u, ws=ws)) and not torch.equal(held, first)


@pytest.mark.parametrize("up", [False, True])
@pytest.mark.parametrize("groups,K,N", [(80, 2048, 576), (48, 2112, 320), (80, 320, 1088), (80, 768, 576), (48, 512, 512), (48, 128, 704)])
def test_product_many_tiles(groups, K, N, up):
    """Several tiles a block, of every tile width, full and partial rows and columns."""
    check_product([(37 * i) % 200 for i in range(groups)], K, N, up, BF16)


def test_product_flags_offsets_that_are_no_offsets():
    """Offsets that run back or past the rows are clamped to them and flagged; nothing outside is touched."""
    a, w, _, offsets = rows_and_weights([30, 20, 14], 256, 64, False)
    ws = moe.Workspace(256)
    good = moe.mx4_product(a, w, offsets.cuda(), ws=ws)
    for bad in ([0, 30, 20, 64], [0, 30, 50, 100], [-5, 30, 50, 64], [3, 30, 50, 64]):
        moe.mx4_product(a, w, torch.tensor(bad, dtype=torch.int32, device="cuda"), ws=ws)
        assert moe.read_device_error(ws) == moe.MOE_ERR_DEVICE_CHECK, bad
    assert torch.equal(good, moe.mx4_product(a, w, offsets.cuda(), ws=ws)) and moe.read_device_error(ws) == 0


def block_values(*values):
    """A row of 32 values a block, all but the first zero."""
    x = torch.zeros(1, 32 * len(values))
    x[0, ::32] = torch.tensor(values)
    return x


@pytest.mark.parametrize("rows", [1, 40, 200])
def test_product_flags_results_beyond_fp16(rows):
    """A sum that rounds to an fp16 infinity is recorded, the largest that rounds to 65504 is not; bf16 holds both."""
    ws = moe.Workspace(256)
    one = moe.mx4_quantize(block_values(1.0, 1.0, 1.0, 1.0).expand(64, -1).contiguous()[None].cuda())
    for parts, flagged in (((65536.0, -32.0, 0, 0), False), ((65536.0, -16.0, -1.0, 0), False),
                           ((65536.0, -16.0, 0, 0), True), ((-65536.0, 0, 0, 0), True), ((98304.0, 0, 0, 0), True)):
        x = torch.zeros(rows, 128)
        x[rows // 2] = block_values(*parts)
        a = moe.mx4_quantize(x.cuda())
        for dtype, bad in ((F16, flagged), (BF16, False)):
            out = moe.mx4_product(a, one, dtype=dtype, ws=ws)
            assert torch.equal(out[rows // 2].cpu(), torch.full((64,), sum(parts)).to(dtype))
            assert moe.read_device_error(ws) == (moe.MOE_ERR_RANGE if bad else moe.MOE_OK), (parts, dtype)
    # gate and up: 512 * 512
    a = moe.mx4_quantize(block_values(512.0, 0).expand(rows, -1).contiguous().cuda())
    w = moe.mx4_quantize(block_values(1.0, 0).expand(64, -1).contiguous()[None].cuda())
    for dtype, bad in ((F16, moe.MOE_ERR_RANGE), (BF16, moe.MOE_OK)):
        moe.mx4_product(a, w, up=w, dtype=dtype, ws=ws)
        assert moe.read_device_error(ws) == bad


def test_product_flags_nothing_but_results():
    """Rows of other groups beside a tile's own are multiplied with it and no result: they are not flagged. Nor is NaN."""
    ws = moe.Workspace(256)
    a = moe.mx4_quantize(torch.cat([block_values(1.0, 0), block_values(32768.0, 0), block_values(float("nan"), 0)]).cuda())
    w = moe.mx4_quantize(torch.stack([block_values(32768.0, 0).expand(64, -1), block_values(1.0, 0).expand(64, -1)]).cuda())
    off = torch.tensor([0, 1, 3], dtype=torch.int32).cuda()
    out = moe.mx4_product(a, w, off, ws=ws)
    assert bool((out[:2] == 32768).all()) and bool(out[2].isnan().all()) and moe.read_device_error(ws) == moe.MOE_OK


@pytest.mark.parametrize("up", [False, True])
def test_product_with_bad_offsets_stays_in_its_rows(up):
    """Whatever the offsets hold, nothing before or behind out is written."""
    n, K, N = 64, 256, 64
    a, w, u, _ = rows_and_weights([30, 20, 14], K, N, up)
    ws = moe.Workspace(256)
    guard = 256
    buf = torch.empty(n + 2 * guard, N, dtype=F16, device="cuda")
    mats = [None if q is None else Mx4Mat(3, N, K, q.codes.data_ptr(), q.scales.data_ptr()) for q in (w, u)]
    ref_of = [None if m is None else ctypes.addressof(m) for m in mats]
    for bad in ([0, 30, 20, 64], [0, 30, 50, 100], [-5, 30, 50, 64], [3, 30, 50, 64], [0, 64, 0, 64],
                [2 ** 31 - 1, -2 ** 31, 5, -1], [0, 0, 0, 2 ** 31 - 1], [-1, -1, -1, -1]):
        buf.fill_(7.0)
        off = torch.tensor(bad, dtype=torch.int32, device="cuda")
        assert moe.lib().moe_mx4_product(a.codes.data_ptr(), a.scales.data_ptr(), n, off.data_ptr(), 3, ref_of[0], ref_of[1],
                                         buf[guard].data_ptr(), moe.F16, ws.buf.data_ptr(), ws.nbytes,
                                         torch.cuda.current_stream().cuda_stream) == 0
        assert moe.read_device_error(ws) == moe.MOE_ERR_DEVICE_CHECK, bad
        assert bool((buf[:guard] == 7).all()) and bool((buf[guard + n:] == 7).all()), bad


@pytest.mark.parametrize("gate", [-64.0, -84.0, -86.0, -88.0, -92.0, -96.0, -0.5, 0.0, 2.0, 88.0, 96.0, 192.0])
def test_silu_of_gates_far_from_zero(gate):
    """silu(gate) up with exact gates and an up that brings the product back into bf16's middle range. CUDA's fast exp is good to
    2 + 1.16 |x| steps of its fp32 result (2^-149 each where that is subnormal), its fast division to 2; two products."""
    big = 2.0 ** 100 if gate < 0 else 1.0
    parts = [math.copysign(p, gate) for p in (64.0, 32.0, 16.0, 8.0, 4.0, 2.0, 0.5) if int(2 * abs(gate)) & int(2 * p)]
    if abs(gate) >= 128:
        parts.append(math.copysign(128.0, gate))
    parts = (parts + [0.0] * 6)[:6]
    assert sum(parts) == gate
    a = moe.mx4_quantize(torch.cat([block_values(*[1.0] * 6)] * 3).cuda())
    w = moe.mx4_quantize(block_values(*parts).expand(64, -1).contiguous()[None].cuda())
    u = moe.mx4_quantize(block_values(big, 0, 0, 0, 0, 0).expand(64, -1).contiguous()[None].cuda())
    ws = moe.Workspace(256)
    got = moe.mx4_product(a, w, up=u, dtype=BF16, ws=ws)
    want = torch.full((3, 64), gate / (1 + math.exp(-gate)) * big, dtype=torch.float64)
    rel = (2 + 1.16 * abs(gate) + 4) * max(2.0 ** -23, 2.0 ** -149 / math.exp(-abs(gate)) if gate < 0 else 0)
    close(got, want, rel * want.abs() + rounded(want, BF16), "silu")
