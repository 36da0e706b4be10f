"""Pairs sorted by expert, dispatched and collected, and their gradients, against plain fp64 loops.

Integers are equal. Bounds: collect adds k products (and a residual) in order, (k + 2) u32 of their
magnitudes; d_w is a sum over H carried by 32 lanes, H/32 + 8 steps; d_rows one product, u32.
"""
import pytest
import torch

import quantized_expert_ffn_gemm_b200 as moe
from tests import block_ref as ref
from tests.block_ref import U32, close, rounded

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


def choices(T, k, E, drop=0.0, seed=0):
    g = torch.Generator().manual_seed(seed * 1000 + T * 7 + k)
    idx = torch.rand(T, E, generator=g).topk(k, 1).indices.to(torch.int32)
    idx[torch.rand(T, k, generator=g) < drop] = -1
    return idx


def space(T, k, E):
    return moe.Workspace(moe.block_workspace_bytes(T, k, E))


def check_sort(idx, E):
    ws = space(*idx.shape, E)
    got = moe.sort_pairs(idx.cuda(), E, ws)
    want = ref.sort_pairs(idx, E)
    for n in want:
        assert torch.equal(got[n].cpu(), want[n]), n
    return got, ws


@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (1, 10, 512), (6, 10, 512), (1, 32, 32), (93, 11, 64), (1023, 1, 3),
                                   (1024, 1, 5), (1025, 1, 5), (512, 2, 2), (205, 10, 512), (341, 3, 16), (700, 8, 4096),
                                   (63, 8, 2050), (64, 8, 2050), (65, 8, 2050), (129, 32, 2048), (2000, 10, 512)])
@pytest.mark.parametrize("drop", [0.0, 0.3])
def test_sort(T, k, E, drop):
    _, ws = check_sort(choices(T, k, E, drop), E)
    assert moe.read_device_error(ws) == 0


@pytest.mark.parametrize("T,k,E", [(14000, 10, 512), (131072, 1, 7), (131073, 1, 40), (9000, 9, 4000), (300000, 3, 64)])
def test_sort_of_long_batches(T, k, E):
    """More chunks than a block adds up itself; against torch's stable sort."""
    g = torch.Generator().manual_seed(T)
    idx = torch.randint(-1, E, (T, k), generator=g, dtype=torch.int32)
    ws = space(T, k, E)
    got = moe.sort_pairs(idx.cuda(), E, ws)
    flat = idx.view(-1).long()
    key, order = torch.where(flat >= 0, flat, E).sort(stable=True)
    kept = int((flat >= 0).sum())
    row_of = torch.full((T * k,), -1, dtype=torch.int32)
    row_of[order[:kept]] = torch.arange(kept, dtype=torch.int32)
    src = torch.full((T * k,), -1, dtype=torch.int32)
    src[:kept] = (order[:kept] // k).to(torch.int32)
    counts = torch.bincount(key, minlength=E + 1)[:E]
    assert torch.equal(got["counts"].cpu().long(), counts) and int(got["offsets"][-1]) == kept
    assert torch.equal(got["offsets"].cpu().long()[1:], counts.cumsum(0))
    assert torch.equal(got["row_of"].cpu().view(-1), row_of) and torch.equal(got["src"].cpu(), src)
    assert moe.read_device_error(ws) == 0


def test_sort_of_extreme_routings():
    check_sort(torch.full((300, 7), -1, dtype=torch.int32), 9)           # every token padded: no row at all
    check_sort(torch.full((300, 7), 8, dtype=torch.int32), 9)            # one expert takes all, the same one in every slot
    check_sort(torch.zeros(5000, 1, dtype=torch.int32), 4096)
    idx = choices(400, 5, 20)
    idx[::3] = -1
    check_sort(idx, 20)
    check_sort(idx.flip(0).contiguous(), 20)


def test_sort_flags_bad_indices_and_drops_them():
    idx = choices(50, 4, 16)
    idx[3, 1], idx[40, 0] = 16, -2
    got, ws = check_sort(idx, 16)
    assert moe.read_device_error(ws) == moe.MOE_ERR_DEVICE_CHECK
    assert int(got["offsets"][-1]) == 198 and moe.read_device_error(ws) == 0


def test_sort_of_no_tokens():
    got = moe.sort_pairs(torch.empty(0, 4, dtype=torch.int32, device="cuda"), 8, space(1, 4, 8))
    assert bool((got["counts"] == 0).all()) and bool((got["offsets"] == 0).all()) and got["src"].numel() == 0


def test_sort_agrees_with_permute():
    T, k, E, H = 600, 10, 512, 64
    idx = choices(T, k, E).cuda()
    ws = moe.Workspace.for_layer(H, E, k, 64, False, T)
    old = moe.permute(idx, E, torch.zeros(T, H, dtype=BF16, device="cuda"), False, ws)
    new = moe.sort_pairs(idx, E, space(T, k, E))
    assert torch.equal(old["counts"][:E], new["counts"]) and torch.equal(old["offsets"][:E + 1], new["offsets"])
    assert torch.equal(old["row_of"], new["row_of"]) and torch.equal(old["src"], new["src"])


CASES = [(1, 1, 1, 64, F32), (1, 10, 512, 2048, BF16), (6, 10, 512, 2048, F16), (77, 3, 16, 320, F32), (33, 32, 40, 1088, BF16),
         (200, 2, 5, 4160, F16), (3, 4, 8, 16384, F32)]


@pytest.mark.parametrize("T,k,E,H,dtype", CASES)
@pytest.mark.parametrize("drop", [0.0, 0.4, 1.0])
def test_out_and_back_and_gradients(T, k, E, H, dtype, drop):
    idx = choices(T, k, E, drop) if drop < 1 else torch.full((T, k), -1, dtype=torch.int32)
    plan = {n: v.cuda() for n, v in ref.sort_pairs(idx, E).items()}
    g = torch.Generator().manual_seed(T + H)
    x = torch.randn(T, H, generator=g).to(dtype)
    row_of, kept = plan["row_of"].cpu(), int(plan["offsets"][-1])
    rows = moe.dispatch(x.cuda(), plan["row_of"], plan["offsets"])
    want = torch.zeros(T * k, H, dtype=dtype)
    src = plan["src"].cpu().long()
    want[:kept] = x[src[:kept]]
    assert torch.equal(rows.cpu(), want)
    # without the offsets the rows behind the last pair stay
    mine = torch.full((T * k, H), 7, dtype=dtype, device="cuda")
    moe.dispatch(x.cuda(), plan["row_of"], rows=mine)
    assert torch.equal(mine[:kept].cpu(), want[:kept]) and bool((mine[kept:] == 7).all())

    back = torch.randn(T * k, H, generator=g).to(dtype)
    back[kept:] = float("nan")  # never read
    w = torch.randn(T, k, generator=g)
    w[idx < 0] = float("inf")   # a dropped pair's weight neither
    res = torch.randn(T, H, generator=g)
    each = ref.spread(row_of, back.double()) * torch.where(row_of >= 0, w, torch.zeros(()))[..., None].double()
    for out, r, ww in ((F32, None, w), (dtype, res, w), (BF16, None, None)):
        got = moe.collect(back.cuda(), plan["row_of"], None if ww is None else w.cuda(), None if r is None else r.cuda(), out)
        e = each if ww is not None else ref.spread(row_of, back.double())
        y = e.sum(1) + (0 if r is None else r.double())
        m = e.abs().sum(1) + (0 if r is None else r.double().abs())
        close(got, y, (k + 2) * U32 * m + rounded(y, out), "y")

    dy = torch.randn(T, H, generator=g).to(BF16)
    d_rows, d_w = moe.collect_backward(dy.cuda(), back.cuda(), plan["row_of"], w.cuda(), plan["offsets"])
    want = torch.zeros(T * k, H, dtype=torch.float64)
    at = row_of[row_of >= 0].long()
    want[at] = (torch.where(row_of >= 0, w, torch.zeros(()))[..., None].double() * dy.double()[:, None])[row_of >= 0]
    close(d_rows, want, U32 * want.abs() + rounded(want, dtype), "d_rows")
    prod = ref.spread(row_of, back.double()) * dy.double()[:, None]
    close(d_w, prod.sum(2), (H / 32 + 8) * U32 * prod.abs().sum(2), "d_w")
    d_rows2, none = moe.collect_backward(dy.cuda(), back.cuda(), plan["row_of"])
    assert none is None and torch.equal(d_rows2[:kept].cpu().float(), dy[src[:kept]].to(dtype).float())


def test_gradients_against_differences():
    """<dy, collect(dispatch(x), w)> moved along x and w; both are linear, so a difference is exact in fp64."""
    T, k, E, H = 20, 4, 8, 128
    idx = choices(T, k, E, 0.2)
    plan = moe.sort_pairs(idx.cuda(), E, space(T, k, E))
    g = torch.Generator().manual_seed(3)
    x, w, dy = torch.randn(T, H, generator=g), torch.randn(T, k, generator=g), torch.randn(T, H, generator=g)
    rows = moe.dispatch(x.cuda(), plan["row_of"], plan["offsets"])
    d_rows, d_w = moe.collect_backward(dy.cuda(), rows, plan["row_of"], w.cuda(), plan["offsets"])
    dx = moe.collect(d_rows, plan["row_of"])
    kept = (idx >= 0).double()

    def loss(x, w):
        return float(((x[:, None] * (w * kept)[..., None]).sum(1) * dy.double()).sum())

    wx, ww = torch.randn(T, H, generator=g).double(), torch.randn(T, k, generator=g).double()
    for slope, grad, way in ((loss(x + wx, w.double()) - loss(x.double(), w.double()), dx, wx),
                             (loss(x.double(), w + ww) - loss(x.double(), w.double()), d_w, ww)):
        terms = grad.cpu().double() * way
        assert abs(slope - float(terms.sum())) <= 4 * (H / 32 + 16) * U32 * (float(terms.abs().sum()) + abs(slope) + 10)


def test_repeatable_in_place_on_a_stream_and_in_a_graph():
    T, k, E, H = 300, 6, 32, 512
    idx = choices(T, k, E, 0.1).cuda()
    ws = space(T, k, E)
    g = torch.Generator().manual_seed(1)
    x, w = torch.randn(T, H, generator=g).cuda().to(BF16), torch.rand(T, k, generator=g).cuda()

    def step():
        plan = moe.sort_pairs(idx, E, ws)
        rows = moe.dispatch(x, plan["row_of"], plan["offsets"])
        y = moe.collect(rows, plan["row_of"], w)
        d_rows, d_w = moe.collect_backward(y, rows, plan["row_of"], w, plan["offsets"])
        return [*plan.values(), rows, y, d_rows, d_w]

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
    idx.copy_(choices(T, k, E, 0.5, seed=4))
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(held, step()))
    assert int(held[1][-1]) < int(first[1][-1])
