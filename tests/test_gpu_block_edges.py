"""The block operators on calls that are allowed and unusual: tensors that start on 16 bytes but not on 32, outputs left
out at the C interface, no rows at all, tensors of more than 2^31 values, and workspaces that are too small."""
import types

import pytest
import torch

import quantized_expert_ffn_gemm_b200 as moe
import synth
from tests import block_ref as ref
from tests.gpu_util import to_dev

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


def shifted(t, by=16):
    """A contiguous copy whose data starts `by` bytes behind a 256-byte boundary."""
    n = by // t.element_size()
    buf = torch.empty(t.numel() + 256, dtype=t.dtype, device="cuda")
    first = (-(buf.data_ptr()) % 256) // t.element_size() + n
    out = buf[first:first + t.numel()].view(t.shape)
    out.copy_(t)
    assert out.data_ptr() % 256 == by and out.is_contiguous()
    return out


@pytest.mark.parametrize("H", [192, 2048, 4160])
@pytest.mark.parametrize("r,y,u", [(F32, F32, F32), (F32, BF16, F16), (BF16, F32, BF16)])
def test_norm_of_tensors_on_16_bytes(H, r, y, u):
    T = 19
    g = torch.Generator().manual_seed(H)
    n = lambda *s, t=F32: torch.randn(*s, generator=g).to(t).cuda()  # noqa: E731
    args = dict(r=n(T, H, t=r), y=n(T, H, t=y), post_gain=n(H), gate=n(H), pre_gain=n(H))
    ws = moe.Workspace(moe.block_workspace_bytes(T, H=H))

    def both(move):
        a = {k: move(v) for k, v in args.items()}
        rr, yy = a.pop("r"), a.pop("y")
        out = moe.block_norm(rr, yy, **a, u_dtype=u, r_out=move(torch.zeros_like(rr)))
        grad = moe.block_norm_backward(move(out[0]), move(out[1]), move(out[0]), move(out[3]), yy, move(out[2]), **a, ws=ws)
        return list(out) + list(grad.values())

    for a, b in zip(both(lambda t: t.clone()), both(shifted)):
        # the same sums in the same order up to the fused multiply-adds that the types' variants use
        tol = 64 * 2.0 ** -24 if a.dtype == F32 else 2 * ref.half(a.dtype)
        scale = float(a.double().abs().max())
        assert float((a.double() - b.double()).abs().max()) <= tol * scale


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_pairs_and_rows_of_tensors_on_16_bytes(dtype):
    T, k, E, H = 33, 4, 8, 320
    g = torch.Generator().manual_seed(3)
    idx = torch.rand(T, E, generator=g).topk(k, 1).indices.to(torch.int32).cuda()
    plan = moe.sort_pairs(shifted(idx), E, moe.Workspace(moe.block_workspace_bytes(T, k, E)))
    x, w = torch.randn(T, H, generator=g).to(dtype).cuda(), torch.rand(T, k, generator=g).cuda()
    row_of = plan["row_of"]
    rows = moe.dispatch(x, row_of, plan["offsets"])
    assert torch.equal(rows, moe.dispatch(shifted(x), shifted(row_of), plan["offsets"], shifted(torch.zeros_like(rows))))
    for out in (F32, dtype):
        assert torch.equal(moe.collect(rows, row_of, w, dtype=out), moe.collect(shifted(rows), row_of, shifted(w), dtype=out))
    one, two = moe.collect_backward(x, rows, row_of, w), moe.collect_backward(shifted(x), shifted(rows), row_of, w)
    assert torch.equal(one[0], two[0])
    # the dot products: eight values a lane either way, in the same order
    assert float((one[1] - two[1]).abs().max()) <= (H / 32 + 8) * 2.0 ** -24 * H
    q = moe.mx4_quantize(x)
    p = moe.mx4_quantize(shifted(x))
    assert torch.equal(q.codes, p.codes) and torch.equal(q.scales, p.scales)
    a = moe.mx4_quantize(rows)
    W = moe.mx4_quantize(torch.randn(E, 64, H, generator=g).cuda())
    ws = moe.Workspace(256)
    assert torch.equal(moe.mx4_product(a, W, plan["offsets"], ws=ws),
                       moe.mx4_product(moe.Mx4(shifted(a.codes), shifted(a.scales)),
                                       moe.Mx4(shifted(W.codes), shifted(W.scales)), shifted(plan["offsets"]), ws=ws))


def test_tensors_on_8_bytes_are_refused():
    x = torch.randn(4, 128).cuda()
    idx = torch.zeros(4, 1, dtype=torch.int32, device="cuda")
    for call in (lambda: moe.block_norm(shifted(x, 8)), lambda: moe.dispatch(shifted(x, 8), idx),
                 lambda: moe.dispatch(x, shifted(idx, 8)), lambda: moe.mx4_quantize(shifted(x, 8))):
        with pytest.raises(moe.MoeError) as e:
            call()
        assert e.value.code == moe.MOE_ERR_ALIGNMENT
    torch.cuda.synchronize()


def test_workspaces_too_small_are_refused():
    idx = torch.zeros(5000, 2, dtype=torch.int32, device="cuda")
    r = torch.randn(8, 128).cuda()
    s = torch.ones(8, device="cuda")
    for call in (lambda: moe.sort_pairs(idx, 64, moe.Workspace(512)),
                 lambda: moe.block_norm_backward(r, r, r, s, ws=moe.Workspace(512))):
        with pytest.raises(moe.MoeError) as e:
            call()
        assert e.value.code == moe.MOE_ERR_WORKSPACE


def test_no_rows_at_all():
    ws = moe.Workspace(moe.block_workspace_bytes(1, 2, 4, 128))
    x, idx = torch.empty(0, 128, device="cuda"), torch.empty(0, 2, dtype=torch.int32, device="cuda")
    for gate in (None, torch.ones(128, device="cuda"), torch.empty(0, 1, device="cuda")):
        r, u, ry, ru = moe.block_norm(x, x, gate=gate)
        grad = moe.block_norm_backward(r, u, r, ru, x, ry, gate=gate, ws=ws)
        assert u.shape == grad["dy"].shape == (0, 128)
        assert gate is None or bool((grad["d_gate"] == 0).all())
    plan = moe.sort_pairs(idx, 4, ws)
    assert moe.dispatch(x, plan["row_of"], plan["offsets"]).shape == (0, 128)
    assert moe.collect(x, plan["row_of"]).shape == (0, 128)
    d_rows, d_w = moe.collect_backward(x, x, plan["row_of"], torch.empty(0, 2, device="cuda"), plan["offsets"])
    assert d_rows.shape == (0, 128) and d_w.shape == (0, 2)
    a = moe.mx4_quantize(x, plan["row_of"], plan["offsets"])
    assert a.codes.shape == (0, 64) and moe.mx4_dequantize(a).shape == (0, 128)
    W = moe.mx4_quantize(torch.randn(4, 64, 128).cuda())
    assert moe.mx4_product(a, W, plan["offsets"], up=W, ws=ws).shape == (0, 64)
    torch.cuda.synchronize()


def test_outputs_left_out_at_the_c_interface():
    T, H, k = 24, 320, 3
    g = torch.Generator().manual_seed(1)
    n = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    r, y, gain, gate = n(T, H), n(T, H), n(H), n(T, 1)
    full = moe.block_norm(r, y, post_gain=gain, gate=gate, pre_gain=gain)
    lib, st = moe.lib(), torch.cuda.current_stream().cuda_stream
    u = torch.empty_like(full[1])
    p = lambda t: t.data_ptr()  # noqa: E731
    assert lib.moe_block_norm(p(r), 0, p(y), 0, T, H, 1, p(gain), p(gate), 2, 1.0, 1e-6, p(gain), None, p(u), 2, None, None,
                              st) == 0
    assert torch.equal(u, full[1])  # without the stream and the statistics
    ws = moe.Workspace(moe.block_workspace_bytes(T, k, 8, H))
    grad = moe.block_norm_backward(r, full[1], full[0], full[3], y, full[2], post_gain=gain, gate=gate, pre_gain=gain, ws=ws)
    dr, dy = torch.empty_like(r), torch.empty_like(y)
    for kept in ("d_gate", "d_pre_gain", None):
        outs = {m: torch.full_like(grad[m], 3.0) for m in ("d_post_gain", "d_gate", "d_pre_gain")}
        args = [p(outs[m]) if m == kept else None for m in outs]
        assert lib.moe_block_norm_backward(p(r), p(full[1]), 2, p(full[0]), 0, p(full[3]), p(y), 0, p(full[2]), T, H, 1,
                                           p(gain), p(gate), 2, 1.0, p(gain), p(dr), p(dy), *args, p(ws.buf), ws.nbytes,
                                           st) == 0
        assert torch.equal(dr, grad["dr"]) and torch.equal(dy, grad["dy"])
        for m in outs:
            assert torch.equal(outs[m], grad[m] if m == kept else torch.full_like(grad[m], 3.0))
    inplace = r.clone()  # dr may be dr_out
    assert lib.moe_block_norm_backward(p(inplace), p(full[1]), 2, p(full[0]), 0, p(full[3]), p(y), 0, p(full[2]), T, H, 1,
                                       p(gain), p(gate), 2, 1.0, p(gain), p(inplace), p(dy), None, None, None, p(ws.buf),
                                       ws.nbytes, st) == 0
    assert torch.equal(inplace, grad["dr"])
    # the way back: one output or the other, and the rows' gradient in the rows' place
    idx = torch.randint(-1, 8, (T, k), generator=g, dtype=torch.int32).cuda()
    plan = moe.sort_pairs(idx, 8, ws)
    rows, w = n(T * k, H), n(T, k)
    d_rows, d_w = moe.collect_backward(y, rows, plan["row_of"], w, plan["offsets"])
    only = torch.empty_like(d_w)
    kept = plan["offsets"].data_ptr() + 4 * 8
    assert lib.moe_collect_backward(p(y), 0, p(rows), 0, T, k, H, p(plan["row_of"]), p(w), kept, None, p(only), st) == 0
    assert torch.equal(only, d_w)
    place = rows.clone()
    assert lib.moe_collect_backward(p(y), 0, p(place), 0, T, k, H, p(plan["row_of"]), p(w), kept, p(place), p(only), st) == 0
    assert torch.equal(place, d_rows) and torch.equal(only, d_w)
    place.zero_()
    assert lib.moe_collect_backward(p(y), 0, None, 0, T, k, H, p(plan["row_of"]), p(w), kept, p(place), None, st) == 0
    assert torch.equal(place, d_rows)
    z = y.clone()  # the residual may be y itself
    want = moe.collect(rows, plan["row_of"], w, residual=y)
    assert lib.moe_collect(p(rows), 0, T, k, H, p(plan["row_of"]), p(w), p(z), p(z), 0, st) == 0
    assert torch.equal(z, want)


def test_more_than_2_to_31_values():
    """Offsets of elements past 32 bits: rows at both ends against the same rows alone."""
    T, k, H, E = 120000, 9, 2048, 16  # 2.2e9 values
    g = torch.Generator(device="cuda").manual_seed(0)
    idx = torch.randint(0, E, (T, k), generator=g, device="cuda", dtype=torch.int32)
    ws = moe.Workspace(moe.block_workspace_bytes(T, k, E, H))
    plan = moe.sort_pairs(idx, E, ws)
    x = torch.randn(T, H, generator=g, device="cuda", dtype=BF16)
    rows = moe.dispatch(x, plan["row_of"], plan["offsets"])
    some = torch.cat([torch.arange(0, 40), torch.arange(T * k // 2, T * k // 2 + 40), torch.arange(T * k - 40, T * k)]).cuda()
    assert torch.equal(rows[some], x[plan["src"][some].long()])
    w = torch.rand(T, k, generator=g, device="cuda")
    toks = torch.cat([torch.arange(0, 20), torch.arange(T - 20, T)]).cuda()
    y = moe.collect(rows, plan["row_of"], w)
    each = rows[plan["row_of"][toks].long()].double() * w[toks][..., None].double()
    assert float((y[toks].double() - each.sum(1)).abs().max()) <= (k + 2) * 2.0 ** -24 * float(each.abs().sum(1).max())
    d_rows, d_w = moe.collect_backward(x, rows, plan["row_of"], w, plan["offsets"])
    pair = plan["row_of"][toks]
    want = (w[toks][..., None] * x[toks][:, None].float()).to(BF16)
    assert torch.equal(d_rows[pair.long()], want)
    del d_rows, y, rows
    q = moe.mx4_quantize(x, plan["row_of"], plan["offsets"])
    alone = moe.mx4_quantize(x[plan["src"][some].long()].contiguous())
    assert torch.equal(q.codes[some], alone.codes) and torch.equal(q.scales[some], alone.scales)
    back = moe.mx4_dequantize(q)
    assert torch.equal(back[some], moe.mx4_dequantize(alone))
    del back
    # 1.08 million rows of 2048 features
    a = moe.mx4_quantize(torch.randn(T * k, 64, generator=g, device="cuda"))
    W = moe.mx4_quantize(torch.randn(E, H, 64, generator=g, device="cuda"))
    out = moe.mx4_product(a, W, plan["offsets"], ws=ws)
    assert moe.read_device_error(ws) == 0
    off = plan["offsets"].tolist()
    for e in (0, E // 2, E - 1):
        r = slice(off[e + 1] - 100, off[e + 1])
        few = moe.mx4_product(moe.Mx4(a.codes[r].clone(), a.scales[r].clone()),
                              moe.Mx4(W.codes[e:e + 1], W.scales[e:e + 1]), ws=ws)
        assert torch.equal(out[r], few)
    del out, a
    r = torch.randn(140000, 16384, generator=g, device="cuda", dtype=BF16)
    _, u, _, rstd = moe.block_norm(r, r_out=r)
    for s in (slice(0, 8), slice(139992, 140000)):
        _, few, _, rs = moe.block_norm(r[s].clone())
        assert torch.equal(u[s], few) and torch.equal(rstd[s], rs)


@pytest.mark.parametrize("T", [1, 2, 5])
def test_one_workspace_for_layers_and_block_operators(T):
    """The decode kernel keeps its launch counts and tagged words in the workspace from call to call; sorts and gradients
    in between leave them alone, whatever they write."""
    shape = synth.LayerShape("block_shared_ws", 8, 512, 32, 4, 256, synth.Q2, True, 1.1, seed=31)
    x, Wr, b, routed, shared = to_dev(synth.make_layer(shape))
    x = x[:T].contiguous()
    run = lambda ws: moe.layer_forward(x, Wr, b, routed, shared, 4, ws)  # noqa: E731
    want = run(moe.Workspace.for_layer(512, 32, 4, 256, True, T)).clone()
    ws = moe.Workspace(max(moe.workspace_bytes(512, 32, 4, 256, True, 8), moe.block_workspace_bytes(3000, 4, 32, 2048)))
    g = torch.Generator().manual_seed(T)
    r, s = torch.randn(700, 2048, generator=g).cuda(), torch.rand(700, generator=g).cuda()
    gain = torch.ones(2048, device="cuda")
    for i in range(6):
        n = 3000 if i % 2 else 7
        idx = torch.rand(n, 32, generator=g).topk(4, 1).indices.to(torch.int32)
        plan = moe.sort_pairs(idx.cuda(), 32, ws)
        grad = moe.block_norm_backward(r, r, r, s, pre_gain=gain, ws=ws)
        assert torch.equal(run(ws), want)
        assert torch.equal(plan["row_of"].cpu(), ref.sort_pairs(idx, 32)["row_of"])
        x64, d = r.double() * s.double()[:, None], r.double()
        assert float((grad["d_pre_gain"].double() - (d * x64).sum(0)).abs().max()) <= 702 * 2.0 ** -24 * float(
            (d * x64).abs().sum(0).max())
    assert moe.read_device_error(ws) == 0
    big = moe.block_workspace_bytes(3000, 4, 32, 2048)
    assert big > moe.block_workspace_bytes(1, 1, 1, 64) > 0


def test_rows_written_and_read_again_without_a_pause():
    """A chain of small calls on the same buffers, each allowed to start while the one before ends: every reader sees what
    its writer left, eagerly and in a replayed graph."""
    T, k, H, n = 6, 10, 2048, 40
    g = torch.Generator().manual_seed(11)
    row_of = torch.randperm(T * k, generator=g).to(torch.int32).view(T, k).cuda()
    xs = torch.randint(-8, 9, (n, T, H), generator=g).float().cuda()  # sums of k equal values are exact
    rows = torch.zeros(T * k, H, device="cuda")
    want = k * xs

    def chain():
        ys = []
        for x in xs:
            moe.dispatch(x, row_of, None, rows)
            ys.append(moe.collect(rows, row_of))
        return torch.stack(ys)

    for _ in range(5):
        assert torch.equal(chain(), want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = chain()
    for sign in (-1, 1):
        xs.mul_(-1)
        rows.zero_()
        graph.replay()
        assert torch.equal(out, k * xs)


def test_quantised_rows_and_products_without_a_pause():
    """As above through the MXFP4 rows: quantised into the same memory (the allocator hands it out again) and multiplied."""
    T, K, N, n = 3, 256, 64, 30
    g = torch.Generator().manual_seed(12)
    w = moe.mx4_quantize(torch.randint(-3, 4, (1, N, K), generator=g).float().cuda())
    xs = torch.randint(-3, 4, (n, T, K), generator=g).float().cuda()  # MXFP4 holds these exactly
    ws = moe.Workspace(256)
    want = [moe.mx4_dequantize(moe.mx4_quantize(x), F32).double() @ moe.mx4_dequantize(w, F32)[0].double().T for x in xs]

    def chain():
        return torch.stack([moe.mx4_product(moe.mx4_quantize(x), w, dtype=F16, ws=ws) for x in xs])

    for _ in range(5):
        assert torch.equal(chain().double(), torch.stack(want))  # integers, far below 2^11: exact in fp16
    assert moe.read_device_error(ws) == 0


def test_offsets_that_swing_are_work_for_nobody():
    """Offsets 0, n, 0, n, ...: every second group would be all rows. The call flags them and multiplies nothing."""
    n, E, K, N = 4000, 512, 256, 64
    a = moe.mx4_quantize(torch.randn(n, K, generator=torch.Generator().manual_seed(5)).cuda())
    w = moe.mx4_quantize(torch.randn(E, N, K, generator=torch.Generator().manual_seed(6)).cuda())
    ws = moe.Workspace(256)
    good = torch.linspace(0, n, E + 1).to(torch.int32).cuda()
    want = moe.mx4_product(a, w, good, ws=ws)
    swing = torch.tensor([0, n], dtype=torch.int32).repeat(E // 2 + 1)[:E + 1].cuda()
    for up in (None, w):
        moe.mx4_product(a, w, swing, up=up, ws=ws)
        assert moe.read_device_error(ws) == moe.MOE_ERR_DEVICE_CHECK
    assert torch.equal(want, moe.mx4_product(a, w, good, ws=ws)) and moe.read_device_error(ws) == 0


@pytest.mark.parametrize("T,H", [(7, 192), (300, 2048), (7, 4160), (3, 16384)])
def test_workspace_on_16_bytes(T, H):
    """Scratch behind a workspace that starts 16 bytes behind a 256-byte boundary: the same results as on the boundary."""
    g = torch.Generator().manual_seed(H)
    n = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    r, y, dr, du, gain, gate = n(T, H), n(T, H), n(T, H), n(T, H), n(H), n(H)
    ry, ru = (v.square().mean(1).rsqrt() for v in (y, r))
    need = moe.block_workspace_bytes(T, H=H)
    idx = torch.randint(-1, 32, (5000, 2), generator=g, dtype=torch.int32).cuda()

    def results(at, nbytes):
        buf = shifted(torch.zeros(nbytes, dtype=torch.uint8), at) if at else torch.zeros(nbytes, dtype=torch.uint8,
                                                                                         device="cuda")
        ws = types.SimpleNamespace(buf=buf, nbytes=nbytes)
        grad = moe.block_norm_backward(dr, du, r, ru, y, ry, post_gain=gain, gate=gate, pre_gain=gain, ws=ws)
        return list(grad.values())

    def sorts(at):
        nbytes = moe.block_workspace_bytes(5000, 2, 32)
        buf = shifted(torch.zeros(nbytes, dtype=torch.uint8), at) if at else torch.zeros(nbytes, dtype=torch.uint8,
                                                                                         device="cuda")
        return list(moe.sort_pairs(idx, 32, types.SimpleNamespace(buf=buf, nbytes=nbytes)).values())

    assert all(torch.equal(a, b) for a, b in zip(results(0, need), results(16, need)))
    assert all(torch.equal(a, b) for a, b in zip(sorts(0), sorts(16)))
