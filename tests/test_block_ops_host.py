"""What the block operators refuse, on the host: no call here reaches a device."""
import ctypes

import pytest
import torch

import quantized_expert_ffn_gemm_b200 as moe
from quantized_expert_ffn_gemm_b200 import build as moe_build
from quantized_expert_ffn_gemm_b200.block import Mx4Mat

P, MIS = 0x10000, 0x10008  # never dereferenced: every call below is refused or has nothing to do
OK, INVALID, ALIGN, WORKSPACE, UNSUPPORTED = (moe.MOE_OK, moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_ALIGNMENT,
                                              moe.MOE_ERR_WORKSPACE, moe.MOE_ERR_UNSUPPORTED)
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    moe_build.build()
    return moe.lib()


def test_workspace_bytes(lib):
    assert moe.block_workspace_bytes(8192, 10, 512, 2048) > 0
    assert moe.block_workspace_bytes(0, 1, 1, 64) > 0
    for bad in ((-1, 1, 1, 64), (1, 0, 1, 64), (1, 33, 64, 64), (1, 3, 2, 64), (1, 1, 4097, 64), (1, 1, 1, 96), (1 << 30, 4, 4, 64)):
        assert moe.block_workspace_bytes(*bad) == 0, bad


def test_scratch_lies_behind_the_control_area(lib):
    """What the decode kernel keeps in a workspace from call to call (624,896 bytes) is not scratch."""
    assert moe.block_workspace_bytes(1, 1, 1, 64) > 624896
    assert norm_grad(lib, wsb=1 << 19) == WORKSPACE
    assert lib.moe_sort_pairs(P, 4, 2, 8, P, P, P, P, P, 1 << 19, None) == WORKSPACE


def norm(lib, r=P, rt=0, y=P, yt=0, T=4, H=128, post=1, pg=P, gate=None, mode=0, eps=1e-6, prg=P, ro=P, u=P, ut=2, ry=P,
         ru=P):
    return lib.moe_block_norm(r, rt, y, yt, T, H, post, pg, gate, mode, 1.0, eps, prg, ro, u, ut, ry, ru, None)


def test_block_norm(lib):
    assert norm(lib, T=0) == OK
    assert norm(lib, T=-1) == INVALID and norm(lib, eps=-1.0) == INVALID and norm(lib, eps=float("nan")) == INVALID
    assert norm(lib, H=100) == INVALID and norm(lib, H=0) == INVALID
    assert norm(lib, H=96) == UNSUPPORTED and norm(lib, H=16448) == UNSUPPORTED
    assert norm(lib, rt=3) == INVALID and norm(lib, yt=-1) == INVALID and norm(lib, ut=7) == INVALID
    assert norm(lib, mode=1) == INVALID and norm(lib, gate=P) == INVALID and norm(lib, gate=P, mode=3) == INVALID
    assert norm(lib, y=None) == INVALID                      # a gain of no block output
    assert norm(lib, post=0) == INVALID                      # statistics of a norm that is left out
    assert norm(lib, u=None) == INVALID                      # a gain of no second norm
    assert norm(lib, ro=None, u=None, prg=None, ru=None) == INVALID  # no output
    assert norm(lib, r=None) == INVALID
    for name in ("r", "y", "pg", "prg", "ro", "u", "ry", "ru"):
        assert norm(lib, **{name: MIS}) == ALIGN, name


def norm_grad(lib, dro=P, du=P, ut=2, r=P, rt=0, ru=P, y=P, yt=0, ry=P, T=4, H=128, post=1, pg=P, gate=None, mode=0, prg=P,
              dr=P, dy=P, dpg=P, dg=None, dprg=P, ws=P, wsb=BIG):
    return lib.moe_block_norm_backward(dro, du, ut, r, rt, ru, y, yt, ry, T, H, post, pg, gate, mode, 1.0, prg, dr, dy, dpg,
                                       dg, dprg, ws, wsb, None)


def test_block_norm_backward(lib):
    assert norm_grad(lib, T=0, dpg=None, dprg=None) == OK
    assert norm_grad(lib, T=-1) == INVALID and norm_grad(lib, H=96) == UNSUPPORTED and norm_grad(lib, rt=5) == INVALID
    assert norm_grad(lib, dro=None, du=None) == INVALID and norm_grad(lib, dr=None) == INVALID
    assert norm_grad(lib, ru=None) == INVALID and norm_grad(lib, ry=None) == INVALID and norm_grad(lib, r=None) == INVALID
    assert norm_grad(lib, dy=None) == INVALID and norm_grad(lib, y=None) == INVALID
    assert norm_grad(lib, dg=P) == INVALID                   # a gate's gradient without the gate
    assert norm_grad(lib, du=None) == INVALID                # a gain's gradient without what reaches it
    assert norm_grad(lib, ws=None) == WORKSPACE and norm_grad(lib, wsb=256) == WORKSPACE
    assert norm_grad(lib, ws=MIS) == ALIGN and norm_grad(lib, dr=MIS) == ALIGN and norm_grad(lib, dprg=MIS) == ALIGN


def test_pairs(lib):
    def sort(idx=P, T=4, k=2, E=8, c=P, o=P, r=P, s=P, ws=P, wsb=BIG):
        return lib.moe_sort_pairs(idx, T, k, E, c, o, r, s, ws, wsb, None)
    assert sort(T=-1) == INVALID and sort(k=0) == INVALID and sort(k=33, E=64) == INVALID and sort(k=9) == INVALID
    assert sort(E=0) == INVALID and sort(E=4097) == INVALID and sort(T=1 << 30) == INVALID
    assert sort(idx=None) == INVALID and sort(c=None) == INVALID and sort(r=None) == INVALID and sort(idx=MIS) == ALIGN
    assert sort(ws=None) == WORKSPACE and sort(wsb=256) == WORKSPACE and sort(ws=MIS) == ALIGN

    def disp(x=P, t=0, T=4, k=2, H=128, r=P, kept=None, rows=P):
        return lib.moe_dispatch(x, t, T, k, H, r, kept, rows, None)
    assert disp(T=0) == OK and disp(T=-1) == INVALID and disp(t=3) == INVALID and disp(k=0) == INVALID
    assert disp(H=100) == INVALID and disp(H=32) == UNSUPPORTED and disp(x=None) == INVALID and disp(rows=None) == INVALID
    assert disp(x=MIS) == ALIGN and disp(kept=0x10001) == ALIGN

    def coll(rows=P, t=0, T=4, k=2, H=128, r=P, w=P, res=None, y=P, yt=0):
        return lib.moe_collect(rows, t, T, k, H, r, w, res, y, yt, None)
    assert coll(T=0) == OK and coll(k=40) == INVALID and coll(yt=3) == INVALID and coll(H=16448) == UNSUPPORTED
    assert coll(rows=None) == INVALID and coll(y=None) == INVALID and coll(y=MIS) == ALIGN and coll(res=MIS) == ALIGN

    def grad(dy=P, dt=0, rows=P, t=0, T=4, k=2, H=128, r=P, w=P, kept=None, dr=P, dw=P):
        return lib.moe_collect_backward(dy, dt, rows, t, T, k, H, r, w, kept, dr, dw, None)
    assert grad(T=0) == OK and grad(dr=None, dw=None) == INVALID and grad(rows=None) == INVALID and grad(dy=None) == INVALID
    assert grad(dt=9) == INVALID and grad(dw=MIS) == ALIGN


def test_mx4(lib):
    def quant(x=P, t=0, T=4, K=128, r=None, k=1, kept=None, c=P, s=P):
        return lib.moe_mx4_quantize(x, t, T, K, r, k, kept, c, s, None)
    assert quant(T=0) == OK and quant(K=96) == UNSUPPORTED and quant(K=100) == INVALID and quant(t=4) == INVALID
    assert quant(kept=P) == INVALID and quant(r=P, k=0) == INVALID and quant(x=None) == INVALID and quant(c=MIS) == ALIGN
    assert lib.moe_mx4_dequantize(P, P, 0, 128, P, 0, None) == OK
    assert lib.moe_mx4_dequantize(P, P, -1, 128, P, 0, None) == INVALID
    assert lib.moe_mx4_dequantize(P, P, 4, 160, P, 0, None) == UNSUPPORTED
    assert lib.moe_mx4_dequantize(P, None, 4, 128, P, 0, None) == INVALID
    assert lib.moe_mx4_dequantize(P, MIS, 4, 128, P, 0, None) == ALIGN

    def prod(a=P, s=P, n=4, off=P, E=2, w=(2, 64, 128), up=None, out=P, t=1, ws=P, wsb=BIG, wc=P):
        m = [None if d is None else Mx4Mat(*d, wc, P) for d in (w, up)]
        ref = [None if d is None else ctypes.addressof(d) for d in m]
        return lib.moe_mx4_product(a, s, n, off, E, ref[0], ref[1], out, t, ws, wsb, None)
    assert prod(n=0) == OK and prod(n=-1) == INVALID and prod(w=None) == INVALID
    assert prod(off=None) == INVALID and prod(w=(3, 64, 128)) == INVALID and prod(E=0, w=(0, 64, 128)) == INVALID
    assert prod(w=(2, 96, 128)) == UNSUPPORTED and prod(w=(2, 64, 160)) == UNSUPPORTED and prod(w=(2, 64, 100)) == INVALID
    assert prod(up=(2, 128, 128)) == INVALID and prod(up=(2, 64, 64)) == INVALID and prod(wc=None) == INVALID
    assert prod(t=0) == UNSUPPORTED and prod(t=5) == INVALID and prod(a=None) == INVALID and prod(out=None) == INVALID
    assert prod(a=MIS) == ALIGN and prod(out=MIS) == ALIGN and prod(wc=MIS) == ALIGN and prod(ws=MIS) == ALIGN
    assert prod(ws=None) == WORKSPACE and prod(wsb=128) == WORKSPACE


def test_tensors_of_another_kind_are_refused():
    r = torch.zeros(4, 128)
    idx = torch.zeros(4, 2, dtype=torch.int32)
    q = moe.Mx4(torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(4, 4, dtype=torch.uint8))
    w = moe.Mx4(torch.zeros(2, 64, 64, dtype=torch.uint8), torch.zeros(2, 64, 4, dtype=torch.uint8))
    calls = [
        (lambda: moe.block_norm(r), "CUDA"),
        (lambda: moe.block_norm(r.double()), "type"),
        (lambda: moe.block_norm(r[0]), "shape"),
        (lambda: moe.block_norm([1.0]), "tensor"),
        (lambda: moe.block_norm_backward(r, r, r, r[:, 0]), "CUDA"),
        (lambda: moe.sort_pairs(idx.long(), 4, None), "type"),
        (lambda: moe.sort_pairs(idx, 4, None), "CUDA"),
        (lambda: moe.dispatch(r, idx), "CUDA"),
        (lambda: moe.collect(r, idx), "CUDA"),
        (lambda: moe.collect_backward(r, r, idx), "CUDA"),
        (lambda: moe.mx4_quantize(r, offsets=idx), "row_of"),
        (lambda: moe.mx4_quantize(r.int()), "type"),
        (lambda: moe.mx4_dequantize(q), "CUDA"),
        (lambda: moe.mx4_product(q, w), "CUDA"),
        (lambda: moe.mx4_product(q, q), "CUDA"),
    ]
    for call, word in calls:
        with pytest.raises(ValueError, match=word):
            call()


def test_workspace_bytes_at_the_ends_of_the_sizes(lib):
    """As many tokens as an int32 holds, and sizes that it does not hold, which are not cut to 32 bits."""
    most = (1 << 31) - 1
    for H in (64, 1088, 2048, 4096, 8256, 16384):
        few, near, last = (moe.block_workspace_bytes(T, 1, 1, H) for T in (most // 2, most - 64, most))
        assert few <= near <= last < 1 << 28, H  # 2 M chunks' counts or 296 blocks' sums
    for T, k, E, H in ((1 << 32) + 1, 1, 1, 64), (1, 1, 1, (1 << 32) + 64), (1, (1 << 32) + 1, 4, 64), (1 << 31, 1, 1, 64), (
            -(1 << 32) + 1, 1, 1, 64):
        assert moe.block_workspace_bytes(T, k, E, H) == 0, (T, k, E, H)


def test_a_binding_of_another_torch_is_built_again_and_not_called(lib, monkeypatch):
    """_bind.so uses torch's C++ interface, which differs from version to version behind the same source."""
    assert not moe_build.bind_stale()
    with monkeypatch.context() as m:
        m.setattr(torch, "__version__", torch.__version__ + ".later")
        assert moe_build.bind_stale()
        m.setattr(moe.block, "_b", None)
        with pytest.raises(RuntimeError, match="build it with"):
            moe.block_norm(torch.zeros(4, 128))
    with pytest.raises(ValueError, match="CUDA"):
        moe.block_norm(torch.zeros(4, 128))
    with monkeypatch.context() as m:  # one that does not say what it was built for
        import quantized_expert_ffn_gemm_b200._bind as b
        m.delattr(b, "built_for")
        m.setattr(moe.block, "_b", None)
        with pytest.raises(RuntimeError, match="build it with"):
            moe.block_norm(torch.zeros(4, 128))
    with monkeypatch.context() as m:  # a shorter version's name is not found in a longer one's
        m.setattr(moe_build, "bind_built_for", lambda: _bind_name()[:-1])
        assert moe_build.bind_stale()


def _bind_name():
    import quantized_expert_ffn_gemm_b200._bind as b
    return b.built_for
