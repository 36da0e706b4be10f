"""The block operators of include/moe_ffn.h for torch tensors: the norms around a block, pairs sorted by
expert and collected again (each with its gradient), MXFP4 rows and their product per expert.

As in the package's other entry points only arguments are marshalled here. Tensors are contiguous CUDA
tensors of one device; a call runs on that device's current stream, whichever device is current, and
allocates its outputs unless they are given. A tensor of another type, shape, layout or device than the
call takes raises ValueError; what the library refuses raises MoeError.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional

import torch

F32, F16, BF16 = 0, 1, 2
TYPE_OF = {torch.float32: F32, torch.float16: F16, torch.bfloat16: BF16}
GATE_NONE, GATE_CHANNEL, GATE_TOKEN = 0, 1, 2

_P, _I, _F, _Z = ctypes.c_void_p, ctypes.c_int32, ctypes.c_float, ctypes.c_size_t
_ARGS = {
    "moe_block_norm": [_P, _I, _P, _I, _I, _I, _I, _P, _P, _I, _F, _F, _P, _P, _P, _I, _P, _P, _P],
    "moe_block_norm_backward": [_P, _P, _I, _P, _I, _P, _P, _I, _P, _I, _I, _I, _P, _P, _I, _F, _P, _P, _P, _P, _P, _P,
                                _P, _Z, _P],
    "moe_sort_pairs": [_P, _I, _I, _I, _P, _P, _P, _P, _P, _Z, _P],
    "moe_dispatch": [_P, _I, _I, _I, _I, _P, _P, _P, _P],
    "moe_collect": [_P, _I, _I, _I, _I, _P, _P, _P, _P, _I, _P],
    "moe_collect_backward": [_P, _I, _P, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P],
    "moe_mx4_quantize": [_P, _I, _I, _I, _P, _I, _P, _P, _P, _P],
    "moe_mx4_dequantize": [_P, _P, _I, _I, _P, _I, _P],
    "moe_mx4_product": [_P, _P, _I, _P, _I, _P, _P, _P, _I, _P, _Z, _P],
}
EXPORTED = ["moe_block_workspace_bytes"] + list(_ARGS)


class Mx4Mat(ctypes.Structure):
    _fields_ = [("n_experts", _I), ("rows", _I), ("K", _I), ("codes", _P), ("scales", _P)]


class Mx4(NamedTuple):
    """MXFP4 rows: codes uint8 [..., rows, K/2] and scales uint8 [..., rows, K/32]."""
    codes: torch.Tensor
    scales: torch.Tensor

    @property
    def K(self) -> int:
        return self.codes.shape[-1] * 2


def bind(lib):
    """Argument types of the block entry points, set once on the loaded library."""
    lib.moe_block_workspace_bytes.restype = _Z
    lib.moe_block_workspace_bytes.argtypes = [_I] * 4
    for name, args in _ARGS.items():
        getattr(lib, name).restype = _I
        getattr(lib, name).argtypes = args


def _pkg():
    import quantized_expert_ffn_gemm_b200 as moe
    return moe


def _call(name: str, dev: torch.device, *args):
    moe = _pkg()
    fn = getattr(moe.lib(), name)
    if dev.index == torch.cuda.current_device():
        code = fn(*args, moe._raw_stream(dev.index))
    else:
        with torch.cuda.device(dev):
            code = fn(*args, moe._raw_stream(dev.index))
    if code != moe.MOE_OK:
        raise moe.MoeError(name, code)


def _want(name: str, t, dtypes, shape, dev=None):
    """Refuses a tensor that is not a contiguous CUDA tensor of these types and this shape (None: any size)."""
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name}: a tensor, got {type(t).__name__}")
    if t.dtype not in dtypes:
        raise ValueError(f"{name}: type {t.dtype}, takes {', '.join(str(d) for d in dtypes)}")
    if t.dim() != len(shape) or any(w is not None and w != n for w, n in zip(shape, t.shape)):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, takes {tuple('any' if w is None else w for w in shape)}")
    if not t.is_cuda:
        raise ValueError(f"{name}: not a CUDA tensor")
    if dev is not None and t.device != dev:
        raise ValueError(f"{name}: on {t.device}, the call's other tensors are on {dev}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: not contiguous")
    return t


_FLOATS = tuple(TYPE_OF)
_F32, _I32, _U8 = (torch.float32,), (torch.int32,), (torch.uint8,)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _ws(ws, dev):
    if ws is None:
        raise ValueError("ws: this call needs a Workspace")
    if ws.buf.device != dev:
        raise ValueError(f"ws: on {ws.buf.device}, the call's tensors are on {dev}")
    return ws.buf.data_ptr(), ws.nbytes


def block_workspace_bytes(T: int, k: int = 1, E: int = 1, H: int = 64) -> int:
    """Bytes of a Workspace that suffices for every block operator of these sizes (0: sizes not taken)."""
    return int(_pkg().lib().moe_block_workspace_bytes(T, k, E, H))


# ----------------------------------------------------------------------------- the norms around a block
def _gate(gate, T, H, dev):
    if gate is None:
        return GATE_NONE
    if gate.dim() == 2:
        _want("gate", gate, _F32, (T, 1), dev)
        return GATE_TOKEN
    _want("gate", gate, _F32, (H,), dev)
    return GATE_CHANNEL


def block_norm(r: torch.Tensor, y: Optional[torch.Tensor] = None, *, post_gain: Optional[torch.Tensor] = None,
               gate: Optional[torch.Tensor] = None, res_scale: float = 1.0, pre_gain: Optional[torch.Tensor] = None,
               eps: float = 1e-6, post_norm: bool = True, pre_norm: bool = True, u_dtype: torch.dtype = torch.bfloat16,
               r_out: Optional[torch.Tensor] = None):
    """r' = res_scale r + gate post_gain N(y) and u = pre_gain N(r'): (r', u, rstd_y, rstd_u).

    r [T,H], y [T,H] or None, each fp32, fp16 or bf16; gains fp32 [H]; gate fp32 [H] (a channel) or [T,1] (a
    token). r' has r's type (r_out may be r, to update the stream in place); u has u_dtype. Without
    pre_norm u and rstd_u are None, without y or post_norm rstd_y is; the statistics are what
    block_norm_backward needs."""
    T, H = _want("r", r, _FLOATS, (None, None)).shape
    dev = r.device
    if y is not None:
        _want("y", y, _FLOATS, (T, H), dev)
    for n, t in (("post_gain", post_gain), ("pre_gain", pre_gain)):
        if t is not None:
            _want(n, t, _F32, (H,), dev)
    mode = _gate(gate, T, H, dev)
    if pre_norm and u_dtype not in TYPE_OF:
        raise ValueError(f"u_dtype: {u_dtype}, takes {', '.join(str(d) for d in _FLOATS)}")
    if r_out is None:
        r_out = torch.empty_like(r)
    else:
        _want("r_out", r_out, (r.dtype,), (T, H), dev)
    u = torch.empty(T, H, dtype=u_dtype, device=dev) if pre_norm else None
    rstd_y = torch.empty(T, dtype=torch.float32, device=dev) if y is not None and post_norm else None
    rstd_u = torch.empty(T, dtype=torch.float32, device=dev) if pre_norm else None
    _call("moe_block_norm", dev, r.data_ptr(), TYPE_OF[r.dtype], _ptr(y), F32 if y is None else TYPE_OF[y.dtype], T, H,
          1 if post_norm else 0, _ptr(post_gain), _ptr(gate), mode, res_scale, eps, _ptr(pre_gain), r_out.data_ptr(),
          _ptr(u), TYPE_OF[u_dtype] if pre_norm else F32, _ptr(rstd_y), _ptr(rstd_u))
    return r_out, u, rstd_y, rstd_u


def block_norm_backward(dr_out: Optional[torch.Tensor], du: Optional[torch.Tensor], r_out: torch.Tensor,
                        rstd_u: Optional[torch.Tensor], y: Optional[torch.Tensor] = None,
                        rstd_y: Optional[torch.Tensor] = None, *, post_gain: Optional[torch.Tensor] = None,
                        gate: Optional[torch.Tensor] = None, res_scale: float = 1.0,
                        pre_gain: Optional[torch.Tensor] = None, post_norm: bool = True, ws=None) -> dict:
    """Gradients of block_norm: a dict of dr, dy, d_post_gain, d_gate and d_pre_gain.

    dr_out and du reach r' and u (None: nothing does); r_out, rstd_u, y and rstd_y as the forward call
    took and returned them. An entry is None where block_norm had no such argument."""
    T, H = _want("r_out", r_out, _FLOATS, (None, None)).shape
    dev = r_out.device
    if dr_out is not None:
        _want("dr_out", dr_out, (r_out.dtype,), (T, H), dev)
    if du is not None:
        _want("du", du, _FLOATS, (T, H), dev)
        _want("rstd_u", rstd_u, _F32, (T,), dev)
    if y is not None:
        _want("y", y, _FLOATS, (T, H), dev)
        if post_norm:
            _want("rstd_y", rstd_y, _F32, (T,), dev)
    for n, t in (("post_gain", post_gain), ("pre_gain", pre_gain)):
        if t is not None:
            _want(n, t, _F32, (H,), dev)
    mode = _gate(gate, T, H, dev)
    ws_ptr, ws_bytes = _ws(ws, dev)
    out = {"dr": torch.empty_like(r_out), "dy": None if y is None else torch.empty_like(y),
           "d_post_gain": None if post_gain is None else torch.empty_like(post_gain),
           "d_gate": None if gate is None else torch.empty_like(gate),
           "d_pre_gain": None if pre_gain is None else torch.empty_like(pre_gain)}
    _call("moe_block_norm_backward", dev, _ptr(dr_out), _ptr(du), F32 if du is None else TYPE_OF[du.dtype],
          r_out.data_ptr(), TYPE_OF[r_out.dtype], _ptr(rstd_u), _ptr(y), F32 if y is None else TYPE_OF[y.dtype],
          _ptr(rstd_y), T, H, 1 if post_norm else 0, _ptr(post_gain), _ptr(gate), mode, res_scale, _ptr(pre_gain),
          out["dr"].data_ptr(), _ptr(out["dy"]), _ptr(out["d_post_gain"]), _ptr(out["d_gate"]),
          _ptr(out["d_pre_gain"]), ws_ptr, ws_bytes)
    return out


# ----------------------------------------------------------------------------- pairs sorted by expert
def sort_pairs(idx: torch.Tensor, E: int, ws) -> dict:
    """The (token, slot) pairs of idx int32 [T,k] (-1: no expert) in expert order: counts [E], offsets [E+1],
    row_of [T,k] (-1: no row) and src [T*k] (-1 behind the last kept pair), all int32."""
    T, k = _want("idx", idx, _I32, (None, None)).shape
    dev = idx.device
    ws_ptr, ws_bytes = _ws(ws, dev)
    counts = torch.empty(max(E, 1), dtype=torch.int32, device=dev)
    offsets = torch.empty(max(E, 1) + 1, dtype=torch.int32, device=dev)
    row_of = torch.empty(T, k, dtype=torch.int32, device=dev)
    src = torch.empty(T * k, dtype=torch.int32, device=dev)
    _call("moe_sort_pairs", dev, idx.data_ptr(), T, k, E, counts.data_ptr(), offsets.data_ptr(), row_of.data_ptr(),
          src.data_ptr(), ws_ptr, ws_bytes)
    return {"counts": counts, "offsets": offsets, "row_of": row_of, "src": src}


def _kept(offsets, dev):
    """Device pointer to the kept pairs' number, the last offset."""
    if offsets is None:
        return None
    E = _want("offsets", offsets, _I32, (None,), dev).shape[0] - 1
    if E < 1:
        raise ValueError("offsets: takes E + 1 entries")
    return offsets.data_ptr() + 4 * E


def dispatch(x: torch.Tensor, row_of: torch.Tensor, offsets: Optional[torch.Tensor] = None,
             rows: Optional[torch.Tensor] = None) -> torch.Tensor:
    """rows[row_of[t,j]] = x[t]: [T*k,H] of x's type. With offsets the rows behind the last kept pair are
    zero, without it they are left as they were (in `rows`, if given)."""
    T, H = _want("x", x, _FLOATS, (None, None)).shape
    dev = x.device
    k = _want("row_of", row_of, _I32, (T, None), dev).shape[1]
    kept = _kept(offsets, dev)
    if rows is None:
        rows = torch.empty(T * k, H, dtype=x.dtype, device=dev)
    else:
        _want("rows", rows, (x.dtype,), (T * k, H), dev)
    _call("moe_dispatch", dev, x.data_ptr(), TYPE_OF[x.dtype], T, k, H, row_of.data_ptr(), kept, rows.data_ptr())
    return rows


def collect(rows: torch.Tensor, row_of: torch.Tensor, w: Optional[torch.Tensor] = None,
            residual: Optional[torch.Tensor] = None, dtype: torch.dtype = torch.float32) -> torch.Tensor:
    """y[t] = sum_j w[t,j] rows[row_of[t,j]] + residual[t], of `dtype`. Without w the gradient of dispatch."""
    T, k = _want("row_of", row_of, _I32, (None, None)).shape
    dev = row_of.device
    H = _want("rows", rows, _FLOATS, (T * k, None), dev).shape[1]
    if w is not None:
        _want("w", w, _F32, (T, k), dev)
    if residual is not None:
        _want("residual", residual, _F32, (T, H), dev)
    if dtype not in TYPE_OF:
        raise ValueError(f"dtype: {dtype}, takes {', '.join(str(d) for d in _FLOATS)}")
    y = torch.empty(T, H, dtype=dtype, device=dev)
    _call("moe_collect", dev, rows.data_ptr(), TYPE_OF[rows.dtype], T, k, H, row_of.data_ptr(), _ptr(w), _ptr(residual),
          y.data_ptr(), TYPE_OF[dtype])
    return y


def collect_backward(dy: torch.Tensor, rows: torch.Tensor, row_of: torch.Tensor, w: Optional[torch.Tensor] = None,
                     offsets: Optional[torch.Tensor] = None):
    """Gradients of collect for dy [T,H]: (d_rows of rows' type, d_w fp32 [T,k], None without w)."""
    T, k = _want("row_of", row_of, _I32, (None, None)).shape
    dev = row_of.device
    H = _want("rows", rows, _FLOATS, (T * k, None), dev).shape[1]
    _want("dy", dy, _FLOATS, (T, H), dev)
    if w is not None:
        _want("w", w, _F32, (T, k), dev)
    kept = _kept(offsets, dev)
    d_rows = torch.empty_like(rows)
    d_w = None if w is None else torch.empty_like(w)
    _call("moe_collect_backward", dev, dy.data_ptr(), TYPE_OF[dy.dtype], rows.data_ptr(), TYPE_OF[rows.dtype], T, k, H,
          row_of.data_ptr(), _ptr(w), kept, d_rows.data_ptr(), _ptr(d_w))
    return d_rows, d_w


# ----------------------------------------------------------------------------- MXFP4
def mx4_quantize(x: torch.Tensor, row_of: Optional[torch.Tensor] = None,
                 offsets: Optional[torch.Tensor] = None) -> Mx4:
    """x [..., K] (fp32, fp16 or bf16) to MXFP4. With row_of int32 [T,k] the quantised token x[t] goes to
    rows row_of[t,:] of T*k rows, as dispatch copies it; offsets as there."""
    if row_of is None:
        if offsets is not None:
            raise ValueError("offsets: goes with row_of")
        if not isinstance(x, torch.Tensor) or x.dim() < 1:
            raise ValueError("x: takes a tensor [..., K]")
        K, lead = x.shape[-1], tuple(x.shape[:-1])
        _want("x", x, _FLOATS, lead + (None,))
        T, k, kept, dev = 1, 1, None, x.device
        for n in lead:
            T *= n
    else:
        T, K = _want("x", x, _FLOATS, (None, None)).shape
        dev = x.device
        k = _want("row_of", row_of, _I32, (T, None), dev).shape[1]
        kept, lead = _kept(offsets, dev), (T * k,)
    codes = torch.empty(lead + (K // 2,), dtype=torch.uint8, device=dev)
    scales = torch.empty(lead + (K // 32,), dtype=torch.uint8, device=dev)
    _call("moe_mx4_quantize", dev, x.data_ptr(), TYPE_OF[x.dtype], T, K, _ptr(row_of), k, kept, codes.data_ptr(),
          scales.data_ptr())
    return Mx4(codes, scales)


def _mx4(name, q, dev, dims=None):
    """(leading sizes, K) of MXFP4 rows."""
    codes, scales = q
    if not isinstance(codes, torch.Tensor) or codes.dim() < 1 or (dims is not None and codes.dim() != dims):
        raise ValueError(f"{name}.codes: takes a tensor of {dims or 'one or more'} dimensions")
    lead = tuple(codes.shape[:-1])
    _want(name + ".codes", codes, _U8, lead + (None,), dev)
    K = 2 * codes.shape[-1]
    if K % 32:
        raise ValueError(f"{name}.codes: K = {K} is not a multiple of 32")
    _want(name + ".scales", scales, _U8, lead + (K // 32,), codes.device)
    return lead, K


def mx4_dequantize(q: Mx4, dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """The values of MXFP4 rows, [..., K] of `dtype`."""
    lead, K = _mx4("q", q, None)
    if dtype not in TYPE_OF:
        raise ValueError(f"dtype: {dtype}, takes {', '.join(str(d) for d in _FLOATS)}")
    rows = 1
    for n in lead:
        rows *= n
    out = torch.empty(lead + (K,), dtype=dtype, device=q.codes.device)
    _call("moe_mx4_dequantize", out.device, q.codes.data_ptr(), q.scales.data_ptr(), rows, K, out.data_ptr(),
          TYPE_OF[dtype])
    return out


def mx4_product(a: Mx4, w: Mx4, offsets: Optional[torch.Tensor] = None, *, up: Optional[Mx4] = None,
                dtype: torch.dtype = torch.float16, ws=None) -> torch.Tensor:
    """out[r] = a[r] w[g]^T for the rows offsets[g] <= r < offsets[g+1], [rows,N] fp16 or bf16; with up
    silu(a w^T) * (a up^T). a: [rows,K]; w, up: [E,N,K]; offsets int32 [E+1] as sort_pairs gives it, or
    None for E = 1. Rows behind offsets[E] become zero."""
    (n_rows,), K = _mx4("a", a, None, 2)
    dev = a.codes.device
    (E, N), Kw = _mx4("w", w, dev, 3)
    if Kw != K:
        raise ValueError(f"w: K = {Kw}, a has {K}")
    if up is not None and _mx4("up", up, dev, 3) != ((E, N), K):
        raise ValueError("up: another shape than w")
    if offsets is not None:
        _want("offsets", offsets, _I32, (E + 1,), dev)
    if dtype not in TYPE_OF:
        raise ValueError(f"dtype: {dtype}, takes {torch.float16}, {torch.bfloat16}")
    ws_ptr, ws_bytes = _ws(ws, dev)
    wm = Mx4Mat(E, N, K, w.codes.data_ptr(), w.scales.data_ptr())
    um = None if up is None else Mx4Mat(E, N, K, up.codes.data_ptr(), up.scales.data_ptr())
    out = torch.empty(n_rows, N, dtype=dtype, device=dev)
    _call("moe_mx4_product", dev, a.codes.data_ptr(), a.scales.data_ptr(), n_rows, _ptr(offsets), E,
          ctypes.addressof(wm), None if um is None else ctypes.addressof(um), out.data_ptr(), TYPE_OF[dtype], ws_ptr,
          ws_bytes)
    return out
