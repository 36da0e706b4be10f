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


_fn = {}                # entry points by name, with their argument types set
_stream_of = None       # device index -> raw handle of its current stream
_MoeError = None
_device = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else torch.cuda.current_device


def bind(lib, stream_of, error):
    """Argument types of the block entry points, set once on the loaded library."""
    global _stream_of, _MoeError
    _stream_of, _MoeError = stream_of, error
    lib.moe_block_workspace_bytes.restype = _Z
    lib.moe_block_workspace_bytes.argtypes = [_I] * 4
    _fn["moe_block_workspace_bytes"] = lib.moe_block_workspace_bytes
    for name, args in _ARGS.items():
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = _I, args
        _fn[name] = fn


def _entry(name: str):
    if name not in _fn:
        import quantized_expert_ffn_gemm_b200 as moe
        moe.lib()
    return _fn[name]


def _call(name: str, dev: torch.device, *args):
    fn = _fn.get(name) or _entry(name)
    i = dev.index
    if i == _device():
        code = fn(*args, _stream_of(i))
    else:
        with torch.cuda.device(dev):
            code = fn(*args, _stream_of(i))
    if code:
        raise _MoeError(name, code)


_Tensor = torch.Tensor


def _want(name: str, t, dtypes, shape, dev=None):
    """Refuses a tensor that is not a contiguous CUDA tensor of these types and this shape (None: any size)."""
    if not isinstance(t, _Tensor):
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


def _same(name: str, t, dtypes, shape, dev):
    """_want for a known shape on the call's (CUDA) device, in the order that is quick when all is well."""
    if not (isinstance(t, _Tensor) and t.dtype in dtypes and t.shape == shape and t.device == dev and t.is_contiguous()):
        _want(name, t, dtypes, shape, dev)


def _matrix(name: str, t, dtypes, dev=None):
    """_want for two dimensions of any size: their sizes."""
    if not (isinstance(t, _Tensor) and t.dtype in dtypes and t.is_cuda and t.dim() == 2 and t.is_contiguous() and
            (dev is None or t.device == dev)):
        _want(name, t, dtypes, (None, None), dev)
    return t.shape


_FLOATS = tuple(TYPE_OF)
_F32, _I32, _U8 = (torch.float32,), (torch.int32,), (torch.uint8,)
_empty, _empty_like, _f32, _i32, _u8 = torch.empty, torch.empty_like, torch.float32, torch.int32, torch.uint8


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
    return int(_entry("moe_block_workspace_bytes")(T, k, E, H))


# ----------------------------------------------------------------------------- the norms around a block
def _gate(gate, T, H, dev):
    if gate is None:
        return GATE_NONE
    if isinstance(gate, _Tensor) and gate.dim() == 2:
        _same("gate", gate, _F32, (T, 1), dev)
        return GATE_TOKEN
    _same("gate", gate, _F32, (H,), dev)
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
    T, H = _matrix("r", r, _FLOATS)
    dev = r.device
    if y is not None:
        _same("y", y, _FLOATS, (T, H), dev)
    for n, t in (("post_gain", post_gain), ("pre_gain", pre_gain)):
        if t is not None:
            _same(n, t, _F32, (H,), dev)
    mode = _gate(gate, T, H, dev)
    if pre_norm and u_dtype not in TYPE_OF:
        raise ValueError(f"u_dtype: {u_dtype}, takes {', '.join(str(d) for d in _FLOATS)}")
    if r_out is None:
        r_out = _empty_like(r)
    else:
        _same("r_out", r_out, (r.dtype,), (T, H), dev)
    u = _empty(T, H, dtype=u_dtype, device=dev) if pre_norm else None
    rstd_y = _empty(T, dtype=_f32, device=dev) if y is not None and post_norm else None
    rstd_u = _empty(T, dtype=_f32, device=dev) if pre_norm else None
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
    T, H = _matrix("r_out", r_out, _FLOATS)
    dev = r_out.device
    if dr_out is not None:
        _same("dr_out", dr_out, (r_out.dtype,), (T, H), dev)
    if du is not None:
        _same("du", du, _FLOATS, (T, H), dev)
        _same("rstd_u", rstd_u, _F32, (T,), dev)
    if y is not None:
        _same("y", y, _FLOATS, (T, H), dev)
        if post_norm:
            _same("rstd_y", rstd_y, _F32, (T,), dev)
    for n, t in (("post_gain", post_gain), ("pre_gain", pre_gain)):
        if t is not None:
            _same(n, t, _F32, (H,), dev)
    mode = _gate(gate, T, H, dev)
    ws_ptr, ws_bytes = _ws(ws, dev)
    out = {"dr": _empty_like(r_out), "dy": None if y is None else _empty_like(y),
           "d_post_gain": None if post_gain is None else _empty_like(post_gain),
           "d_gate": None if gate is None else _empty_like(gate),
           "d_pre_gain": None if pre_gain is None else _empty_like(pre_gain)}
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
    T, k = _matrix("idx", idx, _I32)
    dev = idx.device
    ws_ptr, ws_bytes = _ws(ws, dev)
    counts = _empty(max(E, 1), dtype=_i32, device=dev)
    offsets = _empty(max(E, 1) + 1, dtype=_i32, device=dev)
    row_of = _empty(T, k, dtype=_i32, device=dev)
    src = _empty(T * k, dtype=_i32, device=dev)
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


def _tokens(row_of, T, dev):
    n, k = _matrix("row_of", row_of, _I32, dev)
    if n != T:
        raise ValueError(f"row_of: {n} tokens, x has {T}")
    return k


def dispatch(x: torch.Tensor, row_of: torch.Tensor, offsets: Optional[torch.Tensor] = None,
             rows: Optional[torch.Tensor] = None) -> torch.Tensor:
    """rows[row_of[t,j]] = x[t]: [T*k,H] of x's type. With offsets the rows behind the last kept pair are
    zero, without it they are left as they were (in `rows`, if given)."""
    T, H = _matrix("x", x, _FLOATS)
    dev = x.device
    k = _tokens(row_of, T, dev)
    kept = _kept(offsets, dev)
    if rows is None:
        rows = _empty(T * k, H, dtype=x.dtype, device=dev)
    else:
        _same("rows", rows, (x.dtype,), (T * k, H), dev)
    _call("moe_dispatch", dev, x.data_ptr(), TYPE_OF[x.dtype], T, k, H, row_of.data_ptr(), kept, rows.data_ptr())
    return rows


def collect(rows: torch.Tensor, row_of: torch.Tensor, w: Optional[torch.Tensor] = None,
            residual: Optional[torch.Tensor] = None, dtype: torch.dtype = torch.float32) -> torch.Tensor:
    """y[t] = sum_j w[t,j] rows[row_of[t,j]] + residual[t], of `dtype`. Without w the gradient of dispatch."""
    T, k = _matrix("row_of", row_of, _I32)
    dev = row_of.device
    R, H = _matrix("rows", rows, _FLOATS, dev)
    if R != T * k:
        raise ValueError(f"rows: {R} rows, takes {T * k}, one a pair")
    if w is not None:
        _same("w", w, _F32, (T, k), dev)
    if residual is not None:
        _same("residual", residual, _F32, (T, H), dev)
    if dtype not in TYPE_OF:
        raise ValueError(f"dtype: {dtype}, takes {', '.join(str(d) for d in _FLOATS)}")
    y = _empty(T, H, dtype=dtype, device=dev)
    _call("moe_collect", dev, rows.data_ptr(), TYPE_OF[rows.dtype], T, k, H, row_of.data_ptr(), _ptr(w), _ptr(residual),
          y.data_ptr(), TYPE_OF[dtype])
    return y


def collect_backward(dy: torch.Tensor, rows: torch.Tensor, row_of: torch.Tensor, w: Optional[torch.Tensor] = None,
                     offsets: Optional[torch.Tensor] = None):
    """Gradients of collect for dy [T,H]: (d_rows of rows' type, d_w fp32 [T,k], None without w)."""
    T, k = _matrix("row_of", row_of, _I32)
    dev = row_of.device
    R, H = _matrix("rows", rows, _FLOATS, dev)
    if R != T * k:
        raise ValueError(f"rows: {R} rows, takes {T * k}, one a pair")
    _same("dy", dy, _FLOATS, (T, H), dev)
    if w is not None:
        _same("w", w, _F32, (T, k), dev)
    kept = _kept(offsets, dev)
    d_rows = _empty_like(rows)
    d_w = None if w is None else _empty_like(w)
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
        T, K = _matrix("x", x, _FLOATS)
        dev = x.device
        k = _tokens(row_of, T, dev)
        kept, lead = _kept(offsets, dev), (T * k,)
    codes = _empty(*lead, K // 2, dtype=_u8, device=dev)
    scales = _empty(*lead, K // 32, dtype=_u8, device=dev)
    _call("moe_mx4_quantize", dev, x.data_ptr(), TYPE_OF[x.dtype], T, K, _ptr(row_of), k, kept, codes.data_ptr(),
          scales.data_ptr())
    return Mx4(codes, scales)


def _mx4(name, q, dev=None):
    """(leading sizes, K) of MXFP4 rows."""
    codes, scales = q
    if not isinstance(codes, _Tensor) or codes.dim() < 1:
        raise ValueError(f"{name}.codes: takes a tensor [..., K/2]")
    *lead, half = codes.shape
    if half % 16:
        raise ValueError(f"{name}.codes: K = {2 * half} is not a multiple of 32")
    if not codes.is_cuda or (dev is not None and codes.device != dev) or codes.dtype != _u8 or not codes.is_contiguous():
        _want(name + ".codes", codes, _U8, tuple(codes.shape), dev)
    _same(name + ".scales", scales, _U8, (*lead, half // 16), codes.device)
    return lead, 2 * half


def mx4_dequantize(q: Mx4, dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """The values of MXFP4 rows, [..., K] of `dtype`."""
    lead, K = _mx4("q", q)
    if dtype not in TYPE_OF:
        raise ValueError(f"dtype: {dtype}, takes {', '.join(str(d) for d in _FLOATS)}")
    rows = 1
    for n in lead:
        rows *= n
    out = _empty(*lead, K, dtype=dtype, device=q.codes.device)
    _call("moe_mx4_dequantize", out.device, q.codes.data_ptr(), q.scales.data_ptr(), rows, K, out.data_ptr(),
          TYPE_OF[dtype])
    return out


def mx4_product(a: Mx4, w: Mx4, offsets: Optional[torch.Tensor] = None, *, up: Optional[Mx4] = None,
                dtype: torch.dtype = torch.float16, ws=None) -> torch.Tensor:
    """out[r] = a[r] w[g]^T for the rows offsets[g] <= r < offsets[g+1], [rows,N] fp16 or bf16; with up
    silu(a w^T) * (a up^T). a: [rows,K]; w, up: [E,N,K]; offsets int32 [E+1] as sort_pairs gives it, or
    None for E = 1. Rows behind offsets[E] become zero."""
    lead, K = _mx4("a", a)
    if len(lead) != 1:
        raise ValueError(f"a: takes [rows, K], got {len(lead) + 1} dimensions")
    n_rows, dev = lead[0], a.codes.device
    shape = _mx4("w", w, dev)
    if len(shape[0]) != 2 or shape[1] != K:
        raise ValueError(f"w: takes [E, N, {K}], got {(*shape[0], shape[1])}")
    if up is not None and _mx4("up", up, dev) != shape:
        raise ValueError("up: another shape than w")
    E, N = shape[0]
    if offsets is not None:
        _same("offsets", offsets, _I32, (E + 1,), dev)
    if dtype not in TYPE_OF:
        raise ValueError(f"dtype: {dtype}, takes {torch.float16}, {torch.bfloat16}")
    ws_ptr, ws_bytes = _ws(ws, dev)
    wm = Mx4Mat(E, N, K, w.codes.data_ptr(), w.scales.data_ptr())
    um = None if up is None else Mx4Mat(E, N, K, up.codes.data_ptr(), up.scales.data_ptr())
    out = _empty(n_rows, N, dtype=dtype, device=dev)
    _call("moe_mx4_product", dev, a.codes.data_ptr(), a.scales.data_ptr(), n_rows, _ptr(offsets), E,
          ctypes.addressof(wm), None if um is None else ctypes.addressof(um), out.data_ptr(), TYPE_OF[dtype], ws_ptr,
          ws_bytes)
    return out
