"""The block operators of include/moe_ffn.h for torch tensors: the norms around a block, pairs sorted by
expert and collected again (each with its gradient), MXFP4 rows and their product per expert.

Only arguments are marshalled on the way to the library, in the compiled module _bind (csrc/bind.cpp): these
operators are called with a microsecond or two of work for the GPU, and ctypes alone took longer. Tensors are
contiguous CUDA tensors of one device; a call runs on that device's current stream, whichever device is
current, and allocates its outputs unless they are given (a call's small ones as parts of one allocation). A
tensor of another type, shape, layout or device than the call takes raises ValueError; what the library refuses
raises MoeError.

No call records an autograd graph: the gradients are entry points, to be called from a torch.autograd.Function. Where
torch records and an input requires a gradient, a backward pass that comes to the call raises RuntimeError; a buffer
to write (r_out, rows) goes by torch's rules for tensors changed in place. The codes of mx4_quantize are integers and
take no gradient.
"""
from __future__ import annotations

import ctypes
import os
from typing import NamedTuple, Optional

import torch

BIND_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_bind.so")

F32, F16, BF16 = 0, 1, 2
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


_b = None  # the compiled binding, loaded by the first call


def _load():
    global _b
    import quantized_expert_ffn_gemm_b200 as moe
    moe.lib()  # says what to build where the library is missing
    if not os.path.exists(BIND_PATH):
        raise RuntimeError(f"{BIND_PATH} not found: build it with `python -m quantized_expert_ffn_gemm_b200.build`")
    from . import _bind, build
    built_for, here = getattr(_bind, "built_for", "an older tree"), build.bind_built_for()
    if built_for != here:
        raise RuntimeError(f"{BIND_PATH} was built for {built_for}, this is {here}: build it with "
                           "`python -m quantized_expert_ffn_gemm_b200.build`")
    _bind.init_errors(moe.MoeError, torch.cuda.OutOfMemoryError)
    _b = _bind
    return _b


def bind(lib):
    """Argument types of the C entry points, set once on the loaded library (for calls through ctypes)."""
    lib.moe_block_workspace_bytes.restype = _Z
    lib.moe_block_workspace_bytes.argtypes = [_I] * 4
    for name, args in _ARGS.items():
        getattr(lib, name).restype = _I
        getattr(lib, name).argtypes = args


def block_workspace_bytes(T: int, k: int = 1, E: int = 1, H: int = 64) -> int:
    """Bytes of a Workspace that suffices for every block operator of these sizes (0: sizes not taken)."""
    import quantized_expert_ffn_gemm_b200 as moe
    if not all(0 <= n < 1 << 31 for n in (T, k, E, H)):  # ctypes would cut them to 32 bits
        return 0
    return int(moe.lib().moe_block_workspace_bytes(T, k, E, H))


# ----------------------------------------------------------------------------- the norms around a block
def block_norm(r: torch.Tensor, y: Optional[torch.Tensor] = None, *, post_gain: Optional[torch.Tensor] = None,
               gate: Optional[torch.Tensor] = None, res_scale: float = 1.0, pre_gain: Optional[torch.Tensor] = None,
               eps: float = 1e-6, post_norm: bool = True, pre_norm: bool = True, u_dtype: torch.dtype = torch.bfloat16,
               r_out: Optional[torch.Tensor] = None):
    """r' = res_scale r + gate post_gain N(y) and u = pre_gain N(r'): (r', u, rstd_y, rstd_u).

    r [T,H], y [T,H] or None, each fp32, fp16 or bf16; gains fp32 [H]; gate fp32 [H] (a channel) or [T,1] (a
    token). r' has r's type (r_out may be r, to update the stream in place); u has u_dtype. Without
    pre_norm u and rstd_u are None, without y or post_norm rstd_y is; the statistics are what
    block_norm_backward needs."""
    return (_b or _load()).block_norm(r, y, post_gain, gate, res_scale, pre_gain, eps, post_norm, pre_norm, u_dtype, r_out)


def block_norm_backward(dr_out: Optional[torch.Tensor], du: Optional[torch.Tensor], r_out: torch.Tensor,
                        rstd_u: Optional[torch.Tensor], y: Optional[torch.Tensor] = None,
                        rstd_y: Optional[torch.Tensor] = None, *, post_gain: Optional[torch.Tensor] = None,
                        gate: Optional[torch.Tensor] = None, res_scale: float = 1.0,
                        pre_gain: Optional[torch.Tensor] = None, post_norm: bool = True, ws=None) -> dict:
    """Gradients of block_norm: a dict of dr, dy, d_post_gain, d_gate and d_pre_gain.

    dr_out and du reach r' and u (None: nothing does; not both); r_out, rstd_u, y and rstd_y as the forward call
    took and returned them (rstd_u is not read without du). An entry is None where block_norm had no such
    argument; without du d_pre_gain is zero."""
    dr, dy, d_post, d_gate, d_pre = (_b or _load()).block_norm_backward(
        dr_out, du, r_out, rstd_u, y, rstd_y, post_gain, gate, res_scale, pre_gain, post_norm, ws)
    return {"dr": dr, "dy": dy, "d_post_gain": d_post, "d_gate": d_gate, "d_pre_gain": d_pre}


# ----------------------------------------------------------------------------- pairs sorted by expert
def sort_pairs(idx: torch.Tensor, E: int, ws) -> dict:
    """The (token, slot) pairs of idx int32 [T,k] (-1: no expert) in expert order: counts [E], offsets [E+1],
    row_of [T,k] (-1: no row) and src [T*k] (-1 behind the last kept pair), all int32."""
    counts, offsets, row_of, src = (_b or _load()).sort_pairs(idx, E, ws)
    return {"counts": counts, "offsets": offsets, "row_of": row_of, "src": src}


def dispatch(x: torch.Tensor, row_of: torch.Tensor, offsets: Optional[torch.Tensor] = None,
             rows: Optional[torch.Tensor] = None) -> torch.Tensor:
    """rows[row_of[t,j]] = x[t]: [T*k,H] of x's type. With offsets the rows behind the last kept pair are
    zero, without it they are left as they were (in `rows`, if given)."""
    return (_b or _load()).dispatch(x, row_of, offsets, rows)


def collect(rows: torch.Tensor, row_of: torch.Tensor, w: Optional[torch.Tensor] = None,
            residual: Optional[torch.Tensor] = None, dtype: torch.dtype = torch.float32) -> torch.Tensor:
    """y[t] = sum_j w[t,j] rows[row_of[t,j]] + residual[t], of `dtype`. Without w the gradient of dispatch."""
    return (_b or _load()).collect(rows, row_of, w, residual, dtype)


def collect_backward(dy: torch.Tensor, rows: torch.Tensor, row_of: torch.Tensor, w: Optional[torch.Tensor] = None,
                     offsets: Optional[torch.Tensor] = None):
    """Gradients of collect for dy [T,H]: (d_rows of rows' type, d_w fp32 [T,k], None without w). offsets as in
    dispatch."""
    return (_b or _load()).collect_backward(dy, rows, row_of, w, offsets)


# ----------------------------------------------------------------------------- MXFP4
def mx4_quantize(x: torch.Tensor, row_of: Optional[torch.Tensor] = None,
                 offsets: Optional[torch.Tensor] = None) -> Mx4:
    """x [..., K] (fp32, fp16 or bf16) to MXFP4. With row_of int32 [T,k] the quantised token x[t] goes to
    rows row_of[t,:] of T*k rows, as dispatch copies it; offsets as there."""
    return Mx4(*(_b or _load()).mx4_quantize(x, row_of, offsets))


def mx4_dequantize(q: Mx4, dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """The values of MXFP4 rows, [..., K] of `dtype`."""
    return (_b or _load()).mx4_dequantize(q, dtype)


def mx4_product(a: Mx4, w: Mx4, offsets: Optional[torch.Tensor] = None, *, up: Optional[Mx4] = None,
                dtype: torch.dtype = torch.float16, ws=None) -> torch.Tensor:
    """out[r] = a[r] w[g]^T for the rows offsets[g] <= r < offsets[g+1], [rows,N] fp16 or bf16; with up
    silu(a w^T) * (a up^T). a: [rows,K]; w, up: [E,N,K]; offsets int32 [E+1] as sort_pairs gives it, or
    None for E = 1. Rows behind offsets[E] become zero."""
    return (_b or _load()).mx4_product(a, w, offsets, up, dtype, ws)
