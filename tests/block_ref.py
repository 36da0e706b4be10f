"""The block operators' formulas in fp64 (torch, on the CPU), and the error bounds the tests hold the kernels to.

Bounds: u32 = 2^-24 is half a step of fp32, half(t) half a step of a result's type t. A sum of n terms carried
in fp32 in any order is off by at most n u32 sum|terms|; a shorter chain where the kernels' order gives one.
"""
import torch

U32 = 2.0 ** -24


def half(dtype):
    return torch.finfo(dtype).eps / 2


def rounded(value, dtype):
    """What rounding a result near `value` to dtype may add: half a step, or half the smallest subnormal."""
    return half(dtype) * value.abs() + torch.finfo(dtype).smallest_normal * half(dtype)


def close(got, want, bound, what=""):
    """Every element within its bound (both broadcast); NaN and infinities in the same places."""
    got, want = got.detach().double().cpu(), want.double()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    fine = torch.isfinite(want)
    assert torch.equal(fine, torch.isfinite(got)), (what, "finite in other places")
    assert torch.equal(torch.isnan(got), torch.isnan(want)), (what, "NaN in other places")
    over = ((got - want).abs() - bound)[fine]
    if over.numel():
        assert float(over.max()) <= 0, (what, float(over.max()), float((got - want)[fine].abs().max()))


# ----------------------------------------------------------------------------- norms
def norm(v, eps):
    rstd = (v.square().mean(1, keepdim=True) + eps).rsqrt()
    return v * rstd, rstd


def block_norm(r, y=None, post_gain=None, gate=None, res_scale=1.0, pre_gain=None, eps=1e-6, post_norm=True):
    """fp64 inputs -> (r', u, rstd_y [T,1], rstd_u, the magnitude that r' is summed from)."""
    rstd_y = None
    v, mag = res_scale * r, (res_scale * r).abs()
    if y is not None:
        z = y
        if post_norm:
            z, rstd_y = norm(y, eps)
        if post_gain is not None:
            z = z * post_gain
        if gate is not None:
            z = z * gate
        v, mag = v + z, mag + z.abs()
    u, rstd_u = norm(v, eps)
    if pre_gain is not None:
        u = u * pre_gain
    return v, u, rstd_y, rstd_u, mag


def block_norm_grad(dr_out, du, r, rstd_u, y, rstd_y, post_gain, gate, res_scale, pre_gain, post_norm=True):
    """fp64 gradients and, for each, the sum of magnitudes that its rounding errors go by."""
    T, H = r.shape
    one = torch.ones((), dtype=torch.float64)
    g, G = (dr_out, dr_out.abs()) if dr_out is not None else (torch.zeros_like(r), torch.zeros_like(r))
    out, mag = {}, {}
    if du is not None:
        x = r * rstd_u[:, None]
        h = du * (one if pre_gain is None else pre_gain)
        g = g + rstd_u[:, None] * (h - x * (h * x).mean(1, keepdim=True))
        G = G + rstd_u[:, None] * (h.abs() + x.abs() * (h * x).abs().mean(1, keepdim=True))
        out["d_pre_gain"], mag["d_pre_gain"] = (du * x).sum(0), (du * x).abs().sum(0)
    out["dr"], mag["dr"] = res_scale * g, abs(res_scale) * G
    if y is not None:
        rs = rstd_y[:, None] if post_norm else one
        v = y * rs
        pg, gt = one if post_gain is None else post_gain, one if gate is None else gate
        q, Q = g * gt * pg, G * (gt * pg).abs()
        m = (q * v).mean(1, keepdim=True) if post_norm else 0
        M = (Q * v.abs()).mean(1, keepdim=True) if post_norm else 0
        out["dy"], mag["dy"] = rs * (q - v * m), rs * (Q + v.abs() * M)
        out["d_post_gain"], mag["d_post_gain"] = (g * gt * v).sum(0), (G * gt.abs() * v.abs()).sum(0)
        if gate is not None:
            dim = 1 if gate.dim() == 2 else 0
            out["d_gate"] = (g * pg * v).sum(dim, keepdim=dim == 1)
            mag["d_gate"] = (G * pg.abs() * v.abs()).sum(dim, keepdim=dim == 1)
    return out, mag


# ----------------------------------------------------------------------------- pairs
def sort_pairs(idx, E):
    """Plain loop over the pairs in (expert, token, slot) order."""
    T, k = idx.shape
    flat = idx.reshape(-1).tolist()
    order = sorted((e, p) for p, e in enumerate(flat) if 0 <= e < E)
    row_of, src, counts = [-1] * (T * k), [-1] * (T * k), [0] * E
    for row, (e, p) in enumerate(order):
        row_of[p], src[row] = row, p // k
        counts[e] += 1
    offsets = [0]
    for c in counts:
        offsets.append(offsets[-1] + c)
    as32 = lambda v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    return {"counts": as32(counts), "offsets": as32(offsets), "row_of": as32(row_of).view(T, k), "src": as32(src)}


def spread(row_of, rows):
    """rows[row_of[t,j]] with zeros for -1, [T,k,H]."""
    at = row_of.long()
    return torch.where((at >= 0)[..., None], rows[at.clamp(min=0)], torch.zeros((), dtype=rows.dtype))


# ----------------------------------------------------------------------------- MXFP4
GRID = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64)


def mx4_quantize(x):
    """fp64 [rows,K] -> (codes one a value, scale bytes), from the definition: exact in fp64 for fp32 inputs."""
    b = x.unflatten(-1, (-1, 32))
    top = b.abs().amax(-1)
    bad = ~torch.isfinite(b).all(-1)
    exponent = torch.frexp(torch.where(bad | (top == 0), torch.ones_like(top), top)).exponent - 1
    byte = torch.where(top == 0, torch.zeros_like(exponent), (exponent - 2 + 127).clamp(min=0))
    byte = torch.where(bad, torch.full_like(byte, 255), byte)
    a = torch.where(bad[..., None], torch.zeros_like(b), b.abs() * torch.exp2(127.0 - byte.double())[..., None])
    dist = (a[..., None] - GRID).abs()
    best = dist.amin(-1, keepdim=True)
    near = dist == best  # one code, or two at a tie: then the even one
    code = torch.where(near.sum(-1) == 2, (near & (torch.arange(8) % 2 == 0)).int().argmax(-1), near.int().argmax(-1))
    code = code + 8 * (torch.signbit(b) & ~bad[..., None])
    return code.flatten(-2).to(torch.uint8), byte.to(torch.uint8)


def mx4_value(code, byte):
    v = torch.where(code >= 8, -1.0, 1.0) * GRID[(code % 8).long()]
    unit = torch.where(byte == 255, torch.full((), float("nan"), dtype=torch.float64), torch.exp2(byte.double() - 127))
    return (v.unflatten(-1, (-1, 32)) * unit[..., None]).flatten(-2)


def unpack(packed):
    return torch.stack([packed & 15, packed >> 4], -1).flatten(-2)


def pack(code):
    return (code[..., 0::2] | (code[..., 1::2] << 4)).contiguous()


def mx4_values(q):
    return mx4_value(unpack(q.codes.cpu()), q.scales.cpu())


def mx4_product(a, w, offsets, up=None):
    """fp64 values -> (out, the bound of its error before the result's rounding). A step of the tensor cores adds
    64 products to an fp32 sum and may truncate where it would round (two half steps), so K values are off
    by at most (K/64 + 8) steps of sum|a w|; silu's slope is at most 1.1."""
    out = torch.zeros(a.shape[0], w.shape[1], dtype=torch.float64)
    err = torch.zeros_like(out)
    c = (a.shape[1] / 64 + 8) * 4 * U32
    for g in range(w.shape[0]):
        s = slice(int(offsets[g]), int(offsets[g + 1]))
        p, P = a[s] @ w[g].T, c * (a[s].abs() @ w[g].abs().T)
        if up is None:
            out[s], err[s] = p, P
        else:
            q, Q = a[s] @ up[g].T, c * (a[s].abs() @ up[g].abs().T)
            silu = p / (1 + torch.exp(-p))
            out[s] = silu * q
            err[s] = 1.1 * P * (q.abs() + Q) + silu.abs() * Q + 8 * U32 * (silu * q).abs()
    return out, err
