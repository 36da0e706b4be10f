// C-ABI entry points of the block operators (include/moe_ffn.h): argument checks on the host, then the
// launches of block_norm.cu, pairs.cu and mx4.cu. As everywhere in the library nothing is enqueued by a
// call that is refused, and no call allocates or synchronises.
#include "block.cuh"

using namespace moe;

namespace {

inline bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }  // NULL is aligned
inline moe_status cuda_status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }
inline bool type_ok(int t) { return t == MOE_F32 || t == MOE_F16 || t == MOE_BF16; }

template <class... P>
bool all_aligned(P... p) {
  return (aligned16(p) && ...);
}

moe_status width_status(int n) {
  if (n > 0 && n % 64 == 0 && n <= 16384) return MOE_OK;
  return n > 0 && n % 32 == 0 ? MOE_ERR_UNSUPPORTED : MOE_ERR_INVALID_ARG;
}

bool pairs_ok(int T, int k) { return T >= 0 && k >= 1 && k <= kMaxK && (long long)T * k <= INT32_MAX; }

// a gate for each mode but none; no tokens' gates may be no memory at all
bool gate_ok(int mode, const float *gate, int T) {
  if (mode == MOE_GATE_NONE) return !gate;
  return (mode == MOE_GATE_CHANNEL || mode == MOE_GATE_TOKEN) && (gate || (mode == MOE_GATE_TOKEN && T == 0));
}

// Scratch lies behind the whole control area: what the decode kernel keeps there from one launch to the next (its launch
// counts, words tagged with them) stays valid, so a workspace may serve layers and these operators in turn.
constexpr size_t kScratch = (kControlBytes + 255) / 256 * 256;
size_t sort_bytes(int T, int k, int E) { return kScratch + sort_pairs_scratch((long long)T * k, E); }
size_t norm_grad_bytes(int T, int H) { return kScratch + block_norm_grad_scratch(T, H); }

moe_status check_mx4(const moe_mx4_mat &m, int E, int N, int K) {
  if (m.n_experts != E || m.rows != N || m.K != K || !m.codes || !m.scales) return MOE_ERR_INVALID_ARG;
  return all_aligned(m.codes, m.scales) ? MOE_OK : MOE_ERR_ALIGNMENT;
}

}  // namespace

extern "C" {

size_t moe_block_workspace_bytes(int32_t T, int32_t k, int32_t E, int32_t H) {
  if (!pairs_ok(T, k) || E < 1 || E > kMaxE || k > E || width_status(H) != MOE_OK) return 0;
  const size_t sort = sort_bytes(T, k, E), norm = norm_grad_bytes(T, H);
  return align_up(sort > norm ? sort : norm, 256);
}

moe_status moe_block_norm(const void *r, int32_t r_type, const void *y, int32_t y_type, int32_t T, int32_t H,
                          int32_t post_norm, const float *post_gain, const float *gate, int32_t gate_mode,
                          float res_scale, float eps, const float *pre_gain, void *r_out, void *u, int32_t u_type,
                          float *rstd_y, float *rstd_u, void *stream) {
  const moe_status st = width_status(H);
  if (st != MOE_OK) return st;
  if (T < 0 || !(eps >= 0.0f) || !type_ok(r_type) || (y && !type_ok(y_type)) || (u && !type_ok(u_type)))
    return MOE_ERR_INVALID_ARG;
  if (!gate_ok(gate_mode, gate, T)) return MOE_ERR_INVALID_ARG;
  if (!y && T > 0 && (post_gain || gate || rstd_y)) return MOE_ERR_INVALID_ARG;
  if ((rstd_y && !post_norm) || (!u && T > 0 && (pre_gain || rstd_u))) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (!r || (!r_out && !u)) return MOE_ERR_INVALID_ARG;
  if (!all_aligned(r, y, post_gain, gate, pre_gain, r_out, u, rstd_y, rstd_u)) return MOE_ERR_ALIGNMENT;
  const BlockNormArgs a{r,    y,         r_type,    y_type, T,     H, post_norm ? 1 : 0, post_gain, gate, pre_gain,
                        gate_mode, res_scale, eps, r_out,  u, u_type, rstd_y, rstd_u};
  return cuda_status(launch_block_norm(a, (cudaStream_t)stream));
}

moe_status moe_block_norm_backward(const void *dr_out, const void *du, int32_t u_type, const void *r_out,
                                   int32_t r_type, const float *rstd_u, const void *y, int32_t y_type,
                                   const float *rstd_y, int32_t T, int32_t H, int32_t post_norm,
                                   const float *post_gain, const float *gate, int32_t gate_mode, float res_scale,
                                   const float *pre_gain, void *dr, void *dy, float *d_post_gain, float *d_gate,
                                   float *d_pre_gain, void *ws, size_t ws_bytes, void *stream) {
  const moe_status st = width_status(H);
  if (st != MOE_OK) return st;
  if (T < 0 || !type_ok(r_type) || (du && !type_ok(u_type)) || (y && !type_ok(y_type))) return MOE_ERR_INVALID_ARG;
  if (!gate_ok(gate_mode, gate, T)) return MOE_ERR_INVALID_ARG;
  if (d_gate && !gate) return MOE_ERR_INVALID_ARG;
  if (!all_aligned(dr_out, du, r_out, rstd_u, y, rstd_y, post_gain, gate, pre_gain, dr, dy) ||
      !all_aligned(d_post_gain, d_gate, d_pre_gain))
    return MOE_ERR_ALIGNMENT;
  cudaStream_t s = (cudaStream_t)stream;
  if (T == 0) {
    const size_t n = (size_t)H * 4;
    cudaError_t e = cudaSuccess;
    if (d_post_gain) e = cudaMemsetAsync(d_post_gain, 0, n, s);
    if (e == cudaSuccess && d_pre_gain) e = cudaMemsetAsync(d_pre_gain, 0, n, s);
    if (e == cudaSuccess && d_gate && gate_mode == MOE_GATE_CHANNEL) e = cudaMemsetAsync(d_gate, 0, n, s);
    return cuda_status(e);
  }
  if ((!dr_out && !du) || !dr || (du && (!r_out || !rstd_u)) || (y && post_norm && !rstd_y)) return MOE_ERR_INVALID_ARG;
  if ((y != nullptr) != (dy != nullptr)) return MOE_ERR_INVALID_ARG;
  if (!y && (post_gain || gate || d_post_gain)) return MOE_ERR_INVALID_ARG;
  if (!du && (pre_gain || d_pre_gain)) return MOE_ERR_INVALID_ARG;
  if (!ws || ws_bytes < norm_grad_bytes(T, H)) return MOE_ERR_WORKSPACE;
  if (!aligned16(ws)) return MOE_ERR_ALIGNMENT;
  const BlockNormGradArgs a{dr_out, du,     u_type,    r_out, y,        r_type,    y_type, T,  H,           post_norm ? 1 : 0,
                            rstd_u, rstd_y, post_gain, gate,  pre_gain, gate_mode, res_scale, dr, dy, d_post_gain,
                            d_gate, d_pre_gain};
  float *scratch = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + kScratch);
  return cuda_status(launch_block_norm_grad(a, scratch, s));
}

moe_status moe_sort_pairs(const int32_t *idx, int32_t T, int32_t k, int32_t E, int32_t *counts, int32_t *offsets,
                          int32_t *row_of, int32_t *src, void *ws, size_t ws_bytes, void *stream) {
  if (!pairs_ok(T, k) || E < 1 || E > kMaxE || k > E) return MOE_ERR_INVALID_ARG;
  if (!counts || !offsets) return MOE_ERR_INVALID_ARG;
  if (!all_aligned(idx, counts, offsets, row_of, src)) return MOE_ERR_ALIGNMENT;
  cudaStream_t s = (cudaStream_t)stream;
  if (T == 0) {
    cudaError_t e = cudaMemsetAsync(counts, 0, (size_t)E * 4, s);
    if (e == cudaSuccess) e = cudaMemsetAsync(offsets, 0, (size_t)(E + 1) * 4, s);
    return cuda_status(e);
  }
  if (!idx || !row_of || !src) return MOE_ERR_INVALID_ARG;
  if (!ws || ws_bytes < sort_bytes(T, k, E)) return MOE_ERR_WORKSPACE;
  if (!aligned16(ws)) return MOE_ERR_ALIGNMENT;
  return cuda_status(launch_sort_pairs(idx, T, k, E, counts, offsets, row_of, src,
                                       reinterpret_cast<int32_t *>(static_cast<uint8_t *>(ws) + kScratch),
                                       static_cast<Ctrl *>(ws), s));
}

moe_status moe_dispatch(const void *x, int32_t type, int32_t T, int32_t k, int32_t H, const int32_t *row_of,
                        const int32_t *kept, void *rows, void *stream) {
  const moe_status st = width_status(H);
  if (st != MOE_OK) return st;
  if (!pairs_ok(T, k) || !type_ok(type)) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (!x || !row_of || !rows) return MOE_ERR_INVALID_ARG;
  if (!all_aligned(x, row_of, rows) || ((uintptr_t)kept & 3u)) return MOE_ERR_ALIGNMENT;
  return cuda_status(launch_dispatch(x, type, T, k, H, row_of, kept, rows, (cudaStream_t)stream));
}

moe_status moe_collect(const void *rows, int32_t type, int32_t T, int32_t k, int32_t H, const int32_t *row_of,
                       const float *w, const float *residual, void *y, int32_t y_type, void *stream) {
  const moe_status st = width_status(H);
  if (st != MOE_OK) return st;
  if (!pairs_ok(T, k) || !type_ok(type) || !type_ok(y_type)) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (!rows || !row_of || !y) return MOE_ERR_INVALID_ARG;
  if (!all_aligned(rows, row_of, w, residual, y)) return MOE_ERR_ALIGNMENT;
  return cuda_status(launch_collect(rows, type, T, k, H, row_of, w, residual, y, y_type, (cudaStream_t)stream));
}

moe_status moe_collect_backward(const void *dy, int32_t dy_type, const void *rows, int32_t type, int32_t T, int32_t k,
                                int32_t H, const int32_t *row_of, const float *w, const int32_t *kept, void *d_rows,
                                float *d_w, void *stream) {
  const moe_status st = width_status(H);
  if (st != MOE_OK) return st;
  if (!pairs_ok(T, k) || !type_ok(type) || !type_ok(dy_type)) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (!dy || !row_of || (!d_rows && !d_w) || (d_w && !rows)) return MOE_ERR_INVALID_ARG;
  if (!all_aligned(dy, rows, row_of, w, d_rows, d_w) || ((uintptr_t)kept & 3u)) return MOE_ERR_ALIGNMENT;
  return cuda_status(launch_collect_grad(dy, dy_type, rows, type, T, k, H, row_of, w, kept, d_rows, d_w,
                                         (cudaStream_t)stream));
}

moe_status moe_mx4_quantize(const void *x, int32_t type, int32_t T, int32_t K, const int32_t *row_of, int32_t k,
                            const int32_t *kept, uint8_t *codes, uint8_t *scales, void *stream) {
  const moe_status st = width_status(K);
  if (st != MOE_OK) return st;
  if (!type_ok(type) || !pairs_ok(T, row_of ? k : 1) || (kept && !row_of && T > 0)) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (!x || !codes || !scales) return MOE_ERR_INVALID_ARG;
  if (!all_aligned(x, row_of, codes, scales) || ((uintptr_t)kept & 3u)) return MOE_ERR_ALIGNMENT;
  return cuda_status(launch_mx4_quantize(x, type, T, K, row_of, k, kept, codes, scales, (cudaStream_t)stream));
}

moe_status moe_mx4_dequantize(const uint8_t *codes, const uint8_t *scales, int32_t rows, int32_t K, void *out,
                              int32_t type, void *stream) {
  const moe_status st = width_status(K);
  if (st != MOE_OK) return st;
  if (rows < 0 || !type_ok(type)) return MOE_ERR_INVALID_ARG;
  if (rows == 0) return MOE_OK;
  if (!codes || !scales || !out) return MOE_ERR_INVALID_ARG;
  if (!all_aligned(codes, scales, out)) return MOE_ERR_ALIGNMENT;
  return cuda_status(launch_mx4_dequantize(codes, scales, rows, K, out, type, (cudaStream_t)stream));
}

moe_status moe_mx4_product(const uint8_t *a_codes, const uint8_t *a_scales, int32_t n_rows, const int32_t *offsets,
                           int32_t E, const moe_mx4_mat *w, const moe_mx4_mat *up, void *out, int32_t out_type,
                           void *ws, size_t ws_bytes, void *stream) {
  if (!w || E < 1 || E > kMaxE || n_rows < 0 || !type_ok(out_type) || (!offsets && E != 1)) return MOE_ERR_INVALID_ARG;
  moe_status st = width_status(w->K);
  if (st == MOE_OK) st = width_status(w->rows);
  if (st != MOE_OK) return st;
  if ((st = check_mx4(*w, E, w->rows, w->K)) != MOE_OK) return st;
  if (up && (st = check_mx4(*up, E, w->rows, w->K)) != MOE_OK) return st;
  if (out_type == MOE_F32) return MOE_ERR_UNSUPPORTED;
  if (n_rows == 0) return MOE_OK;
  if (!a_codes || !a_scales || !out) return MOE_ERR_INVALID_ARG;
  if (!all_aligned(a_codes, a_scales, offsets, out)) return MOE_ERR_ALIGNMENT;
  if (!ws || ws_bytes < kCtrlStride) return MOE_ERR_WORKSPACE;
  if (!aligned16(ws)) return MOE_ERR_ALIGNMENT;
  const Mx4ProductArgs a{a_codes, a_scales, n_rows, w->K, w->rows, E, offsets, w->codes, w->scales,
                         up ? up->codes : nullptr, up ? up->scales : nullptr, out, out_type, static_cast<Ctrl *>(ws)};
  return cuda_status(launch_mx4_product(a, (cudaStream_t)stream));
}

}  // extern "C"
