// The norms around a block, in one pass over its rows, and their gradient.
//
//   forward   z = gate * post_gain * N(y),  r' = res_scale * r + z,  u = pre_gain * N(r')
//             N(v) = v * rstd(v),  rstd(v) = 1 / sqrt(mean_h v_h^2 + eps)
// closes one block (its output y normalised, gated and added to the scaled residual stream) and
// opens the next (u is its input); either half can be left out. Written apart the two halves read and
// write the stream twice; here r and y are read once and r' and u written once.
//
//   backward  with x = r' rstd_u, v = y rstd_y, h = du * pre_gain:
//             g = dr' + rstd_u (h - x mean(h x))            the stream's whole gradient
//             dr = res_scale g;   q = g * gate * post_gain;   dy = rstd_y (q - v mean(q v))
//             d_pre_gain = sum_t du x;  d_post_gain = sum_t g gate v;  d_gate = sum g post_gain v
// (sum over t for a gate a channel, over h for a gate a token). With A = sum_t g v (a token's gate
// folded in), d_post_gain = gate A and d_gate = post_gain A for channel gates, so two sums a channel
// are carried whatever the gate.
#include "block.cuh"

namespace moe {

namespace {

constexpr int kMaxWarps = 32;

// Sum over the TPR threads of a row; every thread of the block calls it. `buf` is not reused before
// another block_sum's barrier has passed (callers alternate two).
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float *buf) {
  v = warp_sum(v);
  if constexpr (TPR > 32) {
    const int warp = threadIdx.x >> 5, w0 = (threadIdx.x / TPR) * (TPR / 32);
    if ((threadIdx.x & 31) == 0) buf[warp] = v;
    __syncthreads();
    v = 0.0f;
#pragma unroll
    for (int i = 0; i < TPR / 32; ++i) v += buf[w0 + i];
  }
  return v;
}

__device__ __forceinline__ void ones8(float v[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = 1.0f;
}

// TPR threads a row, CH chunks of eight values a thread
template <int TPR, int CH>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR) block_norm_kernel(const BlockNormArgs a) {
  constexpr int kThreads = TPR < 256 ? 256 : TPR, kRows = kThreads / TPR;
  __shared__ float s_a[kMaxWarps], s_b[kMaxWarps];
  const int sub = threadIdx.x / TPR, lane = threadIdx.x % TPR, H8 = a.H >> 3;
  const float inv_h = 1.0f / (float)a.H;
  for (long long row0 = (long long)blockIdx.x * kRows; row0 < a.T; row0 += (long long)gridDim.x * kRows) {
    const long long t = row0 + sub;
    const bool live = t < a.T;
    const size_t base = (size_t)t * a.H;
    Raw8 rr[CH], ry[CH];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int i = lane + c * TPR;
      if (live && i < H8) {
        rr[c] = load_raw8(a.r, a.r_type, base + 8 * i);
        if (a.y) ry[c] = load_raw8(a.y, a.y_type, base + 8 * i);
      }
    }
    float rstd_y = 1.0f;
    if (a.y && a.post_norm) {
      float ss = 0.0f;
#pragma unroll
      for (int c = 0; c < CH; ++c)
        if (live && lane + c * TPR < H8) {
          float v[8];
          raw8_to_float(ry[c], a.y_type, v);
#pragma unroll
          for (int q = 0; q < 8; ++q) ss = fmaf(v[q], v[q], ss);
        }
      ss = row_sum<TPR>(ss, s_a);
      rstd_y = 1.0f / sqrtf(ss * inv_h + a.eps);
      if (a.rstd_y && live && lane == 0) a.rstd_y[t] = rstd_y;
    }
    const float tok = (a.gate_mode == MOE_GATE_TOKEN && live) ? a.gate[t] : 1.0f;
    float v[CH][8], ss = 0.0f;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int i = lane + c * TPR;
      if (!(live && i < H8)) continue;
      raw8_to_float(rr[c], a.r_type, v[c]);
#pragma unroll
      for (int q = 0; q < 8; ++q) v[c][q] *= a.res_scale;
      if (a.y) {
        float z[8], g[8];
        raw8_to_float(ry[c], a.y_type, z);
#pragma unroll
        for (int q = 0; q < 8; ++q) z[q] *= rstd_y;
        if (a.post_gain) {
          load8(a.post_gain, MOE_F32, 8 * i, g);
#pragma unroll
          for (int q = 0; q < 8; ++q) z[q] *= g[q];
        }
        if (a.gate_mode == MOE_GATE_CHANNEL) {
          load8(a.gate, MOE_F32, 8 * i, g);
#pragma unroll
          for (int q = 0; q < 8; ++q) z[q] *= g[q];
        }
#pragma unroll
        for (int q = 0; q < 8; ++q) v[c][q] = fmaf(tok, z[q], v[c][q]);
      }
      if (a.r_out) store8(a.r_out, a.r_type, base + 8 * i, v[c]);
#pragma unroll
      for (int q = 0; q < 8; ++q) ss = fmaf(v[c][q], v[c][q], ss);
    }
    if (a.u) {  // the norm of r' before its rounding to the stream's type
      ss = row_sum<TPR>(ss, s_b);
      const float rstd_u = 1.0f / sqrtf(ss * inv_h + a.eps);
      if (a.rstd_u && live && lane == 0) a.rstd_u[t] = rstd_u;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int i = lane + c * TPR;
        if (!(live && i < H8)) continue;
        float g[8];
        ones8(g);
        if (a.pre_gain) load8(a.pre_gain, MOE_F32, 8 * i, g);
#pragma unroll
        for (int q = 0; q < 8; ++q) g[q] *= v[c][q] * rstd_u;
        store8(a.u, a.u_type, base + 8 * i, g);
      }
    }
    if constexpr (TPR > 32) {
      if (!(a.u && a.y && a.post_norm)) __syncthreads();  // one reduction a row: its buffer is read before it is reused
    }
  }
}

// HOLD: the row's values stay in registers between the two reductions; otherwise (long rows) they are
// read again, from L2
template <int TPR, int CH, bool HOLD>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR) block_norm_grad_kernel(const BlockNormGradArgs a,
                                                                               float *__restrict__ part) {
  constexpr int kThreads = TPR < 256 ? 256 : TPR, kRows = kThreads / TPR;
  __shared__ float s_a[kMaxWarps], s_b[kMaxWarps];
  const int sub = threadIdx.x / TPR, lane = threadIdx.x % TPR, H8 = a.H >> 3;
  const float inv_h = 1.0f / (float)a.H;
  float sum_v[CH][8], sum_x[CH][8];  // sum over this thread's rows of g v (a token's gate folded in) and du x
#pragma unroll
  for (int c = 0; c < CH; ++c)
#pragma unroll
    for (int q = 0; q < 8; ++q) sum_v[c][q] = sum_x[c][q] = 0.0f;
  for (long long row0 = (long long)blockIdx.x * kRows; row0 < a.T; row0 += (long long)gridDim.x * kRows) {
    const long long t = row0 + sub;
    const bool live = t < a.T;
    const size_t base = (size_t)t * a.H;
    const float rstd_u = (a.du && live) ? a.rstd_u[t] : 0.0f;
    const float rstd_y = (a.y && a.post_norm && live) ? a.rstd_y[t] : 1.0f;
    const float tok = (a.gate_mode == MOE_GATE_TOKEN && live) ? a.gate[t] : 1.0f;
    Raw8 rr[HOLD ? CH : 1], ru[HOLD ? CH : 1], rd[HOLD ? CH : 1], ry[HOLD ? CH : 1];
    auto fetch = [&](int c, int i) {
      const int s = HOLD ? c : 0;
      if (a.du) {
        rr[s] = load_raw8(a.r, a.r_type, base + 8 * i);
        ru[s] = load_raw8(a.du, a.u_type, base + 8 * i);
      }
      if (a.dr_out) rd[s] = load_raw8(a.dr_out, a.r_type, base + 8 * i);
      if (a.y) ry[s] = load_raw8(a.y, a.y_type, base + 8 * i);
    };
    if constexpr (HOLD) {
#pragma unroll
      for (int c = 0; c < CH; ++c)
        if (live && lane + c * TPR < H8) fetch(c, lane + c * TPR);
    }
    // x = r' rstd_u and h = du pre_gain of chunk c
    auto xh = [&](int c, int i, float x[8], float u[8], float h[8]) {
      const int s = HOLD ? c : 0;
      raw8_to_float(rr[s], a.r_type, x);
      raw8_to_float(ru[s], a.u_type, u);
      ones8(h);
      if (a.pre_gain) load8(a.pre_gain, MOE_F32, 8 * i, h);
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        x[q] *= rstd_u;
        h[q] *= u[q];
      }
    };
    float m_u = 0.0f;
    if (a.du) {
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int i = lane + c * TPR;
        if (!(live && i < H8)) continue;
        if constexpr (!HOLD) fetch(c, i);
        float x[8], u[8], h[8];
        xh(c, i, x, u, h);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          m_u = fmaf(h[q], x[q], m_u);
          sum_x[c][q] = fmaf(u[q], x[q], sum_x[c][q]);
        }
      }
      m_u = row_sum<TPR>(m_u, s_a) * inv_h;
    }
    // g: the stream's gradient of chunk c
    auto grad = [&](int c, int i, float g[8]) {
      const int s = HOLD ? c : 0;
      if (a.dr_out) {
        raw8_to_float(rd[s], a.r_type, g);
      } else {
#pragma unroll
        for (int q = 0; q < 8; ++q) g[q] = 0.0f;
      }
      if (a.du) {
        float x[8], u[8], h[8];
        xh(c, i, x, u, h);
#pragma unroll
        for (int q = 0; q < 8; ++q) g[q] = fmaf(rstd_u, fmaf(-x[q], m_u, h[q]), g[q]);
      }
    };
    // f: gate (a channel's) times post_gain of chunk c
    auto factor = [&](int i, float f[8]) {
      ones8(f);
      if (a.post_gain) load8(a.post_gain, MOE_F32, 8 * i, f);
      if (a.gate_mode == MOE_GATE_CHANNEL) {
        float g[8];
        load8(a.gate, MOE_F32, 8 * i, g);
#pragma unroll
        for (int q = 0; q < 8; ++q) f[q] *= g[q];
      }
    };
    float m_y = 0.0f;
    float gh[HOLD ? CH : 1][8];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int i = lane + c * TPR, s = HOLD ? c : 0;
      if (!(live && i < H8)) continue;
      if constexpr (!HOLD) fetch(c, i);
      grad(c, i, gh[s]);
      float d[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) d[q] = a.res_scale * gh[s][q];
      // without a block output, or held in registers, dr can go out at once (it may alias dr_out: each
      // value is read before it is written); otherwise the second reading comes first
      if (HOLD || !a.y) store8(a.dr, a.r_type, base + 8 * i, d);
      if (a.y) {
        float v[8], f[8];
        raw8_to_float(ry[s], a.y_type, v);
        factor(i, f);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          v[q] *= rstd_y;
          sum_v[c][q] = fmaf(tok * gh[s][q], v[q], sum_v[c][q]);
          m_y = fmaf(gh[s][q] * f[q], v[q], m_y);
        }
      }
    }
    if (a.y) {
      const bool need = a.post_norm || (a.d_gate && a.gate_mode == MOE_GATE_TOKEN);
      if (need) m_y = row_sum<TPR>(m_y, s_b);
      if (a.d_gate && a.gate_mode == MOE_GATE_TOKEN && live && lane == 0) a.d_gate[t] = m_y;
      const float mean = a.post_norm ? m_y * tok * inv_h : 0.0f;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int i = lane + c * TPR, s = HOLD ? c : 0;
        if (!(live && i < H8)) continue;
        if constexpr (!HOLD) {
          fetch(c, i);
          grad(c, i, gh[s]);
          float d[8];
#pragma unroll
          for (int q = 0; q < 8; ++q) d[q] = a.res_scale * gh[s][q];
          store8(a.dr, a.r_type, base + 8 * i, d);
        }
        float v[8], f[8];
        raw8_to_float(ry[s], a.y_type, v);
        factor(i, f);
#pragma unroll
        for (int q = 0; q < 8; ++q) f[q] = rstd_y * fmaf(-(v[q] * rstd_y), mean, tok * f[q] * gh[s][q]);
        store8(a.dy, a.y_type, base + 8 * i, f);
      }
    }
    if constexpr (TPR > 32) __syncthreads();
  }
  if (!part) return;
  // this block's sums: the kRows row groups joined in shared memory in order, then one row of partials
  if constexpr (kRows == 1) {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int i = lane + c * TPR;
      if (i >= H8) continue;
      float *p = part + (size_t)blockIdx.x * 2 * a.H + 8 * i;
      store8(p, MOE_F32, 0, sum_v[c]);
      store8(p + a.H, MOE_F32, 0, sum_x[c]);
    }
  } else {
    static_assert(CH == 1, "short rows are one chunk a thread");
    __shared__ float s_p[2][TPR * 8];
    for (int g = 0; g < kRows; ++g) {
      __syncthreads();
      if (sub == g && lane < H8) {
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          float *pv = &s_p[0][q * TPR + lane], *px = &s_p[1][q * TPR + lane];
          *pv = (g ? *pv : 0.0f) + sum_v[0][q];
          *px = (g ? *px : 0.0f) + sum_x[0][q];
        }
      }
    }
    if (sub == kRows - 1 && lane < H8) {
      float v[8], x[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        v[q] = s_p[0][q * TPR + lane];
        x[q] = s_p[1][q * TPR + lane];
      }
      float *p = part + (size_t)blockIdx.x * 2 * a.H + 8 * lane;
      store8(p, MOE_F32, 0, v);
      store8(p + a.H, MOE_F32, 0, x);
    }
  }
}

// the blocks' partial sums added in a fixed order: 32 channels a block, eight row groups
__global__ void __launch_bounds__(256) block_norm_gain_kernel(const BlockNormGradArgs a, const float *__restrict__ part,
                                                             int n) {
  __shared__ float s[2][8][32];
  const int lane = threadIdx.x & 31, grp = threadIdx.x >> 5, h = blockIdx.x * 32 + lane;
  float v = 0.0f, x = 0.0f;
  for (int i = grp; i < n; i += 8) {
    v += part[(size_t)i * 2 * a.H + h];
    x += part[(size_t)i * 2 * a.H + a.H + h];
  }
  s[0][grp][lane] = v;
  s[1][grp][lane] = x;
  __syncthreads();
  if (grp == 0) {
    v = x = 0.0f;
#pragma unroll
    for (int g = 0; g < 8; ++g) {
      v += s[0][g][lane];
      x += s[1][g][lane];
    }
    const float gate = a.gate_mode == MOE_GATE_CHANNEL ? a.gate[h] : 1.0f;
    if (a.d_post_gain) a.d_post_gain[h] = gate * v;
    if (a.d_gate && a.gate_mode == MOE_GATE_CHANNEL) a.d_gate[h] = (a.post_gain ? a.post_gain[h] : 1.0f) * v;
    if (a.d_pre_gain) a.d_pre_gain[h] = x;
  }
}

int tpr_of(int H) {  // threads a row: one chunk of eight values each up to H = 8192
  int t = 32;
  while (t * 8 < H && t < 1024) t *= 2;
  return t;
}

int grad_blocks(int T, int H) {
  const int tpr = tpr_of(H), rows = tpr < 256 ? 256 / tpr : 1;
  const int want = (T + rows - 1) / rows, cap = num_sms() * (tpr <= 256 ? 2 : 1);
  return want < cap ? want : cap;
}

}  // namespace

cudaError_t launch_block_norm(const BlockNormArgs &a, cudaStream_t s) {
  const int tpr = tpr_of(a.H), threads = tpr < 256 ? 256 : tpr, rows = threads / tpr;
  const int grid = (a.T + rows - 1) / rows;
  KTimer kt_(KID_BLOCK_NORM, s);
  switch (tpr) {
    case 32: block_norm_kernel<32, 1><<<grid, threads, 0, s>>>(a); break;
    case 64: block_norm_kernel<64, 1><<<grid, threads, 0, s>>>(a); break;
    case 128: block_norm_kernel<128, 1><<<grid, threads, 0, s>>>(a); break;
    case 256: block_norm_kernel<256, 1><<<grid, threads, 0, s>>>(a); break;
    case 512: block_norm_kernel<512, 1><<<grid, threads, 0, s>>>(a); break;
    default:
      if (a.H <= 8192) block_norm_kernel<1024, 1><<<grid, threads, 0, s>>>(a);
      else block_norm_kernel<1024, 2><<<grid, threads, 0, s>>>(a);
  }
  return cudaGetLastError();
}

size_t block_norm_grad_scratch(int T, int H) { return (size_t)grad_blocks(T, H) * 2 * H * 4; }

cudaError_t launch_block_norm_grad(const BlockNormGradArgs &a, float *scratch, cudaStream_t s) {
  const int tpr = tpr_of(a.H), threads = tpr < 256 ? 256 : tpr, grid = grad_blocks(a.T, a.H);
  const bool sums = a.d_post_gain || a.d_pre_gain || (a.d_gate && a.gate_mode == MOE_GATE_CHANNEL);
  float *part = sums ? scratch : nullptr;
  {
    KTimer kt_(KID_BLOCK_NORM_GRAD, s);
    switch (tpr) {
      case 32: block_norm_grad_kernel<32, 1, true><<<grid, threads, 0, s>>>(a, part); break;
      case 64: block_norm_grad_kernel<64, 1, true><<<grid, threads, 0, s>>>(a, part); break;
      case 128: block_norm_grad_kernel<128, 1, true><<<grid, threads, 0, s>>>(a, part); break;
      case 256: block_norm_grad_kernel<256, 1, true><<<grid, threads, 0, s>>>(a, part); break;
      case 512: block_norm_grad_kernel<512, 1, true><<<grid, threads, 0, s>>>(a, part); break;
      default:
        if (a.H <= 8192) block_norm_grad_kernel<1024, 1, false><<<grid, threads, 0, s>>>(a, part);
        else block_norm_grad_kernel<1024, 2, false><<<grid, threads, 0, s>>>(a, part);
    }
  }
  if (sums) {
    KTimer kt_(KID_BLOCK_NORM_GAIN, s);
    block_norm_gain_kernel<<<a.H / 32, 256, 0, s>>>(a, scratch, grid);
  }
  return cudaGetLastError();
}

}  // namespace moe
