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
#include <initializer_list>
#include <type_traits>

#include "block.cuh"

namespace moe {

namespace {

constexpr int kNormWarps = 16;  // a block has 256 threads, or 512 for rows of more than 2048 values

// Sum over the tpr threads of a row (a power of two from 32 to 512); every thread of the block calls it.
// Calls alternate between two buffers: one is written again only after the barrier of the call between.
struct RowSum {
  float (*buf)[kNormWarps];
  int tpr, k;
  __device__ __forceinline__ float operator()(float v) {
    v = warp_sum(v);
    if (tpr > 32) {
      const int nw = tpr >> 5, lane = threadIdx.x & 31, w0 = (threadIdx.x >> 5) & ~(nw - 1);
      float *b = buf[k];
      k ^= 1;
      if (lane == 0) b[threadIdx.x >> 5] = v;
      __syncthreads();
      v = b[w0 + (lane & (nw - 1))];
#pragma unroll
      for (int o = 8; o > 0; o >>= 1)
        if (o < nw) v += __shfl_xor_sync(0xffffffffu, v, o);
    }
    return v;
  }
};

__device__ __forceinline__ void ones8(float v[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = 1.0f;
}

// post_gain times a channel's gate
template <class Args>
__device__ __forceinline__ void load_post(const Args &a, int gain_type, int i, float v[8]) {
  ones8(v);
  if (a.post_gain) load8(a.post_gain, gain_type, 8 * i, v);
  if (a.gate_mode == MOE_GATE_CHANNEL) {
    float g[8];
    load8(a.gate, gain_type, 8 * i, g);
#pragma unroll
    for (int q = 0; q < 8; ++q) v[q] *= g[q];
  }
}
template <class Args>
__device__ __forceinline__ void load_pre(const Args &a, int gain_type, int i, float v[8]) {
  ones8(v);
  if (a.pre_gain) load8(a.pre_gain, gain_type, 8 * i, v);
}

// tpr threads a row, CH chunks of eight values a thread; R, Y, U: what is known of the types of r, y and u.
// Blocks walk over rows; with one chunk a thread the gains stay in registers, and the next row is loaded
// there while a row's two dependent sums are worked out.
template <int KT, int CH, int R, int Y, int U>
__global__ void __launch_bounds__(KT, KT == 256 ? 3 : 1) block_norm_kernel(const BlockNormArgs a, int tpr) {
  constexpr bool kOne = CH == 1;
  __shared__ float s_sum[2][kNormWarps];
  RowSum row_sum{s_sum, tpr, 0};
  const int rows = KT / tpr, sub = threadIdx.x / tpr, lane = threadIdx.x & (tpr - 1), H8 = a.H >> 3;
  const int rt = known_type<R>(a.r_type), rot = known_type<R>(a.r_out_type), yt = known_type<Y>(a.y_type),
            ut = known_type<U>(a.u_type), gt = R == kAny ? a.gain_type : kF32Wide;
  const float inv_h = 1.0f / (float)a.H;
  const int stride = gridDim.x * rows, first = blockIdx.x * rows + sub;
  pdl_launch_dependents();
  pdl_wait();
  Raw8 rr[CH], ry[CH], nr, ny;
  auto fetch = [&](long long t, int i, Raw8 &r, Raw8 &y) {
    if (t >= a.T || i >= H8) return;
    const size_t at = (size_t)t * a.H + 8 * i;
    r = load_raw8(a.r, rt, at);
    if (a.y) y = load_raw8(a.y, yt, at);
  };
  float post[8], pre[8];
  if constexpr (kOne) {
    fetch(first, lane, nr, ny);
    if (lane < H8) {
      load_post(a, gt, lane, post);
      load_pre(a, gt, lane, pre);
    }
  }
  for (long long t = first; t - sub < a.T; t += stride) {  // every thread of the block stays for the sums
    const bool live = t < a.T;
    const size_t base = (size_t)t * a.H;
    if constexpr (kOne) {
      rr[0] = nr;
      ry[0] = ny;
      fetch(t + stride, lane, nr, ny);
    } else {
#pragma unroll
      for (int c = 0; c < CH; ++c) fetch(t, lane + c * tpr, rr[c], ry[c]);
    }
    float rstd_y = 1.0f;
    if (a.y && a.post_norm) {
      float ss = 0.0f;
#pragma unroll
      for (int c = 0; c < CH; ++c)
        if (live && lane + c * tpr < H8) {
          float v[8];
          raw8_to_float(ry[c], yt, v);
#pragma unroll
          for (int q = 0; q < 8; ++q) ss = fmaf(v[q], v[q], ss);
        }
      rstd_y = 1.0f / sqrtf(row_sum(ss) * inv_h + a.eps);
      if (a.rstd_y && live && lane == 0) a.rstd_y[t] = rstd_y;
    }
    const float yscale = (a.gate_mode == MOE_GATE_TOKEN && live) ? a.gate[t] * rstd_y : rstd_y;
    float v[CH][8], ss = 0.0f;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int i = lane + c * tpr;
      if (!(live && i < H8)) continue;
      raw8_to_float(rr[c], rt, v[c]);
      if constexpr (!kOne) load_post(a, gt, i, post);
#pragma unroll
      for (int q = 0; q < 8; ++q) v[c][q] *= a.res_scale;
      if (a.y) {
        float z[8];
        raw8_to_float(ry[c], yt, z);
#pragma unroll
        for (int q = 0; q < 8; ++q) v[c][q] = fmaf(z[q] * yscale, post[q], v[c][q]);
      }
      if (a.r_out) store8(a.r_out, rot, base + 8 * i, v[c]);
#pragma unroll
      for (int q = 0; q < 8; ++q) ss = fmaf(v[c][q], v[c][q], ss);
    }
    if (a.u) {  // the norm of r' before its rounding to the stream's type
      const float rstd_u = 1.0f / sqrtf(row_sum(ss) * inv_h + a.eps);
      if (a.rstd_u && live && lane == 0) a.rstd_u[t] = rstd_u;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int i = lane + c * tpr;
        if (!(live && i < H8)) continue;
        if constexpr (!kOne) load_pre(a, gt, i, pre);
#pragma unroll
        for (int q = 0; q < 8; ++q) v[c][q] = v[c][q] * rstd_u * pre[q];
        store8(a.u, ut, base + 8 * i, v[c]);
      }
    }
  }
}

// With one chunk a thread the row stays in registers, the next one loaded behind it; with more, each of the three
// passes reads it again (from L2) and works g out again.
template <int KT, int CH, int R, int Y, int U>
__global__ void __launch_bounds__(KT, KT == 256 ? 2 : 1) block_norm_grad_kernel(const BlockNormGradArgs a, float *__restrict__ part, int tpr) {
  constexpr bool kOne = CH == 1;
  __shared__ float s_sum[2][kNormWarps];
  RowSum row_sum{s_sum, tpr, 0};
  const int rows = KT / tpr, sub = threadIdx.x / tpr, lane = threadIdx.x & (tpr - 1), H8 = a.H >> 3;
  const int rt = known_type<R>(a.r_type), dt = known_type<R>(a.d_type), drt = known_type<R>(a.dr_type),
            yt = known_type<Y>(a.y_type), dyt = known_type<Y>(a.dy_type), ut = known_type<U>(a.u_type),
            gt = R == kAny ? a.gain_type : kF32Wide;
  const float inv_h = 1.0f / (float)a.H;
  const int stride = gridDim.x * rows, first = blockIdx.x * rows + sub;
  float sum_v[CH][8], sum_x[CH][8];  // sum over this thread's rows of g v (a token's gate folded in) and du x
#pragma unroll
  for (int c = 0; c < CH; ++c)
#pragma unroll
    for (int q = 0; q < 8; ++q) sum_v[c][q] = sum_x[c][q] = 0.0f;
  pdl_launch_dependents();
  pdl_wait();
  struct Row {
    Raw8 r, u, d, y;
    float su, sy, tok;  // the row's statistics and gate
  };
  auto fetch = [&](long long t, int i, Row &w) {
    if (t >= a.T) return;
    w.su = a.du ? a.rstd_u[t] : 0.0f;
    w.sy = (a.y && a.post_norm) ? a.rstd_y[t] : 1.0f;
    w.tok = a.gate_mode == MOE_GATE_TOKEN ? a.gate[t] : 1.0f;
    if (i >= H8) return;
    const size_t at = (size_t)t * a.H + 8 * i;
    if (a.du) {
      w.r = load_raw8(a.r, rt, at);
      w.u = load_raw8(a.du, ut, at);
    }
    if (a.dr_out) w.d = load_raw8(a.dr_out, dt, at);
    if (a.y) w.y = load_raw8(a.y, yt, at);
  };
  Row w, next;
  if constexpr (kOne) fetch(first, lane, next);
  for (long long t = first; t - sub < a.T; t += stride) {  // every thread of the block stays for the sums
    const bool live = t < a.T;
    const size_t base = (size_t)t * a.H;
    if constexpr (kOne) {
      w = next;
      fetch(t + stride, lane, next);
    } else {
      fetch(t, H8, w);
    }
    const float rstd_u = w.su, rstd_y = w.sy, tok = w.tok;
    // x = r' rstd_u and h = du pre_gain (u: du)
    float x[8], h[8], m_u = 0.0f;
    auto xh = [&](int i, float u[8]) {
      raw8_to_float(w.r, rt, x);
      raw8_to_float(w.u, ut, u);
      load_pre(a, gt, i, h);
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        x[q] *= rstd_u;
        h[q] *= u[q];
      }
    };
    if (a.du) {
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int i = lane + c * tpr;
        if (!(live && i < H8)) continue;
        if constexpr (!kOne) fetch(t, i, w);
        float u[8];
        xh(i, u);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          m_u = fmaf(h[q], x[q], m_u);
          sum_x[c][q] = fmaf(u[q], x[q], sum_x[c][q]);
        }
      }
      m_u = row_sum(m_u) * inv_h;
    }
    // g: the stream's gradient (into h), res_scale g to dr
    auto grad = [&](int i) {
      float d[8];
      if constexpr (!kOne) {
        float u[8];
        if (a.du) xh(i, u);
      }
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        d[q] = 0.0f;
        h[q] = a.du ? rstd_u * fmaf(-x[q], m_u, h[q]) : 0.0f;
      }
      if (a.dr_out) raw8_to_float(w.d, dt, d);
#pragma unroll
      for (int q = 0; q < 8; ++q) h[q] += d[q];
    };
    auto put_dr = [&](int i) {
      float d[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) d[q] = a.res_scale * h[q];
      store8(a.dr, drt, base + 8 * i, d);
    };
    // dr may be dr_out: it is written when the row's dr_out is not needed any more
    float m_y = 0.0f, v[8], f[8];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int i = lane + c * tpr;
      if (!(live && i < H8)) continue;
      if constexpr (!kOne) fetch(t, i, w);
      grad(i);
      if (kOne || !a.y) put_dr(i);
      if (a.y) {
        raw8_to_float(w.y, yt, v);
        load_post(a, gt, i, f);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          v[q] *= rstd_y;
          sum_v[c][q] = fmaf(tok * h[q], v[q], sum_v[c][q]);
          f[q] *= h[q];
          m_y = fmaf(f[q], v[q], m_y);
        }
      }
    }
    if (a.y) {
      const bool token_grad = a.d_gate && a.gate_mode == MOE_GATE_TOKEN;
      if (a.post_norm || token_grad) m_y = row_sum(m_y);
      if (token_grad && live && lane == 0) a.d_gate[t] = m_y;
      const float mean = a.post_norm ? m_y * tok * inv_h : 0.0f;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int i = lane + c * tpr;
        if (!(live && i < H8)) continue;
        if constexpr (!kOne) {
          fetch(t, i, w);
          grad(i);
          put_dr(i);
          raw8_to_float(w.y, yt, v);
          load_post(a, gt, i, f);
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            v[q] *= rstd_y;
            f[q] *= h[q];
          }
        }
#pragma unroll
        for (int q = 0; q < 8; ++q) f[q] = rstd_y * fmaf(-v[q], mean, tok * f[q]);
        store8(a.dy, dyt, base + 8 * i, f);
      }
    }
  }
  if (!part) return;
  // this block's sums: the row groups joined in shared memory in order, then one row of partials
  if (rows == 1) {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int i = lane + c * tpr;
      if (i >= H8) continue;
      float *p = part + (size_t)blockIdx.x * 2 * a.H + 8 * i;
      store8(p, kF32Wide, 0, sum_v[c]);
      store8(p + a.H, kF32Wide, 0, sum_x[c]);
    }
  } else if constexpr (kOne) {  // short rows are one chunk a thread
    __shared__ float s_p[2][128 * 8];
    for (int g = 0; g < rows; ++g) {
      __syncthreads();
      if (sub == g && lane < H8) {
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          float *pv = &s_p[0][q * tpr + lane], *px = &s_p[1][q * tpr + lane];
          *pv = (g ? *pv : 0.0f) + sum_v[0][q];
          *px = (g ? *px : 0.0f) + sum_x[0][q];
        }
      }
    }
    if (sub == rows - 1 && lane < H8) {
      float sv[8], sx[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        sv[q] = s_p[0][q * tpr + lane];
        sx[q] = s_p[1][q * tpr + lane];
      }
      float *p = part + (size_t)blockIdx.x * 2 * a.H + 8 * lane;
      store8(p, kF32Wide, 0, sv);
      store8(p + a.H, kF32Wide, 0, sx);
    }
  }
}

// the blocks' partial sums added in a fixed order: 32 channels a block, 32 row groups, eight loads in flight
__global__ void __launch_bounds__(1024) block_norm_gain_kernel(const BlockNormGradArgs a,
                                                              const float *__restrict__ part, int n) {
  __shared__ float s[2][32][33];
  const int lane = threadIdx.x & 31, grp = threadIdx.x >> 5, h = blockIdx.x * 32 + lane;
  pdl_launch_dependents();
  pdl_wait();
  float v = 0.0f, x = 0.0f;
  for (int i0 = grp; i0 < n; i0 += 32 * 4) {
    float pv[4], px[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int i = i0 + 32 * j;
      pv[j] = i < n ? part[(size_t)i * 2 * a.H + h] : 0.0f;
      px[j] = i < n ? part[(size_t)i * 2 * a.H + a.H + h] : 0.0f;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v += pv[j];
      x += px[j];
    }
  }
  s[0][grp][lane] = v;
  s[1][grp][lane] = x;
  __syncthreads();
  // warp w adds the groups' sums of channel w (lane = group)
  v = warp_sum(s[0][lane][grp]);
  x = warp_sum(s[1][lane][grp]);
  if (lane == 0) {
    const int c = blockIdx.x * 32 + grp;
    const float gate = a.gate_mode == MOE_GATE_CHANNEL ? a.gate[c] : 1.0f;
    if (a.d_post_gain) a.d_post_gain[c] = gate * v;
    if (a.d_gate && a.gate_mode == MOE_GATE_CHANNEL) a.d_gate[c] = (a.post_gain ? a.post_gain[c] : 1.0f) * v;
    if (a.d_pre_gain) a.d_pre_gain[c] = x;
  }
}

int tpr_of(int H) {  // threads a row: one chunk of eight values each up to H = 4096
  int t = 32;
  while (t * 8 < H && t < 512) t *= 2;
  return t;
}
int threads_of(int H) { return tpr_of(H) <= 256 ? 256 : 512; }

int blocks_of(int T, int H, int per_sm) {  // per_sm: blocks of 256 threads an SM holds
  const int threads = threads_of(H), rows = threads / tpr_of(H);
  const int want = (T + rows - 1) / rows, cap = num_sms() * (per_sm * 256 / threads);
  return want < cap ? want : cap;
}
int norm_blocks(int T, int H) { return blocks_of(T, H, threads_of(H) == 256 ? 3 : 2); }
int grad_blocks(int T, int H) { return blocks_of(T, H, 2); }

// calls f with the kernel's template arguments: types are told apart at compile time for rows of one chunk a
// thread whose fp32 tensors are 32-byte aligned
template <class F>
cudaError_t by_types(int H, int r, int y, int u, bool wide_gains, const F &f) {
  using std::integral_constant;
  constexpr integral_constant<int, kAny> any{};
  constexpr integral_constant<int, kF32Wide> w{};
  constexpr integral_constant<int, k16> n{};
  constexpr integral_constant<int, 512> t512{};
  if (H > 8192) return f(t512, integral_constant<int, 4>{}, any, any, any);
  if (H > 4096) return f(t512, integral_constant<int, 2>{}, any, any, any);
  auto typed = [&](auto kt) {
    constexpr integral_constant<int, 1> one{};
    if (!wide_gains || r == kAny || y == kAny || u == kAny) return f(kt, one, any, any, any);
    if (r == kF32Wide) {
      if (y == kF32Wide) return u == kF32Wide ? f(kt, one, w, w, w) : f(kt, one, w, w, n);
      return u == kF32Wide ? f(kt, one, w, n, w) : f(kt, one, w, n, n);
    }
    if (y == kF32Wide) return u == kF32Wide ? f(kt, one, n, w, w) : f(kt, one, n, w, n);
    return u == kF32Wide ? f(kt, one, n, n, w) : f(kt, one, n, n, n);
  };
  return threads_of(H) == 256 ? typed(integral_constant<int, 256>{}) : typed(t512);
}

// what is known of a type: of the tensors that share it all have to be 32-byte aligned; one that is absent
// goes with any (16-bit, so that fewer kernels are in use)
int known(int type, std::initializer_list<const void *> ptrs) {
  uintptr_t all = 0;
  for (const void *p : ptrs) all |= (uintptr_t)p;
  return all == 0 ? k16 : known_of(kernel_type(type, (const void *)all));
}

}  // namespace

cudaError_t launch_block_norm(const BlockNormArgs &args, cudaStream_t s) {
  KTimer kt_(KID_BLOCK_NORM, s);
  BlockNormArgs a = args;
  a.r_out_type = kernel_type(a.r_type, a.r_out);
  a.r_type = kernel_type(a.r_type, a.r);
  a.y_type = kernel_type(a.y_type, a.y);
  a.u_type = kernel_type(a.u_type, a.u);
  const void *gains = (const void *)((uintptr_t)a.post_gain | (uintptr_t)a.pre_gain | (uintptr_t)a.gate);
  a.gain_type = kernel_type(MOE_F32, gains);
  const dim3 grid(norm_blocks(a.T, a.H)), block(threads_of(a.H));
  return by_types(a.H, known(args.r_type, {a.r, a.r_out}), known(args.y_type, {a.y}), known(args.u_type, {a.u}),
                  a.gain_type == kF32Wide, [&](auto kt, auto ch, auto r, auto y, auto u) {
                    return launch_pdl(block_norm_kernel<kt.value, ch.value, r.value, y.value, u.value>, grid, block, 0, s, a,
                                      tpr_of(a.H));
                  });
}

size_t block_norm_grad_scratch(int T, int H) { return (size_t)grad_blocks(T, H) * 2 * H * 4; }

cudaError_t launch_block_norm_grad(const BlockNormGradArgs &args, float *scratch, cudaStream_t s) {
  BlockNormGradArgs a = args;
  a.d_type = kernel_type(a.r_type, a.dr_out);
  a.dr_type = kernel_type(a.r_type, a.dr);
  a.r_type = kernel_type(a.r_type, a.r);
  a.dy_type = kernel_type(a.y_type, a.dy);
  a.y_type = kernel_type(a.y_type, a.y);
  a.u_type = kernel_type(a.u_type, a.du);
  const void *gains = (const void *)((uintptr_t)a.post_gain | (uintptr_t)a.pre_gain | (uintptr_t)a.gate);
  a.gain_type = kernel_type(MOE_F32, gains);
  const int grid = grad_blocks(a.T, a.H);
  const bool sums = a.d_post_gain || a.d_pre_gain || (a.d_gate && a.gate_mode == MOE_GATE_CHANNEL);
  float *part = sums ? scratch : nullptr;
  cudaError_t e;
  {
    KTimer kt_(KID_BLOCK_NORM_GRAD, s);
    e = by_types(a.H, known(args.r_type, {a.r, a.dr_out, a.dr}), known(args.y_type, {a.y, a.dy}),
                 known(args.u_type, {a.du}), a.gain_type == kF32Wide, [&](auto kt, auto ch, auto r, auto y, auto u) {
                   return launch_pdl(block_norm_grad_kernel<kt.value, ch.value, r.value, y.value, u.value>, dim3(grid),
                                     dim3(threads_of(a.H)), 0, s, a, part, tpr_of(a.H));
                 });
  }
  if (e == cudaSuccess && sums) {
    KTimer kt_(KID_BLOCK_NORM_GAIN, s);
    e = launch_pdl(block_norm_gain_kernel, dim3(a.H / 32), dim3(1024), 0, s, a, (const float *)scratch, grid);
  }
  return e;
}

}  // namespace moe
