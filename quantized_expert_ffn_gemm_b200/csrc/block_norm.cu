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
// are carried whatever the gate. mean(q v) depends on mean(h x), but linearly: with e = dr' + rstd_u h,
// c = rstd_u mean(h x) and f = gate * post_gain, g = e - c x and sum f g v = sum f v e - c sum f v x. So a row
// takes one round of three sums, and each of them errs by no more than the terms of g do.
//
// Both are bound by the bytes of their rows, once a row's two dependent sums stop holding the memory up. 8192 rows of
// 2048, fp32 stream, bf16 u: forward with fp32 y 36.6 us (235 MB, 35.8 us of measured copy rate); gradient with
// bf16 y 50.9 us and 3 for the gains' sums (302 MB, 46 us): a ring to fill first, 28 rows a block behind one another
// and 5 MB of partial sums to write last. One row of one token is a launch and two reductions, 2.3 us in a graph.
//
// Rows of more than 4096 values run kernels of their own, further from their bytes: types told apart at run time, no row
// loaded ahead, and in the gradient three passes over a row behind one another, each reading it again. 2048 rows of 8192,
// fp32 stream, bf16 y and u: forward 61 us (201 MB, 31 us of copy rate), gradient 132 (302 MB, 46); of 16384, all bf16:
// 98 (41) and 260 (61).
#include <initializer_list>
#include <type_traits>

#include "block.cuh"

namespace moe {

namespace {

constexpr int kGradBlocks = 2;  // blocks of 256 threads an SM holds in the gradient (three leave two rows each: 80 us)
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

// Three such sums at once, with one barrier; the buffers alternate in the same way.
struct RowSum3 {
  float (*buf)[3][kNormWarps];
  int tpr, k;
  __device__ __forceinline__ void operator()(float v[3]) {
#pragma unroll
    for (int i = 0; i < 3; ++i) v[i] = warp_sum(v[i]);
    if (tpr > 32) {
      const int nw = tpr >> 5, lane = threadIdx.x & 31, w0 = (threadIdx.x >> 5) & ~(nw - 1);
      float(*b)[kNormWarps] = buf[k];
      k ^= 1;
      if (lane == 0)
#pragma unroll
        for (int i = 0; i < 3; ++i) b[i][threadIdx.x >> 5] = v[i];
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 3; ++i) v[i] = b[i][w0 + (lane & (nw - 1))];
#pragma unroll
      for (int o = 8; o > 0; o >>= 1)
        if (o < nw)
#pragma unroll
          for (int i = 0; i < 3; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    }
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

// Two fp32 values in a register pair: one instruction computes on both, each rounded as by itself.
typedef unsigned long long F2;
__device__ __forceinline__ F2 pack2(float a, float b) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ F2 both(float a) { return pack2(a, a); }
__device__ __forceinline__ float2 unpack2(F2 v) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
  return f;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float sum2(F2 v) {
  const float2 f = unpack2(v);
  return f.x + f.y;
}

// Four values of a row, fp32 or 16-bit, as the gradient's rows pass through shared memory.
template <bool F>
__device__ __forceinline__ void get4(const uint8_t *plane, int i, bool bf16, F2 v[2]) {
  if constexpr (F) {
    const ulonglong2 x = reinterpret_cast<const ulonglong2 *>(plane)[i];
    v[0] = x.x;
    v[1] = x.y;
  } else {
    const uint2 w = reinterpret_cast<const uint2 *>(plane)[i];
    const uint32_t p[2] = {w.x, w.y};
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      if (bf16) {
        v[j] = pack2(__uint_as_float(p[j] << 16), __uint_as_float(p[j] & 0xffff0000u));
      } else {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&p[j]));
        v[j] = pack2(f.x, f.y);
      }
    }
  }
}
template <bool F>
__device__ __forceinline__ void put4(void *base, size_t i, bool bf16, const F2 v[2]) {
  if constexpr (F) {
    *reinterpret_cast<ulonglong2 *>(static_cast<float *>(base) + i) = make_ulonglong2(v[0], v[1]);
  } else {
    uint32_t p[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float2 f = unpack2(v[j]);
      if (bf16) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(f.x, f.y);
        p[j] = *reinterpret_cast<const uint32_t *>(&b);
      } else {
        const __half2 h = __floats2half2_rn(f.x, f.y);
        p[j] = *reinterpret_cast<const uint32_t *>(&h);
      }
    }
    *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(base) + i) = make_uint2(p[0], p[1]);
  }
}
// this thread's four values of a row to their place in a plane (16 or 8 bytes, without passing registers)
template <bool F>
__device__ __forceinline__ void copy4(uint8_t *plane, int i, const void *base, size_t at) {
  const uint32_t dst = (uint32_t)__cvta_generic_to_shared(plane) + (uint32_t)i * (F ? 16u : 8u);
  if constexpr (F)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(static_cast<const float *>(base) + at) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(static_cast<const uint16_t *>(base) + at) : "memory");
}
__device__ __forceinline__ void ring_wait(int newer) {  // all but the `newer` youngest groups have landed
  if (newer >= 3) asm volatile("cp.async.wait_group 3;" ::: "memory");
  else if (newer == 2) asm volatile("cp.async.wait_group 2;" ::: "memory");
  else if (newer == 1) asm volatile("cp.async.wait_group 1;" ::: "memory");
  else asm volatile("cp.async.wait_group 0;" ::: "memory");
}
constexpr int kRingStages = 4;

// Rows of up to 8 tpr values, two groups of four a thread (values 4 lane .. and 4 tpr + 4 lane ..: accesses are whole
// lines for every type). RF, YF, UF: r (and its gradients), y, u are fp32, else 16-bit. A row waits for its sums
// (two rounds one behind the other took 54.2 us for 8192 rows of 2048, one round 50.9), so the rows to come pass through a ring in shared memory meanwhile: each thread copies and
// reads its own values, no barrier needed. (The next row held in registers left room for 16 warps an SM
// and took 69 us for 8192 rows of 2048.)
template <int KT, bool RF, bool YF, bool UF>
__global__ void __launch_bounds__(KT, KT == 256 ? kGradBlocks : 1)
block_norm_grad_kernel(const BlockNormGradArgs a, float *__restrict__ part, int tpr, int stages) {
  extern __shared__ __align__(16) uint8_t s_ring[];
  __shared__ float s_sum[2][3][kNormWarps];
  RowSum3 row_sums{s_sum, tpr, 0};
  constexpr int kR = KT * (RF ? 32 : 16), kU = KT * (UF ? 32 : 16), kY = KT * (YF ? 32 : 16);
  constexpr int kD0 = kR, kU0 = 2 * kR, kY0 = 2 * kR + kU, kBytes = 2 * kR + kU + kY;
  const int rows = KT / tpr, sub = threadIdx.x / tpr, lane = threadIdx.x & (tpr - 1);
  const bool rb = a.r_type == MOE_BF16, yb = a.y_type == MOE_BF16, ub = a.u_type == MOE_BF16;
  const float inv_h = 1.0f / (float)a.H;
  const int stride = gridDim.x * rows, first = blockIdx.x * rows + sub;
  const int at[2] = {4 * lane, 4 * tpr + 4 * lane};
  const bool in[2] = {at[0] < a.H, at[1] < a.H};
  F2 sum_v[2][2], sum_x[2][2];  // sum over this thread's rows of g v (a token's gate folded in) and du x
  F2 pre[2][2], f[2][2];        // pre_gain; post_gain times a channel's gate
#pragma unroll
  for (int g = 0; g < 2; ++g)
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      sum_v[g][q] = sum_x[g][q] = both(0.0f);
      pre[g][q] = f[g][q] = both(1.0f);
    }
  pdl_launch_dependents();
  pdl_wait();
  auto fetch = [&](long long t, int s) {
    if (t < a.T) {
      uint8_t *m = s_ring + s * kBytes;
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        if (!in[g]) continue;
        const size_t i = (size_t)t * a.H + at[g];
        const int slot = g * KT + threadIdx.x;
        if (a.du) {
          copy4<RF>(m, slot, a.r, i);
          copy4<UF>(m + kU0, slot, a.du, i);
        }
        if (a.dr_out) copy4<RF>(m + kD0, slot, a.dr_out, i);
        if (a.y) copy4<YF>(m + kY0, slot, a.y, i);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  for (int s = 0; s + 1 < stages; ++s) fetch(first + (long long)s * stride, s);
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    if (!in[g]) continue;
    F2 w[2];
    if (a.pre_gain) get4<true>(reinterpret_cast<const uint8_t *>(a.pre_gain), at[g] / 4, false, pre[g]);
    if (a.post_gain) get4<true>(reinterpret_cast<const uint8_t *>(a.post_gain), at[g] / 4, false, f[g]);
    if (a.gate_mode == MOE_GATE_CHANNEL) {
      get4<true>(reinterpret_cast<const uint8_t *>(a.gate), at[g] / 4, false, w);
#pragma unroll
      for (int q = 0; q < 2; ++q) f[g][q] = mul2(f[g][q], w[q]);
    }
  }
  float su_n = 0.0f, sy_n = 1.0f, tok_n = 1.0f;  // the next row's statistics and gate
  auto stats = [&](long long t) {
    if (t >= a.T) return;
    if (a.du) su_n = a.rstd_u[t];
    if (a.y && a.post_norm) sy_n = a.rstd_y[t];
    if (a.gate_mode == MOE_GATE_TOKEN) tok_n = a.gate[t];
  };
  stats(first);
  int stage = 0;
  for (long long t = first; t - sub < a.T; t += stride) {  // every thread of the block stays for the sums
    const bool live = t < a.T;
    const size_t base = (size_t)t * a.H;
    const float su = su_n, sy = sy_n, tok = tok_n;
    stats(t + stride);
    fetch(t + (long long)(stages - 1) * stride, stage == 0 ? stages - 1 : stage - 1);
    ring_wait(stages - 1);
    const uint8_t *m = s_ring + stage * kBytes;
    F2 x[2][2], e[2][2], v[2][2], dot[3] = {both(0.0f), both(0.0f), both(0.0f)};
    const F2 su2 = both(su), sy2 = both(sy), tok2 = both(tok), res2 = both(a.res_scale);
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      if (!(live && in[g])) continue;
      const int slot = g * KT + threadIdx.x;
      e[g][0] = e[g][1] = both(0.0f);
      if (a.dr_out) get4<RF>(m + kD0, slot, rb, e[g]);
      if (a.du) {
        F2 h[2];
        get4<RF>(m, slot, rb, x[g]);
        get4<UF>(m + kU0, slot, ub, h);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          x[g][q] = mul2(x[g][q], su2);
          sum_x[g][q] = fma2(h[q], x[g][q], sum_x[g][q]);
          h[q] = mul2(h[q], pre[g][q]);
          dot[0] = fma2(h[q], x[g][q], dot[0]);
          e[g][q] = fma2(su2, h[q], e[g][q]);
        }
      }
      if (a.y) {
        get4<YF>(m + kY0, slot, yb, v[g]);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          v[g][q] = mul2(v[g][q], sy2);
          const F2 fv = mul2(f[g][q], v[g][q]);
          dot[1] = fma2(fv, e[g][q], dot[1]);
          if (a.du) dot[2] = fma2(fv, x[g][q], dot[2]);
        }
      }
    }
    float sums[3] = {sum2(dot[0]), sum2(dot[1]), sum2(dot[2])};
    row_sums(sums);
    const float c = su * (sums[0] * inv_h), m_y = fmaf(-c, sums[2], sums[1]);
    if (a.d_gate && a.gate_mode == MOE_GATE_TOKEN && live && lane == 0) a.d_gate[t] = m_y;
    const F2 neg_c = both(-c), neg_mean = both(a.post_norm ? -m_y * inv_h : 0.0f), scale = both(sy * tok);
#pragma unroll
    for (int g = 0; g < 2; ++g) {  // e becomes g
      if (!(live && in[g])) continue;
      F2 o[2];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        if (a.du) e[g][q] = fma2(x[g][q], neg_c, e[g][q]);
        o[q] = mul2(res2, e[g][q]);
      }
      put4<RF>(a.dr, base + at[g], rb, o);
      if (!a.y) continue;
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        sum_v[g][q] = fma2(tok2, mul2(e[g][q], v[g][q]), sum_v[g][q]);
        o[q] = mul2(scale, fma2(v[g][q], neg_mean, mul2(f[g][q], e[g][q])));
      }
      put4<YF>(a.dy, base + at[g], yb, o);
    }
    stage = stage + 1 == stages ? 0 : stage + 1;
  }
  if (!part) return;
  // this block's sums: the row groups joined in shared memory in order, then one row of partials
  if (rows > 1) {
    __shared__ __align__(16) float s_p[2][128 * 8];
    for (int r = 0; r < rows; ++r) {
      __syncthreads();
      if (sub != r) continue;
#pragma unroll
      for (int g = 0; g < 2; ++g)
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          F2 *pv = reinterpret_cast<F2 *>(&s_p[0][at[g] + 2 * q]), *px = reinterpret_cast<F2 *>(&s_p[1][at[g] + 2 * q]);
          *pv = sum_v[g][q] = r ? add2(sum_v[g][q], *pv) : sum_v[g][q];
          *px = sum_x[g][q] = r ? add2(sum_x[g][q], *px) : sum_x[g][q];
        }
    }
    if (sub != rows - 1) return;
  }
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    if (!in[g]) continue;
    float *p = part + (size_t)blockIdx.x * 2 * a.H + at[g];
    put4<true>(p, 0, false, sum_v[g]);
    put4<true>(p, a.H, false, sum_x[g]);
  }
}

// Rows of more than 4096 values: CH chunks of eight a thread; each of the three passes reads the row again (from L2)
// and works g out again.
template <int CH>
__global__ void __launch_bounds__(512, 1) block_norm_grad_long_kernel(const BlockNormGradArgs a, float *__restrict__ part) {
  constexpr int tpr = 512;
  __shared__ float s_sum[2][kNormWarps];
  RowSum row_sum{s_sum, tpr, 0};
  const int lane = threadIdx.x, H8 = a.H >> 3;
  const int rt = a.r_type, dt = a.d_type, drt = a.dr_type, yt = a.y_type, dyt = a.dy_type, ut = a.u_type,
            gt = a.gain_type;
  const float inv_h = 1.0f / (float)a.H;
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
  Row w;
  for (long long t = blockIdx.x; t < a.T; t += gridDim.x) {
    const size_t base = (size_t)t * a.H;
    fetch(t, H8, w);
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
        if (i >= H8) continue;
        fetch(t, i, w);
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
      float u[8];
      if (a.du) xh(i, u);
      if (!a.dr_out) {
#pragma unroll
        for (int q = 0; q < 8; ++q) d[q] = 0.0f;
      } else {
        raw8_to_float(w.d, dt, d);
      }
#pragma unroll
      for (int q = 0; q < 8; ++q) h[q] = a.du ? fmaf(rstd_u, fmaf(-x[q], m_u, h[q]), d[q]) : d[q];
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
      if (i >= H8) continue;
      fetch(t, i, w);
      grad(i);
      if (!a.y) put_dr(i);
      if (a.y) {
        raw8_to_float(w.y, yt, v);
        load_post(a, gt, i, f);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          v[q] *= rstd_y;
          const float hv = h[q] * v[q];
          sum_v[c][q] = fmaf(tok, hv, sum_v[c][q]);
          m_y = fmaf(f[q], hv, m_y);
          f[q] *= h[q];
        }
      }
    }
    if (a.y) {
      const bool token_grad = a.d_gate && a.gate_mode == MOE_GATE_TOKEN;
      if (a.post_norm || token_grad) m_y = row_sum(m_y);
      if (token_grad && lane == 0) a.d_gate[t] = m_y;
      const float mean = a.post_norm ? m_y * inv_h : 0.0f, scale = rstd_y * tok;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int i = lane + c * tpr;
        if (i >= H8) continue;
        fetch(t, i, w);
        grad(i);
        put_dr(i);
        raw8_to_float(w.y, yt, v);
        load_post(a, gt, i, f);
#pragma unroll
        for (int q = 0; q < 8; ++q) f[q] = scale * fmaf(-(v[q] * rstd_y), mean, f[q] * h[q]);
        store8(a.dy, dyt, base + 8 * i, f);
      }
    }
  }
  if (!part) return;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int i = lane + c * tpr;
    if (i >= H8) continue;
    // 16 bytes a store: the scratch is aligned as the workspace is, which may start on any 16 bytes
    float *p = part + (size_t)blockIdx.x * 2 * a.H + 8 * i;
    store8(p, MOE_F32, 0, sum_v[c]);
    store8(p + a.H, MOE_F32, 0, sum_x[c]);
  }
}

// The blocks' partial sums added in a fixed order: 16 channels a block, 64 groups of rows, eight loads in flight.
// The kernel is a few dependent loads long (3 us for 296 rows of 2 x 2048), so it is spread thin.
__global__ void __launch_bounds__(1024) block_norm_gain_kernel(const BlockNormGradArgs a,
                                                              const float *__restrict__ part, int n) {
  __shared__ float s[2][64][17];
  const int ch = threadIdx.x & 15, grp = threadIdx.x >> 4, h = blockIdx.x * 16 + ch;
  pdl_launch_dependents();
  pdl_wait();
  float v = 0.0f, x = 0.0f;
  for (int i0 = grp; i0 < n; i0 += 64 * 4) {
    float pv[4], px[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int i = i0 + 64 * j;
      pv[j] = i < n ? part[(size_t)i * 2 * a.H + h] : 0.0f;
      px[j] = i < n ? part[(size_t)i * 2 * a.H + a.H + h] : 0.0f;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v += pv[j];
      x += px[j];
    }
  }
  s[0][grp][ch] = v;
  s[1][grp][ch] = x;
  __syncthreads();
  // a warp joins the groups of one channel's one sum
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 16 + (warp >> 1);
  const float(*t)[17] = s[warp & 1];
  const float sum = warp_sum(t[lane][warp >> 1] + t[lane + 32][warp >> 1]);
  if (lane) return;
  if (warp & 1) {
    if (a.d_pre_gain) a.d_pre_gain[c] = sum;
  } else {
    if (a.d_post_gain) a.d_post_gain[c] = (a.gate_mode == MOE_GATE_CHANNEL ? a.gate[c] : 1.0f) * sum;
    if (a.d_gate && a.gate_mode == MOE_GATE_CHANNEL) a.d_gate[c] = (a.post_gain ? a.post_gain[c] : 1.0f) * sum;
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
  const int cap = num_sms() * (per_sm * 256 / threads);
  const long long want = ((long long)T + rows - 1) / rows;
  return want < cap ? (int)want : cap;
}
int norm_blocks(int T, int H) { return blocks_of(T, H, threads_of(H) == 256 ? 3 : 2); }
int grad_blocks(int T, int H) { return blocks_of(T, H, threads_of(H) == 256 ? kGradBlocks : 2); }

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

template <int KT, bool RF, bool YF, bool UF>
cudaError_t run_grad(const BlockNormGradArgs &a, float *part, int grid, cudaStream_t s) {
  constexpr int kBytes = KT * (2 * (RF ? 32 : 16) + (YF ? 32 : 16) + (UF ? 32 : 16));
  constexpr int kFit = 208 * 1024 / (KT == 256 ? kGradBlocks : 1) / kBytes;
  const int tpr = tpr_of(a.H), side = KT / tpr;
  const long long rows = ((long long)a.T + side - 1) / side, each = (rows + grid - 1) / grid;
  int stages = kFit < kRingStages ? kFit : kRingStages;
  if (stages > each) stages = (int)each;  // no more than a block's rows
  static_assert(kFit >= 1, "a row fits");
  const cudaError_t e = smem_limit_once(block_norm_grad_kernel<KT, RF, YF, UF>, kRingStages * kBytes < 208 * 1024
                                                                                   ? kRingStages * kBytes
                                                                                   : 208 * 1024);
  if (e != cudaSuccess) return e;
  return launch_pdl(block_norm_grad_kernel<KT, RF, YF, UF>, dim3(grid), dim3(KT), (size_t)stages * kBytes, s, a, part, tpr,
                    stages);
}

template <int KT>
cudaError_t grad_by_types(const BlockNormGradArgs &a, float *part, int grid, cudaStream_t s) {
  const bool r = a.r_type == MOE_F32, y = a.y && a.y_type == MOE_F32, u = a.du && a.u_type == MOE_F32;
  if (r) {
    if (y) return u ? run_grad<KT, true, true, true>(a, part, grid, s) : run_grad<KT, true, true, false>(a, part, grid, s);
    return u ? run_grad<KT, true, false, true>(a, part, grid, s) : run_grad<KT, true, false, false>(a, part, grid, s);
  }
  if (y) return u ? run_grad<KT, false, true, true>(a, part, grid, s) : run_grad<KT, false, true, false>(a, part, grid, s);
  return u ? run_grad<KT, false, false, true>(a, part, grid, s) : run_grad<KT, false, false, false>(a, part, grid, s);
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
    if (a.H > 8192) e = launch_pdl(block_norm_grad_long_kernel<4>, dim3(grid), dim3(512), 0, s, a, part);
    else if (a.H > 4096) e = launch_pdl(block_norm_grad_long_kernel<2>, dim3(grid), dim3(512), 0, s, a, part);
    else if (threads_of(a.H) == 256) e = grad_by_types<256>(args, part, grid, s);
    else e = grad_by_types<512>(args, part, grid, s);
  }
  if (e == cudaSuccess && sums) {
    KTimer kt_(KID_BLOCK_NORM_GAIN, s);
    e = launch_pdl(block_norm_gain_kernel, dim3(a.H / 16), dim3(1024), 0, s, a, (const float *)scratch, grid);
  }
  return e;
}

}  // namespace moe
