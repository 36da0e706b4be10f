// Shared by the block operators (block_norm.cu, pairs.cu, mx4.cu): rows of fp32, fp16 or bf16 values
// handled eight at a time, and the launchers that block_abi.cu calls.
#pragma once

#include "common.cuh"

namespace moe {

// the block operators' kernels, numbered behind the layers' (common.cuh) for the timing hook
enum BlockKernelId {
  KID_BLOCK_NORM = KID_COUNT, KID_BLOCK_NORM_GRAD, KID_BLOCK_NORM_GAIN, KID_PAIR_HIST, KID_PAIR_SCAN, KID_PAIR_PLACE,
  KID_DISPATCH, KID_COLLECT, KID_COLLECT_GRAD, KID_MX4_QUANTIZE, KID_MX4_DEQUANTIZE, KID_MX4_PRODUCT, KID_ALL
};

// The kernels' type codes: the public ones, and fp32 whose base is 32-byte aligned, which moves eight values
// in one access. Two 16-byte accesses 32 bytes apart between lanes touch each 32-byte sector twice.
constexpr int kF32Wide = 3;
inline int kernel_type(int type, const void *p) { return type == MOE_F32 && ((uintptr_t)p & 31u) == 0 ? kF32Wide : type; }
__host__ __device__ constexpr bool is_f32(int type) { return type == MOE_F32 || type == kF32Wide; }
__host__ __device__ constexpr int type_bytes(int type) { return is_f32(type) ? 4 : 2; }

// eight consecutive values as loaded (16 or 32 bytes), so that several loads are in flight before any
// is converted; `type` is the same for every thread of a launch
struct Raw8 {
  uint4 a, b;
};

__device__ __forceinline__ Raw8 load_raw8(const void *base, int type, size_t i) {  // values i .. i+7, i % 8 == 0
  const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(base) + i * type_bytes(type));
  Raw8 r;
  if (type == kF32Wide) {
    asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r.a.x), "=r"(r.a.y), "=r"(r.a.z), "=r"(r.a.w), "=r"(r.b.x), "=r"(r.b.y), "=r"(r.b.z), "=r"(r.b.w)
                 : "l"(p)
                 : "memory");
    return r;
  }
  r.a = p[0];
  r.b = make_uint4(0, 0, 0, 0);
  if (type == MOE_F32) r.b = p[1];
  return r;
}

__device__ __forceinline__ void raw8_to_float(const Raw8 &r, int type, float v[8]) {
  const uint32_t w[4] = {r.a.x, r.a.y, r.a.z, r.a.w};
  if (is_f32(type)) {
    const uint32_t x[4] = {r.b.x, r.b.y, r.b.z, r.b.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = __uint_as_float(w[i]);
      v[4 + i] = __uint_as_float(x[i]);
    }
  } else if (type == MOE_BF16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  }
}

__device__ __forceinline__ void load8(const void *base, int type, size_t i, float v[8]) {
  raw8_to_float(load_raw8(base, type, i), type, v);
}

__device__ __forceinline__ void store_raw8(void *base, int type, size_t i, const Raw8 &r) {
  uint4 *p = reinterpret_cast<uint4 *>(static_cast<uint8_t *>(base) + i * type_bytes(type));
  if (type == kF32Wide) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(r.a.x), "r"(r.a.y), "r"(r.a.z),
                 "r"(r.a.w), "r"(r.b.x), "r"(r.b.y), "r"(r.b.z), "r"(r.b.w)
                 : "memory");
    return;
  }
  p[0] = r.a;
  if (type == MOE_F32) p[1] = r.b;
}

// The inner loops know types at compile time as far as it pays: eight fp32 values in one access, or a 16-bit
// type (fp16 or bf16, told apart by a uniform branch), or any type (kAny). With every type told apart
// at run time a row of the norm cost 58 instructions a value.
constexpr int kAny = -1, k16 = 4;
template <int KT>
__device__ __forceinline__ int known_type(int type) {
  if constexpr (KT == kF32Wide || KT == MOE_F16 || KT == MOE_BF16) return KT;
  else if constexpr (KT == k16) return type == MOE_BF16 ? MOE_BF16 : MOE_F16;
  else return type;
}
inline int known_of(int type) { return type == kF32Wide ? kF32Wide : type == MOE_F32 ? kAny : k16; }

// the one rounding of a result: fp32 as it is, fp16 / bf16 to nearest even
__device__ __forceinline__ void store8(void *base, int type, size_t i, const float v[8]) {
  uint4 *p = reinterpret_cast<uint4 *>(static_cast<uint8_t *>(base) + i * type_bytes(type));
  uint32_t w[4];
  if (is_f32(type)) {
    Raw8 r;
    r.a = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
    r.b = make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7]));
    store_raw8(base, type, i, r);
    return;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (type == MOE_BF16) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
      w[j] = *reinterpret_cast<const uint32_t *>(&b);
    } else {
      const __half2 h = __floats2half2_rn(v[2 * j], v[2 * j + 1]);
      w[j] = *reinterpret_cast<const uint32_t *>(&h);
    }
  }
  p[0] = make_uint4(w[0], w[1], w[2], w[3]);
}

// ---------------------------------------------------------------- block norm (block_norm.cu)
struct BlockNormArgs {
  const void *r, *y;  // y NULL: no block output
  int r_type, y_type, T, H, post_norm;
  const float *post_gain, *gate, *pre_gain;  // each may be NULL
  int gate_mode;
  float res_scale, eps;
  void *r_out, *u;  // either may be NULL
  int u_type;
  float *rstd_y, *rstd_u;  // either may be NULL
  int r_out_type, gain_type;  // set by the launcher
};
cudaError_t launch_block_norm(const BlockNormArgs &a, cudaStream_t s);

struct BlockNormGradArgs {
  const void *dr_out, *du;  // either may be NULL
  int u_type;
  const void *r, *y;  // r: the stream after the block; y NULL: no block output
  int r_type, y_type, T, H, post_norm;
  const float *rstd_u, *rstd_y, *post_gain, *gate, *pre_gain;
  int gate_mode;
  float res_scale;
  void *dr, *dy;  // dy NULL: no block output
  float *d_post_gain, *d_gate, *d_pre_gain;  // each may be NULL
  int d_type, dr_type, dy_type, gain_type;  // set by the launcher
};
// partial sums over the rows of each CTA: [CTAs][2][H] fp32
size_t block_norm_grad_scratch(int T, int H);
cudaError_t launch_block_norm_grad(const BlockNormGradArgs &a, float *scratch, cudaStream_t s);

// ---------------------------------------------------------------- sorted pairs (pairs.cu)
size_t sort_pairs_scratch(long long P, int E);
cudaError_t launch_sort_pairs(const int32_t *idx, int T, int k, int E, int32_t *counts, int32_t *offsets,
                              int32_t *row_of, int32_t *src, int32_t *hist, Ctrl *ctrl, cudaStream_t s);
cudaError_t launch_dispatch(const void *x, int type, int T, int k, int H, const int32_t *row_of, const int32_t *kept,
                            void *rows, cudaStream_t s);
cudaError_t launch_collect(const void *rows, int type, int T, int k, int H, const int32_t *row_of, const float *w,
                           const float *residual, void *y, int y_type, cudaStream_t s);
cudaError_t launch_collect_grad(const void *dy, int dy_type, const void *rows, int type, int T, int k, int H,
                                const int32_t *row_of, const float *w, const int32_t *kept, void *d_rows, float *d_w,
                                cudaStream_t s);

// ---------------------------------------------------------------- MXFP4 (mx4.cu)
cudaError_t launch_mx4_quantize(const void *x, int type, int T, int K, const int32_t *row_of, int k,
                                const int32_t *kept, uint8_t *codes, uint8_t *scales, cudaStream_t s);
cudaError_t launch_mx4_dequantize(const uint8_t *codes, const uint8_t *scales, long long rows, int K, void *out,
                                  int type, cudaStream_t s);
struct Mx4ProductArgs {
  const uint8_t *a_codes, *a_scales;
  int n_rows, K, N, E;
  const int32_t *offsets;  // [E + 1], or NULL: one group of all rows
  const uint8_t *w_codes, *w_scales, *up_codes, *up_scales;  // up: NULL for a plain product
  void *out;
  int out_type;
  Ctrl *ctrl;
};
cudaError_t launch_mx4_product(const Mx4ProductArgs &a, cudaStream_t s);

}  // namespace moe
