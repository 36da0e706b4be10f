// Microscaled 4-bit floating point (MXFP4, the OCP microscaling format): values in blocks of 32 along a
// row, each an e2m1 code (sign, two exponent bits, one mantissa bit: 0 0.5 1 1.5 2 3 4 6) times the
// block's power of two, stored as one e8m0 byte b = exponent + 127.
//
//   quantise   b = max(floor(log2(max |x|)) - 2 + 127, 0);  code = nearest e2m1 of x 2^(127 - b), ties to
//              the even code, magnitudes over 6 become 6; a block with a NaN or an infinity reads back NaN
//   (the product of such rows is in mx4_product.cu)
//
// floor(log2) of an fp32 value is its exponent field less 127, and scaling by a power of two is exact, so
// quantising rounds once, at the code.
//
// Both directions are bound by their bytes: 8192 tokens of 2048 to ten sorted rows each 20.8 us (33 MB in, 89 MB
// out, 18.6 us of measured copy rate), 20,480 such rows back to bf16 18.7 us (106 MB, 16.2 us).
#include <type_traits>

#include "block.cuh"

namespace moe {

namespace {

// 2^(b - 127) of a scale byte; 255 is the format's NaN
__device__ __forceinline__ float e8m0_to_float(uint32_t b) {
  return b == 255u ? __uint_as_float(0x7fffffffu) : b ? __uint_as_float(b << 23) : __uint_as_float(0x00400000u);
}

// two fp32 values to two e2m1 codes, `lo` in the low four bits (nearest even, saturating)
__device__ __forceinline__ uint32_t e2m1_pair(float lo, float hi) {
  uint16_t r;
  asm("{\n.reg .b8 c;\ncvt.rn.satfinite.e2m1x2.f32 c, %1, %2;\ncvt.u16.u8 %0, c;\n}\n" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// the values of two codes, times d
__device__ __forceinline__ float2 e2m1_values(uint32_t pair, float d) {
  uint32_t h;
  asm("{\n.reg .b8 c;\n.reg .b16 w;\ncvt.u16.u32 w, %1;\ncvt.u8.u16 c, w;\ncvt.rn.f16x2.e2m1x2 %0, c;\n}\n" : "=r"(h) : "r"(pair));
  const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
  return make_float2(f.x * d, f.y * d);
}

// index / n and the remainder; 64-bit division only where the index needs it
__device__ __forceinline__ void split(long long i, int n, long long &q, int &r) {
  if (i <= 0xffffffffll) {
    const uint32_t u = (uint32_t)i / (uint32_t)n;
    q = u;
    r = (int)((uint32_t)i - u * (uint32_t)n);
  } else {
    q = i / n;
    r = (int)(i - q * n);
  }
}

// A thread one block of 32: its largest magnitude needs no exchange, its codes are one 16-byte store to each
// of the token's rows, a warp's scales one sector. (Four lanes a block with 4-byte stores: 42 us for 8192 tokens
// of 2048 to ten rows each.)
template <int KT>
__global__ void __launch_bounds__(256) mx4_quantize_kernel(const void *__restrict__ x, int x_type, int T, int K,
                                                          const int32_t *__restrict__ row_of, int k,
                                                          const int32_t *__restrict__ kept,
                                                          uint8_t *__restrict__ codes, uint8_t *__restrict__ scales) {
  const int nb = K >> 5, P = T * k, type = known_type<KT>(x_type);
  pdl_launch_dependents();
  pdl_wait();
  const long long n = (long long)T * nb, stride = (long long)gridDim.x * 256;
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < n; i += stride) {
    Raw8 raw[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) raw[j] = load_raw8(x, type, (size_t)i * 32 + 8 * j);
    long long t;
    int blk;
    split(i, nb, t, blk);
    float v[32];
    uint32_t top = 0;  // the largest magnitude's bits: magnitudes order as their bits do, NaN above all
#pragma unroll
    for (int j = 0; j < 4; ++j) raw8_to_float(raw[j], type, v + 8 * j);
#pragma unroll
    for (int q = 0; q < 32; ++q) top = max(top, __float_as_uint(v[q]) & 0x7fffffffu);
    const int e = (int)(top >> 23);
    const uint32_t b = e == 255 ? 255u : (uint32_t)max(e - 2, 0);
    const float inv = __uint_as_float((254u - b) << 23);  // 2^(127 - b), b <= 252
    uint32_t c[4] = {0, 0, 0, 0};
    if (b != 255u) {
#pragma unroll
      for (int q = 0; q < 16; ++q) c[q >> 2] |= e2m1_pair(v[2 * q] * inv, v[2 * q + 1] * inv) << (8 * (q & 3));
    }
    const uint4 word = make_uint4(c[0], c[1], c[2], c[3]);
    for (int j = 0; j < k; ++j) {
      const long long r = row_of ? row_of[t * k + j] : t;
      if (r < 0 || r >= P) continue;
      reinterpret_cast<uint4 *>(codes)[r * nb + blk] = word;
      scales[r * nb + blk] = (uint8_t)b;
    }
  }
  if (!kept) return;
  // the rows behind the last kept pair hold zeros
  const long long first = (long long)min(max(*kept, 0), P) * nb;
  for (long long i = first + (long long)blockIdx.x * 256 + threadIdx.x; i < (long long)P * nb; i += stride) {
    reinterpret_cast<uint4 *>(codes)[i] = make_uint4(0, 0, 0, 0);
    scales[i] = 0;
  }
}

// eight values a thread: a warp's stores are whole lines
template <int KT>
__global__ void __launch_bounds__(256) mx4_dequantize_kernel(const uint8_t *__restrict__ codes,
                                                            const uint8_t *__restrict__ scales, long long n,
                                                            void *__restrict__ out, int out_type) {
  const int type = known_type<KT>(out_type);
  // its dependents start when it ends: what it writes may be router weights, which a layer call reads early
  pdl_wait();
  const long long stride = (long long)gridDim.x * 256;
  constexpr int kAhead = 4;
  for (long long i0 = (long long)blockIdx.x * 256 + threadIdx.x; i0 < n; i0 += kAhead * stride) {
    uint32_t c[kAhead], b[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const long long i = i0 + j * stride;
      if (i >= n) continue;
      c[j] = reinterpret_cast<const uint32_t *>(codes)[i];
      b[j] = scales[i >> 2];
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const long long i = i0 + j * stride;
      if (i >= n) continue;
      const float d = e8m0_to_float(b[j]);
      float v[8];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float2 f = e2m1_values((c[j] >> (8 * q)) & 255u, d);
        v[2 * q] = f.x;
        v[2 * q + 1] = f.y;
      }
      store8(out, type, (size_t)i * 8, v);
    }
  }
}

int thread_grid(long long n) {
  const long long want = (n + 255) / 256, cap = (long long)num_sms() * 16;
  return (int)(want < cap ? want : cap);
}

// calls f with what is known of a type at compile time
template <class F>
cudaError_t by_type(int type, const F &f) {
  using std::integral_constant;
  if (type == kF32Wide) return f(integral_constant<int, kF32Wide>{});
  if (type == MOE_F16) return f(integral_constant<int, MOE_F16>{});
  if (type == MOE_BF16) return f(integral_constant<int, MOE_BF16>{});
  return f(integral_constant<int, kAny>{});
}

}  // namespace

cudaError_t launch_mx4_quantize(const void *x, int type, int T, int K, const int32_t *row_of, int k,
                                const int32_t *kept, uint8_t *codes, uint8_t *scales, cudaStream_t s) {
  KTimer kt_(KID_MX4_QUANTIZE, s);
  type = kernel_type(type, x);
  return by_type(type, [&](auto kt) {
    return launch_pdl(mx4_quantize_kernel<kt.value>, dim3(thread_grid((long long)T * (K / 32))), dim3(256), 0, s, x, type,
                      T, K, row_of, row_of ? k : 1, kept, codes, scales);
  });
}

cudaError_t launch_mx4_dequantize(const uint8_t *codes, const uint8_t *scales, long long rows, int K, void *out,
                                  int type, cudaStream_t s) {
  KTimer kt_(KID_MX4_DEQUANTIZE, s);
  const long long n = rows * (K / 8);
  type = kernel_type(type, out);
  return by_type(type, [&](auto kt) {
    return launch_pdl(mx4_dequantize_kernel<kt.value>, dim3(thread_grid((n + 3) / 4)), dim3(256), 0, s, codes, scales, n,
                      out, type);
  });
}

}  // namespace moe
