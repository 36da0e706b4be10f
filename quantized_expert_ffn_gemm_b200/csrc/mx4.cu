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

// the value of a code
__device__ __forceinline__ float e2m1_value(uint32_t c) {
  const uint32_t m = c & 7u;
  const float v = m < 2 ? 0.5f * (float)m : __uint_as_float(((126u + (m >> 1)) << 23) | ((m & 1u) << 22));
  return (c & 8u) ? -v : v;
}

// four lanes a block of 32 (eight values each); a token's codes and scales go to all its rows
__global__ void __launch_bounds__(256) mx4_quantize_kernel(const void *__restrict__ x, int type, int T, int K,
                                                          const int32_t *__restrict__ row_of, int k,
                                                          const int32_t *__restrict__ kept,
                                                          uint8_t *__restrict__ codes, uint8_t *__restrict__ scales) {
  const int K8 = K >> 3, P = T * k;
  const long long n = (long long)T * K8, stride = (long long)gridDim.x * 256;
  const long long n4 = (n + 31) / 32 * 32;  // every lane of a warp stays for the shuffles
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < n4; i += stride) {
    const bool ok = i < n;
    float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (ok) load8(x, type, (size_t)i * 8, v);
    uint32_t top = 0;  // the largest magnitude's bits: magnitudes order as their bits do, NaN above all
#pragma unroll
    for (int q = 0; q < 8; ++q) top = max(top, __float_as_uint(v[q]) & 0x7fffffffu);
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const int e = (int)(top >> 23);
    const uint32_t b = e == 255 ? 255u : (uint32_t)max(e - 2, 0);
    const float inv = __uint_as_float((254u - b) << 23);  // 2^(127 - b), b <= 252
    uint32_t c = 0;
    if (b != 255u) {
#pragma unroll
      for (int q = 0; q < 4; ++q) c |= e2m1_pair(v[2 * q] * inv, v[2 * q + 1] * inv) << (8 * q);
    }
    if (!ok) continue;
    const long long t = i / K8;
    const int col = (int)(i % K8);
    for (int j = 0; j < k; ++j) {
      const long long r = row_of ? row_of[t * k + j] : t;
      if (r < 0 || r >= P) continue;
      reinterpret_cast<uint32_t *>(codes)[r * K8 + col] = c;
      if ((col & 3) == 0) scales[r * (K8 >> 2) + (col >> 2)] = (uint8_t)b;
    }
  }
  if (!kept) return;
  // the rows behind the last kept pair hold zeros
  const long long w0 = (long long)min(max(*kept, 0), P) * K8;
  for (long long i = w0 + (long long)blockIdx.x * 256 + threadIdx.x; i < (long long)P * K8; i += stride) {
    reinterpret_cast<uint32_t *>(codes)[i] = 0;
    if ((i & 3) == 0) scales[i >> 2] = 0;
  }
}

__global__ void __launch_bounds__(256) mx4_dequantize_kernel(const uint8_t *__restrict__ codes,
                                                            const uint8_t *__restrict__ scales, long long n,
                                                            void *__restrict__ out, int type) {
  const long long stride = (long long)gridDim.x * 256;
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < n; i += stride) {
    const uint32_t c = reinterpret_cast<const uint32_t *>(codes)[i];
    const float d = e8m0_to_float(scales[i >> 2]);
    float v[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) v[q] = e2m1_value((c >> (4 * q)) & 15u) * d;
    store8(out, type, (size_t)i * 8, v);
  }
}

int thread_grid(long long n) {
  const long long want = (n + 255) / 256, cap = (long long)num_sms() * 16;
  return (int)(want < cap ? want : cap);
}

}  // namespace

cudaError_t launch_mx4_quantize(const void *x, int type, int T, int K, const int32_t *row_of, int k,
                                const int32_t *kept, uint8_t *codes, uint8_t *scales, cudaStream_t s) {
  KTimer kt_(KID_MX4_QUANTIZE, s);
  mx4_quantize_kernel<<<thread_grid((long long)T * (K / 8)), 256, 0, s>>>(x, type, T, K, row_of, row_of ? k : 1, kept,
                                                                         codes, scales);
  return cudaGetLastError();
}

cudaError_t launch_mx4_dequantize(const uint8_t *codes, const uint8_t *scales, long long rows, int K, void *out,
                                  int type, cudaStream_t s) {
  KTimer kt_(KID_MX4_DEQUANTIZE, s);
  const long long n = rows * (K / 8);
  mx4_dequantize_kernel<<<thread_grid(n), 256, 0, s>>>(codes, scales, n, out, type);
  return cudaGetLastError();
}

}  // namespace moe
