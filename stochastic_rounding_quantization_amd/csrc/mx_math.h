// MXFP4 element arithmetic and code layout, shared by the quantized backward
// and the forward rows and products.
#pragma once

#include "s3r_internal.h"

namespace s3r {

// Code layout of every MXFP4 matrix (R rows, K contraction elements, two codes a byte): blocks of
// 256 rows x 128 elements, 64 bytes a row and 16 KiB a block, row-major inside; block (rb, kb)
// starts at rb * ld + kb * 16384 (ld >= 128 K, the stride between 256-row blocks). A GEMM step of
// a 256-row tile is then one contiguous 16 KiB run, which its DMA reads in whole cache lines.
constexpr int kMxBlkBytes = 16384;
__device__ __forceinline__ int64_t mx_code_off(int64_t row, int64_t byte, int64_t ld) {
  return (row >> 8) * ld + (byte >> 6) * kMxBlkBytes + (row & 255) * 64 + (byte & 63);
}

// ------------------------------------------------------ E2M1 rounding ----
// Block exponent of amax bits (ordered fp32 bits): the smallest k with
// a <= 6 * 2^k, clamped; returns 255 (NaN) for a non-finite max.
__device__ __forceinline__ int block_scale_byte(uint32_t abits) {
  if (!(abits < 0x7F800000u)) return 255;
  if (abits == 0) return 0;                                       // k = -127
  int E;
  const float m = __builtin_frexpf(__uint_as_float(abits), &E);  // a = m 2^E, m in [0.5, 1)
  int k = m <= 0.75f ? E - 3 : E - 2;
  k = k < -127 ? -127 : (k > 127 ? 127 : k);
  return k + 127;
}


// E2M1 code of v in a block with scale exponent k (kp1 = k + 1), on the
// block's grid in units of the spacing s = 2^(M - k - 2), M = max(e(v), k + 1)
// with e(v) the frexp exponent (|v| = m 2^e, m in [0.5, 1)), taken from the
// exponent field (zero and subnormals give -126 <= k + 1): s is 0.5, 1 or 2
// as |v / 2^k| lies below 2, in [2, 4) or in [4, 6].  t = v / s * 2^24 is an
// exact power-of-two scaling; n = floor(t / 2^24 + R / 2^24) = (floor(t) + R)
// >> 24 (SR / S3R, R the threshold in units of 2^-24) or rint(v / s) (RTNE).
// |n| + 2 (M - k - 1) is the index into 0, 0.5, 1, 1.5, 2, 3, 4, 6, and the
// dequantized value n s 2^k = n 2^(M - 2).
template <bool RT>
__device__ __forceinline__ uint32_t e2m1_round(float v, int kp1, int32_t R, int& n, int& M) {
  M = max((int)((__float_as_uint(v) >> 23) & 0xFFu) - 126, kp1);
  if constexpr (RT) {
    n = (int)__builtin_rintf(__builtin_ldexpf(v, 2 - M));
  } else {
    const float t = __builtin_ldexpf(v, 26 - M);
    int32_t X;
    asm("v_cvt_flr_i32_f32 %0, %1" : "=v"(X) : "v"(t));
    n = (X + R) >> 24;
  }
  const uint32_t idx = (uint32_t)(abs(n) + 2 * (M - kp1));
  return (n < 0 ? 8u : 0u) | idx;
}

}  // namespace s3r
