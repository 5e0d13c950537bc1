// Rows of any alignment in pieces of 8 elements, and silu(gate) * up of them; shared by what rounds rows to MXFP4
// and to INT8.
#pragma once

#include "swiglu_math.h"

namespace s3r {
namespace {

// 8 consecutive elements of a row as they lie in memory: packed bf16, or fp32.
template <typename TIn> struct Raw8;
template <> struct Raw8<uint16_t> { uint32_t w[4]; };
template <> struct Raw8<float> { float w[8]; };

// The 8 elements at p, of which the row of K has n left (none: zeros).  Words: 16-byte aligned rows with K a
// multiple of 8, so that n is 8 or more, or 0 or less (a path for fewer in an unrolled loop is code that has to
// be fetched, whether it runs or not: a kernel of few instructions per byte was twice as slow with it).  Else
// 16-byte loads at the elements' alignment, for a row's end the row's last 8, which mr_tail moves to their
// place once every load is on its way; element by element where K < 8.  8192 x 4095 bf16: 36 us with elements
// alone, 16 so (8192 x 4096: 14.5); fp32 61 and 28.
typedef uint32_t mr_u4_a2 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t mr_u4_a4 __attribute__((ext_vector_type(4), aligned(4)));
template <typename TIn, bool Words>
__device__ __forceinline__ Raw8<TIn> mr_load8(const TIn* p, int64_t n, int64_t K) {
  Raw8<TIn> r;
  if constexpr (sizeof(TIn) == 2) {
    if constexpr (Words) {
      const uint4 w = n > 0 ? *reinterpret_cast<const uint4*>(p) : make_uint4(0u, 0u, 0u, 0u);
      r.w[0] = w.x; r.w[1] = w.y; r.w[2] = w.z; r.w[3] = w.w;
    } else if (K >= 8) {
      v4u32 w = {0u, 0u, 0u, 0u};
      if (n > 0) w = *reinterpret_cast<const mr_u4_a2*>(p + (n < 8 ? n - 8 : 0));
#pragma unroll
      for (int i = 0; i < 4; ++i) r.w[i] = w[i];
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        r.w[i] = (2 * i < n ? (uint32_t)p[2 * i] : 0u) | (2 * i + 1 < n ? (uint32_t)p[2 * i + 1] << 16 : 0u);
    }
  } else {
    if (Words || K >= 8) {
      v4u32 a = {0u, 0u, 0u, 0u}, b = a;
      if (n > 0) {                     // one branch for both words: with one each, 8192 x 4096 took 60 us instead of 28
        if constexpr (Words) {
          a = reinterpret_cast<const v4u32*>(p)[0];
          b = reinterpret_cast<const v4u32*>(p)[1];
        } else {
          const mr_u4_a4* q = reinterpret_cast<const mr_u4_a4*>(p + (n < 8 ? n - 8 : 0));
          a = q[0];
          b = q[1];
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) { r.w[i] = __uint_as_float(a[i]); r.w[4 + i] = __uint_as_float(b[i]); }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) r.w[i] = i < n ? p[i] : 0.f;
    }
  }
  return r;
}

// The row's last 8 elements to its last n, 0 < n < 8, and zeros after them.
template <bool Words>
__device__ __forceinline__ void mr_tail(Raw8<uint16_t>& r, int64_t n, int64_t K) {
  if constexpr (!Words)
    if (n > 0 && n < 8 && K >= 8) {
      const int by = 16 * (8 - (int)n);
      uint64_t lo = (uint64_t)r.w[1] << 32 | r.w[0], hi = (uint64_t)r.w[3] << 32 | r.w[2];
      lo = by < 64 ? lo >> by | hi << (64 - by) : hi >> (by - 64);
      hi = by < 64 ? hi >> by : 0;
      r.w[0] = (uint32_t)lo; r.w[1] = (uint32_t)(lo >> 32);
      r.w[2] = (uint32_t)hi; r.w[3] = (uint32_t)(hi >> 32);
    }
}
template <bool Words>
__device__ __forceinline__ void mr_tail(Raw8<float>& r, int64_t n, int64_t K) {
  if constexpr (!Words)
    if (n > 0 && n < 8 && K >= 8) {
      const int by = 8 - (int)n;
#pragma unroll
      for (int o = 4; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < 8; ++i) r.w[i] = by & o ? (i + o < 8 ? r.w[i + o] : 0.f) : r.w[i];
    }
}

__device__ __forceinline__ Raw8<float> mr_float8(const Raw8<float>& r) { return r; }
__device__ __forceinline__ Raw8<float> mr_float8(const Raw8<uint16_t>& r) {
  Raw8<float> f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f.w[2 * i] = __uint_as_float(r.w[i] << 16);
    f.w[2 * i + 1] = __uint_as_float(r.w[i] & 0xFFFF0000u);
  }
  return f;
}

// silu(a) * u in fp32 with the glue's exponential and reciprocal.
__device__ __forceinline__ float mr_swiglu(float a, float u) {
  const float d = 1.f + glue_exp32(-a);
  const float s = glue_slow_recip(d) ? __fdiv_rn(1.f, d) : glue_recip(d);
  return (a * s) * u;
}

template <int Ctrl>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, Ctrl, 0xF, 0xF, true);
}
constexpr int kDppXor1 = 0xB1, kDppXor2 = 0x4E, kDppRor4 = 0x124, kDppRor8 = 0x128;

// Largest magnitude of the 8 elements, as fp32 bits.
__device__ __forceinline__ uint32_t mr_amax(const Raw8<float>& r) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(r.w[i]) & 0x7FFFFFFFu);
  return m;
}
__device__ __forceinline__ uint32_t mr_amax(const Raw8<uint16_t>& r) {
  typedef unsigned short u2 __attribute__((ext_vector_type(2)));
  u2 m = __builtin_bit_cast(u2, r.w[0] & 0x7FFF7FFFu);
#pragma unroll
  for (int i = 1; i < 4; ++i) m = __builtin_elementwise_max(m, __builtin_bit_cast(u2, r.w[i] & 0x7FFF7FFFu));
  return (uint32_t)(m.x > m.y ? m.x : m.y) << 16;
}

// The source row of row r, or -1: none (past the end, or an index outside the source).
template <typename TArgs>
__device__ __forceinline__ int64_t mr_source(const TArgs& a, int64_t r) {
  if (r >= a.R) return -1;
  if (!a.index) return r;
  const int i = a.index[r];
  if (i < 0) return -1;
  const int s = (int)((uint32_t)i / (uint32_t)a.index_div);
  return s < a.a_rows ? s : -1;
}

}  // namespace
}  // namespace s3r
