// Tokens to the experts' rows and back: the spread of token rows over their
// expert-sorted rows (dispatch), the weighted sum of a token's expert outputs
// (combine) and the gradients of that sum.
//
// slot_row [T x k] names the row of each (token, choice) slot, as s3r_route
// writes it; an index outside [0, R) is no row: it adds nothing, gets nothing
// and its weight's gradient is 0.
//   dispatch   rows[slot_row[t,j]] = X[t]
//   combine    y[t] = sum_j w[t,j] Y[slot_row[t,j]]        (w = 1 without weights)
//   backward   dY[slot_row[t,j]] = w[t,j] dy[t];  dw[t,j] = <dy[t], Y[slot_row[t,j]]>
// fp32 sums in the order of j (of the columns within a lane, then across lanes),
// one rounding to the output's type.  All three move whole rows between tokens'
// order and experts' order and are bound by HBM.
#include "s3r_internal.h"

namespace s3r {
namespace {

constexpr int kRowThreads = 256;

// Chunks of W elements: 16 bytes of the row type (8 bf16, 4 f32), or one element for rows that are not
// 16-byte aligned.
template <typename T, int W>
struct Chunk {
  static __device__ __forceinline__ void load(const T* p, float (&v)[W]) {
    if constexpr (W == 1) {
      if constexpr (sizeof(T) == 2) v[0] = bf16_to_f32(*reinterpret_cast<const uint16_t*>(p));
      else v[0] = *p;
    } else if constexpr (sizeof(T) == 2) {
      const uint4 w = *reinterpret_cast<const uint4*>(p);
      const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(ww[i] << 16);
        v[2 * i + 1] = __uint_as_float(ww[i] & 0xFFFF0000u);
      }
    } else {
      const float4 w = *reinterpret_cast<const float4*>(p);
      v[0] = w.x; v[1] = w.y; v[2] = w.z; v[3] = w.w;
    }
  }
  static __device__ __forceinline__ void store(T* p, const float (&v)[W]) {
    typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
    typedef float f2 __attribute__((ext_vector_type(2)));
    if constexpr (sizeof(T) == 2) {
      uint32_t w[(W + 1) / 2];
#pragma unroll
      for (int i = 0; i < (W + 1) / 2; ++i) {
        const f2 q = {v[2 * i], W == 1 ? 0.f : v[(2 * i + 1) % W]};
        w[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(q, bf2));
      }
      if constexpr (W == 1) *reinterpret_cast<uint16_t*>(p) = (uint16_t)w[0];
      else *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
      if constexpr (W == 1) *p = v[0];
      else *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    }
  }
};

// One thread per (token, chunk).
template <typename T, int W>
__global__ __launch_bounds__(kRowThreads) void dispatch_kernel(RowMoveArgs a, int chunks) {
  const int64_t i = (int64_t)blockIdx.x * kRowThreads + threadIdx.x;
  const int64_t t = i / chunks;
  if (t >= a.T) return;
  const int64_t c = (i - t * chunks) * W;
  float v[W];
  Chunk<T, W>::load((const T*)a.in + t * a.ld_in + c, v);
  for (int j = 0; j < a.K; ++j) {
    const int64_t r = a.slot_row[t * a.K + j];
    if (r >= 0 && r < a.R) Chunk<T, W>::store((T*)a.out + r * a.ld_out + c, v);
  }
}

template <typename T, int W>
__global__ __launch_bounds__(kRowThreads) void combine_kernel(RowMoveArgs a, int chunks) {
  const int64_t i = (int64_t)blockIdx.x * kRowThreads + threadIdx.x;
  const int64_t t = i / chunks;
  if (t >= a.T) return;
  const int64_t c = (i - t * chunks) * W;
  float s[W];
#pragma unroll
  for (int q = 0; q < W; ++q) s[q] = 0.f;
  for (int j = 0; j < a.K; ++j) {
    const int64_t r = a.slot_row[t * a.K + j];
    if (r < 0 || r >= a.R) continue;
    const float w = a.weights ? a.weights[t * a.K + j] : 1.f;
    float v[W];
    Chunk<T, W>::load((const T*)a.in + r * a.ld_in + c, v);
#pragma unroll
    for (int q = 0; q < W; ++q) s[q] = fmaf(w, v[q], s[q]);
  }
  Chunk<T, W>::store((T*)a.out + t * a.ld_out + c, s);
}

// One wave per token: its dy chunk is read once for every choice; the dot products are lane sums joined
// across the wave.
template <typename T, int W>
__global__ __launch_bounds__(kRowThreads) void combine_backward_kernel(RowMoveArgs a) {
  const int lane = threadIdx.x & 63;
  const int64_t t = (int64_t)blockIdx.x * (kRowThreads / 64) + (threadIdx.x >> 6);
  if (t >= a.T) return;
  for (int j = 0; j < a.K; ++j) {
    const int64_t r = a.slot_row[t * a.K + j];
    const bool ok = r >= 0 && r < a.R;
    const float w = a.weights[t * a.K + j];
    float dot = 0.f;
    if (ok) {
      for (int64_t c = (int64_t)lane * W; c < a.D; c += 64 * W) {
        float g[W], y[W];
        Chunk<T, W>::load((const T*)a.dy + t * a.ld_dy + c, g);
        Chunk<T, W>::load((const T*)a.in + r * a.ld_in + c, y);
#pragma unroll
        for (int q = 0; q < W; ++q) {
          dot = fmaf(g[q], y[q], dot);
          g[q] *= w;
        }
        Chunk<T, W>::store((T*)a.out + r * a.ld_out + c, g);
      }
    }
    dot = wave_sum(dot);
    if (lane == 0) a.dweights[t * a.K + j] = dot;
  }
}

bool rows_vec(const void* p, int64_t ld, int64_t D, int esize) {
  return ((uintptr_t)p & 15u) == 0 && (ld * esize) % 16 == 0 && (D * esize) % 16 == 0;
}

template <typename T>
void run_rows(const RowMoveArgs& a, int what, hipStream_t st) {
  constexpr int W = 16 / (int)sizeof(T);
  const bool vec = rows_vec(a.in, a.ld_in, a.D, sizeof(T)) && rows_vec(a.out, a.ld_out, a.D, sizeof(T)) &&
                   (what != 2 || rows_vec(a.dy, a.ld_dy, a.D, sizeof(T)));
  const int chunks = (int)(vec ? a.D / W : a.D);
  const dim3 grid((unsigned)((a.T * chunks + kRowThreads - 1) / kRowThreads)), block(kRowThreads);
  const dim3 bgrid((unsigned)((a.T + kRowThreads / 64 - 1) / (kRowThreads / 64)));
  if (what == 0) {
    if (vec) hipLaunchKernelGGL((dispatch_kernel<T, W>), grid, block, 0, st, a, chunks);
    else hipLaunchKernelGGL((dispatch_kernel<T, 1>), grid, block, 0, st, a, chunks);
  } else if (what == 1) {
    if (vec) hipLaunchKernelGGL((combine_kernel<T, W>), grid, block, 0, st, a, chunks);
    else hipLaunchKernelGGL((combine_kernel<T, 1>), grid, block, 0, st, a, chunks);
  } else {
    if (vec) hipLaunchKernelGGL((combine_backward_kernel<T, W>), bgrid, block, 0, st, a);
    else hipLaunchKernelGGL((combine_backward_kernel<T, 1>), bgrid, block, 0, st, a);
  }
}

hipError_t launch_rows(const RowMoveArgs& a, int what, hipStream_t st) {
  if (a.T == 0 || (a.D == 0 && what != 2)) return hipSuccess;
  if (a.dtype == S3R_BF16) run_rows<uint16_t>(a, what, st);
  else run_rows<float>(a, what, st);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_dispatch(const RowMoveArgs& a, hipStream_t st) { return launch_rows(a, 0, st); }
hipError_t launch_combine(const RowMoveArgs& a, hipStream_t st) { return launch_rows(a, 1, st); }
hipError_t launch_combine_backward(const RowMoveArgs& a, hipStream_t st) { return launch_rows(a, 2, st); }

}  // namespace s3r
