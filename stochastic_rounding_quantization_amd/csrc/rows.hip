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
// order and experts' order, and with many tokens are bound by HBM: a token's side
// is read or written once, whatever k is.  A thread of combine loads its rows one
// after another (the other waves of the CU cover that: two choices run at a
// large copy's rate); the backward has the rows of up to four choices in flight.
// With few tokens latency bounds them: 16 tokens x 8 x 4096, combine 6.0 us.
#include "s3r_internal.h"

namespace s3r {
namespace {

constexpr int kRowThreads = 256;

typedef uint32_t v4u32_a2 __attribute__((ext_vector_type(4), aligned(2)));     // 16 bytes at a bf16's alignment
typedef uint32_t v4u32_a4 __attribute__((ext_vector_type(4), aligned(4)));     // at an f32's

// Chunks of W elements: 16 bytes of the row type (8 bf16, 4 f32), or one element for rows shorter than that.  Rows
// that are not 16-byte aligned (odd widths, slices) take the same accesses at their elements' alignment.  16384 tokens,
// 2 rows each, 2047 bf16 columns, us, element by element and so: dispatch 113 and 37, combine 155 and 42,
// backward 131 and 70 (2048 columns: 34, 37, 63).
template <typename T, int W, bool NT = false>
struct Chunk {
  // NT: the nontemporal hint, where it measured faster.  16384 tokens, 2 rows each, 2048 bf16 columns, us:
  //   combine:  none 41.3, row loads 37.5, stores 39.4, both 38.3        (202 MB: 5.4 TB/s, a large copy's rate)
  //   backward: none 75.1, row loads 74.0, row stores 78.8, both 67.0, both and dy 76.0      (336 MB: 5.0 TB/s)
  static __device__ __forceinline__ void load(const T* p, float (&v)[W]) {
    if constexpr (W == 1) {
      if constexpr (sizeof(T) == 2) v[0] = bf16_to_f32(*reinterpret_cast<const uint16_t*>(p));
      else v[0] = *p;
    } else if constexpr (sizeof(T) == 2) {
      const v4u32 w = word(p);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      }
    } else {
      const v4u32 w = word(p);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(w[i]);
    }
  }
  static __device__ __forceinline__ v4u32 word(const T* p) {
    if constexpr (sizeof(T) == 2) {
      const v4u32_a2* q = reinterpret_cast<const v4u32_a2*>(p);
      return NT ? __builtin_nontemporal_load(q) : *q;
    } else {
      const v4u32_a4* q = reinterpret_cast<const v4u32_a4*>(p);
      return NT ? __builtin_nontemporal_load(q) : *q;
    }
  }
  static __device__ __forceinline__ void put(T* p, v4u32 w) {
    if constexpr (sizeof(T) == 2) {
      v4u32_a2* q = reinterpret_cast<v4u32_a2*>(p);
      if constexpr (NT) __builtin_nontemporal_store(w, q); else *q = w;
    } else {
      v4u32_a4* q = reinterpret_cast<v4u32_a4*>(p);
      if constexpr (NT) __builtin_nontemporal_store(w, q); else *q = w;
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
      else put(p, v4u32{w[0], w[1], w[2], w[3]});
    } else {
      if constexpr (W == 1) *p = v[0];
      else put(p, v4u32{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])});
    }
  }
};

// One thread per (token, chunk); the last chunk of a row ends with the row, over the one before it.
template <typename T, int W>
__global__ __launch_bounds__(kRowThreads) void dispatch_kernel(RowMoveArgs a, int chunks) {
  const int64_t i = wide_block() * kRowThreads + threadIdx.x;
  const int64_t t = i / chunks;
  if (t >= a.T) return;
  const int64_t c = min((i - t * chunks) * W, a.D - W);
  float v[W];
  Chunk<T, W>::load((const T*)a.in + t * a.ld_in + c, v);
  for (int j = 0; j < a.K; ++j) {
    const int64_t r = a.slot_row[t * a.K + j];
    if (r >= 0 && r < a.R) Chunk<T, W>::store((T*)a.out + r * a.ld_out + c, v);
  }
}

template <typename T, int W>
__global__ __launch_bounds__(kRowThreads) void combine_kernel(RowMoveArgs a, int chunks) {
  const int64_t i = wide_block() * kRowThreads + threadIdx.x;
  const int64_t t = i / chunks;
  if (t >= a.T) return;
  const int64_t c = min((i - t * chunks) * W, a.D - W);
  float s[W];
#pragma unroll
  for (int q = 0; q < W; ++q) s[q] = 0.f;
  for (int j = 0; j < a.K; ++j) {
    const int64_t r = a.slot_row[t * a.K + j];
    if (r < 0 || r >= a.R) continue;
    const float w = a.weights ? a.weights[t * a.K + j] : 1.f;
    float v[W];
    Chunk<T, W, true>::load((const T*)a.in + r * a.ld_in + c, v);
#pragma unroll
    for (int q = 0; q < W; ++q) s[q] = fmaf(w, v[q], s[q]);
  }
  Chunk<T, W>::store((T*)a.out + t * a.ld_out + c, s);
}

// One wave per token and J of its choices: its dy chunk is read once for them; the dot products are lane
// sums joined across the wave.
template <typename T, int W, int J>
__device__ __forceinline__ void combine_backward_choices(const RowMoveArgs& a, int64_t t, int j0, int lane) {
  int64_t r[J];
  float w[J], dot[J];
  bool ok[J];
#pragma unroll
  for (int j = 0; j < J; ++j) {
    r[j] = a.slot_row[t * a.K + j0 + j];
    ok[j] = r[j] >= 0 && r[j] < a.R;
    w[j] = a.weights[t * a.K + j0 + j];
    dot[j] = 0.f;
  }
  for (int64_t at = (int64_t)lane * W; at < a.D; at += 64 * W) {
    const int64_t c = min(at, a.D - W);          // the last chunk ends with the row
    float g[W], y[J][W];
    Chunk<T, W>::load((const T*)a.dy + t * a.ld_dy + c, g);
#pragma unroll
    for (int j = 0; j < J; ++j)
      if (ok[j]) Chunk<T, W, true>::load((const T*)a.in + r[j] * a.ld_in + c, y[j]);
#pragma unroll
    for (int j = 0; j < J; ++j) {
      if (!ok[j]) continue;
      float o[W];
#pragma unroll
      for (int q = 0; q < W; ++q) {
        if (W == 1 || c + q >= at) dot[j] = fmaf(g[q], y[j][q], dot[j]);
        o[q] = g[q] * w[j];
      }
      Chunk<T, W, true>::store((T*)a.out + r[j] * a.ld_out + c, o);
    }
  }
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const float d = wave_sum(dot[j]);
    if (lane == 0) a.dweights[t * a.K + j0 + j] = d;
  }
}

template <typename T, int W>
__global__ __launch_bounds__(kRowThreads) void combine_backward_kernel(RowMoveArgs a) {
  const int lane = threadIdx.x & 63;
  const int64_t t = wide_block() * (kRowThreads / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (t >= a.T) return;
  int j = 0;
  for (; j + 4 <= a.K; j += 4) combine_backward_choices<T, W, 4>(a, t, j, lane);
  if (j + 2 <= a.K) {
    combine_backward_choices<T, W, 2>(a, t, j, lane);
    j += 2;
  }
  if (j < a.K) combine_backward_choices<T, W, 1>(a, t, j, lane);
}

template <typename T>
void run_rows(const RowMoveArgs& a, int what, hipStream_t st) {
  constexpr int W = 16 / (int)sizeof(T);
  const bool vec = a.D >= W;
  const int chunks = (int)(vec ? (a.D + W - 1) / W : a.D);
  const dim3 grid = wide_grid((a.T * chunks + kRowThreads - 1) / kRowThreads), block(kRowThreads);
  const dim3 bgrid = wide_grid((a.T + kRowThreads / 64 - 1) / (kRowThreads / 64));
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
