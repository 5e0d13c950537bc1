// Forward products on MXFP4 operands: rows of any number and any length rounded
// to E2M1 with one E8M0 scale per 32 elements (RTNE, the format and block layout
// of the MXFP4 backward), and y = dq(A) dq(B)^T, dense or over expert-sorted
// rows with one B per group, on the block-scaled FP4 matrix cores.
//
// The contraction K is padded to whole steps of 128 elements with zero codes, so
// K, like the rows and the columns, can have any size.
#include "mx_math.h"
#include "swiglu_math.h"

namespace s3r {
namespace {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));

// ------------------------------------------------------------------ rows ----
// A block of 256 threads takes 16 rows x one 128-element step at a time: 16 lanes
// per row, 8 elements a lane (16 bytes of bf16), so a block of 32 elements is
// four lanes.  Codes leave as 1 KiB and scales as 64 bytes in one run.  With
// `up` the element is silu(A) * up in fp32, not rounded in between.
constexpr int kMrThreads = 256, kMrRows = 16;

template <typename TIn>
__device__ __forceinline__ void mr_load8(const TIn* p, int64_t n, bool vec, float (&v)[8]) {
  if (vec && n >= 8) {
    if constexpr (sizeof(TIn) == 2) {
      const uint4 w = *reinterpret_cast<const uint4*>(p);
      const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(ww[i] << 16);
        v[2 * i + 1] = __uint_as_float(ww[i] & 0xFFFF0000u);
      }
    } else {
      const float4 w0 = reinterpret_cast<const float4*>(p)[0], w1 = reinterpret_cast<const float4*>(p)[1];
      v[0] = w0.x; v[1] = w0.y; v[2] = w0.z; v[3] = w0.w;
      v[4] = w1.x; v[5] = w1.y; v[6] = w1.z; v[7] = w1.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if constexpr (sizeof(TIn) == 2) v[i] = i < n ? bf16_to_f32(*reinterpret_cast<const uint16_t*>(p + i)) : 0.f;
      else v[i] = i < n ? p[i] : 0.f;
    }
  }
}

// silu(a) * u in fp32 with the glue's exponential and reciprocal.
__device__ __forceinline__ float mr_swiglu(float a, float u) {
  const float d = 1.f + glue_exp32(-a);
  const float s = glue_slow_recip(d) ? __fdiv_rn(1.f, d) : glue_recip(d);
  return (a * s) * u;
}

// The codes of this lane's 8 elements (one word) and, in every lane of the row's 16, its step's four
// scale bytes; lanes 4 b .. 4 b + 3 hold block b.
__device__ __forceinline__ uint32_t mr_encode(const float (&v)[8], uint32_t& scales) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  m = max(m, (uint32_t)__shfl_xor((int)m, 1, 64));
  m = max(m, (uint32_t)__shfl_xor((int)m, 2, 64));
  const int sb = block_scale_byte(m);
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    int n, M;
    w |= e2m1_round<true>(v[i], sb - 126, 0, n, M) << (4 * i);
  }
  uint32_t s = (uint32_t)sb << (8 * ((threadIdx.x >> 2) & 3));
  s |= (uint32_t)__shfl_xor((int)s, 4, 64);
  s |= (uint32_t)__shfl_xor((int)s, 8, 64);
  scales = s;
  return sb == 255 ? 0u : w;
}

__device__ __forceinline__ bool mr_nan_scale(uint32_t s) {
  return (s & 0xFFu) == 0xFFu || (s & 0xFF00u) == 0xFF00u || (s & 0xFF0000u) == 0xFF0000u || (s >> 24) == 0xFFu;
}

template <typename TIn>
__global__ __launch_bounds__(kMrThreads) void mx_rows_kernel(MxRowsArgs a, int ksteps) {
  const int sub = threadIdx.x & 15;
  const int64_t r = (int64_t)blockIdx.x * kMrRows + (threadIdx.x >> 4);
  const int64_t g = blockIdx.z;
  const TIn* A = (const TIn*)a.A + g * a.a_stride;
  const TIn* U = a.up ? (const TIn*)a.up + g * a.a_stride : nullptr;
  uint8_t* codes = a.codes + g * a.c_stride;
  uint8_t* scales = a.scales + g * a.s_stride;
  int64_t src = r;
  bool live = r < a.R;
  if (a.index && live) {
    src = (int64_t)a.index[r] / a.index_div;
    live = a.index[r] >= 0 && src < a.a_rows;     // an index outside the source is a row of zeros
  }
  if (!live) src = 0;
  for (int kt = blockIdx.y; kt < ksteps; kt += gridDim.y) {
    const int64_t c = (int64_t)kt * 128 + sub * 8;
    const int64_t n = live ? a.K - c : 0;
    float v[8];
    mr_load8<TIn>(A + src * a.ld + c, n, a.vec != 0, v);
    if (U) {
      float u[8];
      mr_load8<TIn>(U + src * a.ld + c, n, a.vec != 0, u);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = i < n ? mr_swiglu(v[i], u[i]) : 0.f;
    }
    uint32_t s;
    const uint32_t w = mr_encode(v, s);
    if (r < a.R) {
      *reinterpret_cast<uint32_t*>(codes + mx_code_off(r, (int64_t)kt * 64 + sub * 4, a.ld_c)) = w;
      if (sub == 0) {
        *reinterpret_cast<uint32_t*>(scales + (int64_t)kt * a.ld_s + 4 * r) = s;
        if (a.flags && mr_nan_scale(s)) atomicOr(a.flags, S3R_FLAG_NONFINITE);
      }
    }
  }
}

// --------------------------------------------------------------- groups ----
// The m-tile i of `tile` rows in a grouped product: its group e, its first row and the group's end,
// found by one wave from the offsets themselves (prefix sums of the groups' tile counts, 64 groups a
// round).  e = -1 past the last tile.  bad: the offsets are not a non-decreasing sequence from 0 to R.
struct GroupTile { int e; int64_t r0, r1; bool bad; };
__device__ __forceinline__ GroupTile find_group_tile(const int64_t* __restrict__ offsets, int64_t G, int64_t R, int64_t i,
                                                     int tile) {
  const int lane = threadIdx.x & 63;
  GroupTile h{-1, 0, 0, false};
  int64_t carry = 0;                          // tiles of the groups before this round's
  bool bad = lane == 0 && (offsets[0] != 0 || offsets[G] != R);
  for (int64_t g0 = 0; g0 < G; g0 += 64) {
    const int64_t g = g0 + lane;
    const int64_t o0 = g < G ? offsets[g] : 0, o1 = g < G ? offsets[g + 1] : 0;
    bad |= o1 < o0 || o0 < 0 || o1 > R;
    const int64_t n = bad ? 0 : (o1 - o0 + tile - 1) / tile;
    int64_t s = n;
    for (int o = 1; o < 64; o <<= 1) {
      const int64_t b = __shfl_up(s, o, 64);
      if (lane >= o) s += b;
    }
    const bool hit = carry + s > i && carry + s - n <= i;
    const uint64_t m = __builtin_amdgcn_ballot_w64(hit);
    if (m && h.e < 0) {
      const int w = __builtin_ctzll(m);
      h.e = (int)g0 + w;
      h.r1 = __shfl(o1, w, 64);
      h.r0 = __shfl(o0 + (i - (carry + s - n)) * tile, w, 64);
    }
    carry += __shfl(s, 63, 64);
  }
  h.bad = __builtin_amdgcn_ballot_w64(bad) != 0;
  return h;
}

// -------------------------------------------------------------- products ----
struct MxProdK {
  const uint8_t* A; int64_t lda; const uint8_t* As; int64_t ldas;
  const uint8_t* B; int64_t ldb; const uint8_t* Bs; int64_t ldbs;
  int64_t b_stride, bs_stride;
  const int64_t* offsets; int64_t G;          // G = 0: dense
  int64_t M, N; int ksteps, tiles_n;
  void* out; int64_t ld_out;
  uint32_t* flags;
};

__device__ __forceinline__ void store_out(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_out(uint16_t* p, float v) {
  *reinterpret_cast<__bf16*>(p) = (__bf16)v;
}

// Few rows: 16 rows x 16 NJ columns per workgroup, the K steps dealt to its four waves, whose sums are
// joined in LDS in wave order.  Fragments go straight from memory to the matrix cores
// (v_mfma_scale_f32_16x16x128_f8f6f4: lane l holds row or column l % 16, K elements 32 (l / 16) .. + 31,
// 16 bytes, and that block's scale; the result's register r is row 4 (l / 16) + r, column l % 16): 16
// rows of a step are one contiguous KiB of the code layout.
constexpr int kSkThreads = 256;
template <typename TOut, int NJ>
__global__ __launch_bounds__(kSkThreads) void mx_few_rows_kernel(MxProdK p) {
  __shared__ float part[3][NJ][256];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int64_t m0, m1;
  const uint8_t *B = p.B, *Bs = p.Bs;
  const int mt = blockIdx.x / p.tiles_n, nt = blockIdx.x - mt * p.tiles_n;
  if (p.G) {
    const GroupTile h = find_group_tile(p.offsets, p.G, p.M, mt, 16);
    if (h.bad) {
      if (blockIdx.x == 0 && threadIdx.x == 0 && p.flags) atomicOr(p.flags, S3R_FLAG_BAD_GROUPS);
      return;
    }
    if (h.e < 0) return;
    m0 = h.r0;
    m1 = min(h.r1, m0 + 16);
    B += h.e * p.b_stride;
    Bs += h.e * p.bs_stride;
  } else {
    m0 = (int64_t)mt * 16;
    m1 = min(p.M, m0 + 16);
  }
  const int64_t n0 = (int64_t)nt * (16 * NJ);
  const int r15 = lane & 15, kb = lane >> 4;
  // rows and columns past the end repeat the last one; their results are not stored
  const int64_t ar = min(m0 + r15, m1 - 1);
  const uint8_t* pa = p.A + (ar >> 8) * p.lda + (ar & 255) * 64 + kb * 16;
  const uint8_t* psa = p.As + 4 * ar + kb;
  const uint8_t *pb[NJ], *psb[NJ];
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    const int64_t br = min(n0 + 16 * j + r15, p.N - 1);
    pb[j] = B + (br >> 8) * p.ldb + (br & 255) * 64 + kb * 16;
    psb[j] = Bs + 4 * br + kb;
  }
  v4f acc[NJ];
#pragma unroll
  for (int j = 0; j < NJ; ++j) acc[j] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int kt = wave; kt < p.ksteps; kt += kSkThreads / 64) {
    const uint4 x = *reinterpret_cast<const uint4*>(pa + (int64_t)kt * kMxBlkBytes);
    const int sa = psa[kt * p.ldas];
    const v8i fa = v8i{(int)x.x, (int)x.y, (int)x.z, (int)x.w, 0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const uint4 y = *reinterpret_cast<const uint4*>(pb[j] + (int64_t)kt * kMxBlkBytes);
      const int sb = psb[j][kt * p.ldbs];
      const v8i fb = v8i{(int)y.x, (int)y.y, (int)y.z, (int)y.w, 0, 0, 0, 0};
      acc[j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fa, fb, acc[j], 4, 4, 0, sa, 0, sb);
    }
  }
  if (wave > 0) {
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r) part[wave - 1][j][r * 64 + lane] = acc[j][r];
  }
  __syncthreads();
  if (wave > 0) return;
  TOut* out = (TOut*)p.out;
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    const int64_t n = n0 + 16 * j + r15;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int64_t m = m0 + 4 * kb + r;
      const float v = ((acc[j][r] + part[0][j][r * 64 + lane]) + part[1][j][r * 64 + lane]) + part[2][j][r * 64 + lane];
      if (n < p.N && m < m1) store_out(out + m * p.ld_out + n, v);
    }
  }
}

}  // namespace

size_t mx_rows_codes_bytes(int64_t R, int64_t K) { return (size_t)((R + 255) / 256) * (size_t)((K + 127) / 128) * kMxBlkBytes; }
size_t mx_rows_scales_bytes(int64_t R, int64_t K) { return (size_t)((K + 127) / 128) * (size_t)R * 4; }

hipError_t launch_mx_rows(const MxRowsArgs& a, hipStream_t st) {
  if (a.R == 0 || a.K == 0 || a.G == 0) return hipSuccess;
  MxRowsArgs b = a;
  const int esize = a.dtype == S3R_BF16 ? 2 : 4;
  b.vec = ((uintptr_t)a.A & 15u) == 0 && ((uintptr_t)a.up & 15u) == 0 && (a.ld * esize) % 16 == 0 &&
          (a.a_stride * esize) % 16 == 0;
  const int ksteps = (int)((a.K + 127) / 128);
  const dim3 grid((unsigned)((a.R + kMrRows - 1) / kMrRows), (unsigned)std::min(ksteps, 65535), (unsigned)a.G);
  if (a.dtype == S3R_BF16) hipLaunchKernelGGL((mx_rows_kernel<uint16_t>), grid, dim3(kMrThreads), 0, st, b, ksteps);
  else hipLaunchKernelGGL((mx_rows_kernel<float>), grid, dim3(kMrThreads), 0, st, b, ksteps);
  return hipGetLastError();
}

hipError_t launch_mx_product(const MxProductArgs& a, hipStream_t st) {
  if (a.M == 0 || a.N == 0) return hipSuccess;
  MxProdK p{};
  p.A = a.A; p.lda = a.lda; p.As = a.As; p.ldas = a.ldas;
  p.B = a.B; p.ldb = a.ldb; p.Bs = a.Bs; p.ldbs = a.ldbs; p.b_stride = a.b_stride; p.bs_stride = a.bs_stride;
  p.offsets = a.offsets; p.G = a.G; p.M = a.M; p.N = a.N; p.ksteps = (int)((a.K + 127) / 128);
  p.out = a.out; p.ld_out = a.ld_out; p.flags = a.flags;
  // grouped: the tiles of every group, at most one partial tile each
  const int64_t mt = a.G ? a.M / 16 + std::min(a.G, a.M) : (a.M + 15) / 16;
  p.tiles_n = (int)((a.N + 31) / 32);
  if (mt * p.tiles_n > 0x7FFFFFFF) return hipErrorInvalidConfiguration;
  const dim3 grid((unsigned)(mt * p.tiles_n));
  if (a.out_dt == S3R_BF16) hipLaunchKernelGGL((mx_few_rows_kernel<uint16_t, 2>), grid, dim3(kSkThreads), 0, st, p);
  else hipLaunchKernelGGL((mx_few_rows_kernel<float, 2>), grid, dim3(kSkThreads), 0, st, p);
  return hipGetLastError();
}

}  // namespace s3r
