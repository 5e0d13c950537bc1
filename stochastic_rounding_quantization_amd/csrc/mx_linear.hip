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
// A block of 256 threads takes 16 rows x kMrSteps 128-element steps: 16 lanes per
// row, 8 elements a lane and step (16 bytes of bf16), so a block of 32 elements
// is four lanes.  Codes leave as 1 KiB and scales as 64 bytes in one run.  With
// `up` the element is silu(A) * up in fp32, not rounded in between.
// The arithmetic is what bounded the first version (28 instructions an element:
// 35 us for 8192 x 4096 bf16, whose bytes need 15); now two elements convert in
// one instruction, and the maximum of bf16 runs on packed magnitudes.
constexpr int kMrThreads = 256, kMrRows = 16, kMrSteps = 4;

// 8 consecutive elements of a row as they lie in memory: packed bf16, or fp32.
template <typename TIn> struct Raw8;
template <> struct Raw8<uint16_t> { uint32_t w[4]; };
template <> struct Raw8<float> { float w[8]; };

// Elements past the first n are zero.
template <typename TIn>
__device__ __forceinline__ Raw8<TIn> mr_load8(const TIn* p, int64_t n, bool vec) {
  Raw8<TIn> r;
  if constexpr (sizeof(TIn) == 2) {
    if (vec && n >= 8) {
      const uint4 w = *reinterpret_cast<const uint4*>(p);
      r.w[0] = w.x; r.w[1] = w.y; r.w[2] = w.z; r.w[3] = w.w;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        r.w[i] = (2 * i < n ? (uint32_t)p[2 * i] : 0u) | (2 * i + 1 < n ? (uint32_t)p[2 * i + 1] << 16 : 0u);
    }
  } else {
    if (vec && n >= 8) {
      const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
      r.w[0] = a.x; r.w[1] = a.y; r.w[2] = a.z; r.w[3] = a.w;
      r.w[4] = b.x; r.w[5] = b.y; r.w[6] = b.z; r.w[7] = b.w;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) r.w[i] = i < n ? p[i] : 0.f;
    }
  }
  return r;
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

// Codes of 8 elements in a block of scale 2^(sb - 127), 1 <= sb <= 254: the hardware's conversion divides
// by the scale and rounds to nearest, ties to even.  Its sign survives a magnitude of 0; the format here
// has one zero.
__device__ __forceinline__ uint32_t mr_one_zero(uint32_t w) {
  const uint32_t mag = w & 0x77777777u;
  return mag | (w & (mag + 0x77777777u) & 0x88888888u);
}
__device__ __forceinline__ uint32_t mr_codes(const Raw8<float>& r, int sb) {
  const float scale = __uint_as_float((uint32_t)sb << 23);
  uint32_t w = 0;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, r.w[0], r.w[1], scale, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, r.w[2], r.w[3], scale, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, r.w[4], r.w[5], scale, 2);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, r.w[6], r.w[7], scale, 3);
  return mr_one_zero(w);
}
__device__ __forceinline__ uint32_t mr_codes(const Raw8<uint16_t>& r, int sb) {
  typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
  const float scale = __uint_as_float((uint32_t)sb << 23);
  uint32_t w = 0;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf2, r.w[0]), scale, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf2, r.w[1]), scale, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf2, r.w[2]), scale, 2);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf2, r.w[3]), scale, 3);
  return mr_one_zero(w);
}

template <int Ctrl>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, Ctrl, 0xF, 0xF, true);
}
constexpr int kDppXor1 = 0xB1, kDppXor2 = 0x4E, kDppRor4 = 0x124, kDppRor8 = 0x128;

// The codes of this lane's 8 elements (one word) and, in every lane of the row's 16, its step's four
// scale bytes; lanes 4 b .. 4 b + 3 hold block b.
template <typename TRaw>
__device__ __forceinline__ uint32_t mr_encode(const TRaw& v, uint32_t& scales) {
  uint32_t m = mr_amax(v);
  m = max(m, dpp<kDppXor1>(m));
  m = max(m, dpp<kDppXor2>(m));
  const int sb = block_scale_byte(m);
  uint32_t w = mr_codes(v, sb);
  if (sb == 0 || sb == 255) {                  // below the conversion's scales, or not finite
    w = 0;
    if (sb == 0 && m != 0) {
      const Raw8<float> f = mr_float8(v);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        int n, M;
        w |= e2m1_round<true>(f.w[i], sb - 126, 0, n, M) << (4 * i);
      }
    }
  }
  uint32_t s = (uint32_t)sb << (8 * ((threadIdx.x >> 2) & 3));
  s |= dpp<kDppRor4>(s);
  s |= dpp<kDppRor8>(s);
  scales = s;
  return w;
}

__device__ __forceinline__ bool mr_nan_scale(uint32_t s) {
  return (s & 0xFFu) == 0xFFu || (s & 0xFF00u) == 0xFF00u || (s & 0xFF0000u) == 0xFF0000u || (s >> 24) == 0xFFu;
}

// The source row of row r, or -1: none (past the end, or an index outside the source).
__device__ __forceinline__ int64_t mr_source(const MxRowsArgs& a, int64_t r) {
  if (r >= a.R) return -1;
  if (!a.index) return r;
  const int i = a.index[r];
  if (i < 0) return -1;
  const int s = (int)((uint32_t)i / (uint32_t)a.index_div);
  return s < a.a_rows ? s : -1;
}

template <typename TIn, bool UP>
__global__ __launch_bounds__(kMrThreads) void mx_rows_kernel(MxRowsArgs a, int ksteps) {
  const int sub = threadIdx.x & 15;
  const int kblocks = (ksteps + kMrSteps - 1) / kMrSteps;
  const int rb = blockIdx.x / kblocks;
  const int64_t r = (int64_t)rb * kMrRows + (threadIdx.x >> 4);
  const int64_t g = blockIdx.y;
  uint8_t* codes = a.codes + g * a.c_stride;
  uint8_t* scales = a.scales + g * a.s_stride;
  const int64_t src = mr_source(a, r);
  const TIn* A = (const TIn*)a.A + g * a.a_stride + (src < 0 ? 0 : src) * a.ld;
  const TIn* U = UP ? (const TIn*)a.up + g * a.a_stride + (src < 0 ? 0 : src) * a.ld : nullptr;
  const int k0 = (blockIdx.x - rb * kblocks) * kMrSteps;
  Raw8<TIn> v[kMrSteps], u[UP ? kMrSteps : 1];
#pragma unroll
  for (int q = 0; q < kMrSteps; ++q) {           // every load before the first conversion
    const int64_t c = (int64_t)(k0 + q) * 128 + sub * 8;
    const int64_t n = src >= 0 ? a.K - c : 0;
    v[q] = mr_load8<TIn>(A + c, n, a.vec != 0);
    if constexpr (UP) u[q] = mr_load8<TIn>(U + c, n, a.vec != 0);
  }
#pragma unroll
  for (int q = 0; q < kMrSteps; ++q) {
    const int kt = k0 + q;
    if (kt >= ksteps) break;
    uint32_t s, w;
    if constexpr (UP) {
      const Raw8<float> x = mr_float8(v[q]), y = mr_float8(u[q]);
      Raw8<float> h;
#pragma unroll
      for (int i = 0; i < 8; ++i) h.w[i] = mr_swiglu(x.w[i], y.w[i]);        // 0 * 0 past the end
      w = mr_encode(h, s);
    } else {
      w = mr_encode(v[q], s);
    }
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

// Many rows: BM x BN tiles, WM x WN waves of (32 MI) x (32 NI) each, operands staged through LDS by
// buffer-load DMA in a ring of NS steps of 128 elements.  A stage holds the tile's rows of both
// operands, 64 bytes a row with the four 16-byte chunks of a row at permuted places (chunk q of row r
// at q ^ ((r >> 2) & 3), so a quarter-wave's reads hit 16 bank groups), and the rows' scale words.
// v_mfma_scale_f32_32x32x64_f8f6f4: lane l holds row or column l % 32, K elements 32 (l / 32) .. + 31;
// result register r is row (r / 4) 8 + (l / 32) 4 + r % 4, column l % 32.
typedef float v16f __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) void lds_void;
constexpr int kRsrcWord3 = 0x00020000;   // raw buffer, 32-bit dword format

#define S3R_WAIT_VM(n) __builtin_amdgcn_s_waitcnt(((n) & 0xF) | (((n) >> 4) << 14) | 0x70 | 0xF00)
#define S3R_WAIT_LGKM0() __builtin_amdgcn_s_waitcnt(0xC07F)
constexpr int kSgMfma = 0x008, kSgDsRead = 0x100, kSgVmem = 0x010;

template <int MI_, int NI_, int WM_, int WN_, int NS_, int WavesPerSimd_>
struct Tile {
  static constexpr int WavesPerSimd = WavesPerSimd_;
  static constexpr int MI = MI_, NI = NI_, WM = WM_, WN = WN_, NS = NS_;
  static constexpr int Waves = WM * WN, Threads = 64 * Waves;
  static constexpr int BM = 32 * MI * WM, BN = 32 * NI * WN;
  static constexpr int PA = BM / 16 / Waves, PB = BN / 16 / Waves;        // 1 KiB pieces per wave
  static constexpr int SW = (BM + BN) / 64;                               // 64-word scale loads of a step
  static constexpr int PS = (SW + Waves - 1) / Waves;                     // per wave; surplus ones go to a spare place
  static constexpr int Loads = PA + PB + PS;
  static constexpr int OffB = BM * 64, OffS = OffB + BN * 64;
  static constexpr int StageBytes = OffS + Waves * PS * 256;
  static constexpr int EpiLd = 32 * NI + 4;                               // floats per row of the epilogue's staging
  static_assert(BM % (16 * Waves) == 0 && BN % (16 * Waves) == 0, "whole pieces per wave");
};

// One LDS object per stage: the compiler then sees that a stage's reads and the DMA into another touch
// different memory, and does not drain the loads in flight before the reads.
template <typename T, int S>
__device__ __forceinline__ uint8_t* ring() {
  __shared__ __attribute__((aligned(1024))) uint8_t stage[T::StageBytes];
  return stage;
}

__device__ __forceinline__ void dma16(__amdgpu_buffer_rsrc_t r, uint8_t* lds, uint32_t voff, uint32_t soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)lds, 16, voff, soff, 0, 0);
}
__device__ __forceinline__ void dma4(__amdgpu_buffer_rsrc_t r, uint8_t* lds, uint32_t voff, uint32_t soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)lds, 4, voff, soff, 0, 0);
}

__device__ __forceinline__ int chunk_pos(int r, int q) { return q ^ ((r >> 2) & 3); }

template <typename T>
struct TileSrc {
  __amdgpu_buffer_rsrc_t a, b, sa, sb, z;
  uint32_t va[T::PA], vb[T::PB], vs[T::PS];   // this lane's byte offsets in step 0
  uint32_t ldas, ldbs;
  int nk;
};

// Step kt into stage st; past the last step every load reads zeros, so the wait counts stay the same.
template <typename T>
__device__ __forceinline__ void tile_load(const TileSrc<T>& s, uint8_t* st, int kt) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const bool live = kt < s.nk;
  const __amdgpu_buffer_rsrc_t ra = live ? s.a : s.z, rb = live ? s.b : s.z;
  const uint32_t koff = (uint32_t)kt * (uint32_t)kMxBlkBytes;
#pragma unroll
  for (int q = 0; q < T::PA; ++q)
    dma16(ra, st + (wave * T::PA + q) * 1024, s.va[q], koff);
#pragma unroll
  for (int q = 0; q < T::PB; ++q)
    dma16(rb, st + T::OffB + (wave * T::PB + q) * 1024, s.vb[q], koff);
#pragma unroll
  for (int q = 0; q < T::PS; ++q) {
    const int w = q * T::Waves + wave;                       // 64-word run w: A's runs, then B's, then surplus
    const bool is_a = w < T::BM / 64 || w >= T::SW;
    const __amdgpu_buffer_rsrc_t rs = live ? (is_a ? s.sa : s.sb) : s.z;
    dma4(rs, st + T::OffS + w * 256, s.vs[q], (uint32_t)kt * (is_a ? s.ldas : s.ldbs));
  }
}

template <typename T>
struct TileFrag { v8i a[T::MI], b[T::NI]; };

template <typename T>
__device__ __forceinline__ void tile_frag(const uint8_t* st, int h, TileFrag<T>& f) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wm = wave / T::WN, wn = wave % T::WN;
  const int r31 = lane & 31, c = h * 2 + (lane >> 5);
#pragma unroll
  for (int i = 0; i < T::MI; ++i) {
    const int r = (wm * T::MI + i) * 32 + r31;
    const uint4 x = *reinterpret_cast<const uint4*>(st + r * 64 + (chunk_pos(r, c) << 4));
    f.a[i] = v8i{(int)x.x, (int)x.y, (int)x.z, (int)x.w, 0, 0, 0, 0};
  }
#pragma unroll
  for (int j = 0; j < T::NI; ++j) {
    const int r = (wn * T::NI + j) * 32 + r31;
    const uint4 x = *reinterpret_cast<const uint4*>(st + T::OffB + r * 64 + (chunk_pos(r, c) << 4));
    f.b[j] = v8i{(int)x.x, (int)x.y, (int)x.z, (int)x.w, 0, 0, 0, 0};
  }
}

// The scale words of this lane's rows and columns, shifted so that bytes 0 and 2 are its blocks in the
// two half-steps (the instruction picks the byte).
template <typename T>
__device__ __forceinline__ void tile_scales(const uint8_t* st, uint32_t (&sa)[T::MI], uint32_t (&sb)[T::NI]) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wm = wave / T::WN, wn = wave % T::WN;
  const int r31 = lane & 31, sh = (lane >> 5) * 8;
#pragma unroll
  for (int i = 0; i < T::MI; ++i)
    sa[i] = *reinterpret_cast<const uint32_t*>(st + T::OffS + ((wm * T::MI + i) * 32 + r31) * 4) >> sh;
#pragma unroll
  for (int j = 0; j < T::NI; ++j)
    sb[j] = *reinterpret_cast<const uint32_t*>(st + T::OffS + T::BM * 4 + ((wn * T::NI + j) * 32 + r31) * 4) >> sh;
}

template <typename T, int H>
__device__ __forceinline__ void tile_mfma(const TileFrag<T>& f, const uint32_t (&sa)[T::MI], const uint32_t (&sb)[T::NI],
                                          v16f (&acc)[T::MI][T::NI]) {
#pragma unroll
  for (int i = 0; i < T::MI; ++i)
#pragma unroll
    for (int j = 0; j < T::NI; ++j)
      acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(f.a[i], f.b[j], acc[i][j], 4, 4, 2 * H, (int)sa[i],
                                                                  2 * H, (int)sb[j]);
}

// What a wave holds at the start of a step: the fragments of its first half and its scales.
template <typename T>
struct TileHead {
  TileFrag<T> f0;
  uint32_t sa[T::MI], sb[T::NI];
};

template <typename T>
__device__ __forceinline__ void tile_head(const uint8_t* st, TileHead<T>& h) {
  tile_frag<T>(st, 0, h.f0);
  tile_scales<T>(st, h.sa, h.sb);
}

// Step kt on stage S = kt % NS.  The first half's products cover the reads of the second half's
// fragments; the barrier in the middle then makes step kt + 1 visible and retires stage S, which takes
// step kt + NS; the second half's products cover the reads of step kt + 1's head.  So the matrix cores
// wait for no LDS read, and a load has NS - 1 steps and a half to arrive.
template <typename T, int S>
__device__ __forceinline__ void tile_step(const TileSrc<T>& src, int kt, TileHead<T>& h, v16f (&acc)[T::MI][T::NI]) {
  TileFrag<T> f1;
  tile_frag<T>(ring<T, S>(), 1, f1);
  tile_mfma<T, 0>(h.f0, h.sa, h.sb, acc);
  __builtin_amdgcn_sched_group_barrier(kSgDsRead, T::MI + T::NI, 0);
  __builtin_amdgcn_sched_group_barrier(kSgMfma, T::MI * T::NI, 0);
  __builtin_amdgcn_sched_barrier(0);
  S3R_WAIT_VM(T::Loads * (T::NS - 2));
  S3R_WAIT_LGKM0();
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_sched_barrier(0);
  TileHead<T> n;
  tile_load<T>(src, ring<T, S>(), kt + T::NS);
  tile_head<T>(ring<T, (S + 1) % T::NS>(), n);
  tile_mfma<T, 1>(f1, h.sa, h.sb, acc);
#pragma unroll
  for (int x = 0; x < T::MI * T::NI; ++x) {
    __builtin_amdgcn_sched_group_barrier(kSgMfma, 1, 0);
    __builtin_amdgcn_sched_group_barrier(kSgDsRead, (2 * (T::MI + T::NI) + T::MI * T::NI - 1) / (T::MI * T::NI), 0);
    __builtin_amdgcn_sched_group_barrier(kSgVmem, (T::Loads + T::MI * T::NI - 1) / (T::MI * T::NI), 0);
  }
  __builtin_amdgcn_sched_barrier(0);
  h = n;
}

template <typename T, int S>
__device__ __forceinline__ void tile_steps(const TileSrc<T>& src, int kt, TileHead<T>& h, v16f (&acc)[T::MI][T::NI]) {
  if constexpr (S < T::NS) {
    if (kt + S < src.nk) {
      tile_step<T, S>(src, kt + S, h, acc);
      tile_steps<T, S + 1>(src, kt, h, acc);
    }
  }
}

// The wave's results, 32 rows at a time through its own part of the (now free) ring, so that whole
// 16-byte words of consecutive columns are stored.
template <typename T, typename TOut>
__device__ __forceinline__ void tile_store(const MxProdK& p, int64_t m0, int64_t m1, int64_t n0, bool vec,
                                           const v16f (&acc)[T::MI][T::NI]) {
  constexpr int kBuf = 32 * T::EpiLd * 4;
  constexpr int kPer = T::StageBytes / kBuf;                  // waves' buffers in one stage
  static_assert(kPer > 0 && kPer * T::NS >= T::Waves, "the epilogue's staging fits the ring");
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wm = wave / T::WN, wn = wave % T::WN;
  uint8_t* stage = ring<T, 0>();
  if (wave / kPer == 1) stage = ring<T, 1 % T::NS>();
  if (wave / kPer == 2) stage = ring<T, 2 % T::NS>();
  if (T::NS > 3 && wave / kPer == 3) stage = ring<T, 3 % T::NS>();
  float* buf = reinterpret_cast<float*>(stage + (wave % kPer) * kBuf);
  constexpr int W = 16 / (int)sizeof(TOut);                   // elements of a store
  constexpr int LR = 32 * T::NI / W;                          // lanes of a row
  const int lr = lane / LR, lc = (lane % LR) * W;
  const int64_t n = n0 + wn * (32 * T::NI) + lc;
  TOut* out = (TOut*)p.out;
#pragma unroll
  for (int i = 0; i < T::MI; ++i) {
#pragma unroll
    for (int j = 0; j < T::NI; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r)
        buf[((r >> 2) * 8 + (lane >> 5) * 4 + (r & 3)) * T::EpiLd + j * 32 + (lane & 31)] = acc[i][j][r];
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    for (int q = 0; q < 32; q += 64 / LR) {
      const int64_t m = m0 + (wm * T::MI + i) * 32 + q + lr;
      float v[W];
#pragma unroll
      for (int x = 0; x < W; x += 4) {
        const float4 t = *reinterpret_cast<const float4*>(buf + (q + lr) * T::EpiLd + lc + x);
        v[x] = t.x; v[x + 1] = t.y; v[x + 2] = t.z; v[x + 3] = t.w;
      }
      if (m >= m1) continue;
      TOut* o = out + m * p.ld_out + n;
      if (vec && n + W <= p.N) {
        if constexpr (sizeof(TOut) == 2) {
          typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
          typedef float f2 __attribute__((ext_vector_type(2)));
          uint32_t w[4];
#pragma unroll
          for (int x = 0; x < 4; ++x)
            w[x] = __builtin_bit_cast(uint32_t, __builtin_convertvector((f2{v[2 * x], v[2 * x + 1]}), bf2));
          __builtin_nontemporal_store((v4u32{w[0], w[1], w[2], w[3]}), reinterpret_cast<v4u32*>(o));
        } else {
          __builtin_nontemporal_store((v4f32{v[0], v[1], v[2], v[3]}), reinterpret_cast<v4f32*>(o));
        }
      } else {
#pragma unroll
        for (int x = 0; x < W; ++x)
          if (n + x < p.N) store_out(o + x, v[x]);
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
}

template <typename T, typename TOut>
__global__ __launch_bounds__(T::Threads, T::WavesPerSimd) void mx_tile_kernel(MxProdK p, int tiles_m, int vec) {
  int bid = blockIdx.x;
  const int nblocks = tiles_m * p.tiles_n;
  if (nblocks % 8 == 0) bid = (bid % 8) * (nblocks / 8) + bid / 8;   // a contiguous range of tiles per XCD
  const int group = 8 * p.tiles_n;
  const int first_m = (bid / group) * 8;
  const int gsz = min(tiles_m - first_m, 8);
  const int tm = first_m + (bid % group) % gsz, tn = (bid % group) / gsz;
  int64_t m0 = (int64_t)tm * T::BM, m1 = p.M;
  const int64_t n0 = (int64_t)tn * T::BN;
  const uint8_t *B = p.B, *Bs = p.Bs;
  if (p.G) {
    const GroupTile h = find_group_tile(p.offsets, p.G, p.M, tm, T::BM);
    if (h.bad) {
      if (blockIdx.x == 0 && threadIdx.x == 0 && p.flags) atomicOr(p.flags, S3R_FLAG_BAD_GROUPS);
      return;
    }
    const int e = __builtin_amdgcn_readfirstlane(h.e);
    if (e < 0) return;
    m0 = h.r0;
    m1 = h.r1;
    B += e * p.b_stride;
    Bs += e * p.bs_stride;
  }
  TileSrc<T> src;
  src.nk = p.ksteps;
  src.ldas = (uint32_t)p.ldas;
  src.ldbs = (uint32_t)p.ldbs;
  // whole operands, every 256-row block of codes: rows past the end inside the last block reach only
  // outputs that are not stored, and their scale words are the last row's
  src.a = __builtin_amdgcn_make_buffer_rsrc((void*)p.A, (short)0, (int)(uint32_t)(((p.M + 255) >> 8) * p.lda), kRsrcWord3);
  src.b = __builtin_amdgcn_make_buffer_rsrc((void*)B, (short)0, (int)(uint32_t)(((p.N + 255) >> 8) * p.ldb), kRsrcWord3);
  src.sa = __builtin_amdgcn_make_buffer_rsrc((void*)p.As, (short)0, (int)(uint32_t)(((int64_t)p.ksteps - 1) * p.ldas + 4 * p.M), kRsrcWord3);
  src.sb = __builtin_amdgcn_make_buffer_rsrc((void*)Bs, (short)0, (int)(uint32_t)(((int64_t)p.ksteps - 1) * p.ldbs + 4 * p.N), kRsrcWord3);
  src.z = __builtin_amdgcn_make_buffer_rsrc((void*)p.A, (short)0, 0, kRsrcWord3);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
#pragma unroll
  for (int q = 0; q < T::PA; ++q) {
    const int r = (wave * T::PA + q) * 16 + (lane >> 2);
    const int64_t m = m0 + r;
    src.va[q] = (uint32_t)((m >> 8) * p.lda + (m & 255) * 64 + chunk_pos(r, lane & 3) * 16);
  }
#pragma unroll
  for (int q = 0; q < T::PB; ++q) {
    const int r = (wave * T::PB + q) * 16 + (lane >> 2);
    const int64_t n = n0 + r;
    src.vb[q] = (uint32_t)((n >> 8) * p.ldb + (n & 255) * 64 + chunk_pos(r, lane & 3) * 16);
  }
#pragma unroll
  for (int q = 0; q < T::PS; ++q) {
    const int w = q * T::Waves + wave;
    src.vs[q] = w < T::BM / 64 ? (uint32_t)(min(m0 + w * 64 + lane, p.M - 1) * 4)
                : w < T::SW    ? (uint32_t)(min(n0 + (w - T::BM / 64) * 64 + lane, p.N - 1) * 4)
                               : 0u;
  }
  v16f acc[T::MI][T::NI];
#pragma unroll
  for (int i = 0; i < T::MI; ++i)
#pragma unroll
    for (int j = 0; j < T::NI; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
  tile_load<T>(src, ring<T, 0>(), 0);
  tile_load<T>(src, ring<T, 1>(), 1);
  tile_load<T>(src, ring<T, 2>(), 2);
  if constexpr (T::NS > 3) tile_load<T>(src, ring<T, 3>(), 3);
  S3R_WAIT_VM(T::Loads * (T::NS - 1));
  __builtin_amdgcn_s_barrier();
  TileHead<T> head;
  tile_head<T>(ring<T, 0>(), head);
  for (int kt = 0; kt < p.ksteps; kt += T::NS) tile_steps<T, 0>(src, kt, head, acc);
  S3R_WAIT_VM(0);
  S3R_WAIT_LGKM0();
  __builtin_amdgcn_s_barrier();
  tile_store<T, TOut>(p, m0, m1, n0, vec != 0, acc);
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
  const int64_t kblocks = (ksteps + kMrSteps - 1) / kMrSteps, blocks = kblocks * ((a.R + kMrRows - 1) / kMrRows);
  if (blocks > 0x7FFFFFFF) return hipErrorInvalidConfiguration;
  const dim3 grid((unsigned)blocks, (unsigned)a.G);
  const dim3 block(kMrThreads);
  if (a.dtype == S3R_BF16) {
    if (a.up) hipLaunchKernelGGL((mx_rows_kernel<uint16_t, true>), grid, block, 0, st, b, ksteps);
    else hipLaunchKernelGGL((mx_rows_kernel<uint16_t, false>), grid, block, 0, st, b, ksteps);
  } else {
    if (a.up) hipLaunchKernelGGL((mx_rows_kernel<float, true>), grid, block, 0, st, b, ksteps);
    else hipLaunchKernelGGL((mx_rows_kernel<float, false>), grid, block, 0, st, b, ksteps);
  }
  return hipGetLastError();
}

namespace {
#ifndef BIGTILE
#define BIGTILE 4, 2, 2, 4, 3, 2
#endif
#ifndef MIDTILE
#define MIDTILE 2, 2, 4, 2, 3, 4
#endif
#ifndef FEW
#define FEW 32
#endif
using BigTile = Tile<BIGTILE>;
using MidTile = Tile<MIDTILE>;

template <typename T, typename TOut>
hipError_t run_tiles(const MxProductArgs& a, MxProdK p, hipStream_t st) {
  const int64_t mt = a.G ? a.M / T::BM + std::min(a.G, a.M) : (a.M + T::BM - 1) / T::BM;
  p.tiles_n = (int)((a.N + T::BN - 1) / T::BN);
  if (mt * p.tiles_n > 0x7FFFFFFF) return hipErrorInvalidConfiguration;
  const int vec = ((uintptr_t)a.out & 15u) == 0 && (a.ld_out * (int64_t)sizeof(TOut)) % 16 == 0;
  hipLaunchKernelGGL((mx_tile_kernel<T, TOut>), dim3((unsigned)(mt * p.tiles_n)), dim3(T::Threads), 0, st, p, (int)mt, vec);
  return hipGetLastError();
}
}  // namespace

hipError_t launch_mx_product(const MxProductArgs& a, hipStream_t st) {
  if (a.M == 0 || a.N == 0) return hipSuccess;
  MxProdK p{};
  p.A = a.A; p.lda = a.lda; p.As = a.As; p.ldas = a.ldas;
  p.B = a.B; p.ldb = a.ldb; p.Bs = a.Bs; p.ldbs = a.ldbs; p.b_stride = a.b_stride; p.bs_stride = a.bs_stride;
  p.offsets = a.offsets; p.G = a.G; p.M = a.M; p.N = a.N; p.ksteps = (int)((a.K + 127) / 128);
  p.out = a.out; p.ld_out = a.ld_out; p.flags = a.flags;
  const bool bf16 = a.out_dt == S3R_BF16;
  // rows per weight, on average (only the device knows the groups' own)
  const int64_t rows = a.G ? (a.M + a.G - 1) / a.G : a.M;
  if (rows <= FEW) {
    // grouped: the tiles of every group, at most one partial tile each
    const int64_t mt = a.G ? a.M / 16 + std::min(a.G, a.M) : (a.M + 15) / 16;
    p.tiles_n = (int)((a.N + 31) / 32);
    if (mt * p.tiles_n > 0x7FFFFFFF) return hipErrorInvalidConfiguration;
    const dim3 grid((unsigned)(mt * p.tiles_n));
    if (bf16) hipLaunchKernelGGL((mx_few_rows_kernel<uint16_t, 2>), grid, dim3(kSkThreads), 0, st, p);
    else hipLaunchKernelGGL((mx_few_rows_kernel<float, 2>), grid, dim3(kSkThreads), 0, st, p);
  } else {
    const int64_t big = ((a.M + BigTile::BM - 1) / BigTile::BM) * ((a.N + BigTile::BN - 1) / BigTile::BN);
    if (!a.G && big >= 256) return bf16 ? run_tiles<BigTile, uint16_t>(a, p, st) : run_tiles<BigTile, float>(a, p, st);
    return bf16 ? run_tiles<MidTile, uint16_t>(a, p, st) : run_tiles<MidTile, float>(a, p, st);
  }
  return hipGetLastError();
}

}  // namespace s3r
