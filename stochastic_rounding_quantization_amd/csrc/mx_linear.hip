// Forward products on MXFP4 operands: rows of any number and any length rounded
// to E2M1 with one E8M0 scale per 32 elements (RTNE, the format and block layout
// of the MXFP4 backward), and y = dq(A) dq(B)^T, dense or over expert-sorted
// rows with one B per group, on the block-scaled FP4 matrix cores.
//
// The contraction K is padded to whole steps of 128 elements with zero codes, so
// K, like the rows and the columns, can have any size.
//
// What bounds them (MI355X; a large copy moves 5.4 TB/s, the FP4 cores have 10.1 PFLOP/s):
//   rows       HBM: 8192 x 4096 fp32 28 us, 5.5 TB/s, bf16 14.5 - 16; 32768 rows of 2048 gathered 26 us
//   few rows   the weights' bytes: 1 x 14336 x 4096 8.3 us, 3.8 TB/s with the launch
//   tiles      power: 8192 x 14336 x 4096 250 - 270 us, 3.6 - 3.85 PFLOP/s (zero operands: 185 - 205 us; a tile's
//              epilogue, 235 MB of results in all, is a fifth of it); 64 experts, 32768 x 1408 x 2048 82 - 97 us, of
//              which the weights', rows' and results' 225 MB need 42
// Rounding the tokens once and gathering their codes in the product's loads instead of gathering in the rounding
// made the experts' product 126 us (64-byte pieces of 128-byte lines), so the rows are gathered first.
#include <type_traits>

#include "group_tiles.h"
#include "mx_math.h"
#include "rows8.h"
#include "tile_ring.h"

namespace s3r {
namespace {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));

// ------------------------------------------------------------------ rows ----
// A block of 256 threads takes 16 rows x Steps 128-element steps: 16 lanes per
// row, 8 elements a lane and step (16 bytes of bf16), so a block of 32 elements
// is four lanes.  Codes leave as 1 KiB and scales as 64 bytes in one run.  With
// `up` the element is silu(A) * up in fp32, not rounded in between.
// The arithmetic is what bounded the first version (28 instructions an element:
// 35 us for 8192 x 4096 bf16, whose bytes need 15); now two elements convert in
// one instruction, and the maximum of bf16 runs on packed magnitudes.
constexpr int kMrThreads = 256, kMrRows = 16;

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

// Codes of 8 elements of a block with the scale byte sb, any of them: 0 is below the conversion's scales
// (2^-127 is no normal fp32 number), so there elements and scale are taken times 2^64, which is exact.
template <typename TRaw>
__device__ __forceinline__ uint32_t mr_word(const TRaw& v, int sb) {
  uint32_t w = mr_codes(v, sb);
  if (sb == 0) {
    Raw8<float> f = mr_float8(v);
#pragma unroll
    for (int i = 0; i < 8; ++i) f.w[i] *= 0x1p64f;
    w = mr_codes(f, 64);
  }
  return sb == 255 ? 0u : w;                   // a block with a non-finite element
}

// The codes of this lane's 8 elements (one word) and, in every lane of the row's 16, its step's four
// scale bytes; lanes 4 b .. 4 b + 3 hold block b.
template <typename TRaw>
__device__ __forceinline__ uint32_t mr_encode(const TRaw& v, uint32_t& scales) {
  uint32_t m = mr_amax(v);
  m = max(m, dpp<kDppXor1>(m));
  m = max(m, dpp<kDppXor2>(m));
  const int sb = block_scale_byte(m);
  const uint32_t w = mr_word(v, sb);
  uint32_t s = (uint32_t)sb << (8 * ((threadIdx.x >> 2) & 3));
  s |= dpp<kDppRor4>(s);
  s |= dpp<kDppRor8>(s);
  scales = s;
  return w;
}

__device__ __forceinline__ bool mr_nan_scale(uint32_t s) {
  return (s & 0xFFu) == 0xFFu || (s & 0xFF00u) == 0xFF00u || (s & 0xFF0000u) == 0xFF0000u || (s >> 24) == 0xFFu;
}

template <typename TIn, bool UP, bool Words, int Steps>
__global__ __launch_bounds__(kMrThreads) void mx_rows_kernel(MxRowsArgs a, int ksteps) {
  const int sub = threadIdx.x & 15;
  const int kblocks = (ksteps + Steps - 1) / Steps;
  const int rb = blockIdx.x / kblocks;
  const int64_t r = (int64_t)rb * kMrRows + (threadIdx.x >> 4);
  const int64_t g = blockIdx.y;
  uint8_t* codes = a.codes + g * a.c_stride;
  uint8_t* scales = a.scales + g * a.s_stride;
  const int64_t src = mr_source(a, r);
  const TIn* A = (const TIn*)a.A + g * a.a_stride + (src < 0 ? 0 : src) * a.ld;
  const TIn* U = UP ? (const TIn*)a.up + g * a.a_stride + (src < 0 ? 0 : src) * a.ld : nullptr;
  const int k0 = (blockIdx.x - rb * kblocks) * Steps;
  Raw8<TIn> v[Steps], u[UP ? Steps : 1];
#pragma unroll
  for (int q = 0; q < Steps; ++q) {           // every load before the first conversion
    const int64_t c = (int64_t)(k0 + q) * 128 + sub * 8;
    const int64_t n = src >= 0 ? a.K - c : 0;
    v[q] = mr_load8<TIn, Words>(A + c, n, a.K);
    if constexpr (UP) u[q] = mr_load8<TIn, Words>(U + c, n, a.K);
  }
#pragma unroll
  for (int q = 0; q < Steps; ++q) {
    const int kt = k0 + q;
    if (kt >= ksteps) break;
    const int64_t n = src >= 0 ? a.K - (int64_t)kt * 128 - sub * 8 : 0;
    mr_tail<Words>(v[q], n, a.K);
    if constexpr (UP) mr_tail<Words>(u[q], n, a.K);
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
// The offsets of a product without results.
__global__ __launch_bounds__(64) void mx_offsets_kernel(const int64_t* offsets, int64_t G, int64_t R, uint32_t* flags) {
  GroupRound first;
  bool bad;
  group_total(offsets, G, R, 1, first, bad);
  if (bad && threadIdx.x == 0) atomicOr(flags, S3R_FLAG_BAD_GROUPS);
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
// rows of a step are one contiguous KiB of the code layout.  The weights' bytes are the bound, so a wave
// issues the loads of `Depth` steps before its first product.
// With TIn the rows come unquantized (s3r_mx_linear): the workgroup rounds its rows into LDS, as
// mx_rows_kernel does into memory, while its first weights are on the way, so there is no second launch
// and no codes go through memory (every column tile rounds the rows again, from the caches).  Rounding in
// each lane's own fragment instead did the work of 16 rows for one row: 12 us against 9 (N = 14336, K = 4096).
// TIn void: rows already in codes.
constexpr int kSkThreads = 256;
constexpr size_t kSkLdsMax = 65536;               // a workgroup's dynamic LDS
// LDS of the rounded rows: a row's codes (64 bytes a step, 16 to spread the rows over the banks), then
// every row's scale words
__host__ __device__ inline size_t sk_row_bytes(int ksteps) { return (size_t)ksteps * 64 + 16; }
__host__ __device__ inline size_t sk_lds_bytes(int rows, int ksteps) { return rows * (sk_row_bytes(ksteps) + (size_t)ksteps * 4); }

template <typename TOut, typename TIn, bool Words, int MI, int NJ, int Depth>
__global__ __launch_bounds__(kSkThreads) void mx_few_rows_kernel(MxProdK p, MxRowsArgs q, int tile_rows) {
  constexpr bool kFused = !std::is_void<TIn>::value;
  static_assert(!kFused || MI == 1, "rounded rows of one 16-row tile");
  __shared__ float part[3][MI * NJ][256];
  extern __shared__ __attribute__((aligned(16))) uint8_t sk_rows[];
  // The wave's index in a scalar register: the loop over its steps has to branch, since the matrix
  // instructions run whatever the execution mask says.
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int64_t m0, m1;
  const uint8_t *B = p.B, *Bs = p.Bs;
  const int mt = blockIdx.x / p.tiles_n, nt = blockIdx.x - mt * p.tiles_n;
  if (p.G) {
    GroupRound first;
    bool bad;
    const int total = group_total(p.offsets, p.G, p.M, 16 * MI, first, bad);
    if (bad) {
      if (blockIdx.x == 0 && threadIdx.x == 0 && p.flags) atomicOr(p.flags, S3R_FLAG_BAD_GROUPS);
      return;
    }
    if (mt >= total) return;
    const GroupTile h = group_tile(p.offsets, p.G, p.M, 16 * MI, first, mt);
    const int e = __builtin_amdgcn_readfirstlane(h.e);
    m0 = h.r0;
    m1 = min(h.r1, m0 + 16 * MI);
    B += e * p.b_stride;
    Bs += e * p.bs_stride;
  } else {
    m0 = (int64_t)mt * (16 * MI);
    m1 = min(p.M, m0 + 16 * MI);
  }
  const int64_t n0 = (int64_t)nt * (16 * NJ);
  const int r15 = lane & 15, kb = lane >> 4;
  // rows and columns past the end repeat the last one; their results are not stored
  const int rows = (int)(m1 - m0), lr = min(r15, rows - 1);
  const uint8_t *pa[MI], *psa[MI];
  if constexpr (!kFused) {
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      const int64_t ar = m0 + min(16 * i + r15, rows - 1);
      pa[i] = p.A + (ar >> 8) * p.lda + (ar & 255) * 64 + kb * 16;
      psa[i] = p.As + 4 * ar + kb;
    }
  }
  const uint8_t *pb[NJ], *psb[NJ];
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    const int64_t br = min(n0 + 16 * j + r15, p.N - 1);
    pb[j] = B + (br >> 8) * p.ldb + (br & 255) * 64 + kb * 16;
    psb[j] = Bs + 4 * br + kb;
  }
  v4f acc[MI][NJ];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
  uint4 x[Depth][MI], y[Depth][NJ];
  int sa[Depth][MI], sb[Depth][NJ];
  auto load = [&](int kt) {
#pragma unroll
    for (int d = 0; d < Depth; ++d) {
      const int64_t k = kt + 4 * d;
      if (k < p.ksteps) {                          // the same in the whole wave
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          y[d][j] = *reinterpret_cast<const uint4*>(pb[j] + k * kMxBlkBytes);
          sb[d][j] = psb[j][k * p.ldbs];
        }
        if constexpr (!kFused) {
#pragma unroll
          for (int i = 0; i < MI; ++i) {
            x[d][i] = *reinterpret_cast<const uint4*>(pa[i] + k * kMxBlkBytes);
            sa[d][i] = psa[i][k * p.ldas];
          }
        }
      }
    }
  };
  load(wave);
  const int row_bytes = (int)sk_row_bytes(p.ksteps);
  uint8_t* sk_scales = sk_rows + tile_rows * row_bytes;
  if constexpr (kFused) {
    bool bad = false;
    const int sub = threadIdx.x & 15, items = rows * p.ksteps;      // (row, step) pairs, 16 lanes each
    constexpr int kBatch = 2, kApart = kSkThreads / 16;              // pairs of a thread whose loads go out together
    for (int it0 = threadIdx.x >> 4; it0 < items; it0 += kBatch * kApart) {
      Raw8<TIn> v[kBatch];
      int r[kBatch], kt[kBatch], left[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int it = it0 + u * kApart;
        r[u] = it / p.ksteps;
        kt[u] = it - r[u] * p.ksteps;
        const int64_t src = it < items ? mr_source(q, m0 + r[u]) : -1;
        const int c = kt[u] * 128 + sub * 8;
        v[u] = mr_load8<TIn, Words>((const TIn*)q.A + (src < 0 ? 0 : src) * q.ld + c, src < 0 ? 0 : q.K - c, q.K);
        left[u] = src < 0 ? 0 : (int)min(q.K - c, (int64_t)8);
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        uint32_t s;
        mr_tail<Words>(v[u], left[u], q.K);
        const uint32_t w = mr_encode(v[u], s);
        if (it0 + u * kApart < items) {
          *reinterpret_cast<uint32_t*>(sk_rows + r[u] * row_bytes + kt[u] * 64 + sub * 4) = w;
          if (sub == 0) *reinterpret_cast<uint32_t*>(sk_scales + (r[u] * p.ksteps + kt[u]) * 4) = s;
          bad |= mr_nan_scale(s);
        }
      }
    }
    if (bad && nt == 0 && p.flags) atomicOr(p.flags, S3R_FLAG_NONFINITE);
    __syncthreads();
  }
  for (int kt = wave; kt < p.ksteps; kt += 4 * Depth) {
    if (kt != wave) load(kt);
#pragma unroll
    for (int d = 0; d < Depth; ++d) {
      const int k = kt + 4 * d;
      if (k >= p.ksteps) break;
      if constexpr (kFused) {
        x[d][0] = *reinterpret_cast<const uint4*>(sk_rows + lr * row_bytes + k * 64 + kb * 16);
        sa[d][0] = sk_scales[(lr * p.ksteps + k) * 4 + kb];
      }
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        const v8i fa = v8i{(int)x[d][i].x, (int)x[d][i].y, (int)x[d][i].z, (int)x[d][i].w, 0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          const v8i fb = v8i{(int)y[d][j].x, (int)y[d][j].y, (int)y[d][j].z, (int)y[d][j].w, 0, 0, 0, 0};
          acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fa, fb, acc[i][j], 4, 4, 0, sa[d][i], 0, sb[d][j]);
        }
      }
    }
  }
  if (wave > 0) {
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r) part[wave - 1][i * NJ + j][r * 64 + lane] = acc[i][j][r];
  }
  __syncthreads();
  if (wave > 0) return;
  TOut* out = (TOut*)p.out;
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const int64_t n = n0 + 16 * j + r15;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int64_t m = m0 + 16 * i + 4 * kb + r;
        const int at = r * 64 + lane, ij = i * NJ + j;
        const float v = ((acc[i][j][r] + part[0][ij][at]) + part[1][ij][at]) + part[2][ij][at];
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

__device__ __forceinline__ void dma4(__amdgpu_buffer_rsrc_t r, uint8_t* lds, uint32_t voff, uint32_t soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)lds, 4, voff, soff, 0, 0);
}

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
// wait for no LDS read, and a load has NS - 1 steps and a half to arrive.  (A barrier at the step's start, before
// its reads: 4.5 % more for 8192 x 14336 x 4096.)
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

// The first NS steps into the ring.
template <typename T, int S>
__device__ __forceinline__ void tile_fill(const TileSrc<T>& src) {
  if constexpr (S < T::NS) {
    tile_load<T>(src, ring<T, S>(), S);
    tile_fill<T, S + 1>(src);
  }
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
// 16-byte words of consecutive columns are stored, past the last-level cache (fp32 results of
// 8192 x 14336 x 4096: 264 - 272 us, with plain stores 297).  At the elements' alignment, for any width and slice: 8192 x
// 14335 x 4096 in bf16 276 - 281 us, element by element 393 (14336 columns: 250 - 270).
template <typename T, typename TOut>
__device__ __forceinline__ void tile_store(const MxProdK& p, int64_t m0, int64_t m1, int64_t n0,
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
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
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
      if (n + W <= p.N) {
        if constexpr (sizeof(TOut) == 2) {
          typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
          typedef float f2 __attribute__((ext_vector_type(2)));
          uint32_t w[4];
#pragma unroll
          for (int x = 0; x < 4; ++x)
            w[x] = __builtin_bit_cast(uint32_t, __builtin_convertvector((f2{v[2 * x], v[2 * x + 1]}), bf2));
          __builtin_nontemporal_store((v4u32{w[0], w[1], w[2], w[3]}), reinterpret_cast<mr_u4_a2*>(o));
        } else {
          __builtin_nontemporal_store((v4u32{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])}),
                                      reinterpret_cast<mr_u4_a4*>(o));
        }
      } else {
#pragma unroll
        for (int x = 0; x < W; ++x)
          if (n + x < p.N) store_out(o + x, v[x]);
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
}

template <typename T, typename TOut>
__global__ __launch_bounds__(T::Threads, T::WavesPerSimd) void mx_tile_kernel(MxProdK p, int tiles_m) {
  // A contiguous range of tiles per XCD (workgroups go to the 8 XCDs in turn).  Grouped: of the tiles that the
  // groups have, not of the grid's bound on them, whose surplus would all be the last XCD's.
  int bid = blockIdx.x;
  GroupRound first;
  if (p.G) {
    bool bad;
    tiles_m = group_total(p.offsets, p.G, p.M, T::BM, first, bad);
    if (bad) {
      if (blockIdx.x == 0 && threadIdx.x == 0 && p.flags) atomicOr(p.flags, S3R_FLAG_BAD_GROUPS);
      return;
    }
    const int nblocks = tiles_m * p.tiles_n, per = (nblocks + 7) / 8;
    bid = (blockIdx.x % 8) * per + blockIdx.x / 8;
    if ((int)blockIdx.x / 8 >= per || bid >= nblocks) return;
  } else {
    const int nblocks = tiles_m * p.tiles_n;
    if (nblocks % 8 == 0) bid = (bid % 8) * (nblocks / 8) + bid / 8;
  }
  const int group = 8 * p.tiles_n;
  const int first_m = (bid / group) * 8;
  const int gsz = min(tiles_m - first_m, 8);
  const int tm = first_m + (bid % group) % gsz, tn = (bid % group) / gsz;
  int64_t m0 = (int64_t)tm * T::BM, m1 = p.M;
  const int64_t n0 = (int64_t)tn * T::BN;
  const uint8_t *B = p.B, *Bs = p.Bs;
  if (p.G) {
    const GroupTile h = group_tile(p.offsets, p.G, p.M, T::BM, first, tm);
    m0 = h.r0;
    m1 = h.r1;
    B += h.e * p.b_stride;
    Bs += h.e * p.bs_stride;
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
  tile_fill<T, 0>(src);
  S3R_WAIT_VM(T::Loads * (T::NS - 1));
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_sched_barrier(0);
  TileHead<T> head;
  tile_head<T>(ring<T, 0>(), head);
  for (int kt = 0; kt < p.ksteps; kt += T::NS) tile_steps<T, 0>(src, kt, head, acc);
  S3R_WAIT_VM(0);
  S3R_WAIT_LGKM0();
  __builtin_amdgcn_s_barrier();
  tile_store<T, TOut>(p, m0, m1, n0, acc);
}

}  // namespace

size_t mx_rows_codes_bytes(int64_t R, int64_t K) { return (size_t)((R + 255) / 256) * (size_t)((K + 127) / 128) * kMxBlkBytes; }
size_t mx_rows_scales_bytes(int64_t R, int64_t K) { return (size_t)((K + 127) / 128) * (size_t)R * 4; }

namespace {
bool mr_words(const MxRowsArgs& a) {       // rows in whole 16-byte words
  const int esize = a.dtype == S3R_BF16 ? 2 : 4;
  return ((uintptr_t)a.A & 15u) == 0 && ((uintptr_t)a.up & 15u) == 0 && (a.ld * esize) % 16 == 0 &&
         (a.a_stride * esize) % 16 == 0 && a.K % 8 == 0;
}

template <typename TIn, int Steps>
hipError_t run_rows(const MxRowsArgs& a, hipStream_t st) {
  const int ksteps = (int)((a.K + 127) / 128);
  const int64_t blocks = (ksteps + Steps - 1) / Steps * ((a.R + kMrRows - 1) / kMrRows);
  if (blocks * kMrThreads >= (int64_t)1 << 32) return hipErrorInvalidConfiguration;
  const dim3 grid((unsigned)blocks, (unsigned)a.G), block(kMrThreads);
  const bool words = mr_words(a);
  if (a.up && words) hipLaunchKernelGGL((mx_rows_kernel<TIn, true, true, Steps>), grid, block, 0, st, a, ksteps);
  else if (a.up) hipLaunchKernelGGL((mx_rows_kernel<TIn, true, false, Steps>), grid, block, 0, st, a, ksteps);
  else if (words) hipLaunchKernelGGL((mx_rows_kernel<TIn, false, true, Steps>), grid, block, 0, st, a, ksteps);
  else hipLaunchKernelGGL((mx_rows_kernel<TIn, false, false, Steps>), grid, block, 0, st, a, ksteps);
  return hipGetLastError();
}

// Steps of a workgroup: 4 keep more bytes in flight, 1 fills the GPU and has less code to fetch where there
// are few rows.  us with 1 and 4: 333 x 2024 fp32 2.6 and 3.4, 2000 x 2048 bf16 3.6 and 4.5, 2000 x 4096 bf16 5.9 and
// 6.2, 4096 x 4096 bf16 10.0 and 9.1, 8192 x 4096 bf16 16.5 and 14.5 (fp32 27.3 and 27.6).
constexpr int64_t kMrFill = 2048;
}  // namespace

hipError_t launch_mx_rows(const MxRowsArgs& a, hipStream_t st) {
  if (a.R == 0 || a.K == 0 || a.G == 0) return hipSuccess;
  const int64_t one = (a.K + 127) / 128 * ((a.R + kMrRows - 1) / kMrRows) * a.G;       // workgroups of one step
  if (a.dtype == S3R_BF16) return one < kMrFill ? run_rows<uint16_t, 1>(a, st) : run_rows<uint16_t, 4>(a, st);
  return one < kMrFill ? run_rows<float, 1>(a, st) : run_rows<float, 4>(a, st);
}

namespace {
using Tile256 = Tile<4, 2, 2, 4, 3, 2>;        // 256 x 256, 8 waves
using Tile256x128 = Tile<2, 2, 4, 2, 3, 4>;    // 8 waves, two workgroups per CU
using Tile128 = Tile<2, 2, 2, 2, 3, 3>;        // 4 waves, three workgroups per CU
using Tile128x64 = Tile<2, 1, 2, 2, 6, 2>;
using Tile64 = Tile<1, 1, 2, 2, 6, 2>;

// The largest tile that still gives this many workgroups (three quarters of the CUs): larger tiles read
// the operands less often, fewer workgroups leave CUs idle.  N = 14336, K = 4096, rows and product, us:
//   rows   128 x 64  128 x 128  256 x 128
//    128       15.6       19.5       22.7     (224 / 112 / 112 workgroups)
//    384       28.5       24.4       25.0     (672 / 336 / 224)
//   1024       55.7       47.3       40.7     (1792 / 896 / 448)
constexpr int64_t kFillTiles = 192;

template <typename T, typename TOut>
hipError_t run_tiles(const MxProductArgs& a, MxProdK p, hipStream_t st) {
  const int64_t mt = a.G ? a.M / T::BM + std::min(a.G, a.M) : (a.M + T::BM - 1) / T::BM;
  p.tiles_n = (int)((a.N + T::BN - 1) / T::BN);
  if ((mt * p.tiles_n + 7) * T::Threads >= (int64_t)1 << 32) return hipErrorInvalidConfiguration;
  const int64_t blocks = a.G ? (mt * p.tiles_n + 7) / 8 * 8 : mt * p.tiles_n;
  hipLaunchKernelGGL((mx_tile_kernel<T, TOut>), dim3((unsigned)blocks), dim3(T::Threads), 0, st, p, (int)mt);
  return hipGetLastError();
}
}  // namespace

namespace {
MxProdK product_params(const MxProductArgs& a) {
  MxProdK p{};
  p.A = a.A; p.lda = a.lda; p.As = a.As; p.ldas = a.ldas;
  p.B = a.B; p.ldb = a.ldb; p.Bs = a.Bs; p.ldbs = a.ldbs; p.b_stride = a.b_stride; p.bs_stride = a.bs_stride;
  p.offsets = a.offsets; p.G = a.G; p.M = a.M; p.N = a.N; p.ksteps = (int)((a.K + 127) / 128);
  p.out = a.out; p.ld_out = a.ld_out; p.flags = a.flags;
  return p;
}

// rows per weight, on average (only the device knows the groups' own)
int64_t mean_rows(const MxProductArgs& a) { return a.G ? (a.M + a.G - 1) / a.G : a.M; }

template <typename TIn, bool Words, int MI, int NJ, int Depth>
hipError_t run_few_rows(const MxProductArgs& a, const MxRowsArgs& q, hipStream_t st) {
  MxProdK p = product_params(a);
  // grouped: the tiles of every group, at most one partial tile each
  const int64_t mt = a.G ? a.M / (16 * MI) + std::min(a.G, a.M) : (a.M + 16 * MI - 1) / (16 * MI);
  p.tiles_n = (int)((a.N + 16 * NJ - 1) / (16 * NJ));
  if (mt * p.tiles_n * kSkThreads >= (int64_t)1 << 32) return hipErrorInvalidConfiguration;
  const dim3 grid((unsigned)(mt * p.tiles_n)), block(kSkThreads);
  const int rows = (int)std::min<int64_t>(a.M, 16);
  const size_t lds = std::is_void<TIn>::value ? 0 : sk_lds_bytes(rows, p.ksteps);
  if (a.out_dt == S3R_BF16)
    hipLaunchKernelGGL((mx_few_rows_kernel<uint16_t, TIn, Words, MI, NJ, Depth>), grid, block, lds, st, p, q, rows);
  else
    hipLaunchKernelGGL((mx_few_rows_kernel<float, TIn, Words, MI, NJ, Depth>), grid, block, lds, st, p, q, rows);
  return hipGetLastError();
}

template <typename T>
int64_t tile_count(const MxProductArgs& a) { return ((a.M + T::BM - 1) / T::BM) * ((a.N + T::BN - 1) / T::BN); }

template <typename T>
hipError_t run_tiles(const MxProductArgs& a, hipStream_t st) {
  const MxProdK p = product_params(a);
  return a.out_dt == S3R_BF16 ? run_tiles<T, uint16_t>(a, p, st) : run_tiles<T, float>(a, p, st);
}

constexpr int kFewNJ = 2;                       // 16-column tiles of a workgroup
// Largest number of few-rows workgroups of 16 rows before their repeated reads of the weights cost more
// than workgroups of 32 rows or LDS tiles lose to latency.  Rows and product, us:
//   64 rows, N = 1408, K = 2048: 176 of them 6.7, LDS tiles 8.9;  64 rows, N = 4096, K = 4096: 512 10.9, 12.9;
//   32 rows, N = 14336, K = 4096: 896 15.9, of 32 rows 14.0, LDS tiles 13.5; 48 rows: 1344 19.8, LDS tiles 13.7
constexpr int64_t kFewBlocks = 512;
// Rows per weight, on average, up to which a grouped product takes the few-rows kernel.  64 experts,
// N = 1408, K = 2048: 8 rows 21.0 us against 22.4 in 128 x 128 tiles, 16 rows 26.7 against 29.5, 32 rows
// 42.7 against 31.5.
constexpr int64_t kFewGrouped = 16;
// From here on the taller tile: 8 experts, N = K = 4096, 1024 rows each 102.8 against 103.3 us in 128 x 128
// tiles, 4096 rows 350 against 363.
constexpr int64_t kTallGrouped = 1024;
// Rows that the few-rows kernel rounds itself: 1 row, N = 14336, K = 4096 9.2 us against 11.4 with a launch
// of their own, 4 rows 11.8 against 12.0, 8 rows 15.7 against 12.1; grouped, at most a row per weight on average.
constexpr int64_t kRoundRows = 2;

template <typename TIn>
hipError_t run_round_few(const MxProductArgs& a, const MxRowsArgs& q, hipStream_t st) {
  return mr_words(q) ? run_few_rows<TIn, true, 1, kFewNJ, 2>(a, q, st) : run_few_rows<TIn, false, 1, kFewNJ, 2>(a, q, st);
}
}  // namespace

hipError_t launch_check_offsets(const int64_t* offsets, int64_t G, int64_t R, uint32_t* flags, hipStream_t st) {
  if (!G || !flags) return hipSuccess;
  hipLaunchKernelGGL(mx_offsets_kernel, dim3(1), dim3(64), 0, st, offsets, G, R, flags);
  return hipGetLastError();
}

hipError_t launch_mx_product(const MxProductArgs& a, hipStream_t st) {
  if (a.M == 0 || a.N == 0) return launch_check_offsets(a.offsets, a.G, a.M, a.flags, st);
  if (a.G) {
    const int64_t rows = mean_rows(a);
    if (rows <= kFewGrouped) return run_few_rows<void, true, 1, kFewNJ, 2>(a, MxRowsArgs{}, st);
    return rows < kTallGrouped ? run_tiles<Tile128>(a, st) : run_tiles<Tile256x128>(a, st);
  }
  const int64_t few = (a.M + 15) / 16 * ((a.N + 16 * kFewNJ - 1) / (16 * kFewNJ));
  if (a.M <= 16 || (a.M <= 64 && few <= kFewBlocks)) return run_few_rows<void, true, 1, kFewNJ, 4>(a, MxRowsArgs{}, st);
  if (a.M <= 32) return run_few_rows<void, true, 2, kFewNJ, 4>(a, MxRowsArgs{}, st);
  if (tile_count<Tile256>(a) >= kFillTiles) return run_tiles<Tile256>(a, st);
  if (tile_count<Tile256x128>(a) >= kFillTiles) return run_tiles<Tile256x128>(a, st);
  if (tile_count<Tile128>(a) >= kFillTiles) return run_tiles<Tile128>(a, st);
  if (tile_count<Tile128x64>(a) >= kFillTiles) return run_tiles<Tile128x64>(a, st);
  return run_tiles<Tile64>(a, st);
}

// Rows and product; `rows` writes the codes that `prod` reads, unless the few-rows kernel rounds them itself.
hipError_t launch_mx_linear(const MxRowsArgs& rows, const MxProductArgs& prod, hipStream_t st) {
  if (prod.M == 0 || prod.N == 0) return launch_check_offsets(prod.offsets, prod.G, prod.M, prod.flags, st);
  const int ksteps = (int)((prod.K + 127) / 128);
  if (!rows.up && prod.M <= std::max(prod.G, kRoundRows) &&
      sk_lds_bytes((int)std::min<int64_t>(prod.M, 16), ksteps) + 3 * kFewNJ * 1024 <= kSkLdsMax)
    return rows.dtype == S3R_BF16 ? run_round_few<uint16_t>(prod, rows, st) : run_round_few<float>(prod, rows, st);
  const hipError_t e = launch_mx_rows(rows, st);
  return e != hipSuccess ? e : launch_mx_product(prod, st);
}

}  // namespace s3r
