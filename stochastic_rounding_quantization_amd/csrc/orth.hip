// Orthogonalised updates: Newton-Schulz steps that drive a matrix's singular values to about 1,
//   X <- G / (|G|_F + eps),   then   A = X X^T,  B = a I + b A + c A A,  X <- B X   for every step,
// X taken with the smaller side as its rows (m x n, m <= n), so that A and B are m x m.
//
// Precision: the steps multiply small singular values by a each time, and with them every error made before, so the
// products carry about 22 bits: a value is kept as two fp16 planes, v 2^12 = h + l with h and l the nearest fp16, and
// a product is h h' + h l' + l h' in fp32 (three matrix instructions; l l' is below 2^-22).  The factor 2^12 keeps l of
// entries down to 2^-15 normal; entries up to 16 fit, and the singular values of X, A and B stay below 4.
//
// Layout: the planes of 32 consecutive elements of a row share a 128-byte line, 64 bytes of h and 64 of l, so a K step
// of 32 elements of both planes is one line of every row.  Every operand has its contraction along the rows: X for
// X X^T, X^T for B X, A and B as they are (symmetric).  So a step keeps X both ways, written by one epilogue.
// Sides are padded to whole tiles with zeros, which are all in the workspace: the products read and write no edge.
#include <type_traits>

#include "s3r_internal.h"
#include "tile_ring.h"

namespace s3r {
namespace {

typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef float v4f __attribute__((ext_vector_type(4)));

constexpr float kUp = 4096.f, kDown = 1.f / 4096.f;      // the planes' scale
constexpr int kLine = 128, kLineEl = 32;                 // bytes and elements of a line

// ------------------------------------------------------------------ norm ----
// Sum of squares in fp64: no square of an fp32 number leaves its range.  Partial sums of kNormBlocks workgroups a
// matrix, added in a fixed order by whoever needs the norm.
constexpr int kNormThreads = 256, kNormBlocks = 64;

__device__ __forceinline__ float element(const float* p) { return *p; }
__device__ __forceinline__ float element(const uint16_t* p) { return bf16_to_f32(*p); }

__device__ __forceinline__ double block_sum(double v) {
  __shared__ double red[kNormThreads / 64];
  v = wave_sum(v);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  double s = 0.;
#pragma unroll
  for (int w = 0; w < kNormThreads / 64; ++w) s += red[w];
  return s;
}

template <typename TIn>
__global__ __launch_bounds__(kNormThreads) void orth_norm_kernel(OrthArgs a, double* part) {
  const TIn* G = (const TIn*)a.G + (int64_t)blockIdx.y * a.g_stride;
  double s = 0.;
  const int64_t rows = (a.N + kNormBlocks - 1) / kNormBlocks;
  const int64_t r0 = blockIdx.x * rows, r1 = min(r0 + rows, a.N);
  for (int64_t r = r0; r < r1; ++r)
    for (int64_t c = threadIdx.x; c < a.K; c += kNormThreads) {
      const double v = element(G + r * a.ld + c);
      s += v * v;
    }
  s = block_sum(s);
  if (threadIdx.x == 0) part[(int64_t)blockIdx.y * kNormBlocks + blockIdx.x] = s;
}

// 2^12 / (norm + eps) from the partial sums, by one wave; NaN for a matrix that is not finite, 0 for one of zeros
// without an eps.
__device__ __forceinline__ float orth_factor(const double* part, float eps) {
  static_assert(kNormBlocks == 64, "a partial sum a lane");
  const double s = wave_sum(part[threadIdx.x & 63]);
  const double d = sqrt(s) + (double)eps;
  if (!(s < __builtin_inf())) return __builtin_nanf("");
  return d > 0. ? (float)((double)kUp / d) : 0.f;
}

// ---------------------------------------------------------------- planes ----
// The compiler may round what v was computed from to fp16 in one step where h is stored and in two where h is
// subtracted, and near a tie these differ by 2^-11 of v: the empty assembly makes v one number.
__device__ __forceinline__ void split(float v, _Float16& h, _Float16& l) {
  asm("" : "+v"(v));
  h = (_Float16)v;
  l = (_Float16)(v - (float)h);
}
__device__ __forceinline__ int64_t plane_off(int64_t row, int64_t col, int64_t ld) {        // ld in bytes
  return row * ld + (col / kLineEl) * kLine + (col % kLineEl) * 2;
}
// 8 consecutive values (col a multiple of 8) to their planes.
__device__ __forceinline__ void store_planes(uint8_t* p, const float (&v)[8]) {
  v8h h, l;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    _Float16 x, y;
    split(v[i], x, y);
    h[i] = x;
    l[i] = y;
  }
  *reinterpret_cast<v8h*>(p) = h;
  *reinterpret_cast<v8h*>(p + kLine / 2) = l;
}

// G, scaled, to its planes as it lies (`own`) and transposed (`other`), 64 x 64 elements a workgroup, zeros past its
// edges.  rows x cols: the padded sizes, G's orientation.
constexpr int kPrepThreads = 256, kPrepTile = 64;
template <typename TIn>
__global__ __launch_bounds__(kPrepThreads) void orth_prepare_kernel(OrthArgs a, const double* part, uint8_t* own,
                                                                    int64_t own_stride, uint8_t* other, int64_t other_stride,
                                                                    int64_t rows, int64_t cols) {
  __shared__ float tile[kPrepTile][kPrepTile + 1];
  __shared__ float factor;
  const int64_t e = blockIdx.z;
  if (threadIdx.x < 64) {
    const float f = orth_factor(part + e * kNormBlocks, a.eps);
    if (threadIdx.x == 0) factor = f;
  }
  const TIn* G = (const TIn*)a.G + e * a.g_stride;
  const int64_t r0 = (int64_t)blockIdx.y * kPrepTile, c0 = (int64_t)blockIdx.x * kPrepTile;
  for (int i = threadIdx.x; i < kPrepTile * kPrepTile; i += kPrepThreads) {
    const int64_t r = r0 + i / kPrepTile, c = c0 + i % kPrepTile;
    tile[i / kPrepTile][i % kPrepTile] = r < a.N && c < a.K ? element(G + r * a.ld + c) : 0.f;
  }
  __syncthreads();
  const float f = factor;
  own += e * own_stride;
  other += e * other_stride;
  for (int i = threadIdx.x; i < kPrepTile * kPrepTile / 8; i += kPrepThreads) {
    const int q = i / (kPrepTile / 8), p = i % (kPrepTile / 8) * 8;
    float v[8], w[8];
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      v[x] = tile[q][p + x] * f;
      w[x] = tile[p + x][q] * f;
    }
    store_planes(own + plane_off(r0 + q, c0 + p, cols * 4), v);
    store_planes(other + plane_off(c0 + q, r0 + p, rows * 4), w);
  }
}

// -------------------------------------------------------------- products ----
// Tiles of BM x BN, WM x WN waves of (32 MI) x (32 NI) each, operands staged through LDS by buffer-load DMA in a ring
// of NS steps of one line (32 elements, both planes) of every row, the eight 16-byte chunks of a line at permuted places
// (chunk q of row r at q ^ ((r >> 1) & 7): a quarter-wave's reads hit 16 bank groups).
// v_mfma_f32_32x32x16_f16: lane l holds row or column l % 32, elements 8 (l / 32) .. + 7 of 16; result register r is
// row (r / 4) 8 + (l / 32) 4 + r % 4, column l % 32.
template <int MI_, int NI_, int WM_, int WN_, int NS_, int WavesPerSimd_>
struct OrthGeo {
  static constexpr int WavesPerSimd = WavesPerSimd_;
  static constexpr int MI = MI_, NI = NI_, WM = WM_, WN = WN_, NS = NS_;
  static constexpr int Waves = WM * WN, Threads = 64 * Waves;
  static constexpr int BM = 32 * MI * WM, BN = 32 * NI * WN;
  static constexpr int PA = BM / 8 / Waves, PB = BN / 8 / Waves;          // 1 KiB pieces per wave
  static constexpr int Loads = PA + PB;
  static constexpr int OffB = BM * kLine;
  static constexpr int StageBytes = OffB + BN * kLine;
  static constexpr int EpiLd = 32 * NI + 4;                               // floats per row of the epilogue's staging
  static_assert(BM % (8 * Waves) == 0 && BN % (8 * Waves) == 0, "whole pieces per wave");
};

struct OrthGemm {
  const uint8_t *A, *B;                // operands' planes
  int64_t lda, ldb, a_stride, b_stride;        // bytes
  int tiles_m, tiles_n, per_matrix;    // tiles of a matrix; symmetric results: of its upper triangle
  int steps;                           // lines of the contraction
  int full, rest, workers;             // whole tiles, tiles that `workers` workgroups share, after them
  float* partial;                      // two tiles a worker
  // results
  uint8_t *direct, *turned; int64_t ld_direct, ld_turned, d_stride, t_stride;
  const uint8_t* addend;               // A of B = a I + b A + c A A
  float a, b, c;
  void* out; int64_t ld_out, out_stride, rows, cols;
  float scale, keep;
};

// What a product's results become.
enum OrthEpi {
  kEpiGram,        // planes of a symmetric matrix, both triangles
  kEpiPoly,        // a I + b A + c (this), the same
  kEpiBoth,        // planes as the tile lies and transposed
  kEpiOutF32, kEpiOutBf16      // the caller's matrix
};
__host__ __device__ constexpr bool symmetric(OrthEpi e) { return e == kEpiGram || e == kEpiPoly; }

__device__ __forceinline__ int chunk_place(int r, int q) { return q ^ ((r >> 1) & 7); }

template <typename T>
struct OrthSrc {
  __amdgpu_buffer_rsrc_t a, b, z;
  uint32_t va[T::PA], vb[T::PB];              // this lane's byte offsets in step 0
  int k0, nk;                                 // first step, steps
};

// Step kt into stage st; past the last step every load reads zeros, so the wait counts stay the same.
template <typename T>
__device__ __forceinline__ void orth_load(const OrthSrc<T>& s, uint8_t* st, int kt) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const bool live = kt < s.nk;
  const __amdgpu_buffer_rsrc_t ra = live ? s.a : s.z, rb = live ? s.b : s.z;
  const uint32_t koff = (uint32_t)(s.k0 + kt) * (uint32_t)kLine;
#pragma unroll
  for (int q = 0; q < T::PA; ++q) dma16(ra, st + (wave * T::PA + q) * 1024, s.va[q], koff);
#pragma unroll
  for (int q = 0; q < T::PB; ++q) dma16(rb, st + T::OffB + (wave * T::PB + q) * 1024, s.vb[q], koff);
}

template <typename T>
struct OrthFrag { v8h ah[T::MI], al[T::MI], bh[T::NI], bl[T::NI]; };

// The fragments of half h (16 elements) of a stage.
template <typename T>
__device__ __forceinline__ void orth_frag(const uint8_t* st, int h, OrthFrag<T>& f) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wm = wave / T::WN, wn = wave % T::WN;
  const int r31 = lane & 31, c = h * 2 + (lane >> 5);
#pragma unroll
  for (int i = 0; i < T::MI; ++i) {
    const int r = (wm * T::MI + i) * 32 + r31;
    f.ah[i] = *reinterpret_cast<const v8h*>(st + r * kLine + (chunk_place(r, c) << 4));
    f.al[i] = *reinterpret_cast<const v8h*>(st + r * kLine + (chunk_place(r, c + 4) << 4));
  }
#pragma unroll
  for (int j = 0; j < T::NI; ++j) {
    const int r = (wn * T::NI + j) * 32 + r31;
    f.bh[j] = *reinterpret_cast<const v8h*>(st + T::OffB + r * kLine + (chunk_place(r, c) << 4));
    f.bl[j] = *reinterpret_cast<const v8h*>(st + T::OffB + r * kLine + (chunk_place(r, c + 4) << 4));
  }
}

template <typename T>
__device__ __forceinline__ void orth_mfma(const OrthFrag<T>& f, v16f (&acc)[T::MI][T::NI]) {
#pragma unroll
  for (int i = 0; i < T::MI; ++i)
#pragma unroll
    for (int j = 0; j < T::NI; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(f.al[i], f.bh[j], acc[i][j], 0, 0, 0);
#pragma unroll
  for (int i = 0; i < T::MI; ++i)
#pragma unroll
    for (int j = 0; j < T::NI; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(f.ah[i], f.bl[j], acc[i][j], 0, 0, 0);
#pragma unroll
  for (int i = 0; i < T::MI; ++i)
#pragma unroll
    for (int j = 0; j < T::NI; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(f.ah[i], f.bh[j], acc[i][j], 0, 0, 0);
}

// Step kt on stage S = kt % NS, the fragments of its first half in f.  The first half's products cover the reads of the
// second half; the barrier between them makes step kt + 1 visible and retires stage S, which takes step kt + NS.
template <typename T, int S>
__device__ __forceinline__ void orth_step(const OrthSrc<T>& src, int kt, OrthFrag<T>& f, v16f (&acc)[T::MI][T::NI]) {
  constexpr int kReads = 2 * (T::MI + T::NI), kProducts = 3 * T::MI * T::NI;
  OrthFrag<T> n;
  orth_frag<T>(ring<T, S>(), 1, n);
  orth_mfma<T>(f, acc);
#pragma unroll
  for (int x = 0; x < kProducts; ++x) {
    __builtin_amdgcn_sched_group_barrier(kSgDsRead, (kReads + kProducts - 1) / kProducts, 0);
    __builtin_amdgcn_sched_group_barrier(kSgMfma, 1, 0);
  }
  __builtin_amdgcn_sched_barrier(0);
  S3R_WAIT_VM(T::Loads * (T::NS - 2));
  S3R_WAIT_LGKM0();
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_sched_barrier(0);
  orth_load<T>(src, ring<T, S>(), kt + T::NS);
  orth_frag<T>(ring<T, (S + 1) % T::NS>(), 0, f);
  orth_mfma<T>(n, acc);
#pragma unroll
  for (int x = 0; x < kProducts; ++x) {
    __builtin_amdgcn_sched_group_barrier(kSgMfma, 1, 0);
    __builtin_amdgcn_sched_group_barrier(kSgDsRead, (kReads + kProducts - 1) / kProducts, 0);
    __builtin_amdgcn_sched_group_barrier(kSgVmem, (T::Loads + kProducts - 1) / kProducts, 0);
  }
  __builtin_amdgcn_sched_barrier(0);
}

template <typename T, int S>
__device__ __forceinline__ void orth_fill(const OrthSrc<T>& src) {
  if constexpr (S < T::NS) {
    orth_load<T>(src, ring<T, S>(), S);
    orth_fill<T, S + 1>(src);
  }
}

template <typename T, int S>
__device__ __forceinline__ void orth_steps(const OrthSrc<T>& src, int kt, OrthFrag<T>& f, v16f (&acc)[T::MI][T::NI]) {
  if constexpr (S < T::NS) {
    if (kt + S < src.nk) {
      orth_step<T, S>(src, kt + S, f, acc);
      orth_steps<T, S + 1>(src, kt, f, acc);
    }
  }
}

// Tile t of a product: its matrix, its row and its column of tiles.
struct OrthTile { int e, tm, tn; };
template <OrthEpi EPI>
__device__ __forceinline__ OrthTile orth_tile(const OrthGemm& p, int t) {
  OrthTile o;
  o.e = t / p.per_matrix;
  int i = t - o.e * p.per_matrix;
  if constexpr (symmetric(EPI)) {              // the upper triangle, row by row
    o.tm = 0;
    for (int w = p.tiles_n; i >= w; --w) {
      i -= w;
      ++o.tm;
    }
    o.tn = o.tm + i;
  } else {                                     // eight rows of tiles at a time
    const int group = 8 * p.tiles_n, first = i / group * 8;
    const int size = min(p.tiles_m - first, 8), in = i % group;
    o.tm = first + in % size;
    o.tn = in / size;
  }
  return o;
}

// The sums of steps [k0, k1) of a tile.
template <typename T>
__device__ __forceinline__ void orth_sums(const OrthGemm& p, const OrthTile& t, int k0, int k1, v16f (&acc)[T::MI][T::NI]) {
  OrthSrc<T> src;
  src.k0 = k0;
  src.nk = k1 - k0;
  const uint8_t* A = p.A + t.e * p.a_stride + (int64_t)t.tm * T::BM * p.lda;
  const uint8_t* B = p.B + t.e * p.b_stride + (int64_t)t.tn * T::BN * p.ldb;
  src.a = __builtin_amdgcn_make_buffer_rsrc((void*)A, (short)0, (int)(uint32_t)(T::BM * p.lda), kRsrcWord3);
  src.b = __builtin_amdgcn_make_buffer_rsrc((void*)B, (short)0, (int)(uint32_t)(T::BN * p.ldb), kRsrcWord3);
  src.z = __builtin_amdgcn_make_buffer_rsrc((void*)A, (short)0, 0, kRsrcWord3);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
#pragma unroll
  for (int q = 0; q < T::PA; ++q) {
    const int r = (wave * T::PA + q) * 8 + (lane >> 3);
    src.va[q] = (uint32_t)(r * p.lda + chunk_place(r, lane & 7) * 16);
  }
#pragma unroll
  for (int q = 0; q < T::PB; ++q) {
    const int r = (wave * T::PB + q) * 8 + (lane >> 3);
    src.vb[q] = (uint32_t)(r * p.ldb + chunk_place(r, lane & 7) * 16);
  }
#pragma unroll
  for (int i = 0; i < T::MI; ++i)
#pragma unroll
    for (int j = 0; j < T::NI; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
  orth_fill<T, 0>(src);
  S3R_WAIT_VM(T::Loads * (T::NS - 1));
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_sched_barrier(0);
  OrthFrag<T> f;
  orth_frag<T>(ring<T, 0>(), 0, f);
  for (int kt = 0; kt < src.nk; kt += T::NS) orth_steps<T, 0>(src, kt, f, acc);
  S3R_WAIT_VM(0);
  S3R_WAIT_LGKM0();
  __builtin_amdgcn_s_barrier();
}

__device__ __forceinline__ void store_one(float* p, float v, float keep) { *p = keep == 0.f ? v : v + keep * *p; }
__device__ __forceinline__ void store_one(uint16_t* p, float v, float keep) {
  *reinterpret_cast<__bf16*>(p) = (__bf16)(keep == 0.f ? v : v + keep * bf16_to_f32(*p));
}

// A tile's results, 32 rows of a wave at a time through its own part of the (free) ring, read from there along the rows
// and along the columns.
template <typename T, OrthEpi EPI>
__device__ __forceinline__ void orth_store(const OrthGemm& p, const OrthTile& t, const v16f (&acc)[T::MI][T::NI]) {
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
  constexpr int W = 32 * T::NI, LR = W / 8;                   // columns of a wave; lanes of a row, 8 columns each
  const int64_t col0 = (int64_t)t.tn * T::BN + wn * W;
  const bool turned = EPI == kEpiBoth || (symmetric(EPI) && t.tm != t.tn);
#pragma unroll
  for (int i = 0; i < T::MI; ++i) {
    const int64_t row0 = (int64_t)t.tm * T::BM + (wm * T::MI + i) * 32;
#pragma unroll
    for (int j = 0; j < T::NI; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r)
        buf[((r >> 2) * 8 + (lane >> 5) * 4 + (r & 3)) * T::EpiLd + j * 32 + (lane & 31)] = acc[i][j][r] * kDown;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    for (int q = 0; q < 32; q += 64 / LR) {
      const int rr = q + lane / LR, cc = lane % LR * 8;
      const int64_t row = row0 + rr, col = col0 + cc;
      float v[8];
#pragma unroll
      for (int x = 0; x < 8; x += 4) {
        const v4f w = *reinterpret_cast<const v4f*>(buf + rr * T::EpiLd + cc + x);
#pragma unroll
        for (int y = 0; y < 4; ++y) v[x + y] = w[y];
      }
      if constexpr (EPI == kEpiPoly) {
        const uint8_t* at = p.addend + t.e * p.d_stride + plane_off(row, col, p.ld_direct);
        const v8h h = *reinterpret_cast<const v8h*>(at), l = *reinterpret_cast<const v8h*>(at + kLine / 2);
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          v[x] = p.c * v[x] + p.b * ((float)h[x] + (float)l[x]);
          if (row == col + x) v[x] += p.a * kUp;
        }
        if (turned) {
#pragma unroll
          for (int x = 0; x < 8; x += 4)
            *reinterpret_cast<v4f*>(buf + rr * T::EpiLd + cc + x) = v4f{v[x], v[x + 1], v[x + 2], v[x + 3]};
        }
      }
      if constexpr (EPI == kEpiOutF32 || EPI == kEpiOutBf16) {
        using TOut = std::conditional_t<EPI == kEpiOutF32, float, uint16_t>;
        TOut* out = (TOut*)p.out + t.e * p.out_stride + row * p.ld_out + col;
        if (row < p.rows) {
#pragma unroll
          for (int x = 0; x < 8; ++x)
            if (col + x < p.cols) store_one(out + x, v[x] * (kDown * p.scale), p.keep);
        }
      } else {
        store_planes(p.direct + t.e * p.d_stride + plane_off(row, col, p.ld_direct), v);
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    if constexpr (EPI == kEpiBoth || symmetric(EPI)) {
      if (turned)
        for (int q = 0; q < 4 * W; q += 64) {                 // a column's 8 rows a lane
          const int cc = (q + lane) >> 2, rr = (lane & 3) * 8;
          float v[8];
#pragma unroll
          for (int x = 0; x < 8; ++x) v[x] = buf[(rr + x) * T::EpiLd + cc];
          store_planes(p.turned + t.e * p.t_stride + plane_off(col0 + cc, row0 + rr, p.ld_turned), v);
        }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
    }
  }
}

// The steps of all shared tiles in a row, dealt to the workers evenly: worker w has [first(w), first(w + 1)).
__device__ __forceinline__ int64_t first_step(const OrthGemm& p, int w) {
  return (int64_t)w * ((int64_t)p.rest * p.steps) / p.workers;
}

// Workgroups 0 .. full - 1 take a tile each.  What does not fill the GPU evenly, the last `rest` tiles, is dealt to
// `workers` workgroups by steps: each leaves the sums of its part of a tile in memory (at most two tiles are partly its
// own; tiles wholly its own go straight to their results) and orth_join_kernel adds them up, in the order of K.
template <typename T, OrthEpi EPI>
__global__ __launch_bounds__(T::Threads, T::WavesPerSimd) void orth_gemm_kernel(OrthGemm p) {
  v16f acc[T::MI][T::NI];
  int bid = blockIdx.x;
  if (bid < p.full) {
    if (p.full % 8 == 0) bid = (bid % 8) * (p.full / 8) + bid / 8;       // a contiguous range of tiles per XCD
    const OrthTile t = orth_tile<EPI>(p, bid);
    orth_sums<T>(p, t, 0, p.steps, acc);
    orth_store<T, EPI>(p, t, acc);
    return;
  }
  int w = bid - p.full;
  if (p.workers % 8 == 0) w = (w % 8) * (p.workers / 8) + w / 8;
  const int64_t s1 = first_step(p, w + 1);
  int slot = 0;
  for (int64_t s = first_step(p, w); s < s1;) {
    const int tile = (int)(s / p.steps), k0 = (int)(s - (int64_t)tile * p.steps);
    const int k1 = (int)min((int64_t)p.steps, k0 + (s1 - s));
    const OrthTile t = orth_tile<EPI>(p, p.full + tile);
    orth_sums<T>(p, t, k0, k1, acc);
    if (k1 - k0 == p.steps) {
      orth_store<T, EPI>(p, t, acc);
    } else {
      v4f* part = reinterpret_cast<v4f*>(p.partial) + (int64_t)(2 * w + slot) * (T::BM * T::BN / 4) + threadIdx.x;
      slot = 1;
#pragma unroll
      for (int i = 0; i < T::MI; ++i)
#pragma unroll
        for (int j = 0; j < T::NI; ++j)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            part[((i * T::NI + j) * 4 + r) * T::Threads] =
                v4f{acc[i][j][4 * r], acc[i][j][4 * r + 1], acc[i][j][4 * r + 2], acc[i][j][4 * r + 3]};
    }
    S3R_WAIT_VM(0);
    __syncthreads();                   // the ring is free again, and the next loads are counted from none
    s += k1 - k0;
  }
}

template <typename T, OrthEpi EPI>
__global__ __launch_bounds__(T::Threads, T::WavesPerSimd) void orth_join_kernel(OrthGemm p) {
  const int tile = blockIdx.x;
  const int64_t s0 = (int64_t)tile * p.steps, s1 = s0 + p.steps, all = (int64_t)p.rest * p.steps;
  int w = (int)(s0 * p.workers / all);
  while (first_step(p, w + 1) <= s0) ++w;
  while (first_step(p, w) > s0) --w;
  if (first_step(p, w + 1) >= s1) return;              // one worker had all of it
  v16f acc[T::MI][T::NI];
#pragma unroll
  for (int i = 0; i < T::MI; ++i)
#pragma unroll
    for (int j = 0; j < T::NI; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
  for (; first_step(p, w) < s1; ++w) {
    // a worker's second part follows a tile's end; its first one is the tile that its range begins in
    const int64_t b = first_step(p, w);
    if (b == first_step(p, w + 1)) continue;
    const int slot = b < s0 && b % p.steps != 0 ? 1 : 0;
    const v4f* part = reinterpret_cast<const v4f*>(p.partial) + (int64_t)(2 * w + slot) * (T::BM * T::BN / 4) + threadIdx.x;
#pragma unroll
    for (int i = 0; i < T::MI; ++i)
#pragma unroll
      for (int j = 0; j < T::NI; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const v4f v = part[((i * T::NI + j) * 4 + r) * T::Threads];
#pragma unroll
          for (int y = 0; y < 4; ++y) acc[i][j][4 * r + y] += v[y];
        }
  }
  orth_store<T, EPI>(p, orth_tile<EPI>(p, p.full + tile), acc);
}

// -------------------------------------------------------------- launches ----
using Orth256 = OrthGeo<4, 2, 2, 4, 2, 2>;       // 256 x 256, 8 waves, a workgroup per CU
using Orth128 = OrthGeo<2, 2, 2, 2, 2, 2>;       // 128 x 128, 4 waves, two per CU
using Orth64 = OrthGeo<1, 1, 2, 2, 4, 2>;        // 64 x 64, 4 waves, two per CU
template <typename T> constexpr int kSlots = std::is_same<T, Orth256>::value ? 256 : 512;
// Steps of a tile that sharing the last tiles has to save to be worth a launch and the way through memory (~10 us).
template <typename T> constexpr int kShareGain = T::BM == 256 ? 4 : T::BM == 128 ? 8 : 32;
constexpr int kShareLeast = 4;                   // steps of a worker, at least

int tile_side(const OrthArgs& a) {
  const int64_t m = std::min(a.N, a.K), n = std::max(a.N, a.K);
  auto tiles = [&](int64_t side) { return a.E * ((m + side - 1) / side) * ((n + side - 1) / side); };
  if (tiles(128) < 256) return 64;
  const int64_t m128 = (m + 127) / 128 * 128, m256 = (m + 255) / 256 * 256;
  const int64_t n128 = (n + 127) / 128 * 128, n256 = (n + 255) / 256 * 256;
  return tiles(256) >= 256 && (double)m256 * n256 <= 1.05 * (double)m128 * n128 ? 256 : 128;
}

struct OrthLayout {
  int side;
  int64_t m, n, mp, np;
  size_t part, x, xt[2], A, B, partial, total;
};
OrthLayout orth_layout(const OrthArgs& a) {
  OrthLayout l{};
  l.side = tile_side(a);
  l.m = std::min(a.N, a.K);
  l.n = std::max(a.N, a.K);
  l.mp = (l.m + l.side - 1) / l.side * l.side;
  l.np = (l.n + l.side - 1) / l.side * l.side;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += align_up(bytes, 256);
    return here;
  };
  const size_t xs = (size_t)a.E * l.mp * l.np * 4, as = (size_t)a.E * l.mp * l.mp * 4;
  l.part = take((size_t)a.E * kNormBlocks * 8);
  l.x = take(xs);
  l.xt[0] = take(xs);
  l.xt[1] = take(xs);
  l.A = take(as);
  l.B = take(as);
  l.partial = take((size_t)(l.side == 256 ? 256 : 512) * 2 * l.side * l.side * 4);
  l.total = at;
  return l;
}

template <typename T, OrthEpi EPI>
hipError_t run_orth_gemm(OrthGemm p, int64_t E, hipStream_t st) {
  p.per_matrix = symmetric(EPI) ? p.tiles_n * (p.tiles_n + 1) / 2 : p.tiles_m * p.tiles_n;
  const int64_t tiles = E * p.per_matrix;
  if (tiles >= (int64_t)1 << 31 || (tiles + kSlots<T>) * T::Threads >= (int64_t)1 << 32) return hipErrorInvalidConfiguration;
  const int rest = (int)(tiles % kSlots<T>);
  const int64_t workers = std::min<int64_t>(kSlots<T>, (int64_t)rest * p.steps / kShareLeast);
  const bool share = workers > rest && (double)p.steps * (1.0 - (double)rest / workers) >= kShareGain<T>;
  p.rest = share ? rest : 0;
  p.workers = share ? (int)workers : 0;
  p.full = (int)tiles - p.rest;
  hipLaunchKernelGGL((orth_gemm_kernel<T, EPI>), dim3((unsigned)(p.full + p.workers)), dim3(T::Threads), 0, st, p);
  if (share) hipLaunchKernelGGL((orth_join_kernel<T, EPI>), dim3((unsigned)p.rest), dim3(T::Threads), 0, st, p);
  return hipGetLastError();
}

template <typename T>
hipError_t run_orth_steps(const OrthArgs& a, const OrthLayout& l, hipStream_t st) {
  char* ws = (char*)a.ws;
  uint8_t* x = (uint8_t*)ws + l.x;
  uint8_t *A = (uint8_t*)ws + l.A, *B = (uint8_t*)ws + l.B;
  const int64_t ld_x = l.np * 4, ld_t = l.mp * 4, xs = l.mp * l.np * 4, as = l.mp * l.mp * 4;
  const int tm = (int)(l.mp / T::BM), tn = (int)(l.np / T::BM);
  const int along_n = (int)((l.n + kLineEl - 1) / kLineEl), along_m = (int)((l.m + kLineEl - 1) / kLineEl);
  hipError_t err = hipSuccess;
  for (int s = 0; s < a.steps && err == hipSuccess; ++s) {
    const uint8_t* xt = (uint8_t*)ws + l.xt[s & 1];
    OrthGemm p{};
    p.partial = (float*)(ws + l.partial);
    p.a = a.a; p.b = a.b; p.c = a.c;
    p.A = p.B = x; p.lda = p.ldb = ld_x; p.a_stride = p.b_stride = xs;
    p.tiles_m = p.tiles_n = tm; p.steps = along_n;
    p.direct = p.turned = A; p.ld_direct = p.ld_turned = ld_t; p.d_stride = p.t_stride = as;
    if ((err = run_orth_gemm<T, kEpiGram>(p, a.E, st)) != hipSuccess) break;
    p.A = p.B = A; p.lda = p.ldb = ld_t; p.a_stride = p.b_stride = as;
    p.steps = along_m;
    p.addend = A;
    p.direct = p.turned = B;
    if ((err = run_orth_gemm<T, kEpiPoly>(p, a.E, st)) != hipSuccess) break;
    const bool last = s + 1 == a.steps, wide = a.N <= a.K;
    const uint8_t* first = last && wide ? B : xt;             // the tiles' rows: m's or n's
    p.A = first; p.a_stride = first == xt ? xs : as;
    p.B = first == xt ? B : xt; p.b_stride = first == xt ? as : xs;
    p.lda = p.ldb = ld_t;
    p.tiles_m = first == xt ? tn : tm; p.tiles_n = first == xt ? tm : tn;
    if (!last) {
      p.direct = (uint8_t*)ws + l.xt[~s & 1]; p.ld_direct = ld_t; p.d_stride = xs;
      p.turned = x; p.ld_turned = ld_x; p.t_stride = xs;
      err = run_orth_gemm<T, kEpiBoth>(p, a.E, st);
    } else {
      p.out = a.out; p.ld_out = a.ld_out; p.out_stride = a.out_stride; p.rows = a.N; p.cols = a.K;
      p.scale = a.scale; p.keep = a.keep;
      err = a.out_dt == S3R_BF16 ? run_orth_gemm<T, kEpiOutBf16>(p, a.E, st) : run_orth_gemm<T, kEpiOutF32>(p, a.E, st);
    }
  }
  return err;
}

template <typename TIn>
hipError_t run_orth_prepare(const OrthArgs& a, const OrthLayout& l, hipStream_t st) {
  char* ws = (char*)a.ws;
  double* part = (double*)(ws + l.part);
  hipLaunchKernelGGL((orth_norm_kernel<TIn>), dim3(kNormBlocks, (unsigned)a.E), dim3(kNormThreads), 0, st, a, part);
  const bool wide = a.N <= a.K;
  const int64_t rows = wide ? l.mp : l.np, cols = wide ? l.np : l.mp, xs = l.mp * l.np * 4;
  uint8_t *x = (uint8_t*)ws + l.x, *xt = (uint8_t*)ws + l.xt[0];
  hipLaunchKernelGGL((orth_prepare_kernel<TIn>), dim3((unsigned)(cols / kPrepTile), (unsigned)(rows / kPrepTile), (unsigned)a.E),
                     dim3(kPrepThreads), 0, st, a, part, wide ? x : xt, xs, wide ? xt : x, xs, rows, cols);
  return hipGetLastError();
}
}  // namespace

size_t orth_workspace(const OrthArgs& a) { return a.E * a.N * a.K == 0 ? 0 : orth_layout(a).total; }

hipError_t launch_orthogonalize(const OrthArgs& a, hipStream_t st) {
  if (a.E == 0 || a.N == 0 || a.K == 0) return hipSuccess;
  const OrthLayout l = orth_layout(a);
  const hipError_t e = a.g_dtype == S3R_BF16 ? run_orth_prepare<uint16_t>(a, l, st) : run_orth_prepare<float>(a, l, st);
  if (e != hipSuccess) return e;
  if (l.side == 256) return run_orth_steps<Orth256>(a, l, st);
  return l.side == 128 ? run_orth_steps<Orth128>(a, l, st) : run_orth_steps<Orth64>(a, l, st);
}

}  // namespace s3r
