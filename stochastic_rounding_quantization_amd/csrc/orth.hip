// Orthogonalised updates: Newton-Schulz steps that drive a matrix's singular values to about 1,
//   X <- G / (|G|_F + eps),   then   A = X X^T,  B = a I + b A + c A A,  X <- B X   for every step,
// X taken with the smaller side as its rows (m x n, m <= n), so that A and B are m x m.
//
// Precision: the steps multiply small singular values by a each time, and with them every error made before, so the
// products carry about 22 bits: a value is kept as two fp16 planes, v 2^12 = h + l with h and l the nearest fp16, and
// a product is h h' + h l' + l h' in fp32 (three matrix instructions; l l' is below 2^-22).  The factor 2^12 keeps l of
// entries down to 2^-15 normal; entries up to 16 fit, and the singular values of X, A and B stay below 4.
// A result in bf16 takes both planes in every step too: h alone loses 2^-12 of X, which fills the directions that a gradient of
// few tokens leaves empty, and one step multiplies it there by a (two steps: by a^2, 0.0023 - 0.0029 of the matrix at ranks 1 to
// 64, where rounding to bf16 is 0.0017).
//
// Layout: the 32 consecutive elements of a row that make a line of 128 bytes are 64 bytes of h and 64 of l.  A step of the
// products' loops is a line of every row.  Every operand has its
// contraction along the rows: X for X X^T, X^T for B X, A and B as they are (symmetric).  So a step keeps X both ways,
// written by one epilogue.  The matrix cores keep fp16's subnormals, so small h and l lose nothing more.  Sides are padded to whole tiles with zeros, which are all in the workspace: the products read
// and write no edge.
#include <type_traits>

#include "rows8.h"
#include "tile_ring.h"

namespace s3r {
namespace {

typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef float v4f __attribute__((ext_vector_type(4)));

constexpr float kUp = 4096.f, kDown = 1.f / 4096.f;      // the planes' scale
constexpr int kLine = 128;                               // bytes of a line
constexpr int kLineEl = 32, kElBytes = 4;                // elements of a line, bytes of an element

// ------------------------------------------------------------------ norm ----
// Sum of squares in fp64: no square of an fp32 number leaves its range.  A matrix is cut into runs of 2048 elements of a
// row, dealt evenly to `parts` workgroups; whoever needs the norm adds their sums in a fixed order.  Bound by its bytes:
// 4096 x 14336 fp32 42 - 57 us, 4.1 - 5.6 TB/s (in 64 parts 1495).
constexpr int kNormThreads = 256, kNormRun = kNormThreads * 8, kNormMost = 1024;

template <typename TIn>
__global__ __launch_bounds__(kNormThreads) void orth_norm_kernel(OrthArgs a, double* part, int parts) {
  __shared__ double red[kNormThreads / 64];
  const TIn* G = (const TIn*)a.G + (int64_t)blockIdx.y * a.g_stride;
  const int64_t per_row = (a.K + kNormRun - 1) / kNormRun, runs = a.N * per_row;
  const int64_t u0 = runs * blockIdx.x / parts, u1 = runs * (blockIdx.x + 1) / parts;
  double s = 0.;
  constexpr int kBatch = 4;
  for (int64_t u = u0; u < u1; u += kBatch) {
    Raw8<TIn> v[kBatch];
    int64_t left[kBatch];
#pragma unroll
    for (int q = 0; q < kBatch; ++q) {             // every load before the first sum
      const int64_t r = (u + q) / per_row, c = (u + q - r * per_row) * kNormRun + threadIdx.x * 8;
      left[q] = u + q < u1 ? a.K - c : 0;
      v[q] = mr_load8<TIn, false>(G + r * a.ld + c, left[q], a.K);
    }
#pragma unroll
    for (int q = 0; q < kBatch; ++q) {
      mr_tail<false>(v[q], left[q], a.K);
      const Raw8<float> f = mr_float8(v[q]);
#pragma unroll
      for (int x = 0; x < 8; ++x) s += (double)f.w[x] * (double)f.w[x];
    }
  }
  s = wave_sum(s);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x != 0) return;
  s = 0.;
#pragma unroll
  for (int w = 0; w < kNormThreads / 64; ++w) s += red[w];
  part[(int64_t)blockIdx.y * parts + blockIdx.x] = s;
}

// 2^12 / (norm + eps) from the partial sums, by one wave; NaN for a matrix that is not finite, 0 for one of zeros
// without an eps.  As power * rest: norms from 2^-149 on put the factor up to 2^161, which fp32 does not hold, and those
// above 2^138 among its subnormal numbers; the power of two brings elements so small or large to where the rest is normal.
struct OrthFactor {
  float power, rest;
  __device__ __forceinline__ float operator()(float v) const { return v * power * rest; }
};
__device__ __forceinline__ OrthFactor orth_factor(const double* part, int parts, float eps) {
  double s = 0.;
  for (int i = threadIdx.x & 63; i < parts; i += 64) s += part[i];
  s = wave_sum(s);
  const double d = sqrt(s) + (double)eps;
  if (!(s < __builtin_inf())) return OrthFactor{1.f, __builtin_nanf("")};
  const double f = d > 0. ? (double)kUp / d : 0.;
  const float power = f > 0x1p100 ? 0x1p40f : f < 0x1p-100 ? 0x1p-40f : 1.f;
  return OrthFactor{power, (float)(f / (double)power)};
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
  return row * ld + (col >> 5) * kLine + (col & 31) * 2;
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
// edges.  rows x cols: the padded sizes (multiples of 32), G's orientation.  Bound by its bytes: 4 read and 8 written an
// element, 4096 x 14336 146 - 149 us, 4.7 TB/s.
constexpr int kPrepThreads = 256, kPrepTile = 64;
template <typename TIn>
__global__ __launch_bounds__(kPrepThreads) void orth_prepare_kernel(OrthArgs a, const double* part, int parts, uint8_t* own,
                                                                    int64_t own_stride, uint8_t* other, int64_t other_stride,
                                                                    int64_t rows, int64_t cols) {
  __shared__ float tile[kPrepTile][kPrepTile + 1];
  __shared__ OrthFactor factor;
  const int64_t e = blockIdx.z;
  if (threadIdx.x < 64) {
    const OrthFactor f = orth_factor(part + e * parts, parts, a.eps);
    if (threadIdx.x == 0) factor = f;
  }
  const TIn* G = (const TIn*)a.G + e * a.g_stride;
  const int64_t r0 = (int64_t)blockIdx.y * kPrepTile, c0 = (int64_t)blockIdx.x * kPrepTile;
  constexpr int kPer = kPrepTile / 8, kPasses = kPrepTile * kPer / kPrepThreads;       // threads of a row, rows of a thread
  const int q0 = threadIdx.x / kPer, p0 = threadIdx.x % kPer * 8;
  Raw8<TIn> g[kPasses];
#pragma unroll
  for (int x = 0; x < kPasses; ++x) {
    const int64_t r = r0 + q0 + x * (kPrepThreads / kPer);
    g[x] = mr_load8<TIn, false>(G + (r < a.N ? r : 0) * a.ld + c0 + p0, r < a.N ? a.K - c0 - p0 : 0, a.K);
  }
#pragma unroll
  for (int x = 0; x < kPasses; ++x) {
    const int64_t r = r0 + q0 + x * (kPrepThreads / kPer);
    mr_tail<false>(g[x], r < a.N ? a.K - c0 - p0 : 0, a.K);
    const Raw8<float> v = mr_float8(g[x]);
#pragma unroll
    for (int y = 0; y < 8; ++y) tile[q0 + x * (kPrepThreads / kPer)][p0 + y] = v.w[y];
  }
  __syncthreads();
  const OrthFactor f = factor;
  own += e * own_stride;
  other += e * other_stride;
  for (int i = threadIdx.x; i < kPrepTile * kPrepTile / 8; i += kPrepThreads) {
    const int q = i / (kPrepTile / 8), p = i % (kPrepTile / 8) * 8;
    float v[8], w[8];
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      v[x] = f(tile[q][p + x]);
      w[x] = f(tile[p + x][q]);
    }
    if (r0 + q < rows && c0 + p < cols) store_planes(own + plane_off(r0 + q, c0 + p, cols * kElBytes), v);
    if (c0 + q < cols && r0 + p < rows) store_planes(other + plane_off(c0 + q, r0 + p, rows * kElBytes), w);
  }
}

// -------------------------------------------------------------- products ----
// Tiles of BM x BN, WM x WN waves of (32 MI) x (32 NI) each, operands staged through LDS by buffer-load DMA in a ring
// of NS steps of one line of every row, the eight 16-byte chunks of a line at permuted places (chunk q of row r at
// q ^ ((r >> 1) & 7): a quarter-wave's reads hit 16 bank groups).  A line has kParts parts of 16 elements.
// v_mfma_f32_32x32x16_f16: lane l holds row or column l % 32, elements 8 (l / 32) .. + 7 of 16; result register r is
// row (r / 4) 8 + (l / 32) 4 + r % 4, column l % 32.
// Bound by the matrix cores and power.  B X of 4096 x 14336 in tiles of 256: 1.10 - 1.15 ms, 1.3 PFLOP/s counting the three
// products.  64 x 1408 x 2048 in tiles of 128: 1445 - 1500 us, 1.04 - 1.08.
constexpr int kParts = kLineEl / 16, kPlanes = 2, kProducts = 3;
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
struct OrthFrag { v8h a[kPlanes][T::MI], b[kPlanes][T::NI]; };

// The fragments of part h (16 elements) of a stage.
template <typename T>
__device__ __forceinline__ void orth_frag(const uint8_t* st, int h, OrthFrag<T>& f) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wm = wave / T::WN, wn = wave % T::WN;
  const int r31 = lane & 31, c = h * 2 + (lane >> 5);
#pragma unroll
  for (int i = 0; i < T::MI; ++i) {
    const int r = (wm * T::MI + i) * 32 + r31;
#pragma unroll
    for (int l = 0; l < kPlanes; ++l) f.a[l][i] = *reinterpret_cast<const v8h*>(st + r * kLine + (chunk_place(r, c + 4 * l) << 4));
  }
#pragma unroll
  for (int j = 0; j < T::NI; ++j) {
    const int r = (wn * T::NI + j) * 32 + r31;
#pragma unroll
    for (int l = 0; l < kPlanes; ++l)
      f.b[l][j] = *reinterpret_cast<const v8h*>(st + T::OffB + r * kLine + (chunk_place(r, c + 4 * l) << 4));
  }
}

template <typename T>
__device__ __forceinline__ void orth_mfma(const OrthFrag<T>& f, v16f (&acc)[T::MI][T::NI]) {
#pragma unroll
  for (int l = kProducts - 1; l >= 0; --l)               // l h', h l', h h'
#pragma unroll
    for (int i = 0; i < T::MI; ++i)
#pragma unroll
      for (int j = 0; j < T::NI; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(f.a[l == 2][i], f.b[l == 1][j], acc[i][j], 0, 0, 0);
}

// Part h of step kt on stage S, its fragments in f: its products cover the reads of part h + 1.
template <typename T, int S, int H>
__device__ __forceinline__ void orth_parts(OrthFrag<T>& f, v16f (&acc)[T::MI][T::NI]) {
  if constexpr (H + 1 < kParts) {
    constexpr int kReads = kPlanes * (T::MI + T::NI), kMfmas = kProducts * T::MI * T::NI;
    OrthFrag<T> n;
    orth_frag<T>(ring<T, S>(), H + 1, n);
    orth_mfma<T>(f, acc);
#pragma unroll
    for (int x = 0; x < kMfmas; ++x) {
      __builtin_amdgcn_sched_group_barrier(kSgDsRead, (kReads + kMfmas - 1) / kMfmas, 0);
      __builtin_amdgcn_sched_group_barrier(kSgMfma, 1, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
    f = n;
    orth_parts<T, S, H + 1>(f, acc);
  }
}

// Step kt on stage S = kt % NS, the fragments of its first part in f.  Before the last part's products every read of the
// stage has arrived; the barrier there makes step kt + 1 visible and retires stage S, which takes step kt + NS.
template <typename T, int S>
__device__ __forceinline__ void orth_step(const OrthSrc<T>& src, int kt, OrthFrag<T>& f, v16f (&acc)[T::MI][T::NI]) {
  constexpr int kReads = kPlanes * (T::MI + T::NI), kMfmas = kProducts * T::MI * T::NI;
  orth_parts<T, S, 0>(f, acc);
  S3R_WAIT_VM(T::Loads * (T::NS - 2));
  S3R_WAIT_LGKM0();
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_sched_barrier(0);
  OrthFrag<T> n;
  orth_load<T>(src, ring<T, S>(), kt + T::NS);
  orth_frag<T>(ring<T, (S + 1) % T::NS>(), 0, n);
  orth_mfma<T>(f, acc);
#pragma unroll
  for (int x = 0; x < kMfmas; ++x) {
    __builtin_amdgcn_sched_group_barrier(kSgMfma, 1, 0);
    __builtin_amdgcn_sched_group_barrier(kSgDsRead, (kReads + kMfmas - 1) / kMfmas, 0);
    __builtin_amdgcn_sched_group_barrier(kSgVmem, (T::Loads + kMfmas - 1) / kMfmas, 0);
  }
  __builtin_amdgcn_sched_barrier(0);
  f = n;
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
// This does rows 32 i .. of every wave.
template <typename T, OrthEpi EPI>
__device__ __forceinline__ void orth_store_rows(const OrthGemm& p, const OrthTile& t, int i, const v16f (&acc)[T::NI]) {
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
  const int64_t row0 = (int64_t)t.tm * T::BM + (wm * T::MI + i) * 32;
#pragma unroll
  for (int j = 0; j < T::NI; ++j)
#pragma unroll
    for (int r = 0; r < 16; ++r)
      buf[((r >> 2) * 8 + (lane >> 5) * 4 + (r & 3)) * T::EpiLd + j * 32 + (lane & 31)] = acc[j][r] * kDown;
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
      v8h h[kPlanes];
#pragma unroll
      for (int l = 0; l < kPlanes; ++l) h[l] = *reinterpret_cast<const v8h*>(at + l * (kLine / 2));
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        v[x] = p.c * v[x] + p.b * ((float)h[0][x] + (float)h[1][x]);
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

template <typename T, OrthEpi EPI>
__device__ __forceinline__ void orth_store(const OrthGemm& p, const OrthTile& t, const v16f (&acc)[T::MI][T::NI]) {
#pragma unroll
  for (int i = 0; i < T::MI; ++i) orth_store_rows<T, EPI>(p, t, i, acc[i]);
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
  const bool whole = (int)blockIdx.x < p.full;
  int w = whole ? blockIdx.x : blockIdx.x - p.full;
  const int n = whole ? p.full : p.workers;
  if (n % 8 == 0) w = (w % 8) * (n / 8) + w / 8;                // a contiguous range of tiles per XCD
  // from the first of the whole tiles' steps, or the shared ones'
  int64_t s = whole ? (int64_t)w * p.steps : first_step(p, w);
  const int64_t s1 = whole ? s + p.steps : first_step(p, w + 1);
  for (int slot = 0; s < s1;) {
    const int tile = (int)(s / p.steps), k0 = (int)(s - (int64_t)tile * p.steps);
    const int k1 = (int)min((int64_t)p.steps, k0 + (s1 - s));
    const OrthTile t = orth_tile<EPI>(p, whole ? tile : p.full + tile);
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
    s += k1 - k0;
    if (s >= s1) return;
    S3R_WAIT_VM(0);
    __syncthreads();                   // the ring is free again, and the next loads are counted from none
  }
}

// Tile blockIdx.x of the shared ones, rows 32 blockIdx.y .. of every wave (a workgroup for a whole tile of 256 took twice
// as long, few of them adding up in a row what many had left).  136 tiles of 256, 256 workers: 35 - 41 us.
template <typename T, OrthEpi EPI>
__global__ __launch_bounds__(T::Threads, T::WavesPerSimd) void orth_join_kernel(OrthGemm p) {
  const int tile = blockIdx.x, i = blockIdx.y;
  const int64_t s0 = (int64_t)tile * p.steps, s1 = s0 + p.steps, all = (int64_t)p.rest * p.steps;
  int w = (int)(s0 * p.workers / all);
  while (first_step(p, w + 1) <= s0) ++w;
  while (first_step(p, w) > s0) --w;
  if (first_step(p, w + 1) >= s1) return;              // one worker had all of it
  v16f acc[T::NI];
#pragma unroll
  for (int j = 0; j < T::NI; ++j)
#pragma unroll
    for (int r = 0; r < 16; ++r) acc[j][r] = 0.f;
  constexpr int kBatch = 8 / T::NI;
  while (first_step(p, w) < s1) {
    v4f v[kBatch][T::NI * 4];
    bool some[kBatch];
#pragma unroll
    for (int q = 0; q < kBatch; ++q, ++w) {              // every load before the first sum
      // a worker's second part follows a tile's end; its first one is the tile that its range begins in
      const int64_t b = first_step(p, w);
      some[q] = b < s1 && b != first_step(p, w + 1);
      if (!some[q]) continue;
      const int slot = b < s0 && b % p.steps != 0 ? 1 : 0;
      const v4f* part = reinterpret_cast<const v4f*>(p.partial) + (int64_t)(2 * w + slot) * (T::BM * T::BN / 4) +
                        (int64_t)i * T::NI * 4 * T::Threads + threadIdx.x;
#pragma unroll
      for (int x = 0; x < T::NI * 4; ++x) v[q][x] = part[x * T::Threads];
    }
#pragma unroll
    for (int q = 0; q < kBatch; ++q)
      if (some[q])
#pragma unroll
        for (int x = 0; x < T::NI * 4; ++x)
#pragma unroll
          for (int y = 0; y < 4; ++y) acc[x / 4][4 * (x % 4) + y] += v[q][x][y];
  }
  orth_store_rows<T, EPI>(p, orth_tile<EPI>(p, p.full + tile), i, acc);
}

// Small matrices: 32 x 32 results a workgroup, whose eight waves deal the contraction's steps of 32 elements among them and
// join their sums in LDS.  Fragments go straight from the caches to the matrix cores, kBatch steps of a wave at a time, so
// a product of a few hundred elements is one round of loads.  Bound by latency: 256 x 512 4.2 - 5.8 us a product.
constexpr int kFewThreads = 512, kFewWaves = kFewThreads / 64, kFewLd = 36;

template <OrthEpi EPI>
__global__ __launch_bounds__(kFewThreads) void orth_few_kernel(OrthGemm p) {
  __shared__ float part[kFewWaves][32 * kFewLd];
  constexpr int kBatch = 2;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const OrthTile t = orth_tile<EPI>(p, blockIdx.x);
  const int r31 = lane & 31, half = (lane >> 5) * 16;
  const uint8_t* A = p.A + t.e * p.a_stride + ((int64_t)t.tm * 32 + r31) * p.lda + half;
  const uint8_t* B = p.B + t.e * p.b_stride + ((int64_t)t.tn * 32 + r31) * p.ldb + half;
  v16f acc;
#pragma unroll
  for (int r = 0; r < 16; ++r) acc[r] = 0.f;
  for (int k0 = wave; k0 < p.steps; k0 += kFewWaves * kBatch) {
    v8h a[kBatch][2][kPlanes], b[kBatch][2][kPlanes];
#pragma unroll
    for (int q = 0; q < kBatch; ++q) {
      const int k = k0 + q * kFewWaves;
      if (k < p.steps) {                               // the same in the whole wave
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int l = 0; l < kPlanes; ++l) {
            a[q][h][l] = *reinterpret_cast<const v8h*>(A + (int64_t)k * kLine + h * 32 + l * 64);
            b[q][h][l] = *reinterpret_cast<const v8h*>(B + (int64_t)k * kLine + h * 32 + l * 64);
          }
      }
    }
#pragma unroll
    for (int q = 0; q < kBatch; ++q) {
      if (k0 + q * kFewWaves >= p.steps) break;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int l = kProducts - 1; l >= 0; --l)
          acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(a[q][h][l == 2], b[q][h][l == 1], acc, 0, 0, 0);
    }
  }
#pragma unroll
  for (int r = 0; r < 16; ++r) part[wave][((r >> 2) * 8 + (lane >> 5) * 4 + (r & 3)) * kFewLd + r31] = acc[r];
  __syncthreads();
  // 8 results a thread, 128 threads; where they are written transposed as well, 128 others do that
  const bool turned = threadIdx.x >= 128;
  if (threadIdx.x >= 256) return;
  if (turned && !(EPI == kEpiBoth || (symmetric(EPI) && t.tm != t.tn))) return;
  const int at = threadIdx.x & 127, major = at >> 2, minor = (at & 3) * 8;
  float v[8];
#pragma unroll
  for (int x = 0; x < 8; ++x) {
    const int i = turned ? (minor + x) * kFewLd + major : major * kFewLd + minor + x;
    v[x] = part[0][i];
#pragma unroll
    for (int w = 1; w < kFewWaves; ++w) v[x] += part[w][i];
    v[x] *= kDown;
  }
  const int64_t row = (int64_t)t.tm * 32 + (turned ? minor : major), col = (int64_t)t.tn * 32 + (turned ? major : minor);
  if constexpr (EPI == kEpiPoly) {
    // transposed: the addend's other triangle, which its product wrote as a copy of this one
    const uint8_t* add = p.addend + t.e * p.d_stride + (turned ? plane_off(col, row, p.ld_direct) : plane_off(row, col, p.ld_direct));
    v8h h[kPlanes];
#pragma unroll
    for (int l = 0; l < kPlanes; ++l) h[l] = *reinterpret_cast<const v8h*>(add + l * (kLine / 2));
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      v[x] = p.c * v[x] + p.b * ((float)h[0][x] + (float)h[1][x]);
      if (!turned && row == col + x) v[x] += p.a * kUp;
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
  } else if (turned) {
    store_planes(p.turned + t.e * p.t_stride + plane_off(col, row, p.ld_turned), v);
  } else {
    store_planes(p.direct + t.e * p.d_stride + plane_off(row, col, p.ld_direct), v);
  }
}

// -------------------------------------------------------------- launches ----
// Tiles by their side, in two forms: with a deep ring, one workgroup a CU, for products that have no more tiles than that (a
// step then takes the loads' latency over the ring's depth), and with several workgroups a CU.
template <int Side, bool Deep> struct OrthPick;
template <bool Deep> struct OrthPick<32, Deep> { static constexpr int BM = 32, Threads = kFewThreads, PerCu = 1; };
template <bool Deep> struct OrthPick<256, Deep> : OrthGeo<4, 2, 2, 4, 2, 2> { static constexpr int PerCu = 1; };
template <> struct OrthPick<128, false> : OrthGeo<2, 2, 2, 2, 2, 2> { static constexpr int PerCu = 2; };
template <> struct OrthPick<128, true> : OrthGeo<2, 2, 2, 2, 4, 1> { static constexpr int PerCu = 1; };
template <> struct OrthPick<64, false> : OrthGeo<1, 1, 2, 2, 3, 3> { static constexpr int PerCu = 3; };
template <> struct OrthPick<64, true> : OrthGeo<1, 1, 2, 2, 4, 1> { static constexpr int PerCu = 1; };
constexpr int kCus = 256, kMostSlots = 3 * kCus;
// Steps of a tile that sharing the last tiles has to save to be worth a launch and the way through memory.
constexpr int share_gain(int side) { return side == 256 ? 16 : side == 128 ? 16 : 40; }
// Steps of a worker, at least, since a tile's join adds its workers' sums in turn.  us for five steps with these and with 4: 64 x 8192
// 120 and 175 (the join of the one tile 6.5 and 22), 12 x 52 x 2723 158 and 176, 32 x 700 x 1400 1990 and 2056; others within 2 %.
constexpr int share_least(int side) { return side == 64 ? 16 : 8; }

// The tiles' sides, of the symmetric products and of B X.  us for five steps of fp32 results:
//   sides            32    64   128        sides            64   128   128 and 256    256
//   256 x 512       104   110   193        2048 x 2048     834   823
//   512 x 512       135   143   246        4 x 2048 x 2048      2242   2136          2363
//   768 x 768       263   172   303        4096 x 4096    5690  3955   3793          3867
//   64 x 8192       353   120   296        2 x 3000 x 5000      5169   4777          4885
//   16 x 200 x 300  176   118   188        2048 x 8192          2104   2085          1888
//   3 x 1283 x 701  587   290   400        4096 x 14336   15900 10801  10362         10153
// and of the symmetric products' 128 and 256 (B X in 256): 4096 x 5120 4706 4794, 4096 x 6144 5348 5432, 4096 x 8192 6557 6520,
// 2560 x 7168 2721 2643, 2 x 2048 x 6144 3226 3000, 2048 x 8192 2119 1943, 2048 x 10240 2666 2430.
// So the smallest tiles are for matrices that do not fill the GPU with them and whose sums are short, and a larger tile for
// those that give every CU one of it and that it pads no more than 1.4 times as far (12 x 52 x 2723, twice as far: 158 us in
// tiles of 64, 247 of 128), the largest where it pads little; of the symmetric products' triangle only with long sums, which
// the workgroups share.
struct OrthSides { int symmetric, update; };
OrthSides tile_sides(const OrthArgs& a) {
  const int64_t m = std::min(a.N, a.K), n = std::max(a.N, a.K);
  auto padded = [](int64_t x, int64_t side) { return (x + side - 1) / side * side; };
  auto tiles = [&](int64_t side) { return a.E * (padded(m, side) / side) * (padded(n, side) / side); };
  if (tiles(32) <= kCus && n <= 1024) return {32, 32};
  auto area = [&](int64_t side) { return (double)padded(m, side) * padded(n, side); };
  if (tiles(128) < kCus || area(128) > 1.4 * area(64)) return {64, 64};
  const bool most = tiles(256) >= kCus && area(256) <= 1.05 * area(128);
  return {most && n >= 8000 ? 256 : 128, most ? 256 : 128};
}

struct OrthLayout {
  OrthSides sides;
  int parts;
  int64_t m, n, mp, np;
  size_t part, x, xt[2], A, B, partial, total;
};
OrthLayout orth_layout(const OrthArgs& a) {
  OrthLayout l{};
  l.sides = tile_sides(a);
  const int side = l.sides.symmetric, update = l.sides.update;
  // workgroups for the norm: enough for the GPU, of four runs at least (every workgroup that writes the planes adds them up)
  const int64_t runs = a.N * ((a.K + kNormRun - 1) / kNormRun);
  l.parts = (int)std::max<int64_t>(1, std::min<int64_t>({kNormMost, (2048 + a.E - 1) / a.E, runs / 4}));
  l.m = std::min(a.N, a.K);
  l.n = std::max(a.N, a.K);
  // (the symmetric products leave what B's sides are padded with past their own tiles as it is: it reaches only padding)
  l.mp = (l.m + update - 1) / update * update;
  l.np = (l.n + update - 1) / update * update;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += align_up(bytes, 256);
    return here;
  };
  const size_t xs = (size_t)a.E * l.mp * l.np * kElBytes, as = (size_t)a.E * l.mp * l.mp * kElBytes;
  l.part = take((size_t)a.E * l.parts * 8);
  l.x = take(xs);
  l.xt[0] = take(xs);
  l.xt[1] = take(xs);
  l.A = take(as);
  l.B = take(as);
  // two tiles of every worker's sums, of the larger of both sides' (256 x 256 x 256 CUs against 128 x 128 x 512)
  if (side > 32) l.partial = take((size_t)(update == 256 ? kCus * 256 * 256 : kMostSlots * side * side) * 2 * 4);
  l.total = at;
  return l;
}

template <typename T, OrthEpi EPI>
hipError_t run_orth_tiles(OrthGemm p, int64_t tiles, hipStream_t st) {
  constexpr int kSlots = kCus * T::PerCu;
  if (tiles >= (int64_t)1 << 31 || (tiles + kSlots) * T::Threads >= (int64_t)1 << 32) return hipErrorInvalidConfiguration;
  if constexpr (T::BM == 32) {
    hipLaunchKernelGGL((orth_few_kernel<EPI>), dim3((unsigned)tiles), dim3(T::Threads), 0, st, p);
  } else {
    const int rest = (int)(tiles % kSlots);
    const int64_t workers = std::min<int64_t>(kSlots, (int64_t)rest * p.steps / share_least(T::BM));
    const bool share = workers > rest && (double)p.steps * (1.0 - (double)rest / workers) >= share_gain(T::BM);
    p.rest = share ? rest : 0;
    p.workers = share ? (int)workers : 0;
    p.full = (int)tiles - p.rest;
    hipLaunchKernelGGL((orth_gemm_kernel<T, EPI>), dim3((unsigned)(p.full + p.workers)), dim3(T::Threads), 0, st, p);
    if (share) hipLaunchKernelGGL((orth_join_kernel<T, EPI>), dim3((unsigned)p.rest, T::MI), dim3(T::Threads), 0, st, p);
  }
  return hipGetLastError();
}

template <int Side, OrthEpi EPI>
hipError_t run_orth_gemm(OrthGemm p, int64_t E, hipStream_t st) {
  p.per_matrix = symmetric(EPI) ? p.tiles_n * (p.tiles_n + 1) / 2 : p.tiles_m * p.tiles_n;
  const int64_t tiles = E * p.per_matrix;
  if constexpr (Side == 64 || Side == 128)
    if (tiles <= kCus) return run_orth_tiles<OrthPick<Side, true>, EPI>(p, tiles, st);
  return run_orth_tiles<OrthPick<Side, false>, EPI>(p, tiles, st);
}

template <int Side, int Update>
hipError_t run_orth_step(const OrthArgs& a, const OrthLayout& l, int s, hipStream_t st) {
  char* ws = (char*)a.ws;
  uint8_t* x = (uint8_t*)ws + l.x;
  uint8_t *A = (uint8_t*)ws + l.A, *B = (uint8_t*)ws + l.B;
  const uint8_t* xt = (uint8_t*)ws + l.xt[s & 1];
  const int64_t ld_x = l.np * kElBytes, ld_t = l.mp * kElBytes, xs = l.mp * ld_x, as = l.mp * ld_t;
  const int tm = (int)(l.mp / Update), tn = (int)(l.np / Update);
  const int along_n = (int)((l.n + kLineEl - 1) / kLineEl), along_m = (int)((l.m + kLineEl - 1) / kLineEl);      // lines
  OrthGemm p{};
  p.partial = (float*)(ws + l.partial);
  p.a = a.a; p.b = a.b; p.c = a.c;
  p.A = p.B = x; p.lda = p.ldb = ld_x; p.a_stride = p.b_stride = xs;
  p.tiles_m = p.tiles_n = (int)((l.m + Side - 1) / Side); p.steps = along_n;
  p.direct = p.turned = A; p.ld_direct = p.ld_turned = ld_t; p.d_stride = p.t_stride = as;
  hipError_t err = run_orth_gemm<Side, kEpiGram>(p, a.E, st);
  if (err != hipSuccess) return err;
  p.A = p.B = A; p.lda = p.ldb = ld_t; p.a_stride = p.b_stride = as;
  p.steps = along_m;
  p.addend = A;
  p.direct = p.turned = B;
  if ((err = run_orth_gemm<Side, kEpiPoly>(p, a.E, st)) != hipSuccess) return err;
  const bool last = s + 1 == a.steps, wide = a.N <= a.K;
  const uint8_t* first = last && wide ? B : xt;             // the tiles' rows: m's or n's
  p.A = first; p.a_stride = first == xt ? xs : as;
  p.B = first == xt ? B : xt; p.b_stride = first == xt ? as : xs;
  p.lda = p.ldb = ld_t;
  p.tiles_m = first == xt ? tn : tm; p.tiles_n = first == xt ? tm : tn;
  if (!last) {
    p.direct = (uint8_t*)ws + l.xt[~s & 1]; p.ld_direct = ld_t; p.d_stride = xs;
    p.turned = x; p.ld_turned = ld_x; p.t_stride = xs;
    return run_orth_gemm<Update, kEpiBoth>(p, a.E, st);
  }
  p.out = a.out; p.ld_out = a.ld_out; p.out_stride = a.out_stride; p.rows = a.N; p.cols = a.K;
  p.scale = a.scale; p.keep = a.keep;
  return a.out_dt == S3R_BF16 ? run_orth_gemm<Update, kEpiOutBf16>(p, a.E, st) : run_orth_gemm<Update, kEpiOutF32>(p, a.E, st);
}

template <int Side, int Update = Side>
hipError_t run_orth_steps(const OrthArgs& a, const OrthLayout& l, hipStream_t st) {
  hipError_t err = hipSuccess;
  for (int s = 0; s < a.steps && err == hipSuccess; ++s) err = run_orth_step<Side, Update>(a, l, s, st);
  return err;
}

template <typename TIn>
hipError_t run_orth_prepare(const OrthArgs& a, const OrthLayout& l, hipStream_t st) {
  char* ws = (char*)a.ws;
  double* part = (double*)(ws + l.part);
  hipLaunchKernelGGL((orth_norm_kernel<TIn>), dim3((unsigned)l.parts, (unsigned)a.E), dim3(kNormThreads), 0, st, a, part, l.parts);
  const bool wide = a.N <= a.K;
  const int64_t rows = wide ? l.mp : l.np, cols = wide ? l.np : l.mp, xs = l.mp * l.np * kElBytes;
  uint8_t *x = (uint8_t*)ws + l.x, *xt = (uint8_t*)ws + l.xt[0];
  hipLaunchKernelGGL((orth_prepare_kernel<TIn>),
                     dim3((unsigned)((cols + kPrepTile - 1) / kPrepTile), (unsigned)((rows + kPrepTile - 1) / kPrepTile), (unsigned)a.E),
                     dim3(kPrepThreads), 0, st, a, part, l.parts, wide ? x : xt, xs, wide ? xt : x, xs, rows, cols);
  return hipGetLastError();
}
}  // namespace

size_t orth_workspace(const OrthArgs& a) { return a.E * a.N * a.K == 0 ? 0 : orth_layout(a).total; }

hipError_t launch_orthogonalize(const OrthArgs& a, hipStream_t st) {
  if (a.E == 0 || a.N == 0 || a.K == 0) return hipSuccess;
  const OrthLayout l = orth_layout(a);
  const hipError_t e = a.g_dtype == S3R_BF16 ? run_orth_prepare<uint16_t>(a, l, st) : run_orth_prepare<float>(a, l, st);
  if (e != hipSuccess) return e;
  if (l.sides.symmetric == 256) return run_orth_steps<256>(a, l, st);
  if (l.sides.update == 256) return run_orth_steps<128, 256>(a, l, st);
  if (l.sides.symmetric == 128) return run_orth_steps<128>(a, l, st);
  return l.sides.symmetric == 64 ? run_orth_steps<64>(a, l, st) : run_orth_steps<32>(a, l, st);
}

}  // namespace s3r
