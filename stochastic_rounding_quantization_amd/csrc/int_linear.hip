// Forward products on INT8 operands: rows rounded to INT8 with one step a row (RTNE, as the backward's forward
// operands), and y = diag(s_a) A B^T diag(s_b) + bias, dense or over expert-sorted rows with one B per group, on
// the INT8 matrix cores.  Codes are row-major, K (the contraction) along the row: the layout that the backward's
// products take, so one set of codes serves both.  Sums are integers, so every variant gives the same bits.
#include <type_traits>

#include "group_tiles.h"
#include "int8_step.h"
#include "rows8.h"
#include "tile_ring.h"

namespace s3r {
namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v16i __attribute__((ext_vector_type(16)));

// ------------------------------------------------------------------ rows ----
// Threads threads take a row of up to 8 * Threads * Pieces elements, which stay in registers between the maximum and
// the codes; longer rows (Long) are read again for the codes.  Codes are written up to the next multiple of 16
// columns (zeros past K).  With `up` the element is silu(A) * up in fp32, not rounded in between.
// Bound by bytes without `up` (8192 x 4096 bf16 16.6 - 17.3 us, 5.8 - 6.1 TB/s with the last-level cache's help; 64 experts' 32768
// gathered rows of 2048 31.7), by vector instructions with it: 36 an element, 8192 x 14336 142 - 150 us, 3.9 - 4.1 TB/s.
constexpr int kIrBlock = 256;

template <typename TIn, bool UP, bool Words>
struct I8Source {
  const TIn *A, *U;
  int64_t K;
  bool some;
  __device__ __forceinline__ I8Source(const I8RowsArgs& a, int64_t g, int64_t src) {
    some = src >= 0;
    const int64_t at = g * a.a_stride + (some ? src : 0) * a.ld;
    A = (const TIn*)a.A + at;
    U = UP ? (const TIn*)a.up + at : nullptr;
    K = a.K;
  }
  __device__ __forceinline__ int64_t left(int64_t c) const { return some ? K - c : 0; }
};

// The codes of 8 elements, two words.
__device__ __forceinline__ uint2 i8_codes(const Raw8<float>& v, const Step& s) {
  uint32_t y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)       // 1.5 * 2^23: the sum holds the integer nearest to x, ties to even, in its low byte
    y[i] = __float_as_uint(fminf(fmaxf(v.w[i] * s.inv, -127.f), 127.f) + 12582912.f);
  uint2 w;
  w.x = __builtin_amdgcn_perm(y[1], y[0], 0x0C0C0400u) | __builtin_amdgcn_perm(y[3], y[2], 0x04000C0Cu);
  w.y = __builtin_amdgcn_perm(y[5], y[4], 0x0C0C0400u) | __builtin_amdgcn_perm(y[7], y[6], 0x04000C0Cu);
  return s.flag ? make_uint2(0u, 0u) : w;
}

template <typename TRaw>
__device__ __forceinline__ Raw8<float> i8_swiglu(const TRaw& v, const TRaw& u) {
  const Raw8<float> x = mr_float8(v), y = mr_float8(u);
  Raw8<float> d, s;
  bool slow = false;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    d.w[i] = 1.f + glue_exp32(-x.w[i]);
    s.w[i] = glue_recip(d.w[i]);
    slow |= glue_slow_recip(d.w[i]);
  }
  if (__builtin_amdgcn_ballot_w64(slow) != 0) {          // the rare reciprocal below 2^-126: one branch for the wave
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (glue_slow_recip(d.w[i])) s.w[i] = __fdiv_rn(1.f, d.w[i]);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) s.w[i] = (x.w[i] * s.w[i]) * y.w[i];       // 0 * 0 past the end
  return s;
}

// Elements c, c + stride, ... (Pieces of them, 8 each) of a row.
template <typename TIn, bool UP, bool Words, int Pieces>
struct I8Pieces {
  std::conditional_t<UP, Raw8<float>, Raw8<TIn>> v[Pieces];
  Raw8<TIn> a[Pieces], u[UP ? Pieces : 1];
  __device__ __forceinline__ void load(const I8Source<TIn, UP, Words>& s, int64_t c, int stride) {
    ask(s, c, stride);
    take(s, c, stride);
  }
  __device__ __forceinline__ void ask(const I8Source<TIn, UP, Words>& s, int64_t c, int stride) {
#pragma unroll
    for (int q = 0; q < Pieces; ++q) {           // every load before the first conversion
      const int64_t at = c + (int64_t)q * stride;
      a[q] = mr_load8<TIn, Words>(s.A + at, s.left(at), s.K);
      if constexpr (UP) u[q] = mr_load8<TIn, Words>(s.U + at, s.left(at), s.K);
    }
  }
  __device__ __forceinline__ void take(const I8Source<TIn, UP, Words>& s, int64_t c, int stride) {
#pragma unroll
    for (int q = 0; q < Pieces; ++q) {
      const int64_t n = s.left(c + (int64_t)q * stride);
      mr_tail<Words>(a[q], n, s.K);
      if constexpr (UP) {
        mr_tail<Words>(u[q], n, s.K);
        v[q] = i8_swiglu(a[q], u[q]);
        __builtin_amdgcn_sched_barrier(0);         // one piece's registers at a time
      } else {
        v[q] = a[q];
      }
    }
  }
  __device__ __forceinline__ uint32_t amax() const {
    uint32_t m = 0;
#pragma unroll
    for (int q = 0; q < Pieces; ++q) m = max(m, mr_amax(v[q]));
    return m;
  }
  template <typename TStore>
  __device__ __forceinline__ void codes(const Step& s, int64_t c, int stride, TStore store) const {
#pragma unroll
    for (int q = 0; q < Pieces; ++q) store(c + (int64_t)q * stride, i8_codes(mr_float8(v[q]), s));
  }
};

constexpr int ir_block(int threads) { return threads > kIrBlock ? threads : kIrBlock; }
template <typename TIn, bool UP, bool Words, int Threads, int Pieces, bool Long>
__global__ __launch_bounds__(ir_block(Threads)) void i8_rows_kernel(I8RowsArgs a) {
  constexpr int kRows = ir_block(Threads) / Threads, kWaves = Threads / 64;
  __shared__ uint32_t red[ir_block(Threads) / 64];
  const int sub = threadIdx.x % Threads, mine = threadIdx.x / Threads;
  const int64_t r = wide_block() * kRows + mine;
  const int64_t g = blockIdx.z;
  if (kRows == 1 ? r >= a.R : wide_block() * kRows >= a.R) return;       // the same for the whole workgroup
  const I8Source<TIn, UP, Words> s(a, g, mr_source(a, r));
  constexpr int kStride = Threads * 8;
  constexpr int64_t kSpan = (int64_t)kStride * Pieces;
  I8Pieces<TIn, UP, Words, Pieces> p;
  p.load(s, sub * 8, kStride);
  uint32_t m = p.amax();
  if constexpr (Long)
    for (int64_t c = kSpan; c < a.K; c += kSpan) {
      I8Pieces<TIn, UP, Words, Pieces> more;
      more.load(s, c + sub * 8, kStride);
      m = max(m, more.amax());
    }
  m = wave_max_u32(m);
  if constexpr (kWaves > 1) {
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWaves; ++w) m = max(m, red[w]);
  }
  if (r >= a.R) return;
  const Step st = make_step(m);
  if (sub == 0) {
    a.delta[g * a.d_stride + r] = st.delta;
    if (st.flag && a.flags) atomicOr(a.flags, st.flag);
  }
  int8_t* out = a.codes + g * a.c_stride + r * a.ld_c;
  auto store = [&](int64_t c, uint2 w) {
    if (c < a.K_out) *reinterpret_cast<uint2*>(out + c) = w;
  };
  p.codes(st, sub * 8, kStride, store);
  if constexpr (Long)
    for (int64_t c = kSpan; c < a.K_out; c += kSpan) {
      I8Pieces<TIn, UP, Words, Pieces> more;
      more.load(s, c + sub * 8, kStride);
      more.codes(st, c + sub * 8, kStride, store);
    }
}

// -------------------------------------------------------------- products ----
struct I8ProdK {
  const int8_t* A; int64_t lda; const float* sa;
  const int8_t* B; int64_t ldb; const float* sb; const float* bias;
  int64_t b_stride;
  const int64_t* offsets; int64_t G;          // G = 0: dense
  int64_t M, N, K; int tiles_n;
  void* out; int64_t ld_out;
  uint32_t* flags;
};

__device__ __forceinline__ void store_out(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_out(uint16_t* p, float v) {
  *reinterpret_cast<__bf16*>(p) = (__bf16)v;
}
// One result: the sum in fp32, times the product of the steps, one rounding each.
__device__ __forceinline__ float i8_result(int acc, float sa, float sb, float bias) {
  return (sa * sb) * (float)acc + bias;
}

// A buffer of `rows` rows of K codes (whole 16-byte words of the last one); reads past it give zeros.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_rsrc(const int8_t* p, int64_t rows, int64_t ld, int64_t K) {
  const int64_t bytes = rows <= 0 ? 0 : (rows - 1) * ld + (K + 15) / 16 * 16;
  return __builtin_amdgcn_make_buffer_rsrc((void*)p, (short)0, (int)(uint32_t)bytes, kRsrcWord3);
}
// Which of the 16 bytes at column c of a row lie before K, as masks of 4 words.
__device__ __forceinline__ v4i tail_mask(int64_t c, int64_t K) {
  v4i m;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t n = K - c - 4 * i;
    m[i] = n >= 4 ? -1 : n <= 0 ? 0 : (int)((1u << (8 * (int)n)) - 1u);
  }
  return m;
}

// The rows [m0, m1) of tile mt and its weight, or nothing to do.
struct I8Tile { int64_t m0, m1; int e; bool some; };
__device__ __forceinline__ I8Tile i8_tile(const I8ProdK& p, int mt, int tile) {
  const int64_t m0 = (int64_t)mt * tile;
  if (!p.G) return I8Tile{m0, min(p.M, m0 + tile), 0, m0 < p.M};
  GroupRound first;
  bool bad;
  const int total = group_total(p.offsets, p.G, p.M, tile, first, bad);
  if (bad) {
    if (blockIdx.x == 0 && threadIdx.x == 0 && p.flags) atomicOr(p.flags, S3R_FLAG_BAD_GROUPS);
    return I8Tile{0, 0, 0, false};
  }
  if (mt >= total) return I8Tile{0, 0, 0, false};
  const GroupTile h = group_tile(p.offsets, p.G, p.M, tile, first, mt);
  return I8Tile{h.r0, min(h.r1, h.r0 + tile), __builtin_amdgcn_readfirstlane(h.e), true};
}

// Up to four rows: byte dot products.  A wave takes R weight rows, 1 KiB of each at a time (whole lines, 16 bytes a
// lane), against the rows' codes in LDS; `split` of the workgroup's waves share weight rows and deal the 1 KiB pieces of K
// among them.  (The matrix cores would want a weight row in 4 lanes and 16 lines a quarter-wave.)  Bound by the weights'
// bytes: 1 x 14336 x 4096 11.6 - 13.6 us, 4.3 - 5.1 TB/s with the launch; 32 rows of 64 experts of 2816 x 2048 25.4 - 26.0.
// With TIn the rows come unrounded: every workgroup rounds them while its weights are on the way, so there is no
// second launch and no codes go through memory.  TIn void: rows already in codes.  Loads arrive in the order that they were
// asked for, so the rows are asked for first, then kDepth pieces of the weights, always all of them, for the compiler to
// know how many stand between (1 x 4096 x 14336 behind silu(gate) * up: 13.2 us, with the weights first 19.5).
constexpr int kDotPiece = 1024;
// silu(gate) * up of a whole row is 36 instructions an element for every workgroup: wider ones share it among more waves,
// with half of the weights on the way, which is what memory moves meanwhile (and what the registers have room for).
constexpr int dot_waves(bool up) { return up ? 16 : 8; }
constexpr size_t kDotLdsMax = 60000;              // of the 64 KiB that a workgroup has without asking

template <typename TOut, typename TIn, bool UP, bool Words, int MT, int R, int kDepth>
__global__ __launch_bounds__(64 * dot_waves(UP)) void i8_dot_kernel(I8ProdK p, I8RowsArgs q, int split) {
  constexpr int kDotWaves = dot_waves(UP), kDotThreads = 64 * kDotWaves;
  constexpr bool kFused = !std::is_void<TIn>::value;
  __shared__ uint32_t red[kDotWaves];
  __shared__ int part[kDotWaves][R * MT];
  extern __shared__ __attribute__((aligned(16))) int8_t rows[];         // MT rows of kpad codes
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const unsigned block = (unsigned)wide_block();
  const int mt = block / p.tiles_n, nt = block - mt * p.tiles_n;
  const I8Tile t = i8_tile(p, mt, MT);
  if (!t.some) return;
  const int rows_n = (int)(t.m1 - t.m0);
  const int slice = wave % split, group = wave / split;
  const int64_t n0 = ((int64_t)nt * (kDotWaves / split) + group) * R;
  const int pieces = (int)((p.K + kDotPiece - 1) / kDotPiece), kpad = pieces * kDotPiece;
  const __amdgpu_buffer_rsrc_t rb =
      rows_rsrc(p.B + t.e * p.b_stride + (n0 < p.N ? n0 : 0) * p.ldb, min(p.N - n0, (int64_t)R), p.ldb, p.K);
  v4i w[kDepth][R];
  // Past the last piece every load reads zeros: their number is the same for all, and the compiler can count to the row's.
  const __amdgpu_buffer_rsrc_t none = __builtin_amdgcn_make_buffer_rsrc((void*)p.B, (short)0, 0, kRsrcWord3);
  auto load = [&](int d, int pc) {
    const __amdgpu_buffer_rsrc_t from = pc < pieces ? rb : none;
#pragma unroll
    for (int r = 0; r < R; ++r)
      w[d][r] = __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(from, (uint32_t)(pc * kDotPiece + lane * 16),
                                                                              (uint32_t)r * (uint32_t)p.ldb, 0));
  };
  auto load_all = [&]() {
#pragma unroll
    for (int d = 0; d < kDepth; ++d) load(d, slice + d * split);
  };
  float sa[MT];
  if constexpr (kFused) {
    constexpr int kPer = kDotThreads / MT, kStride = kPer * 8, kPieces = UP ? 2 : 4;
    const int mine = threadIdx.x / kPer, c0 = (threadIdx.x % kPer) * 8;
    const I8Source<TIn, UP, Words> s(q, 0, mine < rows_n ? mr_source(q, t.m0 + mine) : -1);
    I8Pieces<TIn, UP, Words, kPieces> v;
    v.ask(s, c0, kStride);
    __builtin_amdgcn_sched_barrier(0);
    load_all();                                    // after the row's: loads arrive in order, and the row is needed first
    __builtin_amdgcn_sched_barrier(0);
    v.take(s, c0, kStride);
    uint32_t m = v.amax();
    for (int64_t c = kPieces * kStride; c < p.K; c += kPieces * kStride) {
      I8Pieces<TIn, UP, Words, kPieces> more;
      more.load(s, c + c0, kStride);
      m = max(m, more.amax());
    }
    m = wave_max_u32(m);
    if (lane == 0) red[wave] = m;
    __syncthreads();
    uint32_t flag = 0;
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      uint32_t a = 0;
#pragma unroll
      for (int x = 0; x < kDotWaves / MT; ++x) a = max(a, red[i * (kDotWaves / MT) + x]);
      const Step st = make_step(a);
      sa[i] = st.delta;
      flag |= st.flag;
      if (i == mine) m = a;
    }
    if (flag && nt == 0 && threadIdx.x == 0 && p.flags) atomicOr(p.flags, flag);
    const Step st = make_step(m);
    auto store = [&](int64_t c, uint2 q8) {
      if (c < kpad) *reinterpret_cast<uint2*>(rows + mine * kpad + c) = q8;
    };
    v.codes(st, c0, kStride, store);
    for (int64_t c = kPieces * kStride; c < kpad; c += kPieces * kStride) {
      I8Pieces<TIn, UP, Words, kPieces> more;
      more.load(s, c + c0, kStride);
      more.codes(st, c + c0, kStride, store);
    }
  } else {
    load_all();
    for (int at = threadIdx.x * 16; at < MT * kpad; at += kDotThreads * 16) {
      const int i = at / kpad, c = at - i * kpad;
      v4i x = {0, 0, 0, 0};
      if (i < rows_n && c < p.K)
        x = *reinterpret_cast<const v4i*>(p.A + (t.m0 + i) * p.lda + c) & tail_mask(c, p.K);
      *reinterpret_cast<v4i*>(rows + at) = x;
    }
#pragma unroll
    for (int i = 0; i < MT; ++i) sa[i] = i < rows_n ? p.sa[t.m0 + i] : 0.f;
  }
  __syncthreads();
  int acc[R][MT];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int i = 0; i < MT; ++i) acc[r][i] = 0;
  for (int p0 = slice; p0 < pieces; p0 += kDepth * split) {
#pragma unroll
    for (int d = 0; d < kDepth; ++d) {
      const int pc = p0 + d * split;
      if (pc >= pieces) break;
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        const v4i x = *reinterpret_cast<const v4i*>(rows + i * kpad + pc * kDotPiece + lane * 16);
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int y = 0; y < 4; ++y) acc[r][i] = __builtin_amdgcn_sdot4(w[d][r][y], x[y], acc[r][i], false);
      }
      load(d, pc + kDepth * split);
    }
  }
  // lane r * MT + i gets the sum of (weight row r, row i)
  int sum = 0;
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      const int all = __builtin_amdgcn_readlane(wave_prefix(acc[r][i]), 63);
      sum = lane == r * MT + i ? all : sum;
    }
  if (split > 1) {
    if (lane < R * MT) part[wave][lane] = sum;
    __syncthreads();
    if (slice > 0) return;
    if (lane < R * MT)
      for (int x = 1; x < split; ++x) sum += part[wave + x][lane];
  }
  const int i = lane % MT;
  const int64_t n = n0 + lane / MT;
  if (lane >= R * MT || i >= rows_n || n >= p.N) return;
  float step = sa[0];
#pragma unroll
  for (int x = 1; x < MT; ++x) step = i == x ? sa[x] : step;
  const int64_t col = t.e * p.N + n;
  store_out((TOut*)p.out + (t.m0 + i) * p.ld_out + n, i8_result(sum, step, p.sb[col], p.bias ? p.bias[col] : 0.f));
}

// Few rows: 16 MI rows x 16 NJ columns per workgroup, whose waves deal K's units of 128 bytes among them and join
// their sums in LDS.  The weights' bytes are the bound, and how they are asked for: a load of 16 rows x 64 bytes (the matrix
// cores' operand) is 64 requests, one of 8 whole lines 16, and the rows' codes cost as much as the weights (24 x 4096 x
// 14336: 20.8 us straight into registers).  So every wave stages its units in LDS by buffer-load DMA, whole lines, in
// a ring of its own of NS units: no wave waits for another before the end (12.0 - 13.2 us, 4.5 - 4.9 TB/s).  Chunks of a line as in the
// tiles below.
// v_mfma_i32_16x16x64_i8: lane l holds row or column l % 16, bytes 16 (l / 16) .. + 15 of 64; the result's register r is
// row 4 (l / 16) + r, column l % 16.
__device__ __forceinline__ int chunk_pos8(int r, int q) { return q ^ ((r >> 1) & 7); }

template <int MI_, int NJ_, int Waves_, int NS_>
struct FewGeo {
  static constexpr int MI = MI_, NJ = NJ_, Waves = Waves_, NS = NS_, Threads = 64 * Waves;
  static constexpr int Loads = 2 * (MI + NJ);                             // 1 KiB pieces of a unit
  static constexpr int UnitBytes = Loads * 1024, StageBytes = Waves * UnitBytes;
};

template <typename T>
struct FewSrc {
  __amdgpu_buffer_rsrc_t a, b, z;
  uint32_t v[T::Loads];                       // this lane's byte offsets in unit 0
  int units;
};

// Unit u into this wave's part of stage st; past the last unit every load reads zeros, so the wait counts stay the same.
template <typename T>
__device__ __forceinline__ void few_load(const FewSrc<T>& s, uint8_t* st, int u) {
  const bool live = u < s.units;
  const __amdgpu_buffer_rsrc_t ra = live ? s.a : s.z, rb = live ? s.b : s.z;
#pragma unroll
  for (int q = 0; q < T::Loads; ++q) dma16(q < 2 * T::MI ? ra : rb, st + q * 1024, s.v[q], (uint32_t)u * 128u);
}

template <typename T, int S>
__device__ __forceinline__ void few_fill(const FewSrc<T>& s, int mine, int wave) {
  if constexpr (S < T::NS) {
    few_load<T>(s, ring<T, S>() + mine, wave + S * T::Waves);
    few_fill<T, S + 1>(s, mine, wave);
  }
}

// Units u, u + Waves, ... on the stages from S on.
template <typename T, int S>
__device__ __forceinline__ void few_units(const FewSrc<T>& s, int mine, int u, int64_t K, v4i (&acc)[T::MI][T::NJ]) {
  if constexpr (S < T::NS) {
    if (u >= s.units) return;
    const int lane = threadIdx.x & 63, r15 = lane & 15, kb = lane >> 4;
    uint8_t* st = ring<T, S>() + mine;
    S3R_WAIT_VM(T::Loads * (T::NS - 1));
    __builtin_amdgcn_sched_barrier(0);
    v4i x[2][T::MI], y[2][T::NJ];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int at = r15 * 128 + (chunk_pos8(r15, 4 * h + kb) << 4);
#pragma unroll
      for (int i = 0; i < T::MI; ++i) x[h][i] = *reinterpret_cast<const v4i*>(st + i * 2048 + at);
#pragma unroll
      for (int j = 0; j < T::NJ; ++j) y[h][j] = *reinterpret_cast<const v4i*>(st + (T::MI + j) * 2048 + at);
    }
    S3R_WAIT_LGKM0();
    __builtin_amdgcn_sched_barrier(0);
    few_load<T>(s, st, u + T::NS * T::Waves);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if ((u + 1) * 128 > K) {                 // the last unit of a K that fills none: the rows' codes past K count as 0
        const v4i m = tail_mask(u * 128 + h * 64 + kb * 16, K);
#pragma unroll
        for (int i = 0; i < T::MI; ++i) x[h][i] &= m;
      }
#pragma unroll
      for (int i = 0; i < T::MI; ++i)
#pragma unroll
        for (int j = 0; j < T::NJ; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(x[h][i], y[h][j], acc[i][j], 0, 0, 0);
    }
    few_units<T, S + 1>(s, mine, u + T::Waves, K, acc);
  }
}

template <typename TOut, typename T>
__global__ __launch_bounds__(T::Threads) void i8_few_rows_kernel(I8ProdK p) {
  // The wave's index in a scalar register: the loop over its units has to branch, since the matrix instructions run
  // whatever the execution mask says.
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const unsigned block = (unsigned)wide_block();
  const int mt = block / p.tiles_n, nt = block - mt * p.tiles_n;
  const I8Tile t = i8_tile(p, mt, 16 * T::MI);
  if (!t.some) return;
  const int64_t n0 = (int64_t)nt * (16 * T::NJ);
  FewSrc<T> s;
  s.units = (int)((p.K + 127) / 128);
  s.a = rows_rsrc(p.A + t.m0 * p.lda, t.m1 - t.m0, p.lda, p.K);
  s.b = rows_rsrc(p.B + t.e * p.b_stride + n0 * p.ldb, min(p.N - n0, (int64_t)(16 * T::NJ)), p.ldb, p.K);
  s.z = __builtin_amdgcn_make_buffer_rsrc((void*)p.A, (short)0, 0, kRsrcWord3);
#pragma unroll
  for (int q = 0; q < T::Loads; ++q) {
    const int r = (q < 2 * T::MI ? q : q - 2 * T::MI) * 8 + (lane >> 3);
    s.v[q] = (uint32_t)(r * (q < 2 * T::MI ? p.lda : p.ldb) + chunk_pos8(r & 15, lane & 7) * 16);
  }
  v4i acc[T::MI][T::NJ];
#pragma unroll
  for (int i = 0; i < T::MI; ++i)
#pragma unroll
    for (int j = 0; j < T::NJ; ++j) acc[i][j] = v4i{0, 0, 0, 0};
  const int mine = wave * T::UnitBytes;
  few_fill<T, 0>(s, mine, wave);
  for (int u = wave; u < s.units; u += T::NS * T::Waves) few_units<T, 0>(s, mine, u, p.K, acc);
  S3R_WAIT_VM(0);
  // the waves' sums over each other's: a wave's part of stage 0 is its own until here
  static_assert(T::UnitBytes >= T::MI * T::NJ * 1024, "a wave's sums fit its unit");
  int* part = reinterpret_cast<int*>(ring<T, 0>());
#pragma unroll
  for (int i = 0; i < T::MI; ++i)
#pragma unroll
    for (int j = 0; j < T::NJ; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r) part[(mine / 4) + ((i * T::NJ + j) * 4 + r) * 64 + lane] = acc[i][j][r];
  __syncthreads();
  // a register of the results (64 of them) a wave and turn
  TOut* out = (TOut*)p.out;
  for (int x = wave; x < T::MI * T::NJ * 4; x += T::Waves) {
    int v = 0;
#pragma unroll
    for (int w = 0; w < T::Waves; ++w) v += part[w * (T::UnitBytes / 4) + x * 64 + lane];
    const int i = x / (T::NJ * 4), j = x / 4 % T::NJ;
    const int64_t m = t.m0 + 16 * i + 4 * (lane >> 4) + x % 4, n = n0 + 16 * j + (lane & 15);
    if (m < t.m1 && n < p.N)
      store_out(out + m * p.ld_out + n, i8_result(v, p.sa[m], p.sb[t.e * p.N + n], p.bias ? p.bias[t.e * p.N + n] : 0.f));
  }
}

// Many rows: BM x BN tiles, WM x WN waves of (32 MI) x (32 NI) each, operands staged through LDS by buffer-load DMA in
// a ring of NS steps of 128 bytes of K.  A stage holds 128 bytes of each of the tile's rows (8 lanes of a load read a
// whole line), the eight 16-byte chunks of a row at permuted places (chunk q of row r at q ^ ((r >> 1) & 7), so a
// quarter-wave's reads hit 16 bank groups).  v_mfma_i32_32x32x32_i8: lane l holds row or column l % 32, bytes
// 16 (l / 32) .. + 15 of 32; result register r is row (r / 4) 8 + (l / 32) 4 + r % 4, column l % 32.
// Bound by power where the tiles are large: 8192 x 14336 x 4096 411 - 439 us, 2.2 - 2.3 POP/s (the whole call with operands of
// zeros 336 us against 418 - 430, in turn on one box, and 448 - 467 over longer runs), 8192 x 4096 x 14336 400 - 421.  64 experts' 32768 x 2816 x 2048 295 - 300 us, 1.3 POP/s:
// partial tiles, 16 steps of K and 185 MB of results.
template <int MI_, int NI_, int WM_, int WN_, int NS_, int WavesPerSimd_>
struct I8Geo {
  static constexpr int WavesPerSimd = WavesPerSimd_;
  static constexpr int MI = MI_, NI = NI_, WM = WM_, WN = WN_, NS = NS_;
  static constexpr int Waves = WM * WN, Threads = 64 * Waves;
  static constexpr int BM = 32 * MI * WM, BN = 32 * NI * WN;
  static constexpr int PA = BM / 8 / Waves, PB = BN / 8 / Waves;          // 1 KiB pieces per wave
  static constexpr int Loads = PA + PB;
  static constexpr int OffB = BM * 128;
  static constexpr int StageBytes = OffB + BN * 128;
  static constexpr int EpiLd = 32 * NI + 4;                               // words per row of the epilogue's staging
  static_assert(BM % (8 * Waves) == 0 && BN % (8 * Waves) == 0, "whole pieces per wave");
};

template <typename T>
struct I8TileSrc {
  __amdgpu_buffer_rsrc_t a, b, z;
  uint32_t va[T::PA], vb[T::PB];              // this lane's byte offsets in step 0
  int nk;
};

// Step kt into stage st; past the last step every load reads zeros, so the wait counts stay the same.
template <typename T>
__device__ __forceinline__ void i8_load(const I8TileSrc<T>& s, uint8_t* st, int kt) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const bool live = kt < s.nk;
  const __amdgpu_buffer_rsrc_t ra = live ? s.a : s.z, rb = live ? s.b : s.z;
  const uint32_t koff = (uint32_t)kt * 128u;
#pragma unroll
  for (int q = 0; q < T::PA; ++q) dma16(ra, st + (wave * T::PA + q) * 1024, s.va[q], koff);
#pragma unroll
  for (int q = 0; q < T::PB; ++q) dma16(rb, st + T::OffB + (wave * T::PB + q) * 1024, s.vb[q], koff);
}

template <typename T>
struct I8Frag { v4i a[T::MI], b[T::NI]; };

// The fragments of quarter h of a stage.
template <typename T>
__device__ __forceinline__ void i8_frag(const uint8_t* st, int h, I8Frag<T>& f) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wm = wave / T::WN, wn = wave % T::WN;
  const int r31 = lane & 31, c = h * 2 + (lane >> 5);
#pragma unroll
  for (int i = 0; i < T::MI; ++i) {
    const int r = (wm * T::MI + i) * 32 + r31;
    f.a[i] = *reinterpret_cast<const v4i*>(st + r * 128 + (chunk_pos8(r, c) << 4));
  }
#pragma unroll
  for (int j = 0; j < T::NI; ++j) {
    const int r = (wn * T::NI + j) * 32 + r31;
    f.b[j] = *reinterpret_cast<const v4i*>(st + T::OffB + r * 128 + (chunk_pos8(r, c) << 4));
  }
}

template <typename T>
__device__ __forceinline__ void i8_mfma(const I8Frag<T>& f, v16i (&acc)[T::MI][T::NI]) {
#pragma unroll
  for (int i = 0; i < T::MI; ++i)
#pragma unroll
    for (int j = 0; j < T::NI; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(f.a[i], f.b[j], acc[i][j], 0, 0, 0);
}

// Quarter h of step kt with the fragments of its first quarter in f: its products cover the reads of quarter h + 1.
template <typename T, int S, int H>
__device__ __forceinline__ void i8_quarter(I8Frag<T>& f, v16i (&acc)[T::MI][T::NI]) {
  I8Frag<T> n;
  i8_frag<T>(ring<T, S>(), H + 1, n);
  i8_mfma<T>(f, acc);
#pragma unroll
  for (int x = 0; x < T::MI * T::NI; ++x) {
    __builtin_amdgcn_sched_group_barrier(kSgDsRead, (T::MI + T::NI + T::MI * T::NI - 1) / (T::MI * T::NI), 0);
    __builtin_amdgcn_sched_group_barrier(kSgMfma, 1, 0);
  }
  __builtin_amdgcn_sched_barrier(0);
  f = n;
}

// Step kt on stage S = kt % NS, the fragments of its first quarter in f.  Before the last quarter's products every read
// of the stage has arrived; the barrier there makes step kt + 1 visible and retires stage S, which takes step kt + NS.
template <typename T, int S>
__device__ __forceinline__ void i8_step(const I8TileSrc<T>& src, int kt, I8Frag<T>& f, v16i (&acc)[T::MI][T::NI]) {
  i8_quarter<T, S, 0>(f, acc);
  i8_quarter<T, S, 1>(f, acc);
  i8_quarter<T, S, 2>(f, acc);
  S3R_WAIT_VM(T::Loads * (T::NS - 2));
  S3R_WAIT_LGKM0();
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_sched_barrier(0);
  I8Frag<T> n;
  i8_load<T>(src, ring<T, S>(), kt + T::NS);
  i8_frag<T>(ring<T, (S + 1) % T::NS>(), 0, n);
  i8_mfma<T>(f, acc);
#pragma unroll
  for (int x = 0; x < T::MI * T::NI; ++x) {
    __builtin_amdgcn_sched_group_barrier(kSgMfma, 1, 0);
    __builtin_amdgcn_sched_group_barrier(kSgDsRead, (T::MI + T::NI + T::MI * T::NI - 1) / (T::MI * T::NI), 0);
    __builtin_amdgcn_sched_group_barrier(kSgVmem, (T::Loads + T::MI * T::NI - 1) / (T::MI * T::NI), 0);
  }
  __builtin_amdgcn_sched_barrier(0);
  f = n;
}

// The first NS steps into the ring.
template <typename T, int S>
__device__ __forceinline__ void i8_fill(const I8TileSrc<T>& src) {
  if constexpr (S < T::NS) {
    i8_load<T>(src, ring<T, S>(), S);
    i8_fill<T, S + 1>(src);
  }
}

template <typename T, int S>
__device__ __forceinline__ void i8_steps(const I8TileSrc<T>& src, int kt, int full, I8Frag<T>& f, v16i (&acc)[T::MI][T::NI]) {
  if constexpr (S < T::NS) {
    if (kt + S < full) {
      i8_step<T, S>(src, kt + S, f, acc);
      i8_steps<T, S + 1>(src, kt, full, f, acc);
    }
  }
}

// The last step where K fills none: the rows' codes past K count as 0 (what lies there may be anything).
template <typename T, int S>
__device__ __forceinline__ void i8_last(int stage, int kt, int64_t K, I8Frag<T>& f, v16i (&acc)[T::MI][T::NI]) {
  if constexpr (S < T::NS) {
    if (stage == S) {
      const int c = (threadIdx.x & 63) >> 5;
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        if (h > 0) i8_frag<T>(ring<T, S>(), h, f);
        const v4i m = tail_mask((int64_t)kt * 128 + (h * 2 + c) * 16, K);
#pragma unroll
        for (int i = 0; i < T::MI; ++i) f.a[i] &= m;
        i8_mfma<T>(f, acc);
      }
    } else {
      i8_last<T, S + 1>(stage, kt, K, f, acc);
    }
  }
}

// The wave's results, 32 rows at a time through its own part of the (now free) ring, so that whole 16-byte words of
// consecutive columns are stored, past the last-level cache, at the elements' alignment.
typedef uint32_t i8_u4_a2 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t i8_u4_a4 __attribute__((ext_vector_type(4), aligned(4)));
template <typename T, typename TOut>
__device__ __forceinline__ void i8_store(const I8ProdK& p, const I8Tile& t, int64_t n0, const v16i (&acc)[T::MI][T::NI]) {
  constexpr int kBuf = 32 * T::EpiLd * 4;
  constexpr int kPer = T::StageBytes / kBuf;                  // waves' buffers in one stage
  static_assert(kPer > 0 && kPer * T::NS >= T::Waves, "the epilogue's staging fits the ring");
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wm = wave / T::WN, wn = wave % T::WN;
  uint8_t* stage = ring<T, 0>();
  if (wave / kPer == 1) stage = ring<T, 1 % T::NS>();
  if (wave / kPer == 2) stage = ring<T, 2 % T::NS>();
  int* buf = reinterpret_cast<int*>(stage + (wave % kPer) * kBuf);
  constexpr int W = 16 / (int)sizeof(TOut);                   // elements of a store
  constexpr int LR = 32 * T::NI / W;                          // lanes of a row
  const int lr = lane / LR, lc = (lane % LR) * W;
  const int64_t n = n0 + wn * (32 * T::NI) + lc;
  TOut* out = (TOut*)p.out;
  float sb[W], bias[W];
#pragma unroll
  for (int x = 0; x < W; ++x) {
    const bool in = n + x < p.N;
    sb[x] = in ? p.sb[t.e * p.N + n + x] : 0.f;
    bias[x] = in && p.bias ? p.bias[t.e * p.N + n + x] : 0.f;
  }
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
      const int64_t m = t.m0 + (wm * T::MI + i) * 32 + q + lr;
      if (m >= t.m1) continue;
      const float sa = p.sa[m];
      float v[W];
#pragma unroll
      for (int x = 0; x < W; x += 4) {
        const v4i c = *reinterpret_cast<const v4i*>(buf + (q + lr) * T::EpiLd + lc + x);
#pragma unroll
        for (int y = 0; y < 4; ++y) v[x + y] = i8_result(c[y], sa, sb[x + y], bias[x + y]);
      }
      TOut* o = out + m * p.ld_out + n;
      if (n + W <= p.N) {
        if constexpr (sizeof(TOut) == 2) {
          typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
          typedef float f2 __attribute__((ext_vector_type(2)));
          uint32_t w[4];
#pragma unroll
          for (int x = 0; x < 4; ++x)
            w[x] = __builtin_bit_cast(uint32_t, __builtin_convertvector((f2{v[2 * x], v[2 * x + 1]}), bf2));
          __builtin_nontemporal_store((v4u32{w[0], w[1], w[2], w[3]}), reinterpret_cast<i8_u4_a2*>(o));
        } else {
          __builtin_nontemporal_store((v4u32{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])}),
                                      reinterpret_cast<i8_u4_a4*>(o));
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
__global__ __launch_bounds__(T::Threads, T::WavesPerSimd) void i8_tile_kernel(I8ProdK p, int tiles_m) {
  // A contiguous range of tiles per XCD (workgroups go to the 8 XCDs in turn).  Grouped: of the tiles that the
  // groups have, not of the grid's bound on them, whose surplus would all be the last XCD's.
  int bid = (int)wide_block();
  GroupRound first;
  if (p.G) {
    bool bad;
    tiles_m = group_total(p.offsets, p.G, p.M, T::BM, first, bad);
    if (bad) {
      if (blockIdx.x == 0 && threadIdx.x == 0 && p.flags) atomicOr(p.flags, S3R_FLAG_BAD_GROUPS);
      return;
    }
    const int nblocks = tiles_m * p.tiles_n, per = (nblocks + 7) / 8;
    const int at = bid / 8;
    bid = (bid % 8) * per + at;
    if (at >= per || bid >= nblocks) return;
  } else {
    const int nblocks = tiles_m * p.tiles_n;
    if (bid >= nblocks) return;
    if (nblocks % 8 == 0) bid = (bid % 8) * (nblocks / 8) + bid / 8;
  }
  const int group = 8 * p.tiles_n;
  const int first_m = (bid / group) * 8;
  const int gsz = min(tiles_m - first_m, 8);
  const int tm = first_m + (bid % group) % gsz, tn = (bid % group) / gsz;
  I8Tile t{(int64_t)tm * T::BM, p.M, 0, true};
  const int64_t n0 = (int64_t)tn * T::BN;
  if (p.G) {
    const GroupTile h = group_tile(p.offsets, p.G, p.M, T::BM, first, tm);
    t = I8Tile{h.r0, h.r1, h.e, true};
  }
  // the tile's rows of both operands; rows past the group's end reach only results that are not stored
  I8TileSrc<T> src;
  src.nk = (int)((p.K + 127) / 128);
  src.a = rows_rsrc(p.A + t.m0 * p.lda, min(p.M - t.m0, (int64_t)T::BM), p.lda, p.K);
  src.b = rows_rsrc(p.B + t.e * p.b_stride + n0 * p.ldb, min(p.N - n0, (int64_t)T::BN), p.ldb, p.K);
  src.z = __builtin_amdgcn_make_buffer_rsrc((void*)p.A, (short)0, 0, kRsrcWord3);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
#pragma unroll
  for (int q = 0; q < T::PA; ++q) {
    const int r = (wave * T::PA + q) * 8 + (lane >> 3);
    src.va[q] = (uint32_t)(r * p.lda + chunk_pos8(r, lane & 7) * 16);
  }
#pragma unroll
  for (int q = 0; q < T::PB; ++q) {
    const int r = (wave * T::PB + q) * 8 + (lane >> 3);
    src.vb[q] = (uint32_t)(r * p.ldb + chunk_pos8(r, lane & 7) * 16);
  }
  v16i acc[T::MI][T::NI];
#pragma unroll
  for (int i = 0; i < T::MI; ++i)
#pragma unroll
    for (int j = 0; j < T::NI; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0;
  i8_fill<T, 0>(src);
  S3R_WAIT_VM(T::Loads * (T::NS - 1));
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_sched_barrier(0);
  I8Frag<T> f;
  i8_frag<T>(ring<T, 0>(), 0, f);
  const int full = (int)(p.K / 128);
  for (int kt = 0; kt < full; kt += T::NS) i8_steps<T, 0>(src, kt, full, f, acc);
  if (full < src.nk) i8_last<T, 0>(full % T::NS, full, p.K, f, acc);
  S3R_WAIT_VM(0);
  S3R_WAIT_LGKM0();
  __builtin_amdgcn_s_barrier();
  i8_store<T, TOut>(p, t, n0, acc);
}

// ----------------------------------------------------------- column sums ----
// A workgroup adds 64 rows of 1024 columns, four columns a thread; integer sums, so the order of its additions into
// memory does not change them.  32768 x 2048 in 64 groups 21.8 us, 8192 x 14336 33 us, 3.1 - 3.6 TB/s, of the codes and the additions;
// 8192 x 4096 19.8 us: 512 workgroups do not fill the GPU.  The clearing before it 1.5 - 4.8 us.
constexpr int kCsRows = 64;
__global__ __launch_bounds__(256) void i8_colsum_clear_kernel(const int64_t* offsets, int64_t G, int64_t R, int64_t K,
                                                              int32_t* sums, uint32_t* flags) {
  if (offsets) {
    GroupRound first;
    bool bad;
    group_total(offsets, G, R, 1, first, bad);
    if (bad) {
      if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0 && flags) atomicOr(flags, S3R_FLAG_BAD_GROUPS);
      return;
    }
  }
  const int64_t i = wide_block() * 256 + threadIdx.x;
  if (i < G * K) sums[i] = 0;
}

__global__ __launch_bounds__(256) void i8_colsum_kernel(const int64_t* offsets, int64_t G, int64_t R, int64_t K,
                                                        const int8_t* Q, int64_t ld, int32_t* sums) {
  const int64_t kblocks = (K + 1023) / 1024;
  const int64_t block = wide_block(), rb = block / kblocks, c = (block - rb * kblocks) * 1024 + threadIdx.x * 4;
  const int64_t r0 = rb * kCsRows, r1 = min(r0 + kCsRows, R);
  if (r0 >= R) return;
  int64_t e = 0;
  if (offsets) {
    GroupRound first;
    bool bad;
    group_total(offsets, G, R, 1, first, bad);
    if (bad) return;
    e = group_tile(offsets, G, R, 1, first, (int)r0).e;
  } else {
    e = r0 / (R / G);
  }
  const __amdgpu_buffer_rsrc_t rq = rows_rsrc(Q + r0 * ld, r1 - r0, ld, K);
  for (int64_t r = r0; r < r1; ++e) {
    const int64_t end = min(r1, offsets ? offsets[e + 1] : (e + 1) * (R / G));
    if (end <= r) continue;
    int s[4] = {0, 0, 0, 0};
#pragma unroll 8
    for (; r < end; ++r) {
      const uint32_t w = __builtin_amdgcn_raw_buffer_load_b32(rq, (uint32_t)((r - r0) * ld + c), 0, 0);
#pragma unroll
      for (int i = 0; i < 4; ++i) s[i] += (int)(w << (24 - 8 * i)) >> 24;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (c + i < K) atomicAdd(sums + e * K + c + i, s[i]);
  }
}

bool i8_words(const I8RowsArgs& a) {       // rows in whole 16-byte words
  const int esize = a.dtype == S3R_BF16 ? 2 : 4;
  return ((uintptr_t)a.A & 15u) == 0 && ((uintptr_t)a.up & 15u) == 0 && (a.ld * esize) % 16 == 0 &&
         (a.a_stride * esize) % 16 == 0 && a.K % 8 == 0;
}

template <typename TIn, bool UP, bool Words, int Threads, int Pieces, bool Long>
hipError_t run_i8_rows(const I8RowsArgs& a, hipStream_t st) {
  constexpr int kBlock = ir_block(Threads), kRows = kBlock / Threads;
  dim3 grid = wide_grid((a.R + kRows - 1) / kRows);
  grid.z = (unsigned)a.G;
  hipLaunchKernelGGL((i8_rows_kernel<TIn, UP, Words, Threads, Pieces, Long>), grid, dim3(kBlock), 0, st, a);
  return hipGetLastError();
}

// Rows from which a wave each is enough: 401 x 1999 fp32 and product 14.9 us with a workgroup each, 16.4 with a wave; 16384 x
// 2048 47.7 and 43.6.
constexpr int64_t kIrFill = 4096;
template <typename TIn, bool UP, bool Words>
hipError_t run_i8_rows(const I8RowsArgs& a, hipStream_t st) {
  if (a.K <= 512) return run_i8_rows<TIn, UP, Words, 64, 1, false>(a, st);
  if (a.K <= 2048)
    return a.R * a.G < kIrFill ? run_i8_rows<TIn, UP, Words, 256, 1, false>(a, st) : run_i8_rows<TIn, UP, Words, 64, 4, false>(a, st);
  if (a.K <= 4096) return run_i8_rows<TIn, UP, Words, 256, 2, false>(a, st);
  if (a.K <= 8192) return run_i8_rows<TIn, UP, Words, 512, 2, false>(a, st);
  if (a.K <= 16384) return run_i8_rows<TIn, UP, Words, 512, 4, false>(a, st);
  return run_i8_rows<TIn, UP, Words, 512, 4, true>(a, st);
}

template <typename TIn>
hipError_t run_i8_rows(const I8RowsArgs& a, hipStream_t st) {
  const bool words = i8_words(a);
  if (a.up) return words ? run_i8_rows<TIn, true, true>(a, st) : run_i8_rows<TIn, true, false>(a, st);
  return words ? run_i8_rows<TIn, false, true>(a, st) : run_i8_rows<TIn, false, false>(a, st);
}
}  // namespace

hipError_t launch_i8_rows(const I8RowsArgs& a, hipStream_t st) {
  if (a.R == 0 || a.G == 0) return hipSuccess;
  return a.dtype == S3R_BF16 ? run_i8_rows<uint16_t>(a, st) : run_i8_rows<float>(a, st);
}

hipError_t launch_i8_colsum(const int64_t* offsets, int64_t G, int64_t R, int64_t K, const int8_t* Q, int64_t ld,
                            int32_t* sums, uint32_t* flags, hipStream_t st) {
  if (G * K == 0) return launch_check_offsets(offsets, offsets ? G : 0, R, flags, st);
  hipLaunchKernelGGL(i8_colsum_clear_kernel, wide_grid((G * K + 255) / 256), dim3(256), 0, st, offsets, G, R, K, sums, flags);
  if (R > 0)
    hipLaunchKernelGGL(i8_colsum_kernel, wide_grid((R + kCsRows - 1) / kCsRows * ((K + 1023) / 1024)), dim3(256), 0, st,
                       offsets, G, R, K, Q, ld, sums);
  return hipGetLastError();
}

namespace {
// Few rows, in one round of workgroups where that can be: 16 columns each give every CU one up to kFewWide columns, past that
// 32 columns read the rows' codes half as often and take one round instead of two.  us with 32 and 16:
//   rows  K        N = 4096       5120         6144         8192         10240        14336
//   16    4096      6.8   6.2    7.3   9.3    8.4   9.8    9.9  10.8   15.1  14.8   18.6  21.6
//   64    4096      9.5   8.6    9.8  13.9   10.4  14.3   11.8  15.0   20.1  21.2   24.2  32.1
//   16    14336    19.2  14.5   20.1  24.1   20.9  25.7   23.5  27.0   38.5  37.4   42.5  49.8
//   64    14336    29.7  24.0   30.4  42.8   31.2  43.4   32.9  45.4   58.2  64.7   61.3  85.9
constexpr int64_t kFewWide = 16 * 256;
using Few16 = FewGeo<1, 1, 8, 4>;
using Few16Wide = FewGeo<1, 2, 4, 4>;
using Few32 = FewGeo<2, 1, 8, 3>;
using Few32Wide = FewGeo<2, 2, 4, 4>;
using Few64 = FewGeo<4, 1, 8, 2>;
using Few64Wide = FewGeo<4, 2, 4, 3>;
using FewGrouped = FewGeo<1, 2, 4, 3>;           // two workgroups a CU
using I8Tile256 = I8Geo<4, 2, 2, 4, 2, 2>;        // 256 x 256, 8 waves
using I8Tile256x128 = I8Geo<2, 2, 4, 2, 3, 2>;    // 8 waves
using I8Tile128 = I8Geo<2, 2, 2, 2, 2, 2>;        // 4 waves, two workgroups per CU
using I8Tile128x64 = I8Geo<2, 1, 2, 2, 3, 2>;
using I8Tile64 = I8Geo<1, 1, 2, 2, 3, 2>;

// The largest tile that still gives this many workgroups (three quarters of the CUs).
constexpr int64_t kFillTiles = 192;

I8ProdK product_params(const I8ProductArgs& a) {
  I8ProdK p{};
  p.A = a.A; p.lda = a.lda; p.sa = a.sa; p.B = a.B; p.ldb = a.ldb; p.sb = a.sb; p.bias = a.bias; p.b_stride = a.b_stride;
  p.offsets = a.offsets; p.G = a.G; p.M = a.M; p.N = a.N; p.K = a.K;
  p.out = a.out; p.ld_out = a.ld_out; p.flags = a.flags;
  return p;
}

// rows per weight, on average (only the device knows the groups' own)
int64_t mean_rows(const I8ProductArgs& a) { return a.G ? (a.M + a.G - 1) / a.G : a.M; }
// Row tiles of a product; grouped: of every group, at most one partial tile each.
int64_t row_tiles(const I8ProductArgs& a, int tile) {
  return a.G ? a.M / tile + std::min(a.G, a.M) : (a.M + tile - 1) / tile;
}
// Workgroups of a grid: numbers of 31 bits, and what a second dimension adds to whole rows of it.
constexpr int64_t kMostBlocks = ((int64_t)1 << 31) - ((int64_t)1 << kWideShift);

template <typename T, typename TOut>
hipError_t run_i8_tiles(const I8ProductArgs& a, I8ProdK p, hipStream_t st) {
  const int64_t mt = row_tiles(a, T::BM);
  p.tiles_n = (int)((a.N + T::BN - 1) / T::BN);
  const int64_t blocks = a.G ? (mt * p.tiles_n + 7) / 8 * 8 : mt * p.tiles_n;
  if (blocks > kMostBlocks) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL((i8_tile_kernel<T, TOut>), wide_grid(blocks), dim3(T::Threads), 0, st, p, (int)mt);
  return hipGetLastError();
}
template <typename T>
hipError_t run_i8_tiles(const I8ProductArgs& a, hipStream_t st) {
  const I8ProdK p = product_params(a);
  return a.out_dt == S3R_BF16 ? run_i8_tiles<T, uint16_t>(a, p, st) : run_i8_tiles<T, float>(a, p, st);
}

template <typename T>
hipError_t run_i8_few(const I8ProductArgs& a, hipStream_t st) {
  I8ProdK p = product_params(a);
  const int64_t mt = row_tiles(a, 16 * T::MI);
  p.tiles_n = (int)((a.N + 16 * T::NJ - 1) / (16 * T::NJ));
  if (mt * p.tiles_n > kMostBlocks) return hipErrorInvalidConfiguration;
  const dim3 grid = wide_grid(mt * p.tiles_n), block(T::Threads);
  if (a.out_dt == S3R_BF16) hipLaunchKernelGGL((i8_few_rows_kernel<uint16_t, T>), grid, block, 0, st, p);
  else hipLaunchKernelGGL((i8_few_rows_kernel<float, T>), grid, block, 0, st, p);
  return hipGetLastError();
}

constexpr int64_t kDotFill = 128, kDotRoom = 16 * 256;            // waves of these kernels that a GPU holds
size_t dot_lds(int rows, int64_t K) { return (size_t)rows * (size_t)((K + kDotPiece - 1) / kDotPiece) * kDotPiece; }

template <typename TIn, bool UP, bool Words, int MT, int R, int Depth>
hipError_t run_i8_dot(const I8ProductArgs& a, const I8RowsArgs& q, hipStream_t st) {
  constexpr int kDotWaves = dot_waves(UP), kDotThreads = 64 * kDotWaves;
  I8ProdK p = product_params(a);
  const int64_t mt = row_tiles(a, MT), groups = (a.N + R - 1) / R;
  // waves that share weight rows: as many as the GPU has room for at once, where K has pieces for them
  int split = 1;
  while (split < kDotWaves && mt * groups * split * 2 <= kDotRoom && split * kDotPiece < a.K) split *= 2;
  p.tiles_n = (int)((groups * split + kDotWaves - 1) / kDotWaves);
  if (mt * p.tiles_n > kMostBlocks) return hipErrorInvalidConfiguration;
  const dim3 grid = wide_grid(mt * p.tiles_n), block(kDotThreads);
  const size_t lds = dot_lds(MT, a.K);
  if (a.out_dt == S3R_BF16)
    hipLaunchKernelGGL((i8_dot_kernel<uint16_t, TIn, UP, Words, MT, R, Depth>), grid, block, lds, st, p, q, split);
  else
    hipLaunchKernelGGL((i8_dot_kernel<float, TIn, UP, Words, MT, R, Depth>), grid, block, lds, st, p, q, split);
  return hipGetLastError();
}
template <typename TIn, bool UP, bool Words, int MT>
hipError_t run_i8_dot(const I8ProductArgs& a, const I8RowsArgs& q, hipStream_t st) {
  // one weight row a wave where four would leave half of the CUs without a workgroup
  const int64_t pieces = (a.K + kDotPiece - 1) / kDotPiece;
  const int64_t waves = row_tiles(a, MT) * ((a.N + 3) / 4) * std::max<int64_t>(1, pieces / 4);
  const bool few = waves < kDotFill * dot_waves(UP);
  // over experts, more workgroups on a CU hide the offsets' and the index' round trips better than deeper loads
  if (a.G) return few ? run_i8_dot<TIn, UP, Words, MT, 1, 8>(a, q, st) : run_i8_dot<TIn, UP, Words, MT, 4, 2>(a, q, st);
  if constexpr (UP) return few ? run_i8_dot<TIn, UP, Words, MT, 1, 8>(a, q, st) : run_i8_dot<TIn, UP, Words, MT, 4, 2>(a, q, st);
  else return few ? run_i8_dot<TIn, UP, Words, MT, 1, 16>(a, q, st) : run_i8_dot<TIn, UP, Words, MT, 4, 4>(a, q, st);
}
// Rows of a workgroup: 1, 2 or 4.
int dot_rows(const I8ProductArgs& a) { return a.M <= 2 ? (int)a.M : 4; }
template <typename TIn, bool UP, bool Words>
hipError_t run_i8_dot(const I8ProductArgs& a, const I8RowsArgs& q, hipStream_t st) {
  const int rows = dot_rows(a);
  if (rows == 1) return run_i8_dot<TIn, UP, Words, 1>(a, q, st);
  return rows == 2 ? run_i8_dot<TIn, UP, Words, 2>(a, q, st) : run_i8_dot<TIn, UP, Words, 4>(a, q, st);
}
template <typename TIn>
hipError_t run_i8_dot(const I8ProductArgs& a, const I8RowsArgs& q, hipStream_t st) {
  const bool words = i8_words(q);
  if (q.up) return words ? run_i8_dot<TIn, true, true>(a, q, st) : run_i8_dot<TIn, true, false>(a, q, st);
  return words ? run_i8_dot<TIn, false, true>(a, q, st) : run_i8_dot<TIn, false, false>(a, q, st);
}

// Rows (per weight, on average) that the byte dot products take.
constexpr int64_t kDotRows = 4, kDotGrouped = 1;
bool takes_dots(const I8ProductArgs& a) {
  return mean_rows(a) <= (a.G ? kDotGrouped : kDotRows) && dot_lds(dot_rows(a), a.K) <= kDotLdsMax;
}
// Rows per weight, on average, up to which a grouped product takes the few-rows kernel.  64 experts, N = 2816, K = 2048: 2 rows
// 55 us against 60 in 128 x 128 tiles, 8 rows 83 against 88, 16 rows 108 against 94.5.
constexpr int64_t kFewGrouped = 12;
// From here on the larger tile: 64 experts, 512 rows each, N = 2816, K = 2048 357 us against 379 in 128 x 128 tiles, 8 experts,
// 1024 rows each, N = K = 4096 216 against 222; 32 experts, 256 rows each, N = 2048, K = 1408 70.4 both.
constexpr int64_t kTallGrouped = 384;

template <typename T>
int64_t tile_count(const I8ProductArgs& a) { return ((a.M + T::BM - 1) / T::BM) * ((a.N + T::BN - 1) / T::BN); }
}  // namespace

hipError_t launch_i8_product(const I8ProductArgs& a, hipStream_t st) {
  if (a.M == 0 || a.N == 0) return launch_check_offsets(a.offsets, a.G, a.M, a.flags, st);
  if (takes_dots(a)) return run_i8_dot<void, false, true>(a, I8RowsArgs{}, st);
  if (a.G) {
    const int64_t rows = mean_rows(a);
    if (rows <= kFewGrouped) return run_i8_few<FewGrouped>(a, st);
    return rows < kTallGrouped ? run_i8_tiles<I8Tile128>(a, st) : run_i8_tiles<I8Tile256>(a, st);
  }
  const bool wide = a.N > kFewWide;
  if (a.M <= 16) return wide ? run_i8_few<Few16Wide>(a, st) : run_i8_few<Few16>(a, st);
  if (a.M <= 32) return wide ? run_i8_few<Few32Wide>(a, st) : run_i8_few<Few32>(a, st);
  if (a.M <= 64) return wide ? run_i8_few<Few64Wide>(a, st) : run_i8_few<Few64>(a, st);
  // Sums that the few-rows kernel spreads over a workgroup's waves, where a tile would walk K alone: with no more than one
  // workgroup a CU (two where K is long).  us of it and of tiles: 128 x 1000 x 8000 15.6 and 28.1, 192 x 1283 x 1999 11.3 and
  // 14.6, 256 x 1283 x 1999 (324 workgroups) 15.2 and 14.0, 96 x 4096 x 14336 (512) 33.1 and 42.8, x 4096 17.5 and 16.8.
  const int64_t few = (a.M + 63) / 64 * ((a.N + 15) / 16);
  if (few <= 256 || (few <= 512 && a.K >= 8192)) return run_i8_few<Few64>(a, st);
  if (tile_count<I8Tile256>(a) >= kFillTiles) return run_i8_tiles<I8Tile256>(a, st);
  if (tile_count<I8Tile256x128>(a) >= kFillTiles) return run_i8_tiles<I8Tile256x128>(a, st);
  if (tile_count<I8Tile128>(a) >= kFillTiles) return run_i8_tiles<I8Tile128>(a, st);
  if (tile_count<I8Tile128x64>(a) >= kFillTiles) return run_i8_tiles<I8Tile128x64>(a, st);
  return run_i8_tiles<I8Tile64>(a, st);
}

// Rows and product; `rows` writes the codes that `prod` reads, unless the product rounds them itself.
hipError_t launch_i8_linear(const I8RowsArgs& rows, const I8ProductArgs& prod, hipStream_t st) {
  if (prod.M == 0 || prod.N == 0) return launch_check_offsets(prod.offsets, prod.G, prod.M, prod.flags, st);
  if (takes_dots(prod)) return rows.dtype == S3R_BF16 ? run_i8_dot<uint16_t>(prod, rows, st) : run_i8_dot<float>(prod, rows, st);
  // (Rounding rows that an index repeats once and gathering their codes in the product's loads: 371 us against 358 for 64
  // experts' 32768 rows of 16384.)
  const hipError_t e = launch_i8_rows(rows, st);
  return e != hipSuccess ? e : launch_i8_product(prod, st);
}

}  // namespace s3r
