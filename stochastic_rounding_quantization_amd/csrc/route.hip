// Routing of tokens to experts: scores, groups, top-k and weights of a router's
// logits, the expert-sorted order of the (token, choice) slots that the grouped
// calls take, and the gradient of the weights.
//
// With logits l [T x E]: scores s = softmax(l) over the row or 1 / (1 + exp(-l)),
// keys s + bias (the bias steers the load, it enters no weight), the experts in
// equal groups of which the best `keep` stay, and the top_k largest keys of the
// rest, ties to the lower index.  Weights w_j = c s_j, or c s_j / sum_i s_i.
//
// A decision between two keys has to be the one of exact arithmetic as far as
// 64 bits tell it: without a bias and without sums of keys the logits themselves
// are compared (the scores are monotone in them), otherwise fp64 keys.
#include <type_traits>

#include "s3r_internal.h"

namespace s3r {
namespace {

constexpr int kRtThreads = 1024;
constexpr int kRtMaxChunks = 256;    // token chunks of one call: the place kernel reads every chunk's counts

template <typename TIn>
__device__ __forceinline__ float rt_load(const TIn* p) {
  if constexpr (sizeof(TIn) == 2) return bf16_to_f32(*reinterpret_cast<const uint16_t*>(p));
  else return *reinterpret_cast<const float*>(p);
}

// V consecutive logits from p, of which the first n exist (the others: NaN, "no expert").
template <typename TIn, int V>
__device__ __forceinline__ void rt_load_row(const TIn* p, int n, bool vec, float (&x)[V]) {
  if (vec && n >= V) {
    if constexpr (sizeof(TIn) == 2) {
#pragma unroll
      for (int q = 0; q < V / 8; ++q) {
        const uint4 w = reinterpret_cast<const uint4*>(p)[q];
        const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[8 * q + 2 * i] = __uint_as_float(ww[i] << 16);
          x[8 * q + 2 * i + 1] = __uint_as_float(ww[i] & 0xFFFF0000u);
        }
      }
    } else {
#pragma unroll
      for (int q = 0; q < V / 4; ++q) {
        const float4 w = reinterpret_cast<const float4*>(p)[q];
        x[4 * q] = w.x; x[4 * q + 1] = w.y; x[4 * q + 2] = w.z; x[4 * q + 3] = w.w;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = i < n ? rt_load(p + i) : __builtin_nanf("");
  }
}

// Reductions over the L lanes of a token.
template <int L, typename T>
__device__ __forceinline__ T rt_sum(T v) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}
template <int L, typename T>
__device__ __forceinline__ T rt_max(T v) {      // NaNs lose
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) {
    const T w = __shfl_xor(v, o, 64);
    if constexpr (sizeof(T) == 8) v = __builtin_fmax(v, w);
    else v = __builtin_fmaxf(v, w);
  }
  return v;
}
template <int L>
__device__ __forceinline__ int rt_min(int v) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) v = min(v, __shfl_xor(v, o, 64));
  return v;
}

template <typename T> __device__ __forceinline__ T rt_neg_inf();
template <> __device__ __forceinline__ float rt_neg_inf<float>() { return -__builtin_inff(); }
template <> __device__ __forceinline__ double rt_neg_inf<double>() { return -__builtin_inf(); }

struct RouteKernelArgs {
  const void* logits; int64_t ld; const float* bias;
  int32_t* ids; float* weights; int64_t* offsets; int32_t* slot_row; int32_t* row_slot;
  int64_t T;
  int E, K, groups, keep, group_top, sigmoid, renorm;
  float scale;
  int32_t* hist;             // [nchunk][E] slots of the chunk's tokens at each expert
  int nchunk; int64_t chunk; // tokens per chunk
  int vec;
};

// The slots [s0, s1) in order, each to row base[e] + (slots of e before it in the range); base is
// advanced.  Every thread of the block takes part.  A wave ranks its 64 slots by matching expert
// indices bit by bit with ballots, and the waves' counts are added in order, so the order is the
// slots' own and no atomic decides it.
__device__ void rt_place(const int32_t* ids, int64_t s0, int64_t s1, int E, int32_t* base,
                         uint16_t* wcnt, int32_t* __restrict__ slot_row, int32_t* __restrict__ row_slot) {
  const int nt = blockDim.x, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, nw = nt >> 6;
  int bits = 0;
  while ((1 << bits) < E) ++bits;
  for (int64_t t0 = s0; t0 < s1; t0 += nt) {
    for (int i = tid; i < nw * E; i += nt) wcnt[i] = 0;
    __syncthreads();
    const int64_t s = t0 + tid;
    const bool act = s < s1;
    const int e = act ? ids[s] : 0;
    uint64_t same = __builtin_amdgcn_ballot_w64(act);
    for (int b = 0; b < bits; ++b) {
      const uint64_t m = __builtin_amdgcn_ballot_w64((e >> b) & 1);
      same &= ((e >> b) & 1) ? m : ~m;
    }
    const int rank = __builtin_popcountll(same & ((1ull << lane) - 1));
    if (act && rank == 0) wcnt[wave * E + e] = (uint16_t)__builtin_popcountll(same);
    __syncthreads();
    int moved = 0;                       // at most one expert per thread: E <= nt
    if (tid < E) {
      for (int w = 0; w < nw; ++w) {
        const int c = wcnt[w * E + tid];
        wcnt[w * E + tid] = (uint16_t)moved;
        moved += c;
      }
    }
    __syncthreads();
    if (act) {
      const int row = base[e] + wcnt[wave * E + e] + rank;
      slot_row[s] = row;
      row_slot[row] = (int32_t)s;
    }
    __syncthreads();
    if (tid < E) base[tid] += moved;
  }
}

// Exclusive sums of v over the block's threads (v = 0 past E), in order; scratch: one int per wave.
__device__ int rt_scan(int v, int32_t* scratch) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int s = v;
  for (int o = 1; o < 64; o <<= 1) {
    const int a = __shfl_up(s, o, 64);
    if (lane >= o) s += a;
  }
  if (lane == 63) scratch[wave] = s;
  __syncthreads();
  int before = 0;
  for (int w = 0; w < wave; ++w) before += scratch[w];
  return before + s - v;
}

// LDS of both kernels: base [E] | scratch [16] | hist or partial sums [2048] | wave counts [16][E] (uint16)
__host__ __device__ inline size_t rt_lds_bytes(int E) {
  return (size_t)E * 4 + 64 + 2048 * 4 + align_up((size_t)16 * E * 2, 16);
}

// L lanes of a wave hold a token's row, V consecutive experts each (L V >= E, L >= top_k, L >= groups).
// The top_k keys are taken one after another: the largest of the token's lanes, then the lowest index
// that holds it; a taken key becomes NaN, which loses every comparison, as do the places past E.
template <typename TIn, int L, int V, bool KEY64>
__global__ __launch_bounds__(kRtThreads) void route_kernel(RouteKernelArgs a) {
  using Key = typename std::conditional<KEY64, double, float>::type;
  extern __shared__ __attribute__((aligned(16))) char rt_lds[];
  int32_t* base = reinterpret_cast<int32_t*>(rt_lds);
  int32_t* scratch = base + a.E;
  int32_t* hist = scratch + 16;
  uint16_t* wcnt = reinterpret_cast<uint16_t*>(hist + 2048);
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, nw = blockDim.x >> 6;
  const int sub = lane % L;
  for (int e = tid; e < a.E; e += blockDim.x) hist[e] = 0;
  __syncthreads();
  const int64_t c0 = (int64_t)blockIdx.x * a.chunk, c1 = min(a.T, c0 + a.chunk);
  const int e0 = sub * V;
  const int per = a.E / a.groups;
  constexpr int TW = 64 / L;
  const TIn* logits = reinterpret_cast<const TIn*>(a.logits);
  for (int64_t tb = c0 + wave * TW; tb < c1; tb += nw * TW) {
    const int64_t t = min(tb + lane / L, c1 - 1);       // lanes past the chunk repeat its last token, unwritten
    const bool act = tb + lane / L < c1;
    float x[V];
    rt_load_row<TIn, V>(logits + t * a.ld + e0, a.E - e0, a.vec != 0, x);
    bool odd = false;                                     // a NaN or +inf logit: the softmax is NaN
    float top = -__builtin_inff();
#pragma unroll
    for (int i = 0; i < V; ++i) {
      odd |= (e0 + i < a.E) && !(x[i] < __builtin_inff());
      top = __builtin_fmaxf(top, x[i]);
    }
    top = rt_max<L>(top);
    const bool row_odd = ((__builtin_amdgcn_ballot_w64(odd) >> (lane / L * L)) & (~0ull >> (64 - L))) != 0;
    const float shift = top == -__builtin_inff() ? 0.f : top;
    Key key[V];
    if constexpr (KEY64) {
      double z = 0.0;
      if (a.sigmoid) {
#pragma unroll
        for (int i = 0; i < V; ++i) key[i] = 1.0 / (1.0 + exp(-(double)x[i]));
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          key[i] = exp((double)x[i] - (double)shift);
          if (e0 + i < a.E) z += key[i];
        }
        z = rt_sum<L>(z);
#pragma unroll
        for (int i = 0; i < V; ++i) key[i] = key[i] / z;
      }
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (e0 + i < a.E && a.bias) key[i] += (double)a.bias[e0 + i];
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) key[i] = x[i];
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (e0 + i < a.E && !(x[i] > -__builtin_inff() && key[i] > rt_neg_inf<Key>())) key[i] = rt_neg_inf<Key>();
    if (a.groups > 1) {
      Key mine = rt_neg_inf<Key>();                       // lane g of the token: the score of group g
      for (int g = 0; g < a.groups; ++g) {
        Key m1 = (Key)__builtin_nan("");
#pragma unroll
        for (int i = 0; i < V; ++i)
          if ((e0 + i) / per == g) m1 = key[i] > m1 || m1 != m1 ? key[i] : m1;
        m1 = rt_max<L>(m1);
        if (a.group_top == 2) {
          int at = 1 << 30;
#pragma unroll
          for (int i = V - 1; i >= 0; --i)
            if ((e0 + i) / per == g && key[i] == m1) at = e0 + i;
          at = rt_min<L>(at);
          Key m2 = rt_neg_inf<Key>();
#pragma unroll
          for (int i = 0; i < V; ++i)
            if ((e0 + i) / per == g && e0 + i != at && key[i] > m2) m2 = key[i];
          m2 = rt_max<L>(m2);
          m1 = m1 + m2;
        }
        if (sub == g) mine = m1;
      }
      int rank = 0;
      for (int h = 0; h < a.groups; ++h) {
        const Key other = __shfl(mine, lane / L * L + h, 64);
        rank += (other > mine || (other == mine && h < sub)) ? 1 : 0;
      }
      const uint64_t kept = __builtin_amdgcn_ballot_w64(sub < a.groups && rank < a.keep) >> (lane / L * L);
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (e0 + i < a.E && !((kept >> ((e0 + i) / per)) & 1)) key[i] = rt_neg_inf<Key>();
    }
    int mine = 0;                                           // lane j of the token: choice j
    for (int j = 0; j < a.K; ++j) {
      Key m = key[0];
#pragma unroll
      for (int i = 1; i < V; ++i) {
        if constexpr (KEY64) m = __builtin_fmax(m, key[i]);
        else m = __builtin_fmaxf(m, key[i]);
      }
      m = rt_max<L>(m);
      int at = 1 << 30;
#pragma unroll
      for (int i = V - 1; i >= 0; --i) at = key[i] == m ? e0 + i : at;
      at = rt_min<L>(at);
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (e0 + i == at) key[i] = (Key)__builtin_nan("");
      if (sub == j) mine = at;
    }
    // weights: lane j < top_k of the token
    const bool live = sub < a.K;
    const float xj = live ? rt_load(logits + t * a.ld + mine) : 0.f;
    float w;
    if (a.sigmoid) {
      w = live ? 1.f / (1.f + expf(-xj)) : 0.f;
      if (a.renorm) {
        float sum = rt_sum<L>(w);
        if (sum < 1e-30f) {      // scores near or below the smallest normal: from their logarithms
          const float ls = live ? fminf(xj, 0.f) - log1pf(expf(-fabsf(xj))) : -__builtin_inff();
          const float m = rt_max<L>(ls);
          w = m == -__builtin_inff() ? 0.f : expf(ls - m);
          sum = rt_sum<L>(w);
        }
        w = sum == 0.f ? 0.f : w / sum;
      }
    } else if (a.renorm) {
      const float m = rt_max<L>(live ? xj : -__builtin_inff());
      w = live && m > -__builtin_inff() ? expf(xj - m) : 0.f;
      const float sum = rt_sum<L>(w);
      w = row_odd ? __builtin_nanf("") : sum == 0.f ? 0.f : w / sum;
    } else {
      float z = 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i) z += e0 + i < a.E ? expf(x[i] - shift) : 0.f;
      z = rt_sum<L>(z);
      w = row_odd ? __builtin_nanf("") : z == 0.f ? 0.f : expf(xj - shift) / z;
    }
    if (act && live) {
      a.ids[t * a.K + sub] = mine;
      a.weights[t * a.K + sub] = w * a.scale;
      atomicAdd(&hist[mine], 1);                            // whole numbers: any order gives the same
    }
  }
  __syncthreads();
  if (a.nchunk > 1) {
    for (int e = tid; e < a.E; e += blockDim.x) a.hist[(int64_t)blockIdx.x * a.E + e] = hist[e];
    return;
  }
  // one chunk: the order too, in this launch
  const int n = tid < a.E ? hist[tid] : 0;
  const int first = rt_scan(n, scratch);
  if (tid < a.E) { base[tid] = first; a.offsets[tid] = first; }
  if (tid == 0) a.offsets[a.E] = a.T * a.K;
  __threadfence_block();
  __syncthreads();
  rt_place(a.ids, 0, a.T * a.K, a.E, base, wcnt, a.slot_row, a.row_slot);
}

// The order of the slots: block b places chunk b's.  Every block adds up the chunks' counts (at most
// kRtMaxChunks x E words, from the caches): all of them for the experts' first rows, those before its
// own for its first row at each expert.
__global__ __launch_bounds__(kRtThreads) void route_place_kernel(RouteKernelArgs a) {
  extern __shared__ __attribute__((aligned(16))) char rt_lds[];
  int32_t* base = reinterpret_cast<int32_t*>(rt_lds);
  int32_t* scratch = base + a.E;
  int32_t* part = scratch + 16;
  uint16_t* wcnt = reinterpret_cast<uint16_t*>(part + 2048);
  const int tid = threadIdx.x, b = blockIdx.x;
  int epad = 1;
  while (epad < a.E) epad <<= 1;
  const int np = kRtThreads / epad, e = tid & (epad - 1), p = tid / epad;
  int before = 0, total = 0;
  if (e < a.E) {
#pragma unroll 8
    for (int c = p; c < a.nchunk; c += np) {
      const int h = a.hist[(int64_t)c * a.E + e];
      total += h;
      before += c < b ? h : 0;
    }
  }
  part[tid] = total;
  part[1024 + tid] = before;
  __syncthreads();
  total = before = 0;
  if (tid < a.E)
    for (int q = 0; q < np; ++q) { total += part[q * epad + tid]; before += part[1024 + q * epad + tid]; }
  const int first = rt_scan(total, scratch);
  if (tid < a.E) {
    base[tid] = first + before;
    if (b == 0) a.offsets[tid] = first;
  }
  if (b == 0 && tid == 0) a.offsets[a.E] = a.T * a.K;
  __syncthreads();
  const int64_t t0 = (int64_t)b * a.chunk, t1 = min(a.T, t0 + a.chunk);
  rt_place(a.ids, t0 * a.K, t1 * a.K, a.E, base, wcnt, a.slot_row, a.row_slot);
}

// ------------------------------------------------------------ gradient ----
// With g = scale * dweights: renormalised weights p = s / sum s depend on the
// chosen scores only, ds_j gives dl_j = p_j (g_j - sum_i p_i g_i), times 1 - s_j
// for the sigmoid; else sigmoid dl_j = g_j s_j (1 - s_j), and softmax
// dl_e = s_e (g_e - sum_j g_j s_j) for every expert, g_e = 0 where not chosen.
// Same lanes as the forward.  The chosen experts' values go through the wave's
// own LDS row, so each lane then writes its V experts in whole words.
constexpr int kRbThreads = 256;
struct RouteBwdKernelArgs {
  const void* logits; int64_t ld; const int32_t* ids; const float* dweights; void* dlogits; int64_t ld_d;
  int64_t T; int E, K, sigmoid, renorm; float scale; int vec, vec_out;
};

template <typename TIn, int V>
__device__ __forceinline__ void rt_store_row(TIn* p, int n, bool vec, const float (&v)[V]) {
  if constexpr (sizeof(TIn) == 2) {
    typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
    typedef float f2 __attribute__((ext_vector_type(2)));
    uint32_t w[V / 2];
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      const f2 q = {v[2 * i], v[2 * i + 1]};
      w[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(q, bf2));
    }
    if (vec && n >= V) {
#pragma unroll
      for (int q = 0; q < V / 8; ++q)
        reinterpret_cast<uint4*>(p)[q] = make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (i < n) reinterpret_cast<uint16_t*>(p)[i] = (uint16_t)(w[i / 2] >> (16 * (i & 1)));
    }
  } else {
    if (vec && n >= V) {
#pragma unroll
      for (int q = 0; q < V / 4; ++q)
        reinterpret_cast<float4*>(p)[q] = make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (i < n) p[i] = v[i];
    }
  }
}

template <typename TIn, int L, int V>
__global__ __launch_bounds__(kRbThreads) void route_backward_kernel(RouteBwdKernelArgs a) {
  __shared__ float spread[kRbThreads / 64][64 * V];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int sub = lane % L, e0 = sub * V;
  constexpr int TW = 64 / L;
  const int64_t tb = ((int64_t)blockIdx.x * (kRbThreads / 64) + wave) * TW + lane / L;
  const bool act = tb < a.T;
  const int64_t t = act ? tb : a.T - 1;
  const TIn* row = reinterpret_cast<const TIn*>(a.logits) + t * a.ld;
  const bool full = !a.sigmoid && !a.renorm;
  const bool live = sub < a.K;
  int id = live ? a.ids[t * a.K + sub] : -1;
  const bool ok = (unsigned)id < (unsigned)a.E;
  id = ok ? id : 0;
  const float g = ok ? a.dweights[t * a.K + sub] * a.scale : 0.f;
  const float xj = ok ? rt_load(row + id) : -__builtin_inff();
  float x[V], val, shift = 0.f, inv = 0.f;
  if (full) {
    rt_load_row<TIn, V>(row + e0, a.E - e0, a.vec != 0, x);
    float top = -__builtin_inff(), z = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) top = __builtin_fmaxf(top, x[i]);
    top = rt_max<L>(top);
    shift = top == -__builtin_inff() ? 0.f : top;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      x[i] = e0 + i < a.E ? expf(x[i] - shift) : 0.f;
      z += x[i];
    }
    z = rt_sum<L>(z);
    inv = z == 0.f ? 0.f : 1.f / z;
    val = g;
  } else if (a.sigmoid) {
    const float up = 1.f / (1.f + expf(xj));                  // 1 - s
    if (a.renorm) {
      const float ls = ok ? fminf(xj, 0.f) - log1pf(expf(-fabsf(xj))) : -__builtin_inff();
      const float m = rt_max<L>(ls);
      const float p0 = m == -__builtin_inff() ? 0.f : expf(ls - m);
      const float sum = rt_sum<L>(p0);
      const float p = sum == 0.f ? 0.f : p0 / sum;
      val = p * up * (g - rt_sum<L>(p * g));
    } else {
      val = ok ? g * up / (1.f + expf(-xj)) : 0.f;
    }
  } else {
    const float m = rt_max<L>(xj);
    const float p0 = m == -__builtin_inff() ? 0.f : expf(xj - m);
    const float sum = rt_sum<L>(p0);
    const float p = sum == 0.f ? 0.f : p0 / sum;
    val = p * (g - rt_sum<L>(p * g));
  }
  float dot = 0.f;
  if (full) dot = rt_sum<L>(ok ? g * expf(xj - shift) * inv : 0.f);
  float* mine = &spread[wave][lane / L * (L * V)];
#pragma unroll
  for (int i = 0; i < V; ++i) mine[e0 + i] = 0.f;
  __syncthreads();
  if (ok) mine[id] = val;
  __syncthreads();
  float o[V];
#pragma unroll
  for (int i = 0; i < V; ++i) o[i] = full ? x[i] * inv * (mine[e0 + i] - dot) : mine[e0 + i];
  if (act && e0 < a.E)
    rt_store_row<TIn, V>(reinterpret_cast<TIn*>(a.dlogits) + t * a.ld_d + e0, a.E - e0, a.vec_out != 0, o);
}

int rt_lanes(int E, int K, int groups) {
  const int need = std::max({(E + 15) / 16, K, groups});
  int L = 8;
  while (L < need) L <<= 1;
  return L;
}

// f(L, V) as compile-time constants.
template <typename F>
void rt_dispatch(int L, int E, F&& f) {
  const bool wide = E > 8 * L;
#define S3R_RT_CASE(l)                                                                          \
  case l:                                                                                       \
    if (wide) f(std::integral_constant<int, l>{}, std::integral_constant<int, 16>{});           \
    else f(std::integral_constant<int, l>{}, std::integral_constant<int, 8>{});                 \
    break;
  switch (L) {
    S3R_RT_CASE(8)
    S3R_RT_CASE(16)
    S3R_RT_CASE(32)
    S3R_RT_CASE(64)
  }
#undef S3R_RT_CASE
}

// One launch, one workgroup, up to this many slots and two passes over the tokens.
bool rt_single(int64_t T, int K, int L) { return T * K <= 1024 && T * L <= 2 * kRtThreads; }

bool rt_rows_aligned(const void* p, int64_t ld, int esize) {
  return ((uintptr_t)p & 15u) == 0 && (ld * esize) % 16 == 0;
}

}  // namespace

size_t route_workspace(int64_t T, int E) {
  return align_up((size_t)std::min<int64_t>(std::max<int64_t>(T, 1), kRtMaxChunks) * E * 4, 256);
}

hipError_t launch_route(const RouteArgs& a, hipStream_t st) {
  RouteKernelArgs k{};
  k.logits = a.logits; k.ld = a.ld; k.bias = a.bias;
  k.ids = a.ids; k.weights = a.weights; k.offsets = a.offsets; k.slot_row = a.slot_row; k.row_slot = a.row_slot;
  k.T = a.T; k.E = a.E; k.K = a.K; k.groups = a.groups; k.keep = a.keep; k.group_top = a.group_top;
  k.sigmoid = a.sigmoid; k.renorm = a.renorm; k.scale = a.scale; k.hist = (int32_t*)a.ws;
  const int esize = a.dtype == S3R_BF16 ? 2 : 4;
  k.vec = rt_rows_aligned(a.logits, a.ld, esize) ? 1 : 0;
  const int L = rt_lanes(a.E, a.K, a.groups);
  const bool key64 = a.bias != nullptr || (a.groups > 1 && a.group_top == 2);
  if (rt_single(a.T, a.K, L)) {
    k.nchunk = 1;
    k.chunk = std::max<int64_t>(a.T, 1);
  } else {
    k.chunk = (a.T + kRtMaxChunks - 1) / kRtMaxChunks;
    k.nchunk = (int)((a.T + k.chunk - 1) / k.chunk);
  }
  const size_t lds = rt_lds_bytes(a.E);
  rt_dispatch(L, a.E, [&](auto l, auto v) {
    constexpr int LL = decltype(l)::value, VV = decltype(v)::value;
    const dim3 grid((unsigned)k.nchunk), block(kRtThreads);
    if (a.dtype == S3R_BF16) {
      if (key64) hipLaunchKernelGGL((route_kernel<uint16_t, LL, VV, true>), grid, block, lds, st, k);
      else hipLaunchKernelGGL((route_kernel<uint16_t, LL, VV, false>), grid, block, lds, st, k);
    } else {
      if (key64) hipLaunchKernelGGL((route_kernel<float, LL, VV, true>), grid, block, lds, st, k);
      else hipLaunchKernelGGL((route_kernel<float, LL, VV, false>), grid, block, lds, st, k);
    }
  });
  if (k.nchunk > 1)
    hipLaunchKernelGGL(route_place_kernel, dim3((unsigned)k.nchunk), dim3(kRtThreads), lds, st, k);
  return hipGetLastError();
}

hipError_t launch_route_backward(const RouteBwdArgs& a, hipStream_t st) {
  if (a.T == 0) return hipSuccess;
  RouteBwdKernelArgs k{};
  k.logits = a.logits; k.ld = a.ld; k.ids = a.ids; k.dweights = a.dweights; k.dlogits = a.dlogits; k.ld_d = a.ld_d;
  k.T = a.T; k.E = a.E; k.K = a.K; k.sigmoid = a.sigmoid; k.renorm = a.renorm; k.scale = a.scale;
  const int esize = a.dtype == S3R_BF16 ? 2 : 4;
  k.vec = rt_rows_aligned(a.logits, a.ld, esize) ? 1 : 0;
  k.vec_out = rt_rows_aligned(a.dlogits, a.ld_d, esize) ? 1 : 0;
  const int L = rt_lanes(a.E, a.K, 1);
  rt_dispatch(L, a.E, [&](auto l, auto v) {
    constexpr int LL = decltype(l)::value, VV = decltype(v)::value;
    const int64_t per = (kRbThreads / 64) * (64 / LL);
    const dim3 grid((unsigned)((a.T + per - 1) / per)), block(kRbThreads);
    if (a.dtype == S3R_BF16) hipLaunchKernelGGL((route_backward_kernel<uint16_t, LL, VV>), grid, block, 0, st, k);
    else hipLaunchKernelGGL((route_backward_kernel<float, LL, VV>), grid, block, 0, st, k);
  });
  return hipGetLastError();
}

}  // namespace s3r
