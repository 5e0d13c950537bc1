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
// 64 bits tell it: without a bias the logits themselves are compared (the scores
// are monotone in them), otherwise, and for the sums of two, fp64 scores.  All keys
// in fp64 cost 179 us for 65536 tokens x 256 experts (8 groups, top 8); fp32 keys
// with an error bound, and fp64 for the tokens whose decisions lie within it
// (0.4 % there), cost 43.
//
// 16384 x 64 bf16, top 2: choice 4.7 us, order 6.5, for 2.6 MB: two launches' latency.
// 65536 x 256 fp32, grouped top 8: choice 43 us (850 vector instructions per four
// tokens take 31, fp64 choices the rest), order 12; the 75 MB alone would take 14.
#include <type_traits>

#include "s3r_internal.h"

namespace s3r {
namespace {

constexpr int kRtThreads = 1024;
constexpr int kRtMaxChunks = 256;    // token chunks of one call: the place kernel reads every chunk's counts
// A chunk fills four waves at least.  Geometric mean of 36 routers of 100 .. 20000 tokens, us: 13.3 with chunks of
// T / 256 tokens, two waves 12.5, four 12.4, eight 12.9 (all with 1024 threads for the order).
constexpr int kRtChunkLanes = 256;

template <typename TIn>
__device__ __forceinline__ float rt_load(const TIn* p) {
  if constexpr (sizeof(TIn) == 2) return bf16_to_f32(*reinterpret_cast<const uint16_t*>(p));
  else return *reinterpret_cast<const float*>(p);
}

// 16 bytes at an element's alignment: rows of any width and any slice of a tensor take them.
typedef uint32_t rt_u4_a2 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t rt_u4_a4 __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t rt_u2_a2 __attribute__((ext_vector_type(2), aligned(2)));
typedef uint32_t rt_u2_a4 __attribute__((ext_vector_type(2), aligned(4)));
typedef uint32_t rt_u1_a2 __attribute__((aligned(2)));

// V consecutive logits of a row from p, which has n left from there (the others: -inf, as masked).  kEnds: the row has
// a 16-byte word at least, so its end is read as its last word and moved to its place (65536 x 255 bf16, top 2: 47 us
// element by element, 30 so); kWhole: no lane sees the row's end; kElements: shorter rows, and where time does not
// count.
enum { kElements, kEnds, kWhole };
template <typename TIn, int V>
__device__ __forceinline__ void rt_load_row(const TIn* p, int n, int words, float (&x)[V]) {
  constexpr int W = 16 / (int)sizeof(TIn);
  if (words != kElements) {
#pragma unroll
    for (int q = 0; q < V / W; ++q) {
      const int left = n - q * W;
      float* y = x + q * W;
      v4u32 w = {0u, 0u, 0u, 0u};
      if (left > 0) {
        const TIn* at = p + q * W + (left < W ? left - W : 0);
        if constexpr (sizeof(TIn) == 2) w = *reinterpret_cast<const rt_u4_a2*>(at);
        else w = *reinterpret_cast<const rt_u4_a4*>(at);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(TIn) == 2) {
          y[2 * i] = __uint_as_float(w[i] << 16);
          y[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        } else {
          y[i] = __uint_as_float(w[i]);
        }
      }
    }
    if (words == kWhole) return;
#pragma unroll
    for (int q = 0; q < V / W; ++q) {
      const int left = n - q * W;
      float* y = x + q * W;
      if (left < W) {
        const int by = left > 0 ? W - left : W;
#pragma unroll
        for (int o = W; o > 0; o >>= 1)
#pragma unroll
          for (int i = 0; i < W; ++i) y[i] = by & o ? (i + o < W ? y[i + o] : -__builtin_inff()) : y[i];
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = i < n ? rt_load(p + i) : -__builtin_inff();
  }
}

// The value of the lane that the reduction's step O pairs this lane with: neighbours, pairs, quads and
// halves of a 16-lane row by DPP moves, which cost no trip through LDS; rows by a shuffle.
template <int O>
__device__ __forceinline__ int rt_partner(int v) {
  if constexpr (O == 1) return __builtin_amdgcn_update_dpp(0, v, 0xB1, 0xF, 0xF, true);        // quad_perm 1 0 3 2
  else if constexpr (O == 2) return __builtin_amdgcn_update_dpp(0, v, 0x4E, 0xF, 0xF, true);   // quad_perm 2 3 0 1
  else if constexpr (O == 4) return __builtin_amdgcn_update_dpp(0, v, 0x141, 0xF, 0xF, true);  // row_half_mirror
  else if constexpr (O == 8) return __builtin_amdgcn_update_dpp(0, v, 0x140, 0xF, 0xF, true);  // row_mirror
  else return __shfl_xor(v, O, 64);
}
template <int O>
__device__ __forceinline__ uint32_t rt_partner(uint32_t v) { return (uint32_t)rt_partner<O>((int)v); }
template <int O>
__device__ __forceinline__ float rt_partner(float v) { return __int_as_float(rt_partner<O>(__float_as_int(v))); }
template <int O>
__device__ __forceinline__ double rt_partner(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)rt_partner<O>((int)(uint32_t)u), hi = (uint32_t)rt_partner<O>((int)(u >> 32));
  return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}

// Reductions over the aligned L lanes of a token (each step joins equal halves, so every lane ends with
// the same value).
template <int L, int O = 1, typename T, typename F>
__device__ __forceinline__ T rt_reduce(T v, F&& join) {
  if constexpr (O < L) return rt_reduce<L, 2 * O>(join(v, rt_partner<O>(v)), join);
  else return v;
}
template <int L, typename T>
__device__ __forceinline__ T rt_sum(T v) {
  return rt_reduce<L>(v, [](T a, T b) { return a + b; });
}
__device__ __forceinline__ float rt_fmax(float a, float b) { return __builtin_fmaxf(a, b); }     // NaNs lose
__device__ __forceinline__ double rt_fmax(double a, double b) { return __builtin_fmax(a, b); }
template <int L, typename T>
__device__ __forceinline__ T rt_max(T v) {
  return rt_reduce<L>(v, [](T a, T b) { return rt_fmax(a, b); });
}
template <int L>
__device__ __forceinline__ int rt_min(int v) {
  return rt_reduce<L>(v, [](int a, int b) { return min(a, b); });
}

template <typename T> __device__ __forceinline__ T rt_neg_inf();
template <> __device__ __forceinline__ float rt_neg_inf<float>() { return -__builtin_inff(); }
template <> __device__ __forceinline__ double rt_neg_inf<double>() { return -__builtin_inf(); }

__host__ __device__ inline int64_t rt_hist_ld(int E) { return (E + 3) / 4 * 4; }

struct RouteKernelArgs {
  const void* logits; int64_t ld; const float* bias;
  int32_t* ids; float* weights; int64_t* offsets; int32_t* slot_row; int32_t* row_slot;
  int64_t T;
  int E, K, groups, keep, group_top, sigmoid, renorm;
  float scale;
  int32_t* hist;             // [nchunk][rt_hist_ld(E)] slots of the chunk's tokens at each expert
  int nchunk; int64_t chunk; // tokens per chunk
  int words;                 // of rt_load_row
  int group_lanes;           // lanes of an expert group where groups are whole power-of-two runs of lanes, else 0
};

// The slots [s0, s1) in order (e_first: the expert of this thread's first), each to row base[e] + (slots of e
// before it in the range); base is advanced.  Every thread of the block takes part.  A wave ranks its 64 slots by matching expert
// indices bit by bit with ballots, and the waves' counts are added in order, so the order is the
// slots' own and no atomic decides it.
__device__ __forceinline__ void rt_place(const int32_t* ids, int e_first, int64_t s0, int64_t s1, int E, int32_t* base,
                         uint16_t* wcnt, int32_t* __restrict__ slot_row, int32_t* __restrict__ row_slot) {
  const int nt = blockDim.x, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, nw = nt >> 6;
  int bits = 0;
  while ((1 << bits) < E) ++bits;
  for (int64_t t0 = s0; t0 < s1; t0 += nt) {
    for (int i = tid; i < (nw * E + 1) / 2; i += nt) reinterpret_cast<uint32_t*>(wcnt)[i] = 0;
    __syncthreads();
    const int64_t s = t0 + tid;
    const bool act = s < s1;
    const int e = t0 == s0 ? e_first : act ? ids[s] : 0;
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

// LDS of both kernels: base [E] | scratch [16] | hist or partial sums [2048] | wave counts [16][E] (uint16),
// in whose place the choice keeps its lanes' bias: L V <= 1024 floats, at most 512 of them where L follows
// top_k or groups (<= E) and not E / V, so 32 E + 1024 bytes hold either.
__host__ __device__ inline size_t rt_lds_bytes(int E) {
  return (size_t)E * 4 + 64 + 2048 * 4 + align_up((size_t)16 * E * 2, 16) + 1024;
}

// Keys of the row in Key's precision; -inf for masked experts and NaN keys.
template <typename Key, int L, int V>
__device__ __forceinline__ void rt_keys(const RouteKernelArgs& a, const float (&x)[V], const float (&bias)[V],
                                        float shift, Key (&key)[V]) {
  if constexpr (sizeof(Key) == 8) {
    if (a.sigmoid) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        key[i] = 1.0 / (1.0 + exp(-(double)x[i]));
        __builtin_amdgcn_sched_barrier(0);     // one after another: interleaved they take twice the registers
      }
    } else {
      double z = 0.0;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        key[i] = exp((double)x[i] - (double)shift);
        z += key[i];
        __builtin_amdgcn_sched_barrier(0);
      }
      z = rt_sum<L>(z);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        key[i] = key[i] / z;
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  } else {
    // The difference of two keys is within 2^-19 of the fp64 keys' (and the rounding of the bias's addition).  In
    // units of 2^-24: a sigmoid has 4 each of the hardware's exponential and reciprocal, 1 of the sum, and 2 |x| of the
    // exponent, which |x| e^-|x| < 0.37 bounds, 20 of two.  A softmax's sum has 21 (15 additions in a lane, 6 across the
    // lanes), its reciprocal 4, and these err in both scores alike: 25 of their difference, which is at most 1, and near
    // 1 only where the other terms, whose 4 of the exponential and 2.25 |x| of the exponent enter, are small.
    constexpr float kLog2e = 1.4426950408889634f;
    if (a.sigmoid) {
#pragma unroll
      for (int i = 0; i < V; ++i) key[i] = __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(x[i] * -kLog2e));
    } else {
      float z = 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        key[i] = __builtin_amdgcn_exp2f((x[i] - shift) * kLog2e);
        z += key[i];
      }
      z = __builtin_amdgcn_rcpf(rt_sum<L>(z));
#pragma unroll
      for (int i = 0; i < V; ++i) key[i] = key[i] * z;
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    key[i] += (Key)bias[i];
    if (!(x[i] > -__builtin_inff() && key[i] > rt_neg_inf<Key>())) key[i] = rt_neg_inf<Key>();
  }
}

// Keys closer than this may be in the other order in exact arithmetic: their errors, the rounding of the bias's
// addition, and the four low bits of both that rt_take32 puts an index in (30 x 2^-23 |key|).
__device__ __forceinline__ float rt_margin(float key) { return 0x1p-19f + 0x1p-18f * fabsf(key); }

// A group's score from its two largest keys; inf - inf is none, and ranks last (a NaN would beat nothing and lose to
// nothing: one group more than `keep` would stay).
template <typename Key>
__device__ __forceinline__ Key rt_pair(Key m1, Key m2) {
  const Key sum = m1 + m2;
  return sum == sum ? sum : rt_neg_inf<Key>();
}

// The best `keep` groups stay, the keys of the others become -inf.  Groups of whole runs of lanes: two
// largest keys in the lane, then across the run.  Any groups: one after another over all lanes.
// Returns whether a kept and a dropped group are within the margin of both.  A sum's margin is that of its keys'
// magnitudes: 256 - 256 is as far off as the 256s are.  Keys of +-inf are exact.
template <typename Key, int L, int V>
__device__ __forceinline__ bool rt_keep_groups(const RouteKernelArgs& a, int group_lanes, int e0, int per, int sub, int lane,
                                               Key (&key)[V]) {
  const bool two = a.group_top == 2;
  Key mine = rt_neg_inf<Key>(), mine2 = mine;             // lane g of the token: the two largest keys of group g
  if (group_lanes) {
    Key m1 = rt_neg_inf<Key>(), m2 = m1;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const Key lo = key[i] > m1 ? m1 : key[i];
      m2 = lo > m2 ? lo : m2;
      m1 = key[i] > m1 ? key[i] : m1;
    }
    for (int o = 1; o < group_lanes; o <<= 1) {
      const Key n1 = __shfl_xor(m1, o, 64), n2 = __shfl_xor(m2, o, 64);
      const Key lo = n1 > m1 ? m1 : n1, hi2 = n2 > m2 ? n2 : m2;
      m2 = lo > hi2 ? lo : hi2;
      m1 = n1 > m1 ? n1 : m1;
    }
    const int from = lane / L * L + (sub < a.groups ? sub : 0) * group_lanes;
    mine = __shfl(m1, from, 64);
    if (two) mine2 = __shfl(m2, from, 64);
  } else {
    for (int g = 0; g < a.groups; ++g) {
      Key m1 = rt_neg_inf<Key>();
#pragma unroll
      for (int i = 0; i < V; ++i)
        if ((e0 + i) / per == g) m1 = key[i] > m1 ? key[i] : m1;
      m1 = rt_max<L>(m1);
      Key m2 = rt_neg_inf<Key>();
      if (two) {
        int at = 1 << 30;
#pragma unroll
        for (int i = V - 1; i >= 0; --i)
          if ((e0 + i) / per == g && key[i] == m1) at = e0 + i;
        at = rt_min<L>(at);
#pragma unroll
        for (int i = 0; i < V; ++i)
          if ((e0 + i) / per == g && e0 + i != at && key[i] > m2) m2 = key[i];
        m2 = rt_max<L>(m2);
      }
      if (sub == g) { mine = m1; mine2 = m2; }
    }
  }
  float margin = 0.f;
  if constexpr (sizeof(Key) == 4) {
    const float inf = __builtin_inff(), m1 = fabsf(mine), m2 = two ? fabsf(mine2) : 0.f;
    margin = rt_margin(m1 < inf && m2 < inf ? m1 + m2 : 0.f);      // inf: a sum that may overflow
  }
  if (two) mine = rt_pair(mine, mine2);
  int rank = 0;
  for (int h = 0; h < a.groups; ++h) {
    const Key other = __shfl(mine, lane / L * L + h, 64);
    rank += (other > mine || (other == mine && h < sub)) ? 1 : 0;
  }
  const bool in = sub < a.groups;
  const uint64_t kept = __builtin_amdgcn_ballot_w64(in && rank < a.keep) >> (lane / L * L);
  bool close = false;
  if constexpr (sizeof(Key) == 4) {
    const float inf = __builtin_inff();
    const float least = -rt_max<L>(in && rank < a.keep ? margin < inf ? margin - mine : inf : -inf);
    const float most = rt_max<L>(in && rank >= a.keep ? margin < inf ? mine + margin : inf : -inf);
    close = most > -inf && !(least > most);               // -inf and -inf: a tie of nothing, decided by index
  }
  if (group_lanes) {
    const bool stay = (kept >> (sub / group_lanes)) & 1;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (!stay) key[i] = rt_neg_inf<Key>();
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (!((kept >> ((e0 + i) / per)) & 1)) key[i] = rt_neg_inf<Key>();
  }
  return close;
}

// fp32 keys as whole numbers of the same order, and back; the two zeros are one number.
__device__ __forceinline__ uint32_t rt_ordered(float f) {
  const uint32_t u = __float_as_uint(f + 0.f);
  return u ^ ((uint32_t)((int)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float rt_float(uint32_t u) {
  return __uint_as_float(u & 0x80000000u ? u ^ 0x80000000u : ~u);
}
constexpr uint32_t kNoKey = 0x007FFFFFu;        // rt_ordered(-inf): no eligible expert from here down

// The top_k fp32 keys: every lane sorts its four largest (whole numbers with the place in the low bits, so a
// maximum brings its index along), and the token's lanes give up their heads, the largest first; when a lane
// has given all four, every lane of the wave sorts again what lies below its last.  Lane j of the token returns
// choice j.  Where that cannot be the exact choice, close is set: a choice without an eligible key, or keys too near
// each other (kMargin: within rt_margin; kBits: equal but for the low bits; kUnique: bf16 logits, which fit the
// upper half, never).
enum { kUnique, kBits, kMargin };
template <int Kind, int L, int V>
__device__ __forceinline__ int rt_take32(const RouteKernelArgs& a, int e0, int sub, const float (&key)[V], bool& close) {
  constexpr int D = V < 4 ? V : 4;
  uint32_t l[D];
  uint32_t below = 0xFFFFFFFFu, last = 0;
  int mine = 0, have = 0;
  for (int j = 0; j < a.K + (Kind == kUnique ? 0 : 1); ++j) {
    if (j == 0 || (V > D && __builtin_amdgcn_ballot_w64(have == 0) != 0)) {
#pragma unroll
      for (int d = 0; d < D; ++d) l[d] = 0u;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        uint32_t t = rt_ordered(key[i]);
        t = Kind == kUnique ? (t & 0xFFFF0000u) | (uint32_t)(0xFFFF - (e0 + i)) : (t & ~15u) | (uint32_t)(15 - i);
        t = t < below ? t : 0u;
#pragma unroll
        for (int d = 0; d < D; ++d) {
          if (d > i) break;
          const uint32_t hi = max(l[d], t);
          t = min(l[d], t);
          l[d] = hi;
        }
      }
      have = D;
    }
    const uint32_t m = rt_reduce<L>(l[0], [](uint32_t x, uint32_t y) { return max(x, y); });
    if constexpr (Kind != kUnique) {
      // kMargin: also where the difference is NaN (two infinite keys, whose low bits make them one)
      if (j > 0) close |= Kind == kBits ? (last ^ m) < 16u : !(rt_float(last) - rt_float(m) > rt_margin(rt_float(last)));
      last = m;
      if (j == a.K) break;
    }
    close |= m <= kNoKey;
    int at;
    bool win = l[0] == m;
    if constexpr (Kind == kUnique) {
      at = 0xFFFF - (int)(m & 0xFFFFu);
    } else {
      at = rt_min<L>(win ? e0 + 15 - (int)(m & 15u) : 1 << 30);
      win = (uint32_t)(at - e0) < (uint32_t)V;
    }
    below = win ? m : below;
#pragma unroll
    for (int d = 0; d < D - 1; ++d) l[d] = win ? l[d + 1] : l[d];
    l[D - 1] = win ? 0u : l[D - 1];
    have -= win ? 1 : 0;
    if (sub == j) mine = at;
  }
  return mine;
}

// The choice of one token by fp64 keys, taken by the whole wave (V experts a lane): one after another the
// largest key, then the lowest index that holds it; a taken key becomes NaN, which loses every
// comparison, as do the places past E.  Lane j returns choice j.
template <typename TIn, int V, bool ByLogit>
__device__ __forceinline__ int rt_choose64(const RouteKernelArgs& a, const TIn* row, int per) {
  const int lane = threadIdx.x & 63, e0 = lane * V, n = a.E - e0;
  float x[V], bias[V], top = -__builtin_inff();
  rt_load_row<TIn, V>(row + e0, n, kElements, x);
  double key[V];
  const bool sums = a.groups > 1 && a.group_top == 2;      // the groups' order needs the scores
  if (!ByLogit || sums) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      bias[i] = a.bias && i < n ? a.bias[e0 + i] : 0.f;
      top = x[i] > top ? x[i] : top;
    }
    top = rt_max<64>(top);
    rt_keys<double, 64, V>(a, x, bias, top == -__builtin_inff() ? 0.f : top, key);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) key[i] = x[i] == x[i] ? (double)x[i] : -__builtin_inf();
  }
  if (a.groups > 1) rt_keep_groups<double, 64, V>(a, a.group_lanes ? per / V : 0, e0, per, lane, lane, key);
  if (ByLogit && sums) {
#pragma unroll
    for (int i = 0; i < V; ++i) key[i] = key[i] > -__builtin_inf() ? (double)x[i] : -__builtin_inf();
  }
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (i >= n) key[i] = __builtin_nan("");
  int mine = 0;
  for (int j = 0; j < a.K; ++j) {
    double m = key[0];
#pragma unroll
    for (int i = 1; i < V; ++i) m = __builtin_fmax(m, key[i]);
    m = rt_max<64>(m);
    int at = 1 << 30;
#pragma unroll
    for (int i = V - 1; i >= 0; --i) at = key[i] == m ? e0 + i : at;
    at = rt_min<64>(at);
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (e0 + i == at) key[i] = __builtin_nan("");
    if (lane == j) mine = at;
  }
  return mine;
}

// L lanes of a wave hold a token's row, V consecutive experts each (L V >= E, L >= top_k, L >= groups).  Whole:
// L V = E; a kernel of its own, since the code for a row's end costs the others registers (65536 x 256 fp32, top 2:
// 30 us, 33 with it).
template <typename TIn, int L, int V, bool ByLogit, bool Whole>
__global__ __launch_bounds__(kRtThreads) void route_kernel(RouteKernelArgs a) {
  extern __shared__ __attribute__((aligned(16))) char rt_lds[];
  int32_t* base = reinterpret_cast<int32_t*>(rt_lds);
  int32_t* scratch = base + a.E;
  int32_t* hist = scratch + 16;
  int32_t* sel = hist + 1024;                              // the choice, for a call of one workgroup
  uint16_t* wcnt = reinterpret_cast<uint16_t*>(hist + 2048);
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, nw = blockDim.x >> 6;
  const int sub = lane % L;
  float* lbias = reinterpret_cast<float*>(wcnt);           // L V values; the waves' counts come after the choice
  for (int e = tid; e < a.E; e += blockDim.x) hist[e] = 0;
  if (tid == 0) scratch[15] = nw;
  if constexpr (!ByLogit)
    for (int e = tid; e < L * V; e += blockDim.x) lbias[e] = a.bias && e < a.E ? a.bias[e] : 0.f;
  __syncthreads();
  const int64_t c0 = (int64_t)blockIdx.x * a.chunk, c1 = min(a.T, c0 + a.chunk);
  const int e0 = sub * V;
  const int groups_per = a.E / a.groups;
  constexpr int TW = 64 / L;
  const TIn* logits = reinterpret_cast<const TIn*>(a.logits);
  // the waves draw their next tokens from a counter (scratch[15], which nothing else uses before the scan):
  // one that has an fp64 choice to make, with code not in the instruction cache, leaves the rest to the others
  for (int64_t tb = c0 + wave * TW; tb < c1;) {
    const int64_t t = min(tb + lane / L, c1 - 1);       // lanes past the chunk repeat its last token, unwritten
    const bool act = tb + lane / L < c1;
    int per = groups_per;
    asm volatile("" : "+v"(per));      // else a quotient per place would be kept for the whole loop, and spilled
    float x[V];
    rt_load_row<TIn, V>(logits + t * a.ld + e0, Whole ? V : a.E - e0, Whole ? kWhole : a.words, x);
    bool row_odd = false;                                 // a NaN or +inf logit: the softmax is NaN
    float shift = 0.f;
    if (!a.sigmoid) {
      bool odd = false;
      float top = -__builtin_inff();
#pragma unroll
      for (int i = 0; i < V; ++i) {
        odd |= !(x[i] < __builtin_inff());
        top = x[i] > top ? x[i] : top;
      }
      top = rt_max<L>(top);
      row_odd = ((__builtin_amdgcn_ballot_w64(odd) >> (lane / L * L)) & (~0ull >> (64 - L))) != 0;
      shift = top == -__builtin_inff() ? 0.f : top;
    }
    float z = 0.f;                                        // the softmax's sum, where the weights need it
    if (!a.sigmoid && !a.renorm) {
#pragma unroll
      for (int i = 0; i < V; ++i) z += expf(x[i] - shift);
      z = rt_sum<L>(z);
    }
    // fp32 keys, and fp64 ones for the tokens in which they may not decide as exact ones
    float key[V];
    bool close = false;
    const bool sums = a.groups > 1 && a.group_top == 2;   // the groups' order needs the scores
    if (!ByLogit || sums) {
      float bias[V];
#pragma unroll
      for (int i = 0; i < V; ++i) bias[i] = ByLogit ? 0.f : lbias[e0 + i];
      rt_keys<float, L, V>(a, x, bias, shift, key);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) key[i] = x[i] == x[i] ? x[i] : -__builtin_inff();
    }
    if (a.groups > 1) {
      const bool near = rt_keep_groups<float, L, V>(a, a.group_lanes, e0, per, sub, lane, key);
      close = (!ByLogit || sums) && near;
    }
    if (ByLogit && sums) {
#pragma unroll
      for (int i = 0; i < V; ++i) key[i] = key[i] > -__builtin_inff() ? x[i] : -__builtin_inff();
    }
    constexpr int kKind = !ByLogit ? kMargin : sizeof(TIn) == 2 ? kUnique : kBits;
    int mine = rt_take32<kKind, L, V>(a, e0, sub, key, close);     // lane j of the token: choice j
    uint64_t left = __builtin_amdgcn_ballot_w64(close);
    while (left) {
      const int tok = __builtin_ctzll(left) / L;
      left &= ~((~0ull >> (64 - L)) << (tok * L));
      const int theirs = rt_choose64<TIn, (L * V + 63) / 64, ByLogit>(a, logits + min(tb + tok, c1 - 1) * a.ld, per);
      const int got = __shfl(theirs, sub, 64);
      if (lane / L == tok) mine = got;
    }
    // weights: lane j < top_k of the token
    const bool live = sub < a.K;
    const float xj = live ? rt_load(logits + t * a.ld + mine) : 0.f;
    float w;
    if (a.sigmoid) {
      w = live ? 1.f / (1.f + expf(-xj)) : 0.f;
      if (a.renorm) {
        float sum = rt_sum<L>(w);
        // a score near or below the smallest normal (e^-80 is 2e-35): all of the token from their logarithms, since
        // its weight among other small scores need not be small
        if (((__builtin_amdgcn_ballot_w64(live && xj < -80.f) >> (lane / L * L)) & (~0ull >> (64 - L))) != 0) {
          const float ls = live ? fminf(xj, 0.f) - log1pf(expf(-fabsf(xj))) : -__builtin_inff();
          const float m = rt_max<L>(ls);
          w = expf(ls - (m == -__builtin_inff() ? 0.f : m));
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
      w = row_odd ? __builtin_nanf("") : z == 0.f ? 0.f : expf(xj - shift) / z;
    }
    if (act && live) {
      a.ids[t * a.K + sub] = mine;
      if (a.nchunk == 1) sel[t * a.K + sub] = mine;
      a.weights[t * a.K + sub] = w * a.scale;
      atomicAdd(&hist[mine], 1);                            // whole numbers: any order gives the same
    }
    int next = 0;
    if (lane == 0) next = atomicAdd(&scratch[15], 1);
    tb = c0 + (int64_t)__builtin_amdgcn_readfirstlane(next) * TW;
  }
  __syncthreads();
  if (a.nchunk > 1) {
    for (int e = tid; e < a.E; e += blockDim.x) a.hist[(int64_t)blockIdx.x * rt_hist_ld(a.E) + e] = hist[e];
    return;
  }
  // one chunk: the order too, in this launch
  const int n = tid < a.E ? hist[tid] : 0;
  const int first = rt_scan(n, scratch);
  if (tid < a.E) { base[tid] = first; a.offsets[tid] = first; }
  if (tid == 0) a.offsets[a.E] = a.T * a.K;
  __syncthreads();
  rt_place(sel, tid < a.T * a.K ? sel[tid] : 0, 0, a.T * a.K, a.E, base, wcnt, a.slot_row, a.row_slot);
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
  const int64_t t0 = (int64_t)b * a.chunk, t1 = min(a.T, t0 + a.chunk);
  const int64_t s0 = t0 * a.K, s1 = t1 * a.K;
  const int e_first = s0 + tid < s1 ? a.ids[s0 + tid] : 0;     // on its way while the counts are added
  int32_t *sum = part, *sum_before = part + 1024;
  for (int e = tid; e < a.E; e += (int)blockDim.x) sum[e] = sum_before[e] = 0;
  __syncthreads();
  // four experts a thread, the chunks dealt to the threads that share them; whole numbers, so the
  // atomics' order changes nothing
  int quads = 1;
  while (quads * 4 < a.E) quads <<= 1;
  const int np = (int)blockDim.x / quads, q = tid & (quads - 1), p = tid / quads;
  int4 total4 = make_int4(0, 0, 0, 0), before4 = total4;
  if (q * 4 < a.E) {
#pragma unroll 16
    for (int c = p; c < a.nchunk; c += np) {
      const int4 h = *reinterpret_cast<const int4*>(a.hist + (int64_t)c * rt_hist_ld(a.E) + q * 4);
      total4.x += h.x; total4.y += h.y; total4.z += h.z; total4.w += h.w;
      if (c < b) { before4.x += h.x; before4.y += h.y; before4.z += h.z; before4.w += h.w; }
    }
    const int t4[4] = {total4.x, total4.y, total4.z, total4.w}, b4[4] = {before4.x, before4.y, before4.z, before4.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (q * 4 + i < a.E) {
        atomicAdd(&sum[q * 4 + i], t4[i]);
        atomicAdd(&sum_before[q * 4 + i], b4[i]);
      }
  }
  __syncthreads();
  const int total = tid < a.E ? sum[tid] : 0, before = tid < a.E ? sum_before[tid] : 0;
  const int first = rt_scan(total, scratch);
  if (tid < a.E) {
    base[tid] = first + before;
    if (b == 0) a.offsets[tid] = first;
  }
  if (b == 0 && tid == 0) a.offsets[a.E] = a.T * a.K;
  __syncthreads();
  rt_place(a.ids, e_first, s0, s1, a.E, base, wcnt, a.slot_row, a.row_slot);
}

// ------------------------------------------------------------ gradient ----
// With g = scale * dweights: renormalised weights p = s / sum s depend on the
// chosen scores only, ds_j gives dl_j = p_j (g_j - sum_i p_i g_i), times 1 - s_j
// for the sigmoid; else sigmoid dl_j = g_j s_j (1 - s_j), and softmax
// dl_e = s_e (g_e - sum_j g_j s_j) for every expert, g_e = 0 where not chosen.
// L lanes per token; lane l holds the 16-byte words l, l + L, .. of the row, so that a token's words leave in
// one run (with V consecutive experts a lane, 40001 x 160 fp32 took 18.5 us instead of 10.9, now 9.1).  The chosen experts'
// values reach their words through the wave's own LDS row.
constexpr int kRbThreads = 256;
struct RouteBwdKernelArgs {
  const void* logits; int64_t ld; const int32_t* ids; const float* dweights; void* dlogits; int64_t ld_d;
  int64_t T; int E, K, sigmoid, renorm; float scale; int words;
};

// Word of W elements at p, of which n exist.
template <typename TIn, int W>
__device__ __forceinline__ void rt_store_word(TIn* p, int n, const float* v) {
  if constexpr (sizeof(TIn) == 2) {
    typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
    typedef float f2 __attribute__((ext_vector_type(2)));
    uint32_t w[W / 2];
#pragma unroll
    for (int i = 0; i < W / 2; ++i) {
      const f2 q = {v[2 * i], v[2 * i + 1]};
      w[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(q, bf2));
    }
    if (n >= W) {
      *reinterpret_cast<rt_u4_a2*>(p) = v4u32{w[0], w[1], w[2], w[3]};
    } else {                           // the row's end: 4, 2 and 1 elements
      uint32_t a = w[0], b = w[1];
      if (n & 4) {
        *reinterpret_cast<rt_u2_a2*>(p) = rt_u2_a2{a, b};
        a = w[2]; b = w[3];
        p += 4;
      }
      if (n & 2) {
        *reinterpret_cast<rt_u1_a2*>(p) = a;
        a = b;
        p += 2;
      }
      if (n & 1) *p = (uint16_t)a;
    }
  } else {
    if (n >= W) {
      *reinterpret_cast<rt_u4_a4*>(p) = v4u32{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])};
    } else {
      float a = v[0];
      if (n & 2) {
        *reinterpret_cast<rt_u2_a4*>(p) = rt_u2_a4{__float_as_uint(a), __float_as_uint(v[1])};
        a = v[2];
        p += 2;
      }
      if (n & 1) *p = a;
    }
  }
}

template <typename TIn, int L, int V>
__global__ __launch_bounds__(kRbThreads) void route_backward_kernel(RouteBwdKernelArgs a) {
  __shared__ __attribute__((aligned(16))) float spread[kRbThreads / 64][64 * V];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int sub = lane % L;
  constexpr int TW = 64 / L, W = 16 / (int)sizeof(TIn), NQ = V / W;
  const int64_t tb = (wide_block() * (kRbThreads / 64) + wave) * TW + lane / L;
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
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      const int e = (q * L + sub) * W;
      float word[W];
      rt_load_row<TIn, W>(row + e, a.E - e, a.words, word);      // -inf past E
#pragma unroll
      for (int i = 0; i < W; ++i) x[q * W + i] = word[i];
    }
    float top = -__builtin_inff(), z = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) top = x[i] > top ? x[i] : top;
    top = rt_max<L>(top);
    shift = top == -__builtin_inff() ? 0.f : top;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      x[i] = expf(x[i] - shift);
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
      const float p0 = expf(ls - (m == -__builtin_inff() ? 0.f : m));       // (m passes over NaNs, the exponential keeps them)
      const float sum = rt_sum<L>(p0);
      const float p = sum == 0.f ? 0.f : p0 / sum;
      val = p * up * (g - rt_sum<L>(p * g));
    } else {
      val = ok ? g * up / (1.f + expf(-xj)) : 0.f;
    }
  } else {
    const float m = rt_max<L>(xj);
    const float p0 = expf(xj - (m == -__builtin_inff() ? 0.f : m));
    const float sum = rt_sum<L>(p0);
    const float p = sum == 0.f ? 0.f : p0 / sum;
    val = p * (g - rt_sum<L>(p * g));
  }
  float dot = 0.f;
  if (full) dot = rt_sum<L>(ok ? g * expf(xj - shift) * inv : 0.f);
  float* mine = &spread[wave][lane / L * (L * V)];
#pragma unroll
  for (int q = 0; q < NQ; ++q)
#pragma unroll
    for (int i = 0; i < W; ++i) mine[(q * L + sub) * W + i] = 0.f;
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");      // the wave's LDS operations keep their order
  __builtin_amdgcn_wave_barrier();
  if (ok) mine[id] = val;
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  TIn* out = reinterpret_cast<TIn*>(a.dlogits) + t * a.ld_d;
#pragma unroll
  for (int q = 0; q < NQ; ++q) {
    const int e = (q * L + sub) * W;
    float o[W];
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const float s = mine[e + i];
      o[i] = full ? x[q * W + i] * inv * (s - dot) : s;
    }
    if (act && e < a.E) rt_store_word<TIn, W>(out + e, a.E - e, o);
  }
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
bool rt_single(int64_t T, int E, int K, int L) { return E <= kRtThreads && T * K <= 1024 && T * L <= 2 * kRtThreads; }

}  // namespace

size_t route_workspace(int64_t T, int E) {
  return align_up((size_t)std::min<int64_t>(std::max<int64_t>(T, 1), kRtMaxChunks) * rt_hist_ld(E) * 4, 256);
}

hipError_t launch_route(const RouteArgs& a, hipStream_t st) {
  RouteKernelArgs k{};
  k.logits = a.logits; k.ld = a.ld; k.bias = a.bias;
  k.ids = a.ids; k.weights = a.weights; k.offsets = a.offsets; k.slot_row = a.slot_row; k.row_slot = a.row_slot;
  k.T = a.T; k.E = a.E; k.K = a.K; k.groups = a.groups; k.keep = a.keep; k.group_top = a.group_top;
  k.sigmoid = a.sigmoid; k.renorm = a.renorm; k.scale = a.scale; k.hist = (int32_t*)a.ws;
  const int esize = a.dtype == S3R_BF16 ? 2 : 4;
  if (a.keep == a.groups) k.groups = k.keep = 1;       // every group stays
  const int L = rt_lanes(a.E, a.K, k.groups);
  k.words = a.E * esize < 16 ? kElements : a.E % (8 * L) ? kEnds : kWhole;      // 8 or 16 experts a lane
  const int per = a.E / k.groups, V = a.E > 8 * L ? 16 : 8, run = per / V;
  if (k.groups > 1 && per % V == 0 && (run & (run - 1)) == 0) k.group_lanes = run;
  const bool by_score = a.bias != nullptr;      // else the logits' order is the scores'
  if (rt_single(a.T, a.E, a.K, L)) {
    k.nchunk = 1;
    k.chunk = std::max<int64_t>(a.T, 1);
  } else {
    k.chunk = std::max<int64_t>((a.T + kRtMaxChunks - 1) / kRtMaxChunks, kRtChunkLanes / L);
    k.nchunk = (int)((a.T + k.chunk - 1) / k.chunk);
  }
  // threads for the chunk's tokens; one workgroup's own order needs one per slot and expert, too
  int64_t threads = std::max<int64_t>(k.chunk * L, 64);
  if (k.nchunk == 1) threads = std::max<int64_t>({threads, k.chunk * a.K, a.E});
  threads = std::min<int64_t>((threads + 63) / 64 * 64, kRtThreads);
  const size_t lds = rt_lds_bytes(a.E);
  rt_dispatch(L, a.E, [&](auto l, auto v) {
    constexpr int LL = decltype(l)::value, VV = decltype(v)::value;
    const dim3 grid((unsigned)k.nchunk), block((unsigned)threads);
    auto go = [&](auto by_logit, auto whole) {
      constexpr bool B = decltype(by_logit)::value, F = decltype(whole)::value;
      if (a.dtype == S3R_BF16) hipLaunchKernelGGL((route_kernel<uint16_t, LL, VV, B, F>), grid, block, lds, st, k);
      else hipLaunchKernelGGL((route_kernel<float, LL, VV, B, F>), grid, block, lds, st, k);
    };
    auto pick = [&](auto by_logit) {
      if (k.words == kWhole) go(by_logit, std::true_type{});
      else go(by_logit, std::false_type{});
    };
    if (by_score) pick(std::false_type{});
    else pick(std::true_type{});
  });
  if (k.nchunk > 1) {
    // A thread per slot of a chunk and per expert, to the next of three sizes: fewer waves meet at each barrier.
    // Geometric mean of 36 routers of 100 .. 20000 tokens, us: 12.4 with 1024 threads for all, 11.1 so; the order
    // of 16384 x 64 top 2 6.9 and 6.5.
    const int64_t want = std::max<int64_t>(k.chunk * a.K, a.E);
    const unsigned place = want <= 256 ? 256 : want <= 512 ? 512 : kRtThreads;
    hipLaunchKernelGGL(route_place_kernel, dim3((unsigned)k.nchunk), dim3(place), lds, st, k);
  }
  return hipGetLastError();
}

hipError_t launch_route_backward(const RouteBwdArgs& a, hipStream_t st) {
  if (a.T == 0) return hipSuccess;
  RouteBwdKernelArgs k{};
  k.logits = a.logits; k.ld = a.ld; k.ids = a.ids; k.dweights = a.dweights; k.dlogits = a.dlogits; k.ld_d = a.ld_d;
  k.T = a.T; k.E = a.E; k.K = a.K; k.sigmoid = a.sigmoid; k.renorm = a.renorm; k.scale = a.scale;
  const int esize = a.dtype == S3R_BF16 ? 2 : 4;
  const int L = rt_lanes(a.E, a.K, 1);
  k.words = a.E * esize < 16 ? kElements : a.E % (8 * L) ? kEnds : kWhole;      // 8 or 16 experts a lane
  rt_dispatch(L, a.E, [&](auto l, auto v) {
    constexpr int LL = decltype(l)::value, VV = decltype(v)::value;
    const int64_t per = (kRbThreads / 64) * (64 / LL);
    const dim3 grid = wide_grid((a.T + per - 1) / per), block(kRbThreads);
    if (a.dtype == S3R_BF16) hipLaunchKernelGGL((route_backward_kernel<uint16_t, LL, VV>), grid, block, 0, st, k);
    else hipLaunchKernelGGL((route_backward_kernel<float, LL, VV>), grid, block, 0, st, k);
  });
  return hipGetLastError();
}

}  // namespace s3r
