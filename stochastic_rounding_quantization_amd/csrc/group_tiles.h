// The row tiles of products over groups of rows; shared by the MXFP4 and the INT8 forward products.
#pragma once

#include "s3r_internal.h"

namespace s3r {
namespace {

// Row tiles of a grouped product, found by one wave from the offsets themselves (prefix sums of the groups'
// tile counts, 64 groups a round).  bad: the offsets are not a non-decreasing sequence from 0 to R.
struct GroupTile { int e; int64_t r0, r1; };
__device__ __forceinline__ int64_t read_lane(int64_t v, int lane) {
  return (int64_t)(((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(v >> 32), lane) << 32) |
                   (uint32_t)__builtin_amdgcn_readlane((int)v, lane));
}
// Inclusive sums over the wave by DPP: shifts within the 16-lane rows, then the rows' last lanes.
__device__ __forceinline__ int wave_prefix(int s) {
  s += __builtin_amdgcn_update_dpp(0, s, 0x111, 0xF, 0xF, true);      // row_shr 1, 2, 4, 8
  s += __builtin_amdgcn_update_dpp(0, s, 0x112, 0xF, 0xF, true);
  s += __builtin_amdgcn_update_dpp(0, s, 0x114, 0xF, 0xF, true);
  s += __builtin_amdgcn_update_dpp(0, s, 0x118, 0xF, 0xF, true);
  s += __builtin_amdgcn_update_dpp(0, s, 0x142, 0xA, 0xF, false);     // row_bcast 15 into rows 1 and 3
  s += __builtin_amdgcn_update_dpp(0, s, 0x143, 0xC, 0xF, false);     // row_bcast 31 into rows 2 and 3
  return s;
}
// One round: groups g0 .. g0 + 63, one a lane; n its tiles, s the inclusive sums of n.
struct GroupRound { int64_t o0, o1; int n, s; bool bad; };
__device__ __forceinline__ GroupRound group_round(const int64_t* __restrict__ offsets, int64_t G, int64_t R, int64_t g0,
                                                  int tile) {
  const int64_t g = g0 + (threadIdx.x & 63);
  const bool in = g < G;
  GroupRound r;
  r.o0 = in ? offsets[g] : 0;
  r.o1 = in ? offsets[g + 1] : 0;
  r.bad = in && (r.o1 < r.o0 || r.o0 < 0 || r.o1 > R || (g == 0 && r.o0 != 0) || (g == G - 1 && r.o1 != R));
  r.n = r.bad ? 0 : (int)(((uint32_t)(r.o1 - r.o0) + (uint32_t)tile - 1u) / (uint32_t)tile);   // rows below 2^31
  r.s = wave_prefix(r.n);
  return r;
}
// All tiles of all groups; first: round 0, to be kept.
__device__ __forceinline__ int group_total(const int64_t* offsets, int64_t G, int64_t R, int tile, GroupRound& first,
                                           bool& bad) {
  first = group_round(offsets, G, R, 0, tile);
  int total = __builtin_amdgcn_readlane(first.s, 63);
  bool b = first.bad;
  for (int64_t g0 = 64; g0 < G; g0 += 64) {
    const GroupRound r = group_round(offsets, G, R, g0, tile);
    total += __builtin_amdgcn_readlane(r.s, 63);
    b |= r.bad;
  }
  bad = __builtin_amdgcn_ballot_w64(b) != 0;
  return total;
}
// Tile i, 0 <= i < total, of valid offsets: its group, its first row and the group's end.
__device__ __forceinline__ GroupTile group_tile(const int64_t* offsets, int64_t G, int64_t R, int tile,
                                                const GroupRound& first, int i) {
  GroupRound r = first;
  int carry = 0;                              // tiles of the groups before this round's
  for (int64_t g0 = 0;;) {
    const uint64_t m = __builtin_amdgcn_ballot_w64(carry + r.s > i);
    if (m || g0 + 64 >= G) {
      const int w = m ? __builtin_ctzll(m) : 0;
      const int before = carry + __builtin_amdgcn_readlane(r.s - r.n, w);
      return GroupTile{(int)g0 + w, read_lane(r.o0, w) + (int64_t)(i - before) * tile, read_lane(r.o1, w)};
    }
    carry += __builtin_amdgcn_readlane(r.s, 63);
    g0 += 64;
    r = group_round(offsets, G, R, g0, tile);
  }
}

}  // namespace
}  // namespace s3r
