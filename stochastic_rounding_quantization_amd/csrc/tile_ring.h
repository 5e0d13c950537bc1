// Staging of a product's operands through a ring of LDS stages by buffer-load DMA; shared by the forward products.
#pragma once

#include "s3r_internal.h"

namespace s3r {
namespace {

typedef __attribute__((address_space(3))) void lds_void;
constexpr int kRsrcWord3 = 0x00020000;   // raw buffer, 32-bit dword format

#define S3R_WAIT_VM(n) __builtin_amdgcn_s_waitcnt(((n) & 0xF) | (((n) >> 4) << 14) | 0x70 | 0xF00)
#define S3R_WAIT_LGKM0() __builtin_amdgcn_s_waitcnt(0xC07F)
constexpr int kSgMfma = 0x008, kSgDsRead = 0x100, kSgVmem = 0x010;

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

__device__ __forceinline__ int chunk_pos(int r, int q) { return q ^ ((r >> 2) & 3); }

}  // namespace
}  // namespace s3r
