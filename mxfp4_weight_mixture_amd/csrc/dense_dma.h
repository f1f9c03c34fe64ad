// Global -> LDS loads and the waits around them.
#pragma once

#include "dense.h"

namespace mxmoe {
namespace {

constexpr uint32_t kOut = 0x80000000u;   // an offset behind every resource's range

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc_at(const void* base) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, 0x7fffffff, 0x00020000);
}
// 16 bytes per lane, global -> LDS (lane i writes dst + 16 i)
__device__ __forceinline__ void dma16(__amdgpu_buffer_rsrc_t r, uint32_t voff, void* dst) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)dst, 16, voff, 0, 0, 0);
}
// 16 bytes per lane to registers
template <typename E>
__device__ __forceinline__ typename Vec<E>::v8 load16(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  return __builtin_bit_cast(typename Vec<E>::v8, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
}

// LDS read beside DMA in flight.  `restrict` gives it alias information; without
// any, the compiler may take it to depend on every LDS DMA and drain them first.
template <typename V>
__device__ __forceinline__ V read_lds(const __attribute__((address_space(3))) V* __restrict__ a) {
  return *a;
}
template <int N>
__device__ __forceinline__ void wait_vm() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
}
__device__ __forceinline__ void wait_lgkm0() { __builtin_amdgcn_s_waitcnt(15 | (3 << 14) | (7 << 4)); }
__device__ __forceinline__ void block_barrier() {
  asm volatile("" ::: "memory");
  wait_lgkm0();
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

}  // namespace
}  // namespace mxmoe
