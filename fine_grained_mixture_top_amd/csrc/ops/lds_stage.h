// Stages of matrix operands on their way into LDS: loads that write LDS directly,
// 16 or 4 bytes per lane, and the waits for them.
#pragma once

#include "../device_common.h"

namespace moe {

typedef int i32x4_v __attribute__((ext_vector_type(4)));
typedef int i32x8_v __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) void lds_void_t;
typedef const __attribute__((address_space(3))) char* lds_ptr_t;
template <typename T> __device__ __forceinline__ T lds_ld(lds_ptr_t p) {
  return *reinterpret_cast<const __attribute__((address_space(3))) T*>(p);
}

constexpr uint32_t OOB = 0x80000000u;  // past every record count

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)bytes, 0x00020000);
}
__device__ __forceinline__ void load16_lds(__amdgpu_buffer_rsrc_t r, char* lds, uint32_t voff, uint32_t soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void_t*)lds, 16, voff, soff, 0, 0);
}
__device__ __forceinline__ void load4_lds(__amdgpu_buffer_rsrc_t r, char* lds, uint32_t voff, uint32_t soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void_t*)lds, 4, voff, soff, 0, 0);
}
// all but the newest N vector memory operations of this wave are complete
// (loads and stores complete in the order they were issued)
template <int N>
__device__ __forceinline__ void wait_vm() {
  static_assert(N < 64, "vmcnt has six bits");
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0x0F70 | (N & 15) | ((N >> 4) << 14));  // lgkmcnt, expcnt at their maximum
  asm volatile("" ::: "memory");
}

}  // namespace moe
