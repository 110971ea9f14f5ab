// ciera_tc_device.cuh -- what the kernels on the tensor cores (tcgen05) share:
// fences, descriptors of operands and instructions, and the maker of tensor maps.
#pragma once

#include <cuda.h>

#include "ciera_device.cuh"

namespace ciera {
namespace {

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}

__device__ __forceinline__ void tmem_ld_wait() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

// One lane of a warp, the same for every call; the compiler then knows that
// what it issues is issued once.
__device__ __forceinline__ bool one_lane() {
  uint32_t one;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.b32 %0, 1, 0, p;\n\t}"
               : "=r"(one));
  return one != 0;
}

// Shared-memory operand: 128-byte swizzle; `stride` bytes between groups of
// eight rows, `lead` between 128-byte columns (operands with the contraction
// along the rows only).
__device__ __forceinline__ uint64_t operand(uint32_t addr, uint32_t stride, uint32_t lead) {
  return static_cast<uint64_t>((addr & 0x3FFFF) >> 4) | static_cast<uint64_t>(lead >> 4) << 16 |
         static_cast<uint64_t>(stride >> 4) << 32 | uint64_t(1) << 46 | uint64_t(2) << 61;
}

// Instruction descriptor: 32-bit float sums, operand types, which operands
// have the contraction along their rows, N and M.
__device__ __forceinline__ uint32_t instruction(bool e4m3, bool a_rows, bool b_rows, int m,
                                                int n) {
  const uint32_t type = e4m3 ? 0u : 1u;
  return 1u << 4 | type << 7 | type << 10 | (a_rows ? 1u << 15 : 0u) | (b_rows ? 1u << 16 : 0u) |
         static_cast<uint32_t>(n >> 3) << 17 | static_cast<uint32_t>(m >> 4) << 24;
}

// Host: cuTensorMapEncodeTiled, null where the driver has none.
using Encode = decltype(&cuTensorMapEncodeTiled);

Encode encode() {
  static const Encode fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                         &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<Encode>(f);
  }();
  return fn;
}

}  // namespace
}  // namespace ciera
