// ciera_moe_device.cuh -- device helpers shared by the kernels of the
// mixture-of-experts operators: bf16 and e4m3 conversion, block sums.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "ciera_moe.h"

namespace ciera {
namespace {

constexpr float kE4m3Max = 448.0f;
constexpr float kTinyAmax = 1e-30f;  // an all-zero row's scale is not 0

__device__ __forceinline__ float bf16_to_f32(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf16_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); }

__device__ __forceinline__ uint16_t f32_to_bf16(float v) {
  return __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

// Two floats to bf16 in one word, `lo` in bits 0..15.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ uint8_t f32_to_e4m3(float v) {
  return static_cast<uint8_t>(__nv_cvt_float_to_fp8(v, __NV_SATFINITE, __NV_E4M3));
}

__device__ __forceinline__ float e4m3_to_f32(uint8_t v) {
  const __half_raw h = __nv_cvt_fp8_to_halfraw(v, __NV_E4M3);
  return __half2float(__half(h));
}

// Scale of a row from the largest |value|'s bits: NaN for a row that holds an
// infinity or a NaN (their bits are the largest).
__device__ __forceinline__ float e4m3_scale(uint32_t amax_bits) {
  if (amax_bits >= 0x7F800000u) return __uint_as_float(0x7FC00000u);
  return fmaxf(__uint_as_float(amax_bits), kTinyAmax) / kE4m3Max;
}

// 16 bytes to shared memory, of which the first `bytes` come from `src`.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void copy16(void* dst, const void* src, int bytes) {
  copy16(static_cast<uint32_t>(__cvta_generic_to_shared(dst)), src, bytes);
}

__device__ __forceinline__ float warp_sum_f32(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sum over the block, the same in every thread; `part` holds 32 floats, and a
// barrier stands between two uses of it.
__device__ __forceinline__ float block_sum(float v, float* part) {
  v = warp_sum_f32(v);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) part[warp] = v;
  __syncthreads();
  const int warps = (blockDim.x + 31) >> 5;
  v = lane < warps ? part[lane] : 0.0f;
  return warp_sum_f32(v);
}

__device__ __forceinline__ uint32_t block_max(uint32_t v, uint32_t* part) {
  v = __reduce_max_sync(0xffffffffu, v);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) part[warp] = v;
  __syncthreads();
  const int warps = (blockDim.x + 31) >> 5;
  v = lane < warps ? part[lane] : 0u;
  return __reduce_max_sync(0xffffffffu, v);
}

// Eight bf16 values of a 16-byte word.
__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf16_lo(w[i]);
    f[2 * i + 1] = bf16_hi(w[i]);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]),
                    pack_bf16(f[6], f[7]));
}

// Four floats to e4m3 in one word.
__device__ __forceinline__ uint32_t pack_e4m3(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | hi << 16;
}

// Words of 8, 2 or 1 bf16 values, for rows that start on 16-, 4- or 2-byte
// boundaries; a Half holds as many e4m3 values.
template <typename W>
struct Word;
template <>
struct Word<uint4> {
  static constexpr int kValues = 8;
  using Half = uint2;
  static __device__ __forceinline__ void unpack(const uint4& v, float (&f)[8]) { unpack8(v, f); }
  static __device__ __forceinline__ uint4 pack(const float (&f)[8]) { return pack8(f); }
  static __device__ __forceinline__ uint2 pack_8bit(const float (&f)[8], float by) {
    return make_uint2(pack_e4m3(f[0] * by, f[1] * by, f[2] * by, f[3] * by),
                      pack_e4m3(f[4] * by, f[5] * by, f[6] * by, f[7] * by));
  }
};
template <>
struct Word<uint32_t> {
  static constexpr int kValues = 2;
  using Half = uint16_t;
  static __device__ __forceinline__ void unpack(uint32_t v, float (&f)[2]) {
    f[0] = bf16_lo(v);
    f[1] = bf16_hi(v);
  }
  static __device__ __forceinline__ uint32_t pack(const float (&f)[2]) {
    return pack_bf16(f[0], f[1]);
  }
  static __device__ __forceinline__ uint16_t pack_8bit(const float (&f)[2], float by) {
    return __nv_cvt_float2_to_fp8x2(make_float2(f[0] * by, f[1] * by), __NV_SATFINITE, __NV_E4M3);
  }
};
template <>
struct Word<uint16_t> {
  static constexpr int kValues = 1;
  using Half = uint8_t;
  static __device__ __forceinline__ void unpack(uint16_t v, float (&f)[1]) {
    f[0] = bf16_to_f32(v);
  }
  static __device__ __forceinline__ uint16_t pack(const float (&f)[1]) { return f32_to_bf16(f[0]); }
  static __device__ __forceinline__ uint8_t pack_8bit(const float (&f)[1], float by) {
    return f32_to_e4m3(f[0] * by);
  }
};

// Offset of group e, clamped to [lo, rows]; `lo` is the one before it.
__device__ __forceinline__ int32_t clamp_offset(int32_t v, int32_t lo, int32_t rows) {
  return v < lo ? lo : v > rows ? rows : v;
}

// Host: lets a kernel have `bytes` of dynamic shared memory, once per device
// (more than 48 KB want asking).
template <auto kKernel>
cudaError_t allow_shared(int bytes) {
  static std::atomic<uint64_t> asked{0};
  int device = 0;
  cudaError_t err = cudaGetDevice(&device);
  if (err != cudaSuccess) return err;
  const uint64_t bit = uint64_t(1) << (device & 63);
  if (asked.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  err = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (err == cudaSuccess) asked.fetch_or(bit, std::memory_order_relaxed);
  return err;
}

}  // namespace
}  // namespace ciera
