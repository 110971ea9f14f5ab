// ciera_attend.cu -- attention over pages of keys and values: which form a call
// takes, and the form that takes any size, stride and alignment.
#include "ciera_attend_device.cuh"

namespace ciera {
namespace {

constexpr int kAnyWarps = 4;
// A warp per row (token and query head).  Bound by the latency of its loads: right for
// every layout, not fast (one token of 4096 keys, 16 heads of 127 values, 1.15 ms, of 72 of
// 8 bits 1.7; the form for few rows takes 15 us of heads of 128).
__global__ void __launch_bounds__(32 * kAnyWarps) k_attend_any(const AttendParams p) {
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kAnyWarps + (threadIdx.x >> 5);
  const int heads = p.heads * p.group;
  const int64_t t = row / heads;
  if (t >= p.tokens) return;
  const int head = static_cast<int>(row - t * heads), lane = threadIdx.x & 31;
  int32_t request, place;
  Slice own{};
  find_row(p, static_cast<int32_t>(t), &request, &place);
  if (request >= 0) {
    const Request r = request_of(p, request);
    const uint16_t* q = p.q + t * p.q_token + head * p.q_head;
    if (p.e4m3)
      warp_attend<kSliceValues, true>(p, q, request, head / p.group, 0, seen_keys(r, place), &own);
    else
      warp_attend<kSliceValues, false>(p, q, request, head / p.group, 0, seen_keys(r, place), &own);
  }
  const float by = inverse_sum(own.sum);
  uint16_t* o = p.o + row * p.head_dim;
#pragma unroll
  for (int i = 0; i < kSliceValues; ++i)
    if (lane + 32 * i < p.head_dim) o[lane + 32 * i] = f32_to_bf16(own.o[i] * by);
}

}  // namespace

namespace {

int sm_count() {
  int device = 0, n = 0;
  if (cudaGetDevice(&device) != cudaSuccess ||
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, device) != cudaSuccess)
    return 1;
  return n;
}

}  // namespace

int64_t attend_workspace_bytes(int64_t, int64_t, int64_t head_dim) {
  const int sms = sm_count();
  int64_t most = split_workspace_bytes(sms);
  if (head_dim <= 128 && wide_workspace_bytes(sms) > most) most = wide_workspace_bytes(sms);
  return (most + 255) / 256 * 256;
}

int launch_attend(const AttendParams& given, void* stream) {
  AttendParams p = given;
  int status = cudaSuccess;
  p.blocks = sm_count();
  if (launch_attend_wide(p, stream, &status)) return status;
  if (launch_attend_split(p, stream, &status)) return status;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int64_t rows = static_cast<int64_t>(p.tokens) * p.heads * p.group;
  k_attend_any<<<static_cast<unsigned>((rows + kAnyWarps - 1) / kAnyWarps), 32 * kAnyWarps, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace ciera
