// ciera_attend_device.cuh -- what the forms of attention over pages share: the
// requests, the pages, and a row computed by one warp value by value.
#pragma once

#include "ciera_attention.h"
#include "ciera_moe_device.cuh"

namespace ciera {
namespace {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr int kSliceValues = 8;   // 256 values of a head over a warp

__device__ __forceinline__ float minus_infinity() { return __uint_as_float(0xFF800000u); }

// Of the weights' sum, 0 of none.
__device__ __forceinline__ float inverse_sum(float sum) { return sum == 0.0f ? 0.0f : 1.0f / sum; }

// A request's tokens and keys as the calls read them.
struct Request {
  int32_t first;   // token
  int32_t tokens;  // new ones
  int32_t keys;    // with the new ones
};

__device__ __forceinline__ int32_t clamp_to(int32_t v, int32_t most) {
  return v < 0 ? 0 : v > most ? most : v;
}

__device__ __forceinline__ Request request_of(const AttendParams& p, int32_t r) {
  const int32_t from = r == 0 ? 0 : clamp_to(p.offsets[r], p.tokens);
  const int32_t to = clamp_to(p.offsets[r + 1], p.tokens);
  return {from, to > from ? to - from : 0, clamp_to(p.context[r], p.keys_most)};
}

// Keys that new token i of a request sees.
__device__ __forceinline__ int32_t seen_keys(const Request& r, int32_t i) {
  const int32_t n = r.keys - r.tokens + i + 1;
  return n > 0 ? n : 0;
}

// Request of token t and its place there; request -1: behind the last.
__device__ void find_row(const AttendParams& p, int32_t t, int32_t* request, int32_t* place) {
  *request = -1;
  *place = 0;
  if (p.requests == 0 || t >= clamp_to(p.offsets[p.requests], p.tokens)) return;
  int32_t lo = 0, hi = p.requests - 1;
  while (lo < hi) {  // the last that begins at t or before
    const int32_t mid = lo + (hi - lo + 1) / 2;
    if (p.offsets[mid] <= t)
      lo = mid;
    else
      hi = mid - 1;
  }
  const Request r = request_of(p, lo);
  if (t < r.first || t - r.first >= r.tokens) return;
  *request = lo;
  *place = t - r.first;
}

// Page that holds a request's key; -1: none.
__device__ __forceinline__ int32_t page_at(const AttendParams& p, int32_t request, int32_t index) {
  const int32_t page = p.table[request * p.table_stride + index];
  return page >= 0 && page < p.pages ? page : -1;
}

__device__ __forceinline__ float scale_of(uint32_t exponent) {
  return exponent == 255 ? __uint_as_float(0x7FC00000u) : __uint_as_float(exponent << 23);
}

// A warp's share of one row: values lane, lane + 32, ... of the head.
struct Slice {
  float most;      // of the scores so far, in powers of two
  float sum;       // of the weights
  float o[kSliceValues];
};

// Row `q` over the keys [from, to) of a request, value by value in 32 bits.
// Keys outside have no part in it.  own->sum 0: no keys.
__device__ __noinline__ void warp_attend(const AttendParams& p, const uint16_t* q, int32_t request,
                                         int32_t head, int32_t from, int32_t to, Slice* own) {
  const int lane = threadIdx.x & 31;
  float qv[kSliceValues], o[kSliceValues];
  float top = minus_infinity(), sum = 0.0f;
#pragma unroll
  for (int i = 0; i < kSliceValues; ++i) {
    const int d = lane + 32 * i;
    qv[i] = d < p.head_dim ? bf16_to_f32(q[d]) : 0.0f;
    o[i] = 0.0f;
  }
  const float scale = p.scale * kLog2e;
  int32_t page = -1, index = -1;
  for (int32_t key = from; key < to; ++key) {
    const int32_t at = key / p.page_size;
    if (at != index) {
      index = at;
      page = page_at(p, request, at);
    }
    const int32_t place = key - at * p.page_size;
    float k[kSliceValues] = {}, v[kSliceValues] = {}, dot = 0.0f;
    if (page >= 0) {
      const Side &ks = p.key, &vs = p.value;
      const int64_t kat = page * ks.stride[0] + place * ks.stride[1] + head * ks.stride[2];
      const int64_t vat = page * vs.stride[0] + place * vs.stride[1] + head * vs.stride[2];
      float k_scale = 1.0f, v_scale = 1.0f;
      if (p.e4m3) {
        k_scale = scale_of(ks.exponent[page * ks.exponent_stride[0] +
                                       place * ks.exponent_stride[1] +
                                       head * ks.exponent_stride[2]]);
        v_scale = scale_of(vs.exponent[page * vs.exponent_stride[0] +
                                       place * vs.exponent_stride[1] +
                                       head * vs.exponent_stride[2]]);
      }
#pragma unroll
      for (int i = 0; i < kSliceValues; ++i) {
        const int d = lane + 32 * i;
        if (d < p.head_dim) {
          if (p.e4m3) {
            k[i] = e4m3_to_f32(static_cast<const uint8_t*>(ks.data)[kat + d]) * k_scale;
            v[i] = e4m3_to_f32(static_cast<const uint8_t*>(vs.data)[vat + d]) * v_scale;
          } else {
            k[i] = bf16_to_f32(static_cast<const uint16_t*>(ks.data)[kat + d]);
            v[i] = bf16_to_f32(static_cast<const uint16_t*>(vs.data)[vat + d]);
          }
          dot += qv[i] * k[i];
        }
      }
    }
    const float score = warp_sum_f32(dot) * scale;
    const float most = score > top || score != score ? score : top;
    // (of scores of minus infinity alone no weight is 0 / 0)
    const float base = most == minus_infinity() ? 0.0f : most;
    const float old = exp2f(top - base), w = exp2f(score - base);
    top = most;
    sum = sum * old + w;
#pragma unroll
    for (int i = 0; i < kSliceValues; ++i) o[i] = o[i] * old + w * v[i];
  }
  own->most = top;
  own->sum = sum;
#pragma unroll
  for (int i = 0; i < kSliceValues; ++i) own->o[i] = o[i];
}

}  // namespace
}  // namespace ciera
