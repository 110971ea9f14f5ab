// ciera_rows.cu -- the row-wise operators of the mixture-of-experts layer:
// the norm with the residual's addition and its gradient, rows to e4m3, the
// router's choice with the expert order, and the combination of the experts'
// rows.
#include <initializer_list>

#include "ciera_moe_device.cuh"

namespace ciera {
namespace {

constexpr int kRowThreads = 256;
constexpr int kRingBytes = 48 * 1024;
constexpr int64_t kManyRows = 2048;    // enough to fill the SMs with half the threads a row
constexpr int64_t kShiftDim = 768;     // values of an odd row from which on it goes by words
constexpr int64_t kShiftGradientDim = 128;  // the same of the gradient
constexpr int kMostRowThreads = 512;  // for one row of the kernels that hold rows in registers

// ------------------------------------------------------------------------
// Norm.  Bound by memory: 8 bytes a value in bf16 with a residual, 7 in e4m3
// (16384 rows of 2048 values: 39.9 us, 6.7 TB/s; in e4m3 40.4 us; rows to e4m3
// without a norm 15.1 us).
//
// k_rmsnorm holds a row in registers, kVecs words per thread, so that it is
// read once; blockDim.x threads take a row (whole warps, one reduction per
// statistic), blockDim.y rows share a block where rows are short.  Words are
// 16 bytes where all rows start on 16-byte boundaries, else 4 or 2.  Rows of odd
// length of matrices laid out alike go by 16-byte words too, but for their ends
// (see Part; 16384 x 2047: 51 us, 74 value by value; in e4m3 66 and 80; of 511
// values 22.5 and 22.5, and 28.7 and 24.6, the ends' words are then most of a
// row's warps).
// k_rmsnorm_any takes rows of any length, none too (whose mean is 0 / 0, and whose
// e4m3 scale that of zeros), value by value, and reads a row once
// per statistic (from L1 or L2 after the first).

__device__ __forceinline__ float norm_input(const NormParams& p, int64_t r, int64_t c) {
  float s = bf16_to_f32(p.x[r * p.x_stride + c]);
  if (p.residual) s += bf16_to_f32(p.residual[r * p.residual_stride + c]);
  return s;
}

__global__ void __launch_bounds__(kRowThreads) k_rmsnorm_any(const NormParams p) {
  __shared__ float part[32];
  __shared__ uint32_t part_max[32];
  for (int64_t r = blockIdx.x; r < p.rows; r += gridDim.x) {
    float rstd = 1.0f;
    if (p.weight) {
      float sum = 0.0f;
      for (int64_t c = threadIdx.x; c < p.dim; c += kRowThreads) {
        const float s = norm_input(p, r, c);
        sum += s * s;
      }
      sum = block_sum(sum, part);
      rstd = rsqrtf(sum / static_cast<float>(p.dim) + p.eps);
      if (p.rstd && threadIdx.x == 0) p.rstd[r] = rstd;
    }
    float scale = 0.0f, inverse = 0.0f;
    if (p.e4m3) {
      uint32_t amax = 0;
      for (int64_t c = threadIdx.x; c < p.dim; c += kRowThreads) {
        const float s = norm_input(p, r, c);
        const float y = p.weight ? s * rstd * bf16_to_f32(p.weight[c]) : s;
        amax = max(amax, __float_as_uint(y) & 0x7FFFFFFFu);
      }
      amax = block_max(amax, part_max);
      scale = e4m3_scale(amax);
      inverse = 1.0f / scale;
      if (threadIdx.x == 0) p.scale[r] = scale;
    }
    for (int64_t c = threadIdx.x; c < p.dim; c += kRowThreads) {
      // s is read before h is written at the same place: h may be the residual
      const float s = norm_input(p, r, c);
      const float y = p.weight ? s * rstd * bf16_to_f32(p.weight[c]) : s;
      if (p.h) p.h[r * p.dim + c] = f32_to_bf16(s);
      if (p.e4m3)
        static_cast<uint8_t*>(p.y)[r * p.dim + c] = f32_to_e4m3(y * inverse);
      else
        static_cast<uint16_t*>(p.y)[r * p.dim + c] = f32_to_bf16(y);
    }
    __syncthreads();  // `part` is free again
  }
}

// Sum over the row's threads (blockDim.x of them), the same in each; `part`
// has blockDim.y rows of 32.
__device__ __forceinline__ float row_sum(float v, float (*part)[32]) {
  v = warp_sum_f32(v);
  if (blockDim.x == 32) return v;
  const int lane = threadIdx.x & 31;
  if (lane == 0) part[threadIdx.y][threadIdx.x >> 5] = v;
  __syncthreads();
  v = lane < blockDim.x >> 5 ? part[threadIdx.y][lane] : 0.0f;
  return warp_sum_f32(v);
}

__device__ __forceinline__ uint32_t row_max(uint32_t v, uint32_t (*part)[32]) {
  v = __reduce_max_sync(0xffffffffu, v);
  if (blockDim.x == 32) return v;
  const int lane = threadIdx.x & 31;
  if (lane == 0) part[threadIdx.y][threadIdx.x >> 5] = v;
  __syncthreads();
  v = lane < blockDim.x >> 5 ? part[threadIdx.y][lane] : 0u;
  return __reduce_max_sync(0xffffffffu, v);
}

// Rows that do not start on 16-byte boundaries, but all of a call's at the same
// place `shift` behind one, are read and written by the 16-byte words that they
// touch.  Of the row's first and last word some values belong to it, `lo` to
// `hi` (never neither end: rows have 16 values and more); those go in up to
// three pieces of 2, 4 and 8 bytes, so that nothing outside the row is touched.
struct Part {
  int lo, hi;
  __device__ __forceinline__ Part(int column, int dim)
      : lo(column < 0 ? -column : 0), hi(dim - column < 8 ? dim - column : 8) {}
  __device__ __forceinline__ bool whole() const { return lo == 0 && hi == 8; }
};

// Pieces of a word as they are loaded, all before the first is needed.
struct Pieces {
  uint32_t one = 0, two = 0;
  uint2 four = {0, 0};
  __device__ __forceinline__ Pieces(const uint4* at, const Part& part) {
    const uint16_t* v = reinterpret_cast<const uint16_t*>(at);
    const int e = part.lo ? (part.lo + 1) & ~1 : part.hi & 4;  // of the two
    if ((part.lo | part.hi) & 1) one = v[part.lo ? part.lo : part.hi - 1];
    if (part.lo ? e & 2 : part.hi & 2) two = *reinterpret_cast<const uint32_t*>(v + e);
    if (part.lo ? part.lo <= 4 : part.hi >= 4)
      four = *reinterpret_cast<const uint2*>(v + (part.lo ? 4 : 0));
  }
  __device__ __forceinline__ uint4 word(const Part& part) const {
    if (part.lo) {
      const uint32_t high = one << 16;
      if (part.lo <= 4)
        return make_uint4(part.lo == 1 ? high : 0u, part.lo == 3 ? high : two, four.x, four.y);
      return make_uint4(0, 0, part.lo == 5 ? high : 0u, part.lo == 7 ? high : two);
    }
    const uint32_t first = part.hi & 2 ? two : one, second = part.hi & 2 ? one : 0u;
    return part.hi & 4 ? make_uint4(four.x, four.y, first, second)
                       : make_uint4(first, second, 0, 0);
  }
};

__device__ __forceinline__ void store_part(uint4* at, const uint4& w, const Part& part) {
  uint16_t* v = reinterpret_cast<uint16_t*>(at);
  if (part.whole()) {
    *at = w;
  } else if (part.lo) {
    const int odd = part.lo & 1, e = part.lo + odd;
    if (odd)
      v[part.lo] = static_cast<uint16_t>(
          (part.lo < 4 ? part.lo < 2 ? w.x : w.y : part.lo < 6 ? w.z : w.w) >> 16);
    if (e & 2) *reinterpret_cast<uint32_t*>(v + e) = e == 2 ? w.y : w.w;
    if (e <= 4) *reinterpret_cast<uint2*>(v + 4) = make_uint2(w.z, w.w);
  } else {
    if (part.hi & 4) *reinterpret_cast<uint2*>(v) = make_uint2(w.x, w.y);
    if (part.hi & 2) *reinterpret_cast<uint32_t*>(v + (part.hi & 4)) = part.hi & 4 ? w.z : w.x;
    if (part.hi & 1)
      v[part.hi - 1] = static_cast<uint16_t>(
          part.hi < 4 ? part.hi < 2 ? w.x : w.y : part.hi < 6 ? w.z : w.w);
  }
}

// The same of eight e4m3 values.
__device__ __forceinline__ void store_part(uint2* at, const uint2& w, const Part& part) {
  uint8_t* v = reinterpret_cast<uint8_t*>(at);
  if (part.whole()) {
    *at = w;
  } else if (part.lo) {
    const int odd = part.lo & 1, e = part.lo + odd;
    if (odd) v[part.lo] = static_cast<uint8_t>((part.lo < 4 ? w.x : w.y) >> (part.lo & 3) * 8);
    if (e & 2)
      *reinterpret_cast<uint16_t*>(v + e) = static_cast<uint16_t>((e == 2 ? w.x : w.y) >> 16);
    if (e <= 4) *reinterpret_cast<uint32_t*>(v + 4) = w.y;
  } else {
    const uint32_t rest = part.hi & 4 ? w.y : w.x;
    if (part.hi & 4) *reinterpret_cast<uint32_t*>(v) = w.x;
    if (part.hi & 2) *reinterpret_cast<uint16_t*>(v + (part.hi & 4)) = static_cast<uint16_t>(rest);
    if (part.hi & 1) v[part.hi - 1] = static_cast<uint8_t>(rest >> (part.hi & 2) * 8);
  }
}

// The weights of a word's columns, from 4-byte words, put together where the
// columns start inside one; `part` of them value by value.
__device__ __forceinline__ uint4 load_weights(const uint16_t* weight, int column) {
  const int odd = column & 1;
  const uint32_t* at = reinterpret_cast<const uint32_t*>(weight + (column - odd));
  uint32_t w[5] = {at[0], at[1], at[2], at[3], odd ? weight[column + 7] : 0u};
  if (odd)
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 16);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ uint4 load_weights(const uint16_t* weight, int column,
                                              const Part& part) {
  uint32_t f[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) f[j] = j >= part.lo && j < part.hi ? weight[column + j] : 0u;
  return make_uint4(f[0] | f[1] << 16, f[2] | f[3] << 16, f[4] | f[5] << 16, f[6] | f[7] << 16);
}

// kNorm false: rows to e4m3 as they are.
template <typename W, int kVecs, bool kNorm, bool kE4m3, bool kShift = false>
__global__ void __launch_bounds__(kMostRowThreads) k_rmsnorm(const NormParams p) {
  __shared__ float part[8][32];
  __shared__ uint32_t part_max[8][32];
  constexpr int kN = Word<W>::kValues;
  const int64_t r = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
  const int dim = static_cast<int>(p.dim), step = blockDim.x;
  const int shift =
      kShift ? static_cast<int>(reinterpret_cast<uintptr_t>(p.x + r * p.x_stride) >> 1 & 7) : 0;
  // words of the row from this thread's first on; a row behind the last has none
  const int words =
      r < p.rows ? (kShift ? (shift + dim + 7) / 8 : dim / kN) - static_cast<int>(threadIdx.x) : 0;
  const auto column = [&](int v) { return static_cast<int>(threadIdx.x + v * step) * 8 - shift; };
  const W* x = reinterpret_cast<const W*>(p.x + r * p.x_stride - shift) + threadIdx.x;
  const W* residual =
      reinterpret_cast<const W*>(p.residual + r * p.residual_stride - shift) + threadIdx.x;
  const W* weights = reinterpret_cast<const W*>(p.weight) + threadIdx.x;
  float s[kVecs][kN];
  W weight[kVecs] = {};
  float sum = 0.0f;
  uint32_t amax = 0;
  W in[kVecs], add[kVecs];
#pragma unroll
  for (int v = 0; v < kVecs; ++v) {
    in[v] = add[v] = W{};
    if (v * step < words) {
      if constexpr (kShift) {
        const Part part(column(v), dim);
        if (part.whole()) {
          in[v] = x[v * step];
          if (kNorm && p.residual) add[v] = residual[v * step];
          if (kNorm) weight[v] = load_weights(p.weight, column(v));
        } else {
          const Pieces of_x(x + v * step, part);
          const Pieces of_residual(kNorm && p.residual ? residual + v * step : x + v * step, part);
          if (kNorm) weight[v] = load_weights(p.weight, column(v), part);
          in[v] = of_x.word(part);
          if (kNorm && p.residual) add[v] = of_residual.word(part);
        }
        continue;
      }
      in[v] = x[v * step];
      if (kNorm && p.residual) add[v] = residual[v * step];
      if (kNorm) weight[v] = weights[v * step];
    }
  }
#pragma unroll
  for (int v = 0; v < kVecs; ++v) {
    Word<W>::unpack(in[v], s[v]);
    if (kNorm && p.residual) {
      float f[kN];
      Word<W>::unpack(add[v], f);
#pragma unroll
      for (int j = 0; j < kN; ++j) s[v][j] += f[j];
    }
#pragma unroll
    for (int j = 0; j < kN; ++j) sum += kNorm ? s[v][j] * s[v][j] : 0.0f;
  }
  if (kNorm) {
    if (p.h) {
      W* h = reinterpret_cast<W*>(p.h + r * p.dim - shift) + threadIdx.x;
#pragma unroll
      for (int v = 0; v < kVecs; ++v)
        if (v * step < words) {
          if constexpr (kShift)
            store_part(h + v * step, Word<W>::pack(s[v]), Part(column(v), dim));
          else
            h[v * step] = Word<W>::pack(s[v]);
        }
    }
    sum = row_sum(sum, part);
    const float rstd = rsqrtf(sum / static_cast<float>(p.dim) + p.eps);
    if (p.rstd && r < p.rows && threadIdx.x == 0) p.rstd[r] = rstd;
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
      float w[kN];
      Word<W>::unpack(weight[v], w);
#pragma unroll
      for (int j = 0; j < kN; ++j) s[v][j] = s[v][j] * rstd * w[j];
    }
  }
  float inverse = 1.0f;
  if (kE4m3) {
    if constexpr (kShift && kNorm) {
#pragma unroll
      for (int v = 0; v < kVecs; ++v) {
        const Part part(column(v), dim);
        if (!part.whole())
#pragma unroll
          for (int j = 0; j < kN; ++j)
            if (j < part.lo || j >= part.hi) s[v][j] = 0.0f;
      }
    }
#pragma unroll
    for (int v = 0; v < kVecs; ++v)
#pragma unroll
      for (int j = 0; j < kN; ++j)
        // behind the row stands 0 times rstd: not a number where rstd is infinite
        if (!kNorm || v * step < words)
          amax = max(amax, __float_as_uint(s[v][j]) & 0x7FFFFFFFu);
    const float scale = e4m3_scale(row_max(amax, part_max));
    inverse = 1.0f / scale;
    if (r < p.rows && threadIdx.x == 0) p.scale[r] = scale;
  }
  using Half = typename Word<W>::Half;
  W* y = reinterpret_cast<W*>(static_cast<uint16_t*>(p.y) + r * p.dim - shift) + threadIdx.x;
  Half* y8 = reinterpret_cast<Half*>(static_cast<uint8_t*>(p.y) + r * p.dim - shift) + threadIdx.x;
#pragma unroll
  for (int v = 0; v < kVecs; ++v)
    if (v * step < words) {
      if constexpr (kShift) {
        const Part part(column(v), dim);
        if (kE4m3)
          store_part(y8 + v * step, Word<W>::pack_8bit(s[v], inverse), part);
        else
          store_part(y + v * step, Word<W>::pack(s[v]), part);
        continue;
      }
      if (kE4m3)
        y8[v * step] = Word<W>::pack_8bit(s[v], inverse);
      else
        y[v * step] = Word<W>::pack(s[v]);
    }
}

// Gradient of the norm: each block takes rows blockIdx.x, + gridDim.x, ... in
// that order and keeps its part of the weight's gradient in its own row of
// `partial`, so that the result does not depend on the blocks' order.
__global__ void __launch_bounds__(kRowThreads) k_rmsnorm_backward_any(const NormBackwardParams p) {
  __shared__ float part[32];
  float* mine = p.partial + static_cast<int64_t>(blockIdx.x) * p.dim;
  for (int64_t r = blockIdx.x; r < p.rows; r += gridDim.x) {
    const float rstd = p.rstd[r];
    float dot = 0.0f;
    for (int64_t c = threadIdx.x; c < p.dim; c += kRowThreads)
      dot += bf16_to_f32(p.dy[r * p.dy_stride + c]) * bf16_to_f32(p.weight[c]) *
             bf16_to_f32(p.h[r * p.h_stride + c]);
    dot = block_sum(dot, part);
    const float pull = dot / static_cast<float>(p.dim) * rstd * rstd * rstd;
    for (int64_t c = threadIdx.x; c < p.dim; c += kRowThreads) {
      const float dy = bf16_to_f32(p.dy[r * p.dy_stride + c]);
      const float h = bf16_to_f32(p.h[r * p.h_stride + c]);
      float dx = rstd * dy * bf16_to_f32(p.weight[c]) - h * pull;
      if (p.dh) dx += bf16_to_f32(p.dh[r * p.dh_stride + c]);
      p.dx[r * p.dim + c] = f32_to_bf16(dx);
      const float dw = dy * h * rstd;
      mine[c] = r == blockIdx.x ? dw : mine[c] + dw;
    }
    __syncthreads();
  }
}

// The same with a row in registers and the weight's gradient too, the next
// row's words under way while this one is reduced.  Bound by memory, 8 bytes a
// value.  kShift: rows of odd length by the 16-byte words they touch; a block's
// rows are a multiple of eight apart, so that all of a thread's start alike
// (16384 x 2047: 82 us, 115 value by value, 109 with 16 values a thread, which
// every row's ends wait for; x 511 37 and 45).
template <typename W, int kVecs, bool kShift = false>
__global__ void __launch_bounds__(kMostRowThreads, kVecs * Word<W>::kValues <= 8 ? 2 : 1)
    k_rmsnorm_backward(const NormBackwardParams p) {
  __shared__ float part[2][8][32];
  constexpr int kN = Word<W>::kValues;
  const int dim = static_cast<int>(p.dim), across = blockDim.x;
  const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.y;
  const float inverse_dim = 1.0f / static_cast<float>(p.dim);
  float dw[kVecs][kN] = {};
  W weight[kVecs], dy[kVecs], h[kVecs], dh[kVecs];
  float rstd = 0.0f;
  int64_t r = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
  const int shift =
      kShift ? static_cast<int>(reinterpret_cast<uintptr_t>(p.dy + r * p.dy_stride) >> 1 & 7) : 0;
  // words of a row from this thread's first on
  const int words = (kShift ? (shift + dim + 7) / 8 : dim / kN) - static_cast<int>(threadIdx.x);
  const auto column_of = [&](int v) {
    return static_cast<int>(threadIdx.x + v * across) * kN - shift;
  };
  const W* dy_at = reinterpret_cast<const W*>(p.dy + r * p.dy_stride - shift) + threadIdx.x;
  const W* h_at = reinterpret_cast<const W*>(p.h + r * p.h_stride - shift) + threadIdx.x;
  const W* dh_at = reinterpret_cast<const W*>(p.dh + r * p.dh_stride - shift) + threadIdx.x;
  W* dx_at = reinterpret_cast<W*>(p.dx + r * p.dim - shift) + threadIdx.x;
  const float* rstd_at = p.rstd + r;
  const int64_t dy_step = step * p.dy_stride / kN, h_step = step * p.h_stride / kN;
  const int64_t dh_step = step * p.dh_stride / kN, dx_step = step * p.dim / kN;
  const auto fetch = [&](bool row) {
    const int have = row ? words : 0;
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
      dy[v] = h[v] = dh[v] = W{};
      if (v * across < have) {
        if constexpr (kShift) {
          const Part part(column_of(v), dim);
          if (!part.whole()) {
            const Pieces of_dy(dy_at + v * across, part), of_h(h_at + v * across, part);
            const Pieces of_dh((p.dh ? dh_at : dy_at) + v * across, part);
            dy[v] = of_dy.word(part);
            h[v] = of_h.word(part);
            if (p.dh) dh[v] = of_dh.word(part);
            continue;
          }
        }
        dy[v] = dy_at[v * across];
        h[v] = h_at[v * across];
        if (p.dh) dh[v] = dh_at[v * across];
      }
    }
    rstd = row ? *rstd_at : 0.0f;
    dy_at += dy_step;
    h_at += h_step;
    dh_at += dh_step;
    rstd_at += step;
  };
#pragma unroll
  for (int v = 0; v < kVecs; ++v) {
    weight[v] = W{};
    if (v * across < words) {
      if constexpr (kShift) {
        const Part part(column_of(v), dim);
        weight[v] = part.whole() ? load_weights(p.weight, column_of(v))
                                 : load_weights(p.weight, column_of(v), part);
      } else {
        weight[v] = reinterpret_cast<const W*>(p.weight)[v * across + threadIdx.x];
      }
    }
  }
  fetch(r < p.rows);
  int turn = 0;  // two reductions' scratch in turn: one barrier each
  for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * blockDim.y; r0 < p.rows; r0 += step) {
    // with n = h rstd:  dx = rstd (g - n mean(g n)) + dh,  dweight += dy n
    float g[kVecs][kN], n[kVecs][kN];
    W more[kVecs];
    float dot = 0.0f;
    const float rs = rstd;
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
      float d[kN], w[kN];
      Word<W>::unpack(dy[v], d);
      Word<W>::unpack(h[v], n[v]);
      Word<W>::unpack(weight[v], w);
      more[v] = dh[v];
#pragma unroll
      for (int j = 0; j < kN; ++j) {
        n[v][j] *= rs;
        g[v][j] = d[j] * w[j];
        dot += g[v][j] * n[v][j];
        dw[v][j] += d[j] * n[v][j];
      }
    }
    const int have = r < p.rows ? words : 0;
    r += step;
    fetch(r < p.rows);
    dot = row_sum(dot, part[turn]);
    turn ^= 1;
    const float mean = dot * inverse_dim;
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
      float out[kN];
      Word<W>::unpack(more[v], out);
#pragma unroll
      for (int j = 0; j < kN; ++j) out[j] += rs * (g[v][j] - n[v][j] * mean);
      if (v * across < have) {
        if constexpr (kShift)
          store_part(dx_at + v * across, Word<W>::pack(out), Part(column_of(v), dim));
        else
          dx_at[v * across] = Word<W>::pack(out);
      }
    }
    dx_at += dx_step;
  }
  // this block's part of the weight's gradient, its rows' in order
  extern __shared__ float column[];  // blockDim.y > 1: dim floats
  float* mine = p.partial + static_cast<int64_t>(blockIdx.x) * p.dim;
  for (int turn_y = 0; turn_y < blockDim.y; ++turn_y) {
    if (threadIdx.y == turn_y) {
#pragma unroll
      for (int v = 0; v < kVecs; ++v) {
        const int i = column_of(v);
        if (v * across >= words) continue;
#pragma unroll
        for (int j = 0; j < kN; ++j) {
          if (kShift && (i + j < 0 || i + j >= dim)) continue;
          const float before = turn_y ? column[i + j] : 0.0f;
          if (turn_y + 1 == blockDim.y)
            mine[i + j] = before + dw[v][j];
          else
            column[i + j] = before + dw[v][j];
        }
      }
    }
    if (blockDim.y > 1) __syncthreads();
  }
}

// The same for rows of 16-byte words that fit: rows come into a ring in shared
// memory by asynchronous copies, kRing - 1 of them ahead, each thread copying
// and reading its own words, so that the bytes under way do not depend on
// registers.  Rows of 16384 x 2048 values not in L2: 47 us with the sum of the
// blocks' parts (57 us with one row ahead in registers); 10007 x 1536: 25 us and 5.
// Wider rows, with all launches and nothing in L2: 16384 x 4096 94 us, 5.7 TB/s; x
// 5120 148, 4.6, and x 7168 170, 5.5, by the form above, of whose rows two do not
// fit the ring; 4096 x 12288 174, 2.3, whose 32 values a thread leave the
// registers; 2048 x 20000 297, 1.1, value by value.
template <int kVecs, int kRing>
__global__ void __launch_bounds__(kMostRowThreads)
    k_rmsnorm_backward_ring(const NormBackwardParams p) {
  extern __shared__ uint4 ring[];  // kRing x 3 x blockDim.y x words
  __shared__ float part[2][8][32];
  const int words = static_cast<int>(p.dim / 8), across = blockDim.x;
  const int have = words - static_cast<int>(threadIdx.x);  // words from this thread's first on
  const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.y;
  const float inverse_dim = 1.0f / static_cast<float>(p.dim);
  float dw[kVecs][8] = {};
  uint4 weight[kVecs];
#pragma unroll
  for (int v = 0; v < kVecs; ++v) {
    weight[v] = make_uint4(0, 0, 0, 0);
    if (v * across < have)
      weight[v] = reinterpret_cast<const uint4*>(p.weight)[v * across + threadIdx.x];
  }
  const int plane = blockDim.y * words;  // words of one tensor's rows in a stage
  uint4* mine = ring + threadIdx.y * words + threadIdx.x;
  const int64_t r_first = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
  // this thread's words of the next row to fetch, and of the row in hand
  const uint16_t* dy_in = p.dy + r_first * p.dy_stride + threadIdx.x * 8;
  const uint16_t* h_in = p.h + r_first * p.h_stride + threadIdx.x * 8;
  const uint16_t* dh_in = p.dh + r_first * p.dh_stride + threadIdx.x * 8;
  uint16_t* dx_out = p.dx + r_first * p.dim + threadIdx.x * 8;
  const int64_t dy_step = step * p.dy_stride, h_step = step * p.h_stride;
  const int64_t dh_step = step * p.dh_stride, dx_step = step * p.dim;
  int64_t left_in = p.rows - r_first, left = left_in;  // rows from that one on
  const auto fetch = [&](int stage) {
    if (left_in > 0) {
      uint4* to = mine + stage * 3 * plane;
#pragma unroll
      for (int v = 0; v < kVecs; ++v)
        if (v * across < have) {
          copy16(to + v * across, dy_in + v * across * 8, 16);
          copy16(to + plane + v * across, h_in + v * across * 8, 16);
          if (p.dh) copy16(to + 2 * plane + v * across, dh_in + v * across * 8, 16);
        }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    left_in -= step;
    dy_in += dy_step;
    h_in += h_step;
    dh_in += dh_step;
  };
#pragma unroll
  for (int i = 0; i + 1 < kRing; ++i) fetch(i);
  const float* rstd_in = p.rstd + r_first;
  float rstd = left > 0 ? *rstd_in : 0.0f;
  int turn = 0, stage = 0;
  for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * blockDim.y; r0 < p.rows; r0 += step) {
    const float rs = rstd;
    rstd_in += step;
    rstd = left > step ? *rstd_in : 0.0f;
    // the stage read in the last turn is free: its reader is this thread
    fetch(stage == 0 ? kRing - 1 : stage - 1);
    asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 1) : "memory");
    const uint4* from = mine + stage * 3 * plane;
    float g[kVecs][8], n[kVecs][8];
    float dot = 0.0f;
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
      float d[8], w[8];
      const bool some = left > 0 && v * across < have;  // else nothing was fetched
      unpack8(some ? from[v * across] : make_uint4(0, 0, 0, 0), d);
      unpack8(some ? from[plane + v * across] : make_uint4(0, 0, 0, 0), n[v]);
      unpack8(weight[v], w);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        n[v][j] *= rs;
        g[v][j] = d[j] * w[j];
        dot += g[v][j] * n[v][j];
        dw[v][j] += d[j] * n[v][j];
      }
    }
    dot = row_sum(dot, part[turn]);
    turn ^= 1;
    const float mean = dot * inverse_dim;
#pragma unroll
    for (int v = 0; v < kVecs; ++v)
      if (left > 0 && v * across < have) {
        float out[8] = {};
        if (p.dh) unpack8(from[2 * plane + v * across], out);
#pragma unroll
        for (int j = 0; j < 8; ++j) out[j] += rs * (g[v][j] - n[v][j] * mean);
        *reinterpret_cast<uint4*>(dx_out + v * across * 8) = pack8(out);
      }
    left -= step;
    dx_out += dx_step;
    stage = stage + 1 == kRing ? 0 : stage + 1;
  }
  // the block's rows' parts in order, through the ring's memory
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();
  float4* column = reinterpret_cast<float4*>(ring) + threadIdx.x * 2;
  float4* out = reinterpret_cast<float4*>(p.partial + static_cast<int64_t>(blockIdx.x) * p.dim) +
                threadIdx.x * 2;
  for (int y = 0; y < blockDim.y; ++y) {
    if (threadIdx.y == y) {
#pragma unroll
      for (int v = 0; v < kVecs; ++v) {
        if (v * across >= have) continue;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          float4 sum = make_float4(dw[v][4 * q], dw[v][4 * q + 1], dw[v][4 * q + 2],
                                   dw[v][4 * q + 3]);
          if (y) {
            const float4 before = column[v * across * 2 + q];
            sum.x += before.x;
            sum.y += before.y;
            sum.z += before.z;
            sum.w += before.w;
          }
          (y + 1 == blockDim.y ? out : column)[v * across * 2 + q] = sum;
        }
      }
    }
    if (blockDim.y > 1) __syncthreads();
  }
}

// Sums of the blocks' parts: 32 columns a block, each by 32 threads that take
// every 32nd part in order, then those 32 sums in order of a tree.
__global__ void __launch_bounds__(1024) k_sum_partials(const float* partial, int blocks,
                                                       int64_t dim, float* out) {
  __shared__ float sums[32][33];
  const int lane = threadIdx.x & 31, way = threadIdx.x >> 5;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  float sum = 0.0f;
  if (c < dim)
#pragma unroll 8
    for (int b = way; b < blocks; b += 32) sum += partial[b * dim + c];
  sums[way][lane] = sum;
  __syncthreads();
  const float total = warp_sum_f32(sums[lane][way]);
  const int64_t to = static_cast<int64_t>(blockIdx.x) * 32 + way;
  if (lane == 0 && to < dim) out[to] = total;
}

// ------------------------------------------------------------------------
// Route.  A warp per token: its logits in registers, topk rounds of "largest
// remaining, lowest index" (the first round's is the softmax's maximum), then
// the softmax's sum and the chosen weights.  Bound by issue slots, about 600
// instructions a token: 16384 tokens, 128 experts, 8 chosen: 13.4 us, and 8.6 for
// k_route_place; one token 3.1 us.  From 257 experts on a lane holds 32 logits, which
// leave the registers, and sorts as many whatever their number: both launches 43 us
// with 256 experts, 365 with 384, 530 with 1024 (the gradient 18, 84, 121).
//
// The order: a token chooses an expert at most once, so a pair's rank among
// its block's pairs of the same expert is the number of earlier tokens of the
// block that chose it.  With a bit per token and expert (32 tokens a block)
// that is a population count, independent of the order in which warps set
// the bits.  k_route leaves ranks and the counts per block and expert;
// k_route_place adds what stands before the block.

// Order-preserving bits of a logit: NaN on top, -inf above 0, 0 for "none".
__device__ __forceinline__ uint32_t logit_key(float l) {
  if (l != l) return 0xFFFFFFFFu;
  if (l == 0.0f) l = 0.0f;  // -0 and +0 tie
  const uint32_t b = __float_as_uint(l);
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
constexpr uint32_t kKeyMinusInf = 0x007FFFFFu;  // logit_key(-inf)

// The logit of a key (+0 for either zero, a NaN for any).
__device__ __forceinline__ float key_logit(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
}

__device__ __forceinline__ float load_logit(const void* logits, int bf16, int64_t i) {
  return bf16 ? bf16_to_f32(static_cast<const uint16_t*>(logits)[i])
              : static_cast<const float*>(logits)[i];
}

// Exclusive sums of v[0 .. n) in place, the total in v[n]; one warp.
__device__ __forceinline__ void exclusive_sums(int32_t* v, int n) {
  const int lane = threadIdx.x & 31;
  int32_t run = 0;
  for (int i0 = 0; i0 < n; i0 += 32) {
    const int i = i0 + lane;
    const int32_t own = i < n ? v[i] : 0;
    int32_t sum = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int32_t left = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += left;
    }
    if (i < n) v[i] = run + sum - own;
    run += __shfl_sync(0xffffffffu, sum, 31);
  }
  if (lane == 0) v[n] = run;
}

constexpr int kRouteWarps = 16;

// Batcher's odd-even merge sort of a lane's V keys, descending; equal keys keep
// the lower place first.
template <int V>
__device__ __forceinline__ void sort_lane(uint32_t (&key)[V], int (&place)[V]) {
#pragma unroll
  for (int p = 1; p < V; p <<= 1)
#pragma unroll
    for (int k = p; k >= 1; k >>= 1)
#pragma unroll
      for (int j = k % p; j + k < V; j += 2 * k)
#pragma unroll
        for (int i = 0; i < k; ++i) {
          const int a = i + j, b = i + j + k;
          if (b < V && a / (2 * p) == b / (2 * p)) {
            const bool swap =
                key[b] > key[a] || (key[b] == key[a] && place[b] < place[a]);
            const uint32_t ka = key[a];
            const int pa = place[a];
            key[a] = swap ? key[b] : ka;
            place[a] = swap ? place[b] : pa;
            key[b] = swap ? ka : key[b];
            place[b] = swap ? pa : place[b];
          }
        }
}

// V: logits per lane (experts <= 32 V).
template <int V>
__global__ void __launch_bounds__(kRouteWarps * 32) k_route(const RouteParams p) {
  __shared__ uint32_t bits[kMaxExperts];  // per expert: a bit per token of this block
  for (int e = threadIdx.x; e < p.experts; e += blockDim.x) bits[e] = 0;
  __syncthreads();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kRouteTokens;
  // the next token's logits are under way while this one's are sorted
  float next[V];
  bool next_live = false;
  const auto fetch = [&](int i) {
    const int64_t t = first + i;
    const bool some = i < kRouteTokens && t < p.tokens;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = v * 32 + lane;
      next[v] = some && e < p.experts ? load_logit(p.logits, p.bf16, t * p.stride + e) : -INFINITY;
    }
    next_live = some && (!p.mask || p.mask[t] != 0);
  };
  fetch(warp);
  for (int i = warp; i < kRouteTokens; i += kRouteWarps) {
    const int64_t t = first + i;
    if (t >= p.tokens) break;
    const bool live = next_live;
    float l[V];
    uint32_t key[V];
#pragma unroll
    for (int v = 0; v < V; ++v) l[v] = next[v];
    fetch(i + kRouteWarps);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = v * 32 + lane;
      key[v] = e < p.experts && live ? logit_key(l[v]) : 0u;
      if (key[v] <= kKeyMinusInf) key[v] = 0u;  // -inf is never chosen
    }
    // Each lane sorts its logits, largest first, lowest index first among
    // equals (V is a power of two: a network of compare-exchanges), and offers
    // its first; the lane that is taken moves up.
    int place[V];
#pragma unroll
    for (int v = 0; v < V; ++v) place[v] = v * 32 + lane;
    sort_lane<V>(key, place);
    uint32_t picked = 0, largest = 0;  // lane j: key and expert of choice j
    int choice = -1;
    for (int j = 0; j < p.topk; ++j) {
      const uint32_t best = __reduce_max_sync(0xffffffffu, key[0]);
      if (best == 0) break;  // nothing left to choose
      if (j == 0) largest = best;
      const uint32_t e =
          __reduce_min_sync(0xffffffffu, key[0] == best ? static_cast<uint32_t>(place[0]) : ~0u);
      if (e == static_cast<uint32_t>(place[0])) {
#pragma unroll
        for (int v = 0; v + 1 < V; ++v) {
          key[v] = key[v + 1];
          place[v] = place[v + 1];
        }
        key[V - 1] = 0u;
      }
      if (lane == j) {
        picked = best;
        choice = static_cast<int>(e);
      }
    }
    const float top = key_logit(largest);
    float sum = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (v * 32 + lane < p.experts) sum += expf(l[v] - top);
    sum = warp_sum_f32(sum);
    float mine = choice >= 0 ? expf(key_logit(picked) - top) / sum : 0.0f;
    if (p.renormalize) {
      const float total = warp_sum_f32(mine);
      if (choice >= 0) mine /= total;
    }
    if (choice >= 0) atomicOr(&bits[choice], 1u << i);
    if (lane < p.topk) {
      p.weights[t * p.topk + lane] = mine;
      p.chosen[t * p.topk + lane] = choice;
    }
  }
  __syncthreads();
  const int64_t pairs = min(static_cast<int64_t>(kRouteTokens), p.tokens - first) * p.topk;
  if (gridDim.x > 1) {
    const int row = count_stride(p.experts);
    for (int e = threadIdx.x; e < row; e += blockDim.x)
      p.counts[static_cast<int64_t>(blockIdx.x) * row + e] =
          e < p.experts ? static_cast<uint8_t>(__popc(bits[e])) : 0;
    for (int64_t i = threadIdx.x; i < pairs; i += blockDim.x) {
      const int e = p.chosen[first * p.topk + i];
      const int token = static_cast<int>(i / p.topk);
      p.slots[first * p.topk + i] = e < 0 ? -1 : __popc(bits[e] & ((1u << token) - 1));
    }
    return;
  }
  // One block has all tokens: the order at once.
  __shared__ int32_t base[kMaxExperts + 1];
  for (int e = threadIdx.x; e < p.experts; e += blockDim.x) base[e] = __popc(bits[e]);
  __syncthreads();
  if (threadIdx.x < 32) exclusive_sums(base, p.experts);
  __syncthreads();
  for (int e = threadIdx.x; e <= p.experts; e += blockDim.x) p.offsets[e] = base[e];
  for (int64_t i = threadIdx.x; i < pairs; i += blockDim.x) {
    const int e = p.chosen[i];
    const int token = static_cast<int>(i / p.topk);
    if (e >= 0) {
      const int32_t slot = base[e] + __popc(bits[e] & ((1u << token) - 1));
      p.slots[i] = slot;
      p.row_tokens[slot] = token;
    } else {
      p.slots[i] = -1;
    }
    if (i >= base[p.experts]) p.row_tokens[i] = -1;
  }
}

// Adds what stands before a block of k_route to its pairs' ranks.  A block
// here takes `group` of those in turn, at most 152 blocks in all: each of them
// sums the counts of all (four experts a word, 16 warps), which costs 64 KB
// from L2 with 16384 tokens and 128 experts.
constexpr int kPlaceThreads = 512;
constexpr int kPlaceBlocks = 152;

__global__ void __launch_bounds__(kPlaceThreads) k_route_place(const RouteParams p, int blocks,
                                                               int group) {
  __shared__ int32_t base[kMaxExperts + 1];  // offsets
  __shared__ int32_t before[kMaxExperts];    // rows of earlier blocks
  for (int e = threadIdx.x; e < p.experts; e += kPlaceThreads) base[e] = before[e] = 0;
  const int lane = threadIdx.x & 31, way = threadIdx.x >> 5;
  const int words = count_stride(p.experts) / 4;
  const int begin = blockIdx.x * group, end = min(begin + group, blocks);
  const uint32_t* counts = reinterpret_cast<const uint32_t*>(p.counts);
  // this thread's first pair is under way meanwhile
  const int64_t all_pairs = static_cast<int64_t>(p.tokens) * p.topk;
  const int block_pairs = kRouteTokens * p.topk;
  int expert = -1, rank = 0;
  const auto fetch = [&](int b) {
    const int64_t pair = static_cast<int64_t>(b) * block_pairs + threadIdx.x;
    const bool some = b < end && static_cast<int>(threadIdx.x) < block_pairs && pair < all_pairs;
    expert = some ? p.chosen[pair] : -1;
    rank = some ? p.slots[pair] : 0;
  };
  fetch(begin);
  __syncthreads();
  for (int w = lane; w < words; w += 32) {
    int32_t all[4] = {}, mine[4] = {};
#pragma unroll 16
    for (int b = way; b < blocks; b += kPlaceThreads / 32) {
      const uint32_t n = counts[static_cast<int64_t>(b) * words + w];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int32_t c = n >> (8 * i) & 0xFF;
        all[i] += c;
        if (b < begin) mine[i] += c;
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (w * 4 + i < p.experts) {  // whole numbers: the order does not matter
        atomicAdd(&base[w * 4 + i], all[i]);
        atomicAdd(&before[w * 4 + i], mine[i]);
      }
  }
  __syncthreads();
  if (threadIdx.x < 32) exclusive_sums(base, p.experts);
  __syncthreads();
  if (blockIdx.x == 0)
    for (int e = threadIdx.x; e <= p.experts; e += kPlaceThreads) p.offsets[e] = base[e];
  const int32_t used = base[p.experts];
  for (int b = begin; b < end; ++b) {
    const int64_t first = static_cast<int64_t>(b) * block_pairs;
    const auto put = [&](int i, int e, int r) {
      const int64_t pair = first + i;
      if (e >= 0) {
        const int32_t slot = base[e] + before[e] + r;
        p.slots[pair] = slot;
        // (counts that someone else wrote to would lead outside)
        if (static_cast<uint32_t>(slot) < static_cast<uint32_t>(all_pairs))
          p.row_tokens[slot] = b * kRouteTokens + i / p.topk;
      }
      if (pair >= used) p.row_tokens[pair] = -1;  // rows past the last group
    };
    const int pairs = static_cast<int>(min(static_cast<int64_t>(block_pairs), all_pairs - first));
    if (static_cast<int>(threadIdx.x) < pairs) put(threadIdx.x, expert, rank);
    for (int i = threadIdx.x + kPlaceThreads; i < pairs; i += kPlaceThreads)
      put(i, p.chosen[first + i], p.slots[first + i]);
    if (b + 1 == end) break;
    fetch(b + 1);
    __syncthreads();
    for (int e = threadIdx.x; e < p.experts; e += kPlaceThreads)
      before[e] += p.counts[static_cast<int64_t>(b) * words * 4 + e];
    __syncthreads();
  }
}

// Gradient of the logits, a warp per token.
template <int V>
__global__ void __launch_bounds__(256) k_route_backward(const RouteBackwardParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t t = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  if (t >= p.tokens) return;
  int choice = -1;
  float pull = 0.0f, w = 0.0f;  // lane j: expert, w_j dw_j and w_j of choice j
  if (lane < p.topk) {
    choice = p.chosen[t * p.topk + lane];
    if (choice >= p.experts) choice = -1;
    w = choice >= 0 ? p.weights[t * p.topk + lane] : 0.0f;
    pull = choice >= 0 ? w * p.dweights[t * p.topk + lane] : 0.0f;
  }
  const float inner = warp_sum_f32(pull);
  const bool any = __any_sync(0xffffffffu, choice >= 0);
  float prob[V], dl[V];
  if (p.renormalize || !any) {
#pragma unroll
    for (int v = 0; v < V; ++v) prob[v] = 0.0f;
  } else {
    float top = -INFINITY;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = v * 32 + lane;
      prob[v] = e < p.experts ? load_logit(p.logits, p.bf16, t * p.stride + e) : -INFINITY;
      top = prob[v] > top || prob[v] != prob[v] ? prob[v] : top;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float other = __shfl_xor_sync(0xffffffffu, top, o);
      top = other > top || other != other ? other : top;
    }
    float sum = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      prob[v] = v * 32 + lane < p.experts ? expf(prob[v] - top) : 0.0f;
      sum += prob[v];
    }
    sum = warp_sum_f32(sum);
#pragma unroll
    for (int v = 0; v < V; ++v) prob[v] /= sum;
  }
#pragma unroll
  for (int v = 0; v < V; ++v) dl[v] = 0.0f;
  for (int j = 0; j < p.topk; ++j) {
    const int e = __shfl_sync(0xffffffffu, choice, j);
    const float at = __shfl_sync(0xffffffffu, pull, j);
    const float wj = __shfl_sync(0xffffffffu, w, j);
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (e == v * 32 + lane) {
        dl[v] += at;
        if (p.renormalize) prob[v] += wj;
      }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = v * 32 + lane;
    if (e >= p.experts) continue;
    const float d = any ? dl[v] - prob[v] * inner : 0.0f;
    const int64_t at = t * p.experts + e;
    if (p.bf16)
      static_cast<uint16_t*>(p.dlogits)[at] = f32_to_bf16(d);
    else
      static_cast<float*>(p.dlogits)[at] = d;
  }
}

// ------------------------------------------------------------------------
// Gather: a warp per row, four words of a lane under way (65536 rows of 2048
// bf16 values: 52 us, 5.2 TB/s of writes).  Words V where bases and strides are
// whole 16-byte words, and what a row has behind its last word element by
// element; else all elements, of type E.

template <typename V, typename E>
__global__ void __launch_bounds__(kRowThreads) k_gather(const GatherParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t r = (static_cast<int64_t>(blockIdx.x) * kRowThreads + threadIdx.x) >> 5;
  if (r >= p.rows) return;
  int64_t t = p.row_tokens[r];
  if (t >= p.x_rows) t = -1;
  constexpr int kOf = sizeof(V) / sizeof(E);
  const int64_t n = p.dim / kOf;
  E* to = static_cast<E*>(p.y) + r * p.y_stride;
  const E* from = static_cast<const E*>(p.x) + (t >= 0 ? t * p.x_stride : 0);
  V* y = reinterpret_cast<V*>(to);
  if (t >= 0) {
    const V* x = reinterpret_cast<const V*>(from);
    int64_t i = lane;
    for (; i + 3 * 32 < n; i += 4 * 32) {
      const V a = x[i], b = x[i + 32], c = x[i + 64], d = x[i + 96];
      y[i] = a;
      y[i + 32] = b;
      y[i + 64] = c;
      y[i + 96] = d;
    }
    for (; i < n; i += 32) y[i] = x[i];
  } else {
    for (int64_t i = lane; i < n; i += 32) y[i] = V{};
  }
  if (n * kOf + lane < p.dim) to[n * kOf + lane] = t >= 0 ? from[n * kOf + lane] : E{};
  if (p.x_scale && lane == 0) p.y_scale[r] = t >= 0 ? p.x_scale[t] : 0.0f;
}

// ------------------------------------------------------------------------
// Combine: a block per token.

__device__ __forceinline__ int64_t slot_of(const CombineParams& p, int64_t pair) {
  const int64_t s = p.slots[pair];
  return s >= 0 && s < p.n_rows ? s : -1;
}

__global__ void __launch_bounds__(kRowThreads) k_combine_any(const CombineParams p) {
  const int64_t t = blockIdx.x;
  for (int64_t c = threadIdx.x; c < p.dim; c += kRowThreads) {
    float sum = 0.0f;
    for (int j = 0; j < p.topk; ++j) {
      const int64_t s = slot_of(p, t * p.topk + j);
      if (s < 0) continue;
      const float v = bf16_to_f32(p.rows[s * p.stride + c]);
      sum += p.weights ? p.weights[t * p.topk + j] * v : v;
    }
    p.y[t * p.dim + c] = f32_to_bf16(sum);
  }
}

// The same 16 bytes at a time, eight rows' words under way at once (333 tokens,
// 8 rows of 2048 values each: 3.0 us).
__global__ void __launch_bounds__(kRowThreads) k_combine(const CombineParams p) {
  const int64_t t = blockIdx.x;
  const int words = static_cast<int>(p.dim / 8);
  __shared__ int32_t slot[kMaxTopk];
  __shared__ float weight[kMaxTopk];
  if (threadIdx.x < p.topk) {
    slot[threadIdx.x] = static_cast<int32_t>(slot_of(p, t * p.topk + threadIdx.x));
    weight[threadIdx.x] = p.weights ? p.weights[t * p.topk + threadIdx.x] : 1.0f;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < words; i += blockDim.x) {
    float sum[8] = {};
    for (int j0 = 0; j0 < p.topk; j0 += 8) {
      uint4 word[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const bool some = j0 + j < p.topk && slot[j0 + j] >= 0;
        word[j] = make_uint4(0, 0, 0, 0);
        if (some)
          word[j] = reinterpret_cast<const uint4*>(
              p.rows + static_cast<int64_t>(slot[j0 + j]) * p.stride)[i];
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (j0 + j >= p.topk || slot[j0 + j] < 0) continue;
        float f[8];
        unpack8(word[j], f);
#pragma unroll
        for (int q = 0; q < 8; ++q) sum[q] += weight[j0 + j] * f[q];
      }
    }
    reinterpret_cast<uint4*>(p.y + t * p.dim)[i] = pack8(sum);
  }
}

// Zeros to the rows past the last group, shared among the blocks.  As the
// products read the offsets, each is at least the one before: the last group ends
// at the highest.
template <typename V>
__device__ __forceinline__ void zero_unused_rows(const CombineParams& p) {
  __shared__ uint32_t part_max[32];
  const int64_t n = p.dim * 2 / static_cast<int64_t>(sizeof(V));
  const int64_t last = p.experts > 0 ? max(p.offsets[p.experts], 0) : 0;
  if (last + blockIdx.x >= p.n_rows) return;  // no row for this block, whatever stands before
  uint32_t highest = 0;
  for (int e = threadIdx.x + 1; e <= p.experts; e += blockDim.x)
    highest = max(highest, static_cast<uint32_t>(max(p.offsets[e], 0)));
  const int64_t used = block_max(highest, part_max);
  for (int64_t r = used + blockIdx.x; r < p.n_rows; r += gridDim.x)
    for (int64_t i = threadIdx.x; i < n; i += blockDim.x)
      reinterpret_cast<V*>(p.drows)[r * n + i] = V{};
}

__global__ void __launch_bounds__(kRowThreads) k_combine_backward_any(const CombineParams p) {
  __shared__ float part[32];
  for (int64_t t = blockIdx.x; t < p.tokens; t += gridDim.x)
    for (int j = 0; j < p.topk; ++j) {
      const int64_t s = slot_of(p, t * p.topk + j);
      const float w = p.weights[t * p.topk + j];
      float dot = 0.0f;
      if (s >= 0)
        for (int64_t c = threadIdx.x; c < p.dim; c += kRowThreads) {
          const float dy = bf16_to_f32(p.dy[t * p.dy_stride + c]);
          dot += dy * bf16_to_f32(p.rows[s * p.stride + c]);
          p.drows[s * p.dim + c] = f32_to_bf16(w * dy);
        }
      dot = block_sum(dot, part);
      if (threadIdx.x == 0) p.dweights[t * p.topk + j] = dot;
      __syncthreads();
    }
  zero_unused_rows<uint16_t>(p);
}

// The same 16 bytes at a time: a block per token, eight rows at once.  The
// eight dot products are reduced together: at each of three exchanges a lane
// hands over half of its sums, so that a warp needs 9 exchanges for 8 sums.
// Bound by memory: 8192 tokens, 8 rows of 2048 values, one in twenty unused, 85 us,
// 6.6 TB/s.
__global__ void __launch_bounds__(kRowThreads) k_combine_backward(const CombineParams p) {
  __shared__ int32_t slot[kMaxTopk];
  __shared__ float weight[kMaxTopk];
  __shared__ float part[32][8];
  const int words = static_cast<int>(p.dim / 8);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = blockIdx.x;
  if (t < p.tokens) {
    if (threadIdx.x < p.topk) {
      slot[threadIdx.x] = static_cast<int32_t>(slot_of(p, t * p.topk + threadIdx.x));
      weight[threadIdx.x] = p.weights[t * p.topk + threadIdx.x];
    }
    __syncthreads();
    for (int j0 = 0; j0 < p.topk; j0 += 8) {
      float dot[8] = {};
      for (int i = threadIdx.x; i < words; i += blockDim.x) {
        uint4 word[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          word[j] = make_uint4(0, 0, 0, 0);
          if (j0 + j < p.topk && slot[j0 + j] >= 0)
            word[j] = reinterpret_cast<const uint4*>(
                p.rows + static_cast<int64_t>(slot[j0 + j]) * p.stride)[i];
        }
        float dy[8];
        unpack8(reinterpret_cast<const uint4*>(p.dy + t * p.dy_stride)[i], dy);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (j0 + j >= p.topk || slot[j0 + j] < 0) continue;
          float f[8], out[8];
          unpack8(word[j], f);
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            dot[j] += dy[q] * f[q];
            out[q] = weight[j0 + j] * dy[q];
          }
          reinterpret_cast<uint4*>(p.drows + static_cast<int64_t>(slot[j0 + j]) * p.dim)[i] =
              pack8(out);
        }
      }
      // lane bits 4, 3, 2 choose sums 4.., 2.., 1..
#pragma unroll
      for (int half = 4; half > 0; half >>= 1) {
        const int o = half * 4;
        const bool upper = lane & o;
#pragma unroll
        for (int j = 0; j < half; ++j) {
          const float give = upper ? dot[j] : dot[j + half];
          const float keep = upper ? dot[j + half] : dot[j];
          dot[j] = keep + __shfl_xor_sync(0xffffffffu, give, o);
        }
      }
      dot[0] += __shfl_xor_sync(0xffffffffu, dot[0], 2);
      dot[0] += __shfl_xor_sync(0xffffffffu, dot[0], 1);
      if ((lane & 3) == 0) part[warp][lane >> 2] = dot[0];
      __syncthreads();
      if (threadIdx.x < 8 && j0 + threadIdx.x < p.topk) {
        float sum = 0.0f;
        for (int w = 0; w < blockDim.x >> 5; ++w) sum += part[w][threadIdx.x];
        p.dweights[t * p.topk + j0 + threadIdx.x] = sum;
      }
      __syncthreads();
    }
  }
  zero_unused_rows<uint4>(p);
}

template <int V>
void route_at(const RouteParams& p, int blocks, cudaStream_t s) {
  k_route<V><<<blocks, kRouteWarps * 32, 0, s>>>(p);
}

template <int V>
void route_backward_at(const RouteBackwardParams& p, int blocks, cudaStream_t s) {
  k_route_backward<V><<<blocks, 256, 0, s>>>(p);
}

int grid_of(int64_t n) { return static_cast<int>(n < (1 << 30) ? n : (1 << 30)); }

bool on16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// Widest words that a call's rows and buffers allow: 8, 2 or 1 values.
int word_values(int64_t dim, std::initializer_list<const void*> at,
                std::initializer_list<int64_t> strides) {
  uintptr_t bytes = static_cast<uintptr_t>(2 * dim);
  for (const void* p : at) bytes |= reinterpret_cast<uintptr_t>(p);  // null counts as aligned
  for (int64_t s : strides) bytes |= static_cast<uintptr_t>(2 * s);
  return bytes % 16 == 0 ? 8 : bytes % 4 == 0 ? 2 : 1;
}

// Words per thread, threads per row, rows per block.  Eight values per thread
// as far as 512 threads reach (with one matrix read and many rows 16, so that
// as many bytes are under way), then 16 and 32; rows of few threads share a
// block of 256.
struct RowShape {
  int values;  // of a thread; 0: the row does not fit
  dim3 block;
};

RowShape row_shape(int64_t dim, int word, int at_first) {
  RowShape s{};
  if (dim == 0) return s;
  for (int values = at_first; values <= (word == 8 ? 32 : 16); values *= 2) {
    const int64_t words = dim / word, vecs = values / word;
    const int64_t threads = (words + 32 * vecs - 1) / (32 * vecs) * 32;
    if (threads > kMostRowThreads) continue;
    s.values = values;
    const unsigned rows = threads <= 128 ? 256 / static_cast<unsigned>(threads) : 1;
    s.block = dim3(static_cast<unsigned>(threads), rows);
    break;
  }
  return s;
}

template <typename W, int kVecs, bool kShift = false>
void norm_at(const NormParams& p, dim3 block, cudaStream_t s) {
  const int grid = grid_of((p.rows + block.y - 1) / block.y);
  if (!p.weight)
    k_rmsnorm<W, kVecs, false, true, kShift><<<grid, block, 0, s>>>(p);
  else if (p.e4m3)
    k_rmsnorm<W, kVecs, true, true, kShift><<<grid, block, 0, s>>>(p);
  else
    k_rmsnorm<W, kVecs, true, false, kShift><<<grid, block, 0, s>>>(p);
}

// Whether all rows of all buffers start at the same place in a 16-byte word.
bool same_shift(int64_t dim, const void* first, std::initializer_list<const void*> at,
                std::initializer_list<int64_t> strides) {
  for (const void* p : at)
    if (p && ((reinterpret_cast<uintptr_t>(p) ^ reinterpret_cast<uintptr_t>(first)) & 15)) return false;
  for (int64_t s : strides)
    if ((s - dim) % 8) return false;
  return true;
}

template <typename W, int kVecs, bool kShift = false>
void norm_backward_at(const NormBackwardParams& p, dim3 block, int blocks, cudaStream_t s) {
  const size_t smem = block.y > 1 ? 4 * static_cast<size_t>(p.dim) : 0;
  k_rmsnorm_backward<W, kVecs, kShift><<<blocks, block, smem, s>>>(p);
}

template <int kVecs, int kRing>
int backward_ring(const NormBackwardParams& p, dim3 block, int blocks, size_t bytes,
                  cudaStream_t s) {
  const cudaError_t err = allow_shared<k_rmsnorm_backward_ring<kVecs, kRing>>(kRingBytes);
  if (err != cudaSuccess) return err;
  k_rmsnorm_backward_ring<kVecs, kRing><<<blocks, block, bytes, s>>>(p);
  return cudaSuccess;
}

}  // namespace

int launch_rmsnorm(const NormParams& p, void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int word = word_values(p.dim, {p.x, p.residual, p.weight, p.h, p.y},
                               {p.x_stride, p.residual ? p.residual_stride : 0});
  const int at_first = !p.residual && p.rows >= kManyRows ? 16 : 8;
  const uintptr_t y_place = reinterpret_cast<uintptr_t>(p.y) * (p.e4m3 ? 2 : 1);
  if (word == 1 && p.dim >= kShiftDim && same_shift(p.dim, p.x, {p.residual, p.h, reinterpret_cast<const void*>(y_place)},
                              {p.x_stride, p.residual ? p.residual_stride : p.dim}) &&
      (reinterpret_cast<uintptr_t>(p.weight) & 3) == 0) {
    // a row touches at most this many words' values
    const RowShape shape = row_shape((p.dim + 14) / 8 * 8, 8, at_first);
    switch (shape.values) {
      case 8: norm_at<uint4, 1, true>(p, shape.block, s); return cudaGetLastError();
      case 16: norm_at<uint4, 2, true>(p, shape.block, s); return cudaGetLastError();
      case 32: norm_at<uint4, 4, true>(p, shape.block, s); return cudaGetLastError();
    }
  }
  const RowShape shape = row_shape(p.dim, word, at_first);
  const dim3 b = shape.block;
  switch (shape.values * 16 + word) {
    case 8 * 16 + 8: norm_at<uint4, 1>(p, b, s); break;
    case 16 * 16 + 8: norm_at<uint4, 2>(p, b, s); break;
    case 32 * 16 + 8: norm_at<uint4, 4>(p, b, s); break;
    case 8 * 16 + 2: norm_at<uint32_t, 4>(p, b, s); break;
    case 16 * 16 + 2: norm_at<uint32_t, 8>(p, b, s); break;
    case 8 * 16 + 1: norm_at<uint16_t, 8>(p, b, s); break;
    case 16 * 16 + 1: norm_at<uint16_t, 16>(p, b, s); break;
    default: k_rmsnorm_any<<<grid_of(p.rows), kRowThreads, 0, s>>>(p);
  }
  return cudaGetLastError();
}

int launch_rmsnorm_backward(const NormBackwardParams& p, int blocks, void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int word = word_values(p.dim, {p.dy, p.h, p.weight, p.dh, p.dx},
                               {p.dy_stride, p.h_stride, p.dh ? p.dh_stride : 0});
  const bool shifted = word == 1 && p.dim >= kShiftGradientDim &&
                       same_shift(p.dim, p.dy, {p.h, p.dh, p.dx},
                                  {p.dy_stride, p.h_stride, p.dh ? p.dh_stride : p.dim}) &&
                       (reinterpret_cast<uintptr_t>(p.weight) & 3) == 0;
  // 16 values per thread where that leaves a warp's worth: half the work of a
  // row's sum and of its addresses per value
  RowShape shape = shifted ? row_shape((p.dim + 14) / 8 * 8, 8, 8)
                           : row_shape(p.dim, word, word == 8 && p.dim >= 512 ? 16 : 8);
  const bool by_words = shifted && shape.values;
  if (shifted && !by_words) shape = row_shape(p.dim, word, 8);
  const dim3 b = shape.block;
  // a ring of four rows as far as it takes 48 KB, else of two
  const int64_t line = 6 * p.dim * b.y;  // bytes of the rows of all three tensors
  const int ring = 4 * line <= kRingBytes ? 4 : 2 * line <= kRingBytes ? 2 : 0;
  const size_t bytes = static_cast<size_t>(ring * line);
  if (shape.values) {
    // as many as are resident at once, 64 registers a thread or shared memory
    // allowing: 1024 threads an SM
    const int64_t resident = 152 * (1024 / static_cast<int64_t>(b.x * b.y));
    const int64_t most = (p.rows + b.y - 1) / b.y;
    if (resident < blocks) blocks = static_cast<int>(resident);
    if (most < blocks) blocks = static_cast<int>(most);
    if (by_words && blocks < most) {  // (blocks > 8 then)
      const int apart = b.y % 8 == 0 ? 1 : b.y % 4 == 0 ? 2 : b.y % 2 == 0 ? 4 : 8;
      blocks = blocks / apart * apart;
    }
  }
  int err = cudaSuccess;
  if (by_words) {
    switch (shape.values) {
      case 8: norm_backward_at<uint4, 1, true>(p, b, blocks, s); break;
      case 16: norm_backward_at<uint4, 2, true>(p, b, blocks, s); break;
      default: norm_backward_at<uint4, 4, true>(p, b, blocks, s);
    }
    k_sum_partials<<<grid_of((p.dim + 31) / 32), 1024, 0, s>>>(p.partial, blocks, p.dim, p.dweight);
    return cudaGetLastError();
  }
  switch (shape.values * 16 + word) {
    case 8 * 16 + 8:  // fewer than 512 values: the ring fits
      err = backward_ring<1, 4>(p, b, blocks, bytes, s);
      break;
    case 16 * 16 + 8:
      if (ring == 4)
        err = backward_ring<2, 4>(p, b, blocks, bytes, s);
      else if (ring == 2)
        err = backward_ring<2, 2>(p, b, blocks, bytes, s);
      else
        norm_backward_at<uint4, 2>(p, b, blocks, s);
      break;
    case 32 * 16 + 8: norm_backward_at<uint4, 4>(p, b, blocks, s); break;
    case 8 * 16 + 2: norm_backward_at<uint32_t, 4>(p, b, blocks, s); break;
    case 16 * 16 + 2: norm_backward_at<uint32_t, 8>(p, b, blocks, s); break;
    case 8 * 16 + 1: norm_backward_at<uint16_t, 8>(p, b, blocks, s); break;
    case 16 * 16 + 1: norm_backward_at<uint16_t, 16>(p, b, blocks, s); break;
    default: k_rmsnorm_backward_any<<<blocks, kRowThreads, 0, s>>>(p);
  }
  if (err != cudaSuccess) return err;
  k_sum_partials<<<grid_of((p.dim + 31) / 32), 1024, 0, s>>>(p.partial, blocks, p.dim, p.dweight);
  return cudaGetLastError();
}

int launch_route(const RouteParams& p, void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int blocks = (p.tokens + kRouteTokens - 1) / kRouteTokens;
  if (p.experts <= 64)
    route_at<2>(p, blocks, s);
  else if (p.experts <= 128)
    route_at<4>(p, blocks, s);
  else if (p.experts <= 256)
    route_at<8>(p, blocks, s);
  else
    route_at<32>(p, blocks, s);
  if (blocks > 1) {
    const int group = (blocks + kPlaceBlocks - 1) / kPlaceBlocks;
    k_route_place<<<(blocks + group - 1) / group, kPlaceThreads, 0, s>>>(p, blocks, group);
  }
  return cudaGetLastError();
}

int launch_route_backward(const RouteBackwardParams& p, void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int blocks = (p.tokens + 7) / 8;
  if (p.experts <= 64)
    route_backward_at<2>(p, blocks, s);
  else if (p.experts <= 128)
    route_backward_at<4>(p, blocks, s);
  else if (p.experts <= 256)
    route_backward_at<8>(p, blocks, s);
  else
    route_backward_at<32>(p, blocks, s);
  return cudaGetLastError();
}

int launch_gather(const GatherParams& p, void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int blocks = static_cast<int>((p.rows + kRowThreads / 32 - 1) / (kRowThreads / 32));
  const uintptr_t at = reinterpret_cast<uintptr_t>(p.x) | reinterpret_cast<uintptr_t>(p.y);
  const bool words = at % 16 == 0 && p.x_stride * p.size % 16 == 0 && p.y_stride * p.size % 16 == 0;
  if (p.size == 2) {
    if (words)
      k_gather<uint4, uint16_t><<<blocks, kRowThreads, 0, s>>>(p);
    else
      k_gather<uint16_t, uint16_t><<<blocks, kRowThreads, 0, s>>>(p);
  } else if (words) {
    k_gather<uint4, uint8_t><<<blocks, kRowThreads, 0, s>>>(p);
  } else {
    k_gather<uint8_t, uint8_t><<<blocks, kRowThreads, 0, s>>>(p);
  }
  return cudaGetLastError();
}

namespace {

// Threads for a row of 16-byte words: one word each up to 256.
int word_threads(int64_t dim) {
  const int64_t words = dim / 8;
  return words >= 256 ? 256 : words <= 32 ? 32 : static_cast<int>((words + 31) / 32 * 32);
}

}  // namespace

int launch_combine(const CombineParams& p, void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (p.dim % 8 == 0 && p.stride % 8 == 0 && on16(p.rows) && on16(p.y))
    k_combine<<<p.tokens, word_threads(p.dim), 0, s>>>(p);
  else
    k_combine_any<<<p.tokens, kRowThreads, 0, s>>>(p);
  return cudaGetLastError();
}

int launch_combine_backward(const CombineParams& p, void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  // without tokens there may still be rows to zero
  const int blocks = p.tokens > 0 ? p.tokens : grid_of(p.n_rows);
  if (p.dim % 8 == 0 && p.stride % 8 == 0 && p.dy_stride % 8 == 0 && on16(p.rows) && on16(p.dy) &&
      on16(p.drows))
    k_combine_backward<<<blocks, word_threads(p.dim), 0, s>>>(p);
  else
    k_combine_backward_any<<<blocks, kRowThreads, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace ciera
