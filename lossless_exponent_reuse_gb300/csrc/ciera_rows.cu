// ciera_rows.cu -- the row-wise operators of the mixture-of-experts layer:
// the norm with the residual's addition and its gradient, rows to e4m3, the
// router's choice with the expert order, and the combination of the experts'
// rows.
#include "ciera_moe_device.cuh"

namespace ciera {
namespace {

constexpr int kRowThreads = 256;

// ------------------------------------------------------------------------
// Norm: one block per row, the row read once for its sum of squares and
// again (from L1 or L2) for the outputs.

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

__global__ void __launch_bounds__(kRowThreads) k_sum_partials(const float* partial, int blocks,
                                                              int64_t dim, float* out) {
  const int64_t c = static_cast<int64_t>(blockIdx.x) * kRowThreads + threadIdx.x;
  if (c >= dim) return;
  float sum = 0.0f;
  for (int b = 0; b < blocks; ++b) sum += partial[b * dim + c];
  out[c] = sum;
}

// ------------------------------------------------------------------------
// Route.  A warp per token: its logits in registers, the softmax's maximum
// and sum, then topk rounds of "largest remaining, lowest index".
//
// The order: a token chooses an expert at most once, so a pair's rank among
// its block's pairs of the same expert is the number of earlier tokens of the
// block that chose it.  With a bit per token and expert (64 tokens a block)
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

__device__ __forceinline__ float load_logit(const void* logits, int bf16, int64_t i) {
  return bf16 ? bf16_to_f32(static_cast<const uint16_t*>(logits)[i])
              : static_cast<const float*>(logits)[i];
}

constexpr int kRouteWarps = 16;

// V: logits per lane (experts <= 32 V).
template <int V>
__global__ void __launch_bounds__(kRouteWarps * 32) k_route(const RouteParams p) {
  extern __shared__ unsigned long long bits[];  // per expert: tokens of this block
  for (int e = threadIdx.x; e < p.experts; e += blockDim.x) bits[e] = 0;
  __syncthreads();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kRouteTokens;
  for (int i = warp; i < kRouteTokens; i += kRouteWarps) {
    const int64_t t = first + i;
    if (t >= p.tokens) break;
    const bool live = !p.mask || p.mask[t] != 0;
    float l[V];
    uint32_t key[V];
    float top = -INFINITY;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = v * 32 + lane;
      l[v] = e < p.experts ? load_logit(p.logits, p.bf16, t * p.stride + e) : -INFINITY;
      key[v] = e < p.experts && live ? logit_key(l[v]) : 0u;
      if (key[v] <= kKeyMinusInf) key[v] = 0u;  // -inf is never chosen
      top = l[v] > top || l[v] != l[v] ? l[v] : top;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float other = __shfl_xor_sync(0xffffffffu, top, o);
      top = other > top || other != other ? other : top;
    }
    float sum = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (v * 32 + lane < p.experts) sum += expf(l[v] - top);
    sum = warp_sum_f32(sum);

    float mine = 0.0f, total = 0.0f;  // lane j: the weight of choice j
    int choice = -1;
    for (int j = 0; j < p.topk; ++j) {
      uint32_t best = 0;
#pragma unroll
      for (int v = 0; v < V; ++v) best = max(best, key[v]);
      const uint32_t all = __reduce_max_sync(0xffffffffu, best);
      if (all == 0) break;  // nothing left to choose
      uint32_t at = 0xFFFFFFFFu;
      float logit = 0.0f;
#pragma unroll
      for (int v = V - 1; v >= 0; --v)
        if (key[v] == all) {
          at = v * 32 + lane;
          logit = l[v];
        }
      const uint32_t e = __reduce_min_sync(0xffffffffu, at);
      logit = __shfl_sync(0xffffffffu, logit, e & 31);
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (e == v * 32 + lane) key[v] = 0u;
      const float w = expf(logit - top) / sum;
      total += w;
      if (lane == j) {
        mine = w;
        choice = static_cast<int>(e);
      }
      if (lane == 0) atomicOr(&bits[e], 1ull << i);
    }
    if (p.renormalize && choice >= 0) mine /= total;
    if (lane < p.topk) {
      p.weights[t * p.topk + lane] = mine;
      p.chosen[t * p.topk + lane] = choice;
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < p.experts; e += blockDim.x)
    p.counts[static_cast<int64_t>(blockIdx.x) * p.experts + e] =
        static_cast<uint8_t>(__popcll(bits[e]));
  const int64_t pairs = min(static_cast<int64_t>(kRouteTokens), p.tokens - first) * p.topk;
  for (int64_t i = threadIdx.x; i < pairs; i += blockDim.x) {
    const int e = p.chosen[first * p.topk + i];
    const int token = static_cast<int>(i / p.topk);
    p.slots[first * p.topk + i] = e < 0 ? -1 : __popcll(bits[e] & ((1ull << token) - 1));
  }
}

constexpr int kPlaceThreads = 256;

__global__ void __launch_bounds__(kPlaceThreads) k_route_place(const RouteParams p) {
  __shared__ int32_t base[kMaxExperts];    // rows before this block's, of each expert
  __shared__ int32_t total[kMaxExperts + 1];
  const int blocks = gridDim.x;
  for (int e = threadIdx.x; e < p.experts; e += kPlaceThreads) {
    int32_t before = 0, all = 0;
    for (int b = 0; b < blocks; ++b) {
      const int32_t n = p.counts[static_cast<int64_t>(b) * p.experts + e];
      all += n;
      if (b < static_cast<int>(blockIdx.x)) before += n;
    }
    base[e] = before;
    total[e] = all;
  }
  __syncthreads();
  if (threadIdx.x < 32) {  // exclusive sum of the totals: the offsets
    int32_t run = 0;
    for (int e0 = 0; e0 < p.experts; e0 += 32) {
      const int e = e0 + threadIdx.x;
      const int32_t n = e < p.experts ? total[e] : 0;
      int32_t s = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int32_t left = __shfl_up_sync(0xffffffffu, s, o);
        if (static_cast<int>(threadIdx.x) >= o) s += left;
      }
      if (e < p.experts) {
        base[e] += run + s - n;
        if (blockIdx.x == 0) p.offsets[e] = run + s - n;
      }
      run += __shfl_sync(0xffffffffu, s, 31);
    }
    if (threadIdx.x == 0) {
      total[p.experts] = run;
      if (blockIdx.x == 0) p.offsets[p.experts] = run;
    }
  }
  __syncthreads();
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kRouteTokens;
  const int64_t pairs = min(static_cast<int64_t>(kRouteTokens), p.tokens - first) * p.topk;
  const int32_t used = total[p.experts];
  for (int64_t i = threadIdx.x; i < pairs; i += kPlaceThreads) {
    const int64_t pair = first * p.topk + i;
    const int e = p.chosen[pair];
    if (e >= 0) {
      const int32_t slot = base[e] + p.slots[pair];
      p.slots[pair] = slot;
      p.row_tokens[slot] = static_cast<int32_t>(first + i / p.topk);
    }
    if (pair >= used) p.row_tokens[pair] = -1;  // rows past the last group
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
// Gather: a warp per row.  V bytes per access: 16 where rows and bases are
// 16-byte aligned, else the element's size.

template <typename V>
__global__ void __launch_bounds__(kRowThreads) k_gather(const GatherParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t r = (static_cast<int64_t>(blockIdx.x) * kRowThreads + threadIdx.x) >> 5;
  if (r >= p.rows) return;
  int64_t t = p.row_tokens[r];
  if (t >= p.x_rows) t = -1;
  const int64_t n = p.dim * p.size / static_cast<int64_t>(sizeof(V));
  V* y = static_cast<V*>(p.y) + r * n;
  if (t >= 0) {
    const V* x = reinterpret_cast<const V*>(static_cast<const unsigned char*>(p.x) +
                                            t * p.x_stride * p.size);
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

// Zeros to the rows past the last group, shared among the blocks.
__device__ __forceinline__ void zero_unused_rows(const CombineParams& p) {
  int64_t used = p.offsets[p.experts];
  used = used < 0 ? 0 : used;
  for (int64_t r = used + blockIdx.x; r < p.n_rows; r += gridDim.x)
    for (int64_t c = threadIdx.x; c < p.dim; c += blockDim.x) p.drows[r * p.dim + c] = 0;
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
  zero_unused_rows(p);
}

template <int V>
void route_at(const RouteParams& p, int blocks, cudaStream_t s) {
  k_route<V><<<blocks, kRouteWarps * 32, 8 * p.experts, s>>>(p);
}

template <int V>
void route_backward_at(const RouteBackwardParams& p, int blocks, cudaStream_t s) {
  k_route_backward<V><<<blocks, 256, 0, s>>>(p);
}

int grid_of(int64_t n) { return static_cast<int>(n < (1 << 30) ? n : (1 << 30)); }

}  // namespace

int launch_rmsnorm(const NormParams& p, void* stream) {
  k_rmsnorm_any<<<grid_of(p.rows), kRowThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
  return cudaGetLastError();
}

int launch_rmsnorm_backward(const NormBackwardParams& p, int blocks, void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  k_rmsnorm_backward_any<<<blocks, kRowThreads, 0, s>>>(p);
  k_sum_partials<<<grid_of((p.dim + kRowThreads - 1) / kRowThreads), kRowThreads, 0, s>>>(
      p.partial, blocks, p.dim, p.dweight);
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
  k_route_place<<<blocks, kPlaceThreads, 0, s>>>(p);
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
  if (at % 16 == 0 && p.dim * p.size % 16 == 0 && p.x_stride * p.size % 16 == 0)
    k_gather<uint4><<<blocks, kRowThreads, 0, s>>>(p);
  else if (p.size == 2)
    k_gather<uint16_t><<<blocks, kRowThreads, 0, s>>>(p);
  else
    k_gather<uint8_t><<<blocks, kRowThreads, 0, s>>>(p);
  return cudaGetLastError();
}

int launch_combine(const CombineParams& p, void* stream) {
  k_combine_any<<<p.tokens, kRowThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
  return cudaGetLastError();
}

int launch_combine_backward(const CombineParams& p, void* stream) {
  // without tokens there may still be rows to zero
  const int blocks = p.tokens > 0 ? p.tokens : grid_of(p.n_rows);
  k_combine_backward_any<<<blocks, kRowThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
  return cudaGetLastError();
}

}  // namespace ciera
