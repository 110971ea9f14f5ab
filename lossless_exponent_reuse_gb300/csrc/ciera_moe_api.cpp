// ciera_moe_api.cpp -- host side of the mixture-of-experts operators:
// argument checks and workspace layout.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "ciera.h"
#include "ciera_moe.h"

using namespace ciera;

namespace {

// Rows that 32-bit indexes can count with a tile's rows to spare.
constexpr int64_t kMaxRows = (int64_t(1) << 31) - 4096;
constexpr int64_t kMaxDim = int64_t(1) << 30;

bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

// A required buffer of elements of `size` bytes; may be null only when empty.
bool buffer(const void* p, int64_t elements, uintptr_t size) {
  return (p || elements == 0) && aligned(p, size);
}

// A matrix of `rows` rows of `dim` elements, `stride` apart.
bool matrix(const void* p, int64_t rows, int64_t dim, int64_t stride, uintptr_t size) {
  return rows >= 0 && dim >= 0 && rows <= kMaxRows && dim <= kMaxDim && stride >= dim &&
         stride <= (int64_t(1) << 40) && buffer(p, rows * dim, size);
}

int status_of(int cuda) { return cuda == cudaSuccess ? CIERA_OK : CIERA_E_CUDA; }

int64_t norm_backward_blocks(int64_t rows) {
  return rows < kNormBackwardBlocks ? rows : kNormBackwardBlocks;
}

int64_t route_blocks(int64_t tokens) { return (tokens + kRouteTokens - 1) / kRouteTokens; }

}  // namespace

namespace ciera {
std::mutex& launches() {
  static std::mutex held;
  return held;
}
}  // namespace ciera

extern "C" {

int64_t ciera_moe_workspace_bytes(int64_t tokens, int64_t experts, int64_t dim) {
  if (tokens < 0 || experts < 0 || dim < 0 || tokens > kMaxRows || experts > kMaxExperts ||
      dim > kMaxDim)
    return 0;
  const int64_t norm = 4 * norm_backward_blocks(tokens) * dim;
  const int64_t route = route_blocks(tokens) * count_stride(static_cast<int>(experts));
  const int64_t most = norm > route ? norm : route;
  return kMoeScratch + (most + 255) / 256 * 256;
}

int ciera_moe_workspace_init(void* workspace_dev, void* stream) {
  if (!workspace_dev || !aligned(workspace_dev, 16)) return CIERA_E_INVAL;
  return status_of(cudaMemsetAsync(workspace_dev, 0, static_cast<size_t>(kMoeScratch),
                                   static_cast<cudaStream_t>(stream)));
}

int ciera_moe_control(void** control_dev) {
  if (!control_dev) return CIERA_E_INVAL;
  return status_of(control_block(control_dev));
}

int ciera_rmsnorm(const uint16_t* x_dev, int64_t x_stride, const uint16_t* residual_dev,
                  int64_t residual_stride, const uint16_t* weight_dev, int64_t rows, int64_t dim,
                  float eps, void* y_dev, int y_type, float* scale_dev, uint16_t* h_dev,
                  float* rstd_dev, void* stream) {
  const bool e4m3 = y_type == CIERA_E4M3;
  if (!e4m3 && y_type != CIERA_BF16) return CIERA_E_INVAL;
  if (!matrix(x_dev, rows, dim, x_stride, 2) || !buffer(weight_dev, dim, 2) ||
      !buffer(y_dev, rows * dim, e4m3 ? 1 : 2) || !aligned(h_dev, 2) || !aligned(rstd_dev, 4) ||
      !(eps >= 0) || !std::isfinite(eps))
    return CIERA_E_INVAL;
  if (residual_dev && !matrix(residual_dev, rows, dim, residual_stride, 2)) return CIERA_E_INVAL;
  if (e4m3 ? !buffer(scale_dev, rows, 4) : scale_dev != nullptr) return CIERA_E_INVAL;
  // s may replace the residual in place, but only row for row
  if (h_dev && h_dev == residual_dev && residual_stride != dim) return CIERA_E_INVAL;
  if (rows == 0) return CIERA_OK;
  NormParams p{};
  p.x = x_dev;
  p.x_stride = x_stride;
  p.residual = residual_dev;
  p.residual_stride = residual_stride;
  // of no columns: not read, but not null, which stands for "no norm"
  p.weight = weight_dev ? weight_dev : reinterpret_cast<const uint16_t*>(rstd_dev);
  p.rows = rows;
  p.dim = dim;
  p.eps = eps;
  p.y = y_dev;
  p.e4m3 = e4m3;
  p.scale = scale_dev;
  p.h = h_dev;
  p.rstd = rstd_dev;
  return status_of(launch_rmsnorm(p, stream));
}

int ciera_quantize_rows(const uint16_t* x_dev, int64_t x_stride, int64_t rows, int64_t dim,
                        uint8_t* y_dev, float* scale_dev, void* stream) {
  if (!matrix(x_dev, rows, dim, x_stride, 2) || !buffer(y_dev, rows * dim, 1) ||
      !buffer(scale_dev, rows, 4))
    return CIERA_E_INVAL;
  if (rows == 0) return CIERA_OK;
  NormParams p{};
  p.x = x_dev;
  p.x_stride = x_stride;
  p.rows = rows;
  p.dim = dim;
  p.y = y_dev;
  p.e4m3 = 1;
  p.scale = scale_dev;
  return status_of(launch_rmsnorm(p, stream));
}

int ciera_rmsnorm_backward(const uint16_t* dy_dev, int64_t dy_stride, const uint16_t* h_dev,
                           int64_t h_stride, const float* rstd_dev, const uint16_t* weight_dev,
                           const uint16_t* dh_dev, int64_t dh_stride, int64_t rows, int64_t dim,
                           uint16_t* dx_dev, float* dweight_dev, void* workspace_dev,
                           int64_t workspace_bytes, void* stream) {
  if (!matrix(dy_dev, rows, dim, dy_stride, 2) || !matrix(h_dev, rows, dim, h_stride, 2) ||
      !buffer(rstd_dev, rows, 4) || !buffer(weight_dev, dim, 2) ||
      !buffer(dx_dev, rows * dim, 2) || !buffer(dweight_dev, dim, 4))
    return CIERA_E_INVAL;
  if (dh_dev && !matrix(dh_dev, rows, dim, dh_stride, 2)) return CIERA_E_INVAL;
  if (!workspace_dev || !aligned(workspace_dev, 16) ||
      workspace_bytes < ciera_moe_workspace_bytes(rows, 0, dim))
    return CIERA_E_INVAL;
  if (dim == 0) return CIERA_OK;
  if (rows == 0)
    return status_of(cudaMemsetAsync(dweight_dev, 0, static_cast<size_t>(4 * dim),
                                     static_cast<cudaStream_t>(stream)));
  NormBackwardParams p{};
  p.dy = dy_dev;
  p.dy_stride = dy_stride;
  p.h = h_dev;
  p.h_stride = h_stride;
  p.rstd = rstd_dev;
  p.weight = weight_dev;
  p.dh = dh_dev;
  p.dh_stride = dh_stride;
  p.rows = rows;
  p.dim = dim;
  p.dx = dx_dev;
  p.dweight = dweight_dev;
  p.partial = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace_dev) + kMoeScratch);
  std::lock_guard<std::mutex> together(launches());
  return status_of(
      launch_rmsnorm_backward(p, static_cast<int>(norm_backward_blocks(rows)), stream));
}

int ciera_route(const void* logits_dev, int logits_type, int64_t logits_stride,
                const uint8_t* token_mask_dev, int64_t tokens, int64_t experts, int topk,
                uint32_t flags, float* weights_dev, int32_t* chosen_dev, int32_t* slots_dev,
                int32_t* row_tokens_dev, int32_t* offsets_dev, void* workspace_dev,
                int64_t workspace_bytes, void* stream) {
  const bool bf16 = logits_type == CIERA_BF16;
  if (!bf16 && logits_type != CIERA_F32) return CIERA_E_INVAL;
  if (experts < 1 || experts > kMaxExperts || topk < 1 || topk > kMaxTopk || topk > experts ||
      tokens < 0 || tokens > kMaxRows / topk || (flags & ~CIERA_ROUTE_RENORMALIZE))
    return CIERA_E_INVAL;
  const int64_t pairs = tokens * topk;
  if (!matrix(logits_dev, tokens, experts, logits_stride, bf16 ? 2 : 4) ||
      !buffer(weights_dev, pairs, 4) || !buffer(chosen_dev, pairs, 4) ||
      !buffer(slots_dev, pairs, 4) || !buffer(row_tokens_dev, pairs, 4) ||
      !buffer(offsets_dev, experts + 1, 4))
    return CIERA_E_INVAL;
  if (!workspace_dev || !aligned(workspace_dev, 16) ||
      workspace_bytes < ciera_moe_workspace_bytes(tokens, experts, 0))
    return CIERA_E_INVAL;
  if (tokens == 0)
    return status_of(cudaMemsetAsync(offsets_dev, 0, static_cast<size_t>(4 * (experts + 1)),
                                     static_cast<cudaStream_t>(stream)));
  RouteParams p{};
  p.logits = logits_dev;
  p.bf16 = bf16;
  p.stride = logits_stride;
  p.mask = token_mask_dev;
  p.tokens = static_cast<int32_t>(tokens);
  p.experts = static_cast<int32_t>(experts);
  p.topk = topk;
  p.renormalize = (flags & CIERA_ROUTE_RENORMALIZE) != 0;
  p.weights = weights_dev;
  p.chosen = chosen_dev;
  p.slots = slots_dev;
  p.row_tokens = row_tokens_dev;
  p.offsets = offsets_dev;
  p.counts = static_cast<uint8_t*>(workspace_dev) + kMoeScratch;
  std::lock_guard<std::mutex> together(launches());
  return status_of(launch_route(p, stream));
}

int ciera_route_backward(const float* dweights_dev, const float* weights_dev,
                         const int32_t* chosen_dev, const void* logits_dev, int logits_type,
                         int64_t logits_stride, int64_t tokens, int64_t experts, int topk,
                         uint32_t flags, void* dlogits_dev, void* stream) {
  const bool bf16 = logits_type == CIERA_BF16;
  if (!bf16 && logits_type != CIERA_F32) return CIERA_E_INVAL;
  if (experts < 1 || experts > kMaxExperts || topk < 1 || topk > kMaxTopk || topk > experts ||
      tokens < 0 || tokens > kMaxRows / topk || (flags & ~CIERA_ROUTE_RENORMALIZE))
    return CIERA_E_INVAL;
  const int64_t pairs = tokens * topk;
  const uintptr_t size = bf16 ? 2 : 4;
  if (!matrix(logits_dev, tokens, experts, logits_stride, size) ||
      !buffer(dweights_dev, pairs, 4) || !buffer(weights_dev, pairs, 4) ||
      !buffer(chosen_dev, pairs, 4) || !buffer(dlogits_dev, tokens * experts, size))
    return CIERA_E_INVAL;
  if (tokens == 0) return CIERA_OK;
  RouteBackwardParams p{};
  p.dweights = dweights_dev;
  p.weights = weights_dev;
  p.chosen = chosen_dev;
  p.logits = logits_dev;
  p.bf16 = bf16;
  p.stride = logits_stride;
  p.tokens = static_cast<int32_t>(tokens);
  p.experts = static_cast<int32_t>(experts);
  p.topk = topk;
  p.renormalize = (flags & CIERA_ROUTE_RENORMALIZE) != 0;
  p.dlogits = dlogits_dev;
  return status_of(launch_route_backward(p, stream));
}

int ciera_gather_rows(const void* x_dev, int64_t x_stride, int64_t x_rows, int type,
                      const float* x_scale_dev, const int32_t* row_tokens_dev, int64_t rows,
                      int64_t dim, void* y_dev, float* y_scale_dev, void* stream) {
  return ciera_gather_rows_strided(x_dev, x_stride, x_rows, type, x_scale_dev, row_tokens_dev,
                                   rows, dim, y_dev, dim, y_scale_dev, stream);
}

int ciera_gather_rows_strided(const void* x_dev, int64_t x_stride, int64_t x_rows, int type,
                              const float* x_scale_dev, const int32_t* row_tokens_dev,
                              int64_t rows, int64_t dim, void* y_dev, int64_t y_stride,
                              float* y_scale_dev, void* stream) {
  const bool e4m3 = type == CIERA_E4M3;
  if (!e4m3 && type != CIERA_BF16) return CIERA_E_INVAL;
  const uintptr_t size = e4m3 ? 1 : 2;
  if (!matrix(x_dev, x_rows, dim, x_stride, size) ||
      !matrix(y_dev, rows, dim, y_stride, size) || !buffer(row_tokens_dev, rows, 4))
    return CIERA_E_INVAL;
  if (e4m3 ? !buffer(x_scale_dev, x_rows, 4) || !buffer(y_scale_dev, rows, 4)
           : x_scale_dev || y_scale_dev)
    return CIERA_E_INVAL;
  if (rows == 0 || (dim == 0 && !e4m3)) return CIERA_OK;
  GatherParams p{};
  p.x = x_dev;
  p.x_stride = x_stride;
  p.x_rows = x_rows;
  p.size = static_cast<int32_t>(size);
  p.x_scale = x_scale_dev;
  p.row_tokens = row_tokens_dev;
  p.rows = rows;
  p.dim = dim;
  p.y = y_dev;
  p.y_stride = y_stride;
  p.y_scale = y_scale_dev;
  return status_of(launch_gather(p, stream));
}

int ciera_combine(const uint16_t* rows_dev, int64_t rows_stride, int64_t rows,
                  const int32_t* slots_dev, const float* weights_dev, int64_t tokens, int topk,
                  int64_t dim, uint16_t* y_dev, void* stream) {
  if (topk < 1 || topk > kMaxTopk || tokens < 0 || tokens > kMaxRows / topk ||
      !matrix(rows_dev, rows, dim, rows_stride, 2) || !buffer(slots_dev, tokens * topk, 4) ||
      !aligned(weights_dev, 4) || !buffer(y_dev, tokens * dim, 2))
    return CIERA_E_INVAL;
  if (tokens == 0 || dim == 0) return CIERA_OK;
  CombineParams p{};
  p.rows = rows_dev;
  p.stride = rows_stride;
  p.n_rows = rows;
  p.slots = slots_dev;
  p.weights = weights_dev;
  p.tokens = static_cast<int32_t>(tokens);
  p.topk = topk;
  p.dim = dim;
  p.y = y_dev;
  return status_of(launch_combine(p, stream));
}

int ciera_combine_backward(const uint16_t* dy_dev, int64_t dy_stride, const uint16_t* rows_dev,
                           int64_t rows_stride, int64_t rows, const int32_t* slots_dev,
                           const float* weights_dev, const int32_t* offsets_dev, int64_t experts,
                           int64_t tokens, int topk, int64_t dim, uint16_t* drows_dev,
                           float* dweights_dev, void* stream) {
  if (topk < 1 || topk > kMaxTopk || tokens < 0 || tokens > kMaxRows / topk || experts < 0 ||
      experts > kMaxExperts || !matrix(dy_dev, tokens, dim, dy_stride, 2) ||
      !matrix(rows_dev, rows, dim, rows_stride, 2) || !buffer(slots_dev, tokens * topk, 4) ||
      !buffer(weights_dev, tokens * topk, 4) || !buffer(offsets_dev, experts + 1, 4) ||
      !buffer(drows_dev, rows * dim, 2) || !buffer(dweights_dev, tokens * topk, 4))
    return CIERA_E_INVAL;
  if (tokens == 0 && (rows == 0 || dim == 0)) return CIERA_OK;
  CombineParams p{};
  p.rows = rows_dev;
  p.stride = rows_stride;
  p.n_rows = rows;
  p.slots = slots_dev;
  p.weights = weights_dev;
  p.tokens = static_cast<int32_t>(tokens);
  p.topk = topk;
  p.dim = dim;
  p.dy = dy_dev;
  p.dy_stride = dy_stride;
  p.offsets = offsets_dev;
  p.experts = static_cast<int32_t>(experts);
  p.drows = drows_dev;
  p.dweights = dweights_dev;
  return status_of(launch_combine_backward(p, stream));
}

}  // extern "C"

namespace {

// What the three products share: the grouped rows, the experts, the sizes.
bool grouped(int64_t rows, int64_t experts, int64_t n, int64_t k, const int32_t* offsets,
             const int32_t* row_tokens, const void* workspace) {
  return rows >= 0 && rows <= kMaxRows && experts >= 0 && experts <= kMaxExperts && n >= 0 &&
         k >= 0 && n <= kMaxDim && k <= kMaxDim && offsets && aligned(offsets, 4) &&
         aligned(row_tokens, 4) && workspace && aligned(workspace, 16);
}

// Weights, or their gradient: `experts` matrices of rows x dim.
bool stacked(const void* p, int64_t experts, int64_t rows, int64_t dim, int64_t stride,
             int64_t expert_stride, uintptr_t size) {
  return matrix(p, experts == 0 ? 0 : rows, dim, stride, size) &&
         (experts <= 1 || expert_stride >= 0) && expert_stride <= (int64_t(1) << 40);
}

}  // namespace

extern "C" {

int ciera_expert_mm(const void* x_dev, int64_t x_stride, int64_t x_rows,
                    const int32_t* row_tokens_dev, const void* w_dev, int64_t w_stride,
                    int64_t w_expert_stride, const float* x_scale_dev, const float* w_scale_dev,
                    const int32_t* offsets_dev, int64_t rows, int64_t experts, int64_t n,
                    int64_t k, int type, uint32_t flags, uint16_t* y_dev, uint16_t* pre_dev,
                    void* workspace_dev, void* stream) {
  const bool e4m3 = type == CIERA_E4M3, gated = (flags & CIERA_GATED) != 0;
  if ((!e4m3 && type != CIERA_BF16) || (flags & ~CIERA_GATED)) return CIERA_E_INVAL;
  if (!grouped(rows, experts, n, k, offsets_dev, row_tokens_dev, workspace_dev))
    return CIERA_E_INVAL;
  const int64_t features = gated ? 2 * n : n;
  if (features > kMaxDim || !matrix(x_dev, x_rows, k, x_stride, e4m3 ? 1 : 2) ||
      (!row_tokens_dev && x_rows < rows) ||
      !stacked(w_dev, experts, features, k, w_stride, w_expert_stride, e4m3 ? 1 : 2) ||
      !buffer(y_dev, rows * n, 2) || !aligned(pre_dev, 2) || (pre_dev && !gated))
    return CIERA_E_INVAL;
  if (e4m3 ? !buffer(x_scale_dev, x_rows, 4) || !buffer(w_scale_dev, experts * features, 4)
           : x_scale_dev || w_scale_dev)
    return CIERA_E_INVAL;
  if (rows == 0 || n == 0) return CIERA_OK;
  ExpertParams p{};
  p.op = kExpertForward;
  p.e4m3 = e4m3;
  p.gated = gated;
  p.x = x_dev;
  p.x_stride = x_stride;
  p.x_rows = x_rows;
  p.row_tokens = row_tokens_dev;
  p.w = w_dev;
  p.w_stride = w_stride;
  p.w_expert_stride = w_expert_stride;
  p.x_scale = x_scale_dev;
  p.w_scale = w_scale_dev;
  p.offsets = offsets_dev;
  p.rows = rows;
  p.experts = static_cast<int32_t>(experts);
  p.n = n;
  p.k = k;
  p.pre_out = pre_dev;
  p.y = y_dev;
  p.ctl = static_cast<Control*>(workspace_dev);
  p.timeout_ns = wait_timeout_ns();
  return status_of(launch_expert(p, stream));
}

int ciera_expert_mm_dx(const uint16_t* dy_dev, int64_t dy_stride, const uint16_t* w_dev,
                       int64_t w_stride, int64_t w_expert_stride, const int32_t* offsets_dev,
                       int64_t rows, int64_t experts, int64_t n, int64_t k,
                       const uint16_t* pre_dev, uint16_t* dx_dev, void* workspace_dev,
                       void* stream) {
  if (!grouped(rows, experts, n, k, offsets_dev, nullptr, workspace_dev)) return CIERA_E_INVAL;
  if (!matrix(dy_dev, rows, n, dy_stride, 2) ||
      !stacked(w_dev, experts, n, k, w_stride, w_expert_stride, 2) || !aligned(pre_dev, 2) ||
      (pre_dev && 2 * k > kMaxDim) || !buffer(dx_dev, rows * k, 2))
    return CIERA_E_INVAL;
  if (rows == 0 || k == 0) return CIERA_OK;
  ExpertParams p{};
  p.op = kExpertDx;
  p.gated = pre_dev != nullptr;
  p.x = dy_dev;
  p.x_stride = dy_stride;
  p.x_rows = rows;
  p.w = w_dev;
  p.w_stride = w_stride;
  p.w_expert_stride = w_expert_stride;
  p.offsets = offsets_dev;
  p.rows = rows;
  p.experts = static_cast<int32_t>(experts);
  p.n = n;
  p.k = k;
  p.pre_in = pre_dev;
  p.y = dx_dev;
  p.ctl = static_cast<Control*>(workspace_dev);
  p.timeout_ns = wait_timeout_ns();
  return status_of(launch_expert(p, stream));
}

int ciera_expert_mm_dw(const uint16_t* dy_dev, int64_t dy_stride, const uint16_t* x_dev,
                       int64_t x_stride, const int32_t* offsets_dev, int64_t rows,
                       int64_t experts, int64_t n, int64_t k, void* dw_dev, int64_t dw_stride,
                       int64_t dw_expert_stride, int dw_type, uint32_t flags,
                       void* workspace_dev, void* stream) {
  const bool f32 = dw_type == CIERA_F32;
  if ((!f32 && dw_type != CIERA_BF16) || (flags & ~CIERA_ACCUMULATE)) return CIERA_E_INVAL;
  if (!grouped(rows, experts, n, k, offsets_dev, nullptr, workspace_dev))
    return CIERA_E_INVAL;
  if (!matrix(dy_dev, rows, n, dy_stride, 2) || !matrix(x_dev, rows, k, x_stride, 2) ||
      !stacked(dw_dev, experts, n, k, dw_stride, dw_expert_stride, f32 ? 4 : 2) ||
      (experts > 1 && dw_expert_stride < k))
    return CIERA_E_INVAL;
  if (experts == 0 || n == 0 || k == 0) return CIERA_OK;
  ExpertParams p{};
  p.op = kExpertDw;
  p.f32_out = f32;
  p.accumulate = (flags & CIERA_ACCUMULATE) != 0;
  p.x = x_dev;
  p.x_stride = x_stride;
  p.x_rows = rows;
  p.w = dy_dev;
  p.w_stride = dy_stride;
  p.offsets = offsets_dev;
  p.rows = rows;
  p.experts = static_cast<int32_t>(experts);
  p.n = n;
  p.k = k;
  p.y = dw_dev;
  p.y_stride = dw_stride;
  p.y_expert_stride = dw_expert_stride;
  p.ctl = static_cast<Control*>(workspace_dev);
  p.timeout_ns = wait_timeout_ns();
  return status_of(launch_expert(p, stream));
}

}  // extern "C"
