// ciera_moe.h -- launch parameters shared by the host API and the kernels of
// the mixture-of-experts operators.  Not part of the public ABI.
#pragma once

#include <cstdint>
#include <mutex>

#include "ciera.h"
#include "ciera_internal.h"

namespace ciera {

constexpr int kMaxExperts = 1024;
constexpr int kMaxTopk = 32;
constexpr int kRouteTokens = 32;        // tokens per block of k_route
constexpr int kNormBackwardBlocks = 760;  // most blocks of a norm's gradient: 5 per SM
constexpr int64_t kMoeScratch = 256;    // offset of the scratch behind the control block

// Limit of every bounded device-side wait (ciera_set_wait_timeout_ns).
uint64_t wait_timeout_ns();

// Held while a call enqueues launches that hand scratch memory on: of calls on
// one stream with the same scratch, from several host threads, each one's
// launches follow one another.
std::mutex& launches();

struct NormParams {
  const uint16_t* x;
  int64_t x_stride;
  const uint16_t* residual;  // may be null
  int64_t residual_stride;
  const uint16_t* weight;    // null: no norm, rows are quantised as they are
  int64_t rows;
  int64_t dim;
  float eps;
  void* y;
  int32_t e4m3;              // y is e4m3 with scale
  float* scale;
  uint16_t* h;               // may be null
  float* rstd;               // may be null
};

struct NormBackwardParams {
  const uint16_t* dy;
  int64_t dy_stride;
  const uint16_t* h;
  int64_t h_stride;
  const float* rstd;
  const uint16_t* weight;
  const uint16_t* dh;        // may be null
  int64_t dh_stride;
  int64_t rows;
  int64_t dim;
  uint16_t* dx;
  float* dweight;
  float* partial;            // blocks x dim
};

struct RouteParams {
  const void* logits;
  int32_t bf16;
  int64_t stride;
  const uint8_t* mask;       // may be null
  int32_t tokens;
  int32_t experts;
  int32_t topk;
  int32_t renormalize;
  float* weights;
  int32_t* chosen;
  int32_t* slots;
  int32_t* row_tokens;
  int32_t* offsets;
  uint8_t* counts;           // per block of tokens: pairs of each expert
};

// Bytes of a block's counts: whole words.
__host__ __device__ inline int count_stride(int experts) { return (experts + 3) & ~3; }

struct RouteBackwardParams {
  const float* dweights;
  const float* weights;
  const int32_t* chosen;
  const void* logits;
  int32_t bf16;
  int64_t stride;
  int32_t tokens;
  int32_t experts;
  int32_t topk;
  int32_t renormalize;
  void* dlogits;
};

struct GatherParams {
  const void* x;
  int64_t x_stride;
  int64_t x_rows;
  int32_t size;              // bytes of an element
  const float* x_scale;      // e4m3
  const int32_t* row_tokens;
  int64_t rows;
  int64_t dim;
  void* y;
  int64_t y_stride;
  float* y_scale;
};

struct CombineParams {
  const uint16_t* rows;
  int64_t stride;
  int64_t n_rows;
  const int32_t* slots;
  const float* weights;      // null: ones (forward only)
  int32_t tokens;
  int32_t topk;
  int64_t dim;
  uint16_t* y;               // forward
  const uint16_t* dy;        // gradient
  int64_t dy_stride;
  const int32_t* offsets;
  int32_t experts;
  uint16_t* drows;
  float* dweights;
};

// One product grouped by expert, D[row, feature]; which of the three it is
// says which of the operands is ragged.
enum ExpertOp : int32_t { kExpertForward = 0, kExpertDx = 1, kExpertDw = 2 };

struct ExpertParams {
  int32_t op;
  int32_t e4m3;
  int32_t gated;             // forward: gated unit; dx: its gradient (pre read)
  int32_t f32_out;           // dw
  int32_t accumulate;        // dw
  const void* x;             // forward: rows; dx: dy; dw: x
  int64_t x_stride;
  int64_t x_rows;
  const int32_t* row_tokens; // forward: may be null
  const void* w;             // forward, dx: weights; dw: dy
  int64_t w_stride;
  int64_t w_expert_stride;   // forward, dx
  const float* x_scale;
  const float* w_scale;
  const int32_t* offsets;
  int64_t rows;
  int32_t experts;
  int64_t n;                 // as in the public header
  int64_t k;
  const uint16_t* pre_in;    // dx, gated
  uint16_t* pre_out;         // forward, gated: may be null
  void* y;
  int64_t y_stride;          // dw
  int64_t y_expert_stride;   // dw
  Control* ctl;
  uint64_t timeout_ns;
};

// Launchers.  Return a cudaError_t value.
int launch_rmsnorm(const NormParams& p, void* stream);
int launch_rmsnorm_backward(const NormBackwardParams& p, int blocks, void* stream);
int launch_route(const RouteParams& p, void* stream);
int launch_route_backward(const RouteBackwardParams& p, void* stream);
int launch_gather(const GatherParams& p, void* stream);
int launch_combine(const CombineParams& p, void* stream);
int launch_combine_backward(const CombineParams& p, void* stream);
int launch_expert(const ExpertParams& p, void* stream);
// Address of the current device's control block.
int control_block(void** control);
// The tensor-core form; false when it cannot take these sizes and strides.
bool launch_expert_tc(const ExpertParams& p, void* stream, int* status);

}  // namespace ciera
