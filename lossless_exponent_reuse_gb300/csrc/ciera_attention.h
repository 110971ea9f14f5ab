// ciera_attention.h -- launch parameters shared by the host API and the kernels
// of the attention half of a layer.  Not part of the public ABI.
#pragma once

#include <cstdint>

#include "ciera.h"
#include "ciera_internal.h"

namespace ciera {

constexpr int kExponentBias = 127;
constexpr int kLowestExponent = -100;   // of an e4m3 row
constexpr int kHighestExponent = 119;

// Tokens x heads of contiguous values.
struct Heads {
  const uint16_t* data;
  int64_t token;   // strides
  int64_t head;
  int64_t heads;
};

// One side (keys or values) of the pages.
struct Side {
  void* data;
  int64_t stride[3];              // page, place, head
  uint8_t* exponent;              // e4m3, else null
  int64_t exponent_stride[3];
};

struct RotaryParams {
  Heads q;                        // rotated into q_out
  uint16_t* out;
  int64_t out_token;
  int64_t out_head;
  Heads k, v;                     // append alone: into the pages
  Side key, value;
  const int32_t* positions;
  const int32_t* slots;           // append alone, else null
  const int64_t* turns;
  int32_t pairs;
  int32_t head_dim;
  int32_t interleaved;
  int32_t inverse;
  int32_t e4m3;
  float amplitude;
  int64_t tokens;
  int32_t pages;
  int32_t page_size;
};

struct PagesParams {
  const int32_t* cached;
  const int32_t* fresh;           // new tokens of each request
  const uint8_t* done;            // release
  int32_t requests;
  int32_t tokens;
  int32_t page_size;
  int32_t* table;
  int64_t table_stride;
  int64_t width;
  int32_t* stack;
  int32_t capacity;
  const int32_t* count;
  int32_t* count_out;
  int32_t* offsets;
  int32_t* context;
  int32_t* lengths;
  int32_t* positions;
  int32_t* slots;
};

// Division of a number below 2^31 by d: with 2^(l-1) < d <= 2^l and
// m = ceil(2^(31+l) / d) the product n m exceeds n 2^(31+l) / d by less than
// 2^(31+l) / d, so that its quotient is exact.
struct Divide {
  uint32_t by, multiplier;
  int32_t shift;
  Divide() = default;
  explicit Divide(uint32_t d) : by(d), shift(31) {
    while ((uint64_t(1) << (shift - 31)) < d) ++shift;
    multiplier = static_cast<uint32_t>(((uint64_t(1) << shift) + d - 1) / d);
  }
#ifdef __CUDACC__
  __device__ __forceinline__ int32_t operator()(int32_t n) const {
    return static_cast<int32_t>((static_cast<uint64_t>(static_cast<uint32_t>(n)) * multiplier) >>
                                shift);
  }
  __device__ __forceinline__ int32_t up(int32_t n) const {  // rounded up
    return (*this)(n + static_cast<int32_t>(by) - 1);
  }
#endif
};

struct AttendParams {
  const uint16_t* q;
  int64_t q_token, q_head;
  Side key, value;
  const int32_t* table;
  int64_t table_stride;
  int32_t keys_most;              // width * page_size
  const int32_t* offsets;
  const int32_t* context;
  uint16_t* o;
  int32_t tokens;
  int32_t requests;
  int32_t heads;                  // of keys and values
  int32_t group;                  // query heads to each
  int32_t head_dim;
  int32_t pages;
  int32_t page_size;
  int32_t e4m3;
  float scale;
  int64_t longest;
  int32_t unit_keys;              // keys of a unit of work
  Divide by_group, by_page, by_unit;
  int32_t blocks;                 // that share the work
  void* workspace;
  Control* ctl;
  uint64_t timeout_ns;
};

// Launchers.  Return a cudaError_t value.
int launch_rotary(const RotaryParams& p, void* stream);
int launch_assign_pages(const PagesParams& p, void* stream);
int launch_release_pages(const PagesParams& p, void* stream);
int launch_attend(const AttendParams& p, void* stream);
int64_t attend_workspace_bytes(int64_t q_heads, int64_t heads, int64_t head_dim);
// Attention in tiles of few rows (mma.sync), and of up to 256 (tcgen05), with
// p.blocks the SMs; false where a call's layout is not one that they take.  And the
// bytes of workspace that they want.
bool launch_attend_split(const AttendParams& p, void* stream, int* status);
int64_t split_workspace_bytes(int sms);
bool launch_attend_wide(const AttendParams& p, void* stream, int* status);
int64_t wide_workspace_bytes(int sms);

}  // namespace ciera
