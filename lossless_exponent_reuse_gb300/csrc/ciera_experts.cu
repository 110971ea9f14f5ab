// ciera_experts.cu -- products grouped by expert, the form that takes any
// size, stride and alignment.
//
// All three products are D[row, col] = sum_c A[row, c] B[col, c]:
//   forward  rows: grouped rows     cols: features n   c: k
//   dx       rows: grouped rows     cols: k            c: features n
//   dw       rows: features n       cols: k            c: the group's rows
// One block computes a 64 x 64 tile with 32-bit sums; operands are converted
// to float on their way into shared memory, so that one loop serves bf16 and
// e4m3.  Bound by its 32-bit multiplications and their operands from shared
// memory, 22 TFLOP/s (65536 rows, 2048 to 2048: 25 ms; the tensor cores' form 0.32).  Grouped rows are cut into tiles per expert; tiles of the rows past
// the last group write zeros.
#include "ciera_moe_device.cuh"

namespace ciera {
namespace {

// Products keep a status there and nothing else, so that calls on different
// streams and in replayed graphs share it.
__device__ Control g_control;

constexpr int kTile = 64;
constexpr int kDepth = 16;
constexpr int kExpertThreads = 256;

// The tile `index` of the grouped rows: its group (experts for the rows past
// the last one), first row and row count; count 0 when there is no such tile.
struct RowTile {
  int32_t group, first, count;
};

__device__ RowTile find_row_tile(const ExpertParams& p, int64_t index) {
  int64_t seen = 0;
  int32_t at = 0;
  for (int32_t e = 0; e <= p.experts; ++e) {
    const int32_t end =
        e < p.experts ? clamp_offset(p.offsets[e + 1], at, static_cast<int32_t>(p.rows))
                      : static_cast<int32_t>(p.rows);
    const int32_t to = end < at ? at : end;
    const int64_t tiles = (static_cast<int64_t>(to) - at + kTile - 1) / kTile;
    if (index < seen + tiles) {
      const int32_t first = at + static_cast<int32_t>(index - seen) * kTile;
      return {e, first, min(kTile, to - first)};
    }
    seen += tiles;
    at = to;
  }
  return {0, 0, 0};
}

// x's row of grouped row r; -1: none (zeros).
__device__ __forceinline__ int64_t x_row_of(const ExpertParams& p, int64_t r) {
  const int64_t t = p.row_tokens ? p.row_tokens[r] : r;
  return t >= 0 && t < p.x_rows ? t : -1;
}

__device__ __forceinline__ float load_value(const void* p, int64_t i, int e4m3) {
  return e4m3 ? e4m3_to_f32(static_cast<const uint8_t*>(p)[i])
              : bf16_to_f32(static_cast<const uint16_t*>(p)[i]);
}

__device__ __forceinline__ float silu(float a) { return a / (1.0f + expf(-a)); }

template <int kOp, bool kGated>
__global__ void __launch_bounds__(kExpertThreads) k_expert_any(const ExpertParams p) {
  constexpr int kParts = kOp == kExpertForward && kGated ? 2 : 1;  // gate and up
  __shared__ float a[kDepth][kTile + 1];
  __shared__ float b[kParts][kDepth][kTile + 1];
  __shared__ RowTile tile;
  if (threadIdx.x == 0) {
    if (kOp == kExpertDw) {
      const int32_t e = blockIdx.z;
      int32_t at = 0;
      for (int32_t i = 0; i < e; ++i)
        at = clamp_offset(p.offsets[i + 1], at, static_cast<int32_t>(p.rows));
      const int32_t to = clamp_offset(p.offsets[e + 1], at, static_cast<int32_t>(p.rows));
      tile = {e, at, to - at};
    } else {
      tile = find_row_tile(p, blockIdx.x);
    }
  }
  __syncthreads();
  const RowTile x = tile;
  if (kOp != kExpertDw && x.count == 0) return;
  const int64_t row0 = kOp == kExpertDw ? static_cast<int64_t>(blockIdx.x) * kTile : x.first;
  const int64_t row_end = kOp == kExpertDw ? p.n : x.first + static_cast<int64_t>(x.count);
  const int64_t cols = kOp == kExpertForward ? p.n : p.k;
  const bool unused = kOp != kExpertDw && x.group == p.experts;
  const int64_t depth = unused ? 0 : kOp == kExpertForward ? p.k : kOp == kExpertDx ? p.n : x.count;
  const int64_t expert = static_cast<int64_t>(x.group) * p.w_expert_stride;

  const int tr = threadIdx.x / 16, tc = threadIdx.x % 16;
  // (a grid has 65535 columns of blocks at most)
  for (int64_t col0 = static_cast<int64_t>(blockIdx.y) * kTile; col0 < cols;
       col0 += static_cast<int64_t>(gridDim.y) * kTile) {
    float acc[kParts][4][4] = {};
    for (int64_t d0 = 0; d0 < depth; d0 += kDepth) {
      for (int i = threadIdx.x; i < kTile * kDepth; i += kExpertThreads) {
        // neighbouring threads read neighbouring addresses of either operand
        const int da = kOp == kExpertDw ? i / kTile : i % kDepth;
        const int ra = kOp == kExpertDw ? i % kTile : i / kDepth;
        const int64_t r = row0 + ra, d = d0 + da;
        float v = 0.0f;
        if (r < row_end && d < depth) {
          if (kOp == kExpertDw) {
            v = load_value(p.w, (x.first + d) * p.w_stride + r, 0);
          } else {
            const int64_t t = kOp == kExpertForward ? x_row_of(p, r) : r;
            if (t >= 0) v = load_value(p.x, t * p.x_stride + d, p.e4m3);
          }
        }
        a[da][ra] = v;
        const int db = kOp == kExpertForward ? i % kDepth : i / kTile;
        const int cb = kOp == kExpertForward ? i / kDepth : i % kTile;
        const int64_t c = col0 + cb, dd = d0 + db;
#pragma unroll
        for (int part = 0; part < kParts; ++part) {
          float w = 0.0f;
          if (c < cols && dd < depth) {
            if (kOp == kExpertForward)
              w = load_value(p.w, expert + (c + part * p.n) * p.w_stride + dd, p.e4m3);
            else if (kOp == kExpertDx)
              w = load_value(p.w, expert + dd * p.w_stride + c, 0);
            else
              w = load_value(p.x, (x.first + dd) * p.x_stride + c, 0);
          }
          b[part][db][cb] = w;
        }
      }
      __syncthreads();
#pragma unroll
      for (int d = 0; d < kDepth; ++d)
#pragma unroll
        for (int part = 0; part < kParts; ++part)
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
              acc[part][i][j] += a[d][tr * 4 + i] * b[part][d][tc + 16 * j];
      __syncthreads();
    }

#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t r = row0 + tr * 4 + i;
      if (r >= row_end) continue;
      float row_scale = 1.0f;
      if (kOp == kExpertForward && p.e4m3 && !unused) {
        const int64_t t = x_row_of(p, r);
        row_scale = t >= 0 ? p.x_scale[t] : 0.0f;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t c = col0 + tc + 16 * j;
        if (c >= cols) continue;
        if (kOp == kExpertDw) {
          const int64_t at = x.group * p.y_expert_stride + r * p.y_stride + c;
          float v = acc[0][i][j];
          if (p.f32_out) {
            float* out = static_cast<float*>(p.y) + at;
            *out = p.accumulate ? *out + v : v;
          } else {
            uint16_t* out = static_cast<uint16_t*>(p.y) + at;
            *out = f32_to_bf16(p.accumulate ? bf16_to_f32(*out) + v : v);
          }
          continue;
        }
        uint16_t* y = static_cast<uint16_t*>(p.y);
        if (kOp == kExpertForward) {
          float v = acc[0][i][j], up = kParts == 2 ? acc[kParts - 1][i][j] : 0.0f;
          if (p.e4m3 && !unused) {
            const float* ws = p.w_scale + static_cast<int64_t>(x.group) * kParts * p.n;
            v *= row_scale * ws[c];
            if (kParts == 2) up *= row_scale * ws[c + p.n];
          }
          if (kParts == 2) {
            if (p.pre_out) {
              p.pre_out[r * 2 * p.n + c] = f32_to_bf16(v);
              p.pre_out[r * 2 * p.n + p.n + c] = f32_to_bf16(up);
            }
            v = silu(v) * up;
          }
          y[r * p.n + c] = f32_to_bf16(v);
        } else if (kGated) {
          float dg = 0.0f, du = 0.0f;
          if (!unused) {  // pre of an unused row is not read
            const float g = bf16_to_f32(p.pre_in[r * 2 * p.k + c]);
            const float u = bf16_to_f32(p.pre_in[r * 2 * p.k + p.k + c]);
            const float s = 1.0f / (1.0f + expf(-g));
            dg = acc[0][i][j] * u * s * (1.0f + g * (1.0f - s));
            du = acc[0][i][j] * g * s;
          }
          y[r * 2 * p.k + c] = f32_to_bf16(dg);
          y[r * 2 * p.k + p.k + c] = f32_to_bf16(du);
        } else {
          y[r * p.k + c] = f32_to_bf16(acc[0][i][j]);
        }
      }
    }
  }
}

int64_t tiles_of(int64_t n) { return (n + kTile - 1) / kTile; }

}  // namespace

int control_block(void** control) { return cudaGetSymbolAddress(control, g_control); }

int launch_expert(const ExpertParams& p, void* stream) {
  int status = cudaSuccess;
  if (launch_expert_tc(p, stream, &status)) return status;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int64_t col_tiles = tiles_of(p.op == kExpertForward ? p.n : p.k);
  const unsigned grid_y = static_cast<unsigned>(col_tiles < 65535 ? col_tiles : 65535);
  if (p.op == kExpertDw) {
    const dim3 grid(static_cast<unsigned>(tiles_of(p.n)), grid_y,
                    static_cast<unsigned>(p.experts));
    k_expert_any<kExpertDw, false><<<grid, kExpertThreads, 0, s>>>(p);
    return cudaGetLastError();
  }
  // Group sizes are known on the device only: at most one partial tile for
  // each group that has rows and one for the rows past the last group.
  const int64_t groups = p.experts + 1 < p.rows ? p.experts + 1 : p.rows;
  const dim3 grid(static_cast<unsigned>(p.rows / kTile + groups), grid_y);
  if (p.op == kExpertForward) {
    if (p.gated)
      k_expert_any<kExpertForward, true><<<grid, kExpertThreads, 0, s>>>(p);
    else
      k_expert_any<kExpertForward, false><<<grid, kExpertThreads, 0, s>>>(p);
  } else {
    if (p.gated)
      k_expert_any<kExpertDx, true><<<grid, kExpertThreads, 0, s>>>(p);
    else
      k_expert_any<kExpertDx, false><<<grid, kExpertThreads, 0, s>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace ciera
