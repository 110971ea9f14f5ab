// ciera_attend_split.cu -- attention of few rows a head over pages.
//
// Bound by memory: every key and value is read once, for all query heads that
// share it.  Four warps of a block take 16 keys each of a unit of 64, on their
// own: each has a ring of stages in shared memory that its lanes fill by
// asynchronous copies, a row of a page at a time, some 16 KB ahead, and joins the
// others at the end of a tile alone.  64 requests of some 4200 keys on average, 16
// heads: 322 us, 6.9 TB/s; in e4m3 213 us, 5.2 TB/s, where issue slots are 60 % used
// (widening takes as many as the products); 4 heads with 8 query heads each 97 us.
//
// The products have the keys as rows and the queries as columns, S^T = K Q^T of
// 16 x 8, so that eight rows (8 query heads, say) cost one instruction per 16
// values of the heads; the weights' fragments are transposed in registers
// (movmatrix) for O^T = V^T P^T, whose values come transposed from shared memory
// (ldmatrix).  mma.sync does: at the rate of memory it is idle.
//
// e4m3 keys are widened to fp16, which holds them exactly, on their way into the
// fragments; queries are fp16 too, scaled by a power of two per row that brings its
// largest finite value to 2^13 or more, so that they lose 2^-38 of it at most (of a row
// whose largest is below 2^-113, which the power's range stops short, 2^-25 of it, and of
// one of bf16's subnormals 2^-18).  The row's power and the scale go on its scores first,
// then the key's power; where the first are beyond 2^96, and a score might pass 32 bits
// between the two (with a scale of 1 / 11, rows of 2^112 and more), the row is computed
// value by value.
// Values go to bf16, whose weights have the range that rows of any exponents
// want: a value's exponent goes on its weight's before a maximum of their own is
// taken (the sum has the scores' maximum).
//
// The running maximum moves only where a score passes it by 2^8 (weights are at
// most 256, which 8 bits of mantissa hold as well as 1): most units then need
// neither the maximum over the lanes nor the sums' scaling.  Weights are rounded to
// bf16 (2^-8 of each at most, as often up as down), the values' own type, whose range
// they need; their sum is of the 32-bit ones.
#include "ciera_attend_device.cuh"
#include "ciera_device.cuh"

namespace ciera {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kUnitKeys = 64;
constexpr int kWarpKeys = kUnitKeys / kWarps;
constexpr float kSlack = 8.0f;
constexpr int kMostPerSm = 3;
constexpr int kMostPartValues = 4096 + 96;  // floats of a part: rows by values, sums, maxima

__device__ __forceinline__ void ldsm(uint32_t addr, uint32_t (&v)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm_t(uint32_t addr, uint32_t (&v)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t transpose(uint32_t v) {
  uint32_t t;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(t) : "r"(v));
  return t;
}
template <bool kHalf>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (kHalf)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Two e4m3 values of the low (0) or high (1) half of a word, as fp16.
template <int kHigh>
__device__ __forceinline__ uint32_t widen(uint32_t v) {
  uint32_t h;
  if (kHigh)
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, hi;\n\t}"
        : "=r"(h)
        : "r"(v));
  else
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}"
        : "=r"(h)
        : "r"(v));
  return h;
}
__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
  uint32_t v;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(v) : "f"(hi), "f"(lo));
  return v;
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

// kDim: values of a row in shared memory, those past the head's own zeros.
// kBlocks: of 8 rows of a tile.
template <int kDim, int kBlocks, bool kE4m3>
struct Form {
  static constexpr int kRows = 8 * kBlocks;
  static constexpr int kRowBytes = kDim * (kE4m3 ? 1 : 2);
  static constexpr int kPieces = kRowBytes / 16;
  static constexpr int kSideBytes = kWarpKeys * kRowBytes;
  static constexpr int kStageBytes = 2 * kSideBytes;
  static constexpr int kRingBytes = 16 * 1024;   // of a warp
  static constexpr int kStages = kStageBytes > kRingBytes / 2 ? 3 : kRingBytes / kStageBytes;
  static constexpr int kQueryStride = kDim + 8;      // 16-bit values; eight rows in different banks
  static constexpr int kSumStride = kDim + 4;        // floats, likewise
  static constexpr int kQueryBytes = kRows * kQueryStride * 2;
  static constexpr int kWarpBytes = kStages * kStageBytes;
  static constexpr int kSumBytes = kWarps * kRows * kSumStride * 4;
  static constexpr int kSmem =
      kQueryBytes + (kWarps * kWarpBytes > kSumBytes ? kWarps * kWarpBytes : kSumBytes);
  // blocks of an SM: what shared memory and registers hold (64 requests in two blocks
  // of 24 KB rings and three of 16, when either took longer: bf16 366, 360 us, 4 heads 109,
  // 105; e4m3 268, 224)
  static constexpr int kPerSm = kDim > 128 ? 1 : kBlocks == 1 ? kMostPerSm : 2;
  static constexpr int kPartValues = kRows * (kDim + 3);
  static constexpr int kSteps = kDim / 16;
  static constexpr bool kKeep = kSteps * kBlocks <= 16;  // queries' fragments in registers
  static_assert(kPartValues <= kMostPartValues, "a part's place in the workspace");
};

// 2^(m - most), of maxima; 1 of none.
__device__ __forceinline__ float since(float m, float most) {
  return most == minus_infinity() ? 1.0f : exp2_fast(m - most);
}

// Bytes from a row's start at which its 16-byte piece lies: eight rows' pieces
// of one place are in different banks.
template <int kPieces>
__device__ __forceinline__ int piece_at(int row, int piece) {
  return kPieces >= 8 ? ((piece ^ (row & 7)) << 4) : ((piece ^ ((row >> 1) & (kPieces - 1))) << 4);
}

struct Shared {
  Share share;
  int64_t part[kWarps + 1];
  float query_scale[32];         // of a score, with the row's power of two
  uint32_t large[kWarps];        // a warp's own rows that are computed value by value
  int32_t seen[32];              // keys that a row sees
  // maxima of the values' weights and of the scores (bf16: the same), sums
  float most[kWarps][32], score[kWarps][32], sum[kWarps][32];
  uint32_t again;                // rows that something out of their sight may have spoilt
};

template <int kDim, int kBlocks, bool kE4m3>
__global__ void __launch_bounds__(kThreads) k_attend_split(const AttendParams p) {
  using F = Form<kDim, kBlocks, kE4m3>;
  extern __shared__ __align__(16) unsigned char raw[];
  __shared__ Shared sh;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int blocks = gridDim.x, block = blockIdx.x;
  const int column = lane & 3, line = lane >> 2;   // of a fragment
  uint16_t* queries = reinterpret_cast<uint16_t*>(raw);
  unsigned char* ring = raw + F::kQueryBytes;
  const uint32_t own_ring = smem_addr(ring) + warp * F::kWarpBytes;
  float* sums = reinterpret_cast<float*>(ring);
  Joint* joint = reinterpret_cast<Joint*>(p.workspace) + block;
  float* parts = reinterpret_cast<float*>(reinterpret_cast<Joint*>(p.workspace) + blocks);

  find_share<F::kRows, kThreads>(p, block, blocks, sh.part, &sh.share);
  Walk<F::kRows> walk(p, sh.share);
  Segment seg;
  bool left_joint = false;
  const int size = kE4m3 ? 1 : 2;
  const int pieces = p.head_dim * size / 16;       // that a row has

  while (walk.next(p, &seg)) {
    const int32_t row0 = seg.tile * F::kRows;
    // ---- queries: a warp a row
    if (threadIdx.x == 0) sh.again = 0;
    uint32_t large = 0;
    for (int r = warp; r < F::kRows; r += kWarps) {
      const bool live = r < seg.rows;
      const uint16_t* q = query_row(p, seg.request.first, seg.head, row0 + (live ? r : 0));
      uint16_t v[kDim / 32];
      uint32_t most = 0;         // of the finite values
#pragma unroll
      for (int i = 0; i < kDim / 32; ++i) {
        const int d = lane + 32 * i;
        v[i] = live && d < p.head_dim ? q[d] : 0;
        const uint32_t size = v[i] & 0x7FFFu;
        most = max(most, size < 0x7F80u ? size : 0);
      }
      float by = 1.0f, scale = p.scale * kLog2e;
      if (kE4m3) {
        // the largest value to 2^13 .. 2^14
        most = __reduce_max_sync(0xffffffffu, most);
        int e = static_cast<int>(most >> 7) - 127 - 13;
        e = most == 0 ? 0 : e < -126 ? -126 : e;
        by = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
        scale *= __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
        // (a product is below 2^14 448 256 < 2^31)
        if (live && fabsf(scale) > 0x1p96f) large |= 1u << r;
      }
#pragma unroll
      for (int i = 0; i < kDim / 32; ++i) {
        uint16_t w = v[i];
        if (kE4m3) w = static_cast<uint16_t>(pack_half(bf16_to_f32(v[i]) * by, 0.0f));
        queries[r * F::kQueryStride + lane + 32 * i] = w;
      }
      if (lane == 0) {
        sh.query_scale[r] = scale;
        sh.seen[r] = live ? seen_keys(seg.request, p.by_group(row0 + r)) : 0;
      }
    }
    if (kE4m3 && lane == 0) sh.large[warp] = large;
    __syncthreads();
    float scale[kBlocks][2], top[kBlocks][2], high[kBlocks][2], sum[kBlocks][2];
    int32_t seen[kBlocks][2];
    int32_t least = 0x7FFFFFFF;
#pragma unroll
    for (int b = 0; b < kBlocks; ++b)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int r = b * 8 + 2 * column + j;
        scale[b][j] = sh.query_scale[r];
        seen[b][j] = sh.seen[r];
        if (r < seg.rows) least = min(least, seen[b][j]);
        top[b][j] = high[b][j] = minus_infinity();
        sum[b][j] = 0.0f;
      }
    least = __reduce_min_sync(0xffffffffu, least);  // all rows see the keys before
    // queries' fragments of one step: bf16 in the heads' order; of e4m3 a lane has four
    // neighbouring values of a row, which a word of keys has too
    const auto query = [&](int step, int b, uint32_t& b0, uint32_t& b1) {
      const uint16_t* row = queries + (b * 8 + line) * F::kQueryStride + step * 16;
      if (kE4m3) {
        const uint2 w = *reinterpret_cast<const uint2*>(row + 4 * column);
        b0 = w.x;
        b1 = w.y;
      } else {
        b0 = *reinterpret_cast<const uint32_t*>(row + 2 * column);
        b1 = *reinterpret_cast<const uint32_t*>(row + 2 * column + 8);
      }
    };
    uint32_t qf[F::kKeep ? F::kSteps : 1][F::kKeep ? kBlocks : 1][2];
    if (F::kKeep)
#pragma unroll
      for (int s = 0; s < F::kSteps; ++s)
#pragma unroll
        for (int b = 0; b < kBlocks; ++b)
          query(s, b, qf[F::kKeep ? s : 0][F::kKeep ? b : 0][0],
                qf[F::kKeep ? s : 0][F::kKeep ? b : 0][1]);
    float o[F::kSteps][kBlocks][4] = {};

    // ---- this warp's units
    const int units = seg.to - seg.from;
    const int32_t key0 = seg.from * kUnitKeys + warp * kWarpKeys;
    const int64_t head_k = seg.head * p.key.stride[2], head_v = seg.head * p.value.stride[2];
    // Lanes 0 to 15 know where the keys of a unit begin, 16 to 31 where its values; -1:
    // zeros.
    const auto locate = [&](int unit) -> int64_t {
      const int32_t key = key0 + unit * kUnitKeys + (lane & 15);
      if (unit >= units || key >= seg.keys) return -1;
      const int32_t at = p.by_page(key), page = page_at(p, seg.index, at);
      if (page < 0) return -1;
      const int32_t place = key - at * p.page_size;
      return lane < 16 ? page * p.key.stride[0] + place * p.key.stride[1] + head_k
                       : page * p.value.stride[0] + place * p.value.stride[1] + head_v;
    };
    const auto exponent_of = [&](int unit) -> uint32_t {
      const int32_t key = key0 + unit * kUnitKeys + (lane & 15);
      if (unit >= units || key >= seg.keys) return kExponentBias;
      const int32_t at = p.by_page(key), page = page_at(p, seg.index, at);
      if (page < 0) return kExponentBias;
      const int32_t place = key - at * p.page_size;
      const Side& s = lane < 16 ? p.key : p.value;
      return s.exponent[page * s.exponent_stride[0] + place * s.exponent_stride[1] +
                        seg.head * s.exponent_stride[2]];
    };
    const auto issue = [&](int unit, int64_t where) {
      if (unit < units) {
        const uint32_t to = own_ring + (unit % F::kStages) * F::kStageBytes;
#pragma unroll
        for (int side = 0; side < 2; ++side)
#pragma unroll
          for (int i = 0; i < kWarpKeys * F::kPieces / 32; ++i) {
            const int at = i * 32 + lane, row = at / F::kPieces, piece = at % F::kPieces;
            const int64_t from = __shfl_sync(0xffffffffu, where, side * 16 + row);
            const unsigned char* base =
                static_cast<const unsigned char*>(side ? p.value.data : p.key.data);
            const bool some = from >= 0 && piece < pieces;
            copy16(to + side * F::kSideBytes + row * F::kRowBytes + piece_at<F::kPieces>(row, piece),
                   some ? base + from * size + piece * 16 : p.workspace, some ? 16 : 0);
          }
      }
      copy_commit();
    };
#pragma unroll 1
    for (int u = 0; u < F::kStages; ++u) issue(u, locate(u));
    int64_t where = locate(F::kStages);
    uint32_t exponent = kE4m3 ? exponent_of(0) : 0;

#pragma unroll 1
    for (int u = 0; u < units; ++u) {
      copy_wait<F::kStages - 1>();
      __syncwarp();
      const uint32_t keys_at = own_ring + (u % F::kStages) * F::kStageBytes;
      const uint32_t values_at = keys_at + F::kSideBytes;
      // ---- scores: 16 keys by 8 rows a block
      float s[kBlocks][4] = {};
      if (kE4m3) {
#pragma unroll
        for (int step = 0; step < F::kSteps; step += 2) {
          uint32_t w[4];
          const int row = lane & 15;
          ldsm(keys_at + row * F::kRowBytes + piece_at<F::kPieces>(row, step + (lane >> 4)), w);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t a[4] = {widen<0>(w[2 * h]), widen<0>(w[2 * h + 1]), widen<1>(w[2 * h]),
                                   widen<1>(w[2 * h + 1])};
#pragma unroll
            for (int b = 0; b < kBlocks; ++b) {
              uint32_t b0, b1;
              if (F::kKeep) {
                b0 = qf[F::kKeep ? step + h : 0][F::kKeep ? b : 0][0];
                b1 = qf[F::kKeep ? step + h : 0][F::kKeep ? b : 0][1];
              } else {
                query(step + h, b, b0, b1);
              }
              mma<true>(s[b], a, b0, b1);
            }
          }
        }
      } else {
#pragma unroll
        for (int step = 0; step < F::kSteps; ++step) {
          uint32_t a[4];
          const int row = lane & 15;
          ldsm(keys_at + row * F::kRowBytes + piece_at<F::kPieces>(row, 2 * step + (lane >> 4)), a);
#pragma unroll
          for (int b = 0; b < kBlocks; ++b) {
            uint32_t b0, b1;
            if (F::kKeep) {
              b0 = qf[F::kKeep ? step : 0][F::kKeep ? b : 0][0];
              b1 = qf[F::kKeep ? step : 0][F::kKeep ? b : 0][1];
            } else {
              query(step, b, b0, b1);
            }
            mma<false>(s[b], a, b0, b1);
          }
        }
      }
      // ---- weights: a lane has keys `line` and `line` + 8 of rows 2 column and the next
      const int32_t key = key0 + u * kUnitKeys + line;
      float shift[2] = {0.0f, 0.0f}, key_scale[2] = {1.0f, 1.0f};
      if (kE4m3) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint32_t ke = __shfl_sync(0xffffffffu, exponent, line + 8 * j);
          const uint32_t ve = __shfl_sync(0xffffffffu, exponent, 16 + line + 8 * j);
          key_scale[j] = scale_of(ke);
          shift[j] = ve == 255 ? __uint_as_float(0x7FC00000u)
                               : static_cast<float>(static_cast<int>(ve) - kExponentBias);
        }
        exponent = exponent_of(u + 1);
      }
      const bool masked = key0 + u * kUnitKeys + kWarpKeys > least;
      bool rises = false;
#pragma unroll
      for (int b = 0; b < kBlocks; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int j = i & 1, k = i >> 1;
          float t = s[b][i] * scale[b][j];
          if (kE4m3) t *= key_scale[k];
          if (masked && key + 8 * k >= seen[b][j]) t = minus_infinity();
          s[b][i] = t;
          rises |= t > high[b][j] + kSlack;
          if (kE4m3) rises |= t + shift[k] > top[b][j] + kSlack;
        }
      if (__any_sync(0xffffffffu, rises)) {
        const auto over_keys = [](float m) {
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
          return m;
        };
#pragma unroll
        for (int b = 0; b < kBlocks; ++b)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float m = fmaxf(over_keys(fmaxf(s[b][j], s[b][2 + j])), high[b][j]);
            const float less = m == minus_infinity() ? 1.0f : exp2_fast(high[b][j] - m);
            high[b][j] = m;
            sum[b][j] *= less;
            float by = less;
            if (kE4m3) {
              const float n =
                  fmaxf(over_keys(fmaxf(s[b][j] + shift[0], s[b][2 + j] + shift[1])), top[b][j]);
              by = n == minus_infinity() ? 1.0f : exp2_fast(top[b][j] - n);
              top[b][j] = n;
            } else {
              top[b][j] = m;
            }
#pragma unroll
            for (int t = 0; t < F::kSteps; ++t) {
              o[t][b][j] *= by;
              o[t][b][2 + j] *= by;
            }
          }
      }
      uint32_t weights[kBlocks][2];
#pragma unroll
      for (int b = 0; b < kBlocks; ++b) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int j = i & 1;
          const float w = exp2_fast(s[b][i] - (high[b][j] == minus_infinity() ? 0.0f : high[b][j]));
          sum[b][j] += w;
          s[b][i] = kE4m3 ? exp2_fast(s[b][i] + shift[i >> 1] -
                                      (top[b][j] == minus_infinity() ? 0.0f : top[b][j]))
                          : w;
        }
#pragma unroll
        for (int k = 0; k < 2; ++k)
          weights[b][k] = transpose(pack_bf16(s[b][2 * k], s[b][2 * k + 1]));
      }
      // ---- sums: 16 values of the heads by 8 rows a block
      if (kE4m3) {
        // a 16-bit element is two values: fragments of even and odd ones
#pragma unroll
        for (int step = 0; step < F::kSteps; step += 2) {
          uint32_t w[4];
          const int row = lane & 15;
          ldsm_t(values_at + row * F::kRowBytes + piece_at<F::kPieces>(row, step + (lane >> 4)), w);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t a[4];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const uint32_t v = __byte_perm(w[2 * h + k], 0, 0x3120);
              a[2 * k] = e4m3_to_bf16<0>(v);
              a[2 * k + 1] = e4m3_to_bf16<1>(v);
            }
#pragma unroll
            for (int b = 0; b < kBlocks; ++b)
              mma<false>(o[step + h][b], a, weights[b][0], weights[b][1]);
          }
        }
      } else {
#pragma unroll
        for (int step = 0; step < F::kSteps; ++step) {
          uint32_t w[4];
          const int row = (lane & 7) + ((lane >> 4) << 3);
          ldsm_t(values_at + row * F::kRowBytes +
                     piece_at<F::kPieces>(row, 2 * step + (lane >> 3 & 1)),
                 w);
#pragma unroll
          for (int b = 0; b < kBlocks; ++b) mma<false>(o[step][b], w, weights[b][0], weights[b][1]);
        }
      }
      __syncwarp();
      issue(u + F::kStages, where);
      where = locate(u + F::kStages + 1);
    }
    copy_wait<0>();

    // ---- the warps' sums, through the ring's memory
    __syncthreads();
#pragma unroll
    for (int b = 0; b < kBlocks; ++b)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float l = sum[b][j];
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
        const int r = b * 8 + 2 * column + j;
        if (line == 0) {
          sh.most[warp][r] = top[b][j];
          sh.score[warp][r] = high[b][j];
          sh.sum[warp][r] = l;
        }
        float* to = sums + (warp * F::kRows + r) * F::kSumStride;
#pragma unroll
        for (int t = 0; t < F::kSteps; ++t) {
          to[t * 16 + (kE4m3 ? 2 * line : line)] = o[t][b][j];
          to[t * 16 + (kE4m3 ? 2 * line + 1 : line + 8)] = o[t][b][2 + j];
        }
      }
    __syncthreads();
    const bool whole = seg.from == 0 && seg.to == seg.all;
    float* part = parts + (2 * block + (seg.from == 0)) * static_cast<int64_t>(F::kPartValues);
    // rows of different sight: what one does not see may have spoilt its products
    const bool differ = p.by_group(row0) != p.by_group(row0 + seg.rows - 1);
    for (int at = threadIdx.x; at < seg.rows * kDim; at += kThreads) {
      const int r = at / kDim, d = at % kDim;
      float m = sh.most[0][r], n = sh.score[0][r];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) {
        m = fmaxf(m, sh.most[w][r]);
        n = fmaxf(n, sh.score[w][r]);
      }
      float l = 0.0f, v = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        l += sh.sum[w][r] * since(sh.score[w][r], n);
        v += sums[(w * F::kRows + r) * F::kSumStride + d] * since(sh.most[w][r], m);
      }
      if (differ && l == l && !(fabsf(v) + fabsf(l) < __uint_as_float(0x7F800000u)))
        atomicOr(&sh.again, 1u << r);
      if (whole) {
        if (d < p.head_dim)
          output_row(p, seg.request.first, seg.head, row0 + r)[d] =
              f32_to_bf16(v * inverse_sum(l) * (kE4m3 ? since(m, n) : 1.0f));
      } else {
        part[3 * F::kRows + at] = v;
        if (d == 0) {
          part[r] = m;
          part[F::kRows + r] = l;
          part[2 * F::kRows + r] = n;
        }
      }
    }
    __syncthreads();
    uint32_t again = sh.again & (0x11111111u << warp);   // this warp's
    if (again)
      again = spoilt_rows(p, seg.index, seg.head, again, sh.seen[lane],
                          min(seg.to * kUnitKeys, seg.keys));
    if (kE4m3) again |= sh.large[warp];
    for (; again; again &= again - 1) {
      const int r = __ffs(again) - 1;
      Slice own;
      const int32_t to = min(seg.to * kUnitKeys, sh.seen[r]);
      warp_attend<kDim / 32, kE4m3>(p, query_row(p, seg.request.first, seg.head, row0 + r),
                                    seg.index, seg.head, seg.from * kUnitKeys, to, &own);
      uint16_t* out = output_row(p, seg.request.first, seg.head, row0 + r);
#pragma unroll
      for (int i = 0; i < kDim / 32; ++i) {
        const int d = lane + 32 * i;
        if (d >= p.head_dim) continue;
        if (whole)
          out[d] = f32_to_bf16(own.o[i] * inverse_sum(own.sum));
        else
          part[3 * F::kRows + r * kDim + d] = own.o[i];
      }
      if (!whole && lane == 0) {
        part[r] = part[2 * F::kRows + r] = own.most;
        part[F::kRows + r] = own.sum;
      }
    }
    if (!whole && seg.from == 0) {
      if (threadIdx.x == 0) leave_joint(joint, &seg, sh.share, row0, block);
      left_joint = true;
    }
    __syncthreads();
  }
  if (!left_joint && threadIdx.x == 0) leave_joint(joint, nullptr, sh.share, 0, block);
}

// Joins a tile's parts, kJoinRows blocks for each of k_attend_split's; rows behind
// the last request become zeros.  A row's parts are shared by the warps of a block
// (one token of 4096 keys, 16 tiles of 20 parts: part by part in every thread 12.3 us).
constexpr int kJoinWarps = 8;
constexpr int kJoinRows = 8;

template <int kDim, int kBlocks>
__global__ void __launch_bounds__(32 * kJoinWarps) k_attend_join(const AttendParams p) {
  using F = Form<kDim, kBlocks, false>;
  constexpr int kLane = kDim / 32;      // values of a lane
  __shared__ float sums[kJoinWarps][kDim];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int blocks = p.blocks, block = blockIdx.x;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Joint j = reinterpret_cast<const Joint*>(p.workspace)[block];
  const float* own =
      reinterpret_cast<const float*>(reinterpret_cast<const Joint*>(p.workspace) + blocks) +
      (2 * block + 1) * static_cast<int64_t>(F::kPartValues);
  const auto part = [&](int i) {  // the block's own slot 1, then the others' slots 0
    return own + (2 * i - (i > 0)) * static_cast<int64_t>(F::kPartValues);
  };
  for (int r = blockIdx.y; j.parts > 0 && r < j.rows; r += kJoinRows) {
    float m = minus_infinity(), n = m, l = 0.0f;
    for (int i = lane; i < j.parts; i += 32) {
      m = fmaxf(m, part(i)[r]);
      n = fmaxf(n, part(i)[2 * F::kRows + r]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      n = fmaxf(n, __shfl_xor_sync(0xffffffffu, n, o));
    }
    for (int i = lane; i < j.parts; i += 32)
      l += part(i)[F::kRows + r] * since(part(i)[2 * F::kRows + r], n);
    l = warp_sum_f32(l);
    float v[kLane] = {};
#pragma unroll 4
    for (int i = warp; i < j.parts; i += kJoinWarps) {
      const float* from = part(i) + 3 * F::kRows + r * kDim + lane * kLane;
      const float by = since(part(i)[r], m);
#pragma unroll
      for (int c = 0; c < kLane; c += 2) {
        const float2 f = *reinterpret_cast<const float2*>(from + c);
        v[c] += f.x * by;
        v[c + 1] += f.y * by;
      }
    }
#pragma unroll
    for (int c = 0; c < kLane; ++c) sums[warp][lane * kLane + c] = v[c];
    __syncthreads();
    const float by = inverse_sum(l) * since(m, n);
    for (int d = threadIdx.x; d < p.head_dim; d += 32 * kJoinWarps) {
      float sum = 0.0f;
#pragma unroll
      for (int w = 0; w < kJoinWarps; ++w) sum += sums[w][d];
      output_row(p, j.first, j.head, j.row + r)[d] = f32_to_bf16(sum * by);
    }
    __syncthreads();
  }
  if (blockIdx.y) return;
  const int64_t width = static_cast<int64_t>(p.heads) * p.group * p.head_dim;
  const int64_t behind = p.requests ? clamp_to(p.offsets[p.requests], p.tokens) : 0;
  for (int64_t at = behind * width + block * 32 * kJoinWarps + threadIdx.x; at < p.tokens * width;
       at += static_cast<int64_t>(blocks) * 32 * kJoinWarps)
    p.o[at] = 0;
}

template <int kDim, int kBlocks, bool kE4m3>
int launch_at(AttendParams p, cudaStream_t s) {
  using F = Form<kDim, kBlocks, kE4m3>;
  const cudaError_t err = allow_shared<k_attend_split<kDim, kBlocks, kE4m3>>(F::kSmem);
  if (err != cudaSuccess) return err;
  p.blocks *= F::kPerSm;
  k_attend_split<kDim, kBlocks, kE4m3><<<p.blocks, kThreads, F::kSmem, s>>>(p);
  return launch_after(k_attend_join<kDim, kBlocks>,
                      dim3(static_cast<unsigned>(p.blocks), kJoinRows), 32 * kJoinWarps, s, p);
}

template <int kDim, int kBlocks>
int launch_with(const AttendParams& p, cudaStream_t s) {
  return p.e4m3 ? launch_at<kDim, kBlocks, true>(p, s) : launch_at<kDim, kBlocks, false>(p, s);
}

bool on_words(const Side& s, int size) {
  return (reinterpret_cast<uintptr_t>(s.data) & 15) == 0 && s.stride[0] * size % 16 == 0 &&
         s.stride[1] * size % 16 == 0 && s.stride[2] * size % 16 == 0;
}

// Rows of whole 16-byte pieces.
bool split_takes(const AttendParams& p) {
  const int size = p.e4m3 ? 1 : 2;
  return p.head_dim * size % 16 == 0 && on_words(p.key, size) && on_words(p.value, size);
}

}  // namespace

int64_t split_workspace_bytes(int sms) {
  return kMostPerSm * static_cast<int64_t>(sms) * (sizeof(Joint) + 2 * 4 * kMostPartValues);
}

bool launch_attend_split(const AttendParams& given, void* stream, int* status) {
  if (!split_takes(given)) return false;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  AttendParams p = given;
  p.unit_keys = kUnitKeys;
  p.by_unit = Divide(kUnitKeys);
  // rows of a tile: as many as a request has at most, by eights
  const int64_t rows = p.longest * p.group;
  if (p.head_dim <= 64)
    *status = rows <= 8 ? launch_with<64, 1>(p, s)
                        : rows <= 16 ? launch_with<64, 2>(p, s) : launch_with<64, 4>(p, s);
  else if (p.head_dim <= 128)
    *status = rows <= 8 ? launch_with<128, 1>(p, s)
                        : rows <= 16 ? launch_with<128, 2>(p, s) : launch_with<128, 4>(p, s);
  else
    *status = rows <= 8 ? launch_with<256, 1>(p, s) : launch_with<256, 2>(p, s);
  return true;
}

}  // namespace ciera
