// ciera_experts_tc.cu -- products grouped by expert on the tensor cores.
//
// Every product is computed as D[feature, row] = sum_c A[feature, c] B[row, c]
// with the output's contiguous dimension as the tensor core's M:
//   forward  A = w_e (c = k contiguous)            B = x rows, gathered or not
//   dx       A = w_e transposed (k contiguous)     B = dy rows
//   dw       A = x transposed (k contiguous)       B = dy transposed; c: the
//                                                  group's rows
// so that a group's rows are the N of the instruction, which may be any
// multiple of 16: a ragged group wastes at most 15 columns where rows in M
// would waste up to 127, and the lanes of a warp hold neighbouring features of
// one row, which they store contiguously without a transposition.
//
// A persistent block of six warps per SM: warp 0 moves tiles of 128 bytes by
// 64 or 128 rows into a ring of stages with TMA (128-byte swizzle; gathered
// rows four per instruction), one lane of warp 1 issues tcgen05.mma into one
// of two accumulators in TMEM, warps 2 to 5 store the other accumulator.
// Tiles are dealt out round-robin over all groups; each block finds the
// groups' tiles from the offsets by itself.
#include <cuda.h>

#include "ciera_device.cuh"
#include "ciera_moe_device.cuh"

namespace ciera {
namespace {

constexpr int kTcThreads = 192;
constexpr int kTileM = 128;             // features of one accumulator
constexpr int kRowBytes = 128;          // bytes of the contraction per stage and row
constexpr int kBoxRows = 64;            // rows of one B load
constexpr int kMaxStages = 12;
constexpr int kMaxN = 256;              // columns of one TMEM accumulator buffer
constexpr int kSmemLimit = 227 * 1024;

struct TcParams {
  ExpertParams e;
  int32_t tile_n;        // most rows of a tile
  int32_t stages;
  int32_t stage_bytes;   // A then B
  int32_t a_bytes;
  int32_t m_tiles;       // tiles of the feature dimension
  int32_t n_tiles;       // dw: tiles of its rows
};

// ------------------------------------------------------------------------
// PTX

__device__ __forceinline__ void tma_2d(uint32_t dst, const CUtensorMap* map, int32_t x, int32_t y,
                                       uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(smem_addr(bar))
      : "memory");
}

__device__ __forceinline__ void tma_3d(uint32_t dst, const CUtensorMap* map, int32_t x, int32_t y,
                                       int32_t z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar))
      : "memory");
}

// Four rows of one box height each; a row outside the matrix arrives as zeros.
__device__ __forceinline__ void tma_gather(uint32_t dst, const CUtensorMap* map, int32_t x,
                                           int4 row, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
      "l"(map), "r"(x), "r"(row.x), "r"(row.y), "r"(row.z), "r"(row.w), "r"(smem_addr(bar))
      : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}

template <bool kE4m3>
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                    uint32_t accumulate) {
  if (kE4m3)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Arrives on `bar` when every MMA issued so far by this thread is done.
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
          smem_addr(bar))
      : "memory");
}

__device__ __forceinline__ void tmem_ld32(uint32_t addr, float (&v)[32]) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr)
      : "memory");
}

__device__ __forceinline__ void tmem_ld16(uint32_t addr, float* v) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(addr)
      : "memory");
}

__device__ __forceinline__ void tmem_ld_wait() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

// Shared-memory operand: 128-byte swizzle; `stride` bytes between groups of
// eight rows, `lead` between 128-byte columns (operands with the contraction
// along the rows only).
__device__ __forceinline__ uint64_t operand(uint32_t addr, uint32_t stride, uint32_t lead) {
  return static_cast<uint64_t>((addr & 0x3FFFF) >> 4) | static_cast<uint64_t>(lead >> 4) << 16 |
         static_cast<uint64_t>(stride >> 4) << 32 | uint64_t(1) << 46 | uint64_t(2) << 61;
}

// Instruction descriptor: 32-bit float sums, operand types, which operands
// have the contraction along their rows, N and M.
__device__ __forceinline__ uint32_t instruction(bool e4m3, bool a_rows, bool b_rows, int n) {
  const uint32_t type = e4m3 ? 0u : 1u;
  return 1u << 4 | type << 7 | type << 10 | (a_rows ? 1u << 15 : 0u) | (b_rows ? 1u << 16 : 0u) |
         static_cast<uint32_t>(n >> 3) << 17 | static_cast<uint32_t>(kTileM >> 4) << 24;
}

// ------------------------------------------------------------------------
// Tiles

struct Shared {
  uint64_t full[kMaxStages];
  uint64_t empty[kMaxStages];
  uint64_t acc_full[2];
  uint64_t acc_empty[2];
  uint32_t tmem;
  uint32_t stop;                     // a wait ran out: every role leaves its loop
  int32_t start[kMaxExperts + 2];    // first row of each group; the unused rows are the last
  int32_t tile[kMaxExperts + 2];     // tiles before each group
};

// Rows per tile of a group of m rows: as few tiles as tile_n allows, of even size.
__device__ __forceinline__ int rows_per_tile(int m, int tile_n) {
  const int tiles = (m + tile_n - 1) / tile_n;
  return tiles <= 1 ? tile_n : ((m + tiles - 1) / tiles + 15) & ~15;
}

template <int kOp>
__device__ __forceinline__ int tiles_of_group(const TcParams& p, int m, bool unused) {
  if (kOp == kExpertDw) return unused ? 0 : p.m_tiles * p.n_tiles;
  const int per = rows_per_tile(m, p.tile_n);
  return (m + per - 1) / per * p.m_tiles;
}

// Fills start[] and tile[]; one warp.
template <int kOp>
__device__ void find_groups(const TcParams& p, Shared& sh) {
  const int lane = threadIdx.x & 31, E = p.e.experts;
  const int32_t rows = static_cast<int32_t>(p.e.rows);
  int32_t highest = 0, before = 0;
  for (int g0 = 0; g0 <= E; g0 += 32) {
    const int g = g0 + lane;  // end of group g
    int32_t end = g < E ? p.e.offsets[g + 1] : rows;
    end = end < 0 ? 0 : end > rows ? rows : end;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int32_t left = __shfl_up_sync(0xffffffffu, end, o);
      if (lane >= o) end = max(end, left);
    }
    end = max(end, highest);
    int32_t begin = __shfl_up_sync(0xffffffffu, end, 1);
    if (lane == 0) begin = highest;
    const int32_t tiles = g <= E ? tiles_of_group<kOp>(p, end - begin, g == E) : 0;
    int32_t sum = tiles;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int32_t left = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += left;
    }
    if (g <= E) {
      sh.start[g] = begin;
      sh.tile[g] = before + sum - tiles;
      if (g == E) {
        sh.start[E + 1] = rows;
        sh.tile[E + 1] = before + sum;
      }
    }
    highest = __shfl_sync(0xffffffffu, end, 31);
    before += __shfl_sync(0xffffffffu, sum, 31);
  }
}

struct OutTile {
  int group;
  int feature;   // first feature
  int row;       // first output row: of the grouped rows, or dw's n
  int rows;      // output rows
  int from;      // dw: first grouped row
  int depth;     // length of the contraction; 0: the tile is zeros
};

// Walks this block's tiles in order.
template <int kOp>
struct Walk {
  int index, group = 0;
  __device__ explicit Walk() : index(blockIdx.x) {}
  __device__ bool next(const TcParams& p, const Shared& sh, OutTile& t) {
    const int E = p.e.experts;
    if (index >= sh.tile[E + 1]) return false;
    while (index >= sh.tile[group + 1]) ++group;
    const int local = index - sh.tile[group];
    const int m = sh.start[group + 1] - sh.start[group];
    t.group = group;
    t.feature = local % p.m_tiles * kTileM;
    const int at = local / p.m_tiles;
    if (kOp == kExpertDw) {
      t.row = at * p.tile_n;
      t.rows = min(p.tile_n, static_cast<int>(p.e.n) - t.row);
      t.from = sh.start[group];
      t.depth = m;
    } else {
      const int per = rows_per_tile(m, p.tile_n);
      t.row = sh.start[group] + at * per;
      t.rows = min(per, m - at * per);
      t.from = 0;
      t.depth = group == E ? 0 : static_cast<int>(kOp == kExpertForward ? p.e.k : p.e.n);
    }
    index += gridDim.x;
    return true;
  }
};

// Bounded wait; false when it ran out here or anywhere in the block.
__device__ __forceinline__ bool wait(const TcParams& p, Shared& sh, uint64_t* bar,
                                     uint32_t parity) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer();
  while (!mbar_try_wait(bar, parity)) {
    if (*reinterpret_cast<volatile uint32_t*>(&sh.stop)) return false;
    if (globaltimer() - t0 > p.e.timeout_ns) {
      *reinterpret_cast<volatile uint32_t*>(&sh.stop) = 1;
      record_status(p.e.ctl, kStatusTimeout);
      return false;
    }
  }
  return true;
}

__device__ __forceinline__ int32_t token_row(const ExpertParams& p, int32_t r, int32_t end) {
  if (r >= end) return static_cast<int32_t>(p.x_rows);  // outside: zeros
  const int32_t t = p.row_tokens[r];
  return t >= 0 && t < p.x_rows ? t : static_cast<int32_t>(p.x_rows);
}

__device__ __forceinline__ int4 token_rows(const ExpertParams& p, int32_t r, int32_t end) {
  return make_int4(token_row(p, r, end), token_row(p, r + 1, end), token_row(p, r + 2, end),
                   token_row(p, r + 3, end));
}

__device__ __forceinline__ float silu(float a) { return a / (1.0f + expf(-a)); }

// ------------------------------------------------------------------------
// Warp 0: loads.

template <int kOp, bool kGated, bool kE4m3>
__device__ void load_tiles(const TcParams& p, const CUtensorMap* map_a, const CUtensorMap* map_b,
                           Shared& sh, uint32_t ring) {
  constexpr int kDepth = kE4m3 ? 128 : 64;  // contraction per stage
  constexpr bool kFused = kOp == kExpertForward && kGated;
  const int lane = threadIdx.x & 31;
  const bool gather = p.e.row_tokens != nullptr;
  int issued = 0;
  Walk<kOp> walk;
  OutTile t;
  bool alive = true;
  while (alive && walk.next(p, sh, t)) {
    const int n = (t.rows + 15) & ~15;
    const int boxes = (n + kBoxRows - 1) / kBoxRows;
    const int32_t end = kOp == kExpertDw ? t.from + t.depth : t.row + t.rows;
    int4 rows_lo{}, rows_hi{};  // forward: this lane's gathered rows
    if (kOp == kExpertForward && gather && t.depth > 0) {
      rows_lo = token_rows(p.e, t.row + 4 * lane, end);
      rows_hi = token_rows(p.e, t.row + 4 * lane + 128, end);
    }
    int4 rows_next{};           // dw: of the next stage, fetched one ahead
    const int quad = (lane & 15) * 4;
    if (kOp == kExpertDw && gather && t.depth > 0) rows_next = token_rows(p.e, t.from + quad, end);
    for (int c = 0; c < t.depth; c += kDepth) {
      const int stage = issued % p.stages;
      const uint32_t parity = (issued / p.stages) & 1;
      alive = wait(p, sh, &sh.empty[stage], parity ^ 1);
      if (!alive) break;
      const uint32_t a = ring + stage * p.stage_bytes, b = a + p.a_bytes;
      uint64_t* bar = &sh.full[stage];
      if (kOp == kExpertDw) {
        const int4 rows = rows_next;
        if (lane == 0) mbar_arrive_expect_tx(bar, p.a_bytes + boxes * kBoxRows * kRowBytes);
        __syncwarp();
        if (gather) {
          if (c + kDepth < t.depth) rows_next = token_rows(p.e, t.from + c + kDepth + quad, end);
          tma_gather(a + (lane >> 4) * 64 * kRowBytes + quad * kRowBytes, map_a,
                     t.feature + (lane >> 4) * 64, rows, bar);
        } else if (lane < 2) {
          tma_2d(a + lane * 64 * kRowBytes, map_a, t.feature + lane * 64, t.from + c, bar);
        }
        if (lane >= 8 && lane < 8 + boxes) {
          const int i = lane - 8;
          tma_2d(b + i * 64 * kRowBytes, map_b, t.row + i * 64, t.from + c, bar);
        }
      } else {
        const bool by_token = kOp == kExpertForward && gather;
        if (lane == 0)
          mbar_arrive_expect_tx(
              bar, p.a_bytes + (by_token ? n : boxes * kBoxRows) * kRowBytes);
        __syncwarp();
        if (kOp == kExpertForward) {
          if (lane == 0) tma_3d(a, map_a, c, t.feature, t.group, bar);
          if (kFused && lane == 1)
            tma_3d(a + kTileM * kRowBytes, map_a, c, static_cast<int>(p.e.n) + t.feature, t.group,
                   bar);
        } else if (lane < 2) {
          tma_3d(a + lane * 64 * kRowBytes, map_a, t.feature + lane * 64, c, t.group, bar);
        }
        if (by_token) {
          if (4 * lane < n) tma_gather(b + 4 * lane * kRowBytes, map_b, c, rows_lo, bar);
          if (4 * lane + 128 < n)
            tma_gather(b + (4 * lane + 128) * kRowBytes, map_b, c, rows_hi, bar);
        } else if (lane >= 8 && lane < 8 + boxes) {
          const int i = lane - 8;
          tma_2d(b + i * kBoxRows * kRowBytes, map_b, c, t.row + i * kBoxRows, bar);
        }
      }
      ++issued;
    }
  }
  // Copies still in flight write this block's shared memory: see them land.
  if (!alive)
    for (int i = issued > p.stages ? issued - p.stages : 0; i < issued; ++i)
      mbar_wait_bounded(&sh.full[i % p.stages], (i / p.stages) & 1, p.e.timeout_ns);
}

// ------------------------------------------------------------------------
// Warp 1: products.

template <int kOp, bool kGated, bool kE4m3>
__device__ void multiply(const TcParams& p, Shared& sh, uint32_t ring, unsigned char* ring_ptr) {
  constexpr int kDepth = kE4m3 ? 128 : 64;
  constexpr int kStep = kE4m3 ? 32 : 16;   // contraction per instruction
  constexpr bool kFused = kOp == kExpertForward && kGated;
  constexpr bool kARows = kOp != kExpertForward, kBRows = kOp == kExpertDw;
  const int lane = threadIdx.x & 31;
  int used = 0, tiles = 0;
  Walk<kOp> walk;
  OutTile t;
  while (walk.next(p, sh, t)) {
    if (t.depth == 0) continue;
    const int buffer = tiles & 1;
    if (!wait(p, sh, &sh.acc_empty[buffer], ((tiles >> 1) & 1) ^ 1)) return;
    tc_fence_after();
    const uint32_t d = sh.tmem + buffer * kMaxN;
    const uint32_t idesc = instruction(kE4m3, kARows, kBRows, (t.rows + 15) & ~15);
    for (int c = 0; c < t.depth; c += kDepth) {
      const int stage = used % p.stages;
      if (!wait(p, sh, &sh.full[stage], (used / p.stages) & 1)) return;
      const uint32_t a = ring + stage * p.stage_bytes, b = a + p.a_bytes;
      int steps = kDepth / kStep;
      if (kOp == kExpertDw && t.depth - c < kDepth) {
        // The stage holds rows of the next group (or stale ones) behind the
        // group's last: whole steps are skipped, the rest is zeroed in both
        // operands, since 0 times an infinity there would be a NaN.
        const int have = t.depth - c;
        steps = (have + kStep - 1) / kStep;
        const int columns = p.a_bytes / (64 * kRowBytes) + (t.rows + 63) / 64;
        const int words = (steps * kStep - have) * (kRowBytes / 16);
        unsigned char* base = ring_ptr + stage * p.stage_bytes;
        for (int i = lane; i < columns * words; i += 32) {
          const int column = i / words, at = i % words;
          *reinterpret_cast<uint4*>(base + column * 64 * kRowBytes + have * kRowBytes + at * 16) =
              make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
        __syncwarp();
      }
      tc_fence_after();
      if (lane == 0) {
        for (int s = 0; s < steps; ++s) {
          // along the row 32 bytes a step, along the rows 16 rows
          const uint32_t step_a = kARows ? s * kStep * kRowBytes : s * 32;
          const uint32_t step_b = kBRows ? s * kStep * kRowBytes : s * 32;
          const uint64_t da = operand(a + step_a, 8 * kRowBytes, kARows ? 64 * kRowBytes : 0);
          const uint64_t db = operand(b + step_b, 8 * kRowBytes, kBRows ? 64 * kRowBytes : 0);
          mma<kE4m3>(d, da, db, idesc, c + s > 0);
          if (kFused) {
            const uint64_t du = operand(a + kTileM * kRowBytes + step_a, 8 * kRowBytes, 0);
            mma<kE4m3>(d + kMaxN / 2, du, db, idesc, c + s > 0);
          }
        }
        mma_commit(&sh.empty[stage]);
      }
      __syncwarp();
      ++used;
    }
    if (lane == 0) mma_commit(&sh.acc_full[buffer]);
    __syncwarp();
    ++tiles;
  }
}

// ------------------------------------------------------------------------
// Warps 2 to 5: outputs.  A thread holds one feature of 32 (or 16) rows; the
// 32 lanes of a warp store 32 neighbouring features of a row.

template <int kOp, bool kGated, bool kE4m3>
__device__ void store_tiles(const TcParams& p, Shared& sh) {
  constexpr bool kFused = kOp == kExpertForward && kGated;
  const ExpertParams& e = p.e;
  const int lane = threadIdx.x & 31, quadrant = (threadIdx.x >> 5) & 3;
  const int64_t features = kOp == kExpertForward ? e.n : e.k;
  int tiles = 0;
  Walk<kOp> walk;
  OutTile t;
  while (walk.next(p, sh, t)) {
    const int64_t f = t.feature + quadrant * 32 + lane;
    const bool mine = f < features;
    const int buffer = tiles & 1;
    const bool zero = t.depth == 0;
    if (!zero) {
      if (!wait(p, sh, &sh.acc_full[buffer], (tiles >> 1) & 1)) return;
      tc_fence_after();
      ++tiles;
    }
    const uint32_t acc =
        sh.tmem + buffer * kMaxN + (static_cast<uint32_t>(quadrant * 32) << 16);
    float scale = 1.0f, scale_up = 1.0f;
    if (kE4m3 && !zero && mine) {
      const float* ws = e.w_scale + static_cast<int64_t>(t.group) * (kFused ? 2 : 1) * e.n;
      scale = ws[f];
      if (kFused) scale_up = ws[f + e.n];
    }
    constexpr int kChunk = kFused ? 16 : 32;
    for (int c = 0; c < t.rows; c += kChunk) {
      float v[kChunk * (kFused ? 2 : 1)];
      if (zero) {
#pragma unroll
        for (int j = 0; j < kChunk * (kFused ? 2 : 1); ++j) v[j] = 0.0f;
      } else {
        if constexpr (kFused) {
          tmem_ld16(acc + c, v);
          tmem_ld16(acc + kMaxN / 2 + c, v + 16);
        } else {
          tmem_ld32(acc + c, v);
        }
        tmem_ld_wait();
      }
#pragma unroll
      for (int j = 0; j < kChunk; ++j) {
        if (c + j >= t.rows || !mine) break;
        const int64_t r = t.row + c + j;
        if (kOp == kExpertDw) {
          const int64_t at = t.group * e.y_expert_stride + r * e.y_stride + f;
          if (e.f32_out) {
            float* out = static_cast<float*>(e.y) + at;
            *out = e.accumulate ? *out + v[j] : v[j];
          } else {
            uint16_t* out = static_cast<uint16_t*>(e.y) + at;
            *out = f32_to_bf16(e.accumulate ? bf16_to_f32(*out) + v[j] : v[j]);
          }
          continue;
        }
        uint16_t* y = static_cast<uint16_t*>(e.y);
        if (kOp == kExpertForward) {
          float a = v[j], up = kFused ? v[kChunk + j - (kFused ? 0 : kChunk)] : 0.0f;
          if (kE4m3 && !zero) {
            int64_t x = r;
            if (e.row_tokens) {
              x = e.row_tokens[r];
              x = x >= 0 && x < e.x_rows ? x : -1;
            }
            const float xs = x >= 0 ? e.x_scale[x] : 0.0f;
            a *= xs * scale;
            if (kFused) up *= xs * scale_up;
          }
          if (kFused) {
            if (e.pre_out) {
              e.pre_out[r * 2 * e.n + f] = f32_to_bf16(a);
              e.pre_out[r * 2 * e.n + e.n + f] = f32_to_bf16(up);
            }
            a = silu(a) * up;
          }
          y[r * e.n + f] = f32_to_bf16(a);
        } else if (kGated) {
          float dg = 0.0f, du = 0.0f;
          if (!zero) {
            const float g = bf16_to_f32(e.pre_in[r * 2 * e.k + f]);
            const float u = bf16_to_f32(e.pre_in[r * 2 * e.k + e.k + f]);
            const float s = 1.0f / (1.0f + expf(-g));
            dg = v[j] * u * s * (1.0f + g * (1.0f - s));
            du = v[j] * g * s;
          }
          y[r * 2 * e.k + f] = f32_to_bf16(dg);
          y[r * 2 * e.k + e.k + f] = f32_to_bf16(du);
        } else {
          y[r * e.k + f] = f32_to_bf16(v[j]);
        }
      }
      __syncwarp();
    }
    if (!zero) {
      tc_fence_before();
      mbar_arrive(&sh.acc_empty[buffer]);
    }
  }
}

template <int kOp, bool kGated, bool kE4m3>
__global__ void __launch_bounds__(kTcThreads, 1)
    k_expert_tc(const TcParams p, const __grid_constant__ CUtensorMap map_a,
                const __grid_constant__ CUtensorMap map_b) {
  extern __shared__ unsigned char raw[];
  __shared__ Shared sh;
  // stages on 1024-byte boundaries: the swizzle's period
  const uint32_t base = smem_addr(raw);
  const uint32_t ring = (base + 1023) & ~1023u;
  unsigned char* ring_ptr = raw + (ring - base);
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.acc_full[i], 1);
      mbar_init(&sh.acc_empty[i], 128);
    }
    sh.stop = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr(&sh.tmem)),
                 "r"(2 * kMaxN)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    tc_fence_before();
  } else if (warp == 2) {
    find_groups<kOp>(p, sh);
  }
  __syncthreads();
  tc_fence_after();
  if (warp == 0)
    load_tiles<kOp, kGated, kE4m3>(p, &map_a, &map_b, sh, ring);
  else if (warp == 1)
    multiply<kOp, kGated, kE4m3>(p, sh, ring, ring_ptr);
  else
    store_tiles<kOp, kGated, kE4m3>(p, sh);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(sh.tmem),
                 "r"(2 * kMaxN)
                 : "memory");
}

// ------------------------------------------------------------------------
// Host

using Encode = decltype(&cuTensorMapEncodeTiled);

Encode encode() {
  static const Encode fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                         &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<Encode>(f);
  }();
  return fn;
}

// A map of `planes` matrices of rows x columns; boxes of 128 bytes by box_rows.
bool make_map(CUtensorMap* map, const void* base, bool e4m3, int64_t columns, int64_t rows,
              int64_t stride, int64_t planes, int64_t plane_stride, int box_rows) {
  const int64_t size = e4m3 ? 1 : 2;
  if ((reinterpret_cast<uintptr_t>(base) & 15) || stride * size % 16 ||
      (planes > 1 && (plane_stride * size % 16 || plane_stride <= 0)) || columns < 1 || rows < 1 ||
      planes < 1)
    return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(columns), static_cast<cuuint64_t>(rows),
                              static_cast<cuuint64_t>(planes)};
  const cuuint64_t strides[2] = {
      static_cast<cuuint64_t>(stride * size),
      static_cast<cuuint64_t>((planes > 1 ? plane_stride : stride * rows) * size)};
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(kRowBytes / size),
                             static_cast<cuuint32_t>(box_rows), 1};
  const cuuint32_t ones[3] = {1, 1, 1};
  return encode()(map, e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                  plane_stride < 0 ? 2 : 3, const_cast<void*>(base), dims, strides, box, ones,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
constexpr int64_t kNoPlanes = -1;

template <int kOp, bool kGated, bool kE4m3>
int launch_at(const TcParams& p, const CUtensorMap& a, const CUtensorMap& b, int grid,
              cudaStream_t s) {
  const int smem = p.stages * p.stage_bytes + 1024;
  static const cudaError_t ready =
      cudaFuncSetAttribute(k_expert_tc<kOp, kGated, kE4m3>,
                           cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit - 12 * 1024);
  if (ready != cudaSuccess) return ready;
  k_expert_tc<kOp, kGated, kE4m3><<<grid, kTcThreads, smem, s>>>(p, a, b);
  return cudaGetLastError();
}

int sm_count() {
  static const int n = [] {
    int dev = 0, v = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
      v = 1;
    return v;
  }();
  return n;
}

}  // namespace

bool launch_expert_tc(const ExpertParams& e, void* stream, int* status) {
  if (!encode()) return false;
  const bool fused = e.op == kExpertForward && e.gated;
  const int64_t features = e.op == kExpertForward ? e.n : e.k;
  const int64_t depth = e.op == kExpertForward ? e.k : e.n;
  if (e.experts < 1 || e.rows < 1 || features < 1 || depth < 1 || e.x_rows < 1) return false;
  TcParams p{};
  p.e = e;
  // Rows of a tile.  With few rows per expert on average the weights' bytes
  // bound the call: small row tiles leave room for more stages in flight.
  const bool small = e.op != kExpertDw && e.rows <= 32 * static_cast<int64_t>(e.experts);
  p.tile_n = small ? 64 : fused ? kMaxN / 2 : kMaxN;
  p.a_bytes = (fused ? 2 : 1) * kTileM * kRowBytes;
  p.stage_bytes = p.a_bytes + p.tile_n * kRowBytes;
  p.stages = (kSmemLimit - 14 * 1024) / p.stage_bytes;
  if (p.stages > kMaxStages) p.stages = kMaxStages;
  const int64_t m_tiles = (features + kTileM - 1) / kTileM;
  const int64_t n_tiles = e.op == kExpertDw ? (e.n + p.tile_n - 1) / p.tile_n : 1;
  const int64_t row_tiles = e.op == kExpertDw ? n_tiles * e.experts
                                              : e.rows / 16 + e.experts + 1;  // at most
  if (m_tiles * row_tiles > (int64_t(1) << 30)) return false;
  p.m_tiles = static_cast<int32_t>(m_tiles);
  p.n_tiles = static_cast<int32_t>(n_tiles);

  CUtensorMap a, b;
  const int gathered = e.row_tokens ? 1 : 0;
  bool ok;
  if (e.op == kExpertForward)
    ok = make_map(&a, e.w, e.e4m3, e.k, fused ? 2 * e.n : e.n, e.w_stride, e.experts,
                  e.w_expert_stride, kTileM) &&
         make_map(&b, e.x, e.e4m3, e.k, e.x_rows, e.x_stride, 1, kNoPlanes,
                  gathered ? 1 : kBoxRows);
  else if (e.op == kExpertDx)
    ok = make_map(&a, e.w, false, e.k, e.n, e.w_stride, e.experts, e.w_expert_stride, 64) &&
         make_map(&b, e.x, false, e.n, e.x_rows, e.x_stride, 1, kNoPlanes, kBoxRows);
  else
    ok = make_map(&a, e.x, false, e.k, e.x_rows, e.x_stride, 1, kNoPlanes, gathered ? 1 : 64) &&
         make_map(&b, e.w, false, e.n, e.rows, e.w_stride, 1, kNoPlanes, 64);
  if (!ok) return false;

  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int64_t most = m_tiles * row_tiles;
  const int grid = most < sm_count() ? static_cast<int>(most) : sm_count();
  if (e.op == kExpertForward) {
    if (e.e4m3)
      *status = e.gated ? launch_at<kExpertForward, true, true>(p, a, b, grid, s)
                        : launch_at<kExpertForward, false, true>(p, a, b, grid, s);
    else
      *status = e.gated ? launch_at<kExpertForward, true, false>(p, a, b, grid, s)
                        : launch_at<kExpertForward, false, false>(p, a, b, grid, s);
  } else if (e.op == kExpertDx) {
    *status = e.gated ? launch_at<kExpertDx, true, false>(p, a, b, grid, s)
                      : launch_at<kExpertDx, false, false>(p, a, b, grid, s);
  } else {
    *status = launch_at<kExpertDw, false, false>(p, a, b, grid, s);
  }
  return true;
}

}  // namespace ciera
