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
// The gated product's M are 64 gates and the 64 ups that go with them in turn,
// so that neighbouring lanes hold the two halves of an output.
//
// A persistent block per SM: warp 0 moves tiles of 128 bytes by 64 or 128 rows
// into a ring of stages with TMA (128-byte swizzle), four warps copy gathered
// rows to the same places, one lane of warp 1 issues tcgen05.mma into one
// of two accumulators in TMEM, eight or twelve store the other accumulator.
// Tiles are dealt out round-robin over all groups; each block finds the
// groups' tiles from the offsets by itself.
//
// With large groups two blocks of a cluster share a product of 256 features by
// 256 rows (cta_group::2), each holding half of either operand: 32 KB of loads
// per block and 512 cycles of products, which L2 can just deliver.  Bound by
// the tensor cores: 2 x 1024 features of 64225 rows of 64 experts, 2048 deep, 322
// us, 1706 TFLOP/s, 16.7 thousand cycles a tile of which 16.4 are the products';
// gated 318 us; gradient of the rows 323 us; of the weights 366 us (ragged ends
// and 537 MB of results); e4m3 238 us with the gather.  With small groups bound
// by the weights' bytes: 24 tokens of the fine-grained layer in e4m3, 142 and 80
// us for gate and up and for down, 6.7 TB/s.
#include <cuda.h>

#include "ciera_device.cuh"
#include "ciera_moe_device.cuh"

namespace ciera {
namespace {

constexpr int kGatherWarps = 4;
// Warps: 0 loads A, 1 issues the products, then the storing warps, one that
// loads B, and those that gather rows (single blocks) or clear (pairs).
template <int kPair>
struct Roles {
  static constexpr int kStoreWarps = kPair == 2 ? 12 : 8;
  static constexpr int kLoadB = 2 + kStoreWarps;
  static constexpr int kThreads = 32 * (kLoadB + 1 + (kPair == 2 ? 1 : kGatherWarps));
};
constexpr int kTileM = 128;             // lanes of one accumulator: features, or gates and ups
constexpr int kRowBytes = 128;          // bytes of the contraction per stage and row
constexpr int kBoxRows = 64;            // rows of one B load
constexpr int kMaxStages = 12;
constexpr int kMaxN = 256;              // columns of one TMEM accumulator buffer
constexpr int kMaxSmallN = 64;          // most rows of a tile with small groups
constexpr int kSmemLimit = 227 * 1024;

struct TcParams {
  ExpertParams e;
  int32_t tile_n;        // most rows of a tile
  int32_t stages;
  int32_t stage_bytes;   // A then B
  int32_t a_bytes;
  int32_t m_tiles;       // tiles of the feature dimension
  uint32_t m_tiles_inverse;  // 2^32 / m_tiles, rounded up (of 2 and more)
  int32_t n_tiles;       // dw: tiles of its rows
};

// ------------------------------------------------------------------------
// PTX

// Loads to this block's shared memory; `bar` counts their bytes: a barrier of
// this block, or (kPair 2) one of the pair's first block.
template <int kPair>
__device__ __forceinline__ void tma_2d(uint32_t dst, const CUtensorMap* map, int32_t x, int32_t y,
                                       uint32_t bar) {
  if (kPair == 2)
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        ".cta_group::2 [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

template <int kPair>
__device__ __forceinline__ void tma_3d(uint32_t dst, const CUtensorMap* map, int32_t x, int32_t y,
                                       int32_t z, uint32_t bar) {
  if (kPair == 2)
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        ".cta_group::2 [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}

template <int kPair>
__device__ __forceinline__ void tma_4d(uint32_t dst, const CUtensorMap* map, int32_t x, int32_t y,
                                       int32_t z, int32_t u, uint32_t bar) {
  if (kPair == 2)
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        ".cta_group::2 [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(u), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(u), "r"(bar)
        : "memory");
}

// Arrives on `bar` (an arrival it counts on) when this thread's copies so far
// have landed.
__device__ __forceinline__ void copy_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(bar))
               : "memory");
}
__device__ __forceinline__ void copy_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}

// kPair: blocks of one product (1, or 2 neighbours of a cluster, whose tensor
// cores take the two halves of its features and share its rows).
template <bool kE4m3, int kPair>
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                    uint32_t accumulate) {
#define CIERA_MMA(group, kind)                                                         \
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\ttcgen05.mma." group kind \
               " [%0], %1, %2, %3, p;\n\t}" ::"r"(d),                                  \
               "l"(a), "l"(b), "r"(idesc), "r"(accumulate)                             \
               : "memory")
  if (kPair == 2) {
    if (kE4m3)
      CIERA_MMA("cta_group::2", ".kind::f8f6f4");
    else
      CIERA_MMA("cta_group::2", ".kind::f16");
  } else {
    if (kE4m3)
      CIERA_MMA("cta_group::1", ".kind::f8f6f4");
    else
      CIERA_MMA("cta_group::1", ".kind::f16");
  }
#undef CIERA_MMA
}

// Arrives on `bar` (of both blocks of a pair) when every MMA issued so far by
// this thread is done.
template <int kPair>
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  if (kPair == 2)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
        "[%0], %1;" ::"r"(smem_addr(bar)),
        "h"(static_cast<uint16_t>(3))
        : "memory");
  else
    asm volatile(
        "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
            smem_addr(bar))
        : "memory");
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

// Address of the barrier at the same place in the pair's first block.
__device__ __forceinline__ uint32_t in_first(const uint64_t* bar) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(a) : "r"(smem_addr(bar)));
  return a;
}

__device__ __forceinline__ void mbar_arrive_first(const uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(in_first(bar)) : "memory");
}

template <int kPair>
__device__ __forceinline__ void sync_all() {
  if (kPair == 2)
    asm volatile(
        "barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
            : "memory");
  else
    __syncthreads();
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

// One lane of a warp, the same for every call; the compiler then knows that
// what it issues is issued once.
__device__ __forceinline__ bool one_lane() {
  uint32_t one;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.b32 %0, 1, 0, p;\n\t}"
               : "=r"(one));
  return one != 0;
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
__device__ __forceinline__ uint32_t instruction(bool e4m3, bool a_rows, bool b_rows, int m,
                                                int n) {
  const uint32_t type = e4m3 ? 0u : 1u;
  return 1u << 4 | type << 7 | type << 10 | (a_rows ? 1u << 15 : 0u) | (b_rows ? 1u << 16 : 0u) |
         static_cast<uint32_t>(n >> 3) << 17 | static_cast<uint32_t>(m >> 4) << 24;
}

// ------------------------------------------------------------------------
// Tiles

struct Shared {
  uint64_t full[kMaxStages];
  uint64_t empty[kMaxStages];
  uint64_t tail[kMaxStages];         // dw: a group's last stage has landed
  uint64_t acc_full[2];
  uint64_t acc_empty[2];
  uint32_t tmem;
  uint32_t stop;                     // a wait ran out: every role leaves its loop
  int32_t start[kMaxExperts + 2];    // first row of each group; the unused rows are the last
  int32_t tile[kMaxExperts + 2];     // tiles before each group
  uint16_t per[kMaxExperts + 1];     // rows of each group's tiles
};

// N of a tile's instructions: multiples of 16, of 32 for a pair.
template <int kPair>
__device__ __forceinline__ int padded(int rows) {
  constexpr int kGrain = 16 * kPair;
  return (rows + kGrain - 1) / kGrain * kGrain;
}

// Rows per tile of a group of m rows: as few tiles as tile_n allows, of even size.
template <int kPair>
__device__ __forceinline__ int rows_per_tile(int m, int tile_n) {
  const int tiles = (m + tile_n - 1) / tile_n;
  return tiles <= 1 ? tile_n : padded<kPair>((m + tiles - 1) / tiles);
}

template <int kOp>
__device__ __forceinline__ int tiles_of_group(const TcParams& p, int m, int per, bool unused) {
  if (kOp == kExpertDw) return unused ? 0 : p.m_tiles * p.n_tiles;
  return (m + per - 1) / per * p.m_tiles;
}

// Fills start[], tile[] and per[]; one warp.
template <int kOp, int kPair>
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
    const int per = kOp == kExpertDw ? p.tile_n : rows_per_tile<kPair>(end - begin, p.tile_n);
    const int32_t tiles = g <= E ? tiles_of_group<kOp>(p, end - begin, per, g == E) : 0;
    int32_t sum = tiles;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int32_t left = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += left;
    }
    if (g <= E) {
      sh.start[g] = begin;
      sh.per[g] = static_cast<uint16_t>(per);
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

// Place in the ring of stages and the parity of its barriers' phase.
struct Place {
  int stage = 0;
  uint32_t parity = 0;
  __device__ __forceinline__ void advance(int stages) {
    if (++stage == stages) {
      stage = 0;
      parity ^= 1;
    }
  }
};

struct OutTile {
  int group;
  int feature;   // first feature of this block
  int row;       // first output row: of the grouped rows, or dw's n
  int rows;      // output rows
  int from;      // dw: first grouped row
  int depth;     // length of the contraction; 0: the tile is zeros
};

// Walks this block's (or pair's) tiles in order.  Every role does so by itself,
// between two tiles: what belongs to a group is kept while the group lasts,
// and the division by m_tiles is a multiplication.
template <int kOp, int kPair, bool kFused>
struct Walk {
  static constexpr int kFeatures = kFused ? kTileM / 2 : kTileM;
  int index, group = -1, end = 0;   // tiles before the group's end
  int begin = 0, first = 0, rows = 0, per = 0;
  __device__ explicit Walk() : index(blockIdx.x / kPair) {}
  __device__ bool next(const TcParams& p, const Shared& sh, OutTile& t) {
    const int E = p.e.experts;
    if (index >= end) {
      if (index >= sh.tile[E + 1]) return false;
      while (index >= end) end = sh.tile[++group + 1];
      begin = sh.tile[group];
      first = sh.start[group];
      rows = sh.start[group + 1] - first;
      per = sh.per[group];
    }
    const int local = index - begin;
    // local / m_tiles; the product is that or one more
    int at = p.m_tiles == 1 ? local : static_cast<int>(__umulhi(local, p.m_tiles_inverse));
    if (at * p.m_tiles > local) --at;
    t.group = group;
    t.feature = (local - at * p.m_tiles) * (kFeatures * kPair) +
                (kPair == 2 ? static_cast<int>(cluster_rank()) * kFeatures : 0);
    if (kOp == kExpertDw) {
      t.row = at * per;
      t.rows = min(per, static_cast<int>(p.e.n) - t.row);
      t.from = first;
      t.depth = rows;
    } else {
      t.row = first + at * per;
      t.rows = min(per, rows - at * per);
      t.from = 0;
      t.depth = group == E ? 0 : static_cast<int>(kOp == kExpertForward ? p.e.k : p.e.n);
    }
    index += gridDim.x / kPair;
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

// x's row behind grouped row r; -1: none (zeros).
__device__ __forceinline__ int32_t token_row(const ExpertParams& p, int32_t r, int32_t end) {
  if (r >= end) return -1;
  const int32_t t = p.row_tokens[r];
  return t >= 0 && t < p.x_rows ? t : -1;
}

// exp and the reciprocal to a few units in the last of 24 bits; the results are
// rounded to 8.  1 / inf is 0.
__device__ __forceinline__ float sigmoid(float a) {
  float s;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(1.0f + __expf(-a)));
  return s;
}
__device__ __forceinline__ float silu(float a) { return a * sigmoid(a); }

// ------------------------------------------------------------------------
// Two warps: loads of A and of B by TMA (one warp for both takes nearly
// as long to issue a stage's loads as the products take).  Gathered rows are
// left to the gathering warps.  The bytes of both operands, and of both blocks
// of a pair, are counted by the first block's barriers, where the products are
// issued; the loader of A announces them.

template <int kOp, bool kGated, bool kE4m3, int kPair, bool kLoadsA>
__device__ void load_tiles(const TcParams& p, const CUtensorMap* map, Shared& sh, uint32_t ring) {
  constexpr int kDepth = kE4m3 ? 128 : 64;  // contraction per stage
  constexpr bool kFused = kOp == kExpertForward && kGated;
  if (!one_lane()) return;
  const bool first = kPair == 1 || cluster_rank() == 0;
  const bool gather = kOp == kExpertForward && kPair == 1 && p.e.row_tokens != nullptr;
  Place at;
  int issued = 0;
  Walk<kOp, kPair, kFused> walk;
  OutTile t;
  bool alive = true;
  while (alive && walk.next(p, sh, t)) {
    // this block's share of the rows
    const int share = padded<kPair>(t.rows) / kPair;
    const int row = t.row + (first ? 0 : share);
    const int boxes = (share + kBoxRows - 1) / kBoxRows;
    const uint32_t bytes = p.a_bytes + (gather ? 0 : boxes * kBoxRows * kRowBytes);
    for (int c = 0; c < t.depth; c += kDepth) {
      uint64_t* full = &sh.full[at.stage];
      alive = wait(p, sh, &sh.empty[at.stage], at.parity ^ 1);
      if (!alive) break;
      const uint32_t a = ring + at.stage * p.stage_bytes, b = a + p.a_bytes;
      // dw's last stage of a group is counted where it lands, and announced
      // by who clears it
      const bool tail = kOp == kExpertDw && t.depth - c < kDepth;
      uint32_t bar = kPair == 2 ? in_first(full) : smem_addr(full);
      if (tail) bar = smem_addr(&sh.tail[at.stage]);
      if constexpr (kLoadsA) {
        if (tail)
          mbar_arrive_expect_tx(&sh.tail[at.stage], bytes);
        else if (first)
          mbar_arrive_expect_tx(full, kPair * bytes);
        else if (kOp == kExpertDw)
          mbar_arrive_first(full);
        if (kOp == kExpertForward) {
          if (kFused)
            tma_4d<kPair>(a, map, c, 0, t.feature, t.group, bar);
          else
            tma_3d<kPair>(a, map, c, t.feature, t.group, bar);
        } else if (kOp == kExpertDx) {
          tma_3d<kPair>(a, map, t.feature, c, t.group, bar);
          tma_3d<kPair>(a + 64 * kRowBytes, map, t.feature + 64, c, t.group, bar);
        } else {
          tma_2d<kPair>(a, map, t.feature, t.from + c, bar);
          tma_2d<kPair>(a + 64 * kRowBytes, map, t.feature + 64, t.from + c, bar);
        }
      } else {
        for (int i = 0; i < boxes; ++i) {
          const uint32_t to = b + i * kBoxRows * kRowBytes;
          if (kOp == kExpertDw)
            tma_2d<kPair>(to, map, row + i * kBoxRows, t.from + c, bar);
          else
            tma_2d<kPair>(to, map, c, row + i * kBoxRows, bar);
        }
      }
      at.advance(p.stages);
      ++issued;
    }
  }
  // What is still under way writes this block's shared memory: see the products'
  // last arrivals come in, or after a wait that ran out the copies land (those
  // of a pair's second block are the first's to see).
  for (int i = issued > p.stages ? issued - p.stages : 0; i < issued; ++i) {
    uint64_t* bar = alive ? &sh.empty[i % p.stages] : &sh.full[i % p.stages];
    if (alive || first) mbar_wait_bounded(bar, (i / p.stages) & 1, p.e.timeout_ns);
  }
}

// ------------------------------------------------------------------------
// Four warps of a single block: gathered rows, 16 bytes per thread and copy, written where
// the 128-byte swizzle has them.  A stage's barrier counts the threads whose
// copies have landed; nobody waits for them but the products.  Right for small
// groups, where it saves a launch; with large ones each row is fetched again
// for every tile of features and the products wait (gated product of 64225
// rows, 2048 to 2 x 1024: 412 us, against 322 us from rows gathered before;
// TMA's own gather, four rows an instruction: 1222 us).

template <bool kFused, bool kE4m3>
__device__ void gather_tiles(const TcParams& p, Shared& sh, uint32_t ring) {
  constexpr int kDepth = kE4m3 ? 128 : 64;
  constexpr int kSize = kE4m3 ? 1 : 2;
  constexpr int kRows = kMaxN / 16;         // rows per thread and stage
  const ExpertParams& e = p.e;
  const int tid = threadIdx.x - 32 * (Roles<1>::kLoadB + 1);
  const int piece = tid & 7, row0 = tid >> 3;  // 16 rows of 8 pieces a sweep
  const unsigned char* x = static_cast<const unsigned char*>(e.x);
  const int64_t stride = e.x_stride * kSize;
  Place at;
  Walk<kExpertForward, 1, kFused> walk;
  OutTile t;
  bool alive = true;
  while (alive && walk.next(p, sh, t)) {
    if (t.depth == 0) continue;
    const int rows = padded<1>(t.rows);
    int32_t token[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) token[i] = token_row(e, t.row + row0 + 16 * i, t.row + t.rows);
    for (int c = 0; c < t.depth; c += kDepth) {
      alive = wait(p, sh, &sh.empty[at.stage], at.parity ^ 1);
      if (!alive) break;
      const uint32_t to = ring + at.stage * p.stage_bytes + p.a_bytes;
      // bytes of the row from this piece on
      const int64_t have = (static_cast<int64_t>(t.depth) - c) * kSize - piece * 16;
      const int bytes = have <= 0 ? 0 : have < 16 ? static_cast<int>(have) : 16;
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const int row = row0 + 16 * i;
        if (row >= rows) break;
        const bool some = token[i] >= 0 && bytes > 0;
        copy16(to + row * kRowBytes + ((piece ^ (row & 7)) << 4),
               some ? x + token[i] * stride + static_cast<int64_t>(c) * kSize + piece * 16 : x,
               some ? bytes : 0);
      }
      copy_arrive(&sh.full[at.stage]);
      at.advance(p.stages);
    }
  }
  copy_wait_all();
}

// ------------------------------------------------------------------------
// Warp 1: products.

template <int kOp, bool kGated, bool kE4m3, int kPair>
__device__ void multiply(const TcParams& p, Shared& sh, uint32_t ring) {
  constexpr int kDepth = kE4m3 ? 128 : 64;
  constexpr int kSteps = 4;                // instructions a stage
  constexpr int kStep = kDepth / kSteps;   // contraction per instruction
  constexpr bool kFused = kOp == kExpertForward && kGated;
  constexpr bool kARows = kOp != kExpertForward, kBRows = kOp == kExpertDw;
  // an operand's next step: 32 bytes along its rows, or 16 rows
  constexpr int kStepA = (kARows ? kStep * kRowBytes : 32) >> 4;
  constexpr int kStepB = (kBRows ? kStep * kRowBytes : 32) >> 4;
  if (!one_lane()) return;
  const bool gather = kOp == kExpertForward && kPair == 1 && p.e.row_tokens != nullptr;
  const uint64_t a0 = operand(ring, 8 * kRowBytes, kARows ? 64 * kRowBytes : 0);
  const uint64_t b0 = operand(ring + p.a_bytes, 8 * kRowBytes, kBRows ? 64 * kRowBytes : 0);
  const uint32_t tmem = sh.tmem;
  Place at;
  int tiles = 0;
  Walk<kOp, kPair, kFused> walk;
  OutTile t, next;
  bool have = walk.next(p, sh, next);
  while (have) {
    t = next;
    if (t.depth == 0) {
      have = walk.next(p, sh, next);
      continue;
    }
    const int buffer = tiles & 1;
    if (!wait(p, sh, &sh.acc_empty[buffer], ((tiles >> 1) & 1) ^ 1)) return;
    tc_fence_after();
    const uint32_t d = tmem + buffer * kMaxN;
    const int n = padded<kPair>(t.rows);
    const uint32_t idesc = instruction(kE4m3, kARows, kBRows, kTileM * kPair, n);
    uint32_t accumulate = 0;
    for (int c = 0; c < t.depth; c += kDepth) {
      const int stage = at.stage;
      if (!wait(p, sh, &sh.full[stage], at.parity)) return;
      // gathered rows came by ordinary copies: order them before the tensor
      // core's reads
      if (gather) fence_proxy_async_smem();
      tc_fence_after();
      const uint32_t offset = static_cast<uint32_t>(stage * p.stage_bytes) >> 4;
      const uint64_t a = a0 + offset, b = b0 + offset;
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        if (kOp == kExpertDw && c + s * kStep >= t.depth) break;
        mma<kE4m3, kPair>(d, a + s * kStepA, b + s * kStepB, idesc, accumulate);
        accumulate = 1;
      }
      mma_commit<kPair>(&sh.empty[stage]);
      at.advance(p.stages);
      // the next tile is looked up behind the third stage, while the tensor
      // core has products in hand
      if (c == 2 * kDepth || (c < 2 * kDepth && c + kDepth >= t.depth))
        have = walk.next(p, sh, next);
    }
    mma_commit<kPair>(&sh.acc_full[buffer]);
    ++tiles;
  }
}

// ------------------------------------------------------------------------
// One warp, dw: zeroes what a group's last stage holds behind the group's last
// row, up to the next whole step: rows of the next group, or stale ones.  Both
// operands, since 0 times an infinity there would be a NaN.  The stage lands
// long before its products are due, so that they do not wait for this (420 us
// for the gradient of 2 x 1024 x 2048 weights from 64225 rows when the issuing
// lane's warp did it).  A stage has a barrier of its own for it, since several
// groups' last stages can be under way; it is used again only when the
// products have read the stage.

__device__ void clear_tails(const TcParams& p, Shared& sh, unsigned char* ring_ptr) {
  const int lane = threadIdx.x & 31;
  int used = 0;
  uint32_t parity = 0;  // of each stage's barrier
  Walk<kExpertDw, 2, false> walk;
  OutTile t;
  while (walk.next(p, sh, t)) {
    if (t.depth == 0) continue;
    used += (t.depth + 63) / 64;  // stages so far
    const int have = t.depth % 64;
    if (have == 0) continue;
    const int stage = (used - 1) % p.stages;
    if (!wait(p, sh, &sh.tail[stage], parity >> stage & 1)) return;
    parity ^= 1u << stage;
    unsigned char* base = ring_ptr + stage * p.stage_bytes;
    const int columns =
        p.a_bytes / (64 * kRowBytes) + (padded<2>(t.rows) / 2 + 63) / 64;
    const int words = (((have + 15) & ~15) - have) * (kRowBytes / 16);
    for (int column = 0; column < columns; ++column)
      for (int i = lane; i < words; i += 32)
        *reinterpret_cast<uint4*>(base + column * 64 * kRowBytes + have * kRowBytes + i * 16) =
            make_uint4(0, 0, 0, 0);
    // each lane's zeros are in shared memory, for this block's tensor core, before
    // the first block hears of it; nothing else is handed over (a fence over
    // the cluster would wait for the storing warps' writes too: 427 instead of
    // 396 us for the gradient of 2 x 1024 x 2048 weights from 64225 rows)
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive_first(&sh.full[stage]);
  }
}

// ------------------------------------------------------------------------
// Storing warps.  A thread holds one feature of 16 rows at a time; the 32 lanes
// of a warp store 32 neighbouring features of a row.  Two or three warps share
// a quarter of the features (a warp can read only the TMEM lanes of its number
// modulo 4) and take chunks of rows in turn.
//
// Nothing in a chunk branches on a row: loads come from the last row where a
// row lies behind the tile, so that sixteen independent rows hide each
// other's latency, and only the stores are predicated.  (With a test per row
// the exponentials, divisions and loads of a chunk ran one after another:
// 2111 instead of 259 us for the
// gradient through the gated unit of 64225 rows, 2048 to 1024.)

// Chunks of 16 rows: two or three warps a quarter make a tile's outputs in 3 to
// 7 thousand cycles while the next tile's products take 8 to 16.
constexpr int kChunk = 16;

// 16 rows of one feature each to bf16, row j at out + j * stride.
__device__ __forceinline__ void store_bf16(uint16_t* out, int64_t stride, const float* v, int left,
                                           bool mine) {
  if (left >= kChunk) {
    if (mine)
#pragma unroll
      for (int j = 0; j < kChunk; ++j) out[j * stride] = f32_to_bf16(v[j]);
  } else {
#pragma unroll
    for (int j = 0; j < kChunk; ++j)
      if (mine && j < left) out[j * stride] = f32_to_bf16(v[j]);
  }
}

// The same for half a chunk, `left` of whose rows are the tile's.
__device__ __forceinline__ void store_half(uint16_t* out, int64_t stride, const float* v, int left,
                                           bool mine) {
  if (left >= kChunk / 2) {
    if (mine)
#pragma unroll
      for (int j = 0; j < kChunk / 2; ++j) out[j * stride] = f32_to_bf16(v[j]);
  } else {
#pragma unroll
    for (int j = 0; j < kChunk / 2; ++j)
      if (mine && j < left) out[j * stride] = f32_to_bf16(v[j]);
  }
}

// Scale of x's row behind grouped row r.
__device__ __forceinline__ float row_scale(const ExpertParams& e, int64_t r) {
  int64_t x = r;
  if (e.row_tokens) {
    x = e.row_tokens[r];
    if (x < 0 || x >= e.x_rows) return 0.0f;
  }
  return e.x_scale[x];
}

// Eight rows of two features f and f + 1 (in one word) at p + j * stride, the
// second feature only where `second`; words where rows start on 4-byte
// boundaries.  Row j is row min(j, last).
__device__ __forceinline__ void load_pairs(const uint16_t* p, int64_t stride, int last, bool wide,
                                           bool second, uint32_t (&v)[kChunk / 2]) {
  if (wide) {
#pragma unroll
    for (int j = 0; j < kChunk / 2; ++j)
      v[j] = *reinterpret_cast<const uint32_t*>(p + min(j, last) * stride);
  } else {
#pragma unroll
    for (int j = 0; j < kChunk / 2; ++j) {
      const uint16_t* at = p + min(j, last) * stride;
      v[j] = at[0] | (second ? static_cast<uint32_t>(at[1]) << 16 : 0u);
    }
  }
}

__device__ __forceinline__ void store_pairs(uint16_t* p, int64_t stride, int rows, bool wide,
                                            bool second, const uint32_t (&v)[kChunk / 2]) {
  if (wide && rows >= kChunk / 2) {
#pragma unroll
    for (int j = 0; j < kChunk / 2; ++j) *reinterpret_cast<uint32_t*>(p + j * stride) = v[j];
  } else {
#pragma unroll
    for (int j = 0; j < kChunk / 2; ++j)
      if (j < rows) {
        p[j * stride] = static_cast<uint16_t>(v[j]);
        if (second) p[j * stride + 1] = static_cast<uint16_t>(v[j] >> 16);
      }
  }
}

template <int kOp, bool kGated, bool kE4m3, int kPair>
__device__ void store_tiles(const TcParams& p, Shared& sh) {
  constexpr bool kFused = kOp == kExpertForward && kGated;
  constexpr bool kReadsPre = kOp == kExpertDx && kGated;
  constexpr int kHalf = kChunk / 2;
  const ExpertParams& e = p.e;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, quadrant = warp & 3;
  constexpr int kTurns = Roles<kPair>::kStoreWarps / 4;  // warps of a quarter
  constexpr int kStride = kTurns * kChunk;        // rows from chunk to chunk
  constexpr int kScales = (kMaxN / kChunk + 2 * kTurns - 1) / (2 * kTurns);
  const int first_row = ((warp - 2) >> 2) * kChunk;
  const bool odd = lane & 1;
  const int64_t features = kOp == kExpertForward ? e.n : e.k;
  uint16_t* y = static_cast<uint16_t*>(e.y);
  const bool wide = kReadsPre && e.k % 2 == 0 &&
                    ((reinterpret_cast<uintptr_t>(e.pre_in) | reinterpret_cast<uintptr_t>(y)) & 3) == 0;
  int tiles = 0;
  Walk<kOp, kPair, kFused> walk;
  OutTile t;
  while (walk.next(p, sh, t)) {
    // this thread's feature: of a gate (even lanes) or up (odd lanes) when they
    // come in turn; the gated unit's gradient takes two lanes' features
    // together, even lanes the first half of a chunk's rows, odd the second
    const int64_t f = t.feature + (kFused     ? quadrant * 16 + (lane >> 1)
                                   : kReadsPre ? quadrant * 32 + (lane & ~1)
                                               : quadrant * 32 + lane);
    const bool mine = f < features, second = f + 1 < features;
    const int64_t f_in = mine ? f : wide ? features - 2 : features - 1;  // for loads
    const int buffer = tiles & 1;
    const bool zero = t.depth == 0;
    // What the outputs need besides the products is fetched before them: e4m3's
    // scales (lanes 0 to 15 of row[q]: the rows of this warp's chunk 2 q, lanes
    // 16 to 31 those of chunk 2 q + 1), and the first chunk
    // of the gated unit's inputs; each further chunk one chunk ahead.
    float scale = 1.0f, scale_up = 1.0f, row[kScales];
    uint32_t gate_in[kHalf], up_in[kHalf];
    const auto fetch_pre = [&](int c) {
      // the last row stands in for rows behind the tile
      const int first = min(c + (odd ? kHalf : 0), t.rows - 1);
      const uint16_t* pre = e.pre_in + (static_cast<int64_t>(t.row) + first) * 2 * e.k + f_in;
      const bool two = f_in + 1 < features;
      load_pairs(pre, 2 * e.k, t.rows - 1 - first, wide, two, gate_in);
      load_pairs(pre + e.k, 2 * e.k, t.rows - 1 - first, wide, two, up_in);
    };
    if (!zero) {
      if (kE4m3) {
        const float* ws = e.w_scale + static_cast<int64_t>(t.group) * (kFused ? 2 : 1) * e.n;
        scale = ws[f_in];
        if (kFused) scale_up = ws[f_in + e.n];
#pragma unroll
        for (int q = 0; q < kScales; ++q) {
          const int at = first_row + (2 * q + (lane >> 4)) * kStride + (lane & 15);
          row[q] = at < t.rows ? row_scale(e, static_cast<int64_t>(t.row) + at) : 0.0f;
        }
      }
      if (kReadsPre && first_row < t.rows) fetch_pre(first_row);
      if (!wait(p, sh, &sh.acc_full[buffer], (tiles >> 1) & 1)) return;
      tc_fence_after();
      ++tiles;
    }
    const uint32_t acc =
        sh.tmem + buffer * kMaxN + (static_cast<uint32_t>(quadrant * 32) << 16);
#pragma unroll 1
    for (int c = first_row, chunk = 0; c < t.rows; c += kStride, ++chunk) {
      const int left = t.rows - c;
      const int64_t r = t.row + c;
      float v[kChunk];
      if (zero) {
#pragma unroll
        for (int j = 0; j < kChunk; ++j) v[j] = 0.0f;
      } else {
        tmem_ld16(acc + c, v);
        tmem_ld_wait();
      }
      // e4m3: this chunk's row scales, row j's in lane from + j
      float scales = 1.0f;
      const int from = (chunk & 1) * kChunk;
      if (kE4m3 && !zero) {
        scales = row[0];
#pragma unroll
        for (int q = 1; q < kScales; ++q)
          if (chunk >> 1 == q) scales = row[q];
      }
      if (kE4m3 && !kFused && !zero) {
#pragma unroll
        for (int j = 0; j < kChunk; ++j)
          v[j] *= __shfl_sync(0xffffffffu, scales, from + j) * scale;
      }
      if (kFused) {
        // even lanes get the ups of the first rows, odd lanes the gates of the last
        const int first = odd ? kHalf : 0;
        float gate[kHalf], up[kHalf];
#pragma unroll
        for (int j = 0; j < kHalf; ++j) {
          const float got = __shfl_xor_sync(0xffffffffu, odd ? v[j] : v[kHalf + j], 1);
          gate[j] = odd ? got : v[j];
          up[j] = odd ? v[kHalf + j] : got;
          if (kE4m3) {
            const float xs = __shfl_sync(0xffffffffu, scales, from + first + j);
            gate[j] *= xs * scale;
            up[j] *= xs * scale_up;
          }
        }
        if (e.pre_out) {
          uint16_t* pre = e.pre_out + (r + first) * 2 * e.n + f;
          store_half(pre, 2 * e.n, gate, left - first, mine);
          store_half(pre + e.n, 2 * e.n, up, left - first, mine);
        }
#pragma unroll
        for (int j = 0; j < kHalf; ++j) gate[j] = silu(gate[j]) * up[j];
        store_half(y + (r + first) * e.n + f, e.n, gate, left - first, mine);
      } else if (kOp == kExpertForward) {
        store_bf16(y + r * e.n + f, e.n, v, left, mine);
      } else if (kReadsPre) {
        uint32_t gate[kHalf], up[kHalf];
#pragma unroll
        for (int j = 0; j < kHalf; ++j) {
          gate[j] = gate_in[j];
          up[j] = up_in[j];
        }
        if (!zero && c + kStride < t.rows) fetch_pre(c + kStride);
#pragma unroll
        for (int j = 0; j < kHalf; ++j) {
          const float got = __shfl_xor_sync(0xffffffffu, odd ? v[j] : v[kHalf + j], 1);
          const float d[2] = {odd ? got : v[j], odd ? v[kHalf + j] : got};
          float dg[2], du[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float g = i ? bf16_hi(gate[j]) : bf16_lo(gate[j]);
            const float u = i ? bf16_hi(up[j]) : bf16_lo(up[j]);
            const float s = sigmoid(g), ds = d[i] * s;
            du[i] = ds * g;
            dg[i] = ds * u * (1.0f + g * (1.0f - s));
          }
          gate[j] = zero ? 0u : pack_bf16(dg[0], dg[1]);
          up[j] = zero ? 0u : pack_bf16(du[0], du[1]);
        }
        const int first = odd ? kHalf : 0;
        uint16_t* to = y + (r + first) * 2 * e.k + f;
        if (mine) {
          store_pairs(to, 2 * e.k, left - first, wide, second, gate);
          store_pairs(to + e.k, 2 * e.k, left - first, wide, second, up);
        }
      } else if (kOp == kExpertDx) {
        store_bf16(y + r * e.k + f, e.k, v, left, mine);
      } else {
        const int64_t at = t.group * e.y_expert_stride + r * e.y_stride + f;
        if (e.f32_out) {
          float* out = static_cast<float*>(e.y) + at;
          if (e.accumulate) {
            float old[kChunk];
#pragma unroll
            for (int j = 0; j < kChunk; ++j)
              old[j] = mine && j < left ? out[j * e.y_stride] : 0.0f;
#pragma unroll
            for (int j = 0; j < kChunk; ++j) v[j] += old[j];
          }
#pragma unroll
          for (int j = 0; j < kChunk; ++j)
            if (mine && j < left) out[j * e.y_stride] = v[j];
        } else {
          uint16_t* out = y + at;
          if (e.accumulate) {
            uint16_t old[kChunk];
#pragma unroll
            for (int j = 0; j < kChunk; ++j) old[j] = mine && j < left ? out[j * e.y_stride] : 0;
#pragma unroll
            for (int j = 0; j < kChunk; ++j) v[j] += bf16_to_f32(old[j]);
          }
          store_bf16(out, e.y_stride, v, left, mine);
        }
      }
      __syncwarp();
    }
    if (!zero) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (kPair == 2)
          mbar_arrive_first(&sh.acc_empty[buffer]);
        else
          mbar_arrive(&sh.acc_empty[buffer]);
      }
    }
  }
}

template <int kOp, bool kGated, bool kE4m3, int kPair>
__global__ void __launch_bounds__(Roles<kPair>::kThreads, 1)
    k_expert_tc(const TcParams p, const __grid_constant__ CUtensorMap map_a,
                const __grid_constant__ CUtensorMap map_b) {
  extern __shared__ unsigned char raw[];
  __shared__ Shared sh;
  // stages on 1024-byte boundaries: the swizzle's period
  const uint32_t base = smem_addr(raw);
  const uint32_t ring = (base + 1023) & ~1023u;
  unsigned char* ring_ptr = raw + (ring - base);
  constexpr int kLoadB = Roles<kPair>::kLoadB;
  const int warp = threadIdx.x >> 5;
  const bool gather = kOp == kExpertForward && kPair == 1 && p.e.row_tokens != nullptr;
  if (threadIdx.x == 0) {
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(&sh.full[i], gather ? 1 + 32 * kGatherWarps
                             : kOp == kExpertDw ? 2 : 1);
      mbar_init(&sh.empty[i], 1);
      mbar_init(&sh.tail[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.acc_full[i], 1);
      mbar_init(&sh.acc_empty[i], Roles<kPair>::kStoreWarps * kPair);
    }
    sh.stop = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    if (kPair == 2) {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                       smem_addr(&sh.tmem)),
                   "r"(2 * kMaxN)
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
      asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                       smem_addr(&sh.tmem)),
                   "r"(2 * kMaxN)
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
  } else if (warp == 2) {
    find_groups<kOp, kPair>(p, sh);
  }
  __syncthreads();
  sync_all<kPair>();
  tc_fence_after();
  if (warp == 0)
    load_tiles<kOp, kGated, kE4m3, kPair, true>(p, &map_a, sh, ring);
  else if (warp == 1 && (kPair == 1 || cluster_rank() == 0))
    multiply<kOp, kGated, kE4m3, kPair>(p, sh, ring);
  else if (warp >= 2 && warp < kLoadB)
    store_tiles<kOp, kGated, kE4m3, kPair>(p, sh);
  else if (warp == kLoadB && !gather)
    load_tiles<kOp, kGated, kE4m3, kPair, false>(p, &map_b, sh, ring);
  else if (warp > kLoadB && kOp == kExpertDw)
    clear_tails(p, sh, ring_ptr);
  else if (warp > kLoadB && gather)
    gather_tiles<kGated, kE4m3>(p, sh, ring);
  tc_fence_before();
  __syncthreads();
  sync_all<kPair>();
  tc_fence_after();
  if (warp == 1) {
    if (kPair == 2)
      asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(sh.tmem),
                   "r"(2 * kMaxN)
                   : "memory");
    else
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(sh.tmem),
                   "r"(2 * kMaxN)
                   : "memory");
  }
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

// A map of matrices of rows x columns, `planes` of them (0: one, without the
// dimension); boxes of 128 bytes by box_rows.  With `parts` 2 a box's rows are
// row i of the first part and row i of the second in turn, part_stride apart.
bool make_map(CUtensorMap* map, const void* base, bool e4m3, int64_t columns, int64_t rows,
              int64_t stride, int64_t planes, int64_t plane_stride, int box_rows, int parts = 1,
              int64_t part_stride = 0) {
  const int64_t size = e4m3 ? 1 : 2;
  if ((reinterpret_cast<uintptr_t>(base) & 15) || stride * size % 16 ||
      (planes > 1 && (plane_stride * size % 16 || plane_stride <= 0)) || columns < 1 || rows < 1)
    return false;
  cuuint64_t dims[4], strides[3];
  cuuint32_t box[4];
  const cuuint32_t ones[4] = {1, 1, 1, 1};
  int rank = 0;
  const auto add = [&](int64_t n, int64_t apart, int64_t of_box) {
    if (rank) strides[rank - 1] = static_cast<cuuint64_t>(apart * size);
    dims[rank] = static_cast<cuuint64_t>(n);
    box[rank++] = static_cast<cuuint32_t>(of_box);
  };
  add(columns, 0, kRowBytes / size);
  if (parts == 2) add(2, part_stride, 2);
  add(rows, stride, box_rows / parts);
  if (planes > 0) add(planes, planes > 1 ? plane_stride : stride * rows * parts, 1);
  return encode()(map, e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                  static_cast<cuuint32_t>(rank), const_cast<void*>(base), dims, strides, box, ones,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int kOp, bool kGated, bool kE4m3, int kPair>
int launch_at(const TcParams& p, const CUtensorMap& a, const CUtensorMap& b, int grid,
              cudaStream_t s) {
  const cudaError_t err =
      allow_shared<k_expert_tc<kOp, kGated, kE4m3, kPair>>(kSmemLimit - 14 * 1024);
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t config{};
  config.gridDim = dim3(static_cast<unsigned>(grid));
  config.blockDim = dim3(Roles<kPair>::kThreads);
  config.dynamicSmemBytes = static_cast<size_t>(p.stages) * p.stage_bytes + 1024;
  config.stream = s;
  cudaLaunchAttribute pair{};
  pair.id = cudaLaunchAttributeClusterDimension;
  pair.val.clusterDim.x = 2;
  pair.val.clusterDim.y = pair.val.clusterDim.z = 1;
  config.attrs = &pair;
  config.numAttrs = kPair == 2 ? 1 : 0;
  return cudaLaunchKernelEx(&config, k_expert_tc<kOp, kGated, kE4m3, kPair>, p, a, b);
}

template <int kPair>
int launch_with(const TcParams& p, const CUtensorMap& a, const CUtensorMap& b, int grid,
                cudaStream_t s) {
  const ExpertParams& e = p.e;  // dw always takes pairs
  if (e.op == kExpertForward) {
    if (e.e4m3)
      return e.gated ? launch_at<kExpertForward, true, true, kPair>(p, a, b, grid, s)
                     : launch_at<kExpertForward, false, true, kPair>(p, a, b, grid, s);
    return e.gated ? launch_at<kExpertForward, true, false, kPair>(p, a, b, grid, s)
                   : launch_at<kExpertForward, false, false, kPair>(p, a, b, grid, s);
  }
  if (e.op == kExpertDx)
    return e.gated ? launch_at<kExpertDx, true, false, kPair>(p, a, b, grid, s)
                   : launch_at<kExpertDx, false, false, kPair>(p, a, b, grid, s);
  return launch_at<kExpertDw, false, false, 2>(p, a, b, grid, s);
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
  const bool small = e.op != kExpertDw && e.rows <= 32 * static_cast<int64_t>(e.experts);
  if (e.experts < 1 || e.rows < 1 || features < 1 || depth < 1 || e.x_rows < 1) return false;
  TcParams p{};
  p.e = e;
  // Rows of a tile.  With few rows per expert on average the weights' bytes
  // bound the call: tiles of 64 rows, a block each, leave room for more stages
  // in flight.  Both forms, gated product over 64 experts of 2048 x 2 x 1024, in
  // us (small, pairs): 16 rows per expert 83.9, 90.0; 32 rows 88.7, 93.1; 64 rows
  // 100.8, 98.6; 128 rows 144.0, 111.3.
  p.tile_n = small ? kMaxSmallN : kMaxN;
  p.a_bytes = kTileM * kRowBytes;
  const int pair = small || e.row_tokens ? 1 : 2;
  p.stage_bytes = p.a_bytes + p.tile_n / pair * kRowBytes;
  p.stages = (kSmemLimit - 16 * 1024) / p.stage_bytes;
  if (p.stages > kMaxStages) p.stages = kMaxStages;
  const int64_t tile_m = (fused ? kTileM / 2 : kTileM) * pair;
  const int64_t m_tiles = (features + tile_m - 1) / tile_m;
  const int64_t n_tiles = e.op == kExpertDw ? (e.n + p.tile_n - 1) / p.tile_n : 1;
  const int64_t row_tiles = e.op == kExpertDw ? n_tiles * e.experts
                                              : e.rows / 16 + e.experts + 1;  // at most
  if (m_tiles * row_tiles > (int64_t(1) << 30)) return false;
  p.m_tiles = static_cast<int32_t>(m_tiles);
  p.m_tiles_inverse = static_cast<uint32_t>(((uint64_t(1) << 32) + m_tiles - 1) / m_tiles);
  p.n_tiles = static_cast<int32_t>(n_tiles);

  CUtensorMap a, b;
  bool ok;
  if (e.op == kExpertForward)
    ok = make_map(&a, e.w, e.e4m3, e.k, e.n, e.w_stride, e.experts, e.w_expert_stride, kTileM,
                  fused ? 2 : 1, e.n * e.w_stride) &&
         make_map(&b, e.x, e.e4m3, e.k, e.x_rows, e.x_stride, 0, 0, kBoxRows);
  else if (e.op == kExpertDx)
    ok = make_map(&a, e.w, false, e.k, e.n, e.w_stride, e.experts, e.w_expert_stride, 64) &&
         make_map(&b, e.x, false, e.n, e.x_rows, e.x_stride, 0, 0, kBoxRows);
  else
    ok = make_map(&a, e.x, false, e.k, e.x_rows, e.x_stride, 0, 0, 64) &&
         make_map(&b, e.w, false, e.n, e.rows, e.w_stride, 0, 0, 64);
  if (!ok) return false;

  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int64_t most = m_tiles * row_tiles, slots = sm_count() / pair;
  const int grid = static_cast<int>(most < slots ? most : slots) * pair;
  *status = pair == 2 ? launch_with<2>(p, a, b, grid, s) : launch_with<1>(p, a, b, grid, s);
  return true;
}

}  // namespace ciera
