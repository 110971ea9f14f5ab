// ciera_experts_tc.cu -- products grouped by expert on the tensor cores.
//
// Every product is computed as D[feature, row] = sum_c A[feature, c] B[row, c]
// with the output's contiguous dimension as the tensor core's M:
//   forward  A = w_e (c = k contiguous)            B = x rows, gathered or not
//   dx       A = w_e transposed (k contiguous)     B = dy rows
//   dw       A = x transposed (k contiguous)       B = dy transposed; c: the
//                                                  group's rows
// so that a group's rows are the N of the instruction, which may be any
// multiple of 16, for pairs of blocks of 32: a ragged group wastes at most 15
// columns, or 31, where rows in M would waste up to 127 or 255, and the lanes of a warp hold neighbouring features of
// one row, which they store contiguously without a transposition.
//
// The gated product's M are 64 gates and the 64 ups that go with them, eight of
// each in turn, so that a thread reads both halves of an output from TMEM.
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
// the tensor cores: 2 x 1024 features of 64225 rows of 64 experts, 2048 deep, 327
// us, 1680 TFLOP/s, 16.6 thousand cycles a tile of which 16.4 are the products';
// gated 317 us; gradient of the rows 311 to 342 us; of the weights 380 us (ragged
// ends and 537 MB of results); e4m3 235 us with the gather.  With small groups bound
// by the weights' bytes: 24 tokens of the fine-grained layer in e4m3, 141 and 80
// us for gate and up and for down, 6.7 TB/s.
#include <cuda.h>

#include "ciera_device.cuh"
#include "ciera_moe_device.cuh"

namespace ciera {
namespace {

constexpr int kGatherWarps = 4;
// Warps: 0 loads A, 1 issues the products, then the storing warps, one that
// loads B, and those that gather rows (single blocks) or clear (pairs).
// A storing warp has 2 KB of shared memory, half of which takes what the gated
// unit's gradient reads (and then there are eight); in e4m3 1 KB, and 512 bytes
// of scales.
constexpr int kStagingBytes = 24 * 1024;
constexpr int kScaleBytes = 6 * 1024;
constexpr int kOutputBytes = 16 * 1024;  // before the scales
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
constexpr int kShallowRows = 256;       // dw: rows per expert up to which two chunks leave at once
constexpr uint64_t kLandNs = 100000000;  // limit for what is under way when a wait ran out
constexpr int kSmemLimit = 227 * 1024;
constexpr int kStaticBytes = 10 * 1024;  // Shared below

struct TcParams {
  ExpertParams e;
  int32_t tile_n;        // most rows of a tile
  int32_t stages;
  int32_t stage_bytes;   // A then B
  int32_t a_bytes;
  int32_t m_tiles;       // tiles of the feature dimension
  uint32_t m_tiles_inverse;  // 2^32 / m_tiles, rounded up (of 2 and more)
  int32_t n_tiles;       // dw: tiles of its rows
  int32_t bulk;          // outputs leave by TMA: a chunk at a time, or two
  int32_t pieces;        // gated: A comes eight rows a load (n is no multiple of 8)
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
__device__ __forceinline__ void tma_5d(uint32_t dst, const CUtensorMap* map, int32_t x, int32_t y,
                                       int32_t z, int32_t u, int32_t v, uint32_t bar) {
  if (kPair == 2)
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        ".cta_group::2 [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(u), "r"(v), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(u), "r"(v), "r"(bar)
        : "memory");
}

// A box from shared memory to a matrix; what lies outside the matrix is left out.
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, uint32_t src, int32_t x,
                                             int32_t y) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::
                   "l"(map),
               "r"(x), "r"(y), "r"(src)
               : "memory");
}
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, uint32_t src, int32_t x,
                                             int32_t y, int32_t z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
          map),
      "r"(x), "r"(y), "r"(z), "r"(src)
      : "memory");
}

// Arrives on `bar` (an arrival it counts on) when this thread's copies so far
// have landed.
__device__ __forceinline__ void copy_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(bar))
               : "memory");
}
// Four bytes to shared memory, of which the first `bytes` come from `src`.
__device__ __forceinline__ void copy4(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes)
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

// Stores to the same place in the pair's other block.
__device__ __forceinline__ void store_peer(const void* at, uint32_t v) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
               : "=r"(a)
               : "r"(smem_addr(at)), "r"(cluster_rank() ^ 1));
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
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

// 16 lanes by 16 columns: lane l of the warp gets, of columns 2 (l % 4) and the
// next, v[0] and v[1] of TMEM lane l / 4, v[2] and v[3] of lane 8 + l / 4; the
// same of columns 8 further on in v[4] to v[7].
__device__ __forceinline__ void tmem_ld(uint32_t addr, float (&v)[8]) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7])
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

// Four 8 x 8 matrices of 16-bit values, transposed on their way: lane l holds, of
// matrix m, elements (l / 4, 2 (l % 4)) and the next in v[m]; in shared memory
// lane 8 m + i points at what is row i there and was column i here.
__device__ __forceinline__ void store_matrices(uint32_t addr, const uint32_t (&v)[4]) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr),
               "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3])
               : "memory");
}
__device__ __forceinline__ void load_matrices(uint32_t addr, uint32_t (&v)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ float load_float(uint32_t addr) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint4 load_shared(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ void store_shared(uint32_t addr, const uint4& v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y),
               "r"(v.z), "r"(v.w)
               : "memory");
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
  uint64_t drain;                    // after a wait that ran out: the products issued are done
  uint32_t tmem;
  uint32_t stop;                     // a wait ran out: every role leaves its loop
  // the same of the pair's other block, told when its roles have left; stages
  // whose loads a loader that left early had issued at most, here and there
  uint32_t peer_stop;
  int32_t issued, peer_issued;
  int32_t start[kMaxExperts + 2];    // first row of each group; the unused rows are the last
  int32_t tile[kMaxExperts + 2];     // tiles before each group
  uint8_t per[kMaxExperts + 1];      // rows of each group's tiles, in sixteens less one
};
static_assert(sizeof(Shared) <= kStaticBytes, "stages and staging take the rest");

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
      sh.per[g] = static_cast<uint8_t>(per / 16 - 1);
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
      per = (sh.per[group] + 1) * 16;
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

// The results are rounded to 8 bits: exp within 2 + 1.173 |a| units in the last
// of 24 (105 where it overflows, 2^-16), the reciprocal within one, below 2^-126 (a
// under -87.3) 0.  1 / inf is 0.
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
  // a bit per stage: dw's tail[] phase to come, and whether the last load counts on it
  uint32_t tail_parity = 0, tails = 0;
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
      if (kOp == kExpertDw) {
        const uint32_t bit = 1u << at.stage;
        tails = tail ? tails | bit : tails & ~bit;
        if (tail) tail_parity ^= bit;
      }
      if (tail) bar = smem_addr(&sh.tail[at.stage]);
      if constexpr (kLoadsA) {
        if (tail)
          mbar_arrive_expect_tx(&sh.tail[at.stage], bytes);
        else if (first)
          mbar_arrive_expect_tx(full, kPair * bytes);
        else if (kOp == kExpertDw)
          mbar_arrive_first(full);
        if (kOp == kExpertForward) {
          if (kFused && !p.pieces)
            tma_5d<kPair>(a, map, c, 0, 0, t.feature / 8, t.group, bar);
          else if (kFused)
            for (int i = 0; i < kTileM / 8; ++i)
              tma_3d<kPair>(a + i * 8 * kRowBytes, map, c,
                            t.feature + i / 2 * 8 + (i & 1 ? static_cast<int>(p.e.n) : 0), t.group,
                            bar);
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
  // What is under way writes this block's shared memory: the products of the
  // last stages have read it, or after a wait that ran out it is seen to land,
  // tails here and the rest in settle().
  for (int i = issued > p.stages ? issued - p.stages : 0; alive && i < issued; ++i)
    alive = wait(p, sh, &sh.empty[i % p.stages], (i / p.stages) & 1);
  if (alive) return;
  atomicMax(&sh.issued, issued);
  for (int i = 0; i < p.stages; ++i)
    if ((tails >> i & 1) &&
        !mbar_wait_bounded(&sh.tail[i], (tail_parity >> i & 1) ^ 1, kLandNs))
      break;
}

// After a wait that ran out in either block of a pair, when the roles of both
// have left: nothing of theirs may still be under way when shared memory and
// TMEM go.  The products issued are seen to end by both blocks.  The loads count on
// the first block's barriers: it waits for every stage that a loader of either
// block has issued and the products have not taken.  Where another loader left
// before its part of a stage the wait runs out, which leaves the others' loads
// kLandNs to land, a thousand times what they take.
template <int kPair>
__device__ void settle(const TcParams& p, Shared& sh) {
  const int warp = threadIdx.x >> 5;
  const bool first = kPair == 1 || cluster_rank() == 0;
  if (warp > 1 || !one_lane()) return;
  if (warp == 1) {  // the lane that issued the products
    if (first) mma_commit<kPair>(&sh.drain);
    mbar_wait_bounded(&sh.drain, 0, kLandNs);
  } else if (first) {
    const int issued = max(sh.issued, sh.peer_issued);
    for (int i = issued > p.stages ? issued - p.stages : 0; i < issued; ++i)
      if (!mbar_wait_bounded(&sh.full[i % p.stages], (i / p.stages) & 1, kLandNs)) break;
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
    bool alive = wait(p, sh, &sh.acc_empty[buffer], ((tiles >> 1) & 1) ^ 1);
    tc_fence_after();
    const uint32_t d = tmem + buffer * kMaxN;
    const int n = padded<kPair>(t.rows);
    const uint32_t idesc = instruction(kE4m3, kARows, kBRows, kTileM * kPair, n);
    uint32_t accumulate = 0;
    for (int c = 0; alive && c < t.depth; c += kDepth) {
      const int stage = at.stage;
      alive = wait(p, sh, &sh.full[stage], at.parity);
      if (!alive) break;
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
    if (!alive) return;
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
// Storing warps.  A chunk is 16 rows of a quarter's 32 lanes; two or three warps
// share a quarter (a warp can read only the TMEM lanes of its number modulo 4)
// and take chunks in turn.  They come out of TMEM as fragments of 8 x 8 matrices
// with the features along the matrices' rows; rounded, they are transposed on
// their way into the warp's shared memory, and 16 bytes of a row at a time go on
// to the output.  What the gated unit's gradient reads takes the same way back.
// (Sixteen 2-byte stores of a thread's feature: 147 instead of 137 us for the
// e4m3 product of 64225 rows, 1024 to 2048.  That product is bound by this chain
// of steps: 6.0 thousand cycles a tile, of which the products take 4.1.)  Large groups' plain outputs leave
// by TMA, whose 64-byte swizzle is the order in which they lie there, where the
// chunk's rows are all the group's: the load and store units, which the
// matrices and the scales' shuffles need, see no global store.
//
// Gradients of weights from few rows an expert leave two chunks at a time: the
// wait for TMEM, the fence and the copy's issue take 590 cycles in turn whether
// 16 rows or 32 go, and short contractions, or a last tile of few features, wait
// for them.  64 experts' 2048 x 2048, one chunk and two, in us: 16 rows an expert
// 112.6, 92.2; 128 rows 118.8, 98.3; 256 rows 131.1, 124.9; 384 rows 155.7, 155.6;
// 512 rows 188.4, 198.7; 1003 rows 309, 318.  128 experts' 4528 x 272 from 37 rows
// 133, 96; but 512 x 2264, whose rows start inside 32-byte sectors, 78, 84.  The
// other products, whose contractions are long, lose by it (2 x 1024 features of
// 64225 rows 329, 351).
//
// Outputs whose rows do not start on 16-byte boundaries, and the weights'
// gradients in 32 bits or added to, are stored value by value: 64 experts' 2048 x
// 2048 from 65536 rows 322 us in bf16, 406 in 32 bits, 616 added to 32 bits, and
// 1440 added to bf16, whose 2-byte words are read and written one by one.

constexpr int kChunk = 16;

// Place of row r's 16-byte piece p in a chunk of 16 rows of 4 pieces, or of 2:
// eight rows of one piece lie in different banks.
__device__ __forceinline__ uint32_t piece4(int r, int p) { return r * 64 + ((p ^ (r >> 1 & 3)) << 4); }
__device__ __forceinline__ uint32_t piece2(int r, int p) { return r * 32 + ((p ^ (r >> 2 & 1)) << 4); }

// 16 rows of 32 features, v[2 fb + cb] the fragment of features 8 fb and rows
// 8 cb, to shared memory.
__device__ __forceinline__ void stage32(uint32_t buf, const uint32_t (&v)[8]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int cb = 0; cb < 2; ++cb) {
    const uint32_t m[4] = {v[cb], v[2 + cb], v[4 + cb], v[6 + cb]};
    store_matrices(buf + piece4(cb * 8 + (lane & 7), lane >> 3), m);
  }
}

// And on to the output, of which `rows` and `features` are.
__device__ __forceinline__ void put32(uint32_t buf, uint16_t* out, int64_t stride,
                                      const uint32_t (&v)[8], int rows, int64_t features) {
  const int lane = threadIdx.x & 31;
  stage32(buf, v);
  __syncwarp();
  const int piece = lane & 3;
#pragma unroll
  for (int cb = 0; cb < 2; ++cb) {
    const int r = cb * 8 + (lane >> 2);
    const uint4 w = load_shared(buf + piece4(r, piece));
    if (r < rows && piece * 8 < features)
      *reinterpret_cast<uint4*>(out + r * stride + piece * 8) = w;
  }
  __syncwarp();
}

// 16 rows of 16 features, v[2 fb + cb].
__device__ __forceinline__ void put16(uint32_t buf, uint16_t* out, int64_t stride,
                                      const uint32_t (&v)[4], int rows, int64_t features) {
  const int lane = threadIdx.x & 31;
  // matrix 2 fb + cb
  store_matrices(buf + piece2((lane >> 3 & 1) * 8 + (lane & 7), lane >> 4), v);
  __syncwarp();
  const int r = lane >> 1, piece = lane & 1;
  const uint4 w = load_shared(buf + piece2(r, piece));
  if (r < rows && piece * 8 < features) *reinterpret_cast<uint4*>(out + r * stride + piece * 8) = w;
  __syncwarp();
}

// The same value by value: v[2 fb + cb]'s two values are rows 8 cb + 2 (lane % 4)
// and the next of feature 8 fb + lane / 4.
template <int kBlocks>
__device__ __forceinline__ void put_values(uint16_t* out, int64_t stride,
                                           const uint32_t (&v)[2 * kBlocks], int rows,
                                           int64_t features) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int fb = 0; fb < kBlocks; ++fb)
#pragma unroll
    for (int cb = 0; cb < 2; ++cb) {
      const int f = fb * 8 + (lane >> 2), r = cb * 8 + 2 * (lane & 3);
      if (f < features && r < rows) out[r * stride + f] = static_cast<uint16_t>(v[2 * fb + cb]);
      if (f < features && r + 1 < rows)
        out[(r + 1) * stride + f] = static_cast<uint16_t>(v[2 * fb + cb] >> 16);
    }
}

// Row of x behind grouped row r; -1: none.
__device__ __forceinline__ int64_t scale_row(const ExpertParams& e, int64_t r) {
  const int64_t x = e.row_tokens ? e.row_tokens[r] : r;
  return x < e.x_rows ? x : -1;
}

__device__ __forceinline__ bool on_words(const void* p, int64_t stride) {
  return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && (stride & 7) == 0;
}

template <int kOp, bool kGated, bool kE4m3, int kPair>
__device__ void store_tiles(const TcParams& p, const CUtensorMap* map_y, Shared& sh,
                            uint32_t staging) {
  constexpr bool kFused = kOp == kExpertForward && kGated;
  constexpr bool kReadsPre = kOp == kExpertDx && kGated;
  const ExpertParams& e = p.e;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, quadrant = warp & 3;
  using R = Roles<kPair>;
  constexpr int kStores = kReadsPre ? 8 : R::kStoreWarps;
  constexpr int kTurns = kStores / 4;             // warps of a quarter
  constexpr int kStride = kTurns * kChunk;        // rows from chunk to chunk
  constexpr int kScales = (kMaxN / kChunk + 2 * kTurns - 1) / (2 * kTurns);
  const int first_row = ((warp - 2) >> 2) * kChunk;
  constexpr int kOwn = kE4m3 ? 1024 : 2048;
  static_assert(kStores * kOwn <= (kE4m3 ? kOutputBytes : kStagingBytes), "the warps' memory");
  const uint32_t buf = staging + (warp - 2) * kOwn, buf_up = buf + 1024;
  const int64_t features = kOp == kExpertForward ? e.n : e.k;
  uint16_t* y = static_cast<uint16_t*>(e.y);
  const bool wide =
      (features & 7) == 0 && on_words(y, kOp == kExpertDw ? e.y_stride | e.y_expert_stride : 0) &&
      on_words(e.pre_out, 0) && on_words(e.pre_in, 0);
  // What the outputs need besides the products is fetched ahead: e4m3's scales
  // for the next tile while this one is stored, into shared memory (32 features'
  // or 16 gates' and 16 ups', then rows: word 32 + 32 q + l is that of row l % 16
  // of this warp's chunk 2 q + l / 16), and the gated unit's inputs for the first
  // chunk before the products, then one chunk ahead (rows lane / 4 and 8 more,
  // features 8 (lane % 4) on).  Loads of scales into registers were waited for in
  // every first chunk, 2000 cycles a tile.
  constexpr int kOwnScales = 128 * (1 + kScales);
  static_assert(kStores * kOwnScales <= kScaleBytes, "the scales' memory");
  const uint32_t scales_at = staging + kOutputBytes + (warp - 2) * kOwnScales;
  const auto fetch_scales = [&](const OutTile& t) {
    const int64_t f0 = t.feature + quadrant * (kFused ? 16 : 32) + (kFused ? lane & 15 : lane);
    const float* ws = e.w_scale + static_cast<int64_t>(t.group) * (kFused ? 2 : 1) * e.n;
    copy4(scales_at + lane * 4, ws + min(f0, features - 1) + (kFused && lane >= 16 ? e.n : 0), 4);
#pragma unroll
    for (int q = 0; q < kScales; ++q) {
      const int at = first_row + (2 * q + (lane >> 4)) * kStride + (lane & 15);
      const int64_t x = at < t.rows ? scale_row(e, static_cast<int64_t>(t.row) + at) : -1;
      copy4(scales_at + 128 + q * 128 + lane * 4, e.x_scale + (x < 0 ? 0 : x), x < 0 ? 0 : 4);
    }
  };
  uint4 gate_in[2], up_in[2];
  const auto fetch_pre = [&](const OutTile& t, int c) {
    const int64_t f0 = t.feature + quadrant * 32 + (lane & 3) * 8, f = min(f0, features - 8);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      // the last row stands in for rows behind the tile
      const int64_t r = t.row + min(c + i * 8 + (lane >> 2), t.rows - 1);
      const uint16_t* pre = e.pre_in + r * 2 * e.k + f;
      gate_in[i] = *reinterpret_cast<const uint4*>(pre);
      up_in[i] = *reinterpret_cast<const uint4*>(pre + e.k);
    }
  };
  int tiles = 0;
  Walk<kOp, kPair, kFused> walk;
  OutTile t, next;
  bool have = walk.next(p, sh, next);
  if (kE4m3 && have && next.depth > 0) fetch_scales(next);
  while (have) {
    t = next;
    const int64_t f0 = t.feature + quadrant * (kFused ? 16 : 32);  // the warp's first feature
    const int64_t left_f = features - f0;
    const int buffer = tiles & 1;
    const bool zero = t.depth == 0;
    have = walk.next(p, sh, next);
    if (!zero) {
      if (kReadsPre && wide && first_row < t.rows) fetch_pre(t, first_row);
      if (!wait(p, sh, &sh.acc_full[buffer], (tiles >> 1) & 1)) break;
      tc_fence_after();
      ++tiles;
    }
    float row[kScales], scale[4];
    if (kE4m3) {
      copy_wait_all();
      __syncwarp();
#pragma unroll
      for (int q = 0; q < kScales; ++q) row[q] = load_float(scales_at + 128 + q * 128 + lane * 4);
#pragma unroll
      for (int i = 0; i < 4; ++i)  // of the fragments' features: 8 i on, or gate and up of 8 (i / 2) on
        scale[i] = load_float(scales_at + 4 * ((kFused ? (i & 1) * 16 + i / 2 * 8 : i * 8) +
                                               (lane >> 2)));
      __syncwarp();
      if (have && next.depth > 0) fetch_scales(next);
    }
    const uint32_t acc =
        sh.tmem + buffer * kMaxN + (static_cast<uint32_t>(quadrant * 32) << 16);
    int rows = left_f > 0 ? t.rows : 0;  // a warp behind the last feature stores none
    if constexpr (kOp == kExpertDw)
      if (p.bulk == 2) {
#pragma unroll 1
        for (int c = 2 * first_row; c < rows; c += 2 * kStride) {
          float v[4][8] = {};
          if (!zero) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              tmem_ld(acc + (static_cast<uint32_t>(16 * (i & 1)) << 16) + c + (i >> 1) * kChunk, v[i]);
            tmem_ld_wait();
          }
          uint32_t out[2][8];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float* w = v[i >> 3 << 1 | (i >> 2 & 1)] + (i & 1) * 4 + (i >> 1 & 1) * 2;
            out[i >> 3][i & 7] = pack_bf16(w[0], w[1]);
          }
          if (lane == 0) bulk_wait_read_all();  // the copy before has read the buffer
          __syncwarp();
          stage32(buf, out[0]);
          stage32(buf_up, out[1]);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_3d(map_y, buf, static_cast<int>(f0), t.row + c, t.group);
            bulk_commit();
          }
        }
        rows = 0;  // all stored
      }
#pragma unroll 1
    for (int c = first_row, chunk = 0; c < rows; c += kStride, ++chunk) {
      const int left = t.rows - c;
      const int64_t r = t.row + c;
      // v[h][4 cb + i]: lanes 16 h + 8 (i / 2) + lane / 4, rows 8 cb + 2 (lane % 4) + i % 2
      float v[2][8];
      if (zero) {
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i / 8][i % 8] = 0.0f;
      } else {
        tmem_ld(acc + c, v[0]);
        tmem_ld(acc + (16u << 16) + c, v[1]);
        tmem_ld_wait();
        if (kE4m3) {
          float scales = row[0];
#pragma unroll
          for (int q = 1; q < kScales; ++q)
            if (chunk >> 1 == q) scales = row[q];
          const int from = (chunk & 1) * kChunk + 2 * (lane & 3);
#pragma unroll
          for (int i = 0; i < 4; ++i) {  // row 8 (i / 2) + i % 2 further on
            const float xs = __shfl_sync(0xffffffffu, scales, from + (i >> 1) * 8 + (i & 1));
            const int at = (i >> 1) * 4 + (i & 1);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              v[h][at] *= xs * scale[2 * h];
              v[h][at + 2] *= xs * scale[2 * h + 1];
            }
          }
        }
      }
      if constexpr (kFused) {
        uint32_t gate[4], up[4], out[4];  // of features 8 h and rows 8 cb at 2 h + cb
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float* w = v[i >> 1] + (i & 1) * 4;
          gate[i] = pack_bf16(w[0], w[1]);
          up[i] = pack_bf16(w[2], w[3]);
          out[i] = pack_bf16(silu(w[0]) * w[2], silu(w[1]) * w[3]);
        }
        uint16_t* pre = e.pre_out + r * 2 * e.n + f0;
        uint16_t* to = y + r * e.n + f0;
        if (wide) {
          if (e.pre_out) {
            put16(buf, pre, 2 * e.n, gate, left, left_f);
            put16(buf, pre + e.n, 2 * e.n, up, left, left_f);
          }
          put16(buf, to, e.n, out, left, left_f);
        } else {
          if (e.pre_out) {
            put_values<2>(pre, 2 * e.n, gate, left, left_f);
            put_values<2>(pre + e.n, 2 * e.n, up, left, left_f);
          }
          put_values<2>(to, e.n, out, left, left_f);
        }
        continue;
      }
      uint32_t out[8];  // of features 8 fb and rows 8 cb at 2 fb + cb
      if constexpr (kReadsPre) {
        uint32_t gate[8] = {}, up[8] = {};
        if (!zero && wide) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t at = piece4(i * 8 + (lane >> 2), lane & 3);
            store_shared(buf + at, gate_in[i]);
            store_shared(buf_up + at, up_in[i]);
          }
          if (c + kStride < t.rows) fetch_pre(t, c + kStride);
          __syncwarp();
#pragma unroll
          for (int cb = 0; cb < 2; ++cb) {
            const uint32_t at = piece4(cb * 8 + (lane & 7), lane >> 3);
            uint32_t m[4];
            load_matrices(buf + at, m);
#pragma unroll
            for (int fb = 0; fb < 4; ++fb) gate[2 * fb + cb] = m[fb];
            load_matrices(buf_up + at, m);
#pragma unroll
            for (int fb = 0; fb < 4; ++fb) up[2 * fb + cb] = m[fb];
          }
          __syncwarp();
        } else if (!zero) {
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int64_t f = min(f0 + (i >> 2) * 8 + (lane >> 2), features - 1);
            const int64_t at = t.row + min(c + (i >> 1 & 1) * 8 + 2 * (lane & 3) + (i & 1),
                                           t.rows - 1);
            const uint16_t* pre = e.pre_in + at * 2 * e.k + f;
            gate[i >> 1] |= static_cast<uint32_t>(pre[0]) << (16 * (i & 1));
            up[i >> 1] |= static_cast<uint32_t>(pre[e.k]) << (16 * (i & 1));
          }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float* d = v[i >> 2] + (i & 1) * 4 + (i >> 1 & 1) * 2;
          float dg[2], du[2];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float g = j ? bf16_hi(gate[i]) : bf16_lo(gate[i]);
            const float u = j ? bf16_hi(up[i]) : bf16_lo(up[i]);
            const float s = sigmoid(g), ds = d[j] * s;
            du[j] = ds * g;
            dg[j] = ds * u * (1.0f + g * (1.0f - s));
          }
          out[i] = zero ? 0u : pack_bf16(dg[0], dg[1]);
          up[i] = zero ? 0u : pack_bf16(du[0], du[1]);
        }
        uint16_t* to = y + r * 2 * e.k + f0;
        if (wide) {
          put32(buf, to, 2 * e.k, out, left, left_f);
          put32(buf_up, to + e.k, 2 * e.k, up, left, left_f);
        } else {
          put_values<4>(to, 2 * e.k, out, left, left_f);
          put_values<4>(to + e.k, 2 * e.k, up, left, left_f);
        }
        continue;
      }
      if (kOp == kExpertDw && (e.f32_out || e.accumulate)) {
        const int64_t base = t.group * e.y_expert_stride + r * e.y_stride + f0;
        // one row of eight features at a time: i counts (h, cb, second lanes, second row)
        float old[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int f = (i >> 3) * 16 + (i >> 1 & 1) * 8 + (lane >> 2);
          const int rr = (i >> 2 & 1) * 8 + 2 * (lane & 3) + (i & 1);
          const int64_t at = base + rr * e.y_stride + f;
          old[i] = 0.0f;
          if (e.accumulate && rr < left && f < left_f)
            old[i] = e.f32_out ? static_cast<const float*>(e.y)[at] : bf16_to_f32(y[at]);
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int f = (i >> 3) * 16 + (i >> 1 & 1) * 8 + (lane >> 2);
          const int rr = (i >> 2 & 1) * 8 + 2 * (lane & 3) + (i & 1);
          const int64_t at = base + rr * e.y_stride + f;
          const float sum = old[i] + v[i >> 3][i & 7];
          if (rr < left && f < left_f) {
            if (e.f32_out)
              static_cast<float*>(e.y)[at] = sum;
            else
              y[at] = f32_to_bf16(sum);
          }
        }
        continue;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float* w = v[i >> 2] + (i & 1) * 4 + (i >> 1 & 1) * 2;
        out[i] = pack_bf16(w[0], w[1]);
      }
      if (p.bulk) {  // the copy before has read the buffer
        if (lane == 0) bulk_wait_read_all();
        __syncwarp();
      }
      if (p.bulk && (kOp == kExpertDw || left >= kChunk)) {
        stage32(buf, out);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          if (kOp == kExpertDw)
            tma_store_3d(map_y, buf, static_cast<int>(f0), static_cast<int>(r), t.group);
          else
            tma_store_2d(map_y, buf, static_cast<int>(f0), static_cast<int>(r));
          bulk_commit();
        }
        continue;
      }
      const int64_t stride = kOp == kExpertDw ? e.y_stride : features;
      uint16_t* to =
          y + (kOp == kExpertDw ? t.group * e.y_expert_stride : 0) + r * stride + f0;
      if (wide)
        put32(buf, to, stride, out, left, left_f);
      else
        put_values<4>(to, stride, out, left, left_f);
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
  // nothing of this warp's is under way when its block's memory goes
  if (kE4m3) copy_wait_all();
  if (p.bulk && lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

template <int kOp, bool kGated, bool kE4m3, int kPair>
__global__ void __launch_bounds__(Roles<kPair>::kThreads, 1)
    k_expert_tc(const TcParams p, const __grid_constant__ CUtensorMap map_a,
                const __grid_constant__ CUtensorMap map_b,
                const __grid_constant__ CUtensorMap map_y) {
  extern __shared__ unsigned char raw[];
  __shared__ Shared sh;
  // stages on 1024-byte boundaries: the swizzle's period; then the storing warps' memory
  const uint32_t base = smem_addr(raw);
  const uint32_t ring = (base + 1023) & ~1023u;
  const uint32_t staging = ring + p.stages * p.stage_bytes;
  unsigned char* ring_ptr = raw + (ring - base);
  // storing warps at work (see kStagingBytes)
  constexpr int kStores = kOp == kExpertDx && kGated ? 8 : Roles<kPair>::kStoreWarps;
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
      mbar_init(&sh.acc_empty[i], kStores * kPair);
    }
    mbar_init(&sh.drain, 1);
    sh.stop = sh.peer_stop = 0;
    sh.issued = sh.peer_issued = 0;
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
  else if (warp >= 2 && warp < 2 + kStores)
    store_tiles<kOp, kGated, kE4m3, kPair>(p, &map_y, sh, staging);
  else if (warp == kLoadB && !gather)
    load_tiles<kOp, kGated, kE4m3, kPair, false>(p, &map_b, sh, ring);
  else if (warp > kLoadB && kOp == kExpertDw)
    clear_tails(p, sh, ring_ptr);
  else if (warp > kLoadB && gather)
    gather_tiles<kGated, kE4m3>(p, sh, ring);
  tc_fence_before();
  __syncthreads();
  if (kPair == 2 && threadIdx.x == 0 && sh.stop) {
    store_peer(&sh.peer_issued, static_cast<uint32_t>(sh.issued));
    store_peer(&sh.peer_stop, 1);
  }
  sync_all<kPair>();
  if (*const_cast<volatile uint32_t*>(&sh.stop) | *const_cast<volatile uint32_t*>(&sh.peer_stop)) {
    settle<kPair>(p, sh);
    __syncthreads();
    sync_all<kPair>();
  }
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
// dimension); boxes of 128 bytes by box_rows.  With part_stride a box is eight
// rows of the first part and the same eight of the second, part_stride further
// on, in turn (rows a multiple of 8).
bool make_map(CUtensorMap* map, const void* base, bool e4m3, int64_t columns, int64_t rows,
              int64_t stride, int64_t planes, int64_t plane_stride, int box_rows,
              int64_t part_stride = 0) {
  const int64_t size = e4m3 ? 1 : 2;
  if ((reinterpret_cast<uintptr_t>(base) & 15) || stride * size % 16 ||
      (planes > 1 && (plane_stride * size % 16 || plane_stride <= 0)) || columns < 1 || rows < 1)
    return false;
  cuuint64_t dims[5], strides[4];
  cuuint32_t box[5];
  const cuuint32_t ones[5] = {1, 1, 1, 1, 1};
  int rank = 0;
  const auto add = [&](int64_t n, int64_t apart, int64_t of_box) {
    if (rank) strides[rank - 1] = static_cast<cuuint64_t>(apart * size);
    dims[rank] = static_cast<cuuint64_t>(n);
    box[rank++] = static_cast<cuuint32_t>(of_box);
  };
  add(columns, 0, kRowBytes / size);
  if (part_stride) {
    add(8, stride, 8);
    add(2, part_stride, 2);
    add(rows / 8, 8 * stride, box_rows / 16);
  } else {
    add(rows, stride, box_rows);
  }
  if (planes > 0) add(planes, planes > 1 ? plane_stride : stride * rows * 2, 1);
  return encode()(map, e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                  static_cast<cuuint32_t>(rank), const_cast<void*>(base), dims, strides, box, ones,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A map of bf16 outputs, boxes of box_rows rows of 32 features.
bool make_out_map(CUtensorMap* map, void* base, int64_t columns, int64_t rows, int64_t stride,
                  int64_t planes, int64_t plane_stride, int box_rows) {
  if (planes > 1 && plane_stride <= 0) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(columns), static_cast<cuuint64_t>(rows),
                              static_cast<cuuint64_t>(planes)};
  const cuuint64_t strides[2] = {
      static_cast<cuuint64_t>(2 * stride),
      static_cast<cuuint64_t>(2 * (planes > 1 ? plane_stride : stride * rows))};
  const cuuint32_t box[3] = {32, static_cast<cuuint32_t>(box_rows), 1}, ones[3] = {1, 1, 1};
  return encode()(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, planes ? 3 : 2, base, dims, strides, box,
                  ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B,
                  CU_TENSOR_MAP_L2_PROMOTION_NONE,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Maps {
  CUtensorMap a, b, y;
};

template <int kOp, bool kGated, bool kE4m3, int kPair>
int launch_at(const TcParams& p, const Maps& m, int grid, cudaStream_t s) {
  const cudaError_t err =
      allow_shared<k_expert_tc<kOp, kGated, kE4m3, kPair>>(kSmemLimit - kStaticBytes);
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t config{};
  config.gridDim = dim3(static_cast<unsigned>(grid));
  config.blockDim = dim3(Roles<kPair>::kThreads);
  config.dynamicSmemBytes = static_cast<size_t>(p.stages) * p.stage_bytes + 1024 + kStagingBytes;
  config.stream = s;
  cudaLaunchAttribute pair{};
  pair.id = cudaLaunchAttributeClusterDimension;
  pair.val.clusterDim.x = 2;
  pair.val.clusterDim.y = pair.val.clusterDim.z = 1;
  config.attrs = &pair;
  config.numAttrs = kPair == 2 ? 1 : 0;
  return cudaLaunchKernelEx(&config, k_expert_tc<kOp, kGated, kE4m3, kPair>, p, m.a, m.b, m.y);
}

template <int kPair>
int launch_with(const TcParams& p, const Maps& m, int grid, cudaStream_t s) {
  const ExpertParams& e = p.e;  // dw always takes pairs
  if (e.op == kExpertForward) {
    if (e.e4m3)
      return e.gated ? launch_at<kExpertForward, true, true, kPair>(p, m, grid, s)
                     : launch_at<kExpertForward, false, true, kPair>(p, m, grid, s);
    return e.gated ? launch_at<kExpertForward, true, false, kPair>(p, m, grid, s)
                   : launch_at<kExpertForward, false, false, kPair>(p, m, grid, s);
  }
  if (e.op == kExpertDx)
    return e.gated ? launch_at<kExpertDx, true, false, kPair>(p, m, grid, s)
                   : launch_at<kExpertDx, false, false, kPair>(p, m, grid, s);
  return launch_at<kExpertDw, false, false, 2>(p, m, grid, s);
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
  p.stages = (kSmemLimit - kStaticBytes - kStagingBytes - 1024) / p.stage_bytes;
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
  p.pieces = fused && e.n % 8 != 0;

  Maps m;
  CUtensorMap &a = m.a, &b = m.b;
  bool ok;
  if (e.op == kExpertForward)
    // gates and ups in turn: one load, or where n is no multiple of 8 sixteen
    // of eight rows each, which may read past the gates (into the ups: not
    // stored) but not past an expert's last row
    ok = (!fused     ? make_map(&a, e.w, e.e4m3, e.k, e.n, e.w_stride, e.experts,
                                e.w_expert_stride, kTileM)
          : p.pieces ? make_map(&a, e.w, e.e4m3, e.k, 2 * e.n, e.w_stride, e.experts,
                                e.w_expert_stride, 8)
                     : make_map(&a, e.w, e.e4m3, e.k, e.n, e.w_stride, e.experts,
                                e.w_expert_stride, kTileM, e.n * e.w_stride)) &&
         make_map(&b, e.x, e.e4m3, e.k, e.x_rows, e.x_stride, 0, 0, kBoxRows);
  else if (e.op == kExpertDx)
    ok = make_map(&a, e.w, false, e.k, e.n, e.w_stride, e.experts, e.w_expert_stride, 64) &&
         make_map(&b, e.x, false, e.n, e.x_rows, e.x_stride, 0, 0, kBoxRows);
  else
    ok = make_map(&a, e.x, false, e.k, e.x_rows, e.x_stride, 0, 0, 64) &&
         make_map(&b, e.w, false, e.n, e.rows, e.w_stride, 0, 0, 64);
  if (!ok) return false;
  const bool shallow = e.rows <= kShallowRows * static_cast<int64_t>(e.experts);
  // plain bf16 outputs of large groups leave by TMA where their rows are words
  if (pair == 2 && !e.gated && !e.f32_out && !e.accumulate && features % 8 == 0 &&
      (reinterpret_cast<uintptr_t>(e.y) & 15) == 0) {
    if (e.op != kExpertDw)
      p.bulk = make_out_map(&m.y, e.y, features, e.rows, features, 0, 0, kChunk);
    else if (e.y_stride % 8 == 0 && e.y_expert_stride % 8 == 0 &&
             make_out_map(&m.y, e.y, e.k, e.n, e.y_stride, e.experts, e.y_expert_stride,
                          shallow ? 2 * kChunk : kChunk))
      p.bulk = shallow ? 2 : 1;
  }
  if (!p.bulk) m.y = m.b;  // not used

  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int64_t most = m_tiles * row_tiles, slots = sm_count() / pair;
  const int grid = static_cast<int>(most < slots ? most : slots) * pair;
  *status = pair == 2 ? launch_with<2>(p, m, grid, s) : launch_with<1>(p, m, grid, s);
  return true;
}

}  // namespace ciera
