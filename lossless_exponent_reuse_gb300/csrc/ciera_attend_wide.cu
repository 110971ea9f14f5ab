// ciera_attend_wide.cu -- attention of many rows a head over pages, on the
// tensor cores (tcgen05).
//
// A persistent block per SM takes 256 rows, in two halves of 128, over units of up
// to 128 keys.  Two warps bring pages' keys and values into a ring of stages by TMA
// (128-byte swizzle; a box is a page, or the largest part of it that a tile holds
// in whole), one lane of another issues S = Q K^T and O += P V, and two groups of
// four warps, one to a half, a thread to a row, turn scores into weights: S from
// TMEM to registers, the running maximum and sum, and the weights in bf16 back to
// TMEM, over the scores, from where the products take them as their A operand, so
// that only keys, values and queries are read from shared memory.  O stays in TMEM;
// it is scaled only where a row's maximum has passed the one in use by 2^8, and
// then by the row's own thread.  While one half's weights are made, the other
// half's products run: S0 S1 | O0 S0' O1 S1' | ...  The products run in the order in
// which the one lane issues them: S0' overwrites the weights that O0 reads.
//
// Weights are rounded to bf16, 2^-8 of each at most and as often up as down: A and B of a
// product are of one type, and values have bf16's range, which fp16 with three bits more
// does not hold.  Their sum is of the 32-bit ones.
//
// Bound by the tensor cores while both halves have units: 1.45 us a unit of 256 x 128 x
// 128, 1759 TFLOP/s; a block's start (9 us), a tile's begin and end (4) and the join
// (5 to 9) come on top.  16 heads of 128: a prompt of 8192 tokens 207 to 214 us (1290 to
// 1330 TFLOP/s, with the clock that power leaves), 512 tokens behind 32256 with 32 heads
// to 4 190 to 193 (1420); 24 requests of 100 to 3000 cached keys and up to 300 new tokens,
// 24 heads to 8, 118 to 119, where some ten units a tile do not hide its begin, and
// queries of three heads to one come by ordinary copies.
//
// e4m3 pages come by TMA as they are; four warps more widen them to bf16, which
// holds every row times its power of two exactly (of an exponent of 3 and more, biased), into
// the ring's stages.
//
// A tile's last keys may lie in a page with others behind them, which hold
// anything: those values are cleared in shared memory before the products.  What a row
// does not see inside a unit has weight 0; where a row came out infinite or NaN the
// values between its last key and the half's are looked at, and where one of them is infinite
// or NaN the row is computed again, value by value.
#include "ciera_attend_device.cuh"
#include "ciera_tc_device.cuh"

namespace ciera {
namespace {

constexpr int kHalf = 128;              // rows of a half: lanes of TMEM
constexpr int kTileRows = 2 * kHalf;
constexpr int kKeys = 128;              // most keys of a unit
constexpr int kStep = 64;               // keys whose weights are handed on at once
constexpr int kRowBytes = 128;          // of a stage's row: 64 values
constexpr int kSoftmaxWarps = 8;
constexpr int kMultiplyWarp = kSoftmaxWarps;
constexpr int kLoadWarp = kSoftmaxWarps + 1;    // keys, and the next warp values
constexpr int kQueryWarp = kSoftmaxWarps + 3;
constexpr int kWidenWarp = kSoftmaxWarps + 4;   // e4m3: four
constexpr float kSlack = 8.0f;
constexpr uint64_t kLandNs = 100000000;  // limit for what is under way when a wait ran out
constexpr int kMostStages = 8;
constexpr int kTmemColumns = 512;       // S0 S1 O0 O1, 128 each
constexpr int kJoinColumns = 16;        // of a block of the launch that joins
constexpr int kJoinGroups = 2;

// Registers a thread: bf16 has three groups of four warps, 168 at launch, 64512 in
// all: 200 for the two that hold a row's scores, 104 for the third, 64512.  e4m3
// has four groups, 128 at launch, 65536: 184, 184, 72 and 72, 65536.
template <int kDim, bool kE4m3 = false>
struct Form {
  static constexpr int kThreads = 32 * (kSoftmaxWarps + (kE4m3 ? 8 : 4));
  static constexpr int kHalves = kDim / 64;                       // columns of 64 values
  static constexpr int kTileBytes = kHalves * kKeys * kRowBytes;  // a stage; half the queries
  static constexpr int kStages = kDim == 128 ? kE4m3 ? 4 : 5 : 8;
  static constexpr int kRawBytes = kKeys * kDim;                  // e4m3: as loaded
  static constexpr int kRaw = kE4m3 ? 2 : 0;
  static constexpr int kSlots = kE4m3 ? kRaw : kStages;           // that TMA fills
  static constexpr int kSmem = (2 + kStages) * kTileBytes + kRaw * kRawBytes + 1024;
};
template <int kDim>
constexpr int64_t kPartValues = kTileRows * (kDim + 2);

struct Shared {
  uint64_t full[kMostStages];
  uint64_t empty[kMostStages];
  uint64_t raw_full[2];    // e4m3
  uint64_t raw_empty[2];
  uint64_t queries[2];     // a half's queries are in shared memory
  uint64_t asked[2];       // and have been read for the last time
  uint64_t scores[2];      // its scores are in TMEM
  uint64_t weights[2][2];  // a step's weights are in TMEM, and the output as scaled
  uint64_t output[2][2];   // a step's weights have gone into the output
  uint64_t cleared;        // a tile's last values have zeros behind the last key
  uint64_t drain;          // after a wait that ran out: the products issued are done
  uint32_t tmem;
  uint32_t stop;           // a wait ran out: every role leaves
  uint32_t busy;           // warps that compute rows again: nobody's wait runs out meanwhile
  int32_t issued;          // loads
  int32_t moved[2];        // loads of keys, of values so far
  Share share;
  int64_t part[kSoftmaxWarps + 9];
};

// Bounded wait; false when it ran out here or anywhere in the block.  kTile: for what comes
// when a tile ends, all of whose units go on meanwhile (some 700 000 of them, 90 million
// keys, take a second): the limit is that of a block whose loads do not go on.
template <bool kTile>
__device__ __forceinline__ bool wait_on(const AttendParams& p, Shared& sh, uint64_t* bar,
                                        uint32_t parity) {
  if (mbar_try_wait(bar, parity)) return true;
  uint64_t t0 = globaltimer();
  int32_t moved = 0;
  while (!mbar_try_wait(bar, parity)) {
    if (*reinterpret_cast<volatile uint32_t*>(&sh.stop)) return false;
    const uint64_t now = globaltimer();
    if (*reinterpret_cast<volatile uint32_t*>(&sh.busy)) t0 = now;
    if (kTile) {
      const volatile int32_t* loads = sh.moved;
      const int32_t so_far = loads[0] + loads[1];
      if (so_far != moved) t0 = now;
      moved = so_far;
    }
    if (now - t0 > p.timeout_ns) {
      *reinterpret_cast<volatile uint32_t*>(&sh.stop) = 1;
      record_status(p.ctl, kStatusTimeout);
      return false;
    }
  }
  return true;
}
// The same for a whole warp, all of whose lanes go on or leave.
template <bool kTile = false>
__device__ __forceinline__ bool wait(const AttendParams& p, Shared& sh, uint64_t* bar,
                                     uint32_t parity) {
  return __all_sync(0xffffffffu, wait_on<kTile>(p, sh, bar, parity));
}

__device__ __forceinline__ void tma_4d(uint32_t dst, const CUtensorMap* map, int32_t x, int32_t y,
                                       int32_t z, int32_t u, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(u), "r"(smem_addr(bar))
      : "memory");
}

// Both operands in shared memory.
__device__ __forceinline__ void mma_shared(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// A in TMEM.
__device__ __forceinline__ void mma_tmem(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void commit(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
          smem_addr(bar))
      : "memory");
}

// 32 columns of this thread's TMEM lane.
__device__ __forceinline__ void tmem_load32(uint32_t addr, float* f) {
  uint32_t* r = reinterpret_cast<uint32_t*>(f);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, "
      "%30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
        "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_store32(uint32_t addr, const float* f) {
  const uint32_t* r = reinterpret_cast<const uint32_t*>(f);
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, "
      "%29, %30, %31, %32};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
      "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]),
      "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]),
      "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_store_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// Waits for the loads from TMEM; what they brought is not looked at before.
template <int kCount>
__device__ __forceinline__ void tmem_arrived(float* f) {
  tmem_ld_wait();
#pragma unroll
  for (int i = 0; i < kCount; i += 8)
    asm volatile(""
                 : "+f"(f[i]), "+f"(f[i + 1]), "+f"(f[i + 2]), "+f"(f[i + 3]), "+f"(f[i + 4]),
                   "+f"(f[i + 5]), "+f"(f[i + 6]), "+f"(f[i + 7]));
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// 16 values as bf16, 32 bytes at once or twice 16.
__device__ __forceinline__ void store16(uint16_t* to, const float* f, float by, bool at_once) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = pack_bf16(f[2 * i] * by, f[2 * i + 1] * by);
  if (at_once) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(w[0]),
                 "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    *reinterpret_cast<uint4*>(to) = make_uint4(w[0], w[1], w[2], w[3]);
    *reinterpret_cast<uint4*>(to + 8) = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

// Two sums or products at once.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)),
        "l"(reinterpret_cast<uint64_t&>(c)));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
  return d;
}

// What every role works out alike of a segment: each half's rows and units.
struct Halves {
  int32_t rows[2];
  int32_t units[2];
  int32_t most;
  __device__ Halves(const AttendParams& p, const Segment& s) {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int32_t left = s.rows - t * kHalf;
      rows[t] = left < 0 ? 0 : left < kHalf ? left : kHalf;
      units[t] = 0;
      if (rows[t] == 0) continue;
      const int32_t last = s.tile * kTileRows + t * kHalf + rows[t] - 1;
      const int32_t all = p.by_unit.up(seen_keys(s.request, p.by_group(last)));
      const int32_t n = (all < s.to ? all : s.to) - s.from;
      units[t] = n > 0 ? n : 0;
    }
    most = units[0] > units[1] ? units[0] : units[1];
  }
};

struct Maps {
  CUtensorMap key, value, query;
  int32_t query_box;  // tokens of a half's queries; 0: they come by ordinary copies
  int32_t box;       // keys of a box, which divide a page's
  Divide by_box;
};

// ------------------------------------------------------------------------
// Two warps: keys and values by TMA, stages in turn.  A lane per box: it looks up
// the page, a unit ahead, and issues the box's loads.  (One warp for both: with
// pages of 16 its 32 loads a unit took as long as the products.)
template <int kDim, bool kE4m3>
__device__ void load(const AttendParams& p, const Maps& maps, Shared& sh, uint32_t ring, int side) {
  using F = Form<kDim, kE4m3>;
  constexpr int kSlots = F::kSlots, kBytes = kE4m3 ? F::kRawBytes : F::kTileBytes;
  constexpr int kLine = kE4m3 ? kDim : kRowBytes;    // of a box
  uint64_t* const full = kE4m3 ? sh.raw_full : sh.full;
  uint64_t* const empty = kE4m3 ? sh.raw_empty : sh.empty;
  const int lane = threadIdx.x & 31;
  const int columns = kE4m3 ? 1 : (p.head_dim + 63) / 64;
  const CUtensorMap* map = side ? &maps.value : &maps.key;
  Walk<kTileRows> walk(p, sh.share);
  Segment s;
  int at = side;      // of all loads
  bool alive = true;
  while (alive && walk.next(p, &s)) {
    const Halves halves(p, s);
    const auto look = [&](int unit, int32_t* page, int32_t* place) {
      const int32_t key = (s.from + unit) * p.unit_keys + lane * maps.box;
      *page = p.pages;     // none: zeros
      *place = 0;
      if (unit >= halves.most || lane * maps.box >= p.unit_keys || key >= s.keys) return;
      const int32_t index = p.by_page(key), found = page_at(p, s.index, index);
      *place = key - index * p.page_size;
      if (found >= 0) *page = found;
    };
    int32_t page, place;
    look(0, &page, &place);
    for (int u = 0; u < halves.most; ++u, at += 2) {
      const int32_t left = s.keys - (s.from + u) * p.unit_keys;
      const int boxes = maps.by_box.up(left < p.unit_keys ? left : p.unit_keys);
      const int slot = at % kSlots;
      alive = wait(p, sh, &empty[slot], ((at / kSlots) & 1) ^ 1);
      if (!alive) break;
      if (lane == 0)
        mbar_arrive_expect_tx(&full[slot], static_cast<uint32_t>(boxes * columns * maps.box * kLine));
      if (lane == 0) *reinterpret_cast<volatile int32_t*>(&sh.moved[side]) = at;
      __syncwarp();
      if (lane < boxes) {
        const uint32_t to = ring + slot * kBytes + lane * maps.box * kLine;
        for (int c = 0; c < columns; ++c)
          tma_4d(to + c * kKeys * kRowBytes, map, c * 64, place, s.head, page, &full[slot]);
      }
      look(u + 1, &page, &place);
    }
  }
  // What is under way writes this block's shared memory: it has been read, or after
  // a wait that ran out it is seen to land (settle).
  const int first = at - 2 * kSlots;
  for (int i = first < side ? side : first; alive && i < at; i += 2)
    if (i >= at - kSlots) alive = wait(p, sh, &empty[i % kSlots], (i / kSlots) & 1);
  if (lane == 0) atomicMax(&sh.issued, at - 1);
}

// ------------------------------------------------------------------------
// Four warps, e4m3: rows as loaded to bf16, times their powers of two, where the
// 128-byte swizzle has them; zeros behind the tile's last key.  A warp takes 32
// rows of a tile, a lane 16 values of four rows in turn and the exponent of one row,
// fetched a stage ahead.  A value goes by way of fp16 and fp32, all of which hold
// it, so that most of the work is the multipliers'; the integer units, which the
// softmax needs, put two together (a prompt of 8192 tokens of 16 heads: 351 us, by
// moving bits 437; two or four rows at once, 380 and 373, spill; now 359).
__device__ __forceinline__ uint32_t times_bf16(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

template <int kDim>
__device__ void widen(const AttendParams& p, Shared& sh, unsigned char* ring, unsigned char* raw,
                      int warp) {
  using F = Form<kDim, true>;
  constexpr int kPieces = kDim / 16, kAtOnce = 32 / kPieces;   // of a row; rows
  const int lane = threadIdx.x & 31, piece = lane % kPieces;
  Walk<kTileRows> walk(p, sh.share);
  Segment s;
  int at = 0;
  while (walk.next(p, &s)) {
    const Halves h(p, s);
    // of this lane's row; 256: none, zeros
    const auto exponent = [&](int load) -> uint32_t {
      const int unit = load >> 1;
      const int32_t row = warp * 32 + lane, key = (s.from + unit) * p.unit_keys + row;
      if (unit >= h.most || row >= p.unit_keys || key >= s.keys) return 256;
      const int32_t index = p.by_page(key), page = page_at(p, s.index, index);
      if (page < 0) return 256;
      const int32_t place = key - index * p.page_size;
      const Side& side = load & 1 ? p.value : p.key;
      return side.exponent[page * side.exponent_stride[0] + place * side.exponent_stride[1] +
                           s.head * side.exponent_stride[2]];
    };
    uint32_t next = exponent(0);
    for (int load = 0; load < 2 * h.most; ++load, ++at) {
      const uint32_t own = next;
      next = exponent(load + 1);
      const int slot = at % F::kRaw, stage = at % F::kStages;
      if (!wait(p, sh, &sh.raw_full[slot], (at / F::kRaw) & 1)) return;
      if (!wait(p, sh, &sh.empty[stage], ((at / F::kStages) & 1) ^ 1)) return;
      const unsigned char* from = raw + slot * F::kRawBytes + warp * 32 * kDim;
      unsigned char* to = ring + stage * F::kTileBytes;
#pragma unroll 1
      for (int i = 0; i < 32 / kAtOnce; ++i) {
        const int r = i * kAtOnce + lane / kPieces, row = warp * 32 + r;
        const uint32_t e = __shfl_sync(0xffffffffu, own, r);
        const uint4 w = *reinterpret_cast<const uint4*>(from + r * kDim + piece * 16);
        const uint32_t words[4] = {w.x, w.y, w.z, w.w};
        uint32_t by = e == 255 ? 0x7FC0u : e ? e << 7 : 0x40u;   // the row's power
        by |= by << 16;
        uint32_t out[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t v = e == 256 ? 0u : words[j];
          out[2 * j] = times_bf16(e4m3_to_bf16<0>(v), by);
          out[2 * j + 1] = times_bf16(e4m3_to_bf16<1>(v), by);
        }
        unsigned char* line = to + (piece / 4) * kKeys * kRowBytes + row * kRowBytes;
        const int first = 2 * (piece & 3);
        *reinterpret_cast<uint4*>(line + ((first ^ (row & 7)) << 4)) =
            make_uint4(out[0], out[1], out[2], out[3]);
        *reinterpret_cast<uint4*>(line + (((first + 1) ^ (row & 7)) << 4)) =
            make_uint4(out[4], out[5], out[6], out[7]);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&sh.raw_empty[slot]);
        mbar_arrive(&sh.full[stage]);
      }
    }
  }
  // the products' last word on each stage comes by itself: it has come before this
  // block's shared memory is another's
  for (int i = at > F::kStages ? at - F::kStages : 0; warp == 0 && i < at; ++i)
    if (!wait(p, sh, &sh.empty[i % F::kStages], (i / F::kStages) & 1)) return;
}

// ------------------------------------------------------------------------
// One lane issues the products.  Everything that it does between two of them
// counts (65 cycles a product): the loops are unrolled, the operands' addresses
// differ by constants, and what has long been there is waited for ahead.
// (Loops with the whole warp: 85 to 120 cycles a product, 230 a wait.)
template <int kDim, bool kE4m3>
__device__ void multiply(const AttendParams& p, Shared& sh, uint32_t queries, uint32_t ring) {
  using F = Form<kDim, kE4m3>;
  if (!one_lane()) return;
  constexpr int kSteps = kDim / 16;
  const int steps = (p.head_dim + 15) / 16;               // of S
  const int key_steps = (p.unit_keys + 15) / 16;          // of O
  const uint32_t scores = instruction(false, false, false, kHalf, kKeys);
  const uint32_t output = instruction(false, false, true, kHalf, steps * 16);
  const uint64_t a0 = operand(queries, 8 * kRowBytes, 0);
  const uint64_t k0 = operand(ring, 8 * kRowBytes, 0);
  const uint64_t v0 = operand(ring, 8 * kRowBytes, kKeys * kRowBytes);
  constexpr uint32_t kTile = F::kTileBytes >> 4, kColumn = (kKeys * kRowBytes) >> 4;
  const uint32_t tmem = sh.tmem;
  Walk<kTileRows> walk(p, sh.share);
  Segment s;
  int taken = 0;                      // stages
  uint32_t query_parity = 0, weight_parity = 0, clear_parity = 0;   // (a bit per half)
  const auto full = [&](int i) {
    return wait_on<false>(p, sh, &sh.full[i % F::kStages], (i / F::kStages) & 1);
  };
  const auto multiply_scores = [&](int t, int stage, bool last) {
    const uint64_t a = a0 + t * kTile, b = k0 + stage * kTile;
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const uint32_t at = (i >> 2) * kColumn + (i & 3) * 2;
      if (i < steps) mma_shared(tmem + t * kHalf, a + at, b + at, scores, i > 0);
    }
    commit(&sh.scores[t]);
    if (last) commit(&sh.asked[t]);
  };
  while (walk.next(p, &s)) {
    const Halves h(p, s);
    if (h.most == 0) continue;
#pragma unroll
    for (int t = 0; t < 2; ++t)
      if (h.units[t] > 0) {
        if (!wait_on<false>(p, sh, &sh.queries[t], query_parity >> t & 1)) return;
        query_parity ^= 1u << t;
      }
    if (!full(taken)) return;
    // queries came by ordinary copies: order them before the tensor core's reads
    fence_proxy_async_smem();
    tc_fence_after();
#pragma unroll
    for (int t = 0; t < 2; ++t)
      if (h.units[t] > 0) multiply_scores(t, taken % F::kStages, h.units[t] == 1);
    commit(&sh.empty[taken % F::kStages]);
    ++taken;
    for (int u = 0; u < h.most; ++u) {
      const int value = taken % F::kStages;                  // this unit's values
      const int next = (taken + 1) % F::kStages;             // the next one's keys
      const bool goes_on = u + 1 < h.most;
      if (!kE4m3 && s.keys - (s.from + u) * p.unit_keys < p.unit_keys) {
        if (!wait_on<false>(p, sh, &sh.cleared, clear_parity)) return;
        clear_parity ^= 1;
      } else if (!full(taken)) {
        return;
      }
      if (goes_on && !full(taken + 1)) return;
      const uint64_t b = v0 + value * kTile;
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        if (u < h.units[t]) {
          const uint32_t from = tmem + t * kHalf, to = from + 2 * kHalf;
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            if (!wait_on<false>(p, sh, &sh.weights[t][half], weight_parity >> t & 1)) return;
            tc_fence_after();
#pragma unroll
            for (int i = half * kStep / 16; i < (half + 1) * kStep / 16; ++i)
              if (i < key_steps)
                mma_tmem(to, from + i * 8, b + i * ((16 * kRowBytes) >> 4), output, u > 0 || i > 0);
            commit(&sh.output[t][half]);
          }
          weight_parity ^= 1u << t;
        }
        if (u + 1 < h.units[t]) multiply_scores(t, next, u + 2 == h.units[t]);
      }
      commit(&sh.empty[value]);
      if (goes_on) commit(&sh.empty[next]);
      taken += goes_on ? 2 : 1;
    }
  }
}

// ------------------------------------------------------------------------
// One warp: queries, while the last tile's weights and output are still made.
// By TMA, a box of whole tokens, where a half is a number of them; else 16
// bytes a copy, written where the 128-byte swizzle has them (6 us a half).  And it
// clears what lies behind a tile's last key in its values.
template <int kDim>
__device__ __forceinline__ void copy_queries(const AttendParams& p, const Segment& s, Shared& sh,
                                             uint32_t queries, int t, int32_t rows) {
  using F = Form<kDim>;
  constexpr int kPieces = kDim / 8, kStride = 32 / kPieces;   // rows at once
  const int lane = threadIdx.x & 31, words = p.head_dim / 8, piece = lane % kPieces;
  const int32_t row0 = s.tile * kTileRows + t * kHalf;
  const uint32_t to = queries + t * F::kTileBytes + (piece / 8) * kKeys * kRowBytes;
  // token and head of a row are counted, not divided for
  int r = lane / kPieces;
  int32_t head = row0 + r - p.by_group(row0 + r) * p.group;
  const int32_t tokens = p.by_group(kStride), heads = kStride - tokens * p.group;
  const uint16_t* from = query_row(p, s.request.first, s.head, row0 + r) + piece * 8;
  const int64_t step = tokens * p.q_token + heads * p.q_head;
  const int64_t carry = p.q_token - p.group * p.q_head;
#pragma unroll 8
  for (int i = 0; i < kHalf / kStride; ++i) {
    const bool some = r < rows && piece < words;
    copy16(to + r * kRowBytes + (((piece & 7) ^ (r & 7)) << 4), some ? from : p.q, some ? 16 : 0);
    r += kStride;
    head += heads;
    from += step;
    if (head >= p.group) {
      head -= p.group;
      from += carry;
    }
  }
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(
                   smem_addr(&sh.queries[t]))
               : "memory");
}

template <int kDim, bool kE4m3>
__device__ void ask(const AttendParams& p, const Maps& maps, Shared& sh, uint32_t queries,
                    unsigned char* ring_ptr) {
  using F = Form<kDim, kE4m3>;
  const int lane = threadIdx.x & 31;
  const int columns = (p.head_dim + 63) / 64;
  Walk<kTileRows> walk(p, sh.share);
  Segment s;
  int tiles[2] = {0, 0}, loaded = 0;
  bool alive = true;
  while (alive && walk.next(p, &s)) {
    const Halves h(p, s);
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      if (h.units[t] == 0) continue;
      // (the last scores of the tile before are waited for below)
      if (!maps.query_box) {
        copy_queries<kDim>(p, s, sh, queries, t, h.rows[t]);
      } else if (lane == 0) {
        const int32_t token = s.request.first + p.by_group(s.tile * kTileRows + t * kHalf);
        mbar_arrive_expect_tx(&sh.queries[t], static_cast<uint32_t>(columns * kHalf * kRowBytes));
        for (int c = 0; c < columns; ++c)
          tma_4d(queries + t * F::kTileBytes + c * kKeys * kRowBytes, &maps.query, c * 64, 0, s.head,
                 token, &sh.queries[t]);
      }
    }
    loaded += 2 * h.most;
    // the tile's last scores: its queries have been read (a barrier is looked at
    // in each of its phases, lest one be taken for the next)
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      if (h.units[t] == 0) continue;
      alive = alive && wait<true>(p, sh, &sh.asked[t], tiles[t] & 1);
      ++tiles[t];
    }
    const int32_t left = s.keys - (s.from + h.most - 1) * p.unit_keys;
    if (!kE4m3 && alive && h.most > 0 && left < p.unit_keys) {
      // its last values' stage is in its last phase
      const int stage = (loaded - 1) % F::kStages;
      alive = wait(p, sh, &sh.full[stage], ((loaded - 1) / F::kStages) & 1);
      if (!alive) break;
      unsigned char* base = ring_ptr + stage * F::kTileBytes;
      const int n = (p.unit_keys - left) * (kRowBytes / 16);
      for (int c = 0; c < F::kHalves; ++c)
        for (int i = lane; i < n; i += 32)
          *reinterpret_cast<uint4*>(base + (c * kKeys + left) * kRowBytes + i * 16) =
              make_uint4(0, 0, 0, 0);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.cleared);
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  if (!alive && maps.query_box) {
    // queries asked for and never read are seen to land
#pragma unroll
    for (int t = 0; t < 2; ++t)
      if (tiles[t]) mbar_wait_bounded(&sh.queries[t], (tiles[t] - 1) & 1, kLandNs);
  }
}

// ------------------------------------------------------------------------
// Of a warp's rows from `row` on, of which those of `odd` came out infinite or NaN: those
// that something out of their sight has spoilt, over the keys [from, to), a warp a row.
// `part`: where the first one's part of the sums lies; null: whole rows.
template <int kDim, bool kE4m3>
__device__ __noinline__ void compute_again(const AttendParams& p, uint32_t* busy, int32_t request,
                                           int32_t head, int32_t first, int32_t row, uint32_t odd,
                                           int32_t seen, int32_t from, int32_t to, float* part) {
  const int lane = threadIdx.x & 31;
  if (lane == 0) atomicAdd(busy, 1u);
  __syncwarp();  // what each lane wrote of its own row is overwritten below
  for (uint32_t again = spoilt_rows(p, request, head, odd, seen, to); again; again &= again - 1) {
    const int who = __ffs(again) - 1;
    Slice own;
    warp_attend<kDim / 32, kE4m3>(p, query_row(p, first, head, row + who), request, head, from,
                                  min(__shfl_sync(0xffffffffu, seen, who), to), &own);
    uint16_t* out = output_row(p, first, head, row + who);
#pragma unroll
    for (int i = 0; i < kDim / 32; ++i) {
      const int d = lane + 32 * i;
      if (d >= p.head_dim) continue;
      if (part)
        part[who + (2 + d) * kTileRows] = own.o[i];
      else
        out[d] = f32_to_bf16(own.o[i] * inverse_sum(own.sum));
    }
    if (part && lane == 0) {
      part[who] = own.most;
      part[who + kTileRows] = own.sum;
    }
    __syncwarp();
  }
  if (lane == 0) atomicSub(busy, 1u);
}

// ------------------------------------------------------------------------
// Four warps, a thread a row.  A unit's weights go in two steps of 64 keys, each
// with its own look at the maximum, so that the first step's products run while
// the second's weights are made: the chain from scores to weights and back is what
// bounds a unit (scores 130 cycles out of TMEM, 64 weights some 330, 130 to
// TMEM and the products' start; products of a half 1024).
template <int kDim, bool kE4m3>
__device__ void soften(const AttendParams& p, Shared& sh, int t) {
  using F = Form<kDim>;
  const int lane = threadIdx.x & 31, tid = threadIdx.x & (kHalf - 1), warp = tid >> 5;
  const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;
  const uint32_t score_at = sh.tmem + lanes + t * kHalf, out_at = score_at + 2 * kHalf;
  const int block = range_of(blockIdx.x, gridDim.x);
  float* parts = reinterpret_cast<float*>(reinterpret_cast<Joint*>(p.workspace) + gridDim.x);
  const float scale = p.scale * kLog2e;
  const bool at_once =
      (reinterpret_cast<uintptr_t>(p.o) & 31) == 0 && p.head_dim % 16 == 0;
  Walk<kTileRows> walk(p, sh.share);
  Segment s;
  uint32_t done = 0;        // units of this half so far
  while (walk.next(p, &s)) {
    const Halves h(p, s);
    const int32_t row0 = s.tile * kTileRows + t * kHalf, rows = t ? h.rows[1] : h.rows[0];
    const int32_t units = t ? h.units[1] : h.units[0];
    float top = minus_infinity(), sum = 0.0f;
    int32_t seen = 0;
    if (tid < rows) seen = seen_keys(s.request, p.by_group(row0 + tid));
    for (int u = 0; u < units; ++u) {
      if (!wait<true>(p, sh, &sh.scores[t], done & 1)) return;
      tc_fence_after();
      float v[kKeys];
      tmem_load32(score_at, v);
      tmem_load32(score_at + 32, v + 32);
      tmem_arrived<kStep>(v);
      tmem_load32(score_at + 64, v + 64);
      tmem_load32(score_at + 96, v + 96);
      const int32_t key0 = (s.from + u) * p.unit_keys;
      int32_t valid = seen - key0;
      valid = valid < p.unit_keys ? valid : p.unit_keys;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        float* x = v + half * kStep;
        if (half == 1) tmem_arrived<kStep>(x);
        if (valid < (half + 1) * kStep) {
#pragma unroll
          for (int c = 0; c < kStep; ++c)
            if (half * kStep + c >= valid) x[c] = minus_infinity();
        }
        float m[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
        for (int c = 4; c < kStep; c += 8)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            m[i] = c + 4 + i < kStep ? max3(m[i], x[c + i], x[c + 4 + i]) : fmaxf(m[i], x[c + i]);
        const float most = fmaxf(max3(m[0], m[1], m[2]), m[3]) * scale;
        if (__any_sync(0xffffffffu, most > top + kSlack)) {
          const float now = fmaxf(top, most);
          const float by = now == minus_infinity() ? 1.0f : exp2_fast(top - now);
          top = now;
          sum *= by;
          if (u > 0 || half == 1) {
            // the step before has gone into the output
            if (!wait(p, sh, &sh.output[t][half ^ 1], half == 1 ? done & 1 : (done - 1) & 1)) return;
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < p.head_dim; c += 32) {
              float o[32];
              tmem_load32(out_at + c, o);
              tmem_arrived<32>(o);
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] *= by;
              tmem_store32(out_at + c, o);
            }
          }
        }
        const float base = top == minus_infinity() ? 0.0f : -top;
        const float2 scale2 = make_float2(scale, scale), base2 = make_float2(base, base);
        float2 sums[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
        uint32_t w[kStep / 2];
#pragma unroll
        for (int i = 0; i < kStep / 2; ++i) {
          float2 y = fma2(make_float2(x[2 * i], x[2 * i + 1]), scale2, base2);
          y.x = exp2_fast(y.x);
          y.y = exp2_fast(y.y);
          sums[i & 1] = add2(sums[i & 1], y);
          w[i] = pack_bf16(y.x, y.y);
        }
        sum += (sums[0].x + sums[0].y) + (sums[1].x + sums[1].y);
        tmem_store32(score_at + half * (kStep / 2), reinterpret_cast<const float*>(w));
        tmem_store_wait();
        tc_fence_before();
        mbar_arrive(&sh.weights[t][half]);
      }
      ++done;
    }
    // ---- output, or this block's part of it
    const bool whole = s.from == 0 && s.to == s.all;
    float* part = parts + (2 * block + (s.from == 0)) * kPartValues<kDim> +
                  t * kHalf + tid;
    const bool live = tid < rows;
    uint16_t* out = live ? output_row(p, s.request.first, s.head, row0 + tid) : nullptr;
    if (units > 0) {
      float o[kDim];
      if (!wait(p, sh, &sh.output[t][1], (done - 1) & 1)) return;
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < kDim; c += 32) tmem_load32(out_at + c, o + c);
      tmem_arrived<kDim>(o);
      float size = fabsf(sum);
#pragma unroll
      for (int c = 0; c < kDim; ++c)
        if (c < p.head_dim) size += fabsf(o[c]);
      if (live && whole) {
        const float by = inverse_sum(sum);
#pragma unroll
        for (int c = 0; c < kDim; c += 16)
          if (c + 16 <= p.head_dim) {
            store16(out + c, o + c, by, at_once);
          } else if (c < p.head_dim) {  // eight
            const float f[8] = {o[c] * by,     o[c + 1] * by, o[c + 2] * by, o[c + 3] * by,
                                o[c + 4] * by, o[c + 5] * by, o[c + 6] * by, o[c + 7] * by};
            *reinterpret_cast<uint4*>(out + c) = pack8(f);
          }
      } else if (live) {
        part[0] = sum == sum ? top : sum;   // (of NaN alone no maximum has come up)
        part[kTileRows] = sum;
#pragma unroll
        for (int c = 0; c < kDim; ++c)
          if (c < p.head_dim) part[(2 + c) * kTileRows] = o[c];
      }
      tc_fence_before();
      const uint32_t odd = __ballot_sync(
          0xffffffffu, live && sum == sum && !(size < __uint_as_float(0x7F800000u)));
      if (odd)
        compute_again<kDim, kE4m3>(p, &sh.busy, s.index, s.head, s.request.first, row0 + warp * 32,
                                   odd, seen, s.from * p.unit_keys,
                                   min((s.from + units) * p.unit_keys, s.keys),
                                   whole ? nullptr : part - lane);
    } else if (live && whole) {
      for (int c = 0; c < p.head_dim; c += 8)
        *reinterpret_cast<uint4*>(out + c) = make_uint4(0, 0, 0, 0);
    } else if (live) {
      part[0] = minus_infinity();   // the join looks no further
    }
  }
  // (the second step's is waited for above; the first step's has come too)
  if (done > 0) mbar_wait_bounded(&sh.output[t][0], (done - 1) & 1, p.timeout_ns);
}

// One lane: what the launch that joins has to know of the block's last tile.
__device__ void announce(const AttendParams& p, const Shared& sh) {
  Walk<kTileRows> walk(p, sh.share);
  Segment s{};
  bool goes_on = false;
  while (walk.next(p, &s)) goes_on = s.from == 0 && s.to < s.all;
  const int block = range_of(blockIdx.x, gridDim.x);
  leave_joint(reinterpret_cast<Joint*>(p.workspace) + block, goes_on ? &s : nullptr, sh.share,
              s.tile * kTileRows, block);
}

template <int kDim, bool kE4m3>
__global__ void __launch_bounds__(Form<kDim, kE4m3>::kThreads, 1)
    k_attend_wide(const AttendParams p, const __grid_constant__ Maps maps) {
  using F = Form<kDim, kE4m3>;
  constexpr int kThreads = F::kThreads;
  extern __shared__ unsigned char raw[];
  __shared__ Shared sh;
  const uint32_t base = smem_addr(raw);
  const uint32_t queries = (base + 1023) & ~1023u, ring = queries + 2 * F::kTileBytes;
  unsigned char* ring_ptr = raw + (ring - base);
  const int warp = threadIdx.x >> 5, blocks = gridDim.x;
  if (threadIdx.x == 0) {
    for (int i = 0; i < F::kStages; ++i) {
      mbar_init(&sh.full[i], kE4m3 ? 4 : 1);
      mbar_init(&sh.empty[i], 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&sh.raw_full[t], 1);
      mbar_init(&sh.raw_empty[t], 4);
      mbar_init(&sh.queries[t], maps.query_box ? 1 : 32);
      mbar_init(&sh.asked[t], 1);
      mbar_init(&sh.scores[t], 1);
      for (int i = 0; i < 2; ++i) {
        mbar_init(&sh.weights[t][i], kHalf);
        mbar_init(&sh.output[t][i], 1);
      }
    }
    mbar_init(&sh.cleared, 1);
    mbar_init(&sh.drain, 1);
    sh.stop = sh.busy = 0;
    sh.issued = 0;
    sh.moved[0] = sh.moved[1] = 0;
    fence_barrier_init();
  }
  if (warp == kMultiplyWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr(&sh.tmem)),
                 "r"(kTmemColumns)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    tc_fence_before();
  }
  // rows of a stage that no load fills
  for (int i = threadIdx.x; i < F::kStages * F::kTileBytes / 16; i += kThreads)
    reinterpret_cast<uint4*>(ring_ptr)[i] = make_uint4(0, 0, 0, 0);
  fence_proxy_async_smem();
  find_share<kTileRows, kThreads>(p, range_of(blockIdx.x, blocks), blocks, sh.part, &sh.share);
  __syncthreads();
  tc_fence_after();
  const uint32_t raw_at = ring + F::kStages * F::kTileBytes;
  if (warp < kSoftmaxWarps) {
    if (kE4m3)
      asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
    else
      asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
    soften<kDim, kE4m3>(p, sh, warp / 4);
  } else {
    if (kE4m3)
      asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    else
      asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
    if (warp == kMultiplyWarp)
      multiply<kDim, kE4m3>(p, sh, queries, ring);
    else if (warp < kQueryWarp)
      load<kDim, kE4m3>(p, maps, sh, kE4m3 ? raw_at : ring, warp - kLoadWarp);
    else if (warp == kQueryWarp)
      ask<kDim, kE4m3>(p, maps, sh, queries, ring_ptr);
    else if constexpr (kE4m3)
      widen<kDim>(p, sh, ring_ptr, ring_ptr + F::kStages * F::kTileBytes, warp - kWidenWarp);
    if (warp == kQueryWarp && one_lane()) announce(p, sh);
  }
  tc_fence_before();
  __syncthreads();
  if (sh.stop) {
    // a wait ran out: the products issued are seen to end, the loads to land
    if (warp == kMultiplyWarp && one_lane()) {
      commit(&sh.drain);
      mbar_wait_bounded(&sh.drain, 0, kLandNs);
    } else if (warp == kLoadWarp) {
      uint64_t* const full = kE4m3 ? sh.raw_full : sh.full;
      for (int i = sh.issued > F::kSlots ? sh.issued - F::kSlots : 0; i < sh.issued; ++i)
        if (!mbar_wait_bounded(&full[i % F::kSlots], (i / F::kSlots) & 1, kLandNs)) break;
    }
    __syncthreads();
  }
  tc_fence_after();
  if (warp == kMultiplyWarp)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(sh.tmem),
                 "r"(kTmemColumns)
                 : "memory");
}

// Joins a tile's parts, kJoinGroups threads a row, kJoinColumns of its values; rows
// behind the last request become zeros.  A thread looks at its parts' maxima first, so
// that what they weigh is read without waiting (one part after the other: 21 us for 152
// parted tiles, 60 for one of 71 parts).
template <int kDim>
__global__ void __launch_bounds__(kJoinGroups* kTileRows) k_attend_wide_join(const AttendParams p) {
  __shared__ float sums[kJoinGroups - 1][kJoinColumns + 2][kTileRows];
  const int blocks = gridDim.x, block = blockIdx.x;
  const int row = threadIdx.x % kTileRows, group = threadIdx.x / kTileRows;
  const int c0 = blockIdx.y * kJoinColumns;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Joint j = reinterpret_cast<const Joint*>(p.workspace)[block];
  const float* own =
      reinterpret_cast<const float*>(reinterpret_cast<const Joint*>(p.workspace) + blocks) +
      (2 * block + 1) * kPartValues<kDim> + row;
  const auto part = [&](int i) {  // the block's own slot 1, then the others' slots 0
    return own + (2 * i - (i > 0)) * kPartValues<kDim>;
  };
  if (j.parts > 0) {
    const bool live = row < j.rows;
    float m = minus_infinity(), l = 0.0f, v[kJoinColumns] = {};
    if (live) {
#pragma unroll 8
      for (int i = group; i < j.parts; i += kJoinGroups) m = fmaxf(m, part(i)[0]);
      const float base = m == minus_infinity() ? 0.0f : m;
#pragma unroll 2
      for (int i = group; i < j.parts; i += kJoinGroups) {
        const float* at = part(i);
        const float top = at[0];
        // of none of its keys seen: no sums were left
        if (top == minus_infinity()) continue;
        const float by = exp2_fast(top - base);
        l += at[kTileRows] * by;
#pragma unroll
        for (int c = 0; c < kJoinColumns; ++c)
          if (c0 + c < p.head_dim) v[c] += at[(2 + c0 + c) * kTileRows] * by;
      }
    }
    if (group > 0) {
      sums[group - 1][0][row] = m;
      sums[group - 1][1][row] = l;
#pragma unroll
      for (int c = 0; c < kJoinColumns; ++c) sums[group - 1][2 + c][row] = v[c];
    }
    __syncthreads();
    if (live && group == 0) {
      float most = m;
#pragma unroll
      for (int g = 1; g < kJoinGroups; ++g) most = fmaxf(most, sums[g - 1][0][row]);
      const float base = most == minus_infinity() ? 0.0f : most;
      const float old = exp2_fast(m - base);
      l *= old;
#pragma unroll
      for (int c = 0; c < kJoinColumns; ++c) v[c] *= old;
#pragma unroll
      for (int g = 1; g < kJoinGroups; ++g) {
        const float by = exp2_fast(sums[g - 1][0][row] - base);
        l += sums[g - 1][1][row] * by;
#pragma unroll
        for (int c = 0; c < kJoinColumns; ++c) v[c] += sums[g - 1][2 + c][row] * by;
      }
      const float by = inverse_sum(l);
      uint16_t* out = output_row(p, j.first, j.head, j.row + row) + c0;
#pragma unroll
      for (int c = 0; c < kJoinColumns; c += 8)
        if (c0 + c < p.head_dim) {
          const float f[8] = {v[c] * by,     v[c + 1] * by, v[c + 2] * by, v[c + 3] * by,
                              v[c + 4] * by, v[c + 5] * by, v[c + 6] * by, v[c + 7] * by};
          *reinterpret_cast<uint4*>(out + c) = pack8(f);
        }
    }
  }
  if (blockIdx.y) return;
  const int64_t width = static_cast<int64_t>(p.heads) * p.group * p.head_dim;
  const int64_t behind = p.requests ? clamp_to(p.offsets[p.requests], p.tokens) : 0;
  for (int64_t at = behind * width + static_cast<int64_t>(block) * blockDim.x + threadIdx.x;
       at < p.tokens * width; at += static_cast<int64_t>(blocks) * blockDim.x)
    p.o[at] = 0;
}

// ------------------------------------------------------------------------
// Host

// Of rows of head_dim values, n[i] of them at[i] elements apart; boxes of `wide`
// values (bf16: 64, swizzled).
bool make_map(CUtensorMap* map, const void* data, const AttendParams& p, bool e4m3, int wide,
              const int64_t (&n)[3], const int64_t (&at)[3], const int (&box)[3]) {
  const int size = e4m3 ? 1 : 2;
  cuuint64_t dims[4] = {static_cast<cuuint64_t>(p.head_dim)}, strides[3];
  for (int i = 0; i < 3; ++i) {
    dims[i + 1] = static_cast<cuuint64_t>(n[i]);
    // (of one: any)
    strides[i] = static_cast<cuuint64_t>(n[i] > 1 ? size * at[i] : 16);
    if (n[i] > 1 && at[i] <= 0) return false;
  }
  const cuuint32_t boxes[4] = {static_cast<cuuint32_t>(wide), static_cast<cuuint32_t>(box[0]),
                               static_cast<cuuint32_t>(box[1]), static_cast<cuuint32_t>(box[2])};
  const cuuint32_t ones[4] = {1, 1, 1, 1};
  return encode()(map, e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
                  const_cast<void*>(data), dims, strides, boxes, ones,
                  CU_TENSOR_MAP_INTERLEAVE_NONE,
                  e4m3 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool make_side_map(CUtensorMap* map, const Side& s, const AttendParams& p, int wide, int box) {
  return make_map(map, s.data, p, p.e4m3, wide, {p.page_size, p.heads, p.pages},
                  {s.stride[1], s.stride[2], s.stride[0]}, {box, 1, 1});
}

bool on_words(const Side& s, int values) {
  return (reinterpret_cast<uintptr_t>(s.data) & 15) == 0 && s.stride[0] % values == 0 &&
         s.stride[1] % values == 0 && s.stride[2] % values == 0;
}

template <int kDim, bool kE4m3>
int launch_at(const AttendParams& p, const Maps& maps, cudaStream_t s) {
  using F = Form<kDim, kE4m3>;
  const cudaError_t err = allow_shared<k_attend_wide<kDim, kE4m3>>(F::kSmem);
  if (err != cudaSuccess) return err;
  k_attend_wide<kDim, kE4m3><<<p.blocks, F::kThreads, F::kSmem, s>>>(p, maps);
  const dim3 grid(static_cast<unsigned>(p.blocks),
                  static_cast<unsigned>((p.head_dim + kJoinColumns - 1) / kJoinColumns));
  return launch_after(k_attend_wide_join<kDim>, grid, kJoinGroups * kTileRows, s, p);
}

// Rows a head (most of any request, as far as the caller knows) up to which a call
// is left to the form for few rows.  64 requests of 5000 keys on average, 4 heads, rows,
// form for few and for many, in us: bf16 8 117, 137; 16 118, 137; 24 159, 137; 32 167,
// 137; 64 235, 138.  e4m3 8 90, 241; 16 110, 241; 32 184, 241; 64 258, 240.
constexpr int kFewRows = 16, kFewRowsE4m3 = 32;
// Of boxes of fewer than eight keys, whose loads take longer, by rows times keys of a box:
// bf16 pages of two and 40 rows 136, 230, 70 rows 199, 231, 100 rows (12 heads) 164, 166;
// of three 44 rows 141, 163; of four 40 rows 133, 135, 70 rows 195, 132; of five 28 rows
// 115, 115, 56 rows 154, 117.  e4m3 of two 100 rows 178, 179; of four 70 rows 211, 139; of
// five 56 rows 168, 135.
constexpr int kSmallBox = 8;
constexpr int kFewSmall = 192, kFewSmallE4m3 = 256;

// Rows of 16-byte words, as queries and outputs are.
bool wide_takes(const AttendParams& p) {
  const int values = p.e4m3 ? 16 : 8;
  return p.head_dim <= 128 && p.head_dim % values == 0 && p.pages > 0 &&
         p.scale > 0.0f && on_words(p.key, values) && on_words(p.value, values) &&
         (reinterpret_cast<uintptr_t>(p.q) & 15) == 0 && p.q_token % 8 == 0 && p.q_head % 8 == 0 &&
         (reinterpret_cast<uintptr_t>(p.o) & 15) == 0 && encode();
}

}  // namespace

int64_t wide_workspace_bytes(int sms) {
  return static_cast<int64_t>(sms) * (sizeof(Joint) + 2 * 4 * kPartValues<128>);
}

bool launch_attend_wide(const AttendParams& given, void* stream, int* status) {
  if (!wide_takes(given)) return false;
  AttendParams p = given;
  Maps maps;
  // Keys of a box: the most that divide a page and fit a unit, by eights of pages of
  // eights.  It may begin at any row of a stage: the swizzle goes by the address in
  // shared memory.  Where a row as loaded has 64 bytes, by twos, as boxes begin on 128
  // bytes.  A unit has 32 boxes at most, a lane each.
  const int by = p.page_size % 8 == 0 ? 8 : p.e4m3 && p.head_dim <= 64 ? 2 : 1;
  maps.box = kKeys;
  while (maps.box > by && p.page_size % maps.box) maps.box -= by;
  if (maps.box < 2 || p.page_size % maps.box) return false;
  const int64_t rows = p.longest * p.group;
  if (rows <= (p.e4m3 ? kFewRowsE4m3 : kFewRows)) return false;
  if (maps.box < kSmallBox && rows * maps.box <= (p.e4m3 ? kFewSmallE4m3 : kFewSmall)) return false;
  p.unit_keys = (kKeys / maps.box < 32 ? kKeys / maps.box : 32) * maps.box;
  maps.by_box = Divide(maps.box);
  p.by_unit = Divide(p.unit_keys);
  const int wide = !p.e4m3 ? 64 : p.head_dim <= 64 ? 64 : 128;
  if (!make_side_map(&maps.key, p.key, p, wide, maps.box) ||
      !make_side_map(&maps.value, p.value, p, wide, maps.box))
    return false;
  maps.query_box = kHalf % p.group ? 0 : kHalf / p.group;
  if (!maps.query_box ||
      !make_map(&maps.query, p.q, p, false, 64, {p.group, p.heads, p.tokens},
                {p.q_head, p.q_head * p.group, p.q_token}, {p.group, 1, maps.query_box})) {
    maps.query_box = 0;
    maps.query = maps.key;  // not used
  }
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (p.e4m3)
    *status = p.head_dim <= 64 ? launch_at<64, true>(p, maps, s) : launch_at<128, true>(p, maps, s);
  else
    *status = p.head_dim <= 64 ? launch_at<64, false>(p, maps, s) : launch_at<128, false>(p, maps, s);
  return true;
}

}  // namespace ciera
