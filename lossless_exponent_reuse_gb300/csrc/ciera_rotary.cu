// ciera_rotary.cu -- rotary positions, keys and values into their pages, and
// the pages of a serving step.
#include <cooperative_groups.h>

#include "ciera_attention.h"
#include "ciera_moe_device.cuh"

namespace ciera {
namespace {

// ------------------------------------------------------------------------
// Rotary positions.  Bound by memory: 4 bytes a value (16384 tokens of 32 heads of 128
// 42.5 us, 6.3 TB/s; 8192 tokens of 32, 8 and 8 heads into 8-bit pages 41.1, 4.5 TB/s: a
// row's exponent has to wait for all of it).  A turn is a whole number
// of 2^-64 turns per position, so that position * turns wraps as the angle does
// and the angle's 24 bits for sin and cos are exact for every position.
//
// A warp takes some rows (a token's heads) of one token: it computes the token's
// sines and cosines once, two a lane for 64 pairs, keeps each lane's in registers
// and goes through the rows, some lanes a row.  A lane holds two words of a row:
// the two halves of its pairs, or two neighbouring words of whole pairs.

constexpr int kRotaryWarps = 4;
constexpr int kMostPairs = 512;

__device__ __forceinline__ float2 turn(const RotaryParams& p, int32_t position, int i) {
  const uint64_t t = static_cast<uint64_t>(static_cast<int64_t>(position)) *
                     static_cast<uint64_t>(p.turns[i]);
  // half turns, from -1 to 1
  float s, c;
  sincospif(static_cast<float>(static_cast<int64_t>(t)) * 0x1p-63f, &s, &c);
  return make_float2(c * p.amplitude, (p.inverse ? -s : s) * p.amplitude);
}

// Biased exponent of an e4m3 row whose values are at most the float of these
// bits: the least e with it <= 448 * 2^e, 448 = 1.75 * 2^8.
__device__ __forceinline__ uint32_t row_exponent(uint32_t most) {
  if (most >= 0x7F800000u) return 255;
  int e = static_cast<int>(most >> 23) - 127 - 8 + ((most & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  e = e < kLowestExponent ? kLowestExponent : e > kHighestExponent ? kHighestExponent : e;
  return static_cast<uint32_t>(e + kExponentBias);
}
// 2^-e of a biased exponent (e in range; of a row of NaN anything).
__device__ __forceinline__ float inverse_scale(uint32_t biased) {
  return __uint_as_float((254 - (biased == 255 ? 127 : biased)) << 23);
}

// Where row j of token t comes from and goes to.  kind 0: a query, 1: a key, 2: a value.
struct RotaryRow {
  int kind;
  const uint16_t* from;
  void* to;              // null: nowhere
  uint8_t* exponent;
};

__device__ __forceinline__ RotaryRow rotary_row(const RotaryParams& p, int64_t t, int64_t j,
                                                int32_t page, int32_t place) {
  RotaryRow r;
  r.exponent = nullptr;
  if (j < p.q.heads) {
    r.kind = 0;
    r.from = p.q.data + t * p.q.token + j * p.q.head;
    r.to = p.out + t * p.out_token + j * p.out_head;
    return r;
  }
  j -= p.q.heads;
  r.kind = j < p.k.heads ? 1 : 2;
  if (r.kind == 2) j -= p.k.heads;
  const Heads& in = r.kind == 1 ? p.k : p.v;
  const Side& side = r.kind == 1 ? p.key : p.value;
  r.from = in.data + t * in.token + j * in.head;
  r.to = nullptr;
  if (page >= 0) {
    const int64_t at = page * side.stride[0] + place * side.stride[1] + j * side.stride[2];
    r.to = p.e4m3 ? static_cast<void*>(static_cast<uint8_t*>(side.data) + at)
                  : static_cast<void*>(static_cast<uint16_t*>(side.data) + at);
    if (p.e4m3)
      r.exponent = side.exponent + page * side.exponent_stride[0] +
                   place * side.exponent_stride[1] + j * side.exponent_stride[2];
  }
  return r;
}

// Page and place of token t's slot; page -1: none.
__device__ __forceinline__ void find_slot(const RotaryParams& p, int64_t t, int32_t* page,
                                          int32_t* place) {
  *page = -1;
  *place = 0;
  if (!p.slots) return;
  const int32_t slot = p.slots[t];
  const int32_t at = slot < 0 ? -1 : slot / p.page_size;
  if (at < 0 || at >= p.pages) return;
  *page = at;
  *place = slot - at * p.page_size;
}

template <int kVec>
struct RotaryWord;
template <>
struct RotaryWord<8> {
  using Word = uint4;
  using Half = uint2;
};
template <>
struct RotaryWord<4> {
  using Word = uint2;
  using Half = uint32_t;
};

template <int kVec>
__device__ __forceinline__ void widen(const typename RotaryWord<kVec>::Word& w, float* f) {
  const uint32_t* v = reinterpret_cast<const uint32_t*>(&w);
#pragma unroll
  for (int i = 0; i < kVec / 2; ++i) {
    f[2 * i] = bf16_lo(v[i]);
    f[2 * i + 1] = bf16_hi(v[i]);
  }
}

template <int kVec>
__device__ __forceinline__ void put_bf16(void* to, const float* f) {
  typename RotaryWord<kVec>::Word w;
  uint32_t* v = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
  for (int i = 0; i < kVec / 2; ++i) v[i] = pack_bf16(f[2 * i], f[2 * i + 1]);
  *static_cast<typename RotaryWord<kVec>::Word*>(to) = w;
}

template <int kVec>
__device__ __forceinline__ void put_e4m3(void* to, const float* f, float by) {
  typename RotaryWord<kVec>::Half w;
  uint32_t* v = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
  for (int i = 0; i < kVec / 4; ++i)
    v[i] = pack_e4m3(f[4 * i] * by, f[4 * i + 1] * by, f[4 * i + 2] * by, f[4 * i + 3] * by);
  *static_cast<typename RotaryWord<kVec>::Half*>(to) = w;
}

// kVec pairs a lane.  lanes: of a row (a power of two); span: rows of a warp,
// spans: warps of a token.
template <int kVec, bool kAppend, bool kInterleaved>
__global__ void __launch_bounds__(32 * kRotaryWarps, kAppend ? 5 : 7)
    k_rotary(const RotaryParams p, int lanes, int span, int spans) {
  using Word = typename RotaryWord<kVec>::Word;
  // Rows that a lane loads before it uses the first, the first ones before it works out
  // the token's turns; into pages, whose rows take longer, the next ones before it
  // stores these.  In us, blocks an SM in brackets: 16384 tokens of 32 heads, two behind
  // the turns 45.8 (6), before them 43.9 (6), 42.5 (7), 43.2 (8), three 45 (5), two and
  // the next 44.4 (5); 8192 tokens into 8-bit pages, three behind the turns 44.5 (5), before
  // them 44.2 (5), two and the next 41.1 (5), 45.5 (4), one and the next 42.8 (6).
  constexpr int kBatch = 2;
  constexpr bool kAhead = kAppend;
  __shared__ float2 turns[kRotaryWarps][kMostPairs];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * kRotaryWarps + warp;
  const int64_t t = item / spans;
  if (t >= p.tokens) return;
  const int64_t rows = p.q.heads + (kAppend ? 2 * p.k.heads : 0);
  const int64_t first = (item - t * spans) * span;
  const int64_t end = first + span < rows ? first + span : rows;

  const int unit = lane & (lanes - 1), turned = p.pairs / kVec, step = 32 / lanes;
  const bool rotates = unit < turned;
  // the lane's two words of a row
  int a = 2 * p.pairs + 2 * (unit - turned) * kVec, b = a + kVec;
  if (rotates) {
    a = kInterleaved ? 2 * unit * kVec : unit * kVec;
    b = kInterleaved ? a + kVec : a + p.pairs;
  }
  const bool has_a = a < p.head_dim, has_b = b < p.head_dim;
  const auto fetch = [&](int64_t j0, Word (&w)[kBatch][2]) {
#pragma unroll
    for (int q = 0; q < kBatch; ++q) {
      const int64_t j = j0 + q * step + lane / lanes;
      w[q][0] = w[q][1] = Word{};
      if (j >= end) continue;
      const uint16_t* from = rotary_row(p, t, j, -1, 0).from;
      if (has_a) w[q][0] = *reinterpret_cast<const Word*>(from + a);
      if (has_b) w[q][1] = *reinterpret_cast<const Word*>(from + b);
    }
  };
  Word w[kBatch][2];
  fetch(first, w);
  const int32_t position = p.positions[t];
  for (int i = lane; i < p.pairs; i += 32) turns[warp][i] = turn(p, position, i);
  int32_t page = -1, place = 0;
  if (kAppend) find_slot(p, t, &page, &place);
  __syncwarp();
  float c[kVec], s[kVec];
  if (rotates) {
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const float2 v = turns[warp][unit * kVec + i];
      c[i] = v.x;
      s[i] = v.y;
    }
  }
  for (int64_t j0 = first; j0 < end; j0 += kBatch * step) {
    // (rows of their own: also where the output is x itself)
    Word next[kBatch][2];
    if (kAhead) fetch(j0 + kBatch * step, next);
#pragma unroll
    for (int q = 0; q < kBatch; ++q) {
      if (j0 + q * step >= end) break;
      const int64_t j = j0 + q * step + lane / lanes;
      RotaryRow row;
      row.to = nullptr;
      row.kind = 2;
      if (j < end) row = rotary_row(p, t, j, page, place);
      float x[2 * kVec];
      widen<kVec>(w[q][0], x);
      widen<kVec>(w[q][1], x + kVec);
      const bool rotate = rotates && row.kind < 2;
      uint32_t most = 0;
      if (kAppend && p.e4m3) {
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
          // the pair's two values: in both words, or side by side
          const float u = fabsf(kInterleaved ? x[2 * i] : x[i]);
          const float v = fabsf(kInterleaved ? x[2 * i + 1] : x[i + kVec]);
          const uint32_t bits = rotate ? __float_as_uint((u + v) * fabsf(p.amplitude))
                                       : max(__float_as_uint(u), __float_as_uint(v));
          most = max(most, bits & 0x7FFFFFFFu);
        }
        for (int o = 1; o < lanes; o <<= 1)
          most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
      }
      if (rotate) {
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
          float& u = kInterleaved ? x[2 * i] : x[i];
          float& v = kInterleaved ? x[2 * i + 1] : x[i + kVec];
          const float y = u * c[i] - v * s[i];
          v = u * s[i] + v * c[i];
          u = y;
        }
      }
      if (!row.to) continue;
      if (kAppend && p.e4m3 && row.kind) {
        const uint32_t e = row_exponent(most);
        const float by = inverse_scale(e);
        uint8_t* to = static_cast<uint8_t*>(row.to);
        if (has_a) put_e4m3<kVec>(to + a, x, by);
        if (has_b) put_e4m3<kVec>(to + b, x + kVec, by);
        if (unit == 0) *row.exponent = static_cast<uint8_t>(e);
      } else {
        uint16_t* to = static_cast<uint16_t*>(row.to);
        if (has_a) put_bf16<kVec>(to + a, x);
        if (has_b) put_bf16<kVec>(to + b, x + kVec);
      }
    }
    if (kAhead) {
#pragma unroll
      for (int q = 0; q < kBatch; ++q) {
        w[q][0] = next[q][0];
        w[q][1] = next[q][1];
      }
    } else {
      fetch(j0 + kBatch * step, w);
    }
  }
}

// Any size and alignment: a warp a row, a pair (or a value behind the pairs) a
// lane at a time; e4m3 rows are read twice.
__global__ void __launch_bounds__(32 * kRotaryWarps) k_rotary_any(const RotaryParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t rows = p.q.heads + (p.slots ? 2 * p.k.heads : 0);
  const int64_t item = static_cast<int64_t>(blockIdx.x) * kRotaryWarps + (threadIdx.x >> 5);
  const int64_t t = item / rows;
  if (t >= p.tokens) return;
  int32_t page, place;
  find_slot(p, t, &page, &place);
  const RotaryRow row = rotary_row(p, t, item - t * rows, page, place);
  if (!row.to) return;
  const int pairs = row.kind < 2 ? p.pairs : 0, units = p.head_dim - pairs;
  const bool narrow = p.e4m3 && row.kind;
  uint32_t exponent = 0;
  if (narrow) {
    uint32_t most = 0;
    for (int i = lane; i < units; i += 32) {
      float m;
      if (i < pairs) {
        const int a = p.interleaved ? 2 * i : i, b = p.interleaved ? a + 1 : a + p.pairs;
        m = (fabsf(bf16_to_f32(row.from[a])) + fabsf(bf16_to_f32(row.from[b]))) *
            fabsf(p.amplitude);
      } else {
        m = fabsf(bf16_to_f32(row.from[i + pairs]));
      }
      most = max(most, __float_as_uint(m) & 0x7FFFFFFFu);
    }
    exponent = row_exponent(__reduce_max_sync(0xffffffffu, most));
    if (lane == 0) *row.exponent = static_cast<uint8_t>(exponent);
  }
  const float by = inverse_scale(exponent);
  const auto put = [&](int at, float v) {
    if (narrow)
      static_cast<uint8_t*>(row.to)[at] = f32_to_e4m3(v * by);
    else
      static_cast<uint16_t*>(row.to)[at] = f32_to_bf16(v);
  };
  const int32_t position = p.positions[t];
  for (int i = lane; i < units; i += 32) {
    if (i >= pairs) {
      put(i + pairs, bf16_to_f32(row.from[i + pairs]));
      continue;
    }
    const int a = p.interleaved ? 2 * i : i, b = p.interleaved ? a + 1 : a + p.pairs;
    const float2 cs = turn(p, position, i);
    const float u = bf16_to_f32(row.from[a]), v = bf16_to_f32(row.from[b]);
    put(a, u * cs.x - v * cs.y);
    put(b, u * cs.y + v * cs.x);
  }
}

// ------------------------------------------------------------------------
// Pages of a step.  A few KB in and out: bound by its launch and the chain of
// loads (8 requests 6.1 us, 200 of up to 80 new tokens 11.7).  The first block of a
// cluster scans the requests and gives out the free pages; then every token of the
// cluster finds its request by bisection.

constexpr int kPagesThreads = 1024;
constexpr int kPagesCluster = 8;
constexpr int64_t kNoPages = int64_t(1) << 40;   // more than any stack holds

__device__ __forceinline__ int64_t warp_scan(int64_t v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t left = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += left;
  }
  return v;
}

// Inclusive sums over the block's threads; `total` gets the last.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* part, int64_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  v = warp_scan(v);
  if (lane == 31) part[warp] = v;
  __syncthreads();
  if (warp == 0) {
    const int64_t w = warp_scan(part[lane]);
    part[lane] = w;
  }
  __syncthreads();
  if (warp > 0) v += part[warp - 1];
  *total = part[31];
  __syncthreads();
  return v;
}

__device__ void assign(const PagesParams& p) {
  __shared__ int64_t part[32];
  const int tid = threadIdx.x, lane = tid & 31;
  const int64_t S = p.page_size;
  const int32_t given = p.count[0];
  const int64_t count = given < 0 ? 0 : given > p.capacity ? p.capacity : given;
  int64_t rows = 0, pages = 0, taken = 0;   // so far; taken: of this thread's requests
  for (int base = 0; base < p.requests; base += kPagesThreads) {
    const int r = base + tid;
    const bool have_r = r < p.requests;
    const int64_t c = have_r ? max(p.cached[r], 0) : 0, n = have_r ? max(p.fresh[r], 0) : 0;
    int64_t all;
    const int64_t to = rows + block_scan(n, part, &all), from = to - n;
    rows += all;
    const int64_t held = (c + S - 1) / S, want = (c + n + S - 1) / S;
    const bool fits = to <= p.tokens && want <= p.width && c + n <= 0x7FFFFFFF;
    const int64_t take = !have_r ? 0 : fits ? want - held : kNoPages;
    const int64_t upto = pages + block_scan(take, part, &all);
    pages += all;
    const bool granted = have_r && fits && (take == 0 || upto <= count);
    if (granted && take) taken = upto;
    if (have_r) {
      p.offsets[r] = static_cast<int32_t>(from < p.tokens ? from : p.tokens);
      p.context[r] = granted ? static_cast<int32_t>(c + n) : 0;
      p.lengths[r] = static_cast<int32_t>(granted ? c + n : c);
    }
    // a warp writes its requests' pages, one request after the other
    for (uint32_t some = __ballot_sync(0xffffffffu, granted && take > 0); some; some &= some - 1) {
      const int who = __ffs(some) - 1;
      const int64_t row = __shfl_sync(0xffffffffu, r, who) * p.table_stride +
                          __shfl_sync(0xffffffffu, held, who);
      const int64_t k = __shfl_sync(0xffffffffu, take, who);
      const int64_t top = count - 1 - (__shfl_sync(0xffffffffu, upto, who) - k);
      for (int64_t i = lane; i < k; i += 32) p.table[row + i] = p.stack[top - i];
    }
  }
  // what was taken: the most of any thread
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) taken = max(taken, __shfl_xor_sync(0xffffffffu, taken, o));
  if (lane == 0) part[tid >> 5] = taken;
  __syncthreads();
  if (tid == 0) {
    for (int i = 1; i < kPagesThreads / 32; ++i) taken = max(taken, part[i]);
    p.offsets[p.requests] = static_cast<int32_t>(rows < p.tokens ? rows : p.tokens);
    p.count_out[0] = static_cast<int32_t>(count - taken);
  }
}

__device__ void place_tokens(const PagesParams& p, int64_t first, int64_t step) {
  const int32_t end = p.offsets[p.requests];
  for (int64_t t = first; t < p.tokens; t += step) {
    int32_t position = 0, slot = -1;
    if (t < end) {
      // the last request that begins at t or before: it has tokens
      int32_t lo = 0, hi = p.requests - 1;
      while (lo < hi) {
        const int32_t mid = lo + (hi - lo + 1) / 2;
        if (p.offsets[mid] <= t)
          lo = mid;
        else
          hi = mid - 1;
      }
      const int32_t begin = p.offsets[lo], n = p.offsets[lo + 1] - begin;
      const int32_t context = p.context[lo];  // 0: no pages
      // (modulo 2^32 where a request that got none says that it holds more)
      position = static_cast<int32_t>(static_cast<uint32_t>(context ? context - n : p.lengths[lo]) +
                                      static_cast<uint32_t>(t - begin));
      if (context) {
        const int32_t index = position / p.page_size, page = p.table[lo * p.table_stride + index];
        const int64_t at = static_cast<int64_t>(page) * p.page_size + position % p.page_size;
        if (page >= 0 && at <= 0x7FFFFFFF) slot = static_cast<int32_t>(at);
      }
    }
    p.positions[t] = position;
    p.slots[t] = slot;
  }
}

__global__ void __launch_bounds__(kPagesThreads) k_assign_pages(const PagesParams p) {
  if (blockIdx.x == 0) assign(p);
  // what the first block wrote is there for the whole cluster
  cooperative_groups::this_cluster().sync();
  place_tokens(p, static_cast<int64_t>(blockIdx.x) * kPagesThreads + threadIdx.x,
               static_cast<int64_t>(gridDim.x) * kPagesThreads);
}

// One block: a warp counts, then pushes, the pages of its requests in turn.
__global__ void __launch_bounds__(kPagesThreads) k_release_pages(const PagesParams p) {
  __shared__ int64_t part[32];
  const int tid = threadIdx.x, lane = tid & 31;
  const int64_t S = p.page_size;
  const int32_t given = p.count[0];
  int64_t top = given < 0 ? 0 : given > p.capacity ? p.capacity : given;
  for (int base = 0; base < p.requests; base += kPagesThreads) {
    const int r = base + tid;
    const bool gone = r < p.requests && p.done[r] != 0;
    int64_t held = gone ? (static_cast<int64_t>(max(p.lengths[r], 0)) + S - 1) / S : 0;
    if (held > p.width) held = p.width;
    const auto valid = [&](int64_t at, bool in) {
      const int32_t page = in ? p.table[at] : -1;
      return page >= 0 && page < p.capacity ? page : -1;
    };
    int64_t good = 0;
    const uint32_t some = __ballot_sync(0xffffffffu, held > 0);
    for (uint32_t left = some; left; left &= left - 1) {
      const int who = __ffs(left) - 1;
      const int64_t row = (base + (tid & ~31) + who) * p.table_stride;
      const int64_t k = __shfl_sync(0xffffffffu, held, who);
      int64_t n = 0;
      for (int64_t i = 0; i < k; i += 32)
        n += __popc(__ballot_sync(0xffffffffu, valid(row + i + lane, i + lane < k) >= 0));
      if (lane == who) good = n;
    }
    int64_t all;
    const int64_t before = top + block_scan(good, part, &all) - good;
    top += all;
    for (uint32_t left = some; left; left &= left - 1) {
      const int who = __ffs(left) - 1;
      const int64_t row = (base + (tid & ~31) + who) * p.table_stride;
      const int64_t k = __shfl_sync(0xffffffffu, held, who);
      int64_t at = __shfl_sync(0xffffffffu, before, who);
      for (int64_t i = 0; i < k; i += 32) {
        const int32_t page = valid(row + i + lane, i + lane < k);
        const uint32_t with = __ballot_sync(0xffffffffu, page >= 0);
        const int64_t to = at + __popc(with & ((1u << lane) - 1));
        if (page >= 0 && to < p.capacity) p.stack[to] = page;
        if (i + lane < k) p.table[row + i + lane] = -1;
        at += __popc(with);
      }
    }
    if (gone) p.lengths[r] = 0;
  }
  if (tid == 0) p.count_out[0] = static_cast<int32_t>(top < p.capacity ? top : p.capacity);
}

// ------------------------------------------------------------------------
// Host

bool on(const void* p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) % bytes) == 0; }

bool on_words(const Heads& h, const void* p, int64_t token, int64_t head, int64_t tokens, int vec) {
  return on(p, 2 * vec) && (tokens <= 1 || token % vec == 0) && (h.heads <= 1 || head % vec == 0);
}

bool on_words(const Side& s, int vec, bool e4m3) {
  return on(s.data, (e4m3 ? 1 : 2) * vec) && s.stride[0] % vec == 0 && s.stride[1] % vec == 0 &&
         s.stride[2] % vec == 0;
}

// Lanes of a row that have work, of words of `vec` values.
int row_units(const RotaryParams& p, int vec) {
  return p.pairs / vec + ((p.head_dim - 2 * p.pairs) / vec + 1) / 2;
}

// Whether rows go by words of `vec` values: whole words of pairs, of the rest, and
// at every row's start, and a row in a warp.
bool by_words(const RotaryParams& p, int vec) {
  if (p.pairs % vec || p.head_dim % vec || row_units(p, vec) > 32 || p.pairs > kMostPairs ||
      !on_words(p.q, p.q.data, p.q.token, p.q.head, p.tokens, vec) ||
      !on_words(p.q, p.out, p.out_token, p.out_head, p.tokens, vec))
    return false;
  return !p.slots || (on_words(p.k, p.k.data, p.k.token, p.k.head, p.tokens, vec) &&
                      on_words(p.v, p.v.data, p.v.token, p.v.head, p.tokens, vec) &&
                      on_words(p.key, vec, p.e4m3) && on_words(p.value, vec, p.e4m3));
}

// Warps that fill the SMs: with fewer rows than these hold, a warp takes what it
// holds at once.
constexpr int64_t kManyWarps = 152 * 32;

template <int kVec>
int launch_words(const RotaryParams& p, int64_t rows, cudaStream_t s) {
  const int units = row_units(p, kVec);
  int lanes = 1;
  while (lanes < units) lanes *= 2;
  const int64_t at_once = 32 / lanes, turns = (rows + at_once - 1) / at_once;
  int64_t each = p.tokens * turns / kManyWarps;
  each = each < 1 ? 1 : each > turns ? turns : each;
  const int64_t span = each * at_once, spans = (rows + span - 1) / span;
  const int64_t blocks = (p.tokens * spans + kRotaryWarps - 1) / kRotaryWarps;
  const auto kernel = p.slots ? p.interleaved ? k_rotary<kVec, true, true>
                                              : k_rotary<kVec, true, false>
                      : p.interleaved ? k_rotary<kVec, false, true>
                                      : k_rotary<kVec, false, false>;
  kernel<<<static_cast<unsigned>(blocks), 32 * kRotaryWarps, 0, s>>>(
      p, lanes, static_cast<int>(span), static_cast<int>(spans));
  return cudaGetLastError();
}

}  // namespace

int launch_rotary(const RotaryParams& p, void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int64_t rows = p.q.heads + (p.slots ? 2 * p.k.heads : 0);
  if (rows == 0) return cudaSuccess;
  if (by_words(p, 8)) return launch_words<8>(p, rows, s);
  if (by_words(p, 4)) return launch_words<4>(p, rows, s);
  const int64_t blocks = (p.tokens * rows + kRotaryWarps - 1) / kRotaryWarps;
  k_rotary_any<<<static_cast<unsigned>(blocks), 32 * kRotaryWarps, 0, s>>>(p);
  return cudaGetLastError();
}

int launch_assign_pages(const PagesParams& p, void* stream) {
  cudaLaunchConfig_t config{};
  config.gridDim = dim3(p.tokens <= 2 * kPagesThreads ? 1 : kPagesCluster);
  config.blockDim = dim3(kPagesThreads);
  config.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute cluster{};
  cluster.id = cudaLaunchAttributeClusterDimension;
  cluster.val.clusterDim.x = config.gridDim.x;
  cluster.val.clusterDim.y = cluster.val.clusterDim.z = 1;
  config.attrs = &cluster;
  config.numAttrs = 1;
  return cudaLaunchKernelEx(&config, k_assign_pages, p);
}

int launch_release_pages(const PagesParams& p, void* stream) {
  k_release_pages<<<1, kPagesThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
  return cudaGetLastError();
}

}  // namespace ciera
