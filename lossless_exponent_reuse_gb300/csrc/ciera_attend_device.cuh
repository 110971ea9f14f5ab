// ciera_attend_device.cuh -- what the forms of attention over pages share: the
// requests, the pages, and a row computed by one warp value by value.
#pragma once

#include "ciera_attention.h"
#include "ciera_moe_device.cuh"

namespace ciera {
namespace {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr int kSliceValues = 8;   // 256 values of a head over a warp

__device__ __forceinline__ float minus_infinity() { return __uint_as_float(0xFF800000u); }

// Of the weights' sum, 0 of none.
__device__ __forceinline__ float inverse_sum(float sum) { return sum == 0.0f ? 0.0f : 1.0f / sum; }

// A request's tokens and keys as the calls read them.
struct Request {
  int32_t first;   // token
  int32_t tokens;  // new ones
  int32_t keys;    // with the new ones
};

__device__ __forceinline__ int32_t clamp_to(int32_t v, int32_t most) {
  return v < 0 ? 0 : v > most ? most : v;
}

__device__ __forceinline__ Request request_of(const AttendParams& p, int32_t r) {
  const int32_t from = r == 0 ? 0 : clamp_to(p.offsets[r], p.tokens);
  const int32_t to = clamp_to(p.offsets[r + 1], p.tokens);
  return {from, to > from ? to - from : 0, clamp_to(p.context[r], p.keys_most)};
}

// Keys that new token i of a request sees.
__device__ __forceinline__ int32_t seen_keys(const Request& r, int32_t i) {
  const int32_t n = r.keys - r.tokens + i + 1;
  return n > 0 ? n : 0;
}

// Request of token t and its place there; request -1: behind the last.
__device__ void find_row(const AttendParams& p, int32_t t, int32_t* request, int32_t* place) {
  *request = -1;
  *place = 0;
  if (p.requests == 0 || t >= clamp_to(p.offsets[p.requests], p.tokens)) return;
  int32_t lo = 0, hi = p.requests - 1;
  while (lo < hi) {  // the last that begins at t or before
    const int32_t mid = lo + (hi - lo + 1) / 2;
    if (p.offsets[mid] <= t)
      lo = mid;
    else
      hi = mid - 1;
  }
  const Request r = request_of(p, lo);
  if (t < r.first || t - r.first >= r.tokens) return;
  *request = lo;
  *place = t - r.first;
}

// Page that holds a request's key; -1: none.
__device__ __forceinline__ int32_t page_at(const AttendParams& p, int32_t request, int32_t index) {
  const int32_t page = p.table[request * p.table_stride + index];
  return page >= 0 && page < p.pages ? page : -1;
}

// 2^(exponent - 127)
__device__ __forceinline__ float scale_of(uint32_t exponent) {
  return __uint_as_float(exponent == 255 ? 0x7FC00000u : exponent ? exponent << 23 : 0x00400000u);
}

// Where a request's key or value starts; -1: nowhere, zeros.  *exponent: of 8 bits.
__device__ __forceinline__ int64_t place_of(const AttendParams& p, const Side& s, int32_t request,
                                            int32_t head, int32_t key, uint32_t* exponent) {
  const int32_t index = p.by_page(key), page = page_at(p, request, index);
  *exponent = kExponentBias;
  if (page < 0) return -1;
  const int32_t place = key - index * p.page_size;
  if (p.e4m3)
    *exponent = s.exponent[page * s.exponent_stride[0] + place * s.exponent_stride[1] +
                           head * s.exponent_stride[2]];
  return page * s.stride[0] + place * s.stride[1] + head * s.stride[2];
}

__device__ __forceinline__ bool whole_words(const AttendParams& p, const Side& s) {
  const int64_t size = p.e4m3 ? 1 : 2;
  return ((reinterpret_cast<uintptr_t>(s.data) | s.stride[0] * size | s.stride[1] * size |
           s.stride[2] * size | p.head_dim * size) & 15) == 0;
}

// Values d .. d + 31 of a row of 16-byte words, or of any; zeros behind the head's last, and
// of no row.  `some`: a row of queries, which is read in place of what is not there: loads that
// nothing depends on go out together.
template <bool kE4m3>
__device__ __forceinline__ void values32(const AttendParams& p, const Side& s, int64_t at,
                                         const uint16_t* some, int d, bool words, float (&f)[32]) {
  constexpr int kSize = kE4m3 ? 1 : 2, kEach = 16 / kSize;
  const uint8_t* own = reinterpret_cast<const uint8_t*>(some);
  const uint8_t* row = at >= 0 ? static_cast<const uint8_t*>(s.data) + at * kSize : own;
  if (words) {
    uint32_t v[32 / kEach * 4];
#pragma unroll
    for (int i = 0; i < 32 / kEach; ++i) {
      uint4 w = make_uint4(0, 0, 0, 0);
      if (at >= 0 && d + i * kEach < p.head_dim)
        w = *reinterpret_cast<const uint4*>(row + (d + i * kEach) * kSize);
      v[4 * i] = w.x;
      v[4 * i + 1] = w.y;
      v[4 * i + 2] = w.z;
      v[4 * i + 3] = w.w;
    }
#pragma unroll
    for (int i = 0; i < 32; ++i)
      f[i] = kE4m3 ? e4m3_to_f32(static_cast<uint8_t>(v[i / 4] >> (i % 4 * 8)))
                   : i % 2 ? bf16_hi(v[i / 2]) : bf16_lo(v[i / 2]);
    return;
  }
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    const int c = min(d + i, p.head_dim - 1);
    f[i] = kE4m3 ? e4m3_to_f32(row[c]) : bf16_to_f32(reinterpret_cast<const uint16_t*>(row)[c]);
  }
#pragma unroll
  for (int i = 0; i < 32; ++i)
    if (at < 0 || d + i >= p.head_dim) f[i] = 0.0f;
}

// A warp's share of one row: values lane, lane + 32, ... of the head.
struct Slice {
  float most;      // of the scores so far, in powers of two
  float sum;       // of the weights
  float o[kSliceValues];
};

// Row `q` over the keys [from, to) of a request, value by value in 32 bits, of heads
// of up to 32 kValues values.  Keys outside have no part in it.  own->sum 0: no keys.
// 32 keys at a time: a lane a key for the scores, then a key after the other, a lane
// some of its values, eight keys' loads at once: 0.2 us a key (a key at a time 1.2 to 1.7; a
// prompt of 8192 tokens of 16 heads, whose last value is NaN, 325 and 56 ms).
template <int kValues, bool kE4m3>
__device__ __noinline__ void warp_attend(const AttendParams& p, const uint16_t* q, int32_t request,
                                         int32_t head, int32_t from, int32_t to, Slice* own) {
  constexpr int kSize = kE4m3 ? 1 : 2, kAtOnce = 8;
  const int lane = threadIdx.x & 31;
  const bool words = whole_words(p, p.key);
  const float scale = p.scale * kLog2e;
  const uint8_t* values = static_cast<const uint8_t*>(p.value.data);
  const uint8_t* some = reinterpret_cast<const uint8_t*>(q);
  float o[kValues] = {};
  float top = minus_infinity(), sum = 0.0f;   // sum: of this lane's keys
  for (int32_t base = from; base < to; base += 32) {
    const int32_t key = base + lane, n = to - base < 32 ? to - base : 32;
    uint32_t ke = kExponentBias, ve = kExponentBias;
    int64_t kat = -1, vat = -1;
    if (key < to) {
      kat = place_of(p, p.key, request, head, key, &ke);
      vat = place_of(p, p.value, request, head, key, &ve);
    }
    float dot = 0.0f;
    const float by = scale_of(ke);
#pragma unroll 1
    for (int d = 0; d < p.head_dim; d += 32) {
      float k[32], x[32];
      values32<kE4m3>(p, p.key, kat, q, d, words, k);
#pragma unroll
      for (int i = 0; i < 32; ++i) x[i] = bf16_to_f32(q[min(d + i, p.head_dim - 1)]);
#pragma unroll
      for (int i = 0; i < 32; ++i) dot += d + i < p.head_dim ? x[i] * (k[i] * by) : 0.0f;
    }
    const float score = key < to ? dot * scale : minus_infinity();
    float most = fmaxf(score, top);   // (of NaN and a number: the number)
#pragma unroll
    for (int i = 16; i > 0; i >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, i));
    if (__any_sync(0xffffffffu, score != score || top != top)) most = __uint_as_float(0x7FC00000u);
    // (of scores of minus infinity alone no weight is 0 / 0)
    const float zero = most == minus_infinity() ? 0.0f : most;
    const float old = exp2f(top - zero), w = exp2f(score - zero);
    top = most;
    sum = sum * old + w;
#pragma unroll
    for (int i = 0; i < kValues; ++i) o[i] *= old;
#pragma unroll 1
    for (int j0 = 0; j0 < n; j0 += kAtOnce) {   // (keys behind the last weigh 0)
      uint32_t raw[kAtOnce][kValues];
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) {
        const int64_t at = __shfl_sync(0xffffffffu, vat, j0 + j);
        const uint8_t* row = at >= 0 ? values + at * kSize : some;
#pragma unroll
        for (int i = 0; i < kValues; ++i) {
          const int d = min(lane + 32 * i, p.head_dim - 1);
          raw[j][i] = kE4m3 ? row[d] : reinterpret_cast<const uint16_t*>(row)[d];
        }
      }
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) {
        const bool there = __shfl_sync(0xffffffffu, vat, j0 + j) >= 0;
        const float weight = __shfl_sync(0xffffffffu, w, j0 + j);
        const float its = scale_of(__shfl_sync(0xffffffffu, ve, j0 + j));
#pragma unroll
        for (int i = 0; i < kValues; ++i) {
          const float v = kE4m3 ? e4m3_to_f32(static_cast<uint8_t>(raw[j][i])) * its
                                : bf16_to_f32(raw[j][i]);
          o[i] += weight * (there ? v : 0.0f);
        }
      }
    }
  }
  own->most = top;
  own->sum = warp_sum_f32(sum);
#pragma unroll
  for (int i = 0; i < kValues; ++i) own->o[i] = o[i];
}

// Whether some value of a request's keys [from, to), in rows of whole 16-byte words, may be
// infinite or NaN; a lane a key.
__device__ __forceinline__ bool some_odd(const AttendParams& p, int32_t request, int32_t head,
                                         int32_t from, int32_t to) {
  const int words = p.head_dim * (p.e4m3 ? 1 : 2) / 16;
  uint32_t odd = 0;
  for (int32_t key = from + (threadIdx.x & 31); key < to; key += 32) {
    uint32_t exponent;
    const int64_t at = place_of(p, p.value, request, head, key, &exponent);
    if (at < 0) continue;
    odd |= exponent > 246;   // (a product with 2^120 may be infinite)
    const uint4* row = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p.value.data) +
                                                      at * (p.e4m3 ? 1 : 2));
#pragma unroll 8
    for (int i = 0; i < words; ++i) {
      const uint4 v = row[i];
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
      // every exponent (and in 8 bits mantissa) bit set: one more carries
#pragma unroll
      for (int j = 0; j < 4; ++j)
        odd |= p.e4m3 ? ((w[j] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u
                      : ((w[j] & 0x7F807F80u) + 0x00800080u) & 0x80008000u;
    }
  }
  return __any_sync(0xffffffffu, odd != 0);
}

// Of `rows` of a warp (bit i: lane i's row, which sees `seen` keys), whose products took
// in a request's keys up to `to`, those that a value out of their sight has spoilt: one
// that is infinite or NaN, which a weight of 0 makes NaN.  A row that sees a NaN in the
// same place of the head is NaN there by right; rows whose weights' sum is NaN are so in all
// places, and not asked about.  Values' rows are whole 16-byte words.  (A prompt of 8192
// tokens of 16 heads, whose first value is NaN: 298 us, without one 214; every row of
// it computed again was some thousand times as long.)
__device__ __noinline__ uint32_t spoilt_rows(const AttendParams& p, int32_t request, int32_t head,
                                             uint32_t rows, int32_t seen, int32_t to) {
  const int lane = threadIdx.x & 31;
  const int32_t least = __reduce_min_sync(0xffffffffu, rows >> lane & 1 ? seen : to);
  if (!some_odd(p, request, head, least, to)) return 0;
  int32_t last[kSliceValues], nan[kSliceValues];  // key of the last such value, of the first NaN
#pragma unroll
  for (int i = 0; i < kSliceValues; ++i) {
    last[i] = -1;
    nan[i] = 0x7FFFFFFF;
  }
  // from the first row's own key on
  for (int32_t base = least > 0 ? least - 1 : 0; base < to; base += 32) {
    uint32_t exponent = kExponentBias;
    const int64_t at =
        base + lane < to ? place_of(p, p.value, request, head, base + lane, &exponent) : -1;
#pragma unroll 4
    for (int j = 0; j < 32; ++j) {
      const int64_t from = __shfl_sync(0xffffffffu, at, j);
      const float by = scale_of(__shfl_sync(0xffffffffu, exponent, j));
#pragma unroll
      for (int i = 0; i < kSliceValues; ++i) {
        const int d = lane + 32 * i;
        float v = 0.0f;
        if (from >= 0 && d < p.head_dim)
          v = p.e4m3 ? e4m3_to_f32(static_cast<const uint8_t*>(p.value.data)[from + d]) * by
                     : bf16_to_f32(static_cast<const uint16_t*>(p.value.data)[from + d]);
        const uint32_t size = __float_as_uint(v) & 0x7FFFFFFFu;
        if (size >= 0x7F800000u) last[i] = base + j;
        if (size > 0x7F800000u) nan[i] = min(nan[i], base + j);
      }
    }
  }
  uint32_t spoilt = 0;
  for (uint32_t left = rows; left; left &= left - 1) {
    const int who = __ffs(left) - 1;
    const int32_t sees = __shfl_sync(0xffffffffu, seen, who);
    bool some = false;
#pragma unroll
    for (int i = 0; i < kSliceValues; ++i) some |= last[i] >= sees && nan[i] >= sees;
    if (__any_sync(0xffffffffu, some)) spoilt |= 1u << who;
  }
  return spoilt;
}

// ------------------------------------------------------------------------
// How a call's work is dealt out.  A tile is up to kRows rows (new tokens by
// query heads of one head of keys, token by token); a unit is p.unit_keys
// keys of a tile, as many units as its last row sees, one if that sees none.
// A unit weighs 1, and a tile has a weight of its own besides (its queries and output).
// All tiles, in order of request, head and tile, are cut into ranges of even
// weight, as many as there are blocks, whatever the lengths are: ragged batches,
// one long context and whole prompts fill the blocks alike.  A block that has a
// part of a tile leaves its sums in the workspace, in a slot of its own: slot 0
// if the tile began before it, slot 1 if it goes on behind it.  The parts of a tile
// are joined by a launch of their own, in the order of the blocks.

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <int kRows>
struct Tiles {
  static __device__ __forceinline__ int32_t count(const AttendParams& p, const Request& r) {
    return (r.tokens * p.group + kRows - 1) / kRows;
  }
  // Keys that a tile's last row sees.
  static __device__ __forceinline__ int32_t keys(const AttendParams& p, const Request& r,
                                                 int32_t tile) {
    const int32_t left = r.tokens * p.group - tile * kRows;
    const int32_t last = tile * kRows + (left < kRows ? left : kRows) - 1;
    return seen_keys(r, p.by_group(last));
  }
  static __device__ __forceinline__ int32_t units(const AttendParams& p, const Request& r,
                                                  int32_t tile) {
    const int32_t n = keys(p, r, tile);
    return n > 0 ? p.by_unit.up(n) : 1;
  }
  // A tile weighs as much as two of its units besides (8192-token prompt of 16
  // heads, 24 chunks, in us: without 234, 172; one 232, 137; two 236, 128; three 240, 124).
  static constexpr int32_t kTileWeight = 2;
  // The least weight of a block: what one more of the wide form's takes to begin and
  // to be joined is as long as some units (24 rows of 9003 keys, 256 of 2256, in us: least 1
  // 45, 21.9; 2 33, 21.4; 3 28, 21.5; 6 28, 24.4).
  static constexpr int32_t kLeast = kRows == 256 ? 3 : 1;
  static __device__ __forceinline__ int32_t weight(const AttendParams& p, const Request& r,
                                                   int32_t tile) {
    return kTileWeight + units(p, r, tile);
  }
  // Of all tiles of a head of each lane's request; a whole warp.  Its lanes share the
  // tiles of a request that has many (a prompt of 8192 tokens of 16 heads to one: 35 us
  // to find the last block's place by one lane).
  static __device__ int64_t of_head(const AttendParams& p, const Request& r) {
    constexpr int32_t kFew = 8;
    const int lane = threadIdx.x & 31;
    const int32_t n = count(p, r);
    int64_t sum = 0;
    if (n <= kFew)
      for (int32_t t = 0; t < n; ++t) sum += weight(p, r, t);
    for (uint32_t many = __ballot_sync(0xffffffffu, n > kFew); many; many &= many - 1) {
      const int who = __ffs(many) - 1;
      const Request its = {__shfl_sync(0xffffffffu, r.first, who),
                           __shfl_sync(0xffffffffu, r.tokens, who),
                           __shfl_sync(0xffffffffu, r.keys, who)};
      const int32_t tiles = count(p, its);
      int64_t part = 0;
      for (int32_t t = lane; t < tiles; t += 32) part += weight(p, its, t);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) part += __shfl_xor_sync(0xffffffffu, part, o);
      if (lane == who) sum = part;
    }
    return sum;
  }
};

// A block's range and where it begins.
struct Share {
  int64_t total, begin, end;
  int64_t into;      // weight of the first request, then of the first tile, before it
  int64_t of_head;   // of the first request
  int32_t request, head, tile;
  int32_t blocks;    // that have a range: of 1 at least
};

// Sums over the block, inclusive; `part` holds a value per warp and one more.
template <int kThreads>
__device__ __forceinline__ int64_t scan_block(int64_t v, int64_t* part, int64_t* all) {
  constexpr int kWarps = kThreads / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t left = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += left;
  }
  __syncthreads();
  if (lane == 31) part[warp] = v;
  __syncthreads();
  int64_t sum = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) v += part[w];
    sum += part[w];
  }
  *all = sum;
  return v;
}

// The range that a block of `blocks` takes.  Neighbouring blocks are on the two dies in
// turn: the even ones take the first half of the work, the odd ones the second, so
// that keys and values that several blocks read stay in one die's L2 (8192-token
// prompt of 16 heads 259 -> 222 us, of 64 heads of 4096 304 -> 260; 24 chunks 134).
__device__ __forceinline__ int range_of(int block, int blocks) {
  return (block & 1) * ((blocks + 1) / 2) + block / 2;
}

// Fills `share` for block `block` of `blocks`; all kThreads threads.
template <int kRows, int kThreads>
__device__ void find_share(const AttendParams& p, int block, int blocks, int64_t* part,
                           Share* share) {
  using T = Tiles<kRows>;
  const auto weight = [&](int32_t r) -> int64_t {
    const Request none{};
    return T::of_head(p, r < p.requests ? request_of(p, r) : none) * p.heads;
  };
  int64_t own = 0, total;
  for (int32_t base = 0; base < p.requests; base += kThreads) own += weight(base + threadIdx.x);
  const int64_t first = own;
  scan_block<kThreads>(own, part, &total);
  if (total < static_cast<int64_t>(blocks) * T::kLeast)
    blocks = total > T::kLeast ? static_cast<int>(total / T::kLeast) : total > 0;
  const int64_t begin = block < blocks ? block * total / blocks : total;
  const int64_t end = block < blocks ? (block + 1) * total / blocks : total;
  if (threadIdx.x == 0) {
    share->blocks = blocks;
    share->total = total;
    share->begin = begin;
    share->end = end;
  }
  if (begin >= end) {
    __syncthreads();
    return;
  }
  int64_t before = 0, all;
  for (int32_t base = 0; base < p.requests && before <= begin; base += kThreads) {
    const int32_t r = base + threadIdx.x;
    const int64_t n = p.requests <= kThreads ? first : weight(r);
    const int64_t to = before + scan_block<kThreads>(n, part, &all);
    if (begin < to && begin >= to - n) {
      share->request = r;
      share->into = begin - (to - n);
      share->of_head = n / p.heads;
    }
    before += all;
  }
  __syncthreads();
  const Request r = request_of(p, share->request);
  const int32_t tiles = T::count(p, r);
  const int32_t head = static_cast<int32_t>(share->into / share->of_head);
  const int64_t into = share->into - head * share->of_head;
  before = 0;
  for (int32_t base = 0; base < tiles && before <= into; base += kThreads) {
    const int32_t t = base + threadIdx.x;
    const int64_t n = t < tiles ? T::weight(p, r, t) : 0;
    const int64_t to = before + scan_block<kThreads>(n, part, &all);  // (all have read `share`)
    if (into < to && into >= to - n) {
      share->head = head;
      share->tile = t;
      share->into = into - (to - n);
    }
    before += all;
  }
  __syncthreads();
}

// Units [from, to) of one tile, of `all`.
struct Segment {
  Request request;
  int32_t index;     // of the request
  int32_t head, tile;
  int32_t from, to, all;
  int32_t keys;      // that the tile's last row sees
  int32_t rows;      // of the tile
  int64_t end;       // of the tile, in the weight of all
};

template <int kRows>
struct Walk {
  using T = Tiles<kRows>;
  Request request;
  int32_t index, head, tile, tiles;
  int32_t into;      // weight of the tile before `at`
  int64_t at, end;

  __device__ Walk(const AttendParams& p, const Share& s) : at(s.begin), end(s.end) {
    if (at >= end) return;
    index = s.request;
    head = s.head;
    tile = s.tile;
    into = static_cast<int32_t>(s.into);
    request = request_of(p, index);
    tiles = T::count(p, request);
  }
  __device__ bool next(const AttendParams& p, Segment* s) {
    while (at < end) {
      const int32_t all = T::units(p, request, tile), of_tile = T::kTileWeight + all;
      const int32_t upto = end - at < of_tile - into ? into + static_cast<int32_t>(end - at) : of_tile;
      // (the tile's own weight comes before its units)
      const int32_t from = into > T::kTileWeight ? into - T::kTileWeight : 0;
      const int32_t to = upto > T::kTileWeight ? upto - T::kTileWeight : 0;
      s->request = request;
      s->index = index;
      s->head = head;
      s->tile = tile;
      s->keys = T::keys(p, request, tile);
      s->all = all;
      const int32_t left = request.tokens * p.group - tile * kRows;
      s->rows = left < kRows ? left : kRows;
      s->from = from;
      s->to = to;
      s->end = at - into + of_tile;
      at += upto - into;
      into = upto;
      if (into == of_tile) {
        into = 0;
        if (++tile == tiles) {
          tile = 0;
          if (++head == p.heads) {
            head = 0;
            while (at < end && ++index < p.requests) {
              request = request_of(p, index);
              if (request.tokens > 0) break;
            }
            if (index >= p.requests) end = at;
            tiles = T::count(p, request);
          }
        }
      }
      if (from < to) return true;
    }
    return false;
  }
};

// What a block says of the tile that begins in it and ends in another: the
// parts to join, its own slot 1 and the next blocks' slots 0.
struct Joint {
  int32_t parts;   // 0: none
  int32_t first;   // the request's first token
  int32_t row;     // the tile's first row
  int32_t rows;
  int32_t head;
  int32_t pad[3];
};

__device__ __forceinline__ void leave_joint(Joint* joint, const Segment* s, const Share& share,
                                            int32_t row, int block) {
  Joint j{};
  if (s) {
    // the last block that begins before the tile's end
    const int64_t last = (s->end * share.blocks + share.total - 1) / share.total - 1;
    j.parts = static_cast<int32_t>(last) - block + 1;
    j.first = s->request.first;
    j.row = row;
    j.rows = s->rows;
    j.head = s->head;
  }
  *joint = j;
}

// Host: a launch that may begin, and waits, while the last blocks of the one before it
// leave (that one says nothing earlier).
inline int launch_after(void (*kernel)(AttendParams), dim3 grid, int threads, cudaStream_t s,
                        const AttendParams& p) {
  cudaLaunchConfig_t config{};
  config.gridDim = grid;
  config.blockDim = dim3(static_cast<unsigned>(threads));
  config.stream = s;
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  config.attrs = &early;
  config.numAttrs = 1;
  const cudaError_t before = cudaGetLastError();  // of the launch before
  return before != cudaSuccess ? before : cudaLaunchKernelEx(&config, kernel, p);
}

// Query and output of a row: row `row` of a head's rows of a request.
__device__ __forceinline__ const uint16_t* query_row(const AttendParams& p, int32_t first,
                                                     int32_t head, int32_t row) {
  const int32_t i = p.by_group(row);
  return p.q + (static_cast<int64_t>(first) + i) * p.q_token +
         (head * p.group + row - i * p.group) * p.q_head;
}
__device__ __forceinline__ uint16_t* output_row(const AttendParams& p, int32_t first, int32_t head,
                                                int32_t row) {
  const int32_t i = p.by_group(row);
  return p.o + ((static_cast<int64_t>(first) + i) * (p.heads * p.group) + head * p.group + row -
                i * p.group) *
                   p.head_dim;
}

}  // namespace
}  // namespace ciera
