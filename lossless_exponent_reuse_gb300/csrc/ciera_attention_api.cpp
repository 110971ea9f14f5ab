// ciera_attention_api.cpp -- host side of the attention half's operators:
// argument checks.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "ciera.h"
#include "ciera_attention.h"
#include "ciera_moe.h"

using namespace ciera;

namespace {

constexpr int64_t kMaxRows = (int64_t(1) << 31) - 4096;
constexpr int64_t kMaxStride = int64_t(1) << 40;
constexpr int64_t kMaxRotaryDim = 1024;
constexpr int64_t kMaxAttendDim = 256;
constexpr int64_t kMaxRequests = int64_t(1) << 20;
constexpr int64_t kMaxSlots = (int64_t(1) << 31) - 1;

bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

bool buffer(const void* p, int64_t elements, uintptr_t size) {
  return (p || elements == 0) && aligned(p, size);
}

// Rows of `dim` elements, n[i] of them `stride[i]` apart in each direction:
// strides in range.  Rows that are written may not overlap: from the shortest
// stride up each has to clear what lies below it.
bool strided(int rank, const int64_t* n, const int64_t* stride, int64_t dim, bool written) {
  int64_t have[3], at[3];
  int used = 0;
  for (int i = 0; i < rank; ++i) {
    if (n[i] < 0 || stride[i] < 0 || stride[i] > kMaxStride) return false;
    if (n[i] == 0) return true;
    if (n[i] > 1) {
      have[used] = n[i];
      at[used++] = stride[i];
    }
  }
  if (!written) return true;
  __int128 extent = dim;
  for (int done = 0; done < used; ++done) {
    int least = done;
    for (int i = done + 1; i < used; ++i)
      if (at[i] < at[least]) least = i;
    const int64_t s = at[least], c = have[least];
    at[least] = at[done];
    have[least] = have[done];
    if (s < extent) return false;
    extent += static_cast<__int128>(s) * (c - 1);
  }
  return extent < (static_cast<__int128>(1) << 62);
}

bool heads_of(const uint16_t* p, int64_t token_stride, int64_t head_stride, int64_t tokens,
              int64_t heads, int64_t dim, bool written) {
  const int64_t n[2] = {tokens, heads}, stride[2] = {token_stride, head_stride};
  return tokens >= 0 && heads >= 0 && tokens <= kMaxRows && heads <= kMaxRows &&
         (heads == 0 || tokens <= kMaxRows / heads) && strided(2, n, stride, dim, written) &&
         buffer(p, tokens * heads, 2);
}

bool side_of(Side* s, void* data, const int64_t* stride, uint8_t* exponent,
             const int64_t* exponent_stride, const ciera_cache& c, bool written) {
  const bool e4m3 = c.type == CIERA_E4M3;
  const int64_t n[3] = {c.pages, c.page_size, c.heads};
  const int64_t rows = c.pages * c.page_size * c.heads;
  if (!strided(3, n, stride, c.head_dim, written) || !buffer(data, rows, e4m3 ? 1 : 2)) return false;
  if (e4m3 ? !strided(3, n, exponent_stride, 1, written) || !buffer(exponent, rows, 1)
           : exponent != nullptr)
    return false;
  s->data = data;
  s->exponent = exponent;
  for (int i = 0; i < 3; ++i) {
    s->stride[i] = stride[i];
    s->exponent_stride[i] = e4m3 ? exponent_stride[i] : 0;
  }
  return true;
}

bool cache_of(const ciera_cache* c, Side* key, Side* value, bool written) {
  if (!c || (c->type != CIERA_BF16 && c->type != CIERA_E4M3) || c->pages < 0 ||
      c->page_size < 1 || c->heads < 0 || c->head_dim < 0 || c->heads > kMaxRows ||
      c->page_size > kMaxSlots || c->pages > kMaxSlots / c->page_size ||
      (c->heads && c->pages * c->page_size > (int64_t(1) << 50) / c->heads))
    return false;
  return side_of(key, c->key_dev, c->key_stride, c->key_exponent_dev, c->key_exponent_stride, *c,
                 written) &&
         side_of(value, c->value_dev, c->value_stride, c->value_exponent_dev,
                 c->value_exponent_stride, *c, written);
}

int status_of(int cuda) { return cuda == cudaSuccess ? CIERA_OK : CIERA_E_CUDA; }

}  // namespace

extern "C" {

int ciera_rotary(const uint16_t *x_dev, int64_t x_token_stride, int64_t x_head_stride,
                 const int32_t *positions_dev, const int64_t *turns_dev, int64_t pairs,
                 float amplitude, int64_t tokens, int64_t heads, int64_t head_dim,
                 uint16_t *y_dev, int64_t y_token_stride, int64_t y_head_stride, uint32_t flags,
                 void *stream) {
  if (head_dim < 0 || head_dim > kMaxRotaryDim || pairs < 0 || pairs > head_dim / 2 ||
      !std::isfinite(amplitude) || (flags & ~(CIERA_INTERLEAVED | CIERA_INVERSE)))
    return CIERA_E_INVAL;
  if (!heads_of(x_dev, x_token_stride, x_head_stride, tokens, heads, head_dim, false) ||
      !heads_of(y_dev, y_token_stride, y_head_stride, tokens, heads, head_dim, true) ||
      !buffer(positions_dev, tokens, 4) || !buffer(turns_dev, pairs, 8))
    return CIERA_E_INVAL;
  if (y_dev == x_dev && ((tokens > 1 && x_token_stride != y_token_stride) ||
                         (heads > 1 && x_head_stride != y_head_stride)))
    return CIERA_E_INVAL;
  if (tokens == 0 || heads == 0 || head_dim == 0) return CIERA_OK;
  RotaryParams p{};
  p.q = {x_dev, x_token_stride, x_head_stride, heads};
  p.out = y_dev;
  p.out_token = y_token_stride;
  p.out_head = y_head_stride;
  p.positions = positions_dev;
  p.turns = turns_dev;
  p.pairs = static_cast<int32_t>(pairs);
  p.head_dim = static_cast<int32_t>(head_dim);
  p.interleaved = (flags & CIERA_INTERLEAVED) != 0;
  p.inverse = (flags & CIERA_INVERSE) != 0;
  p.amplitude = amplitude;
  p.tokens = tokens;
  return status_of(launch_rotary(p, stream));
}

int ciera_append(const uint16_t *q_dev, int64_t q_token_stride, int64_t q_head_stride,
                 const uint16_t *k_dev, int64_t k_token_stride, int64_t k_head_stride,
                 const uint16_t *v_dev, int64_t v_token_stride, int64_t v_head_stride,
                 const int32_t *positions_dev, const int32_t *slots_dev, const int64_t *turns_dev,
                 int64_t pairs, float amplitude, int64_t tokens, int64_t q_heads,
                 uint16_t *q_out_dev, int64_t out_token_stride, int64_t out_head_stride,
                 const ciera_cache *cache, uint32_t flags, void *stream) {
  RotaryParams p{};
  if (!cache_of(cache, &p.key, &p.value, true)) return CIERA_E_INVAL;
  const int64_t dim = cache->head_dim;
  if (dim > kMaxRotaryDim || pairs < 0 || pairs > dim / 2 || !std::isfinite(amplitude) ||
      (flags & ~CIERA_INTERLEAVED))
    return CIERA_E_INVAL;
  if (!heads_of(q_dev, q_token_stride, q_head_stride, tokens, q_heads, dim, false) ||
      !heads_of(q_out_dev, out_token_stride, out_head_stride, tokens, q_heads, dim, true) ||
      !heads_of(k_dev, k_token_stride, k_head_stride, tokens, cache->heads, dim, false) ||
      !heads_of(v_dev, v_token_stride, v_head_stride, tokens, cache->heads, dim, false) ||
      !buffer(positions_dev, tokens, 4) || !buffer(slots_dev, tokens, 4) ||
      !buffer(turns_dev, pairs, 8) || tokens > kMaxRows / (q_heads + 2 * cache->heads + 1))
    return CIERA_E_INVAL;
  if (q_out_dev == q_dev && ((tokens > 1 && q_token_stride != out_token_stride) ||
                             (q_heads > 1 && q_head_stride != out_head_stride)))
    return CIERA_E_INVAL;
  if (tokens == 0 || dim == 0) return CIERA_OK;
  p.q = {q_dev, q_token_stride, q_head_stride, q_heads};
  p.k = {k_dev, k_token_stride, k_head_stride, cache->heads};
  p.v = {v_dev, v_token_stride, v_head_stride, cache->heads};
  p.out = q_out_dev;
  p.out_token = out_token_stride;
  p.out_head = out_head_stride;
  p.positions = positions_dev;
  p.slots = slots_dev;
  p.turns = turns_dev;
  p.pairs = static_cast<int32_t>(pairs);
  p.head_dim = static_cast<int32_t>(dim);
  p.interleaved = (flags & CIERA_INTERLEAVED) != 0;
  p.e4m3 = cache->type == CIERA_E4M3;
  p.amplitude = amplitude;
  p.tokens = tokens;
  p.pages = static_cast<int32_t>(cache->pages);
  p.page_size = static_cast<int32_t>(cache->page_size);
  return status_of(launch_rotary(p, stream));
}

int ciera_assign_pages(const int32_t *cached_dev, const int32_t *new_dev, int64_t requests,
                       int64_t tokens, int64_t page_size, int32_t *table_dev,
                       int64_t table_stride, int64_t width, const int32_t *free_dev,
                       int64_t capacity, const int32_t *count_dev, int32_t *count_out_dev,
                       int32_t *offsets_dev, int32_t *context_dev, int32_t *lengths_dev,
                       int32_t *positions_dev, int32_t *slots_dev, void *stream) {
  if (requests < 0 || requests > kMaxRequests || tokens < 0 || tokens > kMaxRows ||
      page_size < 1 || page_size > kMaxSlots || width < 0 || width > kMaxSlots ||
      table_stride < width || table_stride > kMaxStride || capacity < 0 || capacity > kMaxSlots)
    return CIERA_E_INVAL;
  if (!buffer(cached_dev, requests, 4) || !buffer(new_dev, requests, 4) ||
      !buffer(table_dev, requests * width, 4) || !buffer(free_dev, capacity, 4) ||
      !buffer(count_dev, 1, 4) || !buffer(count_out_dev, 1, 4) || !buffer(offsets_dev, 1, 4) ||
      !buffer(context_dev, requests, 4) || !buffer(lengths_dev, requests, 4) ||
      !buffer(positions_dev, tokens, 4) || !buffer(slots_dev, tokens, 4))
    return CIERA_E_INVAL;
  PagesParams p{};
  p.cached = cached_dev;
  p.fresh = new_dev;
  p.requests = static_cast<int32_t>(requests);
  p.tokens = static_cast<int32_t>(tokens);
  p.page_size = static_cast<int32_t>(page_size);
  p.table = table_dev;
  p.table_stride = table_stride;
  p.width = width;
  p.stack = const_cast<int32_t*>(free_dev);
  p.capacity = static_cast<int32_t>(capacity);
  p.count = count_dev;
  p.count_out = count_out_dev;
  p.offsets = offsets_dev;
  p.context = context_dev;
  p.lengths = lengths_dev;
  p.positions = positions_dev;
  p.slots = slots_dev;
  return status_of(launch_assign_pages(p, stream));
}

int ciera_release_pages(const uint8_t *done_dev, int32_t *lengths_dev, int64_t requests,
                        int64_t page_size, int32_t *table_dev, int64_t table_stride,
                        int64_t width, int32_t *free_dev, int64_t capacity,
                        const int32_t *count_dev, int32_t *count_out_dev, void *stream) {
  if (requests < 0 || requests > kMaxRequests || page_size < 1 || page_size > kMaxSlots ||
      width < 0 || width > kMaxSlots || table_stride < width || table_stride > kMaxStride ||
      capacity < 0 || capacity > kMaxSlots)
    return CIERA_E_INVAL;
  if (!buffer(done_dev, requests, 1) || !buffer(lengths_dev, requests, 4) ||
      !buffer(table_dev, requests * width, 4) || !buffer(free_dev, capacity, 4) ||
      !buffer(count_dev, 1, 4) || !buffer(count_out_dev, 1, 4))
    return CIERA_E_INVAL;
  PagesParams p{};
  p.done = done_dev;
  p.lengths = lengths_dev;
  p.requests = static_cast<int32_t>(requests);
  p.page_size = static_cast<int32_t>(page_size);
  p.table = table_dev;
  p.table_stride = table_stride;
  p.width = width;
  p.stack = free_dev;
  p.capacity = static_cast<int32_t>(capacity);
  p.count = count_dev;
  p.count_out = count_out_dev;
  return status_of(launch_release_pages(p, stream));
}

int64_t ciera_attend_workspace_bytes(int64_t q_heads, int64_t heads, int64_t head_dim) {
  if (heads < 1 || q_heads < heads || q_heads % heads || q_heads > kMaxRows || head_dim < 1 ||
      head_dim > kMaxAttendDim)
    return 0;
  return attend_workspace_bytes(q_heads, heads, head_dim);
}

int ciera_attend(const uint16_t *q_dev, int64_t q_token_stride, int64_t q_head_stride,
                 int64_t tokens, int64_t q_heads, const ciera_cache *cache,
                 const int32_t *table_dev, int64_t table_stride, int64_t width,
                 const int32_t *offsets_dev, const int32_t *context_dev, int64_t requests,
                 int64_t longest, float scale, uint16_t *o_dev, void *workspace_dev,
                 int64_t workspace_bytes, void *control_dev, void *stream) {
  AttendParams p{};
  if (!cache_of(cache, &p.key, &p.value, false)) return CIERA_E_INVAL;
  const int64_t dim = cache->head_dim, heads = cache->heads;
  if (heads < 1 || q_heads < heads || q_heads % heads || dim < 1 || dim > kMaxAttendDim ||
      !std::isfinite(scale) || requests < 0 || requests > kMaxRequests || width < 0 ||
      width > kMaxSlots || table_stride < width || table_stride > kMaxStride || longest < 0)
    return CIERA_E_INVAL;
  if (!heads_of(q_dev, q_token_stride, q_head_stride, tokens, q_heads, dim, false) ||
      !buffer(table_dev, requests * width, 4) || !buffer(offsets_dev, requests + 1, 4) ||
      !buffer(context_dev, requests, 4) || !buffer(o_dev, tokens * q_heads, 2) || !control_dev ||
      !aligned(control_dev, 4))
    return CIERA_E_INVAL;
  if (!workspace_dev || !aligned(workspace_dev, 16) ||
      workspace_bytes < attend_workspace_bytes(q_heads, heads, dim))
    return CIERA_E_INVAL;
  if (tokens == 0) return CIERA_OK;
  const int64_t most = width > kMaxRows / cache->page_size ? kMaxRows : width * cache->page_size;
  p.q = q_dev;
  p.q_token = q_token_stride;
  p.q_head = q_head_stride;
  p.table = table_dev;
  p.table_stride = table_stride;
  p.keys_most = static_cast<int32_t>(most);
  p.offsets = offsets_dev;
  p.context = context_dev;
  p.o = o_dev;
  p.tokens = static_cast<int32_t>(tokens);
  p.requests = static_cast<int32_t>(requests);
  p.heads = static_cast<int32_t>(heads);
  p.group = static_cast<int32_t>(q_heads / heads);
  p.head_dim = static_cast<int32_t>(dim);
  p.pages = static_cast<int32_t>(cache->pages);
  p.page_size = static_cast<int32_t>(cache->page_size);
  p.by_group = Divide(static_cast<uint32_t>(p.group));
  p.by_page = Divide(static_cast<uint32_t>(p.page_size));
  p.e4m3 = cache->type == CIERA_E4M3;
  p.scale = scale;
  p.longest = longest < tokens ? longest : tokens;
  p.workspace = workspace_dev;
  p.ctl = static_cast<Control*>(control_dev);
  p.timeout_ns = wait_timeout_ns();
  std::lock_guard<std::mutex> together(launches());
  return status_of(launch_attend(p, stream));
}

}  // extern "C"
