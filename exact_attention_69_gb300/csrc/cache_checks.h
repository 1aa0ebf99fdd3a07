// cache_checks.h -- host checks that the cache operators' entry points share. All of
// them come before any CUDA call.
#pragma once

#include <algorithm>
#include <cstdint>

#include "attn.h"
#include "attn_host.h"
#include "rope_kernel.h"

namespace attn {
namespace host {

constexpr int64_t kMaxCount = int64_t{1} << 30;  // tokens, rows and units are counted in 32 bits

inline bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// What a call does with a tensor: an input's strides may be anything, a cache's
// places are boxes of a tensor map, a written tensor must not overlap itself.
enum Use { kRead, kMapped, kWritten };

// Element strides of (b, h, n), or of (page, head, slot): given or contiguous.
// A dimension of size 1 has no stride. A written tensor's dimensions, in the
// order of their strides, must each step over all that the ones before reach.
inline int strides(const int64_t in[3], const int64_t size[3], int64_t d, Use use, const char* name, int64_t out[3]) {
  if (in[0] == 0 && in[1] == 0 && in[2] == 0) {
    out[2] = d;
    out[1] = size[2] * d;
    out[0] = size[1] * size[2] * d;
    return ATTN_OK;
  }
  for (int i = 0; i < 3; ++i) {
    out[i] = size[i] == 1 ? 0 : in[i];
    if (out[i] < 0) return fail_with(ATTN_ERR_INVALID_ARG, "%s stride %d is negative", name, i);
    if (out[i] % 8 != 0)
      return fail_with(ATTN_ERR_MISALIGNED, "%s stride %d (%lld elements) is not a multiple of 8", name, i,
                       static_cast<long long>(out[i]));
    if (use != kRead && size[i] > 1 && out[i] < d)
      return fail_with(ATTN_ERR_INVALID_ARG, "%s stride %d (%lld elements) is smaller than d", name, i,
                       static_cast<long long>(out[i]));
  }
  if (use != kWritten) return ATTN_OK;
  int order[3] = {0, 1, 2};
  std::sort(order, order + 3, [&](int a, int b) { return out[a] < out[b]; });
  int64_t reach = d;
  for (int i : order) {
    if (size[i] == 1) continue;
    if (out[i] < reach) return fail_with(ATTN_ERR_INVALID_ARG, "%s overlaps itself", name);
    if (out[i] > (INT64_MAX - reach) / (size[i] - 1)) return fail_with(ATTN_ERR_INVALID_ARG, "%s stride %d is too large", name, i);
    reach += out[i] * (size[i] - 1);
  }
  return ATTN_OK;
}

inline int tensor(const void* p, const int64_t st[3], int B, int H, int N, int d, Use use, const char* name,
           RopeTensor* out) {
  if (p == nullptr) return fail_with(ATTN_ERR_INVALID_ARG, "%s must be non-null", name);
  if (!aligned(p, 16)) return fail_with(ATTN_ERR_MISALIGNED, "%s must be 16-byte aligned", name);
  const int64_t size[3] = {B, H, N};
  int64_t s[3];
  const int rc = strides(st, size, d, use, name, s);
  out->p = const_cast<void*>(p);
  out->sb = s[0];
  out->sh = s[1];
  out->sn = s[2];
  return rc;
}

inline int log2_page(int page_size, int* shift) {
  if (page_size < 16 || page_size > (1 << 24) || (page_size & (page_size - 1)) != 0)
    return fail_with(ATTN_ERR_INVALID_ARG, "page_size must be a power of two >= 16 (got %d)", page_size);
  *shift = 0;
  while ((1 << *shift) < page_size) ++*shift;
  return ATTN_OK;
}

}  // namespace host
}  // namespace attn
