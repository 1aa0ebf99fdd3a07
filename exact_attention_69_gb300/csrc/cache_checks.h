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

// A cache's tensor map: boxes of `rows` slots, or a page if that is less.
inline int encode_pages(PFN_cuTensorMapEncodeTiled_v12000 encode, CUtensorMap* m, const void* base, int d, int page_size,
                 int heads, int pages, int rows, const int64_t st[3], const char* name) {
  const int cols = d >= 64 ? 64 : 32;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(page_size),
                              static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(pages)};
  // a dimension of size 1 may have any stride that the map accepts
  auto bytes = [&](int64_t s) { return static_cast<cuuint64_t>(s > 0 ? s : d) * 2; };
  const cuuint64_t strides[3] = {bytes(st[2]), bytes(st[1]), bytes(st[0])};
  const cuuint32_t box[4] = {static_cast<cuuint32_t>(cols),
                             static_cast<cuuint32_t>(page_size < rows ? page_size : rows), 1, 1};
  const cuuint32_t ones[4] = {1, 1, 1, 1};
  const CUresult r = encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, ones,
                            CU_TENSOR_MAP_INTERLEAVE_NONE,
                            d >= 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS)
    return fail_with(ATTN_ERR_CUDA, "cuTensorMapEncodeTiled(%s) failed with CUresult %d", name, static_cast<int>(r));
  return ATTN_OK;
}

}  // namespace host
}  // namespace attn
