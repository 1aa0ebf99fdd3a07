// cache_host.cu -- C entry points of the per-head norm with rotary positions,
// the cache append and paged attention (declared in include/attn.h). Every
// argument is checked here before any CUDA call; what the device reads
// (lengths, tables, counts) is checked or clamped in the kernels.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "attn.h"
#include "attn_host.h"
#include "attn_kernel.h"
#include "paged_kernel.h"
#include "rope_kernel.h"

namespace {

using attn::host::fail_with;

constexpr int64_t kMaxCount = int64_t{1} << 30;  // tokens, rows and units are counted in 32 bits

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// What a call does with a tensor: an input's strides may be anything, a cache's
// places are boxes of a tensor map, a written tensor must not overlap itself.
enum Use { kRead, kMapped, kWritten };

// Element strides of (b, h, n), or of (page, head, slot): given or contiguous.
// A dimension of size 1 has no stride. A written tensor's dimensions, in the
// order of their strides, must each step over all that the ones before reach.
int strides(const int64_t in[3], const int64_t size[3], int64_t d, Use use, const char* name, int64_t out[3]) {
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

int tensor(const void* p, const int64_t st[3], int B, int H, int N, int d, Use use, const char* name,
           attn::RopeTensor* out) {
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

// The fields that attn_rope_params and attn_rope_bwd_params have in common.
template <typename P>
int check_rope(const P* p) {
  if (p->B < 1 || p->N < 1) return fail_with(ATTN_ERR_INVALID_ARG, "B and N must be >= 1 (got %d, %d)", p->B, p->N);
  if (p->Hq < 0 || p->Hk < 0 || p->Hq + static_cast<int64_t>(p->Hk) < 1 || p->Hq > 16384 || p->Hk > 16384)
    return fail_with(ATTN_ERR_INVALID_ARG, "Hq and Hk must be 0 to 16384 and not both 0 (got %d, %d)", p->Hq, p->Hk);
  if (static_cast<int64_t>(p->B) * p->N >= kMaxCount) return fail_with(ATTN_ERR_INVALID_ARG, "too many tokens");
  if (p->d != 32 && p->d != 64 && p->d != 128)
    return fail_with(ATTN_ERR_UNSUPPORTED, "head dimension %d is not one of 32, 64, 128", p->d);
  if (p->rot < 0 || p->rot > p->d || p->rot % 16 != 0)
    return fail_with(ATTN_ERR_INVALID_ARG, "rot must be a multiple of 16 up to d (got %d)", p->rot);
  if ((p->rot > 0) != (p->inv_freq != nullptr))
    return fail_with(ATTN_ERR_INVALID_ARG, "inv_freq must be given if and only if rot > 0");
  if (!aligned(p->inv_freq, 8)) return fail_with(ATTN_ERR_MISALIGNED, "inv_freq must be 8-byte aligned");
  if (p->norm) {
    if (!std::isfinite(p->eps) || p->eps < 0.f) return fail_with(ATTN_ERR_INVALID_ARG, "eps must be finite and >= 0");
  } else if (p->q_weight != nullptr || p->k_weight != nullptr) {
    return fail_with(ATTN_ERR_INVALID_ARG, "weights without norm");
  }
  for (int i = 0; i < 2; ++i) {
    const int type = i ? p->k_weight_type : p->q_weight_type;
    if (type != ATTN_TYPE_BF16 && type != ATTN_TYPE_FP32) return fail_with(ATTN_ERR_INVALID_ARG, "unknown weight type %d", type);
    if (!aligned(i ? p->k_weight : p->q_weight, type == ATTN_TYPE_FP32 ? 4 : 2))
      return fail_with(ATTN_ERR_MISALIGNED, "weights must be aligned to their type");
  }
  if (p->pos_type < ATTN_POS_NONE || p->pos_type > ATTN_POS_INT64 ||
      (p->pos_type == ATTN_POS_NONE) != (p->positions == nullptr))
    return fail_with(ATTN_ERR_INVALID_ARG, "pos_type must name the type of positions (NONE without)");
  if (!aligned(p->positions, p->pos_type == ATTN_POS_INT64 ? 8 : 4))
    return fail_with(ATTN_ERR_MISALIGNED, "positions must be aligned to their type");
  return ATTN_OK;
}

int log2_page(int page_size, int* shift) {
  if (page_size < 16 || page_size > (1 << 24) || (page_size & (page_size - 1)) != 0)
    return fail_with(ATTN_ERR_INVALID_ARG, "page_size must be a power of two >= 16 (got %d)", page_size);
  *shift = 0;
  while ((1 << *shift) < page_size) ++*shift;
  return ATTN_OK;
}

int fill_rope(const attn_rope_params* p, attn::RopeParams* r) {
  int rc = check_rope(p);
  if (rc != ATTN_OK) return rc;
  std::memset(r, 0, sizeof(*r));
  if (p->Hq > 0) {
    if ((rc = tensor(p->q, p->q_stride, p->B, p->Hq, p->N, p->d, kRead, "q", &r->q)) != ATTN_OK ||
        (rc = tensor(p->q_out, p->q_out_stride, p->B, p->Hq, p->N, p->d, kWritten, "q_out", &r->qo)) != ATTN_OK)
      return rc;
  } else if (p->q || p->q_out || p->q_weight) {
    return fail_with(ATTN_ERR_INVALID_ARG, "q, q_out and q_weight need Hq > 0");
  }
  if (p->Hk > 0) {
    if ((rc = tensor(p->k, p->k_stride, p->B, p->Hk, p->N, p->d, kRead, "k", &r->k)) != ATTN_OK) return rc;
  } else if (p->k || p->k_out || p->k_weight) {
    return fail_with(ATTN_ERR_INVALID_ARG, "k, k_out and k_weight need Hk > 0");
  }
  r->B = p->B;
  r->N = p->N;
  r->Hq = p->Hq;
  r->Hk = p->Hk;
  r->rot = p->rot;
  r->interleaved = p->interleaved != 0;
  r->norm = p->norm != 0;
  r->eps = p->eps;
  r->wq = p->q_weight;
  r->wk = p->k_weight;
  r->wq_type = p->q_weight_type;
  r->wk_type = p->k_weight_type;
  r->inv_freq = p->inv_freq;
  r->pos = p->positions;
  r->pos_type = p->pos_type;
  r->pos_sb = p->pos_stride[0];
  r->pos_sn = p->pos_stride[1];
  r->pos_offset = p->pos_offset;
  return ATTN_OK;
}

// Blocks of 256 threads go over tokens (x) and over the heads in turn (y).
// Few tokens: the heads are dealt to more blocks until the GPU has about
// kBlocksPerSm blocks an SM; the angles are then computed once per block row.
// Measured with 4 / 6 / 12 an SM: B5 N1000 H16+4 d64 appended 9.6 / 9.1 / 13.6 us,
// B4 H16+4 N2048 d128 22.1 / 22.1 / 28.9 us, B2 H20+4 N3000 d64 12.9 / 13.8 / 16.3 us,
// B1 H8+8 N16384 d128 28.9 / 28.9 / 32.1 us.
constexpr int kBlocksPerSm = 6;

int launch_rope(attn::RopeParams* r, int d, int heads, cudaStream_t s) {
  int dev = 0, sms = 0;
  const int rc = attn::host::this_device(&dev, &sms);
  if (rc != ATTN_OK) return rc;
  const int per = attn::rope_tokens_per_block(d);
  const int64_t x = (static_cast<int64_t>(r->B) * r->N + per - 1) / per;
  int64_t y = (static_cast<int64_t>(sms) * kBlocksPerSm + x - 1) / x;
  if (y > heads) y = heads;
  r->heads_per_block = static_cast<int>((heads + y - 1) / y);
  y = (heads + r->heads_per_block - 1) / r->heads_per_block;
  const cudaError_t e = attn::launch_rope(*r, d, dim3(static_cast<unsigned>(x), static_cast<unsigned>(y)), s);
  return e == cudaSuccess ? ATTN_OK : attn::host::cuda_error(e, "norm and rotation launch");
}

// Blocks of the backward: what an SM holds, each over many tokens, so that few rows
// of partial sums are left to add (with 1 / 2 / 4 / 8 blocks an SM, d = 128: B8 H32+8
// N4096 294 / 190 / 193 / 196 us, B4 H16+4 N2048 50.8 / 31.6 / 33.1 / 33.1, B1 H8+8
// N16384 78.4 / 51.7 / 50.6 / 54.7).
constexpr int kBwdBlocksPerSm = 2;

int bwd_blocks(const attn_rope_bwd_params* p, int sms) {
  const int per = attn::rope_tokens_per_block(p->d);
  const int64_t x = (static_cast<int64_t>(p->B) * p->N + per - 1) / per;
  return static_cast<int>(x < static_cast<int64_t>(sms) * kBwdBlocksPerSm ? x : static_cast<int64_t>(sms) * kBwdBlocksPerSm);
}

int64_t bwd_workspace(const attn_rope_bwd_params* p, int blocks) {
  if (!p->norm || (p->dq_weight == nullptr && p->dk_weight == nullptr)) return 0;
  return static_cast<int64_t>(blocks) * 2 * p->d * static_cast<int64_t>(sizeof(float));
}

// ------------------------------------------------------------------ paged attention

int64_t up256(int64_t x) { return (x + 255) & ~int64_t{255}; }

// The join's blocks take four rows each, parts dealt to their warps, if rows are few
// (up to kJoinSplitRows an SM) and may have more than kJoinParts parts; else sixteen.
// Shared blocks and not, d = 128, 256 own keys each: 64 x 8 rows x 2 key heads behind
// 8192 tokens 21.0 and 26.0 us, 32 x 4 x 8 behind 4096 20.4 and 21.0, 8 x 32 x 8 behind
// 2048 19.6 and 19.0; 64 an SM instead of 16: 32 x 16 x 8 behind 512 26.2 and 19.1. Own
// keys only (1024), a task and more a CTA, so a part or two a row: 57 x 4 x 8 44.6 and 42.2.
// Sixteen rows a block: eight parts' loads in flight up to kJoinFewRows rows an SM
// (32 x 16 x 8 behind 2048 24.8 us, four 26.4; 96 x 4 x 8 behind 32768 119.8 and
// 121.7), four above (32 x 32 x 8 behind 2048 29.6 us, eight 30.9; 3 x 512 x 16
// behind 2048 38.2 and 41.7). Shared blocks have eight (four: 64 x 8 x 2 behind 2048
// 19.8 us and not 17.9, behind 8192 23.7 and not 21.2).
constexpr int kJoinSplitRows = 16, kJoinParts = 8, kJoinFewRows = 32;

struct PagedPlan {
  int grid = 0;
  bool batched = false;  // the prefix's tiles once for rows of several sequences
  int64_t tasks = 0, slots = 0, rows_o = 0, rows_ml = 0;  // bytes of the workspace's parts
  int64_t bytes() const { return tasks + slots + rows_o + rows_ml; }
};

int check_paged_sizes(const attn_paged_params* p) {
  if (p == nullptr) return fail_with(ATTN_ERR_INVALID_ARG, "null parameter block");
  if (p->B < 1 || p->Hq < 1 || p->Hk < 1 || p->Nq < 1)
    return fail_with(ATTN_ERR_INVALID_ARG, "B, Hq, Hk and Nq must be >= 1 (got %d, %d, %d, %d)", p->B, p->Hq, p->Hk, p->Nq);
  if (p->Hq % p->Hk != 0) return fail_with(ATTN_ERR_INVALID_ARG, "Hq (%d) must be a multiple of Hk (%d)", p->Hq, p->Hk);
  if (p->d != 32 && p->d != 64 && p->d != 128)
    return fail_with(ATTN_ERR_UNSUPPORTED, "head dimension %d is not one of 32, 64, 128", p->d);
  if (p->prefix_len < 0) return fail_with(ATTN_ERR_INVALID_ARG, "prefix_len must be >= 0");
  if (p->num_ctas < 0) return fail_with(ATTN_ERR_INVALID_ARG, "num_ctas must be >= 0");
  // (in steps, so that no product passes 64 bits)
  int64_t rows = static_cast<int64_t>(p->B) * p->Nq;
  if (rows < kMaxCount) rows *= p->Hq;
  if (rows >= kMaxCount) return fail_with(ATTN_ERR_INVALID_ARG, "too many query rows");
  return ATTN_OK;
}

void plan_paged(const attn_paged_params* p, int sms, PagedPlan* pl) {
  pl->grid = p->num_ctas > 0 && p->num_ctas < sms ? p->num_ctas : sms;
  const int64_t rows = static_cast<int64_t>(p->B) * p->Nq * p->Hq;
  // Batched: 256 rows of the batch read the prefix's tiles together, and each
  // row's prefix part and own part go through the workspace to the join.
  // Otherwise each sequence's tasks go over the prefix and its own keys in one
  // go. What batching saves is tiles, what it costs are the prefix tasks' start
  // and end and a longer join, so it has to save some tiles a CTA: one if a key
  // head's rows fit one query tile, five if not. Measured at d = 128 with 256 own
  // keys, batched and not (sequences x rows x key heads, prefix):
  //   one tile:  16 x 8 x 2, 512: 0.8 saved, 12.0 and 11.7 us; 2048: 3.1, 12.8 and 14.7
  //              4 x 4 x 8, 512: 0.6, 12.1 and 12.0;  16 x 4 x 8, 512: 3.1, 15.1 and 16.5
  //   pairs:     64 x 8 x 2, 512: 3.2, 16.9 and 17.2; 8 x 32 x 8, 2048: 5.8, 19.4 and 18.2
  //              32 x 16 x 8, 512: 6.2, 19.7 and 23.8; 2048: 25, 24.4 and 37.9
  //   96 x 4 x 8 behind 32768: 120 and 1126;  3 x 512 x 16 behind 2048 (saves none): 54 and 38
  constexpr int kGainOne = 1, kGainPair = 5;
  const int64_t rs = static_cast<int64_t>(p->Nq) * (p->Hq / p->Hk), tr = attn::kPagedTaskRows;
  const int64_t own = (rs + tr - 1) / tr, pre = (p->B * rs + tr - 1) / tr, tiles = (static_cast<int64_t>(p->prefix_len) + 127) / 128;
  const int64_t gain = p->Hk * (p->B * own * tiles - pre * (tiles + 1));
  pl->batched = gain > pl->grid * (p->B * rs <= attn::kBM ? kGainOne : kGainPair);
  pl->tasks = up256((p->B * p->Hk * own + (pl->batched ? p->Hk * pre : 0)) * static_cast<int64_t>(sizeof(int2)));
  pl->slots = up256(static_cast<int64_t>(pl->grid) * 4 * 128 * (p->d + 2) * 4);
  if (pl->batched) {
    const int64_t rows32 = attn::paged_rows32(static_cast<int>(rows));
    pl->rows_o = up256(2 * rows32 * p->d * 4);
    pl->rows_ml = up256(2 * rows32 * 8);
  }
}

int encode_pages(PFN_cuTensorMapEncodeTiled_v12000 encode, CUtensorMap* m, const void* base, int d, int page_size,
                 int heads, int pages, const int64_t st[3], const char* name) {
  const int cols = d >= 64 ? 64 : 32;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(page_size),
                              static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(pages)};
  // a dimension of size 1 may have any stride that the map accepts
  auto bytes = [&](int64_t s) { return static_cast<cuuint64_t>(s > 0 ? s : d) * 2; };
  const cuuint64_t strides[3] = {bytes(st[2]), bytes(st[1]), bytes(st[0])};
  const cuuint32_t box[4] = {static_cast<cuuint32_t>(cols),
                             static_cast<cuuint32_t>(page_size < attn::kBN ? page_size : attn::kBN), 1, 1};
  const cuuint32_t ones[4] = {1, 1, 1, 1};
  const CUresult r = encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, ones,
                            CU_TENSOR_MAP_INTERLEAVE_NONE,
                            d >= 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS)
    return fail_with(ATTN_ERR_CUDA, "cuTensorMapEncodeTiled(%s) failed with CUresult %d", name, static_cast<int>(r));
  return ATTN_OK;
}

int encode_queries(PFN_cuTensorMapEncodeTiled_v12000 encode, CUtensorMap* m, const attn_paged_params* p,
                   const attn::RopeTensor& q, int G, bool sequences) {
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(p->d), static_cast<cuuint64_t>(p->Hq),
                              static_cast<cuuint64_t>(p->Nq), static_cast<cuuint64_t>(p->B)};
  auto bytes = [&](int64_t s) { return static_cast<cuuint64_t>(s > 0 ? s : p->d) * 2; };
  const cuuint64_t strides[3] = {bytes(q.sh), bytes(q.sn), bytes(q.sb)};
  const cuuint32_t nq = static_cast<cuuint32_t>(sequences ? p->Nq : 128 / G);
  const cuuint32_t box[4] = {static_cast<cuuint32_t>(p->d >= 64 ? 64 : 32), static_cast<cuuint32_t>(G), nq,
                             128u / (static_cast<cuuint32_t>(G) * nq)};
  const cuuint32_t ones[4] = {1, 1, 1, 1};
  const CUresult r = encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, q.p, dims, strides, box, ones,
                            CU_TENSOR_MAP_INTERLEAVE_NONE,
                            p->d >= 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                            CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS)
    return fail_with(ATTN_ERR_CUDA, "cuTensorMapEncodeTiled(q) failed with CUresult %d", static_cast<int>(r));
  return ATTN_OK;
}

}  // namespace

extern "C" {

void attn_rope_params_init(attn_rope_params* p) {
  if (p) std::memset(p, 0, sizeof(*p));
}

void attn_rope_bwd_params_init(attn_rope_bwd_params* p) {
  if (p) std::memset(p, 0, sizeof(*p));
}

void attn_paged_params_init(attn_paged_params* p) {
  if (p) std::memset(p, 0, sizeof(*p));
}

int attn_struct_size(int which) {
  switch (which) {
    case 0: return static_cast<int>(sizeof(attn_rope_params));
    case 1: return static_cast<int>(sizeof(attn_rope_bwd_params));
    case 2: return static_cast<int>(sizeof(attn_paged_params));
    default: return 0;
  }
}

int attn_qk_norm_rope(const attn_rope_params* p) {
  attn::host::clear_error();
  if (p == nullptr) return fail_with(ATTN_ERR_INVALID_ARG, "null parameter block");
  attn::RopeParams r;
  int rc = fill_rope(p, &r);
  if (rc != ATTN_OK) return rc;
  if (p->v || p->k_cache || p->v_cache || p->block_table || p->starts || p->counts)
    return fail_with(ATTN_ERR_INVALID_ARG, "v and the cache fields are attn_kv_append's");
  if (p->Hk > 0 &&
      (rc = tensor(p->k_out, p->k_out_stride, p->B, p->Hk, p->N, p->d, kWritten, "k_out", &r.ko)) != ATTN_OK)
    return rc;
  return launch_rope(&r, p->d, p->Hq + p->Hk, attn::host::stream_of(p->stream));
}

int attn_kv_append(const attn_rope_params* p) {
  attn::host::clear_error();
  if (p == nullptr) return fail_with(ATTN_ERR_INVALID_ARG, "null parameter block");
  attn::RopeParams r;
  int rc = fill_rope(p, &r);
  if (rc != ATTN_OK) return rc;
  if (p->Hk < 1) return fail_with(ATTN_ERR_INVALID_ARG, "Hk must be >= 1");
  if (p->k_out) return fail_with(ATTN_ERR_INVALID_ARG, "k_out is attn_qk_norm_rope's: the keys go to their pages");
  if ((rc = tensor(p->v, p->v_stride, p->B, p->Hk, p->N, p->d, kRead, "v", &r.v)) != ATTN_OK) return rc;
  if (p->n_pages < 1) return fail_with(ATTN_ERR_INVALID_ARG, "n_pages must be >= 1");
  if ((rc = log2_page(p->page_size, &r.page_shift)) != ATTN_OK) return rc;
  attn::RopeTensor c;
  if ((rc = tensor(p->k_cache, p->k_cache_stride, p->n_pages, p->Hk, p->page_size, p->d, kWritten, "k_cache", &c)) != ATTN_OK)
    return rc;
  r.kc = c.p;
  r.kc_sp = c.sb;
  r.kc_sh = c.sh;
  r.kc_st = c.sn;
  if ((rc = tensor(p->v_cache, p->v_cache_stride, p->n_pages, p->Hk, p->page_size, p->d, kWritten, "v_cache", &c)) != ATTN_OK)
    return rc;
  r.vc = c.p;
  r.vc_sp = c.sb;
  r.vc_sh = c.sh;
  r.vc_st = c.sn;
  if (!p->block_table || !p->starts) return fail_with(ATTN_ERR_INVALID_ARG, "block_table and starts must be non-null");
  if (!aligned(p->block_table, 4) || !aligned(p->starts, 4) || !aligned(p->counts, 4))
    return fail_with(ATTN_ERR_MISALIGNED, "block_table, starts and counts must be 4-byte aligned");
  if (p->table_width < 1 || p->table_stride < 0 || (p->B > 1 && p->table_stride < p->table_width))
    return fail_with(ATTN_ERR_INVALID_ARG, "table_width must be >= 1 and table_stride no smaller");
  r.cache = 1;
  r.n_pages = p->n_pages;
  r.table = p->block_table;
  r.table_sb = p->table_stride;
  r.table_width = p->table_width;
  r.starts = p->starts;
  r.counts = p->counts;
  return launch_rope(&r, p->d, p->Hq + 2 * p->Hk, attn::host::stream_of(p->stream));
}

int64_t attn_qk_norm_rope_bwd_workspace_bytes(const attn_rope_bwd_params* p) {
  attn::host::clear_error();
  if (p == nullptr) return -fail_with(ATTN_ERR_INVALID_ARG, "null parameter block");
  int rc = check_rope(p), dev = 0, sms = 0;
  if (rc != ATTN_OK || (rc = attn::host::this_device(&dev, &sms)) != ATTN_OK) return -rc;
  return bwd_workspace(p, bwd_blocks(p, sms));
}

int attn_qk_norm_rope_bwd(const attn_rope_bwd_params* p) {
  attn::host::clear_error();
  if (p == nullptr) return fail_with(ATTN_ERR_INVALID_ARG, "null parameter block");
  int rc = check_rope(p);
  if (rc != ATTN_OK) return rc;
  attn::RopeBwdParams r;
  std::memset(&r, 0, sizeof(r));
  if (p->Hq > 0) {
    if ((rc = tensor(p->q, p->q_stride, p->B, p->Hq, p->N, p->d, kRead, "q", &r.q)) != ATTN_OK ||
        (rc = tensor(p->dq_out, p->dq_out_stride, p->B, p->Hq, p->N, p->d, kRead, "dq_out", &r.dyq)) != ATTN_OK ||
        (rc = tensor(p->dq, p->dq_stride, p->B, p->Hq, p->N, p->d, kWritten, "dq", &r.dq)) != ATTN_OK)
      return rc;
  } else if (p->dq_weight != nullptr) {
    return fail_with(ATTN_ERR_INVALID_ARG, "dq_weight needs Hq > 0");
  }
  if (p->Hk > 0) {
    if ((rc = tensor(p->k, p->k_stride, p->B, p->Hk, p->N, p->d, kRead, "k", &r.k)) != ATTN_OK ||
        (rc = tensor(p->dk_out, p->dk_out_stride, p->B, p->Hk, p->N, p->d, kRead, "dk_out", &r.dyk)) != ATTN_OK ||
        (rc = tensor(p->dk, p->dk_stride, p->B, p->Hk, p->N, p->d, kWritten, "dk", &r.dk)) != ATTN_OK)
      return rc;
  } else if (p->dk_weight != nullptr) {
    return fail_with(ATTN_ERR_INVALID_ARG, "dk_weight needs Hk > 0");
  }
  if (!p->norm && (p->dq_weight || p->dk_weight)) return fail_with(ATTN_ERR_INVALID_ARG, "weight gradients without norm");
  if (!aligned(p->dq_weight, p->q_weight_type == ATTN_TYPE_FP32 ? 4 : 2) ||
      !aligned(p->dk_weight, p->k_weight_type == ATTN_TYPE_FP32 ? 4 : 2))
    return fail_with(ATTN_ERR_MISALIGNED, "weight gradients must be aligned to their type");
  if (p->workspace && !aligned(p->workspace, 16)) return fail_with(ATTN_ERR_MISALIGNED, "workspace must be 16-byte aligned");
  int dev = 0, sms = 0;
  if ((rc = attn::host::this_device(&dev, &sms)) != ATTN_OK) return rc;
  r.blocks = bwd_blocks(p, sms);
  const int64_t need = bwd_workspace(p, r.blocks);
  if (need > 0 && (p->workspace == nullptr || p->workspace_bytes < static_cast<uint64_t>(need)))
    return fail_with(ATTN_ERR_INVALID_ARG, "workspace of %llu bytes, this call needs %lld",
                     static_cast<unsigned long long>(p->workspace ? p->workspace_bytes : 0), static_cast<long long>(need));
  r.B = p->B;
  r.N = p->N;
  r.Hq = p->Hq;
  r.Hk = p->Hk;
  r.rot = p->rot;
  r.interleaved = p->interleaved != 0;
  r.norm = p->norm != 0;
  r.eps = p->eps;
  r.wq = p->q_weight;
  r.wk = p->k_weight;
  r.wq_type = p->q_weight_type;
  r.wk_type = p->k_weight_type;
  r.inv_freq = p->inv_freq;
  r.pos = p->positions;
  r.pos_type = p->pos_type;
  r.pos_sb = p->pos_stride[0];
  r.pos_sn = p->pos_stride[1];
  r.pos_offset = p->pos_offset;
  r.dwq = p->dq_weight;
  r.dwk = p->dk_weight;
  r.part = static_cast<float*>(p->workspace);
  const cudaError_t e = attn::launch_rope_bwd(r, p->d, attn::host::stream_of(p->stream));
  return e == cudaSuccess ? ATTN_OK : attn::host::cuda_error(e, "norm and rotation backward launch");
}

int64_t attn_paged_workspace_bytes(const attn_paged_params* p) {
  attn::host::clear_error();
  int rc = check_paged_sizes(p), dev = 0, sms = 0;
  if (rc != ATTN_OK || (rc = attn::host::this_device(&dev, &sms)) != ATTN_OK) return -rc;
  PagedPlan pl;
  plan_paged(p, sms, &pl);
  return pl.bytes();
}

int attn_paged(const attn_paged_params* p) {
  attn::host::clear_error();
  int rc = check_paged_sizes(p);
  if (rc != ATTN_OK) return rc;
  if (!std::isfinite(p->scale) || !(p->scale > 0.f)) return fail_with(ATTN_ERR_INVALID_ARG, "scale must be finite and > 0");
  if (p->mask_kind != ATTN_MASK_NONE && p->mask_kind != ATTN_MASK_CAUSAL_BR)
    return fail_with(ATTN_ERR_INVALID_ARG, "mask kind %d is not ATTN_MASK_NONE or ATTN_MASK_CAUSAL_BR", p->mask_kind);
  if (p->inject != 0 && p->inject != 1) return fail_with(ATTN_ERR_INVALID_ARG, "inject must be 0 or 1");
  attn::PagedParams k;
  std::memset(static_cast<void*>(&k), 0, sizeof(k));
  attn::RopeTensor q, o, kc, vc;
  if (p->n_pages < 1) return fail_with(ATTN_ERR_INVALID_ARG, "n_pages must be >= 1");
  if ((rc = log2_page(p->page_size, &k.page_shift)) != ATTN_OK ||
      (rc = tensor(p->q, p->q_stride, p->B, p->Hq, p->Nq, p->d, kRead, "q", &q)) != ATTN_OK ||
      (rc = tensor(p->o, p->o_stride, p->B, p->Hq, p->Nq, p->d, kWritten, "o", &o)) != ATTN_OK ||
      (rc = tensor(p->k_cache, p->k_cache_stride, p->n_pages, p->Hk, p->page_size, p->d, kMapped, "k_cache", &kc)) != ATTN_OK ||
      (rc = tensor(p->v_cache, p->v_cache_stride, p->n_pages, p->Hk, p->page_size, p->d, kMapped, "v_cache", &vc)) != ATTN_OK)
    return rc;
  if (!p->block_table || !p->kv_lens) return fail_with(ATTN_ERR_INVALID_ARG, "block_table and kv_lens must be non-null");
  if (!aligned(p->block_table, 4) || !aligned(p->kv_lens, 4) || !aligned(p->q_lens, 4) || !aligned(p->prefix_table, 4) ||
      !aligned(p->lse, 4))
    return fail_with(ATTN_ERR_MISALIGNED, "tables, lengths and lse must be 4-byte aligned");
  if (p->table_width < 1 || p->table_stride < 0 || (p->B > 1 && p->table_stride < p->table_width))
    return fail_with(ATTN_ERR_INVALID_ARG, "table_width must be >= 1 and table_stride no smaller");
  const int64_t max_len = static_cast<int64_t>(p->table_width) * p->page_size;
  if (max_len + p->prefix_len >= kMaxCount) return fail_with(ATTN_ERR_INVALID_ARG, "table too wide");
  if (p->prefix_len > 0 &&
      (p->prefix_table == nullptr || p->prefix_pages < 0 ||
       static_cast<int64_t>(p->prefix_pages) * p->page_size < p->prefix_len))
    return fail_with(ATTN_ERR_INVALID_ARG, "prefix_table does not hold prefix_len tokens");
  // most units that the lengths can give, each task at its longest
  const int64_t G = p->Hq / p->Hk, tasks_own = (p->Nq * G + attn::kPagedTaskRows - 1) / attn::kPagedTaskRows,
                tasks_pre = (static_cast<int64_t>(p->B) * p->Nq * G + attn::kPagedTaskRows - 1) / attn::kPagedTaskRows;
  const double most = static_cast<double>(p->Hk) * attn::kPagedPairTile *
                      (static_cast<double>(tasks_pre) * (p->prefix_len / 128 + 5) +
                       static_cast<double>(p->B) * tasks_own * (static_cast<double>(max_len + p->prefix_len) / 128 + 6));
  if (most >= static_cast<double>(kMaxCount)) return fail_with(ATTN_ERR_INVALID_ARG, "problem too large");
  if (p->workspace && !aligned(p->workspace, 16)) return fail_with(ATTN_ERR_MISALIGNED, "workspace must be 16-byte aligned");

  PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
  int dev = 0, sms = 0;
  if ((rc = attn::host::tensor_map_encoder(&encode)) != ATTN_OK || (rc = attn::host::this_device(&dev, &sms)) != ATTN_OK)
    return rc;
  PagedPlan pl;
  plan_paged(p, sms, &pl);
  if (p->workspace == nullptr || p->workspace_bytes < static_cast<uint64_t>(pl.bytes()))
    return fail_with(ATTN_ERR_INVALID_ARG, "workspace of %llu bytes, this call needs %lld",
                     static_cast<unsigned long long>(p->workspace ? p->workspace_bytes : 0),
                     static_cast<long long>(pl.bytes()));
  const int64_t ks[3] = {kc.sb, kc.sh, kc.sn}, vs[3] = {vc.sb, vc.sh, vc.sn};
  if ((rc = encode_pages(encode, &k.tm_k, p->k_cache, p->d, p->page_size, p->Hk, p->n_pages, ks, "k_cache")) != ATTN_OK ||
      (rc = encode_pages(encode, &k.tm_v, p->v_cache, p->d, p->page_size, p->Hk, p->n_pages, vs, "v_cache")) != ATTN_OK)
    return rc;
  // Query tiles as boxes of a tensor map: 128 / G queries of a sequence, or all
  // queries of several sequences (batched prefix tasks). Boxes against rows
  // gathered one by one: prompt chunks of 3 x 512 tokens behind 2048 38.2 and
  // 43.8 us, 32 sequences decoding behind 4096 shared tokens 26.7 and 28.4 us.
  const bool several = pl.batched && 128 % (p->Nq * G) == 0;
  if (128 % G == 0 && (p->B == 1 || q.sb > 0) && (p->Hq == 1 || q.sh > 0) && (p->Nq == 1 || q.sn > 0)) {
    if ((rc = encode_queries(encode, &k.tm_q, p, q, static_cast<int>(G), several)) != ATTN_OK) return rc;
    k.q_map = several ? 1 : 2;
  }
  k.q = q.p;
  k.q_sb = q.sb;
  k.q_sh = q.sh;
  k.q_sn = q.sn;
  k.o = o.p;
  k.o_sb = o.sb;
  k.o_sh = o.sh;
  k.o_sn = o.sn;
  k.lse = p->lse;
  k.table = p->block_table;
  k.table_sb = p->table_stride;
  k.kv_lens = p->kv_lens;
  k.q_lens = p->q_lens;
  k.prefix_table = p->prefix_table;
  k.B = p->B;
  k.Hq = p->Hq;
  k.Hk = p->Hk;
  k.Nq = p->Nq;
  k.G = static_cast<int>(G);
  k.prefix_len = p->prefix_len;
  k.prefix_tiles = (p->prefix_len + attn::kBN - 1) / attn::kBN;
  k.prefix_tasks = pl.batched ? static_cast<int>(tasks_pre) : 0;
  const int full = attn::kPagedPairTaskCost + k.prefix_tiles * attn::kPagedPairTile;
  int head = k.prefix_tasks * full;  // (the last task may have one query tile)
  if (p->B * p->Nq * G - (tasks_pre - 1) * attn::kPagedTaskRows <= attn::kBM)
    head -= attn::kPagedPairTaskCost - attn::kPagedTaskCost + k.prefix_tiles * (attn::kPagedPairTile - attn::kPagedTile);
  if (!pl.batched) head = 0;
  k.prefix_units = p->Hk * head;
  k.own_tasks = static_cast<int>(tasks_own);
  k.by_batch_rows = attn::FastDiv(static_cast<uint32_t>(p->B * p->Nq * G));
  k.by_g = attn::FastDiv(static_cast<uint32_t>(G));
  k.by_rows = attn::FastDiv(static_cast<uint32_t>(p->Nq * G));
  k.by_prefix_task = attn::FastDiv(static_cast<uint32_t>(full));
  k.by_prefix_head = attn::FastDiv(static_cast<uint32_t>(head > 0 ? head : 1));
  k.max_len = static_cast<int>(max_len);
  k.causal = p->mask_kind == ATTN_MASK_CAUSAL_BR;
  k.row_limits = p->q_lens != nullptr || (k.causal && p->Nq > 1);
  k.c = p->scale * 1.4426950408889634f;
  char* ws = static_cast<char*>(p->workspace);
  k.tasks = reinterpret_cast<int2*>(ws);
  k.slots = reinterpret_cast<float*>(ws + pl.tasks);
  k.rows_o = reinterpret_cast<float*>(ws + pl.tasks + pl.slots);
  k.rows_ml = reinterpret_cast<float2*>(ws + pl.tasks + pl.slots + pl.rows_o);
  k.timeout_ns = p->timeout_ns ? p->timeout_ns : attn::host::kTimeoutNs;
  k.inject = p->inject;
  k.grid = pl.grid;
  const int64_t fewest = p->Hk * (pl.batched && tasks_pre < p->B * tasks_own ? tasks_pre : p->B * tasks_own);
  const int64_t rows = static_cast<int64_t>(p->B) * p->Nq * p->Hq;
  k.join = rows <= kJoinSplitRows * int64_t{sms} && fewest * kJoinParts < pl.grid ? attn::PagedParams::kJoinSplit
           : rows <= kJoinFewRows * int64_t{sms}                                  ? attn::PagedParams::kJoinFew
                                                                                  : attn::PagedParams::kJoinMany;
  attn::host::paged_used(dev);
  const cudaError_t e = attn::launch_paged(k, p->d, attn::host::stream_of(p->stream));
  return e == cudaSuccess ? ATTN_OK : attn::host::cuda_error(e, "paged attention launch");
}

}  // extern "C"
