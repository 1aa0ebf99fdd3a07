// long_host.cu -- C entry points of the long-cache operators (declared in
// include/attn.h): page bounds and scores, page selection, attention over selected
// pages, received weights, eviction. Every argument is checked here before any CUDA
// call; what the device reads (lengths, tables, lists) is checked in the kernels.
#include <cmath>
#include <cstring>

#include "attn.h"
#include "attn_host.h"
#include "cache_checks.h"
#include "long_kernel.h"

namespace {

using namespace attn::host;
using attn::LongParams;
using attn::RopeTensor;

constexpr int kGridYZ = 65535;  // key heads and sequences are grid dimensions

int check_sizes(const attn_long_params* p, bool queries, bool heads) {
  if (p == nullptr) return fail_with(ATTN_ERR_INVALID_ARG, "null parameter block");
  if (p->B < 1 || p->Hk < 1 || p->B > kGridYZ || p->Hk > kGridYZ)
    return fail_with(ATTN_ERR_INVALID_ARG, "B and Hk must be 1 to %d (got %d, %d)", kGridYZ, p->B, p->Hk);
  if (heads && p->d != 32 && p->d != 64 && p->d != 128)
    return fail_with(ATTN_ERR_UNSUPPORTED, "head dimension %d is not one of 32, 64, 128", p->d);
  if (queries && p->Nq < 1) return fail_with(ATTN_ERR_INVALID_ARG, "Nq must be >= 1 (got %d)", p->Nq);
  if (queries && heads && (p->Hq < 1 || p->Hq % p->Hk != 0))
    return fail_with(ATTN_ERR_INVALID_ARG, "Hq (%d) must be a multiple of Hk (%d)", p->Hq, p->Hk);
  if (queries) {  // (in steps, so that no product passes 64 bits)
    int64_t rows = static_cast<int64_t>(p->B) * p->Nq;
    if (rows < kMaxCount) rows *= heads ? p->Hq : p->Hk;
    if (rows >= kMaxCount) return fail_with(ATTN_ERR_INVALID_ARG, "too many query rows");
  }
  return ATTN_OK;
}

// Sizes, lengths and the table: what every call has.
int fill(const attn_long_params* p, LongParams* r, bool queries, bool heads, bool table) {
  int rc = check_sizes(p, queries, heads);
  if (rc != ATTN_OK) return rc;
  std::memset(static_cast<void*>(r), 0, sizeof(*r));
  if ((rc = log2_page(p->page_size, &r->page_shift)) != ATTN_OK) return rc;
  if (table && p->n_pages < 1) return fail_with(ATTN_ERR_INVALID_ARG, "n_pages must be >= 1");
  if (p->kv_lens == nullptr || (table && p->block_table == nullptr))
    return fail_with(ATTN_ERR_INVALID_ARG, "block_table and kv_lens must be non-null");
  if (!aligned(p->block_table, 4) || !aligned(p->dst_table, 4) || !aligned(p->kv_lens, 4) || !aligned(p->q_lens, 4) ||
      !aligned(p->lse, 4) || !aligned(p->scores, 4) || !aligned(p->blocks, 4) || !aligned(p->weights, 4) ||
      !aligned(p->weights_out, 4) || !aligned(p->kept, 4) || !aligned(p->new_lens, 4))
    return fail_with(ATTN_ERR_MISALIGNED, "tables, lengths, lists, scores, weights and lse must be 4-byte aligned");
  if (p->table_width < 1 || (table && (p->table_stride < 0 || (p->B > 1 && p->table_stride < p->table_width))))
    return fail_with(ATTN_ERR_INVALID_ARG, "table_width must be >= 1 and table_stride no smaller");
  const int64_t max_len = static_cast<int64_t>(p->table_width) * p->page_size;
  if (max_len >= kMaxCount) return fail_with(ATTN_ERR_INVALID_ARG, "table too wide");
  if (queries) {
    if (p->mask_kind != ATTN_MASK_NONE && p->mask_kind != ATTN_MASK_CAUSAL_BR)
      return fail_with(ATTN_ERR_INVALID_ARG, "mask kind %d is not ATTN_MASK_NONE or ATTN_MASK_CAUSAL_BR", p->mask_kind);
    r->causal = p->mask_kind == ATTN_MASK_CAUSAL_BR;
  }
  r->table = p->block_table;
  r->table_sb = p->table_stride;
  r->table_width = p->table_width;
  r->kv_lens = p->kv_lens;
  r->q_lens = p->q_lens;
  r->lse = p->lse;
  r->scores = p->scores;
  r->blocks = p->blocks;
  r->weights = p->weights;
  r->weights_out = p->weights_out;
  r->kept = p->kept;
  r->new_lens = p->new_lens;
  r->bounds = p->bounds;
  r->B = p->B;
  r->Hq = p->Hq;
  r->Hk = p->Hk;
  r->Nq = p->Nq;
  r->G = heads && queries ? p->Hq / p->Hk : 1;
  r->by_g = attn::FastDiv(static_cast<uint32_t>(r->G));
  r->n_pages = p->n_pages;
  r->max_len = static_cast<int>(max_len);
  r->n = p->n;
  r->first = p->first;
  r->last = p->last;
  r->n_new = p->n_new;
  r->decay = p->decay;
  if (p->full_tiles < 0 || p->full_tiles > 2 || p->inject < -1 || p->inject > 1)
    return fail_with(ATTN_ERR_INVALID_ARG, "full_tiles must be 0 to 2, inject -1 to 1");
  r->full_tiles = p->full_tiles;
  r->timeout_ns = p->timeout_ns ? p->timeout_ns : kTimeoutNs;
  r->inject = p->inject;
  return ATTN_OK;
}

int fill_queries(const attn_long_params* p, LongParams* r) {
  RopeTensor q;
  const int rc = tensor(p->q, p->q_stride, p->B, p->Hq, p->Nq, p->d, kRead, "q", &q);
  r->q = q.p;
  r->q_sb = q.sb;
  r->q_sh = q.sh;
  r->q_sn = q.sn;
  return rc;
}

int fill_cache(const attn_long_params* p, LongParams* r, bool keys, bool values, Use use) {
  RopeTensor c;
  int rc;
  if (keys) {
    if ((rc = tensor(p->k_cache, p->k_cache_stride, p->n_pages, p->Hk, p->page_size, p->d, use, "k_cache", &c)) != ATTN_OK)
      return rc;
    r->kc = c.p;
    r->kc_sp = c.sb;
    r->kc_sh = c.sh;
    r->kc_st = c.sn;
  }
  if (values) {
    if ((rc = tensor(p->v_cache, p->v_cache_stride, p->n_pages, p->Hk, p->page_size, p->d, use, "v_cache", &c)) != ATTN_OK)
      return rc;
    r->vc = c.p;
    r->vc_sp = c.sb;
    r->vc_sh = c.sh;
    r->vc_st = c.sn;
  }
  return ATTN_OK;
}

int need(const void* p, const char* name) {
  return p != nullptr ? ATTN_OK : fail_with(ATTN_ERR_INVALID_ARG, "%s must be non-null", name);
}

int check_scale(const attn_long_params* p, LongParams* r) {
  if (!std::isfinite(p->scale) || !(p->scale > 0.f)) return fail_with(ATTN_ERR_INVALID_ARG, "scale must be finite and > 0");
  r->scale = p->scale;
  r->c_hi = p->scale * 1.4426950408889634f;
  return ATTN_OK;
}

int check_taken(const attn_long_params* p, const char* what) {
  if (p->n < 1) return fail_with(ATTN_ERR_INVALID_ARG, "n (%s) must be >= 1", what);
  if (p->first < 0 || p->last < 0 || static_cast<int64_t>(p->first) + p->last > p->n)
    return fail_with(ATTN_ERR_INVALID_ARG, "first and last must be >= 0 and no more than n together");
  return ATTN_OK;
}

// attn_blocks: CTAs that share a tile, a power of two: until there are 1.5 CTAs a SM, while
// every warp has a group of 16 keys.
int blocks_splits(const attn_long_params* p, int sms) {
  const int64_t rows = static_cast<int64_t>(p->Nq) * (p->Hq / p->Hk);
  const int tr = attn::blocks_tile_rows(rows), warps = attn::blocks_warps(tr / 8);
  const int64_t all = (rows + tr - 1) / tr * p->B * p->Hk;
  const int64_t units = static_cast<int64_t>(p->n < p->table_width ? p->n : p->table_width) * (p->page_size / 16);
  int s = 1;
  while (s < attn::kBlocksMaxSplits && 2 * all * s < 3 * static_cast<int64_t>(sms) && 2 * s * warps <= units) s *= 2;
  return s;
}

// attn_blocks, tiles of 128 rows: CTAs that share a tile's stages of 64 keys, each with two of
// them or more and 8 channels of O to join: as many as two CTAs a SM have room for. Work for
// twice as many only makes two rounds, each with a start and a join (us; 64 tiles, by 4 and 8
// CTAs a tile: 34 / 50; 128 tiles, 2 and 4: 40 / 52; 256, 1 and 2: 68 / 80). With q_lens, though,
// a batch is padded, and half of the tiles are taken to have nothing (2 sequences x 512 queries
// x 8 heads of G = 4, 256 tiles, half of the queries padding: 59 by one CTA, 44 by two, 55 by four).
// Lengths are on the device, so this is a guess: q_lens of a batch without padding cost time (without
// them and with them; 1 x 512 queries x 8 heads 40 / 52, 2 x 62 / 76, 4 x 118 / 118).
int blocks_tile_splits(const attn_long_params* p, int sms) {
  const int64_t rows = static_cast<int64_t>(p->Nq) * (p->Hq / p->Hk);
  const int64_t tiles = (rows + 127) / 128 * p->B * p->Hk >> (p->q_lens != nullptr);
  const int64_t stages = (static_cast<int64_t>(p->n < p->table_width ? p->n : p->table_width) * p->page_size + 63) / 64;
  int s = 1;
  while (s < attn::kBlocksMaxSplits && 8 * s < p->d && tiles * s <= sms && 4 * s <= stages) s *= 2;
  return s;
}

// attn_blocks: whether to take tiles of 128 rows. They read a page once for up to 128 rows and
// multiply on full tiles, but take longer to begin and to join. So: where there are 16 rows
// of a sequence and key head, and 12288 pairs of a row and a selected slot a SM in all. Measured
// (us; d = 128, pages of 64, G = 4, 32 pages a query unless said; queries that select much the
// same pages, and pages at random), tiles of 128 and of 16 rows:
//   32 sequences x 8 key heads, 2 queries (8 rows each)   53 /  76   52 /  76
//                               4                         57 / 113   70 / 145
//                               8                         61 / 143  116 / 252
//   32 x 8, G = 16, 1 query                               48         56
//   8 x 8,  4 queries (13800 pairs a SM)                  19 /  38   24 /  44
//         128                                             68 / 216  352 / 843
//   4 x 8,  4 queries (6900)                              15 /  21   17 /  26
//   1 x 8, 16 queries (6900)                              16 /  32   15 /  26
//          32 (13800)                                     18 /  36   21 /  41
//         512                                             40 / 118  190 / 458
//   4 x 2, G = 16, 8 queries, pages of 32, d = 64 (6900)  12 /  17   10 /  10
//   4 x 4, 32 queries, 64 pages of 16, d = 64 (13800)     17 /  31   16 /  29
//         128                                             20 /  45   41 /  90
//   4 x 4, G = 1, 128 queries, 64 pages of 16, d = 64     36 /  54   19 /  56
//   16 x 2, 32 queries, 16 pages of 16, d = 32 (6900)     12 /  29   10 /  17
constexpr int kFullTileRows = 16, kFullPairsPerSm = 12288;

bool blocks_full_tiles(const attn_long_params* p, int sms) {
  if (p->full_tiles != 0) return p->full_tiles == 1;
  const int64_t rows = static_cast<int64_t>(p->Nq) * (p->Hq / p->Hk);
  const int64_t slots = static_cast<int64_t>(p->n < p->table_width ? p->n : p->table_width) * p->page_size;
  return rows >= kFullTileRows &&
         static_cast<double>(rows * p->B * p->Hk) * static_cast<double>(slots) >= static_cast<double>(kFullPairsPerSm) * sms;
}

int this_gpu(LongParams* r) {
  int dev = 0;
  const int rc = this_device(&dev, &r->sms);
  if (rc == ATTN_OK) long_used(dev);
  return rc;
}

// The scores' and weights' form for few rows, where it is asked for by name.
int check_few(const attn_long_params* p, bool fits) {
  if (p->full_tiles == 2 && !fits)
    return fail_with(ATTN_ERR_INVALID_ARG, "full_tiles 2: the form for few rows holds %d rows of a key head", attn::kFewRows);
  return ATTN_OK;
}

int done(cudaError_t e, const char* what) { return e == cudaSuccess ? ATTN_OK : cuda_error(e, what); }

}  // namespace

extern "C" {

void attn_long_params_init(attn_long_params* p) {
  if (p) std::memset(p, 0, sizeof(*p));
}

int attn_kv_bounds(const attn_long_params* p) {
  clear_error();
  LongParams r;
  int rc = fill(p, &r, false, true, true);
  if (rc != ATTN_OK || (rc = fill_cache(p, &r, true, false, kMapped)) != ATTN_OK || (rc = need(p->bounds, "bounds")) != ATTN_OK)
    return rc;
  if (!aligned(p->bounds, 16)) return fail_with(ATTN_ERR_MISALIGNED, "bounds must be 16-byte aligned");
  if (p->n_new < -1) return fail_with(ATTN_ERR_INVALID_ARG, "n_new must be >= 0, or -1 for all tokens");
  if ((rc = this_gpu(&r)) != ATTN_OK) return rc;
  return done(attn::launch_bounds(r, p->d, stream_of(p->stream)), "page bounds launch");
}

int attn_block_scores(const attn_long_params* p) {
  clear_error();
  LongParams r;
  int rc = fill(p, &r, true, true, true);
  if (rc != ATTN_OK || (rc = fill_queries(p, &r)) != ATTN_OK || (rc = check_scale(p, &r)) != ATTN_OK ||
      (rc = need(p->bounds, "bounds")) != ATTN_OK || (rc = need(p->scores, "scores")) != ATTN_OK ||
      (rc = check_few(p, attn::scores_few_rows(r))) != ATTN_OK)
    return rc;
  if (!aligned(p->bounds, 16)) return fail_with(ATTN_ERR_MISALIGNED, "bounds must be 16-byte aligned");
  if ((rc = this_gpu(&r)) != ATTN_OK) return rc;
  return done(attn::launch_scores(r, p->d, stream_of(p->stream)), "page scores launch");
}

int attn_block_select(const attn_long_params* p) {
  clear_error();
  LongParams r;
  int rc = fill(p, &r, true, false, false);
  if (rc != ATTN_OK || (rc = check_taken(p, "pages of a list")) != ATTN_OK || (rc = need(p->scores, "scores")) != ATTN_OK ||
      (rc = need(p->blocks, "blocks")) != ATTN_OK || (rc = this_gpu(&r)) != ATTN_OK)
    return rc;
  return done(attn::launch_select(r, stream_of(p->stream)), "page selection launch");
}

int attn_blocks(const attn_long_params* p) {
  clear_error();
  LongParams r;
  RopeTensor o;
  int rc = fill(p, &r, true, true, true);
  if (rc != ATTN_OK || (rc = fill_queries(p, &r)) != ATTN_OK || (rc = fill_cache(p, &r, true, true, kMapped)) != ATTN_OK ||
      (rc = check_scale(p, &r)) != ATTN_OK || (rc = need(p->blocks, "blocks")) != ATTN_OK ||
      (rc = tensor(p->o, p->o_stride, p->B, p->Hq, p->Nq, p->d, kWritten, "o", &o)) != ATTN_OK)
    return rc;
  if (p->n < 1 || static_cast<int64_t>(p->n) * p->Nq >= kMaxCount)
    return fail_with(ATTN_ERR_INVALID_ARG, "n must be >= 1, and n * Nq below 2^30");
  int dev = 0, sms = 0;
  if ((rc = this_device(&dev, &sms)) != ATTN_OK) return rc;
  r.o = o.p;
  r.o_sb = o.sb;
  r.o_sh = o.sh;
  r.o_sn = o.sn;
  if (blocks_full_tiles(p, sms)) {
    PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
    CUtensorMap tm_k, tm_v;
    const int64_t ks[3] = {r.kc_sp, r.kc_sh, r.kc_st}, vs[3] = {r.vc_sp, r.vc_sh, r.vc_st};
    if ((rc = tensor_map_encoder(&encode)) != ATTN_OK ||
        (rc = encode_pages(encode, &tm_k, r.kc, p->d, p->page_size, p->Hk, p->n_pages, attn::kBlocksBox, ks, "k_cache")) != ATTN_OK ||
        (rc = encode_pages(encode, &tm_v, r.vc, p->d, p->page_size, p->Hk, p->n_pages, attn::kBlocksBox, vs, "v_cache")) != ATTN_OK)
      return rc;
    r.splits = blocks_tile_splits(p, sms);
    long_used(dev);
    return done(attn::launch_blocks_tiles(r, tm_k, tm_v, p->d, stream_of(p->stream)), "attention over selected pages launch");
  }
  r.splits = blocks_splits(p, sms);
  return done(attn::launch_blocks(r, p->d, stream_of(p->stream)), "attention over selected pages launch");
}

int attn_kv_weights(const attn_long_params* p) {
  clear_error();
  LongParams r;
  int rc = fill(p, &r, true, true, true);
  if (rc != ATTN_OK || (rc = fill_queries(p, &r)) != ATTN_OK || (rc = fill_cache(p, &r, true, false, kRead)) != ATTN_OK ||
      (rc = check_scale(p, &r)) != ATTN_OK || (rc = need(p->lse, "lse")) != ATTN_OK ||
      (rc = need(p->weights_out, "weights_out")) != ATTN_OK || (rc = check_few(p, attn::weights_few_rows(r))) != ATTN_OK)
    return rc;
  if (!std::isfinite(p->decay) || p->decay < 0.f) return fail_with(ATTN_ERR_INVALID_ARG, "decay must be finite and >= 0");
  if (p->decay != 0.f && (rc = need(p->weights, "weights")) != ATTN_OK) return rc;
  // scale * log2(e) as an fp32 value below it and what that leaves: both positive, so
  // that a score of -inf stays -inf in the sum of its two products
  const double c = static_cast<double>(p->scale) * 1.4426950408889634074;
  r.c_hi = static_cast<float>(c);
  if (static_cast<double>(r.c_hi) >= c) r.c_hi = std::nextafter(r.c_hi, 0.f);
  r.c_lo = static_cast<float>(c - static_cast<double>(r.c_hi));
  if (!(p->scale >= 0x1p-64f && p->scale <= 0x1p64f) || !(r.c_lo > 0.f))
    return fail_with(ATTN_ERR_INVALID_ARG, "scale must be 2^-64 to 2^64");
  if ((rc = this_gpu(&r)) != ATTN_OK) return rc;
  return done(attn::launch_weights(r, p->d, stream_of(p->stream)), "received weights launch");
}

int attn_kv_evict(const attn_long_params* p) {
  clear_error();
  LongParams r;
  int rc = fill(p, &r, false, true, true);
  if (rc != ATTN_OK || (rc = fill_cache(p, &r, true, true, kWritten)) != ATTN_OK ||
      (rc = check_taken(p, "tokens to keep")) != ATTN_OK || (rc = need(p->weights, "weights")) != ATTN_OK ||
      (rc = need(p->kept, "kept")) != ATTN_OK || (rc = need(p->new_lens, "new_lens")) != ATTN_OK)
    return rc;
  if (!aligned(p->weights, 16)) return fail_with(ATTN_ERR_MISALIGNED, "weights must be 16-byte aligned");
  if (p->new_lens == p->kv_lens) return fail_with(ATTN_ERR_INVALID_ARG, "new_lens must not be kv_lens");
  if (static_cast<int64_t>(p->B) * p->Hk >= kMaxCount || static_cast<int64_t>(p->n) >= kMaxCount)
    return fail_with(ATTN_ERR_INVALID_ARG, "too many rows, or n too large");
  if (p->dst_table != nullptr) {
    const int64_t most = r.n < r.max_len ? r.n : r.max_len;
    if (p->dst_width < 1 || p->dst_stride < 0 || (p->B > 1 && p->dst_stride < p->dst_width))
      return fail_with(ATTN_ERR_INVALID_ARG, "dst_width must be >= 1 and dst_stride no smaller");
    if (static_cast<int64_t>(p->dst_width) * p->page_size < most && p->dst_width < p->table_width)
      return fail_with(ATTN_ERR_INVALID_ARG, "dst_table holds fewer tokens than may be kept");
    r.dst = p->dst_table;
    r.dst_sb = p->dst_stride;
    r.dst_width = p->dst_width;
  }
  r.weights_out = p->weights;
  if ((rc = this_gpu(&r)) != ATTN_OK) return rc;
  return done(attn::launch_evict(r, p->d, stream_of(p->stream)), "eviction launch");
}

}  // extern "C"
