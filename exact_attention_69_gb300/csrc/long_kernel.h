// long_kernel.h -- parameters and launchers of the long-cache operators: page bounds
// and scores (block_scores.cu), page selection and eviction (block_select.cu),
// attention over selected pages (attn_blocks.cu), received weights (kv_weights.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "paged_kernel.h"

namespace attn {

struct LongParams {
  const void* q;                // bf16 [B, Hq, Nq, d], element strides of b, h, n
  int64_t q_sb, q_sh, q_sn;
  void* kc;                     // bf16 pages, element strides of page, head, slot
  int64_t kc_sp, kc_sh, kc_st;
  void* vc;
  int64_t vc_sp, vc_sh, vc_st;
  void* bounds;                 // bf16 [n_pages, Hk, 2, d]
  const int32_t* table;         // [B, table_width]
  int64_t table_sb;
  int table_width;
  const int32_t* dst;           // eviction's destination pages [B, dst_width], or nullptr: in place
  int64_t dst_sb;
  int dst_width;
  const int32_t* kv_lens;       // [B]
  const int32_t* q_lens;        // [B] or nullptr (Nq each)
  void* o;
  int64_t o_sb, o_sh, o_sn;
  float* lse;                   // fp32 [B, Hq, Nq]
  float* scores;                // fp32 [B, Hk, Nq, table_width]
  int32_t* blocks;              // [B, Hk, Nq, n]
  const float* weights;         // fp32 [n_pages, Hk, page_size]
  float* weights_out;
  int32_t* kept;                // [B, Hk, n]
  int32_t* new_lens;            // [B]
  int B, Hq, Hk, Nq, G;
  FastDiv by_g;
  int n_pages, page_shift;
  int max_len;                  // table_width * page size
  int n, first, last;           // selected pages or kept slots, those always taken at either end
  int n_new;                    // kv_bounds: newest tokens of each sequence; < 0: all are new
  int causal;
  float scale;                  // of the scores
  float c_hi, c_lo;             // scale * log2(e), the fp32 value and what it leaves
  float decay;
  int full_tiles;               // 0: by the rule, 1: tiles of 128 rows, 2: the form for few rows
  uint64_t timeout_ns;          // tiles of 128 rows: bound on every wait
  int inject;                   // 1: withhold something once (tests the bounded wait); -1: attn_blocks, values come late
  int splits;                   // CTAs (a cluster) that share a row tile's pages
  int sms;                      // the device's (scores and weights: how finely work is cut)
};

// Keys that query n of a sequence with `len` cached tokens and `ql` queries sees.
#ifdef __CUDACC__
struct LongLens {
  int len, ql;
};
__device__ __forceinline__ LongLens long_lens(const LongParams& p, int b) {
  LongLens s;
  s.len = min(max(p.kv_lens[b], 0), p.max_len);
  s.ql = p.q_lens != nullptr ? min(max(p.q_lens[b], 0), p.Nq) : p.Nq;
  return s;
}
__device__ __forceinline__ int long_seen(const LongParams& p, LongLens s, int n) {
  if (n >= s.ql) return 0;
  return p.causal ? min(max(s.len - s.ql + n + 1, 0), s.len) : s.len;
}
__device__ __forceinline__ int long_pages(const LongParams& p, int tokens) {
  return (tokens + (1 << p.page_shift) - 1) >> p.page_shift;
}
#endif

cudaError_t launch_bounds(const LongParams& p, int d, cudaStream_t s);
cudaError_t launch_scores(const LongParams& p, int d, cudaStream_t s);
cudaError_t launch_select(const LongParams& p, cudaStream_t s);
cudaError_t launch_evict(const LongParams& p, int d, cudaStream_t s);
cudaError_t launch_blocks(const LongParams& p, int d, cudaStream_t s);
cudaError_t launch_weights(const LongParams& p, int d, cudaStream_t s);
// The same for many query rows (long_tiles.cu).
cudaError_t launch_scores_tiles(const LongParams& p, int d, cudaStream_t s);
cudaError_t launch_weights_tiles(const LongParams& p, int d, cudaStream_t s);
// Maps of the caches: boxes of min(page size, kBlocksBox) slots.
cudaError_t launch_blocks_tiles(const LongParams& p, const CUtensorMap& tm_k, const CUtensorMap& tm_v, int d, cudaStream_t s);
constexpr int kBlocksBox = 64;
// Reads and clears the current device's status word of these.
cudaError_t long_take_status(uint32_t word[4]);

// attn_blocks: rows of a tile (a group of 8 columns of the products, or two).
__host__ __device__ constexpr int blocks_tile_rows(int64_t rows) { return rows <= 8 ? 8 : 16; }
// Warps of a CTA, each with keys of its own: two CTAs share a SM's registers.
__host__ __device__ constexpr int blocks_warps(int groups) { return groups == 1 ? 6 : 4; }
constexpr int kBlocksMaxSplits = 8;   // CTAs of a cluster on any GPU

// Rows of a sequence and key head that the scores' and weights' forms for few rows hold (shared memory).
// Up to there they are the faster ones (us, 8, 16 and 32 rows, and the tiles for any of them): 32
// sequences x 8 key heads, d = 128, 16384 tokens, pages of 64: scores 6.4, 8.8, 10.4 and 10.7, weights 160,
// 170, 181 and 380; 4 x 8: 2.7, 2.9, 3.8 and 4.7, 23, 27, 32 and 52.
constexpr int kFewRows = 32;
// Query heads of a key head as the scores' form for few rows pads them, so that groups of 8
// columns hold whole tokens or a token whole groups: 1, 2, 4 or a multiple of 8.
__host__ __device__ constexpr int padded_heads(int g) { return g <= 2 ? g : (g <= 4 ? 4 : (g + 7) / 8 * 8); }
inline bool scores_few_rows(const LongParams& p) { return static_cast<int64_t>(p.Nq) * padded_heads(p.G) <= kFewRows; }
inline bool weights_few_rows(const LongParams& p) { return static_cast<int64_t>(p.Nq) * p.G <= kFewRows; }

}  // namespace attn
