// paged_kernel.h -- parameters of the paged attention kernels (attn_paged.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace attn {

// Rows of a task are numbered r = n * G + g inside one sequence (G query heads
// share a key head) and b * Nq * G + n * G + g over the batch for the prefix.
constexpr int kPagedTaskRows = 256;  // two 128-row query tiles
// Work is dealt out in units of a quarter of a K/V tile of one query tile. A tile
// for two query tiles, where the softmax and not memory sets the pace, takes a
// little longer (with 4 / 5 / 6 units 96 sequences behind 32768 tokens take 135.8 /
// 119.8 / 119.3 us, 3 x 512 tokens x 16 heads behind 2048 38.9 / 38.2 / 38.1 us); a
// task's start and end as long as a tile (2 / 4 / 6 units: 32 sequences behind 4096
// tokens 30.1 / 26.7 / 27.4 us, 16 of up to 4096 own keys at d = 32 12.9 / 10.8 / 11.3
// us), that of two query tiles longer (4 / 8 / 16 units: 64 sequences of 4 rows x 8 key
// heads and 256 own keys behind 512 tokens 33.9 / 29.9 / 29.0 us, the 3 x 512 tokens
// 39.8 / 39.0 / 38.2 us).
constexpr int kPagedTile = 4, kPagedPairTile = 5, kPagedTaskCost = 4, kPagedPairTaskCost = 16;
// Least work that opens another CTA; no less than a tile. (5 / 8 / 16 / 24: 4 sequences
// behind 512 tokens 10.6 / 10.1 / 12.6 / 14.3 us, 7 x 5 tokens behind 1021 12.2 / 11.9 /
// 15.8 / 16.6 us; larger calls have a CTA an SM anyway.)
constexpr int kPagedMinUnits = 8;

// Division of n < 2^31 by a divisor that the host knows: n * mul >> (32 + shift)
// with mul = ceil(2^(32 + shift) / d), shift = ceil(log2 d) - 1 (the error term
// n * (mul * d - 2^(32 + shift)) stays below 2^(32 + shift)); d = 1 is kept apart.
struct FastDiv {
  uint32_t d, mul, shift;
#ifdef __CUDACC__
  __host__ __device__ FastDiv() : d(1), mul(0), shift(0) {}
  __host__ explicit FastDiv(uint32_t div) : d(div), mul(0), shift(0) {
    if (div <= 1) return;
    while ((uint64_t{2} << shift) < div) ++shift;
    mul = static_cast<uint32_t>(((uint64_t{1} << (32 + shift)) + div - 1) / div);
  }
  __device__ __forceinline__ int div(int n) const {
    return d == 1 ? n : static_cast<int>(__umulhi(static_cast<uint32_t>(n), mul) >> shift);
  }
#endif
};

// Rows of a buffer half, whole groups of 32.
__host__ __device__ constexpr int paged_rows32(int rows) { return (rows + 31) & ~31; }

struct PagedParams {
  CUtensorMap tm_k;             // 4-D (d, slot, head, page) bf16 maps, box (swizzle span, min(page, 128), 1, 1)
  CUtensorMap tm_v;
  CUtensorMap tm_q;             // 4-D (d, head, query, sequence); see q_map
  const void* q;                // bf16, element strides of b, h, n
  int64_t q_sb, q_sh, q_sn;
  void* o;
  int64_t o_sb, o_sh, o_sn;
  float* lse;                   // fp32 [B, Hq, Nq] or nullptr
  const int32_t* table;         // [B, table_width] pages of each sequence
  int64_t table_sb;
  const int32_t* kv_lens;       // [B]
  const int32_t* q_lens;        // [B] or nullptr (Nq each)
  const int32_t* prefix_table;  // pages of the shared prefix
  int B, Hq, Hk, Nq, G;
  int prefix_len;
  int page_shift;
  int max_len;                  // table_width * page size: longest own length that the table holds
  FastDiv by_g, by_rows;        // by G; by Nq * G, the rows of a sequence
  FastDiv by_batch_rows;        // by B * Nq * G, the rows of a key head
  FastDiv by_prefix_task;       // by the units of a prefix task of two query tiles
  FastDiv by_prefix_head;       // by the units of the prefix tasks of a key head
  int prefix_tiles;             // K/V tiles of the prefix
  int prefix_tasks, prefix_units;  // batched prefix: tasks of a key head; units of all. 0: each
                                // sequence's tasks go over the prefix's tiles themselves
  int own_tasks;                // tasks of a sequence for one key head
  int q_map;                    // what a box of tm_q holds: 0 nothing (gather), 1 rows of several
                                // sequences (prefix tasks), 2 rows of one
  int row_limits;               // rows of a sequence may see different numbers of keys
  int causal;                   // bottom-right causal over prefix and own keys together
  float c;                      // scale * log2(e)
  // workspace
  int2* tasks;                  // [B * Hk * own_tasks | Hk * prefix_tasks]: first CTA and parts of each
  float* slots;                 // per CTA 2 x 2 query tiles x 128 rows x (d + 2): parts of cut tasks
  float* rows_o;                // [2][paged_rows32(B * Nq * Hq)][d]: uncut prefix and own results
  float2* rows_ml;              // [2][paged_rows32(B * Nq * Hq)]: their running maximum (log2 units) and sum
  enum { kJoinMany, kJoinFew, kJoinSplit };
  int join;                     // the join's form: see the rule's comment in cache_host.cu
  int grid;                     // CTAs of the attention kernel
  uint64_t timeout_ns;
  int inject;
};

// The attention kernel, then the one that joins the parts.
cudaError_t launch_paged(const PagedParams& p, int d, cudaStream_t s);
// Reads and clears the current device's status word of the paged kernels.
cudaError_t paged_take_status(uint32_t word[4]);

}  // namespace attn
