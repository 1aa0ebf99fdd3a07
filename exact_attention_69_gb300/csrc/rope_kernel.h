// rope_kernel.h -- parameters shared by the host entry points and the kernels
// of the per-head norm with rotary position embedding and of the cache append.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace attn {

// One tensor [B, H, N, d] bf16: base and element strides of b, h, n.
struct RopeTensor {
  void* p;
  int64_t sb, sh, sn;
};

struct RopeParams {
  RopeTensor q, k, v;         // inputs (p == nullptr: absent)
  RopeTensor qo, ko;          // outputs; ko unused when the keys go to the cache
  int B, N, Hq, Hk;           // Hq 0: no queries
  int rot, interleaved;       // rotated channels of each head; pairs (2i, 2i+1) or (i, i + rot/2)
  int norm;                   // root-mean-square norm before the rotation
  float eps;
  const void* wq;             // weights [d] or nullptr (ones); type 0 bf16, 1 fp32
  const void* wk;
  int wq_type, wk_type;
  const double* inv_freq;     // [rot / 2] radians per position
  const void* pos;            // positions [B, N] (strides) or nullptr
  int pos_type;               // 1 int32, 2 int64
  int64_t pos_sb, pos_sn;
  int64_t pos_offset;         // without `pos`: position of token n is pos_offset (+ starts[b]) + n
  // cache append
  int cache;                  // 1: keys and values go to their pages
  void* kc;
  void* vc;
  int64_t kc_sp, kc_sh, kc_st;  // element strides of page, head, slot
  int64_t vc_sp, vc_sh, vc_st;
  int n_pages, page_shift;
  const int32_t* table;
  int64_t table_sb;
  int table_width;
  const int32_t* starts;
  const int32_t* counts;      // nullptr: every token is real
  int heads_per_block;        // virtual heads (queries, keys, values in turn) per block row
};

struct RopeBwdParams {
  RopeTensor q, k, dyq, dyk, dq, dk;
  int B, N, Hq, Hk, rot, interleaved, norm;
  float eps;
  const void* wq;
  const void* wk;
  int wq_type, wk_type;
  const double* inv_freq;
  const void* pos;
  int pos_type;
  int64_t pos_sb, pos_sn, pos_offset;
  void* dwq;                  // gradients of the weights, of the weights' types (nullptr: not wanted)
  void* dwk;
  float* part;                // [blocks][2][d] partial sums of the weights' gradients
  int blocks;
};

cudaError_t launch_rope(const RopeParams& p, int d, dim3 grid, cudaStream_t s);
cudaError_t launch_rope_bwd(const RopeBwdParams& p, int d, cudaStream_t s);
// Tokens that a block of the forward (and of the backward's loop) takes at a time.
constexpr int kRopeThreads = 256;
__host__ __device__ constexpr int rope_tokens_per_block(int d) { return kRopeThreads / (d / 8); }

}  // namespace attn
