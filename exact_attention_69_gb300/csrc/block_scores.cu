// block_scores.cu -- bounds of a page's keys and the score that they allow.
//
// Bounds: lower_c = min_j k_jc and upper_c = max_j k_jc over the page's live slots,
// exact in bf16. A key between them has q . k <= sum_c max(q_c lower_c, q_c upper_c)
// = min(q, 0) . lower + max(q, 0) . upper: one product of length 2 d with both halves
// exact in bf16. A page's score for a query token is the largest such bound over the
// query heads that share the key head.
#include "long_dev.cuh"
#include "long_kernel.h"
#ifndef TILE_ROWS
#define TILE_ROWS 33
#endif

namespace attn {
namespace {

using namespace ldev;

// ------------------------------------------------------------------ bounds

constexpr int kBoundsThreads = 128;

// A block per page (x: of the pages that hold new tokens), key head and sequence. D / 8
// threads take a slot's channels 16 bytes at a time; minima and maxima of the slots are
// then joined through shared memory.
template <int D>
__global__ void __launch_bounds__(kBoundsThreads) bounds_kernel(const __grid_constant__ LongParams p) {
  constexpr int kCols = D / 8, kRows = kBoundsThreads / kCols;
  __shared__ uint4 part[2][kRows][kCols];
  grid_dep_wait();
  grid_dep_launch();
  const int b = blockIdx.z, hk = blockIdx.y;
  const int len = min(max(p.kv_lens[b], 0), p.max_len);
  const int from = p.n_new < 0 ? 0 : max(len - p.n_new, 0) >> p.page_shift;
  const int page = from + static_cast<int>(blockIdx.x);
  const int slots = min(len - (page << p.page_shift), 1 << p.page_shift);
  if (page >= p.table_width || slots <= 0) return;
  const int id = p.table[b * p.table_sb + page];
  if (id < 0 || id >= p.n_pages) return;
  const int col = threadIdx.x % kCols, row = threadIdx.x / kCols;
  const __nv_bfloat16* k = static_cast<const __nv_bfloat16*>(p.kc) + id * p.kc_sp + hk * p.kc_sh + col * 8;
  __nv_bfloat162 lo[4], hi[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    lo[i] = __nv_bfloat162(__ushort_as_bfloat16(0x7F80), __ushort_as_bfloat16(0x7F80));
    hi[i] = __nv_bfloat162(__ushort_as_bfloat16(0xFF80), __ushort_as_bfloat16(0xFF80));
  }
#pragma unroll 4
  for (int t = row; t < slots; t += kRows) {
    const uint4 v = ld16(k + t * p.kc_st);
    const __nv_bfloat162* x = reinterpret_cast<const __nv_bfloat162*>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      lo[i] = __hmin2_nan(lo[i], x[i]);
      hi[i] = __hmax2_nan(hi[i], x[i]);
    }
  }
  part[0][row][col] = *reinterpret_cast<uint4*>(lo);
  part[1][row][col] = *reinterpret_cast<uint4*>(hi);
  __syncthreads();
  if (threadIdx.x >= 2 * kCols) return;
  const int side = threadIdx.x / kCols;
  __nv_bfloat162 z[4];
  *reinterpret_cast<uint4*>(z) = part[side][0][col];
  for (int r = 1; r < kRows; ++r) {
    const uint4 v = part[side][r][col];
    const __nv_bfloat162* x = reinterpret_cast<const __nv_bfloat162*>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i) z[i] = side ? __hmax2_nan(z[i], x[i]) : __hmin2_nan(z[i], x[i]);
  }
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.bounds) + ((static_cast<int64_t>(id) * p.Hk + hk) * 2 + side) * D;
  *reinterpret_cast<uint4*>(out + col * 8) = *reinterpret_cast<uint4*>(z);
}

// ------------------------------------------------------------------ scores

constexpr int kScoreWarps = 4, kScorePages = 16 * kScoreWarps, kScoreRows = 64;

// Query heads of a key head, padded so that groups of 8 columns hold whole tokens or a
// token whole groups: 1, 2, 4 or a multiple of 8.
__host__ __device__ constexpr int padded_heads(int g) {
  return g <= 2 ? g : (g <= 4 ? 4 : (g + 7) / 8 * 8);
}

// A warp keeps the bounds of 16 pages in registers and goes over the block's query
// rows 8 at a time; these come into shared memory 64 at a time, the next ones while
// these are used. Columns of a product are rows n * Gp + g (Gp padded heads, GP if that
// is 1 to 8, else 0), so the largest of a token's heads is found among a lane's two
// columns and its neighbours'. Grid: pages x runs of `tokens` tokens, key head, sequence.
template <int D, int GP>
__global__ void __launch_bounds__(32 * kScoreWarps) scores_kernel(const __grid_constant__ LongParams p, int tokens) {
  constexpr int kC = D / 32;  // 16-byte chunks that a lane takes of a vector of d channels
  __shared__ __align__(16) unsigned char qs[2][kScoreRows * row_bytes<D>()];
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, i = lane >> 2, j = lane & 3;
  const int b = blockIdx.z, hk = blockIdx.y;
  const int runs = (p.Nq + tokens - 1) / tokens;
  const int run = blockIdx.x % runs, page0 = (blockIdx.x / runs) * kScorePages + warp * 16;
  const int Gp = GP > 0 ? GP : padded_heads(p.G);
  const int tok0 = run * tokens, tok1 = min(tok0 + tokens, p.Nq);
  const int rows = (tok1 - tok0) * Gp;
  const int ids[2] = {page0 + i < p.table_width ? p.table[b * p.table_sb + page0 + i] : -1,
                      page0 + i + 8 < p.table_width ? p.table[b * p.table_sb + page0 + i + 8] : -1};
  const LongLens lens = long_lens(p, b);
  const int pages = long_pages(p, lens.len);

  uint4 lo[2][kC], hi[2][kC];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const bool real = page0 + i + 8 * h < pages && ids[h] >= 0 && ids[h] < p.n_pages;
    const __nv_bfloat16* v =
        static_cast<const __nv_bfloat16*>(p.bounds) + (static_cast<int64_t>(ids[h]) * p.Hk + hk) * 2 * D + j * 8;
#pragma unroll
    for (int c = 0; c < kC; ++c) {
      lo[h][c] = real ? ld16(v + c * 32) : make_uint4(0, 0, 0, 0);
      hi[h][c] = real ? ld16(v + D + c * 32) : make_uint4(0, 0, 0, 0);
    }
  }
  // rows [base, base + 64) into a buffer; padded heads are zeros
  const auto fetch = [&](int base, int buf) {
    for (int x = threadIdx.x; x < min(kScoreRows, rows - base) * (D / 8); x += 32 * kScoreWarps) {
      const int r = x / (D / 8), c = x % (D / 8), tok = tok0 + (base + r) / Gp, g = (base + r) % Gp;
      const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q) + b * p.q_sb +
                               (static_cast<int64_t>(hk) * p.G + min(g, p.G - 1)) * p.q_sh + tok * p.q_sn + c * 8;
      copy16(smem_addr(qs[buf] + r * row_bytes<D>() + c * 16), q, g < p.G ? 16 : 0);
    }
    copy_commit();
  };
  float* out = p.scores + ((static_cast<int64_t>(b) * p.Hk + hk) * p.Nq + tok0) * p.table_width + page0 + i;
  const bool in[2] = {page0 + i < p.table_width, page0 + i + 8 < p.table_width};
  const auto put = [&](int tok, const float (&v)[2]) {  // counted from tok0
    if (tok >= tok1 - tok0) return;
    const int most = long_pages(p, long_seen(p, lens, tok0 + tok)) - page0 - i;
    float* at = out + static_cast<int64_t>(tok) * p.table_width;
    if (in[0]) at[0] = most > 0 ? v[0] * p.scale : -INFINITY;
    if (in[1]) at[8] = most > 8 ? v[1] * p.scale : -INFINITY;
  };
  const auto top = [](float a, float x) { return a > x || a != a ? a : x; };  // (NaN stays: fmax would drop it)

  float best[2] = {-INFINITY, -INFINITY};  // GP 0: of a token that has several groups of columns
  fetch(0, 0);
  for (int base = 0, buf = 0; base < rows; base += kScoreRows, buf ^= 1) {
    copy_wait();
    __syncthreads();
    if (base + kScoreRows < rows) fetch(base + kScoreRows, buf ^ 1);
#pragma unroll 2
    for (int r0 = 0; r0 < min(kScoreRows, rows - base); r0 += 8) {
      float acc[4] = {0.f, 0.f, 0.f, 0.f};
      if (page0 < pages) {
        const unsigned char* row = qs[buf] + (r0 + i) * row_bytes<D>() + j * 16;
#pragma unroll
        for (int c = 0; c < kC; ++c) {
          uint4 v = *reinterpret_cast<const uint4*>(row + c * 64), neg, pos;
          const __nv_bfloat162 zero(__ushort_as_bfloat16(0), __ushort_as_bfloat16(0));
          const __nv_bfloat162* x = reinterpret_cast<const __nv_bfloat162*>(&v);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            reinterpret_cast<__nv_bfloat162*>(&neg)[e] = __hmin2_nan(x[e], zero);
            reinterpret_cast<__nv_bfloat162*>(&pos)[e] = __hmax2_nan(x[e], zero);
          }
          mma(acc, lo[0][c].x, lo[1][c].x, lo[0][c].y, lo[1][c].y, neg.x, neg.y);
          mma(acc, lo[0][c].z, lo[1][c].z, lo[0][c].w, lo[1][c].w, neg.z, neg.w);
          mma(acc, hi[0][c].x, hi[1][c].x, hi[0][c].y, hi[1][c].y, pos.x, pos.y);
          mma(acc, hi[0][c].z, hi[1][c].z, hi[0][c].w, hi[1][c].w, pos.z, pos.w);
        }
      }
      // columns 2 j and 2 j + 1 are rows r and r + 1
      const int r = base + r0 + 2 * j;
      if constexpr (GP == 1) {
        const float a[2] = {acc[0], acc[2]}, z[2] = {acc[1], acc[3]};
        put(r, a);
        put(r + 1, z);
        continue;
      }
      float v[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int g = r % Gp;
        v[h] = top(g < p.G ? acc[2 * h] : -INFINITY, g + 1 < p.G ? acc[2 * h + 1] : -INFINITY);
        if constexpr (GP != 2) v[h] = top(v[h], __shfl_xor_sync(0xffffffffu, v[h], 1));
        if constexpr (GP == 8 || GP == 0) v[h] = top(v[h], __shfl_xor_sync(0xffffffffu, v[h], 2));
      }
      if constexpr (GP > 0) {
        if (r % GP == 0) put(r / GP, v);
      } else {
        best[0] = top(best[0], v[0]);
        best[1] = top(best[1], v[1]);
        if ((base + r0 + 8) % Gp == 0) {
          if (j == 0) put((base + r0) / Gp, best);
          best[0] = best[1] = -INFINITY;
        }
      }
    }
  }
}

template <int D>
cudaError_t bounds_dim(const LongParams& p, cudaStream_t s) {
  const int page = 1 << p.page_shift;
  int64_t x = p.table_width;
  if (p.n_new >= 0) {
    const int64_t most = (static_cast<int64_t>(p.n_new) + page - 2) / page + 1;  // pages that n_new tokens can touch
    if (p.n_new == 0) return cudaSuccess;
    if (most < x) x = most;
  }
  return launch(bounds_kernel<D>, dim3(static_cast<unsigned>(x), p.Hk, p.B), kBoundsThreads, 0, s, 1, p);
}

// Tokens of a block: enough rows to be worth the pages' bounds (up to kScoreMost), few
// enough for kScoreBlocks blocks.
constexpr int kScoreMost = 1024, kScoreBlocks = 4 * 152;

template <int D>
cudaError_t scores_dim(const LongParams& p, cudaStream_t s) {
  const int Gp = padded_heads(p.G);
  const int64_t cols = (p.table_width + kScorePages - 1) / kScorePages;
  int64_t rows = cols * p.B * p.Hk * p.Nq * Gp / kScoreBlocks;
  rows = rows < kScoreRows ? kScoreRows : (rows > kScoreMost ? kScoreMost : rows / kScoreRows * kScoreRows);
  const int tokens = static_cast<int>(rows / Gp < 1 ? 1 : (rows / Gp < p.Nq ? rows / Gp : p.Nq));
  const int64_t x = cols * ((p.Nq + tokens - 1) / tokens);
  const dim3 grid(static_cast<unsigned>(x), p.Hk, p.B);
  const int threads = 32 * kScoreWarps;
  switch (Gp) {
    case 1: return launch(scores_kernel<D, 1>, grid, threads, 0, s, 1, p, tokens);
    case 2: return launch(scores_kernel<D, 2>, grid, threads, 0, s, 1, p, tokens);
    case 4: return launch(scores_kernel<D, 4>, grid, threads, 0, s, 1, p, tokens);
    case 8: return launch(scores_kernel<D, 8>, grid, threads, 0, s, 1, p, tokens);
    default: return launch(scores_kernel<D, 0>, grid, threads, 0, s, 1, p, tokens);
  }
}

}  // namespace

cudaError_t launch_bounds(const LongParams& p, int d, cudaStream_t s) {
  switch (d) {
    case 32: return bounds_dim<32>(p, s);
    case 64: return bounds_dim<64>(p, s);
    case 128: return bounds_dim<128>(p, s);
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t launch_scores(const LongParams& p, int d, cudaStream_t s) {
  if (static_cast<int64_t>(p.Nq) * p.G >= TILE_ROWS) return launch_scores_tiles(p, d, s);
  switch (d) {
    case 32: return scores_dim<32>(p, s);
    case 64: return scores_dim<64>(p, s);
    case 128: return scores_dim<128>(p, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace attn
