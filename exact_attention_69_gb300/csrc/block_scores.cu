// block_scores.cu -- bounds of a page's keys and the score that they allow.
//
// Bounds: lower_c = min_j k_jc and upper_c = max_j k_jc over the page's live slots,
// exact in bf16. A key between them has q . k <= sum_c max(q_c lower_c, q_c upper_c)
// = min(q, 0) . lower + max(q, 0) . upper: one product of length 2 d with both halves
// exact in bf16. A page's score for a query token is the largest such bound over the
// query heads that share the key head. Sums are the matrix instruction's, in fp32.
//
// Few rows are bound by memory, 4 d bytes of bounds a page and key head: 32 sequences of
// 2048 to 32768 tokens in pages of 64, 8 key heads, d = 128 (27 MB) take 8.1 us, 3.4 TB/s:
// a block's chain (table, bounds, product, store) is long for what it reads. The bounds of the
// newest token's pages take 3.8 us, one block's chain.
#include "long_dev.cuh"
#include "long_kernel.h"

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

constexpr int kScoreWarps = 4, kScorePages = 16 * kScoreWarps;

// Few rows (up to 32, all in shared memory): a warp takes the bounds of 16 pages into
// registers and goes over the rows 8 at a time. Columns of a product are rows n * Gp + g
// (Gp padded heads, GP if that is 1 to 8, else 0), so the largest of a token's heads is
// found among a lane's two columns and its neighbours'. Grid: pages, key head, sequence.
template <int D, int GP>
__global__ void __launch_bounds__(32 * kScoreWarps) scores_kernel(const __grid_constant__ LongParams p) {
  constexpr int kC = D / 32;  // 16-byte chunks that a lane takes of a vector of d channels
  __shared__ __align__(16) unsigned char qs[kFewRows * row_bytes<D>()];
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, i = lane >> 2, j = lane & 3;
  const int b = blockIdx.z, hk = blockIdx.y;
  const int page0 = static_cast<int>(blockIdx.x) * kScorePages + warp * 16;
  const int Gp = GP > 0 ? GP : padded_heads(p.G);
  const int rows = p.Nq * Gp;
  const int ids[2] = {page0 + i < p.table_width ? p.table[b * p.table_sb + page0 + i] : -1,
                      page0 + i + 8 < p.table_width ? p.table[b * p.table_sb + page0 + i + 8] : -1};
  // padded heads are zeros
  for (int x = threadIdx.x; x < rows * (D / 8); x += 32 * kScoreWarps) {
    const int r = x / (D / 8), c = x % (D / 8), tok = r / Gp, g = r % Gp;
    copy16(smem_addr(qs + r * row_bytes<D>() + c * 16),
           static_cast<const __nv_bfloat16*>(p.q) + b * p.q_sb +
               (static_cast<int64_t>(hk) * p.G + min(g, p.G - 1)) * p.q_sh + tok * p.q_sn + c * 8,
           g < p.G ? 16 : 0);
  }
  copy_commit();
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
  copy_wait();
  __syncthreads();
  float* out = p.scores + (static_cast<int64_t>(b) * p.Hk + hk) * p.Nq * p.table_width + page0 + i;
  const bool in[2] = {page0 + i < p.table_width, page0 + i + 8 < p.table_width};
  const auto put = [&](int tok, const float (&v)[2]) {
    if (tok >= p.Nq) return;
    const int most = long_pages(p, long_seen(p, lens, tok)) - page0 - i;
    float* at = out + static_cast<int64_t>(tok) * p.table_width;
    if (in[0]) at[0] = most > 0 ? v[0] * p.scale : -INFINITY;
    if (in[1]) at[8] = most > 8 ? v[1] * p.scale : -INFINITY;
  };
  const auto top = [](float a, float x) { return a > x || a != a ? a : x; };  // (NaN stays: fmax would drop it)

  float best[2] = {-INFINITY, -INFINITY};  // GP 0: of a token that has several groups of columns
#pragma unroll 1
  for (int r0 = 0; r0 < rows; r0 += 8) {
    float acc[2][4] = {};  // (two sums, of the lower and of the upper bounds' products: shorter chains)
    if (page0 < pages) {
      const unsigned char* row = qs + (r0 + i) * row_bytes<D>() + j * 16;
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
        mma(acc[0], lo[0][c].x, lo[1][c].x, lo[0][c].y, lo[1][c].y, neg.x, neg.y);
        mma(acc[1], hi[0][c].x, hi[1][c].x, hi[0][c].y, hi[1][c].y, pos.x, pos.y);
        mma(acc[0], lo[0][c].z, lo[1][c].z, lo[0][c].w, lo[1][c].w, neg.z, neg.w);
        mma(acc[1], hi[0][c].z, hi[1][c].z, hi[0][c].w, hi[1][c].w, pos.z, pos.w);
      }
    }
    // columns 2 j and 2 j + 1 are rows r and r + 1
    const int r = r0 + 2 * j;
    if constexpr (GP == 1) {
      const float v[2] = {acc[0][0] + acc[1][0], acc[0][2] + acc[1][2]}, w[2] = {acc[0][1] + acc[1][1], acc[0][3] + acc[1][3]};
      put(r, v);
      put(r + 1, w);
    } else {
      float v[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int g = r % Gp;
        v[h] = top(g < p.G ? acc[0][2 * h] + acc[1][2 * h] : -INFINITY,
                   g + 1 < p.G ? acc[0][2 * h + 1] + acc[1][2 * h + 1] : -INFINITY);
        if constexpr (GP != 2) v[h] = top(v[h], __shfl_xor_sync(0xffffffffu, v[h], 1));
        if constexpr (GP == 8 || GP == 0) v[h] = top(v[h], __shfl_xor_sync(0xffffffffu, v[h], 2));
      }
      if constexpr (GP > 0) {
        if (r % GP == 0) put(r / GP, v);
      } else {
        best[0] = top(best[0], v[0]);
        best[1] = top(best[1], v[1]);
        if ((r0 + 8) % Gp == 0) {
          if (j == 0) put(r0 / Gp, best);
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

template <int D>
cudaError_t scores_dim(const LongParams& p, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>((p.table_width + kScorePages - 1) / kScorePages), p.Hk, p.B);
  const int threads = 32 * kScoreWarps;
  switch (padded_heads(p.G)) {
    case 1: return launch(scores_kernel<D, 1>, grid, threads, 0, s, 1, p);
    case 2: return launch(scores_kernel<D, 2>, grid, threads, 0, s, 1, p);
    case 4: return launch(scores_kernel<D, 4>, grid, threads, 0, s, 1, p);
    case 8: return launch(scores_kernel<D, 8>, grid, threads, 0, s, 1, p);
    default: return launch(scores_kernel<D, 0>, grid, threads, 0, s, 1, p);
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
  if (p.full_tiles == 1 || !scores_few_rows(p)) return launch_scores_tiles(p, d, s);
  switch (d) {
    case 32: return scores_dim<32>(p, s);
    case 64: return scores_dim<64>(p, s);
    case 128: return scores_dim<128>(p, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace attn
