// kv_weights.cu -- the attention weight that cached tokens receive: for each slot the
// sum over queries and the query heads of its key head of exp(scale q . k - lse), with
// the log-sum-exp that the attention returned.
//
// A weight's relative error is its exponent's absolute one, so the factor scale *
// log2(e) and each lse * log2(e) go in as an fp32 value and what that leaves: s * c_hi -
// lse_hi is one fused operation, exact up to the rounding of a difference that is small
// where the weight is not.
#include "long_dev.cuh"
#include "long_kernel.h"
#ifndef TILE_ROWS
#define TILE_ROWS 33
#endif

namespace attn {
namespace {

using namespace ldev;

constexpr int kWeightWarps = 4, kWarpKeys = 32, kWeightKeys = kWarpKeys * kWeightWarps, kWeightRows = 64;

// A warp keeps 32 keys in registers and goes over the query rows 8 at a time; these come
// into shared memory 64 at a time, the next ones while these are used. A lane's sums are
// over rows 2 j and 2 j + 1 of each group, for keys i, i + 8, i + 16 and i + 24. Grid: key
// groups, key head, sequence.
template <int D>
__global__ void __launch_bounds__(32 * kWeightWarps) weights_kernel(const __grid_constant__ LongParams p) {
  constexpr int kC = D / 32, kM = kWarpKeys / 16;
  struct Rows {
    unsigned char q[kWeightRows * row_bytes<D>()];
    float hi[kWeightRows], lo[kWeightRows];  // -lse * log2(e) in two parts
    int sees[kWeightRows];                   // slots that the row sees
  };
  __shared__ __align__(16) Rows rows_[2];
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, i = lane >> 2, j = lane & 3;
  const int b = blockIdx.z, hk = blockIdx.y;
  const LongLens lens = long_lens(p, b);
  const int block0 = static_cast<int>(blockIdx.x) * kWeightKeys, key0 = block0 + warp * kWarpKeys;
  if (block0 >= lens.len) return;
  const int page_mask = (1 << p.page_shift) - 1;
  int id[kM];
#pragma unroll
  for (int m = 0; m < kM; ++m) {
    id[m] = key0 + 16 * m < lens.len ? p.table[b * p.table_sb + ((key0 + 16 * m) >> p.page_shift)] : -1;
    if (id[m] >= p.n_pages) id[m] = -1;
  }
  uint4 kf[kM][2][kC];
#pragma unroll
  for (int m = 0; m < kM; ++m)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int slot = key0 + 16 * m + 8 * h + i;
      const __nv_bfloat16* k =
          static_cast<const __nv_bfloat16*>(p.kc) + id[m] * p.kc_sp + hk * p.kc_sh + (slot & page_mask) * p.kc_st + j * 8;
#pragma unroll
      for (int c = 0; c < kC; ++c) kf[m][h][c] = id[m] >= 0 && slot < lens.len ? ld16(k + c * 32) : make_uint4(0, 0, 0, 0);
    }
  F2 sum[kM][2];
#pragma unroll
  for (int m = 0; m < kM; ++m) sum[m][0] = sum[m][1] = pair(0.f, 0.f);

  const int rows = lens.ql * p.G;
  const float* lse = p.lse + (static_cast<int64_t>(b) * p.Hq + hk * p.G) * p.Nq;
  const auto fetch = [&](int base, Rows& to) {
    const int here = min(kWeightRows, rows - base);
    for (int x = threadIdx.x; x < here * (D / 8); x += 32 * kWeightWarps) {
      const int r = x / (D / 8), c = x % (D / 8), n = (base + r) / p.G, g = base + r - n * p.G;
      copy16(smem_addr(to.q + r * row_bytes<D>() + c * 16),
             static_cast<const __nv_bfloat16*>(p.q) + b * p.q_sb + (static_cast<int64_t>(hk) * p.G + g) * p.q_sh +
                 n * p.q_sn + c * 8,
             16);
    }
    copy_commit();
    if (threadIdx.x < kWeightRows) {
      const int r = threadIdx.x;
      float hi = 0.f, lo = 0.f;
      int most = 0;
      if (r < here) {
        const int n = (base + r) / p.G, g = base + r - n * p.G;
        const float x = lse[static_cast<int64_t>(g) * p.Nq + n];
        hi = -x * 1.4426950408889634f;
        // (what the product left, and x times log2(e) less its fp32 value)
        lo = fabsf(x) == INFINITY ? 0.f : fmaf(-x, 1.4426950408889634f, -hi) - x * 1.925963033e-8f;
        most = x == -INFINITY ? 0 : long_seen(p, lens, n);
      }
      to.hi[r] = hi;
      to.lo[r] = lo;
      to.sees[r] = most;
    }
  };
  const F2 c_hi = pair(p.c_hi, p.c_hi), c_lo = pair(p.c_lo, p.c_lo);
  if (rows > 0) fetch(0, rows_[0]);
  for (int base = 0, buf = 0; base < rows; base += kWeightRows, buf ^= 1) {
    copy_wait();
    __syncthreads();
    if (base + kWeightRows < rows) fetch(base + kWeightRows, rows_[buf ^ 1]);
    if (key0 >= lens.len) continue;
    const Rows& now = rows_[buf];
    const int here = min(kWeightRows, rows - base);
#pragma unroll 1
    for (int r0 = 0; r0 < here; r0 += 8) {
      float s[kM][4];
#pragma unroll
      for (int m = 0; m < kM; ++m) s[m][0] = s[m][1] = s[m][2] = s[m][3] = 0.f;
      const unsigned char* row = now.q + (r0 + i) * row_bytes<D>() + j * 16;
#pragma unroll
      for (int c = 0; c < kC; ++c) {
        const uint4 v = *reinterpret_cast<const uint4*>(row + c * 64);
#pragma unroll
        for (int m = 0; m < kM; ++m) {
          mma(s[m], kf[m][0][c].x, kf[m][1][c].x, kf[m][0][c].y, kf[m][1][c].y, v.x, v.y);
          mma(s[m], kf[m][0][c].z, kf[m][1][c].z, kf[m][0][c].w, kf[m][1][c].w, v.z, v.w);
        }
      }
      const int r = r0 + 2 * j;
      const float2 zh = *reinterpret_cast<const float2*>(now.hi + r), zl = *reinterpret_cast<const float2*>(now.lo + r);
      const int2 most = *reinterpret_cast<const int2*>(now.sees + r);
      const F2 hi = pair(zh.x, zh.y), lo = pair(zl.x, zl.y);
      const bool whole = __all_sync(0xffffffffu, key0 + kWarpKeys <= min(most.x, most.y));
#pragma unroll
      for (int m = 0; m < kM; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const F2 y = pair(s[m][2 * h], s[m][2 * h + 1]);
          const float2 a = split(add2(fma2(y, c_hi, hi), fma2(y, c_lo, lo)));
          float w0 = ex2(a.x), w1 = ex2(a.y);
          if (!whole) {
            const int slot = key0 + 16 * m + 8 * h + i;
            if (slot >= most.x) w0 = 0.f;
            if (slot >= most.y) w1 = 0.f;
          }
          sum[m][h] = add2(sum[m][h], pair(w0, w1));
        }
    }
  }
#pragma unroll
  for (int m = 0; m < kM; ++m)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float2 x = split(sum[m][h]);
      float z = x.x + x.y;
      z += __shfl_xor_sync(0xffffffffu, z, 1);
      z += __shfl_xor_sync(0xffffffffu, z, 2);
      const int slot = key0 + 16 * m + 8 * h + i;
      if (j != 0 || id[m] < 0 || slot >= lens.len) continue;
      const int64_t at = ((static_cast<int64_t>(id[m]) * p.Hk + hk) << p.page_shift) + (slot & page_mask);
      // the queries' own slots are new in this call: nothing was written there
      const bool old = p.decay != 0.f && !(p.causal && slot >= lens.len - lens.ql);
      p.weights_out[at] = old ? fmaf(p.decay, p.weights[at], z) : z;
    }
}

template <int D>
cudaError_t weights_dim(const LongParams& p, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>((p.max_len + kWeightKeys - 1) / kWeightKeys), p.Hk, p.B);
  return launch(weights_kernel<D>, grid, 32 * kWeightWarps, 0, s, 1, p);
}

}  // namespace

cudaError_t launch_weights(const LongParams& p, int d, cudaStream_t s) {
  if (static_cast<int64_t>(p.Nq) * p.G >= TILE_ROWS) return launch_weights_tiles(p, d, s);
  switch (d) {
    case 32: return weights_dim<32>(p, s);
    case 64: return weights_dim<64>(p, s);
    case 128: return weights_dim<128>(p, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace attn
