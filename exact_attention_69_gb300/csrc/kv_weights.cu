// kv_weights.cu -- the attention weight that cached tokens receive: for each slot the
// sum over queries and the query heads of its key head of exp(scale q . k - lse), with
// the log-sum-exp that the attention returned.
//
// A weight's relative error is its exponent's absolute one, so the factor scale *
// log2(e) and each lse * log2(e) go in as an fp32 value and what that leaves: s * c_hi -
// lse_hi is one fused operation, exact up to the rounding of a difference that is small
// where the weight is not.
//
// Few rows are bound by memory: keys once, weights once each way. 32 sequences of 256 to
// 4224 tokens, 8 key heads, d = 128, pages of 64 (115 MB) take 21.7 us, 5.3 TB/s. (One
// group of 16 keys a warp, nothing on its way meanwhile: 31.6 us.)
#include <cfloat>

#include "long_dev.cuh"
#include "long_kernel.h"

namespace attn {
namespace {

using namespace ldev;

constexpr int kWeightWarps = 4;
// log2(e), and what its fp32 value leaves of it
constexpr float kLog2e = 1.4426950408889634f, kLog2eLeft = static_cast<float>(1.4426950408889634074 - kLog2e);

// Few rows (up to 32, all in shared memory): the keys stream by. A warp takes every
// fourth group of 16 keys of its block's `units` groups a warp, the next group's keys and
// old weights on their way while it works on one; a lane's sums are over rows 2 j and
// 2 j + 1 of each 8, for keys i and i + 8. Grid: runs of keys, key head, sequence.
template <int D>
__global__ void __launch_bounds__(32 * kWeightWarps) weights_kernel(const __grid_constant__ LongParams p, int units) {
  constexpr int kC = D / 32;
  __shared__ __align__(16) unsigned char q[kFewRows * row_bytes<D>()];
  __shared__ float hi[kFewRows], lo[kFewRows];  // -lse * log2(e) in two parts
  __shared__ int sees[kFewRows];                // slots that the row sees
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, i = lane >> 2, j = lane & 3;
  const int b = blockIdx.z, hk = blockIdx.y;
  const int key0 = static_cast<int>(blockIdx.x) * units * kWeightWarps * 16 + warp * 16;  // of the warp's first group
  constexpr int kStride = kWeightWarps * 16;
  // the pages of the warp's groups, one a lane (units <= 32)
  const int mine = (key0 + lane * kStride) >> p.page_shift;
  int id = lane < units && mine < p.table_width ? p.table[b * p.table_sb + mine] : -1;
  if (id >= p.n_pages) id = -1;
  const LongLens lens = long_lens(p, b);
  if (key0 - warp * 16 >= lens.len) return;
  const int rows = lens.ql * p.G, page_mask = (1 << p.page_shift) - 1;
  for (int x = threadIdx.x; x < rows * (D / 8); x += 32 * kWeightWarps) {
    const int r = x / (D / 8), c = x % (D / 8), n = p.by_g.div(r), g = r - n * p.G;
    copy16(smem_addr(q + r * row_bytes<D>() + c * 16),
           static_cast<const __nv_bfloat16*>(p.q) + b * p.q_sb + (static_cast<int64_t>(hk) * p.G + g) * p.q_sh + n * p.q_sn + c * 8,
           16);
  }
  copy_commit();

  struct Group {
    uint4 k[2][kC];
    float old[2];
    int64_t at;  // of slot 0 of the group's page, in the weights
  };
  const __nv_bfloat16* kbase = static_cast<const __nv_bfloat16*>(p.kc) + hk * p.kc_sh + j * 8;
  const int fresh = p.decay == 0.f ? 0 : (p.causal ? lens.len - lens.ql : lens.len);  // slots behind start from zero
  const auto load = [&](int u, Group& to) {
    const int page = __shfl_sync(0xffffffffu, id, u), first = key0 + u * kStride;
    to.at = ((static_cast<int64_t>(page) * p.Hk + hk) << p.page_shift) + (first & page_mask);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int slot = first + i + 8 * h;
      const bool live = page >= 0 && slot < lens.len;
      const __nv_bfloat16* k = kbase + page * p.kc_sp + (slot & page_mask) * p.kc_st;
#pragma unroll
      for (int c = 0; c < kC; ++c) to.k[h][c] = live ? ld16(k + c * 32) : make_uint4(0, 0, 0, 0);
      to.old[h] = j == 0 && live && slot < fresh ? p.weights[to.at + i + 8 * h] : 0.f;
    }
  };
  Group now, next;
  if (key0 < lens.len) load(0, now);
  if (threadIdx.x < kFewRows) {
    const int r = threadIdx.x;
    float zh = 0.f, zl = 0.f;
    int most = 0;
    if (r < rows) {
      const int n = p.by_g.div(r), g = r - n * p.G;
      const float x = p.lse[(static_cast<int64_t>(b) * p.Hq + hk * p.G + g) * p.Nq + n];
      zh = -x * kLog2e;
      // (what the product left, and x times log2(e) less its fp32 value; none of an infinity)
      if (fabsf(x) >= 1e38f) {
        if (fabsf(x) < INFINITY) zh = copysignf(FLT_MAX, -x);  // (finite, as the lse is)
      } else {
        zl = fmaf(-x, kLog2e, -zh) - x * kLog2eLeft;
      }
      most = x == -INFINITY ? 0 : long_seen(p, lens, n);
    }
    hi[r] = zh;
    lo[r] = zl;
    sees[r] = most;
  }
  copy_wait();
  __syncthreads();
  const F2 c_hi = pair(p.c_hi, p.c_hi), c_lo = pair(p.c_lo, p.c_lo);
#pragma unroll 1
  for (int u = 0; u < units && key0 + u * kStride < lens.len; ++u) {
    if (u + 1 < units && key0 + (u + 1) * kStride < lens.len) load(u + 1, next);
    const int first = key0 + u * kStride;
    float sum[2] = {0.f, 0.f};
#pragma unroll 1
    for (int r0 = 0; r0 < rows; r0 += 8) {
      float s[2][4] = {};  // (two sums of half the channels: shorter chains)
      const unsigned char* row = q + (r0 + i) * row_bytes<D>() + j * 16;
#pragma unroll
      for (int c = 0; c < kC; ++c) {
        const uint4 v = *reinterpret_cast<const uint4*>(row + c * 64);
        mma(s[0], now.k[0][c].x, now.k[1][c].x, now.k[0][c].y, now.k[1][c].y, v.x, v.y);
        mma(s[1], now.k[0][c].z, now.k[1][c].z, now.k[0][c].w, now.k[1][c].w, v.z, v.w);
      }
      const int r = r0 + 2 * j;
      const float2 zh = *reinterpret_cast<const float2*>(hi + r), zl = *reinterpret_cast<const float2*>(lo + r);
      const int2 most = *reinterpret_cast<const int2*>(sees + r);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const F2 y = add2(pair(s[0][2 * h], s[0][2 * h + 1]), pair(s[1][2 * h], s[1][2 * h + 1]));
        const float2 a = split(add2(fma2(y, c_hi, pair(zh.x, zh.y)), fma2(y, c_lo, pair(zl.x, zl.y))));
        const int slot = first + i + 8 * h;
        sum[h] += slot < most.x ? ex2(a.x) : 0.f;
        sum[h] += slot < most.y ? ex2(a.y) : 0.f;
      }
    }
    const int page = __shfl_sync(0xffffffffu, id, u);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float z = sum[h];
      z += __shfl_xor_sync(0xffffffffu, z, 1);
      z += __shfl_xor_sync(0xffffffffu, z, 2);
      const int slot = first + i + 8 * h;
      if (j == 0 && page >= 0 && slot < lens.len)
        p.weights_out[now.at + i + 8 * h] = slot < fresh ? fmaf(p.decay, now.old[h], z) : z;
    }
    now = next;
  }
}

// Groups of 16 keys a warp: enough blocks for kWeightBlocks a SM, groups enough to be worth a
// block's start.
constexpr int kWeightBlocks = 8, kWeightUnits = 8;

template <int D>
cudaError_t weights_dim(const LongParams& p, cudaStream_t s) {
  const int64_t groups = p.max_len / 16;
  int64_t units = groups * p.Hk * p.B / (static_cast<int64_t>(kWeightBlocks) * p.sms * kWeightWarps);
  units = units < 1 ? 1 : (units > kWeightUnits ? kWeightUnits : units);
  const int64_t keys = units * kWeightWarps * 16;
  const dim3 grid(static_cast<unsigned>((p.max_len + keys - 1) / keys), p.Hk, p.B);
  return launch(weights_kernel<D>, grid, 32 * kWeightWarps, 0, s, 1, p, static_cast<int>(units));
}

}  // namespace

cudaError_t launch_weights(const LongParams& p, int d, cudaStream_t s) {
  if (p.full_tiles == 1 || !weights_few_rows(p)) return launch_weights_tiles(p, d, s);
  switch (d) {
    case 32: return weights_dim<32>(p, s);
    case 64: return weights_dim<64>(p, s);
    case 128: return weights_dim<128>(p, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace attn
