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

namespace attn {
namespace {

using namespace ldev;

constexpr int kWeightWarps = 4, kWeightKeys = 16 * kWeightWarps, kWeightRows = 64;

// A warp keeps 16 keys in registers and goes over the query rows, which lie in shared
// memory, 8 at a time; a lane's sums are over rows 2 j and 2 j + 1 of each group for
// keys i and i + 8. Grid: key groups, key head, sequence.
template <int D>
__global__ void __launch_bounds__(32 * kWeightWarps) weights_kernel(const __grid_constant__ LongParams p) {
  constexpr int kC = D / 32;
  __shared__ __align__(16) unsigned char qs[kWeightRows * row_bytes<D>()];
  __shared__ float2 lse2[kWeightRows];  // lse * log2(e) in two parts
  __shared__ int sees[kWeightRows];     // slots that the row sees
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, i = lane >> 2, j = lane & 3;
  const int b = blockIdx.z, hk = blockIdx.y;
  const LongLens lens = long_lens(p, b);
  const int block0 = static_cast<int>(blockIdx.x) * kWeightKeys, key0 = block0 + warp * 16;
  if (block0 >= lens.len) return;
  const int page_mask = (1 << p.page_shift) - 1;
  const int id = key0 < lens.len ? p.table[b * p.table_sb + (key0 >> p.page_shift)] : -1;
  const bool real = id >= 0 && id < p.n_pages;
  uint4 kf[2][kC];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int slot = key0 + i + 8 * h;
    const __nv_bfloat16* k =
        static_cast<const __nv_bfloat16*>(p.kc) + id * p.kc_sp + hk * p.kc_sh + (slot & page_mask) * p.kc_st + j * 8;
#pragma unroll
    for (int c = 0; c < kC; ++c) kf[h][c] = real && slot < lens.len ? ld16(k + c * 32) : make_uint4(0, 0, 0, 0);
  }
  float sum[2] = {0.f, 0.f};
  const int rows = min(lens.ql, p.Nq) * p.G;
  for (int base = 0; base < rows; base += kWeightRows) {
    const int here = min(kWeightRows, rows - base);
    __syncthreads();
    for (int x = threadIdx.x; x < here * (D / 8); x += 32 * kWeightWarps) {
      const int r = x / (D / 8), c = x % (D / 8), n = (base + r) / p.G, g = base + r - n * p.G;
      *reinterpret_cast<uint4*>(qs + r * row_bytes<D>() + c * 16) =
          ld16(static_cast<const __nv_bfloat16*>(p.q) + b * p.q_sb + (static_cast<int64_t>(hk) * p.G + g) * p.q_sh +
               n * p.q_sn + c * 8);
    }
    for (int r = threadIdx.x; r < kWeightRows; r += 32 * kWeightWarps) {
      float2 z = make_float2(0.f, 0.f);
      int most = 0;
      if (r < here) {
        const int n = (base + r) / p.G, g = base + r - n * p.G;
        const float x = p.lse[(static_cast<int64_t>(b) * p.Hq + hk * p.G + g) * p.Nq + n];
        z.x = x * 1.4426950408889634f;
        z.y = fmaf(x, 1.4426950408889634f, -z.x) + x * 1.925963033e-8f;  // log2(e) - its fp32 value
        if (x == -INFINITY || x == INFINITY) z.y = 0.f;
        most = x == -INFINITY ? 0 : long_seen(p, lens, n);
      }
      lse2[r] = z;
      sees[r] = most;
    }
    __syncthreads();
    if (key0 >= lens.len) continue;
    for (int r0 = 0; r0 < here; r0 += 8) {
      float s[4] = {0.f, 0.f, 0.f, 0.f};
      const unsigned char* row = qs + (r0 + i) * row_bytes<D>() + j * 16;
#pragma unroll
      for (int c = 0; c < kC; ++c) {
        const uint4 v = *reinterpret_cast<const uint4*>(row + c * 64);
        mma(s, kf[0][c].x, kf[1][c].x, kf[0][c].y, kf[1][c].y, v.x, v.y);
        mma(s, kf[0][c].z, kf[1][c].z, kf[0][c].w, kf[1][c].w, v.z, v.w);
      }
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int r = r0 + 2 * j + x;
        const float2 z = lse2[r];
        const int most = sees[r];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float y = s[2 * h + x];
          const float w = ex2(fmaf(y, p.c_hi, -z.x) + fmaf(y, p.c_lo, -z.y));
          sum[h] += key0 + i + 8 * h < most ? w : 0.f;
        }
      }
    }
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float z = sum[h];
    z += __shfl_xor_sync(0xffffffffu, z, 1);
    z += __shfl_xor_sync(0xffffffffu, z, 2);
    const int slot = key0 + i + 8 * h;
    if (j != 0 || !real || slot >= lens.len) continue;
    const int64_t at = ((static_cast<int64_t>(id) * p.Hk + hk) << p.page_shift) + (slot & page_mask);
    // the queries' own slots are new in this call: nothing was written there
    const bool old = p.decay != 0.f && !(p.causal && slot >= lens.len - lens.ql);
    p.weights_out[at] = old ? fmaf(p.decay, p.weights[at], z) : z;
  }
}

template <int D>
cudaError_t weights_dim(const LongParams& p, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>((p.max_len + kWeightKeys - 1) / kWeightKeys), p.Hk, p.B);
  return launch(weights_kernel<D>, grid, 32 * kWeightWarps, 0, s, p);
}

}  // namespace

cudaError_t launch_weights(const LongParams& p, int d, cudaStream_t s) {
  switch (d) {
    case 32: return weights_dim<32>(p, s);
    case 64: return weights_dim<64>(p, s);
    case 128: return weights_dim<128>(p, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace attn
