// rope.cu -- root-mean-square norm of every head with the rotary position
// embedding in the same pass, its gradient, and the append to a paged cache.
//
//   y = R(pos) (x * r * w),  r = 1 / sqrt(mean(x^2) + eps)
// with R turning each pair of the first `rot` channels by pos * inv_freq.
//
// What bounds it: each row is read once and written once, so device memory; but
// an SM moves only 23 bytes a clock, so it has some 20 instructions for each 16
// bytes read before the arithmetic shows. A row of d channels is d/8 threads of
// 16 bytes each, so a warp reads 512 contiguous bytes of rows; the row sum and the
// exchange with the pair's other half (raw bf16, four words) are warp shuffles. A
// thread keeps one token and one channel chunk and goes over the heads, and
// weights, cosines and sines are folded into two factors a channel that stay in
// registers: y = r (x A + x' B), packed two channels an instruction. The block's
// angles are computed once, into shared memory (a thread for each was half of the
// time with 16 heads). Loads of four heads are in flight at a time.
//
// Measured (rows read and written, with weights and positions):
//   B8 H32+8 N4096 d128 out of a fused projection: 114 us, 5.9 TB/s; gradient 196 us, 5.1 TB/s
//   B4 H16+4 N2048 d128: 23.4 us, 3.6 TB/s; gradient 32.4 us, 3.9 TB/s
//   B1 H8+8 N16384 d128: 29.6 us, 4.5 TB/s; gradient 51.1 us, 3.9 TB/s
// Below the largest size the last, partly filled round of blocks shows (1024
// blocks of 16 tokens on 456 places). Persistent blocks over smaller tiles even
// that out and are slower all the same (43.7 us where one block a tile takes
// 29.6): each tile waits for its angles at a barrier. Head subsets inside a
// block, one tile a block, took 39 to 51 us.
//
// Angles: a frequency becomes a 64-bit fraction of a turn, and position times
// frequency is a 64-bit integer product whose overflow drops whole turns. The
// fraction is exact to 2^-64 * position, where a 32-bit product of position
// and frequency is off by 2^-24 of the angle (0.06 radians at position 10^6).
#include <cuda_bf16.h>
#include <math_constants.h>

#include "rope_kernel.h"

namespace attn {
namespace {

constexpr int kUnroll = 4;

__device__ __forceinline__ void grid_dep_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_dep_launch() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// radians per position -> turns per position as a 64-bit fraction (whole turns
// dropped): f = m 2^e, f / 2pi = m (2^66 / 2pi) 2^(e - 66), times 2^64. Integer
// arithmetic: the double-precision units of this GPU are few.
__device__ __forceinline__ uint64_t turns_of(double f) {
  const uint64_t bits = static_cast<uint64_t>(__double_as_longlong(f));
  const int ex = static_cast<int>((bits >> 52) & 0x7ff);
  if (ex == 0 || ex == 0x7ff) return 0;  // zero, subnormal; infinity and NaN have no angle
  const uint64_t m = (bits & 0xFFFFFFFFFFFFFull) | (1ull << 52);
  const uint64_t kInvTwoPi66 = 11743562013128004906ull;  // round(2^66 / (2 pi))
  const uint64_t hi = __umul64hi(m, kInvTwoPi66), lo = m * kInvTwoPi66;
  const int sh = 2 - (ex - 1075);  // right shift of the 128-bit product
  uint64_t t;
  if (sh <= 0) {
    t = -sh < 64 ? lo << -sh : 0;
  } else if (sh < 64) {
    t = (lo >> sh) | (hi << (64 - sh));
  } else {
    t = sh < 128 ? hi >> (sh - 64) : 0;
  }
  return (bits >> 63) ? 0ull - t : t;
}

// cos and sin of position * frequency.
__device__ __forceinline__ void angle(int64_t pos, uint64_t turns, float& c, float& s) {
  const uint64_t ph = static_cast<uint64_t>(pos) * turns;
  const float half_turns = static_cast<float>(static_cast<int32_t>(ph >> 32)) * 4.656612873077392578125e-10f;  // 2^-31
  sincospif(half_turns, &s, &c);
}

__device__ __forceinline__ void unpack(const uint4& u, float2 (&x)[4]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
}

__device__ __forceinline__ uint32_t pack2(float2 x) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(x.y), "f"(x.x));
  return r;
}

__device__ __forceinline__ uint4 pack(const float2 (&x)[4]) {
  return make_uint4(pack2(x[0]), pack2(x[1]), pack2(x[2]), pack2(x[3]));
}

__device__ __forceinline__ void load_weights(const void* w, int type, int at, float2 (&out)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int j = at + 2 * i;
    if (w == nullptr) {
      out[i] = make_float2(1.f, 1.f);
    } else if (type == 1) {
      out[i] = make_float2(static_cast<const float*>(w)[j], static_cast<const float*>(w)[j + 1]);
    } else {
      const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(w) + j;
      out[i] = make_float2(__bfloat162float(x[0]), __bfloat162float(x[1]));
    }
  }
}

// Sum over the d/8 threads of a row.
template <int D>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int o = D / 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

__device__ __forceinline__ int64_t position(const void* pos, int type, int64_t sb, int64_t sn, int b, int n) {
  const int64_t at = b * sb + n * sn;
  return type == 1 ? static_cast<const int32_t*>(pos)[at] : static_cast<const int64_t*>(pos)[at];
}

// cos and sin of the block's tokens, [token slot][frequency].
template <int D>
struct Angles {
  static constexpr int kTokens = rope_tokens_per_block(D);
  uint64_t turns[D / 2];
  int64_t pos[kTokens];
  float2 cs[kTokens * (D / 2)];
};

// Fills the table for tokens t0 ... of B * N (all threads; P: either parameter block).
template <int D, typename P>
__device__ __forceinline__ void fill_angles(Angles<D>& a, const P& p, int64_t t0, int64_t total, const int32_t* starts,
                                            bool first) {
  constexpr int kT = Angles<D>::kTokens;
  const int n_f = p.rot / 2;
  if (n_f == 0) return;
  __syncthreads();
  if (first)
    for (int i = threadIdx.x; i < n_f; i += kRopeThreads) a.turns[i] = turns_of(p.inv_freq[i]);
  if (threadIdx.x < kT && t0 + threadIdx.x < total) {
    const int64_t tok = t0 + threadIdx.x;
    const int b = static_cast<int>(tok / p.N), n = static_cast<int>(tok - static_cast<int64_t>(b) * p.N);
    a.pos[threadIdx.x] = p.pos != nullptr ? position(p.pos, p.pos_type, p.pos_sb, p.pos_sn, b, n)
                                          : p.pos_offset + n + (starts != nullptr ? starts[b] : 0);
  }
  __syncthreads();
  const int live = static_cast<int>(min(static_cast<int64_t>(kT), total - t0)) * n_f;
  for (int i = threadIdx.x; i < live; i += kRopeThreads) {
    const int tok = i / n_f, f = i - tok * n_f;
    float2 x;
    angle(a.pos[tok], a.turns[f], x.x, x.y);
    a.cs[tok * (D / 2) + f] = x;
  }
  __syncthreads();
}

// A thread's place in its row. Half-split pairs (IL false): channel i turns with
// channel i + rot/2, held by the thread rot/16 chunks away; side by side (IL
// true): both channels of a pair are the thread's own.
template <int D, bool IL>
struct Place {
  int c;         // chunk of 8 channels
  bool on;       // the chunk is rotated
  bool low;      // half-split: the first half of the pairs
  int partner;   // half-split: lane of the other half
  int pchunk;    // half-split: its chunk
  __device__ __forceinline__ explicit Place(int rot) {
    c = threadIdx.x % (D / 8);
    const int lane = threadIdx.x & 31, hc = rot / 16;
    on = c * 8 < rot;
    low = c < hc;
    pchunk = (!IL && on) ? (low ? c + hc : c - hc) : c;
    partner = lane + (pchunk - c);
  }
  // The rotation as factors of the own and the paired channel, y = x A + x' B.
  __device__ __forceinline__ void factors(const float2* cs, float2 (&A)[4], float2 (&B)[4]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      A[i] = make_float2(1.f, 1.f);
      B[i] = make_float2(0.f, 0.f);
    }
    if (!on) return;
    if constexpr (IL) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 x = cs[c * 4 + i];
        A[i] = make_float2(x.x, x.x);
        B[i] = make_float2(-x.y, x.y);
      }
    } else {
      const float2* f = cs + (low ? c : pchunk) * 8;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 x = f[2 * i], y = f[2 * i + 1];
        A[i] = make_float2(x.x, y.x);
        B[i] = low ? make_float2(-x.y, -y.y) : make_float2(x.y, y.y);
      }
    }
  }
  // The paired channels of the thread's chunk; zeros where it is not rotated (an
  // infinity there must not meet the factor 0). All 32 lanes call it.
  __device__ __forceinline__ void paired(const uint4& u, const float2 (&x)[4], float2 (&o)[4]) const {
    if constexpr (IL) {
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = make_float2(x[i].y, x[i].x);
    } else {
      uint4 w = make_uint4(__shfl_sync(0xffffffffu, u.x, partner), __shfl_sync(0xffffffffu, u.y, partner),
                           __shfl_sync(0xffffffffu, u.z, partner), __shfl_sync(0xffffffffu, u.w, partner));
      if (!on) w = make_uint4(0u, 0u, 0u, 0u);
      unpack(w, o);
      return;
    }
    if (!on) {
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = make_float2(0.f, 0.f);
    }
  }
};

__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }

__device__ __forceinline__ uint4 load16(const __nv_bfloat16* p) {
  return __ldcs(reinterpret_cast<const uint4*>(p));
}
__device__ __forceinline__ void store16(__nv_bfloat16* p, const uint4& u) { *reinterpret_cast<uint4*>(p) = u; }

// Heads [h0, h1) of one token: norm, turn, store. in/out: the token's first
// head at this thread's channels. Every lane of the warp goes through the
// same heads; `live` says whether its loads and stores are real. The next
// heads' loads go out before these are worked on, and the first ones' before
// `angles` (the block's table, where it is not there yet).
template <int D, bool IL, bool NORM, typename Fill>
__device__ __forceinline__ void rope_heads(const __nv_bfloat16* in, int64_t in_sh, __nv_bfloat16* out,
                                           int64_t out_sh, int h0, int h1, bool live, const void* w, int w_type,
                                           float eps, const Place<D, IL>& pl, const float2* cs, const Fill& angles) {
  uint4 next[kUnroll];
  auto fetch = [&](int h) {
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      next[u] = make_uint4(0, 0, 0, 0);
      if (live && h + u < h1) next[u] = load16(in + (h + u) * in_sh);
    }
  };
  fetch(h0);
  angles();
  float2 A[4], B[4];
  pl.factors(cs, A, B);
  if constexpr (NORM) {
    if (w != nullptr) {
      float2 wo[4], wp[4];
      load_weights(w, w_type, pl.c * 8, wo);
      load_weights(w, w_type, pl.pchunk * 8, wp);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        A[i] = mul2(A[i], wo[i]);
        B[i] = mul2(B[i], IL ? make_float2(wo[i].y, wo[i].x) : wp[i]);
      }
    }
  }
  for (int h = h0; h < h1; h += kUnroll) {
    uint4 raw[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) raw[u] = next[u];
    if (h + kUnroll < h1) fetch(h + kUnroll);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (h + u >= h1) break;  // the same for the whole block
      float2 x[4], o[4];
      unpack(raw[u], x);
      pl.paired(raw[u], x, o);
      float2 r2 = make_float2(1.f, 1.f);
      if constexpr (NORM) {
        float2 s = mul2(x[0], x[0]);
#pragma unroll
        for (int i = 1; i < 4; ++i) s = fma2(x[i], x[i], s);
        const float r = rsqrtf(row_sum<D>(s.x + s.y) * (1.f / D) + eps);
        r2 = make_float2(r, r);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[i] = fma2(x[i], A[i], mul2(o[i], B[i]));
        if constexpr (NORM) x[i] = mul2(x[i], r2);
      }
      if (live) store16(out + (h + u) * out_sh, pack(x));
    }
  }
}

template <int D, bool IL, bool NORM>
__global__ void __launch_bounds__(kRopeThreads, 3) rope_kernel(const __grid_constant__ RopeParams p) {
  __shared__ Angles<D> ang;
  grid_dep_launch();
  grid_dep_wait();
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * rope_tokens_per_block(D), total = static_cast<int64_t>(p.B) * p.N;
  const int slot_in_block = threadIdx.x / (D / 8);
  const int64_t tok = t0 + slot_in_block;
  const bool live = tok < total;
  const int b = live ? static_cast<int>(tok / p.N) : 0, n = live ? static_cast<int>(tok - static_cast<int64_t>(b) * p.N) : 0;
  const Place<D, IL> pl(p.rot);
  const float2* cs = ang.cs + (live ? slot_in_block : 0) * (D / 2);
  // virtual heads: queries, then keys, then values
  const int v0 = blockIdx.y * p.heads_per_block, v1 = v0 + p.heads_per_block;
  const auto at = [&](const RopeTensor& x) {
    return static_cast<__nv_bfloat16*>(x.p) + b * x.sb + n * x.sn + pl.c * 8;
  };
  const auto fill = [&]() { fill_angles(ang, p, t0, total, p.starts, true); };
  if (v0 < p.Hq)
    rope_heads<D, IL, NORM>(at(p.q), p.q.sh, at(p.qo), p.qo.sh, v0, min(v1, p.Hq), live, p.wq, p.wq_type, p.eps, pl, cs,
                            fill);
  const int k0 = max(v0 - p.Hq, 0), k1 = min(v1 - p.Hq, p.Hk);
  const auto fill_k = [&]() {
    if (v0 >= p.Hq) fill();
  };
  if (!p.cache) {
    if (k0 < k1)
      rope_heads<D, IL, NORM>(at(p.k), p.k.sh, at(p.ko), p.ko.sh, k0, k1, live, p.wk, p.wk_type, p.eps, pl, cs, fill_k);
    return;
  }
  // The token's slot. A token behind its sequence's count, behind the table's
  // end or on a page that the cache does not have leaves the cache as it was.
  const int start = p.starts[b];
  const int64_t slot = static_cast<int64_t>(start) + n;
  bool write = live && start >= 0 && (p.counts == nullptr || n < p.counts[b]) && (slot >> p.page_shift) < p.table_width;
  int page = 0;
  if (write) {
    page = p.table[b * p.table_sb + (slot >> p.page_shift)];
    write = page >= 0 && page < p.n_pages;
  }
  if (!write) page = 0;
  const int in_page = static_cast<int>(slot & ((1 << p.page_shift) - 1));
  const int c8 = pl.c * 8;
  if (k0 < k1)
    rope_heads<D, IL, NORM>(at(p.k), p.k.sh,
                            static_cast<__nv_bfloat16*>(p.kc) + page * p.kc_sp + in_page * p.kc_st + c8, p.kc_sh, k0,
                            k1, write, p.wk, p.wk_type, p.eps, pl, cs, fill_k);
  const int w0 = max(v0 - p.Hq - p.Hk, 0), w1 = min(v1 - p.Hq - p.Hk, p.Hk);
  if (!write) return;
  const __nv_bfloat16* vi = at(p.v);
  __nv_bfloat16* vo = static_cast<__nv_bfloat16*>(p.vc) + page * p.vc_sp + in_page * p.vc_st + c8;
  for (int h = w0; h < w1; h += kUnroll) {
    uint4 raw[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      if (h + u < w1) raw[u] = load16(vi + (h + u) * p.v.sh);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      if (h + u < w1) store16(vo + (h + u) * p.vc_sh, raw[u]);
  }
}

// ---------------------------------------------------------------- backward
//
//   g = R^T dy,  h = g * w,  dx = r h - x r^3 mean(h x),  dw = sum g x r
// A thread keeps one channel chunk over all of its rows, so dw is eight
// registers; the block adds its threads' sums in a fixed order and leaves one
// row of partial sums, which a second kernel adds: no atomics, the same bits
// every time.
template <int D, bool IL, bool NORM, typename Fill>
__device__ __forceinline__ void rope_bwd_heads(const __nv_bfloat16* x_in, int64_t x_sh, const __nv_bfloat16* dy_in,
                                               int64_t dy_sh, __nv_bfloat16* dx_out, int64_t dx_sh, int H, bool live,
                                               const float2 (&w)[4], float eps, const Place<D, IL>& pl,
                                               const float2* cs, const Fill& angles, float2 (&dw)[4]) {
  constexpr int kU = 2;
  uint4 nx[kU], ng[kU];
  auto fetch = [&](int h) {
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      nx[u] = ng[u] = make_uint4(0, 0, 0, 0);
      if (live && h + u < H) {
        if constexpr (NORM) nx[u] = load16(x_in + (h + u) * x_sh);
        ng[u] = load16(dy_in + (h + u) * dy_sh);
      }
    }
  };
  fetch(0);
  angles();
  float2 A[4], B[4];
  pl.factors(cs, A, B);
  for (int h = 0; h < H; h += kU) {
    uint4 rx[kU], rg[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      rx[u] = nx[u];
      rg[u] = ng[u];
    }
    if (h + kU < H) fetch(h + kU);
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      if (h + u >= H) break;
      float2 g[4], o[4];
      unpack(rg[u], g);
      pl.paired(rg[u], g, o);
#pragma unroll
      for (int i = 0; i < 4; ++i) g[i] = fma2(g[i], A[i], mul2(o[i], make_float2(-B[i].x, -B[i].y)));
      if constexpr (NORM) {
        float2 x[4], s = make_float2(0.f, 0.f), dot = make_float2(0.f, 0.f);
        unpack(rx[u], x);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          s = fma2(x[i], x[i], s);
          dot = fma2(mul2(g[i], w[i]), x[i], dot);
        }
        const float r = rsqrtf(row_sum<D>(s.x + s.y) * (1.f / D) + eps);
        const float k = row_sum<D>(dot.x + dot.y) * (-1.f / D) * r * r * r;
        const float2 r2 = make_float2(r, r), k2 = make_float2(k, k);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          g[i] = mul2(g[i], r2);
          if (live) dw[i] = fma2(g[i], x[i], dw[i]);
          g[i] = fma2(g[i], w[i], mul2(x[i], k2));
        }
      }
      if (live) store16(dx_out + (h + u) * dx_sh, pack(g));
    }
  }
}

template <int D>
__device__ __forceinline__ void block_sum(const float2 (&dw)[4], float* smem, float* out) {
  // [token slot][channel]; then one thread per channel adds the slots in order
  constexpr int kRows = rope_tokens_per_block(D);
  __syncthreads();
  const int c = threadIdx.x % (D / 8), row = threadIdx.x / (D / 8);
#pragma unroll
  for (int i = 0; i < 4; ++i) *reinterpret_cast<float2*>(smem + row * D + c * 8 + 2 * i) = dw[i];
  __syncthreads();
  if (threadIdx.x < D) {
    float s = 0.f;
    for (int r = 0; r < kRows; ++r) s += smem[r * D + threadIdx.x];
    out[threadIdx.x] = s;
  }
}

template <int D, bool IL, bool NORM>
__global__ void __launch_bounds__(kRopeThreads, 2) rope_bwd_kernel(const __grid_constant__ RopeBwdParams p) {
  __shared__ Angles<D> ang;
  __shared__ __align__(16) float sums[rope_tokens_per_block(D) * D];
  grid_dep_launch();
  grid_dep_wait();
  const Place<D, IL> pl(p.rot);
  const int64_t total = static_cast<int64_t>(p.B) * p.N;
  constexpr int kTok = rope_tokens_per_block(D);
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kTok;
  // the queries' rows, then the keys': one set of weights and sums in registers at a time
#pragma unroll 1
  for (int side = 0; side < 2; ++side) {
    const int H = side ? p.Hk : p.Hq;
    if (H == 0) continue;
    const RopeTensor &x = side ? p.k : p.q, &dy = side ? p.dyk : p.dyq, &dx = side ? p.dk : p.dq;
    float2 w[4], dw[4];
    load_weights(side ? p.wk : p.wq, side ? p.wk_type : p.wq_type, pl.c * 8, w);
#pragma unroll
    for (int i = 0; i < 4; ++i) dw[i] = make_float2(0.f, 0.f);
#pragma unroll 1
    for (int64_t t0 = first; t0 < total; t0 += static_cast<int64_t>(gridDim.x) * kTok) {
      const int slot = threadIdx.x / (D / 8);
      const int64_t tok = t0 + slot;
      const bool live = tok < total;
      const int b = live ? static_cast<int>(tok / p.N) : 0,
                n = live ? static_cast<int>(tok - static_cast<int64_t>(b) * p.N) : 0;
      const auto at = [&](const RopeTensor& y) {
        return static_cast<__nv_bfloat16*>(y.p) + b * y.sb + n * y.sn + pl.c * 8;
      };
      rope_bwd_heads<D, IL, NORM>(at(x), x.sh, at(dy), dy.sh, at(dx), dx.sh, H, live, w, p.eps, pl,
                                  ang.cs + (live ? slot : 0) * (D / 2),
                                  [&]() { fill_angles(ang, p, t0, total, nullptr, t0 == first && (side == 0 || p.Hq == 0)); },
                                  dw);
    }
    if constexpr (NORM) {
      if ((side ? p.dwk : p.dwq) != nullptr)
        block_sum<D>(dw, sums, p.part + (static_cast<int64_t>(blockIdx.x) * 2 + side) * D);
    }
  }
}

// dw[side][channel] = sum of the blocks' partial sums; a block per side and 32
// channels, a warp per stripe of rows, stripes joined in order.
__global__ void __launch_bounds__(1024) rope_dw_kernel(const float* part, int blocks, int d, void* dwq, int wq_type,
                                                       void* dwk, int wk_type) {
  __shared__ float s[32][33];
  grid_dep_launch();
  grid_dep_wait();
  const int side = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  void* out = side ? dwk : dwq;
  if (out == nullptr) return;
  const int c = blockIdx.x * 32 + lane;
  float a = 0.f;
#pragma unroll 4
  for (int r = warp; r < blocks; r += 32) a += part[(static_cast<int64_t>(r) * 2 + side) * d + c];
  s[warp][lane] = a;
  __syncthreads();
  if (warp == 0) {
    float z = 0.f;
#pragma unroll
    for (int w = 0; w < 32; ++w) z += s[w][lane];
    if ((side ? wk_type : wq_type) == 1)
      static_cast<float*>(out)[c] = z;
    else
      static_cast<__nv_bfloat16*>(out)[c] = __float2bfloat16(z);
  }
}

template <typename... Args, typename... Given>
cudaError_t launch(void (*kern)(Args...), dim3 grid, int threads, cudaStream_t s, const Given&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

template <int D>
cudaError_t launch_rope_dim(const RopeParams& p, dim3 grid, cudaStream_t s) {
  if (p.interleaved)
    return p.norm ? launch(rope_kernel<D, true, true>, grid, kRopeThreads, s, p)
                  : launch(rope_kernel<D, true, false>, grid, kRopeThreads, s, p);
  return p.norm ? launch(rope_kernel<D, false, true>, grid, kRopeThreads, s, p)
                : launch(rope_kernel<D, false, false>, grid, kRopeThreads, s, p);
}

template <int D>
cudaError_t launch_rope_bwd_dim(const RopeBwdParams& p, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>(p.blocks));
  if (p.interleaved)
    return p.norm ? launch(rope_bwd_kernel<D, true, true>, grid, kRopeThreads, s, p)
                  : launch(rope_bwd_kernel<D, true, false>, grid, kRopeThreads, s, p);
  return p.norm ? launch(rope_bwd_kernel<D, false, true>, grid, kRopeThreads, s, p)
                : launch(rope_bwd_kernel<D, false, false>, grid, kRopeThreads, s, p);
}

}  // namespace

cudaError_t launch_rope(const RopeParams& p, int d, dim3 grid, cudaStream_t s) {
  switch (d) {
    case 32: return launch_rope_dim<32>(p, grid, s);
    case 64: return launch_rope_dim<64>(p, grid, s);
    case 128: return launch_rope_dim<128>(p, grid, s);
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t launch_rope_bwd(const RopeBwdParams& p, int d, cudaStream_t s) {
  cudaError_t e;
  switch (d) {
    case 32: e = launch_rope_bwd_dim<32>(p, s); break;
    case 64: e = launch_rope_bwd_dim<64>(p, s); break;
    case 128: e = launch_rope_bwd_dim<128>(p, s); break;
    default: return cudaErrorInvalidValue;
  }
  if (e != cudaSuccess || !p.norm || (p.dwq == nullptr && p.dwk == nullptr)) return e;
  return launch(rope_dw_kernel, dim3(static_cast<unsigned>(d / 32), 2), 1024, s,
                static_cast<const float*>(p.part), p.blocks, d, p.dwq, p.wq_type, p.dwk, p.wk_type);
}

}  // namespace attn
