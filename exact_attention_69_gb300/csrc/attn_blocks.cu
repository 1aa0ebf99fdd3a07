// attn_blocks.cu -- attention of each query over the pages that it selected.
//
// Rows r = n * G + g of one sequence and key head (G query heads share it) go in tiles
// of 8 or 16. A tile reads every page that one of its queries selected once: a bit per
// page and query in shared memory, then the list of pages that have a bit, with the
// queries' bits beside them; a score counts only where the row's query has the bit.
// Products are computed transposed, S^T = K Q^T and O^T = V^T P^T, so that 16 keys (or 16
// channels) fill the matrix instruction's long side and 8 rows its short one: for a few
// rows half the work of the other order. K and V go from global memory to registers
// that are the instruction's operands; nothing is staged. Each warp takes every
// (warps)-th group of 16 keys with a running maximum and sum of its own; the warps' parts
// are joined in shared memory, and those of the CTAs that share a tile, which are a
// cluster, through each other's shared memory: one launch, no workspace, a fixed order.
//
// One or two tokens are bound by memory: 32 sequences x 8 key heads x 32 pages of 64, d = 128
// (269 MB) take 45.3 us, 5.9 TB/s. (In four warps a CTA and up to three CTAs a SM 53 us, with
// two CTAs a tile 64: a CTA's start, some 3 us of lists and first loads, weighs more.)
// Few pages are a chain of latencies: 5.6 us for 16 pages of 16 slots (6.6 with the list of
// one query made into bits first; 6.9 and 15.1 where 32 pages lie among 4096).
//
// The running maximum is a whole number (log2 units) and moves only when a score
// passes it by more than 8: weights stay below 2^8 and rescaling is exact. Weights go into
// the second product as two bf16 parts, 16 bits of each: memory sets the pace, so the second
// half of the products is free, and what is left of the error against 64 bits is the
// output's rounding (one part: 0.0026 of O's norm for rows of few keys, two: 0.0016).
#include <math_constants.h>

#include "long_dev.cuh"
#include "long_kernel.h"

namespace attn {
namespace {

using namespace ldev;

constexpr int kWindow = 1024;  // pages that the bits cover at a time
constexpr int kListThreads = kWindow / 8;  // threads that list them, a byte of the bits each
constexpr float kSlack = 8.f;

// Parts of a row: maxima (log2 units) and sums first, then the weighted values in order.
template <int N>
struct Part {
  float2 ml[N];
  float m, base, sum;
  float4 acc;
  __device__ __forceinline__ void top() {
    m = -INFINITY;
#pragma unroll
    for (int w = 0; w < N; ++w) m = fmaxf(m, ml[w].x);
    base = m == -INFINITY ? 0.f : m;
    sum = 0.f;
    acc = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  __device__ __forceinline__ void add(int w, float4 v) {
    const float f = ex2(ml[w].x - base);
    sum += f * ml[w].y;
    acc.x += f * v.x;
    acc.y += f * v.y;
    acc.z += f * v.z;
    acc.w += f * v.w;
  }
};

struct Entry {
  int block, id;
};

template <int D, int NT>
struct Shared {
  static constexpr int kRows = 8 * NT, kBlocksWarps = blocks_warps(NT);
  struct Lists {
    uint32_t bits[kRows][kWindow / 32];
    Entry entry[kWindow];
    uint16_t who[kWindow];
    int32_t table[kWindow];
    uint32_t sums[kListThreads / 32];
    int next;
  };
  struct Join {
    float o[kBlocksWarps][kRows][D];  // (the first also takes the joined part)
    float2 ml[kBlocksWarps][kRows];
    float2 part[kRows];
  };
  union {
    Lists l;
    Join j;
  };
};

template <int D, int NT>
__global__ void __launch_bounds__(32 * blocks_warps(NT), 2) blocks_kernel(const __grid_constant__ LongParams p) {
  constexpr int kRows = 8 * NT, kC = D / 32, kM = D / 16, kBlocksWarps = blocks_warps(NT), kThreads = 32 * kBlocksWarps;
  constexpr int kVec = D == 32 ? 4 : 8;           // neighbouring channels that a lane takes of V
  constexpr int kVC = D == 128 ? 2 : 1;           // such runs
  extern __shared__ __align__(16) unsigned char smem[];
  Shared<D, NT>& sh = *reinterpret_cast<Shared<D, NT>*>(smem);
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, i = lane >> 2, j = lane & 3;
  const int rows = p.Nq * p.G, tiles = (rows + kRows - 1) / kRows;
  const int split = blockIdx.x % p.splits, tile = blockIdx.x / p.splits % tiles;
  const int hk = blockIdx.y, b = blockIdx.z;
  const int r0 = tile * kRows, rn = min(rows - r0, kRows);
  const int tok0 = r0 / p.G, toks = (r0 + rn - 1) / p.G - tok0 + 1;
  const LongLens lens = long_lens(p, b);
  const int32_t* lists = p.blocks + ((static_cast<int64_t>(b) * p.Hk + hk) * p.Nq + tok0) * p.n;
  const int page_mask = (1 << p.page_shift) - 1;

  // this lane's rows (columns 2 j, 2 j + 1 of each group), what they see, and Q
  int seen[2 * NT];
  uint32_t bit[2 * NT];
  uint32_t qf[NT][kC][4];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int r = 8 * t + 2 * j + x;
      const int n = (r0 + r) / p.G;
      seen[2 * t + x] = r < rn ? long_seen(p, lens, n) : 0;
      bit[2 * t + x] = r < rn ? 1u << (n - tok0) : 0u;
    }
    const int r = min(8 * t + i, rn - 1), n = (r0 + r) / p.G, g = r0 + r - n * p.G;
    const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q) + b * p.q_sb +
                             (static_cast<int64_t>(hk) * p.G + g) * p.q_sh + n * p.q_sn + j * 8;
#pragma unroll
    for (int c = 0; c < kC; ++c) *reinterpret_cast<uint4*>(qf[t][c]) = ld16(q + c * 32);
  }

  float o[NT][kM][4];
  float m[2 * NT], l[2 * NT];
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int c = 0; c < kM; ++c)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[t][c][e] = 0.f;
#pragma unroll
  for (int x = 0; x < 2 * NT; ++x) {
    m[x] = -INFINITY;
    l[x] = 0.f;
  }

  const int pages = min(long_pages(p, long_seen(p, lens, min(tok0 + toks, lens.ql) - 1)), p.table_width);
  const __nv_bfloat16* kbase = static_cast<const __nv_bfloat16*>(p.kc) + hk * p.kc_sh + j * 8;
  const __nv_bfloat16* vbase = static_cast<const __nv_bfloat16*>(p.vc) + hk * p.vc_sh + i * kVec;
  const int shift = p.page_shift - 4;             // groups of 16 keys a page
  const int workers = kBlocksWarps * p.splits, me = split * kBlocksWarps + warp;

  const int total = lens.ql > tok0 ? pages : 0;
  // One query's short list is taken as it is, longer ones and several window by window. (In tiles
  // of 16 rows all: the branch took 0.4 us of 8.5 from calls of several queries there.)
  const bool direct = NT == 1 && toks == 1 && p.n <= kListThreads;
  const int head = static_cast<int>(threadIdx.x) < toks * p.n ? lists[threadIdx.x] : -1;  // this thread's first entry
  int next = total;  // first page of the next window that has a bit
  for (int w0 = 0; w0 < total; w0 = next) {
    __syncthreads();
    uint32_t mine = 0, at = 0;  // pages that this thread lists: bits from `from` on
    int from = 0, id = -1;
    if (direct) {
      const int x = threadIdx.x;
      int page = head;
      if (page >= total) page = -1;
      if (x < kListThreads) sh.l.table[x] = page;
      if (page >= 0) id = p.table[b * p.table_sb + page];
      __syncthreads();
      bool take = page >= 0;  // (named before: counted once)
      for (int e = 0; e < p.n; ++e) take &= e >= x || sh.l.table[e] != page;
      mine = take ? 1u : 0u;
      from = page;
    } else {
      for (int x = threadIdx.x; x < kRows * (kWindow / 32); x += kThreads) (&sh.l.bits[0][0])[x] = 0u;
      if (threadIdx.x == 0) sh.l.next = total;
      for (int x = threadIdx.x; x < min(kWindow, pages - w0); x += kThreads)
        sh.l.table[x] = p.table[b * p.table_sb + w0 + x];
      __syncthreads();
      for (int x = threadIdx.x; x < toks * p.n; x += kThreads) {
        const int t = x / p.n, page = x == static_cast<int>(threadIdx.x) ? head : lists[x];
        if (page < w0 || page >= long_pages(p, long_seen(p, lens, tok0 + t))) continue;
        if (page < w0 + kWindow)
          atomicOr(&sh.l.bits[t][(page - w0) >> 5], 1u << ((page - w0) & 31));
        else
          atomicMin(&sh.l.next, page);
      }
      __syncthreads();
      next = sh.l.next & ~31;  // (a multiple of 32, as all windows' first pages; total: the loop ends)
      if (sh.l.next == total) next = total;
      if (threadIdx.x < kListThreads) {  // 8 pages a thread
        from = threadIdx.x * 8;
        for (int t = 0; t < toks; ++t) mine |= sh.l.bits[t][from >> 5];
        mine = (mine >> (from & 31)) & 255u;
      }
    }
    // the pages that have a bit, in order
    const uint32_t n_mine = __popc(mine);
    if (threadIdx.x < kListThreads) {
      at = n_mine;
#pragma unroll
      for (int s = 1; s < 32; s *= 2) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, at, s);
        if (lane >= s) at += y;
      }
      if (lane == 31) sh.l.sums[warp] = at;
    }
    __syncthreads();
    int count = 0;
    at -= n_mine;
#pragma unroll
    for (int s = 0; s < kListThreads / 32; ++s) {
      if (s < warp) at += sh.l.sums[s];
      count += sh.l.sums[s];
    }
    if (direct) {
      if (mine != 0u) {
        sh.l.entry[at] = Entry{from, id};
        sh.l.who[at] = 1;
      }
    } else {
      for (; mine != 0u; mine &= mine - 1, ++at) {
        const int page = from + __ffs(mine) - 1;
        uint32_t who = 0;
        for (int t = 0; t < toks; ++t) who |= ((sh.l.bits[t][page >> 5] >> (page & 31)) & 1u) << t;
        sh.l.entry[at] = Entry{w0 + page, sh.l.table[page]};
        sh.l.who[at] = static_cast<uint16_t>(who);
      }
    }
    __syncthreads();

    // groups of 16 keys, each warp every workers-th
    const int units = count << shift;
    uint4 kf[2][kC];
    uint32_t vf[4][kVC][kVec / 2];
    const auto load_k = [&](int u) {
      const Entry e = sh.l.entry[u >> shift];
      const int slot = ((u & ((1 << shift) - 1)) << 4) + i;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const bool live = e.id >= 0 && e.id < p.n_pages && (e.block << p.page_shift) + slot + 8 * h < lens.len;
        const __nv_bfloat16* k = kbase + e.id * p.kc_sp + ((slot + 8 * h) & page_mask) * p.kc_st;
#pragma unroll
        for (int c = 0; c < kC; ++c) kf[h][c] = live ? ld16(k + c * 32) : make_uint4(0, 0, 0, 0);
      }
    };
    // keys 2 j, 2 j + 1, 2 j + 8, 2 j + 9 of the group; zeros behind the sequence's end,
    // where a page may hold anything
    const auto load_v = [&](int u) {
      const Entry e = sh.l.entry[u >> shift];
      const int slot = ((u & ((1 << shift) - 1)) << 4) + 2 * j;
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        const int s = slot + (h & 1) + 8 * (h >> 1);
        const bool live = e.id >= 0 && e.id < p.n_pages && (e.block << p.page_shift) + s < lens.len;
        const __nv_bfloat16* v = vbase + e.id * p.vc_sp + s * p.vc_st;
#pragma unroll
        for (int c = 0; c < kVC; ++c) {
          if constexpr (kVec == 8)
            *reinterpret_cast<uint4*>(vf[h][c]) = live ? ld16(v + c * 64) : make_uint4(0, 0, 0, 0);
          else
            *reinterpret_cast<uint2*>(vf[h][c]) = live ? ld8(v) : make_uint2(0, 0);
        }
      }
    };
    int u = me;
    if (u < units) {
      load_k(u);
      load_v(u);
    }
    for (; u < units; u += workers) {
      float s[NT][4];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        s[t][0] = s[t][1] = s[t][2] = s[t][3] = 0.f;
#pragma unroll
        for (int c = 0; c < kC; ++c) {
          mma(s[t], kf[0][c].x, kf[1][c].x, kf[0][c].y, kf[1][c].y, qf[t][c][0], qf[t][c][1]);
          mma(s[t], kf[0][c].z, kf[1][c].z, kf[0][c].w, kf[1][c].w, qf[t][c][2], qf[t][c][3]);
        }
      }
      const Entry e = sh.l.entry[u >> shift];
      const uint32_t who = sh.l.who[u >> shift];
      const int key = (e.block << p.page_shift) + ((u & ((1 << shift) - 1)) << 4) + i;
      if (u + workers < units) load_k(u + workers);
      // s[t][0], s[t][1]: key i, rows 2 j and 2 j + 1; s[t][2], s[t][3]: key i + 8
      bool grow = false;
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int r = 2 * t + (x & 1);
          const bool sees = (who & bit[r]) != 0u && key + (x >> 1) * 8 < seen[r];
          s[t][x] = sees ? s[t][x] * p.c_hi : -INFINITY;
          grow |= s[t][x] > m[r] + kSlack;  // (m -inf: any score above -inf)
        }
      if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int r = 2 * t + x;
            float top = fmaxf(s[t][x], s[t][x + 2]);
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
            top = fmaxf(m[r], ceilf(top));
            const float f = m[r] == top ? 1.f : ex2(m[r] - top);  // (m -inf: 0)
            m[r] = top;
            l[r] *= f;
#pragma unroll
            for (int c = 0; c < kM; ++c) {
              o[t][c][x] *= f;
              o[t][c][x + 2] *= f;
            }
          }
      }
      uint32_t pf[NT][2], pl[NT][2];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int r = 2 * t + (x & 1);
          const float base = m[r] == -INFINITY ? 0.f : m[r];
          s[t][x] = ex2(s[t][x] - base);  // a score of +inf: inf - inf, NaN
          l[r] += s[t][x];
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const uint32_t hi = pack_bf16(s[t][2 * x], s[t][2 * x + 1]);
          pf[t][x] = transpose8(hi);
          pl[t][x] = transpose8(pack_bf16(s[t][2 * x] - __uint_as_float(hi << 16), s[t][2 * x + 1] - __uint_as_float(hi & 0xFFFF0000u)));
        }
      }
#pragma unroll
      for (int c = 0; c < kVC; ++c)
#pragma unroll
        for (int w = 0; w < kVec / 2; ++w) {
          const uint32_t a0 = __byte_perm(vf[0][c][w], vf[1][c][w], 0x5410), a1 = __byte_perm(vf[0][c][w], vf[1][c][w], 0x7632);
          const uint32_t a2 = __byte_perm(vf[2][c][w], vf[3][c][w], 0x5410), a3 = __byte_perm(vf[2][c][w], vf[3][c][w], 0x7632);
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            mma(o[t][c * (kVec / 2) + w], a0, a1, a2, a3, pf[t][0], pf[t][1]);
            mma(o[t][c * (kVec / 2) + w], a0, a1, a2, a3, pl[t][0], pl[t][1]);
          }
        }
      if (u + workers < units) load_v(u + workers);
    }
  }

  // the warps' parts: rows 2 j, 2 j + 1; channels i * kVec + 2 w, + 1 of run c
  __syncthreads();
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int r = 8 * t + 2 * j + x;
      float z = l[2 * t + x];
      z += __shfl_xor_sync(0xffffffffu, z, 4);
      z += __shfl_xor_sync(0xffffffffu, z, 8);
      z += __shfl_xor_sync(0xffffffffu, z, 16);
      if (i == 0) sh.j.ml[warp][r] = make_float2(m[2 * t + x], z);
#pragma unroll
      for (int c = 0; c < kVC; ++c)
#pragma unroll
        for (int w = 0; w < kVec / 2; ++w)
          *reinterpret_cast<float2*>(&sh.j.o[warp][r][c * 64 + i * kVec + 2 * w]) =
              make_float2(o[t][c * (kVec / 2) + w][x], o[t][c * (kVec / 2) + w][x + 2]);
    }
  __syncthreads();
  const auto store = [&](int r, int c, float top, float sum, float4 acc) {
    const int n = (r0 + r) / p.G, h = hk * p.G + r0 + r - n * p.G;
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.o) + b * p.o_sb + h * p.o_sh + n * p.o_sn + c) =
        make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
    if (c == 0 && p.lse != nullptr)
      p.lse[(static_cast<int64_t>(b) * p.Hq + h) * p.Nq + n] = CUDART_LN2_F * (top + log2f(sum));
  };
  for (int x = threadIdx.x; x < rn * (D / 4); x += kThreads) {
    const int r = x / (D / 4), c = (x % (D / 4)) * 4;
    Part<kBlocksWarps> all;
#pragma unroll
    for (int w = 0; w < kBlocksWarps; ++w) all.ml[w] = sh.j.ml[w][r];
    all.top();
#pragma unroll
    for (int w = 0; w < kBlocksWarps; ++w) all.add(w, *reinterpret_cast<const float4*>(&sh.j.o[w][r][c]));
    if (p.splits == 1) {
      store(r, c, all.m, all.sum, all.acc);
    } else {
      *reinterpret_cast<float4*>(&sh.j.o[0][r][c]) = all.acc;
      if (c == 0) sh.j.part[r] = make_float2(all.m, all.sum);
    }
  }
  if (p.splits == 1) return;
  cluster_sync();
  for (int x = split * kThreads + threadIdx.x; x < rn * (D / 4); x += p.splits * kThreads) {
    const int r = x / (D / 4), c = (x % (D / 4)) * 4;
    const uint32_t ml_at = smem_addr(&sh.j.part[r]), o_at = smem_addr(&sh.j.o[0][r][c]);
    Part<kBlocksMaxSplits> all;
#pragma unroll
    for (int w = 0; w < kBlocksMaxSplits; ++w)
      all.ml[w] = w < p.splits ? peer_f2(ml_at, w) : make_float2(-INFINITY, 0.f);
    all.top();
#pragma unroll
    for (int w = 0; w < kBlocksMaxSplits; ++w)
      if (w < p.splits) all.add(w, peer_f4(o_at, w));
    store(r, c, all.m, all.sum, all.acc);
  }
  cluster_sync();  // (no CTA leaves while another reads its part)
}

template <int D, int NT>
cudaError_t blocks_dim(const LongParams& p, cudaStream_t s) {
  constexpr int kRows = 8 * NT;
  const int64_t rows = static_cast<int64_t>(p.Nq) * p.G, tiles = (rows + kRows - 1) / kRows;
  const dim3 grid(static_cast<unsigned>(tiles * p.splits), p.Hk, p.B);
  constexpr size_t kSmem = sizeof(Shared<D, NT>);
  static_assert(kSmem <= 48 * 1024, "no opt-in needed");
  return launch(blocks_kernel<D, NT>, grid, 32 * blocks_warps(NT), kSmem, s, p.splits, p);
}

}  // namespace

cudaError_t launch_blocks(const LongParams& p, int d, cudaStream_t s) {
  const bool one = blocks_tile_rows(static_cast<int64_t>(p.Nq) * p.G) == 8;
  switch (d) {
    case 32: return one ? blocks_dim<32, 1>(p, s) : blocks_dim<32, 2>(p, s);
    case 64: return one ? blocks_dim<64, 1>(p, s) : blocks_dim<64, 2>(p, s);
    case 128: return one ? blocks_dim<128, 1>(p, s) : blocks_dim<128, 2>(p, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace attn
