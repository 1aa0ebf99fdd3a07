// blocks_tiles.cuh -- attention over selected pages for many query rows, on the tensor
// core's full tiles (tcgen05). Included by long_tiles.cu.
//
// A CTA has 128 rows of one sequence and key head (rows r = n * G + g) and goes over the
// pages that any of its queries selected, 64 keys at a time; two CTAs share a SM, so one's
// products run while the other's softmax does.
//   warps 0-3  softmax, one thread a row (a TMEM lane): whether its query selected the page
//              is a bit in shared memory; rows that did not put zeros into P. Where no row
//              of a warp did, nothing is computed.
//   warp 4     loader: TMA of the pages' keys and values into two-stage rings
//   warp 5     products: S = Q K^T, one stage ahead of O += P V (P as bf16 in TMEM over S)
// Neighbouring queries select much the same pages, so a page is read once for (128 / G)
// queries, and its products serve most rows. What pages those are is worked out by all
// warps for kTileWindow pages of the sequence at a time.
//
// The running maximum is a whole number (log2 units) and moves only when a score passes it
// by more than 8, so O in TMEM is seldom rescaled, and exactly.
#pragma once

namespace attn {
namespace dev {

constexpr int kBlocksThreads = 192, kBlocksKeys = 64, kTileWindow = 512;
constexpr float kBlocksSlack = 8.f;
constexpr uint32_t kBlocksCols = 256;  // TMEM: S_0 [0, 64), S_1 [64, 128) (P over their first 32), O from 128

struct BlocksTiles {
  LongParams p;
  CUtensorMap tm_k;  // 4-D (d, slot, head, page), box (swizzle span, min(page, 64), 1, 1)
  CUtensorMap tm_v;
};

template <int D>
struct BlocksSmem {
  static constexpr int kRow = D >= 64 ? 128 : 64, kChunks = D >= 64 ? D / 64 : 1;
  static constexpr int kChunk = kBlocksKeys * kRow;              // bytes of 64 keys, one swizzle span of channels
  static constexpr int kQ = 128 * D * 2, kKV = kBlocksKeys * D * 2;  // a stage of K, or of V
  static constexpr int kOffK = kQ, kOffV = kOffK + 2 * kKV;
  static constexpr int kBytes = kOffV + 2 * kKV + 1024;
  static constexpr uint32_t kLayout = D >= 64 ? 2u : 4u;
};

struct BlocksLists {
  uint32_t bits[128][kTileWindow / 32];  // of each query of the tile
  uint32_t any[kTileWindow / 32];
  uint16_t page[kTileWindow];            // the pages that have a bit, from the window's first
  int32_t id[kTileWindow];
  uint64_t bars[13];
  uint32_t tmem;
  uint32_t abort;
  int count;
};

struct BlocksBars {
  uint32_t base;
  __device__ uint32_t k_full(int s) const { return base + 8 * s; }
  __device__ uint32_t k_empty(int s) const { return base + 16 + 8 * s; }
  __device__ uint32_t v_full(int s) const { return base + 32 + 8 * s; }
  __device__ uint32_t v_empty(int s) const { return base + 48 + 8 * s; }
  __device__ uint32_t s_full(int s) const { return base + 64 + 8 * s; }
  __device__ uint32_t p_full(int s) const { return base + 80 + 8 * s; }
  __device__ uint32_t o_done() const { return base + 96; }
};

// Stages of a window's list, and what a stage has: pages of 64 slots or more are cut
// into stages, smaller ones fill one together.
struct Stages {
  int page_shift, sub, cut;  // log2 of: pages a stage, stages a page
  __device__ __forceinline__ explicit Stages(int shift) : page_shift(shift), sub(max(6 - shift, 0)), cut(max(shift - 6, 0)) {}
  __device__ __forceinline__ int count(int pages) const { return ((pages << cut) + (1 << sub) - 1) >> sub; }
  __device__ __forceinline__ int entry(int s, int i) const { return ((s >> cut) << sub) + i; }  // i-th page of stage s
  __device__ __forceinline__ int slot(int s) const { return (s & ((1 << cut) - 1)) << 6; }     // first slot of the page(s)
  __device__ __forceinline__ int keys() const { return min(64, 1 << page_shift); }             // slots of a page in a stage
};

// The warps that wait as one vote; false: the CTA is aborting.
__device__ __forceinline__ bool blocks_wait(uint32_t bar, uint32_t parity, const Ctl& c, int tile, bool honour = true) {
  return ctl_wait(bar, parity, c, tile, kRoleTiles, honour);
}

template <int D>
__device__ __forceinline__ bool blocks_load(const BlocksTiles& a, const BlocksLists& l, uint32_t base, const BlocksBars& bars,
                                            const Stages& st, int hk, int n, int& gs, const Ctl& ctl) {
  using S = BlocksSmem<D>;
  const uint64_t pol = l2_policy_evict_last();
  for (int s = 0; s < n; ++s, ++gs) {
    const int slot = gs & 1, at = st.slot(s);
    const uint32_t phase = ((gs >> 1) & 1) ^ 1u;
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      if (!blocks_wait(v ? bars.v_empty(slot) : bars.k_empty(slot), phase, ctl, gs)) return false;
      const uint32_t full = v ? bars.v_full(slot) : bars.k_full(slot);
      mbar_expect_tx(full, S::kKV);
      for (int i = 0; i < (1 << st.sub); ++i) {
        const int e = st.entry(s, i);
        const int id = e < l.count ? l.id[e] : -1;  // (a page that the cache has not reads as zeros)
#pragma unroll
        for (int c = 0; c < S::kChunks; ++c)
          tma_load_4d_hint(base + (v ? S::kOffV : S::kOffK) + slot * S::kKV + c * S::kChunk + i * st.keys() * S::kRow,
                           v ? &a.tm_v : &a.tm_k, full, c * 64, at, hk, id, pol);
      }
    }
  }
  return true;
}

// O += P V of stage x (the window's number xs).
template <int D>
__device__ __forceinline__ bool blocks_pv(const BlocksLists& l, uint8_t* smem, uint32_t base, const BlocksBars& bars,
                                          const Stages& st, uint32_t tmem, int len, int w0, int xs, int x, const Ctl& ctl) {
  using S = BlocksSmem<D>;
  const int slot = x & 1;
  const uint32_t parity = (x >> 1) & 1;
  if (!blocks_wait(bars.v_full(slot), parity, ctl, x)) return false;
  // values behind the sequence's end may be anything: 0 * NaN must not reach the sum
  for (int i = 0; i < (1 << st.sub); ++i) {
    const int e = st.entry(xs, i);
    if (e >= l.count) break;
    const int live = len - ((w0 + l.page[e]) << st.page_shift) - st.slot(xs);
    if (live >= st.keys()) continue;
    const int first = i * st.keys() + max(live, 0), rows = (i + 1) * st.keys() - first;
    for (int y = threadIdx.x & 31; y < rows * (D / 8); y += 32) {
      const int r = first + y / (D / 8), c = y % (D / 8);
      *reinterpret_cast<uint4*>(smem + S::kOffV + slot * S::kKV + (c / (S::kRow / 16)) * S::kChunk + r * S::kRow +
                                (c % (S::kRow / 16)) * 16) = make_uint4(0, 0, 0, 0);
    }
    fence_async_smem();
    __syncwarp();
  }
  if (!blocks_wait(bars.p_full(slot), parity, ctl, x)) return false;
  tc_fence_after();
  constexpr uint32_t kIdesc = make_idesc(128, D, true);
  const uint64_t dv = smem_desc(base + S::kOffV + slot * S::kKV, S::kChunk, 8 * S::kRow, S::kLayout);
  mma_ts4<S::kRow, 2 * S::kRow, 3 * S::kRow>(tmem + 128, tmem + slot * 64, dv, kIdesc, x > 0);
  mma_commit(bars.o_done());
  mma_commit(bars.v_empty(slot));
  return true;
}

template <int D>
__device__ __forceinline__ bool blocks_mma(const BlocksLists& l, uint8_t* smem, uint32_t base, const BlocksBars& bars,
                                           const Stages& st, uint32_t tmem, int len, int w0, int n, int& gs, const Ctl& ctl) {
  using S = BlocksSmem<D>;
  for (int s = 0; s < n; ++s, ++gs) {
    const int slot = gs & 1;
    if (!blocks_wait(bars.k_full(slot), (gs >> 1) & 1, ctl, gs)) return false;
    tc_fence_after();
    // (S goes where stage gs - 2 had its P: that product was issued before, and read it)
    issue_tile<D>(tmem + slot * 64, base, base + S::kOffK + slot * S::kKV);
    mma_commit(bars.s_full(slot));
    mma_commit(bars.k_empty(slot));
    if (s > 0 && !blocks_pv<D>(l, smem, base, bars, st, tmem, len, w0, s - 1, gs - 1, ctl)) return false;
  }
  return blocks_pv<D>(l, smem, base, bars, st, tmem, len, w0, n - 1, gs - 1, ctl);
}

template <int D>
__global__ void __launch_bounds__(kBlocksThreads, 2) blocks_tiles(const __grid_constant__ BlocksTiles a) {
  using S = BlocksSmem<D>;
  const LongParams& p = a.p;
  extern __shared__ uint8_t raw[];
  __shared__ BlocksLists l;
  uint8_t* smem = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
  const uint32_t base = smem_u32(smem);
  const BlocksBars bars{smem_u32(l.bars)};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(bars.k_full(s), 1);
      mbar_init(bars.k_empty(s), 1);
      mbar_init(bars.v_full(s), 1);
      mbar_init(bars.v_empty(s), 1);
      mbar_init(bars.s_full(s), 1);
      mbar_init(bars.p_full(s), 4);
    }
    mbar_init(bars.o_done(), 1);
    l.abort = 0;
    fence_barrier_init();
    prefetch_tmap(&a.tm_k);
    prefetch_tmap(&a.tm_v);
  }
  if (warp == 5) {
    tmem_alloc(smem_u32(&l.tmem), kBlocksCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = l.tmem;
  const Ctl ctl{&l.abort, g_long_status, 2000000000ull};
  ldev::grid_dep_launch();
  ldev::grid_dep_wait();

  const int b = blockIdx.z, hk = blockIdx.y, G = p.G;
  const int all = p.Nq * G, r0 = static_cast<int>(blockIdx.x) * 128, rn = min(all - r0, 128);
  const int tok0 = p.by_g.div(r0), toks = p.by_g.div(r0 + rn - 1) - tok0 + 1;
  const LongLens lens = long_lens(p, b);
  const int live = min(tok0 + toks, lens.ql);  // queries of the tile that are real: [tok0, live)
  const int pages = live > tok0 ? min(long_pages(p, long_seen(p, lens, live - 1)), p.table_width) : 0;
  const int32_t* lists = p.blocks + ((static_cast<int64_t>(b) * p.Hk + hk) * p.Nq + tok0) * p.n;
  const Stages st(p.page_shift);

  // the query rows, and of this thread's (warps 0-3) what it sees
  for (int x = threadIdx.x; x < 128 * (D / 8); x += kBlocksThreads) {
    const int r = x / (D / 8), c = x % (D / 8), n = p.by_g.div(r0 + r), g = r0 + r - n * G;
    ldev::copy16(base + operand_at<D>(r, c, 128),
                 static_cast<const __nv_bfloat16*>(p.q) + b * p.q_sb +
                     (r < rn ? (static_cast<int64_t>(hk) * G + g) * p.q_sh + n * p.q_sn : 0) + c * 8,
                 r < rn ? 16 : 0);
  }
  ldev::copy_commit();
  const int row = static_cast<int>(threadIdx.x), n_mine = p.by_g.div(r0 + min(row, rn - 1)), tok = n_mine - tok0;
  const int seen = row < rn ? long_seen(p, lens, n_mine) : 0;
  float m = -INFINITY, sum = 0.f;
  const uint32_t lanes = static_cast<uint32_t>(warp) << 21;
  int gs = 0;  // stages so far
  bool ok = true;

  for (int w0 = 0; w0 < pages; w0 += kTileWindow) {
    __syncthreads();  // the lists of the window before are done with
    for (int x = threadIdx.x; x < toks * (kTileWindow / 32); x += kBlocksThreads) (&l.bits[0][0])[x] = 0u;
    if (threadIdx.x < kTileWindow / 32) l.any[threadIdx.x] = 0u;
    __syncthreads();
    for (int x = threadIdx.x; x < toks * p.n; x += kBlocksThreads) {
      const int t = x / p.n, page = lists[x] - w0;
      const int most = min(long_pages(p, long_seen(p, lens, tok0 + t)) - w0, kTileWindow);
      if (page >= 0 && page < most) {
        atomicOr(&l.bits[t][page >> 5], 1u << (page & 31));
        atomicOr(&l.any[page >> 5], 1u << (page & 31));
      }
    }
    ldev::copy_wait<0>();
    fence_async_smem();
    __syncthreads();
    if (warp == 0) {  // a lane has 16 pages
      static_assert(kTileWindow == 32 * 16, "half a word of the bits a lane");
      uint32_t mine = (l.any[lane >> 1] >> ((lane & 1) * 16)) & 0xFFFFu, at = __popc(mine);
#pragma unroll
      for (int s = 1; s < 32; s *= 2) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, at, s);
        if (lane >= s) at += y;
      }
      if (lane == 31) l.count = static_cast<int>(at);
      at -= __popc(mine);
      for (; mine != 0u; mine &= mine - 1, ++at) l.page[at] = static_cast<uint16_t>(lane * 16 + __ffs(mine) - 1);
    }
    __syncthreads();
    for (int x = threadIdx.x; x < l.count; x += kBlocksThreads) l.id[x] = p.table[b * p.table_sb + w0 + l.page[x]];
    __syncthreads();
    const int n = st.count(l.count);
    if (n > 0) {
      if (warp == 4) {
        ok = blocks_load<D>(a, l, base, bars, st, hk, n, gs, ctl);
      } else if (warp == 5) {
        ok = blocks_mma<D>(l, smem, base, bars, st, tmem, lens.len, w0, n, gs, ctl);
      } else {
        for (int s = 0; s < n; ++s, ++gs) {
          const int slot = gs & 1;
          // of each 16 columns, how many the row sees: keys of pages that its query selected
          int lim[4];
          bool some = false, even = true;
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const int i = g >> (2 - st.sub), e = st.entry(s, i);  // (sub 0: all of the one page; 1: two; 2: four)
            lim[g] = 0;
            if (e < l.count) {
              const int page = l.page[e];
              const int pos = ((w0 + page) << st.page_shift) + st.slot(s) + (g * 16 - i * st.keys());
              if ((l.bits[tok][page >> 5] >> (page & 31)) & 1u) lim[g] = min(max(seen - pos, 0), 16);
            }
            some |= lim[g] > 0;
            even &= lim[g] == 0 || lim[g] == 16;
          }
          ok = blocks_wait(bars.s_full(slot), (gs >> 1) & 1, ctl, gs);
          if (!ok) break;
          tc_fence_after();
          const uint32_t ts = tmem + lanes + slot * 64;
          uint32_t w[32];
          if (!__any_sync(0xffffffffu, some)) {
#pragma unroll
            for (int x = 0; x < 32; ++x) w[x] = 0u;
          } else {
            uint32_t v[2][32];
            tmem_ld32(ts, v[0]);
            tmem_ld32(ts + 32, v[1]);
            const auto at = [&](int c) -> uint32_t& { return v[c >> 5][c & 31]; };
            if (!__all_sync(0xffffffffu, even)) {
#pragma unroll
              for (int c = 0; c < 64; ++c)
                if ((c & 15) >= lim[c >> 4]) at(c) = 0xFF800000u;
            }
            float top = -INFINITY;
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              float z = __uint_as_float(at(16 * g));
#pragma unroll
              for (int c = 1; c < 15; c += 2) z = fmax3(z, __uint_as_float(at(16 * g + c)), __uint_as_float(at(16 * g + c + 1)));
              z = fmaxf(z, __uint_as_float(at(16 * g + 15)));
              top = fmaxf(top, lim[g] > 0 ? z : -INFINITY);
            }
            top *= p.c_hi;
            if (__any_sync(0xffffffffu, top > m + kBlocksSlack)) {
              const float next = fmaxf(m, ceilf(top));
              const float f = m == next ? 1.f : ex2(m - next);  // (m -inf: 0)
              m = next;
              sum *= f;
              if (gs > 0) {
                ok = blocks_wait(bars.o_done(), (gs - 1) & 1, ctl, gs);
                if (!ok) break;
                tc_fence_after();
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                  uint32_t o[32];
                  tmem_ld32(tmem + lanes + 128 + c, o);
#pragma unroll
                  for (int x = 0; x < 32; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * f);
                  tmem_st32(tmem + lanes + 128 + c, o);
                }
                tmem_wait_st();
              }
            }
            const float neg = m == -INFINITY ? 0.f : -m;
            const ldev::F2 c2 = ldev::pair(p.c_hi, p.c_hi), neg2 = ldev::pair(neg, neg);
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              ldev::F2 part = ldev::pair(0.f, 0.f);
#pragma unroll
              for (int c = 16 * g; c < 16 * g + 16; c += 2) {
                const float2 x = ldev::split(ldev::fma2(ldev::pair(__uint_as_float(at(c)), __uint_as_float(at(c + 1))), c2, neg2));
                const float e0 = ex2(x.x), e1 = ex2(x.y);  // (a score of +inf: inf - inf, NaN)
                part = ldev::add2(part, ldev::pair(e0, e1));
                w[c / 2] = lim[g] > 0 ? pack_bf16(e0, e1) : 0u;
              }
              const float2 y = ldev::split(part);
              sum += lim[g] > 0 ? y.x + y.y : 0.f;
            }
          }
          tmem_st32(ts, w);
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bars.p_full(slot));
        }
      }
    }
    if (__syncthreads_or(!ok)) break;
  }

  if (ok && gs > 0 && warp < 4) {
    ok = blocks_wait(bars.o_done(), (gs - 1) & 1, ctl, gs);
    tc_fence_after();
  }
  if (warp < 4) {
    const int g = r0 + row - n_mine * G, h = hk * G + g;
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.o) + b * p.o_sb + h * p.o_sh + n_mine * p.o_sn;
#pragma unroll 1
    for (int c = 0; c < D; c += 32) {
      uint32_t o[32];
      if (gs > 0) tmem_ld32(tmem + lanes + 128 + c, o);
      if (row < rn) {
#pragma unroll
        for (int x = 0; x < 32; x += 8) {
          uint32_t y[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            y[i] = sum == 0.f ? 0u : pack_bf16(__uint_as_float(o[x + 2 * i]) * inv, __uint_as_float(o[x + 2 * i + 1]) * inv);
          *reinterpret_cast<uint4*>(out + c + x) = make_uint4(y[0], y[1], y[2], y[3]);
        }
      }
    }
    if (row < rn && p.lse != nullptr)
      p.lse[(static_cast<int64_t>(b) * p.Hq + h) * p.Nq + n_mine] = CUDART_LN2_F * (m + log2f(sum));
  }
  if (l.abort != 0u && warp == 4) {
    // copies in flight land in this CTA's shared memory: wait (bounded) for the last ones
    for (int x = max(gs - 1, 0); x <= gs; ++x) {
      blocks_wait(bars.k_full(x & 1), (x >> 1) & 1, ctl, x, false);
      blocks_wait(bars.v_full(x & 1), (x >> 1) & 1, ctl, x, false);
    }
  }
  ldev::copy_wait<0>();  // (no page, no wait so far)
  tc_fence_before();
  __syncthreads();
  if (warp == 5) tmem_dealloc(tmem, kBlocksCols);
}

template <int D>
cudaError_t blocks_tiles_dim(const BlocksTiles& a, cudaStream_t s) {
  const int64_t rows = static_cast<int64_t>(a.p.Nq) * a.p.G;
  const cudaError_t e =
      cudaFuncSetAttribute(blocks_tiles<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, BlocksSmem<D>::kBytes);
  if (e != cudaSuccess) return e;
  return ldev::launch(blocks_tiles<D>, dim3(static_cast<unsigned>((rows + 127) / 128), a.p.Hk, a.p.B), kBlocksThreads,
                      static_cast<size_t>(BlocksSmem<D>::kBytes), s, 1, a);
}

}  // namespace dev
}  // namespace attn
