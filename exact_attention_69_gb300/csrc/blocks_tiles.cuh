// blocks_tiles.cuh -- attention over selected pages for many query rows, on the tensor
// core's full tiles (tcgen05). Included by long_tiles.cu.
//
// A CTA has 128 rows of one sequence and key head (rows r = n * G + g) and goes over the
// pages that any of its queries selected, 64 keys at a time; two CTAs share a SM, so one's
// products run while the other's softmax does.
//   warps 0-3  softmax, one thread a row (a TMEM lane). Whether the row's query selected the
//              stage's page is a bit; rows that did not put zeros into P, and where no row
//              of a warp did, nothing is computed.
//   warp 4, 6  loaders of keys and of values: TMA of the pages into two-stage rings
//   warp 5     products: S = Q K^T, one stage ahead of O += P V (P as bf16 in TMEM over S)
// Neighbouring queries select much the same pages, so a page is read once for (128 / G)
// queries, and its products serve most rows. What pages those are is worked out by all
// warps for a window of the sequence at a time. Where tiles are few, the CTAs of a cluster share
// a window's stages and join through each other's shared memory: one launch, a fixed order.
//
// What bounds it is a stage's chain: S, softmax, P V, some 1200 cycles for a CTA alone, 1800
// for two of them on a SM, and around it the lists and the join; 512 queries x 32 heads of two
// sequences, half of them padding, 32 pages of 64 each, d = 128: 44 us (59 by one CTA a tile: 16
// stages on average, but 68 for the longest; 124 by tiles of 16 rows). What made it shorter:
// which pages a row selected as a register word in the list's order rather than three
// dependent reads of shared memory a stage (600 cycles), S read once, loaders of keys and
// values apart.
//
// CTAs of a cluster wait for each other with their TMEM allocated. Registers let no more than
// two CTAs of these kernels into a SM, 512 columns in all, so none of them waits for TMEM that
// another cluster holds; other kernels that hold some wait for no other CTA.
//
// The running maximum is a whole number (log2 units) and moves only when a score passes it
// by more than 8, so O in TMEM is seldom rescaled, and exactly. P is rounded to bf16 once
// (the tensor core's input type; the sum takes the unrounded values): against 64 bits O is off
// by 0.0023 of its norm, the rounding of the output alone is 0.0017. A second part of P, as the
// form for few rows has it (which a caller may ask for), takes the 0.0023 to 0.0017 and 43.5 us to
// 50.6 (512 queries as above; 62 to 79 without padding): some 190 more instructions a stage and thread.
#pragma once

namespace attn {
namespace dev {

constexpr int kBlocksThreads = 224, kBlocksKeys = 64;
constexpr int kWindowMost = 1024, kWindowBits = 256 * 128;  // pages of a window: 256, for fewer queries more
constexpr int kWarpK = 4, kWarpMma = 5, kWarpV = 6;
constexpr float kBlocksSlack = 8.f;
constexpr uint64_t kLateNs = 2000000;  // inject -1 (more than a few polls of a wait, which park for 0.2 ms at most)
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
  static_assert(4 * kKV == 128 * D * 4, "a part of O takes the place of K and V");
};

struct BlocksLists {
  uint32_t bits[kWindowBits / 32];  // of each query of the tile: pages of the window that it selected,
  uint32_t took[kWindowBits / 32];  // and, of the pages listed, which those are
  uint32_t any[kWindowMost / 32];
  uint16_t page[kWindowMost];       // the pages that have a bit, from the window's first
  int32_t id[kWindowMost];
  uint64_t bars[15];
  uint32_t tmem;
  uint32_t abort;
  int count;
  int next;  // the first page behind the window that a query selected
};

struct BlocksBars {
  uint32_t base;
  __device__ uint32_t k_full(int s) const { return base + 8 * s; }
  __device__ uint32_t k_empty(int s) const { return base + 16 + 8 * s; }
  __device__ uint32_t v_full(int s) const { return base + 32 + 8 * s; }
  __device__ uint32_t v_empty(int s) const { return base + 48 + 8 * s; }
  __device__ uint32_t s_full(int s) const { return base + 64 + 8 * s; }
  __device__ uint32_t p_full(int s) const { return base + 80 + 8 * s; }
  // (two, for the stages in turn: S of a stage goes ahead of the product of the stage before, so a
  // row that is through with its last stage waits for the last product but one as well, and a
  // parity tells a phase from the next one, not from the one after it)
  __device__ uint32_t o_done(int s) const { return base + 96 + 8 * s; }
  __device__ uint32_t done() const { return base + 112; }  // every product
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

// Keys (VALUES: values) of stages [first, end) of a window. One warp each: a stage's keys are done with
// earlier than its values, and the next ones need not wait for these.
template <int D, bool VALUES>
__device__ __forceinline__ bool blocks_load(const BlocksTiles& a, const BlocksLists& l, uint32_t base, const BlocksBars& bars,
                                            const Stages& st, int hk, int first, int end, int& gs, const Ctl& ctl) {
  using S = BlocksSmem<D>;
  const uint64_t pol = l2_policy_evict_last();
  for (int s = first; s < end; ++s, ++gs) {
    const int slot = gs & 1, at = st.slot(s);
    if (!blocks_wait(VALUES ? bars.v_empty(slot) : bars.k_empty(slot), ((gs >> 1) & 1) ^ 1u, ctl, gs)) return false;
    const uint32_t full = VALUES ? bars.v_full(slot) : bars.k_full(slot);
    if (!VALUES && gs == 0 && a.p.inject == 1) continue;
    if (VALUES && a.p.inject == -1) {  // (long after the stage's softmax is through)
      for (const uint64_t t0 = global_ns(); global_ns() - t0 < kLateNs;) {
      }
    }
    mbar_expect_tx(full, S::kKV);
    for (int i = 0; i < (1 << st.sub); ++i) {
      const int e = st.entry(s, i);
      const int id = e < l.count ? l.id[e] : -1;  // (a page that the cache has not reads as zeros)
#pragma unroll
      for (int c = 0; c < S::kChunks; ++c)
        tma_load_4d_hint(base + (VALUES ? S::kOffV : S::kOffK) + slot * S::kKV + c * S::kChunk + i * st.keys() * S::kRow,
                         VALUES ? &a.tm_v : &a.tm_k, full, c * 64, at, hk, id, pol);
    }
  }
  return true;
}

// What the warp that issues the products keeps from stage to stage.
template <int D>
struct BlocksMma {
  using S = BlocksSmem<D>;
  uint64_t q, k, v;  // descriptors of Q and of stage 0 of K and V
  uint32_t tmem;
  static constexpr uint64_t kStep = S::kKV >> 4;
  __device__ __forceinline__ BlocksMma(uint32_t base, uint32_t tmem_)
      : q(smem_desc(base, 16, 8 * S::kRow, S::kLayout)),
        k(smem_desc(base + S::kOffK, 16, 8 * S::kRow, S::kLayout)),
        v(smem_desc(base + S::kOffV, S::kChunk, 8 * S::kRow, S::kLayout)),
        tmem(tmem_) {}
  __device__ __forceinline__ void scores(int slot) const {
    constexpr uint32_t kIdesc = make_idesc(128, kBlocksKeys, false);
    const uint64_t ks = k + slot * kStep;
    if constexpr (D == 32) {
      mma_ss2<2>(tmem + slot * 64, q, ks, kIdesc, 0u);
    } else {
      mma_ss4<2, 4, 6>(tmem + slot * 64, q, ks, kIdesc, 0u);
      if constexpr (D == 128)
        mma_ss4<2, 4, 6>(tmem + slot * 64, q + (128 * S::kRow >> 4), ks + (S::kChunk >> 4), kIdesc, 1u);
    }
  }
  __device__ __forceinline__ void values(int slot, bool more) const {
    constexpr uint32_t kIdesc = make_idesc(128, D, true);
    mma_ts4<S::kRow, 2 * S::kRow, 3 * S::kRow>(tmem + 128, tmem + slot * 64, v + slot * kStep, kIdesc, more);
  }
};

// Zeroes the values of stage s that lie behind the sequence's end, where a page may hold
// anything: 0 * NaN must not reach the sum.
template <int D>
__device__ __noinline__ void blocks_clear(const BlocksLists& l, uint8_t* values, int page_shift, int len, int w0, int s) {
  using S = BlocksSmem<D>;
  const Stages st(page_shift);
  for (int i = 0; i < (1 << st.sub); ++i) {
    const int e = st.entry(s, i);
    if (e >= l.count) break;
    const int live = len - ((w0 + l.page[e]) << st.page_shift) - st.slot(s);
    const int first = i * st.keys() + min(max(live, 0), st.keys()), rows = (i + 1) * st.keys() - first;
    for (int y = threadIdx.x & 31; y < rows * (D / 8); y += 32) {
      const int r = first + y / (D / 8), c = y % (D / 8);
      *reinterpret_cast<uint4*>(values + (c / (S::kRow / 16)) * S::kChunk + r * S::kRow + (c % (S::kRow / 16)) * 16) =
          make_uint4(0, 0, 0, 0);
    }
  }
  fence_async_smem();
  __syncwarp();
}

// The products of stages [first, end): S of one, then O += P V of the one before.
template <int D>
__device__ __forceinline__ bool blocks_mma(const BlocksMma<D>& mm, const BlocksLists& l, uint8_t* smem, const BlocksBars& bars,
                                           const Stages& st, int len, int w0, int first, int end, int& gs,
                                           const Ctl& ctl) {
  using S = BlocksSmem<D>;
  // only the last page listed can hold slots behind the sequence's end
  const int last = l.count - 1, dead = ((w0 + l.page[last] + 1) << st.page_shift) > len ? (last << st.cut) >> st.sub : end;
  for (int s = first; s <= end; ++s) {
    if (s < end) {
      const int slot = gs & 1;
      if (!blocks_wait(bars.k_full(slot), (gs >> 1) & 1, ctl, gs)) return false;
      tc_fence_after();
      // (S goes where stage gs - 2 had its P: that product was issued before, and read it)
      mm.scores(slot);
      mma_commit(bars.s_full(slot));
      mma_commit(bars.k_empty(slot));
      ++gs;
    }
    if (s > first) {
      const int x = gs - 1 - (s < end), slot = x & 1;
      const uint32_t parity = (x >> 1) & 1;
      if (!blocks_wait(bars.v_full(slot), parity, ctl, x)) return false;
      if (s - 1 >= dead) blocks_clear<D>(l, smem + S::kOffV + slot * S::kKV, st.page_shift, len, w0, s - 1);
      if (!blocks_wait(bars.p_full(slot), parity, ctl, x)) return false;
      tc_fence_after();
      mm.values(slot, x > 0);
      mma_commit(bars.o_done(slot));
      mma_commit(bars.v_empty(slot));
    }
  }
  return true;
}

// Columns [0, 32) and [32, 64) from an address on, one wait for both.
__device__ __forceinline__ void tmem_ld32x2(uint32_t ta, uint32_t (&a)[32], uint32_t (&b)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%64];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, "
      "%46, %47, %48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, [%65];\n\t"
      "tcgen05.wait::ld.sync.aligned;\n"
      : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3]), "=r"(a[4]), "=r"(a[5]), "=r"(a[6]), "=r"(a[7]), "=r"(a[8]),
        "=r"(a[9]), "=r"(a[10]), "=r"(a[11]), "=r"(a[12]), "=r"(a[13]), "=r"(a[14]), "=r"(a[15]), "=r"(a[16]),
        "=r"(a[17]), "=r"(a[18]), "=r"(a[19]), "=r"(a[20]), "=r"(a[21]), "=r"(a[22]), "=r"(a[23]), "=r"(a[24]),
        "=r"(a[25]), "=r"(a[26]), "=r"(a[27]), "=r"(a[28]), "=r"(a[29]), "=r"(a[30]), "=r"(a[31]), "=r"(b[0]),
        "=r"(b[1]), "=r"(b[2]), "=r"(b[3]), "=r"(b[4]), "=r"(b[5]), "=r"(b[6]), "=r"(b[7]), "=r"(b[8]), "=r"(b[9]),
        "=r"(b[10]), "=r"(b[11]), "=r"(b[12]), "=r"(b[13]), "=r"(b[14]), "=r"(b[15]), "=r"(b[16]), "=r"(b[17]),
        "=r"(b[18]), "=r"(b[19]), "=r"(b[20]), "=r"(b[21]), "=r"(b[22]), "=r"(b[23]), "=r"(b[24]), "=r"(b[25]),
        "=r"(b[26]), "=r"(b[27]), "=r"(b[28]), "=r"(b[29]), "=r"(b[30]), "=r"(b[31])
      : "r"(ta), "r"(ta + 32u)
      : "memory");
}

// What a softmax thread keeps of its row.
struct BlocksRow {
  uint32_t tl;      // TMEM address of its lane
  const uint32_t* took;  // of its query, in shared memory
  int seen;         // slots that it sees
  float c;          // scale * log2(e)
  float m, sum;     // running maximum and sum
  uint32_t word;    // of the 32 pages listed from a multiple of 32 on, which the query selected
};

// How many of 16 columns, from slot `pos` of the sequence on, the row sees.
__device__ __forceinline__ uint32_t blocks_limit(int seen, int pos) { return static_cast<uint32_t>(min(max(seen - pos, 0), 16)); }

// The row of O times f.
template <int D>
__device__ __noinline__ void blocks_rescale(uint32_t to, float f) {
#pragma unroll 1
  for (int c = 0; c < D; c += 32) {
    uint32_t o[32];
    tmem_ld32(to + c, o);
#pragma unroll
    for (int x = 0; x < 32; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * f);
    tmem_st32(to + c, o);
  }
  tmem_wait_st();
}

// One stage of a row's softmax: S to P, the running maximum and sum.
template <int D>
__device__ __forceinline__ bool blocks_softmax(const BlocksLists& l, const BlocksBars& bars, const Stages& st, int w0, int s, int gs,
                                               BlocksRow& r, const Ctl& ctl) {
  const int slot = gs & 1;
  const uint32_t ts = r.tl + slot * 64;
  // of each 16 columns, how many the row sees: keys of pages that its query selected
  uint32_t lim[4] = {0u, 0u, 0u, 0u};
  if (st.sub == 0) {  // one page
    const int e = s >> st.cut;
    if ((e & 31) == 0) r.word = r.took[e >> 5];
    if ((r.word >> (e & 31)) & 1u) {
      const int pos = ((w0 + l.page[e]) << st.page_shift) + st.slot(s);
#pragma unroll
      for (int g = 0; g < 4; ++g) lim[g] = blocks_limit(r.seen, pos + 16 * g);
    }
  } else {  // two or four (their bits lie in one word)
    const int e0 = s << st.sub, left = l.count - e0;
    const uint32_t took = r.took[e0 >> 5] >> (e0 & 31);
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int i = g >> (2 - st.sub);
      if (i < left && ((took >> i) & 1u) != 0u)
        lim[g] = blocks_limit(r.seen, ((w0 + l.page[e0 + i]) << st.page_shift) + g * 16 - i * st.keys());
    }
  }
  const uint32_t some = lim[0] | lim[1] | lim[2] | lim[3];
  if (!blocks_wait(bars.s_full(slot), (gs >> 1) & 1, ctl, gs)) return false;
  tc_fence_after();
  uint32_t w[32];
  if (__any_sync(0xffffffffu, some != 0u)) {
    uint32_t v[2][32];
    tmem_ld32x2(ts, v[0], v[1]);
    if (__any_sync(0xffffffffu, (some & 15u) != 0u)) {  // (else each 16 are seen whole, or not at all)
#pragma unroll
      for (int x = 0; x < 64; ++x)
        if ((x & 15) >= lim[x >> 4]) v[x >> 5][x & 31] = 0xFF800000u;
    }
    const auto at = [&](int x) { return __uint_as_float(v[x >> 5][x & 31]); };
    float top = -INFINITY;
#pragma unroll
    for (int g = 0; g < 64; g += 16) {
      float z = fmaxf(at(g), at(g + 15)), y = fmax3(at(g + 1), at(g + 2), at(g + 3));
#pragma unroll
      for (int x = g + 4; x < g + 15; x += 4) {
        z = fmax3(z, at(x), at(x + 1));
        y = fmax3(y, at(x + 2), x + 3 < g + 15 ? at(x + 3) : y);
      }
      if (lim[g >> 4] != 0u) top = fmaxf(top, fmaxf(z, y));
    }
    top *= r.c;
    if (__any_sync(0xffffffffu, top > r.m + kBlocksSlack)) {
      const float next = fmaxf(r.m, ceilf(top));
      const float f = r.m == next ? 1.f : ex2(r.m - next);  // (m -inf: 0)
      r.m = next;
      r.sum *= f;
      if (gs > 0) {
        if (!blocks_wait(bars.o_done(slot ^ 1), ((gs - 1) >> 1) & 1, ctl, gs)) return false;
        tc_fence_after();
        blocks_rescale<D>(r.tl + 128, f);
      }
    }
    const float neg = r.m == -INFINITY ? 0.f : -r.m;
    const ldev::F2 c2 = ldev::pair(r.c, r.c), neg2 = ldev::pair(neg, neg);
#pragma unroll
    for (int g = 0; g < 64; g += 16) {
      const bool sees = lim[g >> 4] != 0u;
      ldev::F2 part = ldev::pair(0.f, 0.f);
#pragma unroll
      for (int x = g; x < g + 16; x += 2) {
        const float2 y = ldev::split(ldev::fma2(ldev::pair(at(x), at(x + 1)), c2, neg2));
        const float e0 = ex2(y.x), e1 = ex2(y.y);  // (a score of +inf: inf - inf, NaN)
        part = ldev::add2(part, ldev::pair(e0, e1));
        w[x / 2] = sees ? pack_bf16(e0, e1) : 0u;
      }
      const float2 y = ldev::split(part);
      r.sum += sees ? y.x + y.y : 0.f;
    }
  } else {
#pragma unroll
    for (int x = 0; x < 32; ++x) w[x] = 0u;
  }
  tmem_st32(ts, w);
  tmem_wait_st();
  tc_fence_before();
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bars.p_full(slot));
  return true;
}

// A row's part of O, its maximum and sum, to shared memory: 4 channels of all rows after 4
// channels of all rows, in the place of the keys and values, which are done with.
template <int D>
__device__ __forceinline__ void blocks_part(uint8_t* part, float2* ml, const BlocksRow& r, int row, bool some) {
  ml[row] = make_float2(r.m, r.sum);
  if (!some) return;  // (nothing reads O of a sum of 0)
#pragma unroll 1
  for (int c = 0; c < D; c += 32) {
    uint32_t o[32];
    tmem_ld32(r.tl + 128 + c, o);
#pragma unroll
    for (int x = 0; x < 32; x += 4)
      reinterpret_cast<uint4*>(part)[(c + x) / 4 * 128 + row] = make_uint4(o[x], o[x + 1], o[x + 2], o[x + 3]);
  }
}

// The cluster's parts of a row joined, in the order of its CTAs: this CTA's share of the
// channels (8 at least), the first also the LSE.
template <int D>
__device__ __forceinline__ void blocks_join(uint32_t part, uint32_t ml, int splits, int split, int row, __nv_bfloat16* out,
                                            float* lse) {
  float f[kBlocksMaxSplits], top = -INFINITY, sum = 0.f;
  bool some[kBlocksMaxSplits];
#pragma unroll
  for (int i = 0; i < kBlocksMaxSplits; ++i)
    if (i < splits) {
      const float2 y = ldev::peer_f2(ml + row * 8, i);
      f[i] = y.x;
      some[i] = y.y != 0.f;
      top = fmaxf(top, y.x);
    }
#pragma unroll
  for (int i = 0; i < kBlocksMaxSplits; ++i)
    if (i < splits) {
      f[i] = some[i] ? ex2(f[i] - (top == -INFINITY ? 0.f : top)) : 0.f;
      sum += some[i] ? f[i] * ldev::peer_f2(ml + row * 8, i).y : 0.f;
    }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  if (split == 0 && lse != nullptr) *lse = CUDART_LN2_F * (top + log2f(sum));
  if (out == nullptr) return;
  const int per = D / splits;
#pragma unroll 1
  for (int c = split * per; c < (split + 1) * per; c += 8) {
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < kBlocksMaxSplits; ++i)
      if (i < splits && some[i]) {
        const float4 x = ldev::peer_f4(part + (c / 4 * 128 + row) * 16, i), y = ldev::peer_f4(part + (c / 4 * 128 + 128 + row) * 16, i);
        acc[0] += f[i] * x.x, acc[1] += f[i] * x.y, acc[2] += f[i] * x.z, acc[3] += f[i] * x.w;
        acc[4] += f[i] * y.x, acc[5] += f[i] * y.y, acc[6] += f[i] * y.z, acc[7] += f[i] * y.w;
      }
    *reinterpret_cast<uint4*>(out + c) = make_uint4(pack_bf16(acc[0] * inv, acc[1] * inv), pack_bf16(acc[2] * inv, acc[3] * inv),
                                                    pack_bf16(acc[4] * inv, acc[5] * inv), pack_bf16(acc[6] * inv, acc[7] * inv));
  }
}

// Wide: windows of up to 1024 pages, for tables of more than 256: each window is three
// barriers, a pass over the lists and a pipeline that starts anew. (512 queries x 32 heads,
// d = 128, 65536 tokens, 32 pages of much the same ones a query: 43 us and not 53 with pages of
// 64, 34 and not 79 with 16; 32768 tokens, 8 heads, d = 64, 16 pages of 64: 22 both ways. Tables of
// up to 256 pages, one CTA a tile: 59.3 with the width known to the compiler, 61.2 without.)
template <int D, bool Wide>
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
      mbar_init(bars.o_done(s), 1);
    }
    mbar_init(bars.done(), 1);
    l.abort = 0;
    fence_barrier_init();
    prefetch_tmap(&a.tm_k);
    prefetch_tmap(&a.tm_v);
  }
  if (warp == kWarpMma) {
    tmem_alloc(smem_u32(&l.tmem), kBlocksCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = l.tmem;
  const Ctl ctl{&l.abort, g_long_status, p.timeout_ns}, drain{&l.abort, g_long_status, kDrainNs};
  ldev::grid_dep_launch();
  ldev::grid_dep_wait();

  const int b = blockIdx.z, hk = blockIdx.y, G = p.G;
  const int split = static_cast<int>(blockIdx.x) % p.splits;
  const int all = p.Nq * G, r0 = static_cast<int>(blockIdx.x) / p.splits * 128, rn = min(all - r0, 128);
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
  const int row = static_cast<int>(threadIdx.x) & 127, n_mine = p.by_g.div(r0 + min(row, rn - 1));
  BlocksRow r;
  r.tl = tmem + (static_cast<uint32_t>(warp) << 21);
  r.seen = row < rn ? long_seen(p, lens, n_mine) : 0;
  r.c = p.c_hi;
  r.m = -INFINITY;
  r.sum = 0.f;
  r.word = 0;
  int gs = 0;  // stages so far
  bool ok = true;

  // a window: 256 pages, or as many as the bits hold for so many queries
  const int words = Wide ? (toks <= 32 ? 32 : toks <= 64 ? 16 : 8) : 8, window = words * 32;
  r.took = l.took + (n_mine - tok0) * words;
  for (int w0 = 0, next; w0 < pages; w0 = next) {
    __syncthreads();  // the lists of the window before are done with
    for (int x = threadIdx.x; x < toks * words; x += kBlocksThreads) l.bits[x] = l.took[x] = 0u;
    if (static_cast<int>(threadIdx.x) < words) l.any[threadIdx.x] = 0u;
    if (threadIdx.x == 0) l.next = pages;
    __syncthreads();
    constexpr int kBatch = 5;  // entries on their way to a thread at once
    for (int x0 = threadIdx.x; x0 < toks * p.n; x0 += kBatch * kBlocksThreads) {
      int page[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int x = x0 + i * kBlocksThreads;
        page[i] = x < toks * p.n ? lists[x] : -1;
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        if (page[i] < w0) continue;
        const int t = (x0 + i * kBlocksThreads) / p.n, at = page[i] - w0;
        if (page[i] >= long_pages(p, long_seen(p, lens, tok0 + t))) continue;
        if (at >= window) {
          atomicMin(&l.next, page[i]);
          continue;
        }
        atomicOr(&l.bits[t * words + (at >> 5)], 1u << (at & 31));
        atomicOr(&l.any[at >> 5], 1u << (at & 31));
      }
    }
    ldev::copy_wait<0>();
    fence_async_smem();
    __syncthreads();
    next = l.next == pages ? pages : l.next & ~31;  // (all windows begin at a multiple of 32)
    if (warp == 0) {  // a lane has a word of the pages, or part of one
      const int per = words, first = lane * per;
      uint32_t mine = (l.any[first >> 5] >> (first & 31)) & (per == 32 ? 0xFFFFFFFFu : (1u << per) - 1u), at = __popc(mine);
#pragma unroll
      for (int s = 1; s < 32; s *= 2) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, at, s);
        if (lane >= s) at += y;
      }
      if (lane == 31) l.count = static_cast<int>(at);
      at -= __popc(mine);
      for (; mine != 0u; mine &= mine - 1, ++at) l.page[at] = static_cast<uint16_t>(first + __ffs(mine) - 1);
    }
    __syncthreads();
    const int count = l.count;
    for (int x = threadIdx.x; x < count; x += kBlocksThreads) l.id[x] = p.table[b * p.table_sb + w0 + l.page[x]];
    // a query's bits in the order of the list: eight pages a thread at a time
    const int eights = (count + 7) >> 3;
    for (int x = threadIdx.x; x < toks * eights; x += kBlocksThreads) {
      const int t = x / eights, e0 = (x - t * eights) * 8;
      uint32_t z = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int page = l.page[e0 + e];  // (behind the list: a value left there)
        if (e0 + e < count) z |= ((l.bits[t * words + (page >> 5)] >> (page & 31)) & 1u) << e;
      }
      reinterpret_cast<uint8_t*>(l.took + t * words)[e0 >> 3] = static_cast<uint8_t>(z);
    }
    __syncthreads();
    const int n = st.count(count), first = n * split / p.splits, end = n * (split + 1) / p.splits;
    if (first < end) {
      if (warp == kWarpK) {
        ok = blocks_load<D, false>(a, l, base, bars, st, hk, first, end, gs, ctl);
      } else if (warp == kWarpV) {
        ok = blocks_load<D, true>(a, l, base, bars, st, hk, first, end, gs, ctl);
      } else if (warp == kWarpMma) {
        ok = blocks_mma<D>(BlocksMma<D>(base, tmem), l, smem, bars, st, lens.len, w0, first, end, gs, ctl);
      } else {
        r.word = r.took[st.entry(first, 0) >> 5];
        for (int s = first; s < end && ok; ++s, ++gs) ok = blocks_softmax<D>(l, bars, st, w0, s, gs, r, ctl);
      }
    }
    if (__syncthreads_or(!ok)) break;
  }

  if (warp == kWarpMma) {  // products in flight read this CTA's shared memory and write its TMEM: wait (bounded) for all
    mma_commit(bars.done());
    blocks_wait(bars.done(), 0, drain, gs, false);
  }
  if (warp < 4) {
    if (ok && gs > 0) {
      ok = blocks_wait(bars.o_done((gs - 1) & 1), ((gs - 1) >> 1) & 1, ctl, gs);
      tc_fence_after();
    }
    const int g = r0 + row - n_mine * G, h = hk * G + g;
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.o) + b * p.o_sb + h * p.o_sh + n_mine * p.o_sn;
    float* lse = p.lse == nullptr || row >= rn ? nullptr : p.lse + (static_cast<int64_t>(b) * p.Hq + h) * p.Nq + n_mine;
    if (p.splits == 1) {
      const float inv = r.sum == 0.f ? 0.f : 1.f / r.sum;
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        uint32_t o[32];
        if (gs > 0) tmem_ld32(r.tl + 128 + c, o);
        if (row < rn) {
#pragma unroll
          for (int x = 0; x < 32; x += 8) {
            uint32_t y[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              y[i] = r.sum == 0.f ? 0u : pack_bf16(__uint_as_float(o[x + 2 * i]) * inv, __uint_as_float(o[x + 2 * i + 1]) * inv);
            *reinterpret_cast<uint4*>(out + c + x) = make_uint4(y[0], y[1], y[2], y[3]);
          }
        }
      }
      if (lse != nullptr) *lse = CUDART_LN2_F * (r.m + log2f(r.sum));
    } else {
      blocks_part<D>(smem + S::kOffK, reinterpret_cast<float2*>(l.bits), r, row, gs > 0);
      ldev::cluster_sync();
      blocks_join<D>(base + S::kOffK, smem_u32(l.bits), p.splits, split, row, row < rn ? out : nullptr, lse);
    }
  } else if (p.splits > 1) {
    ldev::cluster_sync();
  }
  if (l.abort != 0u && (warp == kWarpK || warp == kWarpV)) {
    // copies in flight land in this CTA's shared memory: wait (bounded) for the last ones
    for (int x = max(gs - 2, warp == kWarpK && p.inject == 1 ? 1 : 0); x < gs; ++x)  // (the keys that inject withheld never come)
      blocks_wait(warp == kWarpV ? bars.v_full(x & 1) : bars.k_full(x & 1), (x >> 1) & 1, drain, x, false);
  }
  ldev::copy_wait<0>();  // (no page, no wait so far)
  tc_fence_before();
  if (p.splits > 1)
    ldev::cluster_sync();  // (no CTA leaves while another reads its part)
  else
    __syncthreads();
  if (warp == kWarpMma) tmem_dealloc(tmem, kBlocksCols);
}

template <int D, bool Wide>
cudaError_t blocks_tiles_dim(const BlocksTiles& a, cudaStream_t s) {
  const int64_t rows = static_cast<int64_t>(a.p.Nq) * a.p.G;
  const cudaError_t e =
      cudaFuncSetAttribute(blocks_tiles<D, Wide>, cudaFuncAttributeMaxDynamicSharedMemorySize, BlocksSmem<D>::kBytes);
  if (e != cudaSuccess) return e;
  return ldev::launch(blocks_tiles<D, Wide>, dim3(static_cast<unsigned>((rows + 127) / 128 * a.p.splits), a.p.Hk, a.p.B),
                      kBlocksThreads, static_cast<size_t>(BlocksSmem<D>::kBytes), s, a.p.splits, a);
}

}  // namespace dev
}  // namespace attn
