// long_tiles.cu -- page scores and received weights for many query rows, on the tensor
// core's full tiles (tcgen05, accumulators in TMEM).
//
// Both are products of 128 cached things (pages' bounds, or keys) with query rows, of
// which only a reduction over rows is kept: the largest over a token's heads, or the sum
// of exponentials over all rows. So the cached side is the long one: it stays in shared
// memory as the A operand, query rows stream by as B, 64 at a time, and a thread owns one
// page or key (a TMEM lane) and walks along the rows (columns) with its running maximum or
// sum in a register: no shuffles, no padding of heads, neighbouring lanes write
// neighbouring places. Eight warps reduce, two threads a lane, each with half of a tile's
// columns (one: 512 tokens' scores 26.5 us, not 24); several CTAs share an SM. While the tensor
// core works on tile t, they reduce tile t - 1 and the rows of tile t + 1 are on their way: for
// scores, where rows are split by sign, brought by the same warps, a block barrier a tile;
// for weights by warps of their own and barriers in shared memory, so that the chains of
// bringing rows, of placing their lse and of the products run next to the sums (333 rows' weights
// 27 us and not 34.5; with one warp that places lse and issues products 32: its chain a
// tile, some 2500 cycles, was longer than the sums').
//
// What bounds them is instructions and those chains. 333 rows x 15 heads of d = 64 over 23204
// tokens: 27 us, 0.35 PFLOP/s (exp2 alone would take 8); 512 tokens x 32 heads of d = 128 over the
// bounds of 1128 pages: 24 us, 25 MB of scores written among it.
//
// Every wait is bounded: when one runs out the CTA notes it in the status word, leaves its
// loop, waits (bounded) for its products in flight, frees TMEM and returns.
#include <math_constants.h>

#include "attn_sm103.cuh"
#include "long_dev.cuh"
#include "long_kernel.h"

namespace attn {
namespace dev {

__device__ uint32_t g_long_status[4];

constexpr int kTileThreads = 256, kTileRows = 64;  // threads: two for each of 128 pages or keys
constexpr uint32_t kTileCols = 2 * kTileRows;      // TMEM columns: two accumulators
constexpr uint32_t kRoleTiles = 4;
// Bound on the wait for copies and products in flight after a wait has run out: theirs, not the
// caller's, which may be shorter than they take.
constexpr uint64_t kDrainNs = 2000000000;

// True once phase `parity` of `bar` is complete; false after the time limit.
__device__ __noinline__ bool tile_wait_slow(uint32_t bar, uint32_t parity, int tile, uint64_t timeout_ns) {
  const uint64_t t0 = global_ns();
  do {
    if (mbar_test_sleep(bar, parity, kSleepHintNs)) return true;
  } while (global_ns() - t0 <= timeout_ns);
  if (atomicCAS(g_long_status, 0u, kStatusTimeout) == 0u) {
    g_long_status[1] = kRoleTiles;
    g_long_status[2] = static_cast<uint32_t>(tile);
    g_long_status[3] = blockIdx.x;
    __threadfence();
  }
  return false;
}
__device__ __forceinline__ bool tile_wait(uint32_t bar, uint32_t parity, int tile, uint64_t timeout_ns) {
  return mbar_test(bar, parity) || tile_wait_slow(bar, parity, tile, timeout_ns);
}

__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Byte of 16-byte piece `c` of row r in a K-major operand of `rows` rows: blocks of 64
// channels one after the other, 128-byte rows swizzled over 8 (32 channels: 64-byte
// rows, swizzled over pairs of 4).
template <int K>
__device__ __forceinline__ uint32_t operand_at(int r, int c, int rows) {
  if constexpr (K >= 64) return (c >> 3) * rows * 128 + r * 128 + (((c & 7) ^ (r & 7)) << 4);
  return r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
}

// D (128 x 64) = A (128 x K) B (64 x K)^T, operands at a and b.
template <int K>
__device__ __forceinline__ void issue_tile(uint32_t d_tmem, uint32_t a, uint32_t b) {
  constexpr uint32_t kIdesc = make_idesc(128, kTileRows, false);
  constexpr int kRow = K >= 64 ? 128 : 64;
  constexpr uint32_t kLayout = K >= 64 ? 2u : 4u;
  const uint64_t da = smem_desc(a, 16, 8 * kRow, kLayout), db = smem_desc(b, 16, 8 * kRow, kLayout);
  if constexpr (K == 32) {
    mma_ss2<2>(d_tmem, da, db, kIdesc, 0u);
  } else {
#pragma unroll
    for (int c = 0; c < K / 64; ++c)
      mma_ss4<2, 4, 6>(d_tmem, da + (c * 128 * kRow >> 4), db + (c * kTileRows * kRow >> 4), kIdesc, c != 0);
  }
}

// D += the product of 16 further channels. Their operands are not swizzled: groups of 8
// rows, 128 bytes (8 rows of 16) for the first 8 channels, then 128 for the others.
__device__ __forceinline__ void issue_more(uint32_t d_tmem, uint32_t a, uint32_t b) {
  constexpr uint32_t kIdesc = make_idesc(128, kTileRows, false);
  mma_ss(d_tmem, smem_desc(a, 128, 256, 0u), smem_desc(b, 128, 256, 0u), kIdesc, 1u);
}
__device__ __forceinline__ uint32_t more_at(int r, int half) { return (r >> 3) * 256 + half * 128 + (r & 7) * 16; }

// Where a thread's piece of a query row is, row by row of a stride: r = n * heads + g
// without a division each.
struct RowWalk {
  const __nv_bfloat16* at;
  int64_t step, wrap;  // elements that a stride adds; what it adds more if g passes the heads
  int g, dg, heads;
  __device__ __forceinline__ RowWalk(const __nv_bfloat16* base, int r, int stride, int heads_, FastDiv by_g, int64_t sh, int64_t sn)
      : heads(heads_) {
    const int n = by_g.div(r), dn = by_g.div(stride);
    g = r - n * heads;
    dg = stride - dn * heads;
    at = base + n * sn + g * sh;
    step = dn * sn + dg * sh;
    wrap = sn - heads * sh;
  }
  __device__ __forceinline__ void next() {
    at += step;
    g += dg;
    if (g >= heads) {
      g -= heads;
      at += wrap;
    }
  }
};

// What the scores' kernel sets up: barriers and TMEM.
struct Tiles2 {
  uint32_t bars;  // of the two accumulators; of all products
  uint32_t tmem;
  uint64_t timeout_ns;
  int inject;
  __device__ __forceinline__ Tiles2(const LongParams& p) : timeout_ns(p.timeout_ns), inject(p.inject) {}
  __device__ __forceinline__ uint32_t bar(int i) const { return bars + 8 * i; }
  __device__ __forceinline__ void commit(int t) const {
    if (inject != 1 || t != 0) mma_commit(bar(t & 1));
  }
  __device__ __forceinline__ uint32_t d(int t) const { return tmem + (t & 1) * kTileRows; }
  __device__ __forceinline__ bool wait(int t) const { return tile_wait(bar(t & 1), (t >> 1) & 1, t, timeout_ns); }
  __device__ __forceinline__ void begin(uint64_t* words, uint32_t* slot) {
    bars = smem_u32(words);
    if (threadIdx.x == 0) {
      for (int i = 0; i < 3; ++i) mbar_init(bar(i), 1);
      fence_barrier_init();
    }
    if (threadIdx.x < 32) {
      tmem_alloc(smem_u32(slot), kTileCols);
      tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    tmem = *slot;
  }
  // The block has given up: the warp that issued its products waits (bounded) for those in flight.
  __device__ __forceinline__ void drain(int t) const {
    if (threadIdx.x >= 32) return;
    mma_commit(bar(2));
    tile_wait(bar(2), 0, t, kDrainNs);
    __syncwarp();
  }
  __device__ __forceinline__ void end() const {
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x < 32) tmem_dealloc(tmem, kTileCols);
  }
};

// ------------------------------------------------------------------ scores

template <int D>
struct ScoreSmem {
  static constexpr int kK = 2 * D;  // lower and upper bounds side by side
  static constexpr int kA = 128 * kK * 2, kB = kTileRows * kK * 2;
  static constexpr int kBytes = kA + kB + 1024;
};

// B holds min(q, 0) in its first D channels and max(q, 0) in the others. G: query heads of a
// key head (0: any number).
template <int D, int G>
__global__ void __launch_bounds__(kTileThreads, 2) scores_tiles(const __grid_constant__ LongParams p, int tokens) {
  using S = ScoreSmem<D>;
  constexpr int kPieces = D / 8, kLoads = kTileRows * kPieces / kTileThreads;
  extern __shared__ uint8_t raw[];
  __shared__ uint64_t bars[3];
  __shared__ uint32_t slot;
  __shared__ int ids[128];  // the pages
  uint8_t* smem = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
  const uint32_t a_at = smem_u32(smem), b_at = a_at + S::kA;
  Tiles2 tl(p);
  tl.begin(bars, &slot);
  ldev::grid_dep_launch();
  ldev::grid_dep_wait();

  const int b = blockIdx.z, hk = blockIdx.y, heads = G > 0 ? G : p.G;
  const int runs = (p.Nq + tokens - 1) / tokens;
  const int tok0 = static_cast<int>(blockIdx.x % runs) * tokens, page0 = static_cast<int>(blockIdx.x / runs) * 128;
  const LongLens lens = long_lens(p, b);
  const int toks = min(tokens, p.Nq - tok0);
  const int half = static_cast<int>(threadIdx.x) >> 7, page = page0 + (static_cast<int>(threadIdx.x) & 127);
  float* out = p.scores + ((static_cast<int64_t>(b) * p.Hk + hk) * p.Nq + tok0) * p.table_width + page;
  // pages of which no query of the run sees anything need no product
  const int live = min(tok0 + toks, lens.ql);
  const int pages = live > tok0 ? long_pages(p, long_seen(p, lens, live - 1)) : 0;
  const bool some = page0 < pages;
  const int rows = some ? (live - tok0) * heads : 0, tiles = (rows + kTileRows - 1) / kTileRows;

  // query rows of a tile: pieces of 16 bytes, D / 8 threads a row
  uint4 q[kLoads], ahead[kLoads];  // of the next tile, and of the one behind it
  const int piece = static_cast<int>(threadIdx.x) % kPieces, row = static_cast<int>(threadIdx.x) / kPieces;
  constexpr int kStep = kTileThreads / kPieces;
  RowWalk walk(static_cast<const __nv_bfloat16*>(p.q) + b * p.q_sb + static_cast<int64_t>(hk) * heads * p.q_sh +
                   tok0 * p.q_sn + piece * 8,
               row, kStep, heads, p.by_g, p.q_sh, p.q_sn);
  int next = row;  // the row that the walk is at
  const auto load = [&]() {
#pragma unroll
    for (int e = 0; e < kLoads; ++e) {
      q[e] = ahead[e];
      ahead[e] = next < rows ? ldev::ld16(walk.at) : make_uint4(0, 0, 0, 0);
      walk.next();
      next += kStep;
    }
  };
  if (tiles > 0) {
    const int mine = half == 0 && page < pages ? p.table[b * p.table_sb + page] : -1;
    load();
    load();
    if (half == 0) ids[threadIdx.x] = mine;
    __syncthreads();
#pragma unroll 4
    for (int x = threadIdx.x; x < 128 * 2 * kPieces; x += kTileThreads) {
      const int r = x / (2 * kPieces), c = x % (2 * kPieces), id = ids[r];
      const bool real = id >= 0 && id < p.n_pages;
      ldev::copy16(a_at + operand_at<S::kK>(r, c, 128),
                   static_cast<const __nv_bfloat16*>(p.bounds) + ((real ? static_cast<int64_t>(id) : 0) * p.Hk + hk) * 2 * D + c * 8,
                   real ? 16 : 0);
    }
    ldev::copy_commit();
  }

  // (other groups: the first of a lane's threads takes all columns; 2048 rows, 2 x 8 key heads of 512 pages,
  // d = 128: 40 to 45 us for groups of 3, 5 and 7, 33 for 16 and 32, 19 to 21 for 4 and 8)
  constexpr int kHalfToks = G > 0 ? kTileRows / 2 / (G > 0 ? G : 1) : 0;
  float best = -INFINITY;
  int tok = half * kHalfToks, g = 0;  // the token and head that the next column is
  float* at = out + static_cast<int64_t>(tok) * p.table_width;
  const uint32_t lanes = ((threadIdx.x >> 5) & 3u) << 21;
  // token n of the run (below live) sees max(first + n * by, 0) slots
  const int first = p.causal ? lens.len - lens.ql + tok0 + 1 : lens.len, by = p.causal ? 1 : 0;
  const auto sees = [&](int n) { return long_pages(p, max(first + n * by, 0)); };
  const bool in = page < p.table_width;
  const auto reduce = [&](int t) {
    uint32_t v[32];
    if constexpr (G > 0) {
      tmem_ld32(tl.d(t) + lanes + half * 32, v);
      const bool whole = page0 + 128 <= sees(tok) && tok + kHalfToks <= live - tok0;  // every page, for every token
#pragma unroll
      for (int n = 0; n < kHalfToks; ++n) {
        float z = __uint_as_float(v[n * G]);
#pragma unroll
        for (int c = n * G + 1; c < (n + 1) * G; ++c) z = max_nan(z, __uint_as_float(v[c]));
        z *= p.scale;
        if (whole) {
          *at = z;
        } else if (in && tok + n < live - tok0) {
          *at = page < sees(tok + n) ? z : -INFINITY;
        }
        at += p.table_width;
      }
      tok += 2 * kHalfToks;
      at += static_cast<int64_t>(kHalfToks) * p.table_width;
    } else {
      if (half != 0) return;
#pragma unroll 1
      for (int h = 0; h < kTileRows; h += 32) {
        tmem_ld32(tl.d(t) + lanes + h, v);
#pragma unroll
        for (int c = 0; c < 32; ++c) {
          best = max_nan(best, __uint_as_float(v[c]));
          if (++g == heads) {
            if (in && tok < live - tok0) *at = page < sees(tok) ? best * p.scale : -INFINITY;
            best = -INFINITY;
            g = 0;
            ++tok;
            at += p.table_width;
          }
        }
      }
    }
  };

  bool ok = true;
  int t = 0;
  for (; t < tiles; ++t) {
    if (t > 0) ok = tl.wait(t - 1);  // its operand may be replaced
#pragma unroll
    for (int e = 0; e < kLoads; ++e) {
      const int r = e * kStep + row;
      const __nv_bfloat162 zero(__ushort_as_bfloat16(0), __ushort_as_bfloat16(0));
      uint4 neg, pos;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 y = reinterpret_cast<const __nv_bfloat162*>(&q[e])[i];
        reinterpret_cast<__nv_bfloat162*>(&neg)[i] = __hmin2_nan(y, zero);
        reinterpret_cast<__nv_bfloat162*>(&pos)[i] = __hmax2_nan(y, zero);
      }
      *reinterpret_cast<uint4*>(smem + S::kA + operand_at<S::kK>(r, piece, kTileRows)) = neg;
      *reinterpret_cast<uint4*>(smem + S::kA + operand_at<S::kK>(r, piece + kPieces, kTileRows)) = pos;
    }
    if (t == 0) ldev::copy_wait<0>();
    fence_async_smem();
    tc_fence_before();
    if (__syncthreads_or(!ok)) break;
    if (threadIdx.x < 32) {
      tc_fence_after();
      issue_tile<S::kK>(tl.d(t), a_at, b_at);
      tl.commit(t);
    }
    tc_fence_after();
    load();
    if (t > 0) reduce(t - 1);
  }
  bool gave_up = t < tiles;  // (the same in all threads)
  if (t > 0 && !gave_up) {
    ok = tl.wait(t - 1);
    tc_fence_after();
    gave_up = __syncthreads_or(!ok);
    if (!gave_up) reduce(t - 1);
  }
  if (gave_up) tl.drain(t);
  // what no query sees
  for (int n = (some ? max(live - tok0, 0) : 0) + half; n < toks; n += 2)
    if (page < p.table_width) out[static_cast<int64_t>(n) * p.table_width] = -INFINITY;
  tl.end();
}

// ------------------------------------------------------------------ weights

// The rows' lse takes part in the product: keys get four further channels of one, query
// row r those of -lse[r] / scale in four parts (three of 8 bits each that hold its fp32
// value, and what that leaves), so a tile's accumulator is q . k - lse / scale, formed in
// fp32 like the sum itself, and a weight is one product and one exp2 of it. The further 16
// channels lie in operands of their own, unswizzled (8 rows of 16 bytes after one another).
template <int D>
struct WeightSmem {
  static constexpr int kA = 128 * D * 2, kB = kTileRows * D * 2, kStages = D == 128 ? 2 : 3;
  static constexpr int kAX = 128 * 32, kBX = kTileRows * 32;
  static constexpr int kOffB = kA, kOffAX = kOffB + kStages * kB, kOffBX = kOffAX + kAX;
  static constexpr int kBytes = kOffBX + kStages * kBX + 1024;
};

// Slots that a tile's rows see.
struct alignas(16) RowNumbers {  // (read 16 bytes at a time)
  int sees[kTileRows];
  int least[4];  // of the first and second half
};

// Warps 0-7 reduce: two threads a key, each with half of a tile's columns. Warp 8 + s brings
// the query rows and lse of stage s, and the last warp issues the products: nothing but
// barriers of its own rows and accumulators makes a warp wait. (A stage has one warp: a
// parity tells a phase from the next, not from the one after it.)
constexpr int kWeightWarps = 8;
constexpr float kBf16Most = 0x1.FEp127f;
template <int D>
constexpr int kWeightThreads = 32 * (kWeightWarps + WeightSmem<D>::kStages + 1);

template <int D>
__global__ void __launch_bounds__(kWeightThreads<D>, 3) weights_tiles(const __grid_constant__ LongParams p) {
  using S = WeightSmem<D>;
  constexpr int kPieces = D / 8, kStages = S::kStages, kRow = D >= 64 ? 128 : 64;
  // a tile's numbers are placed at most kStages + 2 tiles ahead of those that are being read
  constexpr int kNumbers = kStages + 3;
  extern __shared__ uint8_t raw[];
  __shared__ uint64_t bars[2 * kStages + 4];
  __shared__ uint32_t slot, abort;
  __shared__ RowNumbers numbers[kNumbers];
  __shared__ int ids[128];  // the keys' pages; then the sums of the second of a key's threads
  uint8_t* smem = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
  const uint32_t base = smem_u32(smem);
  const int warp = static_cast<int>(threadIdx.x) >> 5, lane = static_cast<int>(threadIdx.x) & 31;
  const uint32_t bar0 = smem_u32(bars);
  const auto full = [&](int s) { return bar0 + 8 * s; };                       // a stage's rows and lse
  const auto empty = [&](int s) { return bar0 + 8 * (kStages + s); };          // its product is done
  const auto d_full = [&](int t) { return bar0 + 8 * (2 * kStages + (t & 1)); };
  const auto d_empty = [&](int t) { return bar0 + 8 * (2 * kStages + 2 + (t & 1)); };
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(d_full(s), 2);  // (the product, and the warp that knows of its rows' numbers)
      mbar_init(d_empty(s), kWeightWarps);
    }
    abort = 0;
    fence_barrier_init();
  }
  if (warp == 0) {
    tmem_alloc(smem_u32(&slot), kTileCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = slot;
  const Ctl ctl{&abort, g_long_status, p.timeout_ns}, drain{&abort, g_long_status, kDrainNs};
  ldev::grid_dep_launch();
  ldev::grid_dep_wait();

  const int b = blockIdx.z, hk = blockIdx.y;
  const LongLens lens = long_lens(p, b);
  const int half = warp >> 2, unit = static_cast<int>(threadIdx.x) & 127;
  const int key0 = static_cast<int>(blockIdx.x) * 128, key = key0 + unit;
  const int page_mask = (1 << p.page_shift) - 1;
  const int rows = key0 < lens.len ? lens.ql * p.G : 0, tiles = (rows + kTileRows - 1) / kTileRows;
  const auto wait = [&](uint32_t bar, uint32_t parity, int t) { return ctl_wait(bar, parity, ctl, t, kRoleTiles); };

  // a tile's query rows and their lse, by one warp
  constexpr int kStep = 32 / kPieces;  // rows between a lane's pieces
  const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q) + b * p.q_sb + static_cast<int64_t>(hk) * p.G * p.q_sh +
                           lane % kPieces * 8;
  const float* lse = p.lse + (static_cast<int64_t>(b) * p.Hq + hk * p.G) * p.Nq;
  const auto bring = [&](int t, int s) {
    float z[2];
    int sees[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = t * kTileRows + i * 32 + lane, n = p.by_g.div(r), g = r - n * p.G;
      z[i] = r < rows ? lse[static_cast<int64_t>(g) * p.Nq + n] : -INFINITY;
      sees[i] = r < rows ? long_seen(p, lens, n) : 0;
    }
    const int row = lane / kPieces;
    RowWalk walk(q, t * kTileRows + row, kStep, p.G, p.by_g, p.q_sh, p.q_sn);
    const uint32_t dst = base + S::kOffB + s * S::kB, to = operand_at<D>(row, lane % kPieces, kTileRows);
    const int left = rows - t * kTileRows - row;  // rows from this lane's first on
#pragma unroll
    for (int x = 0; x < kTileRows; x += kStep) {
      if (x < left) ldev::copy16(dst + (to ^ ((x & 7u) << 4)) + x * kRow, walk.at, 16);
      walk.next();
    }
    ldev::copy_commit();
    RowNumbers& now = numbers[t % kNumbers];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const bool none = z[i] == -INFINITY;          // the row saw nothing
      float x = none ? 0.f : -z[i] * p.c_hi;        // (c_hi + c_lo: 1 / scale)
      float x1 = 0.f, x2 = 0.f, left = 0.f;
      if (fabsf(x) >= 1e38f && fabsf(z[i]) < INFINITY) x = copysignf(kBf16Most, x);  // (finite, as its lse is)
      if (fabsf(x) < 1e38f) {  // (else, or NaN, the first part says it all)
        x1 = x - __bfloat162float(__float2bfloat16_rn(x));
        x2 = x1 - __bfloat162float(__float2bfloat16_rn(x1));
        left = fmaf(-z[i], p.c_hi, -x) - z[i] * p.c_lo;
      }
      *reinterpret_cast<uint2*>(smem + S::kOffBX + s * S::kBX + more_at(i * 32 + lane, 0)) =
          make_uint2(ldev::pack_bf16(x, x1), ldev::pack_bf16(x2, left));
      if (none) sees[i] = 0;
      now.sees[i * 32 + lane] = sees[i];
      const int least = __reduce_min_sync(0xffffffffu, sees[i]);
      if (lane == 0) now.least[i] = least;
    }
    ldev::copy_wait<0>();
    fence_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(full(s));
  };

  ldev::F2 sum = ldev::pair(0.f, 0.f);
  if (tiles > 0) {
    if (threadIdx.x < 128) ids[unit] = key < lens.len ? p.table[b * p.table_sb + (key >> p.page_shift)] : -1;
    __syncthreads();
#pragma unroll 4
    for (int x = threadIdx.x; x < 128 * kPieces; x += kWeightThreads<D>) {
      const int r = x / kPieces, c = x % kPieces, at = key0 + r, id = ids[r];
      const bool real = id >= 0 && id < p.n_pages;
      ldev::copy16(base + operand_at<D>(r, c, 128),
                   static_cast<const __nv_bfloat16*>(p.kc) + (real ? id * p.kc_sp : 0) + hk * p.kc_sh +
                       (at & page_mask) * p.kc_st + c * 8,
                   real ? 16 : 0);
    }
    // the further channels: ones for the keys, zeros behind the four of the rows
    const uint4 zero = make_uint4(0, 0, 0, 0);
    if (warp < kWeightWarps)
      *reinterpret_cast<uint4*>(smem + S::kOffAX + more_at(unit, half)) =
          half == 0 ? make_uint4(0x3F803F80u, 0x3F803F80u, 0, 0) : zero;
    for (int x = threadIdx.x; x < kStages * S::kBX / 16; x += kWeightThreads<D>)
      *reinterpret_cast<uint4*>(smem + S::kOffBX + x * 16) = zero;
    ldev::copy_wait<0>();
    fence_async_smem();
    __syncthreads();

    if (warp < kWeightWarps) {
      const ldev::F2 c = ldev::pair(p.scale, p.scale);  // (scale * log2(e))
      const uint32_t lanes = (static_cast<uint32_t>(warp) & 3u) << 21;
      for (int t = 0; t < tiles; ++t) {
        if (!wait(d_full(t), (t >> 1) & 1, t)) break;
        tc_fence_after();
        uint32_t v[32];
        tmem_ld32(tmem + (t & 1) * kTileRows + lanes + half * 32, v);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(d_empty(t));
        const RowNumbers& now = numbers[t % kNumbers];
        const auto weights = [&](int x, float(&w)[4]) {
          const float2 a0 = ldev::split(ldev::mul2(ldev::pair(__uint_as_float(v[x]), __uint_as_float(v[x + 1])), c));
          const float2 a1 = ldev::split(ldev::mul2(ldev::pair(__uint_as_float(v[x + 2]), __uint_as_float(v[x + 3])), c));
          w[0] = ex2(a0.x), w[1] = ex2(a0.y), w[2] = ex2(a1.x), w[3] = ex2(a1.y);
        };
        const auto add = [&](const float(&w)[4]) {
          sum = ldev::add2(sum, ldev::add2(ldev::pair(w[0], w[1]), ldev::pair(w[2], w[3])));
        };
        if (key0 + 128 <= now.least[half]) {  // all keys are seen by all of these rows
#pragma unroll
          for (int x = 0; x < 32; x += 4) {
            float w[4];
            weights(x, w);
            add(w);
          }
        } else {
#pragma unroll
          for (int x = 0; x < 32; x += 4) {
            float w[4];
            weights(x, w);
            const int4 most = *reinterpret_cast<const int4*>(now.sees + half * 32 + x);
            w[0] = key < most.x ? w[0] : 0.f;
            w[1] = key < most.y ? w[1] : 0.f;
            w[2] = key < most.z ? w[2] : 0.f;
            w[3] = key < most.w ? w[3] : 0.f;
            add(w);
          }
        }
      }
    } else if (warp < kWeightWarps + kStages) {
      const int s = warp - kWeightWarps;
      for (int t = s; t < tiles; t += kStages) {
        if (!wait(empty(s), ((t / kStages) & 1) ^ 1, t)) break;
        bring(t, s);
      }
    } else {
      int t = 0;
      for (; t < tiles; ++t) {
        const int s = t % kStages;
        if (!wait(full(s), (t / kStages) & 1, t) || !wait(d_empty(t), ((t >> 1) & 1) ^ 1, t)) break;
        tc_fence_after();
        const uint32_t d = tmem + (t & 1) * kTileRows;
        issue_tile<D>(d, base, base + S::kOffB + s * S::kB);
        issue_more(d, base + S::kOffAX, base + S::kOffBX + s * S::kBX);
        mma_commit(empty(s));
        if (p.inject != 1 || t != 0) mma_commit(d_full(t));
        if (lane == 0) mbar_arrive(d_full(t));
        __syncwarp();
      }
      // a product in flight reads this CTA's shared memory and writes its TMEM: wait (bounded) for the
      // last one, also where all were issued and only a warp that reduces has given up
      if (t > 0) ctl_wait(empty((t - 1) % kStages), ((t - 1) / kStages) & 1, drain, t, kRoleTiles, false);
    }
  }
  const float2 both = ldev::split(sum);
  if (half == 1) ids[unit] = __float_as_int(both.x + both.y);
  __syncthreads();
  if (half == 0 && key < lens.len && abort == 0) {
    const int id = p.table[b * p.table_sb + (key >> p.page_shift)];
    if (id >= 0 && id < p.n_pages) {
      const int64_t at = ((static_cast<int64_t>(id) * p.Hk + hk) << p.page_shift) + (key & page_mask);
      const float w = both.x + both.y + __int_as_float(ids[unit]);
      const bool old = p.decay != 0.f && !(p.causal && key >= lens.len - lens.ql);
      p.weights_out[at] = old ? fmaf(p.decay, p.weights[at], w) : w;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) tmem_dealloc(tmem, kTileCols);
}

// ------------------------------------------------------------------ launches

template <typename... Args, typename... Given>
cudaError_t launch_tiles(void (*kern)(Args...), dim3 grid, int threads, int bytes, cudaStream_t s, const Given&... args) {
  if (bytes > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
  }
  return ldev::launch(kern, grid, threads, static_cast<size_t>(bytes), s, 1, args...);
}

// Tokens of a CTA: what gives kScoreCtas CTAs a SM at most (two fit there with d = 128), but
// kScoreLeast rows, which are worth loading the pages' bounds for.
constexpr int kScoreLeast = 256, kScoreCtas = 4;

template <int D>
cudaError_t scores_tiles_dim(const LongParams& p, cudaStream_t s) {
  const int64_t cols = (p.table_width + 127) / 128;
  int64_t runs = kScoreCtas * static_cast<int64_t>(p.sms) / (cols * p.B * p.Hk);
  const int64_t most = (static_cast<int64_t>(p.Nq) * p.G + kScoreLeast - 1) / kScoreLeast;
  if (runs > most) runs = most;
  if (runs < 1) runs = 1;
  const int64_t tokens = (p.Nq + runs - 1) / runs;
  const dim3 grid(static_cast<unsigned>(cols * ((p.Nq + tokens - 1) / tokens)), p.Hk, p.B);
  const int n = static_cast<int>(tokens), bytes = ScoreSmem<D>::kBytes;
  switch (p.G) {
    case 1: return launch_tiles(scores_tiles<D, 1>, grid, kTileThreads, bytes, s, p, n);
    case 2: return launch_tiles(scores_tiles<D, 2>, grid, kTileThreads, bytes, s, p, n);
    case 4: return launch_tiles(scores_tiles<D, 4>, grid, kTileThreads, bytes, s, p, n);
    case 8: return launch_tiles(scores_tiles<D, 8>, grid, kTileThreads, bytes, s, p, n);
    default: return launch_tiles(scores_tiles<D, 0>, grid, kTileThreads, bytes, s, p, n);
  }
}

template <int D>
cudaError_t weights_tiles_dim(const LongParams& p, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>((p.max_len + 127) / 128), p.Hk, p.B);
  LongParams r = p;
  const double scale = p.scale, inv = 1.0 / scale;
  r.c_hi = static_cast<float>(inv);
  r.c_lo = static_cast<float>(inv - static_cast<double>(r.c_hi));
  r.scale = static_cast<float>(scale * 1.4426950408889634074);
  return launch_tiles(weights_tiles<D>, grid, kWeightThreads<D>, WeightSmem<D>::kBytes, s, r);
}

}  // namespace dev
}  // namespace attn

#include "blocks_tiles.cuh"

namespace attn {

cudaError_t launch_blocks_tiles(const LongParams& p, const CUtensorMap& tm_k, const CUtensorMap& tm_v, int d, cudaStream_t s) {
  dev::BlocksTiles a;
  a.p = p;
  a.tm_k = tm_k;
  a.tm_v = tm_v;
  const bool wide = p.table_width > 256;
  switch (d) {
    case 32: return wide ? dev::blocks_tiles_dim<32, true>(a, s) : dev::blocks_tiles_dim<32, false>(a, s);
    case 64: return wide ? dev::blocks_tiles_dim<64, true>(a, s) : dev::blocks_tiles_dim<64, false>(a, s);
    case 128: return wide ? dev::blocks_tiles_dim<128, true>(a, s) : dev::blocks_tiles_dim<128, false>(a, s);
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t launch_scores_tiles(const LongParams& p, int d, cudaStream_t s) {
  switch (d) {
    case 32: return dev::scores_tiles_dim<32>(p, s);
    case 64: return dev::scores_tiles_dim<64>(p, s);
    case 128: return dev::scores_tiles_dim<128>(p, s);
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t launch_weights_tiles(const LongParams& p, int d, cudaStream_t s) {
  switch (d) {
    case 32: return dev::weights_tiles_dim<32>(p, s);
    case 64: return dev::weights_tiles_dim<64>(p, s);
    case 128: return dev::weights_tiles_dim<128>(p, s);
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t long_take_status(uint32_t word[4]) {
  cudaError_t e = cudaMemcpyFromSymbol(word, dev::g_long_status, 4 * sizeof(uint32_t), 0, cudaMemcpyDeviceToHost);
  if (e != cudaSuccess || word[0] == 0) return e;
  const uint32_t zero[4] = {0, 0, 0, 0};
  return cudaMemcpyToSymbol(dev::g_long_status, zero, sizeof(zero), 0, cudaMemcpyHostToDevice);
}

}  // namespace attn
