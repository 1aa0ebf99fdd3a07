// attn_paged.cu -- attention over a paged key/value cache: a prefix that every
// sequence of the batch shares, then each sequence's own pages.
//
// Tasks. A task is up to 256 query rows that read the same keys, of one key
// head: rows of one sequence (queries x the heads that share the key head) over the
// prefix's keys and then its own; or, where that saves enough tiles (plan_paged's
// rule), rows of every sequence together over the prefix, whose keys are then read
// once per 256 rows of the batch, and each sequence's over its own. The tasks' K/V tiles of
// 128 keys form one sequence of units (so many for a task's start, then so many
// a tile), and CTA c takes units [c U / G, (c + 1) U / G): every SM has the same
// work whatever the lengths are. The lengths are read on the device, so a
// captured graph follows them. A task cut between CTAs leaves
// parts (row maximum, row sum, unnormalised O in fp32) in the workspace, and a
// second kernel joins the parts of each row, prefix and own, in a fixed order.
//
// A CTA (one per SM):
//   warp 0      loader: page numbers, TMA of the pages of each K and V tile
//   warp 1      MMA issuer: S = Q K^T and O += P V (tcgen05, TMEM)
//   warp 2      gathers the task's query rows into swizzled shared memory
//   warp 3      works out the CTA's tasks and hands them to the others through
//               a small ring: the divisions are done once, not by every role
//   warps 4-7 / 8-11  softmax of stream 0 / 1: one thread per row
// A task of more than 128 rows has two query tiles, one per stream, and each
// K/V tile serves both. A task of up to 128 rows has one query tile and its
// K/V tiles go to the streams in turn, each with its own running maximum, sum
// and O in TMEM; the two are joined in the CTA at the task's end. Either way
// the tensor core works on one stream while the other's softmax runs.
//
// Keys at and behind the task's end inside its last tile are masked, and their
// V rows are set to zero in shared memory first: a page's unused slots may
// hold anything, and 0 * NaN would reach the sum.
//
// What bounds it, and what it takes (GPU time of both kernels, captured calls):
//   - Long keys of few rows: memory. 64 sequences x 2048 own keys, 8 key heads, d = 128,
//     pages of 64: 86.3 us, 6.2 TB/s. 96 sequences behind 32768 tokens, G = 4: 121 us
//     for 556 MB, 4.6 TB/s (softmax of the prefix's two query tiles, and the cuts).
//   - Prompt chunks: the tile of two query tiles, 2900 cycles, the pace of this library's
//     forward kernel with 128 channels; 3 x 512 tokens x 16 heads behind 2048: 38 us.
//   - Short keys: latency. A task of one or two tiles takes 3.7 to 4.2 us, one step after
//     the other: S, softmax (fetching its code: 1700 cycles for the first 64 keys, 530 for
//     the next), O, the exchange, the store. The next task's tiles and queries wait in
//     shared memory meanwhile. A launch takes 5 us to its first tile (lengths, shares,
//     page numbers, tiles, one after the other) and the join some 4 more: 4 sequences
//     behind 512 tokens 10.4 us, 32 behind 4096 27 us.
//
// P is rounded to bf16 for the second product (the tensor core's input type;
// the row sum takes the unrounded values), which moves O by at most 2^-8 of
// sum p |v|, the size of the final rounding to bf16. (Each weight is rounded once; the
// heaviest of the first 64 keys, and one that raises the maximum by 2^8 in the first
// half of a tile, is 1 and not rounded. Against 64 bits O is off by 0.0018 of its norm
// while decoding and in chunks, 0.0022 with one key head of 32 channels; the rounding of
// the output alone is 0.0016.)
#include <cuda_bf16.h>
#include <math_constants.h>

#include "attn_sm103.cuh"
#include "paged_kernel.h"

namespace attn {
namespace dev {

__device__ uint32_t g_paged_status[4];

// One CTA's share of one task, as warp 3 hands it to the other roles.
struct PSeg {
  int rows;        // rows that the task's key head has in all; 0: the CTA is done
  int row0;        // first row of the task
  int pt;          // leading tiles that are the prefix's; the others are the sequence's own
  int k0, k1;      // tiles [k0, k1)
  int hk, b;       // key head; sequence (own tasks)
  int len, ql;     // the sequence's lengths (own tasks)
  int flags;
  int pad[2];
  static constexpr int kPrefix = 1, kTwin = 2, kWhole = 4, kFirst = 8;
  __device__ bool prefix() const { return flags & kPrefix; }
  __device__ bool twin() const { return flags & kTwin; }    // one query tile, tiles in turn
  __device__ bool whole() const { return flags & kWhole; }  // every tile of the task
  __device__ bool first() const { return flags & kFirst; }  // holds the task's first tile
};
static_assert(sizeof(PSeg) == 48, "three 16-byte words");

template <int D>
struct PCfg {
  using C = Cfg<D>;  // tile layout (swizzle, chunks) and MMA descriptors
  // K and V tiles share one ring in the order in which the MMA warp takes
  // them; with 128 channels its five stages are what shared memory holds
  // beside two query tiles (two stages each of K and V kept one tile of four
  // in flight too few: 3600 cycles a tile against 2850).
  static constexpr int kStages = D == 128 ? 5 : (D == 64 ? 10 : 16);
  static constexpr int kSegs = 4;  // ring of task descriptors
  static constexpr int kOffQ = 0;
  static constexpr int kOffKV = 2 * C::kTileBytes;
  static constexpr int kOffX = kOffKV + kStages * C::kTileBytes;  // exchange: [2 streams][m, l][128]
  static constexpr int kXBytes = 2 * 2 * 128 * 4;
  static constexpr int kOffSeg = kOffX + kXBytes;
  static constexpr int kOffBar = kOffSeg + kSegs * static_cast<int>(sizeof(PSeg));
  static constexpr int kBars = 19 + 2 * kSegs + 2 * kStages;
  static constexpr int kSmemBytes = kOffBar + 8 * kBars + 16;
  static_assert(kSmemBytes <= 227 * 1024, "shared memory");
};

template <int D>
struct PBars {
  uint32_t base;
  static constexpr int kSt = PCfg<D>::kStages, kSg = PCfg<D>::kSegs;
  __device__ uint32_t q_full(int s) const { return base + 8 * s; }
  __device__ uint32_t q_empty(int s) const { return base + 16 + 8 * s; }
  __device__ uint32_t s_full(int h) const { return base + 32 + 8 * h; }
  __device__ uint32_t p_full(int h, int part) const { return base + 48 + 8 * (2 * h + part); }
  __device__ uint32_t o_full(int h) const { return base + 80 + 8 * h; }
  __device__ uint32_t o_empty(int h) const { return base + 96 + 8 * h; }
  __device__ uint32_t x_full(int h) const { return base + 112 + 8 * h; }
  __device__ uint32_t done() const { return base + 128; }
  // every product of a one-tile task is complete (o_full: of stream h of a two-tile task).
  // One barrier of its own, that both warpgroups wait for at every such task: none skips a phase.
  __device__ uint32_t t_full() const { return base + 136; }
  __device__ uint32_t q_asked() const { return base + 144; }  // the first task's queries are on their way
  __device__ uint32_t seg_full(int s) const { return base + 152 + 8 * s; }
  __device__ uint32_t seg_empty(int s) const { return base + 152 + 8 * (kSg + s); }
  __device__ uint32_t full(int s) const { return base + 152 + 8 * (2 * kSg + s); }
  __device__ uint32_t empty(int s) const { return base + 152 + 8 * (2 * kSg + kSt + s); }
};

// ------------------------------------------------------------------ work split

__device__ __forceinline__ int clampi(int x, int lo, int hi) { return min(max(x, lo), hi); }

struct SeqLens {
  int len, ql;
};

__device__ __forceinline__ SeqLens raw_lens(const PagedParams& p, int b) {
  return SeqLens{p.kv_lens[b], p.q_lens != nullptr ? p.q_lens[b] : p.Nq};
}
__device__ __forceinline__ SeqLens clamp_lens(const PagedParams& p, SeqLens s) {
  return SeqLens{clampi(s.len, 0, p.max_len), clampi(s.ql, 0, p.Nq)};
}
__device__ __forceinline__ SeqLens seq_lens(const PagedParams& p, int b) { return clamp_lens(p, raw_lens(p, b)); }

// Keys that query n of a sequence sees, counted from the prefix's first.
__device__ __forceinline__ int keys_seen(const PagedParams& p, SeqLens s, int n) {
  if (n >= s.ql) return 0;
  const int total = p.prefix_len + s.len;
  return p.causal ? clampi(total - s.ql + n + 1, 0, total) : total;
}

// K/V tiles that task t (rows [256 t, 256 t + 256)) of a sequence needs: the
// prefix's unless batched tasks go over them, and its own.
struct Tiles {
  int prefix, all;
};
__device__ __forceinline__ Tiles own_tiles(const PagedParams& p, SeqLens s, int t) {
  const int first = p.by_g.div(t * kPagedTaskRows);
  if (first >= s.ql) return Tiles{0, 0};
  const int last = min(p.by_g.div(min((t + 1) * kPagedTaskRows, p.Nq * p.G) - 1), s.ql - 1);
  const int seen = keys_seen(p, s, last);
  const int pre = p.prefix_tasks > 0 ? 0 : (min(seen, p.prefix_len) + kBN - 1) / kBN;
  return Tiles{pre, pre + (max(seen - p.prefix_len, 0) + kBN - 1) / kBN};
}

// Units of a tile of a task that has `rows` rows left, and of the task.
__device__ __forceinline__ int tile_units(int rows) { return rows > kBM ? kPagedPairTile : kPagedTile; }
__device__ __forceinline__ int task_cost(int rows) { return rows > kBM ? kPagedPairTaskCost : kPagedTaskCost; }
__device__ __forceinline__ int task_units(int tiles, int rows) {
  return tiles > 0 ? task_cost(rows) + tiles * tile_units(rows) : 0;
}

// Units of one sequence's tasks for one key head.
__device__ __forceinline__ int own_units(const PagedParams& p, SeqLens s) {
  int u = 0;
  for (int t = 0; t < p.own_tasks; ++t) {
    u += task_units(own_tiles(p, s, t).all, p.Nq * p.G - t * kPagedTaskRows);
  }
  return u;
}

// The split of U units over the CTAs that get some: U / n each, one more for
// the first U mod n.
struct Split {
  int ctas, per, extra;
  __device__ __forceinline__ Split(int u, int grid) : ctas(max(1, min(grid, u / kPagedMinUnits))) {
    per = static_cast<int>(static_cast<uint32_t>(u) / static_cast<uint32_t>(ctas));
    extra = u - per * ctas;
  }
  __device__ __forceinline__ int lo(int c) const { return min(c, ctas) * per + min(c, extra); }
  __device__ __forceinline__ int owner(int u) const {  // the CTA whose range holds unit u
    const int wide = extra * (per + 1);
    const bool in = u < wide;
    return (in ? 0 : extra) + static_cast<int>(static_cast<uint32_t>(in ? u : u - wide) /
                                               static_cast<uint32_t>(in ? per + 1 : max(per, 1)));
  }
};

struct PSegIter {
  int u, hi;       // units left: [u, hi)
  int up;          // units of the prefix tasks
  int b, sb;       // current sequence and its first unit
  SeqLens cur, nxt;  // its lengths, and the next one's as they are in memory (nobody waits for them yet)
  int ub;          // its units per key head
  int at_head = -1, at_a = -1, at_t = 0;  // first unit of the own head and task looked at last, and its number
  int task, parts_end;  // of the segment: index in the task table; its last tile's first unit

  // u0: the CTA's first unit; b0, s0: the sequence that holds it (or the next) and its first unit.
  __device__ __forceinline__ PSegIter(const PagedParams& p, int u0, int u1, int b0, int s0, int ub0, SeqLens lens0)
      : u(u0), hi(u1), up(p.prefix_units), b(b0), sb(s0), cur(lens0), nxt{0, 0}, ub(ub0) {
    if (b + 1 < p.B) nxt = raw_lens(p, b + 1);
  }
  __device__ __forceinline__ bool next(const PagedParams& p, PSeg& s) {
    while (u < hi) {
      int a, tiles;
      if (u < up) {
        tiles = p.prefix_tiles;
        s.hk = p.by_prefix_head.div(u);
        a = s.hk * static_cast<int>(p.by_prefix_head.d);
        const int t = min(p.by_prefix_task.div(u - a), p.prefix_tasks - 1);
        a += t * static_cast<int>(p.by_prefix_task.d);
        s.flags = PSeg::kPrefix;
        s.b = s.len = s.ql = 0;
        s.row0 = t * kPagedTaskRows;
        s.rows = p.B * p.Nq * p.G;
        s.pt = tiles;
        task = p.B * p.Hk * p.own_tasks + s.hk * p.prefix_tasks + t;
      } else {
        while (u >= sb + p.Hk * ub) {
          sb += p.Hk * ub;
          ++b;
          cur = clamp_lens(p, nxt);
          ub = own_units(p, cur);
          if (b + 1 < p.B) nxt = raw_lens(p, b + 1);
        }
        s.flags = 0;
        s.b = b;
        s.len = cur.len;
        s.ql = cur.ql;
        s.hk = (u - sb) / ub;
        // the task that holds u, from where the last look ended if that was in this head
        const int a0 = sb + s.hk * ub;
        if (at_a < a0 || at_head != a0) {
          at_head = at_a = a0;
          at_t = 0;
        }
        Tiles n = own_tiles(p, cur, at_t);
        for (;;) {
          const int per = task_units(n.all, p.Nq * p.G - at_t * kPagedTaskRows);
          if (u < at_a + per) break;
          at_a += per;
          n = own_tiles(p, cur, ++at_t);
        }
        const int t = at_t;
        a = at_a;
        tiles = n.all;
        s.pt = n.prefix;
        task = (b * p.Hk + s.hk) * p.own_tasks + t;
        s.row0 = t * kPagedTaskRows;
        s.rows = p.Nq * p.G;
      }
      // a tile is the share's that holds its first unit
      const int w = tile_units(s.rows - s.row0), first = a + task_cost(s.rows - s.row0), end = first + tiles * w;
      s.k0 = (max(u, first) - first + w - 1) / w;
      s.k1 = (max(min(hi, end), first) - first + w - 1) / w;
      if (s.rows - s.row0 <= kBM) s.flags |= PSeg::kTwin;
      if (s.k0 == 0) s.flags |= s.k1 == tiles ? PSeg::kWhole | PSeg::kFirst : PSeg::kFirst;
      parts_end = end - w;
      u = min(hi, end);
      if (s.k1 > s.k0) return true;
    }
    s.rows = 0;
    return false;
  }
};

// Position of row r of a segment's task.
struct RowPos {
  int b, n, g;
};
__device__ __forceinline__ RowPos row_pos(const PagedParams& p, const PSeg& s, int r) {
  RowPos x;
  x.b = s.prefix() ? p.by_rows.div(r) : s.b;
  const int i = s.prefix() ? r - x.b * p.Nq * p.G : r;
  x.n = p.by_g.div(i);
  x.g = i - x.n * p.G;
  return x;
}

// Loads 64 consecutive 32-bit TMEM columns of this thread's lane, then waits for them.
__device__ __forceinline__ void tmem_ld64(uint32_t taddr, uint32_t (&r)[64]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%64];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, %48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, [%65];\n\t"
      "tcgen05.wait::ld.sync.aligned;\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]), "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]), "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]), "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]), "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
      : "r"(taddr), "r"(taddr + 32u)
      : "memory");
}

// 32 columns at each of two addresses of this thread's lane, one wait for both.
__device__ __forceinline__ void tmem_ld32x2(uint32_t ta, uint32_t (&a)[32], uint32_t tb, uint32_t (&b)[32]) {
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
      : "r"(ta), "r"(tb)
      : "memory");
}

// ------------------------------------------------------------------ roles

// A lane's own TMA (each lane that calls it issues one copy).
__device__ __forceinline__ void tma_lane(uint32_t dst, const CUtensorMap* m, uint32_t bar, int c0, int c1, int c2,
                                         int c3, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%3, %4, %5, %6}], [%2], %7;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "l"(policy)
      : "memory");
}

// Warp 3: reads the lengths, finds the CTA's share of the units (first the
// total, then a running sum over the sequences up to the CTA's first unit) and
// puts its segments into the descriptor ring, one after the other. Whoever
// holds a task's first tile notes who else has parts of it, for the join.
template <int D>
__device__ void paged_scheduler(const PagedParams& p, uint8_t* smem, const PBars<D>& bars, const Ctl& ctl) {
  using P = PCfg<D>;
  const int lane = threadIdx.x & 31;
  grid_dep_wait();  // lengths and tables are the previous kernel's to write
  // (One loop for the total and the running sum, the divisions few: what bounds
  // the start of a launch is fetching this code.)
  int v = 0, sum = 0, u0 = 0, u1 = 0;
  int b0 = 0, s0 = p.prefix_units;  // the sequence that holds u0 (or the first behind it), its first unit
  int ub = 0;                       // and its units per key head
  SeqLens lens{0, 0};               // and its lengths
  Split split(0, 1);
  SeqLens first[4];                 // of the first 128 sequences, all asked for at once
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (32 * j + lane < p.B) first[j] = seq_lens(p, 32 * j + lane);
  SeqLens sl{0, 0};                 // of this lane's sequence of the 32 looked at
  for (int pass = 0, at = 0;; at += 32) {
    if (at >= p.B) {
      if (pass == 1) break;
      pass = 1;
      at = 0;
      split = Split(p.prefix_units + p.Hk * __reduce_add_sync(0xffffffffu, sum), gridDim.x);
      u0 = split.lo(blockIdx.x);
      u1 = split.lo(blockIdx.x + 1);
      if (u0 >= u1) break;
    }
    if (pass == 0 || p.B > 32) {
      sl = first[0];
      if (at > 0) sl = at == 32 ? first[1] : at == 64 ? first[2] : at == 96 ? first[3] : seq_lens(p, min(at + lane, p.B - 1));
      v = at + lane < p.B ? own_units(p, sl) : 0;
    }
    if (pass == 0) {
      sum += v;
      continue;
    }
    int inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += x;
    }
    const uint32_t past = __ballot_sync(0xffffffffu, s0 + p.Hk * inc > u0);
    const int i = u0 < p.prefix_units ? 0 : __ffs(past) - 1;
    if (i >= 0) {
      s0 += p.Hk * __shfl_sync(0xffffffffu, inc - v, i);
      ub = __shfl_sync(0xffffffffu, v, i);
      lens = SeqLens{__shfl_sync(0xffffffffu, sl.len, i), __shfl_sync(0xffffffffu, sl.ql, i)};
      b0 = at + i;
      break;
    }
    s0 += p.Hk * __shfl_sync(0xffffffffu, inc, 31);
  }
  PSegIter it(p, u0, u1, b0, s0, ub, lens);
  RingPos<P::kSegs> r;
  for (bool more = true; more;) {
    PSeg s;
    more = it.next(p, s);
    if (!ctl_wait(bars.seg_empty(r.s), r.ph ^ 1u, ctl, -1, kRoleLoader)) return;
    if (lane == 0) {
      *reinterpret_cast<PSeg*>(smem + P::kOffSeg + r.s * sizeof(PSeg)) = s;
      mbar_arrive(bars.seg_full(r.s));
      if (more && s.first())
        p.tasks[it.task] = make_int2(blockIdx.x, split.owner(it.parts_end) - static_cast<int>(blockIdx.x) + 1);
    }
    __syncwarp();
    r.advance();
  }
}

// A role's view of the ring. take: the next descriptor (rows 0: no more).
template <int D>
struct SegReader {
  RingPos<PCfg<D>::kSegs> r;
  // ROLE softmax waits inline: a call in these warps' loop costs them their registers (2700 bytes of spills).
  template <uint32_t ROLE>
  __device__ __forceinline__ bool take(PSeg& s, const uint8_t* smem, const PBars<D>& bars, const Ctl& ctl) {
    if (ROLE == kRoleSoftmax) {
      if (!warp_wait(bars.seg_full(r.s), r.ph, ctl, -1)) return false;
    } else {
      if (!ctl_wait(bars.seg_full(r.s), r.ph, ctl, -1, ROLE)) return false;
    }
    const int4* src = reinterpret_cast<const int4*>(smem + PCfg<D>::kOffSeg + r.s * sizeof(PSeg));
    const int4 a = src[0], b = src[1], c = src[2];
    s.rows = a.x;
    s.row0 = a.y;
    s.pt = a.z;
    s.k0 = a.w;
    s.k1 = b.x;
    s.hk = b.y;
    s.b = b.z;
    s.len = b.w;
    s.ql = c.x;
    s.flags = c.y;
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bars.seg_empty(r.s));
    r.advance();
    return s.rows > 0;
  }
};

// The ring's order of a segment's n tiles: the K tiles of the first `ahead`
// (one, or two where the streams take tiles in turn), then V(i), K(i + ahead).
// The last position is the last tile's V.
__device__ __forceinline__ int tiles_ahead(const PSeg& s) { return s.twin() ? 2 : 1; }

template <int D>
__device__ void paged_loader(const PagedParams& p, uint8_t* smem, uint32_t sbase, const PBars<D>& bars,
                             const Ctl& ctl) {
  using P = PCfg<D>;
  using C = Cfg<D>;
  const int lane = threadIdx.x & 31;
  const int page = 1 << p.page_shift, box = min(page, kBN);
  const int per_tile = kBN / box;             // pages (or parts of one) of a tile: 1 to 8
  const uint32_t box_bytes = static_cast<uint32_t>(box) * D * 2;
  const uint64_t pol_once = l2_policy_evict_first(), pol_reuse = l2_policy_evict_last();
  RingPos<P::kStages> r;
  uint32_t armed = 0, par = 0;
  int nth = 0;                                // K tiles issued (test hook)
  SegReader<D> segs;
  PSeg s;
  grid_dep_wait();
  while (segs.template take<kRoleLoader>(s, smem, bars, ctl)) {
    const int32_t* own = p.table + s.b * p.table_sb;
    const int ahead = tiles_ahead(s);
    // this lane's first key of tile k among the prefix's or the own keys, and whether
    // it has a page to load (pages behind the last key are not loaded)
    auto key_of = [&](int k) -> int { return (k < s.pt ? k : k - s.pt) * kBN + lane * box; };
    auto has = [&](int k) -> bool { return lane < per_tile && key_of(k) < (k < s.pt ? p.prefix_len : s.len); };
    auto page_of = [&](int k) -> int {
      return k < s.k1 && has(k) ? (k < s.pt ? p.prefix_table : own)[key_of(k) >> p.page_shift] : 0;
    };
    auto load = [&](const CUtensorMap* map, int k, int id, bool withhold) -> bool {
      if (!ctl_wait(bars.empty(r.s), r.ph ^ 1u, ctl, k, kRoleLoader)) return false;
      const bool mine = has(k);
      const uint32_t bytes = static_cast<uint32_t>(__popc(__ballot_sync(0xffffffffu, mine))) * box_bytes;
      if (!withhold) {
        mbar_expect_tx(bars.full(r.s), bytes);
        __syncwarp();
        if (mine) {
          const uint32_t dst = sbase + P::kOffKV + r.s * C::kTileBytes + lane * box * C::kSwizzle;
          const int slot = key_of(k) & (page - 1);
          const uint64_t pol = k < s.pt ? pol_reuse : pol_once;
          for (int c = 0; c < C::kChunks; ++c)
            tma_lane(dst + c * C::kChunkBytes, map, bars.full(r.s), c * C::kBoxCols, slot, s.hk, id, pol);
        }
        __syncwarp();
        armed |= 1u << r.s;
        par = (par & ~(1u << r.s)) | (r.ph << r.s);
      }
      r.advance();
      return true;
    };
    // page numbers are fetched one step before they are used
    int id_k = page_of(s.k0), id_n = page_of(s.k0 + 1), id_v = id_k;
    if (nth == 0) {  // the CTA's first queries go ahead of its first five tiles: behind them they waited 6000 cycles
      if (!ctl_wait(bars.q_asked(), 0, ctl, -1, kRoleLoader)) goto drain;
    }
    for (int i = 0; i < ahead && s.k0 + i < s.k1; ++i) {
      const bool withhold = p.inject && nth == 1;  // test hook: the MMA issuer's wait must run out
      ++nth;
      if (!load(&p.tm_k, s.k0 + i, i ? id_n : id_k, withhold)) goto drain;
    }
    for (int k = s.k0; k < s.k1; ++k) {
      // id_v: pages of tile k; id_n: of tile k + 1
      const int id_2 = page_of(k + 2);
      if (!load(&p.tm_v, k, id_v, false)) goto drain;
      const int kn = k + ahead;
      if (kn < s.k1) {
        const bool withhold = p.inject && nth == 1;
        ++nth;
        if (!load(&p.tm_k, kn, ahead == 2 ? id_2 : id_n, withhold)) goto drain;
      }
      id_v = id_n;
      id_n = id_2;
    }
  }
drain:
  __syncwarp();
  // The last copy armed on each barrier must have landed before the CTA exits.
  for (int st = 0; st < P::kStages; ++st)
    if ((armed >> st) & 1u) ctl_wait(bars.full(st), (par >> st) & 1u, ctl, -1, kRoleLoader, false);
}

// Warp 2: the task's query rows into the swizzled K-major layout that the MMA
// descriptor expects. Where a query tile is a box of a tensor map it is one TMA
// per column chunk: prefix tasks (rows b, n, head) if a sequence's rows divide
// 128, else tasks inside one sequence (rows n, head) if G does.
// Otherwise 16 bytes a copy, every copy of a task in flight at once: each lane
// works out the address of one row of 32, a row's d/8 lanes get it by shuffles.
// The two query tiles are a ring: a one-tile task's queries arrive while the
// task before, in the other slot, is still at work.
template <int D>
__device__ void paged_gather_q(const PagedParams& p, uint32_t sbase, uint8_t* smem, const PBars<D>& bars,
                               const Ctl& ctl) {
  using P = PCfg<D>;
  using C = Cfg<D>;
  constexpr int kLanes = D / 8, kRows = 32 / kLanes;  // lanes of a row; rows per instruction
  const int lane = threadIdx.x & 31;
  const int c = lane % kLanes, sub = lane / kLanes;   // 16-byte chunk of the row; which row of the instruction's
  RingPos<2> r;
  bool asked = false;
  uint32_t armed = 0, par = 0;  // slots whose last queries came as boxes, and their phases
  SegReader<D> segs;
  PSeg s;
  grid_dep_wait();
  while (segs.template take<kRoleLoader>(s, smem, bars, ctl)) {
    const int n = min(s.rows - s.row0, kPagedTaskRows), tiles = n > kBM ? 2 : 1;
    const bool box = p.q_map == (s.prefix() ? 1 : 2);
    // first query, or first sequence, of the task and how many of them a box holds
    const FastDiv& rows = s.prefix() ? p.by_rows : p.by_g;
    const int first = rows.div(s.row0), per = rows.div(kBM);
    const int slot0 = r.s;
    for (int i = 0; i < tiles; ++i) {
      if (!ctl_wait(bars.q_empty(r.s), r.ph ^ 1u, ctl, -1, kRoleLoader)) goto drain;
      const uint32_t tile = sbase + P::kOffQ + r.s * C::kTileBytes;
      if (box) {
        mbar_expect_tx(bars.q_full(r.s), C::kTileBytes);
        for (int ch = 0; ch < C::kChunks; ++ch)
          tma_load_4d(tile + ch * C::kChunkBytes, &p.tm_q, bars.q_full(r.s), ch * C::kBoxCols, s.hk * p.G,
                      s.prefix() ? 0 : first + i * per, s.prefix() ? first + i * per : s.b);
        armed |= 1u << r.s;
        par = (par & ~(1u << r.s)) | (r.ph << r.s);
      } else {
        armed &= ~(1u << r.s);
        const int here = min(n - i * kBM, kBM);  // rows of this query tile
        for (int i0 = 0; i0 < here; i0 += 32) {
          const __nv_bfloat16* src = nullptr;
          if (i0 + lane < here) {
            const RowPos x = row_pos(p, s, s.row0 + i * kBM + i0 + lane);
            src = static_cast<const __nv_bfloat16*>(p.q) + x.b * p.q_sb + static_cast<int64_t>(s.hk * p.G + x.g) * p.q_sh +
                  x.n * p.q_sn;
          }
          const int m = min(32, here - i0);
#pragma unroll 4
          for (int j = 0; j < m; j += kRows) {
            const int k = j + sub;  // row of the 32
            const unsigned long long from = __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(src), k & 31);
            const int row = i0 + k;
            const int swz = C::kSwizzle == 128 ? ((c & 7) ^ (row & 7)) : (c ^ ((row >> 1) & 3));
            const uint32_t dst =
                tile + (C::kSwizzle == 128 ? (c >> 3) * C::kChunkBytes : 0) + row * C::kSwizzle + swz * 16;
            if (k < m)
              asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(from + c * 16) : "memory");
          }
        }
      }
      r.advance();
    }
    if (!asked) {
      asked = true;
      __syncwarp();
      if (lane == 0) mbar_arrive(bars.q_asked());
    }
    if (!box) {
      asm volatile("cp.async.wait_all;" ::: "memory");
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane < tiles) mbar_arrive(bars.q_full(slot0 ^ lane));
    }
  }
drain:
  asm volatile("cp.async.wait_all;" ::: "memory");
  // boxes on their way must have landed before the CTA exits
  for (int i = 0; i < 2; ++i)
    if ((armed >> i) & 1u) ctl_wait(bars.q_full(i), (par >> i) & 1u, ctl, -1, kRoleLoader, false);
}

template <int D>
__device__ void paged_mma(const PagedParams& p, uint8_t* smem, uint32_t sbase, const PBars<D>& bars, uint32_t tmem,
                          const Ctl& ctl) {
  using P = PCfg<D>;
  using C = Cfg<D>;
  const uint64_t q_base = smem_desc(sbase + P::kOffQ, 16, 8 * C::kSwizzle, C::kLayout);
  const uint64_t k_base = smem_desc(sbase + P::kOffKV, 16, 8 * C::kSwizzle, C::kLayout);
  const uint64_t v_base = smem_desc(sbase + P::kOffKV, C::kChunkBytes, 8 * C::kSwizzle, C::kLayout);
  constexpr uint64_t kStep = static_cast<uint64_t>(C::kTileBytes >> 4);
  uint32_t p_par = 0, o_par = 0;  // bit h of p_par, o_par: parity of stream h's next phase
  RingPos<P::kStages> r;
  RingPos<2> q;
  SegReader<D> segs;
  PSeg s;
  grid_dep_wait();  // (the bound on the waits below is not for the kernel before)
  while (segs.template take<kRoleMma>(s, smem, bars, ctl)) {
    const bool twin = s.twin();
    const int slot0 = q.s;  // the task's query tiles: this slot, and the other
    for (int i = 0; i < (twin ? 1 : 2); ++i) {
      if (!ctl_wait(bars.q_full(q.s), q.ph, ctl, -1, kRoleMma)) goto drain;
      q.advance();
    }
    tc_fence_after();
    uint32_t o_ready = 0;
    const uint64_t q0 = q_base + slot0 * kStep, q1 = twin ? q0 : q_base + (slot0 ^ 1) * kStep;
    auto q_done = [&]() {
      mma_commit(bars.q_empty(slot0));
      if (!twin) mma_commit(bars.q_empty(slot0 ^ 1));
    };
    auto scores = [&](int h) {
      issue_s<D>(tmem + static_cast<uint32_t>(h) * C::tm_s(1), h ? q1 : q0, k_base + r.s * kStep);
      mma_commit(bars.s_full(h));
    };
    auto take = [&](int k) -> bool {
      if (!ctl_wait(bars.full(r.s), r.ph, ctl, k, kRoleMma)) return false;
      tc_fence_after();
      return true;
    };
    auto give = [&]() {
      mma_commit(bars.empty(r.s));
      r.advance();
    };
    auto product = [&](int k, int h, uint64_t v) -> bool {
      if (!((o_ready >> h) & 1u) && !ctl_wait(bars.o_empty(h), ((o_par >> h) & 1u) ^ 1u, ctl, k, kRoleMma)) return false;
      const uint32_t par = (p_par >> h) & 1u;
      for (int part = 0; part < 2; ++part) {
        if (!ctl_wait(bars.p_full(h, part), par, ctl, k, kRoleMma)) return false;
        tc_fence_after();
        issue_pv<D>(tmem + C::tm_o(0) + static_cast<uint32_t>(h) * D, tmem + static_cast<uint32_t>(h) * C::tm_p(1), v,
                    part, (((o_ready >> h) & 1u) != 0u || part > 0) ? 1u : 0u);
      }
      p_par ^= 1u << h;
      o_ready |= 1u << h;
      return true;
    };
    const int ahead = tiles_ahead(s);
    for (int i = 0; i < ahead && s.k0 + i < s.k1; ++i) {
      if (!take(s.k0 + i)) goto drain;
      scores(i);
      if (!twin) scores(1);
      give();
    }
    if (s.k0 + ahead >= s.k1) q_done();
    for (int k = s.k0; k < s.k1; ++k) {
      const int kn = k + ahead;
      const bool more = kn < s.k1;
      if (!take(k)) goto drain;
      const uint64_t v = v_base + r.s * kStep;
      const uint32_t v_empty = bars.empty(r.s);
      r.advance();
      if (twin) {
        const int h = (k - s.k0) & 1;
        if (!product(k, h, v)) goto drain;
        mma_commit(v_empty);
        if (more) {
          if (!take(kn)) goto drain;
          scores(h);
          give();
        }
      } else {
        if (!product(k, 0, v)) goto drain;
        if (more) {
          if (!take(kn)) goto drain;
          scores(0);
        }
        if (!product(k, 1, v)) goto drain;
        mma_commit(v_empty);
        if (more) {
          scores(1);
          give();
        }
      }
      if (more && kn + 1 == s.k1) q_done();  // the task's last S is issued
    }
    for (int h = 0; h < 2; ++h) {
      if (!((o_ready >> h) & 1u)) {  // a stream without a tile keeps its phases in step
        if (!ctl_wait(bars.o_empty(h), ((o_par >> h) & 1u) ^ 1u, ctl, -1, kRoleMma)) goto drain;
      }
      if (!twin) mma_commit(bars.o_full(h));
      o_par ^= 1u << h;
    }
    if (twin) mma_commit(bars.t_full());
  }
drain:
  mma_commit(bars.done());
  ctl_wait(bars.done(), 0, ctl, -1, kRoleMma, false);
}

// A part's slot: quarters of 32 rows, each [D/4][32 rows] float4, then m[32], l[32].
template <int D>
__device__ __forceinline__ float* paged_slot(const PagedParams& p, int cta, bool first, int tile, int quarter) {
  return p.slots + (static_cast<int64_t>((2 * cta + (first ? 1 : 0)) * 2 + tile) * 4 + quarter) * 32 * (D + 2);
}

// The buffer of uncut results: the prefix's rows by (key head, sequence, row of
// the sequence), then, from a multiple of 32 on, the own ones by (sequence, key
// head, row); both in groups of 32 rows laid out as the quarters of a slot.
__device__ __forceinline__ int buffer_row(const PagedParams& p, bool prefix, int pair, int r) {
  return pair * (p.Nq * p.G) + r + (prefix ? 0 : paged_rows32(p.B * p.Nq * p.Hq));
}
template <int D>
__device__ __forceinline__ float* buffer_o(const PagedParams& p, int i) {
  return p.rows_o + static_cast<int64_t>(i >> 5) * 32 * D + 4 * (i & 31);
}

template <int D>
__device__ void paged_softmax(const PagedParams& p, uint8_t* smem, const PBars<D>& bars, uint32_t tmem,
                              const Ctl& ctl) {
  using P = PCfg<D>;
  using C = Cfg<D>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h = (warp - 4) >> 2, quarter = warp & 3, row = quarter * 32 + lane;
  const uint32_t lane_base = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
  const uint32_t t_s = lane_base + (h ? C::tm_s(1) : C::tm_s(0)), t_o = lane_base + (h ? C::tm_o(1) : C::tm_o(0)),
                 t_p = lane_base + (h ? C::tm_p(1) : C::tm_p(0));
  float* xch = reinterpret_cast<float*>(smem + P::kOffX);
  const float c = p.c;
  uint32_t s_par = 0, o_par = 0, t_par = 0;
  uint32_t ring = 0;  // K and V tiles that the CTA took before this segment: the ring's position
  SegReader<D> segs;
  PSeg s;
  grid_dep_wait();
  while (segs.template take<kRoleSoftmax>(s, smem, bars, ctl)) {
    // the row inside its sequence's (queries x group) rows; the sequence; the lane has a row
    const int rs = p.Nq * p.G;
    int r = s.row0 + (s.twin() ? 0 : h * kBM) + row, bq = s.b;
    const bool real = r < s.rows;
    SeqLens sl;
    sl.len = s.len;
    sl.ql = s.ql;
    if (s.prefix()) {
      bq = p.by_rows.div(real ? r : s.row0);
      r -= bq * rs;
      if (p.row_limits) sl = seq_lens(p, bq);
    }
    // Keys that the row sees, the prefix's first. Lanes without a row see them
    // all: what they compute is never read, and they ask for no masking.
    int seen = 1 << 30;
    if (real && p.row_limits) seen = keys_seen(p, sl, p.by_g.div(r));
    const bool any = __any_sync(0xffffffffu, real && seen > 0);
    const bool twin = s.twin();
    float m_ref = -CUDART_INF_F, l = 0.f;
    bool first = true;
    for (int k = s.k0 + (twin ? h : 0); k < s.k1; k += twin ? 2 : 1) {
      // the tile's first key among the prefix's or the own keys, and how many of those there are
      const int base = (k < s.pt ? k : k - s.pt) * kBN, end = k < s.pt ? p.prefix_len : s.len;
      if (!warp_wait(bars.s_full(h), s_par, ctl, k)) return;
      s_par ^= 1u;
      tc_fence_after();
      const bool tail = base + kBN > end;
      if (any) {
        // One tile of scores, 64 keys at a time in a rolled loop: mask, running
        // maximum and sum, P as bf16 over S (P of keys [64 j, 64 j + 64) goes over
        // columns [32 j, 32 j + 32), read by then). The code is half of the
        // unrolled tile's, and fetching it is what a tile took when a CTA turned to
        // it once a task: 7000 cycles against 1300 in a long run of tiles. (When the
        // loop came in, 32 keys at a time took 138 us for a long prefix and 96
        // sequences, 64 took 125.)
        // A later piece whose maximum passes the reference by more than 2^8 brings
        // O, the sum and the pieces of P before it to its own (rare).
        const int lim = (k < s.pt ? min(seen, end) : min(seen - p.prefix_len, end)) - base;
        float2 sum2 = make_float2(0.f, 0.f);
#pragma unroll 1
        for (int j = 0; j < 2; ++j) {
          uint32_t sr[64], pk[32];
          tmem_ld64(t_s + 64 * j, sr);
          const int lj = lim - 64 * j;
          if (__any_sync(0xffffffffu, lj < 64)) {
#pragma unroll
            for (int i = 0; i < 64; ++i)
              if (i >= lj) sr[i] = __float_as_uint(-CUDART_INF_F);
          }
          float m4[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) m4[i] = fmaxf(__uint_as_float(sr[i]), __uint_as_float(sr[i + 4]));
#pragma unroll
          for (int i = 8; i < 64; i += 8)
#pragma unroll
            for (int q = 0; q < 4; ++q) m4[q] = fmax3(m4[q], __uint_as_float(sr[i + q]), __uint_as_float(sr[i + q + 4]));
          const float mx = fmax3(fmaxf(m4[0], m4[1]), m4[2], m4[3]);
          const float m_piece = (mx == -CUDART_INF_F) ? -CUDART_INF_F : mx * c;
          const bool grow = m_piece > m_ref + kRescaleLog2;
          if (__any_sync(0xffffffffu, grow)) {
            float alpha = 1.f;
            if (grow) {
              // The heaviest key's weight is 1, exact in bf16 (where it has most of the row, O is
              // some 20 % nearer: 0.0018 and not 0.0024 of its norm). If P of the piece before has
              // to follow, the step is a whole power of two: its weights are not rounded again.
              const float m_new = j > 0 && m_ref > -CUDART_INF_F ? m_ref + ceilf(m_piece - m_ref) : m_piece;
              alpha = ex2(m_ref - m_new);  // 0 while m_ref is still -inf
              m_ref = m_new;
              l *= alpha;
            }
            sum2 = __fmul2_rn(sum2, make_float2(alpha, alpha));
            // The piece before may have scaled O too, and stored P: both are read again here,
            // and stores to TMEM are not in order with the loads behind them.
            if (j > 0) tmem_wait_st();
            if (!first) rescale_o<D>(t_o, alpha);
            if (j > 0) {
              for (int q = 0; q < j; ++q) {
                uint32_t pp[32];
                tmem_ld32(t_p + 32 * q, pp);
#pragma unroll
                for (int i = 0; i < 32; ++i)
                  pp[i] = pack_bf16(__uint_as_float(pp[i] << 16) * alpha, __uint_as_float(pp[i] & 0xffff0000u) * alpha);
                tmem_st32(t_p + 32 * q, pp);
              }
            }
          }
          const float neg_m = (m_ref == -CUDART_INF_F) ? 0.f : -m_ref;
          const float2 c2 = make_float2(c, c), nm2 = make_float2(neg_m, neg_m);
          float2 part = make_float2(0.f, 0.f);
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const float2 y =
                __ffma2_rn(make_float2(__uint_as_float(sr[2 * i]), __uint_as_float(sr[2 * i + 1])), c2, nm2);
            const float2 pe = make_float2(ex2(y.x), ex2(y.y));
            if (i & 1) {
              part = __fadd2_rn(part, pe);
            } else {
              sum2 = __fadd2_rn(sum2, pe);
            }
            pk[i] = pack_bf16(pe.x, pe.y);
          }
          sum2 = __fadd2_rn(sum2, part);
          tmem_st32(t_p + 32 * j, pk);
        }
        l += sum2.x + sum2.y;
        tmem_wait_st();
        if (!tail) {
          tc_fence_before();
          __syncwarp();
          if (lane < 2) mbar_arrive(bars.p_full(h, lane));
        }
      } else if (!tail) {
        // no row of this warp sees a key of the task: its P and O are never read
        tc_fence_before();
        __syncwarp();
        if (lane < 2) mbar_arrive(bars.p_full(h, lane));
      }
      if (tail) {
        // The last tile of the prefix or of the own keys: V rows behind their end
        // become zero before P is announced. (After s_full: this tile's S went
        // out behind whatever held the V's stage before, so `full` is in this
        // tile's phase or past it, and the parity below cannot match an older one.)
        const int i = k - s.k0, n = s.k1 - s.k0, ahead = min(tiles_ahead(s), n);
        const uint32_t at = ring + static_cast<uint32_t>(ahead + i + min(i, n - ahead));
        const int st = static_cast<int>(at % P::kStages);
        if (!warp_wait(bars.full(st), (at / P::kStages) & 1u, ctl, k)) return;
        const int z0 = max(end - base, quarter * 32), z1 = quarter * 32 + 32;
        for (int ch = 0; ch < C::kChunks; ++ch) {
          uint8_t* v = smem + P::kOffKV + st * C::kTileBytes + ch * C::kChunkBytes;
          for (int i2 = z0 * C::kSwizzle + lane * 16; i2 < z1 * C::kSwizzle; i2 += 512)
            *reinterpret_cast<uint4*>(v + i2) = make_uint4(0, 0, 0, 0);
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        tc_fence_before();
        __syncwarp();
        if (lane < 2) mbar_arrive(bars.p_full(h, lane));
      }
      first = false;
    }

    ring += 2u * static_cast<uint32_t>(s.k1 - s.k0);
    // A score that is NaN makes the sum NaN but not the maximum (fmaxf drops it), which may
    // still be -inf, "saw no key", or so low that the join gives the part no weight. +inf
    // brings the NaN through every join: exp2 of inf - inf.
    if (l != l) m_ref = CUDART_INF_F;

    // the end of the segment: O of this row, to its part, its buffer or the result
    float m = m_ref, w0 = 1.f, w1 = 0.f;
    if (twin) {
      // Join the streams: each warpgroup takes half of the columns; the maxima
      // and sums go through shared memory. Both write after t_full, whose
      // products waited for o_empty, that is for every warp's reads of the task
      // before; and neither side can run a whole phase ahead of a warp that has
      // yet to look, since t_full needs them all.
      if (!warp_wait(bars.t_full(), t_par, ctl, -1)) return;
      float* mine = xch + h * 2 * kBM;
      const float* other = xch + (h ^ 1) * 2 * kBM;
      mine[row] = m_ref;
      mine[kBM + row] = l;
      __syncwarp();
      if (lane == 0) mbar_arrive(bars.x_full(h));
      if (!warp_wait(bars.x_full(h ^ 1), t_par, ctl, -1)) return;
      t_par ^= 1u;
      const float mo = other[row], lo = other[kBM + row];
      m = fmaxf(m_ref, mo);
      const float wm = m_ref == -CUDART_INF_F ? 0.f : ex2(m_ref - m), wo = mo == -CUDART_INF_F ? 0.f : ex2(mo - m);
      w0 = h ? wo : wm;
      w1 = h ? wm : wo;
      const float l0 = h ? lo : l, l1 = h ? l : lo;
      l = fmaf(l1, w1, l0 * w0);
    } else {
      if (!warp_wait(bars.o_full(h), o_par, ctl, -1)) return;
      o_par ^= 1u;
    }
    tc_fence_after();
    const bool none = m == -CUDART_INF_F;
    const bool lead = !twin || h == 0;  // writes the row's m and l
    const int n_ch = D / 32;
    const int ch0 = twin ? (h * n_ch + 1) / 2 : 0, ch1 = twin ? (h ? n_ch : (n_ch + 1) / 2) : n_ch;
    const bool direct = s.whole() && p.prefix_tasks == 0;
    if (__any_sync(0xffffffffu, real)) {
      // Where the row goes: its part of a cut task or its place in the buffer of
      // uncut results (float4 i at dst + 128 i in both: 32 rows side by side, so
      // that a warp's store is whole lines), or the result. (Trading 16-byte pieces
      // between lanes, to store the result in whole 64-byte pieces of rows, gained
      // nothing for 256 rows and took 15 % longer for 4: more code to fetch.)
      float* dst = nullptr;
      __nv_bfloat16* out = nullptr;
      float inv = 0.f;
      if (direct) {
        const int n = p.by_g.div(r);
        const int head = s.hk * p.G + r - n * p.G;
        if (real) out = static_cast<__nv_bfloat16*>(p.o) + bq * p.o_sb + head * p.o_sh + n * p.o_sn;
        inv = none ? 0.f : 1.f / l;
        if (real && lead && p.lse != nullptr)
          p.lse[(static_cast<int64_t>(bq) * p.Hq + head) * p.Nq + n] =
              none ? -CUDART_INF_F : (m + log2f(l)) * 0.69314718055994530942f;
      } else {
        float *pm, *pl;
        if (s.whole()) {
          const int i = buffer_row(p, s.prefix(), s.prefix() ? s.hk * p.B + bq : bq * p.Hk + s.hk, r);
          dst = buffer_o<D>(p, i);
          pm = reinterpret_cast<float*>(p.rows_ml + i);
          pl = pm + 1;
        } else {
          dst = paged_slot<D>(p, blockIdx.x, s.first(), twin ? 0 : h, quarter) + 4 * lane;
          pm = dst - 3 * lane + 32 * D;
          pl = pm + 32;
        }
        if (real && lead) {
          *pm = m;
          *pl = l;
        }
        if (!real || none) dst = nullptr;  // (a row that saw no key: its O is never read)
      }
#pragma unroll 1
      for (int ch = ch0; ch < ch1; ++ch) {
        __syncwarp();
        uint32_t a[32];
        float y[32];
        if (twin) {
          uint32_t b[32];
          tmem_ld32x2(lane_base + C::tm_o(0) + ch * 32, a, lane_base + C::tm_o(1) + ch * 32, b);
          if (s.k1 - s.k0 > 1) {
#pragma unroll
            for (int i = 0; i < 32; ++i) y[i] = fmaf(__uint_as_float(b[i]), w1, __uint_as_float(a[i]) * w0);
          } else {  // stream 1 had no tile: its O was not written
#pragma unroll
            for (int i = 0; i < 32; ++i) y[i] = __uint_as_float(a[i]);
          }
        } else {
          tmem_ld32(t_o + ch * 32, a);
#pragma unroll
          for (int i = 0; i < 32; ++i) y[i] = __uint_as_float(a[i]);
        }
        if (direct) {
          if (out != nullptr) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t w[4];
#pragma unroll
              for (int j = 0; j < 4; ++j)
                w[j] = none ? 0u : pack_bf16(y[8 * i + 2 * j] * inv, y[8 * i + 2 * j + 1] * inv);
              *reinterpret_cast<uint4*>(out + ch * 32 + 8 * i) = make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
        } else if (dst != nullptr) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            *reinterpret_cast<float4*>(dst + (ch * 8 + i) * 128) =
                make_float4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
        }
      }
    }
    tc_fence_before();
    __syncwarp();
    // both warpgroups' arrivals free a stream's O: two of a warp when only its own reads it
    if (twin) {
      if (lane < 2) mbar_arrive(bars.o_empty(lane));
    } else if (lane < 2) {
      mbar_arrive(bars.o_empty(h));
    }
    if (*ctl.abort) return;
  }
}

// ------------------------------------------------------------------ kernel

template <int D>
__global__ void __launch_bounds__(kThreads, 1) paged_kernel(const __grid_constant__ PagedParams p) {
  using P = PCfg<D>;
  // The swizzled tiles need 1024-byte alignment. Without static shared memory
  // the dynamic part starts at such an address; the five stages of d = 128
  // leave no room to align by hand, so a CTA that finds it otherwise reports it.
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  if ((sbase & 1023u) != 0u) {
    if (threadIdx.x == 0) atomicCAS(g_paged_status, 0u, 255u);
    return;
  }
  const int warp = threadIdx.x >> 5;
  const PBars<D> bars{sbase + P::kOffBar};
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + P::kOffBar + 8 * P::kBars);
  volatile uint32_t* abort_flag = tmem_slot + 1;

  if (threadIdx.x == 0) {
    for (int h = 0; h < 2; ++h) {
      mbar_init(bars.q_full(h), 1);
      mbar_init(bars.q_empty(h), 1);
      mbar_init(bars.s_full(h), 1);
      mbar_init(bars.p_full(h, 0), 4);
      mbar_init(bars.p_full(h, 1), 4);
      mbar_init(bars.o_full(h), 1);
      mbar_init(bars.o_empty(h), 8);
      mbar_init(bars.x_full(h), 4);
    }
    mbar_init(bars.done(), 1);
    mbar_init(bars.t_full(), 1);
    mbar_init(bars.q_asked(), 1);
    for (int s = 0; s < P::kSegs; ++s) {
      mbar_init(bars.seg_full(s), 1);
      mbar_init(bars.seg_empty(s), kWarps - 1);  // every warp but the scheduler
    }
    for (int s = 0; s < P::kStages; ++s) {
      mbar_init(bars.full(s), 1);
      mbar_init(bars.empty(s), 1);
    }
    *abort_flag = 0u;
    fence_barrier_init();
    prefetch_tmap(&p.tm_k);
    prefetch_tmap(&p.tm_v);
    if (p.q_map != 0) prefetch_tmap(&p.tm_q);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), Cfg<D>::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const Ctl ctl{abort_flag, g_paged_status, p.timeout_ns};
  // So far only shared memory and TMEM are touched; every role waits for the
  // previous kernel on the stream before its first global access.
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  if (warp < 4) {
    set_max_regs_dec<kRegsControl>();
    if (warp == 0) {
      paged_loader<D>(p, smem, sbase, bars, ctl);
    } else if (warp == 1) {
      paged_mma<D>(p, smem, sbase, bars, tmem, ctl);
    } else if (warp == 2) {
      paged_gather_q<D>(p, sbase, smem, bars, ctl);
    } else {
      paged_scheduler<D>(p, smem, bars, ctl);
    }
    __syncwarp();
  } else {
    set_max_regs_inc<kRegsSoftmax>();
    paged_softmax<D>(p, smem, bars, tmem, ctl);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, Cfg<D>::kTmemCols);
  }
}

// ------------------------------------------------------------------ joining the parts
//
// The parts of a row, in order: those of its prefix task, then those of its own
// task; each is a slot of a CTA (cut task) or a row of the row buffers (uncut).
// A warp joins four rows, eight lanes a row: lane j of a row holds part j's
// maximum, sum and address, and adds float4 j, j + 8, ... of every part. The
// slots keep 32 rows' float4 side by side, so four neighbouring rows read whole
// 64-byte pieces (one row a warp took 11 us for 20 parts of 2048 rows, 32 lines
// a load). Few rows may have many parts each: then the block's warps share four
// rows, each taking eight parts of every 32, and the first adds up what they found.
// kBatch parts' loads are in flight together: eight want twice the registers.
constexpr int kJoinWarps = 4;

template <int D, bool SPLIT, int kBatch>
__global__ void __launch_bounds__(kJoinWarps * 32, kBatch > 4 ? 2 : 4) paged_join_kernel(const __grid_constant__ PagedParams p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  grid_dep_wait();
  constexpr int kJ = D / 32;    // float4 of a lane
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane >> 2, which = lane & 3;  // which of the four rows
  const int rows = p.B * p.Nq * p.Hq;  // below 2^30
  // rows in the order (key head, sequence, query, head of the group): neighbours in the prefix's slots too
  const int at = (SPLIT ? static_cast<int>(blockIdx.x) : static_cast<int>(blockIdx.x) * kJoinWarps + warp) * 4 + which;
  const bool live = at < rows;
  const int rs = p.Nq * p.G, batch_rows = p.B * rs;
  const int hk = live ? p.by_batch_rows.div(at) : 0, rp = live ? at - hk * batch_rows : 0;
  const int b = p.by_rows.div(rp), r = rp - b * rs, bh = b * p.Hk + hk;
  const int t = r / kPagedTaskRows, tp = rp / kPagedTaskRows;

  // the row's two tasks: where their parts are, and the row inside the task
  struct Span {
    int c0, parts, in_task;  // parts 0: no key to see; 1: uncut
  };
  Span pre{0, 0, 0}, own{0, 0, 0};
  // (after a wait that ran out some entries were never written: whatever they hold must name slots that exist)
  const auto span = [&](int2 e, int in_task) {
    const int c0 = clampi(e.x, 0, p.grid - 1);
    return Span{c0, clampi(e.y, 0, p.grid - c0), in_task};
  };
  const int2 at_own = p.tasks[bh * p.own_tasks + t];  // (written only if the task has a tile)
  if (p.prefix_tasks > 0) {
    const int2 e = p.tasks[p.B * p.Hk * p.own_tasks + hk * p.prefix_tasks + tp];
    pre = span(e, rp - tp * kPagedTaskRows);
  }
  if (own_tiles(p, seq_lens(p, b), t).all > 0) own = span(at_own, r - t * kPagedTaskRows);
  // an uncut row without a batched prefix was written by the attention kernel
  const bool mine = live && !(p.prefix_tasks == 0 && own.parts == 1);
  const int parts = mine ? pre.parts + own.parts : 0;
  const int most = __reduce_max_sync(0xffffffffu, parts);
  if (SPLIT && warp > 0 && most <= 8) return;  // (the same for all of the block's warps)

  float4 acc[kJ];
#pragma unroll
  for (int j = 0; j < kJ; ++j) acc[j] = make_float4(0.f, 0.f, 0.f, 0.f);
  float M = -CUDART_INF_F, L = 0.f;
  for (int base = SPLIT ? 8 * warp : 0; base < most; base += SPLIT ? 8 * kJoinWarps : 8) {
    const int i = base + sub, count = parts - base;  // of this row, from here on
    const float* src = p.slots;  // float4 j of the row at src + 128 j
    float m = -CUDART_INF_F, l = 0.f;
    if (i < parts) {
      const bool is_pre = i < pre.parts;
      const Span s = is_pre ? pre : own;
      const int k = is_pre ? i : i - pre.parts;
      if (s.parts == 1) {
        const int x = buffer_row(p, is_pre, is_pre ? hk * p.B + b : bh, r);
        const float2 ml = p.rows_ml[x];
        m = ml.x;
        l = ml.y;
        src = buffer_o<D>(p, x);
      } else {
        const int quarter = (s.in_task % kBM) / 32, in_q = s.in_task % 32;
        const float* slot = paged_slot<D>(p, s.c0 + k, k == 0, s.in_task / kBM, quarter);
        m = slot[32 * D + in_q];
        l = slot[32 * D + 32 + in_q];
        src = slot + 4 * in_q;
      }
    }
    // the first batch's data is asked for beside the maxima, before they are known
    float4 v[kBatch][kJ];
    auto fetch = [&](int j0) {
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int holder = ((j0 + u) << 2) | which;
        const float* su = reinterpret_cast<const float*>(
            __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(src), holder));
        if (j0 + u < count) {
#pragma unroll
          for (int j = 0; j < kJ; ++j) v[u][j] = *reinterpret_cast<const float4*>(su + (sub + 8 * j) * 128);
        }
      }
    };
    fetch(0);
    float mx = m;
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    const float M1 = fmaxf(M, mx);
    const float old = M == -CUDART_INF_F ? 0.f : ex2(M - M1);
    const float w = m == -CUDART_INF_F ? 0.f : ex2(m - M1);
    float lw = w > 0.f ? l * w : 0.f;
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) lw += __shfl_xor_sync(0xffffffffu, lw, o);
    L = fmaf(L, old, lw);
    M = M1;
#pragma unroll
    for (int j = 0; j < kJ; ++j) {
      acc[j].x *= old;
      acc[j].y *= old;
      acc[j].z *= old;
      acc[j].w *= old;
    }
#pragma unroll
    for (int j0 = 0; j0 < 8; j0 += kBatch) {
      if (j0 > 0 && base + j0 < most) fetch(j0);
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const float wu = __shfl_sync(0xffffffffu, w, ((j0 + u) << 2) | which);
        // a part that saw no key for this row never wrote its O: left out, not weighted by zero
        if (j0 + u < count && wu > 0.f) {
#pragma unroll
          for (int j = 0; j < kJ; ++j) {
            acc[j].x = fmaf(v[u][j].x, wu, acc[j].x);
            acc[j].y = fmaf(v[u][j].y, wu, acc[j].y);
            acc[j].z = fmaf(v[u][j].z, wu, acc[j].z);
            acc[j].w = fmaf(v[u][j].w, wu, acc[j].w);
          }
        }
      }
    }
  }
  if constexpr (SPLIT) if (most > 8) {
    __shared__ float4 sh_acc[kJoinWarps - 1][kJ][32];
    __shared__ float2 sh_ml[kJoinWarps - 1][32];
    if (warp > 0) {
      sh_ml[warp - 1][lane] = make_float2(M, L);
#pragma unroll
      for (int j = 0; j < kJ; ++j) sh_acc[warp - 1][j][lane] = acc[j];
    }
    __syncthreads();
    if (warp > 0) return;
#pragma unroll
    for (int w = 0; w < kJoinWarps - 1; ++w) {
      const float2 ml = sh_ml[w][lane];
      const float M1 = fmaxf(M, ml.x);
      const float a = M == -CUDART_INF_F ? 0.f : ex2(M - M1), z = ml.x == -CUDART_INF_F ? 0.f : ex2(ml.x - M1);
      M = M1;
      L = fmaf(L, a, ml.y * z);
#pragma unroll
      for (int j = 0; j < kJ; ++j) {
        const float4 v = sh_acc[w][j][lane];
        acc[j].x = fmaf(acc[j].x, a, v.x * z);
        acc[j].y = fmaf(acc[j].y, a, v.y * z);
        acc[j].z = fmaf(acc[j].z, a, v.z * z);
        acc[j].w = fmaf(acc[j].w, a, v.w * z);
      }
    }
  }
  if (!mine) return;
  const int n = p.by_g.div(r), head = hk * p.G + r - n * p.G;
  const bool none = M == -CUDART_INF_F;
  const float inv = none ? 0.f : 1.f / L;
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.o) + b * p.o_sb + head * p.o_sh + n * p.o_sn + sub * 4;
#pragma unroll
  for (int j = 0; j < kJ; ++j) {
    uint2 w = make_uint2(0u, 0u);
    if (!none) w = make_uint2(pack_bf16(acc[j].x * inv, acc[j].y * inv), pack_bf16(acc[j].z * inv, acc[j].w * inv));
    *reinterpret_cast<uint2*>(out + 32 * j) = w;
  }
  if (sub == 0 && p.lse != nullptr)
    p.lse[(static_cast<int64_t>(b) * p.Hq + head) * p.Nq + n] =
        none ? -CUDART_INF_F : (M + log2f(L)) * 0.69314718055994530942f;
}

template <int D>
cudaError_t launch_paged_dim(const PagedParams& p, cudaStream_t s) {
  constexpr int smem = PCfg<D>::kSmemBytes > kMinSmemBytes ? PCfg<D>::kSmemBytes : kMinSmemBytes;  // one CTA an SM
  cudaError_t e = cudaFuncSetAttribute(paged_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.grid));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if ((e = cudaLaunchKernelEx(&cfg, paged_kernel<D>, p)) != cudaSuccess) return e;
  const int64_t rows = static_cast<int64_t>(p.B) * p.Nq * p.Hq;
  const int64_t per_block = p.join == PagedParams::kJoinSplit ? 4 : 4 * kJoinWarps;
  cfg.gridDim = dim3(static_cast<unsigned>((rows + per_block - 1) / per_block));
  cfg.blockDim = dim3(kJoinWarps * 32);
  cfg.dynamicSmemBytes = 0;
  const auto join = p.join == PagedParams::kJoinSplit ? paged_join_kernel<D, true, 8>
                    : p.join == PagedParams::kJoinFew ? paged_join_kernel<D, false, 8>
                                                      : paged_join_kernel<D, false, 4>;
  return cudaLaunchKernelEx(&cfg, join, p);
}

}  // namespace dev

cudaError_t launch_paged(const PagedParams& p, int d, cudaStream_t s) {
  switch (d) {
    case 32: return dev::launch_paged_dim<32>(p, s);
    case 64: return dev::launch_paged_dim<64>(p, s);
    case 128: return dev::launch_paged_dim<128>(p, s);
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t paged_take_status(uint32_t word[4]) {
  cudaError_t e = cudaMemcpyFromSymbol(word, dev::g_paged_status, 4 * sizeof(uint32_t), 0, cudaMemcpyDeviceToHost);
  if (e != cudaSuccess || word[0] == 0) return e;
  const uint32_t zero[4] = {0, 0, 0, 0};
  return cudaMemcpyToSymbol(dev::g_paged_status, zero, sizeof(zero), 0, cudaMemcpyHostToDevice);
}

}  // namespace attn
