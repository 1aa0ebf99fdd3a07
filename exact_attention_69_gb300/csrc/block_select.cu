// block_select.cu -- choosing: the pages that a query reads, the tokens that a cache
// keeps; and moving the kept tokens.
//
// Both choices are the k greatest of a row's values between two runs that are always
// taken (the first ones and the last ones), ties to the lowest index, listed in
// ascending order. Values become unsigned keys of the same order (NaN above
// everything, -0 equal to +0). A team of threads holds a row's keys in registers, each
// warp a run of consecutive ones, and finds the k-th greatest key digit by digit, from the
// highest bit in which keys differ: a count of each digit among the keys that agree so
// far, in shared memory (whole numbers: the order of the additions does not matter), until
// the keys of a digit are wanted all. Ballots then place the keys above it and the
// first of those equal to it. (Bit by bit with a count over the team each: 6.1 us for 256
// rows of 512 pages, 63.7 for an eviction of 48 rows of 32768 tokens; by digits 5.2 and
// 54.8, of which the choice is 23 and instructions set its pace, the move 32, memory, 6.4
// TB/s.) Rows of up to 1024 values take a warp each, longer ones a block, rows beyond what
// a block's registers hold (16384 pages, 32768 tokens) are read again for each digit.
#include "long_dev.cuh"
#include "long_kernel.h"

namespace attn {
namespace {

using namespace ldev;

__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);
  if (x != x) return 0xFFFFFFFFu;
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// A team of T threads: one warp, or a block.
constexpr int kBins = 256;
template <int T>
struct Team {
  static_assert(T == 32 || (T % 32 == 0 && T <= 1024), "team");
  struct Shared {
    __align__(16) uint32_t bins[2][kBins];
    uint32_t words[2][T / 32];
  };
  int rank, turn = 0, pass = 0;
  Shared& sh;
  __device__ __forceinline__ Team(Shared& s) : rank(threadIdx.x % T), sh(s) {}
  __device__ __forceinline__ int lane() const { return rank % 32; }
  __device__ __forceinline__ int warp() const { return rank / 32; }
  __device__ __forceinline__ void barrier() {
    if constexpr (T == 32)
      __syncwarp();
    else
      __syncthreads();
  }
  // A value of every warp, in lane w that of warp w (others 0).
  __device__ __forceinline__ uint32_t gather(uint32_t x) {
    uint32_t* s = sh.words[turn ^= 1];  // (one barrier a call: the other half may still be read)
    if (lane() == 0) s[warp()] = x;
    __syncthreads();
    return lane() < T / 32 ? s[lane()] : 0u;
  }
  __device__ __forceinline__ uint32_t any_of(uint32_t x) {
    x = __reduce_or_sync(0xffffffffu, x);
    return T == 32 ? x : __reduce_or_sync(0xffffffffu, gather(x));
  }
  // Of a count that is the same in all lanes of a warp: that of the warps before; `all`
  // gets the sum.
  __device__ __forceinline__ uint32_t before(uint32_t x, uint32_t* all) {
    if constexpr (T == 32) {
      *all = x;
      return 0u;
    }
    const uint32_t w = gather(x);
    *all = __reduce_add_sync(0xffffffffu, w);
    return __reduce_add_sync(0xffffffffu, lane() < warp() ? w : 0u);
  }
  // Counts of digits, in the two sets in turn: those of the pass before may still be read.
  __device__ __forceinline__ uint32_t* clear() {
    uint32_t* h = sh.bins[pass ^= 1];
    for (int x = rank; x < kBins; x += T) h[x] = 0;
    barrier();
    return h;
  }
  // The digit that holds the `left`-th key from the top; `left` becomes its rank among
  // the digit's keys, `count` their number.
  __device__ __forceinline__ uint32_t digit(const uint32_t* h, uint32_t& left, uint32_t& count) {
    barrier();
    uint32_t v[8], s = 0;  // from the greatest digit down
    const uint4 a = reinterpret_cast<const uint4*>(h)[63 - 2 * lane()], b = reinterpret_cast<const uint4*>(h)[62 - 2 * lane()];
    v[0] = a.w, v[1] = a.z, v[2] = a.y, v[3] = a.x, v[4] = b.w, v[5] = b.z, v[6] = b.y, v[7] = b.x;
#pragma unroll
    for (int x = 0; x < 8; ++x) s += v[x];
    uint32_t up = s;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, up, o);
      if (lane() >= o) up += y;
    }
    const int at = __ffs(__ballot_sync(0xffffffffu, up >= left)) - 1;
    uint32_t rest = left - (up - s), d = 0, c = 0;  // (what matters in lane `at`)
    bool found = false;
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      if (!found && rest <= v[x]) {
        found = true;
        d = 255u - 8u * lane() - x;
        c = v[x];
      }
      if (!found) rest -= v[x];
    }
    left = __shfl_sync(0xffffffffu, rest, at);
    count = __shfl_sync(0xffffffffu, c, at);
    return __shfl_sync(0xffffffffu, d, at);
  }
};

// The k greatest of the values at [lo, hi), 1 <= k < hi - lo, hi <= T * E, ascending to
// out. Warp w has the values 32 E w ..; lane x has runs of V neighbouring ones, run e
// beginning at number 32 V e + V x of them. at(x, v): values x .. x + V - 1 (x a multiple
// of V below hi; what lies behind hi may be anything).
template <int T, int E, int V, typename At>
__device__ __forceinline__ void pick(Team<T>& team, At at, int lo, int hi, int k, int32_t* out) {
  static_assert(E % V == 0, "whole runs");
  uint32_t key[E];
  const int first = team.warp() * 32 * E + team.lane() * V;
  const auto place = [&](int e) { return first + e / V * (32 * V) + e % V; };
  uint32_t ones = 0, zeros = 0;
#pragma unroll
  for (int e = 0; e < E; e += V) {  // (unconditional: all loads at once)
    float v[V];
    at(min(place(e), (hi - 1) / V * V), v);
#pragma unroll
    for (int i = 0; i < V; ++i) key[e + i] = __float_as_uint(v[i]);
  }
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const bool in = place(e) >= lo && place(e) < hi;
    key[e] = in ? key_of(__uint_as_float(key[e])) : 0u;  // (no value has the key 0)
    ones |= key[e];
    zeros |= in ? ~key[e] : 0u;
  }
  ones = team.any_of(ones);
  const uint32_t open = ones & team.any_of(zeros);
  int bits = 32 - __clz(open);  // low bits that are not known yet; the keys agree above them
  uint32_t t = bits == 32 ? 0u : (ones >> bits) << bits, left = static_cast<uint32_t>(k);
  bool ties = true, all_agree = true;  // ties: more keys than wanted may be equal to t
  while (bits > 0) {
    const int shift = max(bits - 8, 0);
    const uint32_t mask = (1u << (bits - shift)) - 1u;
    uint32_t* h = team.clear();
    if (all_agree) {
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (key[e] != 0u) atomicAdd(h + ((key[e] >> shift) & mask), 1u);
    } else {  // (bits < 32)
      // While t is 0 (the k-th value is -inf, or next to the type's lowest) places outside [lo, hi), of key
      // 0, are counted as well, in digit 0. That is below all that is wanted: this digit begins at bit 15 or
      // 16 then, and the least key of a value is 0x007FFFFF, so values have 0x7F or more there; from the
      // next pass on t is not 0.
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (((key[e] ^ t) >> bits) == 0u) atomicAdd(h + ((key[e] >> shift) & mask), 1u);
    }
    uint32_t count;
    t |= team.digit(h, left, count) << shift;
    bits = shift;
    all_agree = false;
    if (count == left) {
      ties = false;
      break;
    }
  }
  if (!ties) t -= 1;  // all keys from t up (t is not 0: some key lies below it)
  uint32_t above = 0, equal = 0, all;
#pragma unroll
  for (int e = 0; e < E; ++e) above += key[e] > t;
  uint32_t a = team.before(__reduce_add_sync(0xffffffffu, above), &all);
  const uint32_t mine = (1u << team.lane()) - 1u;
  if (!ties) {
#pragma unroll
    for (int e = 0; e < E; e += V) {
      uint32_t up[V], n = a;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        up[i] = __ballot_sync(0xffffffffu, key[e + i] > t);
        n += __popc(up[i] & mine);
        a += __popc(up[i]);
      }
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (key[e + i] > t) out[n++] = place(e + i);
    }
    return;
  }
#pragma unroll
  for (int e = 0; e < E; ++e) equal += key[e] == t;
  uint32_t q = team.before(__reduce_add_sync(0xffffffffu, equal), &all);
#pragma unroll
  for (int e = 0; e < E; e += V) {
    uint32_t n = a, m = q;  // of those above t, and equal to it, before this lane's run
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const uint32_t up = __ballot_sync(0xffffffffu, key[e + i] > t), eq = __ballot_sync(0xffffffffu, key[e + i] == t);
      n += __popc(up & mine);
      a += __popc(up);
      m += __popc(eq & mine);
      q += __popc(eq);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const bool eq = key[e + i] == t;
      if (key[e + i] > t || (eq && m < left)) out[n + min(m, left)] = place(e + i);  // (left: of the equal ones, the first)
      n += key[e + i] > t;
      m += eq;
    }
  }
}

// The same for rows of any length: the row is read again for every digit and for the
// placing.
template <int T, typename At>
__device__ __forceinline__ void pick_long(Team<T>& team, At at, int lo, int hi, int k, int32_t* out) {
  uint32_t t = 0, left = static_cast<uint32_t>(k), count;
  for (int bits = 32; bits > 0; bits -= 8) {
    uint32_t* h = team.clear();
    for (int x = lo + team.rank; x < hi; x += T) {
      const uint32_t key = key_of(at(x));
      if (bits == 32 || ((key ^ t) >> bits) == 0u) atomicAdd(h + ((key >> (bits - 8)) & 255u), 1u);
    }
    t |= team.digit(h, left, count) << (bits - 8);
  }
  uint32_t done = 0, tied = 0;
  const uint32_t mine = (1u << team.lane()) - 1u;
  for (int x0 = lo; x0 < hi; x0 += T) {
    const int x = x0 + team.rank;
    const uint32_t key = x < hi ? key_of(at(x)) : 0u;
    const bool eq = x < hi && key == t;
    uint32_t all;
    const uint32_t same = __ballot_sync(0xffffffffu, eq);
    const uint32_t q = tied + team.before(__popc(same), &all) + __popc(same & mine);
    tied += all;
    const bool take = key > t || (eq && q < left);
    const uint32_t took = __ballot_sync(0xffffffffu, take);
    const uint32_t a = done + team.before(__popc(took), &all) + __popc(took & mine);
    done += all;
    if (take) out[a] = x;
  }
}

// A row of `n` values, `take` to be taken, the first `first` and last `last` among them
// for sure; -1 behind them in out[0, width).
template <int T, int E, int V, bool LONG, typename At>
__device__ __forceinline__ void choose(Team<T>& team, At at, int n, int take, int first, int last, int width, int32_t* out) {
  if (n <= take) {
    for (int x = team.rank; x < width; x += T) out[x] = x < n ? x : -1;
    return;
  }
  const int k = take - first - last;
  for (int x = team.rank; x < first; x += T) out[x] = x;
  for (int x = team.rank; x < last; x += T) out[take - last + x] = n - last + x;
  for (int x = take + team.rank; x < width; x += T) out[x] = -1;
  if (k <= 0) return;
  if constexpr (LONG)
    pick_long<T>(
        team,
        [&](int x) {
          float v[1];
          at(x, v);
          return v[0];
        },
        first, n - last, k, out + first);
  else
    pick<T, E, V>(team, at, first, n - last, k, out + first);
}

// ------------------------------------------------------------------ pages of a query

template <int T, int E, bool LONG>
__global__ void __launch_bounds__(T < 128 ? 128 : T) select_kernel(const __grid_constant__ LongParams p) {
  __shared__ typename Team<T>::Shared shared[T == 32 ? 4 : 1];
  grid_dep_wait();
  grid_dep_launch();
  const int64_t row = T == 32 ? static_cast<int64_t>(blockIdx.x) * 4 + threadIdx.x / 32 : blockIdx.x;
  if (row >= static_cast<int64_t>(p.B) * p.Hk * p.Nq) return;  // (a warp's own row: no block barrier follows)
  const int i = static_cast<int>(row % p.Nq), b = static_cast<int>(row / (static_cast<int64_t>(p.Nq) * p.Hk));
  const int n = min(long_pages(p, long_seen(p, long_lens(p, b), i)), p.table_width);
  const float* s = p.scores + row * p.table_width;
  Team<T> team(shared[T == 32 ? threadIdx.x / 32 : 0]);
  choose<T, E, 1, LONG>(team, [&](int x, float(&v)[1]) { v[0] = s[x]; }, n, p.n, p.first, p.last, p.n, p.blocks + row * p.n);
}

// ------------------------------------------------------------------ tokens of a cache

template <int T, int E, bool LONG>
__global__ void __launch_bounds__(T) keep_kernel(const __grid_constant__ LongParams p) {
  __shared__ typename Team<T>::Shared shared;
  grid_dep_wait();
  grid_dep_launch();
  const int hk = blockIdx.x % p.Hk, b = blockIdx.x / p.Hk;
  const int n = min(max(p.kv_lens[b], 0), p.max_len);
  if (hk == 0 && threadIdx.x == 0) p.new_lens[b] = min(n, p.n);
  const int32_t* table = p.table + b * p.table_sb;
  const int mask = (1 << p.page_shift) - 1;
  Team<T> team(shared);
  // (a page's weights are contiguous, and aligned to 16 bytes)
  constexpr int V = LONG ? 1 : 4;
  const auto at = [&](int x, float(&v)[V]) {
    const int id = table[x >> p.page_shift];
    const bool real = id >= 0 && id < p.n_pages;
    const float* w = p.weights + ((static_cast<int64_t>(real ? id : 0) * p.Hk + hk) << p.page_shift) + (x & mask);
    if constexpr (V == 4) {
      const float4 y = *reinterpret_cast<const float4*>(w);
      v[0] = y.x, v[1] = y.y, v[2] = y.z, v[3] = y.w;
    } else {
      v[0] = *w;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = real ? v[i] : 0.f;
  };
  choose<T, E, V, LONG>(team, at, n, p.n, p.first, p.last, p.n, p.kept + (static_cast<int64_t>(b) * p.Hk + hk) * p.n);
}

// Moves the kept tokens. Token x of the list goes to place x, which is no later than
// where it comes from, so in place a block goes over its list in order: what a step
// writes (places below its end) was read in it or before (sources of later steps are
// all at or behind its end). Blocks of one list differ in the bytes of a token that
// they take, never in tokens. Into other pages the lists are cut freely.
constexpr int kMoveThreads = 256, kMoveDeep = 4;  // tokens that a thread has in flight

template <int D, bool IN_PLACE>
__global__ void __launch_bounds__(kMoveThreads) move_kernel(const __grid_constant__ LongParams p) {
  // 16-byte pieces of a token's key, and of its value, that a block takes
  constexpr int kPieces = IN_PLACE ? 4 : D / 8, kSlices = D / 8 / kPieces;
  constexpr int kTokens = kMoveThreads / kPieces;
  grid_dep_wait();
  grid_dep_launch();
  const int slice = blockIdx.x % kSlices, hk = blockIdx.y, b = blockIdx.z;
  const int piece = slice * kPieces + threadIdx.x % kPieces, row = threadIdx.x / kPieces;
  const int n = min(min(max(p.kv_lens[b], 0), p.max_len), p.n);
  const int32_t* kept = p.kept + (static_cast<int64_t>(b) * p.Hk + hk) * p.n;
  const int32_t *from = p.table + b * p.table_sb, *to = IN_PLACE ? from : p.dst + b * p.dst_sb;
  const int to_width = IN_PLACE ? p.table_width : p.dst_width;
  __nv_bfloat16* kc = static_cast<__nv_bfloat16*>(p.kc) + hk * p.kc_sh + piece * 8;
  __nv_bfloat16* vc = static_cast<__nv_bfloat16*>(p.vc) + hk * p.vc_sh + piece * 8;
  const int mask = (1 << p.page_shift) - 1;
  const auto weight = [&](int id, int at) {
    return p.weights_out + (((static_cast<int64_t>(id) * p.Hk + hk) << p.page_shift) + (at & mask));
  };
  int x = IN_PLACE ? 0 : static_cast<int>(blockIdx.x / kSlices) * kTokens * kMoveDeep;
  const int end = IN_PLACE ? n : min(n, x + kTokens * kMoveDeep);
  for (; x < end; x += kTokens * kMoveDeep) {
    int src[kMoveDeep], from_id[kMoveDeep], to_id[kMoveDeep];
    uint4 k[kMoveDeep], v[kMoveDeep];
    float w[kMoveDeep];
#pragma unroll
    for (int e = 0; e < kMoveDeep; ++e) {
      const int at = x + e * kTokens + row;
      src[e] = at < end ? kept[at] : -1;
      to_id[e] = at < end && (at >> p.page_shift) < to_width ? to[at >> p.page_shift] : -1;
    }
#pragma unroll
    for (int e = 0; e < kMoveDeep; ++e) from_id[e] = src[e] >= 0 ? from[src[e] >> p.page_shift] : -1;
#pragma unroll
    for (int e = 0; e < kMoveDeep; ++e) {
      k[e] = v[e] = make_uint4(0, 0, 0, 0);
      w[e] = 0.f;
      if (from_id[e] >= 0 && from_id[e] < p.n_pages) {
        const int64_t at = src[e] & mask;
        k[e] = *reinterpret_cast<const uint4*>(kc + from_id[e] * p.kc_sp + at * p.kc_st);
        v[e] = *reinterpret_cast<const uint4*>(vc + from_id[e] * p.vc_sp + at * p.vc_st);
        if (piece == 0) w[e] = *weight(from_id[e], src[e]);
      }
    }
    if constexpr (IN_PLACE) __syncthreads();
#pragma unroll
    for (int e = 0; e < kMoveDeep; ++e) {
      const int at = x + e * kTokens + row;
      if (to_id[e] < 0 || to_id[e] >= p.n_pages || (IN_PLACE && src[e] == at)) continue;
      const int64_t place = at & mask;
      *reinterpret_cast<uint4*>(kc + to_id[e] * p.kc_sp + place * p.kc_st) = k[e];
      *reinterpret_cast<uint4*>(vc + to_id[e] * p.vc_sp + place * p.vc_st) = v[e];
      if (piece == 0) *weight(to_id[e], at) = w[e];
    }
  }
}

template <int D>
cudaError_t move_dim(const LongParams& p, cudaStream_t s) {
  if (p.dst == nullptr)
    return launch(move_kernel<D, true>, dim3(D / 32, p.Hk, p.B), kMoveThreads, 0, s, 1, p);
  constexpr int kTokens = kMoveThreads / (D / 8) * kMoveDeep;
  const int most = p.n < p.max_len ? p.n : p.max_len;
  return launch(move_kernel<D, false>, dim3(static_cast<unsigned>((most + kTokens - 1) / kTokens), p.Hk, p.B),
                kMoveThreads, 0, s, 1, p);
}

}  // namespace

// A warp takes a row of up to 1024 values, a block longer ones. Both for rows of 100, 500 and 1000 values (us):
// 256 rows 3.7, 5.2, 7.7 by warps and 4.5, 4.5, 4.6 by blocks of 256; 2048 rows 4.4, 6.8, 11.1 and 13.6,
// 14.3, 15.1; 8192 rows 8.6, 15.7, 27.4 and 45, 48, 50.
cudaError_t launch_select(const LongParams& p, cudaStream_t s) {
  const int64_t rows = static_cast<int64_t>(p.B) * p.Hk * p.Nq;
  const dim3 warps(static_cast<unsigned>((rows + 3) / 4)), blocks(static_cast<unsigned>(rows));
  const int w = p.table_width;
  if (w <= 128) return launch(select_kernel<32, 4, false>, warps, 128, 0, s, 1, p);
  if (w <= 512) return launch(select_kernel<32, 16, false>, warps, 128, 0, s, 1, p);
  if (w <= 1024) return launch(select_kernel<32, 32, false>, warps, 128, 0, s, 1, p);
  if (w <= 4096) return launch(select_kernel<256, 16, false>, blocks, 256, 0, s, 1, p);
  if (w <= 16384) return launch(select_kernel<1024, 16, false>, blocks, 1024, 0, s, 1, p);
  return launch(select_kernel<1024, 1, true>, blocks, 1024, 0, s, 1, p);
}

cudaError_t launch_evict(const LongParams& p, int d, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>(p.B) * static_cast<unsigned>(p.Hk));
  cudaError_t e;
  if (p.max_len <= 2048)
    e = launch(keep_kernel<256, 8, false>, grid, 256, 0, s, 1, p);
  else if (p.max_len <= 4096)
    e = launch(keep_kernel<1024, 4, false>, grid, 1024, 0, s, 1, p);
  else if (p.max_len <= 16384)
    e = launch(keep_kernel<1024, 16, false>, grid, 1024, 0, s, 1, p);
  else if (p.max_len <= 32768)
    e = launch(keep_kernel<1024, 32, false>, grid, 1024, 0, s, 1, p);
  else
    e = launch(keep_kernel<1024, 1, true>, grid, 1024, 0, s, 1, p);
  if (e != cudaSuccess) return e;
  switch (d) {
    case 32: return move_dim<32>(p, s);
    case 64: return move_dim<64>(p, s);
    case 128: return move_dim<128>(p, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace attn
