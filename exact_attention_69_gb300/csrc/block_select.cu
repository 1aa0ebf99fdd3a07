// block_select.cu -- choosing: the pages that a query reads, the tokens that a cache
// keeps; and moving the kept tokens.
//
// Both choices are the k greatest of a row's values between two runs that are always
// taken (the first ones and the last ones), ties to the lowest index, listed in
// ascending order. Values become unsigned keys of the same order (NaN above
// everything, -0 equal to +0). A team of threads holds a row's keys in registers, each
// thread a run of consecutive ones, and finds the k-th greatest key bit by bit from the
// top: the largest T that at least k keys reach. One scan over the team then places
// the keys above T and the first of those equal to it. No atomics, so the same row
// always gives the same answer.
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
template <int T>
struct Team {
  static_assert(T == 32 || (T % 32 == 0 && T <= 1024), "team");
  int rank;
  uint32_t* sums;  // shared, two times T / 32 words
  int turn = 0;
  __device__ __forceinline__ Team(uint32_t* s) : rank(threadIdx.x % T), sums(s) {}

  // Sum over the team.
  __device__ __forceinline__ uint32_t sum(uint32_t x) {
    x = __reduce_add_sync(0xffffffffu, x);
    if constexpr (T > 32) {
      uint32_t* s = sums + (turn ^= T / 32);
      if (rank % 32 == 0) s[rank / 32] = x;
      __syncthreads();
      x = __reduce_add_sync(0xffffffffu, rank % 32 < T / 32 ? s[rank % 32] : 0u);
    }
    return x;
  }
  // What the threads before this one have together; `all` gets the team's sum.
  __device__ __forceinline__ uint32_t before(uint32_t x, uint32_t* all) {
    uint32_t z = x;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, z, o);
      if (rank % 32 >= o) z += y;
    }
    if constexpr (T > 32) {
      uint32_t* s = sums + (turn ^= T / 32);
      if (rank % 32 == 31) s[rank / 32] = z;
      __syncthreads();
      uint32_t w = rank % 32 < T / 32 ? s[rank % 32] : 0u;
#pragma unroll
      for (int o = 1; o < 32; o *= 2) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, w, o);
        if (rank % 32 >= o) w += y;
      }
      *all = __shfl_sync(0xffffffffu, w, T / 32 - 1);
      const uint32_t prev = __shfl_sync(0xffffffffu, w, max(rank / 32 - 1, 0));
      return z - x + (rank >= 32 ? prev : 0u);
    }
    *all = __shfl_sync(0xffffffffu, z, 31);
    return z - x;
  }
};

// The k greatest of the values at [lo, hi), 1 <= k < hi - lo <= T * E, ascending to out.
template <int T, int E, typename At>
__device__ __forceinline__ void pick(Team<T>& team, At at, int lo, int hi, int k, int32_t* out) {
  uint32_t key[E];
  const int first = lo + team.rank * E;
#pragma unroll
  for (int e = 0; e < E; ++e) key[e] = first + e < hi ? key_of(at(first + e)) : 0u;
  uint32_t t = 0;
  for (uint32_t bit = 0x80000000u; bit != 0; bit >>= 1) {
    uint32_t c = 0;
#pragma unroll
    for (int e = 0; e < E; ++e) c += key[e] >= (t | bit);
    if (team.sum(c) >= static_cast<uint32_t>(k)) t |= bit;
  }
  // (places behind hi have key 0, which no value has)
  uint32_t above = 0, equal = 0, all;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    above += key[e] > t;
    equal += key[e] == t;
  }
  uint32_t a = team.before(above, &all);
  const uint32_t ties = static_cast<uint32_t>(k) - all;  // of those equal to t, the first
  uint32_t q = team.before(equal, &all);
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const bool up = key[e] > t, eq = key[e] == t;
    if (up || (eq && q < ties)) out[a + min(q, ties)] = first + e;
    a += up;
    q += eq;
  }
}

// The same for rows of any length: the row is read again for every digit of 8 bits and
// for the placing.
template <int T, typename At>
__device__ __forceinline__ void pick_long(Team<T>& team, uint32_t* hist, At at, int lo, int hi, int k, int32_t* out) {
  uint32_t t = 0;
  int left = k;  // of the keys that agree with t so far, how many are wanted
  for (int shift = 24; shift >= 0; shift -= 8) {
    __syncthreads();
    for (int x = team.rank; x < 256; x += T) hist[x] = 0;
    __syncthreads();
    for (int x = lo + team.rank; x < hi; x += T) {
      const uint32_t key = key_of(at(x));
      if (shift == 24 || (key >> (shift + 8)) == (t >> (shift + 8))) atomicAdd(hist + ((key >> shift) & 255u), 1u);
    }
    __syncthreads();
    int digit = 255;
    uint32_t c = 0;
    while (digit > 0 && c + hist[digit] < static_cast<uint32_t>(left)) c += hist[digit--];
    left -= static_cast<int>(c);
    t |= static_cast<uint32_t>(digit) << shift;
  }
  uint32_t done = 0, tied = 0;
  for (int x0 = lo; x0 < hi; x0 += T) {
    const int x = x0 + team.rank;
    const uint32_t key = x < hi ? key_of(at(x)) : 0u;
    const bool eq = x < hi && key == t;
    uint32_t all;
    const uint32_t q = tied + team.before(eq, &all);
    tied += all;
    const bool take = key > t || (eq && q < static_cast<uint32_t>(left));
    const uint32_t a = done + team.before(take, &all);
    done += all;
    if (take) out[a] = x;
  }
}

// A row of `n` values, `take` to be taken, the first `first` and last `last` among them
// for sure; -1 behind them in out[0, width).
template <int T, int E, bool LONG, typename At>
__device__ __forceinline__ void choose(Team<T>& team, uint32_t* hist, At at, int n, int take, int first, int last,
                                       int width, int32_t* out) {
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
    pick_long<T>(team, hist, at, first, n - last, k, out + first);
  else
    pick<T, E>(team, at, first, n - last, k, out + first);
}

// ------------------------------------------------------------------ pages of a query

template <int T, int E, bool LONG>
__global__ void __launch_bounds__(T < 128 ? 128 : T) select_kernel(const __grid_constant__ LongParams p) {
  __shared__ uint32_t sums[T > 32 ? 2 * (T / 32) : 1];
  __shared__ uint32_t hist[LONG ? 256 : 1];
  grid_dep_wait();
  grid_dep_launch();
  const int64_t row = T == 32 ? static_cast<int64_t>(blockIdx.x) * 4 + threadIdx.x / 32 : blockIdx.x;
  if (row >= static_cast<int64_t>(p.B) * p.Hk * p.Nq) return;  // (a warp's own row: no block barrier follows)
  const int i = static_cast<int>(row % p.Nq), b = static_cast<int>(row / (static_cast<int64_t>(p.Nq) * p.Hk));
  const int n = min(long_pages(p, long_seen(p, long_lens(p, b), i)), p.table_width);
  const float* s = p.scores + row * p.table_width;
  Team<T> team(sums);
  choose<T, E, LONG>(team, hist, [&](int x) { return s[x]; }, n, p.n, p.first, p.last, p.n, p.blocks + row * p.n);
}

// ------------------------------------------------------------------ tokens of a cache

template <int T, int E, bool LONG>
__global__ void __launch_bounds__(T) keep_kernel(const __grid_constant__ LongParams p) {
  __shared__ uint32_t sums[2 * (T / 32)];
  __shared__ uint32_t hist[LONG ? 256 : 1];
  grid_dep_wait();
  grid_dep_launch();
  const int hk = blockIdx.x % p.Hk, b = blockIdx.x / p.Hk;
  const int n = min(max(p.kv_lens[b], 0), p.max_len);
  if (hk == 0 && threadIdx.x == 0) p.new_lens[b] = min(n, p.n);
  const int32_t* table = p.table + b * p.table_sb;
  const int mask = (1 << p.page_shift) - 1;
  Team<T> team(sums);
  const auto at = [&](int x) {
    const int id = table[x >> p.page_shift];
    return id >= 0 && id < p.n_pages ? p.weights[((static_cast<int64_t>(id) * p.Hk + hk) << p.page_shift) + (x & mask)] : 0.f;
  };
  choose<T, E, LONG>(team, hist, at, n, p.n, p.first, p.last, p.n, p.kept + (static_cast<int64_t>(b) * p.Hk + hk) * p.n);
}

// Moves the kept tokens. Token x of the list goes to place x, which is no later than
// where it comes from, so in place a block goes over its list in order: what a step
// writes (places below its end) was read in it or before (sources of later steps are
// all at or behind its end). Blocks of one list differ in the bytes of a token that
// they take, never in tokens. Into other pages the lists are cut freely.
constexpr int kMoveThreads = 256;

template <int D, bool IN_PLACE>
__global__ void __launch_bounds__(kMoveThreads) move_kernel(const __grid_constant__ LongParams p, int steps) {
  constexpr int kPieces = 4;                       // 16-byte pieces of a token that a block takes
  constexpr int kSlices = D / 8 / kPieces;         // blocks of K, and of V, for one list
  constexpr int kTokens = kMoveThreads / kPieces;  // tokens a step
  grid_dep_wait();
  grid_dep_launch();
  const int slice = blockIdx.x % (2 * kSlices), hk = blockIdx.y, b = blockIdx.z;
  const bool values = slice >= kSlices;
  const int piece = (slice % kSlices) * kPieces + threadIdx.x % kPieces;
  const int n = min(min(max(p.kv_lens[b], 0), p.max_len), p.n);
  const int32_t* kept = p.kept + (static_cast<int64_t>(b) * p.Hk + hk) * p.n;
  const int32_t *from = p.table + b * p.table_sb, *to = IN_PLACE ? from : p.dst + b * p.dst_sb;
  const int to_width = IN_PLACE ? p.table_width : p.dst_width;
  __nv_bfloat16* cache = static_cast<__nv_bfloat16*>(values ? p.vc : p.kc) + hk * (values ? p.vc_sh : p.kc_sh) + piece * 8;
  const int64_t sp = values ? p.vc_sp : p.kc_sp, st = values ? p.vc_st : p.kc_st;
  const int mask = (1 << p.page_shift) - 1;
  const bool weigh = slice == 0 && threadIdx.x % kPieces == 0 && p.weights_out != nullptr;
  int x = IN_PLACE ? 0 : static_cast<int>(blockIdx.x / (2 * kSlices)) * steps * kTokens;
  const int end = IN_PLACE ? n : min(n, x + steps * kTokens);
  for (; x < end; x += kTokens) {
    const int at = x + static_cast<int>(threadIdx.x) / kPieces;
    int src = -1, to_id = -1, from_id = -1;
    if (at < end) {
      src = kept[at];
      from_id = from[src >> p.page_shift];
      if ((at >> p.page_shift) < to_width) to_id = to[at >> p.page_shift];
    }
    const bool go = to_id >= 0 && to_id < p.n_pages && !(IN_PLACE && src == at), real = from_id >= 0 && from_id < p.n_pages;
    uint4 v = make_uint4(0, 0, 0, 0);
    float w = 0.f;
    if (go && real) {
      v = *reinterpret_cast<const uint4*>(cache + from_id * sp + (src & mask) * st);
      if (weigh) w = p.weights_out[((static_cast<int64_t>(from_id) * p.Hk + hk) << p.page_shift) + (src & mask)];
    }
    if constexpr (IN_PLACE) __syncthreads();
    if (go) {
      *reinterpret_cast<uint4*>(cache + to_id * sp + (at & mask) * st) = v;
      if (weigh) p.weights_out[((static_cast<int64_t>(to_id) * p.Hk + hk) << p.page_shift) + (at & mask)] = w;
    }
  }
}

template <int D>
cudaError_t move_dim(const LongParams& p, cudaStream_t s) {
  constexpr int kSlices = 2 * (D / 8 / 4), kTokens = kMoveThreads / 4, kSteps = 4;
  if (p.dst == nullptr)
    return launch(move_kernel<D, true>, dim3(kSlices, p.Hk, p.B), kMoveThreads, 0, s, p, 0);
  const int most = p.n < p.max_len ? p.n : p.max_len;
  const unsigned cuts = static_cast<unsigned>((most + kTokens * kSteps - 1) / (kTokens * kSteps));
  return launch(move_kernel<D, false>, dim3(kSlices * cuts, p.Hk, p.B), kMoveThreads, 0, s, p, static_cast<int>(kSteps));
}

}  // namespace

cudaError_t launch_select(const LongParams& p, cudaStream_t s) {
  const int64_t rows = static_cast<int64_t>(p.B) * p.Hk * p.Nq;
  const dim3 warps(static_cast<unsigned>((rows + 3) / 4)), blocks(static_cast<unsigned>(rows));
  const int w = p.table_width;
  if (w <= 128) return launch(select_kernel<32, 4, false>, warps, 128, 0, s, p);
  if (w <= 512) return launch(select_kernel<32, 16, false>, warps, 128, 0, s, p);
  if (w <= 1024) return launch(select_kernel<32, 32, false>, warps, 128, 0, s, p);
  if (w <= 4096) return launch(select_kernel<256, 16, false>, blocks, 256, 0, s, p);
  if (w <= 16384) return launch(select_kernel<1024, 16, false>, blocks, 1024, 0, s, p);
  return launch(select_kernel<1024, 1, true>, blocks, 1024, 0, s, p);
}

cudaError_t launch_evict(const LongParams& p, int d, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>(p.B) * static_cast<unsigned>(p.Hk));
  cudaError_t e;
  if (p.max_len <= 4096)
    e = launch(keep_kernel<1024, 4, false>, grid, 1024, 0, s, p);
  else if (p.max_len <= 16384)
    e = launch(keep_kernel<1024, 16, false>, grid, 1024, 0, s, p);
  else if (p.max_len <= 32768)
    e = launch(keep_kernel<1024, 32, false>, grid, 1024, 0, s, p);
  else
    e = launch(keep_kernel<1024, 1, true>, grid, 1024, 0, s, p);
  if (e != cudaSuccess) return e;
  switch (d) {
    case 32: return move_dim<32>(p, s);
    case 64: return move_dim<64>(p, s);
    case 128: return move_dim<128>(p, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace attn
