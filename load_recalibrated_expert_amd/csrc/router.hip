// The router beside the experts: top-K routing with its expert-major pair lists, the balance
// loss with its per-expert counts, the gradient of the logits, and the gradient of the routing
// weights from the saved output rows.
//
// All of it is one pass over [T x E] logits (or, for the routing-weight gradient, over the
// [N x D] output rows), so memory bounds it at large T and launch latency at small T. A group
// of L lanes holds one token's logits in registers, V to a lane.
#include <algorithm>

#include "router_device.h"

namespace lrmoe {
namespace {

// ---------------------------------------------------------------- routing

// Tokens of one top-K block and of one placing block, so that the 256 compute units have about as many
// each: 256 chunks of up to 128 tokens, then 512 (top-K and placing of 300000 x 64 in chunks of 1024
// 27.2 + 16.8 us, of 592 19.3 + 12.7 us; 70000 x 1024 bf16 in chunks of 256 121 us, of 144 70 us). Each
// writes a row of counts, so chunks have at least 128 tokens, or 64 where the top-K gains more by
// smaller ones than the scan loses by more rows: above 320 experts, where a token has sixteen or more
// lanes whatever K (16384 x 512 in chunks of 128 22 us, of 64 14.5 us), and with more than 256 chunks
// (50021 x 257 in chunks of 128 23.6 us, of 104 21.8 us). With 9 to 32 slots sixteen lanes begin at 257
// experts; chunks of 64 there were not measured. Routing by scores costs more a token: 64 tokens always.
int route_chunk(const lrmoe_router* r, bool scored) {
  if (r->T <= kOneChunk) return kOneChunk;
  const int64_t even = align_up((size_t)ceil_div(r->T, r->T <= 256 * 128 ? 256 : 512), 8);
  const int64_t room = (int64_t)kPlaceLds / 4 / r->local * 32;  // whose bits fit
  return (int)std::min(std::max(even, (int64_t)(scored || r->E > 320 || r->T > 256 * 128 ? 64 : 128)),
                       std::min<int64_t>(room, 1024));
}

// One block per chunk of tokens: the K largest logits of each, their weights, and how often the chunk
// chose each expert. With few tokens (rows = 1) the block places the pairs itself.
template <class Lay, int N>
__global__ __launch_bounds__(topk_threads(Lay::L, N)) void route_topk_kernel(RouteArgs a) {
  constexpr int kTopkThreads = topk_threads(Lay::L, N);
  constexpr int L = Lay::L, V = Lay::V, kGroups = kTopkThreads / L;
  constexpr int S = (N + L - 1) / L;  // slots of a lane: k = lane, lane + L, ...
  static_assert(V % N == 0, "whole lists");
  extern __shared__ uint32_t lds[];
  RouteBlock<kTopkThreads> blk(a, lds);
  const int lane = threadIdx.x & (L - 1);
  const int64_t t0 = (int64_t)blockIdx.x * a.C, t1 = min(t0 + a.C, (int64_t)a.T);
  __syncthreads();
  // each wavefront for itself: one that has no tokens left leaves the others the units
  for (int64_t tb = t0 + __builtin_amdgcn_readfirstlane(threadIdx.x / kWave) * (kWave / L); tb < t1; tb += kGroups) {
    const int64_t t = tb + (threadIdx.x & (kWave - 1)) / L;
    const bool in = t < t1;
    float x[V];
    // the keys of bf16 logits hold +inf itself: the largest finite f32 that it stands for is no bf16
    // value, and is above the largest that is
    Lay::template load<Lay::BF16>(a.logits, t, a.E, in && unmasked(a.mask, t), lane, x);
    float top = kNegInf, Z = 0.0f;
    if (!a.renorm) {
#pragma unroll
      for (int v = 0; v < V; ++v) top = fmaxf(top, x[v]);
      top = fminf(group_max<L>(top), kFltMax);
#pragma unroll
      for (int v = 0; v < V; ++v) Z += exp_term((Lay::BF16 ? fminf(x[v], kFltMax) : x[v]) - top);
      Z = group_sum<L>(Z);
    }
    using Key = std::conditional_t<Lay::BF16, uint32_t, double>;
    Key best[N];
#pragma unroll
    for (int q = 0; q < V; q += N) {
      Key d[N];
#pragma unroll
      for (int i = 0; i < N; ++i) to_key(x[q + i], Lay::expert(lane, q + i), &d[i]);
      sort_list<0, N>(d);
      if (q == 0) {
#pragma unroll
        for (int i = 0; i < N; ++i) best[i] = d[i];
      } else {
        merge_lists<N>(best, d);
      }
    }
    merge_lanes<N, L>(best);
    int e[S], top_e;
    float p[S], sum = 0.0f;
    of_key(best[0], &top, &top_e);
#pragma unroll
    for (int q = 0; q < S; ++q) {
      const int k = lane + q * L;
      Key d = 0;
#pragma unroll
      for (int i = q * L; i < N && i < (q + 1) * L; ++i) d = i == k ? best[i] : d;
      float xk;
      of_key(d, &xk, &e[q]);
      if (k >= a.K) e[q] = -1;
      p[q] = e[q] >= 0 ? exp_below<true>(xk - top) : 0.0f;
      sum += p[q];
    }
    if (a.renorm) Z = group_sum<L>(sum);
#pragma unroll
    for (int q = 0; q < S; ++q) {
      const int k = lane + q * L;
      if (in && k < a.K) blk.put(a, t, k, e[q], e[q] >= 0 ? a.scale * (p[q] / Z) : 0.0f);
    }
  }
  blk.finish(a);
}

// Whether every placing block sums all rows of counts itself, a word (two experts' 16-bit counts) of every so many rows to a
// thread, or a launch scans them first. Up to 64 rows, and up to 24 words a thread (22 where a compute unit has more than one
// block); the loads of a thread's last rows go out together too, one after the other they cost 0.7 us. With the scan and
// without: 3584 x 1024 (56 rows of 512 words) 25.0 and 24.5 us, 32768 x 128 (256 rows, 16 words a thread) 17.8 and 15.8,
// 32768 x 192 (256 rows, 24) 20.8 and 20.0, 700000 x 64 (684 rows, 21.4) 147 and 141, 6000000 x 8 (5860 rows, 22.9) 217 and
// 218; but 40000 x 96 (500 rows, 23.4) 20.4 and 20.7.
constexpr int kOwnRows = 64, kOneEach = 256;
bool sums_own(int64_t rows, int64_t E8) {
  return rows <= kOwnRows || rows * (E8 / 2) <= (rows <= kOneEach ? 24 : 22) * kRouteThreads;
}
// Up to so many rows a thread sums one expert's counts, without the other way's sums over threads (1000 x 256, 8 rows: 14.7
// and 15.4 us; 2000 x 128, 16 rows: 11.8 and 12.1 us; but 3000 x 512, 24 rows: 17.0 and 15.7 us).
constexpr int kFewRows = 16;
constexpr int kSumAhead = 8;
constexpr int kScanExperts = 32;
constexpr int kScanKept = 8;  // rows of a run: all of them up to 512 chunks

// Block: 32 experts, the rows in 64 runs. prefix[r][e] = tokens in the rows before r; total[e].
__global__ __launch_bounds__(kRouteThreads) void route_scan_kernel(RouteArgs a) {
  __shared__ int part[kScanExperts][kWave + 1];  // [expert][run]
  const int tid = threadIdx.x, E8 = (a.E + 7) & ~7, p = tid & 15, run = tid >> 4, lane = tid & (kWave - 1);
  const int e = blockIdx.x * kScanExperts + 2 * p, len = (a.rows + kWave - 1) / kWave;
  const int r0 = min(run * len, a.rows), r1 = min(r0 + len, a.rows);
  const uint32_t* h = (const uint32_t*)a.hist + e / 2;
  uint32_t kept[kScanKept];  // a run's first rows stay in registers for the second pass
  int s0 = 0, s1 = 0;
  if (e < E8) {
#pragma unroll
    for (int q = 0; q < kScanKept; ++q) kept[q] = r0 + q < r1 ? h[(int64_t)(r0 + q) * (E8 / 2)] : 0;
#pragma unroll
    for (int q = 0; q < kScanKept; ++q) s0 += (int)(kept[q] & 0xFFFFu), s1 += (int)(kept[q] >> 16);
    for (int r = r0 + kScanKept; r < r1; ++r) {
      const uint32_t v = h[(int64_t)r * (E8 / 2)];
      s0 += (int)(v & 0xFFFFu), s1 += (int)(v >> 16);
    }
  }
  part[2 * p][run] = s0;
  part[2 * p + 1][run] = s1;
  __syncthreads();
  for (int q = tid / kWave; q < kScanExperts; q += kRouteThreads / kWave) {  // a wavefront scans one expert's runs
    const int mine = part[q][lane];
    int inc = mine;
#pragma unroll
    for (int o = 1; o < kWave; o <<= 1) {
      const int up = __shfl_up(inc, o, kWave);
      if (lane >= o) inc += up;
    }
    part[q][lane] = inc - mine;
    const int x = blockIdx.x * kScanExperts + q;
    if (lane == kWave - 1 && x < E8) a.total[x] = inc;
  }
  __syncthreads();
  if (e < E8) {
    s0 = part[2 * p][run], s1 = part[2 * p + 1][run];
    int* out = a.prefix + e;
#pragma unroll
    for (int q = 0; q < kScanKept; ++q) {
      if (r0 + q < r1) *(int2*)(out + (int64_t)(r0 + q) * E8) = make_int2(s0, s1);
      s0 += (int)(kept[q] & 0xFFFFu), s1 += (int)(kept[q] >> 16);
    }
    for (int r = r0 + kScanKept; r < r1; ++r) {
      const uint32_t v = h[(int64_t)r * (E8 / 2)];
      *(int2*)(out + (int64_t)r * E8) = make_int2(s0, s1);
      s0 += (int)(v & 0xFFFFu), s1 += (int)(v >> 16);
    }
  }
}

// One block per chunk. Its experts' tokens in all and in earlier chunks come from the scan, or for few
// rows from the rows themselves.
__global__ __launch_bounds__(kRouteThreads) void route_place_kernel(RouteArgs a) {
  __shared__ int total[1024], before[1024];
  extern __shared__ uint32_t lds[];  // [C / 32, rounded up][local] bits; [2 C K] pairs
  uint32_t* bits = lds;
  const int words = bit_words(a.C, a.local);
  uint32_t* sorted = a.sorted ? lds + words : nullptr;
  const int tid = threadIdx.x, c = blockIdx.x, E8 = (a.E + 7) & ~7;
  const int64_t i0 = (int64_t)c * a.C * a.K;
  const int n = (int)(min((int64_t)(c + 1) * a.C, (int64_t)a.T) * a.K - i0);
  const int e0 = tid < n ? a.idx[i0 + tid] : -1;  // on its way meanwhile
  const float w0 = tid < n ? a.w[i0 + tid] : 0.0f;
  for (int i = tid; i < words; i += kRouteThreads) bits[i] = 0;
  if (a.prefix) {
    if (tid < a.E) {
      total[tid] = a.total[tid];
      before[tid] = a.prefix[(int64_t)c * E8 + tid];
    }
  } else if (a.rows <= kFewRows) {  // a thread has an expert of every row
    int sum = 0, low = 0;
    for (int r = 0; tid < a.E && r < a.rows; r += kSumAhead) {
      int v[kSumAhead];
#pragma unroll
      for (int q = 0; q < kSumAhead; ++q) v[q] = r + q < a.rows ? a.hist[(int64_t)(r + q) * E8 + tid] : 0;
#pragma unroll
      for (int q = 0; q < kSumAhead; ++q) {
        sum += v[q];
        low += r + q < c ? v[q] : 0;
      }
    }
    if (tid < a.E) total[tid] = sum, before[tid] = low;
  } else {
    // a thread has one word of every `step`-th row
    if (tid < a.E) total[tid] = before[tid] = 0;
    __syncthreads();
    const int pairs = E8 / 2, step = kRouteThreads / pairs, w = tid % pairs;
    const uint32_t* h = (const uint32_t*)a.hist + w;
    int s0 = 0, s1 = 0, l0 = 0, l1 = 0;
    if (tid < step * pairs) {
      auto add = [&](auto whole, int r) {  // eight rows whose loads are in flight together, or the fewer that are left
        uint32_t v[kSumAhead];
#pragma unroll
        for (int q = 0; q < kSumAhead; ++q)
          v[q] = decltype(whole)::value || r + q * step < a.rows ? h[(int64_t)(r + q * step) * pairs] : 0;
#pragma unroll
        for (int q = 0; q < kSumAhead; ++q) {
          const int lo = (int)(v[q] & 0xFFFFu), hi = (int)(v[q] >> 16);
          s0 += lo, s1 += hi;
          l0 += r + q * step < c ? lo : 0, l1 += r + q * step < c ? hi : 0;
        }
      };
      int r = tid / pairs;
      for (; r + (kSumAhead - 1) * step < a.rows; r += kSumAhead * step) add(std::true_type(), r);
      if (r < a.rows) add(std::false_type(), r);
      // whole numbers: their order does not matter
      if (2 * w < a.E) atomicAdd(&total[2 * w], s0), atomicAdd(&before[2 * w], l0);
      if (2 * w + 1 < a.E) atomicAdd(&total[2 * w + 1], s1), atomicAdd(&before[2 * w + 1], l1);
    }
  }
  __syncthreads();
  place_chunk<kRouteThreads>(
      a, c, n, total, before, bits, sorted, [&](int i) { return i < kRouteThreads ? e0 : a.idx[i0 + i]; },
      [&](int i) { return i < kRouteThreads ? w0 : a.w[i0 + i]; });
}

// ---------------------------------------------------------------- balance loss

constexpr int kBalThreads = 1024;
constexpr int kMaxTile = 8192;    // its tokens that are live take one byte of LDS each
constexpr int kJoinExperts = 64;  // experts of one joining block, one to a lane

// Sequence s, clamped into [0, T] whatever the offsets hold.
__device__ __forceinline__ void seq_range(const int64_t* __restrict__ off, int s, int T, int64_t* lo, int64_t* hi) {
  if (!off) {
    *lo = 0;
    *hi = T;
    return;
  }
  const int64_t a = off[s], b = off[s + 1];
  *lo = a < 0 ? 0 : (a > T ? T : a);
  *hi = b < *lo ? *lo : (b > T ? T : b);
}

// Tokens of one tile: one pass of a block, or more where the tiles of one sequence would be more than 512,
// which the join takes one after the other (a million tokens of 64 experts: 216 us in tiles of 64,
// 65 us in tiles of 2048). Up to 128 values of a lane are summed in fp32: above 512 experts, where a
// pass takes 16 tokens, tiles end at 2048.
int balance_log_tile(const lrmoe_router* r) {
  int log = 6;
  while ((1 << log) < (r->E > 512 ? kMaxTile / 4 : kMaxTile) && (r->T >> log) > 512) ++log;
  return log;
}

// Sequence s has the tile slots from floor(off[s] / tile) + s on, which are at least as many as it
// has tiles, so tiles need no table: floor(T / tile) + n_seq slots in all.
__device__ __forceinline__ int64_t first_tile(int64_t lo, int s, int log_tile) { return (lo >> log_tile) + s; }

__device__ __forceinline__ int seq_of_tile(const int64_t* __restrict__ off, int n_seq, int T, int log_tile,
                                           int64_t b) {
  int a = 0, z = n_seq - 1;  // the last sequence whose first slot is at or before b
  while (a < z) {
    const int m = (a + z + 1) / 2;
    int64_t lo, hi;
    seq_range(off, m, T, &lo, &hi);
    if (first_tile(lo, m, log_tile) <= b) a = m;
    else z = m - 1;
  }
  return a;
}

struct BalanceWs {
  float* psum;     // [tiles][E] sums of probabilities
  int32_t* count;  // [tiles][E]
  int32_t* live;   // [tiles]
  double* dot;     // [n_seq][parts] sum_e counts psum over a joining block's experts
  int32_t* n;      // [n_seq] live tokens
  uint32_t* done;  // join blocks that are through
};

int64_t balance_tiles(const lrmoe_router* r, int32_t n_seq) { return (r->T >> balance_log_tile(r)) + n_seq; }

size_t balance_layout(const lrmoe_router* r, int32_t n_seq, char* base, BalanceWs* out) {
  const size_t tiles = (size_t)balance_tiles(r, n_seq), parts = (size_t)ceil_div(r->E, kJoinExperts);
  size_t at = 0;
  auto take = [&](size_t b) {
    char* p = base + at;
    at += align_up(b, 256);
    return p;
  };
  BalanceWs w;
  w.psum = (float*)take(tiles * r->E * 4);
  w.count = (int32_t*)take(tiles * r->E * 4);
  w.live = (int32_t*)take(tiles * 4);
  w.dot = (double*)take((size_t)n_seq * parts * 8);
  w.n = (int32_t*)take((size_t)n_seq * 4);
  w.done = (uint32_t*)take(4);
  if (out) *out = w;
  return at;
}

// One block per tile slot; up to 512 experts a pass takes 64 tokens, one to a group of lanes. LONG: tiles of
// more than 64 tokens. (Without its own code for 64, whose loop is one pass, 32768 x 128 took 9.3
// instead of 7.3 us.)
// SIG: p is the token's sigmoid scores over their sum.
template <class Lay, bool LONG, bool SIG>
__global__ __launch_bounds__(kBalThreads) void balance_tile_kernel(int T, int E, int K, int n_seq, int log_long,
                                                                   const void* __restrict__ logits,
                                                                   const uint8_t* __restrict__ mask,
                                                                   const int32_t* __restrict__ idx,
                                                                   const int64_t* __restrict__ off, BalanceWs ws) {
  constexpr int L = Lay::L, V = Lay::V, kGroups = kBalThreads / L, kWaves = kBalThreads / kWave;
  __shared__ int cnt[1024];
  __shared__ float part[kWaves][L * V];
  __shared__ uint8_t live_of[LONG ? kMaxTile : 64];
  __shared__ int live_n;
  const int log_tile = LONG ? log_long : 6;
  const int64_t b = blockIdx.x;
  if (b == 0 && threadIdx.x == 0) *ws.done = 0;
  const int s = off ? seq_of_tile(off, n_seq, T, log_tile, b) : 0;
  int64_t lo, hi;
  seq_range(off, s, T, &lo, &hi);
  const int64_t tile = b - first_tile(lo, s, log_tile);  // negative in slots before the first sequence's
  lo += tile << log_tile;
  hi = min(hi, lo + (1 << log_tile));
  if (tile < 0 || lo >= hi) return;  // a slot that no tile uses: the whole block leaves
  if (!LONG) hi = min(hi, lo + 64);  // what the compiler is to know
  for (int e = threadIdx.x; e < E; e += kBalThreads) cnt[e] = 0;
  if (threadIdx.x == 0) live_n = 0;
  const int lane = threadIdx.x & (L - 1), group = threadIdx.x / L, n = (int)(hi - lo) * K;
  const int e0 = (int)threadIdx.x < n ? idx[lo * K + threadIdx.x] : -1;  // on its way meanwhile
  float acc[V];
#pragma unroll
  for (int v = 0; v < V; ++v) acc[v] = 0.0f;
  for (int64_t tb = lo; tb < hi; tb += kGroups) {
    const int64_t t = tb + group;
    float x[V], top = kNegInf, Z = 0.0f;
    Lay::load(logits, t, E, t < hi && unmasked(mask, t), lane, x);
#pragma unroll
    for (int v = 0; v < V; ++v) top = fmaxf(top, x[v]);
    top = group_max<L>(top);
    const bool live = top > kNegInf;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      x[v] = SIG ? sigmoid_over(x[v], top) : exp_below(x[v] - top);
      Z += x[v];
    }
    Z = group_sum<L>(Z);
    const float rz = live ? 1.0f / Z : 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] += x[v] * rz;
    if (lane == 0 && t < hi) live_of[t - lo] = live ? 1 : 0;
  }
  // the wavefront's groups, then (below) the wavefronts
#pragma unroll
  for (int v = 0; v < V; ++v) {
#pragma unroll
    for (int o = L; o < kWave; o <<= 1) acc[v] += __shfl_xor(acc[v], o, kWave);
  }
  if ((threadIdx.x & (kWave - 1)) < L)
#pragma unroll
    for (int v = 0; v < V; ++v) part[threadIdx.x / kWave][Lay::expert(lane, v)] = acc[v];
  __syncthreads();
  if (LONG) {
    int mine = 0;
    for (int i = threadIdx.x; i < (int)(hi - lo); i += kBalThreads) mine += live_of[i];
    if (mine) atomicAdd(&live_n, mine);
  } else if (threadIdx.x < kWave) {
    const unsigned long long on = __ballot(threadIdx.x < hi - lo && live_of[threadIdx.x] != 0);
    if (threadIdx.x == 0) live_n = __popcll(on);
  }
  for (int i = threadIdx.x; i < n; i += kBalThreads) {
    const int e = i < kBalThreads ? e0 : idx[lo * K + i];
    if (e >= 0 && e < E && live_of[i / K]) atomicAdd(&cnt[e], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += kBalThreads) {
    float a = 0.0f;
#pragma unroll
    for (int g = 0; g < kWaves; ++g) a += part[g][e];
    ws.psum[b * E + e] = a;
    ws.count[b * E + e] = cnt[e];
  }
  if (threadIdx.x == 0) ws.live[b] = live_n;
}

constexpr int kJoinWaves = 16, kJoinWavesMany = 4;  // of a joining block
constexpr int kLossThreads = 1024;
// Joining blocks up to which the last one sums the loss. Their releases follow one another at some 30 ns
// each; above, a launch of its own does it. 131072 x 128: 32 sequences (64 blocks) 28.8 us so and
// 30.2 us with the launch, 64 sequences 29.7 and 28.7, 1024 sequences 79 and 35, 16384 994 and 240.
constexpr int64_t kJoinLast = 64;

// Sum over the wavefront, the same bits in every lane.
template <int S = 1>
__device__ __forceinline__ double lanes_sum(double v) {
  if constexpr (S < kWave)
    return lanes_sum<2 * S>(v + __hiloint2double(lane_swap<S>(__double2hiint(v)), lane_swap<S>(__double2loint(v))));
  else return v;
}

// What of its loss a sequence of m live tokens has beside its own sums, with `alive` sequences that have any.
__device__ __forceinline__ double loss_factor(float coef, int E, int K, int alive, double m) {
  return m > 0 ? (double)coef * E / ((double)alive * K * m * m) : 0.0;
}

// Grid (sequence, 64 experts): the sequence's tiles joined, every WAVES-th by one wavefront and those over
// the wavefronts, always in the same order. LAST: the block that finishes last sums the loss; it reads
// what the others wrote behind their release, in a fixed order, so the result does not depend on
// which block it is. 8.4 us for 512 tiles of 128 experts, 2.5 of them the last block's part, most
// of the rest latency: 16 experts to a block took 7.9 us there, but 9.1 instead of 7.0 us for 37
// sequences of 60 experts, whose releases are then four times as many. Else balance_loss_kernel follows.
template <int WAVES, bool LAST>
__global__ __launch_bounds__(WAVES* kWave) void balance_join_kernel(int T, int E, int K, int n_seq, int log_tile,
                                                                    float coef, const int64_t* __restrict__ off,
                                                                    BalanceWs ws, int32_t* __restrict__ counts,
                                                                    float* __restrict__ psum, float* __restrict__ norm,
                                                                    float* __restrict__ loss) {
  __shared__ double sum_of[WAVES][kWave];
  __shared__ int n_of[WAVES][kWave], live_of;
  const int s = blockIdx.x, part = blockIdx.y, parts = gridDim.y;
  const int wave = threadIdx.x / kWave, lane = threadIdx.x & (kWave - 1);
  const int e = part * kJoinExperts + lane;
  int64_t lo, hi;
  seq_range(off, s, T, &lo, &hi);
  const int64_t b0 = first_tile(lo, s, log_tile);
  const int tiles = (int)((hi - lo + (1 << log_tile) - 1) >> log_tile);
  double a = 0.0;
  int n = 0;
  if (e < E) {
#pragma unroll 8
    for (int i = wave; i < tiles; i += WAVES) {
      a += (double)ws.psum[(b0 + i) * E + e];
      n += ws.count[(b0 + i) * E + e];
    }
  }
  sum_of[wave][lane] = a;
  n_of[wave][lane] = n;
  if (part == 0 && wave == WAVES - 1) {
    int live = 0;
    for (int i = lane; i < tiles; i += kWave) live += ws.live[b0 + i];
    live = group_reduce<kWave>(live, [](int p, int q) { return p + q; });
    if (lane == 0) live_of = live;
  }
  __syncthreads();
  if (wave != 0) return;  // the rest is one wavefront's
  double dot = 0.0;
  if (e < E) {
    a = 0.0;
    n = 0;
    for (int q = 0; q < WAVES; ++q) {
      a += sum_of[q][lane];
      n += n_of[q][lane];
    }
    psum[(int64_t)s * E + e] = (float)a;
    counts[(int64_t)s * E + e] = n;
    dot = a * n;
  }
  dot = lanes_sum(dot);
  if (!LAST) {
    if (lane == 0) {
      ws.dot[(int64_t)s * parts + part] = dot;
      if (part == 0) ws.n[s] = live_of;
    }
    return;
  }
  uint32_t before = 0;
  if (lane == 0) {
    __hip_atomic_store(&ws.dot[(int64_t)s * parts + part], dot, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (part == 0) __hip_atomic_store(&ws.n[s], live_of, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    before = __hip_atomic_fetch_add(ws.done, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT);
  }
  if (__builtin_amdgcn_readfirstlane(before) != gridDim.x * gridDim.y - 1) return;
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");  // lane 0's acquire, for the whole wavefront
  int alive = 0;
  for (int i = lane; i < n_seq; i += kWave)
    alive += __hip_atomic_load(&ws.n[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) > 0 ? 1 : 0;
  alive = group_reduce<kWave>(alive, [](int p, int q) { return p + q; });
  double sum = 0.0;
  for (int i = lane; i < n_seq; i += kWave) {
    const double m = __hip_atomic_load(&ws.n[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    const double f = loss_factor(coef, E, K, alive, m);
    norm[i] = (float)f;
    double d = 0.0;
    for (int q = 0; q < parts; ++q)
      d += __hip_atomic_load(&ws.dot[(int64_t)i * parts + q], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    sum += f * d;
  }
  sum = lanes_sum(sum);
  if (lane == 0) loss[0] = (float)sum;
}

// One block: every sequence's factor, and the loss.
__global__ __launch_bounds__(kLossThreads) void balance_loss_kernel(int E, int K, int n_seq, float coef, BalanceWs ws,
                                                                    float* __restrict__ norm,
                                                                    float* __restrict__ loss) {
  constexpr int kWaves = kLossThreads / kWave;
  __shared__ int alive_of[kWaves];
  __shared__ double sum_of[kWaves];
  const int wave = threadIdx.x / kWave, lane = threadIdx.x & (kWave - 1), parts = (E + kJoinExperts - 1) / kJoinExperts;
  int alive = 0;
#pragma unroll 4
  for (int i = threadIdx.x; i < n_seq; i += kLossThreads) alive += ws.n[i] > 0 ? 1 : 0;
  alive = group_reduce<kWave>(alive, [](int p, int q) { return p + q; });
  if (lane == 0) alive_of[wave] = alive;
  __syncthreads();
  alive = 0;
#pragma unroll
  for (int q = 0; q < kWaves; ++q) alive += alive_of[q];
  double sum = 0.0;
  for (int i = threadIdx.x; i < n_seq; i += kLossThreads) {
    const double f = loss_factor(coef, E, K, alive, ws.n[i]);
    norm[i] = (float)f;
    double d = 0.0;
    for (int q = 0; q < parts; ++q) d += ws.dot[(int64_t)i * parts + q];
    sum += f * d;
  }
  sum = lanes_sum(sum);
  if (lane == 0) sum_of[wave] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    sum = 0.0;
    for (int q = 0; q < kWaves; ++q) sum += sum_of[q];
    loss[0] = (float)sum;
  }
}

// ---------------------------------------------------------------- gradient of the logits

constexpr int kGradThreads = 256;

// The K slots of a token are worked on in K lanes of its group, whose results reach the lanes that
// hold their experts through a row of LDS.
//
// SIG: sigmoid scores s, whose share of the token's sum p has the derivative p_e (1 - s_e) (d_e' - p_e') instead of
// softmax's. Without the balance loss only the chosen experts have a gradient, and only their logits are read.
template <class Lay, int S, bool SIG>  // S: slots of a lane, k = lane, lane + L, ...
__global__ __launch_bounds__(kGradThreads) void route_bwd_kernel(
    int T, int E, int K, int renorm, float scale, const void* __restrict__ logits, const uint8_t* __restrict__ mask,
    const int32_t* __restrict__ idx, const float* __restrict__ dalpha, const int32_t* __restrict__ pmap,
    int64_t n_pairs, const int64_t* __restrict__ off, int n_seq, const int32_t* __restrict__ counts,
    const float* __restrict__ norm, const float* __restrict__ gloss, void* __restrict__ dlogits) {
  constexpr int L = Lay::L, V = Lay::V;
  __shared__ float rows[kGradThreads / L][L * V];
  const int lane = threadIdx.x & (L - 1);
  const int64_t t = (int64_t)blockIdx.x * (kGradThreads / L) + threadIdx.x / L;
  const bool in = t < T, on = in && unmasked(mask, t);
  // the slots' loads start first: dalpha's depends on pmap's
  int e[S];
  float y[S];
  if (dalpha) {
    int64_t j[S];
#pragma unroll
    for (int q = 0; q < S; ++q) {
      const int k = lane + q * L;
      const bool slot = on && k < K;
      e[q] = slot ? idx[t * K + k] : -1;
      j[q] = !slot ? -1 : pmap ? pmap[t * K + k] : t * K + k;
    }
#pragma unroll
    for (int q = 0; q < S; ++q) y[q] = j[q] >= 0 && (!pmap || j[q] < n_pairs) ? scale * dalpha[j[q]] : 0.0f;
  }
  const bool all = !SIG || norm != nullptr;  // uniform
  float x[V], p[V], dx[V], top = kNegInf, Z = 0.0f;
  Lay::load(logits, t, E, on && all, lane, x);
#pragma unroll
  for (int v = 0; v < V; ++v) top = fmaxf(top, x[v]);
  top = group_max<L>(top);
  const bool live = top > kNegInf;
  float xe[S];  // logits of the slots' experts
  if (SIG) {
    if (dalpha) {  // (through the row, as below, took the same time)
#pragma unroll
      for (int q = 0; q < S; ++q) xe[q] = e[q] >= 0 && e[q] < E ? clean(Lay::load_one(logits, t * E + e[q])) : kNegInf;
    }
    if (__any(top < 0.0f)) {
#pragma unroll
      for (int v = 0; v < V; ++v) p[v] = exp_below(fminf(x[v], 0.0f) - fminf(top, 0.0f));
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) p[v] = x[v] >= 0.0f ? 1.0f : exp_below(-fabsf(x[v]));
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float z = exp_below(-fabsf(x[v])), r = __builtin_amdgcn_rcpf(1.0f + z);
      p[v] *= r;
      x[v] = (x[v] >= 0.0f ? z : 1.0f) * r;
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if (!SIG) p[v] = exp_below(x[v] - top);
    Z += p[v];
    dx[v] = 0.0f;
  }
  Z = group_sum<L>(Z);
  const float rz = live ? 1.0f / Z : 0.0f;
#pragma unroll
  for (int v = 0; v < V; ++v) p[v] *= rz;
  if (dalpha) {
    // the row passes the logits of the chosen experts to their slots, then the slots' results back
    float* row = rows[threadIdx.x / L];
    float ref = top, r = rz, q_of[S], s = 0.0f;
    if (!SIG) {
#pragma unroll
      for (int v = 0; v < V; ++v) row[Lay::expert(lane, v)] = x[v];
      wave_sync();
#pragma unroll
      for (int q = 0; q < S; ++q) xe[q] = e[q] >= 0 && e[q] < E ? row[e[q]] : kNegInf;
      wave_sync();
    }
#pragma unroll
    for (int v = 0; v < V; ++v) row[Lay::expert(lane, v)] = 0.0f;
    if (SIG) {
      ref = 0.0f;
      r = 1.0f;
    }
    if (renorm) {  // the chosen experts' shares of their sum
      ref = kNegInf;
#pragma unroll
      for (int q = 0; q < S; ++q) ref = fmaxf(ref, xe[q]);
      ref = group_max<L>(ref);
      r = 1.0f;
    }
#pragma unroll
    for (int q = 0; q < S; ++q)
      q_of[q] = xe[q] > kNegInf ? (SIG ? sigmoid_over<true>(xe[q], ref) : exp_below<true>(xe[q] - ref)) * r : 0.0f;
    if (renorm) {
      float z = 0.0f;
#pragma unroll
      for (int q = 0; q < S; ++q) z += q_of[q];
      z = group_sum<L>(z);
      r = z > 0.0f ? 1.0f / z : 0.0f;
#pragma unroll
      for (int q = 0; q < S; ++q) q_of[q] *= r;
    }
#pragma unroll
    for (int q = 0; q < S; ++q) s += xe[q] > kNegInf ? q_of[q] * y[q] : 0.0f;
    s = group_sum<L>(s);
    wave_sync();
#pragma unroll
    for (int q = 0; q < S; ++q)
      if (xe[q] > kNegInf)
        row[e[q]] = (renorm ? q_of[q] * (y[q] - s) : q_of[q] * y[q]) * (SIG ? sigmoid_over(-xe[q], 0.0f) : 1.0f);
    wave_sync();
#pragma unroll
    for (int v = 0; v < V; ++v) {
      dx[v] = row[Lay::expert(lane, v)];
      if (!SIG && !renorm) dx[v] -= p[v] * s;
    }
  }
  if (norm) {
    int s = 0;
    bool inside = live;
    if (off && in) {  // the last sequence that starts at or before t
      int a = 0, z = n_seq - 1;
      while (a < z) {
        const int m = (a + z + 1) / 2;
        if (off[m] <= t) a = m;
        else z = m - 1;
      }
      s = a;
      inside = live && t >= off[s] && t < off[s + 1];
    }
    // The counts relative to the most probable expert's, as whole numbers: sum_e p_e = 1, so that changes
    // nothing in c - dot, and near balance, where counts in the millions differ by a few, the common part
    // would leave its rounding there. Counts of 2^17 +- 1 over 64 experts: an error of 1.6e-2 of the
    // gradient without, 1.1e-7 with it; 32768 x 128 takes 7.5 and 7.85 us.
    int32_t n[V], ref = INT32_MIN;
    // p of the most probable expert, by the same operations (not by 1 - s, which is 1 for all of them below -17)
    const float most = SIG ? __builtin_amdgcn_rcpf(1.0f + exp_below(-fabsf(top))) * rz : rz;
    Lay::load_counts(counts, s, E, inside, lane, n);
#pragma unroll
    for (int v = 0; v < V; ++v) ref = max(ref, p[v] >= most ? n[v] : INT32_MIN);
    ref = group_reduce<L>(ref, [](int a, int b) { return max(a, b); });
    float c[V], dot = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      c[v] = (float)(int32_t)((uint32_t)n[v] - (uint32_t)ref);
      dot += p[v] * c[v];
    }
    dot = group_sum<L>(dot);
    const float f = inside ? norm[s] * (gloss ? gloss[0] : 1.0f) : 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v)  // zeros where f or, not live, p is 0
      dx[v] += f * (p[v] * (SIG ? x[v] : 1.0f) * (c[v] - dot));
  }
  if (!in) return;
  Lay::store(dlogits, t, E, lane, dx);
}

// ---------------------------------------------------------------- gradient of the routing weights

constexpr int kAlphaThreads = 256;
constexpr int kAlphaRows = 8;  // pairs whose rows a wavefront reads at once
// Tokens up to which a block shares one: any, or those of rows of 4 KB and more (a word to a thread).
constexpr int kAlphaSplit = 1024, kAlphaSplitWide = 8192;

// Products of 16 bytes of two rows, added to s: both in fp64, which holds every product of two f32 or bf16
// values exactly (f32 holds those of bf16 values between 2^-126 and 2^128 only; the time is the same).
template <bool BF16>
__device__ __forceinline__ double dot16(uint4 g, uint4 y, double s) {
  const uint32_t gw[4] = {g.x, g.y, g.z, g.w}, yw[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (BF16) {
      s += (double)bf16_lo(gw[i]) * (double)bf16_lo(yw[i]);
      s += (double)bf16_hi(gw[i]) * (double)bf16_hi(yw[i]);
    } else {
      s += (double)__uint_as_float(gw[i]) * (double)__uint_as_float(yw[i]);
    }
  }
  return s;
}

// One wavefront per token: its gradient row is read once against the rows of up to eight of its
// pairs, whose loads are all in flight before the first product (one row after the other: 256 us for
// 32768 tokens, top-8, 2048 bf16; so: 190 us, 6.4 TB/s, with one or two column blocks at a time;
// four: 207 us). Bound by HBM on the [N x D] rows. SPLIT: the block's four wavefronts share a token's
// columns, which fills the compute units with few tokens and shortens their chains: 8 tokens of 4096 f32
// 18.0 -> 7.6 us, 1024 of 2048 f32 15.6 -> 12.7 us, 8192 of 2048 bf16 53 -> 50 us. With many tokens the
// wavefronts' joins cost more than that: 32768 of 2048 bf16 188 -> 200 us, 65536 of 512 100 -> 211 us.
template <bool BF16, bool SPLIT>
__global__ __launch_bounds__(kAlphaThreads) void alpha_grad_kernel(int T, int K, int D, int64_t N,
                                                                   const uint4* __restrict__ G,
                                                                   const uint4* __restrict__ Y,
                                                                   const float* __restrict__ alpha,
                                                                   const int32_t* __restrict__ pmap,
                                                                   const uint8_t* __restrict__ keep,
                                                                   float* __restrict__ dalpha) {
  constexpr int kWaves = kAlphaThreads / kWave;
  __shared__ double part[SPLIT ? kWaves : 1][kAlphaRows];
  const int lane = threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int64_t t = SPLIT ? blockIdx.x : (int64_t)blockIdx.x * kWaves + wave;
  if (t >= T) return;
  const int words = BF16 ? D / 8 : D / 4;
  for (int k0 = 0; k0 < K; k0 += kAlphaRows) {
    // lane k has slot k0 + k: its pair row, whether that row is read, and its weight
    int j = lane < kAlphaRows && k0 + lane < K ? pmap[t * K + k0 + lane] : -1;
    if (j >= N) j = -1;
    const bool read = j >= 0 && (!keep || keep[j] != 0);
    const float a = j >= 0 ? alpha[j] : 0.0f;
    int row[kAlphaRows];
#pragma unroll
    for (int k = 0; k < kAlphaRows; ++k) row[k] = __builtin_amdgcn_readlane(read ? j : -1, k);
    double s[kAlphaRows] = {0, 0, 0, 0, 0, 0, 0, 0};
    for (int c = SPLIT ? threadIdx.x : lane; c < words; c += SPLIT ? kAlphaThreads : kWave) {
      uint4 y[kAlphaRows];
      const uint4 g = G[t * words + c];
#pragma unroll
      for (int k = 0; k < kAlphaRows; ++k)
        y[k] = row[k] >= 0 ? ld_stream(Y + (int64_t)row[k] * words + c) : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int k = 0; k < kAlphaRows; ++k)
        if (row[k] >= 0) s[k] = dot16<BF16>(g, y[k], s[k]);
    }
    double mine = 0.0;
#pragma unroll
    for (int k = 0; k < kAlphaRows; ++k) {
      if (row[k] < 0) continue;
      const double v = lanes_sum(s[k]);
      mine = lane == k ? v : mine;
    }
    if (SPLIT) {
      if (k0 > 0) __syncthreads();  // the last eight's sums are read
      if (lane < kAlphaRows) part[wave][lane] = mine;
      __syncthreads();
      if (wave != 0) continue;
      mine = 0.0;
      if (lane < kAlphaRows)
#pragma unroll
        for (int q = 0; q < kWaves; ++q) mine += part[q][lane];
    }
    if (j >= 0) dalpha[j] = read && a != 0.0f ? (float)(mine / (double)a) : 0.0f;
  }
}

// Calls f with the layout for E experts and the logits' type: sixteen lanes to a token up to 512
// experts, so that a wavefront takes four tokens and reduces them together, with as few values to a
// lane as hold E. `narrow`: four or eight lanes for up to 64 experts, for callers whose blocks have tokens
// enough to use them all (gradient of 200000 x 16 19.5 -> 7.9 us, of 500000 x 64 bf16 44.9 -> 35.7 us;
// balance loss of 1000000 x 8 60.2 -> 29.6 us; with 128 experts eight lanes gain nothing).
template <bool BF16, class F>
void by_experts(int E, bool narrow, F&& f) {
  if (narrow && E <= 16) f(Layout<4, 4, BF16>());
  else if (narrow && E <= 32) f(Layout<8, 4, BF16>());
  else if (narrow && E <= 64) f(Layout<8, 8, BF16>());
  else if (E <= 64) f(Layout<16, 4, BF16>());
  else if (E <= 128) f(Layout<16, 8, BF16>());
  else if (E <= 192) f(Layout<16, 12, BF16>());
  else if (E <= 256) f(Layout<16, 16, BF16>());
  else if (E <= 320) f(Layout<16, 20, BF16>());
  else if (E <= 384) f(Layout<16, 24, BF16>());
  else if (E <= 512) f(Layout<16, 32, BF16>());
  else f(Layout<64, 16, BF16>());
}
template <class F>
lrmoe_status by_layout(const lrmoe_router* r, bool narrow, F&& f) {
  r->dtype == LRMOE_BF16 ? by_experts<true>(r->E, narrow, f) : by_experts<false>(r->E, narrow, f);
  return launch_status();
}
template <class F>
lrmoe_status by_slots(const lrmoe_router* r, F&& f) {
  r->dtype == LRMOE_BF16 ? by_lists<true>(r->T, r->E, r->K, f) : by_lists<false>(r->T, r->E, r->K, f);
  return launch_status();
}

}  // namespace

size_t route_ws_bytes(const lrmoe_router* r) {
  const size_t rows = (size_t)ceil_div(r->T, route_chunk(r, true)), E8 = align_up(r->E, 8);  // the smaller chunks
  const size_t hist = align_up(rows * E8 * 2, 256);
  return std::max<size_t>(256, hist + align_up((rows + 1) * E8 * 4, 256));
}

lrmoe_status launch_route(const lrmoe_router* r, const lrmoe_scoring* c, const void* logits, const float* bias,
                          const uint8_t* mask, int32_t* idx, float* w, int32_t* counts, int64_t* seg_off, int32_t* tok,
                          int32_t* slot, float* alpha, int32_t* pmap, void* ws, hipStream_t s) {
  const int C = route_chunk(r, c != nullptr), rows = (int)ceil_div(r->T, C);
  const size_t E8 = align_up(r->E, 8);
  int* prefix = sums_own(rows, E8) ? nullptr : (int*)((char*)ws + align_up((size_t)rows * E8 * 2, 256));
  const size_t bits = 4 * (size_t)bit_words(C, r->local), cnt = (size_t)r->E * 4, pairs = (size_t)C * r->K * 8;
  // a chunk's pairs are sorted where they fit beside its bits; without tokens there are no counts to sort by
  const int sorted = rows > 0 && bits + pairs <= kPlaceLds;
  const RouteArgs a{r->T, r->E, r->K, C, rows, r->first, r->local, r->renorm, sorted, r->scale, logits, mask,
                    prefix, prefix ? prefix + (size_t)rows * E8 : nullptr, (uint16_t*)ws,
                    idx, counts, tok, slot, pmap, w, alpha, seg_off};
  if (rows > 0) {
    const size_t lds = rows == 1 ? 2 * cnt + (size_t)C * r->K * 8 + bits : cnt;
    const lrmoe_status st = c ? launch_scored_topk(r, c, a, bias, lds, s) : by_slots(r, [&](auto lay, auto n) {
      using Lay = decltype(lay);
      constexpr int N = decltype(n)::value;
      route_topk_kernel<Lay, N><<<rows, topk_threads(Lay::L, N), lds, s>>>(a);
    });
    if (st != LRMOE_OK || rows == 1) return st;
  }
  if (prefix) {
    route_scan_kernel<<<(unsigned)ceil_div(r->E, kScanExperts), kRouteThreads, 0, s>>>(a);
    if (launch_status() != LRMOE_OK) return LRMOE_ERR_HIP;
  }
  route_place_kernel<<<(unsigned)std::max(1, rows), kRouteThreads, bits + (sorted ? pairs : 0), s>>>(a);
  return launch_status();
}

size_t balance_ws_bytes(const lrmoe_router* r, int32_t n_seq) { return balance_layout(r, n_seq, nullptr, nullptr); }

lrmoe_status launch_balance_loss(const lrmoe_router* r, bool sigmoid, const void* logits, const uint8_t* mask,
                                 const int32_t* idx, const int64_t* seq_off_d, int32_t n_seq, float coef,
                                 int32_t* counts, float* psum, float* norm, float* loss, void* ws, hipStream_t s) {
  BalanceWs b;
  balance_layout(r, n_seq, (char*)ws, &b);
  const int log_tile = balance_log_tile(r);
  // a tile of 64 tokens fills its block with sixteen lanes to each (32768 x 60: 13.7 us, with eight 15.7 us)
  if (by_layout(r, log_tile > 6, [&](auto lay) {
        using Lay = decltype(lay);
        const unsigned g = (unsigned)balance_tiles(r, n_seq);
        auto run = [&](auto kernel) {
          kernel<<<g, kBalThreads, 0, s>>>(r->T, r->E, r->K, n_seq, log_tile, logits, mask, idx, seq_off_d, b);
        };
        if (log_tile > 6) sigmoid ? run(balance_tile_kernel<Lay, true, true>) : run(balance_tile_kernel<Lay, true, false>);
        else if constexpr (Lay::L >= 16)
          sigmoid ? run(balance_tile_kernel<Lay, false, true>) : run(balance_tile_kernel<Lay, false, false>);
      }) != LRMOE_OK)
    return LRMOE_ERR_HIP;
  const dim3 g((unsigned)n_seq, (unsigned)ceil_div(r->E, kJoinExperts));
  if ((int64_t)g.x * g.y <= kJoinLast) {
    balance_join_kernel<kJoinWaves, true><<<g, kJoinWaves * kWave, 0, s>>>(r->T, r->E, r->K, n_seq, log_tile, coef,
                                                                           seq_off_d, b, counts, psum, norm, loss);
    return launch_status();
  }
  balance_join_kernel<kJoinWavesMany, false><<<g, kJoinWavesMany * kWave, 0, s>>>(
      r->T, r->E, r->K, n_seq, log_tile, coef, seq_off_d, b, counts, psum, norm, loss);
  balance_loss_kernel<<<1, kLossThreads, 0, s>>>(r->E, r->K, n_seq, coef, b, norm, loss);
  return launch_status();
}

lrmoe_status launch_route_bwd(const lrmoe_router* r, bool sigmoid, const void* logits, const uint8_t* mask,
                              const int32_t* idx, const float* dalpha, const int32_t* pmap, int64_t n_pairs,
                              const int64_t* seq_off_d, int32_t n_seq, const int32_t* counts, const float* norm,
                              const float* gloss, void* dlogits, hipStream_t s) {
  if (r->E > 512 && r->T > kMaxFours) return LRMOE_ERR_UNSUPPORTED;
  return by_layout(r, true, [&](auto lay) {
    using Lay = decltype(lay);
    constexpr int L = Lay::L, most = std::min(32, L * Lay::V);  // slots: no more than experts
    auto run = [&](auto slots) {
      auto go = [&](auto kernel) {
        kernel<<<(unsigned)ceil_div(r->T, kGradThreads / L), kGradThreads, 0, s>>>(
            r->T, r->E, r->K, r->renorm, r->scale, logits, mask, idx, dalpha, pmap, n_pairs, seq_off_d, n_seq, counts,
            norm, gloss, dlogits);
      };
      constexpr int S = decltype(slots)::value;
      sigmoid ? go(route_bwd_kernel<Lay, S, true>) : go(route_bwd_kernel<Lay, S, false>);
    };
    if (L >= most || r->K <= L) run(std::integral_constant<int, 1>());
    else run(std::integral_constant<int, (most + L - 1) / L>());
  });
}

lrmoe_status launch_alpha_grad(const lrmoe_problem* p, const void* G, const void* Y, const float* alpha,
                               const int32_t* pmap, const uint8_t* keep, float* dalpha, hipStream_t s) {
  const int64_t row = (int64_t)p->D * (p->dtype == LRMOE_BF16 ? 2 : 4);
  const bool split = p->T <= (row >= 16 * kAlphaThreads ? kAlphaSplitWide : kAlphaSplit);
  const unsigned g = (unsigned)(split ? p->T : ceil_div(p->T, kAlphaThreads / kWave));
  auto run = [&](auto kernel) {
    kernel<<<g, kAlphaThreads, 0, s>>>(p->T, p->K, p->D, p->N, (const uint4*)G, (const uint4*)Y, alpha, pmap, keep,
                                       dalpha);
  };
  if (p->dtype == LRMOE_BF16) split ? run(alpha_grad_kernel<true, true>) : run(alpha_grad_kernel<true, false>);
  else split ? run(alpha_grad_kernel<false, true>) : run(alpha_grad_kernel<false, false>);
  return launch_status();
}

}  // namespace lrmoe
