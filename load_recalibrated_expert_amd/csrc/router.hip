// The router beside the experts: top-K routing with its expert-major pair lists, the balance
// loss with its per-expert counts, the gradient of the logits, and the gradient of the routing
// weights from the saved output rows.
//
// All of it is one pass over [T x E] logits (or, for the routing-weight gradient, over the
// [N x D] output rows), so memory bounds it at large T and launch latency at small T. A group
// of L lanes holds one token's logits in registers, V to a lane.
#include <algorithm>
#include <type_traits>

#include "common.h"

namespace lrmoe {
namespace {

constexpr float kFltMax = 3.402823466e+38f;
constexpr float kNegInf = -__builtin_huge_valf();

__device__ __forceinline__ float not_nan(float x) { return fmaxf(x, kNegInf); }  // NaN -> -inf: the maximum is the number
__device__ __forceinline__ float clean(float x) { return fminf(not_nan(x), kFltMax); }  // and +inf -> FLT_MAX

// exp(d) for d = x - max: d is at most 0, or NaN where both are -inf (a token that is not live). h + l is
// d log2(e) to about 2^-48, so the error is that of the 2^h instruction and of d itself. That instruction
// gives 0 below 2^-126, so the result is 0 from d of -87.34 down. Half the instructions of expf, whose
// range checks are not needed here. ALL: subnormal results too, to d of -104, for the K slots of a
// token: a chosen expert's weight is not 0 while f32 has a value for it (routing of 32768 x 128: 17.7 us
// without, 17.9 us with it). The probabilities of all experts do without: below 2^-126 they count as 0.
template <bool ALL = false>
__device__ __forceinline__ float exp_below(float d) {
  d = fmaxf(d, -104.0f);
  const float h = d * 1.44269502f;
  const float l = __builtin_fmaf(d, 1.92596303e-8f, __builtin_fmaf(d, 1.44269502f, -h));
  const bool low = ALL && h < -126.0f;  // h + 64 is exact then
  const float r = __builtin_amdgcn_exp2f(low ? h + 64.0f : h);
  const float e = __builtin_fmaf(r, l * 0.693147181f, r);
  return low ? e * 0x1p-64f : e;
}

// A term of a sum of exp(d): without the part l. Its relative error of 1.2 |d| 2^-24 falls with the term,
// so a whole sum over E values is off by less than 2 ln(E) 2^-24 more. NaN if the token is not live.
__device__ __forceinline__ float exp_term(float d) { return __builtin_amdgcn_exp2f(d * 1.44269502f); }

template <int L>
__device__ __forceinline__ float group_max(float v) {
  return __int_as_float(group_reduce<L>(__float_as_int(v), [](int a, int b) {
    return __float_as_int(fmaxf(__int_as_float(a), __int_as_float(b)));
  }));
}
template <int L>
__device__ __forceinline__ float group_sum(float v) {
  return __int_as_float(group_reduce<L>(__float_as_int(v), [](int a, int b) {
    return __float_as_int(__int_as_float(a) + __int_as_float(b));
  }));
}

// Four logits from or to any element of a row: rows of an odd number of experts are aligned to their
// elements only, which vector loads and stores of global memory take.
typedef float f32x4u_t __attribute__((ext_vector_type(4), aligned(4)));
typedef int32_t i32x4u_t __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t bf16x4u_t __attribute__((ext_vector_type(2), aligned(2)));

// How a token's E logits lie over the L lanes of its group, V to a lane: runs of four, 4 L apart,
// ascending in each lane. One 16-byte (f32) or 8-byte (bf16) access takes a run; the run that E
// cuts is taken singly, so nothing behind the last row is touched.
template <int L_, int V_, bool BF16_>
struct Layout {
  static constexpr int L = L_, V = V_;
  static constexpr bool BF16 = BF16_;
  static __device__ __forceinline__ int expert(int lane, int v) { return (v >> 2) * (4 * L) + lane * 4 + (v & 3); }
  static __device__ __forceinline__ float load_one(const void* __restrict__ logits, int64_t i) {
    return BF16 ? __uint_as_float((uint32_t)((const uint16_t*)logits)[i] << 16) : ((const float*)logits)[i];
  }
  // Token t by the rules of the header; -inf beyond E, and everywhere if `on` is false. INF: +inf stays.
  template <bool INF = false>
  static __device__ __forceinline__ void load(const void* __restrict__ logits, int64_t t, int E, bool on, int lane,
                                              float x[V]) {
#pragma unroll
    for (int q = 0; q < V; q += 4) {
      const int e = expert(lane, q);
      float a = kNegInf, b = kNegInf, c = kNegInf, d = kNegInf;
      if (on && e + 4 <= E) {
        if (BF16) {
          const bf16x4u_t r = *(const bf16x4u_t*)((const uint16_t*)logits + t * E + e);
          a = bf16_lo(r[0]), b = bf16_hi(r[0]), c = bf16_lo(r[1]), d = bf16_hi(r[1]);
        } else {
          const f32x4u_t r = *(const f32x4u_t*)((const float*)logits + t * E + e);
          a = r[0], b = r[1], c = r[2], d = r[3];
        }
      } else if (on && e < E) {
        a = load_one(logits, t * E + e);
        if (e + 1 < E) b = load_one(logits, t * E + e + 1);
        if (e + 2 < E) c = load_one(logits, t * E + e + 2);
      }
      x[q] = a, x[q + 1] = b, x[q + 2] = c, x[q + 3] = d;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) x[v] = INF ? not_nan(x[v]) : clean(x[v]);
  }
  // Row s of the [n_seq x E] counts, zeros beyond E and where `on` is false.
  static __device__ __forceinline__ void load_counts(const int32_t* __restrict__ counts, int64_t s, int E, bool on,
                                                     int lane, int32_t c[V]) {
#pragma unroll
    for (int q = 0; q < V; q += 4) {
      const int e = expert(lane, q);
      const int32_t* row = counts + s * E + e;
      i32x4u_t n = {0, 0, 0, 0};
      if (on && e + 4 <= E) {
        n = *(const i32x4u_t*)row;
      } else if (on && e < E) {
        n[0] = row[0];
        if (e + 1 < E) n[1] = row[1];
        if (e + 2 < E) n[2] = row[2];
      }
      c[q] = n[0], c[q + 1] = n[1], c[q + 2] = n[2], c[q + 3] = n[3];
    }
  }
  static __device__ __forceinline__ void store(void* __restrict__ out, int64_t t, int E, int lane, const float x[V]) {
#pragma unroll
    for (int q = 0; q < V; q += 4) {
      const int e = expert(lane, q);
      if (e + 4 <= E) {
        if (BF16) {
          __builtin_nontemporal_store(bf16x4u_t{pack_bf16x2(x[q], x[q + 1]), pack_bf16x2(x[q + 2], x[q + 3])},
                                      (bf16x4u_t*)((uint16_t*)out + t * E + e));
        } else {
          __builtin_nontemporal_store(f32x4u_t{x[q], x[q + 1], x[q + 2], x[q + 3]},
                                      (f32x4u_t*)((float*)out + t * E + e));
        }
      } else if (e < E) {
#pragma unroll
        for (int i = 0; i < 3; ++i)
          if (e + i < E) {
            if (BF16) ((uint16_t*)out)[t * E + e + i] = (uint16_t)pack_bf16x2(x[q + i], 0.0f);
            else ((float*)out)[t * E + e + i] = x[q + i];
          }
      }
    }
  }
};

__device__ __forceinline__ bool unmasked(const uint8_t* __restrict__ mask, int64_t t) { return !mask || mask[t] != 0; }

// ---------------------------------------------------------------- routing

constexpr int kRouteThreads = 1024;  // scanning and placing blocks
constexpr int kFewTokens = 64;       // one pass of 1024 threads at sixteen lanes to a token
constexpr int kOneChunk = 128;       // up to so many tokens one block does the whole call

constexpr size_t kPlaceLds = 48 * 1024;  // of a placing block, beside its 8 KB of sums

// Words of a placing block's bits, one per (token, local expert); an even number.
__host__ __device__ constexpr int bit_words(int C, int local) { return ((C + 31) / 32 * local + 1) & ~1; }

// Tokens of one top-K block and of one placing block, so that the 256 compute units have about as many
// each: 256 chunks of up to 128 tokens, then 512 (top-K and placing of 300000 x 64 in chunks of 1024
// 27.2 + 16.8 us, of 592 19.3 + 12.7 us; 70000 x 1024 bf16 in chunks of 256 121 us, of 144 70 us). Each
// writes a row of counts, so chunks have at least 128 tokens, or 64 where the top-K gains more by
// smaller ones than the scan loses by more rows: above 320 experts, where a token has sixteen or more
// lanes whatever K (16384 x 512 in chunks of 128 22 us, of 64 14.5 us), and with more than 256 chunks
// (50021 x 257 in chunks of 128 23.6 us, of 104 21.8 us). With 9 to 32 slots sixteen lanes begin at 257
// experts; chunks of 64 there were not measured.
int route_chunk(const lrmoe_router* r) {
  if (r->T <= kOneChunk) return kOneChunk;
  const int64_t even = align_up((size_t)ceil_div(r->T, r->T <= 256 * 128 ? 256 : 512), 8);
  const int64_t room = (int64_t)kPlaceLds / 4 / r->local * 32;  // whose bits fit
  return (int)std::min(std::max(even, (int64_t)(r->E > 320 || r->T > 256 * 128 ? 64 : 128)),
                       std::min<int64_t>(room, 1024));
}

struct RouteArgs {
  int T, E, K, C, rows, first, local, renorm, sorted;
  float scale;
  const void* logits;
  const uint8_t* mask;
  int *prefix, *total;  // [rows][E8], [E8]: the scan's results, NULL if it does not run
  uint16_t* hist;  // [rows][E8] tokens of each chunk per expert, E8 = E rounded up to 8, zeros behind E
  int32_t *idx, *counts, *tok, *slot, *pmap;
  float *w, *alpha;
  int64_t* seg_off;
};

// Pair rows of the n = tokens * K slots of one chunk, whose experts and weights e_of(i), w_of(i) gives.
// total, before (LDS, [E]): tokens per expert in all chunks and in the chunks before this one; before
// becomes the first row of (chunk, expert). The rank of a pair in its chunk is the number of lower
// set bits among its expert's token bits, so no order of atomics enters the result.
// sorted (LDS, [2 n], or NULL): the pairs go through it in the order of their rows, so that a store
// touches a run of rows of each expert instead of a line for every lane (the placing of 32768 x 8
// pairs over 128 experts: 8.0 us without, 7.1 us with it; of 32768 x 32 over 256: 21 and 14 us).
template <int NT, class EOf, class WOf>
__device__ __forceinline__ void place_chunk(const RouteArgs& a, int c, int n, int* total, int* before, uint32_t* bits,
                                            uint32_t* sorted, EOf e_of, WOf w_of) {
  constexpr int kPer = 1024 / NT;  // local experts of one thread in the scan of their totals
  __shared__ unsigned long long wave_total[NT / kWave];
  const int tid = threadIdx.x, lane = tid & (kWave - 1);
  if (c == 0)
    for (int e = tid; e < a.E; e += NT) a.counts[e] = total[e];
  // tokens per local expert, in all chunks (high word) and in this one, scanned together
  unsigned long long v[kPer], mine = 0;
#pragma unroll
  for (int q = 0; q < kPer; ++q) {
    const int l = tid * kPer + q, E8 = (a.E + 7) & ~7;
    v[q] = 0;
    if (l < a.local) {
      const uint32_t here = sorted ? a.hist[(int64_t)c * E8 + a.first + l] : 0u;
      v[q] = (unsigned long long)(uint32_t)total[a.first + l] << 32 | here;
    }
    mine += v[q];
  }
  unsigned long long inc = mine;
#pragma unroll
  for (int o = 1; o < kWave; o <<= 1) {
    const unsigned long long up = __shfl_up(inc, o, kWave);
    if (lane >= o) inc += up;
  }
  if (lane == kWave - 1) wave_total[tid / kWave] = inc;
  __syncthreads();
  unsigned long long base = inc - mine;
  for (int q = 0; q < tid / kWave; ++q) base += wave_total[q];
  int m = 0;  // local pairs of this chunk
  if (sorted)
    for (int q = 0; q < NT / kWave; ++q) m += (int)(uint32_t)wave_total[q];
#pragma unroll
  for (int q = 0; q < kPer; ++q) {
    const int l = tid * kPer + q;
    if (l < a.local) {
      if (c == 0) {
        a.seg_off[l] = (int64_t)(base >> 32);
        if (l == a.local - 1) a.seg_off[a.local] = (int64_t)((base + v[q]) >> 32);
      }
      before[a.first + l] += (int)(base >> 32);
      total[a.first + l] = (int)(uint32_t)base;  // from here on: the expert's first place in `sorted`
      base += v[q];
    }
  }
  for (int i = tid; i < n; i += NT) {
    const int e = e_of(i), l = e - a.first, t = i / a.K;
    if (e >= 0 && l >= 0 && l < a.local) atomicOr(&bits[(t >> 5) * a.local + l], 1u << (t & 31));
  }
  __syncthreads();
  const int64_t t0 = (int64_t)c * a.C;
  for (int i = tid; i < n; i += NT) {
    const int e = e_of(i), l = e - a.first, t = i / a.K;
    int row = -1;
    if (e >= 0 && l >= 0 && l < a.local) {
      int rank = __popc(bits[(t >> 5) * a.local + l] & ((1u << (t & 31)) - 1u));
      for (int q = 0; q < (t >> 5); ++q) rank += __popc(bits[q * a.local + l]);
      row = before[e] + rank;
      if (sorted) {
        sorted[2 * (total[e] + rank)] = (uint32_t)l << 16 | (uint32_t)i;
        sorted[2 * (total[e] + rank) + 1] = __float_as_uint(w_of(i));
      } else {
        a.tok[row] = (int32_t)(t0 + t);
        a.slot[row] = i - t * a.K;
        a.alpha[row] = w_of(i);
      }
    }
    a.pmap[t0 * a.K + i] = row;
  }
  if (!sorted) return;
  __syncthreads();
  for (int p = tid; p < m; p += NT) {
    const uint2 s = *(const uint2*)(sorted + 2 * p);
    const int e = a.first + (int)(s.x >> 16), i = (int)(s.x & 0xFFFFu), t = i / a.K, row = before[e] + p - total[e];
    a.tok[row] = (int32_t)(t0 + t);
    a.slot[row] = i - t * a.K;
    a.alpha[row] = __uint_as_float(s.y);
  }
}

// A top-K block's LDS, one slot's outputs, and the end.
template <int NT>
struct RouteBlock {
  // [E] counts; with one block for all tokens also [E] zeros, [C K] experts, [C K] weights, [C / 32][local] bits
  int *cnt, *before, *e_of;
  float* w_of;
  uint32_t* bits;
  bool one;

  __device__ __forceinline__ RouteBlock(const RouteArgs& a, uint32_t* lds) : one(a.rows == 1) {
    cnt = (int*)lds;
    before = cnt + a.E;
    e_of = before + a.E;
    w_of = (float*)(e_of + a.C * a.K);
    bits = (uint32_t*)(w_of + a.C * a.K);
    for (int e = threadIdx.x; e < (one ? 2 * a.E : a.E); e += NT) cnt[e] = 0;
    if (one)
      for (int i = threadIdx.x; i < a.C / 32 * a.local; i += NT) bits[i] = 0;
  }
  __device__ __forceinline__ void put(const RouteArgs& a, int64_t t, int k, int e, float w) {
    a.idx[t * a.K + k] = e;
    a.w[t * a.K + k] = w;
    if (one) {
      e_of[t * a.K + k] = e;
      w_of[t * a.K + k] = w;
    }
    if (e >= 0) atomicAdd(&cnt[e], 1);
  }
  __device__ __forceinline__ void finish(const RouteArgs& a) {
    __syncthreads();
    if (one) {
      place_chunk<NT>(
          a, 0, a.T * a.K, cnt, before, bits, nullptr, [&](int i) { return e_of[i]; }, [&](int i) { return w_of[i]; });
    } else {
      const int E8 = (a.E + 7) & ~7;
      for (int e = threadIdx.x; e < E8; e += NT)
        a.hist[(int64_t)blockIdx.x * E8 + e] = e < a.E ? (uint16_t)cnt[e] : 0;
    }
  }
};

// A logit and its expert make one key: the logit's bits, mapped so that they order as unsigned numbers,
// above 1023 - e, so one maximum compares both and ties go to the lower index. f32 logits take 63
// bits as a positive double (f64 maxima run at full rate), bf16 logits 32. Lanes sort their keys in
// lists of N = 8, 16 or 32, as many as there are slots or more (odd-even merge sort: 19, 63 or 191
// exchanges of a maximum and a minimum), and the lists are merged, in a lane and then over the
// token's lanes: the larger of one list against the other reversed are the N largest of both,
// sorted by N / 2 log2 N more exchanges. With four lanes to a token (up to 128 experts) and 8 slots
// that is a fifth of the instructions of taking the largest K times over: 32768 x 128 f32 takes
// 8.2 us here and 13.4 us that way.
__device__ __forceinline__ double key_max(double a, double b) { return __builtin_fmax(a, b); }
__device__ __forceinline__ double key_min(double a, double b) { return __builtin_fmin(a, b); }
__device__ __forceinline__ uint32_t key_max(uint32_t a, uint32_t b) { return a > b ? a : b; }
__device__ __forceinline__ uint32_t key_min(uint32_t a, uint32_t b) { return a < b ? a : b; }
template <class Key>
__device__ __forceinline__ void exchange(Key& a, Key& b) {
  const Key hi = key_max(a, b), lo = key_min(a, b);
  a = hi;
  b = lo;
}
// Two sorted lists, interleaved at distance R from LO on, become one.
template <int LO, int N, int R, class Key>
__device__ __forceinline__ void merge_odd_even(Key* a) {
  if constexpr (2 * R < N) {
    merge_odd_even<LO, N, 2 * R>(a);
    merge_odd_even<LO + R, N, 2 * R>(a);
#pragma unroll
    for (int i = LO + R; i + R < LO + N; i += 2 * R) exchange(a[i], a[i + R]);
  } else {
    exchange(a[LO], a[LO + R]);
  }
}
template <int LO, int N, class Key>
__device__ __forceinline__ void sort_list(Key* a) {
  if constexpr (N > 1) {
    sort_list<LO, N / 2>(a);
    sort_list<LO + N / 2, N / 2>(a);
    merge_odd_even<LO, N, 1>(a);
  }
}
template <int N, int D, class Key>
__device__ __forceinline__ void sort_bitonic(Key* a) {
  if constexpr (D > 0) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (!(i & D)) exchange(a[i], a[i + D]);
    sort_bitonic<N, D / 2>(a);
  }
}
// a = the N largest of a and b, both sorted
template <int N, class Key>
__device__ __forceinline__ void merge_lists(Key* a, const Key* b) {
#pragma unroll
  for (int i = 0; i < N; ++i) a[i] = key_max(a[i], b[N - 1 - i]);
  sort_bitonic<N, N / 2>(a);
}
template <int S>
__device__ __forceinline__ double key_swap(double v) {
  return __hiloint2double(lane_swap<S>(__double2hiint(v)), lane_swap<S>(__double2loint(v)));
}
template <int S>
__device__ __forceinline__ uint32_t key_swap(uint32_t v) {
  return (uint32_t)lane_swap<S>((int)v);
}
template <int N, int L, int S = 1, class Key>
__device__ __forceinline__ void merge_lanes(Key* a) {
  if constexpr (S < L) {
    Key b[N];
#pragma unroll
    for (int i = 0; i < N; ++i) b[i] = key_swap<S>(a[i]);
    merge_lists<N>(a, b);
    merge_lanes<N, L, 2 * S>(a);
  }
}
__device__ __forceinline__ uint32_t ordered(float x) {
  const int u = __float_as_int(x + 0.0f);  // -0 ties with 0
  return (uint32_t)u ^ ((uint32_t)(u >> 31) | 0x80000000u);
}
__device__ __forceinline__ void to_key(float x, int e, double* k) {
  const uint32_t u = ordered(x);
  *k = __hiloint2double((int)(u >> 1), (int)(u << 31 | (uint32_t)(1023 - e)));
}
__device__ __forceinline__ void to_key(float x, int e, uint32_t* k) {  // the low half of a bf16's bits is 0 or, mapped, ones
  *k = (ordered(x) & 0xFFFF0000u) | (uint32_t)(1023 - e);
}
__device__ __forceinline__ float unordered(uint32_t u) { return __uint_as_float(u >> 31 ? u ^ 0x80000000u : ~u); }
__device__ __forceinline__ void of_key(double d, float* x, int* e) {  // e = -1 for -inf
  const uint32_t hi = (uint32_t)__double2hiint(d), lo = (uint32_t)__double2loint(d), u = hi << 1 | lo >> 31;
  *x = unordered(u);
  *e = u > 0x007FFFFFu ? 1023 - (int)(lo & 1023u) : -1;
}
__device__ __forceinline__ void of_key(uint32_t k, float* x, int* e) {
  const uint32_t u = k >> 31 ? k & 0xFFFF0000u : k | 0xFFFFu;
  *x = fminf(unordered(u), kFltMax);
  *e = u > 0x007FFFFFu ? 1023 - (int)(k & 1023u) : -1;
}

// Threads of a top-K block: 64 tokens in one pass with sixteen lanes to a token, if 1024 threads have the
// registers (lists of 32 do not). 16384 x 512: 15.5 us with 512 threads, 14.5 us with 1024; with
// eight lanes to a token 50021 x 257 takes 22.9 us with 512 and 24.5 us with 1024.
constexpr int topk_threads(int L, int N) { return L >= 16 && N <= 16 ? 1024 : 512; }

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

// Rows of counts up to which every placing block sums them itself, a thread to an expert and one row
// after the other; above, a launch scans them first. 64 rows of 128 experts: 7.3 us of placing against
// 3.2 us of scan and 5.7 us of placing; 128 rows: 9.9 against 3.1 and 6.1 us. (With 128 experts that
// loop leaves seven eighths of the block's threads idle; sums by all of them were not measured.)
constexpr int kOwnRows = 64;
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
  if (tid < a.E) {
    int sum = 0, low = 0;
    if (a.prefix) {
      sum = a.total[tid];
      low = a.prefix[(int64_t)c * E8 + tid];
    } else {
#pragma unroll 8
      for (int r = 0; r < a.rows; ++r) {
        const int h = a.hist[(int64_t)r * E8 + tid];
        sum += h;
        low += r < c ? h : 0;
      }
    }
    total[tid] = sum;
    before[tid] = low;
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
template <class Lay, bool LONG>
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
      x[v] = exp_below(x[v] - top);
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

// The wavefront's LDS accesses before this point are done and seen by its other lanes.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// The K slots of a token are worked on in K lanes of its group, whose results reach the lanes that
// hold their experts through a row of LDS.
template <class Lay, int S>  // S: slots of a lane, k = lane, lane + L, ...
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
  float x[V], p[V], dx[V], top = kNegInf, Z = 0.0f;
  Lay::load(logits, t, E, on, lane, x);
#pragma unroll
  for (int v = 0; v < V; ++v) top = fmaxf(top, x[v]);
  top = group_max<L>(top);
  const bool live = top > kNegInf;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    p[v] = exp_below(x[v] - top);
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
    float xe[S], ref = top, r = rz, q_of[S], s = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) row[Lay::expert(lane, v)] = x[v];
    wave_sync();
#pragma unroll
    for (int q = 0; q < S; ++q) xe[q] = e[q] >= 0 && e[q] < E ? row[e[q]] : kNegInf;
    wave_sync();
#pragma unroll
    for (int v = 0; v < V; ++v) row[Lay::expert(lane, v)] = 0.0f;
    if (renorm) {  // softmax over the chosen experts
      ref = kNegInf;
#pragma unroll
      for (int q = 0; q < S; ++q) ref = fmaxf(ref, xe[q]);
      ref = group_max<L>(ref);
      r = 1.0f;
    }
#pragma unroll
    for (int q = 0; q < S; ++q) q_of[q] = xe[q] > kNegInf ? exp_below<true>(xe[q] - ref) * r : 0.0f;
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
      if (xe[q] > kNegInf) row[e[q]] = renorm ? q_of[q] * (y[q] - s) : q_of[q] * y[q];
    wave_sync();
#pragma unroll
    for (int v = 0; v < V; ++v) {
      dx[v] = row[Lay::expert(lane, v)];
      if (!renorm) dx[v] -= p[v] * s;
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
    Lay::load_counts(counts, s, E, inside, lane, n);
#pragma unroll
    for (int v = 0; v < V; ++v) ref = max(ref, p[v] >= rz ? n[v] : INT32_MIN);
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
    for (int v = 0; v < V; ++v) dx[v] += f * (p[v] * (c[v] - dot));  // zeros where f or, not live, p is 0
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
// The same for lists of N = 8, 16 or 32 slots: whole lists to a lane, and few lanes to a token. Where one
// pass takes all tokens anyway, more lanes shorten its chain of instructions (16 tokens of 128
// experts: 6.1 us with four lanes to a token, 5.6 us with sixteen; one token of 200: 7.8 and 5.9 us;
// 120 tokens of 128, two passes: 7.6 and 9.4 us). Two lanes for up to 16 experts: 1000000 x 8 60 us with
// four, 44 us with two.
template <bool BF16, class F>
void by_lists(int T, int E, int K, F&& f) {
  using std::integral_constant;
  if (K <= 8) {
    integral_constant<int, 8> n;
    if (T <= kFewTokens && E > 32 && E <= 256) {
      if (E <= 64) f(Layout<8, 8, BF16>(), n);
      else if (E <= 128) f(Layout<16, 8, BF16>(), n);
      else f(Layout<16, 16, BF16>(), n);
    } else if (E <= 16) f(Layout<2, 8, BF16>(), n);
    else if (E <= 32) f(Layout<4, 8, BF16>(), n);
    else if (E <= 64) f(Layout<4, 16, BF16>(), n);
    else if (E <= 128) f(Layout<4, 32, BF16>(), n);
    else if (E <= 192) f(Layout<8, 24, BF16>(), n);
    else if (E <= 256) f(Layout<8, 32, BF16>(), n);
    else if (E <= 320) f(Layout<8, 40, BF16>(), n);
    else if (E <= 512) f(Layout<16, 32, BF16>(), n);
    else f(Layout<32, 32, BF16>(), n);
  } else if (K <= 16) {
    integral_constant<int, 16> n;
    if (E <= 64) f(Layout<4, 16, BF16>(), n);
    else if (E <= 128) f(Layout<4, 32, BF16>(), n);
    else if (E <= 256) f(Layout<8, 32, BF16>(), n);
    else if (E <= 512) f(Layout<16, 32, BF16>(), n);
    else f(Layout<32, 32, BF16>(), n);
  } else {
    integral_constant<int, 32> n;
    if (E <= 128) f(Layout<4, 32, BF16>(), n);
    else if (E <= 256) f(Layout<8, 32, BF16>(), n);
    else if (E <= 512) f(Layout<16, 32, BF16>(), n);
    else f(Layout<32, 32, BF16>(), n);
  }
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
  const size_t rows = (size_t)ceil_div(r->T, route_chunk(r)), E8 = align_up(r->E, 8);
  const size_t hist = align_up(rows * E8 * 2, 256);
  return std::max<size_t>(256, rows > kOwnRows ? hist + align_up((rows + 1) * E8 * 4, 256) : hist);
}

lrmoe_status launch_route(const lrmoe_router* r, const void* logits, const uint8_t* mask, int32_t* idx, float* w,
                          int32_t* counts, int64_t* seg_off, int32_t* tok, int32_t* slot, float* alpha,
                          int32_t* pmap, void* ws, hipStream_t s) {
  const int C = route_chunk(r), rows = (int)ceil_div(r->T, C);
  const size_t E8 = align_up(r->E, 8);
  int* prefix = rows > kOwnRows ? (int*)((char*)ws + align_up((size_t)rows * E8 * 2, 256)) : nullptr;
  const size_t bits = 4 * (size_t)bit_words(C, r->local), cnt = (size_t)r->E * 4, pairs = (size_t)C * r->K * 8;
  // a chunk's pairs are sorted where they fit beside its bits; without tokens there are no counts to sort by
  const int sorted = rows > 0 && bits + pairs <= kPlaceLds;
  const RouteArgs a{r->T, r->E, r->K, C, rows, r->first, r->local, r->renorm, sorted, r->scale, logits, mask,
                    prefix, prefix ? prefix + (size_t)rows * E8 : nullptr, (uint16_t*)ws,
                    idx, counts, tok, slot, pmap, w, alpha, seg_off};
  if (rows > 0) {
    const size_t lds = rows == 1 ? 2 * cnt + (size_t)C * r->K * 8 + bits : cnt;
    const lrmoe_status st = by_slots(r, [&](auto lay, auto n) {
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

lrmoe_status launch_balance_loss(const lrmoe_router* r, const void* logits, const uint8_t* mask, const int32_t* idx,
                                 const int64_t* seq_off_d, int32_t n_seq, float coef, int32_t* counts, float* psum,
                                 float* norm, float* loss, void* ws, hipStream_t s) {
  BalanceWs b;
  balance_layout(r, n_seq, (char*)ws, &b);
  const int log_tile = balance_log_tile(r);
  // a tile of 64 tokens fills its block with sixteen lanes to each (32768 x 60: 13.7 us, with eight 15.7 us)
  if (by_layout(r, log_tile > 6, [&](auto lay) {
        using Lay = decltype(lay);
        const unsigned g = (unsigned)balance_tiles(r, n_seq);
        if (log_tile > 6)
          balance_tile_kernel<Lay, true><<<g, kBalThreads, 0, s>>>(r->T, r->E, r->K, n_seq, log_tile, logits, mask, idx,
                                                                   seq_off_d, b);
        else if constexpr (Lay::L >= 16)
          balance_tile_kernel<Lay, false><<<g, kBalThreads, 0, s>>>(r->T, r->E, r->K, n_seq, log_tile, logits, mask,
                                                                    idx, seq_off_d, b);
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

lrmoe_status launch_route_bwd(const lrmoe_router* r, const void* logits, const uint8_t* mask, const int32_t* idx,
                              const float* dalpha, const int32_t* pmap, int64_t n_pairs, const int64_t* seq_off_d,
                              int32_t n_seq, const int32_t* counts, const float* norm, const float* gloss,
                              void* dlogits, hipStream_t s) {
  return by_layout(r, true, [&](auto lay) {
    using Lay = decltype(lay);
    constexpr int L = Lay::L, most = std::min(32, L * Lay::V);  // slots: no more than experts
    auto run = [&](auto slots) {
      route_bwd_kernel<Lay, decltype(slots)::value>
          <<<(unsigned)ceil_div(r->T, kGradThreads / L), kGradThreads, 0, s>>>(
              r->T, r->E, r->K, r->renorm, r->scale, logits, mask, idx, dalpha, pmap, n_pairs, seq_off_d, n_seq, counts,
              norm, gloss, dlogits);
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
