// What the router's kernels share: how a token's logits lie over lanes, exponentials, the sort of keys, and the
// placing of a chunk's pairs into the pair lists.
#pragma once
#include <type_traits>

#include "common.h"

namespace lrmoe {

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

// sigmoid(x) / exp(min(top, 0)) for x of at most top: exp(min(x, 0) - min(top, 0)) / (1 + exp(-|x|)). With top the largest
// logit of a token the terms of its sum are at most 1 and the largest at least 1/2, however low all scores are. The
// reciprocal is to 1 ulp.
template <bool ALL = false>
__device__ __forceinline__ float sigmoid_over(float x, float top) {
  return exp_below<ALL>(fminf(x, 0.0f) - fminf(top, 0.0f)) * __builtin_amdgcn_rcpf(1.0f + exp_below(-fabsf(x)));
}

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

// The wavefront's LDS accesses before this point are done and seen by its other lanes.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// Calls f with the layout for lists of N = 8, 16 or 32 slots: whole lists to a lane, and few lanes to a token. Where one
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

// Where route's launches are shared with routing by scores.
lrmoe_status launch_scored_topk(const lrmoe_router* r, const lrmoe_scoring* c, const RouteArgs& a, const float* bias,
                                size_t lds, hipStream_t s);

}  // namespace lrmoe
