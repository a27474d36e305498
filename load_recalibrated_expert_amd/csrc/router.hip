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

__device__ __forceinline__ float clean(float x) {  // NaN -> -inf, +inf -> FLT_MAX
  return x != x ? kNegInf : fminf(x, kFltMax);
}

// exp(d) for d = x - max: d is at most 0, or NaN where both are -inf (a token that is not live). h + l is
// d log2(e) to about 2^-48, so the error is that of the 2^h instruction and of d itself; below
// -104 it is 0. Half the instructions of expf, whose range checks are not needed here.
__device__ __forceinline__ float exp_below(float d) {
  d = fmaxf(d, -104.0f);
  const float h = d * 1.44269502f;
  const float l = __builtin_fmaf(d, 1.92596303e-8f, __builtin_fmaf(d, 1.44269502f, -h));
  const float r = __builtin_amdgcn_exp2f(h);
  return __builtin_fmaf(r, l * 0.693147181f, r);
}

// Reductions over the L lanes of a token's group (4 to 64); every lane gets the result, the same bits
// in each, as both lanes of a pair compute the same sum. Up to sixteen lanes the partner's value
// comes by DPP, at register speed, instead of a cross-lane permute through LDS. swap<S> exchanges
// lanes S apart, or mirrored in 2 S lanes, which is the same once S lanes agree.
template <int S>
__device__ __forceinline__ int swap(int v) {
  constexpr int ctrl = S == 1 ? 0xB1 : S == 2 ? 0x4E : S == 4 ? 0x141 : 0x140;
  if (S <= 8) return __builtin_amdgcn_update_dpp(0, v, ctrl, 0xF, 0xF, true);
  return __shfl_xor(v, S, kWave);
}
template <int L, int S = 1, class Op>
__device__ __forceinline__ int group_reduce(int v, Op op) {
  if constexpr (S < L) return group_reduce<L, 2 * S>(op(v, swap<S>(v)), op);
  else return v;
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
template <int L>
__device__ __forceinline__ int group_min(int v) {
  return group_reduce<L>(v, [](int a, int b) { return min(a, b); });
}

// How a token's E logits lie over the L lanes of its group, V to a lane, ascending in each lane.
// VEC (E a multiple of 4, so rows are aligned): runs of four, one 16-byte (f32) or 8-byte (bf16)
// load each; else single logits, L apart.
template <int L_, int V_, bool BF16_, bool VEC_>
struct Layout {
  static constexpr int L = L_, V = V_;
  static constexpr bool BF16 = BF16_, VEC = VEC_;
  static __device__ __forceinline__ int expert(int lane, int v) {
    return VEC ? (v >> 2) * (4 * L) + lane * 4 + (v & 3) : v * L + lane;
  }
  // Token t by the rules of the header; -inf beyond E, and everywhere if `on` is false.
  static __device__ __forceinline__ void load(const void* __restrict__ logits, int64_t t, int E, bool on, int lane,
                                              float x[V]) {
    if (VEC) {
#pragma unroll
      for (int q = 0; q < V; q += 4) {
        const int e = expert(lane, q);
        if (on && e < E) {
          if (BF16) {
            const uint2 r = *(const uint2*)((const uint16_t*)logits + t * E + e);
            x[q] = clean(bf16_lo(r.x));
            x[q + 1] = clean(bf16_hi(r.x));
            x[q + 2] = clean(bf16_lo(r.y));
            x[q + 3] = clean(bf16_hi(r.y));
          } else {
            const float4 r = *(const float4*)((const float*)logits + t * E + e);
            x[q] = clean(r.x);
            x[q + 1] = clean(r.y);
            x[q + 2] = clean(r.z);
            x[q + 3] = clean(r.w);
          }
        } else {
          x[q] = x[q + 1] = x[q + 2] = x[q + 3] = kNegInf;
        }
      }
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int e = expert(lane, v);
        x[v] = kNegInf;
        if (on && e < E) x[v] = load_one(logits, t * E + e);
      }
    }
  }
  static __device__ __forceinline__ float load_one(const void* __restrict__ logits, int64_t i) {
    return clean(BF16 ? __uint_as_float((uint32_t)((const uint16_t*)logits)[i] << 16) : ((const float*)logits)[i]);
  }
  // Row s of the [n_seq x E] counts, zeros beyond E and where `on` is false.
  static __device__ __forceinline__ void load_counts(const int32_t* __restrict__ counts, int64_t s, int E, bool on,
                                                     int lane, float c[V]) {
#pragma unroll
    for (int q = 0; q < V; q += VEC ? 4 : 1) {
      const int e = expert(lane, q);
      if (VEC) {
        const int4 n = on && e < E ? *(const int4*)(counts + s * E + e) : make_int4(0, 0, 0, 0);
        c[q] = (float)n.x;
        c[q + 1] = (float)n.y;
        c[q + 2] = (float)n.z;
        c[q + 3] = (float)n.w;
      } else {
        c[q] = on && e < E ? (float)counts[s * E + e] : 0.0f;
      }
    }
  }
  static __device__ __forceinline__ void store(void* __restrict__ out, int64_t t, int E, int lane, const float x[V]) {
    if (VEC) {
#pragma unroll
      for (int q = 0; q < V; q += 4) {
        const int e = expert(lane, q);
        if (e >= E) continue;
        if (BF16)
          *(uint2*)((uint16_t*)out + t * E + e) = make_uint2(pack_bf16x2(x[q], x[q + 1]), pack_bf16x2(x[q + 2], x[q + 3]));
        else
          *(float4*)((float*)out + t * E + e) = make_float4(x[q], x[q + 1], x[q + 2], x[q + 3]);
      }
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int e = expert(lane, v);
        if (e >= E) continue;
        if (BF16) ((uint16_t*)out)[t * E + e] = (uint16_t)pack_bf16x2(x[v], 0.0f);
        else ((float*)out)[t * E + e] = x[v];
      }
    }
  }
};

__device__ __forceinline__ bool unmasked(const uint8_t* __restrict__ mask, int64_t t) { return !mask || mask[t] != 0; }

// ---------------------------------------------------------------- routing

constexpr int kRouteThreads = 1024;   // placing blocks, and the top-K blocks of more than 8 slots
constexpr int kRoute8Threads = 512;   // the top-K blocks of up to 8 slots
constexpr int kOneChunk = 128;        // up to so many tokens one block does the whole call

// Tokens of one top-K block and of one placing block. Each top-K block writes a row of counts, and a
// placing block reads all rows and holds a bit per (token, local expert) in 48 KB of LDS: chunks
// grow until there are at most 512, as far as those bits let them.
int route_chunk(const lrmoe_router* r) {
  int c = kOneChunk;
  while (c < 1024 && ceil_div(r->T, c) > 512 && (int64_t)r->local * c * 2 / 8 <= 48 * 1024) c *= 2;
  return c;
}

struct RouteArgs {
  int T, E, K, C, rows, first, local, renorm;
  float scale;
  const void* logits;
  const uint8_t* mask;
  uint16_t* hist;  // [rows][E8] tokens of each chunk per expert, E8 = E rounded up to 8, zeros behind E
  int32_t *idx, *counts, *tok, *slot, *pmap;
  float *w, *alpha;
  int64_t* seg_off;
};

// Pair rows of the n = tokens * K slots of one chunk, whose experts and weights e_of(i), w_of(i) gives.
// total, before (LDS, [E]): tokens per expert in all chunks and in the chunks before this one; before
// becomes the first row of (chunk, expert). The rank of a pair in its chunk is the number of lower
// set bits among its expert's token bits, so no order of atomics enters the result.
template <int NT, class EOf, class WOf>
__device__ __forceinline__ void place_chunk(const RouteArgs& a, int c, int n, const int* total, int* before,
                                            uint32_t* bits, EOf e_of, WOf w_of) {
  constexpr int kPer = 1024 / NT;  // local experts of one thread in the scan of their totals
  __shared__ int wave_total[NT / kWave];
  const int tid = threadIdx.x, lane = tid & (kWave - 1);
  if (c == 0)
    for (int e = tid; e < a.E; e += NT) a.counts[e] = total[e];
  int v[kPer], mine = 0;
#pragma unroll
  for (int q = 0; q < kPer; ++q) {
    const int l = tid * kPer + q;
    v[q] = l < a.local ? total[a.first + l] : 0;
    mine += v[q];
  }
  int inc = mine;
#pragma unroll
  for (int o = 1; o < kWave; o <<= 1) {
    const int up = __shfl_up(inc, o, kWave);
    if (lane >= o) inc += up;
  }
  if (lane == kWave - 1) wave_total[tid / kWave] = inc;
  __syncthreads();
  int base = inc - mine;
  for (int q = 0; q < tid / kWave; ++q) base += wave_total[q];
#pragma unroll
  for (int q = 0; q < kPer; ++q) {
    const int l = tid * kPer + q;
    if (l < a.local) {
      if (c == 0) {
        a.seg_off[l] = base;
        if (l == a.local - 1) a.seg_off[a.local] = base + v[q];
      }
      before[a.first + l] += base;
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
      row = before[e] + __popc(bits[(t >> 5) * a.local + l] & ((1u << (t & 31)) - 1u));
      for (int q = 0; q < (t >> 5); ++q) row += __popc(bits[q * a.local + l]);
      a.tok[row] = (int32_t)(t0 + t);
      a.slot[row] = i - t * a.K;
      a.alpha[row] = w_of(i);
    }
    a.pmap[t0 * a.K + i] = row;
  }
}

// What the two top-K kernels have in common: the block's LDS, one slot's outputs, and the end.
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
      place_chunk<NT>(a, 0, a.T * a.K, cnt, before, bits, [&](int i) { return e_of[i]; }, [&](int i) { return w_of[i]; });
    } else {
      const int E8 = (a.E + 7) & ~7;
      for (int e = threadIdx.x; e < E8; e += NT)
        a.hist[(int64_t)blockIdx.x * E8 + e] = e < a.E ? (uint16_t)cnt[e] : 0;
    }
  }
};

// Up to 8 slots. A logit and its expert make one positive double: the logit's bits, mapped so that
// they order as unsigned numbers, above 1023 - e, so one f64 maximum compares both and ties go to
// the lower index. Lanes sort their values in eights (19 exchanges of a maximum and a minimum),
// and lists of eight are merged, in a lane and then over the token's lanes: the larger halves of
// one list against the other reversed are the eight largest of both, sorted by 12 more exchanges.
// With four lanes to a token (up to 128 experts) that is about 45 instructions a token and
// wavefront, where taking the largest K times over costs 240: 32768 x 128 takes TOPK8_US here and
// 13.4 us that way.
#pragma float_control(precise, off, push)  // maxima without NaN handling: there are none among the keys
__device__ __forceinline__ void exchange(double& a, double& b) {
  const double hi = __builtin_fmax(a, b), lo = __builtin_fmin(a, b);
  a = hi;
  b = lo;
}
__device__ __forceinline__ void sort8(double* a) {
  exchange(a[0], a[1]), exchange(a[2], a[3]), exchange(a[4], a[5]), exchange(a[6], a[7]);
  exchange(a[0], a[2]), exchange(a[1], a[3]), exchange(a[4], a[6]), exchange(a[5], a[7]);
  exchange(a[1], a[2]), exchange(a[5], a[6]);
  exchange(a[0], a[4]), exchange(a[1], a[5]), exchange(a[2], a[6]), exchange(a[3], a[7]);
  exchange(a[2], a[4]), exchange(a[3], a[5]);
  exchange(a[1], a[2]), exchange(a[3], a[4]), exchange(a[5], a[6]);
}
// a = the eight largest of a and b, both sorted
__device__ __forceinline__ void merge8(double* a, const double* b) {
#pragma unroll
  for (int i = 0; i < 8; ++i) a[i] = __builtin_fmax(a[i], b[7 - i]);
  exchange(a[0], a[4]), exchange(a[1], a[5]), exchange(a[2], a[6]), exchange(a[3], a[7]);
  exchange(a[0], a[2]), exchange(a[1], a[3]), exchange(a[4], a[6]), exchange(a[5], a[7]);
  exchange(a[0], a[1]), exchange(a[2], a[3]), exchange(a[4], a[5]), exchange(a[6], a[7]);
}
#pragma float_control(pop)
template <int L, int S = 1>
__device__ __forceinline__ void merge_lanes(double* a) {
  if constexpr (S < L) {
    double b[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) b[i] = __hiloint2double(swap<S>(__double2hiint(a[i])), swap<S>(__double2loint(a[i])));
    merge8(a, b);
    merge_lanes<L, 2 * S>(a);
  }
}
__device__ __forceinline__ double key_of(float x, int e) {
  const int u = __float_as_int(x + 0.0f);  // -0 ties with 0
  const uint32_t k = (uint32_t)u ^ ((uint32_t)(u >> 31) | 0x80000000u);
  return __hiloint2double((int)(k >> 1), (int)(k << 31 | (uint32_t)(1023 - e)));
}
__device__ __forceinline__ void of_key(double d, float* x, int* e) {  // e = -1 for -inf
  const uint32_t hi = (uint32_t)__double2hiint(d), lo = (uint32_t)__double2loint(d), k = hi << 1 | lo >> 31;
  *x = __uint_as_float(k >> 31 ? k ^ 0x80000000u : ~k);
  *e = k > 0x007FFFFFu ? 1023 - (int)(lo & 1023u) : -1;
}

template <class Lay>
__global__ __launch_bounds__(kRoute8Threads) void route_topk8_kernel(RouteArgs a) {
  constexpr int L = Lay::L, V = Lay::V, kGroups = kRoute8Threads / L;
  constexpr int S = (8 + L - 1) / L;  // slots of a lane: k = lane, lane + L
  extern __shared__ uint32_t lds[];
  RouteBlock<kRoute8Threads> blk(a, lds);
  const int lane = threadIdx.x & (L - 1), group = threadIdx.x / L;
  const int64_t t0 = (int64_t)blockIdx.x * a.C, t1 = min(t0 + a.C, (int64_t)a.T);
  __syncthreads();
  for (int64_t tb = t0; tb < t1; tb += kGroups) {
    const int64_t t = tb + group;
    const bool in = t < t1;
    float x[V];
    Lay::load(a.logits, t, a.E, in && unmasked(a.mask, t), lane, x);
    float top = kNegInf, Z = 0.0f;
    if (!a.renorm) {
#pragma unroll
      for (int v = 0; v < V; ++v) top = fmaxf(top, x[v]);
      top = group_max<L>(top);
#pragma unroll
      for (int v = 0; v < V; ++v) Z += exp_below(x[v] - top);
      Z = group_sum<L>(Z);
    }
    double best[8];
#pragma unroll
    for (int q = 0; q < V; q += 8) {
      double d[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) d[i] = key_of(x[q + i], Lay::expert(lane, q + i));
      sort8(d);
      if (q == 0) {
#pragma unroll
        for (int i = 0; i < 8; ++i) best[i] = d[i];
      } else {
        merge8(best, d);
      }
    }
    merge_lanes<L>(best);
    int e[S], top_e;
    float p[S], sum = 0.0f;
    of_key(best[0], &top, &top_e);
#pragma unroll
    for (int q = 0; q < S; ++q) {
      const int k = lane + q * L;
      double d = 0.0;
#pragma unroll
      for (int i = q * L; i < 8 && i < (q + 1) * L; ++i) d = i == k ? best[i] : d;
      float xk;
      of_key(d, &xk, &e[q]);
      if (k >= a.K) e[q] = -1;
      p[q] = e[q] >= 0 ? exp_below(xk - top) : 0.0f;
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

// More than 8 slots: the largest value left, K times.
template <class Lay>
__global__ __launch_bounds__(kRouteThreads) void route_topk_kernel(RouteArgs a) {
  constexpr int L = Lay::L, V = Lay::V, kGroups = kRouteThreads / L;
  constexpr int S = (32 + L - 1) / L;  // slots that a lane keeps: k = lane, lane + L
  extern __shared__ uint32_t lds[];
  RouteBlock<kRouteThreads> blk(a, lds);
  const int lane = threadIdx.x & (L - 1), group = threadIdx.x / L;
  const int64_t t0 = (int64_t)blockIdx.x * a.C, t1 = min(t0 + a.C, (int64_t)a.T);
  float next[V];
  Lay::load(a.logits, t0 + group, a.E, t0 + group < t1 && unmasked(a.mask, t0 + group), lane, next);
  __syncthreads();
  for (int64_t tb = t0; tb < t1; tb += kGroups) {
    const int64_t t = tb + group;
    const bool in = t < t1;
    float x[V];
#pragma unroll
    for (int v = 0; v < V; ++v) x[v] = next[v];
    if (tb + kGroups < t1)  // the next pass's row, while this one is ranked
      Lay::load(a.logits, t + kGroups, a.E, t + kGroups < t1 && unmasked(a.mask, t + kGroups), lane, next);
    float top = kNegInf, Z = 0.0f;
    if (!a.renorm) {
#pragma unroll
      for (int v = 0; v < V; ++v) top = fmaxf(top, x[v]);
      top = group_max<L>(top);
#pragma unroll
      for (int v = 0; v < V; ++v) Z += exp_below(x[v] - top);
      Z = group_sum<L>(Z);
    }
    // slot k: the largest value left, and the lowest index that has it
    int my_e[S];
    float my_x[S];
#pragma unroll
    for (int q = 0; q < S; ++q) my_e[q] = -1, my_x[q] = kNegInf;
    for (int k = 0; k < a.K; ++k) {
      float best = kNegInf;
#pragma unroll
      for (int v = 0; v < V; ++v) best = fmaxf(best, x[v]);
      best = group_max<L>(best);
      if (k == 0) top = best;
      int at = 1 << 30;
      bool hit[V], found = false;
#pragma unroll
      for (int v = 0; v < V; ++v) {  // the lane's first value that is the best
        const bool eq = x[v] == best;
        hit[v] = eq && !found;
        found = found || eq;
        at = hit[v] ? Lay::expert(lane, v) : at;
      }
      const int win = group_min<L>(at);
      const bool mine = at == win;
#pragma unroll
      for (int v = 0; v < V; ++v) x[v] = hit[v] && mine ? kNegInf : x[v];
#pragma unroll
      for (int q = 0; q < S; ++q)
        if (lane + q * L == k) {
          my_e[q] = best > kNegInf ? win : -1;
          my_x[q] = best;
        }
    }
    float p[S], sum = 0.0f;
#pragma unroll
    for (int q = 0; q < S; ++q) {
      p[q] = my_e[q] >= 0 ? exp_below(my_x[q] - top) : 0.0f;
      sum += p[q];
    }
    if (a.renorm) Z = group_sum<L>(sum);
#pragma unroll
    for (int q = 0; q < S; ++q) {
      const int k = lane + q * L;
      if (in && k < a.K) blk.put(a, t, k, my_e[q], my_e[q] >= 0 ? a.scale * (p[q] / Z) : 0.0f);
    }
  }
  blk.finish(a);
}

// One block per chunk: sums all rows of counts itself (they are in L2), which saves a launch that scans
// them. Thread: eight experts, every stripes-th row.
__global__ __launch_bounds__(kRouteThreads) void route_place_kernel(RouteArgs a, int log_q) {
  __shared__ int total[1024], before[1024];
  extern __shared__ uint32_t bits[];  // [C / 32][local]
  const int tid = threadIdx.x, c = blockIdx.x;
  const int64_t i0 = (int64_t)c * a.C * a.K;
  const int n = (int)(min((int64_t)(c + 1) * a.C, (int64_t)a.T) * a.K - i0);
  const int e0 = tid < n ? a.idx[i0 + tid] : -1;  // on its way while the rows are summed
  const float w0 = tid < n ? a.w[i0 + tid] : 0.0f;
  total[tid] = before[tid] = 0;
  for (int i = tid; i < a.C / 32 * a.local; i += kRouteThreads) bits[i] = 0;
  __syncthreads();
  const int E8 = (a.E + 7) & ~7, e = 8 * (tid & ((1 << log_q) - 1)), stripes = kRouteThreads >> log_q;
  if (e < E8) {
    int sum[8] = {0, 0, 0, 0, 0, 0, 0, 0}, low[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll 4
    for (int r = tid >> log_q; r < a.rows; r += stripes) {
      const uint4 h = *(const uint4*)(a.hist + (int64_t)r * E8 + e);
      const uint32_t w[4] = {h.x, h.y, h.z, h.w};
      const int m = r < c ? -1 : 0;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int lo = (int)(w[q] & 0xFFFFu), hi = (int)(w[q] >> 16);
        sum[2 * q] += lo, sum[2 * q + 1] += hi;
        low[2 * q] += lo & m, low[2 * q + 1] += hi & m;
      }
    }
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      if (sum[q]) atomicAdd(&total[e + q], sum[q]);
      if (low[q]) atomicAdd(&before[e + q], low[q]);
    }
  }
  __syncthreads();
  place_chunk<kRouteThreads>(
      a, c, n, total, before, bits, [&](int i) { return i < kRouteThreads ? e0 : a.idx[i0 + i]; },
      [&](int i) { return i < kRouteThreads ? w0 : a.w[i0 + i]; });
}

// ---------------------------------------------------------------- balance loss

constexpr int kBalThreads = 1024;
constexpr int kBalTile = 64;  // tokens of one tile

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

// Sequence s has the tile slots from floor(off[s] / tile) + s on, which are at least as many as it
// has tiles, so tiles need no table: floor(T / tile) + n_seq slots in all.
__device__ __forceinline__ int64_t first_tile(int64_t lo, int s) { return lo / kBalTile + s; }

__device__ __forceinline__ int seq_of_tile(const int64_t* __restrict__ off, int n_seq, int T, int64_t b) {
  int a = 0, z = n_seq - 1;  // the last sequence whose first slot is at or before b
  while (a < z) {
    const int m = (a + z + 1) / 2;
    int64_t lo, hi;
    seq_range(off, m, T, &lo, &hi);
    if (first_tile(lo, m) <= b) a = m;
    else z = m - 1;
  }
  return a;
}

struct BalanceWs {
  float* psum;     // [tiles][E] sums of probabilities
  int32_t* count;  // [tiles][E]
  int32_t* live;   // [tiles]
  double* dot;     // [n_seq][parts] sum_e counts psum over 64 experts
  int32_t* n;      // [n_seq] live tokens
  uint32_t* done;  // join blocks that are through
};

int64_t balance_tiles(const lrmoe_router* r, int32_t n_seq) { return r->T / kBalTile + n_seq; }

size_t balance_layout(const lrmoe_router* r, int32_t n_seq, char* base, BalanceWs* out) {
  const size_t tiles = (size_t)balance_tiles(r, n_seq), parts = (size_t)ceil_div(r->E, kWave);
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

// One block per tile slot; up to 512 experts every group of lanes has one token.
template <class Lay>
__global__ __launch_bounds__(kBalThreads) void balance_tile_kernel(int T, int E, int K, int n_seq,
                                                                   const void* __restrict__ logits,
                                                                   const uint8_t* __restrict__ mask,
                                                                   const int32_t* __restrict__ idx,
                                                                   const int64_t* __restrict__ off, BalanceWs ws) {
  constexpr int L = Lay::L, V = Lay::V, kGroups = kBalThreads / L, kWaves = kBalThreads / kWave;
  __shared__ int cnt[1024];
  __shared__ float part[kWaves][L * V];
  __shared__ int live_of[kBalTile];
  const int64_t b = blockIdx.x;
  if (b == 0 && threadIdx.x == 0) *ws.done = 0;
  const int s = off ? seq_of_tile(off, n_seq, T, b) : 0;
  int64_t lo, hi;
  seq_range(off, s, T, &lo, &hi);
  lo += (b - first_tile(lo, s)) * kBalTile;
  hi = min(hi, lo + kBalTile);
  if (lo >= hi) return;  // a slot that no tile uses: the whole block leaves
  for (int e = threadIdx.x; e < E; e += kBalThreads) cnt[e] = 0;
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
  if (threadIdx.x < kBalTile) {
    const unsigned long long on = __ballot(threadIdx.x < hi - lo && live_of[threadIdx.x] != 0);
    if (threadIdx.x == 0) ws.live[b] = __popcll(on);
  }
}

constexpr int kJoinThreads = 1024, kJoinWaves = kJoinThreads / kWave;

__device__ __forceinline__ double block_sum(double v, double* sh) {  // kJoinThreads threads, all get the sum
  v = wave_sum(v);
  if ((threadIdx.x & (kWave - 1)) == 0) sh[threadIdx.x / kWave] = v;
  __syncthreads();
  double a = 0.0;
  for (int i = 0; i < kJoinWaves; ++i) a += sh[i];
  __syncthreads();
  return a;
}

// Grid (sequence, 64 experts): the sequence's tiles joined, wavefront by wavefront and then over
// the wavefronts, always in the same order. The block that finishes last sums the loss; it reads
// what the others wrote behind their release, in a fixed order, so the result does not depend on
// which block it is.
__global__ __launch_bounds__(kJoinThreads) void balance_join_kernel(int T, int E, int K, int n_seq, float coef,
                                                                    const int64_t* __restrict__ off, BalanceWs ws,
                                                                    int32_t* __restrict__ counts,
                                                                    float* __restrict__ psum, float* __restrict__ norm,
                                                                    float* __restrict__ loss) {
  __shared__ double sh[kJoinWaves], sum_of[kJoinWaves][kWave];
  __shared__ int n_of[kJoinWaves][kWave];
  __shared__ bool last;
  const int s = blockIdx.x, part = blockIdx.y, parts = gridDim.y;
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave, e = part * kWave + lane;
  int64_t lo, hi;
  seq_range(off, s, T, &lo, &hi);
  const int64_t b0 = first_tile(lo, s);
  const int tiles = (int)((hi - lo + kBalTile - 1) / kBalTile);
  double a = 0.0;
  int n = 0;
  if (e < E) {
#pragma unroll 16
    for (int i = wave; i < tiles; i += kJoinWaves) {
      a += (double)ws.psum[(b0 + i) * E + e];
      n += ws.count[(b0 + i) * E + e];
    }
  }
  sum_of[wave][lane] = a;
  n_of[wave][lane] = n;
  int live = 0;
  if (part == 0)
    for (int i = threadIdx.x; i < tiles; i += kJoinThreads) live += ws.live[b0 + i];
  __syncthreads();
  double dot = 0.0;
  if (wave == 0 && e < E) {
    a = 0.0;
    n = 0;
    for (int q = 0; q < kJoinWaves; ++q) {
      a += sum_of[q][lane];
      n += n_of[q][lane];
    }
    psum[(int64_t)s * E + e] = (float)a;
    counts[(int64_t)s * E + e] = n;
    dot = a * n;
  }
  dot = wave_sum(dot);
  const double alive_tokens = block_sum((double)live, sh);  // exact: whole numbers
  if (threadIdx.x == 0) {
    __hip_atomic_store(&ws.dot[(int64_t)s * parts + part], dot, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (part == 0) __hip_atomic_store(&ws.n[s], (int)alive_tokens, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    const uint32_t before = __hip_atomic_fetch_add(ws.done, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT);
    last = before == gridDim.x * gridDim.y - 1;
  }
  __syncthreads();
  if (!last) return;
  double alive = 0.0, sum = 0.0;
  for (int i = threadIdx.x; i < n_seq; i += kJoinThreads)
    alive += __hip_atomic_load(&ws.n[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) > 0 ? 1.0 : 0.0;
  alive = block_sum(alive, sh);
  for (int i = threadIdx.x; i < n_seq; i += kJoinThreads) {
    const double m = __hip_atomic_load(&ws.n[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    const double f = m > 0 ? (double)coef * E / (alive * K * m * m) : 0.0;
    norm[i] = (float)f;
    double d = 0.0;
    for (int q = 0; q < parts; ++q)
      d += __hip_atomic_load(&ws.dot[(int64_t)i * parts + q], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    sum += f * d;
  }
  sum = block_sum(sum, sh);
  if (threadIdx.x == 0) loss[0] = (float)sum;
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
template <class Lay>
__global__ __launch_bounds__(kGradThreads) void route_bwd_kernel(
    int T, int E, int K, int renorm, float scale, const void* __restrict__ logits, const uint8_t* __restrict__ mask,
    const int32_t* __restrict__ idx, const float* __restrict__ dalpha, const int32_t* __restrict__ pmap,
    int64_t n_pairs, const int64_t* __restrict__ off, int n_seq, const int32_t* __restrict__ counts,
    const float* __restrict__ norm, const float* __restrict__ gloss, void* __restrict__ dlogits) {
  constexpr int L = Lay::L, V = Lay::V;
  constexpr int S = (32 + L - 1) / L;  // slots of a lane: k = lane, lane + L
  __shared__ float rows[kGradThreads / L][L * V];
  const int lane = threadIdx.x & (L - 1);
  const int64_t t = (int64_t)blockIdx.x * (kGradThreads / L) + threadIdx.x / L;
  const bool in = t < T, on = in && unmasked(mask, t);
  // the slots' loads start first: three of them depend on each other
  int e[S];
  float xe[S], y[S];
  if (dalpha) {
#pragma unroll
    for (int q = 0; q < S; ++q) {
      const int k = lane + q * L;
      e[q] = on && k < K ? idx[t * K + k] : -1;
      y[q] = 0.0f;
      xe[q] = kNegInf;
      if (e[q] >= 0 && e[q] < E) {
        const int64_t j = pmap ? pmap[t * K + k] : t * K + k;
        if (!pmap || (j >= 0 && j < n_pairs)) y[q] = scale * dalpha[j];
        xe[q] = Lay::load_one(logits, t * E + e[q]);
      }
    }
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
    float* row = rows[threadIdx.x / L];
#pragma unroll
    for (int v = 0; v < V; ++v) row[Lay::expert(lane, v)] = 0.0f;
    float ref = top, r = rz, q_of[S], s = 0.0f;
    if (renorm) {  // softmax over the chosen experts
      ref = kNegInf;
#pragma unroll
      for (int q = 0; q < S; ++q) ref = fmaxf(ref, xe[q]);
      ref = group_max<L>(ref);
      r = 1.0f;
    }
#pragma unroll
    for (int q = 0; q < S; ++q) q_of[q] = xe[q] > kNegInf ? exp_below(xe[q] - ref) * r : 0.0f;
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
    float c[V], dot = 0.0f;
    Lay::load_counts(counts, s, E, inside, lane, c);
#pragma unroll
    for (int v = 0; v < V; ++v) dot += p[v] * c[v];
    dot = group_sum<L>(dot);
    const float f = inside ? norm[s] * (gloss ? gloss[0] : 1.0f) : 0.0f;
    if (inside) {
#pragma unroll
      for (int v = 0; v < V; ++v) dx[v] += f * (p[v] * (c[v] - dot));
    }
  }
  if (!in) return;
#pragma unroll
  for (int v = 0; v < V; ++v) dx[v] = live ? dx[v] : 0.0f;
  Lay::store(dlogits, t, E, lane, dx);
}

// ---------------------------------------------------------------- gradient of the routing weights

constexpr int kAlphaThreads = 256;

// One wavefront per token: its gradient row against the rows of its K pairs. Products and sums in
// fp64, as the score's norms.
template <bool BF16>
__global__ __launch_bounds__(kAlphaThreads) void alpha_grad_kernel(int T, int K, int D, int64_t N,
                                                                   const uint4* __restrict__ G,
                                                                   const uint4* __restrict__ Y,
                                                                   const float* __restrict__ alpha,
                                                                   const int32_t* __restrict__ pmap,
                                                                   const uint8_t* __restrict__ keep,
                                                                   float* __restrict__ dalpha) {
  const int lane = threadIdx.x & (kWave - 1);
  const int64_t t = (int64_t)blockIdx.x * (kAlphaThreads / kWave) + __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  if (t >= T) return;
  const int words = BF16 ? D / 8 : D / 4;
  for (int k = 0; k < K; ++k) {
    const int64_t j = pmap[t * K + k];
    if (j < 0 || j >= N) continue;
    double s = 0.0;
    const float a = alpha[j];
    if (a != 0.0f && (!keep || keep[j])) {
      for (int c = lane; c < words; c += kWave) {
        const uint4 g = G[t * words + c], y = ld_stream(Y + j * words + c);
        const uint32_t gw[4] = {g.x, g.y, g.z, g.w}, yw[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (BF16) {
            s += (double)(bf16_lo(gw[i]) * bf16_lo(yw[i]));  // exact in f32
            s += (double)(bf16_hi(gw[i]) * bf16_hi(yw[i]));
          } else {
            s += (double)__uint_as_float(gw[i]) * (double)__uint_as_float(yw[i]);
          }
        }
      }
      s = wave_sum(s) / (double)a;
    }
    if (lane == 0) dalpha[j] = (float)s;
  }
}

// Calls f with the layout for E experts and the logits' type: sixteen lanes to a token up to 512
// experts, so that a wavefront takes four tokens and reduces them together, with as few values to a
// lane as hold E (257 experts in bf16: 73 us with 32 lanes of 16, 41 us with 16 lanes of 20).
template <bool BF16, bool VEC, class F>
void by_experts(int E, F&& f) {
  if (E <= 16) f(Layout<16, 1, BF16, false>());
  else if (E <= 64) f(Layout<16, 4, BF16, VEC>());
  else if (E <= 128) f(Layout<16, 8, BF16, VEC>());
  else if (E <= 192) f(Layout<16, 12, BF16, VEC>());
  else if (E <= 256) f(Layout<16, 16, BF16, VEC>());
  else if (E <= 320) f(Layout<16, 20, BF16, VEC>());
  else if (E <= 384) f(Layout<16, 24, BF16, VEC>());
  else if (E <= 512) f(Layout<16, 32, BF16, VEC>());
  else f(Layout<64, 16, BF16, VEC>());
}
// The same for lists of eight: values by the eight, and as few lanes as hold them in 40 values each.
template <bool BF16, bool VEC, class F>
void by_experts8(int E, F&& f) {
  if (E <= 32) f(Layout<4, 8, BF16, VEC>());
  else if (E <= 64) f(Layout<4, 16, BF16, VEC>());
  else if (E <= 128) f(Layout<4, 32, BF16, VEC>());
  else if (E <= 192) f(Layout<8, 24, BF16, VEC>());
  else if (E <= 256) f(Layout<8, 32, BF16, VEC>());
  else if (E <= 320) f(Layout<8, 40, BF16, VEC>());
  else if (E <= 512) f(Layout<16, 32, BF16, VEC>());
  else f(Layout<32, 32, BF16, VEC>());
}
template <class F>
lrmoe_status by_layout8(const lrmoe_router* r, F&& f) {
  const bool vec = r->E % 4 == 0;
  if (r->dtype == LRMOE_BF16) vec ? by_experts8<true, true>(r->E, f) : by_experts8<true, false>(r->E, f);
  else vec ? by_experts8<false, true>(r->E, f) : by_experts8<false, false>(r->E, f);
  return launch_status();
}
template <class F>
lrmoe_status by_layout(const lrmoe_router* r, F&& f) {
  const bool vec = r->E % 4 == 0;
  if (r->dtype == LRMOE_BF16) vec ? by_experts<true, true>(r->E, f) : by_experts<true, false>(r->E, f);
  else vec ? by_experts<false, true>(r->E, f) : by_experts<false, false>(r->E, f);
  return launch_status();
}

}  // namespace

size_t route_ws_bytes(const lrmoe_router* r) {
  return align_up(std::max<size_t>(16, (size_t)ceil_div(r->T, route_chunk(r)) * align_up(r->E, 8) * 2), 256);
}

lrmoe_status launch_route(const lrmoe_router* r, const void* logits, const uint8_t* mask, int32_t* idx, float* w,
                          int32_t* counts, int64_t* seg_off, int32_t* tok, int32_t* slot, float* alpha,
                          int32_t* pmap, void* ws, hipStream_t s) {
  const int C = route_chunk(r), rows = (int)ceil_div(r->T, C);
  const RouteArgs a{r->T, r->E, r->K, C, rows, r->first, r->local, r->renorm, r->scale, logits, mask,
                    (uint16_t*)ws, idx, counts, tok, slot, pmap, w, alpha, seg_off};
  const size_t bits = (size_t)C / 8 * r->local, cnt = (size_t)r->E * 4;
  if (rows > 0) {
    const size_t lds = rows == 1 ? 2 * cnt + (size_t)C * r->K * 8 + bits : cnt;
    const lrmoe_status st =
        r->K <= 8
            ? by_layout8(r, [&](auto lay) { route_topk8_kernel<decltype(lay)><<<rows, kRoute8Threads, lds, s>>>(a); })
            : by_layout(r, [&](auto lay) { route_topk_kernel<decltype(lay)><<<rows, kRouteThreads, lds, s>>>(a); });
    if (st != LRMOE_OK || rows == 1) return st;
  }
  int log_q = 0;
  while ((8 << log_q) < r->E) ++log_q;
  route_place_kernel<<<(unsigned)std::max(1, rows), kRouteThreads, bits, s>>>(a, log_q);
  return launch_status();
}

size_t balance_ws_bytes(const lrmoe_router* r, int32_t n_seq) { return balance_layout(r, n_seq, nullptr, nullptr); }

lrmoe_status launch_balance_loss(const lrmoe_router* r, const void* logits, const uint8_t* mask, const int32_t* idx,
                                 const int64_t* seq_off_d, int32_t n_seq, float coef, int32_t* counts, float* psum,
                                 float* norm, float* loss, void* ws, hipStream_t s) {
  BalanceWs b;
  balance_layout(r, n_seq, (char*)ws, &b);
  if (by_layout(r, [&](auto lay) {
        balance_tile_kernel<decltype(lay)><<<(unsigned)balance_tiles(r, n_seq), kBalThreads, 0, s>>>(
            r->T, r->E, r->K, n_seq, logits, mask, idx, seq_off_d, b);
      }) != LRMOE_OK)
    return LRMOE_ERR_HIP;
  balance_join_kernel<<<dim3((unsigned)n_seq, (unsigned)ceil_div(r->E, kWave)), kJoinThreads, 0, s>>>(
      r->T, r->E, r->K, n_seq, coef, seq_off_d, b, counts, psum, norm, loss);
  return launch_status();
}

lrmoe_status launch_route_bwd(const lrmoe_router* r, const void* logits, const uint8_t* mask, const int32_t* idx,
                              const float* dalpha, const int32_t* pmap, int64_t n_pairs, const int64_t* seq_off_d,
                              int32_t n_seq, const int32_t* counts, const float* norm, const float* gloss,
                              void* dlogits, hipStream_t s) {
  return by_layout(r, [&](auto lay) {
    using Lay = decltype(lay);
    route_bwd_kernel<Lay><<<(unsigned)ceil_div(r->T, kGradThreads / Lay::L), kGradThreads, 0, s>>>(
        r->T, r->E, r->K, r->renorm, r->scale, logits, mask, idx, dalpha, pmap, n_pairs, seq_off_d, n_seq, counts, norm,
        gloss, dlogits);
  });
}

lrmoe_status launch_alpha_grad(const lrmoe_problem* p, const void* G, const void* Y, const float* alpha,
                               const int32_t* pmap, const uint8_t* keep, float* dalpha, hipStream_t s) {
  const unsigned g = (unsigned)ceil_div(p->T, kAlphaThreads / kWave);
  if (p->dtype == LRMOE_BF16)
    alpha_grad_kernel<true><<<g, kAlphaThreads, 0, s>>>(p->T, p->K, p->D, p->N, (const uint4*)G, (const uint4*)Y,
                                                        alpha, pmap, keep, dalpha);
  else
    alpha_grad_kernel<false><<<g, kAlphaThreads, 0, s>>>(p->T, p->K, p->D, p->N, (const uint4*)G, (const uint4*)Y,
                                                         alpha, pmap, keep, dalpha);
  return launch_status();
}

}  // namespace lrmoe
