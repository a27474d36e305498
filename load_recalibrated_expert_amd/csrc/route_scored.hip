// Top-K routing by scores: softmax or sigmoid scores, a bias per expert that enters the choice but not the weights,
// and groups of experts of which the best are kept. The pair lists behind it are route's. And the bias update.
//
// The choice compares scores that may be as near as rounding lets them be, and experts are whole numbers, so scores are
// computed in f64: exp by its series, one reciprocal. f64 runs at the rate of f32 without packed instructions, and a
// logit costs 30 instructions more than the choice by logits itself.
#include "router_device.h"

namespace lrmoe {
namespace {

constexpr int kMaxGroups = 64;  // their marks are the bits of a word

struct ScoreArgs {
  const float* bias;  // [E] or NULL
  int sigmoid, groups, size, top, best, by_logit;
  uint32_t per_group;  // ceil(2^20 / size): e * per_group >> 20 is e / size for all e below 1024
};

// exp(y) for y in [-745, 700] to a relative 1e-14 (the key that the result goes into keeps 42 bits, 2e-13): y = n ln 2 + r
// with |r| <= ln 2 / 2, the Taylor series of exp(r) to r^11, whose next term is below 7e-15.
__device__ __forceinline__ double exp64(double y) {
  const double n = __builtin_rint(y * 1.4426950408889634074);
  double r = __builtin_fma(n, -0x1.62e42fefap-1, y);  // 36 bits of ln 2: the product is exact
  r = __builtin_fma(n, -0x1.cf79abc9e3b39p-40, r);
  double p = 1.0 / 39916800.0;
  p = __builtin_fma(p, r, 1.0 / 3628800.0);
  p = __builtin_fma(p, r, 1.0 / 362880.0);
  p = __builtin_fma(p, r, 1.0 / 40320.0);
  p = __builtin_fma(p, r, 1.0 / 5040.0);
  p = __builtin_fma(p, r, 1.0 / 720.0);
  p = __builtin_fma(p, r, 1.0 / 120.0);
  p = __builtin_fma(p, r, 1.0 / 24.0);
  p = __builtin_fma(p, r, 1.0 / 6.0);
  p = __builtin_fma(p, r, 0.5);
  p = __builtin_fma(p, r, 1.0);
  p = __builtin_fma(p, r, 1.0);
  return __builtin_amdgcn_ldexp(p, (int)n);
}

// 1 / d for d in [2^-1000, 2^1015]: the instruction's result has over 20 bits, each step doubles them.
__device__ __forceinline__ double rcp64(double d) {
  double r = __builtin_amdgcn_rcp(d);
  r = __builtin_fma(r, __builtin_fma(-d, r, 1.0), r);
  return __builtin_fma(r, __builtin_fma(-d, r, 1.0), r);
}

constexpr double kNoKey = -__builtin_huge_val();

// A choice score and its expert as one f64: the lowest 10 of the score's 52 bits give way to the expert, so that among
// scores that agree in the other 42 the lower index is the larger key.
__device__ __forceinline__ double score_key(double c, int e) {
  c += 0.0;  // -0
  const int lo = __double2loint(c), hi = __double2hiint(c);
  return __hiloint2double(hi, (lo & ~1023) | (hi < 0 ? e : 1023 - e));
}
__device__ __forceinline__ int key_expert(double k) {  // -1 for no expert
  const int lo = __double2loint(k) & 1023;
  return k == kNoKey ? -1 : __double2hiint(k) < 0 ? lo : 1023 - lo;
}

template <int L, int S = 1>
__device__ __forceinline__ double group_sum64(double v) {
  if constexpr (S < L) return group_sum64<L, 2 * S>(v + key_swap<S>(v));
  else return v;
}

constexpr int scored_threads(bool groups, int L, int V) { return groups && V > 16 ? 256 : 512; }

// As route_topk_kernel, with keys of choice scores instead of logits. GROUPS: a token's scores pass through a row of LDS,
// where a lane finds the one or two largest of a group.
template <class Lay, int N, bool GROUPS>
__global__ __launch_bounds__(scored_threads(GROUPS, Lay::L, Lay::V)) void route_scored_kernel(RouteArgs a, ScoreArgs s) {
  constexpr int L = Lay::L, V = Lay::V, NT = scored_threads(GROUPS, L, V), kTokens = NT / L;
  constexpr int S = (N + L - 1) / L;  // slots of a lane: k = lane, lane + L, ...
  static_assert(V % N == 0, "whole lists");
  extern __shared__ uint32_t lds[];
  __shared__ double score_of[GROUPS ? kTokens : 1][GROUPS ? L * V : 1], group_of[GROUPS ? kTokens : 1][GROUPS ? kMaxGroups : 1];
  RouteBlock<NT> blk(a, lds);
  const int lane = threadIdx.x & (L - 1);
  const int64_t t0 = (int64_t)blockIdx.x * a.C, t1 = min(t0 + a.C, (int64_t)a.T);
  float bias[V];
#pragma unroll
  for (int v = 0; v < V; ++v) bias[v] = 0.0f;
  if (s.bias) Layout<L, V, false>::load(s.bias, 0, a.E, true, lane, bias);  // NaN and -inf: no candidate
  __syncthreads();
  for (int64_t tb = t0 + __builtin_amdgcn_readfirstlane(threadIdx.x / kWave) * (kWave / L); tb < t1; tb += kTokens) {
    const int64_t t = tb + (threadIdx.x & (kWave - 1)) / L;
    const bool in = t < t1;
    float x[V], top = kNegInf, Z = 0.0f;
    double c[V];
    Lay::load(a.logits, t, a.E, in && unmasked(a.mask, t), lane, x);
    if (s.by_logit) {
#pragma unroll
      for (int v = 0; v < V; ++v) c[v] = (double)x[v];
    } else {
      if (!s.sigmoid) {
#pragma unroll
        for (int v = 0; v < V; ++v) top = fmaxf(top, x[v]);
        top = group_max<L>(top);
      }
      double sum = 0.0;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const double d = s.sigmoid ? -fmax((double)x[v], -700.0) : fmax((double)x[v] - (double)top, -745.0);
        c[v] = exp64(fmax(d, -745.0));
        sum += x[v] > kNegInf ? c[v] : 0.0;
      }
      double rz = 0.0;
      if (!s.sigmoid) {
        sum = group_sum64<L>(sum);
        Z = (float)sum;
        rz = rcp64(sum);
      }
#pragma unroll
      for (int v = 0; v < V; ++v) {
        c[v] = (s.sigmoid ? rcp64(1.0 + c[v]) : c[v] * rz) + (double)bias[v];
        if (!(x[v] > kNegInf && bias[v] > kNegInf)) c[v] = kNoKey;
      }
    }
    if constexpr (GROUPS) {
      double* row = score_of[threadIdx.x / L];
      double* group = group_of[threadIdx.x / L];
#pragma unroll
      for (int v = 0; v < V; ++v) row[Lay::expert(lane, v)] = c[v];
      wave_sync();
      for (int g = lane; g < s.groups; g += L) {
        double b1 = kNoKey, b2 = kNoKey;
        int at = lane < s.size ? lane : 0;  // lanes begin at different places of their groups: fewer bank conflicts
        for (int i = 0; i < s.size; ++i) {
          const double v = row[g * s.size + at];
          at = at + 1 < s.size ? at + 1 : 0;
          b2 = fmax(b2, fmin(b1, v));
          b1 = fmax(b1, v);
        }
        group[g] = s.best == 2 && b2 > kNoKey ? b1 + b2 : b1;
      }
      wave_sync();
      uint32_t low = 0, high = 0;
      for (int g = lane; g < s.groups; g += L) {
        const double mine = group[g];
        int before = 0;
        for (int h = 0; h < s.groups; ++h) {
          const double o = group[h];
          before += o > mine || (o == mine && h < g) ? 1 : 0;
        }
        const bool kept = before < s.top;
        low |= kept && g < 32 ? 1u << g : 0u;
        high |= kept && g >= 32 ? 1u << (g - 32) : 0u;
      }
      low = (uint32_t)group_reduce<L>((int)low, [](int p, int q) { return p | q; });
      high = (uint32_t)group_reduce<L>((int)high, [](int p, int q) { return p | q; });
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const uint32_t g = (uint32_t)Lay::expert(lane, v) * s.per_group >> 20;
        if (!((g < 32 ? low >> g : high >> (g - 32)) & 1u)) c[v] = kNoKey;
      }
      wave_sync();  // the row is read before the next token's scores are written
    }
    double best[N];
#pragma unroll
    for (int q = 0; q < V; q += N) {
      double d[N];
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const double key = score_key(c[q + i], Lay::expert(lane, q + i));
        d[i] = c[q + i] > kNoKey ? key : kNoKey;
      }
      sort_list<0, N>(d);
      if (q == 0) {
#pragma unroll
        for (int i = 0; i < N; ++i) best[i] = d[i];
      } else {
        merge_lists<N>(best, d);
      }
    }
    merge_lanes<N, L>(best);
    // the weights, from the logits of the chosen experts. Sigmoid scores exp(min(x, 0)) / (1 + exp(-|x|)), renormalised
    // ones relative to the largest exp(min(x, 0)), so that their sum is not 0
    int e[S];
    float xk[S], p[S], ref = kNegInf, sum = 0.0f;
#pragma unroll
    for (int q = 0; q < S; ++q) {
      const int k = lane + q * L;
      double d = kNoKey;
#pragma unroll
      for (int i = q * L; i < N && i < (q + 1) * L; ++i) d = i == k ? best[i] : d;
      e[q] = k < a.K ? key_expert(d) : -1;
      xk[q] = e[q] >= 0 ? clean(Lay::load_one(a.logits, t * a.E + e[q])) : kNegInf;
      ref = fmaxf(ref, s.sigmoid ? fminf(xk[q], 0.0f) : xk[q]);
    }
    ref = a.renorm ? group_max<L>(ref) : s.sigmoid ? 0.0f : top;
#pragma unroll
    for (int q = 0; q < S; ++q) {
      const float up = exp_below<true>((s.sigmoid ? fminf(xk[q], 0.0f) : xk[q]) - ref);
      const float under = s.sigmoid ? 1.0f + exp_below(-fabsf(xk[q])) : 1.0f;
      p[q] = e[q] >= 0 ? up / under : 0.0f;
      sum += p[q];
    }
    if (a.renorm) Z = group_sum<L>(sum);
    else if (s.sigmoid) Z = 1.0f;
#pragma unroll
    for (int q = 0; q < S; ++q) {
      const int k = lane + q * L;
      if (in && k < a.K) blk.put(a, t, k, e[q], e[q] >= 0 ? a.scale * (p[q] / Z) : 0.0f);
    }
  }
  blk.finish(a);
}

// One block: the counts' sum, then each expert's step up or down, compared as whole numbers.
__global__ __launch_bounds__(1024) void bias_update_kernel(int E, const int32_t* __restrict__ counts, float rate,
                                                           const float* bias, float* out) {
  __shared__ int64_t part[1024 / kWave];
  const int e = threadIdx.x, lane = e & (kWave - 1);
  const int64_t n = e < E ? counts[e] : 0;
  int64_t sum = n;
#pragma unroll
  for (int o = 1; o < kWave; o <<= 1) sum += __shfl_xor(sum, o, kWave);
  if (lane == 0) part[e / kWave] = sum;
  __syncthreads();
  sum = 0;
#pragma unroll
  for (int q = 0; q < 1024 / kWave; ++q) sum += part[q];
  if (e < E) out[e] = bias[e] + (sum > E * n ? rate : sum < E * n ? -rate : 0.0f);
}

// Layouts with groups: sixteen lanes or more to a token, so that its row of LDS is one of few.
template <bool BF16, class F>
void by_group_lists(int E, int K, F&& f) {
  using std::integral_constant;
  if (K <= 8) {
    integral_constant<int, 8> n;
    if (E <= 128) f(Layout<16, 8, BF16>(), n);
    else if (E <= 256) f(Layout<16, 16, BF16>(), n);
    else if (E <= 384) f(Layout<16, 24, BF16>(), n);
    else if (E <= 512) f(Layout<16, 32, BF16>(), n);
    else f(Layout<32, 32, BF16>(), n);
  } else if (K <= 16) {
    integral_constant<int, 16> n;
    if (E <= 256) f(Layout<16, 16, BF16>(), n);
    else if (E <= 512) f(Layout<16, 32, BF16>(), n);
    else f(Layout<32, 32, BF16>(), n);
  } else {
    integral_constant<int, 32> n;
    if (E <= 512) f(Layout<16, 32, BF16>(), n);
    else f(Layout<32, 32, BF16>(), n);
  }
}

template <bool BF16>
void run_scored(const RouteArgs& a, const ScoreArgs& s, size_t lds, hipStream_t st) {
  if (s.groups > 1) {
    by_group_lists<BF16>(a.E, a.K, [&](auto lay, auto n) {
      using Lay = decltype(lay);
      route_scored_kernel<Lay, decltype(n)::value, true>
          <<<a.rows, scored_threads(true, Lay::L, Lay::V), lds, st>>>(a, s);
    });
  } else {
    by_lists<BF16>(a.T, a.E, a.K, [&](auto lay, auto n) {
      using Lay = decltype(lay);
      route_scored_kernel<Lay, decltype(n)::value, false>
          <<<a.rows, scored_threads(false, Lay::L, Lay::V), lds, st>>>(a, s);
    });
  }
}

}  // namespace

int max_groups() { return kMaxGroups; }

lrmoe_status launch_scored_topk(const lrmoe_router* r, const lrmoe_scoring* c, const RouteArgs& a, const float* bias,
                                size_t lds, hipStream_t s) {
  const int size = r->E / c->groups;
  // a larger score is a larger logit where nothing else enters the choice
  const int groups = c->groups > c->top_groups ? c->groups : 1;  // where all are kept there are none
  const int by_logit = c->score == LRMOE_SCORE_SIGMOID && !bias && groups == 1;
  const ScoreArgs sc{bias, c->score == LRMOE_SCORE_SIGMOID, groups, size, c->top_groups, c->group_best, by_logit,
                     (uint32_t)(((1 << 20) + size - 1) / size)};
  r->dtype == LRMOE_BF16 ? run_scored<true>(a, sc, lds, s) : run_scored<false>(a, sc, lds, s);
  return launch_status();
}

lrmoe_status launch_bias_update(int32_t E, const int32_t* counts, float rate, const float* bias, float* out,
                                hipStream_t s) {
  bias_update_kernel<<<1, 1024, 0, s>>>(E, counts, rate, bias, out);
  return launch_status();
}

}  // namespace lrmoe
