// Top-K routing by scores: softmax or sigmoid scores, a bias per expert that enters the choice but not the weights,
// and groups of experts of which the best are kept. The pair lists behind it are route's. And the bias update.
//
// The choice compares scores that may be as near as rounding lets them be, and experts are whole numbers, so scores are
// computed in f64: exp by its series, one reciprocal, some 27 instructions a logit, which run at the rate of f32 without
// packed instructions. (f32 scores first, and f64 ones only where two are nearer than their error, took as long: of 32768
// tokens a dozen always need them, and the wavefronts that have those hold the launch up by 2 us.)
#include "router_device.h"

namespace lrmoe {
namespace {

constexpr int kMaxGroups = 64;  // their marks are the bits of a word

struct ScoreArgs {
  const float* bias;  // [E] or NULL: experts are chosen by their logits, whose order is that of the scores
  int sigmoid, groups, size, top, best;
  int log_share;  // 2^log_share lanes look for a group's best, at most 4
  uint32_t per_group;  // ceil(2^20 / size): e * per_group >> 20 is e / size for all e below 1024
};

// exp(y) for y in [-745, 700] to a relative 1e-14 (the key that a score goes into keeps 42 bits, 2e-13): y = n ln 2 + r
// with |r| <= ln 2 / 2, the Taylor series of exp(r) to r^11, whose next term is below 7e-15.
__device__ __forceinline__ double exp64(double y) {
  const double n = __builtin_rint(y * 1.4426950408889634074);
  double r = __builtin_fma(n, -0x1.62e42fefap-1, y);  // 37 bits of ln 2: the product is exact
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

// 1 / d for d in [2^-1000, 2^1015], to 2^-46: the instruction's result has over 23 bits, the step doubles them.
__device__ __forceinline__ double rcp64(double d) {
  const double r = __builtin_amdgcn_rcp(d);
  return __builtin_fma(r, __builtin_fma(-d, r, 1.0), r);
}

// The score of what is no candidate: below every sum of a score and a bias, and finite with any lowest bits.
constexpr double kNoScore = -1e300;

// A choice score and its expert as one f64: the lowest 10 of the score's 52 bits give way to the expert, so that among
// scores that agree in the other 42 the lower index is the larger key. c is not -0.
__device__ __forceinline__ double score_key(double c, int e) {
  const int lo = __double2loint(c), hi = __double2hiint(c);
  return __hiloint2double(hi, (lo & ~1023) | ((e ^ 1023) ^ ((hi >> 31) & 1023)));
}
__device__ __forceinline__ int key_expert(double k) {  // -1 for no expert
  const int lo = __double2loint(k), hi = __double2hiint(k);
  return k < 0.5 * kNoScore ? -1 : (lo ^ 1023 ^ (hi >> 31)) & 1023;
}

template <int L, int S = 1>
__device__ __forceinline__ double group_sum64(double v) {
  if constexpr (S < L) return group_sum64<L, 2 * S>(v + key_swap<S>(v));
  else return v;
}

// The two largest of a run of scores, and of this lane's pair and that of the lane S apart.
__device__ __forceinline__ void add_best(double& b1, double& b2, double v) {
  b2 = fmax(b2, fmin(b1, v));
  b1 = fmax(b1, v);
}
template <int S>
__device__ __forceinline__ void join_best(double& b1, double& b2) {
  const double o1 = key_swap<S>(b1), o2 = key_swap<S>(b2);
  add_best(b1, b2, o1);
  b2 = fmax(b2, o2);
}

// Marks of the groups that a token keeps. A group's scores lie in the token's row of LDS, just written, one place apart
// from the next one's, so that lanes at the same step of their groups read different banks; the place between takes the
// group's score. 2^log_share lanes share a group.
template <int L>
__device__ __forceinline__ uint64_t kept_groups(const ScoreArgs& s, int lane, double* row) {
  wave_sync();
  const int share = 1 << s.log_share, part = lane & (share - 1), pitch = s.size + 1;
  for (int g = lane >> s.log_share; g < s.groups; g += L >> s.log_share) {
    const double* at = row + g * pitch;
    double b1 = kNoScore, b2 = kNoScore;
#pragma unroll 4
    for (int i = part; i < s.size; i += share) add_best(b1, b2, at[i]);
    if (share >= 2) join_best<1>(b1, b2);
    if (share >= 4) join_best<2>(b1, b2);
    if (part == 0) row[g * pitch + s.size] = s.best == 2 && b2 > kNoScore ? b1 + b2 : b1;
  }
  wave_sync();
  uint32_t low = 0, high = 0;
  for (int g = lane; g < s.groups; g += L) {
    const double mine = row[g * pitch + s.size];
    int before = 0;
#pragma unroll 4
    for (int h = 0; h < s.groups; ++h) {
      const double o = row[h * pitch + s.size];
      before += o > mine || (o == mine && h < g) ? 1 : 0;
    }
    const bool kept = before < s.top;
    low |= kept && g < 32 ? 1u << g : 0u;
    high |= kept && g >= 32 ? 1u << (g - 32) : 0u;
  }
  low = (uint32_t)group_reduce<L>((int)low, [](int p, int q) { return p | q; });
  if (s.groups > 32) high = (uint32_t)group_reduce<L>((int)high, [](int p, int q) { return p | q; });
  wave_sync();  // the row is read before the next token's scores are written
  return (uint64_t)high << 32 | low;
}

// g may be the number of groups, of which what is behind the last expert is: its scores are none whatever this gives.
__device__ __forceinline__ bool is_kept(uint64_t marks, uint32_t g) { return (marks >> (g & 63u) & 1u) != 0; }

// Threads of a block: 1024 where they have the registers, which is up to sixteen values to a lane (the layouts with 128
// experts and more; 32768 tokens of 128 experts with eight lanes each: 24.9 us with 512, 24.5 us with 1024; of 256: 38.3
// and 34.4 us; 131072 of 128: 73 and 63 us, all with the masks kept, see below). With groups their rows of LDS do not fit so many tokens.
constexpr int scored_threads(bool groups, int L, int V) {
  return !groups && V <= 16 && L >= 8 && L * V >= 128 ? 1024 : groups && V > 24 ? 256 : 512;
}

// As route_topk_kernel, with keys of choice scores instead of logits.
template <class Lay, int N, bool GROUPS>
__global__ __launch_bounds__(scored_threads(GROUPS, Lay::L, Lay::V)) void route_scored_kernel(RouteArgs a, ScoreArgs s) {
  constexpr int L = Lay::L, V = Lay::V, NT = scored_threads(GROUPS, L, V), kTokens = NT / L;
  constexpr int S = (N + L - 1) / L;  // slots of a lane: k = lane, lane + L, ...
  static_assert(V % N == 0, "whole lists");
  extern __shared__ uint32_t lds[];
  __shared__ double rows[GROUPS ? kTokens : 1][GROUPS ? L * V + kMaxGroups + 1 : 1];
  RouteBlock<NT> blk(a, lds);
  int lane = threadIdx.x & (L - 1);
  const int64_t t0 = (int64_t)blockIdx.x * a.C, t1 = min(t0 + a.C, (int64_t)a.T);
  uint32_t of[V];  // the group of each of the lane's experts; behind the last expert the number of groups
  if (GROUPS)
#pragma unroll
    for (int v = 0; v < V; ++v) of[v] = min((uint32_t)Lay::expert(lane, v) * s.per_group >> 20, (uint32_t)s.groups);
  __syncthreads();
  for (int64_t tb = t0 + __builtin_amdgcn_readfirstlane(threadIdx.x / kWave) * (kWave / L); tb < t1; tb += kTokens) {
    const int64_t t = tb + (threadIdx.x & (kWave - 1)) / L;
    const bool in = t < t1;
    int E = a.E;
    // What only the lane and E decide (the masks of the experts below E, keys' places) is computed where it is used: kept
    // over the loop it takes up to 160 scalar registers that there are not (32768 tokens of 128 experts: 24.9 us, 23.4 so).
    asm volatile("" : "+v"(lane));
    asm volatile("" : "+s"(E));
    double* row = rows[GROUPS ? threadIdx.x / L : 0];
    float x[V], bias[V], top = kNegInf, Z = 0.0f;
    Lay::load(a.logits, t, E, in && unmasked(a.mask, t), lane, x);
    if (s.bias) {  // an expert whose logit or bias is -inf (or NaN) has the bias -inf from here on
      asm volatile("" : "+s"(E));
      Layout<L, V, false>::load(s.bias, 0, E, true, lane, bias);
#pragma unroll
      for (int v = 0; v < V; ++v) bias[v] = x[v] > kNegInf ? bias[v] : kNegInf;
    }
    double c[V];
    if (s.bias || GROUPS) {
      if (s.sigmoid) {
#pragma unroll
        for (int v = 0; v < V; ++v) c[v] = rcp64(1.0 + exp64((double)fminf(fmaxf(-x[v], -745.0f), 700.0f)));
      } else {
#pragma unroll
        for (int v = 0; v < V; ++v) top = fmaxf(top, x[v]);
        top = group_max<L>(top);
        double sum = 0.0;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          c[v] = exp64(fmax((double)x[v] - (double)top, -745.0));
          sum += x[v] > kNegInf ? c[v] : 0.0;
        }
        sum = group_sum64<L>(sum);
        Z = (float)sum;
        const double rz = rcp64(sum);
#pragma unroll
        for (int v = 0; v < V; ++v) c[v] *= rz;
      }
#pragma unroll
      for (int v = 0; v < V; ++v)
        c[v] = fmax(c[v] + (double)(s.bias ? bias[v] : x[v] > kNegInf ? 0.0f : kNegInf), kNoScore);
    }
    uint64_t marks = 0;
    if constexpr (GROUPS) {
#pragma unroll
      for (int v = 0; v < V; ++v) row[Lay::expert(lane, v) + of[v]] = c[v];
      marks = kept_groups<L>(s, lane, row);
    }
    if (!s.bias)
#pragma unroll
      for (int v = 0; v < V; ++v) c[v] = fmax((double)(x[v] + 0.0f), kNoScore);
    double best[N];
#pragma unroll
    for (int q = 0; q < V; q += N) {
      double d[N];
#pragma unroll
      for (int i = 0; i < N; ++i) {
        if (GROUPS) c[q + i] = is_kept(marks, of[q + i]) ? c[q + i] : kNoScore;
        d[i] = score_key(c[q + i], Lay::expert(lane, q + i));
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
    int e[S];
#pragma unroll
    for (int q = 0; q < S; ++q) {
      const int k = lane + q * L;
      double d = kNoScore;
#pragma unroll
      for (int i = q * L; i < N && i < (q + 1) * L; ++i) d = i == k ? best[i] : d;
      e[q] = k < a.K ? key_expert(d) : -1;
    }
    // the weights, from the logits of the chosen experts. Sigmoid scores exp(min(x, 0)) / (1 + exp(-|x|)), renormalised
    // ones relative to the largest exp(min(x, 0)), so that their sum is not 0
    float xk[S], p[S], ref = kNegInf, sum = 0.0f;
#pragma unroll
    for (int q = 0; q < S; ++q) {
      xk[q] = e[q] >= 0 ? clean(Lay::load_one(a.logits, t * E + e[q])) : kNegInf;
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
  const float b = e < E ? bias[e] : 0.0f;  // all are read before any is written: out may share elements with bias
  int64_t sum = n;
#pragma unroll
  for (int o = 1; o < kWave; o <<= 1) sum += __shfl_xor(sum, o, kWave);
  if (lane == 0) part[e / kWave] = sum;
  __syncthreads();
  sum = 0;
#pragma unroll
  for (int q = 0; q < 1024 / kWave; ++q) sum += part[q];
  if (e < E) out[e] = b + (sum > E * n ? rate : sum < E * n ? -rate : 0.0f);
}

// Layouts with groups, whose rows of LDS leave room for a block of eight wavefronts. Eight lanes to a token up to 192
// experts (32768 tokens of 64 experts in 8 groups: 31.8 us with sixteen, 23.2 us with eight; of 128: 33.9 and 30.4 us;
// 20011 of 160: 31.5 and 29.9 us; but of 256: 47.6 and 60.0 us), more lanes above 384 for fewer registers (16384 of 512 in
// 16 groups: 60.3 us with sixteen, 52.7 us with 32; 8192 of 1000: 116 us with 32, 100 us with 64).
template <bool BF16, class F>
void by_group_lists(int E, int K, F&& f) {
  using std::integral_constant;
  if (K <= 8) {
    integral_constant<int, 8> n;
    if (E <= 64) f(Layout<8, 8, BF16>(), n);
    else if (E <= 128) f(Layout<8, 16, BF16>(), n);
    else if (E <= 192) f(Layout<8, 24, BF16>(), n);
    else if (E <= 256) f(Layout<16, 16, BF16>(), n);
    else if (E <= 384) f(Layout<16, 24, BF16>(), n);
    else if (E <= 512) f(Layout<32, 16, BF16>(), n);
    else f(Layout<64, 16, BF16>(), n);
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

// Layouts without groups: those of route, but up to 8 slots sixteen values to a lane where that fits the experts, whose
// f64 scores leave registers for blocks of 1024 (32768 tokens of 128 experts: 24.6 us with four lanes of 32 values, 23.4 us
// with eight of sixteen; 512 tokens 13.5 and 12.6 us; 131072 63.2 and 60.6 us; 32768 of 256: 34.2 and 32.8 us; 16384 of 500:
// 34.8 and 33.9 us; 8192 of 1000: 56.8 and 53.9 us; but of 192 28.4 us with eight lanes of 24 and 31.3 us with sixteen of
// sixteen, of 300 41.6 us with eight of forty and 46.7 us with sixteen of 24, and with 16 slots of 128 27.4 us with
// four lanes and 37.0 us with sixteen).
template <bool BF16, class F>
void by_score_lists(int T, int E, int K, F&& f) {
  std::integral_constant<int, 8> n;
  if (K > 8 || T <= kFewTokens) by_lists<BF16>(T, E, K, f);
  else if (E > 64 && E <= 128) f(Layout<8, 16, BF16>(), n);
  else if (E > 192 && E <= 256) f(Layout<16, 16, BF16>(), n);
  else if (E > 320 && E <= 512) f(Layout<32, 16, BF16>(), n);
  else if (E > 512) f(Layout<64, 16, BF16>(), n);
  else by_lists<BF16>(T, E, K, f);
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
    by_score_lists<BF16>(a.T, a.E, a.K, [&](auto lay, auto n) {
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
  const int groups = c->groups > c->top_groups ? c->groups : 1;  // where all are kept there are none
  const int log_share = groups <= 4 ? 2 : groups <= 8 ? 1 : 0;   // eight lanes at least
  const bool sigmoid = c->score == LRMOE_SCORE_SIGMOID;
  const ScoreArgs sc{bias, sigmoid, groups, size, c->top_groups, c->group_best, log_share,
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
