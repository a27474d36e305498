// Activation checkpoints in 8 bits and the backward's reads of them: rows to codes and back, the LRM score with phi
// from codes, and the weighted rows of the retained pairs.
//
// All are one pass over memory: a code and a scale's part (1.016 bytes a value) beside the 2 or 4 bytes of the rows.
#include <algorithm>
#include <type_traits>

#include "checkpoint_device.h"
#include "score_device.h"

namespace lrmoe {
namespace {

constexpr int kThreads = 256;
// Groups of a lane in flight. 262144 rows of 2 x 768 bf16 saved and restored / their pairs scored (squares in f32) / 60 % of
// them compacted: 393 / 100 / 77 us with one, 360 / 100 / 78 with two, 378 / 119 / 79 with four, 430 / 128 / 83 with eight
// (the restored rows written past the caches, without which four take 414 us; codes written so as well: 381 instead of 360).
constexpr int kUnits = 2;
constexpr int kPerBlock = kThreads / kGroupLanes * kUnits;   // groups of a block

// Words of 16 bytes of gradient rows, read once a pair, up to which scoring takes one launch (8 pairs to a token, rows of
// 2048 bf16: 512 tokens 8.5 us with one launch and 10.7 with two, 1024 tokens 10.9 and 10.8, 2048 tokens 16.7 and 13.6).
constexpr int64_t kFewWords = 1 << 21;

// Where the eight columns of this lane's group `unit` are: rows of `width` in groups of 128, the last one short.
struct Place {
  uint32_t units;
  int width, groups;
  double inv;  // 1 / groups
  bool whole;  // width is whole groups
  __device__ __forceinline__ bool at(uint32_t unit, int lane, int64_t* i) const {
    if (unit >= units) return false;
    if (whole) {
      *i = (int64_t)unit * kGroupCols + lane * 8;
      return true;
    }
    const uint32_t row = (uint32_t)(((double)unit + 0.5) * inv);  // unit / groups: the product is off by far less than 0.5 inv
    const int col = (int)(unit - row * (uint32_t)groups) * kGroupCols + lane * 8;
    *i = (int64_t)row * width + col;
    return col < width;
  }
};

template <bool BF16>
__device__ __forceinline__ void load_rows8(const void* __restrict__ rows, int64_t i, float x[8]) {
  if (BF16) {
    const uint4 v = ld_stream((const uint16_t*)rows + i);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) x[2 * k] = bf16_lo(w[k]), x[2 * k + 1] = bf16_hi(w[k]);
  } else {
    const uint4 a = ld_stream((const float*)rows + i), b = ld_stream((const float*)rows + i + 4);
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] = __uint_as_float(w[k]);
  }
}

template <bool BF16>
__global__ __launch_bounds__(kThreads) void checkpoint_kernel(Place p, const void* __restrict__ rows,
                                                              int8_t* __restrict__ q, uint16_t* __restrict__ scale) {
  const int lane = threadIdx.x & (kGroupLanes - 1);
  const uint32_t u0 = blockIdx.x * (uint32_t)kPerBlock + threadIdx.x / kGroupLanes;
  float x[kUnits][8];
  int64_t i[kUnits];
  bool on[kUnits];
#pragma unroll
  for (int u = 0; u < kUnits; ++u) {
    on[u] = p.at(u0 + u * (kThreads / kGroupLanes), lane, &i[u]);
#pragma unroll
    for (int k = 0; k < 8; ++k) x[u][k] = 0.0f;
    if (on[u]) load_rows8<BF16>(rows, i[u], x[u]);
  }
#pragma unroll
  for (int u = 0; u < kUnits; ++u) {
    const uint32_t unit = u0 + u * (kThreads / kGroupLanes);
    uint16_t s;
    const uint2 c = group_codes<BF16>(x[u], &s);
    if (on[u]) *(uint2*)(q + i[u]) = c;
    if (lane == 0 && unit < p.units) scale[unit] = s;
  }
}

template <bool BF16>
__global__ __launch_bounds__(kThreads) void restore_kernel(Place p, const int8_t* __restrict__ q,
                                                           const uint16_t* __restrict__ scale, void* __restrict__ rows) {
  const int lane = threadIdx.x & (kGroupLanes - 1);
  const uint32_t u0 = blockIdx.x * (uint32_t)kPerBlock + threadIdx.x / kGroupLanes;
  uint2 c[kUnits];
  uint16_t s[kUnits];
  int64_t i[kUnits];
  bool on[kUnits];
#pragma unroll
  for (int u = 0; u < kUnits; ++u) {
    const uint32_t unit = u0 + u * (kThreads / kGroupLanes);
    on[u] = p.at(unit, lane, &i[u]);
    c[u] = make_uint2(0, 0);
    s[u] = 0;
    if (on[u]) {
      c[u] = ld_stream8(q + i[u]);
      s[u] = scale[unit];
    }
  }
#pragma unroll
  for (int u = 0; u < kUnits; ++u) {
    float v[8];
    values8(c[u], scale_of(s[u]), v);
    if (!on[u]) continue;
    if (BF16) {
      const u32x4_t w = {pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                         pack_bf16x2(v[6], v[7])};
      __builtin_nontemporal_store(w, (u32x4_t*)((uint16_t*)rows + i[u]));
    } else {
      typedef float f32x4_t __attribute__((ext_vector_type(4)));
      f32x4_t* o = (f32x4_t*)((float*)rows + i[u]);
      __builtin_nontemporal_store(f32x4_t{v[0], v[1], v[2], v[3]}, o);
      __builtin_nontemporal_store(f32x4_t{v[4], v[5], v[6], v[7]}, o + 1);
    }
  }
}

// Sum of squares of phi of pair j, by sixteen lanes, two groups of its row in flight; squares and sums in fp64.
template <bool SWIGLU>
__device__ __forceinline__ double pair_sqnorm(const int8_t* __restrict__ q, const uint16_t* __restrict__ scale, int64_t j,
                                              bool on, int F) {
  const int lane = threadIdx.x & (kGroupLanes - 1), groups = scale_groups(F), chunks = F / 8;
  double acc = 0.0;
  if (on) {
    for (int c0 = lane; c0 < chunks; c0 += kGroupLanes * kUnits) {
      PhiChunk<SWIGLU> p[kUnits];
#pragma unroll
      for (int u = 0; u < kUnits; ++u) {
        const int c = c0 + u * kGroupLanes;
        if (c < chunks) p[u].load(q, scale, j, F, groups, c);
        else p[u].zero();
      }
#pragma unroll
      for (int u = 0; u < kUnits; ++u) acc = __builtin_fma(p[u].sqnorm_of_codes(), p[u].scale_sq(), acc);
    }
  }
#pragma unroll
  for (int o = kGroupLanes / 2; o > 0; o >>= 1) acc += __shfl_xor(acc, o, kGroupLanes);
  return acc;
}

__device__ __forceinline__ float pair_score(float alpha, double gn, double pn) {
  const double a = (double)alpha;
  return (float)(a * a * gn * pn);
}

// OWN: each pair's lanes take the norm of its gradient row themselves (few pairs, one launch). Else gn has it.
template <bool SWIGLU, bool BF16, bool OWN>
__global__ __launch_bounds__(kThreads) void pair_score_codes_kernel(const uint4* __restrict__ G, int T, int words,
                                                                    const double* __restrict__ gn,
                                                                    const int8_t* __restrict__ q,
                                                                    const uint16_t* __restrict__ scale,
                                                                    const float* __restrict__ alpha,
                                                                    const int32_t* __restrict__ tok, int64_t N, int F,
                                                                    float* __restrict__ R) {
  const int lane = threadIdx.x & (kGroupLanes - 1);
  const int64_t j = (int64_t)blockIdx.x * (kThreads / kGroupLanes) + threadIdx.x / kGroupLanes;
  const int t = j < N ? tok[j] : -1;
  const bool there = t >= 0 && t < T;  // out-of-range tokens score 0
  double g = 0.0;
  if (there && !OWN) g = gn[t];
  if (OWN) {
    if (there) {
      const uint4* row = G + (int64_t)t * words;
#pragma unroll 4
      for (int c = lane; c < words; c += kGroupLanes) g += BF16 ? sumsq_bf16x8(row[c]) : sumsq_f32x4(row[c]);
    }
#pragma unroll
    for (int o = kGroupLanes / 2; o > 0; o >>= 1) g += __shfl_xor(g, o, kGroupLanes);
  }
  const double pn = pair_sqnorm<SWIGLU>(q, scale, j, j < N, F);
  if (lane == 0 && j < N) R[j] = pair_score(alpha[j], g, pn);
}

// Tokens and pairs in one launch, their blocks mixed evenly: the pairs are bound by arithmetic (two transcendental
// instructions a value), the tokens' rows by HBM. The 32768-token share (262144 pairs of 768): 98 us and 4.8 us of the join
// behind it, 100 to 104 us a call, 5.2 TB/s (98 us with squares in f32, which small ones leave), against 116 us with tokens
// and pairs one after the other (20.8 + 99 us); 65536 pairs 31.2 and 33.1 us, in f32 32.1 and 36.3; of 768 without gate and up
// 262144 55.8 and 67.0. The workspace has to have room for the pairs' norms: one that lrmoe_workspace_size gives has it where
// something else needs as much. Block b is the tokens' i-th if the count floor(b step / 2^32) passes i there.
template <bool SWIGLU, bool BF16>
__global__ __launch_bounds__(kThreads) void norms_kernel(uint64_t step, const uint4* __restrict__ G, int T, int words,
                                                         double* __restrict__ gn, const int8_t* __restrict__ q,
                                                         const uint16_t* __restrict__ scale, int64_t N, int F,
                                                         double* __restrict__ pn) {
  const uint64_t before = (blockIdx.x * step) >> 32;
  if (((blockIdx.x + 1ull) * step) >> 32 != before) {
    token_sqnorm<BF16, false>(G, T, words, (int64_t)before, gn);
    return;
  }
  const int64_t j = (int64_t)(blockIdx.x - before) * (kThreads / kGroupLanes) + threadIdx.x / kGroupLanes;
  const double n = pair_sqnorm<SWIGLU>(q, scale, j, j < N, F);
  if ((threadIdx.x & (kGroupLanes - 1)) == 0 && j < N) pn[j] = n;
}

__global__ __launch_bounds__(kThreads) void join_scores_kernel(const double* __restrict__ pn,
                                                               const float* __restrict__ alpha,
                                                               const int32_t* __restrict__ tok,
                                                               const double* __restrict__ gn, int64_t N, int T,
                                                               float* __restrict__ R) {
  const int64_t j = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (j >= N) return;
  const int t = tok[j];
  R[j] = pair_score(alpha[j], t >= 0 && t < T ? gn[t] : 0.0, pn[j]);  // out-of-range tokens score 0
}

// Sixteen lanes to a packed row.
template <bool SWIGLU, bool BF16>
__global__ __launch_bounds__(kThreads) void compact_codes_kernel(int64_t rows, int64_t N, int F,
                                                                 const int32_t* __restrict__ sel,
                                                                 const int8_t* __restrict__ q,
                                                                 const uint16_t* __restrict__ scale,
                                                                 const float* __restrict__ alpha, void* __restrict__ PhiW) {
  const int lane = threadIdx.x & (kGroupLanes - 1), groups = scale_groups(F), chunks = F / 8;
  const int64_t r = (int64_t)blockIdx.x * (kThreads / kGroupLanes) + threadIdx.x / kGroupLanes;
  if (r >= rows) return;
  const int64_t j = sel[r];
  const bool ok = j >= 0 && j < N;  // else a zero row
  const float a = ok ? alpha[j] : 0.0f;
  for (int c0 = lane; c0 < chunks; c0 += kGroupLanes * kUnits) {
    PhiChunk<SWIGLU> p[kUnits];
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      const int c = c0 + u * kGroupLanes;
      if (ok && c < chunks) p[u].load(q, scale, j, F, groups, c);
      else p[u].zero();
    }
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      const int c = c0 + u * kGroupLanes;
      float v[8];
      p[u].phi(v);
      if (c >= chunks) continue;
      if (BF16) {
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
          // phi of a SwiGLU is rounded to f32 already, so its product may be; a restored value's is exact
          w[k] = SWIGLU ? pack_bf16x2(a * v[2 * k], a * v[2 * k + 1])
                        : mul_to_bf16(a, v[2 * k]) | mul_to_bf16(a, v[2 * k + 1]) << 16;
        *(uint4*)((uint16_t*)PhiW + r * F + c * 8) = make_uint4(w[0], w[1], w[2], w[3]);
      } else {
        float4* o = (float4*)((float*)PhiW + r * F + c * 8);
        o[0] = make_float4(a * v[0], a * v[1], a * v[2], a * v[3]);
        o[1] = make_float4(a * v[4], a * v[5], a * v[6], a * v[7]);
      }
    }
  }
}

// A launch has fewer than 2^32 threads.
constexpr int64_t kMaxBlocks = ((int64_t)1 << 32) / kThreads;
constexpr int64_t kLaunchUnits = (kMaxBlocks - 1) * kPerBlock;  // groups of one launch

// Calls f for as many launches as n * parts rows of `width` need (one below 2^29 groups), each with its place, its blocks and
// the values and scales before it.
template <class F>
void by_launches(int64_t n, int32_t parts, int32_t width, F&& f) {
  const int groups = scale_groups(width);
  const int64_t rows = n * parts, step = kLaunchUnits / groups;
  for (int64_t r = 0; r < rows; r += step) {
    const int64_t units = std::min(step, rows - r) * groups;
    f(Place{(uint32_t)units, width, groups, 1.0 / groups, width % kGroupCols == 0}, (unsigned)ceil_div(units, kPerBlock),
      r * width, r * groups);
  }
}

}  // namespace

lrmoe_status launch_checkpoint(int64_t n, int32_t parts, int32_t width, int dtype, const void* rows, int8_t* q,
                               uint16_t* scale, hipStream_t s) {
  by_launches(n, parts, width, [&](const Place& p, unsigned g, int64_t v, int64_t u) {
    if (dtype == LRMOE_BF16) checkpoint_kernel<true><<<g, kThreads, 0, s>>>(p, (const uint16_t*)rows + v, q + v, scale + u);
    else checkpoint_kernel<false><<<g, kThreads, 0, s>>>(p, (const float*)rows + v, q + v, scale + u);
  });
  return launch_status();
}

lrmoe_status launch_restore(int64_t n, int32_t parts, int32_t width, const int8_t* q, const uint16_t* scale, int dtype,
                            void* rows, hipStream_t s) {
  by_launches(n, parts, width, [&](const Place& p, unsigned g, int64_t v, int64_t u) {
    if (dtype == LRMOE_BF16) restore_kernel<true><<<g, kThreads, 0, s>>>(p, q + v, scale + u, (uint16_t*)rows + v);
    else restore_kernel<false><<<g, kThreads, 0, s>>>(p, q + v, scale + u, (float*)rows + v);
  });
  return launch_status();
}

lrmoe_status launch_score_checkpoint(const lrmoe_problem* p, const void* G, const int8_t* q, const uint16_t* scale,
                                     const float* alpha, const int32_t* tok, float* R, void* ws, size_t ws_bytes,
                                     hipStream_t s) {
  double* gn = (double*)ws;
  const bool bf16 = p->dtype == LRMOE_BF16;
  const size_t tokens = align_up(sizeof(double) * (size_t)p->T, 256);
  const int words = p->D / (bf16 ? 8 : 4);
  const int64_t pairs = ceil_div(p->N, kThreads / kGroupLanes), rows = ceil_div(p->T, kThreads / kWave);
  if (p->N == 0) return LRMOE_OK;
  const bool few = p->N * words <= kFewWords;
  if (pairs >= kMaxBlocks || (!few && rows >= kMaxBlocks)) return LRMOE_ERR_UNSUPPORTED;
  // by_type(f): f with SWIGLU and BF16 as constants
  auto by_type = [&](auto f) {
    using std::bool_constant;
    if (bf16) p->swiglu ? f(bool_constant<true>(), bool_constant<true>()) : f(bool_constant<false>(), bool_constant<true>());
    else p->swiglu ? f(bool_constant<true>(), bool_constant<false>()) : f(bool_constant<false>(), bool_constant<false>());
  };
  if (!few && ws_bytes >= tokens + sizeof(double) * (size_t)p->N && pairs + rows < kMaxBlocks) {
    // both norms in one launch: the pairs' need a place until the tokens' are there
    double* pn = (double*)((char*)ws + tokens);
    const uint64_t all = (uint64_t)(pairs + rows), step = (((uint64_t)rows << 32) + all - 1) / all;
    by_type([&](auto sw, auto bf) {
      norms_kernel<decltype(sw)::value, decltype(bf)::value><<<(unsigned)all, kThreads, 0, s>>>(
          step, (const uint4*)G, p->T, words, gn, q, scale, p->N, p->F, pn);
    });
    join_scores_kernel<<<(unsigned)ceil_div(p->N, kThreads), kThreads, 0, s>>>(pn, alpha, tok, gn, p->N, p->T, R);
    return launch_status();
  }
  if (!few) launch_token_sqnorm(p, G, gn, s);
  by_type([&](auto sw, auto bf) {
    auto run = [&](auto kernel) {
      kernel<<<(unsigned)pairs, kThreads, 0, s>>>((const uint4*)G, p->T, words, gn, q, scale, alpha, tok, p->N, p->F, R);
    };
    constexpr bool kSw = decltype(sw)::value, kBf = decltype(bf)::value;
    few ? run(pair_score_codes_kernel<kSw, kBf, true>) : run(pair_score_codes_kernel<kSw, true, false>);
  });
  return launch_status();
}

lrmoe_status launch_compact_checkpoint(const lrmoe_problem* p, int64_t rows, const int32_t* sel, const int8_t* q,
                                       const uint16_t* scale, const float* alpha, void* PhiW, hipStream_t s) {
  if (rows <= 0) return LRMOE_OK;
  const int64_t g = ceil_div(rows, kThreads / kGroupLanes);
  if (g >= kMaxBlocks) return LRMOE_ERR_UNSUPPORTED;
  auto run = [&](auto kernel) { kernel<<<(unsigned)g, kThreads, 0, s>>>(rows, p->N, p->F, sel, q, scale, alpha, PhiW); };
  if (p->dtype == LRMOE_BF16) p->swiglu ? run(compact_codes_kernel<true, true>) : run(compact_codes_kernel<false, true>);
  else p->swiglu ? run(compact_codes_kernel<true, false>) : run(compact_codes_kernel<false, false>);
  return launch_status();
}

}  // namespace lrmoe
