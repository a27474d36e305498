// Activation checkpoints in 8 bits and the backward's reads of them: rows to codes and back, the LRM score with phi
// from codes, and the weighted rows of the retained pairs.
//
// All are one pass over memory: a code and a scale's part (1.016 bytes a value) beside the 2 or 4 bytes of the rows.
#include "checkpoint_device.h"

namespace lrmoe {
namespace {

constexpr int kThreads = 256;
constexpr int kUnits = 4;                                    // groups of a lane in flight
constexpr int kPerBlock = kThreads / kGroupLanes * kUnits;   // groups of a block

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
    const uint2 c = group_codes(x[u], &s);
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
      *(uint4*)((uint16_t*)rows + i[u]) =
          make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
    } else {
      ((float4*)((float*)rows + i[u]))[0] = make_float4(v[0], v[1], v[2], v[3]);
      ((float4*)((float*)rows + i[u]))[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
  }
}

// Sixteen lanes to a pair, four groups of its row in flight. Squares and sums in fp64.
template <bool SWIGLU>
__global__ __launch_bounds__(kThreads) void pair_score_codes_kernel(const int8_t* __restrict__ q,
                                                                    const uint16_t* __restrict__ scale,
                                                                    const float* __restrict__ alpha,
                                                                    const int32_t* __restrict__ tok,
                                                                    const double* __restrict__ gn, int64_t N, int T, int F,
                                                                    float* __restrict__ R) {
  const int lane = threadIdx.x & (kGroupLanes - 1), groups = scale_groups(F), chunks = F / 8;
  const int64_t j = (int64_t)blockIdx.x * (kThreads / kGroupLanes) + threadIdx.x / kGroupLanes;
  double acc = 0.0;
  if (j < N) {
    for (int c0 = lane; c0 < chunks; c0 += kGroupLanes * kUnits) {
      PhiChunk<SWIGLU> p[kUnits];
#pragma unroll
      for (int u = 0; u < kUnits; ++u) {
        const int c = c0 + u * kGroupLanes;
        if (c < chunks) p[u].load(q, scale, j, F, groups, c);
        else p[u].zero();
      }
#pragma unroll
      for (int u = 0; u < kUnits; ++u) {
        float v[8];
        p[u].phi(v);
#pragma unroll
        for (int k = 0; k < 8; ++k) acc = __builtin_fma((double)v[k], (double)v[k], acc);
      }
    }
  }
#pragma unroll
  for (int o = kGroupLanes / 2; o > 0; o >>= 1) acc += __shfl_xor(acc, o, kGroupLanes);
  if (lane == 0 && j < N) {
    const int t = tok[j];
    const double g = (t >= 0 && t < T) ? gn[t] : 0.0;  // out-of-range tokens score 0
    const double a = (double)alpha[j];
    R[j] = (float)(a * a * g * acc);
  }
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

Place place(int64_t n, int32_t parts, int32_t width) {
  const int groups = scale_groups(width);
  return Place{(uint32_t)(n * parts * groups), width, groups, 1.0 / groups, width % kGroupCols == 0};
}

}  // namespace

int64_t checkpoint_units(int64_t n, int32_t parts, int32_t width) { return n * parts * scale_groups(width); }

lrmoe_status launch_checkpoint(int64_t n, int32_t parts, int32_t width, int dtype, const void* rows, int8_t* q,
                               uint16_t* scale, hipStream_t s) {
  const Place p = place(n, parts, width);
  const unsigned g = (unsigned)ceil_div(p.units, kPerBlock);
  if (dtype == LRMOE_BF16) checkpoint_kernel<true><<<g, kThreads, 0, s>>>(p, rows, q, scale);
  else checkpoint_kernel<false><<<g, kThreads, 0, s>>>(p, rows, q, scale);
  return launch_status();
}

lrmoe_status launch_restore(int64_t n, int32_t parts, int32_t width, const int8_t* q, const uint16_t* scale, int dtype,
                            void* rows, hipStream_t s) {
  const Place p = place(n, parts, width);
  const unsigned g = (unsigned)ceil_div(p.units, kPerBlock);
  if (dtype == LRMOE_BF16) restore_kernel<true><<<g, kThreads, 0, s>>>(p, q, scale, rows);
  else restore_kernel<false><<<g, kThreads, 0, s>>>(p, q, scale, rows);
  return launch_status();
}

lrmoe_status launch_score_checkpoint(const lrmoe_problem* p, const void* G, const int8_t* q, const uint16_t* scale,
                                     const float* alpha, const int32_t* tok, float* R, double* gn, hipStream_t s) {
  launch_token_sqnorm(p, G, gn, s);
  if (p->N > 0) {
    const unsigned g = (unsigned)ceil_div(p->N, kThreads / kGroupLanes);
    if (p->swiglu) pair_score_codes_kernel<true><<<g, kThreads, 0, s>>>(q, scale, alpha, tok, gn, p->N, p->T, p->F, R);
    else pair_score_codes_kernel<false><<<g, kThreads, 0, s>>>(q, scale, alpha, tok, gn, p->N, p->T, p->F, R);
  }
  return launch_status();
}

lrmoe_status launch_compact_checkpoint(const lrmoe_problem* p, int64_t rows, const int32_t* sel, const int8_t* q,
                                       const uint16_t* scale, const float* alpha, void* PhiW, hipStream_t s) {
  if (rows <= 0) return LRMOE_OK;
  const unsigned g = (unsigned)ceil_div(rows, kThreads / kGroupLanes);
  auto run = [&](auto kernel) { kernel<<<g, kThreads, 0, s>>>(rows, p->N, p->F, sel, q, scale, alpha, PhiW); };
  if (p->dtype == LRMOE_BF16) p->swiglu ? run(compact_codes_kernel<true, true>) : run(compact_codes_kernel<false, true>);
  else p->swiglu ? run(compact_codes_kernel<true, false>) : run(compact_codes_kernel<false, false>);
  return launch_status();
}

}  // namespace lrmoe
