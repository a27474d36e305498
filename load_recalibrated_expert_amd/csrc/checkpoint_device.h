// Activation rows in 8 bits: codes q int8 with one bf16 scale s for every 128 columns of a part of a row. A row has one
// part, or two of equal width (gate and up); a group of columns lies in one part. The values are q s.
//
// Sixteen lanes hold a group, eight columns each, so that a row's chunk c (eight columns) of lane c % 16 belongs to group
// c / 16: whoever steps through a row by sixteen chunks takes one scale a step.
#pragma once
#include "common.h"

namespace lrmoe {

constexpr int kGroupCols = 128, kGroupLanes = 16;

// unsigned: the sum may be past 2^31
__host__ __device__ constexpr int scale_groups(int width) { return (int)(((uint32_t)width + kGroupCols - 1) / kGroupCols); }

__device__ __forceinline__ uint2 ld_stream8(const void* p) {
  const unsigned long long v = __builtin_nontemporal_load((const unsigned long long*)p);
  return make_uint2((uint32_t)v, (uint32_t)(v >> 32));
}

__device__ __forceinline__ float scale_of(uint16_t bits) { return __uint_as_float((uint32_t)bits << 16); }

// Eight codes times their scale: exact, as 8 bits times 8 fit f32.
__device__ __forceinline__ void values8(uint2 q, float s, float v[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = (float)(int8_t)(q.x >> (8 * i)) * s;
    v[4 + i] = (float)(int8_t)(q.y >> (8 * i)) * s;
  }
}

// The scale of a group whose largest magnitude is amax (finite): the smallest bf16 number that is at least amax / 127 and
// a normal number. 127 times a bf16 number is exact in f32, so the comparison that rounds up is too: the product with the
// rounded 1 / 127 is off by less than 2^-22, so cut to bf16 it is at most two steps low and never too high.
__device__ __forceinline__ float scale_for(float amax) {
  float s = __uint_as_float(__float_as_uint(amax * (1.0f / 127.0f)) & 0xFFFF0000u);
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (127.0f * s < amax) s = __uint_as_float(__float_as_uint(s) + 0x10000u);
  return fmaxf(s, 0x1p-126f);
}

constexpr float kRound = 12582912.0f;  // 1.5 2^23: what is added to it is rounded to a whole number, ties to even

// The lowest bytes of eight whole numbers that kRound has been added to.
__device__ __forceinline__ uint2 pack_codes(const float t[8]) {
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t lo = __builtin_amdgcn_perm(__float_as_uint(t[4 * i + 1]), __float_as_uint(t[4 * i]), 0x0c0c0400u);
    const uint32_t hi = __builtin_amdgcn_perm(__float_as_uint(t[4 * i + 3]), __float_as_uint(t[4 * i + 2]), 0x04000c0cu);
    w[i] = lo | hi;
  }
  return make_uint2(w[0], w[1]);
}

// Codes of eight values of one group, whose sixteen lanes call this together: nearest whole numbers of scales, ties to
// even, exactly. u = x / s is rounded by adding 1.5 2^23, with the reciprocal to 1 ulp instead of the quotient, so next to
// a half the code may be the other neighbour. The remainder r = x - q s tells: it is exact (|r| <= |x| and both are whole
// multiples of the smaller of their last places), and under s / 2 in magnitude where q is right and no tie.
__device__ __forceinline__ uint2 codes8(const float x[8], float s, float inv) {
  const float half = 0.5f * s;
  float t[8], far = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    t[i] = __builtin_fmaf(x[i], inv, kRound);
    far = fmaxf(far, fabsf(__builtin_fmaf(kRound - t[i], s, x[i])));
  }
  if (far >= half) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float r = __builtin_fmaf(kRound - t[i], s, x[i]);
      const bool odd = (__float_as_uint(t[i]) & 1u) != 0;
      if (fabsf(r) > half || (fabsf(r) == half && odd)) t[i] += r > 0.0f ? 1.0f : -1.0f;
    }
  }
  return pack_codes(t);
}

// The same for values that are bf16 numbers, without the second look: the quotient of two 8-bit significands is a half
// exactly or at least 2^-10 away from one (2 x - (2 q + 1) s is a whole multiple of a last place of x or s, and x is at
// least s / 2 there), and the quotient as corrected by its remainder is exact where f32 holds it, as it does all halves.
// The remainder has places down to 2^-31 of s, so tiny scales are taken away from the subnormal numbers first.
__device__ __forceinline__ uint2 codes8_bf16(const float x[8], float s, float inv) {
  float t[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) t[i] = x[i];
  if (s < 0x1p-100f) {
    s *= 0x1p64f;
    inv *= 0x1p-64f;
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] *= 0x1p64f;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float u = t[i] * inv;
    t[i] = __builtin_fmaf(__builtin_fmaf(-u, s, t[i]), inv, u) + kRound;
  }
  return pack_codes(t);
}

// Largest bits of |x| over the group: of finite values the largest magnitude's, else at least infinity's.
__device__ __forceinline__ uint32_t group_amax_bits(const float x[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(x[i]) & 0x7FFFFFFFu);
  return (uint32_t)group_reduce<kGroupLanes>((int)m, [](int a, int b) { return max(a, b); });
}

// A group's codes and the bits of its scale, from the eight values of each of its lanes. BF16: they are bf16 numbers.
template <bool BF16>
__device__ __forceinline__ uint2 group_codes(const float x[8], uint16_t* scale) {
  const uint32_t m = group_amax_bits(x);
  const bool bad = m >= 0x7F800000u;  // infinities or NaN: all of the group counts as NaN
  const float s = scale_for(__uint_as_float(m)), inv = __builtin_amdgcn_rcpf(s);
  const uint2 c = BF16 ? codes8_bf16(x, s, inv) : codes8(x, s, inv);
  *scale = bad ? 0x7FC0 : (uint16_t)(__float_as_uint(s) >> 16);
  return bad ? make_uint2(0, 0) : c;
}

// Eight columns of phi, as an expert's FC2 read it: silu(gate) up from the restored values, or the restored value itself.
template <bool SWIGLU>
struct PhiChunk {
  uint2 a, b;       // codes: gate and up, or phi
  uint16_t sa, sb;  // their scales' bits
  // chunk c of row j, rows of PARTS x F
  __device__ __forceinline__ void load(const int8_t* __restrict__ q, const uint16_t* __restrict__ scale, int64_t j, int F,
                                       int groups, int c) {
    constexpr int kParts = SWIGLU ? 2 : 1;
    const int8_t* row = q + j * kParts * F + c * 8;
    const uint16_t* sc = scale + j * kParts * groups + c / kGroupLanes;
    a = ld_stream8(row);
    sa = sc[0];
    if (SWIGLU) {
      b = ld_stream8(row + F);
      sb = sc[groups];
    }
  }
  __device__ __forceinline__ void zero() { a = b = make_uint2(0, 0), sa = sb = 0; }
  __device__ __forceinline__ void phi(float v[8]) const {
    values8(a, scale_of(sa), v);
    if (!SWIGLU) return;
    float up[8];
    values8(b, scale_of(sb), up);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      // the hardware's base-2 exponential and reciprocal, 1 ulp each: x / (1 + 2^(-x log2 e))
      const float sg = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(v[i] * -1.44269504088896341f));
      v[i] = v[i] * sg * up[i];
    }
  }
  // Sum of squares of the chunk's phi over scale_sq(), in fp64: with a gate of -50 a term is 1e-18, and its square is
  // close to the subnormal f32 numbers.
  __device__ __forceinline__ double sqnorm_of_codes() const {
    const uint32_t qa[2] = {a.x, a.y}, qb[2] = {b.x, b.y};
    const float s = scale_of(sa);
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float g = (float)(int8_t)(qa[i >> 2] >> (8 * (i & 3)));
      float t = g;
      if (SWIGLU) {
        const float u = (float)(int8_t)(qb[i >> 2] >> (8 * (i & 3)));
        t = g * u * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(g * s * -1.44269504088896341f));
      }
      sum = __builtin_fma((double)t, (double)t, sum);
    }
    return sum;
  }
  __device__ __forceinline__ double scale_sq() const {
    const double f = SWIGLU ? (double)scale_of(sa) * (double)scale_of(sb) : (double)scale_of(sa);
    return f * f;
  }
};

}  // namespace lrmoe
