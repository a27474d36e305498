// AdamW over many tensors in one launch, first and second moments in 32 or in 8 bits.
//
// Elementwise over [n]: HBM-bound, every array read and written once. The tensors come in a table,
// cut into chunks of kChunk elements: in the launch's arguments, 48 to a launch, or all of them
// in device memory (a plan). A wavefront finds its chunk's tensor by comparing with 64 first chunks
// at a time.
#include <algorithm>

#include "common.h"

#pragma clang fp contract(off)  // a rounding at each operation, as the header says

namespace lrmoe {
namespace {

constexpr int kThreads = 256;
constexpr int kBlock = 256;   // elements that share a scale: four to a lane of one wavefront
constexpr uint32_t kLaunchChunks = (1u << 24) - 1;  // a launch has fewer than 2^32 threads
constexpr int kChunk = 4 * kThreads;  // elements of one thread block (four times as many: 3 % slower on
                                      // 75 M elements, 7.5 instead of 4.4 us on a small tensor)

// The tensors that have elements, and the first chunk of each.
struct ArgTable {
  lrmoe_adamw_tensor t[kAdamwTensors];
  uint32_t chunk[kAdamwTensors];
  int32_t n;
  __device__ __forceinline__ const lrmoe_adamw_tensor& tensor(int i) const { return t[i]; }
  __device__ __forceinline__ uint32_t first(int i) const { return chunk[i]; }
};
struct PlanTable {
  const lrmoe_adamw_tensor* t;
  const uint32_t* chunk;
  int32_t n;
  __device__ __forceinline__ const lrmoe_adamw_tensor& tensor(int i) const { return t[i]; }
  __device__ __forceinline__ uint32_t first(int i) const { return chunk[i]; }
};

struct AdamwArgs {
  float b1, a1, b2, a2, eps;  // beta, 1 - beta
  lrmoe_adamw_scalars s;
  const lrmoe_adamw_scalars* dyn;
  uint32_t chunk0;  // this launch's first chunk
};

__device__ __forceinline__ uint32_t mix(uint32_t x) {
  x ^= x >> 16;
  x *= 0x9E3779B1u;
  x ^= x >> 15;
  x *= 0x85EBCA77u;
  return x ^ (x >> 13);
}

__device__ __forceinline__ float pow2(int k) { return __uint_as_float((uint32_t)(k + 127) << 23); }

// |x| rounded to e4m3 at random by the 16 bits b: to a multiple of the spacing at x, 2^(e - 3)
// with e at least -6 (exponent field 121). The result is an e4m3 value, so its conversion is exact.
__device__ __forceinline__ float round_e4m3(float x, uint32_t b) {
  const uint32_t t = max(__float_as_uint(x) & 0x7F800000u, 121u << 23);
  const float down = __uint_as_float((257u << 23) - t), up = __uint_as_float(t - (3u << 23));
  return floorf(x * down + __builtin_fmaf((float)b, 0x1p-16f, 0x1p-17f)) * up;  // (b + 0.5) / 65536, exactly
}

// Exponent of a block's scale for its largest finite magnitude: the scaled maximum is in
// [156.8, 313.6), under e4m3's 448 also after rounding up.
__device__ __forceinline__ int scale_exp(float amax) {
  return max((int)(__float_as_uint(amax * 0.8164966f) >> 23) - 127 - 7, -126);
}

// Of magnitudes, whose bits order as whole numbers.
__device__ __forceinline__ float wave_max(float v) {
  return __int_as_float(group_reduce<kWave>(__float_as_int(v), [](int a, int b) { return max(a, b); }));
}

__device__ __forceinline__ bool finite(float x) { return !__builtin_amdgcn_classf(x, 0x207); }  // NaN, -inf, +inf

typedef float f32x4_t __attribute__((ext_vector_type(4)));

// Four elements at i, of which `left` are inside the tensor. NT: past the caches' retention policy.
template <bool BF16, bool NT>
__device__ __forceinline__ void load4(const void* __restrict__ p, int64_t i, int left, float v[4]) {
  if (left >= 4) {
    if (BF16) {
      const uint2 x = *(const uint2*)((const uint16_t*)p + i);
      v[0] = bf16_lo(x.x);
      v[1] = bf16_hi(x.x);
      v[2] = bf16_lo(x.y);
      v[3] = bf16_hi(x.y);
    } else {
      const f32x4_t* at = (const f32x4_t*)((const float*)p + i);
      const f32x4_t x = NT ? __builtin_nontemporal_load(at) : *at;
      v[0] = x[0];
      v[1] = x[1];
      v[2] = x[2];
      v[3] = x[3];
    }
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      v[q] = q >= left ? 0.0f
             : BF16    ? __uint_as_float((uint32_t)((const uint16_t*)p)[i + q] << 16)
                       : ((const float*)p)[i + q];
  }
}

template <bool BF16, bool NT>
__device__ __forceinline__ void store4(void* __restrict__ p, int64_t i, int left, const float v[4]) {
  if (left >= 4) {
    if (BF16) {
      *(uint2*)((uint16_t*)p + i) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
    } else {
      const f32x4_t x = {v[0], v[1], v[2], v[3]};
      f32x4_t* at = (f32x4_t*)((float*)p + i);
      if (NT) __builtin_nontemporal_store(x, at);
      else *at = x;
    }
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (q < left) {
        if (BF16) ((uint16_t*)p)[i + q] = (uint16_t)pack_bf16x2(v[q], 0.0f);
        else ((float*)p)[i + q] = v[q];
      }
  }
}

__device__ __forceinline__ void load_codes(const void* __restrict__ p, int64_t i, int left, float scale, float v[4]) {
  uint32_t c = 0;
  if (left >= 4) {
    c = *(const uint32_t*)((const uint8_t*)p + i);
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (q < left) c |= (uint32_t)((const uint8_t*)p)[i + q] << (8 * q);
  }
  const f32x2_t lo = __builtin_amdgcn_cvt_pk_f32_fp8(c, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8(c, true);
  v[0] = lo[0] * scale;
  v[1] = lo[1] * scale;
  v[2] = hi[0] * scale;
  v[3] = hi[1] * scale;
}

// One wavefront's block of 256: scale, codes, and the scale's store by lane 0. SIGNED: the first
// moment; else the root of the second, whose positive values stay positive. A NaN rounds to the NaN
// code by itself and the maxima pass over it; infinities are looked at only where there are any.
template <bool SIGNED>
__device__ __forceinline__ void store_codes(void* __restrict__ p, float* __restrict__ scale, int64_t i, int left,
                                            const float v[4], const uint32_t rnd[4]) {
  float amax = 0.0f;
#pragma unroll
  for (int q = 0; q < 4; ++q) amax = fmaxf(amax, fabsf(v[q]));  // elements behind the tensor are 0
  amax = wave_max(amax);
  const bool inf = amax > 3.402823466e+38f;
  if (inf) {
    amax = 0.0f;
#pragma unroll
    for (int q = 0; q < 4; ++q) amax = fmaxf(amax, finite(v[q]) ? fabsf(v[q]) : 0.0f);
    amax = wave_max(amax);
  }
  const int k = amax > 0.0f ? scale_exp(amax) : 0;
  const float inv = pow2(-k);
  float c[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    float x = round_e4m3(fabsf(v[q]) * inv, rnd[q]);
    if (!SIGNED && v[q] > 0.0f) x = fmaxf(x, 0x1p-9f);
    if (SIGNED) x = __builtin_copysignf(x, v[q]);
    c[q] = inf && !finite(v[q]) ? __uint_as_float(0x7FC00000u) : x;
  }
  int code = __builtin_amdgcn_cvt_pk_fp8_f32(c[0], c[1], 0, false);
  code = __builtin_amdgcn_cvt_pk_fp8_f32(c[2], c[3], code, true);
  if (left >= 4) {
    *(uint32_t*)((uint8_t*)p + i) = (uint32_t)code;
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (q < left) ((uint8_t*)p)[i + q] = (uint8_t)((uint32_t)code >> (8 * q));
  }
  if ((threadIdx.x & (kWave - 1)) == 0 && left > 0) *scale = pow2(k);
}

// Four elements of one thread, at i; FULL: all inside the tensor.
template <bool Q8, bool W16, bool G16, bool MASTER, bool FULL>
__device__ __forceinline__ void step4(const lrmoe_adamw_tensor& t, const AdamwArgs& a, const lrmoe_adamw_scalars& s,
                                      int64_t i) {
  // f32 arrays stream past the caches: 416 -> 406 us for 75 M elements with 32-bit states; no
  // difference with 8-bit ones, which then keep the plain accesses
  constexpr bool NT = !Q8;
  const int left = FULL ? 4 : (int)max((int64_t)0, min((int64_t)4, t.n - i));
  float w[4], g[4], m[4], v[4], r[4], *sm = nullptr, *sv = nullptr;
  load4<G16, NT>(t.grad, i, left, g);
  if (MASTER) load4<false, NT>(t.master, i, left, w);
  else load4<W16, NT>(t.w, i, left, w);
  if (Q8) {
    const int64_t b = i / kBlock;
    sm = t.m_scale + b;
    sv = t.v_scale + b;
    load_codes(t.m, i, left, FULL || left > 0 ? *sm : 1.0f, m);
    load_codes(t.v, i, left, FULL || left > 0 ? *sv : 1.0f, v);
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] = v[q] * v[q];
  } else {
    load4<false, NT>(t.m, i, left, m);
    load4<false, NT>(t.v, i, left, v);
  }
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const float x = g[q] * s.grad_scale;
    m[q] = m[q] * a.b1 + x * a.a1;
    v[q] = v[q] * a.b2 + (x * x) * a.a2;
    r[q] = sqrtf(v[q]);
    // with 8-bit states the reciprocal instruction (1 ulp) stands for the division, whose ten
    // instructions cost 10 of 253 us there and nothing where the step waits for memory
    const float num = m[q] * s.c1, den = r[q] * s.c2 + a.eps;
    const float u = Q8 ? num * __builtin_amdgcn_rcpf(den) : num / den;
    w[q] = w[q] * s.decay - u * s.lr;
  }
  if (MASTER) store4<false, NT>(t.master, i, left, w);
  store4<W16, NT>(t.w, i, left, w);
  if (Q8) {
    uint32_t rm[4], rr[4];
    const uint64_t c0 = (uint64_t)(t.first + i);  // a multiple of 4: the four share the high half
    const uint32_t base = mix(s.key + (uint32_t)(c0 >> 32) * 0x9E3779B1u) + (uint32_t)c0;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint32_t h = mix(base + q);
      rm[q] = h & 0xFFFFu;
      rr[q] = h >> 16;
    }
    store_codes<true>(t.m, sm, i, left, m, rm);
    store_codes<false>(t.v, sv, i, left, r, rr);
  } else {
    store4<false, NT>(t.m, i, left, m);
    store4<false, NT>(t.v, i, left, v);
  }
}

template <bool Q8, bool W16, bool G16, bool MASTER, class Table>
__global__ __launch_bounds__(kThreads) void adamw_kernel(Table tab, AdamwArgs a) {
  const uint32_t chunk = a.chunk0 + blockIdx.x;
  int at = -1;  // the last tensor whose first chunk is at or before this one
  for (int i = 0; i < tab.n; i += kWave) {
    const int q = i + (int)(threadIdx.x & (kWave - 1));
    at += __popcll(__ballot(q < tab.n && tab.first(q) <= chunk));
  }
  at = __builtin_amdgcn_readfirstlane(at);
  const lrmoe_adamw_tensor t = tab.tensor(at);
  const lrmoe_adamw_scalars s = a.dyn ? *a.dyn : a.s;
  const int64_t i0 = (int64_t)(chunk - tab.first(at)) * kChunk, i = i0 + threadIdx.x * 4;
  // without the bounds' instructions a whole chunk of 8-bit states, which is bound by them, takes 252
  // instead of 276 us for 75 M elements; with 32-bit states it takes 415 instead of 403 us
  if (Q8 && i0 + kChunk <= t.n) step4<Q8, W16, G16, MASTER, true>(t, a, s, i);
  else step4<Q8, W16, G16, MASTER, false>(t, a, s, i);
}

template <class Table>
lrmoe_status run_launch(const lrmoe_adamw_config* c, unsigned grid, const Table& tab, const AdamwArgs& a,
                        hipStream_t s) {
  const int kind = (c->state_bits == 8 ? 8 : 0) + (c->w_dtype == LRMOE_BF16 ? 4 : 0) +
                   (c->grad_dtype == LRMOE_BF16 ? 2 : 0) + (c->master ? 1 : 0);
  switch (kind) {
    case 0: adamw_kernel<false, false, false, false><<<grid, kThreads, 0, s>>>(tab, a); break;
    case 2: adamw_kernel<false, false, true, false><<<grid, kThreads, 0, s>>>(tab, a); break;
    case 4: adamw_kernel<false, true, false, false><<<grid, kThreads, 0, s>>>(tab, a); break;
    case 5: adamw_kernel<false, true, false, true><<<grid, kThreads, 0, s>>>(tab, a); break;
    case 6: adamw_kernel<false, true, true, false><<<grid, kThreads, 0, s>>>(tab, a); break;
    case 7: adamw_kernel<false, true, true, true><<<grid, kThreads, 0, s>>>(tab, a); break;
    case 8: adamw_kernel<true, false, false, false><<<grid, kThreads, 0, s>>>(tab, a); break;
    case 10: adamw_kernel<true, false, true, false><<<grid, kThreads, 0, s>>>(tab, a); break;
    case 12: adamw_kernel<true, true, false, false><<<grid, kThreads, 0, s>>>(tab, a); break;
    case 13: adamw_kernel<true, true, false, true><<<grid, kThreads, 0, s>>>(tab, a); break;
    case 14: adamw_kernel<true, true, true, false><<<grid, kThreads, 0, s>>>(tab, a); break;
    case 15: adamw_kernel<true, true, true, true><<<grid, kThreads, 0, s>>>(tab, a); break;
    default: return LRMOE_ERR_UNSUPPORTED;
  }
  return launch_status();
}

template <class Table>
lrmoe_status run(const lrmoe_adamw_config* c, uint32_t chunks, const Table& tab, AdamwArgs a, hipStream_t s) {
  for (a.chunk0 = 0; a.chunk0 < chunks; a.chunk0 += kLaunchChunks) {
    const lrmoe_status st = run_launch(c, std::min(chunks - a.chunk0, kLaunchChunks), tab, a, s);
    if (st != LRMOE_OK) return st;
  }
  return LRMOE_OK;
}

// Tables as a plan holds them: the tensors that have elements, then their first chunks.
int live_tensors(const lrmoe_adamw_tensor* t, int32_t n) {
  int k = 0;
  for (int32_t i = 0; i < n; ++i) k += t[i].n > 0;
  return k;
}

}  // namespace

size_t adamw_plan_bytes(int32_t n_tensors) {
  return std::max<size_t>(256, align_up((size_t)n_tensors * (sizeof(lrmoe_adamw_tensor) + sizeof(uint32_t)), 256));
}

void adamw_plan(const lrmoe_adamw_tensor* tensors, int32_t n_tensors, void* plan) {
  lrmoe_adamw_tensor* t = (lrmoe_adamw_tensor*)plan;
  uint32_t* first = (uint32_t*)(t + live_tensors(tensors, n_tensors));
  uint32_t chunks = 0;
  for (int32_t i = 0; i < n_tensors; ++i) {
    if (tensors[i].n == 0) continue;
    *t++ = tensors[i];
    *first++ = chunks;
    chunks += (uint32_t)ceil_div(tensors[i].n, kChunk);
  }
}

lrmoe_status launch_adamw(const lrmoe_adamw_tensor* tensors, int32_t n_tensors, const lrmoe_adamw_config* c,
                          const lrmoe_adamw_scalars& host, const void* plan_d, const lrmoe_adamw_scalars* scalars_d,
                          hipStream_t s) {
  AdamwArgs a;
  a.b1 = (float)c->beta1;
  a.a1 = (float)(1.0 - c->beta1);
  a.b2 = (float)c->beta2;
  a.a2 = (float)(1.0 - c->beta2);
  a.eps = (float)c->eps;
  a.s = host;
  a.dyn = scalars_d;
  if (plan_d) {
    const int n = live_tensors(tensors, n_tensors);
    uint64_t chunks = 0;
    for (int32_t i = 0; i < n_tensors; ++i) chunks += (uint64_t)ceil_div(tensors[i].n, kChunk);
    if (n == 0) return LRMOE_OK;
    if (chunks >> 31) return LRMOE_ERR_UNSUPPORTED;
    const lrmoe_adamw_tensor* t = (const lrmoe_adamw_tensor*)plan_d;
    return run(c, (uint32_t)chunks, PlanTable{t, (const uint32_t*)(t + n), n}, a, s);
  }
  int32_t i = 0;
  while (i < n_tensors) {
    ArgTable tab;
    tab.n = 0;
    uint64_t chunks = 0;
    for (; i < n_tensors && tab.n < kAdamwTensors; ++i) {
      const uint64_t more = (uint64_t)ceil_div(tensors[i].n, kChunk);
      if (more == 0) continue;
      if ((chunks + more) >> 31) break;  // the next launch takes it
      tab.t[tab.n] = tensors[i];
      tab.chunk[tab.n++] = (uint32_t)chunks;
      chunks += more;
    }
    if (tab.n == 0) break;
    const lrmoe_status st = run(c, (uint32_t)chunks, tab, a, s);
    if (st != LRMOE_OK) return st;
  }
  return LRMOE_OK;
}

}  // namespace lrmoe
