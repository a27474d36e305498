// The router beside the experts: top-K routing with its expert-major pair lists, the balance
// loss with its per-expert counts, the gradient of the logits, and the gradient of the routing
// weights from the saved output rows.
//
// All of it is one pass over [T x E] logits (or, for the routing-weight gradient, over the
// [N x D] output rows), so memory bounds it at large T and launch latency at small T. A group
// of L lanes holds one token's logits in registers, V to a lane.
#include <algorithm>

#include "common.h"

namespace lrmoe {
namespace {

constexpr float kFltMax = 3.402823466e+38f;
constexpr float kNegInf = -__builtin_huge_valf();

__device__ __forceinline__ float clean(float x) {  // NaN -> -inf, +inf -> FLT_MAX
  return x != x ? kNegInf : fminf(x, kFltMax);
}

template <bool BF16>
__device__ __forceinline__ float load_logit(const void* __restrict__ logits, int64_t i) {
  if (BF16) return __uint_as_float((uint32_t)((const uint16_t*)logits)[i] << 16);
  return ((const float*)logits)[i];
}

// Reductions over the L lanes of a token's group; every lane gets the result.
template <int L>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor(v, o, kWave));
  return v;
}
template <int L>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor(v, o, kWave);
  return v;
}
template <int L>
__device__ __forceinline__ int group_min(int v) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) v = min(v, __shfl_xor(v, o, kWave));
  return v;
}

// Expert of value v of a lane.
template <int L, int V>
__device__ __forceinline__ int expert_of(int lane, int v) {
  return v * L + lane;
}

// A token's logits by the rules of the header; -inf beyond E and for a masked token.
template <int L, int V, bool BF16>
__device__ __forceinline__ void load_row(const void* __restrict__ logits, const uint8_t* __restrict__ mask, int64_t t,
                                         int E, bool in, int lane, float x[V]) {
  const bool on = in && (!mask || mask[t] != 0);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = expert_of<L, V>(lane, v);
    x[v] = on && e < E ? clean(load_logit<BF16>(logits, t * E + e)) : kNegInf;
  }
}

// ---------------------------------------------------------------- routing

constexpr int kRouteThreads = 1024;

// Tokens per chunk: one bit per (chunk token, local expert) has to fit 48 KB of LDS, and the
// placing blocks each read the histograms of all chunks, so there are few of them.
int route_chunk(const lrmoe_router* r) {
  int c = 128;
  while (ceil_div(r->T, c) > 256 && c < 1024 && (int64_t)r->local * c * 2 / 8 <= 48 * 1024) c *= 2;
  return c;
}

// One block per chunk of tokens: the K largest logits of each, their weights, and how often the
// chunk chose each expert.
template <int L, int V, bool BF16>
__global__ __launch_bounds__(kRouteThreads) void route_topk_kernel(int T, int E, int K, int C, int renorm, float scale,
                                                                   const void* __restrict__ logits,
                                                                   const uint8_t* __restrict__ mask,
                                                                   int32_t* __restrict__ idx, float* __restrict__ w,
                                                                   int32_t* __restrict__ hist) {
  __shared__ int cnt[1024];
  for (int e = threadIdx.x; e < E; e += kRouteThreads) cnt[e] = 0;
  __syncthreads();
  const int lane = threadIdx.x & (L - 1), group = threadIdx.x / L;
  constexpr int kGroups = kRouteThreads / L;
  const int64_t t0 = (int64_t)blockIdx.x * C, t1 = min(t0 + C, (int64_t)T);
  for (int64_t tb = t0; tb < t1; tb += kGroups) {
    const int64_t t = tb + group;
    const bool in = t < t1;
    float x[V];
    load_row<L, V, BF16>(logits, mask, t, E, in, lane, x);
    float top = kNegInf;
#pragma unroll
    for (int v = 0; v < V; ++v) top = fmaxf(top, x[v]);
    top = group_max<L>(top);
    float Z = 0.0f;
    if (!renorm) {
#pragma unroll
      for (int v = 0; v < V; ++v) Z += x[v] > kNegInf ? expf(x[v] - top) : 0.0f;
      Z = group_sum<L>(Z);
    }
    // slot k: the largest value left, the lowest index that has it
    int my_e = -1;
    float my_x = kNegInf;
    for (int k = 0; k < K; ++k) {
      float best = kNegInf;
#pragma unroll
      for (int v = 0; v < V; ++v) best = fmaxf(best, x[v]);
      best = group_max<L>(best);
      int at = 1 << 30;
#pragma unroll
      for (int v = V - 1; v >= 0; --v)
        if (x[v] == best && best > kNegInf) at = expert_of<L, V>(lane, v);
      at = group_min<L>(at);
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (expert_of<L, V>(lane, v) == at) x[v] = kNegInf;
      if (lane == k) {
        my_e = at < (1 << 30) ? at : -1;
        my_x = best;
      }
    }
    const float p = my_e >= 0 ? expf(my_x - top) : 0.0f;
    if (renorm) Z = group_sum<L>(p);
    if (in && lane < K) {
      idx[t * K + lane] = my_e;
      w[t * K + lane] = my_e >= 0 ? scale * (p / Z) : 0.0f;
      if (my_e >= 0) atomicAdd(&cnt[my_e], 1);
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += kRouteThreads) hist[(int64_t)blockIdx.x * E + e] = cnt[e];
}

// One block per chunk: where each expert's pairs start and how many earlier chunks hold (from
// all chunks' histograms), then the rank of a pair in its chunk as the number of lower set bits
// of its expert's token bits: no order of atomics enters the result.
__global__ __launch_bounds__(kRouteThreads) void route_place_kernel(
    int T, int E, int K, int C, int chunks, int first, int local, const int32_t* __restrict__ hist,
    const int32_t* __restrict__ idx, const float* __restrict__ w, int32_t* __restrict__ counts,
    int64_t* __restrict__ seg_off, int32_t* __restrict__ tok, int32_t* __restrict__ slot, float* __restrict__ alpha,
    int32_t* __restrict__ pmap) {
  __shared__ int total[1024], before[1024];
  __shared__ int wave_total[kRouteThreads / kWave];
  extern __shared__ uint32_t bits[];  // [C / 32][local]
  const int tid = threadIdx.x, c = blockIdx.x;
  for (int e = tid; e < E; e += kRouteThreads) total[e] = before[e] = 0;
  for (int i = tid; i < C / 32 * local; i += kRouteThreads) bits[i] = 0;
  __syncthreads();
  for (int64_t i = tid; i < (int64_t)chunks * E; i += kRouteThreads) {
    const int ch = (int)(i / E), e = (int)(i - (int64_t)ch * E), h = hist[i];
    if (h) {
      atomicAdd(&total[e], h);
      if (ch < c) atomicAdd(&before[e], h);
    }
  }
  __syncthreads();
  if (c == 0)
    for (int e = tid; e < E; e += kRouteThreads) counts[e] = total[e];
  // exclusive scan of the local experts' totals (local <= 1024 = one value per thread)
  const int mine = tid < local ? total[first + tid] : 0;
  int inc = mine;
#pragma unroll
  for (int o = 1; o < kWave; o <<= 1) {
    const int up = __shfl_up(inc, o, kWave);
    if ((tid & (kWave - 1)) >= o) inc += up;
  }
  if ((tid & (kWave - 1)) == kWave - 1) wave_total[tid / kWave] = inc;
  __syncthreads();
  int base = inc - mine;
  for (int q = 0; q < tid / kWave; ++q) base += wave_total[q];
  if (tid < local) {
    if (c == 0) {
      seg_off[tid] = base;
      if (tid == local - 1) seg_off[local] = base + mine;
    }
    before[first + tid] += base;  // first pair row of (this chunk, expert)
  }
  __syncthreads();
  const int64_t t0 = (int64_t)c * C;
  const int n = (int)(min(t0 + C, (int64_t)T) - t0) * K;
  for (int i = tid; i < n; i += kRouteThreads) {
    const int e = idx[t0 * K + i], l = e - first, t = i / K;
    if (e >= 0 && l >= 0 && l < local) atomicOr(&bits[(t >> 5) * local + l], 1u << (t & 31));
  }
  __syncthreads();
  for (int i = tid; i < n; i += kRouteThreads) {
    const int e = idx[t0 * K + i], l = e - first, t = i / K;
    int row = -1;
    if (e >= 0 && l >= 0 && l < local) {
      row = before[e] + __popc(bits[(t >> 5) * local + l] & ((1u << (t & 31)) - 1u));
      for (int q = 0; q < (t >> 5); ++q) row += __popc(bits[q * local + l]);
      tok[row] = (int32_t)(t0 + t);
      slot[row] = i - t * K;
      alpha[row] = w[t0 * K + i];
    }
    pmap[t0 * K + i] = row;
  }
}

// ---------------------------------------------------------------- balance loss

constexpr int kBalThreads = 256;
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
  double* dot;     // [n_seq] sum_e counts psum
  int32_t* n;      // [n_seq] live tokens
};

int64_t balance_tiles(const lrmoe_router* r, int32_t n_seq) { return r->T / kBalTile + n_seq; }

size_t balance_layout(const lrmoe_router* r, int32_t n_seq, char* base, BalanceWs* out) {
  const size_t tiles = (size_t)balance_tiles(r, n_seq);
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
  w.dot = (double*)take((size_t)n_seq * 8);
  w.n = (int32_t*)take((size_t)n_seq * 4);
  if (out) *out = w;
  return at;
}

template <int L, int V, bool BF16>
__global__ __launch_bounds__(kBalThreads) void balance_tile_kernel(int T, int E, int K, int n_seq,
                                                                   const void* __restrict__ logits,
                                                                   const uint8_t* __restrict__ mask,
                                                                   const int32_t* __restrict__ idx,
                                                                   const int64_t* __restrict__ off, BalanceWs ws) {
  constexpr int kGroups = kBalThreads / L;
  __shared__ int cnt[1024];
  __shared__ float part[kGroups][L * V];
  __shared__ int live_of[kBalTile];
  const int64_t b = blockIdx.x;
  const int s = off ? seq_of_tile(off, n_seq, T, b) : 0;
  int64_t lo, hi;
  seq_range(off, s, T, &lo, &hi);
  lo += (b - first_tile(lo, s)) * kBalTile;
  hi = min(hi, lo + kBalTile);
  if (lo >= hi) return;  // a slot that no tile uses: the whole block leaves
  for (int e = threadIdx.x; e < E; e += kBalThreads) cnt[e] = 0;
  const int lane = threadIdx.x & (L - 1), group = threadIdx.x / L;
  float acc[V];
#pragma unroll
  for (int v = 0; v < V; ++v) acc[v] = 0.0f;
  for (int64_t tb = lo; tb < hi; tb += kGroups) {
    const int64_t t = tb + group;
    float x[V], top = kNegInf, Z = 0.0f;
    load_row<L, V, BF16>(logits, mask, t, E, t < hi, lane, x);
#pragma unroll
    for (int v = 0; v < V; ++v) top = fmaxf(top, x[v]);
    top = group_max<L>(top);
    const bool live = top > kNegInf;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      x[v] = x[v] > kNegInf ? expf(x[v] - top) : 0.0f;
      Z += x[v];
    }
    Z = group_sum<L>(Z);
    const float rz = live ? 1.0f / Z : 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] += x[v] * rz;
    if (lane == 0 && t < hi) live_of[t - lo] = live ? 1 : 0;
  }
#pragma unroll
  for (int v = 0; v < V; ++v) part[group][expert_of<L, V>(lane, v)] = acc[v];
  __syncthreads();
  const int n = (int)(hi - lo) * K;
  for (int i = threadIdx.x; i < n; i += kBalThreads) {
    const int e = idx[lo * K + i];
    if (e >= 0 && e < E && live_of[i / K]) atomicAdd(&cnt[e], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += kBalThreads) {
    float a = 0.0f;
#pragma unroll
    for (int g = 0; g < kGroups; ++g) a += part[g][e];
    ws.psum[b * E + e] = a;
    ws.count[b * E + e] = cnt[e];
  }
  if (threadIdx.x == 0) {
    int a = 0;
    for (int i = 0; i < (int)(hi - lo); ++i) a += live_of[i];
    ws.live[b] = a;
  }
}

__device__ __forceinline__ double block_sum(double v, double* sh) {  // kBalThreads threads, all get the sum
  v = wave_sum(v);
  if ((threadIdx.x & (kWave - 1)) == 0) sh[threadIdx.x / kWave] = v;
  __syncthreads();
  double a = 0.0;
  for (int i = 0; i < kBalThreads / kWave; ++i) a += sh[i];
  __syncthreads();
  return a;
}

// One block per sequence: its tiles joined in order.
__global__ __launch_bounds__(kBalThreads) void balance_join_kernel(int T, int E, const int64_t* __restrict__ off,
                                                                   BalanceWs ws, int32_t* __restrict__ counts,
                                                                   float* __restrict__ psum) {
  __shared__ double sh[kBalThreads / kWave];
  const int s = blockIdx.x;
  int64_t lo, hi;
  seq_range(off, s, T, &lo, &hi);
  const int64_t b0 = first_tile(lo, s);
  const int tiles = (int)((hi - lo + kBalTile - 1) / kBalTile);
  double dot = 0.0;
  for (int e = threadIdx.x; e < E; e += kBalThreads) {
    double a = 0.0;
    int n = 0;
    for (int i = 0; i < tiles; ++i) {
      a += (double)ws.psum[(b0 + i) * E + e];
      n += ws.count[(b0 + i) * E + e];
    }
    psum[(int64_t)s * E + e] = (float)a;
    counts[(int64_t)s * E + e] = n;
    dot += a * n;
  }
  double live = 0.0;
  for (int i = threadIdx.x; i < tiles; i += kBalThreads) live += ws.live[b0 + i];
  dot = block_sum(dot, sh);
  live = block_sum(live, sh);
  if (threadIdx.x == 0) {
    ws.dot[s] = dot;
    ws.n[s] = (int)live;
  }
}

__global__ __launch_bounds__(kBalThreads) void balance_loss_kernel(int E, int K, int n_seq, float coef, BalanceWs ws,
                                                                   float* __restrict__ norm,
                                                                   float* __restrict__ loss) {
  __shared__ double sh[kBalThreads / kWave];
  double alive = 0.0, sum = 0.0;
  for (int s = threadIdx.x; s < n_seq; s += kBalThreads) alive += ws.n[s] > 0 ? 1.0 : 0.0;
  alive = block_sum(alive, sh);
  for (int s = threadIdx.x; s < n_seq; s += kBalThreads) {
    const double n = ws.n[s];
    const double f = n > 0 ? (double)coef * E / (alive * K * n * n) : 0.0;
    norm[s] = (float)f;
    sum += f * ws.dot[s];
  }
  sum = block_sum(sum, sh);
  if (threadIdx.x == 0) loss[0] = (float)sum;
}

// ---------------------------------------------------------------- gradient of the logits

constexpr int kGradThreads = 256;

template <int L, int V, bool BF16>
__global__ __launch_bounds__(kGradThreads) void route_bwd_kernel(
    int T, int E, int K, int renorm, float scale, const void* __restrict__ logits, const uint8_t* __restrict__ mask,
    const int32_t* __restrict__ idx, const float* __restrict__ dalpha, const int32_t* __restrict__ pmap,
    int64_t n_pairs, const int64_t* __restrict__ off, int n_seq, const int32_t* __restrict__ counts,
    const float* __restrict__ norm, const float* __restrict__ gloss, void* __restrict__ dlogits) {
  const int lane = threadIdx.x & (L - 1);
  const int64_t t = (int64_t)blockIdx.x * (kGradThreads / L) + threadIdx.x / L;
  const bool in = t < T;
  float x[V], p[V], dx[V], top = kNegInf, Z = 0.0f;
  load_row<L, V, BF16>(logits, mask, t, E, in, lane, x);
#pragma unroll
  for (int v = 0; v < V; ++v) top = fmaxf(top, x[v]);
  top = group_max<L>(top);
  const bool live = top > kNegInf;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    p[v] = x[v] > kNegInf ? expf(x[v] - top) : 0.0f;
    Z += p[v];
    dx[v] = 0.0f;
  }
  Z = group_sum<L>(Z);
  const float rz = live ? 1.0f / Z : 0.0f;
#pragma unroll
  for (int v = 0; v < V; ++v) p[v] *= rz;
  if (dalpha) {
    // y of every chosen expert, and which they are
    float y[V];
    uint32_t chosen = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) y[v] = 0.0f;
    for (int k = 0; k < K; ++k) {
      const int e = in && live ? idx[t * K + k] : -1;
      float d = 0.0f;
      if (e >= 0) {
        if (pmap) {
          const int j = pmap[t * K + k];
          d = j >= 0 && j < n_pairs ? dalpha[j] : 0.0f;
        } else {
          d = dalpha[t * K + k];
        }
      }
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (e >= 0 && expert_of<L, V>(lane, v) == e && x[v] > kNegInf) {
          y[v] = scale * d;
          chosen |= 1u << v;
        }
    }
    float q[V], s = 0.0f;
    if (renorm) {
      float ct = kNegInf, cz = 0.0f;
#pragma unroll
      for (int v = 0; v < V; ++v) ct = fmaxf(ct, (chosen >> v) & 1 ? x[v] : kNegInf);
      ct = group_max<L>(ct);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        q[v] = (chosen >> v) & 1 ? expf(x[v] - ct) : 0.0f;
        cz += q[v];
      }
      cz = group_sum<L>(cz);
      const float rc = cz > 0.0f ? 1.0f / cz : 0.0f;
#pragma unroll
      for (int v = 0; v < V; ++v) q[v] *= rc;
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) q[v] = p[v];
    }
#pragma unroll
    for (int v = 0; v < V; ++v) s += (chosen >> v) & 1 ? q[v] * y[v] : 0.0f;
    s = group_sum<L>(s);
#pragma unroll
    for (int v = 0; v < V; ++v) dx[v] = q[v] * (y[v] - s);
  }
  if (norm) {
    int s = 0;
    bool on = live;
    if (off && in) {  // the last sequence that starts at or before t
      int a = 0, z = n_seq - 1;
      while (a < z) {
        const int m = (a + z + 1) / 2;
        if (off[m] <= t) a = m;
        else z = m - 1;
      }
      s = a;
      on = live && t >= off[s] && t < off[s + 1];
    }
    float c[V], dot = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = expert_of<L, V>(lane, v);
      c[v] = on && e < E ? (float)counts[(int64_t)s * E + e] : 0.0f;
      dot += p[v] * c[v];
    }
    dot = group_sum<L>(dot);
    const float f = on ? norm[s] * (gloss ? gloss[0] : 1.0f) : 0.0f;
    if (on) {
#pragma unroll
      for (int v = 0; v < V; ++v) dx[v] += f * (p[v] * (c[v] - dot));
    }
  }
  if (!in) return;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = expert_of<L, V>(lane, v);
    if (e >= E) continue;
    const float d = live ? dx[v] : 0.0f;
    if (BF16) ((uint16_t*)dlogits)[t * E + e] = (uint16_t)pack_bf16x2(d, 0.0f);
    else ((float*)dlogits)[t * E + e] = d;
  }
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

// Calls f(L, V) as compile-time values for E experts.
template <class F>
lrmoe_status by_experts(int E, F&& f) {
  const int v = (int)ceil_div(E, kWave);
  if (v <= 1) return f(std::integral_constant<int, 64>(), std::integral_constant<int, 1>());
  if (v <= 2) return f(std::integral_constant<int, 64>(), std::integral_constant<int, 2>());
  if (v <= 4) return f(std::integral_constant<int, 64>(), std::integral_constant<int, 4>());
  if (v <= 8) return f(std::integral_constant<int, 64>(), std::integral_constant<int, 8>());
  return f(std::integral_constant<int, 64>(), std::integral_constant<int, 16>());
}

}  // namespace

size_t route_ws_bytes(const lrmoe_router* r) {
  return align_up(std::max<size_t>(1, (size_t)ceil_div(r->T, route_chunk(r)) * r->E * 4), 256);
}

lrmoe_status launch_route(const lrmoe_router* r, const void* logits, const uint8_t* mask, int32_t* idx, float* w,
                          int32_t* counts, int64_t* seg_off, int32_t* tok, int32_t* slot, float* alpha,
                          int32_t* pmap, void* ws, hipStream_t s) {
  const int C = route_chunk(r);
  const int chunks = (int)ceil_div(r->T, C);
  int32_t* hist = (int32_t*)ws;
  if (chunks > 0) {
    by_experts(r->E, [&](auto l, auto v) {
      constexpr int L = decltype(l)::value, V = decltype(v)::value;
      if (r->dtype == LRMOE_BF16)
        route_topk_kernel<L, V, true><<<chunks, kRouteThreads, 0, s>>>(r->T, r->E, r->K, C, r->renorm, r->scale,
                                                                       logits, mask, idx, w, hist);
      else
        route_topk_kernel<L, V, false><<<chunks, kRouteThreads, 0, s>>>(r->T, r->E, r->K, C, r->renorm, r->scale,
                                                                        logits, mask, idx, w, hist);
      return LRMOE_OK;
    });
    if (launch_status() != LRMOE_OK) return LRMOE_ERR_HIP;
  }
  route_place_kernel<<<std::max(1, chunks), kRouteThreads, (size_t)C / 8 * r->local, s>>>(
      r->T, r->E, r->K, C, chunks, r->first, r->local, hist, idx, w, counts, seg_off, tok, slot, alpha, pmap);
  return launch_status();
}

size_t balance_ws_bytes(const lrmoe_router* r, int32_t n_seq) { return balance_layout(r, n_seq, nullptr, nullptr); }

lrmoe_status launch_balance_loss(const lrmoe_router* r, const void* logits, const uint8_t* mask, const int32_t* idx,
                                 const int64_t* seq_off_d, int32_t n_seq, float coef, int32_t* counts, float* psum,
                                 float* norm, float* loss, void* ws, hipStream_t s) {
  BalanceWs b;
  balance_layout(r, n_seq, (char*)ws, &b);
  if (r->T > 0) {
    const unsigned tiles = (unsigned)balance_tiles(r, n_seq);
    by_experts(r->E, [&](auto l, auto v) {
      constexpr int L = decltype(l)::value, V = decltype(v)::value;
      if (r->dtype == LRMOE_BF16)
        balance_tile_kernel<L, V, true><<<tiles, kBalThreads, 0, s>>>(r->T, r->E, r->K, n_seq, logits, mask, idx,
                                                                      seq_off_d, b);
      else
        balance_tile_kernel<L, V, false><<<tiles, kBalThreads, 0, s>>>(r->T, r->E, r->K, n_seq, logits, mask, idx,
                                                                       seq_off_d, b);
      return LRMOE_OK;
    });
    if (launch_status() != LRMOE_OK) return LRMOE_ERR_HIP;
  }
  balance_join_kernel<<<n_seq, kBalThreads, 0, s>>>(r->T, r->E, seq_off_d, b, counts, psum);
  if (launch_status() != LRMOE_OK) return LRMOE_ERR_HIP;
  balance_loss_kernel<<<1, kBalThreads, 0, s>>>(r->E, r->K, n_seq, coef, b, norm, loss);
  return launch_status();
}

lrmoe_status launch_route_bwd(const lrmoe_router* r, const void* logits, const uint8_t* mask, const int32_t* idx,
                              const float* dalpha, const int32_t* pmap, int64_t n_pairs, const int64_t* seq_off_d,
                              int32_t n_seq, const int32_t* counts, const float* norm, const float* gloss,
                              void* dlogits, hipStream_t s) {
  by_experts(r->E, [&](auto l, auto v) {
    constexpr int L = decltype(l)::value, V = decltype(v)::value;
    const unsigned g = (unsigned)ceil_div(r->T, kGradThreads / L);
    if (r->dtype == LRMOE_BF16)
      route_bwd_kernel<L, V, true><<<g, kGradThreads, 0, s>>>(r->T, r->E, r->K, r->renorm, r->scale, logits, mask, idx,
                                                              dalpha, pmap, n_pairs, seq_off_d, n_seq, counts, norm,
                                                              gloss, dlogits);
    else
      route_bwd_kernel<L, V, false><<<g, kGradThreads, 0, s>>>(r->T, r->E, r->K, r->renorm, r->scale, logits, mask,
                                                               idx, dalpha, pmap, n_pairs, seq_off_d, n_seq, counts,
                                                               norm, gloss, dlogits);
    return LRMOE_OK;
  });
  return launch_status();
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
