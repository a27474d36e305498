// The norms of gradient rows by token, for every kernel that scores.
#pragma once
#include "common.h"

namespace lrmoe {

constexpr int kScoreThreads = 256;
constexpr int kUnroll = 4;

// One wavefront per token row; each lane streams 16-byte chunks. ABS: sum of magnitudes
// instead of squares (the absolute-gradient criterion of the ablation). block: the index among the
// blocks of kScoreThreads threads that do this.
template <bool BF16, bool ABS>
__device__ __forceinline__ void token_sqnorm(const uint4* __restrict__ G, int T, int chunks_per_row, int64_t block,
                                             double* __restrict__ gn) {
  const int lane = threadIdx.x & (kWave - 1);
  const int64_t t = block * (kScoreThreads / kWave) + threadIdx.x / kWave;
  if (t >= T) return;  // the whole wavefront leaves together; no block-level sync follows
  const uint4* row = G + t * chunks_per_row;
  double acc = 0.0;
  for (int c0 = lane; c0 < chunks_per_row; c0 += kWave * kUnroll) {
    uint4 v[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      int c = c0 + u * kWave;
      v[u] = c < chunks_per_row ? ld_stream(row + c) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (ABS) acc += BF16 ? sumabs_bf16x8(v[u]) : sumabs_f32x4(v[u]);
      else acc += BF16 ? sumsq_bf16x8(v[u]) : sumsq_f32x4(v[u]);
    }
  }
  acc = wave_sum(acc);
  if (lane == 0) gn[t] = acc;
}

}  // namespace lrmoe
