// Top-k selection over one row of expert logits by one warp, and the weights of the selected
// experts: shared by the router kernels and the few-token layer.
#pragma once

#include <math.h>

#include "../../include/mm_ops.h"
#include "mm_rows.cuh"

namespace mm {

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  return v;
}

// An unsigned integer of the same order as the float: -0 and 0 alike, NaN (1) below -inf, and
// 0 left for "taken" and "no expert".
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t b = __float_as_uint(v + 0.0f);
  if ((b & 0x7FFFFFFFu) > 0x7F800000u) return 1u;
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

// sigmoid with CUDA's accurate exponential and division; sigmoid(-z) = 1 - sigmoid(z).
__device__ __forceinline__ float sigmoid_accurate(float z) { return 1.0f / (1.0f + expf(-z)); }

// The K largest of the warp's row: key[j] of a lane belongs to expert lane + 32 j. Returns the
// expert of rank `lane` (lanes >= K: -1). Each lane keeps its own largest key, so a round is one
// maximum and one minimum over the warp and a rescan by the lane that lost its key.
template <int NV>
__device__ __forceinline__ int select_topk(uint32_t (&key)[NV], int K, int lane) {
  int mine = -1;
  uint32_t best = 0;
  int at = 0;
  auto scan = [&] {
    best = 0;
    at = 0;
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (key[j] > best) best = key[j], at = j;
  };
  scan();
  for (int k = 0; k < K; ++k) {
    const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, best);
    const uint32_t e = __reduce_min_sync(
        0xFFFFFFFFu, best == top ? (uint32_t)(at * 32 + lane) : 0xFFFFFFFFu);
    if (lane == k) mine = (int)e;
    if ((e & 31u) == (uint32_t)lane) {
      const int j0 = (int)(e >> 5);
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (j == j0) key[j] = 0;
      scan();
    }
  }
  return mine;
}

// The weight of the lane's selected expert with logit z (lane < K), as mm_ops.h defines it.
// row_max, row_sum: max and sum of a over the whole row (used by softmax without `normalize`).
__device__ __forceinline__ float selected_weight(float z, bool has, int score, int normalize,
                                                 float scale, float row_max, float row_sum) {
  float a;
  if (score == MM_SCORE_SIGMOID) {
    a = has ? sigmoid_accurate(z) : 0.f;
  } else {
    float m = row_max;
    if (normalize) m = warp_max(has ? z : -INFINITY);
    if (m == -INFINITY) m = 0.f;  // every logit -inf: all a are 0
    a = has ? expf(z - m) : 0.f;
  }
  float total = 1.f;
  if (normalize)
    total = warp_sum(a);
  else if (score == MM_SCORE_SOFTMAX)
    total = row_sum;
  return total == 0.f ? 0.f : scale * a / total;
}

}  // namespace mm
