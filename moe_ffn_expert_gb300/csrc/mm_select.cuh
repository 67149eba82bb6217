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

// The K largest of the warp's row: key[j] of a lane belongs to expert lane * NV + j, so among
// equal keys the lowest lane has the lowest expert. Returns the expert of rank `lane` (lanes
// >= K: -1); `slot`: shared memory for the K
// experts, of the warp's own. Each lane keeps its largest key
// at hand; a round is one maximum over the warp, a ballot for its lowest holder, which writes its
// expert to the rank's slot and brings up its next key.
//   NV <= 4: a lane's keys are sorted first (adjacent exchanges, so equal keys keep their order)
//   and a round shifts them: 6 moves instead of a search of 13 steps (16384 rows of 128, K = 8:
//   9.9 us, 11.4 with the search).
//   NV == 8: the search, in every lane (shorter than a branch of one; sorting 8 takes as long as
//   nine rounds save). Above that: the search, in the one lane.
template <int NV, typename ID>
__device__ __forceinline__ int select_topk(uint32_t (&key)[NV], int K, int lane,
                                           volatile ID* slot) {
  const uint32_t lower = (1u << lane) - 1;
  int at[NV <= 4 ? NV : 1];
  uint32_t best;
  auto scan = [&] {
    best = key[0];
#pragma unroll
    for (int j = 1; j < NV; ++j) best = max(best, key[j]);
    at[0] = lane * NV + NV - 1;
#pragma unroll
    for (int j = NV - 2; j >= 0; --j) at[0] = key[j] == best ? lane * NV + j : at[0];
  };
  if constexpr (NV <= 4) {
#pragma unroll
    for (int j = 0; j < NV; ++j) at[j] = lane * NV + j;
#pragma unroll
    for (int pass = 0; pass < NV; ++pass)
#pragma unroll
      for (int j = pass & 1; j + 1 < NV; j += 2) {
        const uint32_t x = key[j], y = key[j + 1];
        const int ax = at[j], ay = at[j + 1];
        const bool swap = y > x;
        key[j] = swap ? y : x, key[j + 1] = swap ? x : y;
        at[j] = swap ? ay : ax, at[j + 1] = swap ? ax : ay;
      }
    best = key[0];
  } else {
    scan();
  }
#pragma unroll 1
  for (int k = 0; k < K; ++k) {
    const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, best);
    const bool holds = best == top;
    const uint32_t holders = __ballot_sync(0xFFFFFFFFu, holds);
    const bool owner = holds && (holders & lower) == 0;
    if (owner) slot[k] = (ID)at[0];
    if constexpr (NV <= 4) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        key[j] = owner ? (j + 1 < NV ? key[j + 1 < NV ? j + 1 : 0] : 0u) : key[j];
        if (j + 1 < NV) at[j] = owner ? at[j + 1 < NV ? j + 1 : 0] : at[j];
      }
      best = key[0];
    } else if constexpr (NV <= 8) {
#pragma unroll
      for (int j = 0; j < NV; ++j)
        key[j] = owner && lane * NV + j == at[0] ? 0u : key[j];
      scan();
    } else if (owner) {
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (lane * NV + j == at[0]) key[j] = 0;
      scan();
    }
  }
  __syncwarp();
  const int mine = lane < K ? (int)slot[lane] : -1;
  __syncwarp();  // the slots may be written again
  return mine;
}

// Sums of sigmoids below this: every logit is below -46, where sigmoid(z) is e^z to 32 bits. Ratios are
// then taken of e^(z - largest z), as the sigmoids themselves leave the range of 32 bits from -88 on.
constexpr float kTinySigmoids = 1e-20f;

// (Out of line, as is what follows an infinite logit: in line they took 0.4 of 16.2 us from a selection
// that never comes by.)
static __device__ __noinline__ float shifted_scores(float z, bool has) {
  const float m = warp_max(has ? z : -INFINITY);
  return has && m != -INFINITY ? expf(z - m) : 0.f;
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
  if (normalize) {
    total = warp_sum(a);
    if (score == MM_SCORE_SIGMOID && total < kTinySigmoids) {
      a = shifted_scores(z, has);
      total = warp_sum(a);
    }
  } else if (score == MM_SCORE_SOFTMAX)
    total = row_sum;
  return total == 0.f ? 0.f : scale * (a / total);
}

}  // namespace mm
