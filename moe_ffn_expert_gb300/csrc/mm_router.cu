// Router: top-k selection over expert logits, its weights and loss statistics, and its gradient
// (definitions in mm_ops.h). One warp per token, E / 32 logits per lane in registers.
//
// In terms of logits the gradient is, with p = a / A, w^ the normalised weights of the selected
// experts, c = scale and the upstream gradients dw, dP (prob_sum) and dL (lse):
//   normalize, softmax:  dz_j += c w^_j (dw_j - sum_i dw_i w^_i)            j selected
//   normalize, sigmoid:  the same times (1 - sigmoid z_j)
//   softmax:             dz_j += c dw_j p_j,  dz_e -= p_e sum_j c dw_j p_j
//   sigmoid:             dz_j += c dw_j a_j (1 - a_j)
//   prob_sum:            dz_e += p_e (dP_e - sum_i dP_i p_i)   [sigmoid: times (1 - a_e)]
//   lse:                 dz_e += dL exp(z_e - lse)
//
// A row is a few hundred bytes: the kernels are bound by launch and row latency at serving sizes
// (64 rows of 256, K = 8: 2.7 us; one row: 2.7), and by instructions over many rows (16384 rows of
// 128, K = 8: 10.0 us, of which 2.3 are the selection's last 7 rounds; 15.6 with the loss
// statistics, whose partial sums take a second launch; backward of 8192 rows of 256: 10.6 us, 1.6
// TB/s).
#include <cuda_runtime.h>

#include <algorithm>

#include "mm_kernels.h"
#include "mm_select.cuh"

namespace mm {
namespace {

// Rows in flight per block, at most. The forward's blocks leave partial sums, so it has fewer and
// larger ones (16384 x 128 with them: 15.7 us, 16.7 in blocks of 8; 8192 x 256 backward: 10.8 us in
// blocks of 8, 12.1 of 16).
constexpr int kFwdWarps = 16, kBwdWarps = 8;
// Few rows spread over more SMs (64 rows of 256: 2.7 us in blocks of 4, 3.5 in blocks of 16).
inline int warps_per_block(int64_t T, int most) { return T <= 2048 ? 4 : most; }

struct RouterArgs {
  int64_t T;
  int E, K, score, normalize;
  float scale;
  const void* logits;
  const float* bias;
  int32_t* ids;
  float *weights, *lse, *prob_part;  // prob_part: [gridDim.x][E] partial sums or null
  // backward
  const int32_t* ids_in;
  const float *dw, *dP, *dL;
  void* dz;
};

__device__ __forceinline__ float load_logit(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ float load_logit(const float* p) { return *p; }
__device__ __forceinline__ void store_logit(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void store_logit(float* p, float v) { *p = v; }

// The lane's NV logits, of experts lane * NV on; zero past E. `words`: whole rows of aligned words.
template <typename LT, int NV>
__device__ __forceinline__ void load_logits(const LT* row, int E, int lane, bool words,
                                            float (&z)[NV]) {
  constexpr int BYTES = NV * sizeof(LT);
  if constexpr (BYTES == 8 || BYTES % 16 == 0) {
    if (words) {
      const LT* at = row + lane * NV;
      if constexpr (BYTES == 8) {
        const uint2 v = *reinterpret_cast<const uint2*>(at);
        if constexpr (sizeof(LT) == 2) {
          z[0] = bf16_lo(v.x), z[1] = bf16_hi(v.x), z[2] = bf16_lo(v.y), z[3] = bf16_hi(v.y);
        } else {
          z[0] = __uint_as_float(v.x), z[1] = __uint_as_float(v.y);
        }
      } else {
#pragma unroll
        for (int j = 0; j < BYTES / 16; ++j) {
          const uint4 v = reinterpret_cast<const uint4*>(at)[j];
          const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if constexpr (sizeof(LT) == 2) {
              z[8 * j + 2 * i] = bf16_lo(u[i]);
              z[8 * j + 2 * i + 1] = bf16_hi(u[i]);
            } else {
              z[4 * j + i] = __uint_as_float(u[i]);
            }
          }
        }
      }
      return;
    }
  }
#pragma unroll
  for (int j = 0; j < NV; ++j) z[j] = lane * NV + j < E ? load_logit(row + lane * NV + j) : 0.f;
}

template <int NV>
__device__ __forceinline__ float row_max(const float (&z)[NV], int E, int lane) {
  float m = -INFINITY;
#pragma unroll
  for (int j = 0; j < NV; ++j)
    if (lane * NV + j < E) m = fmaxf(m, z[j]);
  m = warp_max(m);
  return m == -INFINITY ? 0.f : m;  // a row of -inf: exp(z) is 0 without a shift
}

// log sum exp of a row with an infinite logit: infinite, or NaN with a NaN beside it.
template <typename LT>
__device__ __noinline__ float infinite_sum(const LT* row, int E) {
  float sum = INFINITY;
#pragma unroll 1
  for (int e = 0; e < E; ++e) sum += fabsf(load_logit(row + e));
  return sum;
}

// The row's a (in 32 bits up to a common factor, which its uses divide out) and their sum. m: row_max.
template <int NV>
__device__ __forceinline__ float row_scores(const float (&z)[NV], float (&x)[NV], int E, int lane,
                                            bool soft, float m) {
  float A = 0.f;
  if (!soft) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      x[j] = lane * NV + j >= E ? 0.f : sigmoid_accurate(z[j]);
      A += x[j];
    }
    A = warp_sum(A);
    if (!(A < kTinySigmoids)) return A;
    A = 0.f;
  }
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    x[j] = lane * NV + j >= E ? 0.f : expf(z[j] - m);
    A += x[j];
  }
  return warp_sum(A);
}

template <typename LT, int NV>
__global__ void __launch_bounds__(32 * kFwdWarps) k_router_fwd(RouterArgs a) {
  constexpr int SUMS = NV < 4 ? NV : 4;  // probabilities per lane summed over the warps at a time
  __shared__ float part[kFwdWarps][32 * SUMS];
  __shared__ int slot[kFwdWarps][16];
  pdl_wait();
  pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const int E = a.E, K = a.K;
  const bool words = E == 32 * NV && (reinterpret_cast<uintptr_t>(a.logits) & 15) == 0;
  const bool all = a.prob_part != nullptr || (a.score == MM_SCORE_SOFTMAX && !a.normalize);
  float acc[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) acc[j] = 0.f;
  for (int64_t t = (int64_t)blockIdx.x * warps + warp; t < a.T; t += (int64_t)gridDim.x * warps) {
    const LT* row = static_cast<const LT*>(a.logits) + t * E;
    float z[NV];
    uint32_t key[NV];
    load_logits<LT, NV>(row, E, lane, words, z);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int e = lane * NV + j;
      key[j] = 0;
      if (e >= E) continue;
      float k = z[j];
      if (a.bias != nullptr)
        k = (a.score == MM_SCORE_SIGMOID ? sigmoid_accurate(k) : k) + a.bias[e];
      key[j] = order_key(k);
    }
    float m = 0.f, A = 0.f;
    if (all || a.lse != nullptr) m = row_max<NV>(z, E, lane);
    if (all) {
      float x[NV];
      A = row_scores<NV>(z, x, E, lane, a.score == MM_SCORE_SOFTMAX, m);
      if (a.prob_part != nullptr) {
        const float inv = A == 0.f ? 0.f : 1.f / A;
#pragma unroll
        for (int j = 0; j < NV; ++j) acc[j] += x[j] * inv;
      }
    }
    if (a.lse != nullptr) {
      float s = A;
      if (!all || a.score == MM_SCORE_SIGMOID) {
        s = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j)
          if (lane * NV + j < E) s += expf(z[j] - m);
        s = warp_sum(s);
      }
      if (lane == 0) a.lse[t] = m < INFINITY ? m + logf(s) : infinite_sum(row, E);
    }
    const int id = select_topk<NV>(key, K, lane, &slot[warp][0]);
    const float zs = lane < K ? load_logit(row + id) : 0.f;
    const float w = selected_weight(zs, lane < K, a.score, a.normalize, a.scale, m, A);
    if (lane < K) {
      a.ids[t * K + lane] = id;
      a.weights[t * K + lane] = w;
    }
  }
  if (a.prob_part == nullptr) return;
#pragma unroll
  for (int j = 0; j < NV; j += SUMS) {  // the block's warps, in order
#pragma unroll
    for (int i = 0; i < SUMS; ++i) part[warp][lane * SUMS + i] = acc[j + i];
    __syncthreads();
    const int e = (int)threadIdx.x / SUMS * NV + j + (int)threadIdx.x % SUMS;
    if (threadIdx.x < 32 * SUMS && e < E) {
      float s = 0.f;
#pragma unroll 4
      for (int i = 0; i < warps; ++i) s += part[i][threadIdx.x];
      a.prob_part[(int64_t)blockIdx.x * E + e] = s;
    }
    __syncthreads();
  }
}

template <typename LT, int NV>
__global__ void __launch_bounds__(32 * kBwdWarps) k_router_bwd(RouterArgs a) {
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const int E = a.E, K = a.K;
  const bool words = E == 32 * NV && (reinterpret_cast<uintptr_t>(a.logits) & 15) == 0;
  const bool soft = a.score == MM_SCORE_SOFTMAX;
  const bool all = a.dP != nullptr || (soft && !a.normalize);
  for (int64_t t = (int64_t)blockIdx.x * warps + warp; t < a.T; t += (int64_t)gridDim.x * warps) {
    const LT* row = static_cast<const LT*>(a.logits) + t * E;
    float z[NV], dz[NV];
    load_logits<LT, NV>(row, E, lane, words, z);
#pragma unroll
    for (int j = 0; j < NV; ++j) dz[j] = 0.f;
    const int id_in = lane < K ? a.ids_in[t * K + lane] : -1;
    const bool has = id_in >= 0 && id_in < E;
    const float dw = has ? a.scale * a.dw[t * K + lane] : 0.f;
    const float zs = has ? load_logit(row + id_in) : 0.f;
    float m = 0.f, A = 0.f, inv = 0.f;
    if (all || a.dL != nullptr) m = row_max<NV>(z, E, lane);
    float p[NV];
    if (all) {
      A = row_scores<NV>(z, p, E, lane, soft, m);
      inv = A == 0.f ? 0.f : 1.f / A;
#pragma unroll
      for (int j = 0; j < NV; ++j) p[j] *= inv;
    }
    // through the weights: `add` goes to the lane's selected expert, `common` p_e to every one
    float add, common = 0.f;
    if (a.normalize) {
      const float w = selected_weight(zs, has, a.score, 1, 1.f, 0.f, 0.f);
      add = w * (dw - warp_sum(dw * w));
      if (!soft) add *= sigmoid_accurate(-zs);
    } else if (soft) {
      add = has ? dw * expf(zs - m) * inv : 0.f;
      common -= warp_sum(add);
    } else {
      add = dw * sigmoid_accurate(zs) * sigmoid_accurate(-zs);
    }
    if (!has) add = 0.f;
    if (all) {
      float dot = 0.f, g[NV];
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        g[j] = a.dP != nullptr && lane * NV + j < E ? a.dP[lane * NV + j] : 0.f;
        dot += g[j] * p[j];
      }
      dot = warp_sum(dot);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const float to_prob = p[j] * (g[j] - dot);
        dz[j] = (soft ? to_prob : to_prob * sigmoid_accurate(-z[j])) + common * p[j];
      }
    }
    if (a.dL != nullptr) {
      float x[NV], s = 0.f;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        x[j] = lane * NV + j < E ? expf(z[j] - m) : 0.f;
        s += x[j];
      }
      s = warp_sum(s);
      const float f = s == 0.f ? 0.f : a.dL[t] / s;
#pragma unroll
      for (int j = 0; j < NV; ++j) dz[j] += f * x[j];
    }
    for (int k = 0; k < K; ++k) {
      const int e = __shfl_sync(0xFFFFFFFFu, has ? id_in : -1, k);
      const float v = __shfl_sync(0xFFFFFFFFu, add, k);
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (e == lane * NV + j) dz[j] += v;
    }
    LT* const out = static_cast<LT*>(a.dz) + t * E + lane * NV;
    if (NV >= 8 && words && (reinterpret_cast<uintptr_t>(a.dz) & 15) == 0) {
#pragma unroll
      for (int j = 0; j + 8 <= NV; j += 8)
        store_vec<8>(out + j, *reinterpret_cast<const float(*)[8]>(dz + (NV >= 8 ? j : 0)));
    } else {
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (lane * NV + j < E) store_logit(out + j, dz[j]);
    }
  }
}

// LANES x W columns per block, the parts dealt to 512 / LANES slices with 8 loads in flight each;
// the slices' sums are added in order.
template <int LANES, int W>
__global__ void __launch_bounds__(512) k_column_sums(SumArgs a) {
  constexpr int SLICES = 512 / LANES, COLS = LANES * W;
  __shared__ float part[SLICES][COLS + 1];
  pdl_wait();
  int k = 0;
#pragma unroll
  for (int i = 1; i < 3; ++i)
    if (i < a.jobs && (int64_t)blockIdx.y >= a.job[i].first) k = i;
  const SumJob job = a.job[k];
  const int64_t y = (int64_t)blockIdx.y - job.first;
  const int slice = threadIdx.x / LANES, at = threadIdx.x % LANES * W, c = blockIdx.x * COLS + at;
  const float* src = job.src + y * job.parts * a.cols + c;
  float s[W];
#pragma unroll
  for (int i = 0; i < W; ++i) s[i] = 0.f;
  if (c < a.cols) {
#pragma unroll 8
    for (int64_t p = slice; p < job.parts; p += SLICES) {
      if constexpr (W == 4) {
        const float4 v = __ldcg(reinterpret_cast<const float4*>(src + p * a.cols));
        s[0] += v.x, s[1] += v.y, s[2] += v.z, s[3] += v.w;
      } else {
        s[0] += __ldcg(src + p * a.cols);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < W; ++i) part[slice][at + i] = s[i];
  __syncthreads();
  const int col = blockIdx.x * COLS + (int)threadIdx.x;
  if (threadIdx.x < COLS && col < a.cols) {
    float v[1] = {0.f};
#pragma unroll 16
    for (int i = 0; i < SLICES; ++i) v[0] += part[i][threadIdx.x];
    store_any<1>(job.dst, a.type, y * a.cols + col, v);
  }
}

inline bool aligned_to(const void* p, size_t a) {
  return (reinterpret_cast<uintptr_t>(p) % a) == 0;
}

mm_status check_desc(const mm_router_desc* d) {
  if (d == nullptr || d->T < 0 || d->E < 1 || d->K < 1 || d->K > d->E) return MM_ERR_INVALID_ARG;
  if (d->logits_type != MM_BF16 && d->logits_type != MM_FP32) return MM_ERR_INVALID_ARG;
  if (d->score != MM_SCORE_SOFTMAX && d->score != MM_SCORE_SIGMOID) return MM_ERR_INVALID_ARG;
  if (d->E > 1024 || d->K > 16 || d->T >= ((int64_t)1 << 40)) return MM_ERR_UNSUPPORTED;
  return MM_OK;
}

// The forward's or the backward's blocks: at most 64 warps per SM.
int64_t router_blocks(const mm_router_desc& d, int most = kFwdWarps) {
  const int warps = warps_per_block(d.T, most);
  return std::min<int64_t>((d.T + warps - 1) / warps, (int64_t)std::max(1, device_sm_count()) * 64 / warps);
}

RouterArgs router_args(const mm_router_desc& d) {
  RouterArgs a{};
  a.T = d.T;
  a.E = d.E;
  a.K = d.K;
  a.score = d.score;
  a.normalize = d.normalize;
  a.scale = d.scale;
  return a;
}

// Calls f with the number of logits per lane as a compile-time constant.
template <typename F>
cudaError_t for_width(int E, F&& f) {
  if (E <= 32) return f(std::integral_constant<int, 1>());
  if (E <= 64) return f(std::integral_constant<int, 2>());
  if (E <= 128) return f(std::integral_constant<int, 4>());
  if (E <= 256) return f(std::integral_constant<int, 8>());
  if (E <= 512) return f(std::integral_constant<int, 16>());
  return f(std::integral_constant<int, 32>());
}

cudaError_t launch_fwd(const mm_router_desc& d, const RouterArgs& a, cudaStream_t st) {
  const dim3 grid((unsigned)router_blocks(d)), block(32 * warps_per_block(d.T, kFwdWarps));
  return for_width(d.E, [&](auto nv) {
    constexpr int NV = decltype(nv)::value;
    return d.logits_type == MM_BF16
               ? launch_pdl(k_router_fwd<__nv_bfloat16, NV>, grid, block, 0, st, a)
               : launch_pdl(k_router_fwd<float, NV>, grid, block, 0, st, a);
  });
}

}  // namespace

cudaError_t launch_router(const mm_router_desc& d, const float* logits, const float* bias,
                          int32_t* ids, float* weights, cudaStream_t st) {
  RouterArgs a = router_args(d);
  a.logits = logits;
  a.bias = bias;
  a.ids = ids;
  a.weights = weights;
  return launch_fwd(d, a, st);
}

cudaError_t launch_column_sums(const SumArgs& a, int64_t rows, cudaStream_t st) {
  auto grid = [&](int cols) { return dim3((unsigned)((a.cols + cols - 1) / cols), (unsigned)rows); };
  if (a.cols % 4 != 0) return launch_pdl(k_column_sums<32, 1>, grid(32), dim3(512), 0, st, a);
  // 128 columns per block read whole lines; 32 share the parts of few columns among more threads
  // (16384 x 512 backward 45 us with 32 and 51 with 128, 64 x 7168 14 and 11)
  if (a.cols >= 1024)
    return launch_pdl(k_column_sums<32, 4>, grid(128), dim3(512), 0, st, a);
  return launch_pdl(k_column_sums<8, 4>, grid(32), dim3(512), 0, st, a);
}

}  // namespace mm

using namespace mm;

extern "C" {

size_t mm_router_workspace_size(const mm_router_desc* d) {
  if (check_desc(d) != MM_OK) return 0;
  return std::max<size_t>(256, (size_t)router_blocks(*d) * d->E * sizeof(float));
}

mm_status mm_router_forward(const mm_router_desc* d, const void* logits, const float* bias,
                            int32_t* topk_ids, float* topk_weights, float* prob_sum, float* lse,
                            void* workspace, size_t workspace_bytes, void* stream) {
  mm_status s = check_desc(d);
  if (s != MM_OK) return s;
  if (!aligned_to(bias, 4) || !aligned_to(topk_ids, 4) || !aligned_to(topk_weights, 4) ||
      !aligned_to(prob_sum, 4) || !aligned_to(lse, 4) ||
      !aligned_to(logits, d->logits_type == MM_BF16 ? 2 : 4))
    return MM_ERR_INVALID_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (d->T == 0) {
    clear_error();
    if (prob_sum) MM_TRY(cudaMemsetAsync(prob_sum, 0, d->E * sizeof(float), st));
    return MM_OK;
  }
  if (!logits || !topk_ids || !topk_weights) return MM_ERR_INVALID_ARG;
  const int64_t blocks = router_blocks(*d);
  if (prob_sum && (workspace == nullptr || !aligned_to(workspace, 256) ||
                   workspace_bytes < (size_t)blocks * d->E * sizeof(float)))
    return MM_ERR_WORKSPACE;
  clear_error();
  RouterArgs a = router_args(*d);
  a.logits = logits;
  a.bias = bias;
  a.ids = topk_ids;
  a.weights = topk_weights;
  a.lse = lse;
  a.prob_part = prob_sum ? static_cast<float*>(workspace) : nullptr;
  MM_TRY(launch_fwd(*d, a, st));
  if (prob_sum) {
    SumArgs sa{};
    sa.cols = d->E;
    sa.type = MM_FP32;
    sa.jobs = 1;
    sa.job[0] = SumJob{a.prob_part, prob_sum, blocks, 0};
    MM_TRY(launch_column_sums(sa, 1, st));
  }
  return MM_OK;
}

mm_status mm_router_backward(const mm_router_desc* d, const void* logits, const int32_t* topk_ids,
                             const float* d_topk_weights, const float* d_prob_sum,
                             const float* d_lse, void* d_logits, void* stream) {
  mm_status s = check_desc(d);
  if (s != MM_OK) return s;
  const size_t es = d->logits_type == MM_BF16 ? 2 : 4;
  if (!aligned_to(logits, es) || !aligned_to(d_logits, es) || !aligned_to(topk_ids, 4) ||
      !aligned_to(d_topk_weights, 4) || !aligned_to(d_prob_sum, 4) || !aligned_to(d_lse, 4))
    return MM_ERR_INVALID_ARG;
  if (d->T == 0) return MM_OK;
  if (!logits || !topk_ids || !d_topk_weights || !d_logits) return MM_ERR_INVALID_ARG;
  clear_error();
  RouterArgs a = router_args(*d);
  a.logits = logits;
  a.ids_in = topk_ids;
  a.dw = d_topk_weights;
  a.dP = d_prob_sum;
  a.dL = d_lse;
  a.dz = d_logits;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const dim3 blocks((unsigned)router_blocks(*d, kBwdWarps)), threads(32 * warps_per_block(d->T, kBwdWarps));
  MM_TRY(for_width(d->E, [&](auto nv) {
    constexpr int NV = decltype(nv)::value;
    return d->logits_type == MM_BF16
               ? launch_pdl(k_router_bwd<__nv_bfloat16, NV>, blocks, threads, 0, st, a)
               : launch_pdl(k_router_bwd<float, NV>, blocks, threads, 0, st, a);
  }));
  return MM_OK;
}

}  // extern "C"
