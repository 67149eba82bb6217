// The norm of many tensors together, and the tensors scaled down to a largest norm (definitions in
// mm_experts.h).
//
// Bound by HBM: the squares' sum reads every element once, the scaling reads and writes it. Two
// launches: blocks sum the squares of their chunks, which leaves one 64-bit number per block; the
// blocks of the second launch add those numbers in one order, each for itself, and scale their chunks.
// The tensors' addresses travel as the kernels' argument, kRefs at a time, so that a captured call
// holds them by itself.
//
// A chunk is kChunk elements of one tensor. A thread's squares are summed in 32 bits over 64 elements,
// then in 64 bits. Where those 32 bits would overflow or lose what is small (a sum of 2^126 or more, or
// below 2^-80 but not of zeros alone) the 64 squares are summed in 64 bits instead.
#include <algorithm>

#include "../../include/mm_experts.h"
#include "mm_kernels.h"
#include "mm_rows.cuh"

namespace mm {
namespace {

constexpr int kRefs = 1000;    // tensors per launch, at most (32 KB of arguments)
constexpr int kThreads = 256;
constexpr int kSteps = 8;      // vectors of 8 elements per thread and chunk
constexpr int kChunk = kThreads * 8 * kSteps;
constexpr int kBlocks = 8;     // per SM

struct Ref {
  const void* data;
  void* out;
  int64_t count;
  int32_t first;  // chunks of the tensors before
  int16_t type, out_type;
};

template <int N>
struct GradArgs {
  double* parts;  // [launches][blocks] sums of squares
  int n, chunks, part_count;
  double max_norm, eps;
  float* norm;
  int write_norm;
  Ref ref[N];
};

template <int N>
__device__ __forceinline__ int ref_of(const GradArgs<N>& a, int chunk) {
  int lo = 0, hi = a.n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.ref[mid].first <= chunk) lo = mid; else hi = mid;
  }
  return lo;
}

inline __host__ __device__ bool on16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// Elements at `at` .. at + 8 of a tensor, zeros past its end.
template <typename T>
__device__ __forceinline__ void load8(const T* p, int64_t at, int64_t count, bool vec, float (&v)[8]) {
  if (vec && at + 8 <= count) {
    load_vec<8>(p + at, v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float one[1] = {0.f};
      if (at + i < count) load_vec<1>(p + at + i, one);
      v[i] = one[0];
    }
  }
}

template <typename T>
__device__ __forceinline__ double chunk_squares(const T* p, int64_t base, int64_t count) {
  const bool vec = on16(p);
  float v[kSteps][8];
#pragma unroll
  for (int s = 0; s < kSteps; ++s)
    load8(p, base + (int64_t)(s * kThreads + threadIdx.x) * 8, count, vec, v[s]);
  float sum[4] = {};
#pragma unroll
  for (int s = 0; s < kSteps; ++s)
#pragma unroll
    for (int i = 0; i < 8; ++i) sum[i & 3] = fmaf(v[s][i], v[s][i], sum[i & 3]);
  const float total = (sum[0] + sum[1]) + (sum[2] + sum[3]);
  if (total >= 8.2718061e-25f && total < 8.5070592e37f) return total;  // 2^-80, 2^126
  double wide = 0.0;
  bool any = false;
#pragma unroll
  for (int s = 0; s < kSteps; ++s)
#pragma unroll
    for (int i = 0; i < 8; ++i) any |= v[s][i] != 0.f;
  if (!any) return 0.0;
#pragma unroll
  for (int s = 0; s < kSteps; ++s)
#pragma unroll
    for (int i = 0; i < 8; ++i) wide += (double)v[s][i] * (double)v[s][i];
  return wide;
}

__device__ __forceinline__ double block_sum(double v) {
  __shared__ double part[kThreads / 32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  double s = 0.0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) s += part[w];
  return s;
}

template <int N>
__global__ void __launch_bounds__(kThreads) k_squares(const __grid_constant__ GradArgs<N> a) {
  pdl_wait();
  pdl_launch_dependents();
  double sum = 0.0;
  for (int c = blockIdx.x; c < a.chunks; c += gridDim.x) {
    const Ref& r = a.ref[ref_of(a, c)];
    const int64_t base = (int64_t)(c - r.first) * kChunk;
    sum += r.type == MM_BF16 ? chunk_squares(static_cast<const __nv_bfloat16*>(r.data), base, r.count)
                             : chunk_squares(static_cast<const float*>(r.data), base, r.count);
  }
  sum = block_sum(sum);
  if (threadIdx.x == 0) a.parts[blockIdx.x] = sum;
}

template <typename T, typename O>
__device__ __forceinline__ void scale_chunk(const Ref& r, int64_t base, float before, float scale) {
  const T* p = static_cast<const T*>(r.data);
  O* out = static_cast<O*>(r.out);
  const bool vec = on16(p) && on16(out);
  float v[kSteps][8];
#pragma unroll
  for (int s = 0; s < kSteps; ++s)
    load8(p, base + (int64_t)(s * kThreads + threadIdx.x) * 8, r.count, vec, v[s]);
#pragma unroll
  for (int s = 0; s < kSteps; ++s) {
    const int64_t at = base + (int64_t)(s * kThreads + threadIdx.x) * 8;
    if (before != 1.f) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[s][i] *= before;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[s][i] *= scale;
    if (vec && at + 8 <= r.count) {
      store_vec<8>(out + at, v[s]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float one[1] = {v[s][i]};
        if (at + i < r.count) store_vec<1>(out + at + i, one);
      }
    }
  }
}

template <int N>
__global__ void __launch_bounds__(kThreads) k_scale(const __grid_constant__ GradArgs<N> a) {
  pdl_wait();
  pdl_launch_dependents();
  double sum = 0.0;
  for (int p = threadIdx.x; p < a.part_count; p += kThreads) sum += a.parts[p];
  const double norm = sqrt(block_sum(sum));
  if (a.write_norm && blockIdx.x == 0 && threadIdx.x == 0) *a.norm = (float)norm;
  const double share = a.max_norm / (norm + a.eps);
  // A share that 32 bits hold badly is two factors. The first is a power of two that loses nothing of
  // elements whose results are not below 2^-149 anyway.
  const float before = !(share < 0x1p-100) ? 1.f : share < 0x1p-160 ? 0x1p-120f : 0x1p-64f;
  const float scale = share >= 1.0 ? 1.f : (float)(share / before);  // (NaN stays NaN)
  for (int c = blockIdx.x; c < a.chunks; c += gridDim.x) {
    const Ref& r = a.ref[ref_of(a, c)];
    if (scale == 1.f && r.data == r.out) continue;  // nothing changes
    const int64_t base = (int64_t)(c - r.first) * kChunk;
    if (r.type == MM_BF16) {
      if (r.out_type == MM_BF16) scale_chunk<__nv_bfloat16, __nv_bfloat16>(r, base, before, scale);
      else scale_chunk<__nv_bfloat16, float>(r, base, before, scale);
    } else {
      if (r.out_type == MM_BF16) scale_chunk<float, __nv_bfloat16>(r, base, before, scale);
      else scale_chunk<float, float>(r, base, before, scale);
    }
  }
}

// ------------------------------------------------------------------------------------ host side

inline bool aligned_to(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

constexpr int64_t kMostBlocks = 152 * kBlocks;  // sums of a launch

int64_t launches_for(int64_t n) { return std::max<int64_t>(1, (n + kRefs - 1) / kRefs); }

template <int N>
cudaError_t launch_refs(const mm_tensor_ref* t, int count, bool scale, GradArgs<N>& a, cudaStream_t st) {
  int64_t chunks = 0;
  a.n = 0;
  for (int i = 0; i < count; ++i) {
    if (t[i].count == 0) continue;
    a.ref[a.n++] = Ref{t[i].data, t[i].out, t[i].count, (int32_t)chunks, (int16_t)t[i].type,
                       (int16_t)t[i].out_type};
    chunks += (t[i].count + kChunk - 1) / kChunk;
  }
  if (chunks >= (int64_t)1 << 31) return cudaErrorInvalidValue;
  a.chunks = (int)chunks;
  const int64_t most = std::min<int64_t>(kMostBlocks, (int64_t)kBlocks * std::max(1, device_sm_count()));
  const unsigned blocks = (unsigned)std::max<int64_t>(1, std::min(most, chunks));
  if (!scale) a.part_count = (int)blocks;
  return scale ? launch_pdl(k_scale<N>, dim3(blocks), dim3(kThreads), 0, st, a)
               : launch_pdl(k_squares<N>, dim3(blocks), dim3(kThreads), 0, st, a);
}

mm_status run(int64_t n, const mm_tensor_ref* t, bool clip, double max_norm, double eps, float* norm,
              void* workspace, size_t workspace_bytes, void* stream) {
  if (n < 0 || (n > 0 && t == nullptr) || norm == nullptr || !aligned_to(norm, 4)) return MM_ERR_INVALID_ARG;
  if (n >= 1 << 20) return MM_ERR_UNSUPPORTED;
  if (clip && (!(max_norm >= 0.0) || !(eps >= 0.0) || eps > 3e38)) return MM_ERR_INVALID_ARG;
  for (int64_t i = 0; i < n; ++i) {
    const mm_tensor_ref& r = t[i];
    if (r.count < 0 || (r.type != MM_BF16 && r.type != MM_FP32)) return MM_ERR_INVALID_ARG;
    if (r.count >= (int64_t)1 << 44) return MM_ERR_UNSUPPORTED;
    if (r.count > 0 && (!r.data || !aligned_to(r.data, r.type == MM_BF16 ? 2 : 4))) return MM_ERR_INVALID_ARG;
    if (!clip) continue;
    if (r.out_type != MM_BF16 && r.out_type != MM_FP32) return MM_ERR_INVALID_ARG;
    if (r.count > 0 && (!r.out || !aligned_to(r.out, r.out_type == MM_BF16 ? 2 : 4) ||
                        (r.out == r.data && r.out_type != r.type)))
      return MM_ERR_INVALID_ARG;
  }
  if (workspace == nullptr || !aligned_to(workspace, 256) || workspace_bytes < mm_grad_workspace_size(n))
    return MM_ERR_WORKSPACE;
  clear_error();
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  double* parts = static_cast<double*>(workspace);
  auto all = [&](auto args) -> mm_status {
    int total = 0;
    for (int64_t i = 0; i < std::max<int64_t>(1, n); i += kRefs) {
      args.parts = parts + total;
      MM_TRY(launch_refs(t + i, (int)std::min<int64_t>(kRefs, n - i), false, args, st));
      total += args.part_count;
    }
    args.parts = parts;
    args.part_count = total;
    args.max_norm = max_norm;
    args.eps = eps;
    args.norm = norm;
    for (int64_t i = 0; i < std::max<int64_t>(1, n); i += kRefs) {
      args.write_norm = i == 0;
      MM_TRY(launch_refs(t + i, clip ? (int)std::min<int64_t>(kRefs, n - i) : 0, true, args, st));
      if (!clip) break;
    }
    return MM_OK;
  };
  // the argument is as long as it has to be
  if (n <= 64) return all(GradArgs<64>{});
  return all(GradArgs<kRefs>{});
}

}  // namespace
}  // namespace mm

using namespace mm;

extern "C" {

size_t mm_grad_workspace_size(int64_t n) {
  if (n < 0 || n >= 1 << 20) return 0;
  return (size_t)(launches_for(n) * kMostBlocks) * sizeof(double);
}

mm_status mm_grad_norm(int64_t n, const mm_tensor_ref* tensors, float* norm, void* workspace,
                       size_t workspace_bytes, void* stream) {
  return run(n, tensors, false, 0.0, 0.0, norm, workspace, workspace_bytes, stream);
}

mm_status mm_grad_clip(int64_t n, const mm_tensor_ref* tensors, double max_norm, double eps, float* norm,
                       void* workspace, size_t workspace_bytes, void* stream) {
  return run(n, tensors, true, max_norm, eps, norm, workspace, workspace_bytes, stream);
}

}  // extern "C"
