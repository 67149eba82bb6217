// The norm of many tensors together, and the tensors scaled down to a largest norm (definitions in
// mm_experts.h).
//
// Bound by HBM: the squares' sum reads every element once (569 M bf16: 176 us, 6.5 TB/s), the scaling reads
// and writes it (360 us, 6.3 TB/s). Two launches: blocks sum the squares of their chunks, which leaves one 64-bit number per block; the
// blocks of the second launch add those numbers in one order, each for itself, and scale their chunks.
// The tensors' addresses travel as the kernels' argument, kRefs at a time, so that a captured call
// holds them by itself.
//
// A chunk is 32 KB of one tensor; a block has a run of chunks, and the second launch walks the
// runs backwards, from what the first has read last. (L2 gives nothing back all the same: the first pass
// reads with streaming loads, and the second runs at the rate of a copy.) k_squares has 64 registers, for
// four blocks per SM, and spills 36 bytes for it. A thread's squares are summed in
// 32 bits over 64 elements (bf16; fp32: 32), then in 64 bits. Where those 32 bits would overflow or lose what is small (a
// sum of 2^126 or more, or below 2^-80 but not of zeros alone) the squares are summed in 64 bits instead.
#include <algorithm>

#include "../../include/mm_experts.h"
#include "mm_kernels.h"
#include "mm_rows.cuh"

namespace mm {
namespace {

constexpr int kRefs = 1000;    // tensors per launch, at most (32 KB of arguments)
constexpr int kThreads = 256;
constexpr int kBlocks = 4;     // per SM
// Vectors of 8 elements per thread and chunk: eight 16-byte loads in flight of either type.
template <typename T>
constexpr int kSteps = 16 / sizeof(T);
template <typename T>
constexpr int kChunk = kThreads * 8 * kSteps<T>;
inline int64_t chunk_of(int type) { return type == MM_BF16 ? kChunk<__nv_bfloat16> : kChunk<float>; }

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

// 8 elements as they lie in memory.
template <typename T>
struct Raw {
  uint4 w[sizeof(T) / 2];
};

// A thread's vectors of a chunk: elements base + 8 (256 s + thread) on, zeros past the end.
template <typename T>
__device__ __forceinline__ void load_chunk(const T* p, int64_t base, int64_t count, bool vec, Raw<T> (&r)[kSteps<T>]) {
  if (vec && base + kChunk<T> <= count) {
    const uint4* at = reinterpret_cast<const uint4*>(p + base) + threadIdx.x * (sizeof(T) / 2);
#pragma unroll
    for (int s = 0; s < kSteps<T>; ++s)
#pragma unroll
      for (int w = 0; w < (int)sizeof(T) / 2; ++w) r[s].w[w] = __ldcs(at + s * kThreads * (sizeof(T) / 2) + w);
    return;
  }
#pragma unroll
  for (int s = 0; s < kSteps<T>; ++s) {
    const int64_t at = base + (int64_t)(s * kThreads + threadIdx.x) * 8;
    if (vec && at + 8 <= count) {
#pragma unroll
      for (int w = 0; w < (int)sizeof(T) / 2; ++w) r[s].w[w] = reinterpret_cast<const uint4*>(p + at)[w];
    } else {
      r[s] = Raw<T>{};
      if (at >= count) continue;
      alignas(16) T one[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) one[i] = at + i < count ? p[at + i] : T(0.f);
      r[s] = *reinterpret_cast<const Raw<T>*>(one);
    }
  }
}

__device__ __forceinline__ void widen(const Raw<__nv_bfloat16>& r, float (&v)[8]) {
  const uint32_t u[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) v[2 * i] = bf16_lo(u[i]), v[2 * i + 1] = bf16_hi(u[i]);
}
__device__ __forceinline__ void widen(const Raw<float>& r, float (&v)[8]) {
  const uint32_t u[8] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w, r.w[1].x, r.w[1].y, r.w[1].z, r.w[1].w};
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(u[i]);
}

template <typename T>
__device__ __forceinline__ double chunk_squares(const T* p, int64_t base, int64_t count) {
  Raw<T> r[kSteps<T>];
  load_chunk(p, base, count, on16(p), r);
  float sum[4] = {};
#pragma unroll
  for (int s = 0; s < kSteps<T>; ++s) {
    float v[8];
    widen(r[s], v);
#pragma unroll
    for (int i = 0; i < 8; ++i) sum[i & 3] = fmaf(v[i], v[i], sum[i & 3]);
  }
  const float total = (sum[0] + sum[1]) + (sum[2] + sum[3]);
  if (total >= 0x1p-80f && total < 0x1p126f) return total;
  double wide = 0.0;
#pragma unroll
  for (int s = 0; s < kSteps<T>; ++s) {
    float v[8];
    widen(r[s], v);
    bool any = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) any |= v[i] != 0.f;
    if (!any) continue;
#pragma unroll
    for (int i = 0; i < 8; ++i) wide += (double)v[i] * (double)v[i];
  }
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

// The block's run of chunks: first .. end.
template <int N>
__device__ __forceinline__ void run_of(const GradArgs<N>& a, int& first, int& end) {
  first = (int)((int64_t)a.chunks * blockIdx.x / gridDim.x);
  end = (int)((int64_t)a.chunks * (blockIdx.x + 1) / gridDim.x);
}

template <int N>
__global__ void __launch_bounds__(kThreads, kBlocks) k_squares(const __grid_constant__ GradArgs<N> a) {
  pdl_wait();
  pdl_launch_dependents();
  int c, end;
  run_of(a, c, end);
  double sum = 0.0;
  if (c < end) {
    for (int i = ref_of(a, c); c < end; ++i) {
      const int stop = min(end, i + 1 < a.n ? a.ref[i + 1].first : a.chunks), first = a.ref[i].first;
      const int64_t count = a.ref[i].count;
      const void* data = a.ref[i].data;
      if (a.ref[i].type == MM_BF16) {
        for (; c < stop; ++c)
          sum += chunk_squares(static_cast<const __nv_bfloat16*>(data), (int64_t)(c - first) * kChunk<__nv_bfloat16>, count);
      } else {
        for (; c < stop; ++c)
          sum += chunk_squares(static_cast<const float*>(data), (int64_t)(c - first) * kChunk<float>, count);
      }
    }
  }
  sum = block_sum(sum);
  if (threadIdx.x == 0) a.parts[blockIdx.x] = sum;
}

// Chunks end - 1 .. c of a tensor whose chunks start with `first`.
template <typename T, typename O>
__device__ __forceinline__ void scale_chunks(const Ref& ref, int first, int c, int end, float before, float scale) {
  const T* p = static_cast<const T*>(ref.data);
  O* out = static_cast<O*>(ref.out);
  const int64_t count = ref.count;
  const bool vec = on16(p) && on16(out);
  for (int k = end - 1; k >= c; --k) {
    const int64_t base = (int64_t)(k - first) * kChunk<T>;
    Raw<T> r[kSteps<T>];
    load_chunk(p, base, count, vec, r);
#pragma unroll
    for (int s = 0; s < kSteps<T>; ++s) {
      const int64_t at = base + (int64_t)(s * kThreads + threadIdx.x) * 8;
      float v[8];
      widen(r[s], v);
      if (before != 1.f) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= before;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] *= scale;
      if (vec && at + 8 <= count) {
        if constexpr (sizeof(O) == 2) {
          __stcs(reinterpret_cast<uint4*>(out + at), make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]),
                                                                pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])));
        } else {
          __stcs(reinterpret_cast<float4*>(out + at), make_float4(v[0], v[1], v[2], v[3]));
          __stcs(reinterpret_cast<float4*>(out + at) + 1, make_float4(v[4], v[5], v[6], v[7]));
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float one[1] = {v[i]};
          if (at + i < count) store_vec<1>(out + at + i, one);
        }
      }
    }
  }
}

template <int N>
__global__ void __launch_bounds__(kThreads, kBlocks) k_scale(const __grid_constant__ GradArgs<N> a) {
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
  int c, end;
  run_of(a, c, end);
  if (c >= end) return;
  for (int i = ref_of(a, end - 1); c < end; --i) {
    const Ref& r = a.ref[i];
    const int first = r.first, from = max(c, first);
    if (!(scale == 1.f && r.data == r.out)) {  // (nothing changes)
      if (r.type == MM_BF16) {
        if (r.out_type == MM_BF16) scale_chunks<__nv_bfloat16, __nv_bfloat16>(r, first, from, end, before, scale);
        else scale_chunks<__nv_bfloat16, float>(r, first, from, end, before, scale);
      } else {
        if (r.out_type == MM_BF16) scale_chunks<float, __nv_bfloat16>(r, first, from, end, before, scale);
        else scale_chunks<float, float>(r, first, from, end, before, scale);
      }
    }
    end = from;
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
    chunks += (t[i].count + chunk_of(t[i].type) - 1) / chunk_of(t[i].type);
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
