// residual_norm: the step between two transformer blocks, forward and backward (mm_ops.h).
//
//   p = f / rms(f) * w_post;   r' = a r + g p;   n = r' / rms(r') * w_pre
//
// and with q = 1 / rms(r'), s = 1 / rms(f), the upstream gradients u of r' and v of n:
//
//   d  = u + q (w_pre v) - r' q^3 / H <w_pre v, r'>          (the gradient of r' itself)
//   dr = a d,  dg = sum d p,  dw_pre = sum v r' q,  dw_post = sum (g d) f s
//   df = s (e d) - f s^3 / H <e d, f>,  e = w_post g         (df = g d without a post weight)
//
// <e d, f> needs d, which needs <w_pre v, r'>; written out,
//   <e d, f> = <e f, u> + q <e f, w_pre v> - q^3 / H <w_pre v, r'> <e f, r'>,
// so the six sums of a row come from one reduction. Everything is elementwise otherwise: the
// kernels are bound by HBM. A block holds a row in registers, so each tensor moves once.
#include <cuda_runtime.h>
#include <math.h>

#include <algorithm>

#include "../../include/mm_ops.h"
#include "mm_kernels.h"
#include "mm_rows.cuh"

namespace mm {
namespace {

constexpr int kMaxH = 16384;

struct NormArgs {
  int64_t T, rows_per_gate;  // rows_per_gate: T / groups (0: no gate)
  int H, ptype;
  float scale, eps;
  const void *r, *f, *w_post, *w_pre, *gate;
  void *out, *n;                       // forward
  const void *u, *v;                   // backward: gradients of r' and n
  void *dr, *df, *d_gate;
  float *part_post, *part_pre, *part_gate;  // fp32 partial sums over tokens, [parts][H]
  // a piece: up to piece_rows consecutive tokens of one gate group; a block takes pieces
  // blockIdx.x, + gridDim.x, ...
  int64_t pieces, pieces_per_group, piece_rows, group_rows;
};

// Block sum of N values; red: 2 buffers of 32 * N floats, `flip` alternates between calls so that
// one barrier per call suffices (a thread may enter the next call while others still read).
template <int N>
__device__ __forceinline__ void block_sum(float (&v)[N], float* red, int flip) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = (blockDim.x + 31) >> 5;
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = warp_sum(v[i]);
  if (warps == 1) return;
  float* buf = red + flip * 32 * N;
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) buf[warp * N + i] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = warp_sum(lane < warps ? buf[lane * N + i] : 0.f);
}

// One row per block. W: elements per load (8: 16-byte words of bf16), NV loads per thread.
template <typename ST, typename BT, int W, int NV>
__global__ void __launch_bounds__(1024) k_norm_fwd(NormArgs a) {
  __shared__ float red[2 * 32];
  pdl_wait();
  const int64_t t = blockIdx.x;
  const int H = a.H;
  const ST* r = static_cast<const ST*>(a.r) + t * H;
  const BT* f = static_cast<const BT*>(a.f) + t * H;
  float x[NV][W], y[NV][W], sum[1] = {0.f};
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (j * (int)blockDim.x + (int)threadIdx.x) * W;
#pragma unroll
    for (int i = 0; i < W; ++i) x[j][i] = y[j][i] = 0.f;
    if (c >= H) continue;
    load_vec<W>(r + c, x[j]);
    if (a.f != nullptr) load_vec<W>(f + c, y[j]);
#pragma unroll
    for (int i = 0; i < W; ++i) sum[0] += y[j][i] * y[j][i];
  }
  float s = 1.f;
  if (a.w_post != nullptr) {
    block_sum<1>(sum, red, 0);
    s = rsqrtf(sum[0] / (float)H + a.eps);
  }
  const int64_t grow = a.rows_per_gate > 0 ? t / a.rows_per_gate * H : 0;
  sum[0] = 0.f;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (j * (int)blockDim.x + (int)threadIdx.x) * W;
    if (c >= H) continue;
    if (a.w_post != nullptr) {
      float w[W];
      load_any<W>(a.w_post, a.ptype, c, w);
#pragma unroll
      for (int i = 0; i < W; ++i) y[j][i] *= s * w[i];
    }
    if (a.gate != nullptr) {
      float g[W];
      load_any<W>(a.gate, a.ptype, grow + c, g);
#pragma unroll
      for (int i = 0; i < W; ++i) y[j][i] *= g[i];
    }
#pragma unroll
    for (int i = 0; i < W; ++i) {
      x[j][i] = a.scale * x[j][i] + y[j][i];
      sum[0] += x[j][i] * x[j][i];
    }
    if (a.out != nullptr) store_vec<W>(static_cast<ST*>(a.out) + t * H + c, x[j]);
  }
  if (a.w_pre == nullptr) return;
  block_sum<1>(sum, red, 1);
  const float q = rsqrtf(sum[0] / (float)H + a.eps);
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (j * (int)blockDim.x + (int)threadIdx.x) * W;
    if (c >= H) continue;
    float w[W];
    load_any<W>(a.w_pre, a.ptype, c, w);
#pragma unroll
    for (int i = 0; i < W; ++i) x[j][i] *= q * w[i];
    store_vec<W>(static_cast<BT*>(a.n) + t * H + c, x[j]);
  }
}

// A block walks its pieces row by row; the three parameter gradients of its columns stay in
// registers until the block (weights) or the piece (gate) ends.
template <typename ST, typename BT, int W, int NV>
__global__ void __launch_bounds__(1024) k_norm_bwd(NormArgs a) {
  __shared__ float red[2 * 32 * 6];
  pdl_wait();
  const int H = a.H;
  const bool post = a.w_post != nullptr, pre = a.w_pre != nullptr, gated = a.gate != nullptr;
  float d_post[NV][W], d_pre[NV][W], d_gate[NV][W];
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < W; ++i) d_post[j][i] = d_pre[j][i] = d_gate[j][i] = 0.f;
  int flip = 0;
  for (int64_t piece = blockIdx.x; piece < a.pieces; piece += gridDim.x) {
    const int64_t group = piece / a.pieces_per_group;
    const int64_t first = (piece - group * a.pieces_per_group) * a.piece_rows;
    const int64_t t0 = group * a.group_rows + first;
    const int64_t t1 = group * a.group_rows + min(first + a.piece_rows, a.group_rows);
    for (int64_t t = t0; t < t1; ++t, flip ^= 1) {
      float x[NV][W], f[NV][W], u[NV][W], v[NV][W], e[NV][W], g[NV][W];
      float sum[6] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = (j * (int)blockDim.x + (int)threadIdx.x) * W;
#pragma unroll
        for (int i = 0; i < W; ++i) {
          x[j][i] = f[j][i] = u[j][i] = v[j][i] = 0.f;
          e[j][i] = g[j][i] = 1.f;
        }
        if (c >= H) continue;
        load_vec<W>(static_cast<const ST*>(a.r) + t * H + c, x[j]);
        if (a.f != nullptr) load_vec<W>(static_cast<const BT*>(a.f) + t * H + c, f[j]);
        if (a.u != nullptr) load_vec<W>(static_cast<const ST*>(a.u) + t * H + c, u[j]);
        if (pre) {
          float w[W];
          load_vec<W>(static_cast<const BT*>(a.v) + t * H + c, v[j]);
          load_any<W>(a.w_pre, a.ptype, c, w);
#pragma unroll
          for (int i = 0; i < W; ++i) {
            const float wv = w[i] * v[j][i];
            sum[0] += x[j][i] * x[j][i];
            sum[1] += wv * x[j][i];
          }
        }
        if (gated) load_any<W>(a.gate, a.ptype, group * H + c, g[j]);
        if (post) {
          float w[W], wp[W];
          load_any<W>(a.w_post, a.ptype, c, w);
          if (pre) load_any<W>(a.w_pre, a.ptype, c, wp);
#pragma unroll
          for (int i = 0; i < W; ++i) {
            e[j][i] = w[i] * g[j][i];
            const float ef = e[j][i] * f[j][i];
            sum[2] += f[j][i] * f[j][i];
            sum[3] += ef * u[j][i];
            if (pre) sum[4] += ef * wp[i] * v[j][i];
            sum[5] += ef * x[j][i];
          }
        }
      }
      if (pre || post) block_sum<6>(sum, red, flip);
      const float rh = 1.f / (float)H;
      const float q = pre ? rsqrtf(sum[0] * rh + a.eps) : 0.f;
      const float cq = q * q * q * rh * sum[1];
      const float s = post ? rsqrtf(sum[2] * rh + a.eps) : 1.f;
      const float cs = s * s * s * rh * (pre ? sum[3] + q * sum[4] - cq * sum[5] : sum[3]);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = (j * (int)blockDim.x + (int)threadIdx.x) * W;
        if (c >= H) continue;
        float w[W], wq[W], dr[W], df[W];
#pragma unroll
        for (int i = 0; i < W; ++i) w[i] = 1.f, wq[i] = 0.f;
        if (post) load_any<W>(a.w_post, a.ptype, c, w);
        if (pre) load_any<W>(a.w_pre, a.ptype, c, wq);
#pragma unroll
        for (int i = 0; i < W; ++i) {
          const float d = pre ? u[j][i] + q * (wq[i] * v[j][i]) - cq * x[j][i] : u[j][i];
          const float sf = s * f[j][i];
          dr[i] = a.scale * d;
          d_pre[j][i] += v[j][i] * x[j][i] * q;
          d_gate[j][i] += d * (w[i] * sf);
          d_post[j][i] += g[j][i] * d * sf;
          df[i] = post ? s * (e[j][i] * d) - cs * f[j][i] : g[j][i] * d;
        }
        store_vec<W>(static_cast<ST*>(a.dr) + t * H + c, dr);
        if (a.df != nullptr) store_vec<W>(static_cast<BT*>(a.df) + t * H + c, df);
      }
    }
    if (gated) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = (j * (int)blockDim.x + (int)threadIdx.x) * W;
        if (c < H) {
          if (a.part_gate != nullptr)
            store_vec<W>(a.part_gate + piece * H + c, d_gate[j]);
          else
            store_any<W>(a.d_gate, a.ptype, group * H + c, d_gate[j]);
        }
#pragma unroll
        for (int i = 0; i < W; ++i) d_gate[j][i] = 0.f;
      }
    }
  }
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (j * (int)blockDim.x + (int)threadIdx.x) * W;
    if (c >= H) continue;
    if (post) store_vec<W>(a.part_post + (int64_t)blockIdx.x * H + c, d_post[j]);
    if (pre) store_vec<W>(a.part_pre + (int64_t)blockIdx.x * H + c, d_pre[j]);
  }
}

inline bool aligned_to(const void* p, size_t a) {
  return (reinterpret_cast<uintptr_t>(p) % a) == 0;
}

inline size_t type_size(int t) { return t == MM_BF16 ? 2 : 4; }
inline bool type_ok(int t) { return t == MM_BF16 || t == MM_FP32; }

mm_status check_desc(const mm_norm_desc* d) {
  if (d == nullptr || d->T < 0 || d->H < 1 || d->groups < 0) return MM_ERR_INVALID_ARG;
  if (!type_ok(d->stream_type) || !type_ok(d->block_type) || !type_ok(d->param_type) ||
      (d->stream_type == MM_BF16 && d->block_type == MM_FP32))
    return MM_ERR_INVALID_ARG;
  if (d->groups > 0 && d->T % d->groups != 0) return MM_ERR_INVALID_ARG;
  if (!(d->eps >= 0.f) || !isfinite(d->eps)) return MM_ERR_INVALID_ARG;
  if (d->H > kMaxH || d->T >= ((int64_t)1 << 31)) return MM_ERR_UNSUPPORTED;
  return MM_OK;
}

// How the backward's tokens are dealt to blocks.
struct BwdPlan {
  int64_t group_rows, piece_rows, pieces_per_group, pieces, blocks;
  size_t off_post, off_pre, off_gate, total;
};

BwdPlan plan_bwd(const mm_norm_desc& d, int sms) {
  BwdPlan p{};
  const int64_t groups = std::max<int64_t>(1, d.groups);
  const int64_t target = (int64_t)sms * 2;
  p.group_rows = d.T / groups;
  p.piece_rows = std::max<int64_t>(1, std::min(p.group_rows, (d.T + target - 1) / target));
  p.pieces_per_group = (p.group_rows + p.piece_rows - 1) / p.piece_rows;
  p.pieces = groups * p.pieces_per_group;
  p.blocks = std::min(p.pieces, target);
  const size_t slice = ((size_t)d.H * 4 + 255) / 256 * 256;
  p.off_post = 0;
  p.off_pre = slice * (size_t)p.blocks;
  p.off_gate = 2 * slice * (size_t)p.blocks;
  p.total = p.off_gate +
            (d.groups > 0 && p.pieces_per_group > 1 ? slice * (size_t)p.pieces : 0);
  return p;
}

// Rows that can move as 16-byte words.
bool wide(const mm_norm_desc& d, std::initializer_list<const void*> ptrs) {
  if (d.H % 8) return false;
  for (const void* p : ptrs)
    if (!aligned_to(p, 16)) return false;
  return true;
}

bool elements_aligned(size_t size, std::initializer_list<const void*> ptrs) {
  for (const void* p : ptrs)
    if (!aligned_to(p, size)) return false;
  return true;
}

inline int threads_for(int64_t H, int per_thread) {
  return (int)std::min<int64_t>(1024, ((H + per_thread - 1) / per_thread + 31) / 32 * 32);
}

template <typename ST, typename BT>
cudaError_t launch_fwd(const NormArgs& a, bool w8, cudaStream_t st) {
  const dim3 grid((unsigned)a.T);
  if (w8 && a.H <= 8192)
    return launch_pdl(k_norm_fwd<ST, BT, 8, 1>, grid, dim3(threads_for(a.H, 8)), 0, st, a);
  if (w8) return launch_pdl(k_norm_fwd<ST, BT, 8, 2>, grid, dim3(threads_for(a.H, 16)), 0, st, a);
  if (a.H <= 4096)
    return launch_pdl(k_norm_fwd<ST, BT, 1, 4>, grid, dim3(threads_for(a.H, 4)), 0, st, a);
  return launch_pdl(k_norm_fwd<ST, BT, 1, 16>, grid, dim3(threads_for(a.H, 16)), 0, st, a);
}

template <typename ST, typename BT>
cudaError_t launch_bwd(const NormArgs& a, int64_t blocks, bool w8, cudaStream_t st) {
  const dim3 grid((unsigned)blocks);
  if (w8 && a.H <= 8192)
    return launch_pdl(k_norm_bwd<ST, BT, 8, 1>, grid, dim3(threads_for(a.H, 8)), 0, st, a);
  if (w8) return launch_pdl(k_norm_bwd<ST, BT, 8, 2>, grid, dim3(threads_for(a.H, 16)), 0, st, a);
  if (a.H <= 4096)
    return launch_pdl(k_norm_bwd<ST, BT, 1, 4>, grid, dim3(threads_for(a.H, 4)), 0, st, a);
  return launch_pdl(k_norm_bwd<ST, BT, 1, 16>, grid, dim3(threads_for(a.H, 16)), 0, st, a);
}

NormArgs norm_args(const mm_norm_desc& d) {
  NormArgs a{};
  a.T = d.T;
  a.H = (int)d.H;
  a.ptype = d.param_type;
  a.scale = d.residual_scale;
  a.eps = d.eps;
  a.rows_per_gate = d.groups > 0 ? d.T / d.groups : 0;
  return a;
}

}  // namespace
}  // namespace mm

using namespace mm;

extern "C" {

int mm_ops_version(void) { return 1; }

mm_status mm_residual_norm_forward(const mm_norm_desc* d, const void* residual, const void* branch,
                                   const void* post_weight, const void* pre_weight,
                                   const void* gate, void* residual_out, void* normed,
                                   void* stream) {
  mm_status s = check_desc(d);
  if (s != MM_OK) return s;
  if (d->T == 0) return MM_OK;
  if (residual == nullptr || (d->groups > 0) != (gate != nullptr) ||
      (pre_weight != nullptr) != (normed != nullptr) ||
      (branch == nullptr && (post_weight != nullptr || gate != nullptr)))
    return MM_ERR_INVALID_ARG;
  if (!elements_aligned(type_size(d->stream_type), {residual, residual_out}) ||
      !elements_aligned(type_size(d->block_type), {branch, normed}) ||
      !elements_aligned(type_size(d->param_type), {post_weight, pre_weight, gate}))
    return MM_ERR_INVALID_ARG;
  if (residual_out == nullptr && normed == nullptr) return MM_OK;
  clear_error();
  NormArgs a = norm_args(*d);
  a.r = residual;
  a.f = branch;
  a.w_post = post_weight;
  a.w_pre = pre_weight;
  a.gate = gate;
  a.out = residual_out;
  a.n = normed;
  const bool w8 =
      wide(*d, {residual, branch, post_weight, pre_weight, gate, residual_out, normed});
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (d->stream_type == MM_BF16)
    MM_TRY((launch_fwd<__nv_bfloat16, __nv_bfloat16>(a, w8, st)));
  else if (d->block_type == MM_BF16)
    MM_TRY((launch_fwd<float, __nv_bfloat16>(a, w8, st)));
  else
    MM_TRY((launch_fwd<float, float>(a, w8, st)));
  return MM_OK;
}

size_t mm_residual_norm_workspace_size(const mm_norm_desc* d) {
  if (check_desc(d) != MM_OK) return 0;
  return std::max<size_t>(256, plan_bwd(*d, std::max(1, device_sm_count())).total);
}

mm_status mm_residual_norm_backward(const mm_norm_desc* d, const void* residual_out,
                                    const void* branch, const void* post_weight,
                                    const void* pre_weight, const void* gate,
                                    const void* d_residual_out, const void* d_normed,
                                    void* d_residual, void* d_branch, void* d_post_weight,
                                    void* d_pre_weight, void* d_gate, void* workspace,
                                    size_t workspace_bytes, void* stream) {
  mm_status s = check_desc(d);
  if (s != MM_OK) return s;
  if ((d->groups > 0) != (gate != nullptr) || (gate != nullptr) != (d_gate != nullptr) ||
      (post_weight != nullptr) != (d_post_weight != nullptr) ||
      (pre_weight != nullptr) != (d_pre_weight != nullptr))
    return MM_ERR_INVALID_ARG;
  if (!elements_aligned(type_size(d->stream_type), {residual_out, d_residual_out, d_residual}) ||
      !elements_aligned(type_size(d->block_type), {branch, d_normed, d_branch}) ||
      !elements_aligned(type_size(d->param_type),
                        {post_weight, pre_weight, gate, d_post_weight, d_pre_weight, d_gate}))
    return MM_ERR_INVALID_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const size_t ps = type_size(d->param_type);
  if (d->T == 0) {  // no token: the parameter gradients are sums of nothing
    clear_error();
    if (d_post_weight) MM_TRY(cudaMemsetAsync(d_post_weight, 0, d->H * ps, st));
    if (d_pre_weight) MM_TRY(cudaMemsetAsync(d_pre_weight, 0, d->H * ps, st));
    if (d_gate) MM_TRY(cudaMemsetAsync(d_gate, 0, d->groups * d->H * ps, st));
    return MM_OK;
  }
  if (residual_out == nullptr || d_residual == nullptr ||
      (pre_weight != nullptr) != (d_normed != nullptr) ||
      (branch != nullptr) != (d_branch != nullptr) ||
      (branch == nullptr && (post_weight != nullptr || gate != nullptr)) ||
      (d_residual_out == nullptr && d_normed == nullptr))
    return MM_ERR_INVALID_ARG;
  clear_error();
  const BwdPlan p = plan_bwd(*d, std::max(1, device_sm_count()));
  if (workspace == nullptr || !aligned_to(workspace, 256) || workspace_bytes < p.total)
    return MM_ERR_WORKSPACE;
  char* ws = static_cast<char*>(workspace);
  NormArgs a = norm_args(*d);
  a.r = residual_out;
  a.f = branch;
  a.w_post = post_weight;
  a.w_pre = pre_weight;
  a.gate = gate;
  a.u = d_residual_out;
  a.v = d_normed;
  a.dr = d_residual;
  a.df = d_branch;
  a.d_gate = d_gate;
  a.part_post = reinterpret_cast<float*>(ws + p.off_post);
  a.part_pre = reinterpret_cast<float*>(ws + p.off_pre);
  const bool gate_parts = gate != nullptr && p.pieces_per_group > 1;
  a.part_gate = gate_parts ? reinterpret_cast<float*>(ws + p.off_gate) : nullptr;
  a.pieces = p.pieces;
  a.pieces_per_group = p.pieces_per_group;
  a.piece_rows = p.piece_rows;
  a.group_rows = p.group_rows;
  const bool w8 = wide(*d, {residual_out, branch, post_weight, pre_weight, gate, d_residual_out,
                            d_normed, d_residual, d_branch, d_gate});
  if (d->stream_type == MM_BF16)
    MM_TRY((launch_bwd<__nv_bfloat16, __nv_bfloat16>(a, p.blocks, w8, st)));
  else if (d->block_type == MM_BF16)
    MM_TRY((launch_bwd<float, __nv_bfloat16>(a, p.blocks, w8, st)));
  else
    MM_TRY((launch_bwd<float, float>(a, p.blocks, w8, st)));
  SumArgs sa{};
  sa.cols = (int)d->H;
  sa.type = d->param_type;
  int64_t rows = 0;
  auto add = [&](const float* src, void* dst, int64_t parts, int64_t n) {
    sa.job[sa.jobs++] = SumJob{src, dst, parts, rows};
    rows += n;
  };
  if (d_post_weight) add(a.part_post, d_post_weight, p.blocks, 1);
  if (d_pre_weight) add(a.part_pre, d_pre_weight, p.blocks, 1);
  if (gate_parts) add(a.part_gate, d_gate, p.pieces_per_group, d->groups);
  if (rows > 0)
    MM_TRY(launch_column_sums(sa, rows, st));
  return MM_OK;
}

}  // extern "C"
