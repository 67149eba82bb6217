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
// kernels are bound by HBM.
//
// Two forms. Many rows: persistent blocks, 16 columns per thread, whose
// rows arrive by bulk copies into a ring in shared memory several rows ahead, so that HBM stays
// busy through the reductions; weights and the backward's column sums stay in registers
// (k_norm_fwd_rows, k_norm_bwd_rows). Few rows, widths above 7680 and tensors off 16-byte
// boundaries: a row in registers straight from global memory (k_norm_fwd, k_norm_bwd).
//
// Measured, bf16, device time of a call: forward 4096 x 7168 40.5 us, 5.8 TB/s (82 us with a row per
// block); 16384 x 2048 47.1 us, 5.7 TB/s; one row of 2048 2.6 us. Backward 16384 x 2048 73.5 us, 5.5
// TB/s (318 us with a row per block and sums by columns): 66 us for the rows, the rest for the sums of
// 456 blocks' columns; 4096 x 7168 68 us, 5.2 TB/s. fp32 1000 x 2047 23.3 us, 2.1 TB/s: 20 us for the
// rows of 144 blocks, seven each and one after another, 2.8 us a row of single-element loads; then the
// sums' launch.
//
// What spills (ptxas): k_norm_bwd at widths above 7680 or tensors off 16-byte boundaries, 0.6 KB a thread
// up to 8192 and 2.2 to 3.1 KB above in 8-column words (1024 threads leave 64 registers a thread and 32
// column sums beside the row), 1.6 KB in single columns above 4096; it is the form for what the rows'
// ring does not take (4096 x 8192 backward 278 us, floor 59). k_norm_bwd_rows with a part left out
// spills 64 to 180 bytes for its tests (16384 x 2048 without post norm and gate 147 us).
#include <cuda_runtime.h>
#include <math.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "../../include/mm_ops.h"
#include "mm_kernels.h"
#include "mm_rows.cuh"

namespace mm {
namespace {

constexpr int kMaxH = 16384;
constexpr int kMaxRingH = 7680;  // 15 warps of 16 columns per thread (odd rows: 8)

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
  uint64_t timeout_ns;  // of a row's arrival (row rings)
  int stall;            // test hook: block 0's loading warp stops after its first row
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

// A norm's backward takes q^3 / H <.., r'> r' off a row, q = 1 / rms: here the factor of q r', which is
// of unit size as q <.., r'> is of the other factor's. q^3 by itself leaves the range of 32 bits for
// rows of 1e13 (or, with no eps, 1e-13).
__device__ __forceinline__ float unit_factor(float q, float rh, float dot) {
  return (q * rh) * (q * dot);
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
      const float cq = unit_factor(q, rh, sum[1]);
      const float s = post ? rsqrtf(sum[2] * rh + a.eps) : 1.f;
      const float cs = unit_factor(s, rh, pre ? sum[3] + q * sum[4] - cq * (q * sum[5]) : sum[3]);
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
          const float xq = q * x[j][i], sf = s * f[j][i];
          const float d = pre ? u[j][i] + q * (wq[i] * v[j][i]) - cq * xq : u[j][i];
          dr[i] = a.scale * d;
          d_pre[j][i] += v[j][i] * xq;
          d_gate[j][i] += d * (w[i] * sf);
          d_post[j][i] += g[j][i] * d * sf;
          df[i] = post ? s * (e[j][i] * d) - cs * sf : g[j][i] * d;
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

// ---------------------------------------------------------------------------------- row rings

// A stage holds one row of each tensor in use; offsets in bytes, -1: not in use.
struct RowRing {
  int x, f, u, v, g;  // residual (forward: r, backward: r'), branch, the two gradients, gate
  int bytes, depth, odd, tail;  // odd: single elements (see Columns); tail: bytes behind the stages (the backward's sums of d_post)
};

// The rows of a block, piece after piece (see NormArgs).
struct RowWalk {
  int64_t piece, group, t, t1;
  __device__ __forceinline__ void start(const NormArgs& a, int64_t p) {
    piece = p;
    if (p >= a.pieces) return;
    group = a.pieces_per_group == 1 ? p : p / a.pieces_per_group;
    const int64_t first = (p - group * a.pieces_per_group) * a.piece_rows;
    t = group * a.group_rows + first;
    t1 = group * a.group_rows + min(first + a.piece_rows, a.group_rows);
  }
  __device__ __forceinline__ bool more(const NormArgs& a) const { return piece < a.pieces; }
  __device__ __forceinline__ void next(const NormArgs& a) {
    if (++t == t1) start(a, piece + gridDim.x);
  }
};

// ODD rows start off a 16-byte boundary: their copies run from the boundary before to the one
// after (the last row's, to the last one within the tensor: what is left of it, under 16 bytes, the
// loading warp copies itself), and a thread works on single elements, `threads` apart, instead of
// 8 together. Both hold a thread's columns as kVecs x 4 pairs.
struct Span {  // of a row's bytes that are copied
  int64_t from;
  uint32_t bytes;
};
template <bool ODD>
__device__ __forceinline__ Span row_span(int64_t row, int64_t rows, uint32_t row_bytes) {
  const int64_t start = row * row_bytes;
  if (!ODD) return Span{start, row_bytes};
  const int64_t end = min((start + row_bytes + 15) & ~15ll, rows * row_bytes & ~15ll);
  return Span{start & ~15ll, (uint32_t)(end - (start & ~15ll))};
}

// Address of a row's first element in its stage.
template <bool ODD>
__device__ __forceinline__ uint32_t row_at(uint32_t stage, int offset, int64_t row,
                                           uint32_t row_bytes) {
  return stage + offset + (ODD ? (uint32_t)(row * row_bytes) & 15u : 0u);
}

template <bool ODD>
struct Columns {
  int H, threads;
  __device__ __forceinline__ int first(int k) const {
    return ODD ? (int)threadIdx.x + 8 * k * threads : ((int)threadIdx.x + k * threads) * 8;
  }
  __device__ __forceinline__ bool any(int k) const { return first(k) < H; }
  // f(pair, half, column) for every column of group k (ODD)
  template <typename F>
  __device__ __forceinline__ void each(int k, F&& f) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = first(k) + i * threads;
      f(i, c);
    }
  }
  template <typename F>
  __device__ __forceinline__ void gather(int k, f32x2 (&v)[4], F&& value) const {
    float e[8];
    each(k, [&](int i, int c) { e[i] = c < H ? value(c) : 0.f; });
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = pair(e[2 * i], e[2 * i + 1]);
  }
  // from a row in its stage
  template <typename T>
  __device__ __forceinline__ void stage(uint32_t row, int k, f32x2 (&v)[4]) const {
    if constexpr (ODD) {
      gather(k, v, [&](int c) {
        const uint32_t at = row + c * (uint32_t)sizeof(T);
        if constexpr (sizeof(T) == 2) {
          uint16_t w;
          asm volatile("ld.shared.u16 %0, [%1];" : "=h"(w) : "r"(at));
          return __uint_as_float((uint32_t)w << 16);
        } else {
          float w;
          asm volatile("ld.shared.f32 %0, [%1];" : "=f"(w) : "r"(at));
          return w;
        }
      });
    } else {
      lds_pairs<T>(row + first(k) * (uint32_t)sizeof(T), v);
    }
  }
  // from and to rows in global (or, as floats, shared) memory
  template <typename T>
  __device__ __forceinline__ void load(const T* row, int k, f32x2 (&v)[4]) const {
    if constexpr (ODD)
      gather(k, v, [&](int c) { return element(row[c]); });
    else
      load_pairs(row + first(k), v);
  }
  template <typename T>
  __device__ __forceinline__ void store(T* row, int k, const f32x2 (&v)[4]) const {
    if constexpr (ODD) {
      float e[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) split(v[i], e[2 * i], e[2 * i + 1]);
      each(k, [&](int i, int c) {
        if (c < H) put(row + c, e[i]);
      });
    } else {
      store_pairs(row + first(k), v);
    }
  }
  static __device__ __forceinline__ float element(__nv_bfloat16 v) { return __bfloat162float(v); }
  static __device__ __forceinline__ float element(float v) { return v; }
  static __device__ __forceinline__ void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
  static __device__ __forceinline__ void put(float* p, float v) { *p = v; }
};

// One warp: the copies of row t into a stage.
template <typename ST, typename BT, typename PT, bool ODD>
__device__ __forceinline__ void load_row(const NormArgs& a, const RowRing& r, uint32_t stage,
                                         uint32_t bar, int64_t t) {
  const Span ss = row_span<ODD>(t, a.T, a.H * sizeof(ST)), bs = row_span<ODD>(t, a.T, a.H * sizeof(BT));
  Span ps{0, 0};
  const bool last = t + 1 == a.T;
  bool last_gate = false;  // the gate's last row serves several
  if (r.g >= 0) {
    const int64_t gate = t / a.rows_per_gate, gates = a.T / a.rows_per_gate;
    ps = row_span<ODD>(gate, gates, a.H * sizeof(PT));
    last_gate = gate + 1 == gates;
  }
  const int lane = threadIdx.x & 31;
  if (ODD && (last || last_gate)) {  // what the copies leave out, up to 7 words of each tensor
    auto rest = [&](int at, bool use, int offset, const void* base, const Span& span, int64_t total) {
      const int64_t i = span.from + span.bytes + 2 * (lane & 7);
      if (use && offset >= 0 && (lane >> 3) == at && i < total)
        asm volatile("st.shared.u16 [%0], %1;" ::"r"(stage + offset + (uint32_t)(i - span.from)),
                     "h"(*reinterpret_cast<const uint16_t*>(static_cast<const char*>(base) + i))
                     : "memory");
    };
    rest(0, last, r.x, a.r, ss, a.T * a.H * sizeof(ST));
    rest(1, last, r.f, a.f, bs, a.T * a.H * sizeof(BT));
    rest(2, last, r.u, a.u, ss, a.T * a.H * sizeof(ST));
    rest(3, last, r.v, a.v, bs, a.T * a.H * sizeof(BT));
    rest(0, last_gate, r.g, a.gate, ps, r.g >= 0 ? a.T / a.rows_per_gate * a.H * sizeof(PT) : 0);
    __syncwarp();
  }
  if (lane != 0) return;
  mbar_arrive_expect_tx(bar, (r.x >= 0 ? ss.bytes : 0) + (r.f >= 0 ? bs.bytes : 0) +
                                 (r.u >= 0 ? ss.bytes : 0) + (r.v >= 0 ? bs.bytes : 0) + ps.bytes);
  auto copy = [&](int offset, const void* base, const Span& span) {
    if (offset >= 0) bulk_load(stage + offset, static_cast<const char*>(base) + span.from, span.bytes, bar);
  };
  copy(r.x, a.r, ss);
  copy(r.f, a.f, bs);
  copy(r.u, a.u, ss);
  copy(r.v, a.v, bs);
  copy(r.g, a.gate, ps);
}

// A row kernel's last warp issues the copies (a stage's cost hundreds of cycles, which in one of
// the working warps every row would wait for); the others work on the rows and meet at a barrier
// of their own.
__device__ __forceinline__ void row_barrier(int threads) {
  asm volatile("bar.sync 1, %0;" ::"r"(threads) : "memory");
}

// Row loads are this library's own copies from memory that the launch was given: the wait for one
// cannot run out unless the device has failed. It is bounded all the same, and then shows: a thread
// whose wait ran out (kLost, beside the parity that it would wait for next) waits no more, hands no
// stage back and puts NaN into the row's sums (or, without any, in the place of what it would have
// read), so its block's remaining rows and column sums are NaN. A loading warp that gets no stage back
// issues no further copy.
constexpr uint64_t kRowTimeoutNs = 2000000000ull, kTestTimeoutNs = 50000000ull;
constexpr uint32_t kLost = 2;

__device__ __forceinline__ void await_row(uint32_t bar, uint32_t& ph, uint64_t limit_ns) {
  if (ph < kLost && !mbar_wait(bar, ph, limit_ns)) ph |= kLost;
}

__device__ __forceinline__ f32x2 nan_pair() { return both(__int_as_float(0x7FC00000)); }

// Sum over the block: partial sums of the warps in `red` (32 floats, zero beyond the block's
// warps), read back by every thread.
__device__ __forceinline__ float block_sum_1(float v, float* red, int threads) {
  v = warp_sum(v);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  row_barrier(threads);
  const float4* r4 = reinterpret_cast<const float4*>(red);
  float s = 0.f;
#pragma unroll 4
  for (int i = 0; i < (threads + 127) / 128; ++i) {
    const float4 p = r4[i];
    s += (p.x + p.y) + (p.z + p.w);
  }
  return s;
}

template <typename ST, typename BT, typename PT, bool ODD>
__device__ __forceinline__ void produce_rows(const NormArgs& a, const RowRing& ring, uint32_t smem,
                                             uint32_t full, uint32_t empty) {
  RowWalk row;
  row.start(a, blockIdx.x);
  int s = 0;
  uint32_t ph = 1;
  bool stop = false;
  while (row.more(a)) {
    const bool free_stage = mbar_wait(empty + 8u * s, ph, a.timeout_ns);
    if (!__all_sync(0xFFFFFFFFu, free_stage) || stop) break;
    load_row<ST, BT, PT, ODD>(a, ring, smem + s * ring.bytes, full + 8u * s, row.t);
    row.next(a);
    stop = a.stall && blockIdx.x == 0;
    if (++s == ring.depth) s = 0, ph ^= 1u;
  }
  // no block leaves with a copy into its shared memory in flight: the stages before s had their last
  // one in this turn of the ring, the others (if any) in the turn before
  for (int i = 0; i < ring.depth; ++i) mbar_wait(full + 8u * i, i < s ? ph ^ 1u : ph, a.timeout_ns);
}

// FULL: every part is there (branch, both norms, both upstream gradients; OWN: and a gate that comes
// with its row), which takes the tests for the parts out of the loop.
//
// What a thread does per row is the same for 8 columns as for 16 but for the columns themselves:
// with 8, and single floats, 52 instructions went into an element of the forward, and the issue
// slots ran out at 3.6 TB/s. A thread has columns 8 tid .. and 8 (tid + threads) ..; the loop works
// on pairs of floats.
// ODD rows: 8 columns, whose addresses and masks are their own.
constexpr int kRowThreads = 512;  // at most, the loading warp included
template <bool ODD>
struct Shape {
  static constexpr int VECS = ODD ? 1 : 2;
};

template <typename ST, typename BT, typename PT, bool FULL, bool ODD, bool OWN>
__global__ void __launch_bounds__(kRowThreads) k_norm_fwd_rows(NormArgs a, RowRing ring) {
  constexpr int kVecs = Shape<ODD>::VECS;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(16) float red[2][32];
  __shared__ uint64_t bars[16];
  const int tid = threadIdx.x, H = a.H, threads = blockDim.x - 32;
  const Columns<ODD> cols{H, threads};
  const bool post = FULL || a.w_post != nullptr, pre = FULL || a.w_pre != nullptr;
  if (tid < 64) red[tid >> 5][tid & 31] = 0.f;
  if (tid == 0) {
    for (int i = 0; i < ring.depth; ++i) {
      mbar_init(smem_u32(&bars[i]), 1);
      mbar_init(smem_u32(&bars[8 + i]), threads / 32);
    }
    mbar_fence_init();
  }
  __syncthreads();
  pdl_wait();
  if (tid >= threads) {
    produce_rows<ST, BT, PT, ODD>(a, ring, smem_u32(smem), smem_u32(bars), smem_u32(bars + 8));
    return;
  }
  const bool own_gate = FULL ? OWN : ring.g >= 0;  // the gate comes with the row
  RowWalk row;
  row.start(a, blockIdx.x);
  // weights: of the branch (times the gate, where that is the same for many rows) and of the norm
  f32x2 wb[kVecs][4], wn[kVecs][4];
  auto branch_weights = [&](int64_t group) {
#pragma unroll
    for (int k = 0; k < kVecs; ++k) {
      f32x2 g[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) wb[k][i] = both(1.f);
      if (!cols.any(k)) continue;
      if (post) cols.load(static_cast<const PT*>(a.w_post), k, wb[k]);
      if (a.gate != nullptr && !own_gate) {
        cols.load(static_cast<const PT*>(a.gate) + group * H, k, g);
#pragma unroll
        for (int i = 0; i < 4; ++i) wb[k][i] = mul(wb[k][i], g[i]);
      }
    }
  };
#pragma unroll
  for (int k = 0; k < kVecs; ++k) {
#pragma unroll
    for (int i = 0; i < 4; ++i) wn[k][i] = both(1.f);
    if (pre && cols.any(k)) cols.load(static_cast<const PT*>(a.w_pre), k, wn[k]);
  }
  if (row.more(a)) branch_weights(row.group);
  int64_t group = row.group;
  int s = 0, flip = 0;
  uint32_t ph = 0;
  const float rh = 1.f / (float)H;
  const f32x2 scale = both(a.scale);
  while (row.more(a)) {
    const uint32_t stage = smem_u32(smem) + s * ring.bytes;
    if (a.gate != nullptr && !own_gate && row.group != group) branch_weights(group = row.group);
    await_row(smem_u32(&bars[s]), ph, a.timeout_ns);
    f32x2 x[kVecs][4], y[kVecs][4], acc = both(0.f);
    const uint32_t xr = row_at<ODD>(stage, ring.x, row.t, H * sizeof(ST));
    const uint32_t fr = row_at<ODD>(stage, ring.f, row.t, H * sizeof(BT));
#pragma unroll
    for (int k = 0; k < kVecs; ++k) {
      if (!cols.any(k)) continue;
      cols.template stage<ST>(xr, k, x[k]);
      if (FULL || ring.f >= 0) {
        cols.template stage<BT>(fr, k, y[k]);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) y[k][i] = both(0.f);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) acc = fma(y[k][i], y[k][i], acc);
      if (!post && ph >= kLost) {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[k][i] = nan_pair();
      }
    }
    if (post && ph >= kLost) acc = nan_pair();
    f32x2 q = both(1.f);
    // Two sums a row take a buffer each, so that each one's barrier separates the other buffer's reads
    // from its next use; a row's only sum takes them in turn, for the next row's barrier to do it.
    if (post)
      q = both(rsqrtf(block_sum_1(sum_of(acc), red[pre ? 0 : flip], threads) * rh + a.eps));
    acc = both(0.f);
    const int64_t at = row.t * H;
#pragma unroll
    for (int k = 0; k < kVecs; ++k) {
      if (!cols.any(k)) continue;
      if (own_gate) {
        f32x2 g[4];
        const int64_t gate_row = row.t / a.rows_per_gate;
        cols.template stage<PT>(row_at<ODD>(stage, ring.g, gate_row, H * sizeof(PT)), k, g);
#pragma unroll
        for (int i = 0; i < 4; ++i) y[k][i] = mul(y[k][i], g[i]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[k][i] = fma(mul(q, y[k][i]), wb[k][i], mul(scale, x[k][i]));
        acc = fma(x[k][i], x[k][i], acc);
      }
      if (FULL || a.out != nullptr) cols.store(static_cast<ST*>(a.out) + at, k, x[k]);
    }
    __syncwarp();
    if ((tid & 31) == 0 && ph < kLost) mbar_arrive(smem_u32(&bars[8 + s]));  // the stage is read
    float sum = 0.f;
    if (pre)
      sum = block_sum_1(sum_of(acc), red[post ? 1 : flip], threads);
    if (pre) {
      q = both(rsqrtf(sum * rh + a.eps));
#pragma unroll
      for (int k = 0; k < kVecs; ++k) {
        if (!cols.any(k)) continue;
#pragma unroll
        for (int i = 0; i < 4; ++i) x[k][i] = mul(mul(q, x[k][i]), wn[k][i]);
        cols.store(static_cast<BT*>(a.n) + at, k, x[k]);
      }
    }
    row.next(a);
    flip ^= 1;
    if (++s == ring.depth) s = 0, ph ^= 1u;
  }
}

// Sums of 8 values over the block; red: [warps][8]. Every warp adds up the warps' sums itself.
__device__ __forceinline__ void block_sum_8(float (&v)[8], float* red, int threads) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = threads >> 5;
  const float mine = warp_sum_many<8>(v, lane);  // of value lane / 4
  if ((lane & 3) == 0) red[warp * 8 + (lane >> 2)] = mine;
  row_barrier(threads);
  float s = 0.f;
  for (int w = lane >> 3; w < warps; w += 4) s += red[w * 8 + (lane & 7)];
  s += __shfl_xor_sync(0xFFFFFFFFu, s, 8);
  s += __shfl_xor_sync(0xFFFFFFFFu, s, 16);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __shfl_sync(0xFFFFFFFFu, s, i);
}

// A row is read from its stage twice, before and after its sums: its values in registers over the
// reduction would leave no room for the column sums of 16 columns.
// Where the gate is the same over a piece, sum d f s gives both its gradient (times w_post) and,
// times the gate, the piece's share of d_post; a gate per token (own_gate) has its gradient written
// with the row, and the sum is of g d f s.
template <typename ST, typename BT, typename PT, bool FULL, bool ODD, bool OWN>
__global__ void __launch_bounds__(kRowThreads) k_norm_bwd_rows(NormArgs a, RowRing ring) {
  constexpr int kVecs = Shape<ODD>::VECS;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float red[2][kRowThreads / 32 * 8];
  __shared__ uint64_t bars[16];
  const int tid = threadIdx.x, H = a.H, threads = blockDim.x - 32;
  const Columns<ODD> cols{H, threads};
  const bool post = FULL || a.w_post != nullptr, pre = FULL || a.w_pre != nullptr, gated = a.gate != nullptr;
  if (tid == 0) {
    for (int i = 0; i < ring.depth; ++i) {
      mbar_init(smem_u32(&bars[i]), 1);
      mbar_init(smem_u32(&bars[8 + i]), threads / 32);
    }
    mbar_fence_init();
  }
  __syncthreads();
  pdl_wait();
  if (tid >= threads) {
    produce_rows<ST, BT, PT, ODD>(a, ring, smem_u32(smem), smem_u32(bars), smem_u32(bars + 8));
    return;
  }
  RowWalk row;
  row.start(a, blockIdx.x);
  // weights: w_post (times the piece's gate), w_pre; column sums: of d f s, of v r' q, of d_post
  f32x2 wg[kVecs][4], wn[kVecs][4], raw[kVecs][4], d_pre[kVecs][4];
  float* const d_post = reinterpret_cast<float*>(smem + ring.depth * ring.bytes);  // [H]
  const bool own_gate = FULL ? OWN : ring.g >= 0, piece_gate = gated && !own_gate;
  auto post_weights = [&](int k, f32x2 (&w)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = both(1.f);
    if (post && cols.any(k)) cols.load(static_cast<const PT*>(a.w_post), k, w);
  };
#pragma unroll
  for (int k = 0; k < kVecs; ++k) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      wn[k][i] = both(1.f);
      raw[k][i] = d_pre[k][i] = both(0.f);
    }
    if (post && cols.any(k)) cols.store(d_post, k, raw[k]);
    if (pre && cols.any(k)) cols.load(static_cast<const PT*>(a.w_pre), k, wn[k]);
    post_weights(k, wg[k]);
  }
  bool fresh = piece_gate;  // a piece with a gate of its own begins
  int s = 0, flip = 0;
  uint32_t ph = 0;
  const float rh = 1.f / (float)H;
  while (row.more(a)) {
    const uint32_t stage = smem_u32(smem) + s * ring.bytes;
    await_row(smem_u32(&bars[s]), ph, a.timeout_ns);
    if (fresh) {
#pragma unroll
      for (int k = 0; k < kVecs; ++k) {
        if (!cols.any(k)) continue;
        f32x2 g[4];
        post_weights(k, wg[k]);
        cols.load(static_cast<const PT*>(a.gate) + row.group * H, k, g);
#pragma unroll
        for (int i = 0; i < 4; ++i) wg[k][i] = mul(wg[k][i], g[i]);
      }
      fresh = false;
    }
    const uint32_t xr = row_at<ODD>(stage, ring.x, row.t, H * sizeof(ST));
    const uint32_t vr = row_at<ODD>(stage, ring.v, row.t, H * sizeof(BT));
    const uint32_t fr = row_at<ODD>(stage, ring.f, row.t, H * sizeof(BT));
    const uint32_t ur = row_at<ODD>(stage, ring.u, row.t, H * sizeof(ST));
    // a row's values: r', branch, the gradients of r' and of n
    auto read = [&](int k, f32x2 (&x)[4], f32x2 (&f)[4], f32x2 (&u)[4], f32x2 (&v)[4]) {
      auto none = [](f32x2 (&z)[4]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) z[i] = both(0.f);
      };
      if (pre) {
        cols.template stage<ST>(xr, k, x);
        cols.template stage<BT>(vr, k, v);
      } else {
        none(x);
        none(v);
      }
      if (FULL || ring.f >= 0) cols.template stage<BT>(fr, k, f); else none(f);
      if (FULL || ring.u >= 0) cols.template stage<ST>(ur, k, u); else none(u);
    };
    // the row's own gate, and w_post times it
    auto gates = [&](int k, f32x2 (&g)[4], f32x2 (&w)[4]) {
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = wg[k][i];
      if (!own_gate) return;
      cols.template stage<PT>(row_at<ODD>(stage, ring.g, row.t, H * sizeof(PT)), k, g);
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = mul(w[i], g[i]);
    };
    f32x2 acc[6];
#pragma unroll
    for (int i = 0; i < 6; ++i) acc[i] = both(0.f);
#pragma unroll
    for (int k = 0; k < kVecs; ++k) {
      if (!cols.any(k)) continue;
      f32x2 x[4], f[4], u[4], v[4], g[4], w[4];
      read(k, x, f, u, v);
      gates(k, g, w);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const f32x2 wv = mul(wn[k][i], v[i]), ef = mul(w[i], f[i]);
        acc[0] = fma(x[i], x[i], acc[0]);
        acc[1] = fma(wv, x[i], acc[1]);
        acc[2] = fma(f[i], f[i], acc[2]);
        acc[3] = fma(ef, u[i], acc[3]);
        acc[4] = fma(ef, wv, acc[4]);
        acc[5] = fma(ef, x[i], acc[5]);
      }
    }
    float sum[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) sum[i] = i < 6 ? sum_of(acc[i < 6 ? i : 0]) : 0.f;
    if (ph >= kLost) sum[0] = sum[2] = __int_as_float(0x7FC00000);
    block_sum_8(sum, red[flip], threads);
    const float q = pre ? rsqrtf(sum[0] * rh + a.eps) : 0.f;
    const float cq = unit_factor(q, rh, sum[1]);
    const float sf = post ? rsqrtf(sum[2] * rh + a.eps) : 1.f;
    const float cs = post ? unit_factor(sf, rh, pre ? sum[3] + q * sum[4] - cq * (q * sum[5]) : sum[3]) : 0.f;
    const f32x2 q2 = both(q), ncq = both(-cq), sf2 = both(sf), ncs = both(-cs), scale = both(a.scale);
    const int64_t at = row.t * H;
#pragma unroll
    for (int k = 0; k < kVecs; ++k) {
      if (!cols.any(k)) continue;
      f32x2 x[4], f[4], u[4], v[4], g[4], w[4], dr[4];
      read(k, x, f, u, v);
      gates(k, g, w);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f32x2 d = u[i];
        if (pre) {
          const f32x2 xq = mul(q2, x[i]);
          d = fma(ncq, xq, fma(q2, mul(wn[k][i], v[i]), d));
          d_pre[k][i] = fma(v[i], xq, d_pre[k][i]);
        } else if (ph >= kLost) {
          d = nan_pair();
        }
        const f32x2 fs = mul(sf2, f[i]);
        if (own_gate) {  // its gradient leaves with the row; the sum is of g d f s
          const f32x2 own = mul(d, fs);
          raw[k][i] = fma(g[i], own, raw[k][i]);
          g[i] = mul(wg[k][i], own);
        } else {
          raw[k][i] = fma(d, fs, raw[k][i]);
        }
        dr[i] = mul(scale, d);
        // (without a norm the branch's value takes no part, not even an infinite one times zero)
        f[i] = post ? fma(ncs, fs, mul(sf2, mul(w[i], d))) : mul(w[i], d);
      }
      cols.store(static_cast<ST*>(a.dr) + at, k, dr);
      if (FULL || a.df != nullptr) cols.store(static_cast<BT*>(a.df) + at, k, f);
      if (own_gate) cols.store(static_cast<PT*>(a.d_gate) + at, k, g);
    }
    if (piece_gate && row.t + 1 == row.t1) {  // the piece ends
#pragma unroll
      for (int k = 0; k < kVecs; ++k) {
        if (!cols.any(k)) continue;
        f32x2 g[4], w[4], sum_post[4];
        post_weights(k, w);
        cols.load(static_cast<const PT*>(a.gate) + row.group * H, k, g);
        if (post) {
          cols.load(d_post, k, sum_post);
#pragma unroll
          for (int i = 0; i < 4; ++i) sum_post[i] = fma(g[i], raw[k][i], sum_post[i]);
          cols.store(d_post, k, sum_post);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          w[i] = mul(w[i], raw[k][i]);
          raw[k][i] = both(0.f);
        }
        if (a.part_gate != nullptr)
          cols.store(a.part_gate + row.piece * H, k, w);
        else
          cols.store(static_cast<PT*>(a.d_gate) + row.group * H, k, w);
      }
      fresh = true;
    }
    __syncwarp();
    if ((tid & 31) == 0 && ph < kLost) mbar_arrive(smem_u32(&bars[8 + s]));  // the stage is read
    row.next(a);
    flip ^= 1;
    if (++s == ring.depth) s = 0, ph ^= 1u;
  }
#pragma unroll
  for (int k = 0; k < kVecs; ++k) {
    if (!cols.any(k)) continue;
    if (post) {
      f32x2 sum_post[4];
      cols.load(d_post, k, sum_post);  // zero unless pieces have gates
#pragma unroll
      for (int i = 0; i < 4; ++i) sum_post[i] = fma(both(1.f), raw[k][i], sum_post[i]);
      cols.store(a.part_post + (int64_t)blockIdx.x * H, k, sum_post);
    }
    if (pre) cols.store(a.part_pre + (int64_t)blockIdx.x * H, k, d_pre[k]);
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

// How tokens are dealt to blocks.
struct RowPlan {
  int64_t group_rows, piece_rows, pieces_per_group, pieces, blocks;
};

// by_group: a piece lies within one gate's rows.
RowPlan plan_rows(const mm_norm_desc& d, int64_t target, bool by_group = true) {
  RowPlan p{};
  const int64_t groups = by_group ? std::max<int64_t>(1, d.groups) : 1;
  p.group_rows = d.T / groups;
  p.piece_rows = std::max<int64_t>(1, std::min(p.group_rows, (d.T + target - 1) / target));
  p.pieces_per_group = (p.group_rows + p.piece_rows - 1) / p.piece_rows;
  p.pieces = groups * p.pieces_per_group;
  p.blocks = std::min(p.pieces, target);
  return p;
}

struct BwdPlan : RowPlan {
  size_t off_post, off_pre, off_gate, total;
};

// Working threads of a block (see Shape), and the blocks that share an SM: all of its registers.
inline int row_threads(int64_t H, bool odd) {
  const int64_t h = std::min<int64_t>(H, kMaxRingH / (odd ? 2 : 1));
  return (int)(odd ? (h + 255) / 256 * 32 : (h + 511) / 512 * 32);
}
inline int64_t blocks_per_sm(int64_t H, bool odd) {
  return std::max<int64_t>(1, kRowThreads / (row_threads(H, odd) + 32));
}

BwdPlan plan_bwd(const mm_norm_desc& d, int sms) {
  BwdPlan p{};
  static_cast<RowPlan&>(p) = plan_rows(d, sms * std::max(blocks_per_sm(d.H, false), blocks_per_sm(d.H, true)));
  const size_t slice = ((size_t)d.H * 4 + 255) / 256 * 256;
  p.off_post = 0;
  p.off_pre = slice * (size_t)p.blocks;
  p.off_gate = 2 * slice * (size_t)p.blocks;
  p.total = p.off_gate +
            (d.groups > 0 && p.pieces_per_group > 1 ? slice * (size_t)p.pieces : 0);
  return p;
}

// The row ring of a problem with at most `per_sm` blocks on an SM, fewer where rows are so long
// that less than three stages would fit; depth 0: it does not fit.
RowRing plan_ring(const mm_norm_desc& d, const NormArgs& a, bool backward, bool odd,
                  int64_t& per_sm) {
  const int sb = (int)(d.H * (d.stream_type == MM_BF16 ? 2 : 4));
  const int bb = (int)(d.H * (d.block_type == MM_BF16 ? 2 : 4));
  const int pb = (int)(d.H * (d.param_type == MM_BF16 ? 2 : 4));
  RowRing r{-1, -1, -1, -1, -1, 0, 0, odd ? 1 : 0, 0};
  auto add = [&](int& at, bool used, int bytes) {
    if (!used) return;
    at = r.bytes;
    r.bytes += (bytes + (odd ? 30 : 0) + 127) / 128 * 128;
  };
  add(r.x, !backward || a.w_pre != nullptr, sb);
  add(r.f, a.f != nullptr, bb);
  add(r.u, backward && a.u != nullptr, sb);
  add(r.v, backward && a.w_pre != nullptr, bb);
  // a gate that changes every few rows (backward: with every row) travels with them
  add(r.g, a.gate != nullptr && a.rows_per_gate < (backward ? 2 : 8), pb);
  r.tail = backward && a.w_post != nullptr ? (int)(d.H + 3) / 4 * 16 : 0;
  auto fit = [&](int64_t blocks) { return (216 * 1024 / blocks - r.tail) / std::max(1, r.bytes); };
  while (per_sm > 1 && fit(per_sm) < 3) --per_sm;
  r.depth = (int)std::min<int64_t>(8, fit(per_sm));
  return r;
}

// Rows that can move as 16-byte words.
bool wide(const mm_norm_desc& d, std::initializer_list<const void*> ptrs) {
  if (d.H % 8) return false;
  for (const void* p : ptrs)
    if (!aligned_to(p, 16)) return false;
  return true;
}

// Rows off 16-byte boundaries that bulk copies can bring all the same: what is copied starts on one.
bool odd_rows(const mm_norm_desc& d, std::initializer_list<const void*> ptrs) {
  // (from 64 on no row but the last ends within 16 bytes of the tensor's end)
  if (d.H < 64 || d.H > kMaxRingH / 2) return false;
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

// Raises a kernel's dynamic shared memory limit, once per device.
template <auto* KERNEL>
cudaError_t allow_smem(size_t bytes) {
  static std::atomic<uint64_t> done_mask{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (done_mask.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e == cudaSuccess) done_mask.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

template <auto* KERNEL>
cudaError_t launch_rows(const NormArgs& a, const RowRing& r, int64_t blocks, cudaStream_t st) {
  const cudaError_t e = allow_smem<KERNEL>(216 * 1024);
  if (e != cudaSuccess) return e;
  return launch_pdl(KERNEL, dim3((unsigned)blocks), dim3(row_threads(a.H, r.odd) + 32),
                    (size_t)r.bytes * r.depth + r.tail, st, a, r);
}

template <typename ST, typename BT, typename PT>
cudaError_t launch_fwd_rows(const NormArgs& a, const RowRing& r, int64_t blocks, cudaStream_t st) {
  const bool full = a.w_post && a.w_pre && a.out;  // (a post weight has a branch)
  if (r.odd)
    return full && r.g < 0
               ? launch_rows<&k_norm_fwd_rows<ST, BT, PT, true, true, false>>(a, r, blocks, st)
               : launch_rows<&k_norm_fwd_rows<ST, BT, PT, false, true, false>>(a, r, blocks, st);
  if (!full)
    return launch_rows<&k_norm_fwd_rows<ST, BT, PT, false, false, false>>(a, r, blocks, st);
  return r.g < 0 ? launch_rows<&k_norm_fwd_rows<ST, BT, PT, true, false, false>>(a, r, blocks, st)
                 : launch_rows<&k_norm_fwd_rows<ST, BT, PT, true, false, true>>(a, r, blocks, st);
}

template <typename ST, typename BT, typename PT>
cudaError_t launch_bwd_rows(const NormArgs& a, const RowRing& r, int64_t blocks, cudaStream_t st) {
  const bool full = a.w_post && a.w_pre && a.u;  // (a post weight has a branch)
  if (r.odd)
    return full && r.g < 0
               ? launch_rows<&k_norm_bwd_rows<ST, BT, PT, true, true, false>>(a, r, blocks, st)
               : launch_rows<&k_norm_bwd_rows<ST, BT, PT, false, true, false>>(a, r, blocks, st);
  if (!full)
    return launch_rows<&k_norm_bwd_rows<ST, BT, PT, false, false, false>>(a, r, blocks, st);
  return r.g < 0 ? launch_rows<&k_norm_bwd_rows<ST, BT, PT, true, false, false>>(a, r, blocks, st)
                 : launch_rows<&k_norm_bwd_rows<ST, BT, PT, true, false, true>>(a, r, blocks, st);
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

// Calls f with values of the stream, block and parameter types.
template <typename F>
cudaError_t with_types(const mm_norm_desc& d, F&& f) {
  using B = __nv_bfloat16;
  const bool p = d.param_type == MM_BF16;
  if (d.stream_type == MM_BF16) return p ? f(B(), B(), B()) : f(B(), B(), 0.f);
  if (d.block_type == MM_BF16) return p ? f(0.f, B(), B()) : f(0.f, B(), 0.f);
  return p ? f(0.f, 0.f, B()) : f(0.f, 0.f, 0.f);
}

void deal_rows(NormArgs& a, const RowPlan& p) {
  a.pieces = p.pieces;
  a.pieces_per_group = p.pieces_per_group;
  a.piece_rows = p.piece_rows;
  a.group_rows = p.group_rows;
}

thread_local int t_stall = 0;  // mm_residual_norm_test_stall

NormArgs norm_args(const mm_norm_desc& d) {
  NormArgs a{};
  a.T = d.T;
  a.H = (int)d.H;
  a.ptype = d.param_type;
  a.scale = d.residual_scale;
  a.eps = d.eps;
  a.rows_per_gate = d.groups > 0 ? d.T / d.groups : 0;
  a.stall = t_stall;
  a.timeout_ns = t_stall ? kTestTimeoutNs : kRowTimeoutNs;
  return a;
}

}  // namespace
}  // namespace mm

using namespace mm;

extern "C" {

int mm_ops_version(void) { return 1; }

void mm_residual_norm_test_stall(int on) { t_stall = on != 0; }

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
  const int sms = std::max(1, device_sm_count());
  int64_t per_sm = blocks_per_sm(d->H, !w8);
  const RowRing ring = plan_ring(*d, a, false, !w8, per_sm);
  // The ring pays from a few rows per block on (2000 rows of 2048, two per block: 7.3 us, 7.6 without;
  // 500: 4.0 and 3.4) and for rows of some kilobytes, where a block of the other form has few in
  // flight. 2^25 elements, with and without: bf16 512 wide 58 and 51 us, 1024 47 and 52, 2048 48 and
  // 54, 7168 45 and 93; fp32 2048 wide 97 and 85, 4096 89 and 94, 7168 95 and 130.
  const bool bulk = w8 ? d->H >= (d->stream_type == MM_BF16 ? 1024 : 4096) && d->H <= kMaxRingH
                       : odd_rows(*d, {residual, branch, gate});
  if (bulk && d->T > 2 * sms * per_sm && ring.depth >= 2) {
    const RowPlan p = plan_rows(*d, sms * per_sm, ring.g < 0);
    deal_rows(a, p);
    MM_TRY(with_types(*d, [&](auto s0, auto b0, auto p0) {
      return launch_fwd_rows<decltype(s0), decltype(b0), decltype(p0)>(a, ring, p.blocks, st);
    }));
    return MM_OK;
  }
  MM_TRY(with_types(*d, [&](auto s0, auto b0, auto) {
    return launch_fwd<decltype(s0), decltype(b0)>(a, w8, st);
  }));
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
  const int sms = std::max(1, device_sm_count());
  BwdPlan p = plan_bwd(*d, sms);
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
  const bool w8 = wide(*d, {residual_out, branch, post_weight, pre_weight, gate, d_residual_out,
                            d_normed, d_residual, d_branch, d_gate});
  int64_t per_sm = blocks_per_sm(d->H, !w8);  // (no more than the workspace is laid out for)
  const RowRing ring = plan_ring(*d, a, true, !w8, per_sm);
  // (the form without bulk copies takes two to four times as long at every width of 256 to 7168)
  const bool ringed =
      (w8 || odd_rows(*d, {residual_out, branch, gate, d_residual_out, d_normed})) &&
      d->H <= kMaxRingH && ring.depth >= 1;
  const bool own_gate = ringed && ring.g >= 0;
  static_cast<RowPlan&>(p) = plan_rows(*d, sms * per_sm, !own_gate);
  deal_rows(a, p);
  const bool gate_parts = gate != nullptr && !own_gate && p.pieces_per_group > 1;
  a.part_gate = gate_parts ? reinterpret_cast<float*>(ws + p.off_gate) : nullptr;
  MM_TRY(with_types(*d, [&](auto s0, auto b0, auto p0) {
    using ST = decltype(s0);
    using BT = decltype(b0);
    return ringed ? launch_bwd_rows<ST, BT, decltype(p0)>(a, ring, p.blocks, st)
                : launch_bwd<ST, BT>(a, p.blocks, w8, st);
  }));
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
