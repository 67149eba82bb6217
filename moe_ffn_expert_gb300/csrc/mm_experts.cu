// The order of a selection's slots by expert, the tokens' rows in that order, and a token's weighted
// sum of its slots' rows with its gradients (definitions in mm_experts.h).
//
// Order: a stable counting sort. A block takes kSlots slots and counts them per expert (slots without
// an expert are those of one more, the last); the blocks' counts before a block and the experts before
// an expert give where its slots of that expert start, and within a block the warps' counts and the
// lanes before a lane with the same expert the rest. Up to kSlots slots are one launch.
//
// The order is bound by latency: 512 slots of 128 experts 3.6 us, 131072 in two launches 10.5 us (a 2 MB
// read and written).
//
// Dispatch and combine move rows and are bound by HBM: a block has a token's row and its K slots' rows, so
// that each row is read and written once. 16384 x 8 rows of 2048 bf16 dispatched 91 us (6.6 TB/s), 4096 x 8
// of 7168 combined 81 us (6.5 TB/s), the gradients of 8192 x 8 of 2048 88 us (6.5 TB/s). Rows off 16-byte
// boundaries are loaded and stored element by element: the gradients of 1001 x 6 fp32 rows of 2047 20 us (4.9
// TB/s), of bf16 rows 18 us (2.9). Aligned words shifted by a row's offset are not built.
#include <algorithm>
#include <type_traits>

#include "../../include/mm_experts.h"
#include "mm_kernels.h"
#include "mm_rows.cuh"

namespace mm {
namespace {

constexpr int kMaxE = 1024, kMaxK = 16;
constexpr int kTableWarps = 16, kRounds = 4;  // a warp counts kRounds x 32 slots
constexpr int kSlots = kTableWarps * kRounds * 32;
// Blocks whose counts every block adds up by itself; more of them are added up by a launch between.
constexpr int kFewBlocks = 128;

struct TableArgs {
  const int32_t* ids;
  int32_t *offsets, *row_of_slot, *slot_of_row;
  int32_t* counts;  // [blocks + 1][E + 1]; added up: the counts of the blocks before, the totals last
  int S, E, blocks;
};

__device__ __forceinline__ int bucket_of(const TableArgs& a, int s) {
  if (s >= a.S) return -1;
  const int e = a.ids[s];
  return e >= 0 && e < a.E ? e : a.E;
}

__global__ void __launch_bounds__(32 * kTableWarps) k_table_count(TableArgs a) {
  __shared__ int count[kMaxE + 1];
  pdl_wait();
  pdl_launch_dependents();
  for (int e = threadIdx.x; e <= a.E; e += blockDim.x) count[e] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < kSlots; i += blockDim.x) {
    const int b = bucket_of(a, blockIdx.x * kSlots + i);
    if (b >= 0) atomicAdd(&count[b], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e <= a.E; e += blockDim.x)
    a.counts[(int64_t)blockIdx.x * (a.E + 1) + e] = count[e];
}

// 32 buckets a block, a warp for each of 32 runs of blocks: counts become the counts of the blocks
// before, and the totals follow the last.
__global__ void __launch_bounds__(1024) k_table_scan(TableArgs a) {
  __shared__ int sums[32][33];
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, e = blockIdx.x * 32 + lane;
  const int64_t run = (a.blocks + 31) / 32, first = warp * run, end = min(first + run, (int64_t)a.blocks);
  int sum = 0;
  if (e <= a.E)
    for (int64_t b = first; b < end; ++b) sum += a.counts[b * (a.E + 1) + e];
  sums[warp][lane] = sum;
  __syncthreads();
  int before = 0;
  for (int w = 0; w < warp; ++w) before += sums[w][lane];
  if (e > a.E) return;
  for (int64_t b = first; b < end; ++b) {
    int32_t* at = a.counts + b * (a.E + 1) + e;
    const int c = *at;
    *at = before;
    before += c;
  }
  if (warp == 31) a.counts[(int64_t)a.blocks * (a.E + 1) + e] = before;
}

// FEW: no launch between, the blocks' counts are added up here.
template <bool FEW>
__global__ void __launch_bounds__(32 * kTableWarps) k_table_rank(TableArgs a) {
  constexpr int THREADS = 32 * kTableWarps, PER = (kMaxE + THREADS) / THREADS;
  __shared__ __align__(4) uint16_t count[kTableWarps][kMaxE + 2];
  __shared__ int base[kMaxE + 1];    // where a bucket starts, then where this block's slots of it do
  __shared__ int before[kMaxE + 1];  // slots of a bucket in the blocks before
  __shared__ int sums[kTableWarps];
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, buckets = a.E + 1;
  for (int i = threadIdx.x; i < kTableWarps * (kMaxE + 2) / 2; i += THREADS)
    reinterpret_cast<uint32_t*>(&count[0][0])[i] = 0;
  for (int e = threadIdx.x; e < buckets; e += THREADS) {
    base[e] = FEW ? 0 : a.counts[(int64_t)a.blocks * buckets + e];
    before[e] = FEW ? 0 : a.counts[(int64_t)blockIdx.x * buckets + e];
  }
  int b[kRounds];
  unsigned same[kRounds];
  const int s0 = (blockIdx.x * kTableWarps + warp) * kRounds * 32 + lane;
#pragma unroll
  for (int r = 0; r < kRounds; ++r) b[r] = bucket_of(a, s0 + 32 * r);
  __syncthreads();
  if (FEW && a.blocks > 1) {
    // all blocks' counts, 32 buckets of one block at a time, eight loads of a warp in flight
    const int groups = (buckets + 31) / 32, loads = a.blocks * groups;
    for (int i0 = warp; i0 < loads; i0 += 8 * kTableWarps) {
      int c[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int i = i0 + u * kTableWarps, k = i / groups, e = (i - k * groups) * 32 + lane;
        c[u] = i < loads && e < buckets ? a.counts[k * buckets + e] : 0;
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int i = i0 + u * kTableWarps, k = i / groups, e = (i - k * groups) * 32 + lane;
        if (c[u] == 0) continue;
        atomicAdd(&base[e], c[u]);
        if (k < (int)blockIdx.x) atomicAdd(&before[e], c[u]);
      }
    }
  }
#pragma unroll
  for (int r = 0; r < kRounds; ++r) {
    same[r] = __match_any_sync(0xFFFFFFFFu, b[r]);
    if (b[r] >= 0 && lane == __ffs(same[r]) - 1) count[warp][b[r]] += __popc(same[r]);
    __syncwarp();
  }
  __syncthreads();
  for (int e = threadIdx.x; e < buckets; e += THREADS) {
    int run = 0;
#pragma unroll
    for (int w = 0; w < kTableWarps; ++w) {
      const int c = count[w][e];
      count[w][e] = (uint16_t)run;
      run += c;
    }
    if (FEW && a.blocks == 1) base[e] = run;
  }
  __syncthreads();
  // the buckets' totals to where they start
  int total[PER], mine = 0;
#pragma unroll
  for (int p = 0; p < PER; ++p) {
    const int e = threadIdx.x * PER + p;
    total[p] = e < buckets ? base[e] : 0;
    mine += total[p];
  }
  int upto = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int v = __shfl_up_sync(0xFFFFFFFFu, upto, d);
    if (lane >= d) upto += v;
  }
  if (lane == 31) sums[warp] = upto;
  __syncthreads();
  int at = upto - mine;
  for (int w = 0; w < warp; ++w) at += sums[w];
#pragma unroll
  for (int p = 0; p < PER; ++p) {
    const int e = threadIdx.x * PER + p;
    if (e < buckets) {
      base[e] = at + before[e];
      if (blockIdx.x == 0) a.offsets[e] = at;  // (slots without an expert are behind offsets[E])
    }
    at += total[p];
  }
  __syncthreads();
#pragma unroll
  for (int r = 0; r < kRounds; ++r) {
    const int s = s0 + 32 * r;
    int row = 0;
    if (b[r] >= 0) row = base[b[r]] + count[warp][b[r]] + __popc(same[r] & ((1u << lane) - 1u));
    __syncwarp();
    if (b[r] >= 0) {
      if (lane == __ffs(same[r]) - 1) count[warp][b[r]] += __popc(same[r]);
      const bool taken = b[r] < a.E;
      a.row_of_slot[s] = taken ? row : -1;
      a.slot_of_row[row] = taken ? s : -1;
    }
    __syncwarp();
  }
}

// ------------------------------------------------------------------------------------ rows

struct RowArgs {
  const void *x, *rows;  // the tokens' rows, the slots' rows
  const int32_t *offsets, *row_of_slot;
  const float* weights;
  void *out_x, *out_rows;
  float* d_weights;
  int64_t T, S;
  int H, E, K;
  int words;  // of a row, in the words that the kernel moves
};

// Zero rows behind the last expert's, by all blocks of the launch together.
template <typename V>
__device__ __forceinline__ void zero_rows_behind(const RowArgs& a, V* rows) {
  const int64_t first = max(0, a.offsets[a.E]);
  for (int64_t r = first + blockIdx.x; r < a.S; r += gridDim.x)
    for (int w = threadIdx.x; w < a.words; w += blockDim.x) rows[r * a.words + w] = V{};
}

template <typename V>
__global__ void __launch_bounds__(256) k_dispatch(RowArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  const V* x = static_cast<const V*>(a.x);
  V* rows = static_cast<V*>(a.out_rows);
  const int64_t t = blockIdx.x;
  const int32_t* row = a.row_of_slot + t * a.K;
  for (int w = threadIdx.x; w < a.words; w += blockDim.x) {
    const V v = x[t * a.words + w];
    for (int k = 0; k < a.K; ++k) {
      const int64_t r = row[k];
      if (r >= 0 && r < a.S) rows[r * a.words + w] = v;
    }
  }
  zero_rows_behind(a, rows);
}

// Words of W columns of one row that a thread has under way at a time: single columns (rows off 16-byte
// boundaries) need more of them. (1001 x 6 rows of 2047 columns, us, one, two and four at a time: fp32
// backward 38, 20 and 24, bf16 forward 19, 14 and 11.)
template <int W>
constexpr int kAtOnce = W == 1 ? 4 : 1;
template <int W>
constexpr int kAtOnceBwd = W == 1 ? 2 : 1;

// W columns as they lie in memory: half the registers of bf16 numbers that wait for their turn.
template <typename T, int W>
struct Word {
  static_assert(W == 8, "widths 8 and 1");
  uint4 w[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) w[i] = reinterpret_cast<const uint4*>(p)[i];
  }
  __device__ __forceinline__ void widen(float (&v)[W]) const {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) {
      const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if constexpr (sizeof(T) == 2) v[2 * k] = bf16_lo(u[k]), v[2 * k + 1] = bf16_hi(u[k]);
        else v[4 * i + k] = __uint_as_float(u[k]);
      }
    }
  }
};
template <typename T>
struct Word<T, 1> {
  T w{};
  __device__ __forceinline__ void load(const T* p) { w = *p; }
  __device__ __forceinline__ void widen(float (&v)[1]) const {
    if constexpr (sizeof(T) == 2) v[0] = __bfloat162float(w);
    else v[0] = w;
  }
};

// words: H / W.
template <typename T, int W>
__global__ void __launch_bounds__(256) k_combine(RowArgs a) {
  constexpr int U = kAtOnce<W>, N = 4;  // slots whose loads are in flight
  pdl_wait();
  pdl_launch_dependents();
  const T* rows = static_cast<const T*>(a.rows);
  const int64_t t = blockIdx.x;
  const int32_t* row = a.row_of_slot + t * a.K;
  for (int w0 = threadIdx.x; w0 < a.words; w0 += blockDim.x * U) {
    float y[U][W] = {};
    for (int k0 = 0; k0 < a.K; k0 += N) {
      Word<T, W> v[N][U];
      bool there[N];
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const int64_t r = k0 + k < a.K ? row[k0 + k] : -1;
        there[k] = r >= 0 && r < a.S;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int w = w0 + u * (int)blockDim.x;
          v[k][u] = Word<T, W>{};
          if (there[k] && w < a.words) v[k][u].load(rows + r * a.H + (int64_t)w * W);
        }
      }
#pragma unroll
      for (int k = 0; k < N; ++k) {
        if (!there[k]) continue;
        const float g = a.weights ? a.weights[t * a.K + k0 + k] : 1.f;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          float x[W];
          v[k][u].widen(x);
#pragma unroll
          for (int i = 0; i < W; ++i) y[u][i] = fmaf(g, x[i], y[u][i]);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int w = w0 + u * (int)blockDim.x;
      if (w < a.words) store_vec<W>(static_cast<T*>(a.out_x) + t * a.H + (int64_t)w * W, y[u]);
    }
  }
}

// S slots at a time, of which N loads are in flight (fp32 words: what 32 registers hold). Tokens of one or
// two slots have a kernel of fewer registers, as only more blocks bring more loads there (16384 tokens of
// one slot, 1024 columns: 55 us with S = 8).
template <typename T, int W, int S>
__global__ void __launch_bounds__(256, S == 8 ? 3 : 1) k_combine_bwd(RowArgs a) {
  constexpr int U = kAtOnceBwd<W>, N = S == 8 && W == 8 && sizeof(T) == 4 ? 4 : S;
  __shared__ float part[8][S];
  pdl_wait();
  pdl_launch_dependents();
  const T* rows = static_cast<const T*>(a.rows);
  const int64_t t = blockIdx.x;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int k0 = 0; k0 < a.K; k0 += S) {
    float dot[S] = {};
    int row[S];
#pragma unroll
    for (int k = 0; k < S; ++k) {
      row[k] = k0 + k < a.K ? a.row_of_slot[t * a.K + k0 + k] : -1;
      if (row[k] >= a.S) row[k] = -1;
    }
    for (int w0 = threadIdx.x; w0 < a.words; w0 += blockDim.x * U) {
      Word<T, W> d[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int w = w0 + u * (int)blockDim.x;
        d[u] = Word<T, W>{};
        if (w < a.words) d[u].load(static_cast<const T*>(a.x) + t * a.H + (int64_t)w * W);
      }
#pragma unroll
      for (int kn = 0; kn < S; kn += N) {
        Word<T, W> v[N][U];
        if (a.d_weights) {
#pragma unroll
          for (int k = 0; k < N; ++k) {
            const int r = row[kn + k];
#pragma unroll
            for (int u = 0; u < U; ++u) {
              const int w = w0 + u * (int)blockDim.x;
              v[k][u] = Word<T, W>{};
              if (r >= 0 && w < a.words) v[k][u].load(rows + (int64_t)r * a.H + w * W);
            }
          }
        }
#pragma unroll
        for (int k = 0; k < N; ++k) {
          const int64_t r = row[kn + k];
          if (r < 0) continue;
          const float g = a.weights ? a.weights[t * a.K + k0 + kn + k] : 1.f;
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const int w = w0 + u * (int)blockDim.x;
            if (w >= a.words) continue;
            float x[W], y[W];
            d[u].widen(x);
            if (a.d_weights) {
              v[k][u].widen(y);
#pragma unroll
              for (int i = 0; i < W; ++i) dot[kn + k] = fmaf(x[i], y[i], dot[kn + k]);
            }
#pragma unroll
            for (int i = 0; i < W; ++i) y[i] = g * x[i];
            store_vec<W>(static_cast<T*>(a.out_rows) + r * a.H + w * W, y);
          }
        }
      }
    }
    if (a.d_weights) {
      constexpr int LANES = 32 / S;
      const float sum = warp_sum_many<S>(dot, lane);
      if (lane % LANES == 0) part[warp][lane / LANES] = sum;
      __syncthreads();
      if (threadIdx.x < S && k0 + (int)threadIdx.x < a.K) {
        float s = 0.f;
        for (int w = 0; w < (int)blockDim.x / 32; ++w) s += part[w][threadIdx.x];
        a.d_weights[t * a.K + k0 + threadIdx.x] = s;
      }
      __syncthreads();
    }
  }
  // (words of W elements)
  const int64_t first = max(0, a.offsets[a.E]);
  for (int64_t r = first + blockIdx.x; r < a.S; r += gridDim.x)
    for (int w = threadIdx.x; w < a.words; w += blockDim.x) {
      const float zero[W] = {};
      store_vec<W>(static_cast<T*>(a.out_rows) + r * a.H + (int64_t)w * W, zero);
    }
}

// ------------------------------------------------------------------------------------ host side

inline bool aligned_to(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

mm_status check_desc(const mm_expert_desc* d, bool rows) {
  if (d == nullptr || d->T < 0 || d->E < 1 || d->K < 1) return MM_ERR_INVALID_ARG;
  if (d->E > kMaxE || d->K > kMaxK || d->T > ((int64_t)1 << 31) ||
      d->T * d->K >= ((int64_t)1 << 31) - ((int64_t)1 << 16))
    return MM_ERR_UNSUPPORTED;
  if (rows) {
    if (d->H < 1 || (d->type != MM_BF16 && d->type != MM_FP32)) return MM_ERR_INVALID_ARG;
    if (d->H > ((int64_t)1 << 20)) return MM_ERR_UNSUPPORTED;
  }
  return MM_OK;
}

int64_t table_blocks(const mm_expert_desc& d) { return (d.T * d.K + kSlots - 1) / kSlots; }

RowArgs row_args(const mm_expert_desc& d) {
  RowArgs a{};
  a.T = d.T;
  a.S = d.T * d.K;
  a.H = (int)d.H;
  a.E = d.E;
  a.K = d.K;
  return a;
}

inline unsigned threads_for(int words) { return (unsigned)std::min(256, (words + 31) / 32 * 32); }

}  // namespace
}  // namespace mm

using namespace mm;

extern "C" {

size_t mm_expert_table_workspace_size(const mm_expert_desc* d) {
  if (check_desc(d, false) != MM_OK) return 0;
  const int64_t blocks = table_blocks(*d);
  return blocks <= 1 ? 256 : std::max<size_t>(256, (size_t)(blocks + 1) * (d->E + 1) * 4);
}

mm_status mm_expert_table(const mm_expert_desc* d, const int32_t* topk_ids, int32_t* offsets,
                          int32_t* row_of_slot, int32_t* slot_of_row, void* workspace,
                          size_t workspace_bytes, void* stream) {
  mm_status s = check_desc(d, false);
  if (s != MM_OK) return s;
  if (!offsets || !aligned_to(offsets, 4) || !aligned_to(topk_ids, 4) || !aligned_to(row_of_slot, 4) ||
      !aligned_to(slot_of_row, 4))
    return MM_ERR_INVALID_ARG;
  if (d->T * d->K > kSlots && (workspace == nullptr || !aligned_to(workspace, 256) ||
                               workspace_bytes < mm_expert_table_workspace_size(d)))
    return MM_ERR_WORKSPACE;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (d->T > 0 && (!topk_ids || !row_of_slot || !slot_of_row)) return MM_ERR_INVALID_ARG;
  clear_error();
  if (d->T == 0) {
    MM_TRY(cudaMemsetAsync(offsets, 0, (size_t)(d->E + 1) * 4, st));
    return MM_OK;
  }
  TableArgs a{topk_ids, offsets, row_of_slot, slot_of_row, static_cast<int32_t*>(workspace),
              (int)(d->T * d->K), d->E, (int)table_blocks(*d)};
  const dim3 grid((unsigned)a.blocks), threads(32 * kTableWarps);
  if (a.blocks > 1) MM_TRY(launch_pdl(k_table_count, grid, threads, 0, st, a));
  if (a.blocks > kFewBlocks)
    MM_TRY(launch_pdl(k_table_scan, dim3((unsigned)(a.E + 32) / 32), dim3(1024), 0, st, a));
  MM_TRY(launch_pdl(a.blocks > kFewBlocks ? k_table_rank<false> : k_table_rank<true>, grid, threads, 0, st, a));
  return MM_OK;
}

mm_status mm_expert_dispatch(const mm_expert_desc* d, const void* x, const int32_t* offsets,
                             const int32_t* row_of_slot, void* rows, void* stream) {
  mm_status s = check_desc(d, true);
  if (s != MM_OK) return s;
  const size_t es = d->type == MM_BF16 ? 2 : 4;
  if (!aligned_to(x, es) || !aligned_to(rows, es) || !aligned_to(offsets, 4) || !aligned_to(row_of_slot, 4))
    return MM_ERR_INVALID_ARG;
  if (d->T == 0) return MM_OK;
  if (!x || !offsets || !row_of_slot || !rows) return MM_ERR_INVALID_ARG;
  clear_error();
  RowArgs a = row_args(*d);
  a.x = x;
  a.offsets = offsets;
  a.row_of_slot = row_of_slot;
  a.out_rows = rows;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  // the widest words that rows consist of and start at
  const uintptr_t all = reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(rows) |
                        (uintptr_t)(d->H * es);
  const dim3 grid((unsigned)d->T);
  auto go = [&](auto* kernel, int bytes) {
    a.words = (int)(d->H * es / bytes);
    return launch_pdl(kernel, grid, dim3(threads_for(a.words)), 0, st, a);
  };
  if (all % 16 == 0)
    MM_TRY(go(k_dispatch<uint4>, 16));
  else if (all % 8 == 0)
    MM_TRY(go(k_dispatch<uint2>, 8));
  else if (all % 4 == 0)
    MM_TRY(go(k_dispatch<uint32_t>, 4));
  else
    MM_TRY(go(k_dispatch<uint16_t>, 2));
  return MM_OK;
}

mm_status mm_expert_combine(const mm_expert_desc* d, const void* rows, const int32_t* row_of_slot,
                            const float* weights, void* y, void* stream) {
  mm_status s = check_desc(d, true);
  if (s != MM_OK) return s;
  const size_t es = d->type == MM_BF16 ? 2 : 4;
  if (!aligned_to(rows, es) || !aligned_to(y, es) || !aligned_to(row_of_slot, 4) || !aligned_to(weights, 4))
    return MM_ERR_INVALID_ARG;
  if (d->T == 0) return MM_OK;
  if (!rows || !row_of_slot || !y) return MM_ERR_INVALID_ARG;
  clear_error();
  RowArgs a = row_args(*d);
  a.rows = rows;
  a.row_of_slot = row_of_slot;
  a.weights = weights;
  a.out_x = y;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const bool wide = d->H % 8 == 0 && aligned_to(rows, 16) && aligned_to(y, 16);
  a.words = (int)(wide ? d->H / 8 : d->H);
  auto go = [&](auto* kernel) {
    return launch_pdl(kernel, dim3((unsigned)d->T), dim3(threads_for(a.words)), 0, st, a);
  };
  if (d->type == MM_BF16)
    MM_TRY(wide ? go(k_combine<__nv_bfloat16, 8>) : go(k_combine<__nv_bfloat16, 1>));
  else
    MM_TRY(wide ? go(k_combine<float, 8>) : go(k_combine<float, 1>));
  return MM_OK;
}

mm_status mm_expert_combine_backward(const mm_expert_desc* d, const void* dy, const void* rows,
                                     const int32_t* offsets, const int32_t* row_of_slot,
                                     const float* weights, void* d_rows, float* d_weights,
                                     void* stream) {
  mm_status s = check_desc(d, true);
  if (s != MM_OK) return s;
  const size_t es = d->type == MM_BF16 ? 2 : 4;
  if (!aligned_to(dy, es) || !aligned_to(rows, es) || !aligned_to(d_rows, es) || !aligned_to(offsets, 4) ||
      !aligned_to(row_of_slot, 4) || !aligned_to(weights, 4) || !aligned_to(d_weights, 4))
    return MM_ERR_INVALID_ARG;
  if (d->T == 0) return MM_OK;
  if (!dy || !offsets || !row_of_slot || !d_rows || (d_weights && !rows)) return MM_ERR_INVALID_ARG;
  clear_error();
  RowArgs a = row_args(*d);
  a.x = dy;
  a.rows = rows;
  a.offsets = offsets;
  a.row_of_slot = row_of_slot;
  a.weights = weights;
  a.out_rows = d_rows;
  a.d_weights = d_weights;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const bool wide = d->H % 8 == 0 && aligned_to(dy, 16) && aligned_to(rows, 16) && aligned_to(d_rows, 16);
  a.words = (int)(wide ? d->H / 8 : d->H);
  auto go = [&](auto* kernel) {
    return launch_pdl(kernel, dim3((unsigned)d->T), dim3(threads_for(a.words)), 0, st, a);
  };
  auto by_slots = [&](auto type, auto width) {
    using T = decltype(type);
    constexpr int W = decltype(width)::value;
    return d->K <= 2 ? go(k_combine_bwd<T, W, 2>) : go(k_combine_bwd<T, W, 8>);
  };
  using Eight = std::integral_constant<int, 8>;
  using One = std::integral_constant<int, 1>;
  if (d->type == MM_BF16)
    MM_TRY(wide ? by_slots(__nv_bfloat16{}, Eight{}) : by_slots(__nv_bfloat16{}, One{}));
  else
    MM_TRY(wide ? by_slots(float{}, Eight{}) : by_slots(float{}, One{}));
  return MM_OK;
}

}  // extern "C"
