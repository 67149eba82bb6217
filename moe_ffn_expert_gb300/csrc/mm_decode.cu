// The whole MoE layer for a few tokens (mm_decode) and the quantiser of its 8-bit weights.
//
// With few tokens every selected expert's weights are read for a handful of rows: the layer is
// bound by HBM, 3 H I weights per expert against 6 H I multiply-adds per slot. Two launches:
//
//   k_logits  the router product (fp32 sums of bf16 x bf16 or bf16 x fp32 products) over all SMs,
//             and zeroed counters for the second kernel;
//   k_experts one CTA per SM. Every CTA derives the same routing tables from the logits (or the
//             caller's ids) in shared memory, then takes work units from one global counter:
//     GEMM1   (chunk of up to 32 (e4m3: 16) rows of one expert, 64 (e4m3: 128) gate columns and the
//             same of up): w * silu(g) * u
//     GEMM2   (chunk, 128 output columns, part of I): fp32 partial rows
//   and when they are out, sums the partial rows of (token, 128 columns) tasks in slot order, dealt
//   evenly to the warps of the grid.
//
// A GEMM2 unit needs its chunk's GEMM1 units, a sum its columns' GEMM2 units: counters in the
// workspace, waited for at the last moment and only for the small operand, so the weight loads of
// the next units run ahead through the wait. Units are claimed in that order, and a CTA works
// through its units in the order it claimed them, so what a unit waits for is always held by a CTA
// that is running or done: no wait depends on how many CTAs are resident.
//
// From 13 tokens on, the selection runs as a launch of the router's kernel between the two: a CTA
// that selects for 64 tokens itself takes 13 us, one per warp for up to 12 tokens 2.6.
//
// The products run on tcgen05.mma with the weights as the M = 128 operand, straight from the
// row-major tiles that TMA brings (MN-major descriptors), and the chunk's rows as N: 16 or 32
// columns of the accumulator instead of 128 rows of padding. No thread touches a weight.
//
// h goes from the first product to the second as the sum of two bf16 parts, each a column of N of its
// own, so that y's rounding is the only one to 16 bits: y is off by 1.67e-3 in the mean square, as the
// rounded exact y is (one part: 2.36e-3). The second product's N is up to 64 and a stage's rows take twice
// the room, for one stage of weights fewer: 64 tokens of 128 experts 182.6 us, 181.0 with one part.
//
// e4m3 weights meet 16-bit activations: tensor cores take either both in 8 bits or both in 16.
// A bf16 number is the exact sum of two e4m3 numbers, x s = hi + lo / 16 (4 significant bits
// each, s a power of two per row that keeps the row's largest value below 256; what lies 2^-20
// below that is rounded), so both halves of every row are columns of N and the accumulator's two
// columns are added: twice the columns, no conversion of the weights, which outnumber the rows'
// elements many times. The products of 128 x 128 blocks are scaled in 32 bits as they leave the
// tensor memory. h, which has more bits than a bf16 number, is split the same way into three parts
// (2^-12 of a value is left out), with a scale per row and 128 columns: y is off by 1.66e-3, the rounding
// of y, where two parts left 1.77e-3. 64 tokens of 128 experts take 107 us, 109 with two parts; 33 tokens
// of 32 experts with a shared one 41.0, 39.7; one token 24.6, 23.7.
//
// Measured (device time of a call; the floor is the hit experts' bytes at a plain copy's rate):
// 128 experts of 2048 x 768, top-8, bf16: 64 tokens 182 us, 6.5 TB/s (floor 175); 8 tokens 77 (72);
// one token 24.1 (11): logits 2, tables 2.6, the first weights 1.8, GEMM2 behind GEMM1, the sums 2.
// e4m3: one token 24.7 us (5.6), 8 tokens 49 (36), 64 tokens 107 (88); 256 experts of 7168 x 2048, 16
// tokens: 614-637 us, 7.1-7.3 TB/s (663: weights alone stream a little faster than a copy).
#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>

#include "mm_kernels.h"
#include "mm_select.cuh"

namespace mm {
namespace {

constexpr int kMaxT = 64, kMaxSlots = 1024, kMaxE = 1024;
constexpr int kMaxRouted = 12;    // tokens whose selection every CTA repeats, one per warp
constexpr int kRanked = 128;      // slots that are sorted by comparing each with all
constexpr int kCols = 128;        // weight columns per unit
constexpr int kMaxSplit = 4;      // parts of I per GEMM2 column tile
constexpr int kTileBytes = 16384; // one block of weights: 64 x 128 bf16 or 128 x 128 e4m3
constexpr int kThreads = 384;     // weight loads, row loads, MMA, tensor memory; 2 x 4 epilogue
constexpr int kFirstEpilogue = 4;
constexpr int kQueue = 8;         // units claimed ahead
constexpr uint64_t kTimeoutNs = 2000000000ull;

template <bool FP8>
struct Cfg {
  // Rows of one expert per unit. e4m3: 16, so that four accumulators fit per epilogue set; with
  // two the sets' work at the end of a unit stopped the products.
  static constexpr int CHUNK = FP8 ? 16 : 32;
  static constexpr int KB = FP8 ? 128 : 64;   // k of a block: 128 bytes of a row
  // Blocks of weights per stage. e4m3: two, which a warp waits for, issues and commits together:
  // with one the products' warp took some 540 cycles a block, and a block arrives every 690. GEMM1:
  // gate and up columns of the same k; GEMM2: the next two k.
  static constexpr int BLOCKS = FP8 ? 2 : 1;
  static constexpr int KB2 = KB * BLOCKS;             // k per stage of GEMM2
  static constexpr int A_BYTES = BLOCKS * kTileBytes;
  // parts of a row of x and of h (see above), and the rows of a stage: the larger of the two
  static constexpr int X_PARTS = FP8 ? 2 : 1, H_PARTS = FP8 ? 3 : 2;
  static constexpr int B_BYTES = BLOCKS * H_PARTS * CHUNK * 128;
  static constexpr int STAGES = FP8 ? 4 : 7;
  // columns of h that a GEMM1 unit makes. bf16: 64, from stages of 64 gate + 64 up columns. e4m3:
  // 128, so that a block is one box of whole 128-byte lines: two boxes of 64 bytes a row stream at
  // 6.3 TB/s, one of 128 at 7.1.
  static constexpr int H_COLS = FP8 ? 128 : 64;
  // Accumulators in tensor memory, a ring per epilogue set. bf16: a slot per unit (32 columns in GEMM1,
  // 64 in GEMM2). e4m3: a slot per stage in GEMM1 (32 columns, the parts of 16 rows, for each block),
  // one per block in GEMM2 (48 columns).
  static constexpr int SLOT_COLS = 64;
  static constexpr int RING = 512 / SLOT_COLS / 2;
};

// int32 words at the start of the workspace (zeroed by k_logits)
enum { W_STATUS = 0, W_NEXT = 1, W_READY1 = 64 };

struct DecodeArgs {
  CUtensorMap up, down, s_up, s_down;  // weights, boxes of 128 bytes x 64 (e4m3: 128) rows
  CUtensorMap x;                       // token rows (e4m3: hi and lo parts in turn), one per box
  CUtensorMap h_rows, s_h_rows;        // rows of h (their parts in turn), 8 per box
  const float *up_scale, *down_scale, *s_up_scale, *s_down_scale;
  const float* logits;    // with a router
  const float* bias;
  int32_t* ids;           // router: output or null; else input
  float* weights;
  __nv_bfloat16* y;
  int* hdr;
  int *ready1, *ready2;
  void *h, *s_h;           // [S, parts, I], [T, parts, Is]
  const float* x_scale;    // e4m3: [T]
  float *h_scale, *s_h_scale;  // e4m3: [chunk][ceil(I / 128)][16]
  float *o, *s_o;          // [split][S, H], [split][T, H]
  int T, H, I, E, K, S, Is, score, normalize, route;
  float scale;
};

// What a CTA keeps of the routing.
struct Tables {
  float w[kMaxSlots];          // weight of a sorted row
  int16_t tok[kMaxSlots];      // token of a sorted row
  int16_t row[kMaxSlots];      // sorted row of a slot
  uint16_t chunk_row[kMaxSlots];
  uint16_t chunk_e[kMaxSlots];
  uint8_t chunk_n[kMaxSlots];
  int chunks, bad;
};

// What only building the tables needs (in the stage ring's memory).
struct Building {
  float slot_w[kMaxSlots];     // weight of a slot
  int16_t id[kMaxSlots];       // expert of a slot
  uint8_t rank[kMaxSlots];     // slots of the same expert before it in its batch of 32
  uint32_t count[kMaxE];       // slots | chunks << 16, then the exclusive sums
  uint32_t warp_sum[32];
  // then uint16_t [batches][E]: an expert's slots per batch, then those of the batches before; and
  // with a router fp32 [T][E] logits
};

// A work unit as its claimer describes it to the CTA's other warps (one place computes it: code
// that runs once costs more to fetch than to execute).
struct Unit {
  int kind;  // 0 GEMM1, 1 GEMM2, -1 no more units
  int shared, row0, n, e, tile, kb0, kb1, split, ready;  // kb: stages
};

// Work units in claiming order: of each product the shared expert's before the others, as they are
// the longest when it is wider (33 tokens, 1536 beside 768: 53 us, 58 with them last).
struct Work {
  int nc, ncs, nt1, nt1s, nt2, split, splits, kb_h, kb_i, kb_is, t1s, t1, t2s, total, chunk;
};

// A value that all lanes share, in the form the compiler knows to be shared.
__device__ __forceinline__ int uniform(int v) { return __reduce_min_sync(0xFFFFFFFFu, v); }

// A ring's stage barriers as one warp in step walks them. The next stage is asked for before the
// current one's work is issued, so that the answer's latency passes behind it: ~100 cycles of a
// stage's ~350.
template <int STAGES>
struct Walk {
  uint32_t bar0, phase;  // first barrier; parity to wait for
  int s = 0;
  bool ready = false;
  __device__ __forceinline__ Walk(uint32_t bar, uint32_t first) : bar0(bar), phase(first) {}
  // Stage s is there (true in every lane), or the wait ran out.
  __device__ __forceinline__ bool wait() {
    if (__all_sync(0xFFFFFFFFu, ready)) return true;
    return __all_sync(0xFFFFFFFFu, mbar_wait(bar0 + 8u * s, phase, kTimeoutNs));
  }
  __device__ __forceinline__ void ask_next() {
    const bool wrap = s + 1 == STAGES;
    ready = mbar_test_wait(bar0 + 8u * (wrap ? 0 : s + 1), wrap ? phase ^ 1u : phase);
  }
  __device__ __forceinline__ void next() {
    if (++s == STAGES) s = 0, phase ^= 1u;
  }
};

// The e4m3 part of a value below 256, which becomes 16 times what is left of it (below 256 again):
// v = hi + lo / 16 (+ lo2 / 256).
__device__ __forceinline__ uint8_t take_e4m3(float& v) {
  const uint8_t part = __nv_cvt_float_to_fp8(v, __NV_SATFINITE, __NV_E4M3);
  const __half_raw h = __nv_cvt_fp8_to_halfraw(part, __NV_E4M3);
  v = (v - __half2float(*reinterpret_cast<const __half*>(&h))) * 16.f;
  return part;
}

// hi + lo / 16 of two parts' products.
__device__ __forceinline__ float whole(uint32_t hi, uint32_t lo) {
  return fmaf(__uint_as_float(lo), 0.0625f, __uint_as_float(hi));
}

// What a rounded part leaves of a value: nothing of an infinity or a NaN.
__device__ __forceinline__ float rest_of(float v, float part) {
  return fabsf(part) <= 3.4e38f ? v - part : 0.f;
}

__device__ __forceinline__ uint32_t word_of(const uint8_t* b) {
  return (uint32_t)b[0] | (uint32_t)b[1] << 8 | (uint32_t)b[2] << 16 | (uint32_t)b[3] << 24;
}

// The power of two that brings a largest magnitude into [128, 256) and its inverse. `amax` that is
// not finite: the inverse is NaN, so that whatever the row's products are multiplied with it is.
__device__ __forceinline__ float split_scale(float amax, float* inverse) {
  int e = (int)((__float_as_uint(amax) >> 23) & 0xFFu) - 127;
  const bool bad = e == 128;
  e = max(e, -100);  // zero and tiny rows
  *inverse = bad ? __int_as_float(0x7FC00000) : __uint_as_float((uint32_t)(e - 7 + 127) << 23);
  return bad ? 0.f : __uint_as_float((uint32_t)(7 - e + 127) << 23);
}

// ---------------------------------------------------------------------------------- k_logits

struct LogitArgs {
  const __nv_bfloat16* x;
  const void* router;
  float* logits;
  int* zero;  // words to clear
  int zero_n;
  int T, H, E;
  int logit_blocks;  // then, for e4m3 weights, one block per token
  uint8_t* x8;       // [T, 2, H]: hi and lo parts
  float* x_scale;    // [T]
};

// Row t of x as e4m3 hi and lo parts.
__device__ void split_row(const LogitArgs& a, int t, float* red) {
  const int tid = threadIdx.x;
  const __nv_bfloat16* row = a.x + (int64_t)t * a.H;
  float m = 0.f;
  bool nan = false;
  for (int c = tid * 8; c < a.H; c += 256 * 8) {
    float v[8];
    load_vec<8>(row + c, v);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      nan |= v[k] != v[k];
      m = fmaxf(m, fabsf(v[k]));
    }
  }
  m = warp_max(m);
  if ((tid & 31) == 0) red[tid >> 5] = m;
  nan = __syncthreads_or(nan);
  m = red[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) m = fmaxf(m, red[i]);
  float inv;
  const float s = split_scale(nan ? INFINITY : m, &inv);
  if (tid == 0) a.x_scale[t] = inv;
  uint8_t* hi = a.x8 + (int64_t)t * 2 * a.H;
  uint8_t* lo = hi + a.H;
  for (int c = tid * 8; c < a.H; c += 256 * 8) {
    float v[8];
    load_vec<8>(row + c, v);
    uint8_t h[8], l[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      float rest = v[k] * s;
      h[k] = take_e4m3(rest);
      l[k] = take_e4m3(rest);
    }
    *reinterpret_cast<uint2*>(hi + c) = make_uint2(word_of(h), word_of(h + 4));
    *reinterpret_cast<uint2*>(lo + c) = make_uint2(word_of(l), word_of(l + 4));
  }
}

// N experts x N tokens per block, H dealt to the 8 warps; the N^2 sums of a warp's lanes are
// reduced by halving exchanges, the warps' sums in order. N = 4 reads x and the router 4 times
// less; N = 1 is a quarter of the code, which costs more than its reads when they are few.
template <typename RT, int N>
__global__ void __launch_bounds__(256) k_logits(LogitArgs a) {
  __shared__ float part[8][N * N < 8 ? 8 : N * N];
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  for (int i = (int)blockIdx.x * 256 + tid; i < a.zero_n; i += (int)gridDim.x * 256) a.zero[i] = 0;
  if ((int)blockIdx.x >= a.logit_blocks) {
    if (a.x8 != nullptr) split_row(a, (int)blockIdx.x - a.logit_blocks, &part[0][0]);
    return;
  }
  const int eb = (a.E + N - 1) / N;
  const int e0 = (int)blockIdx.x % eb * N, t0 = (int)blockIdx.x / eb * N;
  float acc[N * N];
#pragma unroll
  for (int i = 0; i < N * N; ++i) acc[i] = 0.f;
#pragma unroll 1
  for (int c = tid * 8; c < a.H; c += 256 * 8) {
    float w[N][8], x[N][8];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      load_vec<8>(static_cast<const RT*>(a.router) + (int64_t)min(e0 + i, a.E - 1) * a.H + c, w[i]);
      load_vec<8>(a.x + (int64_t)min(t0 + i, a.T - 1) * a.H + c, x[i]);
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int j = 0; j < N; ++j)
#pragma unroll
        for (int k = 0; k < 8; ++k) acc[i * N + j] = fmaf(w[i][k], x[j][k], acc[i * N + j]);
  }
  const float s = warp_sum_many<N * N>(acc, lane);
  if (lane % (32 / (N * N)) == 0) part[warp][lane / (32 / (N * N))] = s;
  __syncthreads();
  if (tid < N * N) {
    float v = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) v += part[i][tid];
    const int e = e0 + tid / N, t = t0 + tid % N;
    if (e < a.E && t < a.T) a.logits[(int64_t)t * a.E + e] = v;
  }
}

// ---------------------------------------------------------------------------------- k_experts

template <int NV>
__device__ void select_row(const DecodeArgs& a, Building& bd, const float* row, int t, int lane) {
  uint32_t key[NV];
  float z[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int e = lane * NV + j;
    z[j] = e < a.E ? row[e] : 0.f;
  }
  float m = -INFINITY, sum = 0.f;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int e = lane * NV + j;
    key[j] = 0;
    if (e >= a.E) continue;
    float k = z[j];
    if (a.bias != nullptr) k = (a.score == MM_SCORE_SIGMOID ? sigmoid_accurate(k) : k) + a.bias[e];
    key[j] = order_key(k);
    m = fmaxf(m, z[j]);
  }
  if (a.score == MM_SCORE_SOFTMAX && !a.normalize) {
    m = warp_max(m);
    if (m == -INFINITY) m = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (lane * NV + j < a.E) sum += expf(z[j] - m);
    sum = warp_sum(sum);
  }
  const int id = select_topk<NV>(key, a.K, lane, bd.id + t * a.K);
  const float zs = lane < a.K ? row[id] : 0.f;
  const float w = selected_weight(zs, lane < a.K, a.score, a.normalize, a.scale, m, sum);
  if (lane < a.K) {
    bd.slot_w[t * a.K + lane] = w;
    if (blockIdx.x == 0) {
      if (a.ids != nullptr) a.ids[t * a.K + lane] = id;
      if (a.weights != nullptr) a.weights[t * a.K + lane] = w;
    }
  }
}

// Routing tables of the CTA: the slots sorted by expert (stable), cut into chunks. The same in
// every CTA. False if a caller's id is out of range.
__device__ bool build_tables(const DecodeArgs& a, Tables& tb, uint8_t* ring, int chunk) {
  Building& bd = *reinterpret_cast<Building*>(ring);
  uint16_t* before_batch = reinterpret_cast<uint16_t*>(ring + sizeof(Building));
  float* ls = reinterpret_cast<float*>(ring + sizeof(Building));  // (used before it)
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) tb.bad = 0;
  if (tid < 8 && a.S + tid < kMaxSlots) bd.id[a.S + tid] = 0x7FFF;  // above every expert
  if (a.route) {
    // a row's selection starts from shared memory (kMaxRouted rows of at most 1024 fit)
    const int n = a.T * a.E;
#pragma unroll 4
    for (int i = tid; i < n; i += kThreads) ls[i] = __ldcg(a.logits + i);
    __syncthreads();
    for (int t = warp; t < a.T; t += kThreads / 32) {
      const float* row = ls + t * a.E;
      if (a.E <= 32) select_row<1>(a, bd, row, t, lane);
      else if (a.E <= 64) select_row<2>(a, bd, row, t, lane);
      else if (a.E <= 128) select_row<4>(a, bd, row, t, lane);
      else if (a.E <= 256) select_row<8>(a, bd, row, t, lane);
      else if (a.E <= 512) select_row<16>(a, bd, row, t, lane);
      else select_row<32>(a, bd, row, t, lane);
    }
    __syncthreads();
  } else {
    __syncthreads();
    for (int s = tid; s < a.S; s += kThreads) {
      const int e = a.ids[s];
      if (e < 0 || e >= a.E) tb.bad = 1;
      bd.id[s] = (int16_t)e;
      bd.slot_w[s] = a.weights[s];
    }
    __syncthreads();
    if (tb.bad) {
      if (tid == 0) set_status(a.hdr + W_STATUS, MM_ERR_BAD_EXPERT_ID);
      return false;
    }
  }
  if (a.S <= chunk) {  // one warp, one slot per lane; experts in the order of their first slots
    if (warp == 0) {
      const int e = lane < a.S ? bd.id[lane] : -1 - lane;
      const uint32_t same = __match_any_sync(0xFFFFFFFFu, e);
      const int leader = __ffs(same) - 1, n = __popc(same);
      const bool leads = leader == lane && lane < a.S;
      const uint32_t leaders = __ballot_sync(0xFFFFFFFFu, leads);
      int sum = leads ? n : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xFFFFFFFFu, sum, o);
        if (lane >= o) sum += v;
      }
      const int first = __shfl_sync(0xFFFFFFFFu, sum - (leads ? n : 0), leader);
      if (lane < a.S) {
        const int r = first + __popc(same & ((1u << lane) - 1u));
        tb.row[lane] = (int16_t)r;
        tb.tok[r] = (int16_t)(lane / a.K);
        tb.w[r] = bd.slot_w[lane];
        if (leads) {
          const int c = __popc(leaders & ((1u << lane) - 1u));
          tb.chunk_row[c] = (uint16_t)r;
          tb.chunk_e[c] = (uint16_t)e;
          tb.chunk_n[c] = (uint8_t)n;
        }
      }
      if (lane == 0) tb.chunks = __popc(leaders);
    }
    fence_proxy_async_smem();
    __syncthreads();
    return true;
  }
  if (a.S <= kRanked) {
    // A slot's row is the number of slots of a lower expert or of its own and an earlier number, 8
    // comparisons per load; a chunk's number is that of the chunks that begin in rows before. (The
    // way below takes 2 us longer for 64 slots; this one 2 us longer for 198.)
    int e = 0, row = 0, before = 0, same = 0;
    if (tid < a.S) {
      e = bd.id[tid];
      for (int i = 0; i < a.S; i += 8) {
        const uint4 v = *reinterpret_cast<const uint4*>(bd.id + i);
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int x = (int)(u[j >> 1] >> (j & 1) * 16 & 0xFFFFu);
          row += x < e;
          same += x == e;
          before += x == e && i + j < tid;
        }
      }
      row += before;
      tb.row[tid] = (int16_t)row;
      tb.tok[row] = (int16_t)(tid / a.K);
      tb.w[row] = bd.slot_w[tid];
      bd.rank[row] = before % chunk == 0;  // a chunk begins
    }
    __syncthreads();
    if (warp < kRanked / 32) {
      const uint32_t begins = __ballot_sync(0xFFFFFFFFu, tid < a.S && bd.rank[tid]);
      if (lane == 0) bd.warp_sum[warp] = begins;
    }
    __syncthreads();
    int total = 0, c = 0;
#pragma unroll
    for (int i = 0; i < kRanked / 32; ++i) {
      if (i == row >> 5) c = total + __popc(bd.warp_sum[i] & ((1u << (row & 31)) - 1u));
      total += __popc(bd.warp_sum[i]);
    }
    if (tid < a.S && before % chunk == 0) {
      tb.chunk_row[c] = (uint16_t)row;
      tb.chunk_e[c] = (uint16_t)e;
      tb.chunk_n[c] = (uint8_t)min(chunk, same - before);
    }
    if (tid == 0) tb.chunks = total;
    fence_proxy_async_smem();
    __syncthreads();
    return true;
  }
  // A slot's row is the first row of its expert, plus the expert's slots in the batches before,
  // plus those before it in its batch: all batches at once, then all experts, then all slots.
  // (One warp walking the slots took 6 us for 512.)
  const int batches = (a.S + 31) / 32;
  for (int i = tid; i < batches * a.E; i += kThreads) before_batch[i] = 0;
  __syncthreads();
  for (int b = warp; b < batches; b += kThreads / 32) {
    const int s = b * 32 + lane;
    const int e = s < a.S ? bd.id[s] : -1 - lane;
    const uint32_t same = __match_any_sync(0xFFFFFFFFu, e);
    if (s < a.S) {
      const int rank = __popc(same & ((1u << lane) - 1u));
      bd.rank[s] = (uint8_t)rank;
      if (rank == 0) before_batch[b * a.E + e] = (uint16_t)__popc(same);
    }
  }
  __syncthreads();
  // slots (low half) and chunks (high half) of the experts before, summed over the block; a thread
  // takes up to three consecutive experts
  const int per = (a.E + kThreads - 1) / kThreads, e0 = min(a.E, tid * per), e1 = min(a.E, e0 + per);
  uint32_t sum = 0;
  for (int e = e0; e < e1; ++e) {
    uint32_t n = 0;
    for (int b = 0; b < batches; ++b) {
      const uint32_t here = before_batch[b * a.E + e];
      before_batch[b * a.E + e] = (uint16_t)n;
      n += here;
    }
    bd.count[e] = n | ((n + chunk - 1) / (uint32_t)chunk) << 16;
    sum += bd.count[e];
  }
  uint32_t before = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, before, o);
    if (lane >= o) before += v;
  }
  if (lane == 31) bd.warp_sum[warp] = before;
  __syncthreads();
  before -= sum;
  const uint32_t others = lane < kThreads / 32 ? bd.warp_sum[lane] : 0u;
  before += __reduce_add_sync(0xFFFFFFFFu, lane < warp ? others : 0u);
  const uint32_t total = __reduce_add_sync(0xFFFFFFFFu, others);
  if (tid == 0) tb.chunks = (int)(total >> 16);
  for (int e = e0; e < e1; ++e) {
    const uint32_t n = bd.count[e];
    bd.count[e] = before;
    const int first = (int)(before & 0xFFFFu), rows = (int)(n & 0xFFFFu);
    for (int c = 0; c < (int)(n >> 16); ++c) {
      const int at = (int)(before >> 16) + c;
      tb.chunk_row[at] = (uint16_t)(first + c * chunk);
      tb.chunk_e[at] = (uint16_t)e;
      tb.chunk_n[at] = (uint8_t)min(chunk, rows - c * chunk);
    }
    before += n;
  }
  __syncthreads();
  for (int s = tid; s < a.S; s += kThreads) {
    const int e = bd.id[s];
    const int r = (int)(bd.count[e] & 0xFFFFu) + before_batch[(s >> 5) * a.E + e] + bd.rank[s];
    tb.row[s] = (int16_t)r;
    tb.tok[r] = (int16_t)(s / a.K);
    tb.w[r] = bd.slot_w[s];
  }
  // the ring is TMA's from here on
  fence_proxy_async_smem();
  __syncthreads();
  return true;
}

template <bool FP8>
__device__ __forceinline__ Work make_work(const DecodeArgs& a, int chunks) {
  constexpr int KB = Cfg<FP8>::KB, KB2 = Cfg<FP8>::KB2;
  Work w;
  w.nc = chunks;
  constexpr int CHUNK = Cfg<FP8>::CHUNK;
  w.ncs = a.Is > 0 ? (a.T + CHUNK - 1) / CHUNK : 0;
  w.chunk = CHUNK;
  w.nt1 = (a.I + Cfg<FP8>::H_COLS - 1) / Cfg<FP8>::H_COLS;
  w.nt1s = (a.Is + Cfg<FP8>::H_COLS - 1) / Cfg<FP8>::H_COLS;
  w.nt2 = (a.H + kCols - 1) / kCols;
  w.kb_h = (a.H + KB - 1) / KB;
  w.kb_i = (a.I + KB2 - 1) / KB2;
  w.kb_is = (a.Is + KB2 - 1) / KB2;
  // GEMM2 units too few for the SMs are cut along I
  const int units = (w.nc + w.ncs) * w.nt2;
  const int want = max(1, min(kMaxSplit, (int)gridDim.x / max(1, units)));
  w.split = min(want, w.kb_i);
  w.splits = min(want, max(1, w.kb_is));
  w.t1s = w.ncs * w.nt1s;
  w.t1 = w.t1s + w.nc * w.nt1;
  w.t2s = w.t1 + w.ncs * w.nt2 * w.splits;
  w.total = w.t2s + w.nc * w.nt2 * w.split;
  return w;
}

// u / d for 0 <= u < 2^21: a reciprocal and a correction instead of the integer division's code.
__device__ __forceinline__ int div_small(int u, int d) {
  int q = (int)__fdividef((float)u + 0.5f, (float)d);
  if (q * d > u) --q;
  if ((q + 1) * d <= u) ++q;
  return q;
}

__device__ __forceinline__ Unit unit_at(const DecodeArgs& a, const Tables& tb, const Work& w,
                                        int u) {
  Unit r;
  r.kind = -1;
  if (u >= w.total) return r;
  r.shared = 0;
  r.split = 0;
  int c;
  if (u < w.t1) {
    r.kind = 0;
    r.shared = u < w.t1s;
    const int v = r.shared ? u : u - w.t1s, nt = r.shared ? w.nt1s : w.nt1;
    c = div_small(v, nt);
    r.tile = v - c * nt;
    r.kb0 = 0;
    r.kb1 = w.kb_h;
  } else {
    r.kind = 1;
    r.shared = u < w.t2s;
    const int v = u - (r.shared ? w.t1 : w.t2s), sp = r.shared ? w.splits : w.split;
    const int kb = r.shared ? w.kb_is : w.kb_i;
    c = div_small(v, w.nt2 * sp);
    const int rest = v - c * w.nt2 * sp;
    r.tile = sp == 1 ? rest : div_small(rest, sp);
    r.split = rest - r.tile * sp;
    r.kb0 = sp == 1 ? 0 : div_small(kb * r.split, sp);
    r.kb1 = sp == 1 ? kb : div_small(kb * (r.split + 1), sp);
  }
  if (r.shared) {
    r.row0 = c * w.chunk;
    r.n = min(w.chunk, a.T - r.row0);
    r.e = 0;
    r.ready = w.nc + c;
  } else {
    r.row0 = tb.chunk_row[c];
    r.n = tb.chunk_n[c];
    r.e = tb.chunk_e[c];
    r.ready = c;
  }
  return r;
}

template <bool FP8>
__global__ void __launch_bounds__(kThreads, 1) k_experts(const __grid_constant__ DecodeArgs a) {
  using C = Cfg<FP8>;
  constexpr int KB = C::KB, STAGES = C::STAGES, RING = C::RING;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Tables tb;
  __shared__ Unit queue[kQueue];
  __shared__ uint64_t bars[2 * STAGES + 3 * kQueue + 4 * RING + 4 + 1];
  __shared__ uint32_t tmem_slot;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // the stages' weights and rows (1024-byte aligned for the swizzle), then [row][128 columns] of
  // a unit for each epilogue set
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* const aligned = smem_raw + (base - smem_u32(smem_raw));
  const uint32_t rows_at = base + STAGES * C::A_BYTES;
  float* const exchange = reinterpret_cast<float*>(aligned + STAGES * (C::A_BYTES + C::B_BYTES));
  const uint32_t bar0 = smem_u32(bars);
  constexpr int Q = 2 * STAGES, ACC = Q + 3 * kQueue, X = ACC + 4 * RING;
  auto full = [&](int s) { return bar0 + 8u * s; };
  auto empty = [&](int s) { return bar0 + 8u * (STAGES + s); };
  auto q_full = [&](int s) { return bar0 + 8u * (Q + s); };
  auto q_empty = [&](int s) { return bar0 + 8u * (Q + kQueue + s); };
  auto stored = [&](int s) { return bar0 + 8u * (Q + 2 * kQueue + s); };
  auto acc_full = [&](int set, int s) { return bar0 + 8u * (ACC + set * RING + s); };
  auto acc_empty = [&](int set, int s) { return bar0 + 8u * (ACC + (2 + set) * RING + s); };
  auto x_full = [&](int s) { return bar0 + 8u * (X + s); };
  auto x_empty = [&](int s) { return bar0 + 8u * (X + 2 + s); };
  const uint32_t mma_done = bar0 + 8u * (X + 4);
  if (tid == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full(s), 2);  // the weights' and the rows' producers
      mbar_init(empty(s), 1);
    }
    for (int s = 0; s < kQueue; ++s) {
      mbar_init(q_full(s), 1);
      mbar_init(q_empty(s), 3 + 8);  // row loads, MMA, releases, epilogue warps
      mbar_init(stored(s), 4);
    }
    for (int s = 0; s < 2 * RING; ++s) {
      mbar_init(acc_full(0, s), 1);
      mbar_init(acc_empty(0, s), 4);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(x_full(s), 4);
      mbar_init(x_empty(s), 4);
    }
    mbar_init(mma_done, 1);
    mbar_fence_init();
    tma_prefetch_desc(&a.up);
    tma_prefetch_desc(&a.down);
    tma_prefetch_desc(&a.x);
    tma_prefetch_desc(&a.h_rows);
  }
  if (warp == 3) {
    tmem_alloc(smem_u32(&tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  pdl_wait();
  // The first unit is claimed like the others, so that no unit belongs to a CTA that is not running;
  // the claim's latency passes behind the tables.
  int first_unit = 0;
  if (tid == 0) first_unit = atomicAdd(a.hdr + W_NEXT, 1);
  const bool good = build_tables(a, tb, aligned, C::CHUNK);  // (its barriers publish the mbarriers and tmem_slot)
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  const Work work = make_work<FP8>(a, good ? tb.chunks : 0);
  // a wait that runs out ends its role; the roles that depend on it run out in turn
  auto give_up = [&] { set_status(a.hdr + W_STATUS, MM_ERR_TIMEOUT); };
  // entry qi of the queue (null: the wait ran out), every lane
  auto take = [&](int qi) -> const Unit* {
    if (mbar_wait(q_full(qi % kQueue), (qi / kQueue) & 1, kTimeoutNs)) return &queue[qi % kQueue];
    if (lane == 0) give_up();
    return nullptr;
  };
  // the warp has read its entry
  auto taken = [&](int qi) {
    __syncwarp();
    if (lane == 0) mbar_arrive(q_empty(qi % kQueue));
  };

  if (!good && warp < kFirstEpilogue) {
    // a caller's id is out of range: nothing to do but y
  } else if (warp == 0) {
    // ------------------------------------------------ claims units and loads their weights
    int u = __shfl_sync(0xFFFFFFFFu, first_unit, 0), it = 0;
    Walk<STAGES> ring(empty(0), 1);
    bool ok = true;
    for (int qi = 0; ok; ++qi) {
      const int qs = qi % kQueue;
      if (!mbar_wait(q_empty(qs), ((qi / kQueue) & 1) ^ 1, kTimeoutNs)) {
        if (lane == 0) give_up();
        break;
      }
      const Unit un = unit_at(a, tb, work, u);
      if (lane == 0) {
        queue[qs] = un;
        mbar_arrive(q_full(qs));
      }
      if (un.kind < 0) break;
      const CUtensorMap* map = un.kind == 0 ? (un.shared ? &a.s_up : &a.up)
                                            : (un.shared ? &a.s_down : &a.down);
      const int e = uniform(un.e), kb1 = uniform(un.kb1);
      const int c0 = uniform(un.tile * (un.kind == 0 ? C::H_COLS : kCols));
      const int c1 = uniform(un.kind == 0 ? (un.shared ? a.Is : a.I) + c0 : c0 + (FP8 ? 0 : 64));
      // k of the first and from there to the second half (bf16: columns) of a stage
      const int k_step = uniform(un.kind == 0 ? KB : C::KB2), k_half = uniform(FP8 && un.kind == 1 ? KB : 0);
      // The next unit is claimed with two stages of this one left, so that the claim's latency passes
      // behind them. (Not earlier: a CTA stuck in front of a chunk that is not ready should not sit on
      // units that others could take.)
      const int kb0 = uniform(un.kb0), claim_at = max(kb0, kb1 - 2);
      int next = 0;
      for (int kb = kb0; kb < kb1; ++kb, ++it) {
        if (kb == claim_at && lane == 0) next = atomicAdd(a.hdr + W_NEXT, 1);
        if (!ring.wait()) {
          if (lane == 0) give_up();
          ok = false;
          break;
        }
        ring.ask_next();
        if (elect_one()) {
          const uint32_t dst = base + ring.s * C::A_BYTES, bar = full(ring.s);
          mbar_arrive_expect_tx(bar, C::A_BYTES);
          tma_load_3d(dst, map, bar, c0, kb * k_step, e);
          tma_load_3d(dst + C::A_BYTES / 2, map, bar, c1, kb * k_step + k_half, e);
        }
        __syncwarp();
        ring.next();
      }
      u = __shfl_sync(0xFFFFFFFFu, next, 0);
    }
    // no CTA leaves with a copy into its shared memory in flight
    for (int j = max(0, it - STAGES); j < it; ++j)
      mbar_wait(full(j % STAGES), (j / STAGES) & 1, kTimeoutNs);
  } else if (warp == 1) {
    // ------------------------------------------------ loads the rows
    int it = 0;
    Walk<STAGES> ring(empty(0), 1);
    bool ok = true;
    for (int qi = 0; ok; ++qi) {
      const Unit* const entry = take(qi);
      if (entry == nullptr) break;
      const Unit un = *entry;
      taken(qi);
      if (un.kind < 0) break;
      const CUtensorMap* map = un.kind == 0 ? &a.x : un.shared ? &a.s_h_rows : &a.h_rows;
      // a lane loads 4 rows of x by number (e4m3: both parts of 2) or the parts of 8 consecutive rows
      // of h
      constexpr int PARTS = C::X_PARTS, X_ROWS = 4 / PARTS;
      const int groups = un.kind == 0 ? (un.n + X_ROWS - 1) / X_ROWS : (un.n + 7) / 8;
      int r[4] = {0, 0, 0, 0};
      if (un.kind == 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int row = un.row0 + min(lane * X_ROWS + i / PARTS, un.n - 1);
          r[i] = (un.shared ? row : tb.tok[row]) * PARTS + i % PARTS;
        }
      } else {
        // the chunk's rows of h: one count per GEMM1 unit
        const int target = un.shared ? work.nt1s : work.nt1;
        // (every lane acquires what it will load: a shuffle of lane 0's answer would order no memory)
        const bool there = wait_counter(a.ready1 + un.ready, target, kTimeoutNs);
        if (!__all_sync(0xFFFFFFFFu, there)) {
          if (lane == 0) give_up();
          break;
        }
        fence_proxy_async_global();
        r[0] = (un.row0 + 8 * lane) * C::H_PARTS;
      }
      const uint32_t lane_bytes = un.kind == 0 ? 512 : C::H_PARTS * 1024;
      const uint32_t bytes = groups * lane_bytes * (un.kind == 0 ? 1 : C::BLOCKS);
      const uint32_t to = rows_at + lane * lane_bytes;
      for (int kb = un.kb0; kb < un.kb1; ++kb, ++it) {
        if (!ring.wait()) {
          if (lane == 0) give_up();
          ok = false;
          break;
        }
        ring.ask_next();
        if (lane == 0) mbar_arrive_expect_tx(full(ring.s), bytes);
        __syncwarp();
        if (lane < groups) {
          const uint32_t dst = to + ring.s * C::B_BYTES;
          if (un.kind == 0)
            tma_gather4(dst, map, full(ring.s), kb * KB, r[0], r[1], r[2], r[3]);
          else
#pragma unroll
            for (int p = 0; p < C::BLOCKS; ++p)
              tma_load_2d(dst + p * (C::B_BYTES / C::BLOCKS), map, full(ring.s), kb * C::KB2 + p * KB, r[0]);
        }
        __syncwarp();
        ring.next();
      }
    }
    for (int j = max(0, it - STAGES); j < it; ++j)
      mbar_wait(full(j % STAGES), (j / STAGES) & 1, kTimeoutNs);
  } else if (warp == 2) {
    // ------------------------------------------------ issues the products
    // The warp stays in step, an elected lane issues, and what an issue takes is known to be the
    // same in all lanes: operands that are not pass through a move to a uniform register each, and
    // with descriptors built per product in a branch of one lane an issue took 165 cycles instead
    // of 41, longer than its weights take to arrive.
    // (a block of e4m3 weights is 128 columns of 128 bytes a row; of bf16, twice 64)
    const uint64_t wdesc = sdesc_sw128(base, kTileBytes / 2, 1024);
    const uint64_t bdesc = sdesc_sw128(rows_at, 16, 1024);
    Walk<STAGES> ring(full(0), 0);
    Walk<RING> accs[2] = {Walk<RING>(acc_empty(0, 0), 1), Walk<RING>(acc_empty(1, 0), 1)};
    bool ok = true;
    for (int qi = 0; ok; ++qi) {
      const Unit* const entry = take(qi);
      if (!__all_sync(0xFFFFFFFFu, entry != nullptr)) break;
      const int kind = uniform(entry->kind), blocks = uniform(entry->kb1 - entry->kb0);
      const int rows = uniform(entry->n);
      taken(qi);
      if (kind < 0) break;
      const uint32_t n = ((kind == 0 ? C::X_PARTS : C::H_PARTS) * rows + 15) & ~15;  // parts of the chunk's rows
      const uint32_t idesc = FP8 ? idesc_e4m3_f32(128, n, 1, 0) : idesc_bf16_f32(128, n, 1, 0);
      const int set = qi & 1;
      uint32_t d[2] = {0, 0};  // of the two blocks
      int slot[2] = {0, 0};
      auto next_slot = [&](int p) {  // the next accumulator of `set`, free
        Walk<RING>& w = set ? accs[1] : accs[0];
        if (w.wait()) {
          slot[p] = w.s;
          d[p] = tmem + (set * RING + w.s) * C::SLOT_COLS;
          tc_fence_after();
          return true;
        }
        if (lane == 0) give_up();
        return ok = false;
      };
      auto slot_done = [&] {
        Walk<RING>& w = set ? accs[1] : accs[0];
        w.ask_next();
        w.next();
      };
      if (!FP8 && !next_slot(0)) break;
      for (int i = 0; i < blocks; ++i) {
        if (FP8) {
          if (!next_slot(0)) break;
          d[1] = d[0] + C::SLOT_COLS / 2;
          if (kind == 1) {
            slot_done();
            if (!next_slot(1)) break;
          }
        }
        if (!ring.wait()) {
          if (lane == 0) give_up();
          ok = false;
          break;
        }
        ring.ask_next();
        tc_fence_after();
        if (elect_one()) {
          const uint64_t wd = wdesc + (uint32_t)ring.s * (C::A_BYTES / 16);
          const uint64_t bd = bdesc + (uint32_t)ring.s * (C::B_BYTES / 16);
          const uint32_t b_half = kind == 0 ? 0u : C::B_BYTES / 2 / 16;  // e4m3 GEMM1: the same rows
#pragma unroll
          for (int i4 = 0; i4 < 4 * C::BLOCKS; ++i4) {  // 16 (bf16) or 32 (e4m3) rows of weights
            const int p = i4 / 4, ks = i4 % 4;
            const uint64_t wk = wd + i4 * ((FP8 ? 4096 : 2048) / 16), bk = bd + ks * 2 + p * b_half;
            if constexpr (FP8)
              umma_e4m3(d[p], wk, bk, idesc, ks == 0 ? 0u : 1u);
            else
              umma_bf16(d[0], wk, bk, idesc, i == 0 && ks == 0 ? 0u : 1u);
          }
          umma_commit(empty(ring.s));
          if (FP8 || i + 1 == blocks) umma_commit(acc_full(set, slot[0]));
          if (FP8 && kind == 1) umma_commit(acc_full(set, slot[1]));
        }
        __syncwarp();
        ring.next();
        if (FP8) slot_done();
      }
      if (!FP8 && ok) slot_done();
    }
    if (elect_one()) umma_commit(mma_done);
    __syncwarp();
    mbar_wait(mma_done, 0, kTimeoutNs);
  } else if (warp == 3) {
    // ------------------------------------------------ releases the units' results
    // What the epilogue warps stored (ordered before this warp by their arrivals) is released to
    // the other CTAs here: a release waits until the stores are through, some 1000 cycles that
    // would otherwise stand between an epilogue warp's units.
    if (lane == 0) {
      for (int qi = 0;; ++qi) {
        const Unit* const entry = take(qi);
        if (entry == nullptr || entry->kind < 0) break;
        int* const counter = entry->kind == 0 ? a.ready1 + entry->ready : a.ready2 + entry->tile;
        if (!mbar_wait(stored(qi % kQueue), (qi / kQueue) & 1, kTimeoutNs)) {
          give_up();
          break;
        }
        fence_proxy_async_global();
        red_add_release_gpu(counter, 1);
        mbar_arrive(q_empty(qi % kQueue));
      }
    }
  } else if (warp >= kFirstEpilogue) {
    // ------------------------------------------------ accumulators to h, partial rows and y
    // Two sets of four warps take the units in turn.
    const int set = (warp - kFirstEpilogue) >> 2, q = warp & 3;  // q: the warp's quarter of the lanes
    const int col = q * 32 + lane;  // of the unit's 128
    const uint32_t tmem_q = tmem + set * RING * C::SLOT_COLS + ((uint32_t)(q * 32) << 16);
    int acc = 0;                    // accumulators taken from the ring
    int up_units = 0;               // GEMM1 units that this set finished
    bool ok = good;
    for (int qi = 0; ok; ++qi) {
      const Unit* const entry = take(qi);
      if (entry == nullptr) {
        ok = false;
        break;
      }
      const Unit un = *entry;
      taken(qi);
      if (un.kind < 0) break;
      if ((qi & 1) != set) continue;
      float* const ex = exchange + set * C::CHUNK * kCols + col;
      const int n8 = (un.n + 7) & ~7;
      const int I = un.shared ? a.Is : a.I;
      float x_scale = 1.f;  // of row `lane`
      if (FP8 && un.kind == 0 && lane < un.n)
        x_scale = __ldcg(a.x_scale + (un.shared ? un.row0 + lane : tb.tok[un.row0 + lane]));
      auto wait = [&](uint32_t bar, uint32_t phase) {
        if (mbar_wait(bar, phase, kTimeoutNs)) return true;
        if (lane == 0) give_up();
        return ok = false;
      };
      // this thread's column of rows j .. j + 7: GEMM1 to the exchange, GEMM2 to the partial rows
      const int c2 = un.tile * kCols + col;
      float* const o = (un.shared ? a.s_o + (int64_t)un.split * a.T * a.H
                                  : a.o + (int64_t)un.split * a.S * a.H) +
                       (int64_t)un.row0 * a.H + c2;
      auto emit = [&](const float* v, int j) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (j + i >= un.n) continue;
          if (un.kind == 0)
            ex[(j + i) * kCols] = v[i];
          else if (c2 < a.H)
            o[(int64_t)(j + i) * a.H] = v[i];
        }
      };
      if constexpr (!FP8) {
        if (un.kind == 0 && !wait(x_empty(set), (up_units & 1) ^ 1)) break;
        if (!wait(acc_full(set, acc % RING), (acc / RING) & 1)) break;
        tc_fence_after();
        const uint32_t d = tmem_q + acc % RING * C::SLOT_COLS;
#pragma unroll 1
        for (int j = 0; j < n8; j += 8) {
          float v[8];
          if (un.kind == 0) {
            uint32_t r[8];
            tmem_ld_32x8(d + j, r);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
          } else {  // hi and lo parts of the rows in turn
            uint32_t r[16];
            tmem_ld_32x16(d + 2 * j, r);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[2 * i]) + __uint_as_float(r[2 * i + 1]);
          }
          emit(v, j);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(acc_empty(set, acc % RING));
        ++acc;
      } else {
        // The scales of a stage's two blocks of weights (GEMM1: gate and up, whose columns may lie in
        // two blocks of scales; GEMM2: the next two k, a last one past the end with none and weights of
        // zero): lane l holds those of stage kb0 + l, fetched 32 stages at a time, as HBM under load
        // answers later than a few stages.
        const bool up = un.kind == 0;
        const int stride = up ? (2 * I + 127) / 128 : work.nt2, nt = (I + 127) / 128;
        const int up_col = I + un.tile * kCols + q * 32;  // the warp's first up column
        const int block0 = min(up_col / 128, stride - 1), block1 = min((up_col + 31) / 128, stride - 1);
        const bool second = up && (up_col + lane) / 128 != up_col / 128;
        const float* const ws_at =
            (up ? (un.shared ? a.s_up_scale : a.up_scale)
                : (un.shared ? a.s_down_scale : a.down_scale)) +
            (int64_t)un.e * (up ? (a.H + 127) / 128 : nt) * stride;
        auto fetch = [&](int kb) {
          float3 w = make_float3(0.f, 0.f, 0.f);
          if (kb >= un.kb1) return w;
          const float* const at = ws_at + (int64_t)(up ? kb : 2 * kb) * stride;
          w.x = __ldg(at + un.tile);
          if (up)
            w.y = __ldg(at + block0), w.z = __ldg(at + block1);
          else if (2 * kb + 1 < nt)
            w.y = __ldg(at + stride + un.tile);
          return w;
        };
        // and those of the rows of h: lane l holds row l % 16 of block l / 16
        const float* const hs_at =
            (un.shared ? a.s_h_scale + (int64_t)(un.ready - work.nc) * nt * C::CHUNK
                       : a.h_scale + (int64_t)un.ready * nt * C::CHUNK) + lane % C::CHUNK;
        auto row_scale = [&](int kb) {
          return __ldcg(hs_at + min(2 * kb + lane / C::CHUNK, nt - 1) * C::CHUNK);
        };
        // G groups of 8 rows
        auto unit = [&](auto groups) {
          constexpr int G = decltype(groups)::value;
          float v[2][8 * G];
#pragma unroll
          for (int i = 0; i < 8 * G; ++i) v[0][i] = v[1][i] = 0.f;
          float3 held = fetch(un.kb0 + lane), later = fetch(un.kb0 + lane + 32);
          float hs = 1.f;
          int at = 0;  // the lane that holds the stage's
#pragma unroll 1
          for (int kb = un.kb0; kb < un.kb1; ++kb, ++acc, ++at) {
            if (at == 32) {
              at = 0;
              held = later;
              later = fetch(kb + lane + 32);
            }
            float ws[2] = {__shfl_sync(0xFFFFFFFFu, held.x, at), __shfl_sync(0xFFFFFFFFu, held.y, at)};
            const float w2 = __shfl_sync(0xFFFFFFFFu, held.z, at);
            if (second) ws[1] = w2;
            float next_hs = 1.f;
            // (GEMM2: a slot per block, whose products are committed together)
            const int last = up ? acc : acc + 1;
            if (!wait(acc_full(set, last % RING), (last / RING) & 1)) return;
            tc_fence_after();
            if (!up) {  // (the products of h are there, so its scales are)
              if (kb == un.kb0) hs = row_scale(kb);
              if (kb + 1 < un.kb1) next_hs = row_scale(kb + 1);
            }
            if (up) {  // both parts of the rows in turn, both blocks in one slot
#pragma unroll
              for (int half = 0; half < 2; ++half) {
                uint32_t r[16 * G];
#pragma unroll
                for (int j = 0; j < 2 * G; ++j)
                  tmem_ld_32x8(tmem_q + acc % RING * C::SLOT_COLS + half * (C::SLOT_COLS / 2) + 8 * j,
                               *reinterpret_cast<uint32_t(*)[8]>(r + 8 * j));
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 8 * G; ++i)
                  v[half][i] = fmaf(ws[half], whole(r[2 * i], r[2 * i + 1]), v[half][i]);
              }
            } else {  // three parts, a slot per block
#pragma unroll
              for (int half = 0; half < 2; ++half) {
                uint32_t r[24 * G];
#pragma unroll
                for (int j = 0; j < 3 * G; ++j)
                  tmem_ld_32x8(tmem_q + (acc + half) % RING * C::SLOT_COLS + 8 * j,
                               *reinterpret_cast<uint32_t(*)[8]>(r + 8 * j));
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 8 * G; ++i) {
                  const float rest = whole(r[3 * i + 1], r[3 * i + 2]);
                  const float rs = __shfl_sync(0xFFFFFFFFu, hs, half * C::CHUNK + i);
                  v[half][i] = fmaf(ws[half] * rs, whole(r[3 * i], __float_as_uint(rest)), v[half][i]);
                }
              }
            }
            hs = next_hs;
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(acc_empty(set, acc % RING));
              if (!up) mbar_arrive(acc_empty(set, last % RING));
            }
            acc = last;
          }
          if (!up) {
#pragma unroll
            for (int i = 0; i < 8 * G; ++i) v[0][i] += v[1][i];
#pragma unroll
            for (int j = 0; j < G; ++j) emit(v[0] + 8 * j, 8 * j);
            return;
          }
          if (!wait(x_empty(set), (up_units & 1) ^ 1)) return;
#pragma unroll
          for (int i = 0; i < 8 * G; ++i) {
            if (i >= un.n) continue;
            const float xs = __shfl_sync(0xFFFFFFFFu, x_scale, i), g = v[0][i] * xs, u = v[1][i] * xs;
            const float w = un.shared ? 1.f : tb.w[un.row0 + i];
            ex[i * kCols] = un.tile * kCols + col < I ? w * (g * sigmoidf_(g) * u) : 0.f;
          }
        };
        if (n8 == 8) unit(std::integral_constant<int, 1>());
        else unit(std::integral_constant<int, 2>());
        if (!ok) break;
      }
      if (un.kind == 1) {
        __syncwarp();
        if (lane == 0) mbar_arrive(stored(qi % kQueue));
        continue;
      }
      // GEMM1: the set's warps meet in shared memory and take the rows in turn
      __syncwarp();
      if (lane == 0) mbar_arrive(x_full(set));
      if (!wait(x_full(set), up_units & 1)) break;
      ++up_units;
#pragma unroll 1
      for (int i = q; i < un.n; i += 4) {
        const int row = un.row0 + i;
        const float* x = exchange + (set * C::CHUNK + i) * kCols;
        if constexpr (FP8) {  // 128 columns of h, 4 per lane
          const int c = un.tile * kCols + 4 * lane;
          const float4 h = *reinterpret_cast<const float4*>(x + 4 * lane);
          float m = fmaxf(fmaxf(fabsf(h.x), fabsf(h.y)), fmaxf(fabsf(h.z), fabsf(h.w)));
          if (h.x != h.x || h.y != h.y || h.z != h.z || h.w != h.w) m = INFINITY;
          float inv;
          const float s = split_scale(warp_max(m), &inv);
          uint8_t part[C::H_PARTS][4];
          const float hs[4] = {h.x * s, h.y * s, h.z * s, h.w * s};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float rest = hs[j];
#pragma unroll
            for (int k = 0; k < C::H_PARTS; ++k) part[k][j] = take_e4m3(rest);
          }
          uint8_t* dst = static_cast<uint8_t*>(un.shared ? a.s_h : a.h) + (int64_t)row * C::H_PARTS * I + c;
          if (c < I) {
#pragma unroll
            for (int k = 0; k < C::H_PARTS; ++k)
              *reinterpret_cast<uint32_t*>(dst + (int64_t)k * I) = word_of(part[k]);
          }
          const int nt = (I + 127) / 128;
          if (lane == 0)
            (un.shared ? a.s_h_scale + (int64_t)(un.ready - work.nc) * nt * C::CHUNK
                       : a.h_scale + (int64_t)un.ready * nt * C::CHUNK)[un.tile * C::CHUNK + i] = inv;
        } else {  // columns 0..63 are gate, 64..127 up of the same 64: two per lane
          const int c = un.tile * 64 + 2 * lane;
          const float w = un.shared ? 1.f : tb.w[row];
          const float2 g = *reinterpret_cast<const float2*>(x + 2 * lane);
          const float2 l = *reinterpret_cast<const float2*>(x + 64 + 2 * lane);
          if (c < I) {
            uint32_t* const dst = reinterpret_cast<uint32_t*>(
                static_cast<__nv_bfloat16*>(un.shared ? a.s_h : a.h) + (int64_t)row * 2 * I + c);
            const float h0 = w * (g.x * sigmoidf_(g.x) * l.x), h1 = w * (g.y * sigmoidf_(g.y) * l.y);
            const uint32_t hi = pack_bf16(h0, h1);
            dst[0] = hi;
            dst[I / 2] = pack_bf16(rest_of(h0, bf16_lo(hi)), rest_of(h1, bf16_hi(hi)));
          }
        }
      }
      fence_proxy_async_global();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(x_empty(set));
        mbar_arrive(stored(qi % kQueue));
      }
    }
    // ------------------------------------------------ sums of the partial rows
    // (after an error NaN, so that what was not computed does not pass for a result)
    ok = __all_sync(0xFFFFFFFFu, ok);
    const int target = work.nc * work.split + work.ncs * work.splits;
    for (int task = (warp - kFirstEpilogue) * (int)gridDim.x + (int)blockIdx.x;
         task < a.T * work.nt2; task += 8 * (int)gridDim.x) {
      const int t = div_small(task, work.nt2), tile = task - t * work.nt2, c = tile * kCols + lane * 4;
      if (ok) {
        const bool there = wait_counter(a.ready2 + tile, target, kTimeoutNs);  // every lane, as above
        ok = __all_sync(0xFFFFFFFFu, there);
        if (!ok && lane == 0) give_up();
      }
      if (c >= a.H) continue;
      if (!ok) {
        *reinterpret_cast<uint2*>(a.y + (int64_t)t * a.H + c) = make_uint2(0x7FC07FC0u, 0x7FC07FC0u);
        continue;
      }
      float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
      // part by part, a part's rows in slot order with 8 loads in flight; then the shared expert
#pragma unroll 1
      for (int p = 0; p < work.split; ++p) {
        const float* o = a.o + (int64_t)p * a.S * a.H + c;
#pragma unroll 1
        for (int k0 = 0; k0 < a.K; k0 += 8) {
          float4 r[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            r[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (k0 + i < a.K)
              r[i] = __ldcg(reinterpret_cast<const float4*>(
                  o + (int64_t)tb.row[t * a.K + k0 + i] * a.H));
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) s.x += r[i].x, s.y += r[i].y, s.z += r[i].z, s.w += r[i].w;
        }
      }
#pragma unroll 1
      for (int p = 0; p < (work.ncs > 0 ? work.splits : 0); ++p) {
        const float4 r = __ldcg(reinterpret_cast<const float4*>(a.s_o + ((int64_t)p * a.T + t) * a.H + c));
        s.x += r.x, s.y += r.y, s.z += r.z, s.w += r.w;
      }
      *reinterpret_cast<uint2*>(a.y + (int64_t)t * a.H + c) =
          make_uint2(pack_bf16(s.x, s.y), pack_bf16(s.z, s.w));
    }
  }
  tc_fence_before();
  __syncwarp();
  __syncthreads();
  if (warp == 3) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------------------------- quantiser

// One 128 x 128 block per CTA: its largest magnitude, then the quotients. 8 columns per thread.
__global__ void __launch_bounds__(256) k_quantize(int64_t R, int64_t C, const __nv_bfloat16* w,
                                                  uint8_t* q, float* scale) {
  __shared__ float red[8];
  pdl_wait();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t bc = blockIdx.x, br = blockIdx.y, n = blockIdx.z;
  const int64_t c = bc * 128 + (tid & 15) * 8;
  w += n * R * C;
  q += n * R * C;
  float m = 0.f;
  bool bad = false;  // infinity or NaN
  for (int i = tid >> 4; i < 128; i += 16) {
    const int64_t r = br * 128 + i;
    if (r >= R || c >= C) continue;
    float v[8];
    load_vec<8>(w + r * C + c, v);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      bad |= !(fabsf(v[k]) <= 3.4e38f);
      m = fmaxf(m, fabsf(v[k]));
    }
  }
  m = warp_max(m);
  if (lane == 0) red[warp] = m;
  bad = __syncthreads_or(bad);
  m = red[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) m = fmaxf(m, red[i]);
  float s = m == 0.f ? 1.f : m / 448.f;
  if (bad) s = __int_as_float(0x7FC00000);
  if (tid == 0) scale[(n * gridDim.y + br) * gridDim.x + bc] = s;
  for (int i = tid >> 4; i < 128; i += 16) {
    const int64_t r = br * 128 + i;
    if (r >= R || c >= C) continue;
    float v[8];
    load_vec<8>(w + r * C + c, v);
    uint32_t o[2] = {0u, 0u};
#pragma unroll
    for (int k = 0; k < 8; ++k)
      o[k >> 2] |= (uint32_t)__nv_cvt_float_to_fp8(v[k] / s, __NV_SATFINITE, __NV_E4M3) << (8 * (k & 3));
    *reinterpret_cast<uint2*>(q + r * C + c) = make_uint2(o[0], o[1]);
  }
}

// ---------------------------------------------------------------------------------- host side

inline bool aligned_to(const void* p, size_t a) {
  return (reinterpret_cast<uintptr_t>(p) % a) == 0;
}

struct Layout {
  size_t off_ready2, off_logits, off_ids, off_weights, off_x8, off_xs, off_h, off_sh, off_hs, off_shs, off_o, off_so, total;
  int zero_words;
};

mm_status check_desc(const mm_decode_desc* d) {
  if (d == nullptr) return MM_ERR_INVALID_ARG;
  const mm_dims& m = d->dims;
  if (m.T < 0 || m.H < 1 || m.I < 1 || m.E < 1 || m.K < 1 || d->shared_I < 0)
    return MM_ERR_INVALID_ARG;
  if (d->weight_type != MM_BF16 && d->weight_type != MM_E4M3) return MM_ERR_INVALID_ARG;
  if (d->router_type != MM_BF16 && d->router_type != MM_FP32) return MM_ERR_INVALID_ARG;
  if (d->score != MM_SCORE_SOFTMAX && d->score != MM_SCORE_SIGMOID) return MM_ERR_INVALID_ARG;
  const int unit = d->weight_type == MM_E4M3 ? 16 : 8;
  if (m.H % unit || m.I % unit || d->shared_I % unit) return MM_ERR_UNSUPPORTED;
  if (m.T > kMaxT || m.K > 16 || m.T * m.K > kMaxSlots || m.E > kMaxE || m.H > 65536 ||
      m.I > 65536 || d->shared_I > 65536)
    return MM_ERR_UNSUPPORTED;
  return MM_OK;
}

Layout layout(const mm_decode_desc& d) {
  const mm_dims& m = d.dims;
  const size_t S = (size_t)(m.T * m.K);
  Layout l{};
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off = (off + bytes + 255) / 256 * 256;
    return o;
  };
  take((W_READY1 + S + kMaxT / Cfg<true>::CHUNK) * 4);  // header, GEMM1 counters: a chunk has a row
  l.off_ready2 = take((size_t)((m.H + kCols - 1) / kCols) * 4);
  l.zero_words = (int)(off / 4);
  l.off_logits = take((size_t)(m.T * m.E) * 4);
  l.off_ids = take(S * 4);
  l.off_weights = take(S * 4);
  const bool fp8 = d.weight_type == MM_E4M3;
  l.off_x8 = take(fp8 ? (size_t)m.T * m.H * 2 : 0);
  l.off_xs = take(fp8 ? (size_t)m.T * 4 : 0);
  constexpr int chunk = Cfg<true>::CHUNK;
  l.off_hs = take(fp8 ? S * ((m.I + 127) / 128) * chunk * 4 : 0);
  l.off_shs = take(fp8 ? (size_t)(kMaxT / chunk) * ((d.shared_I + 127) / 128) * chunk * 4 : 0);
  const size_t h_bytes = fp8 ? Cfg<true>::H_PARTS : 2 * Cfg<false>::H_PARTS;
  l.off_h = take(S * m.I * h_bytes);
  l.off_sh = take((size_t)m.T * d.shared_I * h_bytes);
  l.off_o = take((size_t)kMaxSplit * S * m.H * 4);
  l.off_so = take(d.shared_I > 0 ? (size_t)kMaxSplit * m.T * m.H * 4 : 0);
  l.total = off;
  return l;
}

bool weight_map(CUtensorMap* m, const void* base, int64_t cols, int64_t rows, int64_t n,
                bool fp8) {
  const uint64_t es = fp8 ? 1 : 2;
  const uint64_t dims[3] = {(uint64_t)cols, (uint64_t)rows, (uint64_t)n};
  const uint64_t strides[2] = {(uint64_t)cols * es, (uint64_t)cols * rows * es};
  const uint32_t box[3] = {fp8 ? 128u : 64u, fp8 ? 128u : 64u, 1};
  return make_map(m, base, 3, dims, strides, box,
                  fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16);
}

// Rows of 128-byte boxes: bf16 or e4m3 [rows, cols].
bool row_map(CUtensorMap* m, const void* base, int64_t cols, int64_t rows, bool fp8,
             uint32_t box_rows) {
  const uint64_t es = fp8 ? 1 : 2;
  const uint64_t dims[2] = {(uint64_t)cols, (uint64_t)rows};
  const uint64_t strides[1] = {(uint64_t)cols * es};
  const uint32_t box[2] = {(uint32_t)(128 / es), box_rows};
  return make_map(m, base, 2, dims, strides, box,
                  fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16);
}

template <bool FP8>
constexpr size_t dynamic_smem() {
  return 1024 + Cfg<FP8>::STAGES * (Cfg<FP8>::A_BYTES + Cfg<FP8>::B_BYTES) + 2 * Cfg<FP8>::CHUNK * kCols * 4;
}

template <bool FP8>
cudaError_t launch_experts(const DecodeArgs& a, int sms, cudaStream_t st) {
  static std::atomic<uint64_t> done_mask{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(done_mask.load(std::memory_order_relaxed) & bit)) {
    e = cudaFuncSetAttribute(k_experts<FP8>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)dynamic_smem<FP8>());
    if (e != cudaSuccess) return e;
    done_mask.fetch_or(bit, std::memory_order_relaxed);
  }
  return launch_pdl(k_experts<FP8>, dim3((unsigned)sms), dim3(kThreads), dynamic_smem<FP8>(), st, a);
}

}  // namespace
}  // namespace mm

using namespace mm;

extern "C" {

size_t mm_decode_workspace_size(const mm_decode_desc* d) {
  if (check_desc(d) != MM_OK) return 0;
  return layout(*d).total;
}

mm_status mm_decode(const mm_decode_desc* d, const mm_decode_weights* w, const void* x,
                    int32_t* topk_ids, float* topk_weights, void* y, void* workspace,
                    size_t workspace_bytes, void* stream) {
  mm_status s = check_desc(d);
  if (s != MM_OK) return s;
  const mm_dims& m = d->dims;
  const bool fp8 = d->weight_type == MM_E4M3, shared = d->shared_I > 0;
  if (w == nullptr || !w->up || !w->down || !aligned_to(w->up, 16) || !aligned_to(w->down, 16))
    return MM_ERR_INVALID_ARG;
  if (shared != (w->shared_up != nullptr) || shared != (w->shared_down != nullptr) ||
      !aligned_to(w->shared_up, 16) || !aligned_to(w->shared_down, 16))
    return MM_ERR_INVALID_ARG;
  if (fp8 != (w->up_scale != nullptr) || fp8 != (w->down_scale != nullptr) ||
      (fp8 && shared) != (w->shared_up_scale != nullptr) ||
      (fp8 && shared) != (w->shared_down_scale != nullptr))
    return MM_ERR_INVALID_ARG;
  if (!aligned_to(w->up_scale, 4) || !aligned_to(w->down_scale, 4) ||
      !aligned_to(w->shared_up_scale, 4) || !aligned_to(w->shared_down_scale, 4))
    return MM_ERR_INVALID_ARG;
  if (!aligned_to(w->router, 16) || !aligned_to(w->router_bias, 4) ||
      (w->router == nullptr && w->router_bias != nullptr) || (w->router && m.K > m.E))
    return MM_ERR_INVALID_ARG;
  if (!aligned_to(topk_ids, 4) || !aligned_to(topk_weights, 4)) return MM_ERR_INVALID_ARG;
  const Layout l = layout(*d);
  if (workspace == nullptr || !aligned_to(workspace, 256) || workspace_bytes < l.total)
    return MM_ERR_WORKSPACE;
  if (m.T > 0 && (!x || !y || !aligned_to(x, 16) || !aligned_to(y, 16))) return MM_ERR_INVALID_ARG;
  if (m.T > 0 && w->router == nullptr && (!topk_ids || !topk_weights)) return MM_ERR_INVALID_ARG;
  clear_error();
  MM_TRY(bind_context());
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  char* ws = static_cast<char*>(workspace);
  if (m.T == 0) {
    MM_TRY(cudaMemsetAsync(ws, 0, (size_t)l.zero_words * 4, st));
    return MM_OK;
  }
  LogitArgs la{};
  la.x = static_cast<const __nv_bfloat16*>(x);
  la.router = w->router;
  la.logits = reinterpret_cast<float*>(ws + l.off_logits);
  la.zero = reinterpret_cast<int*>(ws);
  la.zero_n = l.zero_words;
  la.T = (int)m.T;
  la.H = (int)m.H;
  la.E = (int)m.E;
  DecodeArgs a{};
  char* const x_rows = fp8 ? ws + l.off_x8 : static_cast<char*>(const_cast<void*>(x));
  const int64_t parts = fp8 ? Cfg<true>::X_PARTS : Cfg<false>::X_PARTS;
  const int64_t h_parts = fp8 ? Cfg<true>::H_PARTS : Cfg<false>::H_PARTS;
  bool maps = weight_map(&a.up, w->up, 2 * m.I, m.H, m.E, fp8) &&
              weight_map(&a.down, w->down, m.H, m.I, m.E, fp8) &&
              row_map(&a.x, x_rows, m.H, parts * m.T, fp8, 1) &&
              row_map(&a.h_rows, ws + l.off_h, m.I, h_parts * m.T * m.K, fp8, 8 * h_parts);
  if (shared)
    maps = maps && weight_map(&a.s_up, w->shared_up, 2 * d->shared_I, m.H, 1, fp8) &&
           weight_map(&a.s_down, w->shared_down, m.H, d->shared_I, 1, fp8) &&
           row_map(&a.s_h_rows, ws + l.off_sh, d->shared_I, h_parts * m.T, fp8, 8 * h_parts);
  if (!maps) return cuda_fail(cudaErrorInvalidValue, "decode tensor maps");
  a.up_scale = w->up_scale;
  a.down_scale = w->down_scale;
  a.s_up_scale = w->shared_up_scale;
  a.s_down_scale = w->shared_down_scale;
  a.logits = la.logits;
  a.bias = w->router_bias;
  a.ids = topk_ids;
  a.weights = topk_weights;
  a.y = static_cast<__nv_bfloat16*>(y);
  a.hdr = la.zero;
  a.ready1 = la.zero + W_READY1;
  a.ready2 = reinterpret_cast<int*>(ws + l.off_ready2);
  a.h = ws + l.off_h;
  a.s_h = ws + l.off_sh;
  a.x_scale = reinterpret_cast<float*>(ws + l.off_xs);
  a.h_scale = reinterpret_cast<float*>(ws + l.off_hs);
  a.s_h_scale = reinterpret_cast<float*>(ws + l.off_shs);
  a.o = reinterpret_cast<float*>(ws + l.off_o);
  a.s_o = reinterpret_cast<float*>(ws + l.off_so);
  a.T = la.T;
  a.H = la.H;
  a.I = (int)m.I;
  a.E = la.E;
  a.K = (int)m.K;
  a.S = a.T * a.K;
  a.Is = (int)d->shared_I;
  a.score = d->score;
  a.normalize = d->normalize;
  a.scale = d->scale;
  a.route = w->router != nullptr;
  // k_logits' N. One output per block as long as that makes few blocks per SM, whatever H; from there on
  // the 16 outputs of a block save more reads than they leave SMs idle. A call with 1 and with 4, bf16, H =
  // 512 / 2048 / 7168, us: 512 outputs (8 tokens of 64 experts) 13.1, 19.3, 38.3 and 13.2, 19.5, 39.3;
  // 768 (6 of 128) 13.8, 19.5, 38.8 and 13.9, 19.3, 39.2; 1024 (8 of 128) 14.6, 20.0, 39.6 and 14.4,
  // 19.5, 39.8; 2048 (8 of 256) 15.9, 21.8, 43.0 and 14.8, 20.5, 41.4. One token has no four to read a
  // router row for: of 1024 experts 19.5, 25.8, 43.8 and 20.1, 26.0, 44.9.
  const int sms = std::max(1, device_sm_count());
  const int tile = m.T == 1 || m.T * m.E <= 6 * sms ? 1 : 4;
  la.logit_blocks = a.route ? (int)((m.E + tile - 1) / tile * ((m.T + tile - 1) / tile)) : 0;
  if (fp8) {
    la.x8 = reinterpret_cast<uint8_t*>(ws + l.off_x8);
    la.x_scale = reinterpret_cast<float*>(ws + l.off_xs);
  }
  const dim3 grid((unsigned)std::max(1, la.logit_blocks + (fp8 ? a.T : 0)));
  auto* const logits = d->router_type == MM_BF16
                           ? (tile == 1 ? k_logits<__nv_bfloat16, 1> : k_logits<__nv_bfloat16, 4>)
                           : (tile == 1 ? k_logits<float, 1> : k_logits<float, 4>);
  MM_TRY(launch_pdl(logits, grid, dim3(256), 0, st, la));
  if (a.route && m.T > kMaxRouted) {
    int32_t* ids = topk_ids ? topk_ids : reinterpret_cast<int32_t*>(ws + l.off_ids);
    float* weights = topk_weights ? topk_weights : reinterpret_cast<float*>(ws + l.off_weights);
    const mm_router_desc rd{m.T, (int32_t)m.E, (int32_t)m.K, MM_FP32, d->score, d->normalize,
                            d->scale};
    MM_TRY(launch_router(rd, la.logits, w->router_bias, ids, weights, st));
    a.route = 0;
    a.ids = ids;
    a.weights = weights;
  }
  if (fp8)
    MM_TRY(launch_experts<true>(a, sms, st));
  else
    MM_TRY(launch_experts<false>(a, sms, st));
  return MM_OK;
}

mm_status mm_quantize_blocks(int64_t n, int64_t R, int64_t C, const void* w, void* q, float* scale,
                             void* stream) {
  if (n < 0 || R < 1 || C < 1) return MM_ERR_INVALID_ARG;
  if (C % 8 || n > 65535 || R > 65535 * (int64_t)128 || C > ((int64_t)1 << 31)) return MM_ERR_UNSUPPORTED;
  if (n == 0) return MM_OK;
  if (!w || !q || !scale || !aligned_to(w, 16) || !aligned_to(q, 8) || !aligned_to(scale, 4))
    return MM_ERR_INVALID_ARG;
  clear_error();
  MM_TRY(launch_pdl(k_quantize, dim3((unsigned)((C + 127) / 128), (unsigned)((R + 127) / 128),
                                     (unsigned)n),
                    dim3(256), 0, reinterpret_cast<cudaStream_t>(stream), R, C,
                    static_cast<const __nv_bfloat16*>(w), static_cast<uint8_t*>(q), scale));
  return MM_OK;
}

}  // extern "C"
