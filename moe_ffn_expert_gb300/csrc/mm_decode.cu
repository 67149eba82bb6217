// The whole MoE layer for a few tokens (mm_decode) and the quantiser of its 8-bit weights.
//
// With few tokens every selected expert's weights are read for a handful of rows: the layer is
// bound by HBM, 3 H I weights per expert against 6 H I multiply-adds per slot. Two launches:
//
//   k_logits  the router product (fp32 sums of bf16 x bf16 or bf16 x fp32 products) over all SMs,
//             and zeroed counters for the second kernel;
//   k_experts one CTA per SM. Every CTA derives the same routing tables from the logits (or the
//             caller's ids) in shared memory, then takes work units from one global counter:
//     GEMM1   (chunk of up to 32 rows of one expert, 64 gate + 64 up columns): w * silu(g) * u
//     GEMM2   (chunk, 128 output columns, part of I): fp32 partial rows
//     combine (8 tokens, 128 columns): the sum of a token's partial rows, in slot order
//
// A GEMM2 unit needs its chunk's GEMM1 units, a combine unit its columns' GEMM2 units: counters
// in the workspace, waited for at the last moment and only for the small operand, so the weight
// loads of the next units run ahead through the wait. Units are claimed in that order, and a CTA
// works through its units in the order it claimed them, so what a unit waits for is always held
// by a CTA that is running or done: no wait depends on how many CTAs are resident.
//
// The products run as mma.sync m16n8k16 with the weights as the 16-row operand (its transpose
// comes with ldmatrix.trans from the row-major tiles that TMA brings) and up to 8 tokens per
// instruction: one to 32 rows of an expert cost no padding to 128 rows and no accumulator in
// tensor memory, and the tensor cores are idle for most of the time either way.
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
constexpr int kChunk = 32;        // rows of one expert per unit
constexpr int kCols = 128;        // weight columns per unit
constexpr int kTokens = 8;        // tokens per combine unit
constexpr int kMaxSplit = 4;      // parts of I per GEMM2 column tile
constexpr int kConsumers = 8;     // warps; 4 column groups x 2 halves of a stage's k
constexpr int kThreads = 32 * (kConsumers + 2);
constexpr int kTileBytes = 16384; // one stage of weights: 64 x 128 bf16 or 128 x 128 e4m3
constexpr int kQueue = 4;
constexpr uint64_t kTimeoutNs = 2000000000ull;

template <bool FP8>
struct Cfg {
  static constexpr int KB = FP8 ? 128 : 64;           // k per stage
  static constexpr int PITCH = KB * 2 + 16;           // bytes per row of the token operand
  static constexpr int B_BYTES = kChunk * PITCH;
  static constexpr int STAGES = FP8 ? 7 : 8;
};

// int32 words at the start of the workspace (zeroed by k_logits)
enum { W_STATUS = 0, W_NEXT = 1, W_READY1 = 64 };

struct DecodeArgs {
  CUtensorMap up, down, s_up, s_down;
  const __nv_bfloat16* x;
  const float *up_scale, *down_scale, *s_up_scale, *s_down_scale;
  const float* logits;    // with a router
  const float* bias;
  int32_t* ids;           // router: output or null; else input
  float* weights;
  __nv_bfloat16* y;
  int* hdr;
  int *ready1, *ready2;
  __nv_bfloat16 *h, *s_h;  // [S, I], [T, Is]
  float *o, *s_o;          // [split][S, H], [split][T, H]
  int T, H, I, E, K, S, Is, score, normalize, route;
  float scale;
};

// Everything of a CTA that is derived from the routing.
struct Tables {
  int16_t tok[kMaxSlots];      // token of a sorted row
  int16_t row[kMaxSlots];      // sorted row of a slot
  float w[kMaxSlots];          // weight of a sorted row
  float slot_w[kMaxSlots];     // weight of a slot
  int16_t id[kMaxSlots];       // expert of a slot
  uint16_t chunk_row[kMaxSlots];
  uint16_t chunk_e[kMaxSlots];
  uint32_t count[kMaxE];       // slots | chunks << 16, then the exclusive sums
  uint16_t next[kMaxE];        // rows placed so far
  uint8_t chunk_n[kMaxSlots];
  int chunks, bad;
};

struct Unit {
  int kind;  // 0 GEMM1, 1 GEMM2, 2 combine
  int shared, row0, n, e, tile, kb0, kb1, split, ready;
};

// Work units in claiming order.
struct Work {
  int nc, ncs, nt1, nt1s, nt2, split, splits, kb_h, kb_i, kb_is, t1, t1s, t2, t2s, total;
};

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

__device__ __forceinline__ void ldsm4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// d += a b for a 16 x 16 tile of weights (transposed) and 8 tokens.
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Two e4m3 numbers (low and high byte) as bf16: exact (3 mantissa bits, exponents -9..8), NaN stays.
__device__ __forceinline__ uint32_t e4m3x2_to_bf16x2(uint32_t two) {
  const __half2_raw h =
      __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(two & 0xFFFFu), __NV_E4M3);
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
  return pack_bf16(f.x, f.y);
}

// ---------------------------------------------------------------------------------- k_logits

struct LogitArgs {
  const __nv_bfloat16* x;
  const void* router;
  float* logits;
  int* zero;  // words to clear
  int zero_n;
  int T, H, E;
};

// 4 experts x 4 tokens per block, H dealt to the 8 warps; the 16 sums of a warp's lanes are
// reduced by halving exchanges, the warps' sums in order.
template <typename RT>
__global__ void __launch_bounds__(256) k_logits(LogitArgs a) {
  __shared__ float part[8][16];
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int blocks = gridDim.x * gridDim.y, block = blockIdx.y * gridDim.x + blockIdx.x;
  for (int i = block * 256 + tid; i < a.zero_n; i += blocks * 256) a.zero[i] = 0;
  if (a.router == nullptr) return;
  const int e0 = blockIdx.x * 4, t0 = blockIdx.y * 4;
  float acc[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) acc[i] = 0.f;
  for (int c = tid * 8; c < a.H; c += 256 * 8) {
    float w[4][8], x[4][8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      load_vec<8>(static_cast<const RT*>(a.router) + (int64_t)min(e0 + i, a.E - 1) * a.H + c, w[i]);
      load_vec<8>(a.x + (int64_t)min(t0 + i, a.T - 1) * a.H + c, x[i]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int k = 0; k < 8; ++k) acc[i * 4 + j] = fmaf(w[i][k], x[j][k], acc[i * 4 + j]);
  }
  const float s = warp_sum_many<16>(acc, lane);
  if ((lane & 1) == 0) part[warp][lane >> 1] = s;
  __syncthreads();
  if (tid < 16) {
    float v = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) v += part[i][tid];
    const int e = e0 + (tid >> 2), t = t0 + (tid & 3);
    if (e < a.E && t < a.T) a.logits[(int64_t)t * a.E + e] = v;
  }
}

// ---------------------------------------------------------------------------------- k_experts

template <int NV>
__device__ void select_row(const DecodeArgs& a, Tables& tb, int t, int lane) {
  const float* row = a.logits + (int64_t)t * a.E;
  uint32_t key[NV];
  float z[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int e = lane + 32 * j;
    z[j] = e < a.E ? __ldcg(row + e) : 0.f;
  }
  float m = -INFINITY, sum = 0.f;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int e = lane + 32 * j;
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
      if (lane + 32 * j < a.E) sum += expf(z[j] - m);
    sum = warp_sum(sum);
  }
  const int id = select_topk<NV>(key, a.K, lane);
  const float zs = lane < a.K ? __ldcg(row + id) : 0.f;
  const float w = selected_weight(zs, lane < a.K, a.score, a.normalize, a.scale, m, sum);
  if (lane < a.K) {
    tb.id[t * a.K + lane] = (int16_t)id;
    tb.slot_w[t * a.K + lane] = w;
    if (blockIdx.x == 0) {
      if (a.ids != nullptr) a.ids[t * a.K + lane] = id;
      if (a.weights != nullptr) a.weights[t * a.K + lane] = w;
    }
  }
}

// Routing tables of the CTA: the slots sorted by expert (stable), cut into chunks. The same in
// every CTA. False if a caller's id is out of range.
__device__ bool build_tables(const DecodeArgs& a, Tables& tb) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  for (int e = tid; e < a.E; e += kThreads) tb.count[e] = 0, tb.next[e] = 0;
  if (tid == 0) tb.bad = 0;
  __syncthreads();
  if (a.route) {
    for (int t = warp; t < a.T; t += kThreads / 32) {
      if (a.E <= 32) select_row<1>(a, tb, t, lane);
      else if (a.E <= 64) select_row<2>(a, tb, t, lane);
      else if (a.E <= 128) select_row<4>(a, tb, t, lane);
      else if (a.E <= 256) select_row<8>(a, tb, t, lane);
      else if (a.E <= 512) select_row<16>(a, tb, t, lane);
      else select_row<32>(a, tb, t, lane);
    }
  } else {
    for (int s = tid; s < a.S; s += kThreads) {
      const int e = a.ids[s];
      if (e < 0 || e >= a.E) tb.bad = 1;
      tb.id[s] = (int16_t)e;
      tb.slot_w[s] = a.weights[s];
    }
  }
  __syncthreads();
  if (tb.bad) {
    if (tid == 0) set_status(a.hdr + W_STATUS, MM_ERR_BAD_EXPERT_ID);
    return false;
  }
  for (int s = tid; s < a.S; s += kThreads) atomicAdd(&tb.count[tb.id[s]], 1u);
  __syncthreads();
  if (warp == 0) {
    // exclusive sums of slots (low half) and chunks (high half) over the experts; a lane takes
    // consecutive experts
    const int per = (a.E + 31) / 32, e0 = lane * per, e1 = min(a.E, e0 + per);
    uint32_t sum = 0;
    for (int e = e0; e < e1; ++e) {
      const uint32_t n = tb.count[e];
      tb.count[e] = sum;
      sum += n | ((n + kChunk - 1) / kChunk) << 16;
    }
    uint32_t before = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, before, o);
      if (lane >= o) before += v;
    }
    if (lane == 31) tb.chunks = (int)(before >> 16);
    before -= sum;
    for (int e = e0; e < e1; ++e) tb.count[e] += before;
    __syncwarp();
    // slots in order, 32 at a time: a slot's place among its expert's is what came before
    for (int s0 = 0; s0 < a.S; s0 += 32) {
      const int s = s0 + lane;
      const int e = s < a.S ? tb.id[s] : -1 - lane;
      const uint32_t same = __match_any_sync(0xFFFFFFFFu, e);
      if (s < a.S) {
        const int rank = tb.next[e] + __popc(same & ((1u << lane) - 1u));
        const int r = (int)(tb.count[e] & 0xFFFFu) + rank;
        tb.row[s] = (int16_t)r;
        tb.tok[r] = (int16_t)(s / a.K);
        tb.w[r] = tb.slot_w[s];
        if (rank % kChunk == 0) {  // first row of a chunk
          const int c = (int)(tb.count[e] >> 16) + rank / kChunk;
          tb.chunk_row[c] = (uint16_t)r;
          tb.chunk_e[c] = (uint16_t)e;
        }
      }
      __syncwarp();
      if (s < a.S && (same >> lane) == 1u) tb.next[e] += (uint16_t)__popc(same);
      __syncwarp();
    }
  }
  __syncthreads();
  for (int c = tid; c < tb.chunks; c += kThreads) {
    const int e = tb.chunk_e[c], first = (int)(tb.count[e] & 0xFFFFu);
    tb.chunk_n[c] = (uint8_t)min(kChunk, first + (int)tb.next[e] - (int)tb.chunk_row[c]);
  }
  __syncthreads();
  return true;
}

template <bool FP8>
__device__ __forceinline__ Work make_work(const DecodeArgs& a, int chunks) {
  constexpr int KB = Cfg<FP8>::KB;
  Work w;
  w.nc = chunks;
  w.ncs = a.Is > 0 ? (a.T + kChunk - 1) / kChunk : 0;
  w.nt1 = (a.I + 63) / 64;
  w.nt1s = (a.Is + 63) / 64;
  w.nt2 = (a.H + kCols - 1) / kCols;
  w.kb_h = (a.H + KB - 1) / KB;
  w.kb_i = (a.I + KB - 1) / KB;
  w.kb_is = (a.Is + KB - 1) / KB;
  // GEMM2 units too few for the SMs are cut along I
  const int units = (w.nc + w.ncs) * w.nt2;
  const int want = max(1, min(kMaxSplit, (int)gridDim.x / max(1, units)));
  w.split = min(want, w.kb_i);
  w.splits = min(want, max(1, w.kb_is));
  w.t1 = w.nc * w.nt1;
  w.t1s = w.t1 + w.ncs * w.nt1s;
  w.t2 = w.t1s + w.nc * w.nt2 * w.split;
  w.t2s = w.t2 + w.ncs * w.nt2 * w.splits;
  w.total = w.t2s + w.nt2 * ((a.T + kTokens - 1) / kTokens);
  return w;
}

__device__ __forceinline__ Unit unit_at(const DecodeArgs& a, const Tables& tb, const Work& w,
                                        int u) {
  Unit r;
  r.shared = 0;
  r.split = 0;
  int c;
  if (u < w.t1s) {
    r.kind = 0;
    r.shared = u >= w.t1;
    const int v = r.shared ? u - w.t1 : u, nt = r.shared ? w.nt1s : w.nt1;
    c = v / nt;
    r.tile = v - c * nt;
    r.kb0 = 0;
    r.kb1 = w.kb_h;
  } else if (u < w.t2s) {
    r.kind = 1;
    r.shared = u >= w.t2;
    const int v = u - (r.shared ? w.t2 : w.t1s), sp = r.shared ? w.splits : w.split;
    const int kb = r.shared ? w.kb_is : w.kb_i;
    c = v / (w.nt2 * sp);
    const int rest = v - c * w.nt2 * sp;
    r.tile = rest / sp;
    r.split = rest - r.tile * sp;
    r.kb0 = kb * r.split / sp;
    r.kb1 = kb * (r.split + 1) / sp;
  } else {
    r.kind = 2;
    const int v = u - w.t2s;
    c = v / w.nt2;
    r.tile = v - c * w.nt2;
    r.row0 = c * kTokens;
    r.n = min(kTokens, a.T - r.row0);
    r.e = 0;
    r.kb0 = r.kb1 = 0;
    r.ready = 0;
    return r;
  }
  if (r.shared) {
    r.row0 = c * kChunk;
    r.n = min(kChunk, a.T - r.row0);
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
  constexpr int KB = C::KB, STAGES = C::STAGES, PITCH = C::PITCH;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Tables tb;
  __shared__ uint64_t bars[3 * STAGES + 2 * kQueue + 8];
  __shared__ int queue[kQueue];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // weights of all stages (1024-byte aligned for the swizzle), token rows, the sums of the second
  // k half's warps
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* const aligned = smem_raw + (base - smem_u32(smem_raw));
  const uint32_t rows_at = base + STAGES * kTileBytes;
  float* const halves = reinterpret_cast<float*>(aligned + STAGES * (kTileBytes + C::B_BYTES));
  const uint32_t bar0 = smem_u32(bars);
  auto full_w = [&](int s) { return bar0 + 8u * s; };
  auto full_b = [&](int s) { return bar0 + 8u * (STAGES + s); };
  auto empty = [&](int s) { return bar0 + 8u * (2 * STAGES + s); };
  auto q_full = [&](int s) { return bar0 + 8u * (3 * STAGES + s); };
  auto q_empty = [&](int s) { return bar0 + 8u * (3 * STAGES + kQueue + s); };
  auto half_full = [&](int c) { return bar0 + 8u * (3 * STAGES + 2 * kQueue + c); };
  auto half_empty = [&](int c) { return bar0 + 8u * (3 * STAGES + 2 * kQueue + 4 + c); };
  if (tid == 0) {
    for (int c = 0; c < 4; ++c) {
      mbar_init(half_full(c), 1);
      mbar_init(half_empty(c), 1);
    }
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full_w(s), 1);
      mbar_init(full_b(s), 1);
      mbar_init(empty(s), kConsumers);
    }
    for (int s = 0; s < kQueue; ++s) {
      mbar_init(q_full(s), 1);
      mbar_init(q_empty(s), kConsumers + 1);
    }
    mbar_fence_init();
    tma_prefetch_desc(&a.up);
    tma_prefetch_desc(&a.down);
  }
  pdl_wait();
  if (!build_tables(a, tb)) return;  // (its barriers also publish the initialised mbarriers)
  const Work work = make_work<FP8>(a, tb.chunks);
  // a wait that runs out ends its role; the roles that depend on it run out in turn
  auto give_up = [&] { set_status(a.hdr + W_STATUS, MM_ERR_TIMEOUT); };

  if (warp == kConsumers) {
    // ------------------------------------------------ claims units and loads their weights
    if (lane == 0) {
      int u = blockIdx.x, it = 0;
      bool ok = true;
      for (int qi = 0; ok; ++qi) {
        const int qs = qi % kQueue;
        if (!mbar_wait(q_empty(qs), ((qi / kQueue) & 1) ^ 1, kTimeoutNs)) {
          give_up();
          break;
        }
        queue[qs] = u < work.total ? u : -1;
        mbar_arrive(q_full(qs));
        if (u >= work.total) break;
        const Unit un = unit_at(a, tb, work, u);
        u = gridDim.x + atomicAdd(a.hdr + W_NEXT, 1);
        const CUtensorMap* map = un.kind == 0 ? (un.shared ? &a.s_up : &a.up)
                                              : (un.shared ? &a.s_down : &a.down);
        const int I = un.shared ? a.Is : a.I;
        for (int kb = un.kb0; kb < un.kb1; ++kb, ++it) {
          const int s = it % STAGES;
          if (!mbar_wait(empty(s), ((it / STAGES) & 1) ^ 1, kTimeoutNs)) {
            give_up();
            ok = false;
            break;
          }
          const uint32_t dst = base + s * kTileBytes;
          mbar_arrive_expect_tx(full_w(s), kTileBytes);
          if (un.kind == 0) {
            tma_load_3d(dst, map, full_w(s), un.tile * 64, kb * KB, un.e);
            tma_load_3d(dst + kTileBytes / 2, map, full_w(s), I + un.tile * 64, kb * KB, un.e);
          } else if (FP8) {
            tma_load_3d(dst, map, full_w(s), un.tile * kCols, kb * KB, un.e);
          } else {
            tma_load_3d(dst, map, full_w(s), un.tile * kCols, kb * KB, un.e);
            tma_load_3d(dst + kTileBytes / 2, map, full_w(s), un.tile * kCols + 64, kb * KB, un.e);
          }
        }
      }
      // no CTA leaves with a copy into its shared memory in flight
      for (int j = max(0, it - STAGES); j < it; ++j)
        mbar_wait(full_w(j % STAGES), (j / STAGES) & 1, kTimeoutNs);
    }
  } else if (warp == kConsumers + 1) {
    // ------------------------------------------------ loads the token rows
    int it = 0;
    bool ok = true;
    for (int qi = 0; ok; ++qi) {
      const int qs = qi % kQueue;
      if (!mbar_wait(q_full(qs), (qi / kQueue) & 1, kTimeoutNs)) {
        if (lane == 0) give_up();
        break;
      }
      const int u = queue[qs];
      __syncwarp();
      if (lane == 0) mbar_arrive(q_empty(qs));
      if (u < 0) break;
      const Unit un = unit_at(a, tb, work, u);
      if (un.kind == 2) continue;
      const int I = un.shared ? a.Is : a.I, width = un.kind == 0 ? a.H : I;
      const __nv_bfloat16* src = a.x;
      if (un.kind == 0) {
        if (lane < un.n)
          src += (int64_t)(un.shared ? un.row0 + lane : tb.tok[un.row0 + lane]) * a.H;
      } else {
        // this chunk's rows: every consumer warp of the first k half counts once per unit
        const int target = 4 * (un.shared ? work.nt1s : work.nt1);
        int there = 1;
        if (lane == 0) there = wait_counter(a.ready1 + un.ready, target, kTimeoutNs);
        if (!__shfl_sync(0xFFFFFFFFu, there, 0)) {
          if (lane == 0) give_up();
          break;
        }
        fence_proxy_async_global();
        src = (un.shared ? a.s_h : a.h) + (int64_t)(un.row0 + lane) * I;
      }
      for (int kb = un.kb0; kb < un.kb1; ++kb, ++it) {
        const int s = it % STAGES;
        if (!mbar_wait(empty(s), ((it / STAGES) & 1) ^ 1, kTimeoutNs)) {
          if (lane == 0) give_up();
          ok = false;
          break;
        }
        const uint32_t bytes = (uint32_t)min(KB, width - kb * KB) * 2u;
        if (lane == 0) mbar_arrive_expect_tx(full_b(s), bytes * un.n);
        __syncwarp();
        if (lane < un.n)
          bulk_load(rows_at + s * C::B_BYTES + lane * PITCH, src + kb * KB, bytes, full_b(s));
      }
    }
    for (int j = max(0, it - STAGES); j < it; ++j)
      mbar_wait(full_b(j % STAGES), (j / STAGES) & 1, kTimeoutNs);
  } else {
    // ------------------------------------------------ products, sums and stores
    const int cg = warp & 3, kh = warp >> 2;
    const int bi = lane >> 3, br = lane & 7, g = lane >> 2, q = lane & 3;
    int it = 0, uses = 0;
    bool ok = true;
    for (int qi = 0; ok; ++qi) {
      const int qs = qi % kQueue;
      if (!mbar_wait(q_full(qs), (qi / kQueue) & 1, kTimeoutNs)) {
        if (lane == 0) give_up();
        break;
      }
      const int u = queue[qs];
      __syncwarp();
      if (lane == 0) mbar_arrive(q_empty(qs));
      if (u < 0) break;
      const Unit un = unit_at(a, tb, work, u);
      if (un.kind == 2) {
        const int target = 4 * (work.nc * work.split + work.ncs * work.splits);
        int there = 1;
        if (lane == 0) there = wait_counter(a.ready2 + un.tile, target, kTimeoutNs);
        if (!__shfl_sync(0xFFFFFFFFu, there, 0)) {
          if (lane == 0) give_up();
          break;
        }
        const int t = un.row0 + warp, c = un.tile * kCols + lane * 4;
        if (warp < un.n && c < a.H) {
          float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
          auto add = [&](const float* p) {
            const float4 v = __ldcg(reinterpret_cast<const float4*>(p));
            s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
          };
          for (int k = 0; k < a.K; ++k)
            for (int p = 0; p < work.split; ++p)
              add(a.o + ((int64_t)p * a.S + tb.row[t * a.K + k]) * a.H + c);
          if (work.ncs > 0)
            for (int p = 0; p < work.splits; ++p) add(a.s_o + ((int64_t)p * a.T + t) * a.H + c);
          *reinterpret_cast<uint2*>(a.y + (int64_t)t * a.H + c) =
              make_uint2(pack_bf16(s.x, s.y), pack_bf16(s.z, s.w));
        }
        continue;
      }
      const int nt = (un.n + 7) >> 3;
      const int I = un.shared ? a.Is : a.I, width = un.kind == 0 ? a.H : I;
      float acc[2][4][4];
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[m][j][i] = 0.f;
      // e4m3: the scales of this warp's two column groups, one k block per lane
      const float *sc0 = nullptr, *sc1 = nullptr;
      int sc_stride = 0;
      float scale0 = 0.f, scale1 = 0.f;
      if constexpr (FP8) {
        const float* sc = un.kind == 0 ? (un.shared ? a.s_up_scale : a.up_scale)
                                       : (un.shared ? a.s_down_scale : a.down_scale);
        const int cols = un.kind == 0 ? 2 * I : a.H, nb = (cols + 127) / 128;
        sc_stride = nb;
        sc += (int64_t)un.e * ((width + 127) / 128) * nb;
        const int c0 = un.kind == 0 ? un.tile * 64 + cg * 16 : un.tile * kCols + cg * 32;
        const int c1 = un.kind == 0 ? I + c0 : c0 + 16;
        sc0 = sc + min(c0 / 128, nb - 1);
        sc1 = sc + min(c1 / 128, nb - 1);
      }
      for (int kb = un.kb0; kb < un.kb1; ++kb, ++it) {
        const int s = it % STAGES, ph = (it / STAGES) & 1;
        if constexpr (FP8) {
          if (((kb - un.kb0) & 31) == 0 && kb + lane < un.kb1) {
            scale0 = sc0[(int64_t)(kb + lane) * sc_stride];
            scale1 = sc1[(int64_t)(kb + lane) * sc_stride];
          }
        }
        if (!mbar_wait(full_w(s), ph, kTimeoutNs) || !mbar_wait(full_b(s), ph, kTimeoutNs)) {
          if (lane == 0) give_up();
          ok = false;
          break;
        }
        const uint32_t wt = base + s * kTileBytes, bt = rows_at + s * C::B_BYTES;
        const int kvalid = min(KB, width - kb * KB);  // a multiple of 8
        if constexpr (!FP8) {
          const int k0 = kh * 32;
          if (k0 < kvalid) {
            uint32_t b[4][4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              if (j >= nt) continue;
              ldsm4(bt + (j * 8 + br) * PITCH + (k0 + bi * 8) * 2, b[j]);
              // past the rows' end shared memory holds anything; the weights there are zero
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (k0 + 8 * i >= kvalid) b[j][i] = 0;
            }
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
              const int kr = k0 + ks * 16 + (bi >> 1) * 8 + br;
#pragma unroll
              for (int m = 0; m < 2; ++m) {
                const int box = un.kind == 0 ? (bi & 1) : (cg >> 1);
                const int c16 = un.kind == 0 ? cg * 2 + m : (cg & 1) * 4 + m * 2 + (bi & 1);
                uint32_t r[4];
                ldsm4_trans(wt + box * (kTileBytes / 2) + kr * 128 + ((c16 ^ (kr & 7)) << 4), r);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                  if (j < nt) mma16816(acc[m][j], r[0], r[1], r[2], r[3], b[j][2 * ks], b[j][2 * ks + 1]);
              }
            }
          }
        } else {
          float part[2][4][4];
#pragma unroll
          for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
              for (int i = 0; i < 4; ++i) part[m][j][i] = 0.f;
#pragma unroll
          for (int k32 = 0; k32 < 2; ++k32) {
            const int k0 = kh * 64 + k32 * 32;
            if (k0 >= kvalid) continue;
            uint32_t b[4][4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              if (j >= nt) continue;
              ldsm4(bt + (j * 8 + br) * PITCH + (k0 + bi * 8) * 2, b[j]);
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (k0 + 8 * i >= kvalid) b[j][i] = 0;
            }
            const int kr = k0 + bi * 8 + br;
#pragma unroll
            for (int m = 0; m < 2; ++m) {
              uint32_t r[4];
              if (un.kind == 0)
                ldsm4_trans(wt + m * (kTileBytes / 2) + kr * 64 + ((cg ^ ((kr >> 1) & 3)) << 4), r);
              else
                ldsm4_trans(wt + kr * 128 + (((cg * 2 + m) ^ (kr & 7)) << 4), r);
              // r[i]: bytes (column 2g, 2g + 1) at k = 8 i + 2q, then at the next k
              uint32_t lo[4], hi[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const uint32_t v = __byte_perm(r[i], 0, 0x3120);
                lo[i] = e4m3x2_to_bf16x2(v);
                hi[i] = e4m3x2_to_bf16x2(v >> 16);
              }
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                if (j >= nt) continue;
                mma16816(part[m][j], lo[0], hi[0], lo[1], hi[1], b[j][0], b[j][1]);
                mma16816(part[m][j], lo[2], hi[2], lo[3], hi[3], b[j][2], b[j][3]);
              }
            }
          }
          const float f0 = __shfl_sync(0xFFFFFFFFu, scale0, (kb - un.kb0) & 31);
          const float f1 = __shfl_sync(0xFFFFFFFFu, scale1, (kb - un.kb0) & 31);
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              acc[0][j][i] = fmaf(f0, part[0][j][i], acc[0][j][i]);
              acc[1][j][i] = fmaf(f1, part[1][j][i], acc[1][j][i]);
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(empty(s));
      }
      if (!ok) break;
      // the two k halves of a column group meet: the second hands its sums over
      float* const mine = halves + cg * 32 * 32 + lane;
      if (kh == 1) {
        if (!mbar_wait(half_empty(cg), (uses & 1) ^ 1, kTimeoutNs)) {
          if (lane == 0) give_up();
          break;
        }
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (j < nt)
#pragma unroll
              for (int i = 0; i < 4; ++i) mine[((m * 4 + j) * 4 + i) * 32] = acc[m][j][i];
        __syncwarp();
        if (lane == 0) mbar_arrive(half_full(cg));
        ++uses;
        continue;
      }
      if (!mbar_wait(half_full(cg), uses & 1, kTimeoutNs)) {
        if (lane == 0) give_up();
        break;
      }
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (j < nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[m][j][i] += mine[((m * 4 + j) * 4 + i) * 32];
      __syncwarp();
      if (lane == 0) mbar_arrive(half_empty(cg));
      ++uses;
      if (un.kind == 0) {
        __nv_bfloat16* h = (un.shared ? a.s_h : a.h);
        const int c0 = un.tile * 64 + cg * 16;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (j >= nt) continue;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int n = j * 8 + 2 * q + i;
            if (n >= un.n) continue;
            const int row = un.row0 + n;
            const float w = un.shared ? 1.f : tb.w[row];
            auto swiglu = [&](float gate, float up) { return w * (gate * sigmoidf_(gate) * up); };
            __nv_bfloat16* dst = h + (int64_t)row * I;
            if constexpr (FP8) {
              const int c = c0 + 2 * g;
              if (c < I)
                *reinterpret_cast<uint32_t*>(dst + c) =
                    pack_bf16(swiglu(acc[0][j][i], acc[1][j][i]),
                              swiglu(acc[0][j][2 + i], acc[1][j][2 + i]));
            } else {
#pragma unroll
              for (int m = 0; m < 2; ++m) {
                const int c = c0 + 8 * m + g;
                if (c < I) dst[c] = __float2bfloat16_rn(swiglu(acc[m][j][i], acc[m][j][2 + i]));
              }
            }
          }
        }
        fence_proxy_async_global();
        __syncwarp();
        if (lane == 0) red_add_release_gpu(a.ready1 + un.ready, 1);
      } else {
        float* o = un.shared ? a.s_o + (int64_t)un.split * a.T * a.H
                             : a.o + (int64_t)un.split * a.S * a.H;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (j >= nt) continue;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int n = j * 8 + 2 * q + i;
            if (n >= un.n) continue;
            float* dst = o + (int64_t)(un.row0 + n) * a.H;
#pragma unroll
            for (int m = 0; m < 2; ++m) {
              const int c = un.tile * kCols + cg * 32 + m * 16 + (FP8 ? 2 * g : g);
              if constexpr (FP8) {
                if (c < a.H)
                  *reinterpret_cast<float2*>(dst + c) = make_float2(acc[m][j][i], acc[m][j][2 + i]);
              } else {
                if (c < a.H) dst[c] = acc[m][j][i];
                if (c + 8 < a.H) dst[c + 8] = acc[m][j][2 + i];
              }
            }
          }
        }
        __syncwarp();
        if (lane == 0) red_add_release_gpu(a.ready2 + un.tile, 1);
      }
    }
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
  size_t off_ready2, off_logits, off_h, off_sh, off_o, off_so, total;
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
  take((W_READY1 + S + 2) * 4);  // header, GEMM1 counters: a chunk has a row at least
  l.off_ready2 = take((size_t)((m.H + kCols - 1) / kCols) * 4);
  l.zero_words = (int)(off / 4);
  l.off_logits = take((size_t)(m.T * m.E) * 4);
  l.off_h = take(S * m.I * 2);
  l.off_sh = take((size_t)m.T * d.shared_I * 2);
  l.off_o = take((size_t)kMaxSplit * S * m.H * 4);
  l.off_so = take(d.shared_I > 0 ? (size_t)kMaxSplit * m.T * m.H * 4 : 0);
  l.total = off;
  return l;
}

bool weight_map(CUtensorMap* m, const void* base, int64_t cols, int64_t rows, int64_t n, bool fp8,
                uint32_t box_cols, uint32_t box_rows) {
  const uint64_t es = fp8 ? 1 : 2;
  const uint64_t dims[3] = {(uint64_t)cols, (uint64_t)rows, (uint64_t)n};
  const uint64_t strides[2] = {(uint64_t)cols * es, (uint64_t)cols * rows * es};
  const uint32_t box[3] = {box_cols, box_rows, 1};
  return make_map(m, base, 3, dims, strides, box,
                  fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                  box_cols * es == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B);
}

template <bool FP8>
constexpr size_t dynamic_smem() {
  return 1024 + Cfg<FP8>::STAGES * (kTileBytes + Cfg<FP8>::B_BYTES) + 4 * 32 * 32 * 4;
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
  const uint32_t rows = fp8 ? 128 : 64, down_cols = fp8 ? 128 : 64;
  bool maps = weight_map(&a.up, w->up, 2 * m.I, m.H, m.E, fp8, 64, rows) &&
              weight_map(&a.down, w->down, m.H, m.I, m.E, fp8, down_cols, rows);
  if (shared)
    maps = maps && weight_map(&a.s_up, w->shared_up, 2 * d->shared_I, m.H, 1, fp8, 64, rows) &&
           weight_map(&a.s_down, w->shared_down, m.H, d->shared_I, 1, fp8, down_cols, rows);
  if (!maps) return cuda_fail(cudaErrorInvalidValue, "decode tensor maps");
  a.x = la.x;
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
  a.h = reinterpret_cast<__nv_bfloat16*>(ws + l.off_h);
  a.s_h = reinterpret_cast<__nv_bfloat16*>(ws + l.off_sh);
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
  const dim3 grid = a.route ? dim3((unsigned)((a.E + 3) / 4), (unsigned)((a.T + 3) / 4)) : dim3(1);
  if (d->router_type == MM_BF16)
    MM_TRY(launch_pdl(k_logits<__nv_bfloat16>, grid, dim3(256), 0, st, la));
  else
    MM_TRY(launch_pdl(k_logits<float>, grid, dim3(256), 0, st, la));
  const int sms = std::max(1, device_sm_count());
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
