// Products grouped by expert with ragged sizes, and their weight gradients (definitions in
// mm_experts.h), on tcgen05.
//
// Both are one shape of product: out[j][i] = sum_k A[i][k] B[j][k] with i contiguous in the output.
//   rows:    i = output column, j = row of the expert; A = the expert's matrix, B = its rows.
//   weights: i = the matrix's contiguous dimension, j = the other; k = the expert's rows; A and B are
//            d_out and rows (or the other way round, for transposed matrices).
// The matrix is the M operand (128 columns a CTA) and the rows are N: a tile's N is the number of rows
// of its chunk, rounded up to 16, so that ragged experts cost what they have and not a multiple of
// 128, and one row costs 16. An expert of more than `chunk` rows is cut into equal chunks. Neighbours'
// rows that a chunk's box reaches into are columns of the accumulator that nobody stores.
//
// A CTA: a warp that loads (TMA, a ring of stages of 64 k), a warp that issues the products into two
// accumulators of 256 columns in turn, eight warps that store. PAIR: two CTAs share one M = 256 product
// (.cta_group::2); each holds its 128 columns of the matrix and half of the rows.
//
// With k = rows (weights) the last 16 rows of an expert's sum may reach into the next expert's; those
// rows are set to zero in shared memory, in both operands (0 times an infinity would not be 0).
#include <algorithm>
#include <atomic>

#include "../../include/mm_experts.h"
#include "mm_kernels.h"
#include "mm_rows.cuh"

namespace mm {
namespace {

constexpr int kThreads = 320;      // a warp that loads, one that multiplies, eight that store
constexpr int kStoreWarps = 8;
constexpr int kMaxE = 1024;
constexpr int kTile = 128;         // columns of the M operand per CTA
constexpr int kMaxN = 256;         // rows (or columns of the other dimension) per tile
constexpr int kMaxStages = 12;
constexpr uint32_t kABytes = kTile * 64 * 2;
constexpr uint32_t kBlock = 64 * 64 * 2;  // 64 elements of a MN-major operand over 64 k
constexpr uint32_t kBarBytes = 512;
constexpr uint32_t kTableBytes = 2 * 4 * (kMaxE + 1) + 8;
constexpr uint32_t kMostSmem = 227 * 1024;
constexpr uint64_t kWaitNs = 2000000000ull;

struct Maps {
  CUtensorMap a;     // rows: a box of 128 columns of the matrix (K-major) or 64 (MN-major); weights: 64 x 64
  CUtensorMap b[5];  // rows: boxes of 128, 64, 32, 16, 8 rows; weights: b[0], 64 x 64
};

struct Args {
  const int32_t* offsets;
  void* out;
  int R, E;
  int I, J;       // columns of the output; weights: rows of an expert's output
  int K;          // rows: terms of a sum
  int a_kmajor;   // rows: the matrix's k is contiguous
  int chunk;      // most rows (J) of a tile, a multiple of 16
  int stages;
  uint32_t stage_bytes;
  int f32, accumulate;
};

struct Unit {
  int e, i0, j0;   // i0: first column of this CTA; j0: rows: first row of the chunk in all rows
  int n, n16;      // columns of the accumulator that are stored and computed
  int row0, k;     // weights: the expert's first row; terms of a sum
};

__device__ __forceinline__ bool mbar_wait_cluster(uint32_t bar, uint32_t parity, uint64_t limit_ns) {
  const uint64_t t0 = globaltimer_ns();
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 32; ++i) {
      uint32_t ok;
      asm volatile(
          "{\n\t.reg .pred p;\n\t"
          "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
          "selp.u32 %0, 1, 0, p;\n\t}"
          : "=r"(ok)
          : "r"(bar), "r"(parity)
          : "memory");
      if (ok) return true;
    }
    if (globaltimer_ns() - t0 > limit_ns) return false;
  }
}

__device__ __forceinline__ void mbar_arrive_remote(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr)
               : "memory");
}

// A wait by all lanes of a warp, with one answer for them.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity) {
  return __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity, kWaitNs));
}

// A value that all lanes share, in the form the compiler knows to be shared: what an issue of a copy or a
// product takes is then in uniform registers, and no loop over the lanes' values stands around it.
__device__ __forceinline__ int uniform(int v) { return __reduce_min_sync(0xFFFFFFFFu, v); }

// A ring of barriers as one warp in step walks it. The next one is asked for before the present one's
// work is issued, so that the answer's latency passes behind it.
struct Ring {
  uint32_t bar0, phase;  // first barrier; parity to wait for
  int stages, s = 0;
  bool ready = false;
  __device__ __forceinline__ Ring(uint32_t bar, uint32_t first, int n) : bar0(bar), phase(first), stages(n) {}
  __device__ __forceinline__ bool wait() {
    if (__all_sync(0xFFFFFFFFu, ready)) return true;
    return warp_wait(bar0 + 8u * s, phase);
  }
  __device__ __forceinline__ void ask_next() {
    const bool wrap = s + 1 == stages;
    ready = mbar_test_wait(bar0 + 8u * (wrap ? 0 : s + 1), wrap ? phase ^ 1u : phase);
  }
  __device__ __forceinline__ void next() {
    if (++s == stages) s = 0, phase ^= 1u;
  }
  __device__ __forceinline__ void skip(int n) {  // n stages that another warp walks
    ready = false;
    s += n;
    if (s / stages & 1) phase ^= 1u;
    s %= stages;
  }
};

// Where the experts' rows start (E + 1 numbers) and how many tiles of rows the experts before each
// have, in shared memory. False if the offsets are no such table.
template <bool WEIGHTS>
__device__ __forceinline__ bool build_table(const Args& a, int* start, int* first) {
  __shared__ int sums[kThreads / 32];
  constexpr int PER = (kMaxE + kThreads - 1) / kThreads;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int tiles[PER], mine = 0;
  int bad = 0;
#pragma unroll
  for (int p = 0; p < PER; ++p) {
    const int e = tid * PER + p;
    tiles[p] = 0;
    if (e < a.E) {
      const int s = a.offsets[e], t = a.offsets[e + 1];
      bad |= s < 0 || t < s || t > a.R;
      start[e] = s;
      if (e == a.E - 1) start[a.E] = t;
      tiles[p] = WEIGHTS ? 1 : (t - s + a.chunk - 1) / a.chunk;
    }
    mine += tiles[p];
  }
  if (__syncthreads_or(bad)) return false;
  int upto = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int v = __shfl_up_sync(0xFFFFFFFFu, upto, d);
    if (lane >= d) upto += v;
  }
  if (lane == 31) sums[warp] = upto;
  __syncthreads();
  int base = upto - mine;
  for (int w = 0; w < warp; ++w) base += sums[w];
#pragma unroll
  for (int p = 0; p < PER; ++p) {
    const int e = tid * PER + p;
    if (e < a.E) first[e] = base;
    base += tiles[p];
    if (e == a.E - 1) first[a.E] = base;
  }
  __syncthreads();
  return true;
}

// Unit u of the launch; i_tiles: tiles of the output's columns.
template <bool WEIGHTS, int PAIR>
__device__ __forceinline__ Unit unit_at(const Args& a, const int* start, const int* first, int u,
                                        int i_tiles, int j_tiles, int rank) {
  Unit t;
  if constexpr (WEIGHTS) {
    const int per = i_tiles * j_tiles;
    t.e = u / per;
    const int in = u - t.e * per, jt = in / i_tiles;
    t.i0 = (in - jt * i_tiles) * kTile * PAIR + rank * kTile;
    t.j0 = jt * a.chunk;
    t.n = min(a.chunk, a.J - t.j0);
    t.row0 = start[t.e];
    t.k = start[t.e + 1] - t.row0;
  } else {
    const int q = u / i_tiles;
    int lo = 0, hi = a.E;  // first[lo] <= q < first[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (first[mid] <= q) lo = mid; else hi = mid;
    }
    t.e = lo;
    const int chunks = first[lo + 1] - first[lo], in = u - first[lo] * i_tiles;
    const int it = in / chunks, c = in - it * chunks;
    const int rows = start[lo + 1] - start[lo];
    // equal chunks; as none is above a.chunk the last one has a row at least
    const int per = ((rows + chunks - 1) / chunks + 15) & ~15;
    t.i0 = it * kTile * PAIR + rank * kTile;
    t.j0 = start[lo] + c * per;
    t.n = min(per, rows - c * per);
    t.row0 = 0;
    t.k = a.K;
  }
  t.n16 = (t.n + 15) & ~15;
  return t;
}

// `words` 16-byte words at p set to v by the launch's storing warps.
__device__ __forceinline__ void fill(void* p, int64_t words, uint32_t v, int thread, int threads) {
  uint4* w = static_cast<uint4*>(p);
  for (int64_t i = thread; i < words; i += threads) w[i] = make_uint4(v, v, v, v);
}

// Up to 32 columns of the accumulator (this lane: one i) to rows row .. of the output; n: how many there
// are. The address of a row is that of the one before plus the pitch, as 64-bit products per element were
// most of an epilogue's instructions.
template <bool F32, bool ADD, bool FULL>
__device__ __forceinline__ void store_rows(const Args& a, const float (&v)[32], int64_t row, int i, int n,
                                           int lane) {
  if constexpr (F32) {
    if (i >= a.I) return;
    float* p = static_cast<float*>(a.out) + row * a.I + i;
    float old[32];
    if constexpr (ADD) {
      const float* at = p;
#pragma unroll
      for (int j = 0; j < 32; ++j, at += a.I) old[j] = FULL || j < n ? *at : 0.f;
    }
#pragma unroll
    for (int j = 0; j < 32; ++j, p += a.I)
      if (FULL || j < n) *p = ADD ? v[j] + old[j] : v[j];
  } else {
    // Two neighbouring lanes exchange, so that each has a pair of neighbouring columns of one row: the
    // even lane of row j, the odd one of row j + 1.
    const int odd = lane & 1;
    const bool there = i < a.I;
    const uint32_t halves = odd ? 0x3276 : 0x5410;
    uint32_t* p = reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(a.out) + (row + odd) * a.I + (i & ~1));
#pragma unroll
    for (int j = 0; j < 32; j += 2, p += a.I) {
      if constexpr (ADD) {  // (the sum is rounded, not its addend)
        const float other = __shfl_xor_sync(0xFFFFFFFFu, odd ? v[j] : v[j + 1], 1);
        if (there && (FULL || j + odd < n)) {
          const uint32_t old = *p;
          *p = pack_bf16((odd ? other : v[j]) + bf16_lo(old), (odd ? v[j + 1] : other) + bf16_hi(old));
        }
      } else {
        const uint32_t mine = pack_bf16(v[j], v[j + 1]);
        const uint32_t both = __byte_perm(mine, __shfl_xor_sync(0xFFFFFFFFu, mine, 1), halves);
        if (there && (FULL || j + odd < n)) *p = both;
      }
    }
  }
}

__device__ __forceinline__ void store_columns(const Args& a, const float (&v)[32], int64_t row, int i, int n,
                                              int lane) {
  const bool full = n >= 32;
  if (a.accumulate) {
    if (a.f32) store_rows<true, true, false>(a, v, row, i, n, lane);
    else store_rows<false, true, false>(a, v, row, i, n, lane);
  } else if (a.f32) {
    if (full) store_rows<true, false, true>(a, v, row, i, n, lane);
    else store_rows<true, false, false>(a, v, row, i, n, lane);
  } else {
    if (full) store_rows<false, false, true>(a, v, row, i, n, lane);
    else store_rows<false, false, false>(a, v, row, i, n, lane);
  }
}

template <int PAIR, bool WEIGHTS>
__global__ void __launch_bounds__(kThreads, 1)
    k_grouped(const __grid_constant__ Maps m, const Args a) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ uint32_t tmem_holder;
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  const uint32_t bars = sbase + a.stages * a.stage_bytes;
  int* const start = reinterpret_cast<int*>(smem_raw + (bars + kBarBytes - raw));
  int* const first_tile = start + kMaxE + 1;
  auto full_bar = [&](uint32_t s) { return bars + 8u * s; };
  auto empty_bar = [&](uint32_t s) { return bars + 8u * (kMaxStages + s); };
  // weights, pairs: the odd CTA's part of an expert's last block, loaded and set to zero
  auto tail_bar = [&](uint32_t s) { return bars + 8u * (2 * kMaxStages + s); };
  auto fixed_bar = [&](uint32_t s) { return bars + 8u * (3 * kMaxStages + s); };
  auto accf_bar = [&](uint32_t b) { return bars + 8u * (4 * kMaxStages + b); };
  auto acce_bar = [&](uint32_t b) { return bars + 8u * (4 * kMaxStages + 2 + b); };
  static_assert(8 * (4 * kMaxStages + 4) <= kBarBytes, "barrier area");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = PAIR == 2 ? (int)cluster_ctarank() : 0;
  const int step = (int)gridDim.x / PAIR, mine = (int)blockIdx.x / PAIR;
  if (threadIdx.x == 0) {
    for (int s = 0; s < a.stages; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
      mbar_init(tail_bar(s), 1);
      mbar_init(fixed_bar(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(accf_bar(b), 1);
      mbar_init(acce_bar(b), PAIR * kStoreWarps);
    }
    mbar_fence_init();
    tma_prefetch_desc(&m.a);
    tma_prefetch_desc(&m.b[0]);
  }
  if (warp == 1) {
    if constexpr (PAIR == 2) {
      tmem_alloc_pair(smem_u32(&tmem_holder), 512);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(smem_u32(&tmem_holder), 512);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  pdl_wait();
  const bool good = build_table<WEIGHTS>(a, start, first_tile);  // (a barrier for the block)
  tc_fence_after();
  if constexpr (PAIR == 2) cluster_sync();
  const uint32_t tmem = *static_cast<volatile uint32_t*>(&tmem_holder);

  const int i_tiles = (a.I + kTile * PAIR - 1) / (kTile * PAIR);
  const int j_tiles = WEIGHTS ? (a.J + a.chunk - 1) / a.chunk : 1;
  const int units = !good ? 0 : WEIGHTS ? a.E * i_tiles * j_tiles : first_tile[a.E] * i_tiles;

  if (warp == 0) {
    // ------------------------------------------------ loads
    Ring ring(empty_bar(0), 1, a.stages);
    int it = 0;
    bool ok = true;
    const bool kmajor = a.a_kmajor != 0;
    for (int u = mine; u < units && ok; u += step) {
      const Unit t = unit_at<WEIGHTS, PAIR>(a, start, first_tile, u, i_tiles, j_tiles, rank);
      const int half = uniform(t.n16 / PAIR), blocks = uniform((t.k + 63) / 64);
      const int e = uniform(t.e), i0 = uniform(t.i0), row0 = uniform(t.row0);
      const int j0 = uniform(t.j0 + rank * (t.n16 / PAIR));
      const bool mend = uniform(t.k & 15) != 0;
      const uint32_t bytes = kABytes + (WEIGHTS ? (half + 63) / 64 * kBlock : half * 128u);
      for (int kb = 0; kb < blocks; ++kb, ++it) {
        if (!ring.wait()) {
          ok = false;
          break;
        }
        ring.ask_next();
        if (elect_one()) {
          const uint32_t sa = sbase + ring.s * a.stage_bytes, sb = sa + kABytes;
          const int k0 = kb * 64;
          // the two CTAs' bytes of a stage count on the even one's barrier, but those of a block that
          // is to be mended in place each on its own
          const bool tail = WEIGHTS && PAIR == 2 && kb == blocks - 1 && mend;
          uint32_t bar = full_bar(ring.s);
          if (tail) {
            if (rank == 1) bar = tail_bar(ring.s);
            mbar_arrive_expect_tx(bar, bytes);
          } else if (rank == 0) {
            mbar_arrive_expect_tx(bar, PAIR * bytes);
          }
          if constexpr (PAIR == 2) bar = mapa_shared(bar, tail ? rank : 0);
          auto load2 = [&](uint32_t dst, const CUtensorMap* map, int c0, int c1) {
            if constexpr (PAIR == 2) tma_load_2d_pair(dst, map, bar, c0, c1);
            else tma_load_2d(dst, map, bar, c0, c1);
          };
          auto load3 = [&](uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2) {
            if constexpr (PAIR == 2) tma_load_3d_pair(dst, map, bar, c0, c1, c2);
            else tma_load_3d(dst, map, bar, c0, c1, c2);
          };
          if constexpr (WEIGHTS) {
            load2(sa, &m.a, i0, row0 + k0);
            load2(sa + kBlock, &m.a, i0 + 64, row0 + k0);
#pragma unroll
            for (int c = 0; c < kMaxN / PAIR; c += 64)
              if (c < half) load2(sb + c / 64 * kBlock, &m.b[0], j0 + c, row0 + k0);
          } else {
            if (kmajor) {
              load3(sa, &m.a, k0, i0, e);
            } else {
              load3(sa, &m.a, i0, k0, e);
              load3(sa + kBlock, &m.a, i0 + 64, k0, e);
            }
            // boxes as half's bits are (256: 128 twice)
            int r = 0;
            if (PAIR == 1 && (half & 256)) {
              load2(sb, &m.b[0], k0, j0);
              load2(sb + 128 * 128, &m.b[0], k0, j0 + 128);
            }
#pragma unroll
            for (int p = 0; p < 5; ++p) {
              if (half & (128 >> p)) {
                load2(sb + r * 128, &m.b[p], k0, j0 + r);
                r += 128 >> p;
              }
            }
          }
        }
        __syncwarp();
        ring.next();
      }
    }
    // every stage's last release has landed before this CTA may leave
    for (int s = 0; s < a.stages && s < it && ok; ++s)
      ok = warp_wait(empty_bar(s), (it - 1 - s) / a.stages & 1u);
  } else if (warp == 1) {
    // ------------------------------------------------ multiplies
    // The warp stays in step and an elected lane issues from uniform registers.
    Ring ring(full_bar(0), 0, a.stages);
    const int a_mn = WEIGHTS || !a.a_kmajor, b_mn = WEIGHTS;
    const uint64_t adesc = sdesc_sw128(sbase, a_mn ? kBlock : 16, 1024);
    const uint64_t bdesc = sdesc_sw128(sbase + kABytes, b_mn ? kBlock : 16, 1024);
    const uint32_t a_step = a_mn ? 2048 / 16 : 2, b_step = b_mn ? 2048 / 16 : 2;
    uint32_t acc = 0, tails = 0;
    bool ok = true;
    for (int u = mine; u < units && ok; u += step) {
      const Unit t = unit_at<WEIGHTS, PAIR>(a, start, first_tile, u, i_tiles, j_tiles, rank);
      const int blocks = uniform((t.k + 63) / 64), n16 = uniform(t.n16);
      if (blocks == 0) continue;
      const int last = uniform(t.k) - (blocks - 1) * 64;  // terms in the last block
      const bool mend = WEIGHTS && (last & 15) != 0;
      const uint32_t buf = acc & 1u;
      const uint32_t d = tmem + buf * kMaxN;
      // sets the rows of the next expert to zero in this CTA's part of stage s
      auto zero_rows = [&](uint32_t s) {
        const uint32_t sa = sbase + s * a.stage_bytes;
        const int parts = 2 + (n16 / PAIR + 63) / 64, end = ((last + 15) & ~15) * 128;
        for (int p = 0; p < parts; ++p)
          for (int at = last * 128 + lane * 16; at < end; at += 512)
            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(
                             sa + (p < 2 ? p * kBlock : kABytes + (p - 2) * kBlock) + at),
                         "r"(0)
                         : "memory");
        fence_proxy_async_smem();
        __syncwarp();
      };
      if (PAIR == 2 && rank == 1) {  // the even CTA issues; this one mends its part
        ring.skip(blocks - 1);
        if (mend) {
          const uint32_t s = ring.s;
          if (!warp_wait(tail_bar(s), tails >> s & 1u)) {
            ok = false;
            break;
          }
          tails ^= 1u << s;
          zero_rows(s);
          if (lane == 0) mbar_arrive_remote(mapa_shared(fixed_bar(s), 0));
        }
        ring.next();
        continue;
      }
      if (!warp_wait(acce_bar(buf), (acc >> 1 & 1u) ^ 1u)) break;
      tc_fence_after();
      const uint32_t idesc = idesc_bf16_f32(kTile * PAIR, n16, a_mn, b_mn);
      for (int kb = 0; kb < blocks; ++kb) {
        if (!ring.wait()) {
          ok = false;
          break;
        }
        const uint32_t s = ring.s;
        ring.ask_next();
        int steps = 4;
        if (WEIGHTS && kb == blocks - 1) {
          steps = (last + 15) / 16;
          if (mend) {
            zero_rows(s);
            if constexpr (PAIR == 2) {
              if (!__all_sync(0xFFFFFFFFu, mbar_wait_cluster(fixed_bar(s), tails >> s & 1u, kWaitNs))) {
                ok = false;
                break;
              }
              tails ^= 1u << s;
            }
          }
        }
        tc_fence_after();
        if (elect_one()) {
          const uint64_t ad = adesc + s * (a.stage_bytes / 16), bd = bdesc + s * (a.stage_bytes / 16);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            if (WEIGHTS && kk >= steps) continue;
            if constexpr (PAIR == 2) umma_bf16_pair(d, ad + kk * a_step, bd + kk * b_step, idesc, (kb | kk) != 0);
            else umma_bf16(d, ad + kk * a_step, bd + kk * b_step, idesc, (kb | kk) != 0);
          }
          if constexpr (PAIR == 2) umma_commit_pair_mc(empty_bar(s), 0x3);
          else umma_commit(empty_bar(s));
          if (kb == blocks - 1) {
            if constexpr (PAIR == 2) umma_commit_pair_mc(accf_bar(buf), 0x3);
            else umma_commit(accf_bar(buf));
          }
        }
        __syncwarp();
        ring.next();
      }
      ++acc;
    }
  } else {
    const int q = warp & 3, set = (warp - 2) >> 2;
    const int64_t es = a.f32 ? 4 : 2;
    {
      const int thread = (int)blockIdx.x * (32 * kStoreWarps) + (int)threadIdx.x - 64;
      const int threads = (int)gridDim.x * (32 * kStoreWarps);
      char* out = static_cast<char*>(a.out);
      if (!good) {
        const int64_t rows = WEIGHTS ? (int64_t)a.E * a.J : a.R;
        fill(out, rows * a.I * es / 16, a.f32 ? 0x7FC00000u : 0x7FC07FC0u, thread, threads);
      } else if (!WEIGHTS) {
        fill(out, start[0] * (a.I * es / 16), 0, thread, threads);
        fill(out + start[a.E] * (a.I * es), (a.R - start[a.E]) * (a.I * es / 16), 0, thread, threads);
      }
    }
    uint32_t acc = 0;
    bool ok = true;
    for (int u = mine; u < units; u += step) {
      const Unit t = unit_at<WEIGHTS, PAIR>(a, start, first_tile, u, i_tiles, j_tiles, rank);
      if (t.k == 0 && a.accumulate) continue;  // adding zero changes nothing
      const uint32_t buf = acc & 1u;
      if (t.k > 0 && ok) {
        ok = warp_wait(accf_bar(buf), acc >> 1 & 1u);
      }
      tc_fence_after();
      const int64_t row0 = WEIGHTS ? (int64_t)t.e * a.J + t.j0 : t.j0;
      const int i = t.i0 + q * 32 + lane;
      for (int c = set * 32; c < t.n; c += 64) {
        float v[32];
        if (t.k > 0 && ok) {
          uint32_t r[32];
          tmem_ld_32x32(tmem + ((uint32_t)(q * 32) << 16) + buf * kMaxN + c, r);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(r[j]);
        } else {
          const float none = t.k > 0 ? __int_as_float(0x7FC00000) : 0.f;  // NaN after an error
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = none;
        }
        store_columns(a, v, row0 + c, i, t.n - c, lane);
      }
      if (t.k > 0) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0 && ok) {
          if (PAIR == 2 && rank != 0) mbar_arrive_remote_relaxed(mapa_shared(acce_bar(buf), 0));
          else mbar_arrive(acce_bar(buf));
        }
        ++acc;
      }
    }
  }
  pdl_launch_dependents();
  tc_fence_before();
  __syncthreads();
  if constexpr (PAIR == 2) cluster_sync();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    if constexpr (PAIR == 2) tmem_dealloc_pair(tmem, 512);
    else tmem_dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------------------------------ host side

inline bool aligned_to(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

mm_status check_desc(const mm_grouped_desc* d) {
  if (d == nullptr || d->R < 0 || d->K < 1 || d->N < 1 || d->E < 1) return MM_ERR_INVALID_ARG;
  if (d->out_type != MM_BF16 && d->out_type != MM_FP32) return MM_ERR_INVALID_ARG;
  if (d->flags > 2) return MM_ERR_INVALID_ARG;  // unknown flags, or both forms
  if (d->K % 8 || d->N % 8 || d->K > 65536 || d->N > 65536 || d->E > kMaxE ||
      d->R >= (int64_t)1 << 31)
    return MM_ERR_UNSUPPORTED;
  return MM_OK;
}

bool map2(CUtensorMap* m, const void* base, int64_t cols, int64_t rows, uint32_t box_rows) {
  const uint64_t dims[2] = {(uint64_t)cols, (uint64_t)rows};
  const uint64_t strides[1] = {(uint64_t)cols * 2};
  const uint32_t box[2] = {64, box_rows};
  return make_map(m, base, 2, dims, strides, box);
}

template <int PAIR, bool WEIGHTS>
cudaError_t launch(const Maps& m, Args a, int64_t units, cudaStream_t st) {
  a.stage_bytes = kABytes + (WEIGHTS ? (a.chunk / PAIR + 63) / 64 * kBlock : a.chunk / PAIR * 128u);
  const uint32_t fixed = 1024 + kBarBytes + kTableBytes;
  a.stages = (int)std::min<uint32_t>(kMaxStages, (kMostSmem - 1024 - fixed) / a.stage_bytes);
  const size_t smem = fixed + (size_t)a.stages * a.stage_bytes;
  static std::atomic<uint64_t> ready{0};
  static std::atomic<int> most_clusters[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!(ready.load(std::memory_order_relaxed) >> dev & 1)) {
    e = cudaFuncSetAttribute(k_grouped<PAIR, WEIGHTS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)(kMostSmem - 1024));
    if (e != cudaSuccess) return e;
    ready.fetch_or(1ull << dev, std::memory_order_relaxed);
  }
  int fit = std::max(1, device_sm_count());
  if constexpr (PAIR == 1) {
    return launch_pdl(k_grouped<PAIR, WEIGHTS>, dim3((unsigned)std::max<int64_t>(1, std::min<int64_t>(fit, units))),
                      dim3(kThreads), smem, st, m, a);
  } else {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.gridDim = dim3((unsigned)(fit & ~1));
    // clusters that fit at once, asked once per device with the largest shared memory
    fit = most_clusters[dev].load(std::memory_order_relaxed);
    if (fit == 0) {
      cfg.dynamicSmemBytes = kMostSmem - 1024;
      e = cudaOccupancyMaxActiveClusters(&fit, k_grouped<PAIR, WEIGHTS>, &cfg);
      if (e != cudaSuccess) return e;
      if (fit < 1) return cudaErrorInvalidConfiguration;
      most_clusters[dev].store(fit, std::memory_order_relaxed);
      cfg.dynamicSmemBytes = smem;
    }
    cfg.gridDim = dim3((unsigned)(2 * std::max<int64_t>(1, std::min<int64_t>(fit, units))));
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, k_grouped<PAIR, WEIGHTS>, m, a);
  }
}

}  // namespace
}  // namespace mm

using namespace mm;

extern "C" {

int mm_experts_version(void) { return 1; }

size_t mm_grouped_workspace_size(const mm_grouped_desc* d) {
  return check_desc(d) == MM_OK ? 256 : 0;
}

mm_status mm_grouped_mm(const mm_grouped_desc* d, const void* rows, const void* weight,
                        const int32_t* offsets, void* out, void* workspace, size_t workspace_bytes,
                        void* stream) {
  mm_status s = check_desc(d);
  if (s != MM_OK) return s;
  if (!aligned_to(rows, 16) || !aligned_to(weight, 16) || !aligned_to(out, 16) || !aligned_to(offsets, 4))
    return MM_ERR_INVALID_ARG;
  if (d->R == 0) return MM_OK;
  if (!rows || !weight || !out || !offsets) return MM_ERR_INVALID_ARG;
  if (workspace == nullptr || !aligned_to(workspace, 256) || workspace_bytes < mm_grouped_workspace_size(d))
    return MM_ERR_WORKSPACE;
  clear_error();
  MM_TRY(bind_context());
  // Pairs read half as much of their operands per product. Where a launch has no more tiles of one CTA
  // than SMs, these spread the matrices' columns over twice as many. (us a call, one CTA a tile and pairs:
  // 8 rows of 8 of 128 experts, 2048 -> 1536, 13.1 and 13.8; 512 rows of 128, 768 -> 2048, 73.5 and 66.0;
  // 131072 rows of 128, 2048 -> 1536, 592 and 528.)
  const int64_t chunks = d->R / kMaxN + std::min<int64_t>(d->E, d->R);  // at most
  const bool few = chunks * ((d->N + kTile - 1) / kTile) <= device_sm_count();
  const int pair = d->flags & MM_GROUPED_CTA_PAIRS || (d->flags == 0 && !few) ? 2 : 1;
  Maps m;
  Args a{};
  a.offsets = offsets;
  a.out = out;
  a.R = (int)d->R;
  a.E = d->E;
  a.I = (int)d->N;
  a.K = (int)d->K;
  a.a_kmajor = d->transposed != 0;
  a.f32 = d->out_type == MM_FP32;
  a.chunk = (int)std::min<int64_t>(kMaxN, (d->R + 15) / 16 * 16);
  const int64_t inner = d->transposed ? d->K : d->N, outer = d->transposed ? d->N : d->K;
  const uint64_t dims[3] = {(uint64_t)inner, (uint64_t)outer, (uint64_t)d->E};
  const uint64_t strides[2] = {(uint64_t)inner * 2, (uint64_t)inner * outer * 2};
  const uint32_t box[3] = {64, d->transposed ? 128u : 64u, 1};
  bool ok = make_map(&m.a, weight, 3, dims, strides, box);
  for (int p = 0; p < 5; ++p) ok = ok && map2(&m.b[p], rows, d->K, d->R, 128u >> p);
  if (!ok) return cuda_fail(cudaErrorInvalidValue, "grouped product tensor maps");
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const int64_t units = chunks * ((d->N + kTile * pair - 1) / (kTile * pair));
  if (pair == 2)
    MM_TRY((launch<2, false>(m, a, units, st)));
  else
    MM_TRY((launch<1, false>(m, a, units, st)));
  return MM_OK;
}

mm_status mm_grouped_mm_weight_grad(const mm_grouped_desc* d, const void* rows, const void* d_out,
                                    const int32_t* offsets, void* d_weight, int accumulate,
                                    void* workspace, size_t workspace_bytes, void* stream) {
  mm_status s = check_desc(d);
  if (s != MM_OK) return s;
  if (!aligned_to(rows, 16) || !aligned_to(d_out, 16) || !aligned_to(d_weight, 16) || !aligned_to(offsets, 4))
    return MM_ERR_INVALID_ARG;
  if (!d_weight || !offsets || (d->R > 0 && (!rows || !d_out))) return MM_ERR_INVALID_ARG;
  if (workspace == nullptr || !aligned_to(workspace, 256) || workspace_bytes < mm_grouped_workspace_size(d))
    return MM_ERR_WORKSPACE;
  clear_error();
  MM_TRY(bind_context());
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (d->R == 0) {  // no row: zeros
    if (!accumulate)
      MM_TRY(cudaMemsetAsync(d_weight, 0, (size_t)d->E * d->K * d->N * (d->out_type == MM_FP32 ? 4 : 2), st));
    return MM_OK;
  }
  const int pair = d->flags & MM_GROUPED_SINGLE_CTA ? 1 : 2;
  Maps m;
  Args a{};
  a.offsets = offsets;
  a.out = d_weight;
  a.R = (int)d->R;
  a.E = d->E;
  a.I = (int)(d->transposed ? d->K : d->N);
  a.J = (int)(d->transposed ? d->N : d->K);
  a.f32 = d->out_type == MM_FP32;
  a.accumulate = accumulate != 0;
  a.chunk = std::min(kMaxN, (a.J + 15) / 16 * 16);
  const bool ok = map2(&m.a, d->transposed ? rows : d_out, a.I, d->R, 64) &&
                  map2(&m.b[0], d->transposed ? d_out : rows, a.J, d->R, 64);
  if (!ok) return cuda_fail(cudaErrorInvalidValue, "grouped product tensor maps");
  const int64_t units = (int64_t)d->E * ((a.I + kTile * pair - 1) / (kTile * pair)) *
                        ((a.J + a.chunk - 1) / a.chunk);
  if (pair == 2)
    MM_TRY((launch<2, true>(m, a, units, st)));
  else
    MM_TRY((launch<1, true>(m, a, units, st)));
  return MM_OK;
}

}  // extern "C"
