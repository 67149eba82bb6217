// Products grouped by expert with ragged sizes, and their weight gradients (definitions in
// mm_experts.h), on tcgen05.
//
// Both are one shape of product: out[j][i] = sum_k A[i][k] B[j][k] with i contiguous in the output.
//   rows:    i = output column, j = row of the expert; A = the expert's matrix, B = its rows.
//   weights: i = the matrix's contiguous dimension, j = the other; k = the expert's rows; A and B are
//            d_out and rows (the other way round for transposed matrices).
// The matrix is the M operand (128 columns a CTA) and the rows are N: a tile's N is the number of rows
// of its chunk, rounded up to 16, so that ragged experts cost what they have and not a multiple of
// 128, and one row costs 16. An expert of more than `chunk` rows is cut into equal chunks (full ones and a
// rest are 1 % slower at 1030 rows). Neighbours' rows that a chunk's box reaches into are columns of the
// accumulator that nobody stores.
//
// A CTA: a warp that loads (TMA, a ring of stages of 64 k), a warp that issues the products into two
// accumulators of 256 columns in turn, eight warps that store, and one that deals out the tiles. PAIR: two
// CTAs share one M = 256 product (.cta_group::2); each holds its 128 columns of the matrix and half of
// the rows.
//
// With k = rows (weights) the last 16 rows of an expert's sum may reach into the next expert's, whose
// infinities would not vanish by a zero in the other operand. A launch before copies every expert's last
// rows % 16 rows of both operands to panels of 16 rows filled up with zeros, from where the last step's
// operands are loaded. (Zeros written over the loaded rows in shared memory stood in the way of every
// tile's last block: 65536 rows of 128 experts, 2048 x 1536, 384 us, of which 80 were theirs; boxes of
// exactly the rows there are took 444 for their number.)
//
// The dealing warp of the even CTA tells all others the tiles through a queue, ahead of their use. Rows'
// tiles are dealt in turn, every CTA has every step-th: even for experts of many rows, uneven for skewed
// sizes, where a tile has 16 to 256 columns (6007 skewed rows of 32 experts, counted with a cost of its
// columns, 128 at least: the busiest pair of 76 has 1.2 to 1.5 times the mean; largest first 1.1).
// Weights' tiles go by the experts' rows: they are claimed from a counter, largest sums first.
//
// The tensor cores' sums lose about 2^-30 of their value with every term, always towards zero. Where the
// result has 32 bits a sum is therefore cut into runs of at most kRun blocks, which the storing warps add
// up in registers (8192 rows by 7168 x 2048: 5.6e-6 of the result's norm off without, below 1e-6 with).
//
// What bounds it: with many rows the tensor cores, as far as the power cap and the operands' way through L2
// let them (13 TB/s; 131072 rows of 128 experts, 2048 -> 1536, 467-515 us, 1600-1765 TFLOP/s; 1440-1570 in a
// long run); with few rows the matrices' way from HBM (512 rows of 128 experts, 768 -> 2048, 66.7 us, 6.0
// TB/s); a weight gradient of few rows its result's way there (512 rows of those, 86 us, 4.7 TB/s).
//
// Few tiles, or one expert with most rows, would leave SMs idle: then sums are cut over k, the parts go to
// slices of 32-bit numbers in the workspace, and a launch behind adds the slices in their order.
//
// Sums added to a kept gradient read and write it 4 bytes a lane, row by row, and are far from HBM's rate
// (32768 skewed rows of 128 experts, 768 x 2048: 772 us into 32 bits, 1610 into bf16; 134 as a bf16 result
// of its own).
//
// Waits on barriers have a limit. Without one are: the kernels before (pdl_wait); tensor memory, asked for
// when those have ended and both CTAs run; the registers of the 32-bit kernels (kLaunchRegs); and block and
// cluster barriers, which every warp reaches, as what it does before them is bounded.
#include <algorithm>
#include <atomic>

#include "../../include/mm_experts.h"
#include "mm_kernels.h"
#include "mm_rows.cuh"

namespace mm {
namespace {

constexpr int kThreads = 384;      // warps that load, multiply and deal out tiles (and none), eight that store
constexpr int kStoreWarps = 8, kFirstStore = 4;
// Registers of a thread: the block is launched with 168 x 384, and the storing warps, which hold a tile's
// 128 sums per thread, take over what the first four warps do not need (56 x 128 + 224 x 256 of them). A
// block launched with fewer would wait for them for ever, so the launch asks what the kernel was built with.
constexpr int kLaunchRegs = 168, kFewRegs = 56, kManyRegs = 224;
static_assert(kFewRegs * 32 * kFirstStore + kManyRegs * 32 * kStoreWarps <= kLaunchRegs * kThreads, "register shares");
constexpr int kRun = 8;            // blocks of 64 terms
constexpr int kQueue = 8;          // tiles told and not yet taken by all
constexpr int kMaxE = 1024;
constexpr int kTile = 128;         // columns of the M operand per CTA
constexpr int kMaxN = 256;         // rows (or columns of the other dimension) per tile
constexpr int kMaxStages = 12;
constexpr uint32_t kABytes = kTile * 64 * 2;
constexpr uint32_t kBlock = 64 * 64 * 2;  // 64 elements of a MN-major operand over 64 k
constexpr uint32_t kBarBytes = 512;
constexpr uint32_t kTableBytes = 2 * 4 * (kMaxE + 1) + 8 + 2 * kMaxE;
constexpr uint32_t kOutBytes = 32 * 64;   // a storing warp's share of its set's 32 rows of 128 columns
constexpr uint32_t kMostSmem = 227 * 1024;
constexpr uint64_t kWaitNs = 2000000000ull, kTestWaitNs = 50000000ull;

struct Maps {
  CUtensorMap a;     // rows: a box of 128 columns of the matrix (K-major) or 64 (MN-major); weights: 64 x 64
  CUtensorMap b[5];  // rows: boxes of 128, 64, 32, 16, 8 rows; weights: b[0], 64 x 64
  CUtensorMap a_part[3], b_part[3];  // weights: boxes of 64 columns and 32 and 16 rows, and 16 of the panels
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
  float* slices;  // sums of parts, rows of I
  int64_t slice_rows;  // as many as there are
  int parts;      // rows: parts of every sum, of part_blocks blocks (1: no parts, no slices)
  int part_blocks;
  int part_rows;  // weights: experts with more rows than this have parts of at most as many
  int* next;      // counter of claimed tiles, or null: every step-th
  uint64_t wait_ns;
  int32_t* status;  // the caller's [2], or null
  int stall;      // test hook: CTA 0 withholds its first accumulator
};

// What a wait that ran out was for (numbers of mm_experts.h).
enum Awaited { kFreeStage = 1, kFreeSum, kOperands, kTold, kTaken, kSum };

// Rows that are loaded for n of a chunk: the next power of two from 8 on.
__host__ __device__ constexpr uint32_t box_rows(int n) {
  return n > 128 ? 256 : n > 64 ? 128 : n > 32 ? 64 : n > 16 ? 32 : n > 8 ? 16 : 8;
}

// A tile. 32 bytes, as the queue holds it.
struct __align__(16) Unit {
  int e, i0, j0;   // i0: first column of the (even) CTA; j0: first row of B (rows) or column of B (weights)
  int n;           // columns of the accumulator that are stored; < 0: no more tiles
  int k0, k;       // first term of the sum (weights: a row) and their number
  int row;         // row of the output, or of the slices, of the first column
  int slice;       // whether it goes to the slices
  __device__ __forceinline__ int n16() const { return (n + 15) & ~15; }
  __device__ __forceinline__ int blocks() const { return (k + 63) / 64; }
  // Blocks of a run: all, or (wide results) at most kRun of as many equal runs as it takes.
  __device__ __forceinline__ int run(bool wide) const {
    const int b = blocks(), runs = (b + kRun - 1) / kRun;
    return !wide || runs <= 1 ? b : (b + runs - 1) / runs;
  }
};

// Waits by all lanes of a warp, with one answer for them.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, uint64_t limit_ns) {
  return __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity, limit_ns));
}

// 32 bytes to the other CTA's shared memory, where their arrival completes a phase of the barrier. Without a
// release, which would wait for this thread's accesses to global memory.
__device__ __forceinline__ void send_cluster(uint32_t to, uint32_t bar, int4 lo, int4 hi) {
  asm volatile("mbarrier.arrive.expect_tx.relaxed.cluster.shared::cluster.b64 _, [%0], 32;" ::"r"(bar) : "memory");
  asm volatile(
      "st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(to),
      "r"(lo.x), "r"(lo.y), "r"(lo.z), "r"(lo.w), "r"(bar)
      : "memory");
  asm volatile(
      "st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(
          to + 16),
      "r"(hi.x), "r"(hi.y), "r"(hi.z), "r"(hi.w), "r"(bar)
      : "memory");
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
  uint64_t limit_ns;
  __device__ __forceinline__ Ring(uint32_t bar, uint32_t first, int n, uint64_t limit)
      : bar0(bar), phase(first), stages(n), limit_ns(limit) {}
  __device__ __forceinline__ bool wait() {
    if (__all_sync(0xFFFFFFFFu, ready)) return true;
    return warp_wait(bar0 + 8u * s, phase, limit_ns);
  }
  __device__ __forceinline__ void ask_next() {
    const bool wrap = s + 1 == stages;
    ready = mbar_test_wait(bar0 + 8u * (wrap ? 0 : s + 1), wrap ? phase ^ 1u : phase);
  }
  __device__ __forceinline__ void next() {
    if (++s == stages) s = 0, phase ^= 1u;
  }
};

// Where the experts' rows start (E + 1 numbers), how many chunks of rows the experts before each have,
// and (weights) the experts by falling numbers of rows, in which order the chunks are counted then, in
// shared memory. False if the offsets are no such table.
template <bool WEIGHTS>
__device__ __forceinline__ bool build_table(const Args& a, int* start, int* first, uint16_t* order) {
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
      // (weights: an expert without rows has a tile too, of zeros)
      tiles[p] = WEIGHTS ? max(1, (t - s + a.part_rows - 1) / a.part_rows) : (t - s + a.chunk - 1) / a.chunk;
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
  if constexpr (WEIGHTS) {
    // experts by falling numbers of rows (those with parts as if they had part_rows, so first): the rank
    // of an expert is how many have more, or as many and come first
    __syncthreads();
    for (int e = tid; e < a.E; e += kThreads) {
      const int rows = min(a.part_rows, start[e + 1] - start[e]);
      int rank = 0;
#pragma unroll 4
      for (int o = 0; o < a.E; ++o) {
        const int other = min(a.part_rows, start[o + 1] - start[o]);
        rank += other > rows || (other == rows && o < e);
      }
      order[rank] = (uint16_t)e;
    }
    __syncthreads();
    // first: chunks of the experts before in this order (slices are numbered by it)
    if (tid < 32) {
      int base = 0;
      for (int r0 = 0; r0 < a.E; r0 += 32) {
        const int r = r0 + lane, e = r < a.E ? order[r] : 0;
        const int c = r < a.E ? max(1, (start[e + 1] - start[e] + a.part_rows - 1) / a.part_rows) : 0;
        int upto = c;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int v = __shfl_up_sync(0xFFFFFFFFu, upto, d);
          if (lane >= d) upto += v;
        }
        if (r < a.E) first[r] = base + upto - c;
        base += __shfl_sync(0xFFFFFFFFu, upto, 31);
      }
      if (lane == 0) first[a.E] = base;
    }
  }
  __syncthreads();
  return true;
}

// Tile u of the launch; i_tiles, j_tiles: tiles of an output's columns and (weights) rows.
template <bool WEIGHTS, int PAIR>
__device__ __forceinline__ Unit unit_at(const Args& a, const int* start, const int* first,
                                        const uint16_t* order, int u, int i_tiles, int j_tiles) {
  Unit t{};
  const int per = WEIGHTS ? i_tiles * j_tiles : i_tiles * a.parts;
  const int q = u / per;
  int lo = 0, hi = a.E;  // first[lo] <= q < first[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= q) lo = mid; else hi = mid;
  }
  const int chunks = first[lo + 1] - first[lo];
  t.e = WEIGHTS ? order[lo] : lo;
  const int rows = start[t.e + 1] - start[t.e];
  if constexpr (WEIGHTS) {
    const int in = u - q * per, jt = in / i_tiles, c = q - first[lo];
    t.i0 = (in - jt * i_tiles) * kTile * PAIR;
    t.j0 = jt * a.chunk;
    t.n = min(a.chunk, a.J - t.j0);
    // equal parts of whole blocks
    const int part = chunks == 1 ? rows : ((rows + chunks - 1) / chunks + 63) & ~63;
    t.k0 = start[t.e] + c * part;
    t.k = min(part, rows - c * part);
    t.slice = chunks > 1;
    t.row = (t.slice ? q : t.e) * a.J + t.j0;
  } else {
    const int in = u - first[lo] * per, it = in / (chunks * a.parts);
    const int rest = in - it * chunks * a.parts, c = rest / a.parts, p = rest - c * a.parts;
    t.i0 = it * kTile * PAIR;
    // equal chunks; as none is above a.chunk the last one has a row at least
    const int size = ((rows + chunks - 1) / chunks + 15) & ~15;
    t.j0 = start[t.e] + c * size;
    t.n = min(size, rows - c * size);
    t.k0 = p * a.part_blocks * 64;
    t.k = min(a.part_blocks * 64, a.K - t.k0);
    t.slice = a.parts > 1;
    t.row = p * a.R + t.j0;
  }
  return t;
}

// `words` 16-byte words at p set to v by the launch's storing warps.
__device__ __forceinline__ void fill(void* p, int64_t words, uint32_t v, int thread, int threads) {
  uint4* w = static_cast<uint4*>(p);
  for (int64_t i = thread; i < words; i += threads) w[i] = make_uint4(v, v, v, v);
}

// Up to 32 sums of this lane's column i, to rows row .. of `out`; n: how many there are. The address of a
// row is that of the one before plus the pitch, as 64-bit products per element were most of an epilogue's
// instructions.
template <bool ADD>
__device__ __forceinline__ void store_fp32(const Args& a, float* out, const float (&v)[32], int64_t row, int i,
                                           int n) {
  if (i >= a.I) return;
  float* p = out + row * a.I + i;
  if (!ADD && n >= 32) {
#pragma unroll
    for (int j = 0; j < 32; ++j, p += a.I) *p = v[j];
    return;
  }
#pragma unroll
  for (int j0 = 0; j0 < 32; j0 += 8, p += 8 * (int64_t)a.I) {
    float old[8];
    if constexpr (ADD) {
#pragma unroll
      for (int j = 0; j < 8; ++j) old[j] = j0 + j < n ? p[j * (int64_t)a.I] : 0.f;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j0 + j < n) p[j * (int64_t)a.I] = ADD ? v[j0 + j] + old[j] : v[j0 + j];
  }
}

// The same added to bf16 numbers. Two neighbouring lanes exchange, so that each has a pair of neighbouring
// columns of one row: the even lane of row j, the odd one of row j + 1.
__device__ __forceinline__ void add_bf16(const Args& a, const float (&v)[32], int64_t row, int i, int n, int lane) {
  const int odd = lane & 1;
  uint32_t* p = reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(a.out) + (row + odd) * a.I + (i & ~1));
#pragma unroll
  for (int j = 0; j < 32; j += 2, p += a.I) {
    const float other = __shfl_xor_sync(0xFFFFFFFFu, odd ? v[j] : v[j + 1], 1);
    if (i < a.I && j + odd < n) {
      const uint32_t old = *p;
      *p = pack_bf16((odd ? other : v[j]) + bf16_lo(old), (odd ? v[j + 1] : other) + bf16_hi(old));
    }
  }
}

// 16 lanes x 32 columns of the accumulator: lane l has, of each 8 columns c, elements (l / 4, 2 (l % 4))
// and the one right of it in r[4c], r[4c + 1], and those 8 lanes further down in r[4c + 2], r[4c + 3].
__device__ __forceinline__ void tmem_ld_16x32(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

// 32 lanes x 32 columns of the accumulator as bf16: p[4c + m] is what stmatrix stores as block m of the
// 8 columns c.
__device__ __forceinline__ void load_bf16(uint32_t taddr, uint32_t (&p)[16]) {
  uint32_t lo[16], hi[16];
  tmem_ld_16x32(taddr, lo);
  tmem_ld_16x32(taddr + (16u << 16), hi);
  tmem_ld_wait();
#pragma unroll
  for (int c = 0; c < 4; ++c)
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const uint32_t* r = (m < 2 ? lo : hi) + 4 * c + 2 * (m & 1);
      p[4 * c + m] = pack_bf16(__uint_as_float(r[0]), __uint_as_float(r[1]));
    }
}

// Whether all four warps of a set say so. (Barriers, tensor-memory loads and setmaxnreg in their aligned forms
// want the lanes of a warp together: each stands behind a __syncwarp or a vote.)
__device__ __forceinline__ bool agreed(bool ok, int set) {
  uint32_t all;
  __syncwarp();
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.and.pred q, %2, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(all)
      : "r"((uint32_t)ok), "r"(1 + set)
      : "memory");
  return all != 0;
}

// Those of a set's four warps (the CTA's 128 columns, one of `n` rows row .. at a time) to the output by way
// of shared memory (`stage`, 32 rows of 256 bytes): 8 x 8 blocks are stored transposed, and rows leave in
// words of 16 bytes, 256 bytes of a row at a time; a third of the instructions that an exchange between
// lanes takes, and whole lines (rows of 64 bytes, each warp its own, reached 4.2 TB/s of writes where rows
// of 128 reach 5.7). A row's words are turned by its number, so that eight rows' words of one block lie in
// different banks. i: the CTA's first column.
__device__ __forceinline__ void store_bf16(const Args& a, const uint32_t (&p)[16], uint32_t stage, int set,
                                           int quarter, int64_t row, int i, int n, int lane) {
  const auto sync = [&] {
    __syncwarp();
    asm volatile("bar.sync %0, 128;" ::"r"(1 + set) : "memory");
  };
  sync();  // all have read what was here
  const int jw = lane & 7;
  const uint32_t to = stage + jw * 256 + (((quarter * 4 + (lane >> 3)) ^ jw) << 4);
#pragma unroll
  for (int c = 0; c < 4; ++c)
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(to + c * 2048),
                 "r"(p[4 * c]), "r"(p[4 * c + 1]), "r"(p[4 * c + 2]), "r"(p[4 * c + 3])
                 : "memory");
  sync();
  const int j = quarter * 8 + (lane >> 4), w = lane & 15;  // this warp's 8 rows, two at a time
  __nv_bfloat16* at = static_cast<__nv_bfloat16*>(a.out) + (row + j) * a.I + i + 8 * w;
  const bool there = i + 8 * w < a.I;
#pragma unroll
  for (int c = 0; c < 4; ++c, at += 2 * (int64_t)a.I) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(stage + (j + 2 * c) * 256 + ((w ^ ((j + 2 * c) & 7)) << 4))
                 : "memory");
    if (there && j + 2 * c < n) *reinterpret_cast<uint4*>(at) = v;
  }
}

// WIDE: 32-bit or accumulated results, from runs that are added in registers.
template <int PAIR, bool WEIGHTS, bool WIDE>
__global__ void __launch_bounds__(kThreads, 1)
    k_grouped(const __grid_constant__ Maps m, const Args a) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ uint32_t tmem_holder;
  __shared__ Unit queue[kQueue];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  const uint32_t out_stage = sbase + a.stages * a.stage_bytes;
  const uint32_t bars = out_stage + kStoreWarps * kOutBytes;
  int* const start = reinterpret_cast<int*>(smem_raw + (bars + kBarBytes - raw));
  int* const first_chunk = start + kMaxE + 1;
  uint16_t* const order = reinterpret_cast<uint16_t*>(first_chunk + kMaxE + 1);
  auto full_bar = [&](uint32_t s) { return bars + 8u * s; };
  auto empty_bar = [&](uint32_t s) { return bars + 8u * (kMaxStages + s); };
  auto accf_bar = [&](uint32_t b) { return bars + 8u * (2 * kMaxStages + b); };
  auto acce_bar = [&](uint32_t b) { return bars + 8u * (2 * kMaxStages + 2 + b); };
  auto told_bar = [&](uint32_t s) { return bars + 8u * (2 * kMaxStages + 4 + s); };
  auto taken_bar = [&](uint32_t s) { return bars + 8u * (2 * kMaxStages + 4 + kQueue + s); };
  static_assert(8 * (2 * kMaxStages + 4 + 2 * kQueue) <= kBarBytes, "barrier area");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = PAIR == 2 ? (int)cluster_ctarank() : 0;
  const int step = (int)gridDim.x / PAIR, mine = (int)blockIdx.x / PAIR;
  const uint64_t limit = a.wait_ns;
  if (threadIdx.x == 0) {
    for (int s = 0; s < a.stages; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(accf_bar(b), 1);
      mbar_init(acce_bar(b), PAIR * kStoreWarps);
    }
    for (int q = 0; q < kQueue; ++q) {
      mbar_init(told_bar(q), 1);
      // those who take a tile: the storing and loading warps, the even CTA's multiplying one
      mbar_init(taken_bar(q), PAIR * (kStoreWarps + 1) + 1);
    }
    mbar_fence_init();
    tma_prefetch_desc(&m.a);
    if (WEIGHTS || a.chunk / PAIR > 64) tma_prefetch_desc(&m.b[0]);
  }
  // Tensor memory is asked for, a wait without a limit, when nothing that it needs can be missing any more:
  // the stream's kernels before have ended, so that none of them holds columns on this SM, and both CTAs
  // of a pair, whose warps allocate together, have started.
  pdl_wait();
  if constexpr (PAIR == 2) cluster_sync();
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
  const bool good = build_table<WEIGHTS>(a, start, first_chunk, order);  // (a barrier for the block)
  tc_fence_after();
  if constexpr (PAIR == 2) cluster_sync();
  const uint32_t tmem = *static_cast<volatile uint32_t*>(&tmem_holder);

  const int i_tiles = (a.I + kTile * PAIR - 1) / (kTile * PAIR);
  const int j_tiles = WEIGHTS ? (a.J + a.chunk - 1) / a.chunk : 1;
  const int units = !good ? 0 : first_chunk[a.E] * i_tiles * (WEIGHTS ? j_tiles : a.parts);

  // Records a wait that ran out, if it is the first. By a whole warp.
  auto give_up = [&](Awaited what) {
    if (a.status != nullptr && lane == 0 && atomicCAS(a.status, 0, MM_ERR_TIMEOUT) == 0)
      a.status[1] = what | (int)blockIdx.x << 8;
  };

  // Entry number q of the queue, once it is there; false if the wait ran out. A lane reads a word, so
  // that what frees the slot needs all words to have arrived: the odd CTA's arrival is then one without
  // a release, which would wait for a storing warp's rows to reach memory.
  auto take = [&](int q, Unit& t) {
    const uint32_t slot = q % kQueue, bar = told_bar(slot), phase = q / kQueue & 1u;
    if (!warp_wait(bar, phase, limit)) {
      give_up(kTold);
      return false;
    }
    const int word = static_cast<volatile const int*>(&queue[slot].e)[lane & 7];
    t.e = __shfl_sync(0xFFFFFFFFu, word, 0);
    t.i0 = __shfl_sync(0xFFFFFFFFu, word, 1);
    t.j0 = __shfl_sync(0xFFFFFFFFu, word, 2);
    t.n = __shfl_sync(0xFFFFFFFFu, word, 3);
    t.k0 = __shfl_sync(0xFFFFFFFFu, word, 4);
    t.k = __shfl_sync(0xFFFFFFFFu, word, 5);
    t.row = __shfl_sync(0xFFFFFFFFu, word, 6);
    t.slice = __shfl_sync(0xFFFFFFFFu, word, 7);
    if (lane == 0) {
      if (PAIR == 2 && rank == 1) mbar_arrive_remote_relaxed(mapa_shared(taken_bar(slot), 0));
      else mbar_arrive(taken_bar(slot));
    }
    return true;
  };

  __syncwarp();
  if (warp < kFirstStore) {
    if constexpr (WIDE) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kFewRegs));
    if (warp == 0) {
      // ------------------------------------------------ loads
      Ring ring(empty_bar(0), 1, a.stages, limit);
      int it = 0;
      bool ok = true;
      const bool kmajor = a.a_kmajor != 0;
      for (int q = 0; ok; ++q) {
        Unit t;
        if (!take(q, t) || t.n < 0) break;
        const int half = uniform(t.n16() / PAIR), blocks = uniform(t.blocks());
        const int e = uniform(t.e), i0 = uniform(t.i0) + rank * kTile, first_k = uniform(t.k0);
        const int j0 = uniform(t.j0) + rank * half;
        const int last = WEIGHTS ? uniform(t.k) - (blocks - 1) * 64 : 64;  // rows of the last block
        for (int kb = 0; kb < blocks; ++kb, ++it) {
          if (!ring.wait()) {
            give_up(kFreeStage);
            ok = false;
            break;
          }
          ring.ask_next();
          if (elect_one()) {
            const uint32_t sa = sbase + ring.s * a.stage_bytes, sb = sa + kABytes;
            const int k0 = first_k + kb * 64;
            const bool part = WEIGHTS && kb == blocks - 1 && last < 64;
            const uint32_t bytes = WEIGHTS ? (2 + (half + 63) / 64) * (part ? (last + 15) & ~15 : 64) * 128u
                                           : kABytes + box_rows(half) * 128u;
            // the two CTAs' bytes of a stage count on the even one's barrier
            uint32_t bar = full_bar(ring.s);
            if (rank == 0) mbar_arrive_expect_tx(bar, PAIR * bytes);
            if constexpr (PAIR == 2) bar = mapa_shared(bar, 0);
            auto load2 = [&](uint32_t dst, const CUtensorMap* map, int c0, int c1) {
              if constexpr (PAIR == 2) tma_load_2d_pair(dst, map, bar, c0, c1);
              else tma_load_2d(dst, map, bar, c0, c1);
            };
            auto load3 = [&](uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2) {
              if constexpr (PAIR == 2) tma_load_3d_pair(dst, map, bar, c0, c1, c2);
              else tma_load_3d(dst, map, bar, c0, c1, c2);
            };
            if constexpr (WEIGHTS) {
              // k-rows r .. of the stage from rows `from` of the operands
              auto boxes = [&](const CUtensorMap* ma, const CUtensorMap* mb, int r, int from) {
                load2(sa + r * 128, ma, i0, from);
                load2(sa + kBlock + r * 128, ma, i0 + 64, from);
#pragma unroll
                for (int c = 0; c < kMaxN / PAIR; c += 64)
                  if (c < half) load2(sb + c / 64 * kBlock + r * 128, mb, j0 + c, from);
              };
              if (!part) {
                boxes(&m.a, &m.b[0], 0, k0);
              } else {
                if (last & 32) boxes(&m.a_part[0], &m.b_part[0], 0, k0);
                if (last & 16) boxes(&m.a_part[1], &m.b_part[1], last & 32, k0 + (last & 32));
                if (last & 15) boxes(&m.a_part[2], &m.b_part[2], last & 48, e * 16);
              }
            } else {
              if (kmajor) {
                load3(sa, &m.a, k0, i0, e);
              } else {
                load3(sa, &m.a, i0, k0, e);
                load3(sa + kBlock, &m.a, i0 + 64, k0, e);
              }
              // one box (256: two), not exactly the rows there are in boxes as the bits of their number
              // (experts of 1000 rows, 2048 -> 1536: 1455 TFLOP/s, 1545 this way)
              load2(sb, half > 64 ? &m.b[0] : half > 32 ? &m.b[1] : half > 16 ? &m.b[2] : half > 8 ? &m.b[3] : &m.b[4],
                    k0, j0);
              if (PAIR == 1 && half > 128) load2(sb + 128 * 128, &m.b[0], k0, j0 + 128);
            }
          }
          __syncwarp();
          ring.next();
        }
      }
      // every stage's last release has landed before this CTA may leave
      for (int s = 0; s < a.stages && s < it && ok; ++s) {
        ok = warp_wait(empty_bar(s), (it - 1 - s) / a.stages & 1u, limit);
        if (!ok) give_up(kFreeStage);
      }
    } else if (warp == 1) {
      // ------------------------------------------------ multiplies
      // The warp stays in step and an elected lane of the even CTA issues, from uniform registers (by one
      // lane's branch with operands of its own an issue took 300 cycles: 131072 rows of 128 experts, 2048
      // -> 1536, 1015 us, 528 this way).
      Ring ring(full_bar(0), 0, a.stages, limit);
      const int a_mn = WEIGHTS || !a.a_kmajor, b_mn = WEIGHTS;
      const uint64_t adesc = sdesc_sw128(sbase, a_mn ? kBlock : 16, 1024);
      const uint64_t bdesc = sdesc_sw128(sbase + kABytes, b_mn ? kBlock : 16, 1024);
      const uint32_t a_step = a_mn ? 2048 / 16 : 2, b_step = b_mn ? 2048 / 16 : 2;
      uint32_t acc = 0;
      bool ok = rank == 0;
      for (int q = 0; ok; ++q) {
        Unit t;
        if (!take(q, t) || t.n < 0) break;
        const int blocks = uniform(t.blocks()), n16 = uniform(t.n16());
        const int run = uniform(t.run(WIDE));
        const int last = uniform(t.k) - (blocks - 1) * 64;  // terms in the last block
        const uint32_t idesc = idesc_bf16_f32(kTile * PAIR, n16, a_mn, b_mn);
        uint32_t buf = 0, d = 0;
        for (int kb = 0, left = 0; kb < blocks; ++kb) {
          const bool opens = left == 0;  // a run, in the other accumulator
          if (opens) {
            left = min(run, blocks - kb);
            buf = acc & 1u;
            d = tmem + buf * kMaxN;
            if (!warp_wait(acce_bar(buf), (acc >> 1 & 1u) ^ 1u, limit)) {
              give_up(kFreeSum);
              ok = false;
              break;
            }
            tc_fence_after();
          }
          if (!ring.wait()) {
            give_up(kOperands);
            ok = false;
            break;
          }
          const uint32_t s = ring.s;
          ring.ask_next();
          const int steps = WEIGHTS && kb == blocks - 1 ? (last + 15) / 16 : 4;
          tc_fence_after();
          if (elect_one()) {
            const uint64_t ad = adesc + s * (a.stage_bytes / 16), bd = bdesc + s * (a.stage_bytes / 16);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
              if (WEIGHTS && kk >= steps) continue;
              if constexpr (PAIR == 2) umma_bf16_pair(d, ad + kk * a_step, bd + kk * b_step, idesc, !opens || kk != 0);
              else umma_bf16(d, ad + kk * a_step, bd + kk * b_step, idesc, !opens || kk != 0);
            }
            if constexpr (PAIR == 2) umma_commit_pair_mc(empty_bar(s), 0x3);
            else umma_commit(empty_bar(s));
            if (left == 1 && !(a.stall && blockIdx.x == 0 && acc == 0)) {
              if constexpr (PAIR == 2) umma_commit_pair_mc(accf_bar(buf), 0x3);
              else umma_commit(accf_bar(buf));
            }
          }
          __syncwarp();
          ring.next();
          if (--left == 0) ++acc;
        }
      }
    } else if (warp == 2) {
      // ------------------------------------------------ deals out tiles
      // A claim is made three tiles ahead, so that its answer is there when it is looked at. (Two ahead a
      // tile took 1.1 us at least, and with a release to the other CTA 2.7: 512 rows of 128 experts,
      // 768 x 2048, 110 us in pairs, 88 now.)
      int u = mine, ahead = mine + step, claimed = mine + 2 * step;
      for (int q = 0; rank == 0; ++q) {
        int next = claimed + step;
        if (a.next != nullptr && lane == 0) next = 3 * step + atomicAdd(a.next, 1);
        Unit t{};
        if (u < units) t = unit_at<WEIGHTS, PAIR>(a, start, first_chunk, order, u, i_tiles, j_tiles);
        else t.n = -1;
        const uint32_t slot = q % kQueue;
        if (!warp_wait(taken_bar(slot), (q / kQueue & 1u) ^ 1u, limit)) {
          give_up(kTaken);
          break;
        }
        if (lane == 0) {
          queue[slot] = t;
          mbar_arrive(told_bar(slot));
          if constexpr (PAIR == 2)
            send_cluster(mapa_shared(smem_u32(&queue[slot]), 1), mapa_shared(told_bar(slot), 1),
                         make_int4(t.e, t.i0, t.j0, t.n), make_int4(t.k0, t.k, t.row, t.slice));
        }
        __syncwarp();
        if (t.n < 0) break;
        u = ahead;
        ahead = __shfl_sync(0xFFFFFFFFu, claimed, 0);
        claimed = next;
      }
    }
  } else {
    if constexpr (WIDE) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kManyRegs));
    // ------------------------------------------------ stores
    const int set = (warp - kFirstStore) >> 2, quarter = warp & 3;  // (of the accumulator's lanes)
    const bool to_slices = !WEIGHTS && a.parts > 1;
    const int64_t row_words = a.I * (a.f32 ? 4 : 2) / 16;
    const int64_t all_words = (WEIGHTS ? (int64_t)a.E * a.J : a.R) * row_words;
    const uint32_t nan = a.f32 ? 0x7FC00000u : 0x7FC07FC0u;
    uint4* const out = static_cast<uint4*>(a.out);
    const int thread = (int)blockIdx.x * (32 * kStoreWarps) + (int)threadIdx.x - 32 * kFirstStore;
    const int threads = (int)gridDim.x * (32 * kStoreWarps);
    if (to_slices) {
      // (the launch behind writes the output)
    } else if (!good) {
      fill(out, all_words, nan, thread, threads);
    } else if (!WEIGHTS) {
      fill(out, start[0] * row_words, 0, thread, threads);
      fill(out + start[a.E] * row_words, (a.R - start[a.E]) * row_words, 0, thread, threads);
    }
    const uint32_t stage = out_stage + set * 4 * kOutBytes;
    const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16);
    uint32_t acc = 0;
    // The accumulator of the next run, or false; and its hand-back, when it is in registers.
    auto arrived = [&]() {
      const bool ok = warp_wait(accf_bar(acc & 1u), acc >> 1 & 1u, limit);
      if (!ok) give_up(kSum);
      tc_fence_after();
      return ok;
    };
    auto release = [&]() {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (PAIR == 2 && rank != 0) mbar_arrive_remote_relaxed(mapa_shared(acce_bar(acc & 1u), 0));
        else mbar_arrive(acce_bar(acc & 1u));
      }
      ++acc;
    };
    for (int q = 0;; ++q) {
      Unit t{};
      bool ok = take(q, t);
      if (!WIDE) ok = agreed(ok, set);
      if (ok && t.n < 0) break;
      if (ok && t.k == 0 && a.accumulate) continue;  // adding zero changes nothing
      const int i = t.i0 + rank * kTile + quarter * 32;
      const int blocks = t.blocks();
      if constexpr (WIDE) {
        float sum[kMaxN / 64][32];
#pragma unroll
        for (int g = 0; g < kMaxN / 64; ++g)
#pragma unroll
          for (int j = 0; j < 32; ++j) sum[g][j] = 0.f;
        const int run = t.run(true);
        for (int kb = 0; kb < blocks && ok; kb += run) {
          ok = arrived();
          if (!ok) break;
#pragma unroll
          for (int g = 0; g < kMaxN / 64; ++g) {
            const int c = set * 32 + 64 * g;
            if (c >= t.n) continue;
#pragma unroll
            for (int h = 0; h < 32; h += 16) {
              uint32_t r[16];
              tmem_ld_32x16(lanes + (acc & 1u) * kMaxN + c + h, r);
              tmem_ld_wait();
#pragma unroll
              for (int j = 0; j < 16; ++j) sum[g][h + j] += __uint_as_float(r[j]);
            }
          }
          release();
        }
        if (ok) {
          float* const to = t.slice ? a.slices : static_cast<float*>(a.out);
          const bool add = a.accumulate && !t.slice;
#pragma unroll
          for (int g = 0; g < kMaxN / 64; ++g) {
            const int c = set * 32 + 64 * g;
            if (c >= t.n) continue;
            if (!add) store_fp32<false>(a, to, sum[g], (int64_t)t.row + c, i + lane, t.n - c);
            else if (a.f32) store_fp32<true>(a, to, sum[g], (int64_t)t.row + c, i + lane, t.n - c);
            else add_bf16(a, sum[g], (int64_t)t.row + c, i + lane, t.n - c, lane);
          }
        }
      } else {
        if (ok && blocks > 0) ok = arrived();
        ok = agreed(ok, set);  // (the warps of a set meet at barriers)
        if (ok) {
          for (int c = set * 32; c < t.n; c += 64) {
            __syncwarp();
            if (t.slice) {
              uint32_t r[32];
              tmem_ld_32x32(lanes + (acc & 1u) * kMaxN + c, r);
              tmem_ld_wait();
              float v[32];
#pragma unroll
              for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(r[j]);
              store_fp32<false>(a, a.slices, v, (int64_t)t.row + c, i + lane, t.n - c);
            } else {
              uint32_t p[16] = {};
              if (blocks > 0) load_bf16(lanes + (acc & 1u) * kMaxN + c, p);
              store_bf16(a, p, stage, set, quarter, (int64_t)t.row + c, t.i0 + rank * kTile, t.n - c, lane);
            }
          }
          if (blocks > 0) release();
        }
      }
      if (!ok) {  // the tiles that this CTA has or would have had are nobody's: NaN, if not others' results
        fill(out, all_words, nan, (int)threadIdx.x - 32 * kFirstStore, 32 * kStoreWarps);
        if (a.slices != nullptr)
          fill(a.slices, a.slice_rows * a.I / 4, 0x7FC00000u, (int)threadIdx.x - 32 * kFirstStore,
               32 * kStoreWarps);
        break;
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

struct TailArgs {
  const int32_t* offsets;
  const uint4* from[2];  // the operands, rows of `words` words of 8 elements
  uint4* panel[2];       // [E][16] rows
  int words[2];
  int R;
  int* next;
};

// Block (e, y): the panels of expert e, part y of gridDim.y. And the counter of claimed tiles.
__global__ void __launch_bounds__(256) k_tails(TailArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *a.next = 0;
  const int e = blockIdx.x, s = a.offsets[e], t = a.offsets[e + 1];
  if (s < 0 || t < s || t > a.R) return;  // (no table: the products' launch says so)
  const int n = (t - s) & 15;
  if (n == 0) return;
#pragma unroll
  for (int o = 0; o < 2; ++o) {
    const int words = a.words[o];
    const uint4* from = a.from[o] + (int64_t)(t - n) * words;
    uint4* to = a.panel[o] + (int64_t)e * 16 * words;
    for (int i = blockIdx.y * 256 + threadIdx.x; i < 16 * words; i += gridDim.y * 256)
      to[i] = i < n * words ? from[i] : make_uint4(0, 0, 0, 0);
  }
}

struct JoinArgs {
  const int32_t* offsets;
  const float* slices;
  void* out;
  int R, E, I, J;
  int parts;      // rows
  int part_rows;  // weights
  int f32, accumulate;
};

// Four sums of parts `first`, first + stride, ... in their order, to elements 4 w .. of the output.
__device__ __forceinline__ void join_words(const JoinArgs& a, const float4* slice, int parts, int64_t stride,
                                           int64_t w) {
  float4 s = slice[0];
#pragma unroll 4
  for (int p = 1; p < parts; ++p) {
    const float4 v = slice[p * stride];
    s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
  }
  if (a.f32) {
    float4* at = static_cast<float4*>(a.out) + w;
    if (a.accumulate) {
      const float4 v = *at;
      s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
    }
    *at = s;
  } else {
    uint2* at = static_cast<uint2*>(a.out) + w;
    if (a.accumulate) {
      const uint2 v = *at;
      s.x += bf16_lo(v.x), s.y += bf16_hi(v.x), s.z += bf16_lo(v.y), s.w += bf16_hi(v.y);
    }
    *at = make_uint2(pack_bf16(s.x, s.y), pack_bf16(s.z, s.w));
  }
}

// Rows: the sums of the parts; zeros in no expert's rows, NaN for offsets that are no table.
__global__ void __launch_bounds__(256) k_join_rows(JoinArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  int bad = 0;
  for (int e = threadIdx.x; e < a.E; e += 256) {
    const int s = a.offsets[e], t = a.offsets[e + 1];
    bad |= s < 0 || t < s || t > a.R;
  }
  bad = __syncthreads_or(bad);
  const int words = a.I / 4;
  const int64_t all = (int64_t)a.R * words;
  const int begin = a.offsets[0], end = a.offsets[a.E];
  for (int64_t w = blockIdx.x * 256 + threadIdx.x; w < all; w += (int64_t)gridDim.x * 256) {
    const int64_t r = w / words;
    if (bad || r < begin || r >= end) {
      const uint32_t v = !bad ? 0u : a.f32 ? 0x7FC00000u : 0x7FC07FC0u;
      if (a.f32) static_cast<uint4*>(a.out)[w] = make_uint4(v, v, v, v);
      else static_cast<uint2*>(a.out)[w] = make_uint2(v, v);
    } else {
      join_words(a, reinterpret_cast<const float4*>(a.slices) + w, a.parts, all, w);
    }
  }
}

// Weights: the sums of the parts of the experts that have some.
__global__ void __launch_bounds__(256) k_join_weights(JoinArgs a) {
  constexpr int PER = kMaxE / 256;
  __shared__ int sums[8];
  __shared__ int expert[kMaxE], first[kMaxE];  // those with parts, and their first slices
  __shared__ int count;
  pdl_wait();
  pdl_launch_dependents();
  // Slices are numbered as in build_table: by the experts with part_rows rows or more, in their order.
  // (Offsets that are no table have left NaN in the output, and no parts.)
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int chunks[PER], mine = 0, bad = 0;
#pragma unroll
  for (int p = 0; p < PER; ++p) {
    const int e = tid * PER + p;
    chunks[p] = 0;
    if (e < a.E) {
      const int s = a.offsets[e], t = a.offsets[e + 1];
      bad |= s < 0 || t < s || t > a.R;
      if (t - s >= a.part_rows) chunks[p] = (t - s + a.part_rows - 1) / a.part_rows;
    }
    mine += chunks[p];
  }
  if (tid == 0) count = 0;
  if (__syncthreads_or(bad)) return;
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
    if (chunks[p] > 1) {
      const int at = atomicAdd(&count, 1);  // (in any order)
      expert[at] = tid * PER + p | chunks[p] << 10;
      first[at] = base;
    }
    base += chunks[p];
  }
  __syncthreads();
  const int64_t words = (int64_t)a.J * a.I / 4;
  for (int x = 0; x < count; ++x) {
    const int e = expert[x] & 1023, parts = expert[x] >> 10;
    const float4* slices = reinterpret_cast<const float4*>(a.slices) + first[x] * words;
    for (int64_t w = (int64_t)blockIdx.x * 256 + tid; w < words; w += (int64_t)gridDim.x * 256)
      join_words(a, slices + w, parts, words, e * words + w);
  }
}

// ------------------------------------------------------------------------------------ host side

inline bool aligned_to(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

mm_status check_desc(const mm_grouped_desc* d) {
  if (d == nullptr || d->R < 0 || d->K < 1 || d->N < 1 || d->E < 1) return MM_ERR_INVALID_ARG;
  if (d->out_type != MM_BF16 && d->out_type != MM_FP32) return MM_ERR_INVALID_ARG;
  const uint32_t forms = d->flags & ~MM_GROUPED_TEST_STALL;
  if (forms > 2) return MM_ERR_INVALID_ARG;  // unknown flags, or both forms
  if (d->K % 8 || d->N % 8 || d->K > 65536 || d->N > 65536 || d->E > kMaxE ||
      d->R >= (int64_t)1 << 30)
    return MM_ERR_UNSUPPORTED;
  return MM_OK;
}

inline int64_t div_up(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Parts of the sums of mm_grouped_mm: as many as bring a launch of few tiles to a tile of one CTA per SM,
// of 4 blocks at least. (1 row by a matrix 7168 x 2048, 16 tiles of 112 blocks: 11 us, 31 whole, 0.25 us a
// block. Sums below 32 blocks do not gain the 3 us that the joining launch takes, and 5 of the host.)
struct RowParts {
  int parts, blocks;  // blocks of a part
};
RowParts row_parts(const mm_grouped_desc& d) {
  const int64_t blocks = div_up(d.K, 64);
  const int64_t tiles = (d.R / kMaxN + std::min<int64_t>(d.E, d.R)) * div_up(d.N, kTile);  // at most
  const int64_t want = std::min<int64_t>(device_sm_count() / std::max<int64_t>(1, tiles), blocks / 4);
  if (want < 2 || blocks < 32) return {1, (int)blocks};
  const int64_t part = div_up(blocks, want);
  return {(int)div_up(blocks, part), (int)part};
}

// Rows of an expert from which on its weight gradient has parts: half of what each pair of SMs gets on
// average, so that no expert's tiles outlast the others' by more; and the slices of the experts above it,
// at most (each has fewer than twice its rows / part_rows).
struct WeightParts {
  int64_t rows, slices;
};
WeightParts weight_parts(const mm_grouped_desc& d) {
  const int64_t I = d.transposed ? d.K : d.N, J = d.transposed ? d.N : d.K;
  const int64_t tiles = div_up(I, 2 * kTile) * div_up(J, kMaxN);
  const int64_t rows = std::max<int64_t>(512, div_up(div_up(d.R * tiles, std::max(2, device_sm_count())), 64) * 64);
  if (d.R <= rows) return {d.R + 1, 0};
  return {rows, 2 * d.R / rows};
}

// Workspace of weight gradients: the counter, the panels of both operands, the slices.
constexpr size_t kHeaderBytes = 256;
size_t panel_bytes(int64_t E, int64_t cols) { return ((size_t)E * 16 * cols * 2 + 255) / 256 * 256; }

bool map2(CUtensorMap* m, const void* base, int64_t cols, int64_t rows, uint32_t box_rows) {
  const uint64_t dims[2] = {(uint64_t)cols, (uint64_t)rows};
  const uint64_t strides[1] = {(uint64_t)cols * 2};
  const uint32_t box[2] = {64, box_rows};
  return make_map(m, base, 2, dims, strides, box);
}

// units: tiles, at most.
template <int PAIR, bool WEIGHTS, bool WIDE>
cudaError_t launch_form(const Maps& m, Args a, int64_t units, uint32_t flags, cudaStream_t st) {
  a.stall = (flags & MM_GROUPED_TEST_STALL) != 0;
  a.wait_ns = a.stall ? kTestWaitNs : kWaitNs;
  a.stage_bytes = kABytes + (WEIGHTS ? (a.chunk / PAIR + 63) / 64 * kBlock : box_rows(a.chunk / PAIR) * 128u);
  const uint32_t fixed = 1024 + kStoreWarps * kOutBytes + kBarBytes + kTableBytes;
  a.stages = (int)std::min<uint32_t>(kMaxStages, (kMostSmem - 1024 - fixed) / a.stage_bytes);
  const size_t smem = fixed + (size_t)a.stages * a.stage_bytes;
  static std::atomic<uint64_t> ready{0};
  static std::atomic<int> most_clusters[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!(ready.load(std::memory_order_relaxed) >> dev & 1)) {
    e = cudaFuncSetAttribute(k_grouped<PAIR, WEIGHTS, WIDE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)(kMostSmem - 1024));
    if (e != cudaSuccess) return e;
    if constexpr (WIDE) {
      cudaFuncAttributes built;
      e = cudaFuncGetAttributes(&built, k_grouped<PAIR, WEIGHTS, WIDE>);
      if (e != cudaSuccess) return e;
      if (built.numRegs < kLaunchRegs) return cudaErrorLaunchOutOfResources;
    }
    ready.fetch_or(1ull << dev, std::memory_order_relaxed);
  }
  int fit = std::max(1, device_sm_count());
  if constexpr (PAIR == 1) {
    return launch_pdl(k_grouped<PAIR, WEIGHTS, WIDE>, dim3((unsigned)std::max<int64_t>(1, std::min<int64_t>(fit, units))),
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
      e = cudaOccupancyMaxActiveClusters(&fit, k_grouped<PAIR, WEIGHTS, WIDE>, &cfg);
      if (e != cudaSuccess) return e;
      if (fit < 1) return cudaErrorInvalidConfiguration;
      most_clusters[dev].store(fit, std::memory_order_relaxed);
      cfg.dynamicSmemBytes = smem;
    }
    cfg.gridDim = dim3((unsigned)(2 * std::max<int64_t>(1, std::min<int64_t>(fit, units))));
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, k_grouped<PAIR, WEIGHTS, WIDE>, m, a);
  }
}

template <bool WEIGHTS>
cudaError_t launch(int pair, const Maps& m, const Args& a, int64_t units, uint32_t flags, cudaStream_t st) {
  const bool wide = a.f32 || a.accumulate;
  if (pair == 2)
    return wide ? launch_form<2, WEIGHTS, true>(m, a, units, flags, st)
                : launch_form<2, WEIGHTS, false>(m, a, units, flags, st);
  return wide ? launch_form<1, WEIGHTS, true>(m, a, units, flags, st)
              : launch_form<1, WEIGHTS, false>(m, a, units, flags, st);
}

}  // namespace
}  // namespace mm

using namespace mm;

extern "C" {

int mm_experts_version(void) { return 1; }

size_t mm_grouped_mm_workspace_size(const mm_grouped_desc* d) {
  if (check_desc(d) != MM_OK) return 0;
  const RowParts p = row_parts(*d);  // (256 says that there are no slices)
  return p.parts == 1 ? 256 : std::max<size_t>(512, (size_t)p.parts * d->R * d->N * 4);
}

size_t mm_grouped_weight_grad_workspace_size(const mm_grouped_desc* d) {
  if (check_desc(d) != MM_OK) return 0;
  return kHeaderBytes + panel_bytes(d->E, d->K) + panel_bytes(d->E, d->N) +
         (size_t)weight_parts(*d).slices * d->K * d->N * 4;
}

mm_status mm_grouped_mm(const mm_grouped_desc* d, const void* rows, const void* weight,
                        const int32_t* offsets, void* out, void* workspace, size_t workspace_bytes,
                        void* stream) {
  return mm_grouped_mm_ex(d, rows, weight, offsets, out, workspace, workspace_bytes, nullptr, stream);
}

mm_status mm_grouped_mm_ex(const mm_grouped_desc* d, const void* rows, const void* weight,
                           const int32_t* offsets, void* out, void* workspace, size_t workspace_bytes,
                           int32_t* status, void* stream) {
  mm_status s = check_desc(d);
  if (s != MM_OK) return s;
  if (!aligned_to(rows, 16) || !aligned_to(weight, 16) || !aligned_to(out, 16) || !aligned_to(offsets, 4) ||
      !aligned_to(status, 4))
    return MM_ERR_INVALID_ARG;
  if (d->R == 0) return MM_OK;
  if (!rows || !weight || !out || !offsets) return MM_ERR_INVALID_ARG;
  const RowParts parts = row_parts(*d);
  if (parts.parts > 1 && (workspace == nullptr || !aligned_to(workspace, 256) ||
                          workspace_bytes < mm_grouped_mm_workspace_size(d)))
    return MM_ERR_WORKSPACE;
  clear_error();
  MM_TRY(bind_context());
  // Pairs read half as much of their operands per product. Where a launch has no more tiles of one CTA
  // than SMs, these spread the matrices' columns over twice as many, and up to 128 columns leave a pair's
  // second CTA nothing. (us a call, one CTA a tile and pairs: 8 rows of 8 of 128 experts, 2048 -> 1536, 13.1
  // and 14.1; 512 rows of 128, 768 -> 2048, 71.1 and 66.5; 131072 rows of 128, 2048 -> 1536, 590 and 543;
  // 27494 rows of 8, 2016 -> 128, 26.8 and 31.1, -> 264, 47.7 and 38.5.)
  const int64_t chunks = d->R / kMaxN + std::min<int64_t>(d->E, d->R);  // at most
  const bool few = d->N <= kTile || chunks * div_up(d->N, kTile) <= device_sm_count();
  const int pair = d->flags & MM_GROUPED_CTA_PAIRS || (!(d->flags & MM_GROUPED_SINGLE_CTA) && !few) ? 2 : 1;
  Maps m{};
  Args a{};
  a.offsets = offsets;
  a.status = status;
  a.out = out;
  a.R = (int)d->R;
  a.E = d->E;
  a.I = (int)d->N;
  a.K = (int)d->K;
  a.a_kmajor = d->transposed != 0;
  a.f32 = d->out_type == MM_FP32;
  a.chunk = (int)std::min<int64_t>(kMaxN, (d->R + 15) / 16 * 16);
  a.parts = parts.parts;
  a.part_blocks = parts.blocks;
  if (a.parts > 1) {
    a.slices = static_cast<float*>(workspace);
    a.slice_rows = a.parts * a.R;
  }
  const int64_t inner = d->transposed ? d->K : d->N, outer = d->transposed ? d->N : d->K;
  const uint64_t dims[3] = {(uint64_t)inner, (uint64_t)outer, (uint64_t)d->E};
  const uint64_t strides[2] = {(uint64_t)inner * 2, (uint64_t)inner * outer * 2};
  const uint32_t box[3] = {64, d->transposed ? 128u : 64u, 1};
  bool ok = make_map(&m.a, weight, 3, dims, strides, box);
  for (int p = 0; p < 5; ++p)  // (larger boxes than a chunk's are not used)
    if (128u >> p <= box_rows(a.chunk / pair)) ok = ok && map2(&m.b[p], rows, d->K, d->R, 128u >> p);
  if (!ok) return cuda_fail(cudaErrorInvalidValue, "grouped product tensor maps");
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const int64_t units = chunks * div_up(d->N, kTile * pair) * a.parts;
  MM_TRY(launch<false>(pair, m, a, units, d->flags, st));
  if (a.parts > 1) {
    const JoinArgs j{offsets, a.slices, out, a.R, a.E, a.I, 0, a.parts, 0, a.f32, 0};
    const int64_t blocks = div_up((int64_t)a.R * a.I / 4, 256);
    MM_TRY(launch_pdl(k_join_rows, dim3((unsigned)std::min<int64_t>(blocks, 1024)), dim3(256), 0, st, j));
  }
  return MM_OK;
}

mm_status mm_grouped_mm_weight_grad(const mm_grouped_desc* d, const void* rows, const void* d_out,
                                    const int32_t* offsets, void* d_weight, int accumulate,
                                    void* workspace, size_t workspace_bytes, void* stream) {
  return mm_grouped_mm_weight_grad_ex(d, rows, d_out, offsets, d_weight, accumulate, workspace, workspace_bytes,
                                      nullptr, stream);
}

mm_status mm_grouped_mm_weight_grad_ex(const mm_grouped_desc* d, const void* rows, const void* d_out,
                                       const int32_t* offsets, void* d_weight, int accumulate,
                                       void* workspace, size_t workspace_bytes, int32_t* status,
                                       void* stream) {
  mm_status s = check_desc(d);
  if (s != MM_OK) return s;
  if (!aligned_to(rows, 16) || !aligned_to(d_out, 16) || !aligned_to(d_weight, 16) || !aligned_to(offsets, 4) ||
      !aligned_to(status, 4))
    return MM_ERR_INVALID_ARG;
  if (!d_weight || !offsets || (d->R > 0 && (!rows || !d_out))) return MM_ERR_INVALID_ARG;
  if (workspace == nullptr || !aligned_to(workspace, 256) ||
      workspace_bytes < mm_grouped_weight_grad_workspace_size(d))
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
  const WeightParts parts = weight_parts(*d);
  Maps m;
  Args a{};
  a.offsets = offsets;
  a.status = status;
  a.out = d_weight;
  a.R = (int)d->R;
  a.E = d->E;
  a.I = (int)(d->transposed ? d->K : d->N);
  a.J = (int)(d->transposed ? d->N : d->K);
  a.f32 = d->out_type == MM_FP32;
  a.accumulate = accumulate != 0;
  a.chunk = std::min(kMaxN, (a.J + 15) / 16 * 16);
  a.parts = 1;
  a.part_rows = (int)parts.rows;
  const void *by_i = d->transposed ? rows : d_out, *by_j = d->transposed ? d_out : rows;
  char* const ws = static_cast<char*>(workspace);
  char *const panel_i = ws + kHeaderBytes, *const panel_j = panel_i + panel_bytes(d->E, a.I);
  if (parts.slices > 0) {
    a.slices = reinterpret_cast<float*>(panel_j + panel_bytes(d->E, a.J));
    a.slice_rows = parts.slices * a.J;
  }
  bool ok = map2(&m.a, by_i, a.I, d->R, 64) && map2(&m.b[0], by_j, a.J, d->R, 64);
  for (int p = 0; p < 2; ++p)
    ok = ok && map2(&m.a_part[p], by_i, a.I, d->R, 32u >> p) && map2(&m.b_part[p], by_j, a.J, d->R, 32u >> p);
  ok = ok && map2(&m.a_part[2], panel_i, a.I, 16 * (int64_t)d->E, 16) &&
       map2(&m.b_part[2], panel_j, a.J, 16 * (int64_t)d->E, 16);
  if (!ok) return cuda_fail(cudaErrorInvalidValue, "grouped product tensor maps");
  TailArgs ta{offsets,
              {static_cast<const uint4*>(by_i), static_cast<const uint4*>(by_j)},
              {reinterpret_cast<uint4*>(panel_i), reinterpret_cast<uint4*>(panel_j)},
              {a.I / 8, a.J / 8},
              a.R,
              reinterpret_cast<int*>(ws)};
  a.next = ta.next;
  const int words = 16 * std::max(ta.words[0], ta.words[1]);  // (a few to a thread)
  MM_TRY(launch_pdl(k_tails, dim3((unsigned)d->E, (unsigned)((words + 2047) / 2048)), dim3(256), 0, st, ta));
  const int64_t units = (d->E + parts.slices) * div_up(a.I, kTile * pair) * div_up(a.J, a.chunk);
  MM_TRY(launch<true>(pair, m, a, units, d->flags, st));
  if (parts.slices > 0) {
    const JoinArgs j{offsets, a.slices, d_weight, a.R, a.E, a.I, a.J, 0, a.part_rows, a.f32, a.accumulate};
    const int64_t blocks = std::min<int64_t>(div_up((int64_t)a.I * a.J / 4, 256), 8 * device_sm_count());
    MM_TRY(launch_pdl(k_join_weights, dim3((unsigned)std::max<int64_t>(1, blocks)), dim3(256), 0, st, j));
  }
  return MM_OK;
}

}  // extern "C"
