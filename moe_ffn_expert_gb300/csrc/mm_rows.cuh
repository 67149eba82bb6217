// Device helpers of the row-wise operators (residual_norm, router): typed loads and stores of
// W consecutive elements as 32-bit floats, and sums over a block.
#pragma once

#include "mm_device.cuh"

namespace mm {

// W consecutive elements at p as floats. W = 8: p is 16-byte aligned.
template <int W>
__device__ __forceinline__ void load_vec(const __nv_bfloat16* p, float (&v)[W]) {
  if constexpr (W == 8) {
    const uint4 r = *reinterpret_cast<const uint4*>(p);
    const uint32_t u[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = bf16_lo(u[i]);
      v[2 * i + 1] = bf16_hi(u[i]);
    }
  } else {
    static_assert(W == 1, "widths 8 and 1");
    v[0] = __bfloat162float(p[0]);
  }
}

template <int W>
__device__ __forceinline__ void load_vec(const float* p, float (&v)[W]) {
  if constexpr (W == 8) {
    const float4 a = reinterpret_cast<const float4*>(p)[0];
    const float4 b = reinterpret_cast<const float4*>(p)[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
    static_assert(W == 1, "widths 8 and 1");
    v[0] = p[0];
  }
}

template <int W>
__device__ __forceinline__ void store_vec(__nv_bfloat16* p, const float (&v)[W]) {
  if constexpr (W == 8)
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]),
                                              pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
  else
    p[0] = __float2bfloat16_rn(v[0]);
}

template <int W>
__device__ __forceinline__ void store_vec(float* p, const float (&v)[W]) {
  if constexpr (W == 8) {
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    p[0] = v[0];
  }
}

// The same for a type known at run time (MM_BF16 or MM_FP32); element offset `at`.
template <int W>
__device__ __forceinline__ void load_any(const void* p, int type, int64_t at, float (&v)[W]) {
  if (type == MM_BF16)
    load_vec<W>(static_cast<const __nv_bfloat16*>(p) + at, v);
  else
    load_vec<W>(static_cast<const float*>(p) + at, v);
}

template <int W>
__device__ __forceinline__ void store_any(void* p, int type, int64_t at, const float (&v)[W]) {
  if (type == MM_BF16)
    store_vec<W>(static_cast<__nv_bfloat16*>(p) + at, v);
  else
    store_vec<W>(static_cast<float*>(p) + at, v);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// Sums of N values over the warp (N a power of two up to 32): lane l returns the sum of
// v[l / (32 / N)]. Halving what a lane carries at each exchange takes N - 1 shuffles (plus
// log2(32 / N)) instead of 5 N.
template <int N>
__device__ __forceinline__ float warp_sum_many(float (&v)[N], int lane) {
#pragma unroll
  for (int half = N / 2, o = 16; half > 0; half >>= 1, o >>= 1) {
    const bool hi = (lane & o) != 0;
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      if (i >= half) continue;
      const float keep = hi ? v[i + half] : v[i], send = hi ? v[i] : v[i + half];
      v[i] = keep + __shfl_xor_sync(0xFFFFFFFFu, send, o);
    }
  }
  float s = v[0];
#pragma unroll
  for (int o = 16 / N; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
  return s;
}

// Two 32-bit floats that one instruction works on (sm_100 and later).
struct f32x2 {
  unsigned long long v;
};
__device__ __forceinline__ f32x2 pair(float a, float b) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ f32x2 both(float a) { return pair(a, a); }
__device__ __forceinline__ void split(f32x2 p, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p.v));
}
__device__ __forceinline__ f32x2 mul(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ f32x2 fma(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ float sum_of(f32x2 p) {
  float a, b;
  split(p, a, b);
  return a + b;
}

// 8 elements at p (16-byte aligned) as four pairs, and back with one rounding.
__device__ __forceinline__ void load_pairs(const __nv_bfloat16* p, f32x2 (&v)[4]) {
  const uint4 r = *reinterpret_cast<const uint4*>(p);
  v[0] = pair(bf16_lo(r.x), bf16_hi(r.x));
  v[1] = pair(bf16_lo(r.y), bf16_hi(r.y));
  v[2] = pair(bf16_lo(r.z), bf16_hi(r.z));
  v[3] = pair(bf16_lo(r.w), bf16_hi(r.w));
}
__device__ __forceinline__ void load_pairs(const float* p, f32x2 (&v)[4]) {
  const ulonglong2 a = reinterpret_cast<const ulonglong2*>(p)[0];
  const ulonglong2 b = reinterpret_cast<const ulonglong2*>(p)[1];
  v[0].v = a.x, v[1].v = a.y, v[2].v = b.x, v[3].v = b.y;
}
// The same from shared memory (byte address).
template <typename T>
__device__ __forceinline__ void lds_pairs(uint32_t at, f32x2 (&v)[4]) {
  if constexpr (sizeof(T) == 2) {
    uint32_t r[4];
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at));
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = pair(bf16_lo(r[i]), bf16_hi(r[i]));
  } else {
    asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(v[0].v), "=l"(v[1].v) : "r"(at));
    asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(v[2].v), "=l"(v[3].v) : "r"(at + 16));
  }
}
__device__ __forceinline__ uint32_t pack_pair(f32x2 p) {
  float a, b;
  split(p, a, b);
  return pack_bf16(a, b);
}
__device__ __forceinline__ void store_pairs(__nv_bfloat16* p, const f32x2 (&v)[4]) {
  *reinterpret_cast<uint4*>(p) =
      make_uint4(pack_pair(v[0]), pack_pair(v[1]), pack_pair(v[2]), pack_pair(v[3]));
}
__device__ __forceinline__ void store_pairs(float* p, const f32x2 (&v)[4]) {
  reinterpret_cast<ulonglong2*>(p)[0] = make_ulonglong2(v[0].v, v[1].v);
  reinterpret_cast<ulonglong2*>(p)[1] = make_ulonglong2(v[2].v, v[3].v);
}

// Bytes (a multiple of 16, both addresses too) from global to shared memory, counted on `bar`.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}

}  // namespace mm
