// rows.cuh — building blocks of the kernels that work on one row of
// vocabulary logits with a thread-block cluster: element types, the order of
// a row's entries, and reductions over the threads of a cluster.
//
// A row of V logits is split into `size` contiguous slices, one per CTA of
// its cluster.  Every reduction runs in a fixed order (lanes, warps, CTAs by
// rank), so results repeat bit for bit.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "ptx.cuh"

namespace dfl {

constexpr int kMaxCluster = 8;  // portable cluster size

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) {
  return v;
}
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) {
  return __float2half_rn(v);
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}

// Order of a row's values as unsigned integers: larger value, larger key;
// -0 and +0 share a key; NaN and -inf (masked entries) get 0, below all.
__device__ __forceinline__ uint32_t value_key(float v) {
  const uint32_t b = __float_as_uint(v + 0.f);
  const uint32_t k = b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
  return v > -INFINITY ? k : 0u;
}
__device__ __forceinline__ float key_to_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k ^ 0x80000000u) : ~k);
}
// Entries by descending value, ascending index: larger place, earlier entry.
__device__ __forceinline__ uint64_t place_of(uint32_t key, uint32_t idx) {
  return (static_cast<uint64_t>(key) << 32) | (0xFFFFFFFFu - idx);
}
__device__ __forceinline__ uint32_t place_index(uint64_t p) { return 0xFFFFFFFFu - static_cast<uint32_t>(p); }
// Ordered key of a double (no NaN)
__device__ __forceinline__ uint64_t double_key(double v) {
  const uint64_t b = static_cast<uint64_t>(__double_as_longlong(v + 0.0));
  return (b >> 63) ? ~b : (b | 0x8000000000000000ull);
}

// log2(e) / T as a float pair: an exponent formed with both parts carries
// little more than the rounding of its own last addition.
struct InvT {
  float hi, lo;
};
__device__ __forceinline__ InvT inv_temperature(float t) {
  const double c = 1.4426950408889634 / static_cast<double>(t);
  InvT r;
  r.hi = static_cast<float>(c);
  r.lo = static_cast<float>(c - static_cast<double>(r.hi));
  return r;
}
// log2 of exp((v - m) / T) for v <= m: 0 where both are the same infinity.
// A difference of -inf is brought to -1e38, which the pair's second part
// cannot turn into inf - inf; a NaN stays.
__device__ __forceinline__ float log2_weight(float v, float m, InvT c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(v - m), "f"(-1e38f));
  return v == m ? 0.f : fmaf(d, c.lo, d * c.hi);
}

// ------------------------------------------------------------- clusters ----
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
// All threads of the cluster; memory written before is seen after, shared
// memory of the other CTAs included.
__device__ __forceinline__ void cluster_sync_all(uint32_t size) {
  if (size > 1) {
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  } else {
    __syncthreads();
  }
}
// The address of `p` (this CTA's shared memory) in CTA `rank` of the cluster.
template <typename T>
__device__ __forceinline__ T* peer(T* p, uint32_t rank) {
  uint64_t out;
  asm volatile("mapa.u64 %0, %1, %2;" : "=l"(out) : "l"(reinterpret_cast<uint64_t>(p)), "r"(rank));
  return reinterpret_cast<T*>(out);
}

// Scratch of the cluster reductions below.  Successive reductions use the
// slots in turn, so one cluster barrier per reduction is enough: a slot is
// written again only two barriers after its readers were done.
template <int NW>
struct Exchange {
  uint64_t warp[NW];
  uint64_t slot[3][kMaxCluster];
};

struct OpMaxU64 {
  __device__ __forceinline__ uint64_t operator()(uint64_t a, uint64_t b) const { return a > b ? a : b; }
};
struct OpSumU64 {
  __device__ __forceinline__ uint64_t operator()(uint64_t a, uint64_t b) const { return a + b; }
};

// Reduction of one 64-bit value per thread over the CTA; every thread gets
// the result.
template <int NW, typename Op>
__device__ __forceinline__ uint64_t cta_reduce(uint64_t v, Op op, Exchange<NW>& x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
  if ((threadIdx.x & 31) == 0) x.warp[threadIdx.x >> 5] = v;
  __syncthreads();
  v = x.warp[0];
  for (int w = 1; w < NW; ++w) v = op(v, x.warp[w]);
  __syncthreads();
  return v;
}

// Reduction of one 64-bit value per thread over the cluster; every thread
// gets the result.  `turn` counts the calls (same in all threads).
template <int NW, typename Op>
__device__ __forceinline__ uint64_t cluster_reduce(uint64_t v, Op op, Exchange<NW>& x, uint32_t rank, uint32_t size,
                                                   int& turn) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
  if (lane == 0) x.warp[warp] = v;
  __syncthreads();
  const int s = turn % 3;
  ++turn;
  if (warp == 0) {
    v = lane < NW ? x.warp[lane] : 0;  // 0 leaves a maximum and a sum as they are
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
    if (lane < static_cast<int>(size)) *peer(&x.slot[s][rank], lane) = v;
  }
  cluster_sync_all(size);
  v = x.slot[s][0];
  for (uint32_t r = 1; r < size; ++r) v = op(v, x.slot[s][r]);
  return v;
}

}  // namespace dfl
