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

// log2(e) / T.  Passes over a row form exponents of 2 as x = fma(z, c, -ref) with
// ref = c m rounded, m a maximum.  The fused product is exact, so x carries one
// rounding of its own size, c's rounding counts as a temperature 2^-24 off, and
// ref is a known number, not a rounded one, wherever sums with different
// references meet.
__device__ __forceinline__ float inv_temperature(float t) { return 1.4426950408889634f / t; }
// (a plain product would be fused into the difference of two references, which then is
// not that of the numbers: off by half a unit of c m in its last place)
__device__ __forceinline__ float reference(float m, float c) { return __fmul_rn(m, c); }
// Up to here ref is within 1/4 of c m, so the weights of entries at m are near 1;
// further out (logits of 1e38 as a mask) 2^x could overflow, and (v - m) c is
// taken.
constexpr float kRefMax = 4194304.f;
// log2 of exp((v - m) / T) for v <= m: 0 where both are the same infinity.
__device__ __forceinline__ float log2_weight(float v, float m, float c) { return v == m ? 0.f : (v - m) * c; }

__device__ __forceinline__ float fast_exp2(float x) {  // below 2^-126: 0
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// -------------------------------------------------- 16-byte packs of a row ---
// Four 32-bit words: one fp32 entry each, or two 16-bit ones.
template <typename T>
struct Pack;
template <>
struct Pack<float> {
  static constexpr int kPer = 1;  // entries per word
  static constexpr uint32_t kNegInf = 0xFF800000u;
  static __device__ __forceinline__ void open(uint32_t w, float* v) { v[0] = __uint_as_float(w); }
  static __device__ __forceinline__ uint32_t close(const float* v) { return __float_as_uint(v[0]); }
  static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
  }
};
template <>
struct Pack<__half> {
  static constexpr int kPer = 2;
  static constexpr uint32_t kNegInf = 0xFC00FC00u;
  static __device__ __forceinline__ void open(uint32_t w, float* v) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
    v[0] = f.x;
    v[1] = f.y;
  }
  static __device__ __forceinline__ uint32_t close(const float* v) {
    const __half2 h = __floats2half2_rn(v[0], v[1]);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    const __half2 h = __hmax2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&h);
  }
};
template <>
struct Pack<__nv_bfloat16> {
  static constexpr int kPer = 2;
  static constexpr uint32_t kNegInf = 0xFF80FF80u;
  static __device__ __forceinline__ void open(uint32_t w, float* v) {
    v[0] = __uint_as_float(w << 16);
    v[1] = __uint_as_float(w & 0xFFFF0000u);
  }
  static __device__ __forceinline__ uint32_t close(const float* v) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[0], v[1]);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    const __nv_bfloat162 h =
        __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&h);
  }
};

// One part of a row, read in 16-byte packs.  A row is cut at 16-byte boundaries
// of its addresses, so only its first and last pack can be partial.  Entry e of
// the part (row entry first + e) is element off + e of its packs.
template <typename T>
struct Part {
  static constexpr int kPer = Pack<T>::kPer, kE = 16 / sizeof(T);
  const T* row;
  const uint4* base;  // pack 0
  int64_t first;
  int n, off, packs;
  bool cut_head, cut_tail;

  __device__ __forceinline__ void cut(const T* p, int64_t V, int part, int parts) {  // parts: a power of two
    const int o = static_cast<int>((reinterpret_cast<uintptr_t>(p) & 15) / sizeof(T));
    const int64_t all = (V + o + kE - 1) / kE;
    const int lg = 31 - __clz(parts);
    const int64_t p0 = (all * part) >> lg, p1 = (all * (part + 1)) >> lg;
    const int64_t e0 = p0 * kE - o > 0 ? p0 * kE - o : 0;
    const int64_t e1 = p1 * kE - o < V ? p1 * kE - o : V;
    row = p;
    first = e0;
    n = e1 > e0 ? static_cast<int>(e1 - e0) : 0;
    off = p0 == 0 ? o : 0;
    packs = static_cast<int>(p1 - p0);
    base = reinterpret_cast<const uint4*>(p + first - off);
    cut_head = off > 0;
    cut_tail = (off + n) % kE != 0;
  }
  __device__ __forceinline__ int64_t index_of(int j) const { return first + j * kE - off; }
  __device__ __forceinline__ bool whole(int j) const {
    return (j > 0 || !cut_head) && (j + 1 < packs || !cut_tail);
  }
  // Pack j; elements that are no entries of the part come as -inf, and a pack
  // outside it as nothing else.  kLast: it is not read again.
  template <bool kLast = false>
  __device__ __forceinline__ uint4 pack(int j) const {
    uint4 v = make_uint4(Pack<T>::kNegInf, Pack<T>::kNegInf, Pack<T>::kNegInf, Pack<T>::kNegInf);
    if (j < 0 || j >= packs) return v;
    if (whole(j)) return kLast ? __ldcs(base + j) : base[j];
    T* e = reinterpret_cast<T*>(&v);
#pragma unroll
    for (int h = 0; h < kE; ++h) {
      const int i = j * kE + h - off;
      if (i >= 0 && i < n) e[h] = row[first + i];
    }
    return v;
  }
  // Packs j, j + step, ... into v[kN], with one test where all lie inside.
  template <int kN, bool kLast = false>
  __device__ __forceinline__ void load(int j, int step, uint4* v) const {
    if (j + (kN - 1) * step + 1 < packs && (j > 0 || (j == 0 && !cut_head))) {
      const uint4* p = base + j;
#pragma unroll
      for (int x = 0; x < kN; ++x) v[x] = kLast ? __ldcs(p + x * step) : p[x * step];
    } else {
#pragma unroll
      for (int x = 0; x < kN; ++x) v[x] = pack<kLast>(j + x * step);
    }
  }
  static __device__ __forceinline__ void open(const uint4& w, float* v) {  // kE values
    const uint32_t in[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int x = 0; x < 4; ++x) Pack<T>::open(in[x], v + x * kPer);
  }
  static __device__ __forceinline__ uint32_t max_words(const uint4& w) {
    return Pack<T>::max2(Pack<T>::max2(w.x, w.y), Pack<T>::max2(w.z, w.w));
  }
  static __device__ __forceinline__ float max_of(uint32_t w) {
    float v[kPer];
    Pack<T>::open(w, v);
    float r = v[0];
#pragma unroll
    for (int h = 1; h < kPer; ++h) r = fmaxf(r, v[h]);
    return r;
  }
};

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
