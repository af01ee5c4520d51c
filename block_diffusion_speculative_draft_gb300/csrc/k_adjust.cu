// k_adjust.cu — what a request's history, biases and grammar do to rows of
// logits before a token is drawn from them.  For entry v of a row, c the
// generated tokens equal to v (the row's own path of drafts among them):
//   x = z;  v in the prompt or c > 0: x = x > 0 ? x / rho : x rho
//   x -= frequency c + presence [c > 0];  x += bias[v];  not allowed: -inf
// in fp32, rounded once to the rows' type.
//
// Bound by HBM: a row is read and written once.  One CTA takes one segment of
// the vocabulary for all rows of a sequence, so the history is counted once a
// segment and not once a row: a scan of the whole history (L2 after the first
// CTA) into counters in shared memory, then a list of the entries that it, the
// drafts or the biases touch.  A few rows at a time then stream by as they are,
// but for the grammar's bits, and a warp a row goes through the list and writes
// the touched entries over.  (With the touched entries worked on where they came
// by, nearly every warp had one, and 32 x 32 rows of 151936 bf16 took 426 us in
// place of 144; rows that nothing touches stream at 6.3 TB/s.)  A row's path adds to few entries: they are marked in the
// counters, and the path is walked for those.
#include "kernels.h"
#include "rows.cuh"

namespace dfl {

namespace {

constexpr int kDevBadLength = 0x4, kDevBadParam = 0x8;
// 512 threads and 64 registers, two CTAs an SM: 144 us for 32 x 32 rows of 151936 bf16
// with everything asked for and 31 us for 8 x 16 of fp32, the same rows again and
// again (256 threads: 164 and 32); with rows that are not in L2, 144 and 35.  The
// form without a grammar spills 20 to 116 bytes a thread for its packs in flight.
constexpr int kThreads = 512;
constexpr int kFlight = 4;  // packs a thread has in flight (twice as many without a grammar)
constexpr int kScan = 8;    // tokens of the history

// A counter: generated tokens (bits 0-19), in the prompt, among the drafts,
// and, in bits 22-31, kAdjustMaxBias less the place of the entry's bias in the
// request's list (0: none).
constexpr uint32_t kCount = (1u << 20) - 1, kPrompt = 1u << 20, kDraft = 1u << 21;
constexpr int kSlotShift = 22;

template <typename T>
struct Bits;
template <>
struct Bits<float> {
  static constexpr uint32_t ninf = 0xff800000u, nan = 0x7fffffffu;
};
template <>
struct Bits<__half> {
  static constexpr uint32_t ninf = 0xfc00u, nan = 0x7fffu;
};
template <>
struct Bits<__nv_bfloat16> {
  static constexpr uint32_t ninf = 0xff80u, nan = 0x7fffu;
};
template <typename T>
__device__ __forceinline__ T of_bits(uint32_t b) {
  if constexpr (sizeof(T) == 4) {
    return __uint_as_float(b);
  } else {
    T v;
    *reinterpret_cast<uint16_t*>(&v) = (uint16_t)b;
    return v;
  }
}

// n <= 16 bits of a bit row from bit `at`, ones above them; words past `words`
// are not read.  kIn: they lie in one word.
template <bool kIn>
__device__ __forceinline__ uint32_t bits_at(const uint32_t* w, int64_t at, int n, int64_t words) {
  const int64_t i = at >> 5;
  const int s = (int)(at & 31);
  uint32_t v = w[i] >> s;
  if (!kIn && s + n > 32 && i + 1 < words) v |= w[i + 1] << (32 - s);
  return v | ~((1u << n) - 1u);
}

struct Shared {
  float rho, freq, pres;
  int bad;     // nothing of the sequence can be worked
  int repeat;  // a biased entry is listed twice
  int listed[kThreads / 32 + 1];  // touched entries of each warp's share, and before it
  int bias_idx[kAdjustMaxBias];
  float bias_val[kAdjustMaxBias];
  int draft[kTreeMax];
  int allow_row[kTreeMax];  // -1: no grammar, -2: out of range
};

// Entries before a row's first 16-byte boundary.
template <typename T>
__device__ __forceinline__ int head_of(const T* p) {
  return (int)((16 - ((uintptr_t)p & 15)) & 15) / (int)sizeof(T);
}
template <typename T>
__device__ __forceinline__ uint4 fill(uint32_t bits) {
  const uint32_t w = sizeof(T) == 4 ? bits : bits << 16 | bits;
  return make_uint4(w, w, w, w);
}
// -inf where a bit of `ok` is clear.
template <typename T>
__device__ __forceinline__ uint4 allow_pack(uint4 raw, uint32_t ok) {
  uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 4) {
      if (!(ok >> i & 1)) w[i] = Bits<T>::ninf;
    } else {
      if (!(ok >> (2 * i) & 1)) w[i] = (w[i] & 0xffff0000u) | Bits<T>::ninf;
      if (!(ok >> (2 * i + 1) & 1)) w[i] = (w[i] & 0xffffu) | Bits<T>::ninf << 16;
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// kMasked: rows may have a grammar.
template <typename T, bool kAligned, bool kMasked>
__global__ void __launch_bounds__(kThreads, 2) adjust_kernel(const AdjustArgs a) {
  constexpr int E = 16 / sizeof(T);  // entries of a pack
  constexpr int FL = kMasked ? kFlight : 2 * kFlight;
  extern __shared__ uint32_t s_dyn[];
  uint32_t* const s_count = s_dyn;                                           // [seg]
  uint32_t* const s_touch = s_dyn + a.seg;                                   // [seg / 32] one bit an entry
  uint16_t* const s_list = reinterpret_cast<uint16_t*>(s_touch + a.seg / 32);  // [seg] touched entries
  __shared__ Shared sh;
  pdl_wait();
  const int tid = threadIdx.x;
  const int64_t j = blockIdx.x / a.nseg;
  const int64_t s0 = (int64_t)(blockIdx.x % a.nseg) * a.seg;
  const int64_t s1 = s0 + a.seg < a.V ? s0 + a.seg : a.V;
  const uint32_t len = (uint32_t)(s1 - s0);

  // ---- the sequence's request ----
  const int nh = a.hist ? a.n_hist[j] : 0;
  const int np = a.hist && a.n_prompt ? a.n_prompt[j] : 0;
  if (tid == 0) {
    sh.rho = a.repetition ? a.repetition[j] : 1.f;
    sh.freq = a.frequency ? a.frequency[j] : 0.f;
    sh.pres = a.presence ? a.presence[j] : 0.f;
    int why = 0;
    if (!(sh.rho > 0.f && sh.rho < INFINITY && fabsf(sh.freq) < INFINITY && fabsf(sh.pres) < INFINITY))
      why = kDevBadParam;
    if (np < 0 || np > nh || nh > a.H) why |= kDevBadLength;
    sh.bad = why;
    sh.repeat = 0;
  }
  for (int i = tid; i < a.seg + a.seg / 32; i += kThreads) s_dyn[i] = 0;
  for (int i = tid; i < a.K; i += kThreads) {
    sh.bias_idx[i] = a.bias_idx[j * a.K + i];
    sh.bias_val[i] = a.bias_val[j * a.K + i];
  }
  for (int i = tid; i < a.D; i += kThreads) sh.draft[i] = a.draft[j * a.D + i];
  for (int i = tid; i < a.R; i += kThreads) {
    int64_t r = -1;
    if (a.allow) {
      r = a.allow_row ? a.allow_row[j * a.R + i] : j * a.R + i;
      if (r < -1 || r >= a.n_allow) {
        r = -2;
        if (s0 == 0) atomicOr(a.status, kDevBadParam);
      }
    }
    sh.allow_row[i] = (int)r;
  }
  __syncthreads();
  auto mark = [&](uint32_t e) { atomicOr(&s_touch[e >> 5], 1u << (e & 31)); };
  if (!sh.bad) {
    const int* h = a.hist + j * a.ld_hist;
    auto take = [&](int t, bool made) {
      const uint32_t e = (uint32_t)t - (uint32_t)s0;  // below the segment, or negative: out of range
      if (t < 0 || e >= len) return;
      if (made) atomicAdd(&s_count[e], 1u);
      else atomicOr(&s_count[e], kPrompt);
      mark(e);
    };
    for (int i = tid; i < nh; i += kThreads * kScan) {
      int t[kScan];
#pragma unroll
      for (int q = 0; q < kScan; ++q) t[q] = i + q * kThreads < nh ? h[i + q * kThreads] : -1;
#pragma unroll
      for (int q = 0; q < kScan; ++q) take(t[q], i + q * kThreads >= np);
    }
    for (int i = tid; i < a.D; i += kThreads) {
      const int t = sh.draft[i];
      const uint32_t e = (uint32_t)t - (uint32_t)s0;
      if (t < 0 || e >= len) continue;
      atomicOr(&s_count[e], kDraft);
      mark(e);
    }
    // The counters' low parts are done before slots go above them: the largest
    // number wins, so an entry belongs to the first that lists it.
    __syncthreads();
    for (int i = tid; i < a.K; i += kThreads) {
      const int t = sh.bias_idx[i];
      if (t < 0 || t >= a.V) continue;
      if (!(sh.bias_val[i] < INFINITY)) atomicOr(&sh.bad, kDevBadParam);
      const uint32_t e = (uint32_t)t - (uint32_t)s0;
      if ((int64_t)t < s0 || e >= len) continue;
      const uint32_t slot = (uint32_t)(kAdjustMaxBias - i) << kSlotShift;
      const uint32_t low = s_count[e] & ((1u << kSlotShift) - 1u);
      if (atomicMax(&s_count[e], slot | low) >> kSlotShift) sh.repeat = 1;
      mark(e);
    }
    __syncthreads();
    // an entry listed again adds up, in the list's order: the first of an entry
    // writes the sum to its own place, which no other sum reads
    if (sh.repeat)
      for (int i = tid; i < a.K; i += kThreads) {
        const int t = sh.bias_idx[i];
        const uint32_t e = (uint32_t)t - (uint32_t)s0;
        if (t < 0 || (int64_t)t < s0 || e >= len || s_count[e] >> kSlotShift != (uint32_t)(kAdjustMaxBias - i)) continue;
        float sum = sh.bias_val[i];
        for (int k = i + 1; k < a.K; ++k)
          if (sh.bias_idx[k] == t) sum += sh.bias_val[k];
        sh.bias_val[i] = sum;
      }
    __syncthreads();
  }
  const int bad = sh.bad;
  if (bad && tid == 0 && s0 == 0) atomicOr(a.status, bad);

  // ---- the touched entries, in order ----
  const int lane = tid & 31, warp = tid >> 5;
  int listed = 0;
  if (!bad) {
    const int words = a.seg / 32;
    const uint32_t w = tid < words ? s_touch[tid] : 0u;
    int n = __popc(w);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, n, o);
      if (lane >= o) n += y;
    }
    if (lane == 31) sh.listed[warp] = n;
    __syncthreads();
    int at = n - __popc(w);
    for (int i = 0; i < kThreads / 32; ++i) {
      if (i < warp) at += sh.listed[i];
      listed += sh.listed[i];
    }
    for (uint32_t m = w; m; m &= m - 1) s_list[at++] = (uint16_t)(tid * 32 + __ffs(m) - 1);
    __syncthreads();
  }

  // ---- the rows, up to one a warp at a time ----
  const int64_t aw = (a.V + 31) / 32;
  const T* const in0 = static_cast<const T*>(a.logits) + j * a.R * a.ld + s0;
  T* const out0 = static_cast<T*>(a.out) + j * a.R * a.ld_out + s0;
  const uint32_t shift = 31 - __clz(a.seg / E);  // packs of a whole segment, a power of two
  for (int r0 = 0; r0 < a.R; r0 += kThreads / 32) {
    const int rn = min(kThreads / 32, a.R - r0);
    // Whole packs on 16-byte boundaries, then (unaligned rows) the entries before
    // the first and behind the last of them.
    for (uint32_t p0 = tid; p0 < (uint32_t)rn << shift; p0 += kThreads * FL) {
      uint4 raw[FL];
      uint32_t ok[FL];
#pragma unroll
      for (int q = 0; q < FL; ++q) {
        const uint32_t p = p0 + q * kThreads;
        const int r = r0 + (int)(p >> shift);
        if (r >= r0 + rn) continue;
        const T* in = in0 + r * a.ld;
        const int at = (int)(p & ((1u << shift) - 1u)) * E + (kAligned ? 0 : head_of(in));
        if (at + E > (int)len) continue;
        raw[q] = *reinterpret_cast<const uint4*>(in + at);
        if (!kMasked) continue;
        ok[q] = ~0u;
        const int ar = sh.allow_row[r];
        if (ar >= 0) ok[q] = bits_at<kAligned>(a.allow + ar * a.ld_allow, s0 + at, E, aw);
      }
#pragma unroll
      for (int q = 0; q < FL; ++q) {
        const uint32_t p = p0 + q * kThreads;
        const int r = r0 + (int)(p >> shift);
        if (r >= r0 + rn) continue;
        const int at = (int)(p & ((1u << shift) - 1u)) * E + (kAligned ? 0 : head_of(in0 + r * a.ld));
        if (at + E > (int)len) continue;
        if (bad || (kMasked && sh.allow_row[r] == -2)) raw[q] = fill<T>(Bits<T>::nan);
        else if (kMasked && ok[q] != ~0u) raw[q] = allow_pack<T>(raw[q], ok[q]);
        T* out = out0 + r * a.ld_out + at;
        if (kAligned || ((uintptr_t)out & 15) == 0) {
          *reinterpret_cast<uint4*>(out) = raw[q];
        } else {
          const T* x = reinterpret_cast<const T*>(&raw[q]);
#pragma unroll
          for (int i = 0; i < E; ++i) out[i] = x[i];
        }
      }
    }
    if (!kAligned || len % E) {
      for (int i = tid; i < rn * 2 * E; i += kThreads) {
        const int r = r0 + i / (2 * E), e = i % (2 * E);
        const T* in = in0 + r * a.ld;
        const int head = kAligned ? 0 : min(head_of(in), (int)len);
        const int at = e < E ? e : head + ((int)len - head) / E * E + e - E;
        if (e < E ? e >= head : at >= (int)len) continue;
        const int ar = sh.allow_row[r];
        T x = in[at];
        if (ar >= 0 && !(a.allow[ar * a.ld_allow + ((s0 + at) >> 5)] >> ((s0 + at) & 31) & 1)) x = of_bits<T>(Bits<T>::ninf);
        if (bad || ar == -2) x = of_bits<T>(Bits<T>::nan);
        out0[r * a.ld_out + at] = x;
      }
    }
    if (!listed) continue;
    __syncthreads();  // the rows' entries are written, the touched ones as they were
    const int share = kThreads / 32 / rn;  // warps a row
    const int r = r0 + warp % rn;
    const int ar = sh.allow_row[r];
    if (warp / rn >= share || ar == -2) continue;
    const uint32_t* const path = a.path ? a.path + (j * a.R + r) * ((a.D + 31) / 32) : nullptr;
    for (int i0 = warp / rn * 32 + lane; i0 < listed; i0 += share * 32 * kFlight) {
      T z[kFlight];
      int entry[kFlight];  // -1: none, or not allowed
#pragma unroll
      for (int q = 0; q < kFlight; ++q) {
        const int i = i0 + q * share * 32;
        entry[q] = i < listed ? s_list[i] : -1;
        if (entry[q] >= 0 && ar >= 0) {
          const int64_t v = s0 + entry[q];
          if (!(a.allow[ar * a.ld_allow + (v >> 5)] >> (v & 31) & 1)) entry[q] = -1;
        }
        if (entry[q] >= 0) z[q] = in0[r * a.ld + entry[q]];
      }
#pragma unroll
      for (int q = 0; q < kFlight; ++q) {
        const int e = entry[q];
        if (e < 0) continue;
        const uint32_t w = s_count[e];
        uint32_t c = w & kCount;
        if (w & kDraft) {
          const int v = (int)s0 + e;
          if (path) {
            for (int k = 0; k * 32 < a.D; ++k)
              for (uint32_t m = path[k]; m; m &= m - 1) {
                const int d = k * 32 + __ffs(m) - 1;
                c += d < a.D && sh.draft[d] == v;
              }
          } else {
            for (int d = 0; d < min(r, a.D); ++d) c += sh.draft[d] == v;
          }
        }
        float f = to_f32(z[q]);
        if (c || (w & kPrompt)) f = f > 0.f ? f / sh.rho : f * sh.rho;
        if (c) f = f - sh.freq * (float)c - sh.pres;
        const uint32_t slot = w >> kSlotShift;
        if (slot) f += sh.bias_val[kAdjustMaxBias - slot];
        out0[r * a.ld_out + e] = from_f32<T>(f);
      }
    }
  }
}

template <typename T>
const void* pick(bool aligned, bool masked) {
  if (aligned) return masked ? (const void*)adjust_kernel<T, true, true> : (const void*)adjust_kernel<T, true, false>;
  return masked ? (const void*)adjust_kernel<T, false, true> : (const void*)adjust_kernel<T, false, false>;
}

}  // namespace

cudaError_t adjust_logits(const AdjustArgs& a0, int dtype, int64_t b, cudaStream_t st) {
  AdjustArgs a = a0;
  const int es = dtype == 0 ? 4 : 2;
  // Segments: as long as they go (the history is scanned once a segment), but
  // two CTAs an SM where the call has so much to share out.
  a.seg = 8192;
  while (a.seg > 1024 && b * ((a.V + a.seg - 1) / a.seg) < 2 * num_sms()) a.seg /= 2;
  a.nseg = (unsigned)((a.V + a.seg - 1) / a.seg);
  if (b * (int64_t)a.nseg > 0x7fffffffll) return cudaErrorInvalidValue;
  const bool aligned = ((uintptr_t)a.logits & 15) == 0 && ((uintptr_t)a.out & 15) == 0 && a.ld * es % 16 == 0 &&
                       a.ld_out * es % 16 == 0;
  const void* fn = dtype == 0   ? pick<float>(aligned, a.allow)
                   : dtype == 1 ? pick<__half>(aligned, a.allow)
                                : pick<__nv_bfloat16>(aligned, a.allow);
  const size_t smem = (size_t)(a.seg + a.seg / 32) * 4 + (size_t)a.seg * 2;
  static unsigned long long done[12];
  if (cudaError_t e = allow_smem(fn, 8192 * 4 + 8192 / 8 + 8192 * 2, &done[dtype * 4 + aligned * 2 + (a.allow != nullptr)])) return e;
  void* args[] = {&a};
  return launch_k(fn, dim3((unsigned)(b * a.nseg)), dim3(kThreads), smem, st, true, args);
}

}  // namespace dfl
