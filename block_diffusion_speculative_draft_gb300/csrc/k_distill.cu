// k_distill.cu — distillation of a student's logits from a teacher's top
// logits: loss and gradient.
//
// Per row, with student logits z[0..V), the teacher's entries (t_k, i_k),
// k < K (S the set of their tokens), and temperature T:
//   q = softmax(z / T);   p_k = exp(t_k / T - Lt)
//   Lt = log sum_k exp(t_k / T), or the caller's log-sum-exp over the whole
//   vocabulary; then p_r = max(0, 1 - sum_k p_k) is the teacher's probability
//   of every other token together, and q_r = sum of q outside S
//   KL = sum_k p_k (ln p_k - ln q_{i_k}) + p_r (ln p_r - ln q_r)
//   dKL/dz_j = (P q_j - p_j) / T                     j in S, P = sum p + p_r
//            = exp(z_j / T) (P / E' - p_r / E'_r) / T  outside, E' and E'_r
//              the sums of exp(z / T) over the row and outside S
// The sums over the entries outside S are kept apart from those in S, and
// scaled by their own maximum, so q_r keeps its precision when the student
// puts nearly everything on S.
//
// Bound by HBM: the row is read, and its gradient written.  A row belongs to
// a cluster of up to eight CTAs whose shared memory holds it (one bulk copy
// each), so maximum, sum and gradient take one read of HBM; one exchange of
// (maximum, sum, refusal) joins the parts.  The listed entries become -inf in
// shared memory: the loops over the part then need no membership test, and
// the listed gradients are written after them.
#include "kernels.h"
#include "rows.cuh"

namespace dfl {

namespace {

constexpr int kDevBadToken = 0x2;
constexpr float kMassOne = 1099511627776.f;  // 2^40: probabilities are summed as integers
constexpr float kLn2 = 0.6931471805599453f;

// Shared memory of one CTA: this header, the teacher's entries (three arrays
// of K), the bitmap of the part's listed entries, then the part itself.
template <int NW>
struct alignas(16) Shared {
  Exchange<NW> x;
  float4 warp[2][NW];
  uint64_t warp_mass[NW];
  float4 part[kMaxCluster];  // (maximum, sum, refused) of each CTA's part
  uint64_t bar;
};

struct Entries {
  float* p;   // the teacher's logits, then its probabilities
  float* z;   // the student's logits at its tokens
  int* at;    // the tokens, -1: no entry
};
__device__ __forceinline__ Entries entries_at(uint8_t* base, int K) {
  Entries e;
  e.p = reinterpret_cast<float*>(base);
  e.z = e.p + K;
  e.at = reinterpret_cast<int*>(e.z + K);
  return e;
}
__host__ __device__ inline size_t entries_bytes(int K) { return (static_cast<size_t>(K) * 12 + 15) & ~size_t(15); }
size_t bitmap_bytes(int64_t n) { return (static_cast<size_t>((n + 31) / 32) * 4 + 15) & ~size_t(15); }

// Sum / maximum of a float over the CTA in a fixed order (every thread gets it).
template <int NW>
__device__ __forceinline__ float cta_sum(float v, float4* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5].x = v;
  __syncthreads();
  v = 0.f;
#pragma unroll
  for (int w = 0; w < NW; ++w) v += red[w].x;
  return v;
}
template <int NW>
__device__ __forceinline__ float cta_max(float v, float4* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5].x = v;
  __syncthreads();
  v = red[0].x;
#pragma unroll
  for (int w = 1; w < NW; ++w) v = fmaxf(v, red[w].x);
  return v;
}

// What the teacher's entries contribute, with the student's logits at them.
// Exponents are in units of log2 (x = z log2(e) / T).
struct Teacher {
  float tm;    // largest listed logit (-inf: nothing is listed)
  bool bad;    // refused by this CTA's view of the row
  float P;     // sum p + p_r
  float pr;
  float ref;   // reference of the listed student logits
  float es;    // sum of 2^(x_k - ref)
  float self;  // sum p_k (ln p_k - ln 2 (x_k - ref))
};

// A reference for exponents whose maximum is m: its own exponent, held within
// +-kRefMax.  Logits beyond that (the type's lowest value as a mask, infinities
// aside from -inf) count as the bound, so that rows of nothing else still have
// a distribution.
__device__ __forceinline__ float ref_of(float m, float c) {
  const float r = m * c;
  return r > kRefMax ? kRefMax : (r > -kRefMax ? r : -kRefMax);
}
__device__ __forceinline__ float exponent(float v, float c, float ref) {
  const float r = v * c;
  if (fabsf(r) < kRefMax || !(v > -INFINITY)) return fmaf(v, c, -ref);  // -inf and NaN stay
  return (r > 0.f ? kRefMax : -kRefMax) - ref;
}
// Calls f(weight) with weight(v) = 2^(exponent of v): the bare form where the
// reference, and so every entry below it, is inside the bound.
template <typename F>
__device__ __forceinline__ void with_weight(float c, float ref, F f) {
  if (fabsf(ref) < kRefMax) {
    f([=](float v) { return fast_exp2(fmaf(v, c, -ref)); });
  } else {
    f([=](float v) { return fast_exp2(exponent(v, c, ref)); });
  }
}

// Reads the row's entries.  `bits` (zero) marks the listed tokens in [c0, c1);
// a mark that is there already, or a token out of range, refuses the row.
// `row_z`: the student's logits are wanted for every entry (read from global
// memory); else es and self are not formed.
template <typename T, int NT>
__device__ __forceinline__ Teacher read_teacher(const DistillArgs& a, int64_t row, const T* z, int64_t c0, int64_t c1,
                                                bool row_z, Entries e, uint32_t* bits, Shared<NT / 32>& s) {
  constexpr int NW = NT / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool some = warp * 32 < a.K;  // this warp holds entries
  Teacher t;
  bool bad = false;
  float tm = -INFINITY, zm = -INFINITY;
  for (int k = threadIdx.x; k < a.K; k += NT) {
    const int i = a.t_idx[row * a.K + k];
    const float v = a.t_val[row * a.K + k];
    const bool in = i >= 0 && i < a.V, own = in && i >= c0 && i < c1;
    const float zk = own || (in && row_z) ? to_f32(z[i]) : -INFINITY;
    bad |= !in && i != -1;
    if (own) {
      const uint32_t bit = 1u << ((i - c0) & 31);
      bad |= (atomicOr(&bits[(i - c0) >> 5], bit) & bit) != 0;
    }
    e.at[k] = in ? i : -1;
    e.p[k] = in ? v : -INFINITY;
    e.z[k] = zk;
    tm = fmaxf(tm, in ? v : -INFINITY);
    zm = fmaxf(zm, zk);
  }
  if (some) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      tm = fmaxf(tm, __shfl_xor_sync(0xffffffffu, tm, o));
      zm = fmaxf(zm, __shfl_xor_sync(0xffffffffu, zm, o));
    }
  }
  if (lane == 0) s.warp[0][warp] = make_float4(tm, zm, 0.f, 0.f);
  t.bad = __syncthreads_or(bad);
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    tm = fmaxf(tm, s.warp[0][w].x);
    zm = fmaxf(zm, s.warp[0][w].y);
  }
  t.tm = tm;
  t.ref = ref_of(zm, a.c);
  double lt;
  if (a.t_lse) {
    lt = static_cast<double>(a.t_lse[row]);
  } else {
    float sp = 0.f;
    for (int k = threadIdx.x; k < a.K; k += NT) sp += exp2f(log2_weight(e.p[k], tm, a.c));
    lt = static_cast<double>(tm) * a.inv_t + static_cast<double>(logf(cta_sum<NW>(sp, s.warp[1])));
    __syncthreads();
  }
  // ln p_k = t_k / T - Lt, formed in double: where t_lse is given, p_r is a
  // difference from one.  The probabilities' sum is an integer sum for the
  // same reason.
  uint64_t fixed = 0;
  float es = 0.f, self = 0.f;
  for (int k = threadIdx.x; k < a.K; k += NT) {
    const double lp = static_cast<double>(e.p[k]) * a.inv_t - lt;
    const float hi = static_cast<float>(lp);
    float p = expf(hi);
    if (hi > -INFINITY) p = fmaf(p, static_cast<float>(lp - static_cast<double>(hi)), p);
    e.p[k] = p;
    fixed += __float2ull_rn(fminf(p, 256.f) * kMassOne);
    if (row_z && e.at[k] >= 0) {
      const float x = exponent(e.z[k], a.c, t.ref);
      es += exp2f(x);
      if (p > 0.f) self += p * (hi - x * kLn2);
    }
  }
  if (some) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      fixed += __shfl_xor_sync(0xffffffffu, fixed, o);
      es += __shfl_xor_sync(0xffffffffu, es, o);
      self += __shfl_xor_sync(0xffffffffu, self, o);
    }
  }
  if (lane == 0) {
    s.warp_mass[warp] = fixed;
    s.warp[1][warp] = make_float4(es, self, 0.f, 0.f);
  }
  __syncthreads();
  fixed = 0;
  t.es = 0.f;
  t.self = 0.f;
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    fixed += s.warp_mass[w];
    t.es += s.warp[1][w].x;
    t.self += s.warp[1][w].y;
  }
  // in units of 2^-40: one minus the sum, exactly
  const int64_t rest = (static_cast<int64_t>(1) << 40) - static_cast<int64_t>(fixed);
  const float mass = static_cast<float>(fixed) * (1.f / kMassOne);
  t.pr = a.t_lse && rest > 0 ? static_cast<float>(rest) * (1.f / kMassOne) : 0.f;
  t.P = mass + t.pr;
  return t;
}

// What the row's gradient needs: reference and sum of 2^(x - reference) over
// the row (m, E) and outside S (mr, Er).  E = 0 stands for a row without a
// gradient.
struct RowSums {
  float m, E, mr, Er;
};

// Joins the sums outside S with the listed entries'; thread 0 of the row's
// first CTA writes the loss.
__device__ __forceinline__ RowSums join_row(const DistillArgs& a, int64_t row, const Teacher& t, float mr, float Er,
                                            float w, bool writes) {
  RowSums s;
  s.mr = mr;
  s.Er = Er;
  // a part without a finite logit does not set the reference
  s.m = t.es > 0.f && Er > 0.f ? fmaxf(t.ref, mr) : (Er > 0.f ? mr : t.ref);
  s.E = t.es * exp2f(t.ref - s.m) + Er * exp2f(mr - s.m);
  // a row without any finite logit has no distribution
  if (s.E == 0.f) s.E = NAN;
  if (writes) {
    const float log_e = log2f(s.E);
    // sum p (ln p - ln q), ln q = ln 2 (x - m - log2 E)
    float l = t.self + (t.P - t.pr) * (log_e + (s.m - t.ref)) * kLn2;
    if (t.pr > 0.f) l += t.pr * (logf(t.pr) - (log2f(Er) + (mr - s.m) - log_e) * kLn2);
    a.loss[row] = w * l;
    if (a.stats) a.stats[row] = make_float4(s.m, s.E, s.mr, s.Er);
  }
  return s;
}

__device__ __forceinline__ void leave_out(const DistillArgs& a, int64_t row, bool bad) {
  a.loss[row] = bad ? NAN : 0.f;
  if (a.stats) a.stats[row] = make_float4(0.f, 0.f, 0.f, 0.f);
}

// Factor of 2^(x_j - mr) outside S.
__device__ __forceinline__ float outside_factor(const RowSums& s, const Teacher& t, float g) {
  return s.Er > 0.f ? g * (t.P * exp2f(s.mr - s.m) / s.E - t.pr / s.Er) : 0.f;
}

// Gradients of the listed entries in [c0, c1).
template <typename T, int NT>
__device__ __forceinline__ void listed_gradients(const DistillArgs& a, T* dz, Entries e, int64_t c0, int64_t c1,
                                                 const RowSums& s, const Teacher& t, float g) {
  const float f = t.P / s.E;
  for (int k = threadIdx.x; k < a.K; k += NT) {
    const int i = e.at[k];
    if (i >= c0 && i < c1) dz[i] = from_f32<T>(g * (f * exp2f(exponent(e.z[k], a.c, s.m)) - e.p[k]));
  }
}

// Writes f(entry) of a part to dz: whole packs where source and destination
// share their alignment, else 32-bit words of the destination, each from the
// one or two words of the buffer that hold its entries.
template <typename T, int NT, typename F>
__device__ __forceinline__ void write_part(const Part<T>& q, const T* buf, T* dz, F f) {
  constexpr int kPer = Pack<T>::kPer;
  T* out = dz + q.first;  // entry 0 of the part
  const uint32_t* words = reinterpret_cast<const uint32_t*>(buf);
  const int phase = static_cast<int>((reinterpret_cast<uintptr_t>(out) & 15) / sizeof(T));
  if (phase == q.off) {
    const uint4* src = reinterpret_cast<const uint4*>(buf);
    T* dst = out - q.off;
    const bool cut_tail = (q.off + q.n) % Part<T>::kE != 0;
    for (int j = threadIdx.x; j < q.packs; j += NT) {
      const uint4 v = src[j];
      const uint32_t in[4] = {v.x, v.y, v.z, v.w};
      uint32_t o[4];
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        float t[kPer];
        Pack<T>::open(in[w], t);
#pragma unroll
        for (int h = 0; h < kPer; ++h) t[h] = f(t[h]);
        o[w] = Pack<T>::close(t);
      }
      if ((j > 0 || q.off == 0) && (j + 1 < q.packs || !cut_tail)) {
        reinterpret_cast<uint4*>(dst)[j] = make_uint4(o[0], o[1], o[2], o[3]);
      } else {
        const T* t = reinterpret_cast<const T*>(o);
#pragma unroll
        for (int h = 0; h < Part<T>::kE; ++h) {
          const int e = j * Part<T>::kE + h - q.off;
          if (e >= 0 && e < q.n) out[e] = t[h];
        }
      }
    }
    return;
  }
  // words of the destination: entry e = kPer * j - shift is the first of word j
  const int shift = kPer == 2 ? phase & 1 : 0;
  uint32_t* dst = reinterpret_cast<uint32_t*>(out - shift);
  const int count = (q.n + shift + kPer - 1) / kPer;
  for (int j = threadIdx.x; j < count; j += NT) {
    const int e = kPer * j - shift, b = q.off + e;
    uint32_t w;
    if (kPer == 1) {
      w = words[b];
    } else {
      // b + 1 may pass the part's last pack only where e + 1 is no entry
      const uint32_t lo = b >= 0 ? words[b >> 1] : 0u;
      const uint32_t hi = (b & 1) && e + 1 < q.n ? words[(b + 1) >> 1] : 0u;
      w = (b & 1) ? __byte_perm(lo, hi, 0x5432) : lo;
    }
    float t[kPer];
    Pack<T>::open(w, t);
#pragma unroll
    for (int h = 0; h < kPer; ++h) t[h] = f(t[h]);
    w = Pack<T>::close(t);
    if (kPer == 1 || (e >= 0 && e + 1 < q.n)) {
      dst[j] = w;
    } else {
      const T* h = reinterpret_cast<const T*>(&w);
      if (e >= 0 && e < q.n) out[e] = h[0];
      if (e + 1 >= 0 && e + 1 < q.n) out[e + 1] = h[1];
    }
  }
}

// A row held in the shared memory of its cluster (`parts` CTAs), or in the
// backward call one part of it per CTA: the statistics are given, so the parts
// need nothing of one another.
template <typename T, int NT, bool kBackward>
__global__ void __launch_bounds__(NT, NT == 256 ? 5 : 2) distill_kernel(const DistillArgs a, const int parts,
                                                                       const uint32_t part_bytes) {
  constexpr int NW = NT / 32, kPer = Pack<T>::kPer;
  extern __shared__ __align__(16) uint8_t raw[];
  Shared<NW>& s = *reinterpret_cast<Shared<NW>*>(raw);
  T* buf = reinterpret_cast<T*>(raw + sizeof(Shared<NW>));
  uint8_t* after = raw + sizeof(Shared<NW>) + part_bytes;
  const Entries e = entries_at(after, a.K);
  uint32_t* bits = reinterpret_cast<uint32_t*>(after + entries_bytes(a.K));
  const int64_t row = blockIdx.x >> (31 - __clz(parts));
  const int part = static_cast<int>(blockIdx.x & (parts - 1));
  const T* z = static_cast<const T*>(a.logits) + row * a.ld;
  T* dz = a.dlogits ? static_cast<T*>(a.dlogits) + row * a.ldd : nullptr;
  Part<T> q;
  q.cut(z, a.V, part, parts);
  const int64_t c0 = q.first, c1 = q.first + q.n;
  if (threadIdx.x == 0) {
    mbar_init(&s.bar, 1);
    fence_mbar_init();
  }
  for (int i = threadIdx.x; i < (q.n + 31) / 32; i += NT) bits[i] = 0;
  __syncthreads();
  if (!kBackward && parts > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  pdl_wait();
  q.load(z, buf, &s.bar);
  const float w = a.weight ? a.weight[row] : 1.f;
  const Teacher t = read_teacher<T, NT>(a, row, z, c0, c1, !kBackward, e, bits, s);
  mbar_wait(&s.bar, 0, a.status);
  __syncthreads();
  for (int k = threadIdx.x; k < a.K; k += NT) {
    const int i = e.at[k];
    if (i >= c0 && i < c1) buf[q.off + i - c0] = from_f32<T>(-INFINITY);
  }
  __syncthreads();
  RowSums r;
  if (!kBackward) {
    // maximum and exponential sum of the part, relative to its own maximum
    const uint4* src = reinterpret_cast<const uint4*>(buf);
    uint32_t mx = Pack<T>::kNegInf;
    for (int j = threadIdx.x; j < q.packs; j += NT) {
      const uint4 v = src[j];
      mx = Pack<T>::max2(mx, Pack<T>::max2(Pack<T>::max2(v.x, v.y), Pack<T>::max2(v.z, v.w)));
    }
    float v[kPer];
    Pack<T>::open(mx, v);
    float pm = v[0];
#pragma unroll
    for (int h = 1; h < kPer; ++h) pm = fmaxf(pm, v[h]);
    float ref = ref_of(cta_max<NW>(pm, s.warp[0]), a.c);
    float sum = 0.f;
    with_weight(a.c, ref, [&](auto weight) {
      for (int j = threadIdx.x; j < q.packs; j += NT) {
        const uint4 y = src[j];
        const uint32_t in[4] = {y.x, y.y, y.z, y.w};
        float some = 0.f;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          Pack<T>::open(in[x], v);
#pragma unroll
          for (int h = 0; h < kPer; ++h) some += weight(v[h]);
        }
        sum += some;
      }
    });
    sum = cta_sum<NW>(sum, s.warp[1]);
    bool bad = t.bad;
    if (parts > 1) {
      asm volatile("barrier.cluster.wait.aligned;" ::: "memory");  // the other CTAs have started
      if (threadIdx.x < parts) *peer(&s.part[part], threadIdx.x) = make_float4(ref, sum, bad ? 1.f : 0.f, 0.f);
      cluster_sync_all(parts);
      // references are finite, and below every other where nothing is left
      ref = -kRefMax;
      for (int o = 0; o < parts; ++o) {
        ref = fmaxf(ref, s.part[o].x);
        bad |= s.part[o].z != 0.f;
      }
      sum = 0.f;
      for (int o = 0; o < parts; ++o) sum += s.part[o].y * exp2f(s.part[o].x - ref);
    }
    r = RowSums{0.f, 0.f, 0.f, 0.f};
    if (bad || w == 0.f || t.tm == -INFINITY) {
      if (part == 0 && threadIdx.x == 0) {
        leave_out(a, row, bad);
        if (bad) atomicOr(a.status, kDevBadToken);
      }
    } else if (dz || part == 0) {
      r = join_row(a, row, t, ref, sum, w, part == 0 && threadIdx.x == 0);
    }
    if (!dz) return;
  } else {
    if (t.bad && threadIdx.x == 0) atomicOr(a.status, kDevBadToken);
    const float4 st = a.stats[row];
    r = RowSums{st.x, t.bad || w == 0.f ? 0.f : st.y, st.z, st.w};
  }
  if (r.E == 0.f) {  // left out or refused
    write_part<T, NT>(q, buf, dz, [](float) { return 0.f; });
    return;
  }
  const float g = w / a.T, f = outside_factor(r, t, g);
  with_weight(a.c, r.mr, [&](auto weight) {
    write_part<T, NT>(q, buf, dz, [=](float v) { return f * weight(v); });
  });
  __syncthreads();
  listed_gradients<T, NT>(a, dz, e, c0, c1, r, t, g);
}

// A row too long for the shared memory of a cluster: the same sums by reading
// the row from global memory for each of them, with the listed entries told by
// the bitmap.
constexpr int kLongThr = 512;

template <typename T>
__global__ void __launch_bounds__(kLongThr) distill_long_kernel(const DistillArgs a, const bool backward) {
  constexpr int NT = kLongThr, NW = NT / 32;
  extern __shared__ __align__(16) uint8_t raw[];
  Shared<NW>& s = *reinterpret_cast<Shared<NW>*>(raw);
  const Entries e = entries_at(raw + sizeof(Shared<NW>), a.K);
  uint32_t* bits = reinterpret_cast<uint32_t*>(raw + sizeof(Shared<NW>) + entries_bytes(a.K));
  pdl_wait();
  const uint32_t rank = cluster_rank(), size = cluster_size();
  const int64_t row = blockIdx.x / size;
  const T* z = static_cast<const T*>(a.logits) + row * a.ld;
  T* dz = a.dlogits ? static_cast<T*>(a.dlogits) + row * a.ldd : nullptr;
  const int64_t chunk = (a.V + size - 1) / size;
  const int64_t c0 = chunk * rank < a.V ? chunk * rank : a.V, c1 = c0 + chunk < a.V ? c0 + chunk : a.V;
  int turn = 0;
  const float w = a.weight ? a.weight[row] : 1.f;
  for (int64_t i = threadIdx.x; i < (c1 - c0 + 31) / 32; i += NT) bits[i] = 0;
  __syncthreads();
  const Teacher t = read_teacher<T, NT>(a, row, z, c0, c1, true, e, bits, s);
  cluster_sync_all(size);  // the other CTAs have started
  const bool bad = cluster_reduce<NW>(t.bad, OpMaxU64(), s.x, rank, size, turn) != 0;
  auto outside = [&](int64_t i) { return !(bits[(i - c0) >> 5] >> ((i - c0) & 31) & 1); };
  RowSums r{0.f, 0.f, 0.f, 0.f};
  if (bad || w == 0.f || t.tm == -INFINITY) {
    if (rank == 0 && threadIdx.x == 0) {
      if (!backward) leave_out(a, row, bad);
      if (bad) atomicOr(a.status, kDevBadToken);
    }
  } else if (!backward) {
    float v = -INFINITY;
    for (int64_t i = c0 + threadIdx.x; i < c1; i += NT)
      if (outside(i)) v = fmaxf(v, to_f32(z[i]));
    const uint64_t key = cluster_reduce<NW>(max(value_key(v), 0x007FFFFFu), OpMaxU64(), s.x, rank, size, turn);
    const float ref = ref_of(key_to_value(static_cast<uint32_t>(key)), a.c);
    float sum = 0.f;
    for (int64_t i = c0 + threadIdx.x; i < c1; i += NT)
      if (outside(i)) sum += fast_exp2(exponent(to_f32(z[i]), a.c, ref));
    sum = cta_sum<NW>(sum, s.warp[0]);
    if (threadIdx.x < size) peer(&s.part[rank], threadIdx.x)->x = sum;
    cluster_sync_all(size);
    sum = 0.f;
    for (uint32_t o = 0; o < size; ++o) sum += s.part[o].x;
    r = join_row(a, row, t, ref, sum, w, rank == 0 && threadIdx.x == 0);
  } else {
    const float4 st = a.stats[row];
    r = RowSums{st.x, st.y, st.z, st.w};
  }
  if (!dz) return;
  if (r.E == 0.f) {
    for (int64_t i = c0 + threadIdx.x; i < c1; i += NT) dz[i] = from_f32<T>(0.f);
    return;
  }
  const float g = w / a.T, f = outside_factor(r, t, g);
  for (int64_t i = c0 + threadIdx.x; i < c1; i += NT)
    if (outside(i)) dz[i] = from_f32<T>(f * fast_exp2(exponent(to_f32(z[i]), a.c, r.mr)));
  listed_gradients<T, NT>(a, dz, e, c0, c1, r, t, g);
}

template <typename T, int NT, bool kBackward>
cudaError_t launch_resident(const DistillArgs& a, int64_t rows, int parts, cudaStream_t st) {
  const uint32_t pb = static_cast<uint32_t>(Part<T>::bytes(a.V, parts));
  const size_t smem = sizeof(Shared<NT / 32>) + pb + entries_bytes(a.K) + bitmap_bytes(pb / sizeof(T));
  const void* kern = (const void*)distill_kernel<T, NT, kBackward>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  DistillArgs b = a;
  void* args[] = {&b, &parts, const_cast<uint32_t*>(&pb)};
  return launch_kc(kern, dim3((unsigned)(rows * parts)), dim3(NT), smem, st, true, dim3(kBackward ? 1 : parts), args);
}

// Largest part a CTA keeps beside the entries and the bitmap.
constexpr size_t kPartMax = 180 * 1024;

template <typename T>
cudaError_t launch(const DistillArgs& a, int64_t rows, bool backward, cudaStream_t st) {
  // parts of at most 40 KB let five CTAs share an SM; rows that do not fill the
  // GPU are cut further
  int parts = 1;
  while (parts < kMaxCluster && (Part<T>::bytes(a.V, parts) > 40 * 1024 ||
                                 (rows * parts < 2 * num_sms() && Part<T>::bytes(a.V, 2 * parts) >= 4096)))
    parts *= 2;
  const size_t pb = Part<T>::bytes(a.V, parts);
  if (pb <= kPartMax) {
    if (pb <= 40 * 1024)
      return backward ? launch_resident<T, 256, true>(a, rows, parts, st)
                      : launch_resident<T, 256, false>(a, rows, parts, st);
    return backward ? launch_resident<T, 512, true>(a, rows, parts, st)
                    : launch_resident<T, 512, false>(a, rows, parts, st);
  }
  const size_t smem = sizeof(Shared<kLongThr / 32>) + entries_bytes(a.K) +
                      bitmap_bytes((a.V + kMaxCluster - 1) / kMaxCluster);
  const void* kern = (const void*)distill_long_kernel<T>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  DistillArgs b = a;
  void* args[] = {&b, &backward};
  return launch_kc(kern, dim3((unsigned)(rows * kMaxCluster)), dim3(kLongThr), smem, st, true, dim3(kMaxCluster),
                   args);
}

}  // namespace

cudaError_t distill(DistillArgs a, int dtype, int64_t rows, bool backward, cudaStream_t st) {
  a.c = static_cast<float>(1.4426950408889634 / static_cast<double>(a.T));
  a.inv_t = 1.0 / static_cast<double>(a.T);
  if (dtype == 0) return launch<float>(a, rows, backward, st);
  if (dtype == 1) return launch<__half>(a, rows, backward, st);
  return launch<__nv_bfloat16>(a, rows, backward, st);
}

}  // namespace dfl
