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
constexpr double kMassOne = 1099511627776.0;  // 2^40: probabilities are summed as integers

// Shared memory of one CTA: this header, the teacher's entries (four arrays
// of K), the bitmap of the part's listed entries, then the part itself.
template <int NW>
struct Shared {
  Exchange<NW> x;
  float red[NW];
  float4 part[kMaxCluster];  // (maximum, sum, refused) of each CTA's part
  uint64_t bar;
};

struct Entries {
  float* lp;  // the teacher's logits, then log-probabilities
  float* p;   // its probabilities
  float* z;   // the student's logits at its tokens
  int* at;    // the tokens, -1: no entry
};
__device__ __forceinline__ Entries entries_at(uint8_t* base, int K) {
  Entries e;
  e.lp = reinterpret_cast<float*>(base);
  e.p = e.lp + K;
  e.z = e.p + K;
  e.at = reinterpret_cast<int*>(e.z + K);
  return e;
}
size_t entries_bytes(int K) { return (static_cast<size_t>(K) * 16 + 15) & ~size_t(15); }
size_t bitmap_bytes(int64_t n) { return (static_cast<size_t>((n + 31) / 32) * 4 + 15) & ~size_t(15); }

// Sum / maximum of a float over the CTA in a fixed order (every thread gets it).
template <int NW>
__device__ __forceinline__ float cta_sum(float v, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.f;
#pragma unroll
  for (int w = 0; w < NW; ++w) v += red[w];
  __syncthreads();
  return v;
}
template <int NW>
__device__ __forceinline__ float cta_max(float v, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = red[0];
#pragma unroll
  for (int w = 1; w < NW; ++w) v = fmaxf(v, red[w]);
  __syncthreads();
  return v;
}

// exp((v - m) / T) for v <= m
__device__ __forceinline__ float exp_diff(float v, float m, InvT c) { return exp2f(log2_weight(v, m, c)); }

// The teacher's entries of a row.  `bits` (zero) marks the listed entries of
// [c0, c1); a mark that is there already, or a token out of range, refuses the
// row.  z is gathered for every entry, or for those in [c0, c1) alone.
// Returns the largest t of this thread's entries.
template <typename T, int NT>
__device__ __forceinline__ float list_entries(const DistillArgs& a, int64_t row, const T* z, int64_t c0, int64_t c1,
                                              bool own_only, Entries e, uint32_t* bits, bool& bad) {
  float tm = -INFINITY;
  for (int k = threadIdx.x; k < a.K; k += NT) {
    const int i = a.t_idx[row * a.K + k];
    const float t = a.t_val[row * a.K + k];
    const bool in = i >= 0 && i < a.V, own = in && i >= c0 && i < c1;
    bad |= !in && i != -1;
    if (own) {
      const uint32_t bit = 1u << ((i - c0) & 31);
      bad |= (atomicOr(&bits[(i - c0) >> 5], bit) & bit) != 0;
    }
    e.at[k] = in ? i : -1;
    e.lp[k] = in ? t : -INFINITY;
    e.z[k] = own || (in && !own_only) ? to_f32(z[i]) : -INFINITY;
    tm = fmaxf(tm, in ? t : -INFINITY);
  }
  return tm;
}

// Turns the entries' logits into log-probabilities and probabilities; tm is
// the largest logit.  Returns sum p and p_r.
template <int NT>
__device__ __forceinline__ float2 teacher_mass(const DistillArgs& a, int64_t row, Entries e, float tm, InvT c,
                                               Exchange<NT / 32>& x, float* red) {
  const double inv_t = 1.0 / static_cast<double>(a.T);
  double lt;
  if (a.t_lse) {
    lt = static_cast<double>(a.t_lse[row]);
  } else {
    float sp = 0.f;
    for (int k = threadIdx.x; k < a.K; k += NT) sp += exp_diff(e.lp[k], tm, c);
    lt = static_cast<double>(tm) * inv_t + static_cast<double>(logf(cta_sum<NT / 32>(sp, red)));
  }
  // ln p_k = t_k / T - Lt, formed in double: where t_lse is given, p_r is a
  // difference from one.  The probabilities' sum is an integer sum for the
  // same reason.
  uint64_t fixed = 0;
  for (int k = threadIdx.x; k < a.K; k += NT) {
    const double lp = static_cast<double>(e.lp[k]) * inv_t - lt;
    const float hi = static_cast<float>(lp);
    float p = expf(hi);
    if (hi > -INFINITY) p = fmaf(p, static_cast<float>(lp - static_cast<double>(hi)), p);
    e.lp[k] = hi;
    e.p[k] = p;
    fixed += __float2ull_rn(fminf(p, 256.f) * static_cast<float>(kMassOne));
  }
  const double total = static_cast<double>(cta_reduce<NT / 32>(fixed, OpSumU64(), x)) / kMassOne;
  return make_float2(static_cast<float>(total),
                     a.t_lse && total < 1.0 ? static_cast<float>(1.0 - total) : 0.f);
}

// What the row's gradient needs: the maximum and exponential sum over the row
// (m, E) and outside S (mr, Er).  E = 0 stands for a row without a gradient.
struct RowSums {
  float m, E, mr, Er;
};

// The row's sums from those outside S, and its loss (rank 0's threads).
template <int NT>
__device__ __forceinline__ RowSums join_entries(const DistillArgs& a, int64_t row, Entries e, float2 mass, float mr,
                                                float Er, float w, InvT c, bool first, float* red) {
  RowSums s;
  s.mr = mr;
  s.Er = Er;
  float zm = -INFINITY;
  for (int k = threadIdx.x; k < a.K; k += NT) zm = fmaxf(zm, e.z[k]);
  s.m = fmaxf(cta_max<NT / 32>(zm, red), mr);
  float es = 0.f;
  for (int k = threadIdx.x; k < a.K; k += NT)
    if (e.at[k] >= 0) es += exp_diff(e.z[k], s.m, c);
  // a row without any finite logit has no distribution
  es = cta_sum<NT / 32>(es, red);
  s.E = s.m == -INFINITY ? NAN : es + Er * exp_diff(mr, s.m, c);
  if (first) {
    const float log_e = logf(s.E);
    float l = 0.f;
    for (int k = threadIdx.x; k < a.K; k += NT) {
      const float lp = e.lp[k];
      if (lp > -INFINITY) l += e.p[k] * (lp - ((e.z[k] - s.m) / a.T - log_e));
    }
    l = cta_sum<NT / 32>(l, red);
    if (mass.y > 0.f) l += mass.y * (logf(mass.y) - ((mr - s.m) / a.T + logf(s.Er) - log_e));
    if (threadIdx.x == 0) {
      a.loss[row] = w * l;
      if (a.stats) a.stats[row] = make_float4(s.m, s.E, s.mr, s.Er);
    }
  }
  return s;
}

// Factor of exp((z_j - mr) / T) outside S.
__device__ __forceinline__ float outside_factor(const RowSums& s, float2 mass, float g, InvT c) {
  return s.Er > 0.f ? g * ((mass.x + mass.y) * exp_diff(s.mr, s.m, c) / s.E - mass.y / s.Er) : 0.f;
}

// Gradients of the listed entries in [c0, c1).
template <typename T, int NT>
__device__ __forceinline__ void listed_gradients(T* dz, int K, Entries e, int64_t c0, int64_t c1, const RowSums& s,
                                                 float2 mass, float g, InvT c) {
  const float f = (mass.x + mass.y) / s.E;
  for (int k = threadIdx.x; k < K; k += NT) {
    const int i = e.at[k];
    if (i >= c0 && i < c1) dz[i] = from_f32<T>(g * (f * exp_diff(e.z[k], s.m, c) - e.p[k]));
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
  constexpr int NW = NT / 32;
  extern __shared__ __align__(16) uint8_t raw[];
  Shared<NW>& s = *reinterpret_cast<Shared<NW>*>(raw);
  T* buf = reinterpret_cast<T*>(raw + sizeof(Shared<NW>));
  uint8_t* after = raw + sizeof(Shared<NW>) + part_bytes;
  const Entries e = entries_at(after, a.K);
  uint32_t* bits = reinterpret_cast<uint32_t*>(after + ((static_cast<size_t>(a.K) * 16 + 15) & ~size_t(15)));
  const int64_t row = blockIdx.x / parts;
  const int part = static_cast<int>(blockIdx.x % parts);
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
  const InvT c = inv_temperature(a.T);
  bool bad = false;
  float tm = list_entries<T, NT>(a, row, z, c0, c1, kBackward, e, bits, bad);
  tm = cta_max<NW>(tm, s.red);
  const float2 mass = teacher_mass<NT>(a, row, e, tm, c, s.x, s.red);
  mbar_wait(&s.bar, 0, a.status);
  bad = __syncthreads_or(bad);
  T* body = buf + q.off;
  for (int k = threadIdx.x; k < a.K; k += NT) {
    const int i = e.at[k];
    if (i >= c0 && i < c1) body[i - c0] = from_f32<T>(-INFINITY);
  }
  RowSums r;
  if (!kBackward) {
    // maximum and exponential sum of the part, relative to its own maximum
    __syncthreads();
    const uint4* src = reinterpret_cast<const uint4*>(buf);
    uint32_t mx = Pack<T>::kNegInf;
    for (int j = threadIdx.x; j < q.packs; j += NT) {
      const uint4 v = src[j];
      mx = Pack<T>::max2(mx, Pack<T>::max2(Pack<T>::max2(v.x, v.y), Pack<T>::max2(v.z, v.w)));
    }
    float t[Pack<T>::kPer];
    Pack<T>::open(mx, t);
    float pm = t[0];
#pragma unroll
    for (int h = 1; h < Pack<T>::kPer; ++h) pm = fmaxf(pm, t[h]);
    pm = cta_max<NW>(pm, s.red);
    const float ref = pm == -INFINITY ? 0.f : pm;
    float sum = 0.f;
    for (int j = threadIdx.x; j < q.packs; j += NT) {
      const uint4 v = src[j];
      const uint32_t in[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        Pack<T>::open(in[x], t);
#pragma unroll
        for (int h = 0; h < Pack<T>::kPer; ++h) sum += fast_exp2((t[h] - ref) * c.hi);
      }
    }
    sum = cta_sum<NW>(sum, s.red);
    if (parts > 1) {
      asm volatile("barrier.cluster.wait.aligned;" ::: "memory");  // the other CTAs have started
      if (threadIdx.x < parts) *peer(&s.part[part], threadIdx.x) = make_float4(pm, sum, bad ? 1.f : 0.f, 0.f);
      cluster_sync_all(parts);
      pm = -INFINITY;
      for (int o = 0; o < parts; ++o) {
        pm = fmaxf(pm, s.part[o].x);
        bad |= s.part[o].z != 0.f;
      }
      sum = 0.f;
      for (int o = 0; o < parts; ++o) sum += s.part[o].y * exp_diff(s.part[o].x, pm, c);
    }
    const bool out = bad || w == 0.f || tm == -INFINITY;
    if (out) {
      if (part == 0 && threadIdx.x == 0) {
        a.loss[row] = bad ? NAN : 0.f;
        if (a.stats) a.stats[row] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (bad) atomicOr(a.status, kDevBadToken);
      }
      r.E = 0.f;
    } else if (dz || part == 0) {
      r = join_entries<NT>(a, row, e, mass, pm, sum, w, c, part == 0, s.red);
    }
    if (!dz) return;
  } else {
    if (bad && threadIdx.x == 0) atomicOr(a.status, kDevBadToken);
    const float4 st = a.stats[row];
    r = RowSums{st.x, bad || w == 0.f ? 0.f : st.y, st.z, st.w};
    __syncthreads();
  }
  if (r.E == 0.f) {  // left out or refused
    write_part<T, NT>(q, buf, dz, [](float) { return 0.f; });
    return;
  }
  const float g = w / a.T, f = outside_factor(r, mass, g, c);
  const float ref = r.mr == -INFINITY ? 0.f : r.mr, ch = c.hi;
  write_part<T, NT>(q, buf, dz, [=](float v) { return f * fast_exp2((v - ref) * ch); });
  __syncthreads();
  listed_gradients<T, NT>(dz, a.K, e, c0, c1, r, mass, g, c);
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
  uint32_t* bits = reinterpret_cast<uint32_t*>(raw + sizeof(Shared<NW>) +
                                               ((static_cast<size_t>(a.K) * 16 + 15) & ~size_t(15)));
  pdl_wait();
  const uint32_t rank = cluster_rank(), size = cluster_size();
  const int64_t row = blockIdx.x / size;
  const T* z = static_cast<const T*>(a.logits) + row * a.ld;
  T* dz = a.dlogits ? static_cast<T*>(a.dlogits) + row * a.ldd : nullptr;
  const int64_t chunk = (a.V + size - 1) / size;
  const int64_t c0 = chunk * rank < a.V ? chunk * rank : a.V, c1 = c0 + chunk < a.V ? c0 + chunk : a.V;
  int turn = 0;
  const float w = a.weight ? a.weight[row] : 1.f;
  const InvT c = inv_temperature(a.T);
  for (int64_t i = threadIdx.x; i < (c1 - c0 + 31) / 32; i += NT) bits[i] = 0;
  __syncthreads();
  bool bad = false;
  float tm = list_entries<T, NT>(a, row, z, c0, c1, false, e, bits, bad);
  cluster_sync_all(size);
  bad = cluster_reduce<NW>(bad, OpMaxU64(), s.x, rank, size, turn) != 0;
  tm = cta_max<NW>(tm, s.red);
  const float2 mass = teacher_mass<NT>(a, row, e, tm, c, s.x, s.red);
  auto outside = [&](int64_t i) { return !(bits[(i - c0) >> 5] >> ((i - c0) & 31) & 1); };
  RowSums r;
  if (bad || w == 0.f || tm == -INFINITY) {
    if (rank == 0 && threadIdx.x == 0) {
      if (!backward) a.loss[row] = bad ? NAN : 0.f;
      if (!backward && a.stats) a.stats[row] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (bad) atomicOr(a.status, kDevBadToken);
    }
    r.E = 0.f;
  } else if (!backward) {
    float v = -INFINITY;
    for (int64_t i = c0 + threadIdx.x; i < c1; i += NT)
      if (outside(i)) v = fmaxf(v, to_f32(z[i]));
    v = cta_max<NW>(v, s.red);
    const float mr = key_to_value(static_cast<uint32_t>(
        cluster_reduce<NW>(max(value_key(v), 0x007FFFFFu), OpMaxU64(), s.x, rank, size, turn)));
    const float ref = mr == -INFINITY ? 0.f : mr;
    float sum = 0.f;
    for (int64_t i = c0 + threadIdx.x; i < c1; i += NT)
      if (outside(i)) sum += exp_diff(to_f32(z[i]), ref, c);
    sum = cta_sum<NW>(sum, s.red);
    if (threadIdx.x < size) peer(&s.part[rank], threadIdx.x)->x = sum;
    cluster_sync_all(size);
    sum = 0.f;
    for (uint32_t o = 0; o < size; ++o) sum += s.part[o].x;
    r = join_entries<NT>(a, row, e, mass, mr, sum, w, c, rank == 0, s.red);
  } else {
    const float4 st = a.stats[row];
    r = RowSums{st.x, st.y, st.z, st.w};
  }
  if (!dz) return;
  if (r.E == 0.f) {
    for (int64_t i = c0 + threadIdx.x; i < c1; i += NT) dz[i] = from_f32<T>(0.f);
    return;
  }
  const float g = w / a.T, f = outside_factor(r, mass, g, c);
  for (int64_t i = c0 + threadIdx.x; i < c1; i += NT)
    if (outside(i)) dz[i] = from_f32<T>(f * exp_diff(to_f32(z[i]), r.mr == -INFINITY ? 0.f : r.mr, c));
  listed_gradients<T, NT>(dz, a.K, e, c0, c1, r, mass, g, c);
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

cudaError_t distill(const DistillArgs& a, int dtype, int64_t rows, bool backward, cudaStream_t st) {
  if (dtype == 0) return launch<float>(a, rows, backward, st);
  if (dtype == 1) return launch<__half>(a, rows, backward, st);
  return launch<__nv_bfloat16>(a, rows, backward, st);
}

}  // namespace dfl
