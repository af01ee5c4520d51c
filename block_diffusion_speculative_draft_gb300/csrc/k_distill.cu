// k_distill.cu — distillation of a student's logits from a teacher's top
// logits: loss and gradient.
//
// Per row, with student logits z[0..V), the teacher's entries (t_k, i_k),
// k < K (S the set of their tokens), and temperature T:
//   q = softmax(z / T);   p_k = exp(t_k / T - Lt)
//   Lt = log sum_k exp(t_k / T), or the caller's log-sum-exp over the whole
//   vocabulary; then p_r = max(0, 1 - sum_k p_k) is the teacher's probability
//   of every other token together, and q_r = sum of q outside S; a p_r that the
//   rounding of the log-sum-exp explains counts as 0 where q_r does (rest_of)
//   KL = sum_k p_k (ln p_k - ln q_{i_k}) + p_r (ln p_r - ln q_r)
//   dKL/dz_j = (P q_j - p_j) / T                     j in S, P = sum p + p_r
//            = exp(z_j / T) (P / E' - p_r / E'_r) / T  outside, E' and E'_r
//              the sums of exp(z / T) over the row and outside S
// The sums over the entries outside S are kept apart from those in S, and
// scaled by their own maximum, so q_r keeps its precision when the student
// puts nearly everything on S.
//
// Bound by HBM: the row is read, and its gradient written.  A cluster of CTAs
// takes a row, each a part of it: one pass for the sums, one exchange of them,
// and a second pass for the gradient, which finds the part in L2 (the CTAs on
// the GPU hold some 70 MB of parts of its 129 MB).  Nothing but the entries'
// bookkeeping is kept on chip, so enough loads are in flight to fill HBM while
// other CTAs exchange.  Entries of S are told by a bitmap of the part, which
// also shows a token listed twice; the listed gradients are written last.
// 2048 x 151936 bf16, K = 128: loss 112 us (5.6 TB/s), with gradient 255 us (4.9
// TB/s: a cluster waits for its slowest CTA); 15 x 151936 fp32 with gradient 12 us.
#include "kernels.h"
#include "rows.cuh"

namespace dfl {

namespace {

constexpr int kDevBadToken = 0x2, kDevBadParam = 0x8;  // why a row is refused
constexpr int kSome = 0x1;  // beside them: an entry above -inf is listed
constexpr float kMassOne = 1099511627776.f;  // 2^40: probabilities are summed as integers
constexpr float kMostP = 256.f;               // up to here: 1024 of them stay below 2^58
constexpr float kLn2 = 0.6931471805599453f;
// A log-sum-exp in fp32 is off by its rounding, 2^-24 of its size, and by its
// sum's, some 12 2^-24 (exponentials to 2^-22, the scaled logits' own rounding): a
// p_r up to 2^-20 (1 + |t_lse|) may be nothing else.
constexpr float kFaintRest = 9.5367431640625e-07f;

// What a part of a row contributes: the entries outside S (maximum and sum of
// 2^((z - maximum) c)), those listed in it (the same, sum p_k (ln p_k - (z_k -
// maximum) / T) and sum p_k), and its CTA's flags.  Without an entry above -inf the
// maximum is -inf and the sum 0.
struct PartSums {
  float top, sum, ltop, lsum, self, p;
  int flags;
};

// Shared memory of one CTA: this header, the teacher's entries (four arrays of
// K), and the bitmap of the part's listed tokens.
template <int NW>
struct alignas(16) Shared {
  float4 warp[NW];
  float2 top[NW];
  uint64_t mass[NW];
  PartSums part[kMaxCluster];
  struct {
    float f, mr, g, in, m;  // factor and maximum outside S, weight / T, P / E and the row's maximum
    int zero;                // no gradient
  } plan;
  int flags;  // reasons to refuse the row, and kSome
};

struct Entries {
  float* lp;  // the teacher's logits, then log-probabilities
  float* p;   // its probabilities
  float* z;   // the student's logits at the tokens of this part
  int* at;    // place of the token in this part, -1: not here
};
__device__ __forceinline__ Entries entries_at(uint8_t* base, int K) {
  Entries e;
  e.lp = reinterpret_cast<float*>(base);
  e.p = e.lp + K;
  e.z = e.p + K;
  e.at = reinterpret_cast<int*>(e.z + K);
  return e;
}
__host__ __device__ inline size_t entries_bytes(int K) { return (static_cast<size_t>(K) * 16 + 15) & ~size_t(15); }
// (with room for the packs that a loop's last round passes the part by)
size_t bitmap_bytes(int64_t n, int slack) {
  return (static_cast<size_t>((n + 31) / 32) * 4 + slack + 15) & ~size_t(15);
}

// Sums of 2^(v c) are kept relative to a maximum m of theirs.  In a pass over
// the entries the exponent is fma(v, c, -ref) with ref = m c rounded, while that
// rounding is small (is_near); lead() tells how far it is off.  Past that (the
// type's lowest value as a mask, say) it is (v - m) c.
__device__ __forceinline__ bool is_near(float ref) { return fabsf(ref) < kRefMax; }
__device__ __forceinline__ float lead(float m, float c) {
  const float ref = reference(m, c);
  return is_near(ref) ? fmaf(-m, c, ref) : 0.f;
}
// Calls f(weight) with weight(v) = 2^(exponent of v) in the form that m asks for.
template <typename F>
__device__ __forceinline__ void with_weight(float c, float ref, float m, F f) {
  if (is_near(ref)) {
    f([=](float v) { return fast_exp2(fmaf(v, c, -ref)); });
  } else {
    f([=](float v) { return fast_exp2(log2_weight(v, m, c)); });
  }
}

// A sum of two floats that carries twice their digits.
struct Pair {
  float hi, lo;
};
__device__ __forceinline__ Pair two_sum(float a, float b) {  // a + b exactly
  const float s = a + b, t = s - a;
  return Pair{s, (a - (s - t)) + (b - t)};
}
// v / T, from the launcher's pair of 1 / T
__device__ __forceinline__ Pair over_t(const DistillArgs& a, float v) {
  const float h = __fmul_rn(v, a.inv_hi);  // (not to be fused into the sums it goes to)
  return Pair{h, fmaf(v, a.inv_hi, -h) + v * a.inv_lo};
}

struct Teacher {
  int flags;   // this CTA's view of the row: reasons to refuse it, and kSome
  bool faint;  // p_r is within the rounding of t_lse
  float mass;  // sum p
  float pr;
};

// Why a row of weight w is refused (0: it is not).
__device__ __forceinline__ int reasons(int flags, float w) {
  return flags & (w != 0.f ? kDevBadToken | kDevBadParam : kDevBadToken);
}

// Reads the row's entries, with the student's logits at those of this part, and
// forms the teacher's probabilities.  `bits` (zero) marks the part's listed
// elements; a mark that is there already, or a token out of range, refuses the
// row; a logit that is NaN or +inf, or a t_lse that is not finite or so low that a p
// is above kMostP, does so unless the row's weight leaves it out (reasons).
template <typename T, int NT>
__device__ __forceinline__ Teacher read_teacher(const DistillArgs& a, int64_t row, const Part<T>& q, Entries e,
                                                uint32_t* bits, Shared<NT / 32>& s) {
  constexpr int NW = NT / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool holds = warp * 32 < a.K;  // this warp holds entries
  const int used = a.K < NT ? (a.K + 31) / 32 : NW;
  int flags = 0;
  float tm = -INFINITY;
  float lt = a.t_lse ? a.t_lse[row] : 0.f;
  for (int k = threadIdx.x; k < a.K; k += NT) {
    const int i = a.t_idx[row * a.K + k];
    const float v = a.t_val[row * a.K + k];
    const int64_t at = i - q.first;
    const bool in = i >= 0 && i < a.V, own = in && at >= 0 && at < q.n;
    if (!in && i != -1) flags |= kDevBadToken;
    if (own) {
      const uint32_t x = static_cast<uint32_t>(q.off + at), bit = 1u << (x & 31);
      if (atomicOr(&bits[x >> 5], bit) & bit) flags |= kDevBadToken;
      e.z[k] = to_f32(q.row[i]);
    }
    e.at[k] = own ? static_cast<int>(at) : -1;
    e.lp[k] = in ? v : -INFINITY;
    tm = fmaxf(tm, in ? v : -INFINITY);
  }
  if (!a.t_lse) {  // log of the sum over the listed entries
    if (holds) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) tm = fmaxf(tm, __shfl_xor_sync(0xffffffffu, tm, o));
    }
    if (lane == 0) s.top[warp].x = tm;
    __syncthreads();
    for (int w = 0; w < used; ++w) tm = fmaxf(tm, s.top[w].x);
    float sp = 0.f;
    for (int k = threadIdx.x; k < a.K; k += NT) sp += exp2f(log2_weight(e.lp[k], tm, a.c));
    if (holds) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sp += __shfl_xor_sync(0xffffffffu, sp, o);
    }
    if (lane == 0) s.warp[warp].x = sp;
    __syncthreads();
    sp = 0.f;
    for (int w = 0; w < used; ++w) sp += s.warp[w].x;
    lt = logf(sp);
  }
  // ln p_k = t_k / T - Lt, to twice a float's digits: where t_lse is given, p_r is
  // a difference from one.  The probabilities' sum is an integer sum for the
  // same reason.  Without t_lse both are taken relative to the largest t_k.
  const float base = a.t_lse ? 0.f : tm;
  uint64_t fixed = 0;
  for (int k = threadIdx.x; k < a.K; k += NT) {
    const float v = e.lp[k];
    const Pair y = two_sum(v, -base), x = over_t(a, y.hi), d = two_sum(x.hi, -lt);
    Pair lp{v > -INFINITY ? d.hi : v, 0.f};
    // (the low parts are as large as the difference where t / T and t_lse are far out)
    if (lp.hi > -INFINITY) lp = two_sum(d.hi, d.lo + fmaf(y.lo, a.inv_hi, x.lo));
    float p = expf(lp.hi);
    p = fmaf(p, lp.lo, p);
    if (!(p <= kMostP)) flags |= kDevBadParam;
    e.lp[k] = lp.hi;
    e.p[k] = p;
    fixed += __float2ull_rn(p * kMassOne);
  }
  if (holds) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) fixed += __shfl_xor_sync(0xffffffffu, fixed, o);
  }
  if (lane == 0) s.mass[warp] = fixed;
  if (tm > -INFINITY) flags |= kSome | (fabsf(lt) < INFINITY ? 0 : kDevBadParam);
  if (flags) atomicOr(&s.flags, flags);
  __syncthreads();
  Teacher t;
  t.flags = s.flags;
  fixed = 0;
  for (int w = 0; w < used; ++w) fixed += s.mass[w];
  // in units of 2^-40: one minus the sum, exactly
  const int64_t rest = (static_cast<int64_t>(1) << 40) - static_cast<int64_t>(fixed);
  t.mass = static_cast<float>(fixed) * (1.f / kMassOne);
  t.pr = a.t_lse && rest > 0 ? static_cast<float>(rest) * (1.f / kMassOne) : 0.f;
  t.faint = t.pr <= kFaintRest * (1.f + fabsf(lt));
  return t;
}

// The maxima of a part: of its entries outside S, whose maximum over this
// thread's is `top`, and of its listed ones.
template <int NW>
__device__ __forceinline__ float2 part_tops(int K, float top, Entries e, Shared<NW>& s) {
  float l = -INFINITY;
  for (int k = threadIdx.x; k < K; k += NW * 32)
    if (e.at[k] >= 0) l = fmaxf(l, e.z[k]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    l = fmaxf(l, __shfl_xor_sync(0xffffffffu, l, o));
  }
  if ((threadIdx.x & 31) == 0) s.top[threadIdx.x >> 5] = make_float2(top, l);
  __syncthreads();
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    const float2 v = s.top[w];
    top = fmaxf(top, v.x);
    l = fmaxf(l, v.y);
  }
  return make_float2(top, l);
}

// Adds up a part (`sum`: this thread's outside S) and sends it to every CTA of
// the cluster; complete after a cluster barrier.
template <int NW>
__device__ __forceinline__ void send_part(const DistillArgs& a, float2 tops, float sum, int flags, Entries e,
                                          Shared<NW>& s, int part, int parts) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float4 v = make_float4(sum, 0.f, 0.f, 0.f);  // sum, lsum, self, p
  for (int k = threadIdx.x; k < a.K; k += NW * 32) {
    if (e.at[k] < 0) continue;
    const float z = e.z[k], p = e.p[k];
    const float x = z == -INFINITY ? z : log2_weight(z, tops.y, a.c);
    v.y += exp2f(x);
    if (p > 0.f) v.z += p * (e.lp[k] - x * kLn2);
    v.w += p;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
  if (warp * 32 < a.K) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
      v.z += __shfl_xor_sync(0xffffffffu, v.z, o);
      v.w += __shfl_xor_sync(0xffffffffu, v.w, o);
    }
  }
  if (lane == 0) s.warp[warp] = v;
  __syncthreads();
  if (warp == 0) {
    v = lane < NW ? s.warp[lane] : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
      v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
      v.z += __shfl_xor_sync(0xffffffffu, v.z, o);
      v.w += __shfl_xor_sync(0xffffffffu, v.w, o);
    }
    if (lane < parts) *peer(&s.part[part], lane) = PartSums{tops.x, v.x, tops.y, v.y, v.z, v.w, flags};
  }
}

// What the row's gradient needs: maximum and sum of 2^((z - maximum) c) over the
// row (m, E) and outside S (mr, Er).  E = 0 stands for a row without a gradient.
struct RowSums {
  float m, E, mr, Er;
};

// p_r where it counts: a faint one meets no q_r below fp32's range, of a row whose
// unmasked tokens are all listed, say.  It would weigh ln q_r, as large as
// the mask is low, or infinite, by a rounding.
__device__ __forceinline__ float rest_of(const DistillArgs& a, const RowSums& r, const Teacher& t) {
  if (!t.faint) return t.pr;
  return log2f(r.Er) + log2_weight(r.mr, r.m, a.c) - log2f(r.E) < -126.f ? 0.f : t.pr;
}

// What the gradient pass needs of a row of weight w whose rest counts pr, worked
// out once per CTA.
template <int NW>
__device__ __forceinline__ void make_plan(const DistillArgs& a, Shared<NW>& s, const RowSums& r, const Teacher& t, float w, float pr) {
  const float g = w * a.inv_hi;
  s.plan.zero = r.E == 0.f;
  s.plan.g = g;
  s.plan.mr = r.mr;
  s.plan.m = r.m;
  const float P = t.mass + pr;
  s.plan.in = P / r.E;
  // factor of the weights outside S, in the form of with_weight
  const float f = r.Er > 0.f ? g * (P * exp2f(log2_weight(r.mr, r.m, a.c)) / r.E - pr / r.Er) : 0.f;
  s.plan.f = f * exp2f(lead(r.mr, a.c));
}

// Joins the parts, in rank order, makes the plan and, in the row's first CTA,
// writes the loss (the first warp).
template <int NW>
__device__ __forceinline__ void join_parts(const DistillArgs& a, int64_t row, const Teacher& t, float w,
                                           Shared<NW>& s, int part, int parts) {
  const int lane = threadIdx.x & 31;
  const PartSums q = lane < parts ? s.part[lane] : PartSums{-INFINITY, 0.f, -INFINITY, 0.f, 0.f, 0.f, 0};
  const int bad = reasons(__reduce_or_sync(0xffffffffu, q.flags), w);
  RowSums r;
  r.mr = q.top;
  r.m = fmaxf(q.top, q.ltop);
#pragma unroll
  for (int o = kMaxCluster / 2; o > 0; o >>= 1) {
    r.mr = fmaxf(r.mr, __shfl_xor_sync(0xffffffffu, r.mr, o));
    r.m = fmaxf(r.m, __shfl_xor_sync(0xffffffffu, r.m, o));
  }
  r.Er = q.sum * exp2f(log2_weight(q.top, r.mr, a.c));
  r.E = q.sum * exp2f(log2_weight(q.top, r.m, a.c)) + q.lsum * exp2f(log2_weight(q.ltop, r.m, a.c));
#pragma unroll
  for (int o = kMaxCluster / 2; o > 0; o >>= 1) {
    r.Er += __shfl_xor_sync(0xffffffffu, r.Er, o);
    r.E += __shfl_xor_sync(0xffffffffu, r.E, o);
  }
  if (r.E == 0.f) r.E = NAN;  // a row without any finite logit has no distribution
  const float log_e = log2f(r.E);
  // sum p (ln p - ln q), ln q = (z - m) / T - ln E
  float l = q.p > 0.f ? q.self + q.p * (log_e - log2_weight(q.ltop, r.m, a.c)) * kLn2 : 0.f;
#pragma unroll
  for (int o = kMaxCluster / 2; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  if (lane != 0) return;
  const float pr = rest_of(a, r, t);
  const bool out = bad || w == 0.f || !(t.flags & kSome);
  if (part == 0) {
    if (pr > 0.f) l += pr * (logf(pr) - (log2f(r.Er) + log2_weight(r.mr, r.m, a.c) - log_e) * kLn2);
    a.loss[row] = out ? (bad ? NAN : 0.f) : w * l;
    if (a.stats) a.stats[row] = out ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(r.m, r.E, r.mr, r.Er);
    if (bad) atomicOr(a.status, bad);
  }
  if (out) r.E = 0.f;
  make_plan(a, s, r, t, w, pr);
}

// Gradients of the part's listed entries; out: its first entry's.
template <typename T, int NT>
__device__ __forceinline__ void listed_gradients(const DistillArgs& a, const Shared<NT / 32>& s, T* out, Entries e) {
  const float f = s.plan.in, g = s.plan.g, m = s.plan.m;
  for (int k = threadIdx.x; k < a.K; k += NT) {
    const int i = e.at[k];
    if (i >= 0) out[i] = from_f32<T>(g * (f * exp2f(log2_weight(e.z[k], m, a.c)) - e.p[k]));
  }
}

constexpr int kFlight = 3;  // packs a thread loads at a time

// The listed elements of pack j become -inf.
template <typename T>
__device__ __forceinline__ void mask_listed(const uint32_t* bits, int j, uint4& w) {
  constexpr int kE = Part<T>::kE;
  const uint32_t byte = reinterpret_cast<const uint8_t*>(bits)[kE == 8 ? j : j >> 1];
  const uint32_t m = kE == 8 ? byte : byte >> (4 * (j & 1)) & 15;
  if (m == 0) return;
  uint32_t in[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int h = 0; h < kE; ++h) {
    constexpr int kPer = Pack<T>::kPer;
    if (!(m >> h & 1)) continue;
    const uint32_t lane = kPer == 1 ? 0xFFFFFFFFu : (h & 1 ? 0xFFFF0000u : 0xFFFFu);
    in[h / kPer] = (in[h / kPer] & ~lane) | (Pack<T>::kNegInf & lane);
  }
  w = make_uint4(in[0], in[1], in[2], in[3]);
}

// Writes f(entry) of a part to dz, in 16-byte packs of the destination.  Where
// those do not line up with the row's, each is cut out of two of them: the
// distance is the same for the whole part.
template <typename T, int NT, typename F>
__device__ __forceinline__ void write_part(const Part<T>& q, T* dz, F f) {
  constexpr int kPer = Pack<T>::kPer, kE = Part<T>::kE;
  T* out = dz + q.first;  // entry 0 of the part
  const int phase = static_cast<int>((reinterpret_cast<uintptr_t>(out) & 15) / sizeof(T));
  // destination pack j holds entries j kE - phase ..., which start `shift`
  // elements into the row's pack j + back
  const int delta = q.off - phase, back = delta < 0 ? -1 : 0, shift = delta < 0 ? delta + kE : delta;
  const int packs = (phase + q.n + kE - 1) / kE;
  T* dst = out - phase;
  auto put = [&](int j, const uint32_t* in, bool inside) {
    uint32_t o[4];
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      float t[kPer];
      Pack<T>::open(in[w], t);
#pragma unroll
      for (int h = 0; h < kPer; ++h) t[h] = f(t[h]);
      o[w] = Pack<T>::close(t);
    }
    if (inside) {
      __stcs(reinterpret_cast<uint4*>(dst) + j, make_uint4(o[0], o[1], o[2], o[3]));
      return;
    }
    const int e0 = j * kE - phase;
#pragma unroll
    for (int h = 0; h < kE; ++h) {
      const uint32_t word = o[h / kPer];
      if (e0 + h < 0 || e0 + h >= q.n) continue;
      if (kPer == 1)
        reinterpret_cast<uint32_t*>(out)[e0 + h] = word;
      else
        reinterpret_cast<uint16_t*>(out)[e0 + h] = static_cast<uint16_t>(h & 1 ? word >> 16 : word);
    }
  };
  if (shift == 0) {
    for (int j = threadIdx.x; j < packs; j += kFlight * NT) {
      uint4 v[kFlight];
      q.template load<kFlight, true>(j, NT, v);
      if (j + (kFlight - 1) * NT + 1 < packs && (j > 0 || phase == 0)) {
#pragma unroll
        for (int x = 0; x < kFlight; ++x) {
          const uint32_t in[4] = {v[x].x, v[x].y, v[x].z, v[x].w};
          put(j + x * NT, in, true);
        }
      } else {
#pragma unroll 1
        for (int x = 0; x < kFlight; ++x) {
          const uint4 y = q.template pack<true>(j + x * NT);
          const uint32_t in[4] = {y.x, y.y, y.z, y.w};
          const int e0 = (j + x * NT) * kE - phase;
          if (j + x * NT < packs) put(j + x * NT, in, e0 >= 0 && e0 + kE <= q.n);
        }
      }
    }
    return;
  }
  const int words = shift / kPer;
  for (int j = threadIdx.x; j < packs; j += 2 * NT) {
    uint4 v[2][2];
#pragma unroll
    for (int x = 0; x < 2; ++x) q.template load<2>(j + x * NT + back, 1, v[x]);
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      uint32_t in[8] = {v[x][0].x, v[x][0].y, v[x][0].z, v[x][0].w, v[x][1].x, v[x][1].y, v[x][1].z, v[x][1].w};
      if (words & 2) {
#pragma unroll
        for (int w = 0; w < 6; ++w) in[w] = in[w + 2];
      }
      if (words & 1) {
#pragma unroll
        for (int w = 0; w < 5; ++w) in[w] = in[w + 1];
      }
      if (kPer == 2 && (shift & 1)) {
#pragma unroll
        for (int w = 0; w < 4; ++w) in[w] = __byte_perm(in[w], in[w + 1], 0x5432);
      }
      const int e0 = (j + x * NT) * kE - phase;
      if (j + x * NT < packs) put(j + x * NT, in, e0 >= 0 && e0 + kE <= q.n);
    }
  }
}

// A row by a cluster of `parts` CTAs, or in the backward call, where the sums
// are given, by `parts` CTAs that need nothing of one another.
template <typename T, int NT, bool kBackward>
__global__ void __launch_bounds__(NT, NT == 256 ? 5 : 1) distill_kernel(const DistillArgs a, const int parts) {
  constexpr int NW = NT / 32, kE = Part<T>::kE;
  extern __shared__ __align__(16) uint8_t raw[];
  Shared<NW>& s = *reinterpret_cast<Shared<NW>*>(raw);
  const Entries e = entries_at(raw + sizeof(Shared<NW>), a.K);
  uint32_t* bits = reinterpret_cast<uint32_t*>(raw + sizeof(Shared<NW>) + entries_bytes(a.K));
  const int64_t row = blockIdx.x >> (31 - __clz(parts));
  const int part = static_cast<int>(blockIdx.x & (parts - 1));
  T* dz = a.dlogits ? static_cast<T*>(a.dlogits) + row * a.ldd : nullptr;
  Part<T> q;
  q.cut(static_cast<const T*>(a.logits) + row * a.ld, a.V, part, parts);
  pdl_wait();
  uint4 v[kFlight];  // the first packs are on their way while the entries are read
  if (!kBackward) q.template load<kFlight>(threadIdx.x, NT, v);
  constexpr int kSlack = kFlight * NT * kE / 8;  // bytes
  for (int i = threadIdx.x; i < (q.off + q.n + 31) / 32 + kSlack / 4; i += NT) bits[i] = 0;
  if (threadIdx.x == 0) s.flags = 0;
  const float w = a.weight ? a.weight[row] : 1.f;
  __syncthreads();
  if (!kBackward && parts > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  const Teacher t = read_teacher<T, NT>(a, row, q, e, bits, s);
  if (!kBackward) {
    // the sum relative to this thread's maximum, which it follows, then to the
    // part's
    float top = -INFINITY, ref = 0.f, sum = 0.f;
    for (int j = threadIdx.x; j < q.packs; j += kFlight * NT) {
#pragma unroll
      for (int x = 0; x < kFlight; ++x) mask_listed<T>(bits, j + x * NT, v[x]);
      uint32_t mx = Part<T>::max_words(v[0]);
#pragma unroll
      for (int x = 1; x < kFlight; ++x) mx = Pack<T>::max2(mx, Part<T>::max_words(v[x]));
      const float m = Part<T>::max_of(mx);
      if (m > top) {
        const float next = reference(m, a.c);
        if (top > -INFINITY)
          sum *= fast_exp2(is_near(ref) && is_near(next)
                               ? ref - next
                               : log2_weight(top, m, a.c) + (lead(top, a.c) - lead(m, a.c)));
        ref = next;
        top = m;
      }
      with_weight(a.c, ref, top, [&](auto weight) {
#pragma unroll
        for (int x = 0; x < kFlight; ++x) {
          float z[kE], some = 0.f;
          Part<T>::open(v[x], z);
#pragma unroll
          for (int h = 0; h < kE; ++h) some += weight(z[h]);
          sum += some;
        }
      });
      q.template load<kFlight>(j + kFlight * NT, NT, v);
    }
    const float2 tops = part_tops<NW>(a.K, top, e, s);
    if (top > -INFINITY) sum *= fast_exp2(log2_weight(top, tops.x, a.c) + lead(top, a.c));
    if (parts > 1) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");  // the other CTAs have started
    send_part<NW>(a, tops, sum, t.flags, e, s, part, parts);
    cluster_sync_all(parts);
    if (threadIdx.x < 32) join_parts<NW>(a, row, t, w, s, part, parts);
    if (!dz) return;
  } else if (threadIdx.x == 0) {
    const int bad = reasons(t.flags, w);
    if (bad) atomicOr(a.status, bad);
    const float4 st = a.stats[row];
    const RowSums r{st.x, bad || w == 0.f ? 0.f : st.y, st.z, st.w};
    make_plan(a, s, r, t, w, rest_of(a, r, t));
  }
  __syncthreads();
  if (s.plan.zero) {  // left out or refused
    write_part<T, NT>(q, dz, [](float) { return 0.f; });
    return;
  }
  const float f = s.plan.f;
  with_weight(a.c, reference(s.plan.mr, a.c), s.plan.mr, [&](auto weight) {
    write_part<T, NT>(q, dz, [=](float z) { return f * weight(z); });
  });
  __syncthreads();
  listed_gradients<T, NT>(a, s, dz + q.first, e);
}

template <typename T, int NT, bool kBackward>
cudaError_t launch_kernel(const DistillArgs& a, int64_t rows, int parts, cudaStream_t st) {
  const int64_t most = a.V / parts + 2 * Part<T>::kE;
  const size_t smem = sizeof(Shared<NT / 32>) + entries_bytes(a.K) + bitmap_bytes(most, kFlight * NT * Part<T>::kE / 8);
  const void* kern = (const void*)distill_kernel<T, NT, kBackward>;
  if (smem > 48 * 1024) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  DistillArgs b = a;
  void* args[] = {&b, &parts};
  return launch_kc(kern, dim3((unsigned)(rows * parts)), dim3(NT), smem, st, true, dim3(kBackward ? 1 : parts), args);
}

template <typename T>
cudaError_t launch(const DistillArgs& a, int64_t rows, bool backward, cudaStream_t st) {
  // Loss with gradient: parts of at most 80 KB keep what the GPU's CTAs read
  // twice well inside L2 (2048 x 151936 bf16: 347 / 264 / 270 / 293 us at 40 / 80 /
  // 160 / 320 KB).  One pass alone wants few CTAs a row (loss: 231 / 159 / 131 / 120
  // us).  Rows that do not fill the GPU are cut further.
  const int64_t most = (backward || !a.dlogits ? 320 : 80) * 1024;
  int parts = 1;
  while (parts < kMaxCluster && (a.V * (int64_t)sizeof(T) / parts > most ||
                                 (rows * parts < 2 * num_sms() && a.V * (int64_t)sizeof(T) / (2 * parts) >= 4096)))
    parts *= 2;
  // few rows: one large CTA an SM, whose threads have little to do one after
  // another (15 x 151936 fp32: 12.1 us, with 256 threads 14.6)
  if (rows * parts <= num_sms())
    return backward ? launch_kernel<T, 1024, true>(a, rows, parts, st)
                    : launch_kernel<T, 1024, false>(a, rows, parts, st);
  return backward ? launch_kernel<T, 256, true>(a, rows, parts, st)
                  : launch_kernel<T, 256, false>(a, rows, parts, st);
}

}  // namespace

cudaError_t distill(DistillArgs a, int dtype, int64_t rows, bool backward, cudaStream_t st) {
  a.c = static_cast<float>(1.4426950408889634 / static_cast<double>(a.T));
  const double inv = 1.0 / static_cast<double>(a.T);
  a.inv_hi = static_cast<float>(inv);
  a.inv_lo = static_cast<float>(inv - static_cast<double>(a.inv_hi));
  if (dtype == 0) return launch<float>(a, rows, backward, st);
  if (dtype == 1) return launch<__half>(a, rows, backward, st);
  return launch<__nv_bfloat16>(a, rows, backward, st);
}

}  // namespace dfl
