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
// puts nearly everything on S.  Entries of S are found through a bitmap of
// the CTA's slice, which also shows a token listed twice.
//
// Bound by HBM: the row is read, and its gradient written.
#include "kernels.h"
#include "rows.cuh"

namespace dfl {

namespace {

constexpr int kThr = 512;
constexpr int kWarps = kThr / 32;
constexpr int kDevBadToken = 0x2;
constexpr double kMassOne = 1099511627776.0;  // 2^40: probabilities are summed as integers

struct Shared {
  Exchange<kWarps> x;
  float p[kDistillMaxK];    // the teacher's logits, then log-probabilities
  float pk[kDistillMaxK];   // its probabilities
  float z[kDistillMaxK];    // the student's logits at its tokens
  int at[kDistillMaxK];     // their tokens, -1: no entry
  float red[2][kWarps];
};

// Sum of a float over the CTA in a fixed order (every thread gets it).
__device__ __forceinline__ float cta_sum(float v, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.f;
  for (int w = 0; w < kWarps; ++w) v += red[w];
  __syncthreads();
  return v;
}
__device__ __forceinline__ float cta_max(float v, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = red[0];
  for (int w = 1; w < kWarps; ++w) v = fmaxf(v, red[w]);
  __syncthreads();
  return v;
}

// Sum of a float over the cluster, CTAs in rank order.
__device__ __forceinline__ float cluster_sum(float v, Shared& s, uint32_t rank, uint32_t size, int& turn) {
  v = cta_sum(v, s.red[0]);
  const int k = turn % 3;
  ++turn;
  if (threadIdx.x < size) *peer(&s.x.slot[k][rank], threadIdx.x) = __float_as_uint(v);
  cluster_sync_all(size);
  v = 0.f;
  for (uint32_t r = 0; r < size; ++r) v += __uint_as_float(static_cast<uint32_t>(s.x.slot[k][r]));
  return v;
}

// exp((v - m) / T) for v <= m
__device__ __forceinline__ float exp_diff(float v, float m, InvT c) { return exp2f(log2_weight(v, m, c)); }

template <typename T>
__global__ void __launch_bounds__(kThr) distill_kernel(const DistillArgs a, const bool backward) {
  extern __shared__ __align__(16) uint8_t raw[];
  Shared& s = *reinterpret_cast<Shared*>(raw);
  uint32_t* bits = reinterpret_cast<uint32_t*>(raw + sizeof(Shared));  // slice entries in S
  pdl_wait();
  const uint32_t rank = cluster_rank(), size = cluster_size();
  const int64_t row = blockIdx.x / size;
  const T* z = static_cast<const T*>(a.logits) + row * a.ld;
  T* dz = a.dlogits ? static_cast<T*>(a.dlogits) + row * a.ldd : nullptr;
  const int64_t chunk = (a.V + size - 1) / size;
  const int64_t c0 = chunk * rank < a.V ? chunk * rank : a.V, c1 = c0 + chunk < a.V ? c0 + chunk : a.V;
  int turn = 0;
  const float w = a.weight ? a.weight[row] : 1.f;

  // the teacher's entries: every CTA of the cluster reads them all
  for (int64_t i = threadIdx.x; i < (c1 - c0 + 31) / 32; i += kThr) bits[i] = 0;
  __syncthreads();
  bool bad = false;
  float tm = -INFINITY;
  for (int k = threadIdx.x; k < a.K; k += kThr) {
    const int i = a.t_idx[row * a.K + k];
    const float t = a.t_val[row * a.K + k];
    int at = -1;
    if (i >= 0 && i < a.V) {
      at = i;
      if (i >= c0 && i < c1) {
        const uint32_t bit = 1u << ((i - c0) & 31);
        bad |= (atomicOr(&bits[(i - c0) >> 5], bit) & bit) != 0;
      }
    } else if (i != -1) {
      bad = true;
    }
    s.at[k] = at;
    s.p[k] = at >= 0 ? t : -INFINITY;
    s.z[k] = at >= 0 ? to_f32(z[at]) : -INFINITY;
    tm = fmaxf(tm, s.p[k]);
  }
  cluster_sync_all(size);
  bad = cluster_reduce<kWarps>(bad, OpMaxU64(), s.x, rank, size, turn) != 0;
  tm = cta_max(tm, s.red[0]);
  if (bad || w == 0.f || tm == -INFINITY) {
    // a row left out (or refused): no gradient
    if (rank == 0 && threadIdx.x == 0) {
      if (a.loss) a.loss[row] = bad ? NAN : 0.f;
      if (!backward && a.stats) a.stats[row] = make_float4(0.f, 1.f, 0.f, 1.f);
      if (bad) atomicOr(a.status, kDevBadToken);
    }
    if (dz)
      for (int64_t i = c0 + threadIdx.x; i < c1; i += kThr) dz[i] = from_f32<T>(0.f);
    return;  // the last access to other CTAs was before the reduction's barrier
  }

  const double inv_t = 1.0 / static_cast<double>(a.T);
  const InvT c = inv_temperature(a.T);
  float sp = 0.f, zm = -INFINITY;
  for (int k = threadIdx.x; k < a.K; k += kThr) {
    sp += a.t_lse ? 0.f : exp_diff(s.p[k], tm, c);
    zm = fmaxf(zm, s.z[k]);
  }
  sp = cta_sum(sp, s.red[0]);
  // ln p_k = t_k / T - Lt, formed in double: where t_lse is given, p_r is a
  // difference from one.  The probabilities' sum is an integer sum for the
  // same reason.
  const double lt = a.t_lse ? static_cast<double>(a.t_lse[row])
                            : static_cast<double>(tm) * inv_t + static_cast<double>(logf(sp));
  uint64_t fixed = 0;
  for (int k = threadIdx.x; k < a.K; k += kThr) {
    const double lp = static_cast<double>(s.p[k]) * inv_t - lt;
    const float hi = static_cast<float>(lp);
    float p = expf(hi);
    if (hi > -INFINITY) p = fmaf(p, static_cast<float>(lp - static_cast<double>(hi)), p);
    s.p[k] = hi;
    s.pk[k] = p;
    fixed += __float2ull_rn(fminf(p, 256.f) * static_cast<float>(kMassOne));
  }
  fixed = cta_reduce<kWarps>(fixed, OpSumU64(), s.x);
  const double total = static_cast<double>(fixed) / kMassOne;
  const float mass = static_cast<float>(total);
  const float pr = a.t_lse && total < 1.0 ? static_cast<float>(1.0 - total) : 0.f;
  const float P = mass + pr;

  float m, E, mr, Er;
  if (!backward) {
    // maximum and exponential sum outside S
    float v = -INFINITY;
    for (int64_t i = c0 + threadIdx.x; i < c1; i += kThr)
      if (!(bits[(i - c0) >> 5] >> ((i - c0) & 31) & 1)) v = fmaxf(v, to_f32(z[i]));
    v = cta_max(v, s.red[0]);
    mr = key_to_value(static_cast<uint32_t>(
        cluster_reduce<kWarps>(max(value_key(v), 0x007FFFFFu), OpMaxU64(), s.x, rank, size, turn)));
    float e = 0.f;
    for (int64_t i = c0 + threadIdx.x; i < c1; i += kThr)
      if (!(bits[(i - c0) >> 5] >> ((i - c0) & 31) & 1)) e += exp_diff(to_f32(z[i]), mr, c);
    Er = cluster_sum(mr == -INFINITY ? 0.f : e, s, rank, size, turn);
    // and over the whole row
    zm = cta_max(zm, s.red[0]);
    m = fmaxf(zm, mr);
    e = 0.f;
    for (int k = threadIdx.x; k < a.K; k += kThr)
      if (s.at[k] >= 0) e += exp_diff(s.z[k], m, c);
    // a row without any finite logit has no distribution
    E = m == -INFINITY ? NAN : cta_sum(e, s.red[0]) + (mr == -INFINITY ? 0.f : Er * exp_diff(mr, m, c));
    if (rank == 0) {
      const float log_e = logf(E);
      float l = 0.f;
      for (int k = threadIdx.x; k < a.K; k += kThr) {
        const float lp = s.p[k];
        if (lp > -INFINITY) l += s.pk[k] * (lp - ((s.z[k] - m) / a.T - log_e));
      }
      l = cta_sum(l, s.red[0]);
      if (pr > 0.f) l += pr * (logf(pr) - ((mr - m) / a.T + logf(Er) - log_e));
      if (threadIdx.x == 0) {
        a.loss[row] = w * l;
        if (a.stats) a.stats[row] = make_float4(m, E, mr, Er);
      }
    }
  } else {
    const float4 st = a.stats[row];
    m = st.x;
    E = st.y;
    mr = st.z;
    Er = st.w;
  }
  if (dz) {
    const float g = w / a.T;
    const float out = Er > 0.f ? g * (P * exp_diff(mr, m, c) / E - pr / Er) : 0.f;
    for (int64_t i = c0 + threadIdx.x; i < c1; i += kThr)
      if (!(bits[(i - c0) >> 5] >> ((i - c0) & 31) & 1)) dz[i] = from_f32<T>(out * exp_diff(to_f32(z[i]), mr, c));
    for (int k = threadIdx.x; k < a.K; k += kThr) {
      const int i = s.at[k];
      if (i >= c0 && i < c1) dz[i] = from_f32<T>(g * (P * exp_diff(s.z[k], m, c) / E - s.pk[k]));
    }
  }
}

template <typename T>
cudaError_t launch(const DistillArgs& a, int64_t rows, bool backward, cudaStream_t st) {
  int c = 1;
  while (c < kMaxCluster && rows * c < 2 * num_sms() && a.V / (2 * c) >= 2048) c *= 2;
  // the bitmap of a slice fits beside the entries
  while (c < kMaxCluster && (a.V + c - 1) / c > (int64_t)8 * 160 * 1024) c *= 2;
  const size_t smem = sizeof(Shared) + (size_t)(((a.V + c - 1) / c + 31) / 32) * 4;
  cudaError_t e = cudaFuncSetAttribute((const void*)distill_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)smem);
  if (e != cudaSuccess) return e;
  DistillArgs b = a;
  void* args[] = {&b, &backward};
  return launch_kc((const void*)distill_kernel<T>, dim3((unsigned)(rows * c)), dim3(kThr), smem, st, true, dim3(c),
                   args);
}

}  // namespace

cudaError_t distill(const DistillArgs& a, int dtype, int64_t rows, bool backward, cudaStream_t st) {
  if (dtype == 0) return launch<float>(a, rows, backward, st);
  if (dtype == 1) return launch<__half>(a, rows, backward, st);
  return launch<__nv_bfloat16>(a, rows, backward, st);
}

}  // namespace dfl
