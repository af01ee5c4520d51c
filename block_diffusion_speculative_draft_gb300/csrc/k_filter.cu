// k_filter.cu — filtered sampling over rows of vocabulary logits: one token a
// row, the speculative accept under the same filters, and a row's K largest
// logits with its log-sum-exp.
//
// A row z[0..V) with temperature T: masked entries (NaN, -inf) never count,
//   w_v = exp((z_v - max z) / T);  order: z descending, index ascending;
//   top-k keeps the first k of the order, top-p of those each entry whose
//   predecessors sum to less than p times what top-k kept (the first always),
//   min-p of those the entries with z_v >= max z + T ln(min_p);
//   P(v) = w_v / (sum of the kept w).
// What is kept is always a prefix of the order, so a row's filters reduce to
// one 64-bit cut (value key, complemented index): an entry is kept iff its
// place is at or above the cut.  The token is the Gumbel maximum
// argmax (z_v - max z)/T - log(-log u_v) over the kept entries.
//
// Weights are summed as 64-bit integers (w scaled by a power of two that
// keeps V of them below 2^62): the sums do not depend on the order of the
// additions, so the cut and every result repeat bit for bit; the rounding of
// one weight, 2^-45 of the largest at V = 152 k, is far below the 2^-23 of
// its exponential.
#include "kernels.h"
#include "rows.cuh"

namespace dfl {

namespace {

constexpr int kThr = 512;
constexpr int kWarps = kThr / 32;
constexpr int kBins = 2048;
constexpr int kDevBadParam = 0x8;

// What one row asks for.
struct Ask {
  float T;
  int k;      // V: no bound
  float p;    // 1: off
  float mp;   // 0: off
  bool ok, greedy;
};

__device__ __forceinline__ Ask read_ask(const FilterArgs& a, int64_t i) {
  Ask q;
  q.T = a.temperature ? a.temperature[i] : a.T;
  q.k = a.top_k ? a.top_k[i] : 0;
  q.p = a.top_p ? a.top_p[i] : 1.f;
  q.mp = a.min_p ? a.min_p[i] : 0.f;
  // comparisons that a NaN fails
  q.ok = (q.T == 0.f || (q.T >= kFilterMinT && q.T <= kFilterMaxT)) && q.k >= 0 && q.p >= 0.f && q.p <= 1.f &&
         q.mp >= 0.f && q.mp <= 1.f;
  q.greedy = q.T == 0.f;
  if (q.greedy) {
    q.T = 1.f;
    q.k = 1;
    q.p = 1.f;
    q.mp = 0.f;
  }
  if (q.k == 0 || q.k > a.V) q.k = static_cast<int>(a.V);
  return q;
}

struct Shared {
  Exchange<kWarps> x;
  unsigned long long mass[kBins];
  uint32_t count[kBins];
  uint64_t total[kMaxCluster];   // mass or count of each CTA's share of the bins
  uint64_t pick[4];              // the level's choice: bin, sum before it, its count, found
  uint64_t warp_sum[kWarps];
};

// One row as a cluster sees it.
template <typename T>
struct Row {
  const T* p;
  int64_t c0, c1;  // this CTA's slice
  uint32_t rank, size;
  float m;         // the row's maximum
  InvT c;
  float scale;       // weights become integers by this power of two
  int turn;

  __device__ __forceinline__ float at(int64_t i) const { return to_f32(p[i]); }
  __device__ __forceinline__ float log2w(float v) const { return log2_weight(v, m, c); }
  __device__ __forceinline__ unsigned long long weight(float v) const {
    return __float2ull_rn(exp2f(log2w(v)) * scale);
  }
};

// The place of the last entry kept when entries at or above `lo` are taken in
// order until the taken ones reach `need` (by count, or by weight): a radix
// descent over the places, 11 bits of the value key at a time and, where
// equal values straddle the border, over the index bits.  Each level is one
// pass over the row that adds every entry with the prefix found so far to its
// digit's bin.  need is in [1, sum over the entries at or above lo].
template <typename T, bool kMass>
__device__ uint64_t find_cut(Row<T>& r, Shared& s, uint64_t lo, uint64_t need, int idx_bits) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint64_t pre = 0;
  int top = 64;  // bits of the place above `top` are `pre`
  while (true) {
    int bits;
    if (top > 32) {
      bits = top == 64 ? 11 : (top == 53 ? 11 : 10);
    } else {
      if (top == 32) {  // the index bits above V are all ones
        pre = (pre << (32 - idx_bits)) | ((1ull << (32 - idx_bits)) - 1);
        top = idx_bits;
        if (top == 0) return pre;
      }
      bits = top < 11 ? top : 11;
    }
    const int shift = top - bits;
    for (int b = threadIdx.x; b < kBins; b += kThr) {
      s.count[b] = 0;
      s.mass[b] = 0;
    }
    __syncthreads();
    for (int64_t i = r.c0 + threadIdx.x; i < r.c1; i += kThr) {
      const float v = r.at(i);
      const uint32_t key = value_key(v);
      const uint64_t c = place_of(key, static_cast<uint32_t>(i));
      if (key == 0 || c < lo || (top < 64 && (c >> top) != pre)) continue;
      const int b = static_cast<int>((c >> shift) & ((1u << bits) - 1));
      atomicAdd(&s.count[b], 1u);
      if (kMass) atomicAdd(&s.mass[b], r.weight(v));
    }
    cluster_sync_all(r.size);
    // bins in falling order, cut into one contiguous share per CTA; a share's
    // bins are summed over the cluster, four per thread and warp-scanned
    const int share = kBins / static_cast<int>(r.size);
    uint64_t mine[kBins / kThr];
    uint32_t cnt[kBins / kThr];
    uint64_t sum = 0;
    const int per = (share + kThr - 1) / kThr;
#pragma unroll
    for (int q = 0; q < kBins / kThr; ++q) {
      mine[q] = 0;
      cnt[q] = 0;
      const int j = threadIdx.x * per + q;
      if (q < per && j < share) {
        const int b = kBins - 1 - (static_cast<int>(r.rank) * share + j);
        for (uint32_t o = 0; o < r.size; ++o) {
          cnt[q] += *peer(&s.count[b], o);
          if (kMass) mine[q] += *peer(&s.mass[b], o);
        }
        if (!kMass) mine[q] = cnt[q];
      }
      sum += mine[q];
    }
    uint64_t inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t u = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += u;
    }
    if (lane == 31) s.warp_sum[warp] = inc;
    __syncthreads();
    uint64_t before = inc - sum, all = 0;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += s.warp_sum[w];
      all += s.warp_sum[w];
    }
    if (threadIdx.x < r.size) *peer(&s.total[r.rank], threadIdx.x) = all;
    cluster_sync_all(r.size);
    for (uint32_t o = 0; o < r.rank; ++o) before += s.total[o];
#pragma unroll
    for (int q = 0; q < kBins / kThr; ++q) {
      if (before < need && before + mine[q] >= need) {
        const int b = kBins - 1 - (static_cast<int>(r.rank) * share + threadIdx.x * per + q);
        for (uint32_t o = 0; o < r.size; ++o) {
          uint64_t* pk = peer(s.pick, o);
          pk[0] = static_cast<uint64_t>(b);
          pk[1] = before;
          pk[2] = cnt[q];
        }
      }
      before += mine[q];
    }
    cluster_sync_all(r.size);
    const uint64_t b = s.pick[0];
    need -= s.pick[1];
    const uint64_t in_bin = s.pick[2];
    pre = (top < 64 ? pre << bits : 0) | b;
    top = shift;
    __syncthreads();  // pick is read before the next level writes it
    // the whole bin is taken, or it holds only the border entry
    if (top == 0 || in_bin == 1 || (!kMass && in_bin == need)) return pre << top;
  }
}

template <typename T>
__device__ uint64_t mass_from(Row<T>& r, Shared& s, uint64_t cut) {
  uint64_t w = 0;
  for (int64_t i = r.c0 + threadIdx.x; i < r.c1; i += kThr) {
    const float v = r.at(i);
    const uint32_t key = value_key(v);
    if (key != 0 && place_of(key, static_cast<uint32_t>(i)) >= cut) w += r.weight(v);
  }
  return cluster_reduce<kWarps>(w, OpSumU64(), s.x, r.rank, r.size, r.turn);
}

// Row set-up: slice, maximum, temperature.  False: no entry counts.
template <typename T>
__device__ bool open_row(Row<T>& r, Shared& s, const FilterArgs& a, int64_t row, float temp) {
  r.p = static_cast<const T*>(a.logits) + row * a.ld;
  r.rank = cluster_rank();
  r.size = cluster_size();
  const int64_t chunk = (a.V + r.size - 1) / r.size;
  r.c0 = chunk * r.rank < a.V ? chunk * r.rank : a.V;
  r.c1 = r.c0 + chunk < a.V ? r.c0 + chunk : a.V;
  r.turn = 0;
  r.scale = a.scale;
  r.c = inv_temperature(temp);
  uint32_t k = 0;
  for (int64_t i = r.c0 + threadIdx.x; i < r.c1; i += kThr) {
    const uint32_t q = value_key(r.at(i));
    k = q > k ? q : k;
  }
  cluster_sync_all(r.size);  // the other CTAs have started
  k = static_cast<uint32_t>(cluster_reduce<kWarps>(k, OpMaxU64(), s.x, r.rank, r.size, r.turn));
  r.m = key_to_value(k);
  return k != 0;
}

// The row's cut and the sum of the weights at or above it.
template <typename T>
__device__ uint64_t kept_cut(Row<T>& r, Shared& s, const FilterArgs& a, const Ask& q, uint64_t* kept_mass) {
  uint64_t cut = 1ull << 32;  // every unmasked entry
  uint64_t valid = 0;
  if (q.k < a.V) {
    for (int64_t i = r.c0 + threadIdx.x; i < r.c1; i += kThr) valid += value_key(r.at(i)) != 0;
    valid = cluster_reduce<kWarps>(valid, OpSumU64(), s.x, r.rank, r.size, r.turn);
    if (static_cast<uint64_t>(q.k) < valid) cut = find_cut<T, false>(r, s, cut, q.k, a.idx_bits);
  }
  uint64_t w = mass_from(r, s, cut);
  const uint64_t had = cut;
  if (q.p < 1.f) {
    // entries are taken while the sum before them is below p times w
    uint64_t need = static_cast<uint64_t>(ceil(static_cast<double>(q.p) * static_cast<double>(w)));
    if (need < 1) need = 1;
    if (need < w) cut = find_cut<T, true>(r, s, cut, need, a.idx_bits);
  }
  if (q.mp > 0.f) {
    const double t = static_cast<double>(r.m) + static_cast<double>(q.T) * log(static_cast<double>(q.mp));
    float f = static_cast<float>(t);
    if (static_cast<double>(f) < t) f = nextafterf(f, INFINITY);
    if (f > r.m) f = r.m;
    const uint64_t c = place_of(value_key(f), 0xFFFFFFFFu);
    if (c > cut) cut = c;
  }
  *kept_mass = cut == had ? w : mass_from(r, s, cut);
  return cut;
}

// Gumbel maximum over the kept entries but `drop`: decided in fp32, entries
// whose fp32 scores nearly tie again in double (the thread's own runner-up
// aside).  -1 when nothing is kept.
template <typename T>
__device__ int gumbel_pick(Row<T>& r, Shared& s, const float* u, uint64_t cut, int drop, float temp) {
  float best = 0.f;
  int at = -1;
  const float c = 0.6931471805599453f;
  for (int64_t i = r.c0 + threadIdx.x; i < r.c1; i += kThr) {
    const float v = r.at(i);
    const uint32_t key = value_key(v);
    if (key == 0 || place_of(key, static_cast<uint32_t>(i)) < cut || i == drop) continue;
    const float sc = r.log2w(v) * c - logf(-logf(u[i]));
    if (at < 0 || sc > best) {
      best = sc;
      at = static_cast<int>(i);
    }
  }
  const uint64_t k = at >= 0 ? argmax_key(best, static_cast<uint32_t>(at)) : 0ull;
  const uint64_t win = cluster_reduce<kWarps>(k, OpMaxU64(), s.x, r.rank, r.size, r.turn);
  if (win == 0) return -1;
  const float top = key_value(win);
  const bool close = at >= 0 && best >= top - (1e-5f + 1e-6f * fabsf(top));
  const uint64_t n = cluster_reduce<kWarps>(close, OpSumU64(), s.x, r.rank, r.size, r.turn);
  if (n <= 1) return static_cast<int>(key_index(win));
  double d = 0.0;
  if (close) {
    const float v = r.at(at);
    d = (v == r.m ? 0.0 : (static_cast<double>(v) - static_cast<double>(r.m)) / static_cast<double>(temp)) -
        log(-log(static_cast<double>(u[at])));
  }
  const uint64_t dk = close ? double_key(d) : 0ull;
  const uint64_t dbest = cluster_reduce<kWarps>(dk, OpMaxU64(), s.x, r.rank, r.size, r.turn);
  const uint64_t low = close && dk == dbest ? 0xFFFFFFFFull - static_cast<uint32_t>(at) : 0ull;
  return static_cast<int>(0xFFFFFFFFull -
                          cluster_reduce<kWarps>(low, OpMaxU64(), s.x, r.rank, r.size, r.turn));
}

template <typename T>
__device__ __forceinline__ float log_prob(const Row<T>& r, int tok, uint64_t kept) {
  return r.log2w(r.at(tok)) * 0.6931471805599453f - logf(static_cast<float>(kept) / r.scale);
}

template <typename T>
__global__ void __launch_bounds__(kThr) sample_rows_kernel(const FilterArgs a) {
  extern __shared__ __align__(16) uint8_t raw[];
  Shared& s = *reinterpret_cast<Shared*>(raw);
  pdl_wait();
  const int64_t row = blockIdx.x / cluster_size();
  const Ask q = read_ask(a, row);
  Row<T> r;
  const bool some = open_row(r, s, a, row, q.T);
  int tok = -1;
  float lp = -INFINITY;
  if (q.ok && some) {
    uint64_t kept;
    const uint64_t cut = kept_cut(r, s, a, q, &kept);
    tok = gumbel_pick(r, s, a.u + row * a.ld_u, cut, -1, q.T);
    lp = log_prob(r, tok, kept);
  }
  if (r.rank == 0 && threadIdx.x == 0) {
    a.tok[row] = tok;
    if (a.logprob) a.logprob[row] = lp;
    if (!q.ok) atomicOr(a.status, kDevBadParam);
  }
  cluster_sync_all(r.size);
}

// Verified row r of sequence j: its cut, and for r < D the probability of the
// draft token under the filters.
template <typename T>
__global__ void __launch_bounds__(kThr) accept_rows_kernel(const FilterArgs a) {
  extern __shared__ __align__(16) uint8_t raw[];
  Shared& s = *reinterpret_cast<Shared*>(raw);
  pdl_wait();
  const int64_t row = blockIdx.x / cluster_size();
  const int64_t j = row / a.R;
  const int rr = static_cast<int>(row - j * a.R);
  const Ask q = read_ask(a, j);
  Row<T> r;
  const bool some = open_row(r, s, a, row, q.T);
  RowCut out;
  out.cut = ~0ull;
  out.m = r.m;
  out.accept = 0;
  if (q.ok && some) {
    uint64_t kept;
    out.cut = kept_cut(r, s, a, q, &kept);
    if (rr < a.D) {
      const int x = a.draft[j * a.D + rr];
      if (x >= 0 && x < a.V) {
        const float v = r.at(x);
        const uint32_t key = value_key(v);
        if (key != 0 && place_of(key, static_cast<uint32_t>(x)) >= out.cut)
          out.accept = static_cast<double>(a.u_accept[j * a.D + rr]) <
                       static_cast<double>(r.weight(v)) / static_cast<double>(kept);
      }
    }
  }
  if (r.rank == 0 && threadIdx.x == 0) a.cuts[row] = out;
  cluster_sync_all(r.size);
}

// One cluster per sequence: leading accepts, the draw at the row after them
// and the outputs.
template <typename T>
__global__ void __launch_bounds__(kThr) accept_pick_kernel(const FilterArgs a) {
  extern __shared__ __align__(16) uint8_t raw[];
  Shared& s = *reinterpret_cast<Shared*>(raw);
  pdl_wait();
  const int64_t j = blockIdx.x / cluster_size();
  const Ask q = read_ask(a, j);
  int n = 0;
  while (n < a.D && a.cuts[j * a.R + n].accept) ++n;
  const int* dr = a.draft + j * a.D;
  int corr = -1;
  const uint32_t rank = cluster_rank(), size = cluster_size();
  cluster_sync_all(size);
  if (q.ok && n < a.R) {
    const int64_t row = j * a.R + n;
    const RowCut c = a.cuts[row];
    Row<T> r;
    r.p = static_cast<const T*>(a.logits) + row * a.ld;
    r.rank = rank;
    r.size = size;
    const int64_t chunk = (a.V + size - 1) / size;
    r.c0 = chunk * rank < a.V ? chunk * rank : a.V;
    r.c1 = r.c0 + chunk < a.V ? r.c0 + chunk : a.V;
    r.turn = 0;
    r.m = c.m;
    r.c = inv_temperature(q.T);
    corr = gumbel_pick(r, s, a.u + j * a.ld_u, c.cut, n < a.D ? dr[n] : -1, q.T);
  }
  if (rank == 0 && threadIdx.x == 0) {
    if (!q.ok) {
      n = -1;  // a commit of this length appends nothing
      atomicOr(a.status, kDevBadParam);
    }
    a.n_out[j] = n;
    a.corr_out[j] = corr;
    if (a.next_tok) a.next_tok[j] = corr >= 0 ? corr : (n > 0 ? dr[n - 1] : -1);
    if (a.emitted)
      for (int i = 0; i < a.R; ++i) a.emitted[j * a.R + i] = i < n ? dr[i] : (i == n ? corr : -1);
  }
  cluster_sync_all(size);
}

// The K first entries of the order, sorted, and the row's log-sum-exp.
constexpr int kListMax = kTopLogitsMax;

struct TopShared {
  Shared s;
  uint64_t list[kListMax];
  int n;
};

__device__ void bitonic_desc(uint64_t* list, int n) {  // n a power of two
  for (int k = 2; k <= n; k <<= 1)
    for (int j = k >> 1; j > 0; j >>= 1) {
      for (int i = threadIdx.x; i < n / 2; i += kThr) {
        const int lo = 2 * i - (i & (j - 1)), hi = lo + j;
        const uint64_t x = list[lo], y = list[hi];
        if ((x < y) == ((lo & k) == 0)) {
          list[lo] = y;
          list[hi] = x;
        }
      }
      __syncthreads();
    }
}

template <typename T>
__global__ void __launch_bounds__(kThr) top_rows_kernel(const FilterArgs a) {
  extern __shared__ __align__(16) uint8_t raw[];
  TopShared& t = *reinterpret_cast<TopShared*>(raw);
  Shared& s = t.s;
  pdl_wait();
  const int64_t row = blockIdx.x / cluster_size();
  Row<T> r;
  int np = 1;
  while (np < a.K) np <<= 1;
  for (int i = threadIdx.x; i < np; i += kThr) t.list[i] = 0;
  if (threadIdx.x == 0) t.n = 0;
  const bool some = open_row(r, s, a, row, a.T);
  uint64_t w = 0;
  if (some) {
    Ask q;
    q.T = a.T;
    q.k = a.K < a.V ? a.K : static_cast<int>(a.V);
    q.p = 1.f;
    q.mp = 0.f;
    uint64_t kept;
    const uint64_t cut = kept_cut(r, s, a, q, &kept);
    w = mass_from(r, s, 1ull << 32);
    int* n0 = peer(&t.n, 0);
    uint64_t* l0 = peer(t.list, 0);
    for (int64_t i = r.c0 + threadIdx.x; i < r.c1; i += kThr) {
      const uint32_t key = value_key(r.at(i));
      const uint64_t c = place_of(key, static_cast<uint32_t>(i));
      if (key != 0 && c >= cut) {
        const int at = atomicAdd(n0, 1);
        if (at < a.K) l0[at] = c;
      }
    }
  }
  cluster_sync_all(r.size);
  if (r.rank == 0) {
    if (np > 1) bitonic_desc(t.list, np);
    for (int i = threadIdx.x; i < a.K; i += kThr) {
      const uint64_t c = t.list[i];
      a.val[row * a.K + i] = c ? key_to_value(static_cast<uint32_t>(c >> 32)) : -INFINITY;
      a.idx[row * a.K + i] = c ? static_cast<int>(place_index(c)) : -1;
    }
    if (a.lse && threadIdx.x == 0)
      a.lse[row] = some ? static_cast<float>(static_cast<double>(r.m) / static_cast<double>(a.T) +
                                             static_cast<double>(logf(static_cast<float>(w) / r.scale)))
                        : -INFINITY;
  }
}

template <typename K>
cudaError_t launch_rows(K kern, int64_t rows, size_t smem, const FilterArgs& a, cudaStream_t st) {
  // enough CTAs to occupy the GPU, at least 2048 entries each
  int c = 1;
  while (c < kMaxCluster && rows * c < 2 * num_sms() && a.V / (2 * c) >= 2048) c *= 2;
  cudaError_t e = cudaFuncSetAttribute((const void*)kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  FilterArgs b = a;
  void* args[] = {&b};
  return launch_kc((const void*)kern, dim3((unsigned)(rows * c)), dim3(kThr), smem, st, true, dim3(c), args);
}

void finish(FilterArgs& a) {
  a.idx_bits = 0;
  while (((int64_t)1 << a.idx_bits) < a.V) ++a.idx_bits;
  a.scale = ldexpf(1.f, 62 - a.idx_bits);
}

}  // namespace

cudaError_t filter_sample(FilterArgs a, int dtype, int64_t rows, cudaStream_t st) {
  finish(a);
  if (dtype == 0) return launch_rows(sample_rows_kernel<float>, rows, sizeof(Shared), a, st);
  if (dtype == 1) return launch_rows(sample_rows_kernel<__half>, rows, sizeof(Shared), a, st);
  return launch_rows(sample_rows_kernel<__nv_bfloat16>, rows, sizeof(Shared), a, st);
}

cudaError_t filter_accept(FilterArgs a, int dtype, int64_t b, cudaStream_t st) {
  finish(a);
  const int64_t rows = b * a.R;
  cudaError_t e;
  if (dtype == 0) {
    if ((e = launch_rows(accept_rows_kernel<float>, rows, sizeof(Shared), a, st)) != cudaSuccess) return e;
    return launch_rows(accept_pick_kernel<float>, b, sizeof(Shared), a, st);
  }
  if (dtype == 1) {
    if ((e = launch_rows(accept_rows_kernel<__half>, rows, sizeof(Shared), a, st)) != cudaSuccess) return e;
    return launch_rows(accept_pick_kernel<__half>, b, sizeof(Shared), a, st);
  }
  if ((e = launch_rows(accept_rows_kernel<__nv_bfloat16>, rows, sizeof(Shared), a, st)) != cudaSuccess) return e;
  return launch_rows(accept_pick_kernel<__nv_bfloat16>, b, sizeof(Shared), a, st);
}

cudaError_t top_logits(FilterArgs a, int dtype, int64_t rows, cudaStream_t st) {
  finish(a);
  if (dtype == 0) return launch_rows(top_rows_kernel<float>, rows, sizeof(TopShared), a, st);
  if (dtype == 1) return launch_rows(top_rows_kernel<__half>, rows, sizeof(TopShared), a, st);
  return launch_rows(top_rows_kernel<__nv_bfloat16>, rows, sizeof(TopShared), a, st);
}

}  // namespace dfl
