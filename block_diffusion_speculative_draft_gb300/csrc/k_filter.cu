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

constexpr int kDigit = 9;             // bits of a place per level of the descent
constexpr int kBins = 1 << kDigit;
constexpr int kGroupBins = 256;       // bins of the threads' maxima
constexpr int kDevBadParam = 0x8;
constexpr int kFewTarget = 128;       // entries the short list aims at where top-k does not say
constexpr float kLn2 = 0.6931471805599453f;

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
  if (q.greedy || !q.ok) {
    q.T = 1.f;
    q.k = 1;
    q.p = 1.f;
    q.mp = 0.f;
  }
  if (q.k == 0 || q.k > a.V) q.k = static_cast<int>(a.V);
  return q;
}

// Shared memory of a CTA; the part of the row follows.
template <int NT, int kCap>
struct alignas(16) Shared {
  Exchange<NT / 32> x;
  uint64_t bar;
  uint64_t total[kMaxCluster];       // a level's sum over each CTA's share of the bins
  uint64_t pick[3];                  // a level's choice: bin, sum before it, its count
  uint64_t warp_sum[NT / 32];
  uint64_t list_mass[kMaxCluster];   // what each CTA put on the list, by weight and by count
  uint32_t list_count[kMaxCluster];
  uint32_t highest[kMaxCluster], lowest[kMaxCluster];  // of each CTA's threads' maxima
  double mass[kMaxCluster];          // each CTA's sum of weights
  uint64_t own_mass;
  uint32_t own_count, taken;
  uint32_t groups[kGroupBins];
  union {
    uint64_t list[kCap];  // places; complete in rank 0
    struct {
      unsigned long long mass[kBins];
      uint32_t count[kBins];
    } bin;
  };
};

// One row as a cluster sees it: held in the CTAs' shared memory, or read from
// global memory by every pass where it is too long for that.
template <typename T, int NT, bool kHeld>
struct Row {
  const T* p;
  Part<T> part;    // held
  const T* buf;
  int64_t c0, c1;  // read
  uint32_t rank, size;
  float m;         // the row's maximum
  float c;         // log2(e) / temperature
  float scale;     // weights become integers by this power of two
  int turn;

  __device__ __forceinline__ float at(int64_t i) const { return to_f32(p[i]); }
  __device__ __forceinline__ float log2w(float v) const { return log2_weight(v, m, c); }
  __device__ __forceinline__ unsigned long long weight(float v) const {
    return __float2ull_rn(exp2f(log2w(v)) * scale);
  }
  // f(value, index) for this thread's entries, in ascending order.  Fillers of
  // a held part come as -inf.
  template <typename F>
  __device__ __forceinline__ void each(F f) const {
    if (kHeld) {
      constexpr int kPer = Pack<T>::kPer;
      const uint4* src = reinterpret_cast<const uint4*>(buf);
      for (int j = threadIdx.x; j < part.packs; j += NT) {
        const uint4 w = src[j];
        const uint32_t in[4] = {w.x, w.y, w.z, w.w};
        const int64_t i = part.first + j * Part<T>::kE - part.off;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          float t[kPer];
          Pack<T>::open(in[x], t);
#pragma unroll
          for (int h = 0; h < kPer; ++h) f(t[h], i + x * kPer + h);
        }
      }
    } else {
      for (int64_t i = c0 + threadIdx.x; i < c1; i += NT) f(at(i), i);
    }
  }
  // Maximum of this thread's entries.
  __device__ __forceinline__ float own_max() const {
    if (kHeld) {
      const uint4* src = reinterpret_cast<const uint4*>(buf);
      uint32_t mx = Pack<T>::kNegInf;
      for (int j = threadIdx.x; j < part.packs; j += NT) {
        const uint4 v = src[j];
        mx = Pack<T>::max2(mx, Pack<T>::max2(Pack<T>::max2(v.x, v.y), Pack<T>::max2(v.z, v.w)));
      }
      float t[Pack<T>::kPer];
      Pack<T>::open(mx, t);
      float r = t[0];
#pragma unroll
      for (int h = 1; h < Pack<T>::kPer; ++h) r = fmaxf(r, t[h]);
      return r;
    }
    float r = -INFINITY;
    each([&](float v, int64_t) { r = fmaxf(r, v); });
    return r;
  }
};

// The place of the last entry kept when entries at or above `lo` are taken in
// order until the taken ones reach `need` (by count, or by weight): a radix
// descent over the places, kDigit bits of the value key at a time and, where
// equal values straddle the border, over the index bits.  Each level is one
// pass over the row that adds every entry with the prefix found so far to its
// digit's bin.  need is in [1, sum over the entries at or above lo].
template <typename T, int NT, bool kHeld, int kCap, bool kMass>
__device__ __noinline__ uint64_t find_cut(Row<T, NT, kHeld>& r, Shared<NT, kCap>& s, uint64_t lo, uint64_t need,
                                          int idx_bits) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint64_t pre = 0;
  int top = 64;  // bits of the place above `top` are `pre`
  while (true) {
    if (top == 32) {  // the index bits above V are all ones
      pre = (pre << (32 - idx_bits)) | ((1ull << (32 - idx_bits)) - 1);
      top = idx_bits;
      if (top == 0) return pre;
    }
    const int left = top > 32 ? top - 32 : top;
    const int bits = left < kDigit ? left : kDigit;
    const int shift = top - bits;
    for (int b = threadIdx.x; b < kBins; b += NT) {
      s.bin.count[b] = 0;
      s.bin.mass[b] = 0;
    }
    __syncthreads();
    r.each([&](float v, int64_t i) {
      const uint32_t key = value_key(v);
      const uint64_t c = place_of(key, static_cast<uint32_t>(i));
      if (key == 0 || c < lo || (top < 64 && (c >> top) != pre)) return;
      const int b = static_cast<int>((c >> shift) & ((1u << bits) - 1));
      atomicAdd(&s.bin.count[b], 1u);
      if (kMass) atomicAdd(&s.bin.mass[b], r.weight(v));
    });
    cluster_sync_all(r.size);
    // bins in falling order, cut into one contiguous share per CTA; a share's
    // bins are summed over the cluster and scanned
    constexpr int kMost = (kBins + NT - 1) / NT;
    const int share = kBins / static_cast<int>(r.size);
    const int per = (share + NT - 1) / NT;
    uint64_t mine[kMost];
    uint32_t cnt[kMost];
    uint64_t sum = 0;
#pragma unroll
    for (int q = 0; q < kMost; ++q) {
      mine[q] = 0;
      cnt[q] = 0;
      const int j = threadIdx.x * per + q;
      if (q < per && j < share) {
        const int b = kBins - 1 - (static_cast<int>(r.rank) * share + j);
        for (uint32_t o = 0; o < r.size; ++o) {
          cnt[q] += *peer(&s.bin.count[b], o);
          if (kMass) mine[q] += *peer(&s.bin.mass[b], o);
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
    for (int w = 0; w < NT / 32; ++w) {
      if (w < warp) before += s.warp_sum[w];
      all += s.warp_sum[w];
    }
    if (threadIdx.x < r.size) *peer(&s.total[r.rank], threadIdx.x) = all;
    cluster_sync_all(r.size);
    for (uint32_t o = 0; o < r.rank; ++o) before += s.total[o];
#pragma unroll
    for (int q = 0; q < kMost; ++q) {
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
    // the whole bin is taken, or it holds only the border entry
    if (top == 0 || in_bin == 1 || (!kMass && in_bin == need)) return pre << top;
  }
}

// Sum of the weights at or above a cut.
template <typename T, int NT, bool kHeld, int kCap>
__device__ uint64_t mass_from(Row<T, NT, kHeld>& r, Shared<NT, kCap>& s, uint64_t cut) {
  uint64_t w = 0;
  r.each([&](float v, int64_t i) {
    const uint32_t key = value_key(v);
    if (key != 0 && place_of(key, static_cast<uint32_t>(i)) >= cut) w += r.weight(v);
  });
  return cluster_reduce<NT / 32>(w, OpSumU64(), s.x, r.rank, r.size, r.turn);
}

// Smallest float at or above the bound that min-p puts on a logit.
__device__ __forceinline__ float min_p_bound(float m, const Ask& q) {
  const double t = static_cast<double>(m) + static_cast<double>(q.T) * log(static_cast<double>(q.mp));
  float f = static_cast<float>(t);
  if (static_cast<double>(f) < t) f = nextafterf(f, INFINITY);
  return f > m ? m : f;
}

// Sets up a row; in a held row its copy is started.
template <typename T, int NT, bool kHeld, int kCap>
__device__ void open_row(Row<T, NT, kHeld>& r, Shared<NT, kCap>& s, const FilterArgs& a, int64_t row, T* buf) {
  r.p = static_cast<const T*>(a.logits) + row * a.ld;
  r.rank = cluster_rank();
  r.size = cluster_size();
  r.turn = 0;
  r.scale = a.scale;
  if (threadIdx.x == 0) {
    mbar_init(&s.bar, 1);
    fence_mbar_init();
    s.own_mass = 0;
    s.own_count = 0;
    s.taken = 0;
  }
  for (int b = threadIdx.x; b < kGroupBins; b += NT) s.groups[b] = 0;
  __syncthreads();
  if (r.size > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  pdl_wait();
  if (kHeld) {
    r.part.cut(r.p, a.V, static_cast<int>(r.rank), static_cast<int>(r.size));
    r.buf = buf;
    r.part.load(r.p, buf, &s.bar);
  } else {
    const int64_t chunk = (a.V + r.size - 1) / r.size;
    r.c0 = chunk * r.rank < a.V ? chunk * r.rank : a.V;
    r.c1 = r.c0 + chunk < a.V ? r.c0 + chunk : a.V;
  }
}

// The row's maximum (false: no entry counts), the maximum of this thread's
// entries and the lowest of the threads' maxima that are not -inf.
template <typename T, int NT, bool kHeld, int kCap>
__device__ bool row_max(Row<T, NT, kHeld>& r, Shared<NT, kCap>& s, const FilterArgs& a, float* own, float* low) {
  if (kHeld) {
    mbar_wait(&s.bar, 0, a.status);
    __syncthreads();
  }
  *own = r.own_max();
  const uint32_t key = value_key(*own);
  const uint32_t hi = __reduce_max_sync(0xffffffffu, key);
  const uint32_t lo = __reduce_min_sync(0xffffffffu, key ? key : 0xFFFFFFFFu);
  if ((threadIdx.x & 31) == 0) s.warp_sum[threadIdx.x >> 5] = (static_cast<uint64_t>(hi) << 32) | lo;
  __syncthreads();
  if (r.size > 1) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");  // the other CTAs have started
  uint32_t h = 0, l = 0xFFFFFFFFu;
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) {
    h = max(h, static_cast<uint32_t>(s.warp_sum[w] >> 32));
    l = min(l, static_cast<uint32_t>(s.warp_sum[w]));
  }
  if (threadIdx.x < r.size) {
    *peer(&s.highest[r.rank], threadIdx.x) = h;
    *peer(&s.lowest[r.rank], threadIdx.x) = l;
  }
  cluster_sync_all(r.size);
  for (uint32_t o = 0; o < r.size; ++o) {
    h = max(h, s.highest[o]);
    l = min(l, s.lowest[o]);
  }
  r.m = key_to_value(h);
  *low = key_to_value(l);
  return h != 0;
}

// The short list.  A value t with at least `target` entries at or above it is
// read off a histogram of the threads' maxima (each the largest of a few dozen
// entries, so few entries beyond the target pass), and the places of the
// entries that reach t go to rank 0's list.  Only threads whose maximum
// reaches t look at their entries again.
//   target 0: t is given.  want_mass: the row's whole sum of weights is formed
//   on the way (the cluster barrier is shared).
// Returns false where the list would not hold them; else count and mass are
// those of the list.
struct Listed {
  uint32_t count;
  uint64_t mass;
  double row_mass;
};

template <typename T, int NT, bool kHeld, int kCap>
__device__ bool short_list(Row<T, NT, kHeld>& r, Shared<NT, kCap>& s, int64_t V, float own, float low, int target,
                           float t, bool want_mass, Listed* out) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const float range = r.m - low;
  bool fits = r.m < INFINITY && range < 1e30f;
  if (target > 0 || want_mass) {
    // (maxima that are all but equal share a bin)
    const float per = range > 1e-30f ? (kGroupBins - 0.01f) / range : 0.f;
    if (target > 0 && own > -INFINITY) {
      const int b = static_cast<int>((r.m - own) * per);
      atomicAdd(&s.groups[b < 0 ? 0 : (b < kGroupBins ? b : kGroupBins - 1)], 1u);
    }
    if (want_mass) {
      float w = 0.f;
      r.each([&](float v, int64_t) { w += v > -INFINITY ? fast_exp2(r.log2w(v)) : 0.f; });
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) w += __shfl_xor_sync(0xffffffffu, w, o);
      if (lane == 0) s.warp_sum[warp] = __float_as_uint(w);
    }
    __syncthreads();
    if (want_mass && threadIdx.x < r.size) {
      double w = 0.0;
      for (int x = 0; x < NT / 32; ++x) w += static_cast<double>(__uint_as_float(static_cast<uint32_t>(s.warp_sum[x])));
      *peer(&s.mass[r.rank], threadIdx.x) = w;
    }
    cluster_sync_all(r.size);
    if (want_mass) {
      out->row_mass = 0.0;
      for (uint32_t o = 0; o < r.size; ++o) out->row_mass += s.mass[o];
    }
    if (target > 0) {
      // the bin in which the maxima, from the highest, reach the target
      static_assert(kGroupBins <= NT, "one thread per bin");
      uint32_t n = 0;
      if (threadIdx.x < kGroupBins)
        for (uint32_t o = 0; o < r.size; ++o) n += *peer(&s.groups[threadIdx.x], o);
      uint32_t inc = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t u = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += u;
      }
      if (lane == 31) s.warp_sum[warp] = inc;
      if (threadIdx.x == 0) s.pick[0] = kGroupBins;
      __syncthreads();
      for (int w = 0; w < warp; ++w) inc += static_cast<uint32_t>(s.warp_sum[w]);
      if (inc - n < static_cast<uint32_t>(target) && inc >= static_cast<uint32_t>(target)) s.pick[0] = threadIdx.x;
      __syncthreads();
      const int b = static_cast<int>(s.pick[0]);
      if (b < kGroupBins) {
        // its lower edge, less what the bins' arithmetic may round
        t = per > 0.f ? r.m - (static_cast<float>(b) + 1.f) / per * 1.0001f - fabsf(r.m) * 1e-6f : low;
      } else {
        t = -INFINITY;  // fewer threads hold entries than the target
        fits = fits && V <= kCap;
      }
    }
  }
  if (!fits) return false;
  if (own >= t && own > -INFINITY) {
    uint32_t* taken = peer(&s.taken, 0);
    uint64_t* list = peer(s.list, 0);
    r.each([&](float v, int64_t i) {
      if (v >= t && v > -INFINITY) {
        const unsigned act = __activemask();
        const int first = __ffs(act) - 1;
        uint32_t base = 0;
        if (lane == first) {
          base = atomicAdd(taken, static_cast<uint32_t>(__popc(act)));
          atomicAdd(&s.own_count, static_cast<uint32_t>(__popc(act)));
        }
        base = __shfl_sync(act, base, first) + __popc(act & ((1u << lane) - 1));
        if (base < kCap) list[base] = place_of(value_key(v), static_cast<uint32_t>(i));
        if (want_mass) atomicAdd(reinterpret_cast<unsigned long long*>(&s.own_mass), r.weight(v));
      }
    });
  }
  __syncthreads();
  if (threadIdx.x < r.size) {
    *peer(&s.list_count[r.rank], threadIdx.x) = s.own_count;
    *peer(&s.list_mass[r.rank], threadIdx.x) = s.own_mass;
  }
  cluster_sync_all(r.size);
  out->count = 0;
  out->mass = 0;
  for (uint32_t o = 0; o < r.size; ++o) {
    out->count += s.list_count[o];
    out->mass += s.list_mass[o];
  }
  return out->count <= kCap;
}

// Sorts n places of the list (room for the next power of two), falling.
// Exchanges closer than a warp run on registers.
template <int NT>
__device__ void sort_list(uint64_t* list, int n) {
  int np = 32;
  while (np < n) np <<= 1;
  for (int i = n + threadIdx.x; i < np; i += NT) list[i] = 0;
  __syncthreads();
  const int lane = threadIdx.x & 31;
  for (int k = 32; k <= np; k <<= 1) {
    for (int j = k >> 1; j >= 32; j >>= 1) {
      for (int i = threadIdx.x; i < np / 2; i += NT) {
        const int lo = 2 * i - (i & (j - 1)), hi = lo + j;
        const uint64_t x = list[lo], y = list[hi];
        if ((x < y) == ((lo & k) == 0)) {
          list[lo] = y;
          list[hi] = x;
        }
      }
      __syncthreads();
    }
    for (int i = threadIdx.x; i < np; i += NT) {  // whole warps: np is a multiple of 32
      uint64_t x = list[i];
      for (int kk = k == 32 ? 2 : k; kk <= k; kk <<= 1) {
        const bool down = (i & kk) == 0;
        for (int j = kk >> 1 < 16 ? kk >> 1 : 16; j > 0; j >>= 1) {
          const uint64_t y = __shfl_xor_sync(0xffffffffu, x, j);
          const bool keep_max = ((lane & j) == 0) == down;
          x = (x > y) == keep_max ? x : y;
        }
      }
      list[i] = x;
    }
    __syncthreads();
  }
}

// Filters a sorted list (rank 0's threads): how many of its n entries are kept
// and the sum of their weights.  Without top-p the sum is formed all the same.
template <typename T, int NT, bool kHeld, int kCap>
__device__ int filter_list(const Row<T, NT, kHeld>& r, Shared<NT, kCap>& s, const Ask& q, int n, double row_mass,
                           uint64_t* kept_mass) {
  constexpr int kMost = (kCap + NT - 1) / NT;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int kk = q.k < n ? q.k : n;
  const int per = (kk + NT - 1) / NT;
  uint64_t w[kMost];
  uint64_t sum = 0;
  for (int x = 0; x < per; ++x) {
    const int i = threadIdx.x * per + x;
    const uint64_t v = i < kk ? r.weight(key_to_value(static_cast<uint32_t>(s.list[i] >> 32))) : 0ull;
    if (x < kMost) w[x] = v;
    sum += v;
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
  for (int x = 0; x < NT / 32; ++x) {
    if (x < warp) before += s.warp_sum[x];
    all += s.warp_sum[x];
  }
  // top-k bounds the mass that top-p refers to; without it the whole row does
  const double whole = row_mass > 0.0 ? row_mass * static_cast<double>(r.scale) : static_cast<double>(all);
  const double need = static_cast<double>(q.p) * whole;
  const float bound = q.mp > 0.f ? min_p_bound(r.m, q) : -INFINITY;
  int kept = 0;
  uint64_t mass = 0;
  for (int x = 0; x < per; ++x) {
    const int i = threadIdx.x * per + x;
    if (i < kk && (i == 0 || q.p >= 1.f || static_cast<double>(before) < need) &&
        key_to_value(static_cast<uint32_t>(s.list[i] >> 32)) >= bound) {
      ++kept;
      mass += w[x];
    }
    before += w[x];
  }
  *kept_mass = cta_reduce<NT / 32>(mass, OpSumU64(), s.x);
  return static_cast<int>(cta_reduce<NT / 32>(static_cast<uint64_t>(kept), OpSumU64(), s.x));
}

// The score of an entry, (v - m)/T - log(-log u), in fp32 and in double.
__device__ __forceinline__ float gumbel(float u) { return -logf(-logf(u)); }
__device__ __forceinline__ double score64(float v, float m, float temp, float u) {
  return (v == m ? 0.0 : (static_cast<double>(v) - static_cast<double>(m)) / static_cast<double>(temp)) -
         log(-log(static_cast<double>(u)));
}
// fp32 scores this close to the best are compared again in double
__device__ __forceinline__ bool near_best(float sc, float best) {
  return sc >= best - (1e-5f + 1e-6f * fabsf(best));
}

// Gumbel maximum over the first `kept` entries of the sorted list but `drop`
// (rank 0's threads); -1 when nothing is left.
template <typename T, int NT, bool kHeld, int kCap>
__device__ int pick_listed(const Row<T, NT, kHeld>& r, Shared<NT, kCap>& s, const float* u, int kept, int drop,
                           float temp) {
  float best = 0.f;
  int at = -1;
  for (int i = threadIdx.x; i < kept; i += NT) {
    const uint32_t v = place_index(s.list[i]);
    if (static_cast<int>(v) == drop) continue;
    const float sc = r.log2w(key_to_value(static_cast<uint32_t>(s.list[i] >> 32))) * kLn2 + gumbel(u[v]);
    if (at < 0 || argmax_key(sc, v) > argmax_key(best, place_index(s.list[at]))) {
      best = sc;
      at = i;
    }
  }
  const uint32_t v = at >= 0 ? place_index(s.list[at]) : 0;
  const uint64_t win = cta_reduce<NT / 32>(at >= 0 ? argmax_key(best, v) : 0ull, OpMaxU64(), s.x);
  if (win == 0) return -1;
  const bool close = at >= 0 && near_best(best, key_value(win));
  if (__syncthreads_count(close) <= 1) return static_cast<int>(key_index(win));
  const uint64_t dk =
      close ? double_key(score64(key_to_value(static_cast<uint32_t>(s.list[at] >> 32)), r.m, temp, u[v])) : 0ull;
  const uint64_t dbest = cta_reduce<NT / 32>(dk, OpMaxU64(), s.x);
  const uint64_t low = close && dk == dbest ? 0xFFFFFFFFull - v : 0ull;
  return static_cast<int>(0xFFFFFFFFull - cta_reduce<NT / 32>(low, OpMaxU64(), s.x));
}

// The same over the whole row: the entries at or above the cut.
template <typename T, int NT, bool kHeld, int kCap>
__device__ int pick_row(Row<T, NT, kHeld>& r, Shared<NT, kCap>& s, const float* u, uint64_t cut, int drop,
                        float temp) {
  constexpr int NW = NT / 32;
  float best = 0.f, val = 0.f;
  int at = -1;
  r.each([&](float v, int64_t i) {
    const uint32_t key = value_key(v);
    if (key == 0 || place_of(key, static_cast<uint32_t>(i)) < cut || i == drop) return;
    const float sc = r.log2w(v) * kLn2 + gumbel(u[i]);
    if (at < 0 || sc > best) {
      best = sc;
      val = v;
      at = static_cast<int>(i);
    }
  });
  const uint64_t k = at >= 0 ? argmax_key(best, static_cast<uint32_t>(at)) : 0ull;
  const uint64_t win = cluster_reduce<NW>(k, OpMaxU64(), s.x, r.rank, r.size, r.turn);
  if (win == 0) return -1;
  const bool close = at >= 0 && near_best(best, key_value(win));
  const uint64_t n = cluster_reduce<NW>(close, OpSumU64(), s.x, r.rank, r.size, r.turn);
  if (n <= 1) return static_cast<int>(key_index(win));
  const uint64_t dk = close ? double_key(score64(val, r.m, temp, u[at])) : 0ull;
  const uint64_t dbest = cluster_reduce<NW>(dk, OpMaxU64(), s.x, r.rank, r.size, r.turn);
  const uint64_t low = close && dk == dbest ? 0xFFFFFFFFull - static_cast<uint32_t>(at) : 0ull;
  return static_cast<int>(0xFFFFFFFFull - cluster_reduce<NW>(low, OpMaxU64(), s.x, r.rank, r.size, r.turn));
}

// The cut and the kept mass of a row whose kept entries may be many.
template <typename T, int NT, bool kHeld, int kCap>
__device__ uint64_t wide_cut(Row<T, NT, kHeld>& r, Shared<NT, kCap>& s, const FilterArgs& a, const Ask& q,
                             uint64_t* kept_mass) {
  uint64_t cut = 1ull << 32;  // every unmasked entry
  if (q.k < a.V) {
    uint64_t valid = 0;
    r.each([&](float v, int64_t) { valid += v > -INFINITY; });
    valid = cluster_reduce<NT / 32>(valid, OpSumU64(), s.x, r.rank, r.size, r.turn);
    if (static_cast<uint64_t>(q.k) < valid) cut = find_cut<T, NT, kHeld, kCap, false>(r, s, cut, q.k, a.idx_bits);
  }
  uint64_t w = mass_from(r, s, cut);
  const uint64_t had = cut;
  if (q.p < 1.f) {
    // entries are taken while the sum before them is below p times w
    uint64_t need = static_cast<uint64_t>(ceil(static_cast<double>(q.p) * static_cast<double>(w)));
    if (need < 1) need = 1;
    if (need < w) cut = find_cut<T, NT, kHeld, kCap, true>(r, s, cut, need, a.idx_bits);
  }
  if (q.mp > 0.f) {
    const uint64_t c = place_of(value_key(min_p_bound(r.m, q)), 0xFFFFFFFFu);
    if (c > cut) cut = c;
  }
  *kept_mass = cut == had ? w : mass_from(r, s, cut);
  return cut;
}

// Tries the short list for a row's filters; true: rank 0 holds the sorted list,
// of which it keeps *kept entries (rank 0's threads only know).
template <typename T, int NT, bool kHeld, int kCap>
__device__ bool listed_row(Row<T, NT, kHeld>& r, Shared<NT, kCap>& s, const FilterArgs& a, const Ask& q, float own,
                           float low, int* kept, uint64_t* kept_mass) {
  int target = 0;
  float t = -INFINITY;
  bool want_mass = false;
  if (q.k == 1) {
    t = r.m;
  } else if (q.k < a.V) {
    target = q.k;
  } else if (q.p < 1.f) {
    target = kFewTarget;
    want_mass = true;
  } else if (q.mp > 0.f) {
    t = min_p_bound(r.m, q);
  } else {
    return false;
  }
  if (target > kCap) return false;
  Listed l;
  l.row_mass = 0.0;
  if (!short_list(r, s, a.V, own, low, target, t, want_mass, &l)) return false;
  // top-p of the whole row: the list has to hold its border
  if (want_mass &&
      static_cast<double>(l.mass) < static_cast<double>(q.p) * l.row_mass * static_cast<double>(r.scale) &&
      static_cast<int64_t>(l.count) < a.V)
    return false;
  if (r.rank != 0) return true;
  sort_list<NT>(s.list, static_cast<int>(l.count));
  *kept = filter_list(r, s, q, static_cast<int>(l.count), l.row_mass, kept_mass);
  return true;
}

template <typename T, int NT, bool kHeld>
__device__ __forceinline__ float log_prob(const Row<T, NT, kHeld>& r, int tok, uint64_t kept) {
  return r.log2w(r.at(tok)) * kLn2 - logf(static_cast<float>(kept) / r.scale);
}

constexpr int kShortCap = 1024;

template <typename T, int NT, bool kHeld>
__global__ void __launch_bounds__(NT, NT == 256 ? 4 : 2) sample_rows_kernel(const FilterArgs a) {
  extern __shared__ __align__(16) uint8_t raw[];
  using S = Shared<NT, kShortCap>;
  S& s = *reinterpret_cast<S*>(raw);
  const int64_t row = blockIdx.x / cluster_size();
  Row<T, NT, kHeld> r;
  open_row(r, s, a, row, reinterpret_cast<T*>(raw + sizeof(S)));
  const Ask q = read_ask(a, row);
  r.c = inv_temperature(q.T);
  float own, low;
  const bool some = row_max(r, s, a, &own, &low);
  const float* u = a.u + row * a.ld_u;
  int tok = -1;
  float lp = -INFINITY;
  if (q.ok && some) {
    int n;
    uint64_t mass;
    if (listed_row(r, s, a, q, own, low, &n, &mass)) {
      if (r.rank != 0) return;
      tok = q.greedy ? static_cast<int>(place_index(s.list[0])) : pick_listed(r, s, u, n, -1, q.T);
    } else {
      const uint64_t cut = wide_cut(r, s, a, q, &mass);
      tok = q.greedy ? static_cast<int>(place_index(cut)) : pick_row(r, s, u, cut, -1, q.T);
    }
    if (tok >= 0) lp = log_prob(r, tok, mass);
  }
  if (r.rank == 0 && threadIdx.x == 0) {
    a.tok[row] = tok;
    if (a.logprob) a.logprob[row] = lp;
    if (!q.ok) atomicOr(a.status, kDevBadParam);
  }
}

// Verified row rr of sequence j: whether its draft is accepted, and the token
// drawn here if it is not (or if rr = D).  A row without a short list leaves
// the draw, which few rows need, to the second kernel.
template <typename T, int NT, bool kHeld>
__global__ void __launch_bounds__(NT, NT == 256 ? 4 : 2) accept_rows_kernel(const FilterArgs a) {
  extern __shared__ __align__(16) uint8_t raw[];
  using S = Shared<NT, kShortCap>;
  S& s = *reinterpret_cast<S*>(raw);
  const int64_t j = blockIdx.x / cluster_size() / a.rows_used;
  const int rr = static_cast<int>(blockIdx.x / cluster_size() - j * a.rows_used);
  const int64_t row = j * a.R + rr;
  Row<T, NT, kHeld> r;
  open_row(r, s, a, row, reinterpret_cast<T*>(raw + sizeof(S)));
  const Ask q = read_ask(a, j);
  r.c = inv_temperature(q.T);
  float own, low;
  const bool some = row_max(r, s, a, &own, &low);
  RowCut out;
  out.cut = ~0ull;
  out.m = r.m;
  out.accept = 0;
  out.tok = -1;
  if (q.ok && some) {
    int n;
    uint64_t kept;
    const bool listed = listed_row(r, s, a, q, own, low, &n, &kept);
    if (listed && r.rank != 0) return;
    out.cut = listed ? s.list[n - 1] : wide_cut(r, s, a, q, &kept);
    int drop = -1;
    if (rr < a.D) {
      drop = a.draft[j * a.D + rr];
      if (drop >= 0 && drop < a.V) {
        const float v = r.at(drop);
        const uint32_t key = value_key(v);
        if (key != 0 && place_of(key, static_cast<uint32_t>(drop)) >= out.cut)
          out.accept = static_cast<double>(a.u_accept[j * a.D + rr]) <
                       static_cast<double>(r.weight(v)) / static_cast<double>(kept);
      }
    }
    out.tok = -2;  // not drawn yet
    if (listed && !out.accept) out.tok = pick_listed(r, s, a.u + j * a.ld_u, n, drop, q.T);
  }
  if (r.rank == 0 && threadIdx.x == 0) a.cuts[row] = out;
}

// One cluster per sequence: leading accepts, the draw at the row after them if
// it is still to be made, and the outputs.
template <typename T>
__global__ void __launch_bounds__(512) accept_pick_kernel(const FilterArgs a) {
  extern __shared__ __align__(16) uint8_t raw[];
  using S = Shared<512, kShortCap>;
  S& s = *reinterpret_cast<S*>(raw);
  pdl_wait();
  const int64_t j = blockIdx.x / cluster_size();
  const uint32_t rank = cluster_rank(), size = cluster_size();
  const Ask q = read_ask(a, j);
  int n = 0;
  while (n < a.D && a.cuts[j * a.R + n].accept) ++n;
  const int* dr = a.draft + j * a.D;
  int corr = -1;
  if (q.ok && n < a.R) {
    const int64_t row = j * a.R + n;
    const RowCut c = a.cuts[row];
    corr = c.tok;
    if (corr == -2) {
      Row<T, 512, false> r;
      r.p = static_cast<const T*>(a.logits) + row * a.ld;
      r.rank = rank;
      r.size = size;
      const int64_t chunk = (a.V + size - 1) / size;
      r.c0 = chunk * rank < a.V ? chunk * rank : a.V;
      r.c1 = r.c0 + chunk < a.V ? r.c0 + chunk : a.V;
      r.turn = 0;
      r.m = c.m;
      r.c = inv_temperature(q.T);
      cluster_sync_all(size);
      corr = pick_row(r, s, a.u + j * a.ld_u, c.cut, n < a.D ? dr[n] : -1, q.T);
    }
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
}

constexpr int kTopCap = 2048;
static_assert(kTopCap >= kTopLogitsMax, "the K entries fit the list");

// The K first entries of the order, sorted, and the row's log-sum-exp.
template <typename T, int NT, bool kHeld>
__global__ void __launch_bounds__(NT, NT == 256 ? 4 : 2) top_rows_kernel(const FilterArgs a) {
  extern __shared__ __align__(16) uint8_t raw[];
  using S = Shared<NT, kTopCap>;
  S& s = *reinterpret_cast<S*>(raw);
  const int64_t row = blockIdx.x / cluster_size();
  Row<T, NT, kHeld> r;
  open_row(r, s, a, row, reinterpret_cast<T*>(raw + sizeof(S)));
  r.c = inv_temperature(a.T);
  float own, low;
  const bool some = row_max(r, s, a, &own, &low);
  Listed l;
  l.count = 0;
  l.row_mass = 0.0;
  if (some && !short_list(r, s, a.V, own, low, a.K, -INFINITY, true, &l)) {
    // ties or a clustered row: find the exact border, then list
    uint64_t cut = 1ull << 32, valid = 0;
    r.each([&](float v, int64_t) { valid += v > -INFINITY; });
    valid = cluster_reduce<NT / 32>(valid, OpSumU64(), s.x, r.rank, r.size, r.turn);
    if (static_cast<uint64_t>(a.K) < valid)
      cut = find_cut<T, NT, kHeld, kTopCap, false>(r, s, cut, a.K, a.idx_bits);
    if (r.rank == 0 && threadIdx.x == 0) s.taken = 0;
    cluster_sync_all(r.size);
    uint32_t* taken = peer(&s.taken, 0);
    uint64_t* list = peer(s.list, 0);
    r.each([&](float v, int64_t i) {
      const uint32_t key = value_key(v);
      const uint64_t c = place_of(key, static_cast<uint32_t>(i));
      if (key != 0 && c >= cut) {
        const uint32_t at = atomicAdd(taken, 1u);
        if (at < kTopCap) list[at] = c;
      }
    });
    cluster_sync_all(r.size);
    l.count = static_cast<uint64_t>(a.K) < valid ? static_cast<uint32_t>(a.K) : static_cast<uint32_t>(valid);
  }
  if (r.rank != 0) return;
  const int n = static_cast<int>(l.count);
  sort_list<NT>(s.list, n);
  for (int i = threadIdx.x; i < a.K; i += NT) {
    const uint64_t c = i < n ? s.list[i] : 0;
    a.val[row * a.K + i] = c ? key_to_value(static_cast<uint32_t>(c >> 32)) : -INFINITY;
    a.idx[row * a.K + i] = c ? static_cast<int>(place_index(c)) : -1;
  }
  if (a.lse && threadIdx.x == 0)
    a.lse[row] = some ? static_cast<float>(static_cast<double>(r.m) / static_cast<double>(a.T) +
                                           static_cast<double>(logf(static_cast<float>(l.row_mass))))
                      : -INFINITY;
}

cudaError_t launch_rows(const void* kern, int nt, int64_t rows, int parts, size_t smem, const FilterArgs& a,
                        cudaStream_t st) {
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  FilterArgs b = a;
  void* args[] = {&b};
  return launch_kc(kern, dim3((unsigned)(rows * parts)), dim3(nt), smem, st, true, dim3(parts), args);
}

// Parts of at most 40 KB let several CTAs share an SM; rows that do not fill
// the GPU are cut further; what does not fit is read from global memory.
template <typename T>
int pick_parts(int64_t V, int64_t rows) {
  int parts = 1;
  while (parts < kMaxCluster && (Part<T>::bytes(V, parts) > 40 * 1024 ||
                                 (rows * parts < 2 * num_sms() && Part<T>::bytes(V, 2 * parts) >= 4096)))
    parts *= 2;
  return parts;
}

#define DFL_ROWS(KERNEL, CAP)                                                                                     \
  template <typename T>                                                                                           \
  cudaError_t launch_##KERNEL(const FilterArgs& a, int64_t rows, cudaStream_t st) {                               \
    const int parts = pick_parts<T>(a.V, rows);                                                                   \
    const size_t pb = Part<T>::bytes(a.V, parts);                                                                 \
    if (pb <= 40 * 1024)                                                                                          \
      return launch_rows((const void*)KERNEL<T, 256, true>, 256, rows, parts, sizeof(Shared<256, CAP>) + pb, a,    \
                         st);                                                                                     \
    if (pb <= 190 * 1024)                                                                                         \
      return launch_rows((const void*)KERNEL<T, 512, true>, 512, rows, parts, sizeof(Shared<512, CAP>) + pb, a,    \
                         st);                                                                                     \
    return launch_rows((const void*)KERNEL<T, 512, false>, 512, rows, kMaxCluster, sizeof(Shared<512, CAP>), a,    \
                       st);                                                                                       \
  }
DFL_ROWS(sample_rows_kernel, kShortCap)
DFL_ROWS(accept_rows_kernel, kShortCap)
DFL_ROWS(top_rows_kernel, kTopCap)
#undef DFL_ROWS

template <typename T>
cudaError_t launch_accept(const FilterArgs& a, int64_t b, cudaStream_t st) {
  cudaError_t e = launch_accept_rows_kernel<T>(a, b * a.rows_used, st);
  if (e != cudaSuccess) return e;
  return launch_rows((const void*)accept_pick_kernel<T>, 512, b, pick_parts<T>(a.V, b), sizeof(Shared<512, kShortCap>),
                     a, st);
}

void finish(FilterArgs& a) {
  a.idx_bits = 0;
  while (((int64_t)1 << a.idx_bits) < a.V) ++a.idx_bits;
  a.scale = ldexpf(1.f, 62 - a.idx_bits);
}

}  // namespace

cudaError_t filter_sample(FilterArgs a, int dtype, int64_t rows, cudaStream_t st) {
  finish(a);
  if (dtype == 0) return launch_sample_rows_kernel<float>(a, rows, st);
  if (dtype == 1) return launch_sample_rows_kernel<__half>(a, rows, st);
  return launch_sample_rows_kernel<__nv_bfloat16>(a, rows, st);
}

cudaError_t filter_accept(FilterArgs a, int dtype, int64_t b, cudaStream_t st) {
  finish(a);
  a.rows_used = a.R <= a.D ? a.R : a.D + 1;  // no answer depends on the rows behind
  if (dtype == 0) return launch_accept<float>(a, b, st);
  if (dtype == 1) return launch_accept<__half>(a, b, st);
  return launch_accept<__nv_bfloat16>(a, b, st);
}

cudaError_t top_logits(FilterArgs a, int dtype, int64_t rows, cudaStream_t st) {
  finish(a);
  if (dtype == 0) return launch_top_rows_kernel<float>(a, rows, st);
  if (dtype == 1) return launch_top_rows_kernel<__half>(a, rows, st);
  return launch_top_rows_kernel<__nv_bfloat16>(a, rows, st);
}

}  // namespace dfl
