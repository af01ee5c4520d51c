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
constexpr int kGroups = 8;            // groups of entries per thread whose maxima are kept
constexpr int kGroupBins = 256;       // bins of the groups' maxima
constexpr int kLineBins = 1024;       // bins of the weights, linear in the logit
constexpr int kDevBadParam = 0x8;
constexpr int kFewTarget = 96;        // entries the short list aims at where top-k does not say
constexpr int kQuick = 128;           // lists up to this length are ranked, longer ones sorted
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

// Shared memory of a CTA.
template <int NT, int kCap>
struct alignas(16) Shared {
  Exchange<NT / 32> x;
  uint64_t total[kMaxCluster];       // a level's sum over each CTA's share of the bins
  uint64_t pick[3];                  // a level's choice: bin, sum before it, its count
  uint64_t warp_sum[NT / 32];
  uint64_t list_mass[kMaxCluster];   // what each CTA put on the list, by weight and by count
  uint32_t list_count[kMaxCluster];
  uint32_t highest[kMaxCluster], lowest[kMaxCluster];  // of each CTA's groups' maxima
  double mass[kMaxCluster];          // each CTA's sum of weights
  uint64_t own_mass;
  uint32_t own_count, taken, queued;
  uint32_t groups[kGroupBins];
  union {
    uint64_t list[kCap];  // places; complete in rank 0
    struct {
      unsigned long long mass[kBins];
      uint32_t count[kBins];
    } bin;
  };
  uint32_t line[kLineBins];
  ulonglong2 entry[kQuick];          // a quick list's places and weights
  uint64_t half_before[kQuick];
  uint32_t half_rank[kQuick];
  uint64_t join[NT / 32][3];
};

// One row as a cluster sees it.  Each CTA reads its part of the row from
// global memory in 16-byte packs, thread t the packs t, t + NT, ...; a pass
// after the first finds them in L2.
template <typename T, int NT>
struct Row {
  static constexpr int kPer = Pack<T>::kPer, kE = Part<T>::kE;
  const T* p;
  Part<T> part;
  const uint4* packs;  // pack 0 (its first `off` entries lie before the part)
  bool cut_head, cut_tail;
  uint32_t rank, size;
  float m;             // the row's maximum
  float c;             // log2(e) / temperature
  float scale;         // weights become integers by this power of two
  int turn;

  __device__ __forceinline__ void open(const FilterArgs& a, int64_t row) {
    p = static_cast<const T*>(a.logits) + row * a.ld;
    rank = cluster_rank();
    size = cluster_size();
    turn = 0;
    scale = a.scale;
    part.cut(p, a.V, static_cast<int>(rank), static_cast<int>(size));
    packs = reinterpret_cast<const uint4*>(p + part.first - part.off);
    cut_head = part.off > 0;
    cut_tail = (part.off + part.n) % kE != 0;
  }
  __device__ __forceinline__ float at(int64_t i) const { return to_f32(p[i]); }
  __device__ __forceinline__ int64_t index_of(int j) const { return part.first + j * kE - part.off; }
  __device__ __forceinline__ float log2w(float v) const { return log2_weight(v, m, c); }
  __device__ __forceinline__ unsigned long long weight(float v) const {
    return __float2ull_rn(exp2f(log2w(v)) * scale);
  }
  // Pack j; entries that are not the row's come as -inf, and a pack past the
  // part as nothing else.
  __device__ __forceinline__ uint4 pack(int j) const {
    uint4 v = make_uint4(Pack<T>::kNegInf, Pack<T>::kNegInf, Pack<T>::kNegInf, Pack<T>::kNegInf);
    if (j >= part.packs) return v;
    if ((j > 0 || !cut_head) && (j + 1 < part.packs || !cut_tail)) return packs[j];
    T* e = reinterpret_cast<T*>(&v);
#pragma unroll
    for (int h = 0; h < kE; ++h) {
      const int i = j * kE + h - part.off;
      if (i >= 0 && i < part.n) e[h] = p[part.first + i];
    }
    return v;
  }
  static __device__ __forceinline__ void open_pack(const uint4& w, float* v) {  // kE values
    const uint32_t in[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int x = 0; x < 4; ++x) Pack<T>::open(in[x], v + x * kPer);
  }
  static __device__ __forceinline__ uint32_t max_pack(const uint4& w) {
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
  // f(pack, its number) for this thread's packs, four loads at a time.
  template <typename F>
  __device__ __forceinline__ void each_pack(F f) const {
    for (int j = threadIdx.x; j < part.packs; j += 4 * NT) {
      uint4 w[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) w[x] = pack(j + x * NT);
#pragma unroll
      for (int x = 0; x < 4; ++x)
        if (j + x * NT < part.packs) f(w[x], j + x * NT);
    }
  }
  // f(value, index) for this thread's entries.
  template <typename F>
  __device__ __forceinline__ void each(F f) const {
    each_pack([&](const uint4& w, int j) {
      float v[kE];
      open_pack(w, v);
      const int64_t i = index_of(j);
#pragma unroll
      for (int h = 0; h < kE; ++h) f(v[h], i + h);
    });
  }
};

// The place of the last entry kept when entries at or above `lo` are taken in
// order until the taken ones reach `need` (by count, or by weight): a radix
// descent over the places, kDigit bits of the value key at a time and, where
// equal values straddle the border, over the index bits.  Each level is one
// pass over the row that adds every entry with the prefix found so far to its
// digit's bin.  need is in [1, sum over the entries at or above lo].
template <typename T, int NT, int kCap, bool kMass>
__device__ __noinline__ uint64_t find_cut(Row<T, NT>& r, Shared<NT, kCap>& s, uint64_t lo, uint64_t need,
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

// The value of a cut's entry; -inf where every unmasked entry is kept.
__device__ __forceinline__ float cut_value(uint64_t cut) {
  const uint32_t k = static_cast<uint32_t>(cut >> 32);
  return k > 0x007FFFFFu ? key_to_value(k) : -INFINITY;
}

// Sum of the weights at or above a cut.
template <typename T, int NT, int kCap>
__device__ uint64_t mass_from(Row<T, NT>& r, Shared<NT, kCap>& s, uint64_t cut) {
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

// What one pass over the row leaves in a thread: the maxima of its groups
// (the packs whose turn is the group's number, modulo kGroups) and, where asked
// for, its exponential sum relative to its own maximum.
template <typename T, int NT>
struct Scan {
  float group[kGroups];
  float top;     // the thread's maximum
  float ref;     // exponent of the sum's reference
  float sum;     // sum of 2^(x - ref); of the weights relative to top if `careful`
  bool careful;
};

template <typename T, int NT>
__device__ __forceinline__ void scan_row(const Row<T, NT>& r, bool want_mass, Scan<T, NT>& t) {
  constexpr int kE = Row<T, NT>::kE;
  uint32_t g[kGroups];
#pragma unroll
  for (int x = 0; x < kGroups; ++x) g[x] = Pack<T>::kNegInf;
  t.ref = 0.f;
  t.sum = 0.f;
  bool any = false, odd = false;
  for (int j = threadIdx.x; j < r.part.packs; j += kGroups * NT) {
    uint4 w[kGroups];
#pragma unroll
    for (int x = 0; x < kGroups; ++x) w[x] = r.pack(j + x * NT);
    uint32_t all = Pack<T>::kNegInf;
#pragma unroll
    for (int x = 0; x < kGroups; ++x) {
      const uint32_t mx = Row<T, NT>::max_pack(w[x]);
      g[x] = Pack<T>::max2(g[x], mx);
      all = Pack<T>::max2(all, mx);
    }
    if (want_mass) {
      const float top = Row<T, NT>::max_of(all);
      if (top > -INFINITY) {
        const float ref = top * r.c;
        if (!any || ref > t.ref) {
          if (any) t.sum *= fast_exp2(t.ref - ref);
          t.ref = ref;
          any = true;
          odd |= !(fabsf(ref) < kRefMax);
        }
#pragma unroll
        for (int x = 0; x < kGroups; ++x) {
          float v[kE];
          Row<T, NT>::open_pack(w[x], v);
          float some = 0.f;
#pragma unroll
          for (int h = 0; h < kE; ++h) some += fast_exp2(fmaf(v[h], r.c, -t.ref));
          t.sum += some;
        }
      }
    }
  }
  t.top = -INFINITY;
#pragma unroll
  for (int x = 0; x < kGroups; ++x) {
    t.group[x] = Row<T, NT>::max_of(g[x]);
    t.top = fmaxf(t.top, t.group[x]);
  }
  // masked entries that are NaN, or logits at the type's end: again, with care
  t.careful = want_mass && (odd || !(t.sum < INFINITY));
  if (t.careful) {
    t.sum = 0.f;
    r.each([&](float v, int64_t) {
      if (v > -INFINITY) t.sum += fast_exp2(log2_weight(v, t.top, r.c));
    });
  }
}

// The row's maximum (false: no entry counts), the lowest of the groups' maxima
// that are not -inf, and where wanted the row's sum of weights.
template <typename T, int NT, int kCap>
__device__ bool join_scan(Row<T, NT>& r, Shared<NT, kCap>& s, const Scan<T, NT>& t, bool want_mass, float* low,
                          double* row_mass) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t lo = 0xFFFFFFFFu;
#pragma unroll
  for (int x = 0; x < kGroups; ++x) {
    const uint32_t k = value_key(t.group[x]);
    lo = k && k < lo ? k : lo;
  }
  uint32_t hi = __reduce_max_sync(0xffffffffu, value_key(t.top));
  lo = __reduce_min_sync(0xffffffffu, lo);
  if (lane == 0) s.warp_sum[warp] = (static_cast<uint64_t>(hi) << 32) | lo;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) {
    hi = max(hi, static_cast<uint32_t>(s.warp_sum[w] >> 32));
    lo = min(lo, static_cast<uint32_t>(s.warp_sum[w]));
  }
  // the CTA's sum relative to its own maximum
  const float cta_top = key_to_value(hi);
  float sum = 0.f;
  if (want_mass) {
    if (t.top > -INFINITY)
      sum = t.sum * fast_exp2(t.careful ? log2_weight(t.top, cta_top, r.c) : fmaf(-cta_top, r.c, t.ref));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    __syncthreads();
    if (lane == 0) s.warp_sum[warp] = __float_as_uint(sum);
    __syncthreads();
  }
  if (r.size > 1) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");  // the other CTAs have started
  if (threadIdx.x < r.size) {
    *peer(&s.highest[r.rank], threadIdx.x) = hi;
    *peer(&s.lowest[r.rank], threadIdx.x) = lo;
    if (want_mass) {
      double w = 0.0;
      for (int x = 0; x < NT / 32; ++x) w += static_cast<double>(__uint_as_float(static_cast<uint32_t>(s.warp_sum[x])));
      *peer(&s.mass[r.rank], threadIdx.x) = w;
    }
  }
  cluster_sync_all(r.size);
  for (uint32_t o = 0; o < r.size; ++o) {
    hi = max(hi, s.highest[o]);
    lo = min(lo, s.lowest[o]);
  }
  r.m = key_to_value(hi);
  *low = key_to_value(lo);
  *row_mass = 0.0;
  if (want_mass && hi != 0)
    for (uint32_t o = 0; o < r.size; ++o)
      if (s.highest[o]) *row_mass += s.mass[o] * static_cast<double>(fast_exp2(r.log2w(key_to_value(s.highest[o]))));
  return hi != 0;
}

// Puts the places of the entries at or above t on rank 0's list and counts them
// in own_count (own_mass: their weights, if wanted).  Only groups whose maximum
// reaches t are read again: their numbers go to a queue, whose packs all
// threads share, so that one round trip to L2 serves most rows.
template <typename T, int NT, int kCap>
__device__ __forceinline__ void list_entries(const Row<T, NT>& r, Shared<NT, kCap>& s, const Scan<T, NT>& sc, float t,
                                             bool want_mass) {
  constexpr int kE = Row<T, NT>::kE;
  static_assert(NT * kGroups * sizeof(uint16_t) <= sizeof(s.line) && NT * kGroups <= 65536, "the queue fits");
  uint16_t* queue = reinterpret_cast<uint16_t*>(s.line);
#pragma unroll
  for (int x = 0; x < kGroups; ++x)
    if (sc.group[x] >= t && sc.group[x] > -INFINITY)
      queue[atomicAdd(&s.queued, 1u)] = static_cast<uint16_t>(threadIdx.x + x * NT);
  __syncthreads();
  const int lane = threadIdx.x & 31;
  uint32_t* taken = peer(&s.taken, 0);
  uint64_t* list = peer(s.list, 0);
  const uint32_t deep = (r.part.packs + kGroups * NT - 1) / (kGroups * NT), units = s.queued * deep;
  for (uint32_t y = threadIdx.x; y < units; y += NT) {
    const uint32_t g = y / deep;
    const int j = queue[g] + static_cast<int>(y - g * deep) * (kGroups * NT);
    if (j >= r.part.packs) continue;
    const uint4 w = r.pack(j);
    if (!(Row<T, NT>::max_of(Row<T, NT>::max_pack(w)) >= t)) continue;
    float v[kE];
    Row<T, NT>::open_pack(w, v);
    const int64_t i = r.index_of(j);
#pragma unroll
    for (int h = 0; h < kE; ++h) {
      if (v[h] >= t && v[h] > -INFINITY) {
        const unsigned act = __activemask();
        const int first = __ffs(act) - 1;
        uint32_t base = 0;
        if (lane == first) {
          base = atomicAdd(taken, static_cast<uint32_t>(__popc(act)));
          atomicAdd(&s.own_count, static_cast<uint32_t>(__popc(act)));
        }
        base = __shfl_sync(act, base, first) + __popc(act & ((1u << lane) - 1));
        if (base < kCap) list[base] = place_of(value_key(v[h]), static_cast<uint32_t>(i + h));
        if (want_mass) atomicAdd(reinterpret_cast<unsigned long long*>(&s.own_mass), r.weight(v[h]));
      }
    }
  }
}

// Sum of the CTAs' own counts and masses; complete lists are seen after it.
template <typename T, int NT, int kCap>
__device__ __forceinline__ void close_list(const Row<T, NT>& r, Shared<NT, kCap>& s, uint32_t* count, uint64_t* mass) {
  __syncthreads();
  if (threadIdx.x < r.size) {
    *peer(&s.list_count[r.rank], threadIdx.x) = s.own_count;
    *peer(&s.list_mass[r.rank], threadIdx.x) = s.own_mass;
  }
  cluster_sync_all(r.size);
  *count = 0;
  *mass = 0;
  for (uint32_t o = 0; o < r.size; ++o) {
    *count += s.list_count[o];
    *mass += s.list_mass[o];
  }
}

// The short list.  A value t with at least `target` entries at or above it is
// read off a histogram of the groups' maxima (each the largest of a few dozen
// entries, so few entries beyond the target pass), and the places of the
// entries that reach t go to rank 0's list.  target 0: t is given.  Returns
// false where the list would not hold them; else count and mass (if wanted)
// are those of the list.
template <typename T, int NT, int kCap>
__device__ bool short_list(Row<T, NT>& r, Shared<NT, kCap>& s, const Scan<T, NT>& sc, int64_t V, float low, int target,
                           float* bound, bool want_mass, uint32_t* count, uint64_t* mass) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const float range = r.m - low;
  float t = *bound;
  if (!(r.m < INFINITY) || !(range < 1e30f)) return false;
  if (target > 0) {
    // (maxima that are all but equal share a bin)
    const float per = range > 1e-30f ? (kGroupBins - 0.01f) / range : 0.f;
#pragma unroll
    for (int x = 0; x < kGroups; ++x) {
      if (sc.group[x] > -INFINITY) {
        const int b = static_cast<int>((r.m - sc.group[x]) * per);
        atomicAdd(&s.groups[b < 0 ? 0 : (b < kGroupBins ? b : kGroupBins - 1)], 1u);
      }
    }
    cluster_sync_all(r.size);
    // the bin in which the maxima, from the highest, reach the target
    static_assert(kGroupBins <= NT, "one thread per bin");
    uint32_t n = 0;
    if (threadIdx.x < kGroupBins) {
      uint32_t c[kMaxCluster];
#pragma unroll
      for (uint32_t o = 0; o < kMaxCluster; ++o) c[o] = o < r.size ? *peer(&s.groups[threadIdx.x], o) : 0u;
#pragma unroll
      for (uint32_t o = 0; o < kMaxCluster; ++o) n += c[o];
    }
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
      t = -INFINITY;  // fewer groups hold entries than the target
      if (V > kCap) return false;
    }
  }
  list_entries(r, s, sc, t, want_mass);
  close_list(r, s, count, mass);
  *bound = t;
  return *count <= kCap;
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
// and the sum of their weights.  `above` is the weight of the entries before
// the list; whole > 0 is the weight that top-p refers to, else what top-k keeps.
template <typename T, int NT, int kCap>
__device__ int filter_list(const Row<T, NT>& r, Shared<NT, kCap>& s, const Ask& q, int n, double above, double whole,
                           double* kept_mass) {
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
  const double scale = static_cast<double>(r.scale);
  const double need = static_cast<double>(q.p) * (whole > 0.0 ? whole * scale : static_cast<double>(all));
  above *= scale;
  const float bound = q.mp > 0.f ? min_p_bound(r.m, q) : -INFINITY;
  int kept = 0;
  uint64_t mass = 0;
  for (int x = 0; x < per; ++x) {
    const int i = threadIdx.x * per + x;
    if (i < kk && (i == 0 || q.p >= 1.f || above + static_cast<double>(before) < need) &&
        key_to_value(static_cast<uint32_t>(s.list[i] >> 32)) >= bound) {
      ++kept;
      mass += w[x];
    }
    before += w[x];
  }
  *kept_mass = (above + static_cast<double>(cta_reduce<NT / 32>(mass, OpSumU64(), s.x))) / scale;
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
template <typename T, int NT, int kCap>
__device__ int pick_listed(const Row<T, NT>& r, Shared<NT, kCap>& s, const float* u, int kept, int drop,
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

// What a list says of its row (rank 0's threads).
struct Verdict {
  double mass;   // sum of the kept weights
  uint64_t cut;  // place of the last entry kept
  int tok;       // Gumbel maximum of the kept entries but `drop` (u given)
};

// Filters a short list and draws from it.  Up to kQuick entries, each one's
// rank and the sum of the weights before it come from comparing it with all
// others (two threads an entry), which needs neither a sort nor a scan; longer
// lists are sorted.  above, whole: as in filter_list.
template <typename T, int NT, int kCap>
__device__ __noinline__ Verdict settle_list(const Row<T, NT>& r, Shared<NT, kCap>& s, const Ask& q, int n, double above,
                                            double whole, const float* u, int drop) {
  Verdict out;
  if (n > kQuick) {
    sort_list<NT>(s.list, n);
    const int kept = filter_list(r, s, q, n, above, whole, &out.mass);
    out.cut = s.list[kept - 1];
    out.tok = u ? pick_listed(r, s, u, kept, drop, q.T) : -1;
    return out;
  }
  static_assert(NT == 2 * kQuick, "two threads an entry");
  const int e = threadIdx.x & (kQuick - 1), half = threadIdx.x / kQuick;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint64_t place = e < n ? s.list[e] : 0;
  const float v = key_to_value(static_cast<uint32_t>(place >> 32));
  const uint32_t at = place_index(place);
  uint64_t w = 0;
  float ue = 0.f;
  if (half == 0 && e < n) {
    if (u && !q.greedy) ue = u[at];
    w = r.weight(v);
    s.entry[e] = make_ulonglong2(place, w);
  }
  __syncthreads();
  uint32_t rank = 0;
  uint64_t before = 0;
  const int i1 = half ? n : (n < kQuick / 2 ? n : kQuick / 2);
  for (int i = half * (kQuick / 2); i < i1; ++i) {
    const ulonglong2 o = s.entry[i];
    if (o.x > place) {
      ++rank;
      before += o.y;
    }
  }
  if (half == 1) {
    s.half_rank[e] = rank;
    s.half_before[e] = before;
  }
  __syncthreads();
  const bool mine = half == 0 && e < n;
  if (mine) {
    rank += s.half_rank[e];
    before += s.half_before[e];
  }
  const bool in_k = mine && rank < static_cast<uint32_t>(q.k);
  double need = static_cast<double>(q.p) * whole * static_cast<double>(r.scale);
  if (q.p < 1.f && whole == 0.0) {  // top-p of what top-k keeps
    uint64_t x = in_k ? w : 0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    if (lane == 0) s.join[warp][0] = x;
    __syncthreads();
    x = 0;
#pragma unroll
    for (int y = 0; y < kQuick / 32; ++y) x += s.join[y][0];
    need = static_cast<double>(q.p) * static_cast<double>(x);
    __syncthreads();
  }
  const double over = above * static_cast<double>(r.scale);
  const float bound = q.mp > 0.f ? min_p_bound(r.m, q) : -INFINITY;
  const bool kept =
      in_k && (rank == 0 || q.p >= 1.f || over + static_cast<double>(before) < need) && v >= bound;
  const bool runs = kept && u && !q.greedy && static_cast<int>(at) != drop;
  const float sc = runs ? fmaf(r.log2w(v), kLn2, gumbel(ue)) : -INFINITY;
  uint64_t sum = kept ? w : 0, last = kept ? ~place : 0, key = runs ? argmax_key(sc, at) : 0;
  if (q.greedy && kept && static_cast<int>(at) != drop) key = argmax_key(0.f, at);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const uint64_t y = __shfl_xor_sync(0xffffffffu, last, o), z = __shfl_xor_sync(0xffffffffu, key, o);
    last = y > last ? y : last;
    key = z > key ? z : key;
  }
  if (lane == 0) {
    s.join[warp][0] = sum;
    s.join[warp][1] = last;
    s.join[warp][2] = key;
  }
  __syncthreads();
  sum = 0;
  last = 0;
  key = 0;
#pragma unroll
  for (int y = 0; y < kQuick / 32; ++y) {
    sum += s.join[y][0];
    last = s.join[y][1] > last ? s.join[y][1] : last;
    key = s.join[y][2] > key ? s.join[y][2] : key;
  }
  out.mass = above + static_cast<double>(sum) / static_cast<double>(r.scale);
  out.cut = ~last;
  out.tok = key ? static_cast<int>(key_index(key)) : -1;
  const bool close = runs && near_best(sc, key_value(key));
  if (__syncthreads_count(close) > 1) {
    const uint64_t dk = close ? double_key(score64(v, r.m, q.T, ue)) : 0ull;
    const uint64_t best = cta_reduce<NT / 32>(dk, OpMaxU64(), s.x);
    const uint64_t low = close && dk == best ? 0xFFFFFFFFull - at : 0ull;
    out.tok = static_cast<int>(0xFFFFFFFFull - cta_reduce<NT / 32>(low, OpMaxU64(), s.x));
  }
  return out;
}

// log2 by the special-function unit (2^-22 of the result; -inf at 0)
__device__ __forceinline__ float fast_log2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A thread's best entry so far.
struct Best {
  float score;  // (z - max)/T - log(-log u); starts at -inf
  float val;
  int at;       // -1: none yet
};

// Takes one more entry into account; equal scores keep the lower index.
__device__ __forceinline__ void offer(Best& b, float v, int i, float log2w, float u) {
  const float sc = fmaf(log2w, kLn2, gumbel(u));
  if (b.at < 0 || sc > b.score || (sc == b.score && i < b.at)) b = Best{sc, v, i};
}

// One pass over this thread's entries with v >= low: f(v, i) for each, and the
// best of those for which it returns true.  A score needs two logarithms; as
// -log u >= 1 - u, (z - max)/T - log(1 - u) bounds it, and few entries pass the best
// score so far by that.  Uniforms are loaded for the packs that hold such an
// entry.
template <typename T, int NT, typename F>
__device__ __forceinline__ void draw_pass(const Row<T, NT>& r, const float* u, float low, Best& best, F f) {
  constexpr int kE = Row<T, NT>::kE, kB = 16 / kE;  // packs in flight
  const float* u0 = u + (r.part.first - r.part.off);
  const bool wide = (reinterpret_cast<uintptr_t>(u0) & 15) == 0;
  for (int j = threadIdx.x; j < r.part.packs; j += kB * NT) {
    uint4 w[kB];
    float uu[kB][kE];
    bool some[kB];
#pragma unroll
    for (int x = 0; x < kB; ++x) w[x] = r.pack(j + x * NT);
#pragma unroll
    for (int x = 0; x < kB; ++x) {
      const int k = j + x * NT;
      const float top = Row<T, NT>::max_of(Row<T, NT>::max_pack(w[x]));
      some[x] = top >= low && top > -INFINITY;
#pragma unroll
      for (int h = 0; h < kE; ++h) uu[x][h] = 0.f;
      if (!some[x]) continue;
      if (wide && (k > 0 || !r.cut_head) && (k + 1 < r.part.packs || !r.cut_tail)) {
        const float4* q = reinterpret_cast<const float4*>(u0 + static_cast<int64_t>(k) * kE);
#pragma unroll
        for (int h = 0; h < kE; h += 4) {
          const float4 y = __ldcs(q + h / 4);
          uu[x][h] = y.x;
          uu[x][h + 1] = y.y;
          uu[x][h + 2] = y.z;
          uu[x][h + 3] = y.w;
        }
      } else {
#pragma unroll
        for (int h = 0; h < kE; ++h) {
          const int e = k * kE + h - r.part.off;
          if (e >= 0 && e < r.part.n) uu[x][h] = __ldcs(u + r.part.first + e);
        }
      }
    }
#pragma unroll
    for (int x = 0; x < kB; ++x) {
      if (!some[x]) continue;
      float v[kE];
      Row<T, NT>::open_pack(w[x], v);
      const int i = static_cast<int>(r.index_of(j + x * NT));
      // bounds in units of log2, and 2^-10 to be safe
      const float bar = best.score * 1.4426950408889634f - 0.0009765625f - fabsf(best.score) * 1e-5f;
#pragma unroll
      for (int h = 0; h < kE; ++h) {
        if (!(v[h] >= low) || !(v[h] > -INFINITY)) continue;
        const bool counts = f(v[h], i + h);
        const float x2 = (v[h] - r.m) * r.c;
        if (counts && !(x2 - fast_log2(1.f - uu[x][h]) < bar)) offer(best, v[h], i + h, x2, uu[x][h]);
      }
    }
  }
}

// The best entry over the cluster; scores that fp32 cannot tell apart are
// formed again in double (a thread's own runner-up aside).
template <typename T, int NT, int kCap>
__device__ int join_best(Row<T, NT>& r, Shared<NT, kCap>& s, const float* u, const Best& b, float temp) {
  constexpr int NW = NT / 32;
  const uint64_t k = b.at >= 0 ? argmax_key(b.score, static_cast<uint32_t>(b.at)) : 0ull;
  const uint64_t win = cluster_reduce<NW>(k, OpMaxU64(), s.x, r.rank, r.size, r.turn);
  if (win == 0) return -1;
  const bool close = b.at >= 0 && near_best(b.score, key_value(win));
  const uint64_t n = cluster_reduce<NW>(close, OpSumU64(), s.x, r.rank, r.size, r.turn);
  if (n <= 1) return static_cast<int>(key_index(win));
  const uint64_t dk = close ? double_key(score64(b.val, r.m, temp, u[b.at])) : 0ull;
  const uint64_t dbest = cluster_reduce<NW>(dk, OpMaxU64(), s.x, r.rank, r.size, r.turn);
  const uint64_t low = close && dk == dbest ? 0xFFFFFFFFull - static_cast<uint32_t>(b.at) : 0ull;
  return static_cast<int>(0xFFFFFFFFull - cluster_reduce<NW>(low, OpMaxU64(), s.x, r.rank, r.size, r.turn));
}

// Gumbel maximum over the row's entries at or above the cut but `drop`.
template <typename T, int NT, int kCap>
__device__ __noinline__ int pick_row(Row<T, NT>& r, Shared<NT, kCap>& s, const float* u, uint64_t cut, int drop,
                                     float temp) {
  Best b{-INFINITY, 0.f, -1};
  if (r.m < INFINITY) {
    const float low = cut_value(cut);
    const int last = static_cast<int>(place_index(cut) < 0x7FFFFFFFu ? place_index(cut) : 0x7FFFFFFFu);
    draw_pass(r, u, low, b, [=](float v, int i) { return i != drop && (v > low || i <= last); });
  } else {  // only the infinite entries have weight
    r.each([&](float v, int64_t i) {
      if (v == r.m && place_of(value_key(v), static_cast<uint32_t>(i)) >= cut && i != drop)
        offer(b, v, static_cast<int>(i), 0.f, u[i]);
    });
  }
  return join_best(r, s, u, b, temp);
}

// Cluster sum of a double, CTAs in rank order.
template <typename T, int NT, int kCap>
__device__ __forceinline__ double cluster_mass(Row<T, NT>& r, Shared<NT, kCap>& s, float w) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) w += __shfl_xor_sync(0xffffffffu, w, o);
  __syncthreads();
  if (lane == 0) s.warp_sum[warp] = __float_as_uint(w);
  __syncthreads();
  if (threadIdx.x < r.size) {
    double d = 0.0;
    for (int x = 0; x < NT / 32; ++x) d += static_cast<double>(__uint_as_float(static_cast<uint32_t>(s.warp_sum[x])));
    *peer(&s.mass[r.rank], threadIdx.x) = d;
  }
  cluster_sync_all(r.size);
  double d = 0.0;
  for (uint32_t o = 0; o < r.size; ++o) d += s.mass[o];
  return d;
}

// Top-p over the whole row where its border lies deep in the row.  A histogram
// linear in the logit, of weights relative to their bin's upper edge (integers:
// nearly equal within a bin, exact sums), finds the bin of the border; a second
// pass sums the weights above that bin, draws among them (`u` given) and lists
// the bin's own entries, which are sorted and filtered as a short list is.
// False: the border fell too close to a bin's edge, or the bin does not fit the
// list.  Else rank 0 holds the list, of which it keeps *kept.
template <typename T, int NT, int kCap>
__device__ __noinline__ bool deep_top_p(Row<T, NT>& r, Shared<NT, kCap>& s, const Ask& q, int64_t V, double row_mass,
                                        const float* u, int* kept, double* kept_mass, Best* best) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const double need = static_cast<double>(q.p) * row_mass;
  // entries this far below the maximum sum to less than (1 - p) / 2 of the row
  const float span = logf(2.f * static_cast<float>(V) / ((1.f - q.p) * static_cast<float>(row_mass))) * q.T;
  if (!(r.m < INFINITY) || !(span > 1e-20f) || !(span < 1e30f)) return false;
  const float per = kLineBins / span, step = r.c / per;  // log2 of a bin's fall
  // the unit of the bins' integers: 2^31 holds every entry of the longest part
  const int most = static_cast<int>(V / r.size) + 2 * Part<T>::kE;
  const float one = static_cast<float>(0x80000000u >> (32 - __clz(most - 1)));
  for (int b = threadIdx.x; b < kLineBins; b += NT) s.line[b] = 0;
  if (threadIdx.x == 0) {
    s.own_count = 0;
    s.own_mass = 0;
    s.taken = 0;
    s.pick[0] = kLineBins;
  }
  __syncthreads();
  const float m = r.m;
  r.each([&](float v, int64_t) {
    const float d = (m - v) * per;
    if (d < static_cast<float>(kLineBins)) {
      const int b = static_cast<int>(d);
      atomicAdd(&s.line[b], __float2uint_rn(fast_exp2((static_cast<float>(b) - d) * step) * one));
    }
  });
  cluster_sync_all(r.size);
  constexpr int kMine = kLineBins / NT;
  double mine[kMine], sum = 0.0;
#pragma unroll
  for (int x = 0; x < kMine; ++x) {
    const int b = threadIdx.x * kMine + x;
    float h = 0.f;
    uint32_t c[kMaxCluster];
#pragma unroll
    for (uint32_t o = 0; o < kMaxCluster; ++o) c[o] = o < r.size ? *peer(&s.line[b], o) : 0u;
#pragma unroll
    for (uint32_t o = 0; o < kMaxCluster; ++o) h += static_cast<float>(c[o]);
    mine[x] = static_cast<double>(h / one * fast_exp2(-static_cast<float>(b) * step));
    sum += mine[x];
  }
  double inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  if (lane == 31) s.warp_sum[warp] = __double_as_longlong(inc);
  __syncthreads();
  double before = inc - sum;
  for (int w = 0; w < warp; ++w) before += __longlong_as_double(s.warp_sum[w]);
#pragma unroll
  for (int x = 0; x < kMine; ++x) {
    if (before < need && before + mine[x] >= need) s.pick[0] = threadIdx.x * kMine + x;
    before += mine[x];
  }
  __syncthreads();
  const int bin = static_cast<int>(s.pick[0]);
  if (bin == kLineBins) return false;
  // second pass
  const float edge = static_cast<float>(bin), end = edge + 1.f;
  float w = 0.f;
  uint32_t* taken = peer(&s.taken, 0);
  uint64_t* list = peer(s.list, 0);
  const float low = m - end / per * 1.0001f - fabsf(m) * 1e-6f;  // no entry of the bin lies below
  auto visit = [&](float v, int i) {
    const float d = (m - v) * per;
    if (d < edge) {
      w += fast_exp2((v - m) * r.c);
      return true;
    }
    if (d < end) {
      const uint32_t at = atomicAdd(taken, 1u);
      if (at < kCap) list[at] = place_of(value_key(v), static_cast<uint32_t>(i));
      atomicAdd(&s.own_count, 1u);
      atomicAdd(reinterpret_cast<unsigned long long*>(&s.own_mass), r.weight(v));
    }
    return false;
  };
  if (u) {
    draw_pass(r, u, low, *best, visit);
  } else {
    r.each([&](float v, int64_t i) {
      if (v >= low) visit(v, static_cast<int>(i));
    });
  }
  const double above = cluster_mass(r, s, w);
  uint32_t count;
  uint64_t mass;
  close_list(r, s, &count, &mass);
  if (count > kCap || !(above < need) ||
      above + static_cast<double>(mass) / static_cast<double>(r.scale) < need)
    return false;
  if (r.rank == 0) {
    sort_list<NT>(s.list, static_cast<int>(count));
    *kept = filter_list(r, s, q, static_cast<int>(count), above, row_mass, kept_mass);
  }
  return true;
}

// The cut and the kept mass of any row, by radix descents.
template <typename T, int NT, int kCap>
__device__ __noinline__ uint64_t wide_cut(Row<T, NT>& r, Shared<NT, kCap>& s, const FilterArgs& a, const Ask& q,
                                          double* kept_mass) {
  uint64_t cut = 1ull << 32;  // every unmasked entry
  if (q.k < a.V) {
    uint64_t valid = 0;
    r.each([&](float v, int64_t) { valid += v > -INFINITY; });
    valid = cluster_reduce<NT / 32>(valid, OpSumU64(), s.x, r.rank, r.size, r.turn);
    if (static_cast<uint64_t>(q.k) < valid) cut = find_cut<T, NT, kCap, false>(r, s, cut, q.k, a.idx_bits);
  }
  if (q.p < 1.f) {
    // entries are taken while the sum before them is below p times w
    const uint64_t w = mass_from(r, s, cut);
    uint64_t need = static_cast<uint64_t>(ceil(static_cast<double>(q.p) * static_cast<double>(w)));
    if (need < 1) need = 1;
    if (need < w) cut = find_cut<T, NT, kCap, true>(r, s, cut, need, a.idx_bits);
  }
  if (q.mp > 0.f) {
    const uint64_t c = place_of(value_key(min_p_bound(r.m, q)), 0xFFFFFFFFu);
    if (c > cut) cut = c;
  }
  const float low = cut_value(cut);
  const int64_t last = place_index(cut);
  float w = 0.f;
  r.each([&](float v, int64_t i) {
    if (v > -INFINITY && (v > low || (v == low && i <= last))) w += fast_exp2(r.log2w(v));
  });
  *kept_mass = cluster_mass(r, s, w);
  return cut;
}

// Tries the short list for a row's filters; true: rank 0's threads have the
// verdict (with a draw from u, if given).
template <typename T, int NT, int kCap>
__device__ bool listed_row(Row<T, NT>& r, Shared<NT, kCap>& s, const Scan<T, NT>& sc, const FilterArgs& a,
                           const Ask& q, float low, double row_mass, const float* u, int drop, Verdict* out) {
  int target = 0;
  float t = -INFINITY;
  const bool of_row = q.k >= a.V && q.p < 1.f;  // top-p refers to the whole row
  if (q.k == 1) {
    t = r.m;
  } else if (q.k < a.V) {
    target = q.k;
  } else if (of_row) {
    target = kFewTarget;
  } else if (q.mp > 0.f) {
    t = min_p_bound(r.m, q);
  } else {
    return false;
  }
  if (target > kCap) return false;
  uint32_t count;
  uint64_t mass;
  if (!short_list(r, s, sc, a.V, low, target, &t, of_row, &count, &mass)) return false;
  // the list has to hold top-p's border, or all that min-p leaves
  if (of_row && static_cast<double>(mass) < static_cast<double>(q.p) * row_mass * static_cast<double>(r.scale) &&
      static_cast<int64_t>(count) < a.V && !(q.mp > 0.f && min_p_bound(r.m, q) >= t))
    return false;
  if (r.rank == 0) *out = settle_list(r, s, q, static_cast<int>(count), 0.0, of_row ? row_mass : 0.0, u, drop);
  return true;
}

template <typename T, int NT>
__device__ __forceinline__ float log_prob(const Row<T, NT>& r, int tok, double kept) {
  return r.log2w(r.at(tok)) * kLn2 - logf(static_cast<float>(kept));
}

// A row whose sum of weights the scan has to form: nothing filters it, or
// top-p refers to all of it.
__device__ __forceinline__ bool wants_mass(const FilterArgs& a, const Ask& q) {
  return q.k >= a.V && (q.p < 1.f || q.mp == 0.f) && !q.greedy;
}

// Common start of the kernels: shared counters, the other kernels' results.
template <int NT, int kCap>
__device__ __forceinline__ void start(Shared<NT, kCap>& s, uint32_t size) {
  if (threadIdx.x == 0) {
    s.own_mass = 0;
    s.own_count = 0;
    s.taken = 0;
    s.queued = 0;
  }
  for (int b = threadIdx.x; b < kGroupBins; b += NT) s.groups[b] = 0;
  __syncthreads();
  if (size > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  pdl_wait();
}

constexpr int kShortCap = 1024;
constexpr int kThr = 256;

template <typename T>
__global__ void __launch_bounds__(kThr, 4) sample_rows_kernel(const FilterArgs a) {
  extern __shared__ __align__(16) uint8_t raw[];
  using S = Shared<kThr, kShortCap>;
  S& s = *reinterpret_cast<S*>(raw);
  const uint32_t size = cluster_size();
  const int64_t row = blockIdx.x / size;
  start(s, size);
  const Ask q = read_ask(a, row);
  Row<T, kThr> r;
  r.c = inv_temperature(q.T);
  r.open(a, row);
  const bool want_mass = wants_mass(a, q);
  Scan<T, kThr> sc;
  scan_row(r, want_mass, sc);
  float low;
  double row_mass;
  const bool some = join_scan(r, s, sc, want_mass, &low, &row_mass);
  const float* u = a.u + row * a.ld_u;
  int tok = -1;
  float lp = -INFINITY;
  if (q.ok && some) {
    Verdict v;
    Best best{-INFINITY, 0.f, -1};
    int n = 0;
    if (listed_row(r, s, sc, a, q, low, row_mass, u, -1, &v)) {
      if (r.rank != 0) return;
      tok = v.tok;
    } else if (q.k >= a.V && q.p < 1.f && q.mp == 0.f &&
               deep_top_p(r, s, q, a.V, row_mass, u, &n, &v.mass, &best)) {
      if (r.rank == 0) {
        for (int i = threadIdx.x; i < n; i += kThr) {
          const uint32_t x = place_index(s.list[i]);
          const float z = key_to_value(static_cast<uint32_t>(s.list[i] >> 32));
          offer(best, z, static_cast<int>(x), r.log2w(z), u[x]);
        }
      }
      tok = join_best(r, s, u, best, q.T);
    } else {
      uint64_t cut = 1ull << 32;
      if (want_mass && q.p >= 1.f) {
        v.mass = row_mass;
      } else {
        cut = wide_cut(r, s, a, q, &v.mass);
      }
      tok = q.greedy ? static_cast<int>(place_index(cut)) : pick_row(r, s, u, cut, -1, q.T);
    }
    if (tok >= 0) lp = log_prob(r, tok, v.mass);
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
template <typename T>
__global__ void __launch_bounds__(kThr, 4) accept_rows_kernel(const FilterArgs a) {
  extern __shared__ __align__(16) uint8_t raw[];
  using S = Shared<kThr, kShortCap>;
  S& s = *reinterpret_cast<S*>(raw);
  const uint32_t size = cluster_size();
  const int64_t j = blockIdx.x / size / a.rows_used;
  const int rr = static_cast<int>(blockIdx.x / size - j * a.rows_used);
  const int64_t row = j * a.R + rr;
  start(s, size);
  const Ask q = read_ask(a, j);
  Row<T, kThr> r;
  r.c = inv_temperature(q.T);
  r.open(a, row);
  const bool want_mass = wants_mass(a, q);
  Scan<T, kThr> sc;
  scan_row(r, want_mass, sc);
  float low;
  double row_mass;
  const bool some = join_scan(r, s, sc, want_mass, &low, &row_mass);
  RowCut out;
  out.cut = ~0ull;
  out.m = r.m;
  out.accept = 0;
  out.tok = -1;
  if (q.ok && some) {
    const int drop = rr < a.D ? a.draft[j * a.D + rr] : -1;
    Verdict v;
    int n = 0;
    if (listed_row(r, s, sc, a, q, low, row_mass, a.u + j * a.ld_u, drop, &v)) {
      if (r.rank != 0) return;
      out.cut = v.cut;
      out.tok = v.tok;
    } else {
      out.tok = -2;  // not drawn yet
      if (q.k >= a.V && q.p < 1.f && q.mp == 0.f &&
          deep_top_p(r, s, q, a.V, row_mass, static_cast<const float*>(nullptr), &n, &v.mass,
                     static_cast<Best*>(nullptr))) {
        if (r.rank != 0) return;
        out.cut = s.list[n - 1];
      } else if (want_mass && q.p >= 1.f) {
        out.cut = 1ull << 32;
        v.mass = row_mass;
      } else {
        out.cut = wide_cut(r, s, a, q, &v.mass);
      }
    }
    if (drop >= 0 && drop < a.V) {
      const float z = r.at(drop);
      const uint32_t key = value_key(z);
      if (key != 0 && place_of(key, static_cast<uint32_t>(drop)) >= out.cut)
        out.accept = static_cast<double>(a.u_accept[j * a.D + rr]) <
                     static_cast<double>(r.weight(z)) / static_cast<double>(r.scale) / v.mass;
    }
  }
  if (r.rank == 0 && threadIdx.x == 0) a.cuts[row] = out;
}

// One cluster per sequence: leading accepts, the draw at the row after them if
// it is still to be made, and the outputs.
template <typename T>
__global__ void __launch_bounds__(kThr) accept_pick_kernel(const FilterArgs a) {
  extern __shared__ __align__(16) uint8_t raw[];
  using S = Shared<kThr, kShortCap>;
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
      Row<T, kThr> r;
      r.c = inv_temperature(q.T);
      r.open(a, row);
      r.m = c.m;
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
template <typename T>
__global__ void __launch_bounds__(kThr, 4) top_rows_kernel(const FilterArgs a) {
  extern __shared__ __align__(16) uint8_t raw[];
  using S = Shared<kThr, kTopCap>;
  S& s = *reinterpret_cast<S*>(raw);
  const uint32_t size = cluster_size();
  const int64_t row = blockIdx.x / size;
  start(s, size);
  Row<T, kThr> r;
  r.c = inv_temperature(a.T);
  r.open(a, row);
  Scan<T, kThr> sc;
  const bool want_mass = a.lse != nullptr;
  scan_row(r, want_mass, sc);
  float low, t = -INFINITY;
  double row_mass;
  const bool some = join_scan(r, s, sc, want_mass, &low, &row_mass);
  uint32_t n = 0;
  uint64_t mass;
  if (some && !short_list(r, s, sc, a.V, low, a.K, &t, false, &n, &mass)) {
    // ties or a clustered row: find the exact border, then list
    uint64_t cut = 1ull << 32, valid = 0;
    r.each([&](float v, int64_t) { valid += v > -INFINITY; });
    valid = cluster_reduce<kThr / 32>(valid, OpSumU64(), s.x, r.rank, r.size, r.turn);
    if (static_cast<uint64_t>(a.K) < valid)
      cut = find_cut<T, kThr, kTopCap, false>(r, s, cut, a.K, a.idx_bits);
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
    n = static_cast<uint64_t>(a.K) < valid ? static_cast<uint32_t>(a.K) : static_cast<uint32_t>(valid);
  }
  if (r.rank != 0) return;
  sort_list<kThr>(s.list, static_cast<int>(n));
  for (uint32_t i = threadIdx.x; i < static_cast<uint32_t>(a.K); i += kThr) {
    const uint64_t c = i < n ? s.list[i] : 0;
    a.val[row * a.K + i] = c ? key_to_value(static_cast<uint32_t>(c >> 32)) : -INFINITY;
    a.idx[row * a.K + i] = c ? static_cast<int>(place_index(c)) : -1;
  }
  if (a.lse && threadIdx.x == 0) {
    // an infinite maximum is the sum
    const float l = r.m < INFINITY ? static_cast<float>(static_cast<double>(r.m) / static_cast<double>(a.T) +
                                                        static_cast<double>(logf(static_cast<float>(row_mass))))
                                   : r.m;
    a.lse[row] = some ? l : -INFINITY;
  }
}

cudaError_t launch_rows(const void* kern, int64_t rows, int parts, size_t smem, const FilterArgs& a,
                        cudaStream_t st) {
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  FilterArgs b = a;
  void* args[] = {&b};
  return launch_kc(kern, dim3((unsigned)(rows * parts)), dim3(kThr), smem, st, true, dim3(parts), args);
}

// CTAs per row: enough to occupy the GPU, at least 4 KB each.
int pick_parts(int64_t V, int64_t rows, size_t esize) {
  int parts = 1;
  while (parts < kMaxCluster && rows * parts < 4 * num_sms() && V * (int64_t)esize / (2 * parts) >= 4096) parts *= 2;
  return parts;
}

template <typename T>
cudaError_t launch_sample(const FilterArgs& a, int64_t rows, cudaStream_t st) {
  return launch_rows((const void*)sample_rows_kernel<T>, rows, pick_parts(a.V, rows, sizeof(T)),
                     sizeof(Shared<kThr, kShortCap>), a, st);
}
template <typename T>
cudaError_t launch_accept(const FilterArgs& a, int64_t b, cudaStream_t st) {
  const int64_t rows = b * a.rows_used;
  const size_t smem = sizeof(Shared<kThr, kShortCap>);
  cudaError_t e = launch_rows((const void*)accept_rows_kernel<T>, rows, pick_parts(a.V, rows, sizeof(T)), smem, a, st);
  if (e != cudaSuccess) return e;
  return launch_rows((const void*)accept_pick_kernel<T>, b, pick_parts(a.V, b, sizeof(T)), smem, a, st);
}
template <typename T>
cudaError_t launch_top(const FilterArgs& a, int64_t rows, cudaStream_t st) {
  return launch_rows((const void*)top_rows_kernel<T>, rows, pick_parts(a.V, rows, sizeof(T)),
                     sizeof(Shared<kThr, kTopCap>), a, st);
}

void finish(FilterArgs& a) {
  a.idx_bits = 0;
  while (((int64_t)1 << a.idx_bits) < a.V) ++a.idx_bits;
  a.scale = ldexpf(1.f, 62 - a.idx_bits);
}

}  // namespace

cudaError_t filter_sample(FilterArgs a, int dtype, int64_t rows, cudaStream_t st) {
  finish(a);
  if (dtype == 0) return launch_sample<float>(a, rows, st);
  if (dtype == 1) return launch_sample<__half>(a, rows, st);
  return launch_sample<__nv_bfloat16>(a, rows, st);
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
  if (dtype == 0) return launch_top<float>(a, rows, st);
  if (dtype == 1) return launch_top<__half>(a, rows, st);
  return launch_top<__nv_bfloat16>(a, rows, st);
}

}  // namespace dfl
