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
// A row is one cluster's: one pass from HBM takes the row's maximum, the maxima
// of its groups of entries and, where top-p refers to the whole row, its sum of
// weights.  Rows whose answer is among a few hundred entries (top-k, a peaked
// top-p, min-p) list the entries above a bound read off the groups' maxima, and
// rank 0 settles them.  Others take a histogram of the weights and one more pass
// (deep top-p), one more pass (min-p), the scan's own draw (no filter), or, for
// what none of these can hold (top-k above 1024, thousands of equal values), radix
// descents over the places.  All passes after the first read from L2.
//
// Sums that decide which entries are kept are of integers wherever their order
// is not fixed (w scaled by a power of two that keeps V of them below 2^62; the
// rounding of one weight, 2^-45 of the largest at V = 152 k, is far below the
// 2^-23 of its exponential), and floats in a fixed order elsewhere, so every
// result repeats bit for bit.
//
// Large batches are bound by HBM while they stream, and then by random re-reads
// and one CTA's ranking (512 x 151936 bf16, top-k with top-p: 52 us, 32 of them at
// 4.9 TB/s; unfiltered, where every uniform counts too, 86 us, 5.4 TB/s); small
// ones by the chain of launch, cluster barriers and L2 round trips (one row 12 us).
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
// Groups the short list takes at most where top-k does not say (512 x 151936 bf16,
// top-p: 180 / 149 / 153 / 166 us with 128 / 192 / 256 / 512).
constexpr int kGroupTarget = 192;
constexpr float kGroupOne = 131072.f;  // 2^17: a weight of one in sums over groups (at most 2^14 of them)
constexpr int kShareRows = 2048;      // rows looked through at a time by a second launch
constexpr int kShareMost = 64;        // of which a cluster takes at most so many
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
  int beside[2];                     // the bins before and after it that hold entries
  uint64_t warp_sum[NT / 32];
  uint64_t list_mass[kMaxCluster];   // what each CTA put on the list, by weight and by count
  uint32_t list_count[kMaxCluster];
  uint32_t highest[kMaxCluster], lowest[kMaxCluster];  // of each CTA's groups' maxima
  float mass[kMaxCluster];           // each CTA's sum of weights, from the scan
  float sums[kMaxCluster];           // and from a pass over the entries kept
  uint64_t own_mass;
  uint64_t need;                     // top-p keeps entries while the sum before them is below this
  float bound;                       // min-p's bound on a logit
  uint32_t own_count, taken, queued;
  uint32_t groups[kGroupBins], weights[kGroupBins];  // groups' maxima: their number and weights
  union {
    uint64_t list[kCap];  // places; complete in rank 0
    struct {
      unsigned long long mass[kBins];
      uint32_t count[kBins];
    } bin;
  };
  alignas(16) uint32_t line[kLineBins];
  ulonglong2 entry[kQuick];          // a quick list's places and weights
  uint64_t half_before[kQuick];
  uint32_t half_rank[kQuick];
  uint64_t join[NT / 32][3];
  float val;
  uint32_t bar;                      // key of the best score seen by any thread of the CTA
  int64_t rows[kShareMost];          // a cluster's rows of a second launch
};

// One row as a cluster sees it.  Each CTA reads its part of the row from
// global memory in 16-byte packs, thread t the packs t, t + NT, ...; a pass
// after the first finds them in L2.
template <typename T, int NT>
struct Row {
  static constexpr int kPer = Pack<T>::kPer, kE = Part<T>::kE;
  const T* p;
  Part<T> part;
  uint32_t rank, size;
  float m;             // the row's maximum
  float c;             // log2(e) / temperature
  float scale;         // weights become integers by this power of two
  float unit;          // its inverse
  int turn;

  __device__ __forceinline__ void open(const FilterArgs& a, int64_t row) {
    p = static_cast<const T*>(a.logits) + row * a.ld;
    rank = cluster_rank();
    size = cluster_size();
    turn = 0;
    scale = a.scale;
    unit = a.unit;
    part.cut(p, a.V, static_cast<int>(rank), static_cast<int>(size));
  }
  __device__ __forceinline__ float at(int64_t i) const { return to_f32(p[i]); }
  __device__ __forceinline__ int64_t index_of(int j) const { return part.index_of(j); }
  __device__ __forceinline__ float log2w(float v) const { return log2_weight(v, m, c); }
  __device__ __forceinline__ unsigned long long weight(float v) const {
    return __float2ull_rn(exp2f(log2w(v)) * scale);
  }
  __device__ __forceinline__ uint4 pack(int j) const { return part.pack(j); }
  static __device__ __forceinline__ void open_pack(const uint4& w, float* v) { Part<T>::open(w, v); }
  static __device__ __forceinline__ uint32_t max_pack(const uint4& w) { return Part<T>::max_words(w); }
  static __device__ __forceinline__ float max_of(uint32_t w) { return Part<T>::max_of(w); }
  // Entry h (not a constant) of a pack.
  static __device__ __forceinline__ float pick_of(const uint4& w, int h) {
    const int x = h / kPer;
    const uint32_t word = x == 0 ? w.x : (x == 1 ? w.y : (x == 2 ? w.z : w.w));
    float v[kPer];
    Pack<T>::open(word, v);
    return h % kPer ? v[kPer - 1] : v[0];
  }
  // The uniforms of pack j's entries (0 where it has none); `wide`: u0, those
  // of pack 0, allows 16-byte loads.
  __device__ __forceinline__ void uniforms(const float* u, const float* u0, bool wide, int j, float* out) const {
#pragma unroll
    for (int h = 0; h < kE; ++h) out[h] = 0.f;
    if (j >= part.packs) return;
    if (wide && part.whole(j)) {
      const float4* q = reinterpret_cast<const float4*>(u0 + static_cast<int64_t>(j) * kE);
#pragma unroll
      for (int h = 0; h < kE; h += 4) {
        const float4 y = __ldcs(q + h / 4);
        out[h] = y.x;
        out[h + 1] = y.y;
        out[h + 2] = y.z;
        out[h + 3] = y.w;
      }
      return;
    }
#pragma unroll
    for (int h = 0; h < kE; ++h) {
      const int e = j * kE + h - part.off;
      if (e >= 0 && e < part.n) out[h] = __ldcs(u + part.first + e);
    }
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

// A cut after the last entry kept when entries at or above `lo` are taken in
// order until the taken ones reach `need` (by count, or by weight): no entry lies
// between the two, but the cut's low bits need not be the entry's.  A radix
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
    // the whole bin is taken, or it holds only the border entry; entries below `lo`
    // may lie in it too
    if (top == 0 || in_bin == 1 || (!kMass && in_bin == need)) return pre << top > lo ? pre << top : lo;
  }
}

// The value of a cut's entry; -inf where every unmasked entry is kept.
__device__ __forceinline__ float cut_value(uint64_t cut) {
  const uint32_t k = static_cast<uint32_t>(cut >> 32);
  return k > 0x007FFFFFu ? key_to_value(k) : -INFINITY;
}

// Place of the row's first entry.
template <typename T, int NT, int kCap>
__device__ uint64_t first_place(Row<T, NT>& r, Shared<NT, kCap>& s) {
  uint64_t best = 0;
  r.each([&](float v, int64_t i) {
    const uint64_t c = place_of(value_key(v), static_cast<uint32_t>(i));
    if (v == r.m && c > best) best = c;
  });
  return cluster_reduce<NT / 32>(best, OpMaxU64(), s.x, r.rank, r.size, r.turn);
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

// The two borders that are formed in double, by one thread (the unit is narrow);
// seen by all after the next barrier.  min-p: the smallest float at or above
// its bound.  top-p: sums are integers, so "below p times the whole" is "below
// the next integer", and as the first entry is kept whatever p, 1 stands for 0.
template <int NT, int kCap>
__device__ __forceinline__ void set_bound(Shared<NT, kCap>& s, float m, const Ask& q) {
  if (threadIdx.x != 0) return;
  const double t = static_cast<double>(m) + static_cast<double>(q.T) * log(static_cast<double>(q.mp));
  float f = static_cast<float>(t);
  if (static_cast<double>(f) < t) f = nextafterf(f, INFINITY);
  s.bound = f > m ? m : f;
}
template <int NT, int kCap>
__device__ __forceinline__ void set_need(Shared<NT, kCap>& s, float p, uint64_t whole) {
  if (threadIdx.x != 0) return;
  const uint64_t sum = static_cast<uint64_t>(ceil(static_cast<double>(p) * static_cast<double>(whole)));
  s.need = p >= 1.f ? ~0ull : sum > 0 ? sum : 1;
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

// log2 by the special-function unit (2^-22 of the result; -inf at 0)
__device__ __forceinline__ float fast_log2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <int N>
__device__ __forceinline__ float pick_float(const float* v, int h) {
  float r = v[0];
#pragma unroll
  for (int x = 1; x < N; ++x) r = x == h ? v[x] : r;
  return r;
}

// A thread's best entry so far.  Scores are formed in fp32, and those that it cannot
// tell apart again in double: at once where a few threads hold the listed entries
// (offer<true>); a pass over a row has no registers for that, and keeps the score of
// the next best.  Where that comes as near as the row's best, one more pass settles
// the row (settle_row: some 1e-5 apart, so not once in 10^5 rows).
struct Best {
  float score;  // (z - max)/T, or z/T, - log(-log u); starts at -inf
  float next;   // the highest of the thread's others
  float val;
  int at;       // -1: none yet
};
__device__ __forceinline__ Best no_best() { return Best{-INFINITY, -INFINITY, 0.f, -1}; }

// Whether an entry comes before another by its score in double, equal ones by
// index.
__device__ __noinline__ bool beats64(const float* u, float v, int i, float bv, int bi, float m, float temp) {
  const double x = score64(v, m, temp, u[i]), y = score64(bv, m, temp, u[bi]);
  return x > y || (x == y && i < bi);
}

// Takes one more entry into account, whose uniform is ui; equal scores keep the lower
// index.  With kExact: u, the row's uniforms, its maximum and temperature.
template <bool kExact = false>
__device__ __forceinline__ void offer(Best& b, float v, int i, float log2w, float ui, const float* u = nullptr,
                                      float m = 0.f, float temp = 1.f) {
  const float sc = fmaf(log2w, kLn2, gumbel(ui));
  bool better = b.at < 0 || sc > b.score || (sc == b.score && i < b.at);
  if (kExact) {
    if (b.at >= 0 && near_best(sc, b.score) && near_best(b.score, sc)) better = beats64(u, v, i, b.val, b.at, m, temp);
  } else {
    b.next = fmaxf(b.next, fminf(sc, b.score));
  }
  if (better) b = Best{sc, b.next, v, i};
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

// A thread's sum of weights relative to its maximum, whatever its entries are.
template <typename T, int NT>
__device__ __noinline__ float careful_sum(const Part<T> part, const float c, const float top) {
  float sum = 0.f;
  for (int j = threadIdx.x; j < part.packs; j += NT) {
    float v[Part<T>::kE];
    Part<T>::open(part.pack(j), v);
#pragma unroll
    for (int h = 0; h < Part<T>::kE; ++h)
      if (v[h] > -INFINITY) sum += fast_exp2(log2_weight(v[h], top, c));
  }
  return sum;
}

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
        const float ref = reference(top, r.c);
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
  if (t.careful) t.sum = careful_sum<T, NT>(r.part, r.c, t.top);
}

// A first bar for a drawing pass, below the best score among the entries of the
// threads' first packs with v >= from: -log u <= (1 - u) / u bounds a score from
// below without a logarithm of a number next to one.  Without a bar every thread
// would score its first entries in full.
template <typename T, int NT, int kCap>
__device__ __forceinline__ void first_bar(const Row<T, NT>& r, Shared<NT, kCap>& s, const float* u, const float* u0,
                                          bool wide, float from, float m) {
  constexpr int kE = Row<T, NT>::kE;
  const int j = threadIdx.x;
  float uu[kE], v[kE], best = -INFINITY;
  Row<T, NT>::open_pack(r.pack(j), v);
  r.uniforms(u, u0, wide, j, uu);
#pragma unroll
  for (int h = 0; h < kE; ++h) {
    const float g = (v[h] - m) * r.c - fast_log2(1.f - uu[h]) + fast_log2(uu[h]);  // u = 0: -inf
    if (v[h] >= from && v[h] > -INFINITY) best = fmaxf(best, g);
  }
  const uint32_t key = __reduce_max_sync(0xffffffffu, value_key(best * kLn2 - 0.00390625f - fabsf(best) * 1e-5f));
  if ((threadIdx.x & 31) == 0) atomicMax(&s.bar, key);
  __syncthreads();
}

// The scan of a row that nothing filters, and its draw, in one pass over the
// logits and the uniforms: scores are taken as z/T - log(-log u), before the
// maximum is known (the caller draws again where z/T is too large for that).
template <typename T, int NT, int kCap>
__device__ __forceinline__ void scan_and_draw(const Row<T, NT>& r, Shared<NT, kCap>& s, const float* u,
                                              Scan<T, NT>& t, Best& best) {
  constexpr int kE = Row<T, NT>::kE, kB = 16 / kE;
  const float* u0 = u + (r.part.first - r.part.off);
  const bool wide = (reinterpret_cast<uintptr_t>(u0) & 15) == 0;
  uint32_t mx = Pack<T>::kNegInf;
  t.ref = 0.f;
  t.sum = 0.f;
  bool any = false, odd = false;
  first_bar(r, s, u, u0, wide, -INFINITY, 0.f);
  for (int j = threadIdx.x; j < r.part.packs; j += kB * NT) {
    uint4 w[kB];
    float uu[kB][kE];
#pragma unroll
    for (int x = 0; x < kB; ++x) {
      w[x] = r.pack(j + x * NT);
      r.uniforms(u, u0, wide, j + x * NT, uu[x]);
    }
#pragma unroll
    for (int x = 0; x < kB; ++x) {
      const uint32_t pm = Row<T, NT>::max_pack(w[x]);
      mx = Pack<T>::max2(mx, pm);
      const float top = Row<T, NT>::max_of(pm);
      if (!(top > -INFINITY)) continue;
      const float ref = reference(top, r.c);
      if (!any || ref > t.ref) {
        if (any) t.sum *= fast_exp2(t.ref - ref);
        t.ref = ref;
        any = true;
        odd |= !(fabsf(ref) < kRefMax);
      }
      const float seen = key_to_value(*reinterpret_cast<volatile uint32_t*>(&s.bar));
      const float bar = seen * 1.4426950408889634f - 0.0009765625f - fabsf(seen) * 1e-5f;
      const float reach = fminf(fast_exp2(bar - t.ref), 1e30f);
      float v[kE], some = 0.f, peak = -INFINITY;
      Row<T, NT>::open_pack(w[x], v);
#pragma unroll
      for (int h = 0; h < kE; ++h) {
        const float e = fast_exp2(fmaf(v[h], r.c, -t.ref));
        some += e;
        peak = fmaxf(peak, fmaf(uu[x][h], reach, e));  // w >= 2^bar (1 - u)
      }
      t.sum += some;
      if (peak >= reach) {
        const int i = static_cast<int>(r.index_of(j + x * NT));
#pragma unroll 1
        for (int h = 0; h < kE; ++h) {
          const float z = Row<T, NT>::pick_of(w[x], h), y = pick_float<kE>(uu[x], h);
          if (z > -INFINITY && !(fmaf(z, r.c, -fast_log2(1.f - y)) < bar)) offer(best, z, i + h, z * r.c, y);
        }
        const uint32_t key = value_key(best.score);
        if (key > *reinterpret_cast<volatile uint32_t*>(&s.bar)) atomicMax(&s.bar, key);
      }
    }
  }
  t.top = Row<T, NT>::max_of(mx);
#pragma unroll
  for (int x = 0; x < kGroups; ++x) t.group[x] = t.top;
  t.careful = odd || !(t.sum < INFINITY);  // (see scan_row)
  if (t.careful) t.sum = careful_sum<T, NT>(r.part, r.c, t.top);
}

// The row's maximum (false: no entry counts), the lowest of the groups' maxima
// that are not -inf, and where wanted the row's sum of weights.
template <typename T, int NT, int kCap>
__device__ bool join_scan(Row<T, NT>& r, Shared<NT, kCap>& s, const Scan<T, NT>& t, bool want_mass, float* low,
                          float* row_mass) {
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
      float w = 0.f;
#pragma unroll
      for (int x = 0; x < NT / 32; ++x) w += __uint_as_float(static_cast<uint32_t>(s.warp_sum[x]));
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
  *row_mass = 0.f;
  if (want_mass && hi != 0)
    for (uint32_t o = 0; o < r.size; ++o)
      if (s.highest[o]) *row_mass += s.mass[o] * fast_exp2(r.log2w(key_to_value(s.highest[o])));
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
  if (s.queued > kCap) {  // more groups than the list holds entries
    if (threadIdx.x == 0) s.own_count = kCap + 1;
    return;
  }
  uint64_t* list = peer(s.list, 0);
  const int lane = threadIdx.x & 31;
  const uint32_t deep = (r.part.packs + kGroups * NT - 1) / (kGroups * NT), units = s.queued * deep;
  uint64_t listed = 0;  // as integers: which thread takes which pack is not fixed
  uint32_t count = 0;
  for (uint32_t y0 = threadIdx.x - lane; y0 < units; y0 += 4 * NT) {
    uint4 w[4];
    int at[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const uint32_t y = y0 + lane + x * NT, g = y / deep;
      at[x] = y < units ? queue[g] + static_cast<int>(y - g * deep) * (kGroups * NT) : r.part.packs;
      w[x] = r.pack(at[x]);
    }
    uint32_t hits = 0;  // kE bits a pack
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      float v[kE];
      Row<T, NT>::open_pack(w[x], v);
#pragma unroll
      for (int h = 0; h < kE; ++h) hits |= (v[h] >= t && v[h] > -INFINITY ? 1u : 0u) << (x * kE + h);
    }
    // one reservation a warp: a round trip to rank 0 for all of its packs
    const uint32_t n = __popc(hits);
    uint32_t before = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, before, o);
      if (lane >= o) before += y;
    }
    uint32_t base = 0;
    if (lane == 31 && before > 0) {
      count += before;
      base = r.size == 1 ? atomicAdd(&s.taken, before) : atomicAdd(peer(&s.taken, 0), before);
    }
    base = __shfl_sync(0xffffffffu, base, 31) + before - n;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      uint32_t some = hits >> (x * kE) & ((1u << kE) - 1);
      const int64_t i = r.index_of(at[x]);
      while (some) {
        const int h = __ffs(some) - 1;
        some &= some - 1;
        const float z = Row<T, NT>::pick_of(w[x], h);
        if (base < kCap) list[base] = place_of(value_key(z), static_cast<uint32_t>(i + h));
        ++base;
        if (want_mass) listed += r.weight(z);
      }
    }
  }
  if (count > 0) atomicAdd(&s.own_count, count);
  if (listed > 0) atomicAdd(reinterpret_cast<unsigned long long*>(&s.own_mass), static_cast<unsigned long long>(listed));
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
// entries that reach t go to rank 0's list.  With want > 0, t may come earlier:
// where the maxima's own weights, a lower bound of the entries', sum to `want`;
// a row whose first `target` groups hold less than half of it is not listed
// (unless `sure`).  target 0: t is given.  Returns false where there is no list;
// else count and, with want, mass are those of the list.
template <typename T, int NT, int kCap>
__device__ bool short_list(Row<T, NT>& r, Shared<NT, kCap>& s, const Scan<T, NT>& sc, int64_t V, float low, int target,
                           float* bound, float want, bool sure, uint32_t* count, uint64_t* mass) {
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
        const int at = b < 0 ? 0 : (b < kGroupBins ? b : kGroupBins - 1);
        atomicAdd(&s.groups[at], 1u);
        if (want > 0.f) atomicAdd(&s.weights[at], __float2uint_rz(fast_exp2(r.log2w(sc.group[x])) * kGroupOne));
      }
    }
    cluster_sync_all(r.size);
    // the bin in which the maxima, from the highest, reach the target: number
    // and weight side by side in one word
    static_assert(kGroupBins == NT, "one thread per bin");
    uint64_t c[kMaxCluster], n = 0;
#pragma unroll
    for (uint32_t o = 0; o < kMaxCluster; ++o) {
      c[o] = 0;
      if (o < r.size) {
        c[o] = static_cast<uint64_t>(*peer(&s.groups[threadIdx.x], o)) << 32;
        if (want > 0.f) c[o] += *peer(&s.weights[threadIdx.x], o);
      }
    }
#pragma unroll
    for (uint32_t o = 0; o < kMaxCluster; ++o) n += c[o];
    uint64_t inc = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t u = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += u;
    }
    if (lane == 31) s.warp_sum[warp] = inc;
    if (threadIdx.x == 0) s.pick[0] = kGroupBins;
    __syncthreads();
    for (int w = 0; w < warp; ++w) inc += s.warp_sum[w];
    // (a margin of 2^-10: the list's own sum is compared with what is needed)
    const uint32_t weight = want > 0.f ? __float2uint_ru(want * kGroupOne * 1.0009765625f) : 0xFFFFFFFFu;
    const auto reached = [=](uint64_t x) {
      return (x >> 32) >= static_cast<uint32_t>(target) || static_cast<uint32_t>(x) >= weight;
    };
    if (reached(inc) && !reached(inc - n)) {
      s.pick[0] = threadIdx.x;
      s.pick[1] = static_cast<uint32_t>(inc) < weight / 2 && !sure;
    }
    __syncthreads();
    const int b = static_cast<int>(s.pick[0]);
    // the first groups hold too little, or fewer groups hold entries than the target
    if (b < kGroupBins ? want > 0.f && s.pick[1] : V > kCap) {
      // Peers may still be reading this CTA's bins, and its own threads its pick:
      // nothing is written anew, and no CTA ends, before all of them are done
      cluster_sync_all(r.size);
      return false;
    }
    // the bin's lower edge, less what the bins' arithmetic may round
    t = b >= kGroupBins ? -INFINITY
        : per > 0.f     ? r.m - (static_cast<float>(b) + 1.f) / per * 1.0001f - fabsf(r.m) * 1e-6f
                        : low;
  }
  list_entries(r, s, sc, t, want > 0.f);
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
__device__ int filter_list(const Row<T, NT>& r, Shared<NT, kCap>& s, const Ask& q, int n, uint64_t above,
                           uint64_t whole, uint64_t* kept_mass) {
  constexpr int kMost = (kCap + NT - 1) / NT;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int kk = q.k < n ? q.k : n;
  const int per = (kk + NT - 1) / NT;
  uint64_t w[kMost];
  uint64_t sum = 0;
#pragma unroll
  for (int x = 0; x < kMost; ++x) {
    const int i = threadIdx.x * per + x;
    w[x] = x < per && i < kk ? r.weight(key_to_value(static_cast<uint32_t>(s.list[i] >> 32))) : 0ull;
    sum += w[x];
  }
  uint64_t inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t u = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += u;
  }
  if (lane == 31) s.warp_sum[warp] = inc;
  __syncthreads();
  uint64_t before = above + inc - sum, all = 0;
#pragma unroll
  for (int x = 0; x < NT / 32; ++x) {
    if (x < warp) before += s.warp_sum[x];
    all += s.warp_sum[x];
  }
  set_need(s, q.p, whole ? whole : all);
  __syncthreads();
  const float bound = q.mp > 0.f ? s.bound : -INFINITY;
  const uint64_t need = s.need;
  uint64_t mass = 0, kept = 0;
#pragma unroll
  for (int x = 0; x < kMost; ++x) {
    const int i = threadIdx.x * per + x;
    if (x < per && i < kk && (i == 0 || before < need) &&
        key_to_value(static_cast<uint32_t>(s.list[i] >> 32)) >= bound) {
      ++kept;
      mass += w[x];
    }
    before += w[x];
  }
  *kept_mass = above + cta_reduce<NT / 32>(mass, OpSumU64(), s.x);
  return static_cast<int>(cta_reduce<NT / 32>(kept, OpSumU64(), s.x));
}

// What a list says of its row (rank 0's threads).
struct Verdict {
  uint64_t mass;  // sum of the kept weights
  uint64_t cut;  // entries at or above it are kept
  int tok;       // Gumbel maximum of the kept entries but `drop` (u given)
  float val;     // its logit
};

// Filters a list of at most kQuick entries and draws from it: each one's rank
// and the sum of the weights before it come from comparing it with all others
// (two threads an entry), which needs neither a sort nor a scan: one row of 151936
// 11.8 us, by the sort 13.0 (512 rows, four CTAs an SM: 55 and 52).  above, whole: as
// in filter_list.
template <typename T, int NT, int kCap>
__device__ __noinline__ Verdict quick_list(const Row<T, NT>& r, Shared<NT, kCap>& s, const Ask& q, int n,
                                           uint64_t above, uint64_t whole, const float* u, int drop) {
  Verdict out;
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
  // each of an entry's two threads looks at every other entry; whole warps
  // without entries of their own pass by
  if ((e & ~31) < n) {
#pragma unroll 4
    for (int i = half; i < n; i += 2) {
      const ulonglong2 o = s.entry[i];
      if (o.x > place) {
        ++rank;
        before += o.y;
      }
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
  uint64_t need = ~0ull;
  if (q.p < 1.f) {
    if (whole == 0) {  // top-p of what top-k keeps
      uint64_t x = in_k ? w : 0;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
      if (lane == 0) s.join[warp][0] = x;
      __syncthreads();
#pragma unroll
      for (int y = 0; y < kQuick / 32; ++y) whole += s.join[y][0];
    }
    set_need(s, q.p, whole);
    __syncthreads();
    need = s.need;
  }
  const float bound = q.mp > 0.f ? s.bound : -INFINITY;
  const bool kept = in_k && (rank == 0 || above + before < need) && v >= bound;
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
  out.mass = above + sum;
  out.cut = ~last;
  out.tok = key ? static_cast<int>(key_index(key)) : -1;
  const bool close = runs && near_best(sc, key_value(key));
  if (__syncthreads_count(close) > 1) {
    const uint64_t dk = close ? double_key(score64(v, r.m, q.T, ue)) : 0ull;
    const uint64_t best = cta_reduce<NT / 32>(dk, OpMaxU64(), s.x);
    const uint64_t low = close && dk == best ? 0xFFFFFFFFull - at : 0ull;
    out.tok = static_cast<int>(0xFFFFFFFFull - cta_reduce<NT / 32>(low, OpMaxU64(), s.x));
  }
  if (kept && static_cast<int>(at) == out.tok) s.val = v;
  __syncthreads();
  out.val = s.val;
  return out;
}

// One pass over this thread's entries with v >= low: f(v, i) for each, and the
// best of those for which it returns true.  A score needs two logarithms; as
// -log u >= 1 - u, (z - max)/T - log(1 - u) bounds it, and few entries pass the CTA's
// best score so far by that.  Uniforms are loaded for the packs that hold such an
// entry, or with kDense for all, without waiting for the logits.
template <bool kDense, int kCap, typename T, int NT, typename F>
__device__ __forceinline__ void draw_pass(const Row<T, NT>& r, Shared<NT, kCap>& s, const float* u, float low,
                                          Best& best, F f) {
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
      if (kDense || some[x]) r.uniforms(u, u0, wide, k, uu[x]);
    }
#pragma unroll
    for (int x = 0; x < kB; ++x) {
      if (!some[x]) continue;
      float v[kE];
      Row<T, NT>::open_pack(w[x], v);
      const int i = static_cast<int>(r.index_of(j + x * NT));
      // the CTA's best so far in units of log2, less 2^-10 to be safe: whatever
      // comes near the final best is scored
      const float seen = key_to_value(*reinterpret_cast<volatile uint32_t*>(&s.bar));
      const float bar = seen * 1.4426950408889634f - 0.0009765625f - fabsf(seen) * 1e-5f;
#pragma unroll
      for (int h = 0; h < kE; ++h) {
        if (!(v[h] >= low) || !(v[h] > -INFINITY)) continue;
        const bool counts = f(v[h], i + h);
        const float x2 = (v[h] - r.m) * r.c;
        if (counts && !(x2 - fast_log2(1.f - uu[x][h]) < bar)) {
          offer(best, v[h], i + h, x2, uu[x][h]);
          const uint32_t key = value_key(best.score);
          if (best.at == i + h && key > *reinterpret_cast<volatile uint32_t*>(&s.bar)) atomicMax(&s.bar, key);
        }
      }
    }
  }
}

// Gumbel maximum over the row's entries at or above the cut (as rank 0 has it) but
// `drop`, by scores in double; `win` is the entry with the best score in fp32.
template <typename T, int NT, int kCap>
__device__ __noinline__ int settle_row(Shared<NT, kCap>& s, const T* p, int64_t V, float m, float c, const float* u,
                                       uint64_t cut, int drop, int win, float temp, int turn) {
  constexpr int NW = NT / 32;
  Row<T, NT> r;
  r.rank = cluster_rank();
  r.size = cluster_size();
  r.m = m;
  r.c = c;
  r.part.cut(p, V, static_cast<int>(r.rank), static_cast<int>(r.size));
  if (r.rank == 0 && threadIdx.x < r.size) *peer(&s.pick[0], threadIdx.x) = cut;
  cluster_sync_all(r.size);
  cut = s.pick[0];
  const float best = static_cast<float>(score64(to_f32(p[win]), m, temp, u[win]));
  uint64_t mine = 0;
  uint32_t at = 0;
  r.each([&](float v, int64_t i) {
    const uint32_t key = value_key(v), x = static_cast<uint32_t>(i);
    if (key == 0 || place_of(key, x) < cut || static_cast<int>(x) == drop) return;
    if (m == INFINITY && v != m) return;  // probability 0: not even where u = 0 leaves no score above -inf
    const float ui = u[i];
    if (!near_best(fmaf(r.log2w(v), kLn2, gumbel(ui)), best)) return;
    const uint64_t k = double_key(score64(v, m, temp, ui));
    if (k > mine || (k == mine && x < at)) {
      mine = k;
      at = x;
    }
  });
  const uint64_t top = cluster_reduce<NW>(mine, OpMaxU64(), s.x, r.rank, r.size, turn);
  const uint64_t low = mine == top ? 0xFFFFFFFFull - at : 0ull;
  return static_cast<int>(0xFFFFFFFFull - cluster_reduce<NW>(low, OpMaxU64(), s.x, r.rank, r.size, turn));
}

// The best entry over the cluster, of a draw among the row's entries at or above the
// cut (as rank 0 has it) but `drop`.  A call of its own, to which the row comes in
// pieces, so that the loops before it keep their registers (512 x 151936 bf16, top-k
// with top-p 51.5 us, inlined 54.3; top-p 138.4 and 140.0; unfiltered 87 both).
template <typename T, int NT, int kCap>
__device__ __noinline__ int join_pieces(Shared<NT, kCap>& s, const T* p, int64_t V, float m, float c, const float* u,
                                        const Best b, uint64_t cut, int drop, float temp, int turn) {
  constexpr int NW = NT / 32;
  const uint32_t rank = cluster_rank(), size = cluster_size();
  const uint64_t k = b.at >= 0 ? argmax_key(b.score, static_cast<uint32_t>(b.at)) : 0ull;
  const uint64_t win = cluster_reduce<NW>(k, OpMaxU64(), s.x, rank, size, turn);
  if (win == 0) return -1;
  // threads near the best, and above bit 32 those of them with more than one entry there
  const bool close = b.at >= 0 && near_best(b.score, key_value(win));
  const uint64_t more = close && near_best(b.next, key_value(win)) ? 1ull << 32 : 0ull;
  const uint64_t n = cluster_reduce<NW>(more + close, OpSumU64(), s.x, rank, size, turn);
  if (n <= 1) return static_cast<int>(key_index(win));
  if (n >> 32) return settle_row(s, p, V, m, c, u, cut, drop, static_cast<int>(key_index(win)), temp, turn);
  const uint64_t dk = close ? double_key(score64(b.val, m, temp, u[b.at])) : 0ull;
  const uint64_t dbest = cluster_reduce<NW>(dk, OpMaxU64(), s.x, rank, size, turn);
  const uint64_t low = close && dk == dbest ? 0xFFFFFFFFull - static_cast<uint32_t>(b.at) : 0ull;
  return static_cast<int>(0xFFFFFFFFull - cluster_reduce<NW>(low, OpMaxU64(), s.x, rank, size, turn));
}

template <typename T, int NT, int kCap>
__device__ __forceinline__ int join_best(const Row<T, NT>& r, Shared<NT, kCap>& s, const float* u, const Best& b,
                                         int64_t V, uint64_t cut, int drop, float temp) {
  return join_pieces(s, r.p, V, r.m, r.c, u, b, cut, drop, temp, r.turn);
}

// Gumbel maximum over the row's entries at or above the cut but `drop`.
template <typename T, int NT, int kCap>
__device__ __noinline__ int pick_row(const Row<T, NT>& r, Shared<NT, kCap>& s, const float* u, int64_t V,
                                     uint64_t cut, int drop, float temp) {
  Best b = no_best();
  if (threadIdx.x == 0) s.bar = 0x007FFFFFu;  // -inf
  __syncthreads();
  if (r.m < INFINITY) {
    const float low = cut_value(cut);
    const int last = static_cast<int>(place_index(cut) < 0x7FFFFFFFu ? place_index(cut) : 0x7FFFFFFFu);
    const auto takes = [=](float v, int i) { return i != drop && (v > low || i <= last); };
    if (low == -INFINITY) {
      draw_pass<true>(r, s, u, low, b, takes);
    } else {
      draw_pass<false>(r, s, u, low, b, takes);
    }
  } else {  // only the infinite entries have weight
    r.each([&](float v, int64_t i) {
      if (v == r.m && place_of(value_key(v), static_cast<uint32_t>(i)) >= cut && i != drop)
        offer(b, v, static_cast<int>(i), 0.f, u[i]);
    });
  }
  return join_best(r, s, u, b, V, cut, drop, temp);
}

// Cluster sum of a float, CTAs in rank order.
template <typename T, int NT, int kCap>
__device__ __forceinline__ float cluster_mass(Row<T, NT>& r, Shared<NT, kCap>& s, float w) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) w += __shfl_xor_sync(0xffffffffu, w, o);
  __syncthreads();
  if (lane == 0) s.warp_sum[warp] = __float_as_uint(w);
  __syncthreads();
  if (threadIdx.x < r.size) {
    float d = 0.f;
#pragma unroll
    for (int x = 0; x < NT / 32; ++x) d += __uint_as_float(static_cast<uint32_t>(s.warp_sum[x]));
    *peer(&s.sums[r.rank], threadIdx.x) = d;
  }
  cluster_sync_all(r.size);
  float d = 0.f;
  for (uint32_t o = 0; o < r.size; ++o) d += s.sums[o];
  return d;
}

// One pass over a row of which many entries may be kept: those with v > over (or
// v >= over, kFrom).  Their weights are summed, and with kDraw the best of them
// found; entries with under < v that are not kept go to the CTA's own list.
// Decisions are taken per pack, so that a warp leaves the straight path for the
// few packs that hold a candidate.
template <bool kDraw, bool kFrom, int kCap, typename T, int NT>
__device__ __forceinline__ float deep_pass(const Row<T, NT>& r, Shared<NT, kCap>& s, const float* u, float over,
                                           float under, Best* best) {
  constexpr int kE = Row<T, NT>::kE, kB = 16 / kE;  // packs in flight
  const float* u0 = u + (r.part.first - r.part.off);
  const bool wide = (reinterpret_cast<uintptr_t>(u0) & 15) == 0;
  const float m = r.m, c = r.c;
  float sum = 0.f;
  if (kDraw) first_bar(r, s, u, u0, wide, kFrom ? over : nextafterf(over, INFINITY), m);
  float listed = 0.f;
  for (int j = threadIdx.x; j < r.part.packs; j += kB * NT) {
    uint4 w[kB];
    float uu[kB][kE];
#pragma unroll
    for (int x = 0; x < kB; ++x) {
      w[x] = r.pack(j + x * NT);
      if (kDraw) r.uniforms(u, u0, wide, j + x * NT, uu[x]);
    }
    // the CTA's best so far in units of log2, less 2^-10 to be safe: whatever
    // comes near the final best is scored
    const float seen = key_to_value(*reinterpret_cast<volatile uint32_t*>(&s.bar));
    const float bar = seen * 1.4426950408889634f - 0.0009765625f - fabsf(seen) * 1e-5f;
    const float reach = fminf(fast_exp2(bar), 1e30f);
#pragma unroll
    for (int x = 0; x < kB; ++x) {
      if (!(Row<T, NT>::max_of(Row<T, NT>::max_pack(w[x])) >= under)) continue;
      float v[kE], some = 0.f, peak = -INFINITY;
      bool edge = false;
      Row<T, NT>::open_pack(w[x], v);
#pragma unroll
      for (int h = 0; h < kE; ++h) {
        const bool k = kFrom ? v[h] >= over : v[h] > over;
        const float e = fast_exp2((v[h] - m) * c);
        if (k) some += e;
        // the bound in the weights' own terms: w >= 2^bar (1 - u)
        if (kDraw && k) peak = fmaxf(peak, fmaf(uu[x][h], reach, e));
        if (!kFrom) edge |= !k && v[h] > under;
      }
      sum += some;
      const int i = static_cast<int>(r.index_of(j + x * NT));
      if (kDraw && peak >= reach) {
#pragma unroll 1
        for (int h = 0; h < kE; ++h) {
          const float z = Row<T, NT>::pick_of(w[x], h), t = pick_float<kE>(uu[x], h), y = (z - m) * c;
          if ((kFrom ? z >= over : z > over) && !(y - fast_log2(1.f - t) < bar)) offer(*best, z, i + h, y, t);
        }
        const uint32_t key = value_key(best->score);
        if (key > *reinterpret_cast<volatile uint32_t*>(&s.bar)) atomicMax(&s.bar, key);
      }
      if (!kFrom && edge) {
        uint32_t hits = 0;
#pragma unroll
        for (int h = 0; h < kE; ++h) hits |= (v[h] > under && !(v[h] > over) ? 1u : 0u) << h;
        uint32_t at = atomicAdd(&s.own_count, static_cast<uint32_t>(__popc(hits)));
        while (hits) {
          const int h = __ffs(hits) - 1;
          hits &= hits - 1;
          const float z = Row<T, NT>::pick_of(w[x], h);
          if (at < kCap) s.list[at] = place_of(value_key(z), static_cast<uint32_t>(i + h));
          ++at;
          listed += fast_exp2((z - m) * c);
        }
      }
    }
  }
  if (!kFrom && listed > 0.f)
    atomicAdd(reinterpret_cast<unsigned long long*>(&s.own_mass), __float2ull_rn(listed * r.scale));
  return sum;
}

// Best of the entries that rank 0's threads hold, each the best of its own in double.
template <typename T, int NT, int kCap>
__device__ int join_best_cta(const Row<T, NT>& r, Shared<NT, kCap>& s, const float* u, const Best& b, float temp) {
  const uint64_t win = cta_reduce<NT / 32>(b.at >= 0 ? argmax_key(b.score, static_cast<uint32_t>(b.at)) : 0ull,
                                           OpMaxU64(), s.x);
  if (win == 0) return -1;
  const bool close = b.at >= 0 && near_best(b.score, key_value(win));
  if (__syncthreads_count(close) <= 1) return static_cast<int>(key_index(win));
  const uint64_t dk = close ? double_key(score64(b.val, r.m, temp, u[b.at])) : 0ull;
  const uint64_t dbest = cta_reduce<NT / 32>(dk, OpMaxU64(), s.x);
  const uint64_t low = close && dk == dbest ? 0xFFFFFFFFull - static_cast<uint32_t>(b.at) : 0ull;
  return static_cast<int>(0xFFFFFFFFull - cta_reduce<NT / 32>(low, OpMaxU64(), s.x));
}

// Gumbel maximum over the first `kept` entries of the sorted list but `drop`
// (rank 0's threads); -1 when nothing is left.
template <typename T, int NT, int kCap>
__device__ int pick_listed(const Row<T, NT>& r, Shared<NT, kCap>& s, const float* u, int kept, int drop,
                           float temp) {
  Best best = no_best();
  for (int x = threadIdx.x; x < kept; x += NT) {
    const float v = key_to_value(static_cast<uint32_t>(s.list[x] >> 32));
    const int i = static_cast<int>(place_index(s.list[x]));
    if (i != drop) offer<true>(best, v, i, r.log2w(v), u[i], u, r.m, temp);
  }
  return join_best_cta(r, s, u, best, temp);
}

// A long list that top-k does not cut (rank 0's threads).  Top-p's border is
// found by 256 bins of exact weights, linear in the place over the list's range
// (so that equal values are told apart by their indices); the border's bin is
// cut again until it leaves a few entries to rank.  `above` is the weight before the
// list, `whole` what top-p refers to.  With u the kept entries but `drop` are
// offered to `best`.
template <typename T, int NT, int kCap>
__device__ Verdict long_list(const Row<T, NT>& r, Shared<NT, kCap>& s, const Ask& q, int n, uint64_t above,
                             uint64_t whole, const float* u, int drop, Best* best) {
  static_assert(NT == 256 && kCap % NT == 0 && sizeof(s.line) >= 256 * sizeof(uint64_t), "one thread a bin");
  constexpr int kMine = kCap / NT;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const float bound = q.mp > 0.f ? s.bound : -INFINITY;
  unsigned long long* sub = reinterpret_cast<unsigned long long*>(s.line);
  uint64_t place[kMine], all = 0, low = ~0ull, high = 0;
  sub[threadIdx.x] = 0;
#pragma unroll
  for (int x = 0; x < kMine; ++x) {
    const int i = threadIdx.x + x * NT;
    place[x] = i < n ? s.list[i] : 0;
    if (i < n && key_to_value(static_cast<uint32_t>(place[x] >> 32)) < bound) place[x] = 0;  // min-p drops it
    if (place[x]) {
      all += r.weight(key_to_value(static_cast<uint32_t>(place[x] >> 32)));
      low = place[x] < low ? place[x] : low;
      high = place[x] > high ? place[x] : high;
    }
  }
  Verdict out{0, 0, -1, 0.f};
  all = cta_reduce<NT / 32>(all, OpSumU64(), s.x);
  low = ~cta_reduce<NT / 32>(~low, OpMaxU64(), s.x);
  out.mass = above + all;
  out.cut = low;
  if (q.p < 1.f) {
    set_need(s, q.p, whole);
    if (threadIdx.x == 0) s.taken = 0;
    high = cta_reduce<NT / 32>(high, OpMaxU64(), s.x);
    if (out.mass > s.need) {  // the border is among these entries
      const uint64_t need = s.need;
      uint64_t over = above;
      int few;
      do {
        const int bits = 64 - __clzll(static_cast<long long>(high - low)), shift = bits > 8 ? bits - 8 : 0;
        sub[threadIdx.x] = 0;
        __syncthreads();
#pragma unroll
        for (int x = 0; x < kMine; ++x)
          if (place[x] >= low && place[x] <= high)
            atomicAdd(&sub[(high - place[x]) >> shift], r.weight(key_to_value(static_cast<uint32_t>(place[x] >> 32))));
        __syncthreads();
        const uint64_t mine = sub[threadIdx.x];
        uint64_t inc = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint64_t y = __shfl_up_sync(0xffffffffu, inc, o);
          if (lane >= o) inc += y;
        }
        if (lane == 31) s.warp_sum[warp] = inc;
        __syncthreads();
        uint64_t before = over + inc - mine;
        for (int w = 0; w < warp; ++w) before += s.warp_sum[w];
        if (before < need && before + mine >= need) {
          s.pick[0] = threadIdx.x;
          s.pick[1] = before;
        }
        __syncthreads();
        const uint64_t at = s.pick[0];
        over = s.pick[1];
        high -= at << shift;
        const uint64_t end = high - ((1ull << shift) - 1);
        if (end > low) low = end;
        // what is left: their number, and the range that they fill
        uint64_t first = 0, last = 0;
        few = 0;
#pragma unroll
        for (int x = 0; x < kMine; ++x) {
          if (place[x] < low || place[x] > high) continue;
          ++few;
          first = place[x] > first ? place[x] : first;
          last = ~place[x] > last ? ~place[x] : last;
        }
        few = __reduce_add_sync(0xffffffffu, few);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
          const uint64_t y = __shfl_xor_sync(0xffffffffu, first, o), z = __shfl_xor_sync(0xffffffffu, last, o);
          first = y > first ? y : first;
          last = z > last ? z : last;
        }
        if (lane == 0) {
          s.join[warp][0] = static_cast<uint64_t>(few);
          s.join[warp][1] = first;
          s.join[warp][2] = last;
        }
        __syncthreads();
        few = 0;
#pragma unroll
        for (int w = 0; w < NT / 32; ++w) {
          few += static_cast<int>(s.join[w][0]);
          first = s.join[w][1] > first ? s.join[w][1] : first;
          last = s.join[w][2] > last ? s.join[w][2] : last;
        }
        high = first;
        low = ~last;
      } while (few > kQuick);
#pragma unroll
      for (int x = 0; x < kMine; ++x)
        if (place[x] >= low && place[x] <= high) s.list[atomicAdd(&s.taken, 1u)] = place[x];
      __syncthreads();
      out = quick_list(r, s, q, few, over, whole, static_cast<const float*>(nullptr), -1);
    }
  }
  out.tok = -1;
  if (u) {
#pragma unroll
    for (int x = 0; x < kMine; ++x) {
      if (place[x] && place[x] >= out.cut) {
        const float v = key_to_value(static_cast<uint32_t>(place[x] >> 32));
        const int i = static_cast<int>(place_index(place[x]));
        if (i != drop) offer<true>(*best, v, i, r.log2w(v), u[i], u, r.m, q.T);
      }
    }
  }
  return out;
}

// Filters a list and draws from it (rank 0's threads).
template <typename T, int NT, int kCap>
__device__ __forceinline__ Verdict settle_list(const Row<T, NT>& r, Shared<NT, kCap>& s, const Ask& q, int n,
                                               uint64_t whole, const float* u, int drop) {
  if (n <= kQuick) return quick_list(r, s, q, n, 0, whole, u, drop);
  Verdict out;
  if (q.k >= n && (q.p >= 1.f || whole > 0)) {
    Best best = no_best();
    out = long_list(r, s, q, n, 0, whole, u, drop, &best);
    if (u) out.tok = join_best_cta(r, s, u, best, q.T);
  } else {
    sort_list<NT>(s.list, n);
    const int kept = filter_list(r, s, q, n, 0, whole, &out.mass);
    out.cut = s.list[kept - 1];
    out.tok = u ? pick_listed(r, s, u, kept, drop, q.T) : -1;
  }
  out.val = out.tok >= 0 ? r.at(out.tok) : 0.f;
  return out;
}

// Top-p over the whole row where its border lies deep in the row.  A histogram
// linear in the logit, of weights relative to their bin's middle (integers:
// nearly equal within a bin, exact sums), finds the bin of the border; a second
// pass sums the weights above that bin, draws among them (`u` given) and lists
// the bin's own entries.  False: the border fell too close to a bin's edge, or
// the bin does not fit the list.  Else rank 0 has the verdict, and the draw is
// left in `best` of the cluster's threads.
template <typename T, int NT, int kCap>
__device__ __noinline__ bool deep_top_p(const Row<T, NT>& row, Shared<NT, kCap>& s, const Ask& q, int64_t V, float row_mass,
                                        const float* u, Best* best, Verdict* out) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  Row<T, NT> r = row;
  const uint64_t whole = __float2ull_rn(row_mass * r.scale);
  // entries this far below the maximum, in units of log2, sum to less than
  // (1 - p) / 2 of the row
  const float span = log2f(2.f * static_cast<float>(V) / ((1.f - q.p) * row_mass));
  if (!(fabsf(r.m) < 1e30f) || !(span > 0.f) || !(span < 1e6f)) return false;
  const float per = kLineBins / span, step = span / kLineBins;
  // the unit of the bins' integers: 2^31 holds every entry of the longest part
  const int most = static_cast<int>(V / r.size) + 2 * Part<T>::kE;
  const float one = fminf(static_cast<float>(0x80000000u >> (32 - __clz(most - 1))), 2097152.f);
  for (int b = threadIdx.x; b < kLineBins; b += NT) s.line[b] = 0;
  if (threadIdx.x == 0) {
    s.own_count = 0;
    s.own_mass = 0;
    s.pick[0] = kLineBins;
    s.beside[0] = -1;
    s.beside[1] = kLineBins;
    s.bar = 0x007FFFFFu;  // -inf
  }
  set_need(s, q.p, whole);
  __syncthreads();
  const float m = r.m, c = r.c;
  // bin and weight without conversions or exponentials: adding 1.5 2^23 rounds a
  // float to an integer in its low bits, and within half a bin 2^(-f step) is a
  // parabola to (step ln 2)^3 / 48
  const float magic = 12582912.f, t1 = -step * kLn2 * one, t2 = 0.5f * step * kLn2 * step * kLn2 * one;
  const float slope = -c * per;
  r.each([&](float v, int64_t) {
    const float d = (v - m) * slope;
    if (d < static_cast<float>(kLineBins) - 0.5f) {
      const float near = d + magic, f = d - (near - magic);
      const float part = fmaf(fmaf(t2, f, t1), f, one) + magic;
      atomicAdd(&s.line[__float_as_int(near) & (kLineBins - 1)],
                static_cast<uint32_t>(__float_as_int(part) - __float_as_int(magic)));
    }
  });
  cluster_sync_all(r.size);
  constexpr int kMine = kLineBins / NT;
  static_assert(kMine == 4, "a thread's bins are one 16-byte load");
  const uint64_t need = s.need;
  uint4 bins[kMaxCluster];
#pragma unroll
  for (uint32_t o = 0; o < kMaxCluster; ++o)
    bins[o] = o < r.size ? *peer(reinterpret_cast<const uint4*>(s.line) + threadIdx.x, o) : make_uint4(0, 0, 0, 0);
  float h[kMine] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (uint32_t o = 0; o < kMaxCluster; ++o) {
    h[0] += static_cast<float>(bins[o].x);
    h[1] += static_cast<float>(bins[o].y);
    h[2] += static_cast<float>(bins[o].z);
    h[3] += static_cast<float>(bins[o].w);
  }
  uint64_t mine[kMine], sum = 0;
#pragma unroll
  for (int x = 0; x < kMine; ++x) {
    const float b = static_cast<float>(threadIdx.x * kMine + x);
    mine[x] = __float2ull_rn(h[x] / one * fast_exp2(-b * step) * r.scale);
    sum += mine[x];
  }
  uint64_t inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  if (lane == 31) s.warp_sum[warp] = inc;
  __syncthreads();
  uint64_t before = inc - sum;
  for (int w = 0; w < warp; ++w) before += s.warp_sum[w];
#pragma unroll
  for (int x = 0; x < kMine; ++x) {
    if (before < need && before + mine[x] >= need) s.pick[0] = threadIdx.x * kMine + x;
    before += mine[x];
  }
  __syncthreads();
  int bin = static_cast<int>(s.pick[0]);
  if (bin == kLineBins) return false;
#pragma unroll
  for (int x = 0; x < kMine; ++x) {
    const int b = threadIdx.x * kMine + x;
    if (mine[x] && b < bin) atomicMax(&s.beside[0], b);
    if (mine[x] && b > bin) atomicMin(&s.beside[1], b);
  }
  // second pass: exact sums, by values in place of bins.  Where rounding put the
  // border into a neighbour of its bin they tell, and the next bin that holds
  // entries is taken.
  uint64_t above;
  uint32_t count;
  for (int attempt = 0;; ++attempt) {
    const float over = m - (static_cast<float>(bin) - 0.5f) * step / c;
    const float under = m - (static_cast<float>(bin) + 0.5f) * step / c;
    const float w = u ? deep_pass<true, false>(r, s, u, over, under, best)
                      : deep_pass<false, false>(r, s, u, over, under, best);
    above = __float2ull_rn(cluster_mass(r, s, w) * r.scale);
    uint64_t mass;
    close_list(r, s, &count, &mass);
    if (count <= kCap && above < need && above + mass >= need) break;
    bin = s.beside[above >= need ? 0 : 1];
    if (attempt == 1 || count > kCap || bin < 0 || bin >= kLineBins) return false;
    if (best) *best = no_best();
    if (threadIdx.x == 0) {
      s.own_count = 0;
      s.own_mass = 0;
      s.bar = 0x007FFFFFu;  // -inf
    }
    __syncthreads();
  }
  if (r.rank != 0) {  // behind the entries of the CTAs before
    uint32_t at = 0;
    for (uint32_t o = 0; o < r.rank; ++o) at += s.list_count[o];
    uint64_t* list = peer(s.list, 0);
    for (uint32_t i = threadIdx.x; i < s.own_count; i += NT) list[at + i] = s.list[i];
  }
  cluster_sync_all(r.size);
  if (r.rank == 0) {
    if (count <= kQuick) {
      *out = quick_list(row, s, q, static_cast<int>(count), above, whole, static_cast<const float*>(nullptr), -1);
      if (u && threadIdx.x < count && s.list[threadIdx.x] >= out->cut) {
        const uint32_t i = place_index(s.list[threadIdx.x]);
        const float v = key_to_value(static_cast<uint32_t>(s.list[threadIdx.x] >> 32));
        offer<true>(*best, v, static_cast<int>(i), r.log2w(v), u[i], u, r.m, q.T);
      }
    } else {
      *out = long_list(row, s, q, static_cast<int>(count), above, whole, u, -1, best);
    }
  }
  return true;
}

// Min-p alone over a row of which it keeps many entries: their mass, and the
// draw left in `best`.
template <typename T, int NT, int kCap>
__device__ __noinline__ uint64_t deep_min_p(const Row<T, NT>& row, Shared<NT, kCap>& s, const float* u, Best* best) {
  Row<T, NT> r = row;
  const float low = s.bound;
  if (threadIdx.x == 0) s.bar = 0x007FFFFFu;  // -inf
  __syncthreads();
  const float w =
      u ? deep_pass<true, true>(r, s, u, low, low, best) : deep_pass<false, true>(r, s, u, low, low, best);
  return __float2ull_rn(cluster_mass(r, s, w) * r.scale);
}

// The cut and the kept mass of any row, by radix descents.
template <typename T, int NT, int kCap>
__device__ __noinline__ uint64_t wide_cut(Row<T, NT>& r, Shared<NT, kCap>& s, const FilterArgs& a, const Ask& q,
                                          uint64_t* kept_mass) {
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
    set_need(s, q.p, w);
    __syncthreads();
    const uint64_t need = s.need;
    if (need < w) cut = find_cut<T, NT, kCap, true>(r, s, cut, need, a.idx_bits);
  }
  if (q.mp > 0.f) {
    set_bound(s, r.m, q);
    __syncthreads();
    const uint64_t c = place_of(value_key(s.bound), 0xFFFFFFFFu);
    if (c > cut) cut = c;
  }
  const float low = cut_value(cut);
  const int64_t last = place_index(cut);
  float w = 0.f;
  r.each([&](float v, int64_t i) {
    if (v > -INFINITY && (v > low || (v == low && i <= last))) w += fast_exp2(r.log2w(v));
  });
  *kept_mass = __float2ull_rn(cluster_mass(r, s, w) * r.scale);
  return cut;
}

// Tries the short list for a row's filters; true: rank 0's threads have the
// verdict (with a draw from u, if given).
template <typename T, int NT, int kCap>
__device__ bool listed_row(Row<T, NT>& r, Shared<NT, kCap>& s, const Scan<T, NT>& sc, const FilterArgs& a,
                           const Ask& q, float low, float row_mass, const float* u, int drop, Verdict* out) {
  int target = 0;
  float t = -INFINITY;
  if (q.mp > 0.f) {
    set_bound(s, r.m, q);
    __syncthreads();
  }
  const bool of_row = q.k >= a.V && q.p < 1.f;  // top-p refers to the whole row
  if (q.k == 1) {
    t = r.m;
  } else if (q.k < a.V) {
    target = q.k;
  } else if (of_row) {
    target = kGroupTarget;
  } else if (q.mp > 0.f) {
    t = s.bound;
  } else {
    return false;
  }
  if (target > kCap) return false;
  uint32_t count;
  uint64_t mass;
  const float want = of_row ? fmaxf(q.p * row_mass, 1.f) : 0.f;  // (the first entry is kept whatever p)
  if (!short_list(r, s, sc, a.V, low, target, &t, want, q.mp > 0.f, &count, &mass)) return false;
  // the list has to hold top-p's border (with a margin for these roundings), or
  // all that min-p leaves
  const uint64_t whole = of_row ? __float2ull_rn(row_mass * r.scale) : 0;
  if (of_row && __ull2float_rz(mass) < q.p * __ull2float_ru(whole) * 1.000001f && static_cast<int64_t>(count) < a.V &&
      !(q.mp > 0.f && s.bound >= t))
    return false;
  if (r.rank == 0) {
    const Row<T, NT> far = r;  // (a copy for calls: the row of the hot loops stays in registers)
    *out = settle_list(far, s, q, static_cast<int>(count), whole, u, drop);
  }
  return true;
}

template <typename T, int NT>
__device__ __forceinline__ float log_prob(const Row<T, NT>& r, float v, uint64_t kept) {
  return r.log2w(v) * kLn2 - logf(__ull2float_rn(kept) * r.unit);
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
    s.bar = 0x007FFFFFu;  // -inf
  }
  for (int b = threadIdx.x; b < kGroupBins; b += NT) s.groups[b] = s.weights[b] = 0;
  __syncthreads();
  if (size > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  pdl_wait();
}

constexpr int kShortCap = 1024;
constexpr int kThr = 256;

constexpr int kDeferred = -2;  // tok of a row that is left to the wide kernel, or whose draw is
using Short = Shared<kThr, kShortCap>;

// A row without a short list: its mass and cut, and with u the token drawn.
// mass and cut are known to rank 0's threads, the token to all.
template <typename T>
__device__ __forceinline__ int wide_row(Row<T, kThr>& r, Short& s, const FilterArgs& a, const Ask& q, float row_mass,
                                        const float* u, Verdict* v) {
  Best best = no_best();
  const bool ordinary = q.k >= a.V && fabsf(r.m) < 1e30f;
  if (q.mp > 0.f) {
    set_bound(s, r.m, q);
    __syncthreads();
  }
  if (ordinary && q.p < 1.f && q.mp == 0.f && deep_top_p(r, s, q, a.V, row_mass, u, &best, v))
    return u ? join_best(r, s, u, best, a.V, v->cut, -1, q.T) : -1;
  if (ordinary && q.p >= 1.f && q.mp > 0.f) {
    v->mass = deep_min_p(r, s, u, &best);
    v->cut = place_of(value_key(s.bound), 0xFFFFFFFFu);
    return u ? join_best(r, s, u, best, a.V, v->cut, -1, q.T) : -1;
  }
  if (q.greedy) {  // the first entry of the order
    v->cut = first_place(r, s);
    v->mass = r.weight(r.m);
    return u ? static_cast<int>(place_index(v->cut)) : -1;
  }
  if (q.k >= a.V && q.p >= 1.f && q.mp == 0.f) {  // nothing filters
    v->mass = __float2ull_rn(row_mass * r.scale);
    v->cut = 1ull << 32;
  } else {
    v->cut = wide_cut(r, s, a, q, &v->mass);
  }
  return u ? pick_row(r, s, u, a.V, v->cut, -1, q.T) : -1;
}

template <typename T>
__device__ __forceinline__ void write_sample(const FilterArgs& a, const Row<T, kThr>& r, int64_t row, int tok,
                                             const Verdict& v, bool ok) {
  if (r.rank != 0 || threadIdx.x != 0) return;
  a.tok[row] = tok;
  if (a.logprob) a.logprob[row] = tok >= 0 ? log_prob(r, tok == v.tok ? v.val : r.at(tok), v.mass) : -INFINITY;
  if (!ok) atomicOr(a.status, kDevBadParam);
}

// Few CTAs serve a row whose filters leave a short list.  A row that needs more
// passes is left to a second launch, whose clusters share out such rows, unless
// this one has many CTAs a row already: kDefer keeps those passes' registers out
// of the scan (512 x 151936 bf16, top-k with top-p, as one kernel for both: 57 to
// 62 us; so: 54).
template <typename T, bool kDefer>
__global__ void __launch_bounds__(kThr, 4) sample_rows_kernel(const FilterArgs a) {
  extern __shared__ __align__(16) uint8_t raw[];
  Short& s = *reinterpret_cast<Short*>(raw);
  const uint32_t size = cluster_size();
  const int64_t row = blockIdx.x / size;
  start(s, size);
  const Ask q = read_ask(a, row);
  Row<T, kThr> r;
  r.c = inv_temperature(q.T);
  r.open(a, row);
  const bool want_mass = wants_mass(a, q), unfiltered = want_mass && q.p >= 1.f && q.ok;
  const float* u = a.u + row * a.ld_u;
  Scan<T, kThr> sc;
  Best best = no_best();
  if (unfiltered) {
    scan_and_draw(r, s, u, sc, best);
  } else {
    scan_row(r, want_mass, sc);
  }
  float low, row_mass;
  const bool some = join_scan(r, s, sc, want_mass, &low, &row_mass);
  int tok = -1, left = 0;
  Verdict v{0, 0, -1, 0.f};
  if (q.ok && some) {
    if (unfiltered && fabsf(r.m * r.c) < 1e3f) {
      v.mass = __float2ull_rn(row_mass * r.scale);
      tok = join_best(r, s, u, best, a.V, 1ull << 32, -1, q.T);
    } else if (listed_row(r, s, sc, a, q, low, row_mass, u, -1, &v)) {
      if (r.rank != 0) return;
      tok = v.tok;
    } else if constexpr (kDefer) {
      left = 1;
    } else {
      Row<T, kThr> far = r;
      tok = wide_row(far, s, a, q, row_mass, u, &v);
    }
  }
  if (kDefer && r.rank == 0 && threadIdx.x == 0) a.states[row] = RowState{r.m, row_mass, left};
  if (!left) write_sample(a, r, row, tok, v, q.ok);
}

// Visits, in all CTAs of cluster `id` alike, its share of the rows that
// left(row) tells: the id-th such row, and every `clusters`-th after it.
template <typename L, typename F>
__device__ __forceinline__ void share_rows(Short& s, int64_t rows, uint32_t id, uint32_t clusters, L left, F visit) {
  constexpr int kEach = kShareRows / kThr;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int64_t carry = 0;
  for (int64_t base = 0; base < rows; base += kThr * kEach) {
    uint32_t bits = 0;
#pragma unroll
    for (int x = 0; x < kEach; ++x) {
      const int64_t i = base + threadIdx.x * kEach + x;
      if (i < rows && left(i)) bits |= 1u << x;
    }
    const uint32_t n = __popc(bits);
    uint32_t inc = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    if (lane == 31) s.warp_sum[warp] = inc;
    __syncthreads();
    uint32_t before = inc - n, all = 0;
    for (int w = 0; w < kThr / 32; ++w) {
      if (w < warp) before += static_cast<uint32_t>(s.warp_sum[w]);
      all += static_cast<uint32_t>(s.warp_sum[w]);
    }
    // ordinals id + t clusters, t >= first, are this cluster's
    const int64_t first = carry > id ? (carry - id + clusters - 1) / clusters : 0;
#pragma unroll
    for (int x = 0; x < kEach; ++x) {
      if (!(bits >> x & 1)) continue;
      const int64_t ord = carry + before++;
      if (ord % clusters == id) s.rows[ord / clusters - first] = base + threadIdx.x * kEach + x;
    }
    carry += all;
    const int64_t end = carry > id ? (carry - id + clusters - 1) / clusters : 0;
    __syncthreads();
    for (int64_t t = first; t < end; ++t) {
      cluster_sync_all(cluster_size());  // the other CTAs have started, or are done with the last row
      visit(s.rows[t - first]);
    }
    __syncthreads();
  }
}

template <typename T>
__global__ void __launch_bounds__(kThr, 4) sample_wide_kernel(const FilterArgs a, const int64_t rows) {
  extern __shared__ __align__(16) uint8_t raw[];
  Short& s = *reinterpret_cast<Short*>(raw);
  pdl_wait();
  const uint32_t size = cluster_size();
  share_rows(
      s, rows, blockIdx.x / size, gridDim.x / size, [&](int64_t i) { return a.states[i].left != 0; },
      [&](int64_t row) {
        const Ask q = read_ask(a, row);
        const RowState st = a.states[row];
        Row<T, kThr> r;
        r.c = inv_temperature(q.T);
        r.open(a, row);
        r.m = st.m;
        Verdict v{0, 0, -1, 0.f};
        const int tok = wide_row(r, s, a, q, st.mass, a.u + row * a.ld_u, &v);
        write_sample(a, r, row, tok, v, true);
      });
}

// Whether the draft of verified row rr of sequence j is accepted (one thread).
template <typename T>
__device__ __forceinline__ int accepts(const FilterArgs& a, const Row<T, kThr>& r, int64_t j, int rr, uint64_t cut,
                                       uint64_t mass) {
  const int x = rr < a.D ? a.draft[j * a.D + rr] : -1;
  if (x < 0 || x >= a.V) return 0;
  const float z = r.at(x);
  const uint32_t key = value_key(z);
  return key != 0 && place_of(key, static_cast<uint32_t>(x)) >= cut &&
         static_cast<double>(a.u_accept[j * a.D + rr]) * static_cast<double>(mass) <
             static_cast<double>(r.weight(z));
}

// A sequence's outputs from its rows (one warp): leading accepts, and the token
// drawn at the row after them, or `drawn` where that is still to be drawn.
__device__ __forceinline__ int leading_accepts(const FilterArgs& a, int64_t j) {
  const int lane = threadIdx.x & 31;
  for (int base = 0; base < a.D; base += 32) {
    const int i = base + lane;
    const bool ok = i < a.D && __ldcg(&a.cuts[j * a.R + i].accept);
    const uint32_t no = ~__ballot_sync(0xffffffffu, ok);
    if (no) {
      const int n = base + __ffs(no) - 1;
      return n < a.D ? n : a.D;
    }
  }
  return a.D;
}
__device__ __forceinline__ void write_sequence(const FilterArgs& a, int64_t j, int n, int corr, bool ok) {
  const int lane = threadIdx.x & 31;
  const int* dr = a.draft + j * a.D;
  if (!ok) {
    n = -1;  // a commit of this length appends nothing
    corr = -1;
  }
  if (lane == 0) {
    if (!ok) atomicOr(a.status, kDevBadParam);
    a.n_out[j] = n;
    a.corr_out[j] = corr;
    if (a.next_tok) a.next_tok[j] = corr >= 0 ? corr : (n > 0 ? dr[n - 1] : -1);
  }
  if (a.emitted)
    for (int i = lane; i < a.R; i += 32) a.emitted[j * a.R + i] = i < n ? dr[i] : (i == n ? corr : -1);
}

// One thread, after its row's result is written: whether it was the sequence's
// last (then the ticket starts anew).  A ticket lies in the record of its
// sequence's first row, where no batch of another shape over the same workspace
// writes anything else.
__device__ __forceinline__ bool finishes(const FilterArgs& a, int64_t j) {
  __threadfence();
  int* ticket = &a.cuts[j * a.R].ticket;
  if (atomicAdd(ticket, 1) != a.rows_used - 1) return false;
  *ticket = 0;
  __threadfence();
  return true;
}

// Verified row rr of sequence j: whether its draft is accepted, and the token
// drawn here if it is not (or if rr = D).  The CTA that finishes a sequence's
// last row (a ticket) writes the outputs.  With kDefer, rows without a short
// list are left to a second launch.
template <typename T, bool kDefer>
__global__ void __launch_bounds__(kThr, 4) accept_rows_kernel(const FilterArgs a) {
  extern __shared__ __align__(16) uint8_t raw[];
  Short& s = *reinterpret_cast<Short*>(raw);
  const uint32_t size = cluster_size(), at = blockIdx.x / size;
  const int64_t j = at / a.rows_used;
  const int rr = static_cast<int>(at - j * a.rows_used);
  const int64_t row = j * a.R + rr;
  start(s, size);
  const Ask q = read_ask(a, j);
  Row<T, kThr> r;
  r.c = inv_temperature(q.T);
  r.open(a, row);
  const bool want_mass = wants_mass(a, q);
  Scan<T, kThr> sc;
  scan_row(r, want_mass, sc);
  float low, row_mass;
  const bool some = join_scan(r, s, sc, want_mass, &low, &row_mass);
  RowCut out;
  out.cut = ~0ull;
  out.m = r.m;
  out.accept = 0;
  out.tok = -1;
  out.left = 0;
  out.mass = row_mass;
  if (q.ok && some) {
    const int drop = rr < a.D ? a.draft[j * a.D + rr] : -1;
    const float* u = a.u + j * a.ld_u;
    Verdict v{0, 0, -1, 0.f};
    const bool listed = listed_row(r, s, sc, a, q, low, row_mass, u, drop, &v);
    if (listed && r.rank != 0) return;
    Row<T, kThr> far = r;
    if (listed) {
      out.tok = v.tok;
    } else {
      out.tok = kDeferred;
      if constexpr (kDefer) {
        out.left = 1;
      } else {
        wide_row(far, s, a, q, row_mass, static_cast<const float*>(nullptr), &v);
      }
    }
    out.cut = v.cut;
    if (r.rank == 0 && threadIdx.x == 0 && !out.left) out.accept = accepts(a, r, j, rr, v.cut, v.mass);
    if constexpr (!kDefer) {
      if (!listed) {  // a wide row draws where it has to
        if (r.rank == 0 && threadIdx.x == 0) {
          for (uint32_t o = 0; o < size; ++o) {
            uint64_t* p = peer(s.pick, o);
            p[0] = out.cut;
            p[1] = static_cast<uint64_t>(out.accept);
          }
        }
        cluster_sync_all(size);
        if (s.pick[1] == 0) out.tok = pick_row(far, s, u, a.V, s.pick[0], drop, q.T);
      }
    }
  }
  if (r.rank != 0) return;
  if (threadIdx.x == 0) {
    RowCut& c = a.cuts[row];  // (all but the ticket)
    c.cut = out.cut;
    c.m = out.m;
    c.accept = out.accept;
    c.tok = out.tok;
    c.left = out.left;
    c.mass = out.mass;
    s.taken = !out.left && finishes(a, j);
  }
  __syncthreads();
  if (!s.taken || threadIdx.x >= 32) return;
  const int n = leading_accepts(a, j);
  write_sequence(a, j, n, n < a.R ? __ldcg(&a.cuts[j * a.R + n].tok) : -1, q.ok);
}

// The rows left by it; the cluster that finishes a sequence's last row makes the one
// draw that it needs, if that row was left too, and writes the outputs.
template <typename T>
__global__ void __launch_bounds__(kThr, 4) accept_wide_kernel(const FilterArgs a, const int64_t rows) {
  extern __shared__ __align__(16) uint8_t raw[];
  Short& s = *reinterpret_cast<Short*>(raw);
  pdl_wait();
  const uint32_t size = cluster_size();
  const auto row_of = [&](int64_t at) { return at / a.rows_used * a.R + at % a.rows_used; };
  share_rows(
      s, rows, blockIdx.x / size, gridDim.x / size, [&](int64_t at) { return a.cuts[row_of(at)].left != 0; },
      [&](int64_t at) {
        const int64_t j = at / a.rows_used;
        const int rr = static_cast<int>(at - j * a.rows_used);
        const Ask q = read_ask(a, j);
        RowCut* c = a.cuts + row_of(at);
        Row<T, kThr> r;
        r.c = inv_temperature(q.T);
        r.open(a, row_of(at));
        r.m = c->m;
        Verdict v{0, 0, -1, 0.f};
        wide_row(r, s, a, q, c->mass, static_cast<const float*>(nullptr), &v);
        if (r.rank == 0 && threadIdx.x == 0) {  // `left` stays: other clusters read it
          c->cut = v.cut;
          c->accept = accepts(a, r, j, rr, v.cut, v.mass);
          const bool last = finishes(a, j);
          for (uint32_t o = 0; o < size; ++o) *peer(s.pick, o) = last;
        }
        cluster_sync_all(size);
        if (s.pick[0] == 0) return;
        const int n = leading_accepts(a, j);
        int corr = -1;
        if (n < a.R) {
          const RowCut* e = a.cuts + j * a.R + n;
          corr = __ldcg(&e->tok);
          if (corr == kDeferred) {
            r.open(a, j * a.R + n);
            r.m = __ldcg(&e->m);
            corr = pick_row(r, s, a.u + j * a.ld_u, a.V, __ldcg(&e->cut), n < a.D ? a.draft[j * a.D + n] : -1, q.T);
          }
        }
        if (r.rank == 0 && threadIdx.x < 32) write_sequence(a, j, n, corr, true);
      });
}

constexpr int kTopCap = 2048;
static_assert(kTopCap >= kTopLogitsMax, "the K entries fit the list");

// The K first entries of the order, sorted, and the row's log-sum-exp.  16 x 151936
// fp32, K = 64: 15 us; 1024 x 151936 bf16, K = 256: 108 us, 60 of them streaming
// (5.2 TB/s), the rest the list and its sort by one CTA a row.
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
  float row_mass;
  const bool some = join_scan(r, s, sc, want_mass, &low, &row_mass);
  uint32_t n = 0;
  uint64_t mass;
  if (some && !short_list(r, s, sc, a.V, low, a.K, &t, 0.f, false, &n, &mass)) {
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
                                                        static_cast<double>(logf(row_mass)))
                                   : r.m;
    a.lse[row] = some ? l : -INFINITY;
  }
}

static_assert(sizeof(Shared<kThr, kTopCap>) <= 48 * 1024, "more would have to be asked for");
cudaError_t launch_rows(const void* kern, int64_t rows, int parts, size_t smem, const FilterArgs& a,
                        cudaStream_t st) {
  FilterArgs b = a;
  void* args[] = {&b};
  return launch_kc(kern, dim3((unsigned)(rows * parts)), dim3(kThr), smem, st, true, dim3(parts), args);
}

// CTAs per row: as many as the GPU holds at once (four an SM), at least 4 KB
// each.  More of them spread the rows' waves: 512 x 151936 bf16, top-k with top-p, 66
// us with one a row, 83 with two; 128 rows, 28 us with four, 39 with eight.  Small
// rows (16 x 8000 fp32), one CTA / eight: top-k with top-p 10 / 11 us, top-p 31 / 27.
int pick_parts(int64_t V, int64_t rows, size_t esize) {
  int parts = 1;
  while (parts < kMaxCluster && rows * parts * 2 <= 4 * num_sms() && V * (int64_t)esize / (2 * parts) >= 4096)
    parts *= 2;
  return parts;
}
// Whether wide rows are left to a second launch: worth it where a CTA of the first
// has a long part to work alone.  bf16, us inline / deferred: parts of 83 KB (300 x
// 83000) top-p 78 / 86, top-k with top-p 28 / 31; of 152 KB (300 x 151936) 122 / 116,
// 40 / 44; of 304 KB (512 x 151936) 192 / 138, 53 / 55.  (Up to kInlineRows rows need
// no workspace; they have eight CTAs each or short parts.)
bool defers(int64_t V, int64_t rows, size_t esize, int parts) {
  return rows > kInlineRows && parts < kMaxCluster && V * (int64_t)esize / parts > 160 * 1024;
}

// The second launch: clusters that fill the GPU share out the rows.  Of eight CTAs:
// 512 x 151936 bf16, top-p / min-p / mixed 138 / 83 / 133 us; of four 138 / 87 / 142.
cudaError_t launch_wide(const void* kern, int64_t rows, size_t smem, const FilterArgs& a, cudaStream_t st) {
  FilterArgs b = a;
  void* args[] = {&b, &rows};
  const int parts = 8;
  int64_t clusters = 4 * num_sms() / parts;
  if (clusters < kShareRows / kShareMost) clusters = kShareRows / kShareMost;
  if (clusters > rows) clusters = rows;
  return launch_kc(kern, dim3((unsigned)(clusters * parts)), dim3(kThr), smem, st, true, dim3(parts), args);
}

template <typename T>
cudaError_t launch_sample(FilterArgs a, int64_t rows, cudaStream_t st) {
  const int parts = pick_parts(a.V, rows, sizeof(T));
  const bool defer = defers(a.V, rows, sizeof(T), parts);
  const void* kern = defer ? (const void*)sample_rows_kernel<T, true> : (const void*)sample_rows_kernel<T, false>;
  cudaError_t e = launch_rows(kern, rows, parts, sizeof(Short), a, st);
  if (e != cudaSuccess || !defer) return e;
  return launch_wide((const void*)sample_wide_kernel<T>, rows, sizeof(Short), a, st);
}
template <typename T>
cudaError_t launch_accept(FilterArgs a, int64_t b, cudaStream_t st) {
  const int64_t rows = b * a.rows_used;
  const int parts = pick_parts(a.V, rows, sizeof(T));
  const bool defer = defers(a.V, rows, sizeof(T), parts);
  const void* kern = defer ? (const void*)accept_rows_kernel<T, true> : (const void*)accept_rows_kernel<T, false>;
  cudaError_t e = launch_rows(kern, rows, parts, sizeof(Short), a, st);
  if (e != cudaSuccess || !defer) return e;
  return launch_wide((const void*)accept_wide_kernel<T>, rows, sizeof(Short), a, st);
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
  a.unit = ldexpf(1.f, a.idx_bits - 62);
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
