// k_tree_attn.cu — attention of a tree's nodes over a cache.  For node i, head
// h of a sequence with `len` cached keys and n nodes,
//   o = sum_t p_t v_t / sum_t p_t,  p_t = exp(scale q.k_t - m),  lse = m + ln sum_t p_t
// over t in the whole cache and the nodes that mask(i) has; no key: o = 0 and
// lse = -inf.
//
// The N nodes times the nq / nkv heads that share a kv head are the rows of a
// query tile, so a key's bytes serve them all: 4 flops a key, dimension and
// row against 4 bytes a key and dimension, and HBM is the bound up to about
// 280 rows.
//
// Work is shared out by keys, not by sequences: the key tiles (64 or 128 keys) of
// all (sequence, kv head, query tile) items, in that order, are cut into as many
// equal runs as CTAs are resident, whatever the lengths (which only the device
// knows).  A CTA walks its run with the online softmax (running maximum and
// sum, O rescaled when the maximum rises); an item that lies within one run is
// written straight out, the parts of the others go to the workspace as fp32
// (O, m, sum) and a second launch joins them in the order of the keys, so
// results repeat bit for bit.  (Joined by the last of an item's runs instead,
// one CTA's loads in place of many: 31 us against 18 for one sequence of 8192
// keys and 16 rows.)
#include "kernels.h"
#include "ptx.cuh"
#include "rows.cuh"
#include "runs.h"
#include "tcgen05.cuh"

namespace dfl {

namespace {

constexpr int kDevBadLength = 0x4;
constexpr int kKT = 64;           // keys of a tile
constexpr int kMaxCtas = 320;     // runs at most (two parts each in the workspace)
constexpr float kLog2e = 1.4426950408889634f;

// Lengths of sequence j; a length or a count out of range leaves it without work.
struct Seq {
  int len, n;
  int tiles;   // key tiles of an item
  int qtiles;  // query tiles of a kv head
  __device__ __forceinline__ long long units(int nkv) const { return (long long)tiles * qtiles * nkv; }
};
template <typename P>
__device__ __forceinline__ Seq seq_of(const TreeAttnArgs& a, int j, int* status = nullptr) {
  Seq s;
  s.len = a.len[j];
  s.n = a.n_nodes ? a.n_nodes[j] : a.N;
  if (s.len < 0 || s.len > a.cap || s.n < 0 || s.n > a.N) {
    if (status) atomicOr(status, kDevBadLength);
    s.len = s.n = 0;
  }
  s.tiles = s.n ? P::tiles(s.len, s.n) : 0;
  s.qtiles = (s.n * a.g + P::ROWS - 1) / P::ROWS;
  return s;
}

// Word w of the set of nodes that a node sees.
__device__ __forceinline__ uint32_t node_bits(const TreeAttnArgs& a, int j, int node, int w) {
  if (w >= (a.N + 31) / 32) return 0u;
  if (a.mask) return a.mask[((size_t)j * a.N + node) * ((a.N + 31) / 32) + w];
  const int own = node - w * 32;  // the last node it sees, in this word
  return own < 0 ? 0u : own >= 31 ? ~0u : (2u << own) - 1u;
}

// A CTA's run: the tiles [u0, u1), and the sequence that holds u0 (base tiles
// come before it).  Every warp finds it by itself, so without a barrier; up to
// 32 sequences are one load a lane.  False: there is nothing for this CTA.
struct Run {
  Runs all;
  long long u0, u1, base;
  int j;
  Seq s;
};
__device__ __forceinline__ long long warp_scan(long long x) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    if ((int)(threadIdx.x & 31) >= o) x += y;
  }
  return x;
}
template <typename P>
__device__ __forceinline__ bool locate(const TreeAttnArgs& a, int cta, int ctas, Run& r) {
  const int lane = threadIdx.x & 31;
  auto units = [&](int i, Seq& q) {
    if (i >= a.b) return 0ll;
    q = seq_of<P>(a, i, a.status);  // (a length out of range is told wherever it is seen)
    return q.units(a.nkv);
  };
  Seq q = {0, 0, 0, 0};
  const long long mine = units(lane, q);
  const long long upto = warp_scan(mine);
  r.all.all = __shfl_sync(0xffffffffu, upto, 31);
  if (a.b > 32) {
    long long more = 0;
    Seq none;
    for (int i = 32 + lane; i < a.b; i += 32) more += units(i, none);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) more += __shfl_xor_sync(0xffffffffu, more, o);
    r.all.all += more;
  }
  const long long most = Runs::ratio(r.all.all + P::MIN_TILES - 1, P::MIN_TILES);
  r.all.runs = most < ctas ? most : ctas;
  if (cta >= r.all.runs) return false;
  r.u0 = r.all.start(cta);
  r.u1 = r.all.start(cta + 1);
  unsigned in = __ballot_sync(0xffffffffu, upto > r.u0);  // from the sequence that holds u0
  r.base = 0;
  r.j = 0;
  long long x = upto, t = mine;
  while (!in) {  // (more than 32 sequences)
    r.base += __shfl_sync(0xffffffffu, x, 31);
    r.j += 32;
    t = units(r.j + lane, q);
    x = warp_scan(t);
    in = __ballot_sync(0xffffffffu, r.base + x > r.u0);
  }
  const int l = __ffs(in) - 1;
  r.base += __shfl_sync(0xffffffffu, x - t, l);
  r.j += l;
  r.s.len = __shfl_sync(0xffffffffu, q.len, l);
  r.s.n = __shfl_sync(0xffffffffu, q.n, l);
  r.s.tiles = __shfl_sync(0xffffffffu, q.tiles, l);
  r.s.qtiles = __shfl_sync(0xffffffffu, q.qtiles, l);
  return true;
}

// What the second launch has to join: a record a run.  An item whose parts lie
// in several runs belongs to the second of them.
struct Join {
  int j, item;      // sequence, item of the sequence; j < 0: nothing
  int first, last;  // runs
  int slot;         // of the part in the first run; 0 in the others
  int n;            // nodes of the sequence
  int pad[2];
};

// Node and place in the group of a query row: x / g by a product with 2^32 / g
// rounded up, exact for x g < 2^32 (x is below 256 g, g at most 1024).
struct Group {
  uint32_t g, inv;
  __device__ __forceinline__ explicit Group(const TreeAttnArgs& a) : g(a.g), inv(a.g_inv) {}
  __device__ __forceinline__ int node(int x) const { return g == 1 ? x : (int)__umulhi((uint32_t)x, inv); }
  __device__ __forceinline__ int place(int x, int node) const { return x - node * (int)g; }
};

// A part in the workspace: O of rows x D fp32, then (m, sum) of each row, m in
// log2 units.  A run has two: of its first item, and of its last.  O lies by
// rows, or (the tensor-memory form, a thread a row) in columns of four, so that
// a warp's 16-byte stores lie side by side either way.
template <int D, int ROWS>
struct PartOf {
  float o[ROWS * D];
  float2 ml[ROWS];
  __device__ __forceinline__ static int by_row(int r, int c) { return r * D + c; }
  __device__ __forceinline__ static int by_four(int r, int c) { return (c / 4 * ROWS + r) * 4; }
};
// The workspace: the parts, then the records.
__device__ __forceinline__ uint8_t* aligned32(void* p) {
  return reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(p) + 31) & ~uintptr_t(31));
}
template <int D, int ROWS>
__device__ __forceinline__ PartOf<D, ROWS>* parts_of(const TreeAttnArgs& a) {
  return reinterpret_cast<PartOf<D, ROWS>*>(aligned32(a.ws));
}
template <int D, int ROWS>
__device__ __forceinline__ Join* joins_of(const TreeAttnArgs& a) {
  return reinterpret_cast<Join*>(parts_of<D, ROWS>(a) + 2 * kMaxCtas);
}
// CTA c's record; u0 its first tile, which is tile t0 of an item of `tiles`.
__device__ __forceinline__ void leave_join(Join* joins, const Runs& r, int c, long long u0, int j, int item, int t0,
                                           const Seq& s) {
  const int tiles = s.tiles;
  Join x;
  x.n = s.n;
  x.j = -1;
  const long long ub = u0 - t0;
  if (t0 > 0 && r.of(ub) == c - 1) {
    x.j = j;
    x.item = item;
    x.first = c - 1;
    x.last = (int)r.of(ub + tiles - 1);
    x.slot = r.start(c - 1) < ub;
  }
  joins[c] = x;
}

// Byte offset of 16-byte unit ch (of D / 8) of row r in a K, V or Q tile of
// `rows` rows: [D / 64 column halves][rows][128 bytes], unit c of a row at
// c ^ (r % 8), so the eight rows of a matrix load lie in different banks.
__device__ __forceinline__ int tile_off(int r, int ch, int rows) {
  return (ch >> 3) * rows * 128 + (r << 7) + (((ch & 7) ^ (r & 7)) << 4);
}

template <typename T>
__device__ __forceinline__ void mma16816(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  if constexpr (sizeof(T) == 2 && __is_same(T, __half)) mma_f16(d, a, b0, b1);
  else mma_bf16(d, a, b0, b1);
}
template <typename T>
__device__ __forceinline__ uint32_t pack2(float x, float y) {
  if constexpr (__is_same(T, __half)) {
    __half2 h = __floats2half2_rn(x, y);
    return *reinterpret_cast<uint32_t*>(&h);
  } else {
    __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<uint32_t*>(&h);
  }
}
// Exponent bits all set in either half of a pair: an infinity or NaN.
template <typename T>
__device__ __forceinline__ bool not_finite(uint32_t pair) {
  const uint32_t e = __is_same(T, __half) ? 0x7c00u : 0x7f80u;
  return (pair & e) == e || (pair >> 16 & e) == e;
}

// ---------------------------------------------------------------------------
// The warp-level form, for few rows a key: RW row warps of 16 query rows, KW
// groups of warps that share out a tile's keys.  Each warp keeps its own running
// maximum, sum and O over its keys; the groups are joined when the item or the
// run ends.  Bound by HBM: 64 sequences of 2000 keys with one token each (32 / 8
// heads) run at 5.6 TB/s; small calls by their two launches (12 us at 1024 keys).
template <int D, int RW>
struct Shape {
  static_assert(RW == 1 || RW == 2, "");
  static constexpr int KW = 4;
  static constexpr int THREADS = RW * KW * 32;
  static constexpr int ROWS = RW * 16;  // of a query tile
  // cached keys and the tree's side by side
  __host__ __device__ static int64_t tiles(int64_t len, int n) { return (len + n + kKT - 1) / kKT; }
  static constexpr int MIN_TILES = 2;  // of a run: fewer cost more in joining parts
  static constexpr int CTAS = RW == 1 || D == 64 ? 2 : 1;  // of an SM, by registers
  static constexpr int STAGES = CTAS == 2 ? 3 : 6;
  static constexpr int TILE = kKT * D * 2;  // bytes of a K or V tile
  static constexpr int SMEM = STAGES * 2 * TILE + ROWS * (kTreeMax / 32) * 4;
};

template <typename T, int D, int RW>
__global__ void __launch_bounds__(Shape<D, RW>::THREADS, Shape<D, RW>::CTAS)
    tree_attn_kernel(const TreeAttnArgs a) {
  using S = Shape<D, RW>;
  constexpr int KW = S::KW, ROWS = S::ROWS, THREADS = S::THREADS, NST = S::STAGES, TILE = S::TILE;
  constexpr int KEYS = kKT / KW;  // of a warp and tile
  constexpr int CH = D / 8;       // 16-byte units of a row
  extern __shared__ __align__(128) uint8_t sKV[];                                 // [NST][K, V]
  uint32_t* const sMask = reinterpret_cast<uint32_t*>(sKV + NST * 2 * TILE);  // [ROWS][W] of the rows' nodes
  __shared__ float2 s_ml[KW][ROWS];
  __shared__ uint32_t s_odd[kTreeMax / 32];  // tree keys whose V has an infinity or NaN

  pdl_wait();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rw = warp % RW, kg = warp / RW;
  const int g = a.g;
  const Group grp(a);
  const int W = (a.N + 31) / 32;
  Join* const joins = joins_of<D, ROWS>(a);
  Run run;
  if (!locate<S>(a, blockIdx.x, gridDim.x, run)) {
    if (tid == 0) joins[blockIdx.x].j = -1;
    return;
  }
  const long long u0 = run.u0, u1 = run.u1;

  // A place in the run: sequence, item of the sequence (kv head, query tile), tile.
  struct Place {
    int j, item, tile;
    Seq s;
  };
  auto next = [&](Place& p) {
    if (++p.tile < p.s.tiles) return;
    p.tile = 0;
    if (++p.item < a.nkv * p.s.qtiles) return;
    p.item = 0;
    do {
      if (++p.j >= a.b) return;
      p.s = seq_of<S>(a, p.j);
    } while (!p.s.tiles);
  };
  Place cur;
  cur.j = run.j;
  cur.s = run.s;
  cur.item = (int)Runs::ratio(u0 - run.base, cur.s.tiles);
  cur.tile = (int)(u0 - run.base - (long long)cur.item * cur.s.tiles);
  const int item0 = cur.item, tile0 = cur.tile;
  Place pre = cur;  // the tile to copy next

  // K and V of a tile: cached keys, then the tree's, then zeros
  auto copy = [&](const Place& p, int stg) {
    const int h = p.item / p.s.qtiles;
    const int t0 = p.tile * kKT, total = p.s.len + p.s.n;
    const size_t crow = ((size_t)p.j * a.nkv + h) * a.cap;
    uint8_t* dst = sKV + stg * 2 * TILE;
    for (int c = tid; c < kKT * CH; c += THREADS) {
      const int r = c / CH, ch = c % CH, t = t0 + r;
      const uint16_t *k = a.kc, *v = a.vc;
      if (t < p.s.len) {
        const size_t off = (crow + t) * D + ch * 8;
        k += off;
        v += off;
      } else if (t < total) {
        const int64_t off = p.j * a.t_seq + (t - p.s.len) * a.t_tok + h * D + ch * 8;
        k = a.kt + off;
        v = a.vt + off;
      }
      const int o = tile_off(r, ch, kKT);
      cp_async16(dst + o, k, t < total);
      cp_async16(dst + TILE + o, v, t < total);
    }
  };

  float m[2], l[2], o[D / 8][4];
  uint32_t qf[D / 16][4];
  const float sl2 = a.scale * kLog2e;
  long long u = u0;
  int stg = 0;
#pragma unroll
  for (int i = 0; i < NST - 1; ++i) {
    if (u0 + i < u1) {
      copy(pre, i);
      next(pre);
    }
    cp_async_commit();
  }
  bool first = true;  // the run's first item
  while (u < u1) {
    // ---------------- an item, or the run's part of it ----------------
    const int h = cur.item / cur.s.qtiles, row0 = (cur.item % cur.s.qtiles) * ROWS, j = cur.j;
    const int tiles = cur.s.tiles, t_first = cur.tile;
    const int t_last = (int)min((long long)tiles, t_first + (u1 - u));
    const int len = cur.s.len, n = cur.s.n;
    const int rows = min(ROWS, n * g - row0);
    __syncthreads();  // the last item's rows are no longer read
    for (int c = tid; c < ROWS * W; c += THREADS) {
      const int r = c / W, w = c % W;
      uint32_t x = 0;
      if (r < rows) {
        const int node = grp.node(row0 + r);
        x = node_bits(a, j, node, w);
        const int left = n - w * 32;  // nodes past the count are not there
        if (left < 32) x &= left <= 0 ? 0u : (1u << left) - 1u;
      }
      sMask[c] = x;
    }
    if (tid < kTreeMax / 32) s_odd[tid] = 0;
    __syncthreads();
    // Q, as the products take it: pairs of columns of rows lane / 4 and lane / 4 + 8
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int r = rw * 16 + (lane >> 2) + x * 8;
      const bool there = r < rows;
      const int node = there ? grp.node(row0 + r) : 0, hh = there ? grp.place(row0 + r, node) : 0;
      const uint16_t* q = a.q + j * a.q_seq + node * a.q_tok + (h * g + hh) * D + (lane & 3) * 2;
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        qf[k][x] = there ? *reinterpret_cast<const uint32_t*>(q + k * 16) : 0u;
        qf[k][x + 2] = there ? *reinterpret_cast<const uint32_t*>(q + k * 16 + 8) : 0u;
      }
    }
#pragma unroll
    for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    m[0] = m[1] = -INFINITY;
    l[0] = l[1] = 0.f;

    for (int tile = t_first; tile < t_last; ++tile, ++u) {
      cp_async_wait<NST - 2>();
      const int t0 = tile * kKT;
      uint8_t* const sK = sKV + stg * 2 * TILE;
      uint8_t* const sV = sK + TILE;
      const bool edge = t0 + kKT > len;  // holds keys of the tree, or none
      if (edge) {
        // 0 x V has to be 0 where a row does not see the key: infinities and
        // NaN of the tree's V are taken out and added to the rows that see them
        for (int c = tid; c < kKT * CH; c += THREADS) {
          const int r = c / CH, t = t0 + r - len;
          if (t < 0 || t >= n) continue;
          uint4* x = reinterpret_cast<uint4*>(sV + tile_off(r, c % CH, kKT));
          uint4 v = *x;
          if (!(not_finite<T>(v.x) | not_finite<T>(v.y) | not_finite<T>(v.z) | not_finite<T>(v.w))) continue;
          uint16_t* e = reinterpret_cast<uint16_t*>(&v);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (not_finite<T>(e[i])) e[i] = 0;
          *x = v;
          atomicOr(&s_odd[t >> 5], 1u << (t & 31));
        }
      }
      __syncthreads();  // the tile has landed; the stage before it is no longer read
      if (u + NST - 1 < u1) {
        copy(pre, (stg + NST - 1) % NST);
        next(pre);
      }
      cp_async_commit();

      // S = Q K^T over the warp's keys
      float s[KEYS / 8][4];
      const int key0 = kg * KEYS;
#pragma unroll
      for (int i = 0; i < KEYS / 8; ++i) s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.f;
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
#pragma unroll
        for (int i = 0; i < KEYS / 16; ++i) {
          uint32_t b[4];
          ldsm_x4(smem_u32(sK + tile_off(key0 + i * 16 + (lane & 7) + (lane >> 4) * 8, 2 * k + ((lane >> 3) & 1), kKT)),
                  b[0], b[1], b[2], b[3]);
          mma16816<T>(s[2 * i], qf[k], b[0], b[1]);
          mma16816<T>(s[2 * i + 1], qf[k], b[2], b[3]);
        }
      if (edge) {
#pragma unroll
        for (int i = 0; i < KEYS / 8; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int t = t0 + key0 + i * 8 + (lane & 3) * 2 + (e & 1) - len;
            const int r = rw * 16 + (lane >> 2) + (e >> 1) * 8;
            if (t >= 0 && !(t < n && (sMask[r * W + (t >> 5)] >> (t & 31) & 1))) s[i][e] = -INFINITY;
          }
      }
      // the running maximum and sum of rows lane / 4 and lane / 4 + 8
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        float mx = -INFINITY;
#pragma unroll
        for (int i = 0; i < KEYS / 8; ++i) mx = fmaxf(mx, fmaxf(s[i][2 * x], s[i][2 * x + 1]));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const float mn = fmaxf(m[x], mx * sl2);
        const float ref = mn == -INFINITY ? 0.f : mn;
        const float corr = fast_exp2(m[x] - ref);
        m[x] = mn;
        l[x] *= corr;
#pragma unroll
        for (int i = 0; i < KEYS / 8; ++i) {
          s[i][2 * x] = fast_exp2(fmaf(s[i][2 * x], sl2, -ref));
          s[i][2 * x + 1] = fast_exp2(fmaf(s[i][2 * x + 1], sl2, -ref));
          l[x] += s[i][2 * x] + s[i][2 * x + 1];
        }
        if (corr != 1.f) {
#pragma unroll
          for (int i = 0; i < D / 8; ++i) {
            o[i][2 * x] *= corr;
            o[i][2 * x + 1] *= corr;
          }
        }
      }
      // O += P V; P is rounded to the values' type, as the products take it:
      // half a step of a number below one, against V's own half step
#pragma unroll
      for (int i = 0; i < KEYS / 16; ++i) {
        const uint32_t p[4] = {pack2<T>(s[2 * i][0], s[2 * i][1]), pack2<T>(s[2 * i][2], s[2 * i][3]),
                               pack2<T>(s[2 * i + 1][0], s[2 * i + 1][1]), pack2<T>(s[2 * i + 1][2], s[2 * i + 1][3])};
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
          uint32_t b[4];
          ldsm_x4_t(smem_u32(sV + tile_off(key0 + i * 16 + (lane & 7) + ((lane >> 3) & 1) * 8, 2 * c + (lane >> 4), kKT)),
                    b[0], b[1], b[2], b[3]);
          mma16816<T>(o[2 * c], p, b[0], b[1]);
          mma16816<T>(o[2 * c + 1], p, b[2], b[3]);
        }
      }
      stg = (stg + 1) % NST;
    }

    // ---------------- join the key groups ----------------
    // the stage just read is free until the next tile's copy: it holds the
    // groups' O, ROWS x D fp32 each, half of them a round
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      l[x] += __shfl_xor_sync(0xffffffffu, l[x], 1);
      l[x] += __shfl_xor_sync(0xffffffffu, l[x], 2);
      if ((lane & 3) == 0) s_ml[kg][rw * 16 + (lane >> 2) + x * 8] = make_float2(m[x], l[x]);
    }
    __syncthreads();
    float mt[2], lt[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int r = rw * 16 + (lane >> 2) + x * 8;
      mt[x] = -INFINITY;
      lt[x] = 0.f;
#pragma unroll
      for (int k = 0; k < KW; ++k) mt[x] = fmaxf(mt[x], s_ml[k][r].x);
      const float ref = mt[x] == -INFINITY ? 0.f : mt[x];
#pragma unroll
      for (int k = 0; k < KW; ++k) lt[x] += s_ml[k][r].y * fast_exp2(s_ml[k][r].x - ref);
      const float w = fast_exp2(m[x] - ref);
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        o[i][2 * x] *= w;
        o[i][2 * x + 1] *= w;
      }
    }
    {
      float* const red = reinterpret_cast<float*>(sKV + ((stg + NST - 1) % NST) * 2 * TILE);
#pragma unroll
      for (int half = KW / 2; half > 0; half /= 2) {
        float* mine = red + (size_t)(kg % half) * ROWS * D + (rw * 32 + lane) * 4;
        if (kg >= half && kg < 2 * half) {
#pragma unroll
          for (int i = 0; i < D / 8; ++i)
            *reinterpret_cast<float4*>(mine + i * RW * 128) = make_float4(o[i][0], o[i][1], o[i][2], o[i][3]);
        }
        __syncthreads();
        if (kg < half) {
#pragma unroll
          for (int i = 0; i < D / 8; ++i) {
            const float4 v = *reinterpret_cast<const float4*>(mine + i * RW * 128);
            o[i][0] += v.x;
            o[i][1] += v.y;
            o[i][2] += v.z;
            o[i][3] += v.w;
          }
        }
        __syncthreads();
      }
    }
    const bool whole = t_first == 0 && t_last == tiles;
    if (kg == 0) {
      PartOf<D, ROWS>* part = parts_of<D, ROWS>(a) + (size_t)blockIdx.x * 2 + (first ? 0 : 1);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int r = rw * 16 + (lane >> 2) + x * 8;
        if (r >= rows) continue;
        const int node = grp.node(row0 + r), head = h * g + grp.place(row0 + r, node);
        for (int w = 0; w < W; ++w)
          for (uint32_t z = s_odd[w] & sMask[r * W + w]; z; z &= z - 1) {
            const uint16_t* v = a.vt + j * a.t_seq + (w * 32 + __ffs(z) - 1) * a.t_tok + h * D;
#pragma unroll
            for (int i = 0; i < D / 8; ++i)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const uint16_t b = v[i * 8 + (lane & 3) * 2 + e];
                if (not_finite<T>(b)) o[i][2 * x + e] += to_f32(*reinterpret_cast<const T*>(&b));
              }
          }
        if (whole) {
          const float inv = lt[x] > 0.f || lt[x] != lt[x] ? 1.f / lt[x] : 0.f;
          const size_t row = ((size_t)j * a.N + node) * a.nq + head;
          uint16_t* out = a.out + row * D + (lane & 3) * 2;
#pragma unroll
          for (int i = 0; i < D / 8; ++i)
            *reinterpret_cast<uint32_t*>(out + i * 8) = pack2<T>(o[i][2 * x] * inv, o[i][2 * x + 1] * inv);
          if (a.lse && (lane & 3) == 0)
            a.lse[row] = lt[x] == 0.f ? -INFINITY : (mt[x] + log2f(lt[x])) * (1.f / kLog2e);
        } else {
#pragma unroll
          for (int i = 0; i < D / 8; ++i)
            *reinterpret_cast<float2*>(&part->o[part->by_row(r, i * 8 + (lane & 3) * 2)]) =
                make_float2(o[i][2 * x], o[i][2 * x + 1]);
          if ((lane & 3) == 0) part->ml[r] = make_float2(mt[x], lt[x]);
        }
      }
    }
    first = false;
    cur.tile = t_last - 1;
    next(cur);
  }
  cp_async_wait<0>();
  if (tid == 0) leave_join(joins, run.all, blockIdx.x, u0, run.j, item0, tile0, run.s);
}

// Joins the parts of the items that have several.  Every CTA lists the records
// that ask for it, so that none is started for nothing, and takes (item, chunk)
// pairs in turn.  Bound by the loads' latency where an item has few rows, by L2
// where it has many.
constexpr int kJoinThreads = 256;

// The runs with a record, in s_run; their number.
__device__ __forceinline__ int list_joins(const Join* joins, int ctas, int* s_run, int* s_count) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int items = 0;
  for (int c0 = 0; c0 < ctas; c0 += kJoinThreads) {
    const int c = c0 + threadIdx.x;
    const bool some = c < ctas && joins[c].j >= 0;
    const unsigned in = __ballot_sync(0xffffffffu, some);
    if (lane == 0) s_count[warp] = __popc(in);
    __syncthreads();
    int at = items + __popc(in & ((1u << lane) - 1u));
    for (int w = 0; w < kJoinThreads / 32; ++w) {
      if (w < warp) at += s_count[w];
      items += s_count[w];
    }
    if (some) s_run[at] = c;
    __syncthreads();
  }
  return items;
}

// Parts by rows: JR query rows a chunk, 8 / JR warps a row that share out its
// parts (each the same ones every time; the shares are added in order).
template <typename T, int D, int ROWS, int JR>
__global__ void __launch_bounds__(kJoinThreads) tree_join_kernel(const TreeAttnArgs a, int ctas, int chunks) {
  constexpr int LANES = D / 4;                  // of a row: four columns each
  constexpr int SHARES = 8 / JR * (32 / LANES);  // of a row's parts
  __shared__ float4 s_o[JR][SHARES][LANES];
  __shared__ int s_count[kJoinThreads / 32], s_run[kMaxCtas];
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = a.g;
  const Join* const joins = joins_of<D, ROWS>(a);
  const int items = list_joins(joins, ctas, s_run, s_count);
  for (int work = blockIdx.x; work < items * chunks; work += gridDim.x) {
    const Join x = joins[s_run[work / chunks]];
    const int qtiles = (x.n * g + ROWS - 1) / ROWS;
    const int row0 = (x.item % qtiles) * ROWS, rows = min(ROWS, x.n * g - row0);
    const int lr = warp % JR, chunk = work % chunks, r = chunk * JR + lr;
    const int share = warp / JR * (32 / LANES) + lane / LANES, c = lane % LANES;
    if (chunk * JR >= rows) continue;
    const PartOf<D, ROWS>* parts = parts_of<D, ROWS>(a);
    const int n = x.last - x.first + 1;
    auto part = [&](int k) { return parts + 2 * (x.first + k) + (k ? 0 : x.slot); };
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r < rows) {
      for (int k = lane; k < n; k += 32) m = fmaxf(m, part(k)->ml[r].x);
#pragma unroll
      for (int q = 16; q > 0; q >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, q));
      const float ref = m == -INFINITY ? 0.f : m;
      for (int k0 = 0; k0 < n; k0 += 32) {
        const float2 ml = k0 + lane < n ? part(k0 + lane)->ml[r] : make_float2(-INFINITY, 0.f);
        const float w = fast_exp2(ml.x - ref);
        l += ml.y * w;
        const int ke = min(32, n - k0);
        for (int k = share; k - share < ke; k += 8 * SHARES) {
          float4 v[8];
          float wk[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int q = k + i * SHARES;
            wk[i] = __shfl_sync(0xffffffffu, w, q & 31);
            v[i] = q < ke ? *reinterpret_cast<const float4*>(&part(k0 + q)->o[PartOf<D, ROWS>::by_row(r, 4 * c)]) : make_float4(0.f, 0.f, 0.f, 0.f);
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (k + i * SHARES >= ke) continue;
            o.x += v[i].x * wk[i];
            o.y += v[i].y * wk[i];
            o.z += v[i].z * wk[i];
            o.w += v[i].w * wk[i];
          }
        }
      }
#pragma unroll
      for (int q = 16; q > 0; q >>= 1) l += __shfl_xor_sync(0xffffffffu, l, q);
    }
    if (SHARES > 1) {
      __syncthreads();  // (the last turn's are read)
      s_o[lr][share][c] = o;
      __syncthreads();
      if (share) continue;
#pragma unroll
      for (int k = 1; k < SHARES; ++k) {
        const float4 v = s_o[lr][k][c];
        o.x += v.x;
        o.y += v.y;
        o.z += v.z;
        o.w += v.w;
      }
    }
    if (r >= rows) continue;
    const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
    const Group grp(a);
    const int node = grp.node(row0 + r), head = x.item / qtiles * g + grp.place(row0 + r, node);
    const size_t row = ((size_t)x.j * a.N + node) * a.nq + head;
    *reinterpret_cast<uint2*>(a.out + row * D + 4 * c) =
        make_uint2(pack2<T>(o.x * inv, o.y * inv), pack2<T>(o.z * inv, o.w * inv));
    if (a.lse && c == 0) a.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * (1.f / kLog2e);
  }
}

// Parts by columns of four: 32 rows and 32 columns a chunk, a lane a row and a
// warp four columns, BATCH parts in flight.
template <typename T, int D, int ROWS, int BATCH>
__global__ void __launch_bounds__(kJoinThreads) tree_join_cols_kernel(const TreeAttnArgs a, int ctas, int chunks) {
  using Part = PartOf<D, ROWS>;
  __shared__ int s_count[kJoinThreads / 32], s_run[kMaxCtas];
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = a.g;
  const Join* const joins = joins_of<D, ROWS>(a);
  const int items = list_joins(joins, ctas, s_run, s_count);
  for (int work = blockIdx.x; work < items * chunks; work += gridDim.x) {
    const Join x = joins[s_run[work / chunks]];
    const int qtiles = (x.n * g + ROWS - 1) / ROWS;
    const int row0 = (x.item % qtiles) * ROWS, rows = min(ROWS, x.n * g - row0);
    const int chunk = work % chunks, r = chunk / (D / 32) * 32 + lane, c = chunk % (D / 32) * 32 + warp * 4;
    if (r >= rows) continue;
    const Part* parts = parts_of<D, ROWS>(a);
    const int n = x.last - x.first + 1;
    auto part = [&](int k) { return parts + 2 * (x.first + k) + (k ? 0 : x.slot); };
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k0 = 0; k0 < n; k0 += BATCH) {  // (the maximum runs along)
      float4 v[BATCH];
      float2 ml[BATCH];
      float top = m;
#pragma unroll
      for (int i = 0; i < BATCH; ++i) {
        ml[i] = k0 + i < n ? part(k0 + i)->ml[r] : make_float2(-INFINITY, 0.f);
        v[i] = k0 + i < n ? *reinterpret_cast<const float4*>(&part(k0 + i)->o[Part::by_four(r, c)])
                          : make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
      for (int i = 0; i < BATCH; ++i) top = fmaxf(top, ml[i].x);
      const float ref = top == -INFINITY ? 0.f : top, old = fast_exp2(m - ref);
      m = top;
      l *= old;
      o = make_float4(o.x * old, o.y * old, o.z * old, o.w * old);
#pragma unroll
      for (int i = 0; i < BATCH; ++i) {
        if (k0 + i >= n) continue;
        const float w = fast_exp2(ml[i].x - ref);
        l += ml[i].y * w;
        o.x += v[i].x * w;
        o.y += v[i].y * w;
        o.z += v[i].z * w;
        o.w += v[i].w * w;
      }
    }
    const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
    const Group grp(a);
    const int node = grp.node(row0 + r), head = x.item / qtiles * g + grp.place(row0 + r, node);
    const size_t row = ((size_t)x.j * a.N + node) * a.nq + head;
    *reinterpret_cast<uint2*>(a.out + row * D + c) = make_uint2(pack2<T>(o.x * inv, o.y * inv), pack2<T>(o.z * inv, o.w * inv));
    if (a.lse && c == 0) a.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * (1.f / kLog2e);
  }
}

// fn: the joining kernel, whose items have `chunks` chunks.
cudaError_t launch_join(const void* fn, TreeAttnArgs& a, int ctas, int chunks, cudaStream_t st) {
  int64_t grid = (int64_t)(ctas - 1) * chunks;  // an item has its second run's record: at most so many
  if (grid < 1) return cudaSuccess;             // one run: nothing is split
  if (grid > 4 * num_sms()) grid = 4 * num_sms();
  void* args[] = {&a, &ctas, &chunks};
  return launch_k(fn, dim3((unsigned)grid), dim3(kJoinThreads), 0, st, true, args);
}

template <typename T, int D, int RW>
cudaError_t launch(const TreeAttnArgs& a0, cudaStream_t st) {
  using S = Shape<D, RW>;
  TreeAttnArgs a = a0;
  const void* fn = (const void*)tree_attn_kernel<T, D, RW>;
  static unsigned long long done;  // devices that the kernel may use so much shared memory on
  cudaError_t e = allow_smem(fn, S::SMEM, &done);
  if (e != cudaSuccess) return e;
  int ctas = S::CTAS * num_sms();
  if (ctas > kMaxCtas) ctas = kMaxCtas;
  const int g = a.g;
  const int64_t items = (int64_t)a.b * a.nkv * ((a.N * g + S::ROWS - 1) / S::ROWS);
  const int64_t most = (items * S::tiles(a.cap, a.N) + S::MIN_TILES - 1) / S::MIN_TILES;  // were every cache full
  if (most < ctas) ctas = (int)most;
  void* args[] = {&a};
  e = launch_k(fn, dim3(ctas), dim3(S::THREADS), S::SMEM, st, true, args);
  if (e != cudaSuccess) return e;
  constexpr int JR = S::ROWS <= 16 ? 2 : 4;
  const int rows = a.N * a.g < S::ROWS ? a.N * a.g : S::ROWS;
  return launch_join((const void*)tree_join_kernel<T, D, S::ROWS, JR>, a, ctas, (rows + JR - 1) / JR, st);
}

// ---------------------------------------------------------------------------
// The tensor-memory form.  Two streams of 128 query rows each have O and two
// buffers of S (64 keys, fp32; P over its first half) in tensor memory: two
// blocks of a query tile of 256 rows, each over every tile; or, with up to 128
// rows (PAR), the same rows over every other tile, joined at the end.  One
// thread copies tiles of 128 keys (TMA, one ring of K and V tiles in the order
// of their use); a warp a stream issues the products of half a tile after
// another,
//   wait for P(i); O += P(i) V;  S(i + 2) = Q K^T, in the buffer of P(i)
// and four warps a stream make P(i + 1) of the other buffer meanwhile, a thread
// a row: neither waits for the other while both keep up.  (With one buffer of
// 128 keys each row's chain, weights then products, took 4.3 thousand cycles a
// tile of 256 rows; its products take 2.6.)
// Cached keys fill tiles of their own, the last one padded, and the tree's keys
// follow in theirs.  Tiles with absent keys have those rows of V zeroed by the
// threads that mask S, before they hand over P.
constexpr int kTcKeys = 128;
constexpr int kTcThreads = 352;  // warps 0-7: rows; 8, 9: the streams' products; 10: copies
constexpr int kTcMma = 8, kTcCopy = 10;
constexpr int kTcStep = 64;  // keys of a buffer of S

template <int D, bool PAR>
struct TcShape {
  static constexpr int ROWS = PAR ? 128 : 256;
  static constexpr int MIN_TILES = 1;
  __host__ __device__ static int64_t tiles(int64_t len, int n) {
    return (len + kTcKeys - 1) / kTcKeys + (n + kTcKeys - 1) / kTcKeys;
  }
  static constexpr int TILE = kTcKeys * D * 2;
  static constexpr int HALF = kTcKeys * 128;  // bytes of 64 columns of a tile
  static constexpr int QTILES = PAR ? 1 : 2;  // the streams' own rows of Q, or the same
  // as many tiles in flight as fit: with 5 in place of 6, 64 sequences of 2000 keys
  // and 32 rows took 118 us in place of 99
  static constexpr int SLOTS = D == 64 ? 12 : PAR ? 6 : 5;
  static constexpr int CTRL = 2 * 128 * 8 + 512;  // row statistics, then barriers and small change
  static constexpr int SMEM = (QTILES + SLOTS) * TILE + CTRL;
};

struct TcCtrl {
  float2 ml[2][128];
  uint64_t full[12], empty[12], s_ready[2][2], p_ready[2][2], pv_done[2], q_ready[2], o_done;
  uint32_t odd[2][kTreeMax / 32];
  uint32_t tmem;
};
static_assert(sizeof(TcCtrl) <= 2 * 128 * 8 + 512, "");

// 64 consecutive tensor-memory columns of this warp's 32 lanes to registers.
__device__ __forceinline__ void tmem_ld64_wait(uint32_t taddr, uint32_t (&v)[64]) {
#define R8(i) "=r"(v[i]), "=r"(v[i + 1]), "=r"(v[i + 2]), "=r"(v[i + 3]), "=r"(v[i + 4]), "=r"(v[i + 5]), "=r"(v[i + 6]), "=r"(v[i + 7])
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
      "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%64];\n"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,%48,%49,"
      "%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%65];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : R8(0), R8(8), R8(16), R8(24), R8(32), R8(40), R8(48), R8(56)
      : "r"(taddr), "r"(taddr + 32)
      : "memory");
#undef R8
}
#undef R8
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
// Whether a phase has completed.  Where it has, this answers some 150 cycles
// before the try_wait of mbar_wait does.
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
// One box of a tensor map of four dimensions (the rule of tma_load_2d for x).
__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, int x, int y, int z, int w, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
      "[%6];" ::"r"(smem_u32(dst)),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar))
      : "memory");
}
// The products and commits of tcgen05.cuh, called by a whole warp and issued by
// one of its lanes.  The choice stands beside each instruction: with a predicate
// kept from before, 4 x 64 nodes over 65536 keys took 243 us in place of 228.
__device__ __forceinline__ void mma_ss_elect(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{ .reg .pred p, q; setp.ne.u32 p, %4, 0; elect.sync _|q, 0xffffffff;\n"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_ts_elect(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{ .reg .pred p, q; setp.ne.u32 p, %4, 0; elect.sync _|q, 0xffffffff;\n"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p; }" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void commit_elect(uint64_t* bar) {
  asm volatile(
      "{ .reg .pred q; elect.sync _|q, 0xffffffff;\n"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0]; }" ::"r"(smem_u32(bar))
      : "memory");
}
// Two fp32 numbers in a register pair, worked on by one instruction.
__device__ __forceinline__ uint64_t pair(float x, float y) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(x), "f"(y));
  return v;
}
__device__ __forceinline__ float2 halves(uint64_t v) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
  return f;
}
__device__ __forceinline__ uint64_t fma2(uint64_t x, uint64_t y, uint64_t z) {
  uint64_t v;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(v) : "l"(x), "l"(y), "l"(z));
  return v;
}
__device__ __forceinline__ uint64_t add2(uint64_t x, uint64_t y) {
  uint64_t v;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(x), "l"(y));
  return v;
}
__device__ __forceinline__ void rows_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

template <typename T, int D, bool PAR>
__global__ void __launch_bounds__(kTcThreads, 1)
    tree_attn_tc_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                        const __grid_constant__ CUtensorMap ktmap, const __grid_constant__ CUtensorMap vtmap,
                        const TreeAttnArgs a) {
  using S = TcShape<D, PAR>;
  using Part = PartOf<D, S::ROWS>;
  constexpr int TILE = S::TILE, HALF = S::HALF, SLOTS = S::SLOTS, CH = D / 8;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* const sQ = smem;                      // [QTILES][D / 64][128 rows][128 bytes]
  uint8_t* const sKV = smem + S::QTILES * TILE;  // the ring
  TcCtrl& sh = *reinterpret_cast<TcCtrl*>(sKV + SLOTS * TILE);

  pdl_wait();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = a.g;
  const Group grp(a);
  Join* const joins = joins_of<D, S::ROWS>(a);
  Run run;
  if (!locate<S>(a, blockIdx.x, gridDim.x, run)) {
    if (tid == 0) joins[blockIdx.x].j = -1;
    return;
  }
  // The run's items, walked by every role by itself.
  struct Item {
    int j, item;   // sequence, its item
    int t0, t1;    // tiles of the run
    Seq s;
    int head, row0, ctx;  // kv head, first query row, tiles of cached keys
  };
  int left = (int)(run.u1 - run.u0);  // tiles of the run from the item on (a cache that fits the device has fewer than 2^31)
  Item it;
  it.j = run.j;
  it.s = run.s;
  it.item = (int)Runs::ratio(run.u0 - run.base, it.s.tiles);
  it.t0 = (int)(run.u0 - run.base - (long long)it.item * it.s.tiles);
  auto enter = [&]() {  // the rest of the item's places
    it.t1 = min(it.s.tiles, it.t0 + left);
    it.head = it.item / it.s.qtiles;
    it.row0 = (it.item % it.s.qtiles) * S::ROWS;
    it.ctx = (it.s.len + kTcKeys - 1) / kTcKeys;
  };
  auto leave = [&]() {  // to the next item; false at the run's end
    left -= it.t1 - it.t0;
    if (left <= 0) return false;
    it.t0 = 0;
    if (++it.item >= a.nkv * it.s.qtiles) {
      it.item = 0;
      do it.s = seq_of<S>(a, ++it.j);
      while (!it.s.tiles);
    }
    enter();
    return true;
  };
  enter();
  // Keys of tile t (of the run's item; 128 or more: all), and its halves that hold any.
  auto keys_of = [&](int t) { return t < it.ctx ? it.s.len - t * kTcKeys : it.s.n - (t - it.ctx) * kTcKeys; };
  auto halves_of = [&](int t) { return keys_of(t) > kTcStep ? 2 : 1; };
  // Q of the tile's rows (zero where there is none), a row by neighbouring threads
  auto copy_q = [&]() {
    const int rows = min(S::ROWS, it.s.n * g - it.row0);
    const uint16_t* q = a.q + it.j * a.q_seq + it.head * g * D;
#pragma unroll 4
    for (int i = 0; i < S::ROWS * CH / 256; ++i) {
      const int x = i * 256 + tid, r = x / CH, c = x % CH;
      const bool ok = r < rows;
      const int nd = ok ? grp.node(it.row0 + r) : 0, hd = ok ? grp.place(it.row0 + r, nd) : 0;
      cp_async16(sQ + (r >> 7) * TILE + tile_off(r & 127, c, 128), q + nd * a.q_tok + hd * D + c * 8, ok);
    }
    cp_async_commit();
  };
  // The first item's Q before any tile: behind the ring's first tiles of all
  // CTAs it would arrive 4 us later.
  if (warp < 8) copy_q();
  if (warp == kTcMma) tmem_alloc(&sh.tmem, 512);
  if (warp == kTcCopy && lane == 0) {
    for (int i = 0; i < SLOTS; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.empty[i], PAR ? 1 : 2);  // streams that read a tile
    }
    for (int m = 0; m < 2; ++m) {
      for (int i = 0; i < 2; ++i) {
        mbar_init(&sh.s_ready[m][i], 1);
        mbar_init(&sh.p_ready[m][i], 4);
      }
      mbar_init(&sh.pv_done[m], 1);
      mbar_init(&sh.q_ready[m], 8);
    }
    mbar_init(&sh.o_done, 2);
    fence_mbar_init();
    prefetch_tmap(&kmap);
    prefetch_tmap(&vmap);
    prefetch_tmap(&ktmap);
    prefetch_tmap(&vtmap);
  }
  if (tid < 2 * (kTreeMax / 32)) sh.odd[tid / (kTreeMax / 32)][tid % (kTreeMax / 32)] = 0;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  constexpr uint32_t kS = 2 * D;  // columns: O of the two streams, then the buffers of S of each
  bool dead = false;  // a wait gave up: the status is raised, the rest only drains
  auto wait = [&](uint64_t* bar, uint32_t n) {  // for the bar's n-th completion, from 0
    if (!dead && !mbar_test(bar, n & 1) && !mbar_wait(bar, n & 1, a.status)) dead = true;
  };
  // For the ring's x-th tile.  A barrier tells a phase from the one before it,
  // not from the one two before, so the one before has to be over: of the same
  // rows' earlier tiles it is, but with PAR the slot may have held the other
  // stream's, which can land after later ones.  Its release is waited for first
  // (the release before that is over: the tile in between was sent for after
  // it, and before the stream's last one, which was used; none but this stream
  // gives the next one).
  auto landed = [&](uint32_t x) {
    if (PAR && x >= SLOTS) wait(&sh.empty[x % SLOTS], x / SLOTS - 1);
    wait(&sh.full[x % SLOTS], x / SLOTS);
  };

  if (warp == kTcCopy) {
    if (lane == 0) {
      uint32_t x = 0;  // K and V tiles so far
      const int j = it.j, item = it.item, t0 = it.t0;  // (the first item's)
      fence_proxy_async_global();  // the inputs were written by generic stores
      do {
        for (int t = it.t0; t < it.t1; ++t)
#pragma unroll
          for (int kv = 0; kv < 2; ++kv) {
            const uint32_t slot = x % SLOTS;
            if (x >= SLOTS) wait(&sh.empty[slot], x / SLOTS - 1);
            if (dead) break;
            ++x;
            mbar_arrive_expect_tx(&sh.full[slot], TILE);
#pragma unroll
            for (int h = 0; h < D / 64; ++h) {
              uint8_t* dst = sKV + slot * TILE + h * HALF;
              if (t < it.ctx)
                tma_load_3d(dst, kv ? &vmap : &kmap, h * 64, t * kTcKeys, it.j * a.nkv + it.head, &sh.full[slot]);
              else
                tma_load_4d(dst, kv ? &vtmap : &ktmap, h * 64, it.head, (t - it.ctx) * kTcKeys, it.j, &sh.full[slot]);
            }
          }
      } while (!dead && leave());
      leave_join(joins, run.all, blockIdx.x, run.u0, j, item, t0, run.s);
      // nothing is in flight when the CTA ends (in order: each slot's last copy)
      if (dead)
        for (uint32_t i = x > SLOTS ? x - SLOTS : 0; i < x; ++i) mbar_wait(&sh.full[i % SLOTS], i / SLOTS & 1, nullptr);
    }
  } else if (warp >= kTcMma) {
    // All lanes walk along, so that descriptors and addresses are the warp's and
    // not a thread's.
    const uint32_t m = __reduce_max_sync(0xffffffffu, (unsigned)(warp - kTcMma));
    const uint32_t tmem = __reduce_max_sync(0xffffffffu, sh.tmem);
    constexpr uint32_t idesc_s = __is_same(T, __half) ? tc_idesc_f16(kTcStep) : tc_idesc_bf16(128, kTcStep);
    constexpr uint32_t idesc_o = (__is_same(T, __half) ? tc_idesc_f16(D) : tc_idesc_bf16(128, D)) | (1u << 16);
    constexpr uint32_t kHalfTile = kTcStep * 128;  // bytes from a half's rows to the other's
    const uint32_t kv_at = smem_u32(sKV), s_at = tmem + kS + 128 * m, o_at = tmem + D * m;
    const uint64_t qd = tc_sdesc_sw128(smem_u32(sQ) + (PAR ? 0 : m * TILE));
    uint32_t x0 = 0;  // K and V tiles before the item
    uint32_t item = 0, ns = 0, np = 0;  // items, halves sent for and added so far
    do {
      const int tiles = (int)__reduce_max_sync(0xffffffffu, (unsigned)(it.t1 - it.t0));
      constexpr int STEP = PAR ? 2 : 1;
      const int k0 = PAR ? (int)m : 0;
      int kq = k0, hq = 0;  // tile and half that the next S is of
      auto qk = [&]() {
        const uint32_t x = x0 + 2 * (uint32_t)kq, slot = x % SLOTS;
        if (hq == 0) landed(x);
        if ((dead = __any_sync(0xffffffffu, dead))) return;
        tc_fence_after();
        const uint64_t kd = tc_sdesc_sw128(kv_at + slot * TILE + hq * kHalfTile);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t o = ((k >> 2) * HALF + (k & 3) * 32) >> 4;  // (of the address field)
          mma_ss_elect(s_at + kTcStep * (ns & 1), qd + o, kd + o, idesc_s, k != 0);
        }
        commit_elect(&sh.s_ready[m][ns & 1]);
        ++ns;
        if (++hq == halves_of(it.t0 + kq)) {
          commit_elect(&sh.empty[slot]);
          hq = 0;
          kq += STEP;
        }
      };
      wait(&sh.q_ready[m], item);
      if (kq < tiles) qk();
      if (kq < tiles) qk();
      bool first = true;
      for (int k = k0; k < tiles && !dead; k += STEP) {
        const uint32_t x = x0 + 2 * (uint32_t)k + 1, slot = x % SLOTS;
        const int halves = halves_of(it.t0 + k);
        for (int h = 0; h < halves; ++h) {
          if (h == 0) landed(x);
          wait(&sh.p_ready[m][np & 1], np >> 1);
          if ((dead = __any_sync(0xffffffffu, dead))) break;
          tc_fence_after();
          const uint64_t vd = tc_sdesc_mn_sw128(kv_at + slot * TILE + h * kHalfTile, HALF, 1024);
#pragma unroll
          for (int c = 0; c < kTcStep / 16; ++c)
            mma_ts_elect(o_at, s_at + kTcStep * (np & 1) + 8 * c, vd + c * (2048 >> 4), idesc_o, !first || c != 0);
          first = false;
          commit_elect(&sh.pv_done[m]);
          ++np;
          if (h + 1 == halves) commit_elect(&sh.empty[slot]);
          if (kq < tiles) qk();
        }
      }
      commit_elect(&sh.o_done);
      x0 += 2 * (uint32_t)tiles;
      ++item;
    } while (__reduce_max_sync(0xffffffffu, (unsigned)leave()));
  } else if (warp < 8) {
    const int m = warp >> 2, lr = (warp & 3) * 32 + lane;  // stream, row of the stream
    const int rt = PAR ? lr : m * 128 + lr;                 // row of the query tile
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const float sl2 = a.scale * kLog2e;
    const int W = (a.N + 31) / 32;
    uint32_t x0 = 0, item = 0, ns = 0;
    for (;;) {
      const int rows = min(S::ROWS, it.s.n * g - it.row0);
      const bool there = rt < rows, some = rt - lane < rows;
      const int node = there ? grp.node(it.row0 + rt) : 0, hh = there ? grp.place(it.row0 + rt, node) : 0;
      {  // Q of the stream's rows
        cp_async_wait<0>();
        fence_proxy_async_shared();
        __syncwarp();
        if (lane < 2) mbar_arrive(&sh.q_ready[lane]);  // (its copies are of rows of either stream)
      }
      float mref = -INFINITY, lsum = 0.f;  // reference maximum (raw scores) and sum of the row
      const int tiles = it.t1 - it.t0;
      uint32_t* const odd = sh.odd[item & 1];
      for (int k = PAR ? m : 0; k < tiles; k += PAR ? 2 : 1) {
        const int t = it.t0 + k, keys = keys_of(t), halves_t = halves_of(t);
        const bool tree = t >= it.ctx;
        const int first = (tree ? t - it.ctx : t) * kTcKeys;  // the tile's first key or node
        for (int h = 0; h < halves_t; ++h, ++ns) {
          const int here = keys - h * kTcStep;  // keys of the half (64 or more: all)
          const bool edge = tree || here < kTcStep;
          const uint32_t sa = tmem + lanes + kS + 128 * m + kTcStep * (ns & 1);
          wait(&sh.s_ready[m][ns & 1], ns >> 1);
          tc_fence_after();
          if (some) {
            if (edge) {  // keys that the row does not see
#pragma unroll 1
              for (int w = 0; w < 2; ++w) {
                const int rest = here - w * 32;
                uint32_t bits = rest >= 32 ? ~0u : rest <= 0 ? 0u : (1u << rest) - 1u;
                if (tree) bits &= there ? node_bits(a, it.j, node, (first + h * kTcStep) / 32 + w) : 0u;
                uint32_t y[32];
                tmem_ld32_wait(sa + 32 * w, y);
#pragma unroll
                for (int n = 0; n < 32; ++n)
                  if (!(bits >> n & 1)) y[n] = 0xff800000u;
                tmem_st32(sa + 32 * w, y);
              }
              asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
            }
            // two passes over S: in registers for the maximum, 32 keys at a time for
            // the weights (a short loop; all 64 at once: 248 us in place of 243)
            uint32_t s[64];
            tmem_ld64_wait(sa, s);
            float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int n = 0; n < 64; n += 2)
              mx[n / 2 & 3] = fmaxf(mx[n / 2 & 3], fmaxf(__uint_as_float(s[n]), __uint_as_float(s[n + 1])));
            const float mnew = fmaxf(mref, fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])));
            // The reference follows the maximum where it lags by more than 8 in
            // log2 units: weights stay below 2^8, which P and the sums hold, and
            // O is seldom rescaled.
            const bool resc = mref != -INFINITY && (mnew - mref) * sl2 > 8.f;
            if (__any_sync(0xffffffffu, resc)) {
              const float corr = resc ? fast_exp2((mref - mnew) * sl2) : 1.f;
              lsum *= corr;
              // O holds what was added before this half: the last of it has to be
              // over (the one before it is, S was sent for after it)
              wait(&sh.pv_done[m], ns - 1);
              tc_fence_after();
#pragma unroll 1
              for (int c = 0; c < D; c += 32) {
                uint32_t o[32];
                tmem_ld32_wait(tmem + lanes + m * D + c, o);
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * corr);
                tmem_st32(tmem + lanes + m * D + c, o);
              }
            }
            if (mref == -INFINITY || resc) mref = mnew;
            const float nb = mref == -INFINITY ? 0.f : -mref * sl2;
            const uint64_t sl22 = pair(sl2, sl2), nb2 = pair(nb, nb);
            uint64_t sum[2] = {0, 0};  // pairs of zeros
#pragma unroll 1
            for (int w = 0; w < 2; ++w) {
              uint32_t y[32], p[16];
              tmem_ld32_wait(sa + 32 * w, y);
#pragma unroll
              for (int c = 0; c < 16; ++c) {
                const float2 e = halves(fma2(pair(__uint_as_float(y[2 * c]), __uint_as_float(y[2 * c + 1])), sl22, nb2));
                const float p0 = fast_exp2(e.x), p1 = fast_exp2(e.y);
                sum[c & 1] = add2(sum[c & 1], pair(p0, p1));
                p[c] = pack2<T>(p0, p1);
              }
              tmem_st16(sa + 16 * w, p);
            }
            const float2 total = halves(add2(sum[0], sum[1]));
            lsum += total.x + total.y;
            asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
          }
          if (edge) {
            // rows of V that are not there become zero, and so do a tree's
            // infinities and NaN: they are added to the rows that see them
            const uint32_t x = x0 + 2 * (uint32_t)k + 1;
            landed(x);
            const int r = lr % kTcStep;  // two threads a row of the half
            uint8_t* const sV = sKV + x % SLOTS * TILE;
            bool bad = false;
#pragma unroll 4
            for (int c = lr / kTcStep * (CH / 2), ce = c + CH / 2; c < ce; ++c) {
              uint4* e = reinterpret_cast<uint4*>(sV + tile_off(h * kTcStep + r, c, 128));
              if (r >= here) {
                *e = make_uint4(0u, 0u, 0u, 0u);
              } else if (tree) {
                uint4 y = *e;
                if (not_finite<T>(y.x) | not_finite<T>(y.y) | not_finite<T>(y.z) | not_finite<T>(y.w)) {
                  uint16_t* z = reinterpret_cast<uint16_t*>(&y);
#pragma unroll
                  for (int i = 0; i < 8; ++i)
                    if (not_finite<T>(z[i])) z[i] = 0;
                  *e = y;
                  bad = true;
                }
              }
            }
            if (bad) atomicOr(&odd[(first + h * kTcStep + r) >> 5], 1u << (r & 31));
            fence_proxy_async_shared();
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.p_ready[m][ns & 1]);
        }
      }
      // ---------------- the item's rows ----------------
      wait(&sh.o_done, item);
      tc_fence_after();
      const Item at = it;
      const bool more = leave();
      if (more) copy_q();  // the next one's Q: no product reads this one's any more
      float mt = mref * sl2, lt = lsum, w[2] = {1.f, 1.f};  // m in log2 units; weights of the streams' O
      if (mref == -INFINITY) mt = -INFINITY;
      if (PAR) sh.ml[m][lr] = make_float2(mt, lt);
      rows_sync();
      if (PAR) {
        const float2 o = sh.ml[m ^ 1][lr];
        const float top = fmaxf(mt, o.x), ref = top == -INFINITY ? 0.f : top;
        const float mine = fast_exp2(mt - ref), theirs = fast_exp2(o.x - ref);
        w[m] = mine;
        w[m ^ 1] = theirs;
        lt = m ? o.y * theirs + lt * mine : lt * mine + o.y * theirs;  // the same sum in both streams
        mt = top;
      }
      const bool whole = at.t0 == 0 && at.t1 == at.s.tiles;
      if (some) {
        const float inv = lt > 0.f || lt != lt ? 1.f / lt : 0.f;
        const size_t row = ((size_t)at.j * a.N + node) * a.nq + at.head * g + hh;
        Part* part = parts_of<D, S::ROWS>(a) + (size_t)blockIdx.x * 2 + (item ? 1 : 0);
        constexpr int COLS = PAR ? D / 2 : D;  // of this thread
#pragma unroll 1
        for (int c0 = PAR ? m * COLS : 0, ce = c0 + COLS; c0 < ce; c0 += 32) {
          float o[32];
          {
            uint32_t y[32];
            tmem_ld32_wait(tmem + lanes + (PAR ? 0 : m * D) + c0, y);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __uint_as_float(y[e]);
            if (PAR) {
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] *= w[0];
              if (tiles > 1) {
                tmem_ld32_wait(tmem + lanes + D + c0, y);
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = fmaf(__uint_as_float(y[e]), w[1], o[e]);
              }
            }
          }
          for (int k = 0; k < W; ++k) {
            uint32_t z = there ? odd[k] : 0u;
            if (z) z &= node_bits(a, at.j, node, k);
            for (; z; z &= z - 1) {
              const uint16_t* v = a.vt + at.j * a.t_seq + (k * 32 + __ffs(z) - 1) * a.t_tok + at.head * D + c0;
#pragma unroll
              for (int e = 0; e < 32; ++e) {
                const uint16_t y = v[e];
                if (not_finite<T>(y)) o[e] += to_f32(*reinterpret_cast<const T*>(&y));
              }
            }
          }
          if (there && whole) {
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] *= inv;
#pragma unroll
            for (int e = 0; e < 4; ++e)
              *reinterpret_cast<uint4*>(a.out + row * D + c0 + 8 * e) =
                  make_uint4(pack2<T>(o[8 * e], o[8 * e + 1]), pack2<T>(o[8 * e + 2], o[8 * e + 3]),
                             pack2<T>(o[8 * e + 4], o[8 * e + 5]), pack2<T>(o[8 * e + 6], o[8 * e + 7]));
          } else if (there) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              *reinterpret_cast<float4*>(&part->o[Part::by_four(rt, c0 + 4 * e)]) =
                  make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
          }
          __syncwarp();
        }
        if (there && (!PAR || m == 0)) {
          if (!whole) part->ml[rt] = make_float2(mt, lt);
          else if (a.lse) a.lse[row] = lt == 0.f ? -INFINITY : (mt + log2f(lt)) * (1.f / kLog2e);
        }
      }
      if (tid < kTreeMax / 32) sh.odd[(item & 1) ^ 1][tid] = 0;  // (last read before the barrier above)
      tc_fence_before();
      rows_sync();  // O is read, the statistics too
      x0 += 2 * (uint32_t)tiles;
      ++item;
      if (!more) break;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kTcMma) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <typename T, int D, bool PAR>
cudaError_t launch_tc(const TreeAttnArgs& a0, cudaStream_t st) {
  using S = TcShape<D, PAR>;
  TreeAttnArgs a = a0;
  const void* fn = (const void*)tree_attn_tc_kernel<T, D, PAR>;
  static unsigned long long done;
  cudaError_t e = allow_smem(fn, S::SMEM, &done);
  if (e != cudaSuccess) return e;
  const CUtensorMapDataType dt = __is_same(T, __half) ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  CUtensorMap maps[4];
  for (int v = 0; v < 2; ++v) {
    const uint64_t cd[3] = {(uint64_t)D, (uint64_t)a.cap, (uint64_t)a.b * a.nkv};
    const uint64_t cs[2] = {(uint64_t)D * 2, (uint64_t)a.cap * D * 2};
    const uint32_t cb[3] = {64, kTcKeys, 1};
    const uint64_t td[4] = {(uint64_t)D, (uint64_t)a.nkv, (uint64_t)a.N, (uint64_t)a.b};
    const uint64_t ts[3] = {(uint64_t)D * 2, (uint64_t)(a.N > 1 ? a.t_tok : a.nkv * D) * 2,
                            (uint64_t)(a.b > 1 ? a.t_seq : a.N * a.nkv * D) * 2};
    const uint32_t tb[4] = {64, 1, kTcKeys, 1};
    if (!encode_tmap(&maps[v], dt, v ? a.vc : a.kc, 3, cd, cs, cb, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_tmap(&maps[2 + v], dt, v ? a.vt : a.kt, 4, td, ts, tb, CU_TENSOR_MAP_SWIZZLE_128B))
      return cudaErrorInvalidValue;
  }
  int ctas = num_sms();
  if (ctas > kMaxCtas) ctas = kMaxCtas;
  const int g = a.g;
  const int64_t items = (int64_t)a.b * a.nkv * ((a.N * g + S::ROWS - 1) / S::ROWS);
  const int64_t most = (items * S::tiles(a.cap, a.N) + S::MIN_TILES - 1) / S::MIN_TILES;  // were every cache full
  if (most < ctas) ctas = (int)most;
  void* args[] = {&maps[0], &maps[1], &maps[2], &maps[3], &a};
  e = launch_k(fn, dim3(ctas), dim3(kTcThreads), S::SMEM, st, true, args);
  if (e != cudaSuccess) return e;
  const int rows = a.N * a.g < S::ROWS ? a.N * a.g : S::ROWS;
  // Items of many parts wait for loads: 16 in flight (39 rows of 3 x 2999 keys, 25
  // runs an item, 11.7 us in place of 13.7); of few parts or many rows, for the
  // CTAs that so many registers keep out (8 x 32 nodes over 4096 keys, 52.7 us in
  // place of 44.9).
  const bool many = PAR && items * 8 < ctas;
  const void* join = many ? (const void*)tree_join_cols_kernel<T, D, S::ROWS, 16>
                          : (const void*)tree_join_cols_kernel<T, D, S::ROWS, 8>;
  return launch_join(join, a, ctas, (rows + 31) / 32 * (D / 32), st);
}

// Query tiles of more than kWarpRows rows go to the tensor cores' own memory.
// Device time, us, warp-level / tensor-memory form, 8 kv heads, by rows of one:
//                             4          8          16           32
//   d 128, 64 x 2000 keys   94 / 96    98 / 96   107 / 97    150 / 99
//           8 x 4096        33 / 35    33 / 35    36 / 35     47 / 36
//           1 x 8192      17.2/17.4  17.3/17.3  17.7/17.4   19.3/17.2
//   d  64, 64 x 2000        63 / 79               71 / 79     89 / 79
//           1 x 8192                            14.3/14.6
// Sixteen rows are one of the warp-level form's tiles, 17 and more two: it wins
// at 64 dimensions up to there, and at 128 up to 8 rows; from 9 to 16 rows of 128
// the tensor-memory form would be up to a tenth faster, for a workspace of eight
// times the size.
constexpr int kWarpRows = 16;

// Tensor maps take strides below 2^40 bytes; that they grow with the dimension is
// what a cut out of larger tensors has, but not every order of dimensions, and
// other orders (or a repeated token's 0) are left to the warp-level form.
bool maps_fit(const TreeAttnArgs& a) {
  const int64_t tok = (int64_t)a.nkv * a.d, most = (int64_t)1 << 39;
  return (a.N == 1 || (a.t_tok >= tok && a.t_tok < most)) &&
         (a.b == 1 || (a.t_seq >= (a.N > 1 ? a.t_tok : tok) && a.t_seq < most));
}

template <typename T, int D>
cudaError_t launch_rows(const TreeAttnArgs& a, cudaStream_t st) {
  const int rows = a.N * a.g;
  if (rows > kWarpRows && maps_fit(a)) return rows <= 128 ? launch_tc<T, D, true>(a, st) : launch_tc<T, D, false>(a, st);
  return rows <= 16 ? launch<T, D, 1>(a, st) : launch<T, D, 2>(a, st);
}

template <typename T>
cudaError_t launch_type(const TreeAttnArgs& a, cudaStream_t st) {
  return a.d == 128 ? launch_rows<T, 128>(a, st) : launch_rows<T, 64>(a, st);
}

}  // namespace

size_t tree_attn_ws_bytes(int64_t b, int N, int nq, int nkv, int d) {
  (void)b;
  const int rows = N * (nq / nkv);
  const int tile = rows <= 16 ? 16 : rows <= 128 ? 128 : 256;
  return (size_t)kMaxCtas * (2 * (size_t)tile * (d + 2) * 4 + sizeof(Join)) + 32;
}

cudaError_t tree_attention(const TreeAttnArgs& a, int dtype, cudaStream_t st) {
  return dtype == 1 ? launch_type<__half>(a, st) : launch_type<__nv_bfloat16>(a, st);
}

}  // namespace dfl
