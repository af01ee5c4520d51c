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
// Work is shared out by keys, not by sequences: the 64-key tiles of all
// (sequence, kv head, query tile) items, in that order, are cut into as many
// equal runs as CTAs are resident, whatever the lengths (which only the device
// knows).  A CTA walks its run with the online softmax (running maximum and
// sum, O rescaled when the maximum rises); an item that lies within one run is
// written straight out, the parts of the others go to the workspace as fp32
// (O, m, sum) and a second launch joins them in the order of the keys, so
// results repeat bit for bit.
#include "kernels.h"
#include "ptx.cuh"
#include "rows.cuh"
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
  s.qtiles = (s.n * (a.nq / a.nkv) + P::ROWS - 1) / P::ROWS;
  return s;
}

// Word w of the set of nodes that a node sees.
__device__ __forceinline__ uint32_t node_bits(const TreeAttnArgs& a, int j, int node, int w) {
  if (w >= (a.N + 31) / 32) return 0u;
  if (a.mask) return a.mask[((size_t)j * a.N + node) * ((a.N + 31) / 32) + w];
  const int own = node - w * 32;  // the last node it sees, in this word
  return own < 0 ? 0u : own >= 31 ? ~0u : (2u << own) - 1u;
}

// Sum over the block of a 64-bit number, and over the threads before this one.
__device__ __forceinline__ long long block_scan(long long v, long long* s_warp, long long& before) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
  before = x - v;
  long long all = 0;
  for (int w = 0; w < (int)blockDim.x / 32; ++w) {
    if (w < warp) before += s_warp[w];
    all += s_warp[w];
  }
  return all;
}

// Tiles of all items, and of the sequences before j.
template <typename P>
__device__ __forceinline__ long long count_tiles(const TreeAttnArgs& a, int j, long long* s_warp, long long& before) {
  long long x = 0, y = 0, none;
  for (int i = threadIdx.x; i < a.b; i += blockDim.x) {
    const long long t = seq_of<P>(a, i).units(a.nkv);
    y += t;
    if (i < j) x += t;
  }
  before = j ? block_scan(x, s_warp, none) : 0;
  return block_scan(y, s_warp, none);
}

// Runs: tiles [run_start(c), run_start(c + 1)) of `all` belong to CTA c < ctas.
template <typename P>
__device__ __forceinline__ long long run_count(long long all, int ctas) {
  const long long most = (all + P::MIN_TILES - 1) / P::MIN_TILES;
  return most < ctas ? most : ctas;
}
__device__ __forceinline__ long long run_start(long long all, long long runs, long long c) { return c * all / runs; }
__device__ __forceinline__ long long run_of(long long all, long long runs, long long u) {
  return ((u + 1) * runs - 1) / all;
}

// A part in the workspace: O of rows x D fp32, then (m, sum) of each row, m in
// log2 units.  O lies by rows, or, where a thread writes a whole row, in
// columns of four, so that a warp's 16-byte stores lie side by side.
template <int D, int ROWS, bool BY_ROW>
struct PartOf {
  float4 o[ROWS * D / 4];
  float2 ml[ROWS];
  static __device__ __forceinline__ int at(int r, int c) { return BY_ROW ? r * (D / 4) + c / 4 : (c / 4) * ROWS + r; }
};

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
// RW row warps of 16 query rows, KW groups of warps that share out a tile's
// keys.  Each warp keeps its own running maximum, sum and O over its keys; the
// groups are joined when the item or the run ends.
template <int D, int RW>
struct Shape {
  static constexpr int KW = RW == 1 ? 4 : 8 / RW;
  static constexpr int THREADS = RW * KW * 32;
  static constexpr int ROWS = RW * 16;  // of a query tile
  static constexpr bool BY_ROW = true;
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
  __shared__ long long s_warp[THREADS / 32];
  __shared__ float2 s_ml[KW][ROWS];
  __shared__ uint32_t s_odd[kTreeMax / 32];  // tree keys whose V has an infinity or NaN
  __shared__ int s_j0;
  __shared__ long long s_base;

  pdl_wait();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rw = warp % RW, kg = warp / RW;
  const int g = a.nq / a.nkv;
  const int W = (a.N + 31) / 32;
  long long none;
  const long long all = count_tiles<S>(a, 0, s_warp, none);
  if (blockIdx.x == 0)
    for (int i = tid; i < a.b; i += THREADS) seq_of<S>(a, i, a.status);  // out of range: told once
  if (all == 0) return;
  const long long runs = run_count<S>(all, gridDim.x);
  if (blockIdx.x >= runs) return;
  const long long u0 = run_start(all, runs, blockIdx.x), u1 = run_start(all, runs, blockIdx.x + 1);

  // the sequence that holds tile u0, and the tiles before it
  for (long long c = 0, base = 0; base <= u0; c += THREADS) {
    const long long i = c + tid;
    const long long t = i < a.b ? seq_of<S>(a, (int)i).units(a.nkv) : 0;
    long long before;
    const long long sum = block_scan(t, s_warp, before);
    before += base;
    if (before <= u0 && u0 < before + t) {
      s_j0 = (int)i;
      s_base = before;
    }
    base += sum;
  }
  __syncthreads();

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
  cur.j = s_j0;
  cur.s = seq_of<S>(a, cur.j);
  cur.item = (int)((u0 - s_base) / cur.s.tiles);
  cur.tile = (int)((u0 - s_base) % cur.s.tiles);
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
        const int node = (row0 + r) / g;
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
      const int node = there ? (row0 + r) / g : 0, hh = there ? (row0 + r) % g : 0;
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
    if (kg == 0) {
      const bool whole = t_first == 0 && t_last == tiles;
      using Part = PartOf<D, ROWS, true>;
      Part* part = static_cast<Part*>(a.ws) + (size_t)blockIdx.x * 2 + (first ? 0 : 1);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int r = rw * 16 + (lane >> 2) + x * 8;
        if (r >= rows) continue;
        const int node = (row0 + r) / g, head = h * g + (row0 + r) % g;
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
            reinterpret_cast<float2*>(&part->o[Part::at(r, i * 8)])[lane & 3] = make_float2(o[i][2 * x], o[i][2 * x + 1]);
          if ((lane & 3) == 0) part->ml[r] = make_float2(mt[x], lt[x]);
        }
      }
    }
    first = false;
    cur.tile = t_last - 1;
    next(cur);
  }
  cp_async_wait<0>();
}

// Joins the parts of one item: 16 query rows a CTA, a thread per row and four
// columns, the parts in the order of their keys.
constexpr int kJoinRows = 16, kJoinThreads = 256;

template <typename T, int D, typename S>
__global__ void __launch_bounds__(kJoinThreads) tree_join_kernel(const TreeAttnArgs a, int ctas) {
  constexpr int ROWS = S::ROWS;
  using Part = PartOf<D, ROWS, S::BY_ROW>;
  __shared__ long long s_warp[kJoinThreads / 32];
  pdl_wait();
  const int g = a.nq / a.nkv, most = (a.N * g + ROWS - 1) / ROWS;  // query tiles of a kv head
  constexpr int BLK = ROWS / kJoinRows;
  const int blk = blockIdx.x % BLK, qt = blockIdx.x / BLK % most;
  const int h = (int)(blockIdx.x / (BLK * most) % a.nkv), j = (int)(blockIdx.x / (BLK * most) / a.nkv);
  const Seq s = seq_of<S>(a, j);
  const int row0 = qt * ROWS, rows = min(ROWS, s.n * g - row0);
  if (rows <= blk * kJoinRows) return;  // (the same for the whole block)
  long long before;
  const long long all = count_tiles<S>(a, j, s_warp, before);
  const long long runs = run_count<S>(all, ctas);
  const long long ub = before + (long long)(h * s.qtiles + qt) * s.tiles;
  const long long c0 = run_of(all, runs, ub), c1 = run_of(all, runs, ub + s.tiles - 1);
  if (c0 == c1) return;  // written by the run itself
  const Part* parts = static_cast<const Part*>(a.ws);
  // the item is its run's first unless the run has tiles before it
  const Part* p0 = parts + 2 * c0 + (run_start(all, runs, c0) < ub ? 1 : 0);
  for (int it = threadIdx.x; it < kJoinRows * (D / 4); it += kJoinThreads) {
    // neighbouring threads read neighbouring places of a part
    const int r = blk * kJoinRows + (S::BY_ROW ? it / (D / 4) : it % kJoinRows);
    const int c = (S::BY_ROW ? it % (D / 4) : it / kJoinRows) * 4;
    if (r >= rows) continue;
    float m = p0->ml[r].x;
    for (long long k = c0 + 1; k <= c1; ++k) m = fmaxf(m, parts[2 * k].ml[r].x);
    const float ref = m == -INFINITY ? 0.f : m;
    float l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (long long k = c0; k <= c1; ++k) {
      const Part* p = k == c0 ? p0 : parts + 2 * k;
      const float2 ml = p->ml[r];
      const float4 v = p->o[Part::at(r, c)];
      const float w = fast_exp2(ml.x - ref);
      l += ml.y * w;
      o.x += v.x * w;
      o.y += v.y * w;
      o.z += v.z * w;
      o.w += v.w * w;
    }
    const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
    const int node = (row0 + r) / g, head = h * g + (row0 + r) % g;
    const size_t row = ((size_t)j * a.N + node) * a.nq + head;
    uint2 x;
    x.x = pack2<T>(o.x * inv, o.y * inv);
    x.y = pack2<T>(o.z * inv, o.w * inv);
    *reinterpret_cast<uint2*>(a.out + row * D + c) = x;
    if (a.lse && c == 0) a.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * (1.f / kLog2e);
  }
}

template <typename T, int D, int RW>
cudaError_t launch(const TreeAttnArgs& a0, cudaStream_t st) {
  using S = Shape<D, RW>;
  TreeAttnArgs a = a0;
  const void* fn = (const void*)tree_attn_kernel<T, D, RW>;
  cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM);
  if (e != cudaSuccess) return e;
  int ctas = S::CTAS * num_sms();
  if (ctas > kMaxCtas) ctas = kMaxCtas;
  const int g = a.nq / a.nkv;
  const int64_t items = (int64_t)a.b * a.nkv * ((a.N * g + S::ROWS - 1) / S::ROWS);
  const int64_t most = (items * S::tiles(a.cap, a.N) + S::MIN_TILES - 1) / S::MIN_TILES;  // were every cache full
  if (most < ctas) ctas = (int)most;
  void* args[] = {&a};
  e = launch_k(fn, dim3(ctas), dim3(S::THREADS), S::SMEM, st, true, args);
  if (e != cudaSuccess) return e;
  void* jargs[] = {&a, &ctas};
  return launch_k((const void*)tree_join_kernel<T, D, S>, dim3((unsigned)(items * (S::ROWS / kJoinRows))),
                  dim3(kJoinThreads), 0, st, true, jargs);
}

// ---------------------------------------------------------------------------
// The tensor-memory form.  Two streams of 128 query rows each have S (128 keys,
// fp32; P over its first half) and O in tensor memory: two blocks of a query
// tile of 256 rows, each over every tile; or, with up to 128 rows (PAR), the
// same rows over every other tile, joined at the end.  While one stream's four
// warps make P of its S (a thread a row, no exchange), the tensor cores work
// for the other.  One thread copies tiles (TMA, one ring of K and V tiles in
// the order of their use), one issues the products:
//   step v: wait for P of v; O += P V; S of step v + 2 = Q K^T
// Cached keys fill tiles of their own, the last one padded, and the tree's keys
// follow in theirs.  Tiles with absent keys have those rows of V zeroed by the
// threads that mask S, before they hand over P.
constexpr int kTcKeys = 128;
constexpr int kTcThreads = 320;  // warps 0-7: rows; 8: tensor memory and products; 9: copies
constexpr int kTcMma = 8, kTcCopy = 9;

template <int D, bool PAR>
struct TcShape {
  static constexpr int ROWS = PAR ? 128 : 256;
  static constexpr bool BY_ROW = false;
  static constexpr int MIN_TILES = 1;
  __host__ __device__ static int64_t tiles(int64_t len, int n) {
    return (len + kTcKeys - 1) / kTcKeys + (n + kTcKeys - 1) / kTcKeys;
  }
  static constexpr int TILE = kTcKeys * D * 2;
  static constexpr int HALF = kTcKeys * 128;  // bytes of 64 columns of a tile
  static constexpr int SLOTS = D == 128 ? 5 : 8;
  static constexpr int CTRL = 2 * 128 * 8 + 512;  // row statistics, then barriers and small change
  static constexpr int SMEM = 2 * TILE + SLOTS * TILE + CTRL;
};

struct TcCtrl {
  float2 ml[2][128];
  uint64_t full[8], empty[8], s_ready[2], p_ready[2], q_ready[2], o_done;
  long long warp[kTcThreads / 32], base;
  uint32_t odd[2][kTreeMax / 32];
  int j0;
  uint32_t tmem;
};
static_assert(sizeof(TcCtrl) <= 2 * 128 * 8 + 512, "");

// Waits for this thread's tensor-memory loads; names the registers of one, so
// that no use of them is scheduled before.
__device__ __forceinline__ void tmem_wait_ld(uint32_t (&v)[32]) {
#define R8(i) "+r"(v[i]), "+r"(v[i + 1]), "+r"(v[i + 2]), "+r"(v[i + 3]), "+r"(v[i + 4]), "+r"(v[i + 5]), "+r"(v[i + 6]), "+r"(v[i + 7])
  asm volatile("tcgen05.wait::ld.sync.aligned;" : R8(0), R8(8), R8(16), R8(24)::"memory");
#undef R8
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
// One box of a tensor map of four dimensions (the rule of tma_load_2d for x).
__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, int x, int y, int z, int w, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
      "[%6];" ::"r"(smem_u32(dst)),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void rows_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

template <typename T, int D, bool PAR>
__global__ void __launch_bounds__(kTcThreads, 1)
    tree_attn_tc_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                        const __grid_constant__ CUtensorMap ktmap, const __grid_constant__ CUtensorMap vtmap,
                        const TreeAttnArgs a) {
  using S = TcShape<D, PAR>;
  using Part = PartOf<D, S::ROWS, false>;
  constexpr int TILE = S::TILE, HALF = S::HALF, SLOTS = S::SLOTS, CH = D / 8;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* const sQ = smem;              // [2 streams][D / 64][128 rows][128 bytes]
  uint8_t* const sKV = smem + 2 * TILE;  // the ring
  TcCtrl& sh = *reinterpret_cast<TcCtrl*>(sKV + SLOTS * TILE);

  pdl_wait();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = a.nq / a.nkv;
  long long none;
  const long long all = count_tiles<S>(a, 0, sh.warp, none);
  if (blockIdx.x == 0)
    for (int i = tid; i < a.b; i += kTcThreads) seq_of<S>(a, i, a.status);  // out of range: told once
  if (all == 0) return;
  const long long runs = run_count<S>(all, gridDim.x);
  if (blockIdx.x >= runs) return;
  const long long u0 = run_start(all, runs, blockIdx.x), u1 = run_start(all, runs, blockIdx.x + 1);
  for (long long c = 0, base = 0; base <= u0; c += kTcThreads) {
    const long long i = c + tid;
    const long long t = i < a.b ? seq_of<S>(a, (int)i).units(a.nkv) : 0;
    long long before;
    const long long sum = block_scan(t, sh.warp, before);
    before += base;
    if (before <= u0 && u0 < before + t) {
      sh.j0 = (int)i;
      sh.base = before;
    }
    base += sum;
  }
  if (warp == kTcMma) tmem_alloc(&sh.tmem, 512);
  if (warp == kTcCopy && lane == 0) {
    for (int i = 0; i < SLOTS; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.empty[i], 1);
    }
    for (int m = 0; m < 2; ++m) {
      mbar_init(&sh.s_ready[m], 1);
      mbar_init(&sh.p_ready[m], 4);
      mbar_init(&sh.q_ready[m], 4);
    }
    mbar_init(&sh.o_done, 1);
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
  constexpr uint32_t kS = 2 * D;  // columns: O of the two streams, then their S

  // The run's items, walked by every role by itself.
  struct Item {
    int j, item;   // sequence, its item
    int t0, t1;    // tiles of the run
    Seq s;
    int head, row0, ctx;  // kv head, first query row, tiles of cached keys
  };
  long long u = u0;
  Item it;
  it.j = sh.j0;
  it.s = seq_of<S>(a, it.j);
  it.item = (int)((u0 - sh.base) / it.s.tiles);
  it.t0 = (int)((u0 - sh.base) % it.s.tiles);
  auto enter = [&]() {  // the rest of the item's places
    it.t1 = (int)min((long long)it.s.tiles, it.t0 + (u1 - u));
    it.head = it.item / it.s.qtiles;
    it.row0 = (it.item % it.s.qtiles) * S::ROWS;
    it.ctx = (it.s.len + kTcKeys - 1) / kTcKeys;
  };
  auto leave = [&]() {  // to the next item; false at the run's end
    u += it.t1 - it.t0;
    if (u >= u1) return false;
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
  bool dead = false;  // a wait gave up: the status is raised, the rest only drains
  auto wait = [&](uint64_t* bar, uint32_t n) {  // for the bar's n-th completion, from 0
    if (!dead && !mbar_wait(bar, n & 1, a.status)) dead = true;
  };

  if (warp == kTcCopy) {
    if (lane == 0) {
      uint32_t x = 0;  // K and V tiles so far
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
      // nothing is in flight when the CTA ends (in order: each slot's last copy)
      if (dead)
        for (uint32_t i = x > SLOTS ? x - SLOTS : 0; i < x; ++i) mbar_wait(&sh.full[i % SLOTS], i / SLOTS & 1, nullptr);
    }
  } else if (warp == kTcMma) {
    if (lane == 0) {
      constexpr uint32_t idesc_s = __is_same(T, __half) ? tc_idesc_f16(kTcKeys) : tc_idesc_bf16(128, kTcKeys);
      constexpr uint32_t idesc_o = (__is_same(T, __half) ? tc_idesc_f16(D) : tc_idesc_bf16(128, D)) | (1u << 16);
      uint32_t x0 = 0;             // K and V tiles before the item
      uint32_t item = 0, np[2] = {0, 0};
      do {
        const int steps = (it.t1 - it.t0) * (PAR ? 1 : 2);
        auto tile_of = [&](int v) { return x0 + 2 * (uint32_t)(PAR ? v : v >> 1); };
        auto last_use = [&](int v) { return PAR || (v & 1); };
        auto qk = [&](int v) {
          const int m = v & 1;
          const uint32_t x = tile_of(v), slot = x % SLOTS;
          wait(&sh.full[slot], x / SLOTS);
          if (dead) return;
          tc_fence_after();
          const uint32_t qa = smem_u32(sQ + m * TILE), kb = smem_u32(sKV + slot * TILE);
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint32_t o = (k >> 2) * HALF + (k & 3) * 32;
            tc_mma_ss(tmem + kS + 128 * m, tc_sdesc_sw128(qa + o), tc_sdesc_sw128(kb + o), idesc_s, k != 0);
          }
          tc_commit(&sh.s_ready[m]);
          if (last_use(v)) tc_commit(&sh.empty[slot]);
        };
        wait(&sh.q_ready[0], item);
        wait(&sh.q_ready[1], item);
        tc_fence_after();
        qk(0);
        if (steps > 1) qk(1);
        for (int v = 0; v < steps; ++v) {
          const int m = v & 1;
          const uint32_t x = tile_of(v) + 1, slot = x % SLOTS;
          wait(&sh.full[slot], x / SLOTS);
          wait(&sh.p_ready[m], np[m]++);
          if (dead) break;
          tc_fence_after();
          const uint32_t vb = smem_u32(sKV + slot * TILE);
#pragma unroll
          for (int k = 0; k < kTcKeys / 16; ++k)
            tc_mma_f16_ta(tmem + D * m, tmem + kS + 128 * m + 8 * k, tc_sdesc_mn_sw128(vb + k * 2048, HALF, 1024), idesc_o,
                          v > 1 || k != 0);
          if (last_use(v)) tc_commit(&sh.empty[slot]);
          if (v + 2 < steps) qk(v + 2);
        }
        tc_commit(&sh.o_done);
        x0 += 2 * (it.t1 - it.t0);
        ++item;
      } while (leave());
    }
  } else if (warp < 8) {
    const int m = warp >> 2, lr = (warp & 3) * 32 + lane;  // stream, row of the stream
    const int rt = PAR ? lr : m * 128 + lr;                 // row of the query tile
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const float sl2 = a.scale * kLog2e;
    const int W = (a.N + 31) / 32;
    uint32_t x0 = 0, item = 0, ns = 0;
    do {
      const int rows = min(S::ROWS, it.s.n * g - it.row0);
      const bool there = rt < rows, some = rt - lane < rows;
      const int node = there ? (it.row0 + rt) / g : 0, hh = there ? (it.row0 + rt) % g : 0;
      {  // this row of Q (zero where there is none)
        const uint16_t* q = a.q + it.j * a.q_seq + node * a.q_tok + (it.head * g + hh) * D;
#pragma unroll
        for (int c = 0; c < CH; ++c)
          *reinterpret_cast<uint4*>(sQ + m * TILE + tile_off(lr, c, 128)) =
              there ? *reinterpret_cast<const uint4*>(q + c * 8) : make_uint4(0u, 0u, 0u, 0u);
        fence_proxy_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.q_ready[m]);
      }
      float mref = -INFINITY, lsum = 0.f;  // reference maximum (raw scores) and sum of the row
      const int steps = (it.t1 - it.t0) * (PAR ? 1 : 2);
      uint32_t* const odd = sh.odd[item & 1];
      for (int v = m; v < steps; v += 2) {
        const int t = it.t0 + (PAR ? v : v >> 1);
        const bool tree = t >= it.ctx;
        const int first = (tree ? t - it.ctx : t) * kTcKeys;         // the tile's first key or node
        const int here = (tree ? it.s.n : it.s.len) - first;  // keys of the tile (128 or more: all)
        wait(&sh.s_ready[m], ns++);
        tc_fence_after();
        if (some) {
          // Two passes over S, 32 keys at a time (the next ones on their way):
          // the maximum, then the weights.  P of 32 keys takes half the columns
          // of their S, which lie behind all that is still to be read.
          const uint32_t sa = tmem + lanes + kS + 128 * m;
          const bool edge = tree || here < kTcKeys;
          uint32_t bits[4];  // keys that the row sees
          if (edge) {
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              const int left = here - w * 32;
              bits[w] = left >= 32 ? ~0u : left <= 0 ? 0u : (1u << left) - 1u;
              if (tree) bits[w] &= there ? node_bits(a, it.j, node, (first >> 5) + w) : 0u;
            }
          }
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
          uint32_t x[2][32];
          auto seen = [&](uint32_t (&y)[32], int w) {
            if (edge) {
#pragma unroll
              for (int n = 0; n < 32; ++n)
                if (!(bits[w] >> n & 1)) y[n] = 0xff800000u;
            }
          };
          tmem_ld32(sa, x[0]);
          tmem_wait_ld(x[0]);
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            tmem_ld32(sa + 32 * ((w + 1) & 3), x[(w + 1) & 1]);
            uint32_t(&y)[32] = x[w & 1];
            seen(y, w);
#pragma unroll
            for (int n = 0; n < 32; ++n) mx[n & 3] = fmaxf(mx[n & 3], __uint_as_float(y[n]));
            tmem_wait_ld(x[(w + 1) & 1]);
          }
          const float mnew = fmaxf(mref, fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])));
          // The reference follows the maximum where it lags by more than 8 in
          // log2 units: weights stay below 2^8, which P and the sums hold, and
          // O is seldom rescaled.
          const bool resc = mref != -INFINITY && (mnew - mref) * sl2 > 8.f;
          const float corr = resc ? fast_exp2((mref - mnew) * sl2) : 1.f;
          if (mref == -INFINITY || resc) mref = mnew;
          if (__any_sync(0xffffffffu, resc)) {
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {  // (the stream's earlier products were committed before this S)
              uint32_t o[32];
              tmem_ld32_wait(tmem + lanes + m * D + c, o);
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * corr);
              tmem_st32(tmem + lanes + m * D + c, o);
            }
          }
          const float nb = mref == -INFINITY ? 0.f : -mref * sl2;
          float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int w = 0; w < 4; ++w) {  // (the first 32 are in x[0] again)
            if (w < 3) tmem_ld32(sa + 32 * (w + 1), x[(w + 1) & 1]);
            uint32_t(&y)[32] = x[w & 1];
            seen(y, w);
            uint32_t p[16];
#pragma unroll
            for (int c = 0; c < 16; ++c) {
              const float p0 = fast_exp2(fmaf(__uint_as_float(y[2 * c]), sl2, nb));
              const float p1 = fast_exp2(fmaf(__uint_as_float(y[2 * c + 1]), sl2, nb));
              sum[c & 3] += p0 + p1;
              p[c] = pack2<T>(p0, p1);
            }
            if (w < 3) tmem_wait_ld(x[(w + 1) & 1]);
            tmem_st16(sa + 16 * w, p);
          }
          lsum = lsum * corr + ((sum[0] + sum[1]) + (sum[2] + sum[3]));
          asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        }
        if (here < kTcKeys || tree) {
          // rows of V that are not there become zero, and so do a tree's
          // infinities and NaN: they are added to the rows that see them
          const uint32_t x = x0 + 2 * (uint32_t)(t - it.t0) + 1, slot = x % SLOTS;
          wait(&sh.full[slot], x / SLOTS);
          uint8_t* const sV = sKV + slot * TILE;
          bool bad = false;
#pragma unroll 4
          for (int c = 0; c < CH; ++c) {
            uint4* e = reinterpret_cast<uint4*>(sV + tile_off(lr, c, 128));
            if (lr >= here) {
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
          if (bad) atomicOr(&odd[(first + lr) >> 5], 1u << (lr & 31));
          fence_proxy_async_shared();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.p_ready[m]);
      }
      // ---------------- the item's rows ----------------
      wait(&sh.o_done, item);
      tc_fence_after();
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
      const bool whole = it.t0 == 0 && it.t1 == it.s.tiles;
      if (some) {
        const float inv = lt > 0.f || lt != lt ? 1.f / lt : 0.f;
        const size_t row = ((size_t)it.j * a.N + node) * a.nq + it.head * g + hh;
        Part* part = static_cast<Part*>(a.ws) + (size_t)blockIdx.x * 2 + (item ? 1 : 0);
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
              if (steps > 1) {
                tmem_ld32_wait(tmem + lanes + D + c0, y);
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = fmaf(__uint_as_float(y[e]), w[1], o[e]);
              }
            }
          }
          if (there) {
          for (int k = 0; k < W; ++k) {
            uint32_t z = odd[k];
            if (z) z &= node_bits(a, it.j, node, k);
            for (; z; z &= z - 1) {
              const uint16_t* v = a.vt + it.j * a.t_seq + (k * 32 + __ffs(z) - 1) * a.t_tok + it.head * D + c0;
#pragma unroll
              for (int e = 0; e < 32; ++e) {
                const uint16_t y = v[e];
                if (not_finite<T>(y)) o[e] += to_f32(*reinterpret_cast<const T*>(&y));
              }
            }
          }
          if (whole) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float* y = o + 8 * e;
              *reinterpret_cast<uint4*>(a.out + row * D + c0 + 8 * e) =
                  make_uint4(pack2<T>(y[0] * inv, y[1] * inv), pack2<T>(y[2] * inv, y[3] * inv),
                             pack2<T>(y[4] * inv, y[5] * inv), pack2<T>(y[6] * inv, y[7] * inv));
            }
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              part->o[Part::at(rt, c0 + 4 * e)] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
          }
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
      x0 += 2 * (uint32_t)(it.t1 - it.t0);
      ++item;
    } while (leave());
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
  cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM);
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
  const int g = a.nq / a.nkv;
  const int64_t items = (int64_t)a.b * a.nkv * ((a.N * g + S::ROWS - 1) / S::ROWS);
  const int64_t most = (items * S::tiles(a.cap, a.N) + S::MIN_TILES - 1) / S::MIN_TILES;  // were every cache full
  if (most < ctas) ctas = (int)most;
  void* args[] = {&maps[0], &maps[1], &maps[2], &maps[3], &a};
  e = launch_k(fn, dim3(ctas), dim3(kTcThreads), S::SMEM, st, true, args);
  if (e != cudaSuccess) return e;
  void* jargs[] = {&a, &ctas};
  return launch_k((const void*)tree_join_kernel<T, D, S>, dim3((unsigned)(items * (S::ROWS / kJoinRows))),
                  dim3(kJoinThreads), 0, st, true, jargs);
}

// Query tiles of more than kWarpRows rows go to the tensor cores' own memory.
constexpr int kWarpRows = 64;

// The tensor maps want the tree's strides to grow: what a cut out of larger
// tensors has, but not every order of dimensions.
bool maps_fit(const TreeAttnArgs& a) {
  const int64_t tok = (int64_t)a.nkv * a.d;
  return (a.N == 1 || a.t_tok >= tok) && (a.b == 1 || a.t_seq >= (a.N > 1 ? a.t_tok : tok));
}

template <typename T, int D>
cudaError_t launch_rows(const TreeAttnArgs& a, cudaStream_t st) {
  const int rows = a.N * (a.nq / a.nkv);
  if (rows > kWarpRows && maps_fit(a)) return rows <= 128 ? launch_tc<T, D, true>(a, st) : launch_tc<T, D, false>(a, st);
  return rows <= 16 ? launch<T, D, 1>(a, st) : rows <= 32 ? launch<T, D, 2>(a, st) : launch<T, D, 4>(a, st);
}

template <typename T>
cudaError_t launch_type(const TreeAttnArgs& a, cudaStream_t st) {
  return a.d == 128 ? launch_rows<T, 128>(a, st) : launch_rows<T, 64>(a, st);
}

}  // namespace

size_t tree_attn_ws_bytes(int64_t b, int N, int nq, int nkv, int d) {
  (void)b;
  const int rows = N * (nq / nkv);
  const int tile = rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : rows <= 128 ? 128 : 256;
  return (size_t)kMaxCtas * 2 * tile * (d + 2) * 4;
}

cudaError_t tree_attention(const TreeAttnArgs& a, int dtype, cudaStream_t st) {
  return dtype == 1 ? launch_type<__half>(a, st) : launch_type<__nv_bfloat16>(a, st);
}

}  // namespace dfl
