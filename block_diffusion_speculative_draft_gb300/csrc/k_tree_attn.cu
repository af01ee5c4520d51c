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

namespace dfl {

namespace {

constexpr int kDevBadLength = 0x4;
constexpr int kKT = 64;           // keys of a tile
constexpr int kMaxCtas = 320;     // runs at most (two parts each in the workspace)
constexpr int kMinTiles = 2;      // tiles of a run at least: less is spent on joining parts
constexpr float kLog2e = 1.4426950408889634f;

// Lengths of sequence j; a length or a count out of range leaves it without work.
struct Seq {
  int len, n;
  int tiles;   // 64-key tiles of an item
  int qtiles;  // query tiles of a kv head
  __device__ __forceinline__ long long units(int nkv) const { return (long long)tiles * qtiles * nkv; }
};
template <int ROWS>
__device__ __forceinline__ Seq seq_of(const TreeAttnArgs& a, int j, int* status = nullptr) {
  Seq s;
  s.len = a.len[j];
  s.n = a.n_nodes ? a.n_nodes[j] : a.N;
  if (s.len < 0 || s.len > a.cap || s.n < 0 || s.n > a.N) {
    if (status) atomicOr(status, kDevBadLength);
    s.len = s.n = 0;
  }
  s.tiles = s.n ? (s.len + s.n + kKT - 1) / kKT : 0;
  s.qtiles = (s.n * (a.nq / a.nkv) + ROWS - 1) / ROWS;
  return s;
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
template <int ROWS>
__device__ __forceinline__ long long count_tiles(const TreeAttnArgs& a, int j, long long* s_warp, long long& before) {
  long long x = 0, y = 0, none;
  for (int i = threadIdx.x; i < a.b; i += blockDim.x) {
    const long long t = seq_of<ROWS>(a, i).units(a.nkv);
    y += t;
    if (i < j) x += t;
  }
  before = j ? block_scan(x, s_warp, none) : 0;
  return block_scan(y, s_warp, none);
}

// Runs: tiles [run_start(c), run_start(c + 1)) of `all` belong to CTA c < ctas.
__device__ __forceinline__ long long run_count(long long all, int ctas) {
  const long long most = (all + kMinTiles - 1) / kMinTiles;
  return most < ctas ? most : ctas;
}
__device__ __forceinline__ long long run_start(long long all, long long runs, long long c) { return c * all / runs; }
__device__ __forceinline__ long long run_of(long long all, long long runs, long long u) {
  return ((u + 1) * runs - 1) / all;
}

// A part in the workspace: O [rows][D] fp32, then (m, sum) [rows], m in log2 units.
template <int D, int ROWS>
struct Part {
  float o[ROWS][D];
  float2 ml[ROWS];
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
  static constexpr int ROWS = RW * 16;
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
  const long long all = count_tiles<ROWS>(a, 0, s_warp, none);
  if (blockIdx.x == 0)
    for (int i = tid; i < a.b; i += THREADS) seq_of<ROWS>(a, i, a.status);  // out of range: told once
  if (all == 0) return;
  const long long runs = run_count(all, gridDim.x);
  if (blockIdx.x >= runs) return;
  const long long u0 = run_start(all, runs, blockIdx.x), u1 = run_start(all, runs, blockIdx.x + 1);

  // the sequence that holds tile u0, and the tiles before it
  for (long long c = 0, base = 0; base <= u0; c += THREADS) {
    const long long i = c + tid;
    const long long t = i < a.b ? seq_of<ROWS>(a, (int)i).units(a.nkv) : 0;
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
      p.s = seq_of<ROWS>(a, p.j);
    } while (!p.s.tiles);
  };
  Place cur;
  cur.j = s_j0;
  cur.s = seq_of<ROWS>(a, cur.j);
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
        const int own = node - w * 32;  // the last node seen without a mask, in this word
        x = a.mask ? a.mask[((size_t)j * a.N + node) * W + w] : own < 0 ? 0u : own >= 31 ? ~0u : (2u << own) - 1u;
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
      Part<D, ROWS>* part = static_cast<Part<D, ROWS>*>(a.ws) + (size_t)blockIdx.x * 2 + (first ? 0 : 1);
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
            *reinterpret_cast<float2*>(&part->o[r][i * 8 + (lane & 3) * 2]) = make_float2(o[i][2 * x], o[i][2 * x + 1]);
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

template <typename T, int D, int ROWS>
__global__ void __launch_bounds__(kJoinThreads) tree_join_kernel(const TreeAttnArgs a, int ctas) {
  __shared__ long long s_warp[kJoinThreads / 32];
  pdl_wait();
  const int g = a.nq / a.nkv, most = (a.N * g + ROWS - 1) / ROWS;  // query tiles of a kv head
  constexpr int BLK = ROWS / kJoinRows;
  const int blk = blockIdx.x % BLK, qt = blockIdx.x / BLK % most;
  const int h = (int)(blockIdx.x / (BLK * most) % a.nkv), j = (int)(blockIdx.x / (BLK * most) / a.nkv);
  const Seq s = seq_of<ROWS>(a, j);
  const int row0 = qt * ROWS, rows = min(ROWS, s.n * g - row0);
  if (rows <= blk * kJoinRows) return;  // (the same for the whole block)
  long long before;
  const long long all = count_tiles<ROWS>(a, j, s_warp, before);
  const long long runs = run_count(all, ctas);
  const long long ub = before + (long long)(h * s.qtiles + qt) * s.tiles;
  const long long c0 = run_of(all, runs, ub), c1 = run_of(all, runs, ub + s.tiles - 1);
  if (c0 == c1) return;  // written by the run itself
  const Part<D, ROWS>* parts = static_cast<const Part<D, ROWS>*>(a.ws);
  // the item is its run's first unless the run has tiles before it
  const Part<D, ROWS>* p0 = parts + 2 * c0 + (run_start(all, runs, c0) < ub ? 1 : 0);
  for (int it = threadIdx.x; it < kJoinRows * (D / 4); it += kJoinThreads) {
    const int r = blk * kJoinRows + it / (D / 4), c = (it % (D / 4)) * 4;
    if (r >= rows) continue;
    float m = p0->ml[r].x;
    for (long long k = c0 + 1; k <= c1; ++k) m = fmaxf(m, parts[2 * k].ml[r].x);
    const float ref = m == -INFINITY ? 0.f : m;
    float l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (long long k = c0; k <= c1; ++k) {
      const Part<D, ROWS>* p = k == c0 ? p0 : parts + 2 * k;
      const float2 ml = p->ml[r];
      const float4 v = *reinterpret_cast<const float4*>(&p->o[r][c]);
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
  const int64_t most = items * ((a.cap + (int64_t)a.N + kKT - 1) / kKT);  // tiles, were every cache full
  if ((most + kMinTiles - 1) / kMinTiles < ctas) ctas = (int)((most + kMinTiles - 1) / kMinTiles);
  void* args[] = {&a};
  e = launch_k(fn, dim3(ctas), dim3(S::THREADS), S::SMEM, st, true, args);
  if (e != cudaSuccess) return e;
  void* jargs[] = {&a, &ctas};
  return launch_k((const void*)tree_join_kernel<T, D, S::ROWS>, dim3((unsigned)(items * (S::ROWS / kJoinRows))),
                  dim3(kJoinThreads), 0, st, true, jargs);
}

template <typename T>
cudaError_t launch_type(const TreeAttnArgs& a, cudaStream_t st) {
  const int rows = a.N * (a.nq / a.nkv);
  if (a.d == 128)
    return rows <= 16 ? launch<T, 128, 1>(a, st) : rows <= 32 ? launch<T, 128, 2>(a, st) : launch<T, 128, 4>(a, st);
  return rows <= 16 ? launch<T, 64, 1>(a, st) : rows <= 32 ? launch<T, 64, 2>(a, st) : launch<T, 64, 4>(a, st);
}

}  // namespace

size_t tree_attn_ws_bytes(int64_t b, int N, int nq, int nkv, int d) {
  (void)b;
  const int rows = N * (nq / nkv);
  const int tile = rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
  return (size_t)kMaxCtas * 2 * tile * (d + 2) * 4;
}

cudaError_t tree_attention(const TreeAttnArgs& a, int dtype, cudaStream_t st) {
  return dtype == 1 ? launch_type<__half>(a, st) : launch_type<__nv_bfloat16>(a, st);
}

}  // namespace dfl
