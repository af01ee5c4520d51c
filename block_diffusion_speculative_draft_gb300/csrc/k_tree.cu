// k_tree.cu — bookkeeping of a tree of drafts: each node's set of ancestors,
// the walk that accepts a path, and the path's commit to a cache.
//
// A tree has up to kTreeMax nodes; parent[i] < i, -1 for a root; node 0 is the
// root of the walk (the last emitted token).
//
// All three move little: masks and walk are bound by latency (one CTA a
// sequence, chains of shared-memory reads), the commit by launch and one
// round trip to HBM until it moves tens of megabytes.
#include "kernels.h"
#include "ptx.cuh"

namespace dfl {

namespace {

constexpr int kDevCapacity = 0x1, kDevBadLength = 0x4, kDevBadTree = 0x10;

// Nodes of sequence j: its own count, or N; one out of range is none.
__device__ __forceinline__ int node_count(const int* n_nodes, int j, int N, int* status) {
  const int n = n_nodes ? n_nodes[j] : N;
  if (n >= 0 && n <= N) return n;
  if (threadIdx.x == 0) atomicOr(status, kDevBadLength);
  return 0;
}

// mask(i) = {i} + mask(parent(i)): every node keeps a link to an ancestor and
// the set of nodes up to that link.  A round joins the link's set and follows
// its link, which doubles the reach, so log2(depth) rounds end it.  A node
// whose parent is out of range, and all that hang from it, gets the empty set.
__global__ void __launch_bounds__(kTreeMax) tree_mask_kernel(const TreeMaskArgs a) {
  __shared__ uint32_t set[2][kTreeMax][kTreeMax / 32 + 1];  // odd stride: nodes of a warp in different banks
  __shared__ int link[2][kTreeMax];
  constexpr int kTop = -1, kBad = -2;
  pdl_wait();
  const int j = blockIdx.x, i = threadIdx.x, W = (a.N + 31) / 32;
  const int n = node_count(a.n_nodes, j, a.N, a.status);
  int up = kBad;
  if (i < n) {
    up = a.parent[(size_t)j * a.N + i];
    if (up < -1 || up >= i) {
      atomicOr(a.status, kDevBadTree);
      up = kBad;
    }
  }
  for (int w = 0; w < W; ++w) set[0][i][w] = i < n && (i >> 5) == w ? 1u << (i & 31) : 0u;
  link[0][i] = up;
  int cur = 0;
  while (__syncthreads_or(i < n && link[cur][i] >= 0)) {
    const int l = link[cur][i];
    for (int w = 0; w < W; ++w) set[cur ^ 1][i][w] = set[cur][i][w] | (l >= 0 ? set[cur][l][w] : 0u);
    link[cur ^ 1][i] = l >= 0 ? link[cur][l] : l;
    cur ^= 1;
  }
  if (i >= a.N) return;
  const bool ok = link[cur][i] == kTop;
  int depth = -1;
  uint32_t* out = a.mask + ((size_t)j * a.N + i) * W;
  for (int w = 0; w < W; ++w) {
    const uint32_t s = ok ? set[cur][i][w] : 0u;
    out[w] = s;
    depth += __popc(s);
  }
  if (a.depth) a.depth[(size_t)j * a.N + i] = depth;
}

// The walk: from node 0, the first child whose token is the target's token at
// the node, until there is none or the path is full.  Each node's next step is
// found for all nodes at once; one thread then follows the links.
__global__ void __launch_bounds__(kTreeMax) tree_accept_kernel(const TreeAcceptArgs a) {
  __shared__ int next[kTreeMax], want[kTreeMax], tok[kTreeMax], path[kTreeMax], last;
  pdl_wait();
  const int j = blockIdx.x, i = threadIdx.x;
  const int n = node_count(a.n_nodes, j, a.N, a.status);
  const size_t row = (size_t)j * a.N;
  int up = -1;
  next[i] = a.N;
  if (i < n) {
    want[i] = a.tok[row + i];
    tok[i] = a.tree_tok[row + i];
    up = a.parent[row + i];
    if (up < -1 || up >= i) {
      atomicOr(a.status, kDevBadTree);
      up = -1;
    }
  }
  __syncthreads();
  if (up >= 0 && want[up] >= 0 && want[up] == tok[i]) atomicMin(&next[up], i);
  __syncthreads();
  if (i == 0) {
    int m = -1;  // accepted drafts; the path has one node more
    if (n > 0) {
      path[0] = m = 0;
      for (int c = next[0]; c < a.N && m + 1 < a.R; c = next[c]) path[++m] = c;
    }
    last = m;
    const int corr = m >= 0 ? want[path[m]] : -1;
    a.n_out[j] = m;
    a.corr_out[j] = corr >= 0 ? corr : -1;
    // without a correction the block ends with the last token on the path
    if (a.next_tok) a.next_tok[j] = corr >= 0 ? corr : m >= 0 ? tok[path[m]] : -1;
  }
  __syncthreads();
  for (int r = i; r < a.R; r += blockDim.x) {
    a.path_out[(size_t)j * a.R + r] = r <= last ? path[r] : -1;
    if (a.emitted) {
      const int t = r < last ? tok[path[r + 1]] : r == last ? want[path[r]] : -1;
      a.emitted[(size_t)j * a.R + r] = t >= 0 ? t : -1;
    }
  }
}

// Rows of the path to the cache.  One warp takes one token's K or V of one
// layer (its heads lie side by side in the tree, cap rows apart in the cache),
// or 2 KB of a hidden row; four 16-byte loads a lane are issued before the
// stores.
constexpr int kCommitThreads = 256;
constexpr int kHidPiece = 128;  // 16-byte units of a hidden row's piece

__global__ void __launch_bounds__(kCommitThreads) tree_commit_kernel(const TreeCommitArgs a) {
  __shared__ int s_path[kTreeMax];
  pdl_wait();
  const int j = blockIdx.y, lane = threadIdx.x & 31;
  const int n = a.n[j], L0 = a.len[j];
  int fault = 0;
  if (n < -1 || n >= a.R || L0 < 0) fault = kDevBadLength;
  else if ((int64_t)L0 + n + 1 > a.cap) fault = kDevCapacity;
  const int c = fault ? 0 : n + 1;
  bool bad = false;
  for (int i = threadIdx.x; i < c; i += blockDim.x) {
    const int p = a.path[(size_t)j * a.R + i];
    s_path[i] = p;
    bad |= p < 0 || p >= a.N;
  }
  if (__syncthreads_or(bad)) fault = kDevBadTree;
  if (!fault) {
    const int ch = a.d / 8;          // 16-byte units of a head
    const int units = a.nkv * ch;    // of a token's K or V
    const int hp = a.hid ? (a.hid_units + kHidPiece - 1) / kHidPiece : 0;
    const int kv_items = 2 * a.L * c, items = kv_items + c * hp;
    const int warps = gridDim.x * (kCommitThreads / 32);
    for (int it = blockIdx.x * (kCommitThreads / 32) + (threadIdx.x >> 5); it < items; it += warps) {
      const uint4* src;
      uint4* dst;
      int len;
      size_t head = 0;  // extra distance of the cache's next head, in units
      if (it < kv_items) {
        const int i = it % c, lv = it / c, l = lv >> 1;
        const uint16_t* tree = (lv & 1) ? a.v_tree : a.k_tree;
        uint16_t* cache = (lv & 1) ? a.v : a.k;
        src = reinterpret_cast<const uint4*>(tree + (int64_t)l * a.ld_layer + (int64_t)j * a.ld_seq +
                                             (int64_t)s_path[i] * a.ld_tok);
        dst = reinterpret_cast<uint4*>(cache + ((((size_t)l * a.b + j) * a.nkv) * a.cap + L0 + i) * a.d);
        len = units;
        head = (size_t)(a.cap - 1) * ch;
      } else {
        const int x = it - kv_items, i = x / hp, p0 = (x % hp) * kHidPiece;
        src = reinterpret_cast<const uint4*>(a.hid) + ((size_t)j * a.N + s_path[i]) * a.hid_units + p0;
        dst = reinterpret_cast<uint4*>(a.hid_out) + ((size_t)j * a.R + i) * a.hid_units + p0;
        len = min(kHidPiece, a.hid_units - p0);
      }
      for (int u = lane; u < len; u += 128) {
        uint4 v[4];
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (u + 32 * q < len) v[q] = src[u + 32 * q];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int x = u + 32 * q;
          if (x < len) dst[x + (head ? (size_t)(x / ch) * head : 0)] = v[q];
        }
      }
    }
  }
  // The new length: where it goes to another place any CTA may write it; where
  // it replaces the old one, the last CTA of the sequence to have read that.
  bool mine = blockIdx.x == 0;
  if (a.tickets) {
    __shared__ int s_last;
    __syncthreads();
    if (threadIdx.x == 0) {
      s_last = atomicAdd(&a.tickets[j], 1) == (int)gridDim.x - 1;
      if (s_last) a.tickets[j] = 0;
    }
    __syncthreads();
    mine = s_last;
  }
  if (mine && threadIdx.x == 0) {
    if (fault) atomicOr(a.status, fault);
    a.len_out[j] = L0 + (fault ? 0 : c);
  }
}

}  // namespace

cudaError_t tree_mask(const TreeMaskArgs& a0, int b, cudaStream_t st) {
  TreeMaskArgs a = a0;
  void* args[] = {&a};
  return launch_k((const void*)tree_mask_kernel, dim3(b), dim3((a.N + 31) / 32 * 32), 0, st, true, args);
}

cudaError_t tree_accept(const TreeAcceptArgs& a0, int b, cudaStream_t st) {
  TreeAcceptArgs a = a0;
  void* args[] = {&a};
  return launch_k((const void*)tree_accept_kernel, dim3(b), dim3((a.N + 31) / 32 * 32), 0, st, true, args);
}

cudaError_t tree_commit(const TreeCommitArgs& a0, cudaStream_t st) {
  TreeCommitArgs a = a0;
  // a warp an item of a full path, up to eight CTAs an SM in all
  const int64_t items = (int64_t)a.R * (2 * a.L + (a.hid ? (a.hid_units + kHidPiece - 1) / kHidPiece : 0));
  const int64_t most = (8 * (int64_t)num_sms() + a.b - 1) / a.b;
  int64_t x = (items + kCommitThreads / 32 - 1) / (kCommitThreads / 32);
  x = x < most ? x : most;
  void* args[] = {&a};
  return launch_k((const void*)tree_commit_kernel, dim3((unsigned)(x < 1 ? 1 : x), a.b), dim3(kCommitThreads), 0, st,
                  true, args);
}

}  // namespace dfl
