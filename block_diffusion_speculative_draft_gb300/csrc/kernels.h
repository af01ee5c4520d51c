// kernels.h — host-side launchers shared between the C-ABI translation unit
// and the kernel translation units.  Plain C++ declarations, no device code.
#pragma once
#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace dfl {

constexpr int kTile = 128;            // packed weight tile edge (rows x k-columns)
constexpr int kLayersPerLaunch = 8;   // layers batched into one commit GEMM launch
constexpr int kTileBytes = 16384;     // one packed int8 tile

// Streaming multiprocessors of the current device (queried once per device).
int num_sms();

// Whether launches may start early as programmatic dependents of the
// previous kernel in their stream (the library's launch mode).
bool launch_early();
void set_launch_mode(int mode);
int get_launch_mode();

enum Epi : int {
  EPI_STORE_F32 = 0,  // out[m][n] = y
  EPI_RESID_F32 = 1,  // out[m][n] += y
  EPI_SWIGLU = 2,     // g[m][j] = silu(gate_j) * up_j  (fp16)
  EPI_QKV = 3,        // per-head Q/K RMSNorm + RoPE; q, block k, block v (fp16)
  EPI_KVCOMMIT = 4,   // per-head K RMSNorm + RoPE; K, V appended to the cache
};

struct W8Args {
  const uint8_t* q;  // packed tiles
  const __half* s;   // logical-order scales (int8 weights only)
  int N, K, layout;
  int bits;  // 8: int8 tiles + per-row scales; 4: int4 tiles carrying their group scales
  int row0;   // first packed row used (multiple of 128)
  int nrows;  // packed rows used (multiple of 128)
  int M;      // activation rows
  int splits;  // k-splits = cluster size along y
  int epi;
  float* out_f32;
  int ldo;
  __half* out_h;  // EPI_SWIGLU: g [M][F]; EPI_QKV: q [M][nq d]
  __half* kout;   // EPI_QKV: block k [M][nkv d]; EPI_KVCOMMIT: layer's K cache
  __half* vout;
  const float* gq;
  const float* gk;
  int nq, nkv, d, F;
  float theta, eps;
  const int* len;    // [b] committed lengths
  const int* nacc;   // EPI_KVCOMMIT: accept lengths
  int rows_per_seq;  // activation rows per sequence
  int b, cap;
  int* status;
  // Deferred RMSNorm.  Reader side: when ss_in is set, the activations are
  // x * gamma (not yet normalised) and the epilogue scales each row's result
  // by rsqrt(sum_i ss_in[m][i] / K + eps), i < nss_in.  Writer side (STORE /
  // RESID): when xg_out is set, also write fp16(y * g_next) and each row's
  // sum of squares over this 128-column tile into ss_out[m][tile].
  const float* ss_in;
  int nss_in;
  float* ss_out;
  int nss_out;
  __half* xg_out;
  const float* g_next;
  // Lm-head input (RESID): when set, rows with slot m % hb_rps > 0 also go to
  // hb_out, compacted to row (m / hb_rps) (hb_rps - 1) + slot - 1, as
  // bf16(y * g_next): the final RMSNorm's per-row factor is left out, which
  // the argmax over each row's logits does not see.
  __nv_bfloat16* hb_out;
  int hb_rps;
  // A commit folded into the draft's QKV projection (EPI_QKV only; c_nacc
  // null: none): rows m >= mc0 are target-context rows, c_rps per sequence,
  // whose K/V go into this layer's cache ck / cv at len + slot for the
  // committed slots; the block's rows sit after the new length.
  int mc0;
  const int* c_nacc;
  int c_rps;
  __half* ck;
  __half* cv;
  // Several layers' projections in one launch (the K/V rows of every
  // layer's qkv for a commit): tile columns [i ntl, (i + 1) ntl) of the grid
  // belong to layer i < nl and use lq/ls/lk/lv/lgk[i] in place of
  // q/s/kout/vout/gk.  nl = 0: a single projection.
  int nl, ntl;
  const uint8_t* lq[kLayersPerLaunch];
  const __half* ls[kLayersPerLaunch];
  __half* lk[kLayersPerLaunch];
  __half* lv[kLayersPerLaunch];
  const float* lgk[kLayersPerLaunch];
  // RoPE frequencies theta^(-2p/d), p < d/2, as float pairs hi + lo of the
  // double value (per-head epilogues)
  float inv_hi[64];
  float inv_lo[64];
};

// Tensor-map encoder of the CUDA driver API (resolved once through the runtime).
bool encode_tmap_2d(CUtensorMap* map, CUtensorMapDataType dt, const void* base, uint64_t inner, uint64_t outer,
                    uint64_t row_bytes, uint32_t box_inner, uint32_t box_outer, CUtensorMapSwizzle swz);
// Same for a 3-D tensor: dims innermost first, strides (bytes) of dims 1 and 2.
bool encode_tmap_3d(CUtensorMap* map, CUtensorMapDataType dt, const void* base, const uint64_t dims[3],
                    const uint64_t strides[2], const uint32_t box[3], CUtensorMapSwizzle swz);
// Same for `rank` (2 to 5) dimensions: rank - 1 strides.
bool encode_tmap(CUtensorMap* map, CUtensorMapDataType dt, const void* base, int rank, const uint64_t* dims,
                 const uint64_t* strides, const uint32_t* box, CUtensorMapSwizzle swz);

// Lets a kernel use so much dynamic shared memory, once a device: `done` has a
// bit for each where that has been asked for.
cudaError_t allow_smem(const void* fn, int bytes, unsigned long long* done);

// Launch helpers: the programmatic-dependent-launch attribute is set when
// `pdl` is requested and the library's launch mode allows early launches
// (launch_early()); launch_kc also groups blocks into thread-block clusters
// of shape `cluster` (no cluster when 1x1x1).
cudaError_t launch_k(const void* fn, dim3 grid, dim3 block, size_t smem, cudaStream_t st, bool pdl, void** args);
cudaError_t launch_kc(const void* fn, dim3 grid, dim3 block, size_t smem, cudaStream_t st, bool pdl, dim3 cluster,
                      void** args);

// --- W8A16 GEMM (k_gemm_w8.cu) ---
int w8_pick_splits(int units, int KT);
cudaError_t w8_gemm(const W8Args& a, const __half* x, cudaStream_t st, bool pdl);
cudaError_t w8_pack(const void* w, int w_dtype, int64_t N, int64_t K, int layout, uint8_t* q_out, __half* s_out,
                    cudaStream_t st);
// int4 packing: s_out [N][K/128] group scales in logical order, q_out the
// packed tiles of kW4TileBytes each (nibbles + the tile's rows' scales)
cudaError_t w4_pack(const void* w, int w_dtype, int64_t N, int64_t K, int layout, uint8_t* q_out, __half* s_out,
                    cudaStream_t st);
constexpr int64_t kW4TileBytes = 8192 + 256;

// --- lm-head GEMM + argmax (k_lmhead.cu) ---
size_t lmhead_ws_bytes(int64_t M);
// Vocabulary tiles the lm-head kernel reads first (lmhead_tile_rows rows
// each): tiles [0, n) start every CTA's stream.
int lmhead_first_tiles(int M, int V, int H);
// Vocabulary rows per lm-head tile for M rows (the stride of the tiles that
// lmhead_first_tiles counts).
int lmhead_tile_rows(int M, int H);
cudaError_t lmhead_argmax(const __nv_bfloat16* h, const __nv_bfloat16* w, int M, int V, int H, int* idx_out,
                          float* maxlogit, float* logits, void* ws, cudaStream_t st, bool pdl, int* status);

// --- block attention (k_attn.cu) ---
struct AttnArgs {
  const __half* q;     // [M][nq][d]
  const __half* kblk;  // [M][nkv][d]
  const __half* vblk;
  const __half* kc;  // layer's K cache [b][nkv][cap][d]
  const __half* vc;
  const int* len;
  __half* out;  // [M][nq][d]
  int b, B, nq, nkv, d, cap;
  int* status;
  int nwc;  // compute warps (16 query rows each); the rest help with loads and the merge
  // a commit folded into this pass (null: none): the context grows by
  // commit_count(len, nacc, rps, cap) rows, written by this layer's QKV kernel
  const int* nacc;
  int rps;
  // L2 prefetch issued while the kernel would otherwise leave HBM idle:
  // pieces [pf_i0, pf_i1) of base + i * pf_stride, pf_bytes each (or none)
  const uint8_t* pf_base;
  size_t pf_stride;
  uint32_t pf_bytes;
  int pf_i0, pf_i1;
};
cudaError_t attention(const AttnArgs& a, cudaStream_t st, bool pdl);

// --- small kernels (k_small.cu) ---
// ss_out null: u = RMSNorm(x; gamma).  Else the deferred form: u = x * gamma
// and ss_out[m][H/128] = sums of squares per 128-column tile.
cudaError_t embed_rmsnorm(const __nv_bfloat16* E, const int* last_tok, int mask_id, int V, int b, int B, int H,
                          const float* gamma, float eps, float* x, __half* u, float* ss_out, cudaStream_t st,
                          bool pdl, int* status);

// Rows of a sequence a commit appends: min(n + 1, rps), or 0 when n is out
// of [-1, rps], the length is negative or the rows would pass cap (the
// length-update kernel flags those cases).
__device__ __forceinline__ int commit_count(int len, int n, int rps, int cap) {
  int c = n + 1 < rps ? n + 1 : rps;
  if (c < 0) c = 0;
  return (n >= -1 && n <= rps && len >= 0 && len + c <= cap) ? c : 0;
}
cudaError_t final_norm(const float* x, int b, int B, int H, const float* gamma, float eps, __nv_bfloat16* h,
                       float* hidden_out, cudaStream_t st, bool pdl);
cudaError_t commit_len_update(int* len, const int* nacc, int b, int rows_per_seq, int cap, cudaStream_t st,
                              bool pdl, int* status);
// --- temperature speculative-sampling accept (k_sample.cu) ---
struct SampleArgs {
  const float* logits;    // [b][R][V]
  const int* draft;       // [b][D]
  const float* u_acc;     // [b][D] uniforms in (0, 1)
  const float* u_sample;  // [b][V] uniforms in (0, 1)
  int b, R, D;
  int64_t V;
  float T;
  int P, P2;              // vocabulary slices per row (stats) / per sequence (pick)
  int64_t chunk, chunk2;  // slice lengths
  int* tickets;           // [2b] zero between calls
  float2* part;           // [b R][P] (max, exp-sum) of z / T per slice
  float* zx;              // [b R] z / T of each row's draft token
  int* sel;               // [b][2] row to sample (-1: none), token it excludes
  unsigned long long* keys;  // [b][P2]
  int* n_out;
  int* corr_out;
  int* emitted;
  int* next_tok;
};
int sample_parts(int b, int R, int64_t V);
int sample_parts2(int b, int64_t V);
size_t sample_ws_bytes(int b, int R, int64_t V);
cudaError_t verify_sample(const float* logits, const int* draft, int b, int R, int D, int64_t V, float T,
                          const float* u_acc, const float* u_sample, int* n_out, int* corr_out, int* emitted,
                          int* next_tok, void* ws, cudaStream_t st, bool pdl);
size_t verify_ws_bytes(int b, int R, int64_t V);
cudaError_t verify_accept(const float* logits, const int* draft, int b, int R, int D, int64_t V, int* n_out,
                          int* corr_out, int* emitted, int* next_tok, void* ws, cudaStream_t st, bool pdl);

// --- filtered sampling, filtered accept, top logits (k_filter.cu) ---
constexpr float kFilterMinT = 1e-6f, kFilterMaxT = 1e6f;  // sampling temperatures (0: greedy)
constexpr int kTopLogitsMax = 1024;
constexpr int kInlineRows = 64;  // up to so many sampled rows need no state between launches
struct RowCut {  // one verified row; the workspace of every call is a run of these
  uint64_t cut;  // an entry is kept iff its place is at or above it
  float m;       // the row's maximum
  int accept;    // the row's draft token is accepted
  int tok;       // the token drawn where it is not; -2: still to be drawn
  int left;      // the row is left to the second launch
  float mass;    // its sum of weights, for that
  int ticket;    // rows done of the sequence that starts here; zero between calls
};
struct RowState {  // one sampled row between its launches
  float m, mass;   // the row's maximum and sum of weights
  int left;        // it is left to the second launch
};
struct FilterArgs {
  const void* logits;  // [rows] of V entries, ld apart
  int64_t V, ld;
  const float* temperature;  // per row (per sequence in the accept); null: T
  float T;
  const int* top_k;  // the filters, each nullable
  const float* top_p;
  const float* min_p;
  const float* u;  // uniforms, ld_u apart
  int64_t ld_u;
  int* tok;        // sample
  RowState* states;
  float* logprob;
  int R, D;        // accept
  int rows_used;   // rows of a sequence that can matter, set by the launcher
  const int* draft;
  const float* u_accept;
  RowCut* cuts;
  int* n_out;
  int* corr_out;
  int* emitted;
  int* next_tok;
  int K;           // top logits
  float* val;
  int* idx;
  float* lse;
  int* status;
  int idx_bits;    // set by the launchers: bits of V - 1, scale of the weights
  float scale;
  float unit;      // 1 / scale
};
cudaError_t filter_sample(FilterArgs a, int dtype, int64_t rows, cudaStream_t st);
inline size_t accept_ws_bytes(int64_t b, int R) { return (size_t)b * R * sizeof(RowCut); }
cudaError_t filter_accept(FilterArgs a, int dtype, int64_t b, cudaStream_t st);
cudaError_t top_logits(FilterArgs a, int dtype, int64_t rows, cudaStream_t st);

// --- distillation from a teacher's top logits (k_distill.cu) ---
constexpr int kDistillMaxK = 1024;
struct DistillArgs {
  const void* logits;  // student [rows] of V entries, ld apart
  int64_t V, ld;
  const float* t_val;  // teacher [rows][K]
  const int* t_idx;
  const float* t_lse;  // nullable
  int K;
  float T;
  const float* weight;  // nullable; the upstream gradient in the backward call
  float* loss;          // null in the backward call
  float4* stats;        // nullable: the row's sums (RowSums); input of the backward call
  void* dlogits;        // nullable
  int64_t ldd;
  int* status;
  float c;               // log2(e) / T and 1 / T as a float pair, set by the launcher
  float inv_hi, inv_lo;
};
cudaError_t distill(DistillArgs a, int dtype, int64_t rows, bool backward, cudaStream_t st);

// --- a tree of drafts: masks, accepted path, commit (k_tree.cu) ---
constexpr int kTreeMax = 256;  // nodes of a tree
struct TreeMaskArgs {
  const int* parent;   // [b][N]
  const int* n_nodes;  // [b], nullable
  int N;
  uint32_t* mask;  // [b][N][(N + 31) / 32]
  int* depth;      // [b][N], nullable
  int* status;
};
cudaError_t tree_mask(const TreeMaskArgs& a, int b, cudaStream_t st);
struct TreeAcceptArgs {
  const int* tok;       // [b][N] the target's token at each node
  const int* tree_tok;  // [b][N] the nodes' own tokens
  const int* parent;
  const int* n_nodes;  // nullable
  int N, R;
  int* n_out;
  int* corr_out;
  int* path_out;  // [b][R]
  int* emitted;   // [b][R], nullable
  int* next_tok;  // nullable
  int* status;
};
cudaError_t tree_accept(const TreeAcceptArgs& a, int b, cudaStream_t st);
struct TreeCommitArgs {
  uint16_t* k;  // cache [L][b][nkv][cap][d]
  uint16_t* v;
  const int* len;
  int* len_out;
  int b, cap, L, nkv, d, N, R;
  const uint16_t* k_tree;  // layer l, sequence j, node i at l ld_layer + j ld_seq + i ld_tok
  const uint16_t* v_tree;
  int64_t ld_layer, ld_seq, ld_tok;
  const int* path;  // [b][R]
  const int* n;     // [b]
  const uint16_t* hid;  // [b][N] rows of hid_units 16-byte units, nullable
  uint16_t* hid_out;    // [b][R]
  int hid_units;
  int* tickets;  // [b], zero between calls; null: len_out is not len
  int* status;
};
cudaError_t tree_commit(const TreeCommitArgs& a, cudaStream_t st);

// --- penalties, biases and grammar masks on rows of logits (k_adjust.cu) ---
constexpr int kAdjustMaxBias = 512;
constexpr int kAdjustMaxHist = (1 << 20) - 1 - kTreeMax;  // counts have 20 bits
struct AdjustArgs {
  const void* logits;  // sequence j's row r at (j R + r) ld
  void* out;
  int64_t V, ld, ld_out;
  int R;
  const int* hist;  // [b] rows of H tokens, ld_hist apart; nullable
  int64_t ld_hist;
  int H;
  const int* n_hist;
  const int* n_prompt;  // nullable: 0
  const int* draft;     // [b][D], nullable
  int D;
  const uint32_t* path;  // [b][R][(D + 31) / 32]; null: row r follows drafts 0..r-1
  const float* repetition;  // [b] each, nullable
  const float* frequency;
  const float* presence;
  const int* bias_idx;  // [b][K], nullable
  const float* bias_val;
  int K;
  const uint32_t* allow;  // rows of bits, ld_allow words apart; nullable
  int64_t n_allow, ld_allow;
  const int* allow_row;  // [b R], nullable: its own number
  int* status;
  int seg;        // set by the launcher: entries of a CTA's segment, segments of a row
  unsigned nseg;
};
cudaError_t adjust_logits(const AdjustArgs& a, int dtype, int64_t b, cudaStream_t st);

// --- attention of a tree's nodes over a cache (k_tree_attn.cu) ---
struct TreeAttnArgs {
  const uint16_t* q;   // node i, head h of sequence j at j q_seq + i q_tok + h d
  const uint16_t* kt;  // node i, kv head h at j t_seq + i t_tok + h d
  const uint16_t* vt;
  int64_t q_seq, q_tok, t_seq, t_tok;
  const uint16_t* kc;  // the layer's cache [b][nkv][cap][d]
  const uint16_t* vc;
  const int* len;
  const int* n_nodes;    // nullable
  const uint32_t* mask;  // [b][N][(N + 31) / 32]; null: node i sees nodes 0..i
  uint16_t* out;         // [b][N][nq][d]
  float* lse;            // [b][N][nq], nullable
  int b, N, nq, nkv, d, cap;
  int g;           // nq / nkv, and 2^32 / g rounded up
  uint32_t g_inv;
  float scale;
  void* ws;
  int* status;
};
constexpr int kTreeMaxGroup = 1024;  // query heads of a kv head
size_t tree_attn_ws_bytes(int64_t b, int N, int nq, int nkv, int d);
cudaError_t tree_attention(const TreeAttnArgs& a, int dtype, cudaStream_t st);

// Allocation-free variant of verify_accept: scratch lives in a fixed device
// array of kNoAllocScratchBytes inside the library (k_small.cu).
constexpr size_t kNoAllocScratchBytes = 64 * 1024;
size_t verify_noalloc_need(int b, int R, int64_t V);
cudaError_t verify_accept_noalloc(const float* logits, const int* draft, int b, int R, int D, int64_t V, int* n_out,
                                  int* corr_out, int* emitted, int* next_tok, cudaStream_t st);

}  // namespace dfl
