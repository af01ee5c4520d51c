/*
 * dflash.h — C ABI of libdflash.so: one DFlash block-diffusion draft step, the
 * greedy verify-accept that follows it, and the draft-KV commit, on one GB300
 * (sm_103a).
 *
 * The method (sources are web pages on DFlash, cited by title and section):
 *  - The drafter is a few-layer transformer that fills a block of B positions
 *    in ONE parallel non-causal pass; position 0 holds the last accepted token,
 *    the other positions hold the mask-token embedding; it reuses the target's
 *    embedding and lm-head (mlx-dspark v0.0.3 release notes, "Highlights").
 *  - It is conditioned on intermediate target activations, not logits
 *    (dflash-mlx summary, "What It Does").
 *  - Projections are int8 with per-output-channel fp16 scales (W8A16), Q/K get
 *    a per-head RMSNorm over head_dim values, RoPE is neox split-half
 *    (mirror-sd README, "The Story", Phases 2 and 3; "How It Works").
 *  - Verify: the target scores the block in one pass; the longest prefix on
 *    which the drafts equal the target's greedy choice is accepted and the
 *    target supplies one correction token (mirror-sd README, "How It Works",
 *    step 3; agentlens dflash-mlx, "How it works").
 *
 * Conventions for every entry point:
 *  - All tensor pointers are DEVICE pointers unless stated otherwise; the
 *    caller allocates and owns every buffer.  The library never allocates or
 *    frees device memory; scratch comes from a caller workspace.
 *  - fp16 and bf16 tensors are passed as uint16_t bit patterns.
 *  - `stream` is a cudaStream_t passed as void*; NULL means the legacy default
 *    stream.  Every call is asynchronous and stream-ordered: it enqueues work
 *    and returns.  Accept lengths and next tokens stay on the device.
 *  - Return value: DFLASH_OK or a negative dflash_status.  Host-checkable
 *    faults (null pointers, bad sizes, unsupported shapes, workspace too
 *    small) return before anything is enqueued.  A failed kernel launch
 *    returns DFLASH_ECUDA.  Faults only the device can see (KV capacity
 *    exceeded, a token or length out of range) set bits in a device status
 *    word, skip the offending writes and never trap; read it with
 *    dflash_get_status().
 *  - Workspaces: scratch regions contain counters that must be zero before
 *    the first call; zero-fill a workspace once after allocating it.  Every
 *    call leaves them zero again.  Calls that share a workspace must not
 *    overlap on the GPU (stream order them).
 */
#ifndef DFLASH_H
#define DFLASH_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define DFLASH_API __attribute__((visibility("default")))
#else
#define DFLASH_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum dflash_status {
  DFLASH_OK = 0,
  DFLASH_EINVAL = -1,       /* null pointer, negative or inconsistent size */
  DFLASH_EUNSUPPORTED = -2, /* shape outside what the kernels implement    */
  DFLASH_ECUDA = -3,        /* a CUDA runtime/launch error                  */
  DFLASH_ECAPACITY = -4,    /* KV cache capacity exceeded (device flag)    */
  DFLASH_EWORKSPACE = -5    /* workspace missing or too small              */
} dflash_status;

/* Bits of the device status word (dflash_get_status). */
#define DFLASH_DEV_KV_CAPACITY 0x1 /* a commit would pass `cap`: skipped   */
#define DFLASH_DEV_BAD_TOKEN 0x2   /* a token id outside [0, V): row zeroed */
#define DFLASH_DEV_BAD_LENGTH 0x4  /* len < 0 or n outside [-1, B]         */
#define DFLASH_DEV_BAD_PARAM 0x8   /* a row's temperature, top_k, top_p, min_p
                                      or teacher's value outside its range  */
#define DFLASH_DEV_BAD_TREE 0x10  /* a node's parent outside [-1, node), or a
                                      path's node outside the tree          */

/* Element types accepted by dflash_pack_w8a16 and by the calls on logits that
 * take a dtype. */
#define DFLASH_DTYPE_F32 0
#define DFLASH_DTYPE_F16 1
#define DFLASH_DTYPE_BF16 2

/* Row layouts of a packed W8A16 matrix. */
#define DFLASH_LAYOUT_PLAIN 0  /* rows in logical order                    */
#define DFLASH_LAYOUT_GATEUP 1 /* logical rows [gate F | up F]; packed so
                                  each 128-row tile holds 64 gate rows and
                                  the 64 matching up rows                  */

/* Drafter shape.  Supported: d in {64, 128}; H, nq*d, nkv*d, F, k*H multiples
 * of 128; nq a multiple of nkv; B in [2, 32]; V >= 1. */
typedef struct dflash_config {
  int32_t L;        /* drafter layers                                     */
  int32_t H;        /* hidden size                                        */
  int32_t nq, nkv;  /* query / key-value heads (GQA group = nq / nkv)     */
  int32_t d;        /* head_dim                                           */
  int32_t F;        /* SwiGLU width                                       */
  int32_t V;        /* vocabulary (rows of embedding and lm-head)         */
  int32_t B;        /* block size                                         */
  int32_t k;        /* hooked target layers: hidden rows are k*H wide     */
  int32_t mask_id;  /* token whose embedding fills block slots 1..B-1     */
  float rope_theta; /* RoPE base                                          */
  float eps;        /* RMSNorm epsilon                                    */
} dflash_config;

/* A packed weight matrix, int8 or int4 codes with fp16 scales.
 *  bits 8 (or 0), output of dflash_pack_w8a16: W[N][K] = q[N][K] * s[N];
 *    `q` is N*K bytes in the library's tiled layout, `s` is N fp16 scales in
 *    logical row order.
 *  bits 4, output of dflash_pack_w4a16: W[N][K] = q[N][K] * s[N][K/128]
 *    with q in [-7, 7]; `q` is dflash_w4a16_packed_bytes(N, K) bytes of
 *    tiles that carry their own scales, so `s` is not read and may be NULL.
 * Borrowed device pointers.  All matrices of one dflash_weights use the same
 * `bits`. */
typedef struct dflash_w8 {
  const void* q;
  const uint16_t* s;
  int64_t N, K;
  int32_t layout; /* DFLASH_LAYOUT_* */
  int32_t bits;   /* 8 (or 0) or 4 */
} dflash_w8;

/* Drafter weights.  qkv/o/gu/down point to HOST arrays of L descriptors
 * (read during the call); every tensor they describe is on the device.
 *   qkv[l]:  N = (nq + 2 nkv) d, K = H; rows q heads | k heads | v heads
 *   o[l]:    N = H, K = nq d
 *   gu[l]:   N = 2F, K = H, layout DFLASH_LAYOUT_GATEUP
 *   down[l]: N = H, K = F
 *   fc:      N = H, K = k H  (target hidden -> drafter width)
 * Gammas are fp32; embed and lm_head are the target's bf16 [V][H] tables. */
typedef struct dflash_weights {
  dflash_config cfg;
  dflash_w8 fc;
  const dflash_w8* qkv;
  const dflash_w8* o;
  const dflash_w8* gu;
  const dflash_w8* down;
  const float* gamma_hid;   /* [H]    norm after fc                        */
  const float* gamma_in;    /* [L][H] pre-attention norm                 */
  const float* gamma_post;  /* [L][H] pre-FFN norm                       */
  const float* gamma_q;     /* [L][d] per-head Q norm                    */
  const float* gamma_k;     /* [L][d] per-head K norm                    */
  const float* gamma_final; /* [H]    norm before the lm-head            */
  const uint16_t* embed;    /* bf16 [V][H]                               */
  const uint16_t* lm_head;  /* bf16 [V][H]                               */
} dflash_weights;

/* Draft KV cache: K after Q/K-norm and RoPE, V as projected, fp16,
 * k and v each [L][b][nkv][cap][d]; len[b] (device int32) = committed rows of
 * each sequence.  Context row j of a sequence sits at position j. */
typedef struct dflash_kv {
  uint16_t* k;
  uint16_t* v;
  int32_t* len;
  int32_t b;   /* sequences */
  int32_t cap; /* rows per sequence; at most 2^24 - 64 (positions are carried
                  exactly in fp32 by the RoPE epilogues), else the calls that
                  take a dflash_kv return DFLASH_EUNSUPPORTED */
} dflash_kv;

/* Library version string (static storage). */
DFLASH_API const char* dflash_version(void);

/* Human-readable name of a dflash_status (static storage). */
DFLASH_API const char* dflash_status_string(int32_t status);

/* Workspace bytes for dflash_draft_block, dflash_kv_commit and
 * dflash_commit_draft_block with b sequences and up to rows_per_seq hidden
 * rows per commit call (use B for the decode loop).  One workspace serves all
 * three calls.  Returns DFLASH_EINVAL / DFLASH_EUNSUPPORTED for a bad
 * config. */
DFLASH_API int32_t dflash_workspace_size(const dflash_config* cfg, int32_t b,
                              int32_t rows_per_seq, size_t* bytes);

/* W8A16 packing (mirror-sd README, "The Story", Phase 3: int8 weights with
 * per-output-channel fp16 scales).  w: device [N][K] of w_dtype.
 *   s[n] = fp16_rne(absmax_n / 127)            (division in fp32)
 *   q[n][k] = clamp(rint(w[n][k] / s[n]), -127, 127), 0 where s[n] == 0
 * and writes q in the tiled layout the GEMM streams (q_out: N*K bytes, 16-byte
 * aligned) and s in logical order (s_out: N fp16).  N, K multiples of 128;
 * layout DFLASH_LAYOUT_GATEUP needs N/2 a multiple of 64.  Offline, once per
 * weight; not on the timed path. */
DFLASH_API int32_t dflash_pack_w8a16(const void* w, int32_t w_dtype, int64_t N, int64_t K,
                          int32_t layout, void* q_out, uint16_t* s_out,
                          void* stream);

/* Bytes of the packed tiles of an int4 matrix: (N/128)(K/128) tiles of
 * 8448 bytes (8192 of codes, then the tile's 128 rows' fp16 scales).
 * N, K multiples of 128 (else DFLASH_EUNSUPPORTED). */
DFLASH_API int32_t dflash_w4a16_packed_bytes(int64_t N, int64_t K, size_t* bytes);

/* Symmetric int4 quantisation with one scale per row and 128-column group
 * (W4A16; a 4-bit drafter is the default of mlx-dspark v0.0.3, release
 * notes "Notes"; the symmetric [-7, 7] format and the group size of 128 are
 * this library's choice) of w[N][K] (device, w_dtype DFLASH_DTYPE_*):
 *   s[n][g] = fp16_rn(max_{k in group g} |w[n][k]| / 7)  (fp32 division)
 *   q[n][k] = clamp(rint(w[n][k] / s[n][k/128]), -7, 7)  (fp32 division;
 *             0 where the scale is 0)
 * q_out (16-byte aligned, dflash_w4a16_packed_bytes(N, K) bytes) receives
 * the tiles, s_out (device, N*K/128 fp16) the scales in logical order; both
 * caller-owned.  s_out is only a by-product once packing has finished (the
 * tiles hold a copy).  Layouts, shape limits and errors as dflash_pack_w8a16.
 * Asynchronous on `stream`. */
DFLASH_API int32_t dflash_pack_w4a16(const void* w, int32_t w_dtype, int64_t N, int64_t K,
                          int32_t layout, void* q_out, uint16_t* s_out,
                          void* stream);

/* Workspace bytes for dflash_w8a16_linear (0: split-K partial sums are
 * reduced on chip, so the call needs no scratch; ws may be NULL). */
DFLASH_API int32_t dflash_w8a16_linear_workspace_size(int64_t M, int64_t N, int64_t K,
                                           size_t* bytes);

/* The W8A16 projection alone (the kernel every drafter matmul runs on):
 * y[m][n] = s[n] * sum_k x[m][k] q[n][k] (int4: sum over groups g of
 * s[n][g] * sum_{k in g} x[m][k] q[n][k]) with fp16 activations x [M][K]
 * (16-byte aligned), fp32 accumulation, fp32 output y [M][N] in logical row
 * order (mirror-sd README, "The Story", Phase 3).  M in [1, 4096]. */
DFLASH_API int32_t dflash_w8a16_linear(const dflash_w8* w, const uint16_t* x, int64_t M,
                            float* y, void* ws, size_t ws_bytes, void* stream);

/* One draft step for b = kv->b sequences (mlx-dspark v0.0.3, "Highlights";
 * mirror-sd README, "How It Works"):
 *   x[slot 0] = embed[last_tok], x[slots 1..B-1] = embed[mask_id];
 *   slot i of sequence j sits at position len[j] + i;
 *   per layer: u = RMSNorm(x; gamma_in); [q|k|v] = W8(qkv) u;
 *              q, k = RoPE(per-head RMSNorm(q|k)); attention of the block's
 *              queries over [context K/V (len[j] rows) || block K/V], no mask;
 *              x += W8(o) attn; u = RMSNorm(x; gamma_post);
 *              x += W8(down)(silu(gate) * up), [gate|up] = W8(gu) u;
 *   h = RMSNorm(x[slots 1..B-1]; gamma_final) (rounded to bf16);
 *   draft[j][i] = argmax_v h[i] . lm_head[v] (lowest index on ties).
 * last_tok: [b] int32.  draft_out: [b][B-1] int32.
 * hidden_out (nullable): [b][B-1][H] fp32, h before bf16 rounding.
 * logits_out (nullable): [b][B-1][V] fp32.
 * When both are null the lm-head's input is bf16(x * gamma_final) without
 * the final RMSNorm's positive per-row factor, which leaves each row's
 * argmax unchanged (up to bf16 rounding of near ties).
 * The cache is read, never written: the block's own K/V live in the
 * workspace, so rejecting drafts needs no cache rollback. */
DFLASH_API int32_t dflash_draft_block(const dflash_weights* w, const dflash_kv* kv,
                           const int32_t* last_tok, int32_t* draft_out,
                           float* hidden_out, float* logits_out, void* ws,
                           size_t ws_bytes, void* stream);

/* Workspace bytes for dflash_lmhead_argmax with M rows. */
DFLASH_API int32_t dflash_lmhead_workspace_size(int64_t M, size_t* bytes);

/* idx_out[m] = argmax_v sum_k h[m][k] * w[v][k] (bf16 inputs, fp32
 * accumulation, lowest index on ties), the drafter's shared lm-head
 * (mlx-dspark v0.0.3, "Highlights").  h: [M][H] bf16, w: [V][H] bf16,
 * M in [1, 128], H a multiple of 64, rows 16-byte aligned.
 * maxlogit_out (nullable): [M] fp32.  logits_out (nullable): [M][V] fp32. */
DFLASH_API int32_t dflash_lmhead_argmax(const uint16_t* h, const uint16_t* w, int64_t M,
                             int64_t V, int64_t H, int32_t* idx_out,
                             float* maxlogit_out, float* logits_out, void* ws,
                             size_t ws_bytes, void* stream);

/* Workspace bytes for dflash_verify_accept. */
DFLASH_API int32_t dflash_verify_workspace_size(int32_t b, int32_t R, int64_t V,
                                     size_t* bytes);

/* Greedy verify-accept (mirror-sd README, "How It Works", step 3; agentlens
 * dflash-mlx, "How it works").  For each sequence j:
 *   a_r = argmax_v logits[j][r][v]  (fp32, lowest index on ties)
 *   n   = number of leading i < D with draft[j][i] == a_i
 *   corr = a_n if n < R else -1
 *   emitted[j] = draft[j][0..n) ++ [corr], padded with -1 to R entries
 *   next_tok[j] = last emitted token (slot 0 of the next block)
 * logits: [b][R][V] fp32; draft: [b][D] int32, 1 <= D <= R.
 * n_out, corr_out, next_tok_out: [b] int32 (next_tok_out nullable);
 * emitted_out: [b][R] int32 (nullable).  n_out feeds dflash_kv_commit. */
DFLASH_API int32_t dflash_verify_accept(const float* logits, const int32_t* draft,
                             int32_t b, int32_t R, int32_t D, int64_t V,
                             int32_t* n_out, int32_t* corr_out,
                             int32_t* emitted_out, int32_t* next_tok_out,
                             void* ws, size_t ws_bytes, void* stream);

/* Allocation-free verify-accept.  The pages describe no counterpart to this call;
 * it exists for callers that cannot allocate device memory themselves (for
 * example code running inside a stream capture that forbids allocation,
 * embedders whose memory is fully pre-reserved by another allocator, or
 * plain C hosts without a CUDA allocator wrapper).  It computes exactly what
 * dflash_verify_accept computes, with the same arguments minus the
 * workspace: its scratch is a fixed 64 KiB array inside the library's device
 * image, resident on every GPU that loads the library until the process
 * exits.  Shapes whose scratch would exceed that (more than 1024 sequences,
 * or b*R*slices keys beyond the array) return DFLASH_EWORKSPACE.  The first
 * call on a device resolves the array's device address (cudaGetSymbolAddress
 * with that device current) and keeps it for the life of the process; make
 * that first call before any stream capture, and do not call it again on a
 * device after cudaDeviceReset there (the kept address would be stale).  Each call clears the per-sequence counters it needs with
 * cudaMemsetAsync on the stream.  All calls share the one array, which keeps
 * the last call's contents, so calls that can overlap on the GPU (different
 * streams without ordering) race: serialise them.  No cudaMalloc, cudaFree
 * or other allocating routine is ever called. */
DFLASH_API int32_t dflash_verify_accept_noalloc(const float* logits,
                                                const int32_t* draft,
                                                int32_t b, int32_t R,
                                                int32_t D, int64_t V,
                                                int32_t* n_out,
                                                int32_t* corr_out,
                                                int32_t* emitted_out,
                                                int32_t* next_tok_out,
                                                void* stream);

/* Workspace bytes for dflash_verify_accept_sample. */
DFLASH_API int32_t dflash_verify_sample_workspace_size(int32_t b, int32_t R, int64_t V,
                                                       size_t* bytes);

/* Temperature speculative-sampling accept (mlx-dspark v0.0.3 release notes,
 * "Highlights": with temperature T > 0 the loop stays lossless, each emitted
 * token an exact sample from the target at T, "via the same acceptance rule
 * as DSpark").  The pages do not write the rule out; this is the standard
 * speculative-sampling rule for this drafter's greedy (one-hot) proposals.
 * For each sequence j, with p_r = softmax(logits[j][r] / T):
 *   draft i, in order, is accepted iff u_accept[j][i] < p_i(draft[j][i])
 *   n    = number of leading accepted drafts
 *   corr = a draw from p_n with draft[j][n] removed (renormalised) if n < D,
 *          a draw from p_D if n = D < R, else -1
 *   emitted / next_tok as in dflash_verify_accept.
 * The draw is argmax_v logits[j][row][v] / T - log(-log u_sample[j][v])
 * (Gumbel-max, decided in fp32, lowest index on ties).  The random numbers
 * are inputs: u_accept [b][D] and u_sample [b][V] fp32 on the device, every
 * value in the open interval (0, 1); values outside it give unspecified
 * tokens.  temperature: finite, > 0.  Accept probabilities are formed in
 * fp32 (max and exp-sum per vocabulary slice, merged in a fixed order).
 * Other arguments, layouts and errors as in dflash_verify_accept; ws holds
 * dflash_verify_sample_workspace_size bytes, zero-filled once (every call
 * leaves its counters zero).  A draft token outside [0, V) has probability 0
 * (rejected). */
DFLASH_API int32_t dflash_verify_accept_sample(const float* logits, const int32_t* draft,
                                               int32_t b, int32_t R, int32_t D, int64_t V,
                                               float temperature, const float* u_accept,
                                               const float* u_sample, int32_t* n_out,
                                               int32_t* corr_out, int32_t* emitted_out,
                                               int32_t* next_tok_out, void* ws,
                                               size_t ws_bytes, void* stream);

/* Commit and draft in one pass: the same results as dflash_kv_commit(w, kv,
 * hid, rows_per_seq, n, ...) followed by dflash_draft_block(w, kv, last_tok,
 * ...) on the same stream (up to fp32 summation order).  The committed rows'
 * K/V projections ride along in each layer's QKV GEMM of the draft, so the
 * K/V weights are read once and the separate K/V launch disappears; the
 * block is drafted against the grown context and len[] is advanced at the
 * end.  Arguments and errors are the union of the two calls'; ws is sized by
 * dflash_workspace_size(cfg, b, rows_per_seq). */
DFLASH_API int32_t dflash_commit_draft_block(const dflash_weights* w, const dflash_kv* kv,
                                             const uint16_t* hid, int32_t rows_per_seq,
                                             const int32_t* n, const int32_t* last_tok,
                                             int32_t* draft_out, float* hidden_out,
                                             float* logits_out, void* ws, size_t ws_bytes,
                                             void* stream);

/* ---------------------------------------------------------------------------
 * Operators on rows of vocabulary logits.  Common to the calls below:
 *  - logits: [rows] of V entries of `dtype` (DFLASH_DTYPE_*), consecutive rows
 *    ld >= V elements apart, the base aligned to an element; nothing is read
 *    between V and ld.  1 <= V < 2^31, 1 <= rows < 2^28.
 *  - An entry that is NaN or -inf is masked: it has probability 0 and is never
 *    returned (the distillation calls instead propagate a NaN).  Every finite
 *    value counts, the type's lowest included; where the largest is +inf, the
 *    entries that are +inf share the probability.
 *  - The order of a row is by descending logit, equal logits by ascending
 *    index (-0 equals +0).
 *  - Results depend on the arguments alone: they repeat bit for bit.
 * Arguments are checked, and errors returned, as for the other calls.
 * ------------------------------------------------------------------------- */

/* Workspace bytes for dflash_sample (0 for up to 64 rows: ws may be NULL). */
DFLASH_API int32_t dflash_sample_workspace_size(int64_t rows, int64_t V, size_t* bytes);

/* One token per row, drawn from softmax(z / T) under the row's filters.  With
 * m = max z and w_v = exp((z_v - m) / T):
 *   top_k keeps the first top_k entries of the order (0 or >= V: all);
 *   top_p keeps, of those, each entry whose predecessors' w sum to less than
 *     top_p times the sum over what top_k kept (the first always; 1: all).
 *     The sums are of fp32 exponentials: an entry within 1e-6 of the whole from
 *     that border may fall on its other side;
 *   min_p keeps, of those, the entries with z_v >= m + T ln(min_p) (0: all);
 *   P(v) = w_v / (sum of the kept w), 0 for the others;
 *   tok = argmax over the kept v of (z_v - m) / T - log(-log u_v), lowest
 *     index on ties (Gumbel maximum: an exact draw from P), formed in 64 bits
 *     where 32 cannot tell entries apart; logprob = ln P(tok).
 * T = 0 takes the first entry of the order (logprob 0), whatever the filters.
 * temperature [rows] fp32; top_k [rows] int32, top_p and min_p [rows] fp32,
 * each nullable (no filter).  T must be 0 or in [1e-6, 1e6], top_k >= 0, top_p
 * and min_p in [0, 1]; a row outside that gets tok -1 and logprob -inf, and
 * sets DFLASH_DEV_BAD_PARAM.  u: uniforms in [0, 1), [rows] of V fp32, ld_u >= V
 * apart; those of entries that are not kept do not matter.  tok_out [rows] int32, logprob_out
 * [rows] fp32 (nullable).  A row without an unmasked entry gets tok -1 and
 * logprob -inf.  ws holds dflash_sample_workspace_size bytes, 16-byte aligned;
 * it needs no zero fill and keeps nothing between calls. */
DFLASH_API int32_t dflash_sample(const void* logits, int32_t dtype, int64_t rows, int64_t V, int64_t ld,
                                 const float* temperature, const int32_t* top_k, const float* top_p,
                                 const float* min_p, const float* u, int64_t ld_u, int32_t* tok_out,
                                 float* logprob_out, void* ws, size_t ws_bytes, void* stream);

/* Workspace bytes for dflash_verify_accept_filtered. */
DFLASH_API int32_t dflash_verify_filtered_workspace_size(int32_t b, int32_t R, int64_t V, size_t* bytes);

/* dflash_verify_accept_sample with each sequence's own temperature, top_k,
 * top_p and min_p (as in dflash_sample, [b] each; a sequence at T = 0 is
 * verified greedily).  With P_r the filtered distribution of row r:
 *   draft i, in order, is accepted iff u_accept[j][i] < P_i(draft[j][i])
 *   n    = number of leading accepted drafts
 *   corr = the draw of dflash_sample at row n without draft[j][n] if n < D,
 *          at row D if n = D < R, else -1 (-1 too where nothing is left)
 *   emitted / next_tok as in dflash_verify_accept.
 * logits: [b][R] rows of V entries, ld apart (sequences R * ld apart).  draft
 * [b][D] int32; an entry outside [0, V) is rejected, so a sequence with fewer
 * drafts pads with -1.  u_accept [b][D] and u_sample ([b] of V entries, ld_u
 * apart) are uniforms in [0, 1).  A sequence with a parameter out of range gets
 * n = -1 (a commit of which appends nothing), corr and next_tok -1, and sets
 * DFLASH_DEV_BAD_PARAM.  ws holds dflash_verify_filtered_workspace_size bytes,
 * 16-byte aligned, zero-filled once (every call leaves its counters zero).  It
 * may be larger, and serve batches of other b, R and D, one call at a time; no
 * other function may write to it in between. */
DFLASH_API int32_t dflash_verify_accept_filtered(const void* logits, int32_t dtype, int64_t ld, const int32_t* draft,
                                                 int32_t b, int32_t R, int32_t D, int64_t V,
                                                 const float* temperature, const int32_t* top_k, const float* top_p,
                                                 const float* min_p, const float* u_accept, const float* u_sample,
                                                 int64_t ld_u, int32_t* n_out, int32_t* corr_out,
                                                 int32_t* emitted_out, int32_t* next_tok_out, void* ws,
                                                 size_t ws_bytes, void* stream);

/* The first K entries of each row's order, 1 <= K <= 1024: val_out [rows][K]
 * fp32 (the logits themselves, falling) and idx_out [rows][K] int32; where a
 * row has fewer unmasked entries the rest is -inf with index -1.  lse_out
 * [rows] fp32 (nullable) = log sum_v exp(z_v / T) over the whole row (-inf when
 * nothing counts), temperature T in [1e-6, 1e6].  A target's rows give the
 * teacher side of dflash_distill_loss.  No workspace. */
DFLASH_API int32_t dflash_top_logits(const void* logits, int32_t dtype, int64_t rows, int64_t V, int64_t ld,
                                     int32_t K, float temperature, float* val_out, int32_t* idx_out, float* lse_out,
                                     void* stream);

/* Distillation of a student's logits from a teacher's top logits.  Per row,
 * with q = softmax(z / T), the teacher's entries t_val[k], t_idx[k] (k < K, S
 * the set of their tokens) and p_k = exp(t_val[k] / T - Lt):
 *   Lt = log sum_k exp(t_val[k] / T) when t_lse is null, else t_lse[row], the
 *     log-sum-exp of the teacher's whole row at this T; then the tokens outside
 *     S count as one entry with p_r = max(0, 1 - sum_k p_k) and q_r = their sum
 *     of q (without t_lse: p_r = 0).  Where q_r is below 2^-126 (S holds every
 *     token, or the student masks the others) a p_r up to 2^-20 (1 + |t_lse|),
 *     which the rounding of t_lse explains, counts as 0
 *   loss = weight * [sum_k p_k (ln p_k - ln q_{t_idx[k]}) + p_r (ln p_r - ln q_r)]
 *   dlogits[j] = weight / T * (P q_j - p_j) for j in S, and
 *                weight / T * q_j (P - p_r / q_r) outside, P = sum_k p_k + p_r
 * t_val [rows][K] fp32 (finite or -inf), t_idx [rows][K] int32, 1 <= K <= 1024;
 * an entry with index -1 is no entry.  t_lse [rows] (nullable), weight [rows]
 * (nullable: 1) and loss_out [rows] are fp32.  V <= 2^23; T in [1e-6, 1e6].
 *  - dlogits (nullable): [rows] of V entries of `dtype`, ldd >= V apart, all V
 *    written; it may be the logits' own buffer with ldd = ld (else the two must
 *    not overlap).
 *  - stats_out (nullable): [rows][4] fp32, 16-byte aligned, what
 *    dflash_distill_backward needs.
 *  - A row with weight 0, or whose teacher lists nothing above -inf, is left
 *    out: loss 0, gradient 0, its student logits do not matter.
 *  - A row with an index listed twice, or outside [-1, V), is refused: loss
 *    NaN, gradient 0, DFLASH_DEV_BAD_TOKEN set.  So is one that is not left out
 *    and has a listed t_val that is NaN or +inf, or a t_lse that is not finite
 *    (of a teacher's row with a +inf logit, say) or so far below a t_val / T that
 *    p_k > 256: DFLASH_DEV_BAD_PARAM set.  (In fp32 t_lse is off by up to 2^-24 of
 *    its size, which p_k shows: teacher logits far from 0 are better shifted.)
 *  - A student row without a logit above -inf has no distribution: loss NaN,
 *    gradient undefined.  The loss is +inf where a p_k or p_r above 0 meets a q
 *    below fp32's range of logarithms (a -inf logit, or one 3e38 T below the others).
 * No workspace. */
DFLASH_API int32_t dflash_distill_loss(const void* logits, int32_t dtype, int64_t rows, int64_t V, int64_t ld,
                                       const float* t_val, const int32_t* t_idx, int32_t K, const float* t_lse,
                                       float temperature, const float* weight, float* loss_out, float* stats_out,
                                       void* dlogits, int64_t ldd, void* stream);

/* The gradient of the unweighted loss for a given upstream gradient:
 * dlogits = grad_loss[row] * dloss/dlogits, with stats [rows][4] of a
 * dflash_distill_loss call on the same logits, teacher entries and T.
 * grad_loss: [rows] fp32 (0: a zero row).  A row that call left out or refused
 * stays so.  The rest as in that call. */
DFLASH_API int32_t dflash_distill_backward(const void* logits, int32_t dtype, int64_t rows, int64_t V, int64_t ld,
                                           const float* t_val, const int32_t* t_idx, int32_t K, const float* t_lse,
                                           float temperature, const float* stats, const float* grad_loss,
                                           void* dlogits, int64_t ldd, void* stream);

/* What a request's history, biases and grammar do to its rows of logits, before
 * a token is drawn from them (dflash_sample, dflash_verify_accept_filtered) or
 * they are read otherwise.  Sequence j's row r, of R a sequence, is row j R + r.
 * With c_v the generated tokens that equal v (those of the history and those
 * among the row's own drafts):
 *   x = z_v
 *   v in the prompt or c_v > 0:  x = x > 0 ? x / repetition : x * repetition
 *   x = x - frequency * c_v - (c_v > 0 ? presence : 0)
 *   x = x + the sum of v's biases;   where the grammar does not allow v: -inf
 * formed in fp32 and rounded once to `dtype` (to an infinity beyond its range).
 * Entries that nothing changes are copied; a NaN stays one unless disallowed.
 *  - out: rows ld_out >= V apart; it may be the logits' own buffer with
 *    ld_out = ld (else the two must not overlap).  Only V entries a row are
 *    written.  b * R < 2^28, R <= 256.
 *  - hist (nullable): [b] rows of up to H tokens, ld_hist apart; of sequence j
 *    the first n_prompt[j] (nullable: 0) are the prompt, those up to n_hist[j]
 *    were generated.  0 <= n_prompt <= n_hist <= H < 2^20 - 256.
 *  - draft (nullable): [b][D] tokens, D <= 256, that the rows verify, and path
 *    (nullable): [b][R][(D + 31) / 32] bits, which of them come before row r's
 *    token (of a tree: the masks of dflash_tree_mask, D = R).  Without path row
 *    r follows drafts 0 to r - 1.  They count beside the history, so a token
 *    that is in it already (a tree's root) is given as -1 in one of the two.
 *  - repetition, frequency, presence (each nullable: 1, 0, 0): [b] fp32,
 *    repetition finite and > 0, the others finite.
 *  - bias_idx, bias_val (both or neither): [b][K], K <= 512; a token listed
 *    again adds up in the list's order; a value is finite or -inf.
 *  - allow (nullable): n_allow rows of bits, ld_allow >= (V + 31) / 32 words
 *    apart, bit v % 32 of word v / 32 set where v is allowed; allow_row
 *    (nullable: the row's own number) [b][R] names each row's, -1: no grammar.
 *  - A token outside [0, V) in hist, draft or bias_idx is no token.
 *  - A sequence with a parameter out of range gets rows of NaN, which the calls
 *    on rows take as masked, and sets DFLASH_DEV_BAD_PARAM (a length:
 *    DFLASH_DEV_BAD_LENGTH); so does a row whose allow_row is out of range.
 * No workspace. */
DFLASH_API int32_t dflash_adjust_logits(const void* logits, int32_t dtype, int64_t b, int32_t R, int64_t V, int64_t ld,
                                        void* out, int64_t ld_out, const int32_t* hist, int64_t ld_hist, int32_t H,
                                        const int32_t* n_hist, const int32_t* n_prompt, const int32_t* draft,
                                        int32_t D, const uint32_t* path, const float* repetition,
                                        const float* frequency, const float* presence, const int32_t* bias_idx,
                                        const float* bias_val, int32_t K, const uint32_t* allow, int64_t n_allow,
                                        int64_t ld_allow, const int32_t* allow_row, void* stream);

/* ---------------------------------------------------------------------------
 * A tree of drafts: several continuations verified in one target pass.  Common
 * to the calls below:
 *  - A sequence's tree has up to N nodes, 1 <= N <= 256, of which it uses the
 *    first n_nodes[j] (nullable: all N; 0 <= n_nodes <= N, else it has none and
 *    DFLASH_DEV_BAD_LENGTH is set).  What belongs to other nodes does not matter,
 *    whatever its bits, and is not written in outputs, unless a call says so.
 *  - parent: [b][N] int32, parent[i] in [-1, i), -1 for a root.  Node 0 is where
 *    the walk begins: the last emitted token, whose keys and values are not in
 *    the cache yet (as slot 0 of a draft block).
 *  - b <= 65535.
 * One block of a target: dflash_tree_mask; in each layer dflash_tree_attention;
 * on the nodes' logits dflash_adjust_logits and dflash_sample (or
 * dflash_lmhead_argmax); dflash_tree_accept; dflash_tree_commit.
 * ------------------------------------------------------------------------- */

/* mask [b][N][(N + 31) / 32]: bit t % 32 of word t / 32 of node i's row is set
 * where t is i or one of its ancestors; depth_out (nullable) [b][N] int32: the
 * number of ancestors, so node i's position is len + depth.  Nodes that are not
 * there get no bits and depth -1; so do one whose parent is out of range and
 * all that hang from it (DFLASH_DEV_BAD_TREE). */
DFLASH_API int32_t dflash_tree_mask(const int32_t* parent, const int32_t* n_nodes, int32_t b, int32_t N,
                                    uint32_t* mask, int32_t* depth_out, void* stream);

/* Workspace bytes for dflash_tree_attention. */
DFLASH_API int32_t dflash_tree_attention_workspace_size(int32_t b, int32_t N, int32_t nq, int32_t nkv, int32_t d,
                                                        size_t* bytes);

/* Attention of a tree's nodes over a cache and one another.  For node i and head
 * h of sequence j, over the len[j] cached keys of kv head h nkv / nq and the
 * nodes that mask has for i:
 *   o = sum_t exp(s_t) v_t / sum_t exp(s_t),  s_t = scale q . k_t
 *   lse = ln sum_t exp(s_t)
 * in fp32 (probabilities enter the product with v rounded to dtype); a node that
 * sees no key gets o = 0, lse = -inf.  Values of keys that a node does not see
 * do not matter to it, infinities and NaN included.
 *  - kv: the cache of any model, k and v [layers][b][nkv][cap][d] of `dtype`
 *    (DFLASH_DTYPE_F16 or _BF16, as all tensors here); `layer` is read at len.
 *  - q: node i of sequence j at j q_seq + i q_tok elements, its nq heads of d
 *    side by side; k_tree, v_tree likewise, nkv heads, at j t_seq + i t_tok (so
 *    all three may lie in one projection's output).  16-byte aligned, strides
 *    multiples of 8 elements.  Any order will do, but above 16 rows (N nq / nkv)
 *    others than t_seq >= t_tok >= nkv d read the cache again for every 32 rows
 *    (256 rows over 4 x 16384 keys, 8 kv heads of 128: 480 us in place of 74).
 *  - mask: as of dflash_tree_mask, any bits (of nodes that are not there they
 *    count for nothing); null: node i sees nodes 0 to i, a chain (N = 1: one
 *    token's step).
 *  - out [b][N][nq][d] of dtype, lse_out (nullable) [b][N][nq] fp32.
 *  - d is 64 or 128, nq a multiple of nkv (1024 times at most), scale finite and
 *    > 0.
 * A len[j] outside [0, cap] leaves the sequence out (DFLASH_DEV_BAD_LENGTH).  ws
 * holds dflash_tree_attention_workspace_size bytes, 16-byte aligned; it needs no
 * zero fill and keeps nothing between calls. */
DFLASH_API int32_t dflash_tree_attention(const void* q, int64_t q_seq, int64_t q_tok, int32_t dtype,
                                         const dflash_kv* kv, int32_t layer, int32_t N, int32_t nq, int32_t nkv,
                                         int32_t d, const void* k_tree, const void* v_tree, int64_t t_seq,
                                         int64_t t_tok, const uint32_t* mask, const int32_t* n_nodes, float scale,
                                         void* out, float* lse_out, void* ws, size_t ws_bytes, void* stream);

/* The path that the target accepts.  tok [b][N]: the target's token at each node
 * (its argmax, or a draw: each emitted token is then an exact sample, because the
 * walk only asks which of a node's children the drawn token is); tree_tok
 * [b][N]: the nodes' own tokens.  From node 0, while a child's token is the
 * target's token at the node (the first such child) and the path has less than R
 * nodes, the walk steps to that child.
 *   path_out [b][R]: the walk's nodes, then -1;  n_out [b]: its steps (accepted
 *     drafts; -1 for a sequence without nodes)
 *   corr_out [b]: the target's token at the last node (-1: none)
 *   emitted_out (nullable) [b][R]: the accepted drafts' tokens, then corr, then -1
 *   next_tok_out (nullable) [b]: corr; where that is -1 the last node's token.
 * 1 <= R <= N.  A tok below 0 equals no child's.  A node whose parent is out of
 * range is no child (DFLASH_DEV_BAD_TREE). */
DFLASH_API int32_t dflash_tree_accept(const int32_t* tok, const int32_t* tree_tok, const int32_t* parent,
                                      const int32_t* n_nodes, int32_t b, int32_t N, int32_t R, int32_t* n_out,
                                      int32_t* corr_out, int32_t* path_out, int32_t* emitted_out,
                                      int32_t* next_tok_out, void* stream);

/* Workspace bytes for dflash_tree_commit. */
DFLASH_API int32_t dflash_tree_commit_workspace_size(int32_t b, size_t* bytes);

/* Commit of an accepted path to the cache.  Of sequence j the nodes
 * path[j][0..n[j]] (n + 1 of them, none for n = -1; n, path as of
 * dflash_tree_accept) become rows len[j] + i of all L layers of kv, and its length
 * grows by as many; hid (nullable): [b][N] rows of hid_cols 16-bit elements, whose
 * nodes of the path become rows i of hid_out [b][R] (for dflash_kv_commit, which
 * takes n too).
 *  - k_tree, v_tree: layer l, sequence j, node i at l t_layer + j t_seq + i t_tok
 *    elements (16 bits each), nkv heads of d side by side; 16-byte aligned,
 *    strides, d and hid_cols multiples of 8.
 *  - len_out (nullable: kv->len itself) [b]: the new lengths.
 *  - A sequence that would pass cap, whose n is outside [-1, R) or len below 0, or
 *    whose path has a node outside [0, N) is left as it is, hidden rows included,
 *    and sets DFLASH_DEV_KV_CAPACITY, _BAD_LENGTH or _BAD_TREE.
 * ws holds dflash_tree_commit_workspace_size bytes, zero-filled once (every call
 * leaves them zero). */
DFLASH_API int32_t dflash_tree_commit(const dflash_kv* kv, int32_t L, int32_t nkv, int32_t d, int32_t N,
                                      const void* k_tree, const void* v_tree, int64_t t_layer, int64_t t_seq,
                                      int64_t t_tok, const int32_t* path, const int32_t* n, int32_t R,
                                      const uint16_t* hid, int64_t hid_cols, uint16_t* hid_out, int32_t* len_out,
                                      void* ws, size_t ws_bytes, void* stream);

/* Draft-KV commit with rollback of the rejected suffix (mlx-dspark v0.0.3,
 * "Notes": KV rollback; dflash-mlx "What It Does": conditioning on target
 * hidden states).  hid: [b][rows_per_seq][k*H] fp16 target hidden rows of the
 * verified block; n: [b] int32 (device) accept lengths, n[j] in [-1, B].
 * For each sequence j, rows r < c_j = min(n[j] + 1, rows_per_seq):
 *   c = RMSNorm(W8(fc) hid[j][r]; gamma_hid)
 *   per layer l: K = RoPE(per-head RMSNorm(W8(Wk_l) c; gamma_k[l]),
 *                         pos = len[j] + r),  V = W8(Wv_l) c
 *   written at cache row len[j] + r;  then len[j] += c_j.
 * Rows r >= c_j are never written.  A sequence whose len[j] + c_j would pass
 * `cap` is skipped whole and flags DFLASH_DEV_KV_CAPACITY.  rows_per_seq in
 * [1, 256] with b * rows_per_seq <= 4096. */
DFLASH_API int32_t dflash_kv_commit(const dflash_weights* w, const dflash_kv* kv,
                         const uint16_t* hid, int32_t rows_per_seq,
                         const int32_t* n, void* ws, size_t ws_bytes,
                         void* stream);

/* Launch modes (dflash_set_launch_mode).
 *  DFLASH_LAUNCH_STREAM_ORDER (the default): every kernel starts after the
 *    previous work of its stream has finished.  Correct whatever else runs
 *    on the GPU at the same time.
 *  DFLASH_LAUNCH_EARLY: every kernel is launched as a programmatic dependent
 *    of the previous kernel of its stream and lets its own dependents launch
 *    early, so each kernel's weight copies start while the previous kernel
 *    finishes (about 10 % shorter draft steps on a dedicated GPU).  Only for
 *    callers that own the GPU and issue the library's calls from one stream:
 *    on GB300 (driver 580), early-launched kernels gave wrong results, now
 *    and then, while other kernels (the library's on another stream, or any
 *    other work) ran on the same GPU. */
#define DFLASH_LAUNCH_STREAM_ORDER 0
#define DFLASH_LAUNCH_EARLY 1

/* Sets the launch mode of every later call in this process (all devices,
 * all threads).  A CUDA graph keeps the mode its kernels were captured with.
 * DFLASH_EINVAL for an unknown mode.  No page describes this; it is a
 * property of this library's kernels. */
DFLASH_API int32_t dflash_set_launch_mode(int32_t mode);

/* The current launch mode. */
DFLASH_API int32_t dflash_get_launch_mode(void);

/* Reads (and, when clear != 0, resets) the device status word of the current
 * device into *host_status.  Synchronises the device. */
DFLASH_API int32_t dflash_get_status(int32_t* host_status, int32_t clear);

#ifdef __cplusplus
}
#endif
#endif /* DFLASH_H */
