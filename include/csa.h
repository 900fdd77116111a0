/*
 * csa.h -- C ABI of the B200 (sm_100a) CSA / HCA compressed-attention operator.
 *
 * One attention layer of DeepSeek-V4's hybrid attention, as the explainer
 * pages describe it:
 *
 *   CSA ("compressed sparse attention"): every m consecutive raw KV rows are
 *   pooled into one compressed entry with learned per-channel gate logits and
 *   positional biases over an overlapping 2m-row window; a lightning indexer
 *   scores the causally complete entries against the query; the top-k
 *   entries plus a sliding window of the w most recent raw rows are attended
 *   by shared-KV multi-query attention with a per-head sink logit, RMSNorm on
 *   queries and entries, rotary embedding on the last 64 dims only, and the
 *   inverse rotation applied to the output.
 *     - "DeepSeek-V4: Making a Million Tokens Affordable", section "Two ways
 *       to shrink attention, interleaved" (m=4, top-k=1024, overlap 2m, sink,
 *       RMSNorm, partial RoPE, inverse RoPE on the output, 128-token window).
 *     - "DeepSeek-V4 Explained: Compressed Sparse Attention and 1M Context at
 *       10% KV", section "The attention stack, and why it is two mechanisms"
 *       (compression weights and positional biases, lightning indexer,
 *       shared-KV multi-query layout, BF16 rotary dims + FP8 remainder).
 *   HCA ("heavily compressed attention"): the same path with m'=128, no
 *   overlap, no indexer and dense attention over every visible entry.
 *     - same page, same section (m' = 128, and attention dense over all the
 *       remaining entries).
 *
 * The pages give no formula for the indexer or the gate and no storage
 * layout; the definitions this library implements are stated at each call.
 *
 * Conventions (every call):
 *   - Returns csa_status_t; CSA_OK = 0.  Argument errors are detected on the
 *     host, before any launch, and leave all buffers untouched;
 *     csa_last_error() then describes the failure (thread-local string).
 *   - Every pointer is a DEVICE pointer owned by the caller, 16-byte aligned,
 *     unless marked "host".  The library allocates nothing on the hot calls.
 *   - Calls are asynchronous on the given CUDA stream (a cudaStream_t passed
 *     as void*; NULL = legacy default stream).  Device-side faults surface at
 *     the caller's next synchronisation.  Kernels contain only bounded waits:
 *     a wait that gives up sets a bit in the workspace's device error word,
 *     read back by csa_device_error().
 *   - Workspace: csa_workspace_size() bytes of device memory, zero-filled by
 *     the caller before its FIRST use (the library leaves its counters and
 *     histograms at zero after every call but the paged cache's, whose
 *     workspace is its own; zero it again after a device error).  Concurrent calls must not share a workspace.
 *   - Positions: q_pos[b * Tq + j] (device int64) is the absolute position t
 *     of query token j of sequence b; raw row index r = t - pos0.
 *
 * Stored-row formats (kv_format), one row = one compressed entry or one
 * window row, row_bytes = csa_row_bytes():
 *   CSA_FMT_F32   D float32.
 *   CSA_FMT_BF16  D bfloat16.
 *   CSA_FMT_MIXED D+80 bytes: FP8-e4m3 codes of dims [0, D-64) at byte 0,
 *                 bfloat16 of the 64 rotary dims at byte D-64, float32 scale
 *                 sigma at byte D+64, zero padding.  value = code * sigma for
 *                 the FP8 part; sigma is the smallest power of two with
 *                 max|x| / sigma <= 448 (1 for an all-zero part), codes are
 *                 round-to-nearest-even with saturation.
 *
 * Index-key formats (idx_format), one key of d_I dims per entry:
 *   CSA_FMT_F32   d_I float32, idx_key_scale all 1.
 *   CSA_FMT_E4M3  d_I e4m3 codes; idx_key_scale[i] = the key's power-of-two scale.
 *   CSA_FMT_E2M1  d_I / 2 bytes of FP4 e2m1 codes (1 sign, 2 exponent bits with bias 1, 1 mantissa
 *                 bit; magnitudes 0, .5, 1, 1.5, 2, 3, 4, 6), two per byte with the even dim in the
 *                 low nibble; idx_key_scale[i] holds a uint32 scale word (stored in the float
 *                 array's 4 bytes): bits 0..7 = e + 127 for the key scale sigma = 2^e, bits
 *                 8+4b..11+4b = the offset delta_b (0..7) of dims [32b, 32b+32); the value of dim d
 *                 is code * sigma * 2^-delta_b.  d_I a multiple of 32.  Index queries stay e4m3.
 *                 ("DeepSeek-V4: Making a Million Tokens Affordable", "Two ways to shrink
 *                 attention, interleaved": the indexer's attention runs in FP4.)
 *
 * Rotary convention: interleaved pairs (D-64+2u, D-64+2u+1), u < 32, angle
 * pos * base^(-2u/64) formed and reduced in float64.
 */
#ifndef CSA_B200_CSA_H_
#define CSA_B200_CSA_H_

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define CSA_API __attribute__((visibility("default")))
#else
#define CSA_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum csa_status {
  CSA_OK = 0,
  CSA_ERR_INVALID_ARG = 1,     /* bad pointer, size, alignment or layer field */
  CSA_ERR_UNSUPPORTED = 2,     /* valid, but no kernel for this shape / format */
  CSA_ERR_WORKSPACE = 3,       /* workspace missing or smaller than csa_workspace_size() */
  CSA_ERR_CUDA = 4,            /* a CUDA runtime call failed (message in csa_last_error) */
  CSA_ERR_DEVICE_TIMEOUT = 5,  /* a kernel set bit 1 or 2 of a device error word (csa_device_error) */
  CSA_ERR_DEVICE_PAGE = 6      /* bit 4 alone was set: a paged-cache call left something out */
} csa_status_t;

enum {
  CSA_FMT_F32 = 0,
  CSA_FMT_BF16 = 1,
  CSA_FMT_MIXED = 2,           /* kv_format only */
  CSA_FMT_E4M3 = 3,            /* idx_format only */
  CSA_FMT_E2M1 = 4             /* idx_format only: FP4 index keys, e4m3 index queries (see below) */
};

enum { CSA_KIND_CSA = 0, CSA_KIND_HCA = 1 };

/* One layer's hyper-parameters. */
typedef struct csa_layer {
  int32_t kind;          /* CSA_KIND_CSA or CSA_KIND_HCA */
  int32_t B;             /* sequences */
  int32_t H;             /* query heads (all share the one KV head) */
  int32_t D;             /* KV / head dim; the last d_rope dims are rotary */
  int32_t d_rope;        /* must be 64 */
  int32_t m;             /* raw rows per compressed entry (4 for CSA, 128 for HCA) */
  int32_t overlap;       /* 1: entry i pools raw rows [(i-1)m, (i+1)m); 0: [im, (i+1)m) */
  int32_t top_k;         /* CSA: entries kept per query; ignored for HCA */
  int32_t window;        /* w: most recent raw rows attended uncompressed (incl. current) */
  int32_t H_I;           /* CSA: indexer heads */
  int32_t d_I;           /* CSA: indexer head dim */
  int32_t kv_format;     /* CSA_FMT_F32 | CSA_FMT_BF16 | CSA_FMT_MIXED */
  int32_t idx_format;    /* CSA_FMT_F32 | CSA_FMT_E4M3 | CSA_FMT_E2M1 (index keys; queries e4m3 for E2M1) */
  int32_t act_format;    /* CSA_FMT_F32 | CSA_FMT_BF16: queries, raw rows, gate logits, output */
  double rope_base;      /* rotary base (10000) */
  float eps;             /* RMSNorm epsilon (1e-6) */
  float softmax_scale;   /* logit scale; 0 selects 1/sqrt(D) */
  int64_t pos0;          /* absolute position of raw row 0 */
} csa_layer_t;

/* Per-layer caches (state carried across decode steps; caller-owned). */
typedef struct csa_cache {
  void* entries;          /* [B][entry_cap][row_bytes] compressed entries, entry i at slot i */
  int64_t entry_cap;      /* capacity in entries per sequence */
  void* idx_keys;         /* CSA: [B][entry_cap][d_I] index keys (e4m3 codes or float32) */
  const float* idx_key_scale; /* CSA: [B][entry_cap] per-key scale (all 1 for float32 keys) */
  void* window;           /* [B][window_cap][row_bytes]: raw row r's rotated row at slot r mod window_cap */
  int64_t window_cap;     /* >= window; >= Tq + window - 1 for a Tq-token chunk */
  void* raw;              /* [B][raw_cap][D] un-rotated raw rows (act_format); row r at slot (r - raw_base) mod raw_cap */
  void* gate;             /* [B][raw_cap][D] gate logits, same indexing as raw */
  int64_t raw_cap;        /* decode: >= (1+overlap)*m; prefill: the chunk plus overlap*m look-back rows */
  int64_t raw_base;       /* raw row stored at slot 0 (0 for a ring) */
} csa_cache_t;

/* Learned per-layer parameters. */
typedef struct csa_params {
  const float* pos_bias;  /* [(1+overlap)*m][D] positional bias per window slot and channel */
  const float* gamma_kv;  /* [D] RMSNorm weight of compressed entries, or NULL (= 1) */
  const float* gamma_q;   /* [D] RMSNorm weight of queries, or NULL (= 1) */
  const float* sinks;     /* [H] per-head sink logits */
} csa_params_t;

/* Operation selector for csa_workspace_size(). */
enum {
  CSA_OP_INDEX_TOPK = 0,
  CSA_OP_SPARSE_ATTEND = 1,
  CSA_OP_HCA_ATTEND = 2,
  CSA_OP_DECODE_STEP = 3,   /* csa_decode_step / hca_decode_step */
  CSA_OP_PREFILL = 4,       /* csa_prefill */
  CSA_OP_DECODE_STEP_INDEXED = 5  /* csa_decode_step_indexed */
};

/* Index-key stream of a CSA layer: per token one index row and one row of gate logits of d_I
 * values (act_format), kept in rings with the same slots as cache->raw / cache->gate
 * (row r at slot (r - raw_base) mod raw_cap), and the slot biases of their compression. */
typedef struct csa_index_stream {
  void* raw;              /* [B][raw_cap][d_I] index rows */
  void* gate;             /* [B][raw_cap][d_I] gate logits */
  const float* pos_bias;  /* [(1+overlap)*m][d_I] positional bias per window slot and channel */
} csa_index_stream_t;

/* Bytes of one stored row for the layer's kv_format (host). */
CSA_API size_t csa_row_bytes(const csa_layer_t* L);

/* Workspace bytes an operation needs for Tq queries per sequence and caches
 * of entry_cap entries (host; 0 if the layer is invalid). */
CSA_API size_t csa_workspace_size(const csa_layer_t* L, int32_t op, int32_t Tq, int64_t entry_cap);

/* Thread-local text of the last error returned on this thread (host). */
CSA_API const char* csa_last_error(void);

/* Library version string (host). */
CSA_API const char* csa_version(void);

/* Reads and clears the device error words (synchronises the stream): the
 * workspace's word (workspace may be NULL: then it is skipped) and the
 * library's own word on the current device, where the kernels of the calls
 * that take no workspace (csa_append, csa_compress) report.  With workspace
 * NULL also the device's word of the paged-cache calls that take none; a
 * call with a workspace leaves that one to whoever made those calls.  *code
 * gets the OR of the bits kernels set (0 = none):
 *   1  a bounded wait (mbarrier / tensor-memory pipeline / cluster
 *      reduction) gave up; the results of that launch are incomplete;
 *   2  the multi-CTA top-k found its score histogram inconsistent with the
 *      scores; that row's top-k output is incomplete (padded with -1);
 *   4  a paged-cache call met an index out of range or a token without a page
 *      of its own and left it out (see the paged cache below).
 * Returns CSA_ERR_DEVICE_TIMEOUT if bit 1 or 2 was set, CSA_ERR_DEVICE_PAGE
 * if bit 4 was set alone. */
CSA_API csa_status_t csa_device_error(void* workspace, size_t ws_bytes, void* stream, int32_t* code);

/* Test and diagnostic aids (no counterpart on the pages). */

/* Workspace segments, for csa_debug_workspace_segment. */
enum {
  CSA_SEG_ERROR_WORD = 0,      /* the int32 device error word */
  CSA_SEG_SCORES = 1,          /* indexer scores [rows][entry_cap] float32 */
  CSA_SEG_TOPK_HISTOGRAM = 2,  /* multi-CTA top-k: [rows][4096] uint32 score histogram, then
                                  [rows][4] counters, then [rows][4096] second histogram */
  CSA_SEG_TOPK = 3,            /* top-k indices of the fused calls [rows][top_k] int32 */
  CSA_SEG_PARTIALS = 4,        /* attention partials */
  CSA_SEG_INDEX_QUERY = 5,     /* csa_decode_step_indexed: the produced index query [B][H_I][d_I] */
  CSA_SEG_INDEX_QUERY_SCALE = 6  /* ... and its per-head scales [B][H_I] float32 */
};

/* Byte offset and size of one segment of the workspace that
 * csa_workspace_size(L, op, Tq, entry_cap) describes (host; *bytes = 0 when
 * the operation has no such segment).  Lets a test inject state (e.g. an
 * inconsistent score histogram) into a caller-owned workspace. */
CSA_API csa_status_t csa_debug_workspace_segment(const csa_layer_t* L, int32_t op, int32_t Tq, int64_t entry_cap,
                                                 int32_t segment, size_t* offset, size_t* bytes);

/* Launches one CTA that waits, with the library's bounded wait and a limit
 * of limit_ns nanoseconds (0 < limit_ns <= 1e9), on an mbarrier phase that
 * nothing completes; when the limit passes it sets bit 1 of the workspace's
 * error word and returns.  Nothing is in flight in the CTA when it gives up,
 * so the context stays usable.  Lets a test drive the failure-reporting path
 * (csa_device_error -> CSA_ERR_DEVICE_TIMEOUT) without a device fault. */
CSA_API csa_status_t csa_debug_wait_probe(void* workspace, size_t ws_bytes, uint64_t limit_ns, void* stream);

/* Profiling aid (no counterpart on the pages).  When ev_start and ev_stop (cudaEvent_t handles
 * created with timing enabled) are both non-NULL, every later call made from this host thread
 * records ev_start immediately before and ev_stop immediately after the launch of the indexer
 * score kernel (the dominant kernel of a CSA decode step), with the external-record flag so the
 * records become event nodes when the stream is being captured into a CUDA graph.  NULL, NULL
 * turns it off.  Host only; never fails. */
CSA_API void csa_profile_events(void* ev_start, void* ev_stop);

/* Profiling aid (no counterpart on the pages).  Arms a timeline on this host thread: later
 * calls record events[0], events[1], ... (cudaEvent_t handles with timing enabled), one just
 * before each kernel launch or memset they issue, until `capacity` events are used; the records
 * use the external flag, so they become event nodes under stream capture.  The caller records
 * one more event after the last call to close the last interval.  NULL disarms it. */
CSA_API void csa_profile_timeline(void** events, int32_t capacity);

/* Events of the armed timeline used so far. */
CSA_API int32_t csa_profile_timeline_count(void);

/* Number of kernels this process has launched through the library so far (host counter). */
CSA_API uint64_t csa_launch_count(void);

/* Append Tq new tokens per sequence: raw rows x_new[b][j] (and gate rows
 * g_new) are written into the raw / gate rings at slot (r - raw_base) mod
 * raw_cap (skipped when x_new is NULL: the rows are then already in the raw
 * buffer), and each token's window row RoPE_t(x) -- rotated at its own
 * position, not normalised -- is stored at window slot r mod window_cap.
 *   x_new, g_new: [B][Tq][D] act_format, or both NULL.
 * The sliding window is the pages' short branch over the most recent tokens,
 * kept uncompressed ("DeepSeek-V4 Explained: ...", "The attention stack, and
 * why it is two mechanisms"). */
CSA_API csa_status_t csa_append(const csa_layer_t* L, const csa_cache_t* cache,
                        const void* x_new, const void* g_new,
                        const int64_t* q_pos, int32_t Tq, void* stream);

/* Compress every entry completed by the Tq tokens at q_pos (entry i is
 * completed by raw row (i+1)m - 1).  Entry i = RoPE_{pos0 + i m}(RMSNorm(e) *
 * gamma_kv) with e_c = sum_r softmax_r(gate[r][c] + pos_bias[r - (i-ov)m][c])
 * * raw[r][c] over raw rows r in [(i-ov)m, (i+1)m) clipped at 0, written to
 * entries[b][i] in kv_format.  The raw buffer must hold those rows.
 * Pages: each group of m consecutive tokens becomes one entry, pooled with
 * learned weights and per-slot position biases ("DeepSeek-V4 Explained: ...");
 * an entry reads 2m source rows, yet the sequence still shrinks m-fold
 * ("DeepSeek-V4: Making a Million Tokens Affordable", "Two ways to shrink
 * attention"). */
CSA_API csa_status_t csa_compress(const csa_layer_t* L, const csa_cache_t* cache,
                          const csa_params_t* P, const int64_t* q_pos, int32_t Tq,
                          void* stream);

/* Lightning indexer + top-k (CSA).  For query (b, j) at position t, entry i
 * is visible iff pos0 + (i+1)m - 1 <= t; its score is
 *   s_i = sum_h head_w[h] * max(0, idx_q_scale[h] * idx_key_scale[i] * <idx_q[h], idx_key[i]>)
 * and the k highest scores are kept, ties to the smaller index, written in
 * ascending entry order to topk_idx[b][j][0..k), padded with -1 when fewer
 * than k entries are visible.
 *   idx_q:       [B][Tq][H_I][d_I] e4m3 codes or float32
 *   idx_q_scale: [B][Tq][H_I] float32;  head_w: [B][Tq][H_I] float32
 *   n_max:       entries scored per query (<= entry_cap; entries beyond the
 *                query's visible count are excluded)
 *   topk_idx:    [B][Tq][top_k] int32 (output)
 *   scores:      [B][Tq][n_max] float32 (output, optional: NULL keeps them in the workspace)
 * Pages: a cheap low-rank indexer scores the compressed entries and each query
 * attends only to its k best ("DeepSeek-V4 Explained"); the indexer uses a
 * few small FP8 heads ("DeepSeek-V4, explained.", step 3). */
CSA_API csa_status_t csa_index_topk(const csa_layer_t* L, const csa_cache_t* cache,
                            const void* idx_q, const float* idx_q_scale, const float* head_w,
                            const int64_t* q_pos, int32_t Tq, int64_t n_max,
                            int32_t* topk_idx, float* scores,
                            void* workspace, size_t ws_bytes, void* stream);

/* Sparse shared-KV multi-query attention (CSA).  For query (b, j) at t:
 *   q~_h = RoPE_t(RMSNorm(q_h) * gamma_q);   keys = values = the selected
 *   entries topk_idx[b][j][*] (-1 skipped) plus the window rows r in
 *   [max(0, r_t - w + 1), r_t];  l_j = <q~_h, k_j> * softmax_scale;
 *   o_h = sum_j e^{l_j} k_j / (e^{sink_h} + sum_j e^{l_j});  out = RoPE_{-t}(o_h).
 *   q:   [B][Tq][H][D] act_format;  out: [B][Tq][H][D] act_format.
 * Pages: an entry is both key and value, the output is rotated back by the
 * query's position, and each head has a learned sink ("DeepSeek-V4: Making a
 * Million Tokens Affordable"). */
CSA_API csa_status_t csa_sparse_attend(const csa_layer_t* L, const csa_cache_t* cache,
                               const csa_params_t* P, const void* q, const int64_t* q_pos,
                               int32_t Tq, const int32_t* topk_idx, void* out,
                               void* workspace, size_t ws_bytes, void* stream);

/* Dense attention over every visible entry i < n_visible(t) (HCA) plus the
 * window rows, otherwise as csa_sparse_attend.  n_max bounds the visible
 * entries (<= entry_cap).
 * Pages: after the heavy compression, attention stays dense, without an
 * indexer or a top-k ("DeepSeek-V4: Making a Million Tokens Affordable"). */
CSA_API csa_status_t hca_attend(const csa_layer_t* L, const csa_cache_t* cache,
                        const csa_params_t* P, const void* q, const int64_t* q_pos,
                        int32_t Tq, int64_t n_max, void* out,
                        void* workspace, size_t ws_bytes, void* stream);

/* One fused CSA decode step for token t = q_pos[b] of every sequence:
 * csa_append (x_new, g_new) -> csa_compress (when t completes a group) ->
 * csa_index_topk over entry_cap entries -> csa_sparse_attend.  Tq = 1.
 * topk_idx: [B][top_k] int32 output, or NULL (kept in the workspace).
 * The index keys are inputs, so append+compress does not feed the indexer:
 * the library runs it on an internal second stream (one per thread and
 * device, created by the first call made outside stream capture), forked
 * from and joined back into `stream` before attention.  Ordering with
 * respect to `stream` is unchanged, and the pattern is graph-capturable. */
CSA_API csa_status_t csa_decode_step(const csa_layer_t* L, const csa_cache_t* cache,
                             const csa_params_t* P, const void* q,
                             const void* idx_q, const float* idx_q_scale, const float* head_w,
                             const void* x_new, const void* g_new, const int64_t* q_pos,
                             void* out, int32_t* topk_idx,
                             void* workspace, size_t ws_bytes, void* stream);

/* Index keys produced from the index-key stream.  Appends the Tq tokens' index rows x_new / g_new
 * ([B][Tq][d_I] act_format; both NULL when the rows are already in S->raw / S->gate) to the stream's
 * rings, then writes the key of every entry the tokens complete: the entry's window rows
 * [(i-ov)m, (i+1)m) clipped at 0 pooled with a per-channel softmax of gate + S->pos_bias[slot], no
 * RMSNorm, no rotation, into cache->idx_keys[b][i] (e4m3 codes of k / sigma with sigma the smallest
 * power of two with max|k| / sigma <= 448, into cache->idx_key_scale[b][i]; float32 keys get scale 1).
 * Reading of the pages: the lightning indexer scores the compressed entries "in a low-rank way"
 * ("DeepSeek-V4 Explained: ...", "The attention stack, and why it is two mechanisms"); its keys are
 * read as compressed like the entries themselves.  Needs d_I a multiple of 32, <= 128. */
CSA_API csa_status_t csa_index_keys(const csa_layer_t* L, const csa_cache_t* cache, const csa_index_stream_t* S,
                                    const void* x_new, const void* g_new, const int64_t* q_pos, int32_t Tq,
                                    void* stream);

/* Low-rank index queries: for each of `rows` query tokens, q_h = W_h c with c [rows][rank] (bf16,
 * the query's low-rank latent) and W [H_I * d_I][rank] (bf16, row h*d_I + d of W is output dim d of
 * head h), stored as idx_q [rows][H_I][d_I] e4m3 codes of q_h / sigma_h with idx_q_scale
 * [rows][H_I] the per-head power-of-two scale (the same rule as the keys), or float32 values with
 * scale 1.  rank a multiple of 16; d_I a multiple of 32, <= 128.  Same page and section (a low-rank
 * indexer); the up-projection of a latent is this library's reading of it. */
CSA_API csa_status_t csa_index_query(const csa_layer_t* L, const void* c, const void* W, int32_t rank,
                                     int32_t rows, void* idx_q, float* idx_q_scale, void* stream);

/* csa_decode_step with the index side produced in the step: csa_index_keys for the token (its
 * index row idx_x_new / idx_g_new [B][d_I]) and csa_index_query from its latent c [B][rank] run
 * first, on `stream`, and the indexer then scores the keys and queries they wrote (the index query
 * lives in the workspace of CSA_OP_DECODE_STEP_INDEXED).  Other arguments as csa_decode_step. */
CSA_API csa_status_t csa_decode_step_indexed(const csa_layer_t* L, const csa_cache_t* cache,
                                             const csa_params_t* P, const csa_index_stream_t* S,
                                             const void* q, const void* c, const void* W, int32_t rank,
                                             const float* head_w, const void* x_new, const void* g_new,
                                             const void* idx_x_new, const void* idx_g_new,
                                             const int64_t* q_pos, void* out, int32_t* topk_idx,
                                             void* workspace, size_t ws_bytes, void* stream);

/* Context-sharded CSA decode (one sequence's entries and index keys split into contiguous shards,
 * one per rank).  A rank holding entries [entry_offset, entry_offset + n_local) at slots 0.. of its
 * cache runs, for the B decode queries:
 *   1. csa_index_topk over its shard, with a layer whose pos0 is pos0 + entry_offset * m (so each
 *      shard entry's visibility is that of its global position) and n_max = n_local;
 *   2. csa_shard_candidates: (score, global index) of its local top-k;
 *   3. an all-gather of the candidates, [shards][B][top_k] each (the caller's collective);
 *   4. csa_shard_select: the global top-k of the gathered candidates, identical on every rank;
 *   5. csa_sparse_attend_partial over the selected entries it holds (one rank also the window rows);
 *   6. an all-gather of the partials, [shards][B][H][D + 2] (the caller's collective);
 *   7. csa_attend_merge: the output, with the sink counted once and the inverse rotation.
 * The result equals csa_sparse_attend with the unsharded top-k: an entry of the global top-k is in
 * its own shard's top-k, and attention over disjoint key sets merges by log-sum-exp weights.  The
 * pages describe one layer, not its distribution; the sink and the inverse rotation are those of
 * "DeepSeek-V4: Making a Million Tokens Affordable", "Two ways to shrink attention, interleaved". */

/* Step 2.  scores: [B][n_local] float32 of the shard (csa_index_topk's optional output); topk_local:
 * [B][top_k] its local top-k (-1 padded).  Writes cand_score [B][top_k] (-inf for padding) and
 * cand_idx [B][top_k] = local index + entry_offset (-1 for padding). */
CSA_API csa_status_t csa_shard_candidates(const csa_layer_t* L, const float* scores, int64_t n_local,
                                          const int32_t* topk_local, int64_t entry_offset, float* cand_score,
                                          int32_t* cand_idx, void* stream);

/* Step 4.  cand_score / cand_idx: [shards][B][top_k], shard s's lists in ascending index order and
 * the shards in ascending entry_offset order.  Writes topk_idx [B][top_k]: the top_k largest scores,
 * ties to the smaller global index, in ascending index order, -1 padded when fewer exist.
 * shards * top_k <= 262144. */
CSA_API csa_status_t csa_shard_select(const csa_layer_t* L, int32_t shards, const float* cand_score,
                                      const int32_t* cand_idx, int32_t* topk_idx, void* stream);

/* Step 5.  topk_idx [B][top_k] holds global indices; the entries in [entry_offset, entry_offset +
 * cache->entry_cap) are attended from cache slot (index - entry_offset), the others skipped; the
 * window rows only when with_window != 0.  partial: [B][H][D + 2] float32, per (query, head) the
 * weighted mean O/l of the attended rows (before the inverse rotation), then m and l in base 2
 * (max logit * log2 e and the sum of 2^(logit * log2 e - m)); no sink.  Needs H = 128, D = 512,
 * bf16 or mixed rows, B <= 8; workspace of CSA_OP_SPARSE_ATTEND. */
CSA_API csa_status_t csa_sparse_attend_partial(const csa_layer_t* L, const csa_cache_t* cache,
                                               const csa_params_t* P, const void* q, const int64_t* q_pos,
                                               const int32_t* topk_idx, int64_t entry_offset, int32_t with_window,
                                               float* partial, void* workspace, size_t ws_bytes, void* stream);

/* Step 7.  partials: [parts][B][H][D + 2] as written by csa_sparse_attend_partial; out [B][H][D]
 * act_format. */
CSA_API csa_status_t csa_attend_merge(const csa_layer_t* L, const csa_params_t* P, const int64_t* q_pos,
                                      int32_t parts, const float* partials, void* out, void* stream);

/* Bytes of the static device scratch used by csa_decode_step_scratch. */
#define CSA_SCRATCH_BYTES ((size_t)16 << 20)

/* csa_decode_step without a caller workspace (no counterpart on the pages:
 * a convenience of this library).  The workspace is a fixed array of
 * CSA_SCRATCH_BYTES in the library's static device memory, one per device,
 * so the call allocates nothing.
 *   - Limit: csa_workspace_size(L, CSA_OP_DECODE_STEP, 1, cache->entry_cap)
 *     must be <= CSA_SCRATCH_BYTES (B = 1 covers entry_cap up to 2^18, i.e.
 *     a 1M-token context at m = 4); a larger call returns CSA_ERR_WORKSPACE
 *     and touches no device state.
 *   - The array's address is looked up (cudaGetSymbolAddress, which may load
 *     the module) on the first call on each device: make that first call
 *     outside any CUDA stream capture.
 *   - Every call on a device shares its one array: two calls whose executions
 *     overlap (different streams or threads, concurrent graph replays) race
 *     on it and give undefined results.  Serialise them.
 *   - device_error: NULL, or a host int32 that receives the device error word
 *     (see csa_device_error); non-NULL synchronises the stream (not allowed
 *     during stream capture) and, when the word is non-zero, zero-fills the
 *     scratch again and returns CSA_ERR_DEVICE_TIMEOUT.  A call with NULL
 *     leaves any bits its kernels set in the scratch's word: the next call
 *     with a non-NULL device_error reports them (with its own), so after
 *     NULL calls that report covers every call since the last non-NULL one.
 *   - After a device error the scratch's histograms may be left non-zero.
 *     Every call therefore starts with a small guard kernel that, when the
 *     scratch's error word is set, zero-fills the scratch's top-k histograms
 *     and counters (keeping the word), so later calls, NULL or not, select
 *     from clean histograms.
 * Other arguments, layouts and errors as csa_decode_step. */
CSA_API csa_status_t csa_decode_step_scratch(const csa_layer_t* L, const csa_cache_t* cache,
                             const csa_params_t* P, const void* q,
                             const void* idx_q, const float* idx_q_scale, const float* head_w,
                             const void* x_new, const void* g_new, const int64_t* q_pos,
                             void* out, int32_t* topk_idx, int32_t* device_error,
                             void* stream);

/* Test aid for csa_decode_step_scratch (no counterpart on the pages): copies `bytes` bytes between
 * `buf` (host or device memory) and the current device's static scratch at byte `offset`, in the
 * direction `to_scratch` (1: buf -> scratch, 0: scratch -> buf), on `stream`, and synchronises it.
 * Offsets of the scratch's segments are those csa_debug_workspace_segment gives for the decode step.
 * Lets a test plant a device error and dirty histograms in the scratch.  A range outside the
 * CSA_SCRATCH_BYTES array returns CSA_ERR_INVALID_ARG with no device work. */
CSA_API csa_status_t csa_debug_scratch_copy(size_t offset, void* buf, size_t bytes, int32_t to_scratch,
                                            void* stream);

/* One fused HCA decode step: csa_append -> csa_compress -> hca_attend. */
CSA_API csa_status_t hca_decode_step(const csa_layer_t* L, const csa_cache_t* cache,
                             const csa_params_t* P, const void* q,
                             const void* x_new, const void* g_new, const int64_t* q_pos,
                             void* out, void* workspace, size_t ws_bytes, void* stream);

/* Chunked prefill of Tq tokens per sequence (CSA or HCA): csa_append of the
 * chunk's window rows (raw rows already in cache->raw), csa_compress of the
 * entries the chunk completes, then per query the indexer + top-k (CSA) and
 * attention.  n_max = entries visible to the chunk's last query. */
CSA_API csa_status_t csa_prefill(const csa_layer_t* L, const csa_cache_t* cache,
                         const csa_params_t* P, const void* q,
                         const void* idx_q, const float* idx_q_scale, const float* head_w,
                         const int64_t* q_pos, int32_t Tq, int64_t n_max,
                         void* out, int32_t* topk_idx,
                         void* workspace, size_t ws_bytes, void* stream);

/* ============================================================================================
 * Paged 8-bit key/value cache of grouped-query attention: appending to it, attending over it
 * (dense, or a sliding window with a few first tokens that stay visible), and the copying, forking,
 * freeing and compacting of its pages.  For the layers of a stack that are not compressed; the pages
 * compare the compressed caches against such a grouped-query cache ("DeepSeek-V4: Making a Million
 * Tokens Affordable") and give none of its details, so the definitions below are this library's.
 *
 * Layout.  A page holds `page` consecutive tokens of one sequence: k / v [n_pages][Hkv][page][D] e4m3
 * codes and one scale per page and KV head, k_scale / v_scale [n_pages][Hkv], a power of two in
 * [2^-126, 2^120]; value = code * scale.  table[b][p] is the page of tokens [p*page, (p+1)*page) of
 * sequence b, negative where there is none; refs[g] counts the table entries that name page g (0: free).
 * Several rows may name one page (after csa_pages_fork); the layers of a stack share one table and
 * have a pool each.
 *
 * Tokens.  A call passes up to Tq new tokens per sequence, j < n_new[b] (all Tq when n_new is NULL),
 * at positions start[b] + j; n_new[b] is taken into [0, Tq], and a sequence with start[b] < 0 has none.
 *
 * Errors on the device.  A page-table entry or page index of n_pages or more, a row index outside [0, B), a position
 * behind the table, a token without a page of its own, or a reference count that would fall below
 * zero sets bit 4 of a device error word: the workspace's for csa_paged_attend, for the calls without a
 * workspace one word per device that csa_device_error reads when it gets no workspace; the page or token
 * concerned is left out, nothing is read or written out of range.
 * ============================================================================================ */

/* One grouped-query attention layer over the cache. */
typedef struct csa_gqa {
  int32_t H;             /* query heads, a multiple of Hkv; query head h reads KV head h / (H / Hkv) */
  int32_t Hkv;           /* KV heads */
  int32_t D;             /* head dim: 64 or 128 */
  int32_t act_format;    /* CSA_FMT_F32 | CSA_FMT_BF16: queries, new keys and values, output */
  int32_t window;        /* keys seen behind the query, itself included; 0: all of them */
  int32_t first;         /* with a window: the first tokens, which every later query still sees */
  float softmax_scale;   /* logit scale; 0 selects 1/sqrt(D) */
  int32_t reserved;      /* 0 */
} csa_gqa_t;

/* One layer's pages. */
typedef struct csa_page_pool {
  void* k;               /* [n_pages][Hkv][page][D] e4m3 codes */
  void* v;               /* [n_pages][Hkv][page][D] e4m3 codes */
  float* k_scale;        /* [n_pages][Hkv] */
  float* v_scale;        /* [n_pages][Hkv] */
} csa_page_pool_t;

/* The bookkeeping of the pages, shared by the layers. */
typedef struct csa_page_table {
  int32_t* table;        /* [B][table_cap]; 4-byte aligned, so that some rows of a table are a table */
  int32_t* refs;         /* [n_pages] */
  int64_t table_cap;     /* entries of a row */
  int64_t n_pages;       /* pages of every pool, at most 2^30 */
  int32_t B;             /* rows (sequences) */
  int32_t page;          /* tokens per page: 16, 32, 64 or 128 */
} csa_page_table_t;

/* Encodes the new tokens' keys and values into their pages.  k_new, v_new: [B][Tq] tokens of Hkv * D
 * values in act_format, kv_stride elements apart (0: Hkv * D), a multiple of 16 bytes.  Per page and
 * KV head: scale = the larger of the scale its tokens before start[b] have (nothing when there are
 * none) and the smallest power of two, at least 2^-126, with max|x| / scale <= 448 over the finite new
 * values; new codes are x / scale rounded to nearest even, infinities saturated to +-448, NaN kept.
 * When the scale of a page grows, the codes of its earlier tokens are rounded once more, to the new
 * scale.  Slots behind the new tokens keep their bytes.  A token is left out, with error bit 4, where
 * the table has no page for it or refs (unless NULL) says that the page is shared: make the pages
 * ready with csa_pages_reserve. */
CSA_API csa_status_t csa_paged_append(const csa_gqa_t* L, const csa_page_pool_t* pool, const csa_page_table_t* T,
                                      const void* k_new, const void* v_new, int64_t kv_stride,
                                      const int64_t* start, const int32_t* n_new, int32_t Tq, void* stream);

/* Workspace bytes of csa_paged_attend (host; 0 if an argument is invalid).  One workspace serves paged calls of all
 * shapes that it is large enough for, one after the other.  It does not serve the other calls of the library: they need
 * theirs at zero, and a paged call leaves its records in it (zero-fill it before such a use). */
CSA_API size_t csa_paged_workspace_size(const csa_gqa_t* L, const csa_page_table_t* T, int32_t Tq, int64_t n_max);

/* Attention over the cache.  The query at position t = start[b] + j sees key i of its sequence iff
 *   i <= t, and (window == 0 or i > t - window or i < first), and table[b][i / page] is a page;
 *   z_i = <q_h, k_i> * softmax_scale;  o_h = sum_i e^{z_i} v_i / (e^{sinks[h]} + sum_i e^{z_i}),
 * without the sink's term when sinks is NULL; a query that sees nothing gets 0.  Keys and queries are
 * taken as they are: rotate them before the call where the layer does.
 *   q:     [B][Tq] tokens of H * D values in act_format, q_stride elements apart (0: H * D), a multiple
 *          of 16 bytes; the new tokens' own keys are in the cache already (csa_paged_append)
 *   sinks: [H] float32 or NULL
 *   n_max: a bound of every start[b] + n_new[b], at most table_cap * page and 2^30: tokens at n_max or
 *          behind it are neither attended nor answered
 *   out:   [B][Tq][H][D] act_format; the rows of tokens j >= n_new[b] are left as they are
 * Slots that no query sees are not read as numbers: whatever bytes they hold, NaN codes among them,
 * change nothing.  A NaN among the keys or values that a query sees makes that query's output NaN, at
 * least in the channels concerned.  Products and sums are float32 or wider (logits too: their magnitude has to
 * stay below 2^23).  What is rounded is w_i = p_i * (value scale of key i's page), the factor of key i's codes:
 * to 11 bits, where it is below 2^-18 of the query's largest w to 2^-29 of that largest (act_format float32: to
 * 22 bits, below 2^-17 to 2^-40).  Beside a page of a large scale, keys on pages of a far smaller one therefore
 * lose digits in every channel, also in channels where the large page's codes are 0.  Results depend on the
 * arguments and the number of SMs alone. */
CSA_API csa_status_t csa_paged_attend(const csa_gqa_t* L, const csa_page_pool_t* pool, const csa_page_table_t* T,
                                      const void* q, int64_t q_stride, const float* sinks,
                                      const int64_t* start, const int32_t* n_new, int32_t Tq, int64_t n_max,
                                      void* out, void* workspace, size_t ws_bytes, void* stream);

/* Test aid: the second launch of csa_paged_attend alone, which joins the parts of the sequences that were cut, over what
 * the workspace holds from an earlier call with the same arguments.  From byte 256 on the workspace has two int32 per
 * (sequence, block of query rows, KV head), the first and the last CTA with a part (equal: nothing to join).  They are the
 * first launch's; where one of its waits gave up (error bit 1) an entry may be an earlier call's bytes, and one that names
 * no CTA is left out, its rows as they were. */
CSA_API csa_status_t csa_debug_paged_join(const csa_gqa_t* L, const csa_page_table_t* T, const float* sinks,
                                          const int64_t* start, const int32_t* n_new, int32_t Tq, int64_t n_max,
                                          void* out, void* workspace, size_t ws_bytes, void* stream);

/* Row dst[i] of the table becomes a copy of row src[i] (i < n; both int32 on the device), so that the
 * two share their pages; the pages row dst[i] held before are released.  Pairs are taken from the rows
 * as they were before the call.  A pair whose src or dst is out of range, whose dst is a src of the
 * call or the dst of an earlier pair, is left out with error bit 4 (src = dst = -1: left out silently).
 * n <= 4096. */
CSA_API csa_status_t csa_pages_fork(const csa_page_table_t* T, const int32_t* src, const int32_t* dst, int32_t n,
                                    void* stream);

/* Gives every sequence pages of its own for the tokens it is about to write, [start[b], start[b] +
 * n_new[b]): where the table has none, and where the page there is shared (refs > 1).  When every table
 * entry that names a shared page is about to write it, the highest row keeps it.  New pages are the
 * lowest free ones, in the order of rows and positions.  copy_src / copy_dst [B] int32 (output): the
 * page to copy for row b because it holds tokens before start[b], -1 where there is none; pass them to
 * csa_pages_copy for every layer before the append.  missing [1] int32 (output): 0, or how many pages
 * there are too few; then nothing else changes (copy_src, copy_dst all -1).  A sequence whose tokens
 * pass the end of its row gets nothing, with error bit 4. */
CSA_API csa_status_t csa_pages_reserve(const csa_page_table_t* T, const int64_t* start, const int32_t* n_new,
                                       int32_t Tq, int32_t* copy_src, int32_t* copy_dst, int32_t* missing,
                                       void* stream);

/* Releases pages: entry p of row b is set to -1 and its page's count lowered where
 *   keep[b] >= 0 and p * page >= keep[b]            (tokens from keep[b] on are dropped; 0 ends the sequence), or
 *   p * page >= first and (p + 1) * page <= begin[b]  (tokens that a window has left behind for good).
 * keep, begin: [B] int64 or NULL (at least one given). */
CSA_API csa_status_t csa_pages_free(const csa_page_table_t* T, const int64_t* keep, const int64_t* begin,
                                    int64_t first, void* stream);

/* Moves pages down into free ones: the i-th highest page in use goes to the i-th lowest free page, as
 * long as that is lower and i < max_moves; table and refs are rewritten.  move_src / move_dst
 * [max_moves] int32 (output, -1 behind the last move) and count [1] int32 (output): pass them to
 * csa_pages_copy for every layer before the pages are read again.  max_moves <= n_pages. */
CSA_API csa_status_t csa_pages_compact(const csa_page_table_t* T, int32_t max_moves, int32_t* move_src,
                                       int32_t* move_dst, int32_t* count, void* stream);

/* Copies page src[i] to page dst[i], codes and scales of keys and values, for i < min(n, count[0])
 * (count NULL: i < n); src[i] < 0 or dst[i] < 0: nothing.  A page that is named as a dst twice, or as
 * both a src and a dst, ends with unspecified contents. */
CSA_API csa_status_t csa_pages_copy(const csa_gqa_t* L, const csa_page_pool_t* pool, const csa_page_table_t* T,
                                    const int32_t* src, const int32_t* dst, const int32_t* count, int32_t n,
                                    void* stream);

#ifdef __cplusplus
}
#endif

#endif  /* CSA_B200_CSA_H_ */
