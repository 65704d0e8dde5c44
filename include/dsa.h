/*
 * dsa.h -- C ABI of the DSA (Dynamic Sparse Attention) hot path for GB300 (sm_103a).
 *
 * The path, as the public pages on Kimi K3.1 Pro inference describe it:
 *   1. Lightning Indexer: score the query against every cached key with per-head weights
 *      ("Inference Optimization for Kimi K3.1 Pro: Decoding Architecture Evolution and Systems
 *      Engineering Practices", section 1, DSA step 1; "Day0 Inference Adaptation for Next-Gen
 *      LLMs ... CANN", section 3.1),
 *   2. keep the top-K positions, fused with scoring so that no score reaches global memory
 *      (first page, section 2 "Operator-Level Deep Fusion"),
 *   3. Sparse Flash Attention over only those positions of the paged MLA latent cache, blockwise
 *      with a cross-block softmax reduction ("Optimizing Kimi K3.1 Pro Sparse Attention
 *      Inference ...", section "Inheritance and Extension of Core Operators").
 *
 * Conventions shared by every call:
 *   - Every pointer in an args struct is a DEVICE pointer owned by the caller.  The library never
 *     allocates, never frees, never synchronises and keeps no pointer after it returns.  Work is
 *     enqueued on `stream` (a cudaStream_t; NULL = the legacy default stream) and runs
 *     asynchronously.
 *   - Synchronous errors (bad shape, null pointer, unsupported specialisation) are returned
 *     before anything is launched; dsa_last_error() then holds a one-line reason for the calling
 *     thread.  A failed launch returns DSA_ERR_CUDA.
 *   - Device-side checks (an index, length or page id out of range, a bounded wait that ran out)
 *     never trap: the kernel skips the offending work and stores a DSA_ERR_* code into *status
 *     (when status is not NULL; first error wins).  The caller reads it after synchronising.
 *   - Caches are paged with `page_size` rows per page.  Logical position j of sequence b lives at
 *     physical row page_table[b * max_pages + j / page_size] * page_size + j % page_size.
 *   - Query tokens are packed over sequences: the tokens of sequence b are q_start[b] ..
 *     q_start[b+1]-1; they are the last n_b = q_start[b+1]-q_start[b] positions of the sequence,
 *     so token i of sequence b sits at position seq_lens[b] - n_b + i (the keys and latent rows of
 *     the new tokens are already in the caches) and sees positions 0 .. that position.
 *   - Indices are LOGICAL positions, so results do not depend on where pages are placed.
 */
#ifndef DSA_H
#define DSA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Raised when a struct or a call changes so that an older caller would go wrong; an entry point that is only
 * added is found by its symbol. */
#define DSA_ABI_VERSION 7

/* Same type as cudaStream_t. */
typedef struct CUstream_st* dsa_stream_t;

typedef enum {
  DSA_OK = 0,
  DSA_ERR_INVALID_ARG = 1,  /* null pointer, negative or inconsistent size                    */
  DSA_ERR_UNSUPPORTED = 2,  /* valid, but no compiled specialisation covers it                */
  DSA_ERR_CUDA = 3,         /* a CUDA runtime/driver call or a launch failed                  */
  DSA_ERR_DEVICE_CHECK = 4, /* (in *status) a device-side range check failed                  */
  DSA_ERR_TIMEOUT = 5       /* (in *status) a bounded device-side wait gave up                */
} dsa_status;

/* DSA_MXFP8_E4M3: e4m3 elements with one E8M0 (power-of-two) scale per 32 consecutive elements. */
typedef enum { DSA_BF16 = 0, DSA_FP8_E4M3 = 1, DSA_MXFP8_E4M3 = 2 } dsa_dtype;

/* Human-readable name of a status code (static storage). */
const char* dsa_status_string(dsa_status s);

/* Reason for the last synchronous error returned on the calling thread ("" if none). */
const char* dsa_last_error(void);

/* DSA_ABI_VERSION of the built library. */
int dsa_abi_version(void);

/* ------------------------------------------------------------------------------------------ */
/* Lightning Indexer + top-K                                                                   */
/* ------------------------------------------------------------------------------------------ */

/*
 * For every query token t (at position p):
 *   s(t, j) = sum_{h < H_I} w[t][h] * max(0, q[t][h][:] . k[j][:])      for 0 <= j <= p,
 * with one index key row k[j] (d_I wide) per position, shared by all index heads; in FP8 mode
 * q[t][h][:] = q8 * q_scale[t][h] and k[j][:] = k8 * k_scale[row(j)]; in MXFP8 mode
 * ("Inference Optimization for Kimi K3.1 Pro", section 4: the indexer's fully quantised path,
 * group size 32) q[t][h][d] = q8 * 2^(q_sf[t][h][d/32] - 127) and
 * k[j][d] = k8 * 2^(k_sf[row(j)][d/32] - 127) (E8M0 bytes; 255 is not a valid scale).  The
 * selected set is the
 * first min(K, p+1) positions in the order (score descending, position ascending) -- ties go to
 * the lower position, and -0.0 equals +0.0.  Scores never leave the chip.
 *
 * Supported: page_size 64; (H_I, d_I) in {(8, 64), (64, 128)}; dtype BF16, or FP8_E4M3 and
 * MXFP8_E4M3 with (H_I, d_I) = (64, 128);
 * 1 <= K <= 2048; max_seq_len <= 131072; any number of tokens per sequence (decode, speculative
 * multi-token decode, chunked prefill).
 *
 * Position units (decode and two-token groups, max_seq_len > 32768, B <= 256): a sequence longer than one
 * cluster's span (32768 positions) is split into equal units, each selecting the top-K of its own
 * positions (with their scores) into `workspace`; a second kernel then merges each such token's
 * units ("Inference Optimization for Kimi K3.1 Pro", section 5: a local Top-K before the
 * merge, here over ranges of one sequence on one GPU), so that a batch of short and long
 * sequences spreads evenly over the SMs.  The result is the same set, in the same order.
 * dsa_li_workspace_bytes() says how much scratch that takes (0 when no sequence can be split).
 */
typedef struct {
  int B;            /* sequences                                                         */
  int n_q;          /* query tokens over all sequences (= q_start[B])                    */
  int H_I, d_I;     /* index heads, index head dim                                        */
  int K;            /* top-K                                                              */
  int page_size;    /* rows per page (64)                                                 */
  int max_pages;    /* row stride of page_table                                           */
  int num_pages;    /* pages in k_pool (device check on every page id)                     */
  int max_seq_len;  /* host-known upper bound of seq_lens[] (sizes the launch)            */
  int max_q_per_seq;/* host-known upper bound of q_start[b+1]-q_start[b]                  */
  dsa_dtype dtype;
  const void* q;          /* [n_q][H_I][d_I]   bf16 | e4m3                                */
  const float* q_scale;   /* [n_q][H_I] fp32, FP8 only (per-token scales: replicate)      */
  const float* w;         /* [n_q][H_I] fp32 head weights                                 */
  const void* k_pool;     /* [num_pages][page_size][d_I]  bf16 | e4m3                     */
  const float* k_scale;   /* [num_pages][page_size] fp32, FP8 only                        */
  const int32_t* page_table; /* [B][max_pages] physical page ids                          */
  const int32_t* seq_lens;   /* [B] positions, new tokens included                        */
  const int32_t* q_start;    /* [B+1] prefix offsets of the query tokens                  */
  int32_t* out_idx;       /* [n_q][K] selected positions, ascending, then -1 padding      */
  int32_t* out_cnt;       /* [n_q] number selected = min(K, p+1), or NULL                 */
  int32_t* status;        /* device int32 error word, or NULL                             */
  const uint8_t* q_sf;    /* [n_q][H_I][d_I/32] E8M0 group scales, MXFP8 only (else NULL) */
  const uint8_t* k_sf;    /* [num_pages][page_size][d_I/32] E8M0, MXFP8 only; the 4-byte
                             row of scales must be 4-byte aligned (d_I = 128)              */
  float* out_score;       /* [n_q][K] fp32 score of each position in out_idx (-inf for the
                             padding), or NULL: the candidates of a context-parallel shard  */
  void* workspace;        /* device scratch of dsa_li_workspace_bytes() bytes, 256-B aligned,
                             or NULL when that is 0; owned by the caller, no initial value */
  size_t workspace_bytes;
} dsa_li_args;

/* Scratch that dsa_li_topk needs for these arguments (0 if none).  Host only: reads B, K,
 * max_seq_len and max_q_per_seq; no CUDA call. */
size_t dsa_li_workspace_bytes(const dsa_li_args* args);

dsa_status dsa_li_topk(const dsa_li_args* args, dsa_stream_t stream);

/* ------------------------------------------------------------------------------------------ */
/* Sparse Flash Attention                                                                      */
/* ------------------------------------------------------------------------------------------ */

/*
 * For every query token t and head h, over the index set S_t = {idx[t][r] : idx[t][r] >= 0}:
 *   z_j = softmax_scale * q[t][h][0:d_qk] . kv[j][0:d_qk]
 *   out[t][h][:] = sum_j exp(z_j - m) kv[j][0:d_v] / sum_j exp(z_j - m),   m = max_j z_j
 *   lse[t][h]    = m + ln(sum_j exp(z_j - m))
 * The value is the leading d_v columns of the same latent row (MLA), so each selected row is
 * read once.  An empty set gives out = 0 and lse = -inf.  An index >= seq_lens[b] or < -1 is a
 * device check failure: the row is skipped and *status set.
 *
 * dsa_sfa_decode targets few tokens per sequence: it splits each token's K rows over several CTA
 * pairs and merges the partial softmax states through `workspace` (dsa_sfa_workspace_bytes()
 * bytes; with two splits, the usual case, each split finalises half of the heads);
 * dsa_sfa_prefill targets many tokens per sequence (one token per CTA pair, no workspace).  Both
 * give the same result up to fp32 rounding.
 *
 * Stream order: both are launched as programmatic dependents of the preceding kernel in the
 * stream, so their CTAs may start (barrier set-up, tensor-memory allocation) while that kernel
 * finishes; they read no device memory (inputs included) before it has completed.  Stream order
 * is therefore kept for every input, whichever kernel wrote it.
 *
 * Supported: page_size 64; d_qk 576; d_v 512; H in {16, 128} (decode) and 128 (prefill);
 * 1 <= K <= 2048; bf16 q/out; latent cache bf16 or FP8 (kv_dtype).
 *
 * FP8 latent cache (kv_dtype DSA_FP8_E4M3; "Inference Optimization for Kimi K3.1 Pro",
 * section 4, SFA KV cache quantisation per token and 128-column tile): each row of kv_pool is
 * 608 bytes: the 576 columns as e4m3 codes, then one fp32 scale per 128-column tile (5; the
 * last covers the 64 rope columns), then 12 unused bytes.  The attention runs on the BF16
 * values bf16(fp32(code * scale)) (both roundings to nearest even).
 */
typedef struct {
  int B, n_q;
  int H;              /* query heads                                                     */
  int d_qk, d_v;      /* 576, 512                                                        */
  int K;              /* row stride of idx                                               */
  int page_size, max_pages, num_pages;
  int max_seq_len, max_q_per_seq;
  float softmax_scale;
  const void* q;             /* [n_q][H][d_qk] bf16                                      */
  const void* kv_pool;       /* [num_pages][page_size][d_qk] bf16                        */
  const int32_t* page_table; /* [B][max_pages]                                           */
  const int32_t* seq_lens;   /* [B]                                                      */
  const int32_t* q_start;    /* [B+1]                                                    */
  const int32_t* idx;        /* [n_q][K] logical positions, -1 = empty slot              */
  void* out;                 /* [n_q][H][d_v] bf16                                       */
  float* lse;                /* [n_q][H] fp32, or NULL                                   */
  int32_t* status;           /* device int32 error word, or NULL                         */
  void* workspace;           /* device scratch of dsa_sfa_workspace_bytes(), 256-B aligned */
  size_t workspace_bytes;
  dsa_dtype kv_dtype;        /* DSA_BF16 (rows of 576 bf16) or DSA_FP8_E4M3 (608-byte rows) */
  int row_splits;            /* dsa_sfa_decode: CTA pairs that share one token's K rows
                                (0 = chosen from the SM count; the result does not depend on
                                it beyond fp32 rounding); ignored by dsa_sfa_prefill        */
} dsa_sfa_args;

/* Scratch that dsa_sfa_decode needs for these arguments (0 if none).  Host only: it reads the
 * current device's SM count (the split plan depends on it; 152 when no device is visible) and
 * launches nothing.  Only n_q, H, K and row_splits are read. */
size_t dsa_sfa_workspace_bytes(const dsa_sfa_args* args);

dsa_status dsa_sfa_decode(const dsa_sfa_args* args, dsa_stream_t stream);
dsa_status dsa_sfa_prefill(const dsa_sfa_args* args, dsa_stream_t stream);

/*
 * dsa_sfa_decode without a caller workspace, for callers that cannot allocate device memory: an
 * operator inside a framework that plans all device memory itself and passes the operator only
 * its inputs and outputs, or a path on which allocating is not allowed.  The pages have no
 * counterpart of this; it is an interface convenience of this library.
 *
 * The split-merge scratch is a fixed device array of DSA_SFA_STATIC_SCRATCH_BYTES inside the
 * library, held by every GPU that loads the library until the process exits.  args->workspace and
 * args->workspace_bytes are ignored; everything else is exactly dsa_sfa_decode (same kernel, same
 * result).  Arguments whose dsa_sfa_workspace_bytes() exceeds the capacity are rejected with
 * DSA_ERR_UNSUPPORTED and a reason in dsa_last_error().  No call allocates or frees memory.
 *  - The first call on a device looks up the array's device address (once per device, with that
 *    device current); make that first call before capturing a stream.
 *  - All calls on a device share the one array, which keeps the last call's contents; the call
 *    clears what must start at zero.  Calls whose work overlaps on the GPU (other streams, other
 *    host threads) race on the array: serialise them.
 *  - Capacity: with row_splits = 0 and K <= 2048 the library never plans more CTA pairs than
 *    one wave holds (2 * n_q * splits <= SMs), and a plan needs at most
 *    n_q * splits * 263,168 bytes (+ 512 for alignment and counters), so 20 MiB covers every such
 *    plan on a GPU of 159 SMs or fewer (152 on GB300).  An explicit row_splits or a larger K can
 *    exceed it; such calls are rejected as above.
 */
#define DSA_SFA_STATIC_SCRATCH_BYTES (20u * 1024u * 1024u)
dsa_status dsa_sfa_decode_static(const dsa_sfa_args* args, dsa_stream_t stream);

/* ------------------------------------------------------------------------------------------ */
/* Dense latent attention                                                                      */
/* ------------------------------------------------------------------------------------------ */

/*
 * Attention over every position a token sees, absorbed form: dsa_sfa_decode without the selection,
 * for contexts up to top-K, for layers without an indexer and for draft layers.  For query token t
 * (at position p = seq_lens[b] - n_b + i of sequence b) and head h, over j = 0 .. p:
 *   z_j = softmax_scale * q[t][h][0:d_qk] . kv[j][0:d_qk]
 *   out[t][h][:] = sum_j exp(z_j - m) kv[j][0:d_v] / sum_j exp(z_j - m),   m = max_j z_j
 *   lse[t][h]    = m + ln(sum_j exp(z_j - m))
 * q is the query with the keys' up-projection absorbed; the value is the leading d_v columns of
 * the latent row.  A token that sees nothing (p < 0, or only pages that do not exist) gets out = 0 and
 * lse = -inf; one whose logits, which are held in fp32, are all -inf, or one of them +inf, gets NaN in both.
 *
 * A value that a token does not see never reaches its output, whatever it holds: cache rows past
 * a sequence's length may hold NaN or infinities, and so may the rows of a sequence's later tokens.
 * A NaN or an infinity that a token does see makes its whole output row (and lse) NaN, or leaves NaN in the
 * columns it is in; an infinity among the d_qk - d_v last columns whose score is -inf has a weight of 0.
 * Rows of out and lse of tokens that no sequence owns (before q_start[0], from q_start[B] on) are
 * left as they were.  A length below 0 or above max_pages * page_size, a page id outside
 * [0, num_pages), and a q_start that decreases or leaves [0, n_q] set DSA_ERR_DEVICE_CHECK; the
 * length is clamped, the page's positions are skipped, the sequence is skipped.  (Tokens that two of the
 * remaining sequences then claim get rows of either.)
 *
 * Workspace: dsa_mla_decode_workspace_bytes() bytes, no initial value; a call leaves nothing in it
 * that a later call needs.  Calls that may overlap on the GPU need one each.
 *
 * Supported: page_size 64; d_qk 576; d_v 512; 1 <= H <= 128; bf16 q/out; latent cache bf16 or FP8
 * (608-byte rows, as for dsa_sfa_decode); any lengths that the page table covers; any number of
 * tokens per sequence.  max_q_per_seq (at least 1) is the host's bound of q_start[b+1]-q_start[b];
 * it sizes the groups of tokens that share a pass over the cache, and more tokens than it says
 * only take more passes.  q and kv_pool 16-byte aligned, out 32-byte aligned.
 */
typedef struct {
  int B, n_q;
  int H;              /* query heads                                                     */
  int d_qk, d_v;      /* 576, 512                                                        */
  int page_size, max_pages, num_pages;
  int max_q_per_seq;
  float softmax_scale;
  dsa_dtype kv_dtype;        /* DSA_BF16 (rows of 576 bf16) or DSA_FP8_E4M3 (608-byte rows) */
  const void* q;             /* [n_q][H][d_qk] bf16                                      */
  const void* kv_pool;       /* [num_pages][page_size][576 bf16 | 608 bytes]             */
  const int32_t* page_table; /* [B][max_pages]                                           */
  const int32_t* seq_lens;   /* [B] positions, new tokens included                       */
  const int32_t* q_start;    /* [B+1]                                                    */
  void* out;                 /* [n_q][H][d_v] bf16                                       */
  float* lse;                /* [n_q][H] fp32, or NULL                                   */
  int32_t* status;           /* device int32 error word, or NULL                         */
  void* workspace;           /* device scratch, 256-B aligned                            */
  size_t workspace_bytes;
} dsa_mla_decode_args;

/* Scratch that dsa_mla_decode needs for these arguments (only n_q, H and max_q_per_seq are read;
 * host only, it reads the current device's SM count and launches nothing). */
size_t dsa_mla_decode_workspace_bytes(const dsa_mla_decode_args* args);
dsa_status dsa_mla_decode(const dsa_mla_decode_args* args, dsa_stream_t stream);

/*
 * The same attention in its expanded form, for many new tokens: every head has its own keys and
 * values, the up-projection of the latent rows (a matrix product on the rows that dsa_cache_read
 * returns), and all heads share one rope key.  Keys and values are packed over sequences:
 * those of sequence b are kv_start[b] .. kv_start[b+1]-1, n_kv_b of them, and its n_b query
 * tokens are the last n_b positions, so token i sees j = 0 .. n_kv_b - n_b + i of them:
 *   z_j = softmax_scale * (q[t][h][0:128] . kv[j][h][0:128] + q[t][h][128:192] . k_rope[j])
 *   out[t][h][:] = softmax(z) . kv[:][h][128:256],   lse[t][h] = ln sum_j exp(z_j)
 * With q_absorbed = [W_uk[h]^T q_nope | q_rope], dsa_mla_decode followed by W_uv gives the same
 * output up to rounding.  A token that sees nothing gets out = 0 and lse = -inf, one whose logits (fp32)
 * are all -inf, or one of them +inf, NaN in both; tokens that no sequence owns keep their rows.  Keys and values of other sequences, and of later tokens, never
 * reach a token's output, whatever they hold; a NaN or infinity among the values that a token
 * does see may make its whole output row NaN.  A q_start or kv_start that decreases or leaves its
 * array sets DSA_ERR_DEVICE_CHECK, and the sequence is skipped; so is, after a q_start that decreases, a
 * sequence whose tokens start before an earlier one's end (a token belongs to the first that claims it).
 * More tokens in a sequence than max_q_per_seq set it too, and are computed all the same.
 *
 * Supported: d_nope 128, d_rope 64, d_v 128; 1 <= H <= 1024; bf16; (n_q / 256 + B) * max(H, 16) below
 * 2^31; q, kv and k_rope 16-byte aligned, out 32-byte aligned, k_rope_stride a multiple of 8.
 */
typedef struct {
  int B, n_q, n_kv;
  int H;
  int d_nope, d_rope, d_v;   /* 128, 64, 128                                             */
  int max_q_per_seq;         /* host-known upper bound of q_start[b+1]-q_start[b]        */
  float softmax_scale;
  long long k_rope_stride;   /* elements from one row of k_rope to the next (576: a view of the
                                latent rows' last columns)                               */
  const void* q;             /* [n_q][H][192] bf16                                       */
  const void* kv;            /* [n_kv][H][256] bf16: 128 key columns, then 128 value columns */
  const void* k_rope;        /* [n_kv][64] bf16                                          */
  const int32_t* q_start;    /* [B+1]                                                    */
  const int32_t* kv_start;   /* [B+1]                                                    */
  void* out;                 /* [n_q][H][128] bf16                                       */
  float* lse;                /* [n_q][H] fp32, or NULL                                   */
  int32_t* status;           /* device int32 error word, or NULL                         */
} dsa_mla_prefill_args;

dsa_status dsa_mla_prefill(const dsa_mla_prefill_args* args, dsa_stream_t stream);

/* ------------------------------------------------------------------------------------------ */
/* 8-bit rows and their product                                                                */
/* ------------------------------------------------------------------------------------------ */

/*
 * What stands between the residual stream and the calls above in a model that is served in FP8 ("Inference
 * Optimization for Kimi K3.1 Pro", section 4: one scale per token and 128 columns, as in the latent cache): the
 * norm before a projection, the projection, and what the attention leaves on its way into the next one.  The
 * pages define no interface for these.
 *
 * An 8-bit row is dim e4m3 codes and ceil(dim / 128) fp32 scales, each of 128 columns (the last of what is left):
 * with a the largest finite magnitude of a group's values, s = fp32(a / 448), 1 when a = 0 and at least 2^-126,
 * code = e4m3(value / s), to nearest even, saturated at 448 (infinities too); a NaN is kept.
 */
typedef enum { DSA_ELEM_BF16 = 0, DSA_ELEM_FP16 = 1, DSA_ELEM_FP32 = 2 } dsa_elem;

/*
 * Root-mean-square norm with the residual's addition, into 8-bit rows; T is the type of x:
 *   h = T(x + residual)  (h = x without a residual),   stored to sum
 *   r = 1 / sqrt(mean(h^2) + eps),   v[d] = h[d] * weight[d] * r   -> codes, scale, and T(v) -> y
 * mean(h^2) and r are held in fp32: a row whose sum of squares is beyond fp32 has r = 0, one with a NaN is all
 * NaN; squares below 2^-126 keep fewer bits and those below 2^-150 none, so that without eps a row that has no other
 * is taken as a row of zeros, r = infinity.  h * weight is rounded to fp32 (exact for 16-bit types within its normal
 * range); v itself is not rounded before it is quantised, but counts as infinite where it is beyond fp32 (it
 * saturates, and its group's scale is that of the others) and is rounded below fp32's normal range.
 *
 * sum and y may be x or residual themselves (same address and stride); outputs overlap nothing else.  Launched as a
 * programmatic dependent, as dsa_sfa_decode is (see above).  Supported: dim a multiple of 8, up to 32768; weight of T
 * or fp32; rows of x, residual, sum, y and weight 16-byte aligned, those of codes 8-byte aligned; strides (of more than
 * one row) from the row's length up to 2^40.
 */
typedef struct {
  int n_rows;
  int dim;
  dsa_elem elem;           /* T: type of x, residual, sum and y                              */
  dsa_elem weight_elem;    /* T or DSA_ELEM_FP32                                             */
  float eps;               /* >= 0                                                           */
  long long x_stride, residual_stride, sum_stride, y_stride; /* elements from row to row     */
  long long codes_stride;  /* bytes                                                          */
  long long scale_stride;  /* elements                                                       */
  const void* x;           /* [n_rows][dim]                                                  */
  const void* weight;      /* [dim]                                                          */
  const void* residual;    /* [n_rows][dim], or NULL                                         */
  void* sum;               /* [n_rows][dim]: with a residual only                            */
  void* y;                 /* [n_rows][dim], or NULL                                         */
  void* codes;             /* [n_rows][dim] e4m3                                             */
  float* scale;            /* [n_rows][ceil(dim / 128)]                                      */
} dsa_rms_norm_quant_args;

dsa_status dsa_rms_norm_quant(const dsa_rms_norm_quant_args* args, dsa_stream_t stream);

/* Rows as they are into 8-bit rows.  Launched as a programmatic dependent, as dsa_sfa_decode is (see above).  Supported:
 * dim a multiple of 8, up to 2^30; rows of x 16-byte, of codes 8-byte aligned; n_rows times ceil(dim / 128) below 2^29;
 * strides as above. */
typedef struct {
  int n_rows;
  int dim;
  dsa_elem elem;           /* type of x                                                      */
  long long x_stride;      /* elements                                                       */
  long long codes_stride;  /* bytes                                                          */
  long long scale_stride;  /* elements                                                       */
  const void* x;           /* [n_rows][dim]                                                  */
  void* codes;             /* [n_rows][dim] e4m3                                             */
  float* scale;            /* [n_rows][ceil(dim / 128)]                                      */
} dsa_quant_rows_args;

dsa_status dsa_quant_rows(const dsa_quant_rows_args* args, dsa_stream_t stream);

/*
 * Product of 8-bit rows with e4m3 weights that have one fp32 scale per block of 128 rows and 128 columns:
 *   out[m][n] = sum_i fp32(a_scale[m][i] * b_scale[n / 128][i]) * sum_{k in columns of block i} a[m][k] * b[n][k]
 * for i < ceil(K / 128).  A block's products are added by the tensor cores with fp32 accumulators, the blocks'
 * sums with fp32 multiply-adds, and the result is rounded once to the type of out.  A NaN in a row of either operand,
 * or a NaN or an infinity in a scale, reaches the outputs of the rows that it belongs to alone: one row of out for a
 * row of a, one column for a row of b, the 128 columns of its block for a scale of b.
 *
 * a may be the rows of an FP8 latent cache as they lie there (a_stride 608, a_scale 576 bytes on, a_scale_stride
 * 152): the up-projection of dsa_mla_prefill's keys and values reads no converted copy.
 *
 * Few rows stream the weights, many run on tiles of 256 x 256; each output is added up in an order that
 * depends on the sizes and the GPU's number of SMs alone, so that a call gives the same bits every time.  Rows of out that start 16-byte
 * aligned are stored fastest.  Launched as a programmatic dependent, as dsa_sfa_decode is (see above).
 *
 * Supported: K a multiple of 16; M, N and K up to 2^31 - 256, and M times N in no more than 0x70000000 tiles of
 * 256 x 256; rows of a and b 16-byte aligned; rows (of more than one) at least their length and less than 2^40 bytes
 * apart; out overlaps no input.
 */
typedef struct {
  int M, N, K;
  dsa_elem elem;             /* type of out                                                  */
  long long a_stride;        /* bytes from row to row                                        */
  long long a_scale_stride;  /* elements                                                     */
  long long b_stride;        /* bytes                                                        */
  long long b_scale_stride;  /* elements                                                     */
  long long out_stride;      /* elements                                                     */
  const void* a;             /* [M][K] e4m3                                                  */
  const float* a_scale;      /* [M][ceil(K / 128)]                                           */
  const void* b;             /* [N][K] e4m3                                                  */
  const float* b_scale;      /* [ceil(N / 128)][ceil(K / 128)]                               */
  void* out;                 /* [M][N]                                                       */
  int32_t* status;           /* device int32 error word, or NULL                             */
} dsa_matmul_fp8_args;

dsa_status dsa_matmul_fp8(const dsa_matmul_fp8_args* args, dsa_stream_t stream);

/* ------------------------------------------------------------------------------------------ */
/* Context-parallel top-K merge                                                                */
/* ------------------------------------------------------------------------------------------ */

/*
 * "Inference Optimization for Kimi K3.1 Pro", section 5 (local Top-K before communication): a
 * long sequence's positions are split over S shards; each shard runs dsa_li_topk on its own
 * range (with out_score) and the shards' (score, position) candidates are gathered -- the one
 * exchange step -- and merged here.  For each query t the result is the first min(K, valid)
 * candidates in the order (score descending, position ascending), emitted in ascending
 * position order with -1 padding: the same set dsa_li_topk selects over the whole range, since
 * every position's score does not depend on the split.
 *   cand_idx   [S][n_q][K_in] shard-local positions (-1 = none); position + shard_offset[s] is
 *              the sequence position (shards own disjoint ranges)
 *   cand_score [S][n_q][K_in] their scores
 * Supported: S * K_in <= 16384, K <= K_in * S.  Device pointers; asynchronous on stream.
 */
typedef struct {
  int S, n_q, K_in, K;
  const int32_t* cand_idx;
  const float* cand_score;
  const int32_t* shard_offset; /* [S] device array                                          */
  int32_t* out_idx;            /* [n_q][K]                                                   */
  int32_t* out_cnt;            /* [n_q] or NULL                                              */
} dsa_topk_merge_args;

dsa_status dsa_topk_merge(const dsa_topk_merge_args* args, dsa_stream_t stream);

/* ------------------------------------------------------------------------------------------ */
/* Indexer Prolog                                                                              */
/* ------------------------------------------------------------------------------------------ */

/*
 * The indexer's input preparation for the new tokens ("Inference Optimization for Kimi K3.1 Pro",
 * section 3, Indexer Prolog, and section 4, MXFP8 indexer path; "Day0 Inference Adaptation ...
 * CANN", section 3.3).  For each new token t (sequence b, position p = seq_lens[b] - n_b + i):
 *   q[t][h][:] = W_q[h*d_I .. h*d_I+d_I) . xq[t]                 -> q_out (+ q_sf)
 *   k[t]       = LayerNorm(W_k . x[t]) * ln_gamma + ln_beta        -> key-cache row of p
 *   w[t][h]    = w_scale * (W_w[h] . x[t])                         -> w_out (fp32)
 * LayerNorm: mean and biased variance over the d_I features, then (v - mean) / sqrt(var + eps).
 * dtype DSA_MXFP8_E4M3: q and k become e4m3 codes with one E8M0 scale byte per 32 features
 * (shared exponent floor(log2(max |v|)) - 8, clamped to [-127, 127], 0 for an all-zero group;
 * elements v / 2^e rounded to nearest even, saturated at 448; a zero is +0) -- the layout
 * dsa_li_topk reads in its MXFP8 mode; dtype DSA_BF16: bf16, round to nearest even.
 * The three projections run as concurrent CTA roles of one launch (no stream fork).
 *
 * Supported: H_I = 64, d_I = 128, page_size 64; d_q and d_model multiples of 8; bf16 inputs and
 * weights, 16-byte aligned.  A position whose page id is outside [0, num_pages) sets
 * DSA_ERR_DEVICE_CHECK and its key row is not written.
 */
typedef struct {
  int n_q;              /* new tokens (= q_start[B])                                       */
  int B;
  int d_q;              /* input width of the Q projection                                 */
  int d_model;          /* input width of the K and head-weight projections                */
  int H_I, d_I;         /* 64, 128                                                         */
  dsa_dtype dtype;      /* DSA_MXFP8_E4M3 or DSA_BF16: format of q_out and of the key cache */
  int page_size;        /* 64                                                              */
  int max_pages;        /* row stride of page_table                                        */
  int num_pages;        /* pages in k_pool                                                 */
  float ln_eps;
  float w_scale;        /* head-weight scale                                               */
  const void* xq;       /* [n_q][d_q] bf16                                                 */
  const void* x;        /* [n_q][d_model] bf16                                             */
  const void* w_q;      /* [H_I*d_I][d_q] bf16                                             */
  const void* w_k;      /* [d_I][d_model] bf16                                             */
  const void* w_w;      /* [H_I][d_model] bf16                                             */
  const float* ln_gamma;/* [d_I]                                                           */
  const float* ln_beta; /* [d_I]                                                           */
  const int32_t* page_table; /* [B][max_pages] of the key cache                           */
  const int32_t* seq_lens;   /* [B] positions, new tokens included                        */
  const int32_t* q_start;    /* [B+1]                                                     */
  void* q_out;          /* [n_q][H_I][d_I] e4m3 codes or bf16                              */
  uint8_t* q_sf;        /* [n_q][H_I][d_I/32] (MXFP8)                                      */
  float* w_out;         /* [n_q][H_I]                                                      */
  void* k_pool;         /* [num_pages][page_size][d_I] e4m3 codes or bf16 (written rows only) */
  uint8_t* k_sf;        /* [num_pages][page_size][d_I/32] (MXFP8)                          */
  void* workspace;      /* unused: dsa_prolog_workspace_bytes() is 0 (the slices of a tile
                           meet in distributed shared memory); may be NULL                */
  size_t workspace_bytes;
  int32_t* status;      /* device int32 error word, or NULL                                */
} dsa_prolog_args;

/* Scratch bytes dsa_indexer_prolog needs for these sizes (only the size fields are read): 0 --
 * this implementation needs none; kept so that callers size the field the same way as the
 * other entry points' workspaces. */
size_t dsa_prolog_workspace_bytes(const dsa_prolog_args* args);
dsa_status dsa_indexer_prolog(const dsa_prolog_args* args, dsa_stream_t stream);

/* ------------------------------------------------------------------------------------------ */
/* Cache layout and page-table helpers                                                         */
/* ------------------------------------------------------------------------------------------ */

/*
 * The caches are paged: the indexer reads the paged key cache directly ("Day0 Inference
 * Adaptation for Next-Gen LLMs ... CANN", section 3.1), and the selected indices address the
 * paged KV cache page by page ("Inference Optimization for Kimi K3.1 Pro", section 2, "Inlined
 * Top-K Selection": on-demand in-page addressing).  The helpers below describe and maintain
 * that layout; they are host-side conveniences (the pages define no interface).
 */

/* Bytes of one page of `rows` rows of `dim` elements of `dtype` (0 on invalid input); for
 * MXFP8 the elements only (the E8M0 scales are a separate [rows][dim/32] byte array, the
 * group-32 scales of "Inference Optimization for Kimi K3.1 Pro", section 4). */
size_t dsa_page_bytes(dsa_dtype dtype, int rows, int dim);

/*
 * Host-side check of a page table (host pointers) before it drives the in-page addressing of
 * the kernels ("Inference Optimization for Kimi K3.1 Pro", section 2, "Inlined Top-K
 * Selection"): for every sequence b, the pages
 * 0 .. ceil(seq_lens[b]/page_size)-1 hold ids in [0, num_pages), and (if require_unique) no id
 * is used twice over the whole table.  Entries past a sequence's last page are ignored.
 * Returns DSA_OK or DSA_ERR_INVALID_ARG (reason in dsa_last_error()).
 */
dsa_status dsa_page_table_validate(const int32_t* page_table_host, int B, int max_pages,
                                   const int32_t* seq_lens_host, int page_size, int num_pages,
                                   int require_unique);

/*
 * Append new rows to a paged cache: the write of the new tokens' keys that the indexer's input
 * preparation performs ("Inference Optimization for Kimi K3.1 Pro", section 3, "Three-Stream
 * Parallel Architecture", the K normalisation stream; dsa_indexer_prolog does this itself for
 * the key cache), or of latent rows for the attention cache.  Scatter n_rows rows (device
 * pointers):
 *   pool[page_table[seq[r]][pos[r] / page_size]][pos[r] % page_size][:] = rows[r][:]
 * and, when row_scales is not NULL, scale_pool[same page][same slot] = row_scales[r] (the
 * per-row fp32 scale of an FP8 key cache).  elem_bytes is 2 (bf16) or 1 (e4m3); dim*elem_bytes
 * must be a multiple of 16.  Out-of-range seq/pos/page entries are skipped and flagged in
 * *status.
 */
dsa_status dsa_cache_write(void* pool, float* scale_pool, int num_pages, int page_size, int dim,
                           int elem_bytes, const int32_t* page_table, int max_pages, int B,
                           const int32_t* seq, const int32_t* pos, const void* rows,
                           const float* row_scales, int n_rows, int32_t* status,
                           dsa_stream_t stream);

/*
 * Rows of activations into a quantised paged cache (dsa_cache_write_quant), and cache rows back
 * out (dsa_cache_read): "Inference Optimization for Kimi K3.1 Pro", section 4, the latent cache
 * in FP8 with one scale per token and 128-column tile and the index keys in FP8 with group
 * scales, in the layouts that dsa_li_topk, dsa_sfa_* and dsa_mla_decode read.  Row r goes to, or
 * comes from, physical row page_table[seq[r]][pos[r] / page_size] * page_size + pos[r] % page_size.
 *
 *   DSA_ROW_LATENT_FP8  pool [num_pages][page_size][608 bytes]: 576 e4m3 codes, one fp32 scale per
 *                       128 columns (5; the last covers 64), 12 bytes that a write sets to zero
 *   DSA_ROW_FP8         pool e4m3 [num_pages][page_size][dim], scale_pool fp32 [num_pages][page_size]
 *   DSA_ROW_MXFP8       pool e4m3 [num_pages][page_size][dim], sf_pool E8M0 [...][dim / 32]
 *   DSA_ROW_BF16        pool bf16 [num_pages][page_size][dim]; read only (dsa_cache_write writes it)
 *
 * Write: with a the largest finite magnitude of a group of columns (the scale's columns),
 *   FP8:   s = fp32(a / 448), 1 when a = 0 and at least 2^-126; code = e4m3(x / s)
 *   MXFP8: e = max(floor(log2 a) - 8, -127), 0 when a = 0;      code = e4m3(x * 2^-e), sf = e + 127
 * e4m3() rounds to nearest even, saturates at 448 (infinities too) and keeps a NaN; x / s is not
 * rounded before it.  Read: y = rows' type(fp32(code * scale)), to nearest even (to bf16: the
 * operand that the attention over an FP8 latent cache forms); an E8M0 byte of 255 gives NaN.
 *
 * A row whose seq, pos or page id is out of range sets DSA_ERR_DEVICE_CHECK; a write skips it, a
 * read fills it with zeros.  Two rows of one write to the same place leave either one's codes and
 * scales, possibly mixed.  A read may name a place any number of times.
 *
 * Supported: dim 576 (LATENT_FP8); 32, 64, 128, 256 (FP8, MXFP8); any multiple of 8 (BF16).  rows
 * and pool 16-byte aligned, row_stride * element size a multiple of 16, row_stride >= dim.
 */
typedef enum { DSA_ROW_BF16 = 0, DSA_ROW_FP8 = 1, DSA_ROW_MXFP8 = 2, DSA_ROW_LATENT_FP8 = 3 } dsa_row_format;

typedef struct {
  int n_rows;
  int dim;               /* columns of a row                                               */
  int B;                 /* sequences (rows of page_table)                                 */
  int page_size;         /* cache rows per page (any)                                      */
  int max_pages;         /* row stride of page_table                                       */
  int num_pages;         /* pages in pool                                                  */
  dsa_row_format format; /* of the cache                                                   */
  dsa_elem elem;         /* type of rows                                                   */
  long long row_stride;  /* elements from one row of rows to the next                      */
  void* rows;            /* [n_rows][dim]: read by dsa_cache_write_quant, written by dsa_cache_read */
  void* pool;
  float* scale_pool;     /* FP8 only                                                       */
  uint8_t* sf_pool;      /* MXFP8 only                                                     */
  const int32_t* page_table; /* [B][max_pages]                                             */
  const int32_t* seq;    /* [n_rows]                                                       */
  const int32_t* pos;    /* [n_rows]                                                       */
  int32_t* status;       /* device int32 error word, or NULL                               */
} dsa_cache_rows_args;

dsa_status dsa_cache_write_quant(const dsa_cache_rows_args* args, dsa_stream_t stream);
dsa_status dsa_cache_read(const dsa_cache_rows_args* args, dsa_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* DSA_H */
