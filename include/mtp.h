/*
 * mtp.h -- C ABI of the GB300 MTP speculative-decoding hot path.
 *
 * Eleven operations, all asynchronous on a caller-supplied CUDA stream:
 *
 *   mtp_draft_block    N chained draft steps of an MTP assistant head that
 *                      cross-attends into the target's KV cache, in ONE
 *                      persistent launch (token -> embedding -> hidden-state
 *                      chain stays on the device between steps).
 *   mtp_verify_greedy  longest greedy-matching prefix + bonus token from the
 *                      target's (1+N) x V verify logits.
 *   mtp_verify_sample  exact speculative sampling at temp > 0.
 *   mtp_sample_drafts  the draws of a sampling drafter from given draft
 *                      logits (the q the sampling verifier checks against).
 *   mtp_nextn_draft    the dense NextN self-speculation drafter: its own
 *                      block and its own KV, the catch-up on the accepted
 *                      rows, then N chained draft steps, in ONE launch.
 *   mtp_kv_append      the target's new key and value rows into its paged KV
 *                      cache (fp32, bf16, or e4m3 with a scale per page and
 *                      KV head), key norm and RoPE on the way.
 *   mtp_paged_attention  the target's 1..64 new rows per sequence (a verify
 *                      step, or plain decoding) attend that cache.
 *   mtp_token_logprobs log probability, entropy and top alternatives of given
 *                      tokens from rows of logits.
 *   mtp_rotate_axes    query and key rows normed and rotated by several
 *                      positions (time, height, width of images and video).
 *   mtp_prompt_attention  the rows of whole prompts, packed one after another,
 *                      attend that cache.
 *   mtp_prefix_attention  the new rows of sequences that share long prefixes
 *                      attend that cache, a group's prefix once for its rows.
 *
 * Definitions are those of the pages this library implements:
 *   [G4] "Gemma 4 MTP -- Multi-Token Prediction speculative decoding":
 *        sec. 4 "Per-step MTP graph" (the draft step), sec. 5 "KV sharing"
 *        (read-only cross-attention, one mask for all steps), sec. 6 (the
 *        public API this one replaces: llama_decode_mtp_async / _wait).
 *   [NX] "MTP decoding (--mtp)": "Requirements" (enorm / hnorm / eh_proj) and
 *        "How it is wired" (greedy longest-prefix accept + bonus token).
 *   [FN] "Fused NextN draft graph": one launch + one readback for N steps;
 *        delta 6 (frozen-prefix cross-attention).
 *   [SP] "opus-mtp-turbo: Track 1 report", item 4 (exact temp > 0
 *        verification: sample_dist, accept with p/q, residual max(p - q, 0)).
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * - Every pointer argument is DEVICE memory owned by the caller, unless its
 *   comment says "host".  The library never allocates, frees or copies
 *   buffers of its own, never synchronizes the stream (except
 *   mtp_last_error, which says so) and keeps no state between calls.
 * - Scratch space is the caller's workspace `ws` (`ws_bytes` bytes, 256-byte
 *   aligned, device memory), sized by mtp_workspace_size().  Calls that share
 *   a workspace must be ordered on one stream.
 * - Return value: MTP_OK, or a negative MTP_ERR_* code when the arguments are
 *   rejected on the host (nothing is launched then) or a launch fails.
 *   Errors found while the kernels run (a grid barrier that timed out, a
 *   candidate set that overflowed) are written to a status word inside the
 *   workspace and read back with mtp_last_error().
 * - Row-major layouts; every row start must be 16-byte aligned (row lengths
 *   in elements: multiples of 8 for bf16, 4 for fp32).
 */
#ifndef MTP_H
#define MTP_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* a cudaStream_t; NULL is the legacy default stream */
typedef struct CUstream_st *mtp_stream_t;

enum {
    MTP_OK = 0,
    MTP_ERR_ARG = -1,          /* a pointer, size or layout argument is invalid */
    MTP_ERR_UNSUPPORTED = -2,  /* valid, but outside what the kernels implement */
    MTP_ERR_WORKSPACE = -3,    /* ws is NULL, misaligned or smaller than required */
    MTP_ERR_CUDA = -4,         /* a CUDA launch failed */
    MTP_ERR_TIMEOUT = -5,      /* (device status) a grid barrier gave up waiting */
    MTP_ERR_CAPACITY = -6      /* (device status) a sampling candidate set overflowed */
};

enum { MTP_DTYPE_F32 = 0, MTP_DTYPE_BF16 = 1,
       MTP_DTYPE_E4M3 = 2 };       /* only as mtp_kv_cache.kv_dtype */
/* projection weight formats (mtp_config.wquant) */
enum { MTP_WQ_NONE = 0, MTP_WQ_Q8_0 = 1, MTP_WQ_Q4_0 = 2 };

#define MTP_MAX_BLOCKS 8
#define MTP_MAX_VIEWS 4
#define MTP_MAX_BATCH 64            /* sequences of one mtp_draft_block call */
#define MTP_MAX_VERIFY_BATCH 65536  /* sequences of one verify or draw call */
#define MTP_MAX_CENTROIDS 8192      /* centroids of a centroid-routed LM head */
#define MTP_MAX_CATCHUP 16          /* catch-up rows per sequence of one mtp_nextn_draft call */
#define MTP_MAX_PAGED_BATCH 1024    /* sequences of one mtp_kv_append or attention call over a paged cache */
#define MTP_MAX_APPEND_ROWS 65536   /* rows per sequence of one mtp_kv_append call */
#define MTP_MAX_ATTN_ROWS 64        /* rows per sequence of one mtp_paged_attention call */
#define MTP_MAX_PAGE_SIZE 256       /* slots of a page */
#define MTP_MAX_TOP 32              /* alternatives per row of mtp_token_logprobs */
#define MTP_MAX_PROMPT_ROWS 1048576 /* packed rows of one mtp_prompt_attention or mtp_rotate_axes call */
#define MTP_MAX_AXES 4              /* positions per row of mtp_rotate_axes */

/* Sizes and scalars of the assistant head ([G4] sec. 3-4).
 *   d_t        backbone (target) width: token embedding, h_prev, LM head input
 *   d_a        assistant width
 *   n_blocks   assistant blocks (<= MTP_MAX_BLOCKS)
 *   n_q_heads, head_dim, n_kv_heads   query heads, their width, KV heads of the
 *              target layers cross-attended (n_q_heads % n_kv_heads == 0)
 *   d_ff       GeGLU hidden width
 *   vocab      rows of the tied token-embedding table
 *   wdtype     MTP_DTYPE_BF16 or MTP_DTYPE_F32: weight matrices and KV
 *   rms_eps    RMSNorm epsilon; attn_scale softmax scale, 0 = the default
 *              1/sqrt(head_dim) (rounded to fp32);
 *   emb_scale  token-embedding scale, 0 = the default sqrt(d_t) (Gemma's);
 *   logit_softcap  > 0 applies cap * tanh(z / cap) to the logits, 0 = off
 *   n_centroids    0: the dense tied LM head.  > 0: the centroid-routed head
 *                  of ordered-embedding models ([G4] sec. 3 "Centroid /
 *                  ordered-embeddings LM head"), n_centroids <=
 *                  MTP_MAX_CENTROIDS dividing vocab (MTP_ERR_ARG otherwise;
 *                  above the maximum MTP_ERR_UNSUPPORTED)
 *   centroid_top_k centroids whose candidate lists are scored per step,
 *                  1..n_centroids (ignored for the dense head, must be >= 0)
 *   wquant         MTP_WQ_NONE: the projections (w_pre, w_post and every
 *                  block's w_q, w_o, w_gate, w_up, w_down) are in wdtype.
 *                  MTP_WQ_Q8_0 ("opus-mtp-turbo: Track 1 report", item 3):
 *                  they are Q8_0 codes, int8 [out, in], each with its
 *                  block scales, binary16 [out, in / 32] (see
 *                  mtp_quantize_q8_0); requires wdtype MTP_DTYPE_BF16 (the
 *                  table and KV), head_dim 64, 128 or 256, every input
 *                  width a multiple of 32; runs on the CUDA-core paths.
 *                  MTP_WQ_Q4_0 (the same item's Q4_0 column): Q4_0 codes,
 *                  uint8 [out, in / 2] -- per block of 32 weights 16 bytes,
 *                  byte j holding the code of weight j in its low four bits
 *                  and of weight j + 16 in its high four; the weight is
 *                  (code - 8) times the block's binary16 scale [out, in / 32]
 *                  (see mtp_quantize_q4_0); the same requirements as Q8_0 */
typedef struct mtp_config {
    int32_t d_t, d_a, n_blocks, n_q_heads, head_dim, n_kv_heads, d_ff, vocab;
    int32_t wdtype;
    float rms_eps, attn_scale, emb_scale, logit_softcap;
    int32_t n_centroids, centroid_top_k;
    int32_t wquant, pad_;
} mtp_config;

/* One assistant block.  Matrices are row-major [out, in] in `wdtype`; RMSNorm
 * gains are fp32.  kv_view selects which mtp_kv_view the block attends. */
typedef struct mtp_block_weights {
    const void *attn_norm;       /* fp32 [d_a] */
    const void *w_q;             /* [n_q_heads * head_dim, d_a] */
    const void *q_norm;          /* fp32 [head_dim], shared by all heads */
    const void *w_o;             /* [d_a, n_q_heads * head_dim] */
    const void *post_attn_norm;  /* fp32 [d_a] */
    const void *pre_ffn_norm;    /* fp32 [d_a] */
    const void *w_gate;          /* [d_ff, d_a] */
    const void *w_up;            /* [d_ff, d_a] */
    const void *w_down;          /* [d_a, d_ff] */
    const void *post_ffn_norm;   /* fp32 [d_a] */
    int32_t kv_view;
    int32_t pad_;
    /* MTP_WQ_Q8_0 only (NULL otherwise): block scales of w_q, w_o, w_gate, w_up, w_down */
    const uint16_t *w_q_scale, *w_o_scale, *w_gate_scale, *w_up_scale, *w_down_scale;
    /* mtp_nextn_draft only (NULL otherwise): fp32 [head_dim] key norm, shared by all KV heads */
    const void *k_norm;
} mtp_block_weights;

typedef struct mtp_weights {
    const void *tok_embd;    /* [vocab, d_t]: the TARGET's table, also the tied LM head */
    const void *norm_e;      /* fp32 [d_t]: norm of the scaled token embedding */
    const void *norm_h;      /* fp32 [d_t]: norm of h_prev */
    const void *w_pre;       /* [d_a, 2 d_t]: pre-projection of [norm_e(e); norm_h(h)] */
    const void *final_norm;  /* fp32 [d_a] */
    const void *w_post;      /* [d_t, d_a]: post-projection -> next h_prev */
    mtp_block_weights blk[MTP_MAX_BLOCKS];
    /* centroid-routed head only (NULL for the dense head): */
    const void *centroids;           /* [n_centroids, d_t] in wdtype, 16-byte aligned */
    const int32_t *token_ordering;   /* [vocab]: n_centroids consecutive lists of
                                      * vocab / n_centroids token ids, list j the
                                      * candidates of centroid j */
    /* MTP_WQ_Q8_0 only (NULL otherwise): block scales of w_pre and w_post */
    const uint16_t *w_pre_scale, *w_post_scale;
} mtp_weights;

/* A read-only view of one target KV layer ([G4] sec. 5).  K and V share the
 * layout: element (b, kv head g, slot s, d) at b*stride_b + g*stride_h +
 * s*stride_t + d (elements of `wdtype`; d contiguous).  window == 0 reads
 * positions [0, kv_len[b]) (requires kv_len[b] <= cap, sink == 0); window
 * W > 0 reads the last W positions [lo, kv_len[b]), lo = max(0, kv_len[b] - W),
 * plus the attention sink [0, min(sink, lo)) ("opus-mtp-turbo: Track 1
 * report", item 2: the draft attention reads the first `sink` cells and the
 * window).  Storage: position t lives in slot t for t < sink and in slot
 * sink + (t - sink) % (cap - sink) from there on (a ring of `cap` slots when
 * sink == 0); requires W + sink <= cap.  K is stored after RoPE; V is used as
 * stored.  rope_theta is the RoPE base of the target layer type (applied to
 * the drafter's queries). */
typedef struct mtp_kv_view {
    const void *k, *v;
    int64_t stride_b, stride_h, stride_t;
    int32_t cap, window;
    float rope_theta;
    int32_t sink;
} mtp_kv_view;

/* sample_dist settings ([SP] item 4): repetition penalty (z > 0: z / r, else
 * z * r) and presence penalty (z - pres), once per distinct token of the
 * penalty set, then temperature, min-p (keep p >= min_p * p_max), top-p (keep
 * the shortest prefix, by probability desc / id asc, whose mass reaches
 * top_p), renormalising after each cut.  top_k must be 0 (off). */
typedef struct mtp_sample_params {
    float temp, top_p, min_p, rep_penalty, presence_penalty;
    int32_t top_k;
} mtp_sample_params;

/* The paged KV cache of one target layer.  Position t of sequence b lives in
 * slot t % page_size of page page_table[b * max_pages + t / page_size]; element
 * (page, kv head g, slot s, d) of k and of v at page*stride_p + g*stride_h +
 * s*stride_t + d (elements of kv_dtype, d contiguous).  Consecutive pages of
 * one sequence with stride_p == page_size * stride_t are a mtp_kv_view of the
 * same memory (window 0), which the drafters read.
 *   kv_dtype   MTP_DTYPE_F32, MTP_DTYPE_BF16, or MTP_DTYPE_E4M3: 8-bit codes,
 *              the value is code * k_scale[page * n_kv_heads + g] (v_scale
 *              for v), fp32 [n_pages, n_kv_heads], powers of two within
 *              [2^-40, 2^40] (what mtp_kv_append writes); an attended page
 *              with any other scale counts as absent
 *   head_dim   32, 64, 128, 256 or 512 (strides: multiples of 16 bytes, k and
 *              v 16-byte aligned)
 *   page_size  16, 32, 64, 128 or 256
 *   window, sink  window W > 0: a row at position p attends the last W
 *              positions (p - W, p] and the attention sink, positions
 *              [0, min(sink, p + 1 - W)), as in mtp_kv_view; window 0 (sink 0)
 *              attends [0, p].  Pages outside what is attended are not read
 *              and may be absent.
 *   rope_theta > 0: RoPE base, NeoX pairs (i, i + head_dim/2), of the keys on
 *              their way in and of the queries; 0: neither is rotated
 * An entry of page_table is a page in [0, n_pages); any other value means
 * that the page is absent. */
typedef struct mtp_kv_cache {
    void *k, *v;
    float *k_scale, *v_scale;      /* MTP_DTYPE_E4M3 only (NULL otherwise) */
    const int32_t *page_table;     /* [B, max_pages] */
    int64_t stride_p, stride_h, stride_t;
    int32_t n_pages, page_size, max_pages;
    int32_t n_kv_heads, head_dim, kv_dtype;
    int32_t window, sink;
    float rope_theta;
    int32_t pad_;
} mtp_kv_cache;

/* Q8_0 quantisation of a row-major fp32 matrix [rows, cols] on the host
 * ("opus-mtp-turbo: Track 1 report", item 3, ggml's Q8_0 rule): per block of
 * 32 consecutive weights of a row, d = max |w| / 127 (fp32), stored as
 * binary16 (round to nearest even); codes q = round(w * (1 / d)) in fp32,
 * halves away from zero, 0 when d = 0.  The weight a code stands for is
 * binary16(d) * q.  Host pointers: w [rows, cols], codes [rows, cols] int8,
 * scales [rows, cols / 32].  cols must be a multiple of 32 (MTP_ERR_ARG).
 * Synchronous, no device work. */
int mtp_quantize_q8_0(const float *w, int64_t rows, int64_t cols, int8_t *codes, uint16_t *scales);
/* Q4_0 quantisation on the host ("opus-mtp-turbo: Track 1 report", item 3,
 * the Q4_0 format; the scale by ggml's rule, where the report's quantiser
 * picks it by Lloyd iterations): per block of 32 consecutive weights of a row,
 * m = the weight of largest magnitude (the first on ties), d = m / -8 (fp32),
 * stored as binary16 (round to nearest even); codes q = min(15, trunc(w * (1 /
 * d) + 8.5)) in fp32, 8 when d = 0.  Host pointers: w [rows, cols], codes
 * [rows, cols / 2] uint8 (layout as for MTP_WQ_Q4_0), scales [rows, cols /
 * 32].  cols must be a multiple of 32 (MTP_ERR_ARG).  Synchronous, no device
 * work. */
int mtp_quantize_q4_0(const float *w, int64_t rows, int64_t cols, uint8_t *codes, uint16_t *scales);

/* Workspace bytes needed by any of the operations for these sizes (B
 * sequences, N drafts, vocabulary V).  cfg may be NULL when only the verify
 * and draw calls will use the workspace (then B <= MTP_MAX_VERIFY_BATCH,
 * else B <= MTP_MAX_BATCH).  Returns 0 for invalid sizes. */
size_t mtp_workspace_size(const mtp_config *cfg, int B, int N, int V);

/* N chained draft steps for B sequences ([G4] sec. 4-5, [NX], [FN]).
 * Step k of sequence b consumes token tok_k (last_tok[b] for k = 0, the draft
 * of step k-1 after) and hidden state h_k (h_prev[b] for k = 0, the previous
 * step's post-projection after):
 *   e = tok_embd[tok_k] * emb_scale
 *   x = w_pre [rmsnorm(e; norm_e); rmsnorm(h_k; norm_h)]
 *   per block: q = rope(qnorm(w_q rmsnorm(x)), pos = kv_len[b] + k);
 *              o = GQA softmax cross-attention of q into the block's view;
 *              x += rmsnorm(w_o o); x += rmsnorm(w_down(gelu_tanh(w_gate n) * w_up n)),
 *              n = rmsnorm(x; pre_ffn_norm)
 *   h_{k+1} = w_post rmsnorm(x; final_norm);  z = tok_embd h_{k+1} (softcap)
 *   (centroid-routed head, cfg->n_centroids > 0: z is -1e30 except at the
 *   candidates, the lists of the centroid_top_k centroids with the largest
 *   centroids[j] . h_{k+1} (lower j on ties), where z_t = tok_embd[t] h_{k+1}
 *   (softcap); an ordering entry outside [0, vocab) is skipped and sets the
 *   status word to MTP_ERR_ARG)
 *   draft_k = argmax z (lowest index on ties), or, when sp != NULL and
 *   sp->temp > 0, a draw from sample_dist(z) with penalty set hist[b] u
 *   {draft_0..draft_{k-1}} and the Philox-4x32-10 uniform of counter
 *   (b, 4k + 0, offset lo, offset hi), key (seed lo, seed hi).
 * Arguments:
 *   views[n_views]       KV views (host array of structs; data on device)
 *   kv_len [B] int32     attn_pos + 1 of each sequence, >= 1
 *   last_tok [B] int32   the last accepted token
 *   h_prev [B, d_t] fp32 the target's hidden state at that token
 *   sp                   host pointer or NULL (greedy); with temp > 0 the
 *                        settings are checked as for mtp_verify_sample
 *                        (MTP_ERR_ARG; top_k != 0: MTP_ERR_UNSUPPORTED), and
 *                        a kept set over 4096 candidates sets the status word
 *                        to MTP_ERR_CAPACITY
 *   hist [B, H] int32    penalty history (newest last; entries < 0 ignored);
 *                        used only when sampling; may be NULL when H == 0
 *   out_drafts [B, N] int32
 *   out_h_last [B, d_t] fp32, or NULL: h after the last step
 *   out_logits [B, N, vocab] fp32, or NULL: every step's logits (diagnostic)
 *   out_conf [B, N] fp32, or NULL: each step's confidence, the softmax
 *                        probability of its largest logit, 1 / sum_v
 *                        exp(z_v - max z) over the step's logits (after the
 *                        softcap, NaN left out) -- the draft loop's
 *                        confidence that [NX] "Stopping early when the head
 *                        is unsure" compares with p_min.  The caller trims a
 *                        row's drafts at the first step below its p_min
 *                        before verifying; the drafts themselves do not
 *                        depend on it.
 * B <= MTP_MAX_BATCH, 1 <= N <= 16.  One cooperative launch (plus a 256-byte
 * workspace memset); no host round-trip between steps. */
int mtp_draft_block(const mtp_config *cfg, const mtp_weights *w,
                    const mtp_kv_view *views, int n_views,
                    const int32_t *kv_len, int B, int N,
                    const int32_t *last_tok, const float *h_prev,
                    const mtp_sample_params *sp, uint64_t seed, uint64_t offset,
                    const int32_t *hist, int H,
                    int32_t *out_drafts, float *out_h_last, float *out_logits,
                    float *out_conf, void *ws, size_t ws_bytes, mtp_stream_t stream);

/* The dense NextN drafter ([NX] "Requirements", "How it is wired", "The
 * catch-up runs on the accepted prefix"; [FN] "The two MTP lanes": NextN runs
 * its own block over its own KV).  One block at the backbone width d = d_t.
 * The drafter's KV `dkv` holds kv_len[b] rows of sequence b, the row of
 * position t in slot t (window 0, sink 0, kv_len[b] + n_cu[b] + N <= cap);
 * this call WRITES rows kv_len[b] .. kv_len[b] + n_cu[b] + N - 1 of it.
 * A row consumes a token t at position pos and a hidden state h:
 *   x = w_pre [rmsnorm(tok_embd[t] * emb_scale; norm_e); rmsnorm(h; norm_h)]
 *       (w_pre the eh_proj [d, 2d]; emb_scale 0 = the default 1)
 *   a = rmsnorm(x; attn_norm);  [q; k; v] = w_q a  (w_q [(Hq + 2 Hkv) hd, d]:
 *       query rows, then key rows, then value rows)
 *   per KV head: key = rope(rmsnorm(k_g; k_norm), pos), value = v_g, both
 *       stored at slot pos rounded to wdtype
 * Catch-up rows stop there.  A draft step goes on:
 *   per query head: q_h = rope(rmsnorm(q_h; q_norm), pos) attends (GQA,
 *       scale attn_scale) to the rows [0, pos] of KV head h / (Hq / Hkv)
 *   x += w_o o;  x += w_down(silu(w_gate n) * w_up n), n = rmsnorm(x; pre_ffn_norm)
 *   h' = x (the next step's hidden state);  z = tok_embd rmsnorm(x; final_norm)
 *       (final_norm the shared head's norm; optional softcap); draft = argmax z
 *       (lowest index on ties)
 * Rows of sequence b: catch-up row j < n_cu[b] consumes (cu_tok[b, j],
 * cu_h[b, j]) at position kv_len[b] + j -- the accepted drafts with the
 * target's hidden states at the positions before them; draft step k consumes
 * (last_tok[b], h_prev[b]) for k = 0 -- the bonus token with the target's
 * hidden state before it -- and (draft k-1, h' of step k-1) after, at
 * position kv_len[b] + n_cu[b] + k.  The next call's kv_len is kv_len +
 * n_cu + 1: the rows of steps k >= 1 are the drafter's own guesses, and the
 * next call's catch-up rewrites the accepted ones (no rollback is needed).
 * Arguments:
 *   cfg        d_a == d_t, n_blocks == 1, n_centroids == 0; wquant NONE,
 *              Q8_0 or Q4_0 (then w_pre_scale and blk[0]'s w_q, w_o,
 *              w_gate, w_up, w_down scales are required); rope_theta comes
 *              from dkv
 *   w          tok_embd, norm_e, norm_h, w_pre (eh_proj), final_norm (head
 *              norm); blk[0]: attn_norm, w_q (fused), q_norm, k_norm, w_o,
 *              pre_ffn_norm, w_gate, w_up, w_down (w_post, post_attn_norm,
 *              post_ffn_norm, centroids and w_post_scale unused, may be NULL)
 *   dkv        host pointer to one view (data on device, written)
 *   kv_len [B] int32 >= 0;  n_cu [B] int32 in [0, M] (NULL: all 0)
 *   cu_tok [B, M] int32, cu_h [B, M, d] fp32 (only rows j < n_cu[b] are read;
 *              NULL when M == 0);  0 <= M <= MTP_MAX_CATCHUP
 *   last_tok [B] int32;  h_prev [B, d] fp32
 *   out_drafts [B, N] int32;  out_h_last [B, d] fp32 or NULL: h' of the last
 *              step;  out_logits [B, N, vocab] fp32 or NULL;  out_conf [B, N]
 *              fp32 or NULL (as for mtp_draft_block)
 * Greedy only ([NX]: speculation there requires greedy decoding).  B <=
 * MTP_MAX_BATCH, 1 <= N <= 16.  Host-checked arguments return MTP_ERR_ARG /
 * MTP_ERR_UNSUPPORTED; a kv_len, n_cu or token out of range sets the status
 * word to MTP_ERR_ARG and the kernel returns before writing anything.  One
 * cooperative launch (plus a 256-byte workspace memset). */
int mtp_nextn_draft(const mtp_config *cfg, const mtp_weights *w, const mtp_kv_view *dkv,
                    const int32_t *kv_len, int B, int N,
                    const int32_t *n_cu, const int32_t *cu_tok, const float *cu_h, int M,
                    const int32_t *last_tok, const float *h_prev,
                    int32_t *out_drafts, float *out_h_last, float *out_logits, float *out_conf,
                    void *ws, size_t ws_bytes, mtp_stream_t stream);
/* Greedy verify ([NX] How it is wired).  B <= MTP_MAX_VERIFY_BATCH.  logits [B, 1+N, V] in ldtype (row i
 * is the target's distribution after consuming the last token and drafts
 * 0..i-1); t_i = argmax of row i (lowest index on ties, NaN never wins, an
 * all-NaN row gives 0).  n_accept[b] = the largest k <= N with
 * drafts[b, j] == t_j for all j < k; out_tokens[b] = drafts[b, 0..k-1], t_k,
 * then -1 up to 1+N entries.  drafts [B, N] int32, out_tokens [B, 1+N] int32,
 * out_n_accept [B] int32.  0 <= N, B >= 1, V >= 1. */
int mtp_verify_greedy(const void *logits, int ldtype, int B, int N, int V,
                      const int32_t *drafts, int32_t *out_tokens, int32_t *out_n_accept,
                      void *ws, size_t ws_bytes, mtp_stream_t stream);

/* Exact speculative sampling ([SP] item 4), B <= MTP_MAX_VERIFY_BATCH
 * sequences.  For row i < N of sequence b:
 * p_i = sample_dist(target row i), q_i = sample_dist(draft row i), both with
 * penalty set hist[b] u {drafts[b, 0..i-1]}; x = drafts[b, i] is accepted iff
 * u < p_i(x) / q_i(x) (u of counter (b, 4i + 1, ...)).  At the first
 * rejection the emitted token is drawn from norm(max(p_i - q_i, 0)) (from p_i
 * if that is empty) with u of (b, 4i + 2, ...) and the window ends; when all
 * N drafts are accepted the bonus token is drawn from p_N with u of
 * (b, 4N + 3, ...).  Draws walk the candidates in (probability desc, id asc)
 * order.  Uniforms: Philox-4x32-10, counter (b, 4i + purpose, offset lo,
 * offset hi), key (seed lo, seed hi), u = (word0 >> 8) * 2^-24.
 *   tgt_logits [B, 1+N, V], dft_logits [B, N, V] in ldtype; drafts [B, N];
 *   hist [B, H] int32 (newest last, entries < 0 ignored; NULL when H == 0);
 *   sp host pointer (temp > 0, top_k == 0); out_tokens [B, 1+N] (-1 padded);
 *   out_n_accept [B].  sample_dist's weights are exp(l - lmax) rounded once
 *   to fp32 (the exponential in fp64); every other step feeding a decision
 *   is IEEE fp32 in the order written above, sums sequential in (w desc,
 *   id asc) order.  A row whose min-p set exceeds 4096 candidates sets
 *   MTP_ERR_CAPACITY in the status word.  One launch (plus a memset of the
 *   workspace's counters); one pass over the logits. */
int mtp_verify_sample(const void *tgt_logits, const void *dft_logits, int ldtype,
                      int B, int N, int V, const int32_t *drafts,
                      const int32_t *hist, int H, const mtp_sample_params *sp,
                      uint64_t seed, uint64_t offset,
                      int32_t *out_tokens, int32_t *out_n_accept,
                      void *ws, size_t ws_bytes, mtp_stream_t stream);

/* Draws of a sampling drafter ([SP] item 4: the token drafted at window
 * position i is a draw from q_i = sample_dist(draft row i)).  For every
 * sequence b and i = 0..N-1 in order: q_i = sample_dist(dft_logits[b, i]) with
 * penalty set hist[b] u {out_drafts[b, 0..i-1]}, and out_drafts[b, i] = the
 * inverse-CDF pick of q_i with the uniform of counter (b, 4i + 0, offset lo,
 * offset hi), key (seed lo, seed hi) -- the same draw mtp_draft_block makes
 * at temp > 0, so mtp_verify_sample can then check these drafts exactly.
 *   dft_logits [B, N, V] in ldtype; hist [B, H] int32 (NULL when H == 0);
 *   sp host pointer (as for mtp_verify_sample); out_drafts [B, N] int32.
 * 1 <= N <= 16, B <= MTP_MAX_VERIFY_BATCH.  N launches (window position i
 * depends on the draws before it) plus one workspace memset. */
int mtp_sample_drafts(const void *dft_logits, int ldtype, int B, int N, int V,
                      const int32_t *hist, int H, const mtp_sample_params *sp,
                      uint64_t seed, uint64_t offset, int32_t *out_drafts,
                      void *ws, size_t ws_bytes, mtp_stream_t stream);

/* Workspace bytes of mtp_kv_append and mtp_paged_attention on this cache for at
 * most B sequences of at most M rows each (beyond MTP_MAX_ATTN_ROWS only
 * appended) and n_q_heads query heads.  Returns 0 for invalid sizes. */
size_t mtp_kv_workspace_size(const mtp_kv_cache *c, int B, int M, int n_q_heads);

/* Append rows to the cache: row j < n_new[b] of sequence b goes to position
 * kv_len[b] + j as key = rope(rmsnorm(k_j; k_norm)), value = v_j (per KV head;
 * the norm only where k_norm is given, the rotation where rope_theta > 0), each
 * rounded once to kv_dtype, nearest even.
 *   k, v       rows in in_dtype (F32 or BF16): row (b, j, kv head g) at
 *              b*in_stride_b + j*in_stride_m + g*in_stride_h (elements; 16-byte
 *              multiples, 16-byte aligned), head_dim contiguous -- slices of a
 *              fused projection's output, for example
 *   kv_len [B] int32 >= 0: positions already cached;  n_new [B] int32 in
 *              [0, M] (NULL: all M);  kv_len + n_new <= max_pages * page_size
 *   k_norm     fp32 [head_dim] or NULL;  rms_eps its epsilon
 * MTP_DTYPE_E4M3: the scale of a (page, KV head) is the smallest power of two s
 * with max |x| <= 448 s over this call's finite values in it, at least 2^-40
 * and at most 2^40 (larger values saturate), and at least the scale it has if
 * the page already holds positions of the sequence (slot kv_len % page_size >
 * 0): its older codes are then re-rounded to the larger scale.  A page whose
 * first slot is written starts anew.  NaN and infinities are stored as NaN.
 * Slots behind the last row keep their bytes.  The pages that one call writes
 * must be distinct between sequences.
 * A sequence whose kv_len or n_new is out of range is left out, rows whose
 * page is absent are dropped, and both set the status word to MTP_ERR_ARG.
 * 1 <= B <= MTP_MAX_PAGED_BATCH, 1 <= M <= MTP_MAX_APPEND_ROWS.  One launch. */
int mtp_kv_append(const mtp_kv_cache *c, int B, int M, const int32_t *kv_len, const int32_t *n_new,
                  const void *k, const void *v, int in_dtype,
                  int64_t in_stride_b, int64_t in_stride_m, int64_t in_stride_h,
                  const float *k_norm, float rms_eps, void *ws, size_t ws_bytes, mtp_stream_t stream);

/* Attention of the appended rows over the cache: row j < n_new[b] of sequence
 * b, at position p = kv_len[b] + j, query head h (KV head h / (n_q_heads /
 * n_kv_heads)):
 *   q' = rope(rmsnorm(q; q_norm), p)   (norm and rotation as for the keys)
 *   out = sum_t softmax_t(attn_scale q' . k_t) v_t  over the positions t that
 *         p attends (see mtp_kv_cache); kv_len is the length BEFORE the rows,
 *         whose keys and values are in the cache already (mtp_kv_append)
 *   q          rows in dtype (F32 or BF16): row (b, j, head h) at b*q_stride_b
 *              + j*q_stride_m + h*q_stride_h (elements; 16-byte multiples,
 *              16-byte aligned)
 *   q_norm     fp32 [head_dim] or NULL;  rms_eps its epsilon
 *   attn_scale 0 = the default 1/sqrt(head_dim)
 *   out [B, M, n_q_heads, head_dim] in dtype; rows j >= n_new[b] keep their
 *              bytes
 * fp32 queries are computed in fp32 throughout.  bf16 queries against a bf16
 * or e4m3 cache with head_dim 64, 128, 256 or 512 run on the tensor cores: the
 * rotated queries then keep 16 bits (bf16 cache) or 12 (e4m3 cache), the
 * probabilities 16 or 9, sums and maxima 32.  Against e4m3 what keeps 9 bits is
 * a probability times its page's value scale, down to 2^-19 of the row's
 * largest; below it keeps fewer, and none under 2^-28.
 * Slots that hold no attended position are never used, whatever they contain.
 * An attended value that is infinite gives that infinity in its dimension, NaN
 * or infinities of both signs give NaN; other dimensions and rows that do not
 * attend it are not touched.  An attended key that is not finite may make the
 * row's outputs NaN.
 * A row that attends nothing (all its pages absent) gives zeros.  A sequence
 * whose kv_len or n_new is out of range is left out, positions on absent pages
 * are masked, and both set the status word to MTP_ERR_ARG.
 * 1 <= B <= MTP_MAX_PAGED_BATCH, 1 <= M <= MTP_MAX_ATTN_ROWS, at most 16
 * query heads per KV head.  Two launches. */
int mtp_paged_attention(const mtp_kv_cache *c, int B, int M, int n_q_heads, const int32_t *kv_len,
                        const int32_t *n_new, const void *q, int dtype,
                        int64_t q_stride_b, int64_t q_stride_m, int64_t q_stride_h,
                        const float *q_norm, float rms_eps, float attn_scale, void *out,
                        void *ws, size_t ws_bytes, mtp_stream_t stream);

/* Rows normed and rotated by several positions, for targets whose tokens have a
 * place in time, height and width: row t, head h (queries and, where k is given,
 * keys; each with its own norm),
 *   y = rope(rmsnorm(x; norm)), the norm only where it is given; with P = the sum
 *       of sections, the pairs (i, i + P), i < P, turn by
 *       positions[axis(i), t] * theta^(-i / P), dimensions from 2 P on are not
 *       turned
 *   interleaved 0: axis(i) is the section that holds i (the sections one after
 *       another); otherwise axis(i) = i mod n_axes while i < n_axes *
 *       sections[i mod n_axes], else 0
 * rounded once to dtype.  The rows then go to a cache with rope_theta 0
 * (mtp_kv_append without k_norm) and attend it without q_norm.  The drafters
 * (mtp_draft_block, mtp_nextn_draft) rotate by the slot: behind an image, where a
 * target's next position is not its next slot, they do not follow these positions.
 *   positions  int32 [n_axes, rows], any sign
 *   sections   HOST pointer, [n_axes] >= 0; P a multiple of 8, 2 P <= head_dim
 *   q, k       rows in dtype (F32 or BF16): row (t, head h) at t*stride_m +
 *              h*stride_h (elements; 16-byte multiples, 16-byte aligned),
 *              head_dim (32, 64, 128, 256 or 512) contiguous; k NULL: queries
 *              alone
 *   out_q, out_k  the same with their own strides.  An output may be its input
 *              (the same address and strides); else it overlaps no input
 *   q_norm, k_norm  fp32 [head_dim] or NULL;  rms_eps their epsilon
 * 1 <= rows <= MTP_MAX_PROMPT_ROWS, 1 <= n_axes <= MTP_MAX_AXES, theta > 0.  One
 * launch, no workspace. */
int mtp_rotate_axes(int64_t rows, int n_axes, const int32_t *positions, const int32_t *sections, int interleaved,
                    float theta, int head_dim, int dtype,
                    const void *q, int n_q_heads, int64_t q_stride_m, int64_t q_stride_h,
                    const void *k, int n_k_heads, int64_t k_stride_m, int64_t k_stride_h,
                    const float *q_norm, const float *k_norm, float rms_eps,
                    void *out_q, int64_t out_q_stride_m, int64_t out_q_stride_h,
                    void *out_k, int64_t out_k_stride_m, int64_t out_k_stride_h, mtp_stream_t stream);

/* Workspace bytes of mtp_prompt_attention on this cache for at most B sequences
 * with at most T rows in all, and of mtp_prefix_attention for at most B sequences
 * of at most M rows.  0 for invalid sizes. */
size_t mtp_prompt_workspace_size(const mtp_kv_cache *c, int B, int64_t T, int n_q_heads);
size_t mtp_prefix_workspace_size(const mtp_kv_cache *c, int B, int M, int n_q_heads);

/* Attention of whole prompts (or pieces of them) over the cache: the rows of B
 * sequences lie one after another, sequence b's are rows [row_start[b],
 * row_start[b + 1]) of T; row row_start[b] + j, at position kv_len[b] + j, attends
 * as a row of mtp_paged_attention does (norm, rotation, scale, window and sink,
 * absent pages, values that are not finite).  The keys and values of all rows are
 * in the cache already.
 *   kv_len [B] int32: positions cached before the rows
 *   row_start [B + 1] int32, ascending, within [0, T]; rows of no sequence (in
 *              front of row_start[0], behind row_start[B]) keep their bytes.
 *              Where it does not ascend, a sequence is left out unless all bounds
 *              in front of its rows are at most row_start[b] and all behind them
 *              at least row_start[b + 1]: rows that two would claim are no one's
 *   q          rows in dtype (F32 or BF16): row (t, head h) at t*q_stride_m +
 *              h*q_stride_h (elements; 16-byte multiples, 16-byte aligned)
 *   out [T, n_q_heads, head_dim] in dtype, 16-byte aligned; it overlaps no input
 * fp32 queries or caches and head_dim 32 and 512 are computed in fp32 throughout,
 * a row at a time (slower by two orders of magnitude).  bf16 queries against a bf16
 * or e4m3 cache with head_dim 64, 128 or 256 run on the tensor cores: against bf16,
 * rotated queries and probabilities are then rounded to bf16 (8 bits, half of what
 * mtp_paged_attention keeps); against e4m3 both to fp16: a query's elements to 11
 * bits down to 2^-21 of their row's largest (below, to 2^-32 of it), and of the
 * probabilities each times its page's value scale, to 11 bits down to 2^-25 of the
 * row's largest such product (below, to 2^-36 of it).  Maxima, sums and accumulators
 * are fp32.
 * A sequence whose kv_len or rows are out of range is left out, positions on
 * absent pages are masked, and both set the status word to MTP_ERR_ARG.
 * 1 <= B <= MTP_MAX_PAGED_BATCH, 1 <= T <= MTP_MAX_PROMPT_ROWS, T * n_q_heads <
 * 2^31, at most 16 query heads per KV head. */
int mtp_prompt_attention(const mtp_kv_cache *c, int B, int64_t T, int n_q_heads, const int32_t *kv_len,
                         const int32_t *row_start, const void *q, int dtype, int64_t q_stride_m, int64_t q_stride_h,
                         const float *q_norm, float rms_eps, float attn_scale, void *out,
                         void *ws, size_t ws_bytes, mtp_stream_t stream);

/* Attention of the new rows of sequences that share prefixes: as
 * mtp_paged_attention, but the sequences [group_start[i], group_start[i + 1]) have
 * their positions [0, prefix_len[i]) in common, on the pages of sequence
 * group_start[i]'s row of page_table (the other sequences' entries for whole pages
 * of it are not read).  On the tensor cores a group's prefix is read and computed
 * once for 256 of its rows of a KV head, and every sequence's own positions
 * [prefix_len[i], kv_len + j] for itself; fp32 queries or caches and head_dim 32
 * and 512 read the prefix for every row.
 * It pays where many sequences read a long prefix: measured from 8 sequences on
 * behind 32768 positions, 16 behind 8192, 32 to 128 behind 2048, none behind 512.
 * Where it does not, mtp_paged_attention with the prefix's pages in every row of
 * page_table takes down to half the time, and it keeps more bits of queries and
 * probabilities over a bf16 cache.
 *   kv_len [B] int32 >= prefix_len of its group: the prefix counts;  n_new [B] or
 *              NULL, q, q_norm, attn_scale, out: as for mtp_paged_attention
 *   group_start [n_groups + 1] int32, ascending, within [0, B]; sequences of no
 *              group have no prefix
 *   prefix_len [n_groups] int32 >= 0, of any length (a prefix may end inside a page)
 * The cache's window must be 0 (MTP_ERR_UNSUPPORTED otherwise: a sliding layer's
 * rows attend few positions of a long prefix, and mtp_paged_attention reads only
 * those).  Types and roundings as for mtp_prompt_attention.
 * A sequence whose kv_len, n_new, prefix_len or group is out of range is left out
 * (all of them are where group_start does not ascend), positions on absent pages
 * are masked, and both set the status word to MTP_ERR_ARG.
 * 1 <= B <= MTP_MAX_PAGED_BATCH, 1 <= M <= MTP_MAX_ATTN_ROWS, 0 <= n_groups <= B,
 * at most 16 query heads per KV head, B * (max_pages * page_size / 128 + 2) <
 * 2^31. */
int mtp_prefix_attention(const mtp_kv_cache *c, int B, int M, int n_q_heads, const int32_t *kv_len, const int32_t *n_new,
                         int n_groups, const int32_t *group_start, const int32_t *prefix_len,
                         const void *q, int dtype, int64_t q_stride_b, int64_t q_stride_m, int64_t q_stride_h,
                         const float *q_norm, float rms_eps, float attn_scale, void *out,
                         void *ws, size_t ws_bytes, mtp_stream_t stream);

/* Log probabilities of given tokens: for row r of logits [rows, V] in ldtype
 * (rows row_stride elements apart), with lse = log sum_v exp z_v,
 *   out_logprob[r]  = z_t - lse, t = tokens[r]
 *   out_entropy[r]  = -sum_v p_v log p_v (natural), p = exp(z - lse)
 *   out_top_ids / out_top_logprobs [rows, top_k]: the largest logits with
 *                     their z - lse, by value descending, lowest index first
 *                     on ties; -1 and -inf behind the last one
 * NaN logits are left out as if they were -inf; -inf is never an alternative.
 * A row with a +inf logit, or with nothing above -inf, gives NaN log
 * probabilities and entropy.  A row whose logits do not reach the kernel within
 * a second gives NaN, and -1 for every alternative.  A row whose token is outside
 * [0, V) (the -1 padding of a verify's out_tokens) is not read and its
 * outputs keep their values; tokens NULL: every row, out_logprob not written.
 * Each output may be NULL (top_k 0: both alternatives' arrays unused).
 * 1 <= rows <= 17 * MTP_MAX_VERIFY_BATCH, 0 <= top_k <= MTP_MAX_TOP, V >= 1,
 * row_stride >= V.  One launch, no workspace. */
int mtp_token_logprobs(const void *logits, int ldtype, int64_t rows, int V, int64_t row_stride,
                       const int32_t *tokens, int top_k, float *out_logprob, float *out_entropy,
                       int32_t *out_top_ids, float *out_top_logprobs, mtp_stream_t stream);

/* Greedy verify without a workspace.  The pages have no counterpart of this
 * call; it exists for callers that may not allocate device memory at all --
 * for example a serving loop that has already handed every byte of the GPU to
 * its weights and KV cache and forbids further allocations, or code that must
 * not call cudaMalloc because it can synchronize the device in the middle of a
 * decode step.  Same arguments, results and errors as mtp_verify_greedy, minus
 * `ws` / `ws_bytes`: the scratch is a 4 KiB array built into the library (held
 * on every GPU that loads it until the process exits), so B * (1 + N) may be
 * at most 480; larger sizes return MTP_ERR_UNSUPPORTED and launch nothing.
 * Allocates nothing.  The first call on a device looks up the array's device
 * address (with that device current); make that first call before any stream
 * capture.  All calls share the one array and every call clears it first, so
 * calls that may overlap on the GPU (different streams, or several host
 * threads) race and must be serialized by the caller.  The looked-up address
 * is kept for the life of the process: do not use this call on a device after
 * cudaDeviceReset() in the same process. */
int mtp_verify_greedy_noalloc(const void *logits, int ldtype, int B, int N, int V,
                              const int32_t *drafts, int32_t *out_tokens, int32_t *out_n_accept,
                              mtp_stream_t stream);

/* Device status of the most recent call that used `ws`: MTP_OK,
 * MTP_ERR_TIMEOUT or MTP_ERR_CAPACITY.  SYNCHRONIZES `stream` (a 4-byte
 * device-to-host copy).  Returns MTP_ERR_CUDA if the copy fails. */
int mtp_last_error(const void *ws, mtp_stream_t stream);

/* Static description of an error code. */
const char *mtp_strerror(int code);

/* Fault-detection check: launches the grid barrier of the draft kernel with
 * an arrival count that can never be reached and a wait limit of
 * `timeout_us` microseconds (1..1000000).  Every block gives up, the status
 * word becomes MTP_ERR_TIMEOUT and the kernel returns; the context stays
 * usable.  For tests of the timeout path; computes nothing. */
int mtp_debug_barrier_timeout(void *ws, size_t ws_bytes, int timeout_us, mtp_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MTP_H */
