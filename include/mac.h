/*
 * mac.h -- C ABI of the MAC-Attention per-step decode-attention library
 * (libmac_gb300.so, hand-written CUDA for GB300 / sm_103a).
 *
 * The method (sources cited per entry point below):
 *   [MAC]  "MAC-Attention: Match-Amend-Complete attention reuse, up to 99% fewer
 *          KV reads in long-context decoding (MLSys 2026)", pinghaoyang.com.cn
 *   [MACS] "MAC-Attention: A Match-Amend-Complete Scheme for Fast and Accurate
 *          Attention Computation (MLSys 2026)", awesome-system-papers summary
 *   [ACSP] "Attention Cache and Sequence Parallelism", shaojiemike.top
 *
 * Conventions shared by every entry point
 *   - Positions are 1-based.  For request b, m = seq_len[b] is the current
 *     length and the K/V of position m is already in the cache: the caller
 *     writes K/V, keys already rotated by RoPE ([ACSP] MHA decode pseudo-code).
 *   - Query head h reads KV head h / (Hq/Hkv) ([ACSP] repeat_kv).
 *   - Every pointer argument is a DEVICE pointer unless stated otherwise; the
 *     caller owns all memory.  The library never allocates device memory.
 *     It owns two CUDA events per ring workspace (created on first use,
 *     destroyed by mac_release_ring).
 *   - Every call is asynchronous on the given stream(s) and returns a status
 *     code: MAC_OK, or a negative MAC_ERR_* for an invalid argument, an
 *     unsupported configuration or a CUDA launch error; nothing was enqueued
 *     when the return value is negative.  Errors that depend on device data
 *     (bad lengths or page ids, a bounded wait that gave up) never fault: the
 *     kernels skip the offending work, write zeros for it, and set bits of a
 *     device status word read by mac_last_status.
 *   - Buffers must be 16-byte aligned (K/V, queries, rings) and do not alias.
 */
#ifndef MAC_H_
#define MAC_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* ---- status codes (return values) --------------------------------------- */
#define MAC_OK 0
#define MAC_ERR_INVALID_ARG (-1)   /* NULL pointer, bad size, misaligned buffer */
#define MAC_ERR_UNSUPPORTED (-2)   /* configuration the kernels do not cover */
#define MAC_ERR_CUDA (-3)          /* a CUDA runtime call or launch failed */

/* ---- device status bits (mac_last_status) ------------------------------- */
#define MAC_DEV_BAD_SEQ_LEN 0x1    /* m < 1 or m beyond the cache: request skipped, output 0 */
#define MAC_DEV_BAD_PAGE 0x2       /* page id outside [0, n_pages): its tokens skipped */
#define MAC_DEV_WAIT_TIMEOUT 0x4   /* a bounded wait on a copy gave up: item skipped */
#define MAC_DEV_NONFINITE_Q 0x8    /* non-finite query: treated as a miss */
#define MAC_DEV_BAD_COPY 0x10      /* a copy outside its tile was refused (internal check) */
#define MAC_DEV_NO_ROOM 0x20       /* free pages or token rows ran out: request not admitted */
#define MAC_DEV_BAD_PARENT 0x40    /* a slot's parent outside its group: the slot keeps what it has */
#define MAC_DEV_NONFINITE_LOGIT 0x80 /* NaN or +inf among a beam's logits, or in its score: no candidates of it */

/* ---- configuration ------------------------------------------------------ */
enum { MAC_BF16 = 0, MAC_F32 = 1 };
/* Threshold reading: [MAC] "Match (2)" accepts ||q~_m - q~_p|| < (1-tau) sqrt(2d)
 * (d=128, tau=0.45 -> 8.8; larger tau is stricter); [MACS] writes
 * tau sqrt(2d).  Both are offered; the first is the default. */
enum { MAC_THR_ONE_MINUS_TAU = 0, MAC_THR_TAU = 1 };
/* RoPE pairing of the query rotation R(m): half-split (j, j+d/2), interleaved
 * (2j, 2j+1), or none.  Frequencies base^(-2j/d), angle (m-1) w_j. */
enum { MAC_ROPE_HALF = 0, MAC_ROPE_INTERLEAVED = 1, MAC_ROPE_NONE = 2 };

typedef struct {
  int32_t batch;       /* B: request slots */
  int32_t n_q_heads;   /* Hq */
  int32_t n_kv_heads;  /* Hkv; Hq/Hkv in {1, 2, 4, 8} */
  int32_t head_dim;    /* d; 128 */
  int32_t ring_k;      /* K: ring capacity = candidate window [m-K, m-1] ([MAC] "Match (3)") */
  int32_t band_r;      /* r: rectification band ([MAC] "Amend"); r >= 0 */
  double tau;          /* match threshold parameter ([MAC] "Match (2)") */
  int32_t thr_mode;    /* MAC_THR_* */
  double rope_base;    /* RoPE base, e.g. 10000 */
  int32_t rope_mode;   /* MAC_ROPE_* */
  int32_t dtype;       /* MAC_BF16 | MAC_F32: element type of queries, ring queries, K, V */
  int32_t page_size;   /* 0 = contiguous K/V; 16 = paged K/V */
  int32_t min_context; /* steps with m < min_context never reuse ([MAC] production defaults) */
  int64_t max_context; /* largest m any call will see; sizes the scratch workspace */
  int32_t front_sink;  /* F >= 0: front-sink isolation ([MAC] "Production version"): tokens
                          [1, F] stay out of the reused summaries (seeded and appended) and
                          are attended exactly at every decode step; 0 = none; negative:
                          MAC_ERR_INVALID_ARG, above 2^30 - 1: MAC_ERR_UNSUPPORTED */
} mac_config;

/* K/V cache.  Contiguous (page_size 0): k, v are [B][Hkv][capacity][d].
 * Paged (page_size 16): k, v are [n_pages][Hkv][16][d] and page_table is
 * [B][max_pages] int32 (device); token t of request b lives in page
 * page_table[b][(t-1)/16], row (t-1)%16. */
typedef struct {
  const void *k;
  const void *v;
  const int32_t *page_table;
  int64_t capacity;  /* contiguous only: tokens per (b, kv-head) block */
  int32_t max_pages; /* paged only */
  int32_t n_pages;   /* paged only: physical pages (bounds check) */
} mac_kv;

/* Where the requests' tokens live, for mac_build_tables.  Paged: the table
 * and page count of the cache (as in mac_kv) and a stack of free page ids,
 * entries [0, *n_free_in) of free_pages, the last one on top.  Contiguous:
 * capacity only. */
typedef struct {
  int32_t *page_table;      /* paged: [B][max_pages], extended in place */
  int32_t *free_pages;      /* paged: [n_pages] */
  const int32_t *n_free_in; /* paged: one int32, entries of the stack before the call */
  int32_t *n_free_out;      /* paged: one int32, entries after it (may be n_free_in) */
  int64_t capacity;         /* contiguous only: tokens per (b, kv-head) block */
  int32_t max_pages;        /* paged only */
  int32_t n_pages;          /* paged only: physical pages */
} mac_pages;

/* Byte offsets of the parts of a ring workspace (for inspection/snapshots). */
typedef struct {
  size_t pos;        /* int32 [B][K]: position held by each slot, 0 = empty */
  size_t q;          /* dtype [B][Hq][K][d]: pre-RoPE query ring */
  size_t o;          /* f32 [B][Hq][K][d]: rectified summaries, normalised (S/Z) */
  size_t lse;        /* f32 [B][Hq][K]: their natural-log LSE (running max + ln Z) */
  size_t stage_q;    /* dtype [B][Hq][d]: this step's pre-RoPE query, for the append */
  size_t stage_o;    /* f32 [B][Hq][d]: this step's AS_{1:m-r}, normalised */
  size_t stage_lse;  /* f32 [B][Hq]: its LSE */
  size_t ctl;        /* the running step's match state (GQA groups up to 4): uint32 step
                        count, uint32 [2] chunk counters, uint64 [2][B][Hq] per-head minima
                        (the step count's parity selects the copy in use) */
  size_t total;      /* bytes */
} mac_ring_layout;

/* ---- entry points ------------------------------------------------------- */

/* Workspace sizes for cfg.  ring_bytes: one per layer (the two per-request
 * rings of capacity K, [MAC] "Paper version: K1/K2/K3": a pre-RoPE query
 * ring and a rectified-summary ring with its ln-LSE, plus a small staging
 * area).  scratch_bytes: shared by all calls on one stream (per-head match
 * minima, split-K piece partials, grid-barrier counter, device status word);
 * it must be zero-filled before its first use (mac_init_rings does it).  Its
 * size does not depend on the context length.  Either pointer may be NULL.
 * Returns MAC_ERR_INVALID_ARG / MAC_ERR_UNSUPPORTED for a bad cfg. */
int mac_workspace_size(const mac_config *cfg, size_t *ring_bytes, size_t *scratch_bytes);

/* Offsets of the ring workspace parts for cfg. */
int mac_ring_layout_of(const mac_config *cfg, mac_ring_layout *layout);

/* Reset the rings and scratch; optionally seed them.  q_seed == NULL: every
 * slot is emptied and all requests miss until decode steps fill the rings
 * (requests whose rings are not ready fall back to exact attention, [MAC]
 * "Production version").  q_seed != NULL: [B][Hq][n_seed][d] pre-RoPE queries
 * of positions L-n_seed+1 .. L with L = prompt_len[b] (device int32 [B]);
 * slot p mod K receives position p, its query and the exact rectified
 * summary AS_{1:p-r} of R(p) q_seed over the prompt K/V -- the state exact
 * decoding of those positions would have left ([MACS] "Design trade-offs":
 * prefill stays on the exact path).  n_seed <= K; positions < 1 are skipped.
 * Enqueued on stream (NULL = default stream). */
int mac_init_rings(const mac_config *cfg, void *ring_ws, void *scratch_ws, const void *q_seed,
                   const int32_t *prompt_len, int32_t n_seed, const mac_kv *kv, void *stream);

/* One MAC decode step for all B requests and Hq heads ([MAC] "Paper version:
 * K1/K2/K3", [MACS] "Core method"):
 *   Match     ring L2 nearest neighbour of the pre-RoPE query q_pre[b][h]
 *             (dtype [B][Hq][d]) among slots with position in [m-K, m-1];
 *             hit iff min ||q~_m - q~_c||^2 < thr^2 (thr per cfg.thr_mode,
 *             rounded to fp32); ties go to the most recent position.
 *   Complete  a hit at p attends q_m = R(m) q~_m over [p-r+1, m] only and
 *             merges it in log domain with the cached summary AS_{1:p-r};
 *             a miss attends over [1, m] (split-K full attention).
 *   Append    on stream_aux after an event: slot m mod K <- (m, q~_m,
 *             AS_{1:m-r}), where AS_{1:m-r} = cached part (+) fresh tokens up
 *             to m-r (the rectified summary; the band and tail are
 *             accumulated separately, so no log-domain subtraction is needed).
 * out: f32 [B][Hq][d] attention output.  match_pos: int32 [B][Hq] matched
 * position, -1 on a miss (may be NULL).  stream_aux NULL: the step kernel
 * writes the rings' slot itself once it has merged a head (the match has
 * read the rings before that), so there is no second kernel and no event.
 * stream_aux == stream_main: the append kernel runs on stream_main after the
 * step.  Another stream: the append kernel runs there after an event, and
 * the next step on the same ring_ws makes stream_main wait for it; a
 * captured CUDA graph must then call mac_join_aux before its capture ends.
 * The three give bitwise identical rings and outputs. */
int mac_decode_step(const mac_config *cfg, void *ring_ws, void *scratch_ws, const void *q_pre,
                    const int32_t *seq_len, const mac_kv *kv, float *out, int32_t *match_pos,
                    void *stream_main, void *stream_aux);

/* Exact split-K decode attention over [1, m] for every (b, h): the miss
 * fallback as a call of its own ([MAC] "Match (1)": a miss reproduces full
 * attention; [ACSP] MHA decode).  The query is rotated by R(m).  out: f32
 * [B][Hq][d]; lse: f32 [B][Hq] natural-log softmax denominator, or NULL.
 * Uses the same chunking and merge order as a decode step in which every
 * head misses, so such a step's output is bitwise equal to this call's; a
 * missing head in a step where others hit attends the same tokens with a
 * chunking that depends on the other units' bands (equal to rounding).  The
 * config's front_sink is ignored (attention over [1, m] is exact either way;
 * with F > 0 a decode step's miss equals this call to rounding). */
int mac_full_attention(const mac_config *cfg, void *scratch_ws, const void *q_pre,
                       const int32_t *seq_len, const mac_kv *kv, float *out, float *lse,
                       void *stream);

/* Largest scratch workspace mac_full_attention_noalloc can use (16 MiB). */
#define MAC_NOALLOC_SCRATCH_BYTES ((size_t)16 << 20)

/* mac_full_attention without a caller-provided scratch workspace.  (The
 * pages have no counterpart; this is a packaging variant.)  For callers that
 * cannot allocate device memory: code whose device memory is owned by
 * another allocator it may not call into, code that must not trigger the
 * device-wide synchronisation cudaMalloc can cause, or code running under a
 * fixed memory budget decided at start-up.  The scratch lives in a 16 MiB
 * array compiled into this library (MAC_NOALLOC_SCRATCH_BYTES); every GPU
 * that loads the library holds that array until the process exits.
 *   - Same arguments and results as mac_full_attention, minus scratch_ws.
 *   - Returns MAC_ERR_UNSUPPORTED, without enqueueing anything, when the
 *     configuration's scratch (mac_workspace_size) exceeds
 *     MAC_NOALLOC_SCRATCH_BYTES.
 *   - Allocates nothing: no cudaMalloc/cudaFree and no allocating library
 *     call.  The first call on a device looks up the array's device address
 *     (once per device, with that device current); make that first call
 *     before any stream capture.
 *   - Every call on a device shares the one array.  Each call clears the
 *     array's counters on its stream before launching, so calls on one
 *     stream are fine; calls that overlap on the GPU (different streams, or
 *     different host threads without ordering) race on the array and give
 *     wrong results.  The device status word of these calls is cleared by
 *     the next call and is not readable through mac_last_status. */
int mac_full_attention_noalloc(const mac_config *cfg, const void *q_pre, const int32_t *seq_len,
                               const mac_kv *kv, float *out, float *lse, void *stream);

/* ---- batches of new tokens ----------------------------------------------
 * A step that brings new tokens into the cache (prompts, chunks of prompts,
 * or one token per request ahead of a decode step) is three calls on one
 * stream: mac_build_tables lays the tokens out, mac_write_kv rotates and
 * stores them, mac_chunk_attention attends them.  ([MAC] "Production
 * version" keeps prefill on the exact path and the cache in pages; the
 * pages describe neither call, so the interfaces are this library's own.)
 *
 * The batch is n_tokens packed rows, in request order: request b's new
 * tokens are rows q_start[b] .. q_start[b+1] - 1, and rows from q_start[B]
 * on belong to nobody (a captured graph keeps n_tokens fixed while the
 * device arrays change).  chunk_ws: a workspace of
 * mac_chunk_workspace_size bytes, zero-filled before its first use, for one
 * stream at a time (two graphs that may run at once need one each); its
 * device status word is read by mac_last_status(cfg, chunk_ws, ..). */

/* Bytes of chunk_ws for batches of up to n_tokens rows.  Does not depend on
 * the context length. */
int mac_chunk_workspace_size(const mac_config *cfg, int32_t n_tokens, size_t *chunk_bytes);

/* Page tables, slots and positions of a batch, from its lengths alone, on
 * the device.  Request b holds len_in[b] tokens and brings new_len[b] >= 0.
 *   reset_flags (device int32 [B] or NULL): a request whose flag is set
 *     first gives its ceil(len_in/16) pages back and starts at length 0: in
 *     order of request and page they go on top of the stack.  The flags
 *     are not cleared (mac_reset_requests on the same flags, after this
 *     call, empties the request's rings and clears them).  Slots that share
 *     pages are given back by mac_reorder_tables, not so; beams that share
 *     none may be, but this call does not reach what mac_reorder_tables
 *     holds of their common positions (shared_in there).
 *   Pages: the k-th new page, in order of request and page, is the stack's
 *     k-th entry from the top.  Entries above the count stay as they are.
 *   A request is admitted whole or not at all: while the pages and the rows
 *     asked for by it and all requests before it fit (one that asks for no
 *     page needs only the rows).  One that is not admitted keeps its length
 *     and pages, gets no row, and sets MAC_DEV_NO_ROOM.  A negative length,
 *     or one that would pass max_context, max_pages * 16 or capacity, is
 *     not admitted and sets MAC_DEV_BAD_SEQ_LEN (with a reset flag and
 *     len_in itself out of range, no page is given back and the length
 *     stays).  A free or held page id outside [0, n_pages) sets
 *     MAC_DEV_BAD_PAGE; its tokens get slot -1, a new table entry is -1.
 * Outputs: len_out [B] (may be len_in); q_start int32 [B+1]; pos int32
 * [n_tokens], 1-based; slot int64 [n_tokens]: page * 16 + row (paged) or
 * b * capacity + pos - 1 (contiguous); rows that belong to nobody get pos 0
 * and slot -1.  n_tokens >= 1.  (mac_decode_step takes a query of every
 * request: one that brings no token, or is not admitted, decodes the position
 * of its last token again, and its row of out is to be dropped.) */
int mac_build_tables(const mac_config *cfg, void *chunk_ws, const mac_pages *pages,
                     const int32_t *reset_flags, const int32_t *len_in, const int32_t *new_len,
                     int32_t n_tokens, int32_t *len_out, int32_t *q_start, int32_t *pos,
                     int64_t *slot, void *stream);

/* Rotate and store the batch's rows: q_out[t] = R(pos[t]) q[t], and the K/V
 * of slot[t] <- (R(pos[t]) k[t], v[t]), with cfg's rotation ([MAC] "Match
 * (1)"; keys are kept rotated, [ACSP] "Why only K/V are cached"); angles
 * are exact to fp32, one rounding to dtype.  q, k, v: dtype rows of Hq, Hkv
 * and Hkv heads of d, row t at element t * {q,k,v}_stride (multiples of 16
 * bytes; a fused projection's rows have stride (Hq + 2 Hkv) d).  q and
 * q_out NULL: keys and values only (a decode step takes q unrotated).
 * q_out: [n_tokens][Hq][d], may be q itself if q_stride is Hq * d.  The
 * caches kv->k and kv->v are written (kv->page_table is not read).  A row
 * with a negative slot is skipped, its q_out row left as it was; one with
 * a slot outside the cache too, setting MAC_DEV_BAD_PAGE, and one with
 * pos < 1, setting MAC_DEV_BAD_SEQ_LEN.  Of two rows with the same slot the
 * cache gets an unspecified mixture: mac_build_tables makes none. */
int mac_write_kv(const mac_config *cfg, void *chunk_ws, const void *q, int64_t q_stride,
                 const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                 const int32_t *pos, const int64_t *slot, int32_t n_tokens, const mac_kv *kv,
                 void *q_out, void *stream);

/* Exact causal attention of the batch's rows over the cache: row t of
 * request b, the i-th of its n = q_start[b+1] - q_start[b] new tokens, is
 * position p = seq_len[b] - n + i (i from 1) and attends [1, p]
 * ([ACSP] MHA with repeat_kv; the miss path of [MAC] for many queries).
 * q: [n_tokens][Hq][d] of dtype, already rotated (mac_write_kv's q_out);
 * seq_len[b] counts the new tokens, whose K/V are in the cache.  out:
 * [n_tokens][Hq][d] of dtype; lse: f32 [n_tokens][Hq] natural-log softmax
 * denominators, or NULL.  Requests with n = 0 are passed over; rows that
 * belong to nobody keep what out and lse held.  Tokens on a page id outside
 * [0, n_pages) are left out (MAC_DEV_BAD_PAGE); a row that so has nothing
 * to attend gets out 0 and lse -inf, and so does every row of a request
 * whose seq_len is below n or beyond the cache (MAC_DEV_BAD_SEQ_LEN);
 * a request whose rows q_start puts outside [0, n_tokens], or ends before
 * they start, is passed over (MAC_DEV_BAD_SEQ_LEN); of rows that q_start so
 * gives to several requests out and lse are unspecified.  Cache rows beyond
 * seq_len may hold anything.  V of positions up to seq_len must be finite
 * even where a row of the same call does not attend them yet: they meet its
 * zero weights (K may be anything).  dtype bf16: products of bf16, sums and
 * statistics in fp32, the probabilities rounded to bf16 before they meet V.
 * dtype f32: weights, sums and statistics in fp32, each product to 2^-21 of
 * its size (2^-24 on average); a row that attends an infinite element is
 * NaN. */
int mac_chunk_attention(const mac_config *cfg, void *chunk_ws, const void *q,
                        const int32_t *q_start, const int32_t *seq_len, int32_t n_tokens,
                        const mac_kv *kv, void *out, float *lse, void *stream);

/* Attention over another sequence's states ([ACSP] MHA with repeat_kv, its
 * keys and values those of an encoder; the pages do not describe the call):
 * every row of the batch attends the whole memory of its source, [1,
 * mem_len[b]], with no causal mask.  cfg->batch counts the sources, kv is
 * their cache (mac_write_kv fills it, with MAC_ROPE_NONE where the keys keep
 * no position), mem_len: int32 [B].  The rows of source b are those of its
 * `group` >= 1 slots, which lie next to one another (its beams, say): rows
 * q_start[b group] .. q_start[(b+1) group] - 1, q_start int32 [B group + 1]
 * as mac_build_tables writes it for the slots (the entries between are not
 * looked at).  q, out, lse, chunk_ws, n_tokens as in mac_chunk_attention, of
 * this cfg; the query is taken as it is.  A source without states (mem_len
 * 0) gives its rows out 0 and lse -inf.  Bad lengths, pages and rows are
 * reported and left out as there.  Cache rows beyond mem_len may hold
 * anything; an infinity that is attended makes its outputs infinite or NaN.
 * cfg->max_context bounds mem_len, as the cache's room does, and with the
 * number of rows it says which kernels run: a caller that knows its memories
 * to be shorter than the cache gives that bound (one row of 8 / 2 heads over
 * 57 keys 4.4 us, 5.9 where 32768 would fit; five rows of 32 / 8 heads over
 * 128 5.0 and 9.4).  The numerics are mac_chunk_attention's; where there are at most
 * 16 rows of a KV head per source (n_tokens Hq / Hkv <= 16 B), or few more
 * and the memory is short, in bf16 the probabilities are not rounded to bf16,
 * and in fp32 each product is good to 2^-20 of its size (2^-24 on average),
 * sums over the memory round to nearest, tile by tile, however long it is,
 * and elements beyond 3.39e38 count as infinite. */
int mac_cross_attention(const mac_config *cfg, void *chunk_ws, const void *q, const int32_t *q_start,
                        int32_t group, const int32_t *mem_len, int32_t n_tokens, const mac_kv *kv,
                        void *out, float *lse, void *stream);

/* ---- beam search --------------------------------------------------------
 * The batch's slots form groups of n_beams slots next to one another: group g
 * is slots g n_beams .. (g+1) n_beams - 1, a sequence's beams (cfg->batch is
 * a multiple of n_beams).  A step decodes one token per slot, then:
 * mac_beam_select chooses the next beams from the logits, mac_reorder_tables
 * gives every slot its parent's history (pages, length), mac_reorder_state
 * moves what each layer keeps per slot.  (The pages describe none of the
 * three: the interfaces are this library's own.) */
#define MAC_MAX_BEAMS 16
#define MAC_MAX_CANDIDATES 32

/* Bytes of beam_ws for mac_beam_select: zero-filled before its first use, for
 * one stream at a time; calls of other n_beams, vocab and n_out may use it if
 * it is large enough for each.  Its device status word is read by
 * mac_last_status(cfg, beam_ws, ..). */
int mac_beam_workspace_size(const mac_config *cfg, int32_t n_beams, int32_t vocab, int32_t n_out,
                            size_t *beam_bytes);

/* The n_out <= MAC_MAX_CANDIDATES best next tokens of every group's beams.
 * logits: logits_dtype (MAC_BF16 | MAC_F32) rows of vocab <= 2^20 of every
 * slot, row_stride >= vocab elements apart, on any element boundary.  scores:
 * f32 [batch], the beams' sums of log probabilities; -inf: the beam has no
 * candidates (all but one slot of a group before its first token), and its
 * logits may be anything (a very low number in its place makes it a live beam,
 * and the choice, whose first threshold in fp32 allows for the largest score,
 * ranks many more candidates: of 5 beams of 128000 logits, -1e9 for four of
 * them, the 10 best take 130 us, not 13).  A candidate is (beam j, token v) with score s =
 * scores[j] + x_jv - ln sum_v exp x_jv; logits of -inf are no candidates.
 * The order is that of the exact scores (by s, rounded no coarser than 2^-36
 * or, where that is more, 2^-51 |s|), ties to the lowest (j, v), whatever the
 * card's sums in fp32 make of it.
 * done (int32 [batch] or NULL): a beam whose flag is set is finished and is
 * one candidate, end_token with the beam's score; its logits may be anything.
 * end_token: a token, or any other number if there is none (then done must be
 * NULL).
 * Outputs, [batch / n_beams][n_out], best first: scores_out f32; parent int32,
 * the beam's place in its group; token int32; done_out int32 or NULL: whether
 * the token is end_token.  Where a group has fewer candidates: score -inf,
 * parent -1, token -1, done 1.  placed != 0 (n_out = n_beams): instead of
 * best first, the best child of each parent in the parent's slot and the
 * others, best first, in the slots that are left, so that mac_reorder_state
 * has the least to move.  A beam with a NaN or +inf logit (or score) has no
 * candidates (MAC_DEV_NONFINITE_LOGIT).  scores_out and done_out may be scores
 * and done themselves. */
int mac_beam_select(const mac_config *cfg, void *beam_ws, int32_t n_beams, const void *logits,
                    int32_t logits_dtype, int64_t row_stride, int32_t vocab, const float *scores,
                    const int32_t *done, int32_t end_token, int32_t n_out, int32_t placed,
                    float *scores_out, int32_t *parent, int32_t *token, int32_t *done_out,
                    void *stream);

/* Slots take over the histories of their parents.  parent: int32 [batch], the
 * place in its group of the slot whose history a slot goes on from (as
 * mac_beam_select gives it with n_out = n_beams), or -1: the slot is given
 * up and is empty afterwards.  len_in, len_out: int32 [batch] tokens of every
 * slot; a child has its parent's.  shared_in, shared_out: int32
 * [batch][n_beams], for each slot of a group how many leading positions a
 * slot has in common with it; the caller keeps the array, zero-filled at
 * first.  These calls write it, and take its counts at their word: positions
 * that two slots have in common are not moved.  So a slot begins anew with
 * parent -1, which clears its counts (then its rings by mac_reset_requests,
 * its new tokens by mac_build_tables).  Where it begins anew in another way,
 * or goes back to a shorter history (reset_flags of slots without a common
 * page, lengths written by the caller), the caller clears its row, and its
 * column in the rows of its group, before the next call: what it had in
 * common would be taken for the beginning of its new history.
 *   Pages (pages == NULL for a contiguous cache): children share their
 *     parent's pages.  A history whose last page is not full is parted: its
 *     slot keeps that page if it goes on as its own child, else the child of
 *     the lowest slot does, and every other child gets a free page, the k-th
 *     from the top for the k-th such child of the batch.  Pages that no slot
 *     of the group holds any more are put on the stack first, in order of
 *     group, place in the table and slot, each once.  Table entries past a
 *     slot's pages stay as they are.  Pages are shared within a group only,
 *     and slots that share pages are given back here, with parent -1, not
 *     with mac_build_tables' reset_flags.
 *   A child whose free page is missing (MAC_DEV_NO_ROOM) is empty afterwards
 *     (len_out 0, parent >= 0) and has nothing in common with any slot: its
 *     rings are to be reset as after parent -1, and the caller sets its score
 *     to -inf, or the next selection counts it as a beam.
 *     A parent outside [-1, n_beams) (MAC_DEV_BAD_PARENT) is taken for the
 *     slot itself.  A group with a length outside [0, limit]
 *     (MAC_DEV_BAD_SEQ_LEN) is passed over.  A held page id outside
 *     [0, n_pages) is not put on the stack (MAC_DEV_BAD_PAGE), a page
 *     parted from or to one is not copied.
 * moves: int32 [batch][8] (16-byte aligned), what mac_reorder_state has to
 * move into every slot: the slot copied from (-1: nothing to do), the first and
 * last position whose ring entries may differ, the new length, the page
 * parted from, the page that its rows are copied to (-1: none), those rows, 0.
 * len_out may be len_in, shared_out shared_in.  The workspace is that of
 * the batch calls, of any number of rows. */
int mac_reorder_tables(const mac_config *cfg, void *chunk_ws, const mac_pages *pages, int32_t n_beams,
                       const int32_t *parent, const int32_t *len_in, int32_t *len_out,
                       const int32_t *shared_in, int32_t *shared_out, int32_t *moves, void *stream);

/* One layer's part of the moves that mac_reorder_tables has left, in place,
 * each slot from what its parent held before the call (slots may change
 * places).  ring_ws (or NULL): the layer's rings, where the entries of the
 * positions that parent and child do not share are moved.  Their mac_reset_requests
 * goes with parent -1.  kv (or NULL): the layer's cache; contiguous, the
 * keys and values of those positions; paged, the rows of parted pages
 * (kv->page_table is not read).  Moves outside a group, the cache or its pages are
 * reported (MAC_DEV_BAD_PARENT, _BAD_SEQ_LEN, _BAD_PAGE in chunk_ws) and
 * left out.  Runs after an append still pending on an auxiliary stream for
 * ring_ws, as mac_reset_requests does. */
int mac_reorder_state(const mac_config *cfg, void *chunk_ws, void *ring_ws, int32_t n_beams,
                      const int32_t *moves, const mac_kv *kv, void *stream);

/* Make stream_main wait for the last append enqueued on ring_ws (no-op if
 * none is pending).  Needed before ending a stream capture that used a
 * separate aux stream. */
int mac_join_aux(void *ring_ws, void *stream_main);

/* Ready gate ([MAC] "Production version": request state gated so that a
 * captured CUDA graph stays valid).  reset_flags: device int32 [B].  For
 * every request b whose flag is non-zero, its rings start over empty: no
 * slot holds a position any more, so its next decode step has no match
 * candidate, misses on every head and attends [1, m] exactly, and the
 * appends of its next steps refill the rings.  The flags are read and
 * cleared on the device, on `stream`, after any append still pending on an
 * auxiliary stream for ring_ws; the call can be captured into a graph and
 * the caller sets flags between replays (a new request in a reused slot,
 * a request whose cache was rewritten).  Returns MAC_ERR_INVALID_ARG for a
 * null or misaligned pointer; the flags' values are not checked. */
int mac_reset_requests(const mac_config *cfg, void *ring_ws, int32_t *reset_flags, void *stream);

/* Test hook for the bounded waits (no counterpart on the pages): the next
 * step or chunk-attention kernel launched by the calling thread gives every
 * wait (a stage's copy, a flag, the grid barrier, a piece count) `cycles` SM
 * cycles instead of about a second, and, if withhold_use >= 0, never issues
 * the copy of that stage use (per CTA; per warp in the ring kernel; of the K
 * ring in chunk attention), so the wait for it runs out: the kernel sets
 * MAC_DEV_WAIT_TIMEOUT, stops its work, lets its other copies land and returns.  The launch's outputs
 * are then undefined; its scratch workspace must be cleared (or replaced)
 * before the next launch.  1 <= cycles <= 2^31, withhold_use >= -1; the
 * hook clears itself. */
int mac_test_wait_budget(int64_t cycles, int32_t withhold_use);

/* Destroy the events the library keeps for ring_ws (call before freeing it). */
int mac_release_ring(void *ring_ws);

/* Synchronise stream, copy the device status word (MAC_DEV_* bits, 0 = clean)
 * to *device_status (host pointer) and clear it. */
int mac_last_status(const mac_config *cfg, void *scratch_ws, int32_t *device_status,
                    void *stream);

/* Profiling hook (no counterpart on the pages): the next mac_decode_step
 * issued by the calling thread records these CUDA events (cudaEvent_t
 * handles, each may be NULL): before and after the step kernel (match and
 * attention) on stream_main, and after the append kernel on the stream it
 * runs on; then the hook clears itself.  Lets a caller time the kernels on
 * the stream they run on, also inside a captured graph. */
int mac_set_phase_events(void *before_step, void *after_step, void *after_append);

/* Profiling hook (no counterpart on the pages): the next step kernel
 * launched by the calling thread (decode step or full attention) writes, per
 * CTA, MAC_TRACE_POINTS uint64 %globaltimer stamps (ns) into device_buffer
 * [grid][MAC_TRACE_POINTS]:
 *    0 start            1 end of the match       2 end of the tail pieces
 *    3 bands laid out   4 end of the band pieces and merges
 *    5 decisions read   6 end              7 tail layout published
 *    8 first match chunk arrived   9 producer: short-band tiles issued
 *   10 after the grid barrier
 *   11/12 first tail piece: first tile arrived / tiles done
 *   13/14 first band piece: first tile arrived / tiles done
 *   15 first band piece's partial written
 *   16/17 the SM's clock64() at start / end (cycles; with 0 and 6 they give
 *         the SM clock during the launch)
 *   18/19 time spent merging units (ns) / units merged
 *   20/21 the longest merge (ns) / its pieces
 *   22/23 band tokens / band pieces the CTA attended
 *   24 last band piece's tiles done   25 time spent waiting for band tiles (ns)
 *   26/27 producer: short-band list seen / long-band layout published
 *   28/29 time spent waiting for match chunks (ns) / match chunks scanned
 *   30/31 producer: first match copies issued / tail layout seen
 * Configurations with Hq/Hkv = 8 run the ring kernel (every warp feeds its
 * own stage ring; no producer warp), whose stamps are:
 *    0 start            1 warp 0's window tiles and match items done
 *    2 after the grid barrier         3 decisions and long bands laid out
 *    4 boundary pieces and hit merges done   5 long bands done
 *    6 end              7 the CTA's exit
 *   13/19 warps 0 / 1: owner merge's list read   14/15 owner merge's
 *         states written / combined  18 owner merge start
 *   16/17 the SM's clock64() at start / end
 * Stamps of phases a launch does not run are left as they were.  The span
 * kernel's stamps are compiled into one instantiation only, bf16 K/V without
 * a front sink, which the launch then runs; other span-kernel launches leave
 * the buffer as it was.  The buffer must hold MAC_TRACE_POINTS * (number of
 * SMs) uint64.  The hook clears itself. */
#define MAC_TRACE_POINTS 32
int mac_set_trace(void *device_buffer);

/* Static string for a MAC_OK / MAC_ERR_* code. */
const char *mac_status_string(int code);

/* Squared match threshold the kernels compare against (fp64 formula rounded
 * once to fp32), for reporting. */
float mac_threshold_sq(const mac_config *cfg);

#ifdef __cplusplus
}
#endif
#endif /* MAC_H_ */
