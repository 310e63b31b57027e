/*
 * pace_serve.h -- serving sets of sequences that change and that are drafted ahead, beside the layers of pace.h and pace_kv.h:
 * the gated delta rule over fp32 states in slots (prompts of unequal length, single tokens, trees of drafts, accepted paths),
 * verification of drafted tokens against the target's probabilities, and the pages of the caches (shared, taken, given back,
 * compacted, copied).
 *
 * Conventions are those of pace.h and pace_kv.h: device pointers owned by the caller, no device allocation, work enqueued on
 * `stream`, argument errors returned on the host before anything is launched, pace_last_error() for the message. Calls on one
 * handle must not overlap on the GPU (same stream, or ordered by events). Indices that only the device sees are checked there: a
 * bad one touches nothing outside the handle's arrays, and sets a bit that the handle's get_status call reports.
 */
#ifndef PACE_SERVE_H
#define PACE_SERVE_H

#include "pace_kv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- the gated delta rule over states in slots ------------------------------------------------------------------
 *   S_t = a_t S_{t-1} + k_t u_t^T,   u_t = beta_t (v_t - a_t S_{t-1}^T k_t),   o_t = S_t^T q_t
 * for every sequence and head, from and into an fp32 state [d][d] (key index first) of the sequence's slot. As in pace.h, k is
 * not normalised and q not scaled; a is the decay itself. Values are finite; one that is not spoils the outputs and the state of
 * its own sequence and head. */
typedef struct {
  int heads;               /* value heads, 1..PACE_MAX_HEADS */
  int key_heads;           /* heads of q and k (0: = heads); divides heads, value head h uses key head h / (heads/key_heads) */
  int d;                   /* 64 or 128 */
  int n_slots;             /* states */
  int io_dtype;            /* PACE_IO_* of q, k, v and o; a and beta are fp32 */
} pace_delta_config;

typedef struct pace_delta pace_delta;   /* opaque host handle */

/* Most tokens of a call of pace_delta_draft. */
#define PACE_DELTA_MAX_DRAFT 64

/* Bits of a handle's device status word. */
enum {
  PACE_DELTA_BAD_SLOT = 1, /* a slot outside the states, or one that an earlier sequence of the call with tokens has too:
                              the sequence was left out (its outputs are zeros) */
  PACE_DELTA_BAD_KEEP = 2, /* a kept index outside the drafts or not increasing (it and later ones were left), or a kept
                              count outside 0..n_idx (taken as the nearest) */
  PACE_DELTA_TIMEOUT = 4   /* a bounded device wait gave up: the call's outputs are not to be used; each head's state is whole,
                              as before the call or as after it */
};

/* The sequences of one call: sequence b has n_b = n_new[b] tokens, clamped to 0..n_tokens (n_new NULL: n_tokens), and the state
 * of slot slots[b] (slots NULL: slot b). lens, when given, says which sequences begin: where lens[b] == 0 the state before the
 * call counts as zero, whatever the slot holds, so that one vector of lengths serves these calls and those of pace_kv.h. A
 * sequence that may begin with drafts (a slot used before, a prompt of one token) needs it in draft and keep too. */
typedef struct {
  int batch, n_tokens;
  const int32_t *slots;    /* [batch] or NULL */
  const int32_t *lens;     /* [batch] or NULL */
  const int32_t *n_new;    /* [batch] or NULL */
} pace_delta_step;

/* Device bytes of a handle: the states [n_slots][heads][d][d] at its start, and a status word. */
pace_status pace_delta_bytes(const pace_delta_config *cfg, size_t *bytes_out);
/* Bind a caller-owned, 256-byte aligned region to a handle; enqueues its clearing (zero states). */
pace_status pace_delta_alloc(const pace_delta_config *cfg, void *device_mem, size_t bytes, void *stream, pace_delta **out);
void pace_delta_free(pace_delta *delta);

/* All tensors below are [batch][n_tokens][heads][d] by strides as in pace_kv.h: q, k of key_heads, v, o of heads, 16-byte
 * aligned with strides of 16-byte multiples; a and beta [batch][n_tokens][heads] by strides (4-byte aligned, any strides).
 *
 * Advance the states by the new tokens (a prompt chunk of any length, or single tokens): o, and S_{n_b} into the slot. Rows of
 * o at and past n_b are zeros; a sequence without tokens keeps its slot as it is. q and o may both be NULL (states only). No two
 * sequences with tokens share a slot. One launch. A few tokens go one by one in fp32; more by chunks of 64 whose products are of
 * fp32 values in parts of 8 bits, three of each, but where bf16 outputs are formed two (16 bits) of the states in S^T q, of u and
 * of q k^T. States then differ from those in 64 bits by 2e-7 of their norm with decays from 0.95 to 1, up to 7e-7 from 0.999. */
pace_status pace_delta_chunk(pace_delta *delta, const pace_delta_step *step, const pace_tensor *q, const pace_tensor *k,
                             const pace_tensor *v, const pace_tensor *a, const pace_tensor *beta, const pace_tensor *o,
                             void *stream);

/* Outputs of up to PACE_DELTA_MAX_DRAFT drafted tokens; no state changes, and sequences may share a slot. mask as for
 * pace_kv_attend: bit s % 32 of mask[b][t][s / 32] says that token s < t is an ancestor of token t (its own and later bits are
 * not looked at), or every earlier token where mask is NULL. The state before t is then that after its ancestors, in order, from
 * the slot's; the ancestors of an ancestor are ancestors. */
pace_status pace_delta_draft(pace_delta *delta, const pace_delta_step *step, const pace_tensor *q, const pace_tensor *k,
                             const pace_tensor *v, const pace_tensor *a, const pace_tensor *beta, const uint32_t *mask,
                             const pace_tensor *o, void *stream);

/* Advance the states along an accepted path of drafts: the rows idx[b][0 .. n_keep[b] - 1] of k, v, a and beta, in order, as
 * pace_delta_chunk would. idx [batch][n_idx] (int32) rises strictly in each row, below n_b. */
pace_status pace_delta_keep(pace_delta *delta, const pace_delta_step *step, const pace_tensor *k, const pace_tensor *v,
                            const pace_tensor *a, const pace_tensor *beta, const int32_t *idx, int n_idx,
                            const int32_t *n_keep, void *stream);

/* The status word (synchronises `stream`): PACE_ERR_TIMEOUT / PACE_ERR_STATE when a bit is set; cleared when `clear` is non-zero. */
pace_status pace_delta_get_status(const pace_delta *delta, int clear, int *status_out, void *stream);

/* ---- verification of drafts ------------------------------------------------------------------------------------------
 * Each sequence has up to n_nodes nodes: node 0 is the last token that the target has (it is always kept), the others are drafts. The parent
 * of node i is its nearest ancestor by mask (as for pace_delta_draft: the highest bit below i; without one the node hangs
 * nowhere and is never kept), or node i - 1 where mask is NULL. p[b][i] is the target's distribution of the token after node i,
 * q[b][i] that of the draft model (q NULL: the drafts were named without probabilities, each counts as certain to its
 * model), u [batch][n_nodes] are random numbers in [0, 1).
 *
 * From node 0 on, the drafts that hang from the node so far are tried in order. With R = p of the node and Z = 1 at first, draft i with
 * token y is kept if u_i q(y) Z < R(y); the walk then goes on from it. If not, R <- max(R - q Z, 0) and Z <- sum R (q NULL:
 * R(y) <- 0 and Z <- max(Z - R(y), 0)), and the next draft of the node is tried. Where none is left, the next token is the
 * smallest v with R(0) + .. + R(v) > u_0 sum R. So tokens are distributed as the target's own, where rows of p sum to 1 and drafts of one
 * node are drawn from q independently of one another, or named by any rule that does not look at u. Z begins at 1 whatever p sums to:
 * a row whose sum is off by a factor 1 + e (bf16: up to 2^-9) moves what drafts are kept by as much.
 *
 * Probabilities count as their clamp to 0..1, NaN as 0. Sums are taken in fixed point, so that the same call gives the same tokens: in units of
 * 2^-46 below 2^17 tokens, twice as large for each doubling from there, so that rows of any sum (all ones, say) are summed right.
 * A draft outside the vocabulary is not kept. Where nothing of R is left, the next token is drawn from p of the node; it is -1 where that is
 * zero too, and for sequences without nodes (n_nodes of sequence b: n_new[b], clamped to 0..n_nodes).
 *
 * idx [batch][n_nodes]: the kept nodes in order (rows go on with the last one), as pace_kv_keep and pace_delta_keep take them;
 * n_keep [batch]: their number; next [batch]. tokens [batch][n_nodes]. p, q: [batch][n_nodes][vocab] by the strides stride_b and
 * stride_t (stride_h unused), of io_dtype, aligned to their elements. One launch. */
#define PACE_VERIFY_MAX_NODES 256
#define PACE_VERIFY_MAX_VOCAB (1 << 24)
pace_status pace_verify(int batch, int n_nodes, int vocab, int io_dtype, const int32_t *tokens, const pace_tensor *p,
                        const pace_tensor *q, const float *u, const uint32_t *mask, const int32_t *n_new, int32_t *idx,
                        int32_t *n_keep, int32_t *next, void *stream);

/* ---- pages of the caches ---------------------------------------------------------------------------------------------
 * One set of page numbers serves the caches of all layers. A handle counts how many rows of the page table hold each page
 * (refs [n_pages]; 0: free); the table [batch][table_cols] and lens [batch] are the caller's, as for pace_kv_step, with -1 in
 * cells that hold no page. Row b holds the pages of its lens[b] tokens, and any that pace_pages_take added. */
typedef struct {
  int n_pages;             /* as the caches' */
  int page_tokens;         /* as the caches' */
  int max_batch;           /* rows of a table, 1..PACE_KV_MAX_BATCH */
} pace_pages_config;

typedef struct pace_pages pace_pages;   /* opaque host handle */

/* Byte offsets in a handle's region: refs [n_pages], the last call's moves (pages src[i] to copy to dst[i], [n_pages] each) and
 * their number. All int32. */
typedef struct {
  size_t refs, src, dst, n_moves, total_bytes;
} pace_pages_layout;

/* Bits of a handle's device status word. */
enum {
  PACE_PAGES_BAD_CELL = 1, /* a cell outside the pool (taken as -1), or a row whose last page is missing or free, or that
                              ends before its new tokens do (pace_pages_take: the row got nothing) */
  PACE_PAGES_BAD_ROW = 2   /* a source row outside the table (the row was left as it is) */
};

pace_status pace_pages_get_layout(const pace_pages_config *cfg, pace_pages_layout *out);
/* Bind a caller-owned, 256-byte aligned region of at least total_bytes; enqueues its clearing (every page free). */
pace_status pace_pages_alloc(const pace_pages_config *cfg, void *device_mem, size_t bytes, void *stream, pace_pages **out);
void pace_pages_free(pace_pages *pages);

/* Row b becomes what row src[b] was before the call (every row is read before any is written): its pages as far as its lens covers them
 * (pages taken for tokens that were not kept go back), and its length; src[b] = -1 leaves the row empty. src NULL: every row itself. One
 * call forks, reorders, shortens and frees rows. One launch. */
pace_status pace_pages_select(pace_pages *pages, int batch, int32_t *table, int table_cols, int32_t *lens, const int32_t *src,
                              void *stream);

/* Give each row the pages that its next n_new[b] tokens (slots lens[b] ..) need: one for each empty cell of them, and one in the
 * place of a page that they begin in and that other rows hold too, whose tokens are then to be copied (src, dst of the moves).
 * Where all holders of such a page take part, the one with the most tokens in it keeps it (of several the first). Free pages go
 * out from the lowest number, to the rows in order; from the first row on that the pool cannot serve, rows that need pages get
 * none, and fits[b] is 0 (else 1). The table has at most 2^31 - 1 cells. One launch. */
pace_status pace_pages_take(pace_pages *pages, int batch, int32_t *table, int table_cols, const int32_t *lens,
                            const int32_t *n_new, int32_t *fits, void *stream);

/* Renumber so that the pages in use are the lowest: used pages above their count move to free ones below it, both in rising order
 * (src, dst of the moves), and the table follows. All rows that hold pages are in the table. Two launches. */
pace_status pace_pages_compact(pace_pages *pages, int batch, int32_t *table, int table_cols, void *stream);

/* The status word (synchronises `stream`): PACE_ERR_STATE when a bit is set; cleared when `clear` is non-zero. */
pace_status pace_pages_get_status(const pace_pages *pages, int clear, int *status_out, void *stream);

/* Copy pages src[i] to dst[i] of a cache, i < min(*n, max_n) (n device memory; NULL: max_n). No dst is a src, or twice there. A page
 * outside the pool is not copied and sets PACE_KV_BAD_PAGE. One launch. */
pace_status pace_kv_copy_pages(pace_kv *kv, const int32_t *src, const int32_t *dst, const int32_t *n, int max_n, void *stream);
/* The pages of a cache: [n_pages] of page_bytes each, from *pool on (to hold them elsewhere, or to look at them). */
pace_status pace_kv_pool(const pace_kv *kv, void **pool, size_t *page_bytes);

#ifdef __cplusplus
}
#endif
#endif /* PACE_SERVE_H */
