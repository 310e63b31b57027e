/*
 * pace_kv.h -- the softmax-attention layers of a hybrid model, beside the gated-delta layers of pace.h:
 * rotary positions, a paged KV cache held at 4 or 8 bits, and attention over it for single tokens, trees of
 * drafted tokens and prompt chunks.
 *
 * Conventions are those of pace.h: device pointers owned by the caller, no device allocation, work enqueued on
 * `stream`, argument errors returned on the host before anything is launched, pace_last_error() for the message.
 * Calls on one cache must not overlap on the GPU (same stream, or ordered by events): they share its pages and
 * its work area. Indices that only the device sees (page numbers, lengths, positions, kept drafts) are checked
 * there: a bad one touches nothing outside the cache, and sets a bit that pace_kv_get_status reports. A slot without a
 * valid page is not written, reads as zeros, and is seen by no query.
 *
 * Cached values. Each head vector is held in groups of PACE_KV_GROUP consecutive elements with the quantizer of
 * the states (every operation rounds once to fp32; elements are first clamped to +-2^120, NaN counts as 0):
 *   8 bits  s = bf16(max|x| / 127), code = clamp(rint(x * (1/s)), -127, 127),       value s * code
 *   4 bits  lo = min(0, x), hi = max(0, x), s = bf16((hi - lo) / 15), z = clamp(rint(-lo * (1/s)), 0, 15),
 *           code = clamp(rint(x * (1/s)) + z, 0, 15),                                value s * (code - z)
 * A zero or subnormal s makes the group zero.
 *
 * Pages. A sequence's token t sits in page table[b][t / page_tokens]. Of a page every KV head has page_tokens / 32
 * tiles of 32 tokens, each contiguous (pace_kv_tile_bytes): key codes, value codes, key scales, value scales and
 * (4 bits) key and value zero points, in the order in which the attention kernels' matrix fragments read them.
 */
#ifndef PACE_KV_H
#define PACE_KV_H

#include "pace.h"

#ifdef __cplusplus
extern "C" {
#endif

#define PACE_KV_GROUP 64
#define PACE_KV_TILE 32
#define PACE_KV_MAX_BATCH 1024
#define PACE_KV_MAX_NEW 4096

/* Bits of the device status word (pace_kv_get_status). */
enum {
  PACE_KV_BAD_PAGE = 1,      /* a slot outside the page table or a page number outside the pool */
  PACE_KV_BAD_POSITION = 2,  /* a rotary position outside the table (the nearest row was used) */
  PACE_KV_BAD_KEEP = 4,      /* a kept index outside the drafts or not increasing (it and later ones were left), or a kept
                                count outside 0..n_tokens (taken as the nearest) */
  PACE_KV_TIMEOUT = 8        /* a bounded device wait gave up (the call's outputs are not to be used) */
};

/* ---- rotary positions ---------------------------------------------------------------------------------------
 * Pair i of the first `rot` elements of a head turns by pos * theta_i, theta_i = base^(-2i/rot):
 *   y_a = x_a c - x_b s, y_b = x_b c + x_a s, c = m cos, s = m sin (fp32, each operation rounds once),
 * the other elements pass unchanged. The inverse rotation (s negated) is the gradient of the rotation.
 * Long contexts, `factor` times the trained one:
 *   LINEAR  theta_i / factor (positions squeezed)
 *   NTK     base * factor^(rot / (rot - 2)) in place of base (the slowest pair is stretched by factor, the
 *           fastest is unchanged)
 *   PARTS   per pair by its turns over the trained context r_i = orig_pos theta_i / (2 pi):
 *           g = clamp((r_i - beta_slow) / (beta_fast - beta_slow), 0, 1), theta_i (g + (1 - g) / factor),
 *           with m = 0.1 ln(factor) + 1 (m = 1 for the other kinds). The ramp is linear in the turns, as published; checkpoints
 *           whose code ramps linearly over the pair index i, between the pairs that turn beta_fast and beta_slow times, have
 *           other angles between those pairs */
enum { PACE_ROPE_HALF = 0, PACE_ROPE_INTERLEAVED = 1 };    /* pairs (i, i + rot/2) or (2i, 2i + 1) */
enum { PACE_ROPE_PLAIN = 0, PACE_ROPE_LINEAR = 1, PACE_ROPE_NTK = 2, PACE_ROPE_PARTS = 3 };

typedef struct {
  int rot;                 /* rotated elements, a multiple of 16, 16..256 */
  int max_pos;             /* table rows: positions 0..max_pos-1 */
  int layout;              /* PACE_ROPE_HALF / PACE_ROPE_INTERLEAVED */
  int scaling;             /* PACE_ROPE_PLAIN .. PACE_ROPE_PARTS */
  double base, factor;     /* base > 1; factor >= 1 */
  int orig_pos;            /* PARTS: trained context */
  double beta_fast, beta_slow;   /* PARTS: 32 and 1 are usual */
  double mscale;           /* factor m on cos and sin; 0: the kind's own */
} pace_rope_config;

/* A [batch][tokens][heads][d] tensor: strides in elements, d contiguous. Pointer and strides are multiples of
 * 16 bytes (pace_rope_apply takes token and head strides only). */
typedef struct {
  void *data;
  int64_t stride_b, stride_t, stride_h;
} pace_tensor;

/* Bytes of the cos/sin table (fp32 pairs, [max_pos][rot/2]) and its construction in 64 bits. */
pace_status pace_rope_bytes(const pace_rope_config *cfg, size_t *bytes_out);
pace_status pace_rope_table(const pace_rope_config *cfg, void *table, size_t bytes, void *stream);
/* Rotate x [n][heads][d] (d a multiple of 8, rot <= d <= 256) at positions[n] (int32, device) into out, which may be x itself
 * (same strides). inverse != 0: by the negative angle. A position outside the table uses the nearest row. */
pace_status pace_rope_apply(const pace_rope_config *cfg, const void *table, int n, int heads, int d, int io_dtype,
                            const pace_tensor *x, const int32_t *positions, const pace_tensor *out, int inverse,
                            void *stream);

/* ---- the cache -------------------------------------------------------------------------------------------- */
typedef struct {
  int q_heads, kv_heads;   /* 1..PACE_MAX_HEADS; kv_heads divides q_heads; query head h reads KV head h / (q/kv) */
  int d;                   /* 64, 128 or 256 */
  int bits;                /* 4 or 8 */
  int page_tokens;         /* a multiple of 32, 32..4096 */
  int n_pages;             /* pages of the pool */
  int max_batch;           /* 1..PACE_KV_MAX_BATCH */
  int max_new;             /* most new tokens a sequence and call, 1..PACE_KV_MAX_NEW */
  int io_dtype;            /* PACE_IO_* of q, k, v and outputs */
} pace_kv_config;

typedef struct pace_kv pace_kv;   /* opaque host handle */

/* The sequences of one call. lens[b] tokens are in the cache before the call's new tokens, which take slots
 * lens[b] .. lens[b] + n_b - 1, n_b = n_new[b] clamped to 0..n_tokens, or n_tokens where n_new is NULL. Lengths and
 * page tables are the caller's (one set serves every layer) and are not advanced by any call. */
typedef struct {
  int batch, n_tokens;
  const int32_t *lens;      /* [batch] */
  const int32_t *n_new;     /* [batch] or NULL */
  const int32_t *table;     /* [batch][table_cols] page numbers */
  int table_cols;
} pace_kv_step;

size_t pace_kv_tile_bytes(const pace_kv_config *cfg);      /* 0 for an invalid config */
pace_status pace_kv_bytes(const pace_kv_config *cfg, size_t *bytes_out);
/* Bind a caller-owned, 256-byte aligned region of at least pace_kv_bytes to a handle; enqueues its clearing. */
pace_status pace_kv_alloc(const pace_kv_config *cfg, void *device_mem, size_t bytes, void *stream, pace_kv **out);
void pace_kv_free(pace_kv *kv);

/* Write the new tokens' k and v [batch][n_tokens][kv_heads][d] into the cache. With a rope config (and its table) k
 * is rotated first, and q [..][q_heads][d], when given, is rotated into q_out (which may be q); without one q and q_out
 * are NULL. positions [batch][n_tokens] (int32) or NULL for lens[b] + t. One launch. */
pace_status pace_kv_append(pace_kv *kv, const pace_kv_step *step, const pace_tensor *q, const pace_tensor *k,
                           const pace_tensor *v, const pace_tensor *q_out, const pace_rope_config *rope,
                           const void *rope_table, const int32_t *positions, void *stream);

/* The held values of slots first[b] .. first[b] + n - 1 (first NULL: from 0) as k_out and v_out [batch][n][kv_heads][d]
 * of the I/O type; zeros at and past end[b] (end NULL: no bound but the page table's). step->lens, n_new unused. */
pace_status pace_kv_read(const pace_kv *kv, const pace_kv_step *step, const int32_t *first, const int32_t *end,
                         const pace_tensor *k_out, const pace_tensor *v_out, void *stream);

/* Attention of the new tokens' queries over the cache (their k and v appended before):
 *   o_t = sum_j p_j v_j, p = softmax over visible slots j of scale * q_t . k_j
 * Every slot below lens[b] is visible; of the new tokens, t sees j where bit j%32 of mask[b][t][j/32] is set (uint32,
 * (n_tokens + 31)/32 words a row; a tree's ancestor bits, itself included), or j <= t where mask is NULL. A row
 * that sees nothing, and rows t >= n_new[b], get zeros. q, o [batch][n_tokens][q_heads][d]. Scores, maxima, sums and
 * the output accumulate in fp32. With fp32 I/O, and where a KV head has up to 32 rows (new tokens times query heads of
 * it), codes enter the products as exact integers; with bf16 I/O queries and weights are rounded to 11 bits, and above 32
 * rows held keys and values too. Tokens keep these bits whatever the size of others that weigh less. Within one head
 * vector a group of values (above 32 rows of keys too) keeps them down to 2^-12 of the largest group and loses them gradually
 * below; what is lost is below 2^-22 of the vector's largest element. With bf16 I/O and up to 32 rows, values whose scale is
 * below 2^-80 lose bits, and below 2^-90 count as zero. The same call gives the same bits. One launch, or two above 32 rows (more only where a batch or a sequence
 * could hold 2^31 tiles of work). */
pace_status pace_kv_attend(pace_kv *kv, const pace_kv_step *step, const pace_tensor *q, const uint32_t *mask, float scale,
                           const pace_tensor *o, void *stream);

/* Keep an accepted path: for i < n_keep[b], the row of draft idx[b][i] (slot lens[b] + idx) moves to slot lens[b] + i,
 * codes and scales unchanged. idx [batch][n_tokens] int32 rises strictly in each row (as a root-to-leaf path does), below
 * max_new. The caller then advances lens[b] by n_keep[b]. */
pace_status pace_kv_keep(pace_kv *kv, const pace_kv_step *step, const int32_t *idx, const int32_t *n_keep, void *stream);

/* The status word (bits above); synchronises `stream`. PACE_ERR_TIMEOUT / PACE_ERR_STATE when a bit is set; cleared when
 * `clear` is non-zero. */
pace_status pace_kv_get_status(const pace_kv *kv, int clear, int *status_out, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* PACE_KV_H */
