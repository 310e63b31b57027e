// Host side of the attention-layer calls (pace_kv.h): argument checks, the cache's region, dispatch. Every entry point checks
// on the host and returns before any launch on error.
#include <math.h>
#include <string.h>

#include <new>

#include "kv_common.cuh"

struct pace_kv {
  pace_kv_config cfg;
  KvDev dev;                // the per-call fields are filled per call
};

namespace {

using pace::fail;
using pace::ok;

pace_status cuda_fail(cudaError_t e, const char *what) { return fail(PACE_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e)); }

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

pace_status check_config(const pace_kv_config *c) {
  if (!c) return fail(PACE_ERR_INVALID_ARG, "config is NULL");
  if (c->q_heads < 1 || c->q_heads > PACE_MAX_HEADS || c->kv_heads < 1 || c->kv_heads > c->q_heads)
    return fail(PACE_ERR_INVALID_ARG, "q_heads %d, kv_heads %d: need 1 <= kv_heads <= q_heads <= %d", c->q_heads, c->kv_heads,
                PACE_MAX_HEADS);
  if (c->q_heads % c->kv_heads)
    return fail(PACE_ERR_INVALID_ARG, "kv_heads %d does not divide q_heads %d", c->kv_heads, c->q_heads);
  if (c->d != 64 && c->d != 128 && c->d != 256) return fail(PACE_ERR_UNSUPPORTED, "d = %d: supported 64, 128, 256", c->d);
  if (c->bits != 4 && c->bits != 8) return fail(PACE_ERR_UNSUPPORTED, "bits = %d: supported 4, 8", c->bits);
  if (c->page_tokens < PACE_KV_TILE || c->page_tokens > 4096 || c->page_tokens % PACE_KV_TILE)
    return fail(PACE_ERR_INVALID_ARG, "page_tokens %d is not a multiple of %d in %d..4096", c->page_tokens, PACE_KV_TILE,
                PACE_KV_TILE);
  if (c->n_pages < 1) return fail(PACE_ERR_INVALID_ARG, "n_pages %d < 1", c->n_pages);
  if ((int64_t)c->n_pages * c->kv_heads * (c->page_tokens / PACE_KV_TILE) > (int64_t)INT32_MAX)
    return fail(PACE_ERR_UNSUPPORTED, "the pool has more than 2^31 - 1 tiles of %d tokens", PACE_KV_TILE);
  if (c->max_batch < 1 || c->max_batch > PACE_KV_MAX_BATCH)
    return fail(PACE_ERR_INVALID_ARG, "max_batch %d outside 1..%d", c->max_batch, PACE_KV_MAX_BATCH);
  if (c->max_new < 1 || c->max_new > PACE_KV_MAX_NEW)
    return fail(PACE_ERR_INVALID_ARG, "max_new %d outside 1..%d", c->max_new, PACE_KV_MAX_NEW);
  if (c->io_dtype != PACE_IO_BF16 && c->io_dtype != PACE_IO_F32) return fail(PACE_ERR_INVALID_ARG, "bad io_dtype");
  return PACE_OK;
}

size_t tile_bytes(const pace_kv_config *c) {
  const size_t ng = c->d / PACE_KV_GROUP;
  return 2 * PACE_KV_TILE * ((size_t)c->d * c->bits / 8 + ng * 2 + (c->bits == 4 ? ng : 0));
}
size_t pool_bytes(const pace_kv_config *c) {
  return (size_t)c->n_pages * c->kv_heads * (c->page_tokens / PACE_KV_TILE) * tile_bytes(c);
}

// Regions: status (256 bytes), counters, partial results, pool.
struct Regions {
  size_t count, part, pool, total;
};
Regions regions(const pace_kv_config *c) {
  size_t nc = 0, np = 0;
  pace_kv_attend_work(*c, &nc, &np);
  Regions r;
  r.count = 256;
  r.part = align256(r.count + nc);
  r.pool = align256(r.part + np);
  r.total = align256(r.pool + pool_bytes(c));
  return r;
}

pace_status check_rope(const pace_rope_config *r) {
  if (!r) return fail(PACE_ERR_INVALID_ARG, "rope config is NULL");
  if (r->rot < 16 || r->rot > 256 || r->rot % 16)
    return fail(PACE_ERR_INVALID_ARG, "rot %d is not a multiple of 16 in 16..256", r->rot);
  if (r->max_pos < 1) return fail(PACE_ERR_INVALID_ARG, "max_pos %d < 1", r->max_pos);
  if (r->layout != PACE_ROPE_HALF && r->layout != PACE_ROPE_INTERLEAVED) return fail(PACE_ERR_INVALID_ARG, "bad rope layout");
  if (r->scaling < PACE_ROPE_PLAIN || r->scaling > PACE_ROPE_PARTS) return fail(PACE_ERR_INVALID_ARG, "bad rope scaling");
  if (!(r->base > 1.0) || !isfinite(r->base)) return fail(PACE_ERR_INVALID_ARG, "rope base must be finite and > 1");
  if (r->scaling != PACE_ROPE_PLAIN && (!(r->factor >= 1.0) || !isfinite(r->factor)))
    return fail(PACE_ERR_INVALID_ARG, "rope factor must be finite and >= 1");
  if (!(r->mscale >= 0.0) || !isfinite(r->mscale)) return fail(PACE_ERR_INVALID_ARG, "rope mscale must be finite and >= 0");
  if (r->scaling == PACE_ROPE_PARTS && (r->orig_pos < 1 || !(r->beta_slow >= 0.0) || !(r->beta_fast > r->beta_slow) ||
                                        !isfinite(r->beta_fast)))
    return fail(PACE_ERR_INVALID_ARG, "rope by parts needs orig_pos >= 1 and 0 <= beta_slow < beta_fast");
  return PACE_OK;
}
size_t rope_bytes(const pace_rope_config *r) { return (size_t)r->max_pos * (r->rot / 2) * sizeof(float2); }

bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

pace_status check_tensor(const pace_tensor *t, int io, const char *call, const char *name, KvTensor *out) {
  if (!t || !t->data) return fail(PACE_ERR_INVALID_ARG, "%s: %s is NULL", call, name);
  const int64_t per = io == PACE_IO_F32 ? 4 : 8;     // elements of 16 bytes
  if (!aligned(t->data, 16) || t->stride_b % per || t->stride_t % per || t->stride_h % per)
    return fail(PACE_ERR_INVALID_ARG, "%s: %s must be 16-byte aligned with strides of 16-byte multiples", call, name);
  *out = KvTensor{static_cast<char *>(t->data), t->stride_b, t->stride_t, t->stride_h};
  return PACE_OK;
}

// Checks what every call on a cache has in common and fills the device view.
pace_status check_step(const pace_kv *kv, const pace_kv_step *s, const char *call, bool lens, KvDev *d) {
  if (!kv) return fail(PACE_ERR_INVALID_ARG, "%s: cache is NULL", call);
  if (!s) return fail(PACE_ERR_INVALID_ARG, "%s: step is NULL", call);
  if (s->batch < 0 || s->batch > kv->cfg.max_batch)
    return fail(PACE_ERR_INVALID_ARG, "%s: batch %d outside 0..max_batch (%d)", call, s->batch, kv->cfg.max_batch);
  if (s->n_tokens < 0 || (lens && s->n_tokens > kv->cfg.max_new))
    return fail(PACE_ERR_INVALID_ARG, "%s: n_tokens %d outside 0..max_new (%d)", call, s->n_tokens, kv->cfg.max_new);
  if (s->batch == 0 || s->n_tokens == 0) return PACE_OK;
  if ((lens && !s->lens) || !s->table) return fail(PACE_ERR_INVALID_ARG, "%s: lens or table is NULL", call);
  if (!aligned(s->lens, 4) || !aligned(s->n_new, 4) || !aligned(s->table, 4))
    return fail(PACE_ERR_INVALID_ARG, "%s: lens, n_new and table must be 4-byte aligned", call);
  if (s->table_cols < 1 || (int64_t)s->table_cols * kv->cfg.page_tokens > (int64_t)1 << 30)
    return fail(PACE_ERR_INVALID_ARG, "%s: table_cols %d outside 1..2^30 tokens' pages", call, s->table_cols);
  *d = kv->dev;
  d->batch = s->batch;
  d->n_tokens = s->n_tokens;
  d->lens = s->lens;
  d->n_new = s->n_new;
  d->table = s->table;
  d->table_cols = s->table_cols;
  return PACE_OK;
}
bool empty(const pace_kv_step *s) { return s->batch == 0 || s->n_tokens == 0; }

}  // namespace

extern "C" {

pace_status pace_rope_bytes(const pace_rope_config *cfg, size_t *bytes_out) {
  pace_status st = check_rope(cfg);
  if (st != PACE_OK) return st;
  if (!bytes_out) return fail(PACE_ERR_INVALID_ARG, "bytes_out is NULL");
  *bytes_out = rope_bytes(cfg);
  return ok();
}

pace_status pace_rope_table(const pace_rope_config *cfg, void *table, size_t bytes, void *stream) {
  pace_status st = check_rope(cfg);
  if (st != PACE_OK) return st;
  if (!table || !aligned(table, 16)) return fail(PACE_ERR_INVALID_ARG, "rope_table: table is NULL or not 16-byte aligned");
  if (bytes < rope_bytes(cfg))
    return fail(PACE_ERR_INVALID_ARG, "rope_table: %zu bytes are fewer than the %zu the table needs", bytes, rope_bytes(cfg));
  const cudaError_t e = pace_launch_rope_table(*cfg, static_cast<float2 *>(table), static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ok() : cuda_fail(e, "rope_table launch");
}

pace_status pace_rope_apply(const pace_rope_config *cfg, const void *table, int n, int heads, int d, int io_dtype,
                            const pace_tensor *x, const int32_t *positions, const pace_tensor *out, int inverse, void *stream) {
  pace_status st = check_rope(cfg);
  if (st != PACE_OK) return st;
  if (n < 0 || heads < 0) return fail(PACE_ERR_INVALID_ARG, "rope_apply: n %d or heads %d < 0", n, heads);
  if (d < 16 || d > 256 || d % 8) return fail(PACE_ERR_UNSUPPORTED, "rope_apply: d = %d: multiples of 8 in 16..256", d);
  if (cfg->rot > d) return fail(PACE_ERR_INVALID_ARG, "rope_apply: rot %d > d %d", cfg->rot, d);
  if (io_dtype != PACE_IO_BF16 && io_dtype != PACE_IO_F32) return fail(PACE_ERR_INVALID_ARG, "rope_apply: bad io_dtype");
  if (n == 0 || heads == 0) return ok();
  if ((int64_t)n * heads > (int64_t)1 << 30) return fail(PACE_ERR_UNSUPPORTED, "rope_apply: more than 2^30 head vectors");
  if (!table || !aligned(table, 16)) return fail(PACE_ERR_INVALID_ARG, "rope_apply: table is NULL or not 16-byte aligned");
  if (!positions || !aligned(positions, 4)) return fail(PACE_ERR_INVALID_ARG, "rope_apply: positions is NULL or misaligned");
  KvTensor tx, to;
  if ((st = check_tensor(x, io_dtype, "rope_apply", "x", &tx)) != PACE_OK) return st;
  if ((st = check_tensor(out, io_dtype, "rope_apply", "out", &to)) != PACE_OK) return st;
  const KvRope r{static_cast<const float2 *>(table), cfg->rot, cfg->max_pos, cfg->layout};
  const cudaError_t e = pace_launch_rope(r, n, heads, d, io_dtype, tx, positions, to, inverse, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ok() : cuda_fail(e, "rope_apply launch");
}

size_t pace_kv_tile_bytes(const pace_kv_config *cfg) { return check_config(cfg) == PACE_OK ? tile_bytes(cfg) : 0; }

pace_status pace_kv_bytes(const pace_kv_config *cfg, size_t *bytes_out) {
  pace_status st = check_config(cfg);
  if (st != PACE_OK) return st;
  if (!bytes_out) return fail(PACE_ERR_INVALID_ARG, "bytes_out is NULL");
  *bytes_out = regions(cfg).total;
  return ok();
}

pace_status pace_kv_alloc(const pace_kv_config *cfg, void *device_mem, size_t bytes, void *stream, pace_kv **out) {
  pace_status st = check_config(cfg);
  if (st != PACE_OK) return st;
  if (!out) return fail(PACE_ERR_INVALID_ARG, "out is NULL");
  *out = nullptr;
  if (!device_mem || !aligned(device_mem, 256)) return fail(PACE_ERR_INVALID_ARG, "device_mem is NULL or not 256-byte aligned");
  const Regions r = regions(cfg);
  if (bytes < r.total)
    return fail(PACE_ERR_INVALID_ARG, "device region of %zu bytes is smaller than the %zu the cache needs", bytes, r.total);
  pace_kv *kv = new (std::nothrow) pace_kv;
  if (!kv) return fail(PACE_ERR_INVALID_ARG, "host allocation of the handle failed");
  char *base = static_cast<char *>(device_mem);
  kv->cfg = *cfg;
  memset(&kv->dev, 0, sizeof kv->dev);
  KvDev &d = kv->dev;
  d.pool = base + r.pool;
  d.status = reinterpret_cast<int32_t *>(base);
  d.count = reinterpret_cast<int32_t *>(base + r.count);
  d.part = reinterpret_cast<float *>(base + r.part);
  d.Hq = cfg->q_heads;
  d.Hkv = cfg->kv_heads;
  d.group = cfg->q_heads / cfg->kv_heads;
  d.d = cfg->d;
  d.bits = cfg->bits;
  d.page = cfg->page_tokens;
  d.n_pages = cfg->n_pages;
  d.io = cfg->io_dtype;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaMemsetAsync(base, 0, r.part, cs);                        // status and counters
  if (e == cudaSuccess) e = cudaMemsetAsync(d.pool, 0, pool_bytes(cfg), cs);   // slots never written hold zeros
  if (e != cudaSuccess) {
    delete kv;
    return cuda_fail(e, "clearing the cache");
  }
  *out = kv;
  return ok();
}

void pace_kv_free(pace_kv *kv) { delete kv; }

pace_status pace_kv_append(pace_kv *kv, const pace_kv_step *step, const pace_tensor *q, const pace_tensor *k,
                           const pace_tensor *v, const pace_tensor *q_out, const pace_rope_config *rope,
                           const void *rope_table, const int32_t *positions, void *stream) {
  KvDev c;
  pace_status st = check_step(kv, step, "kv_append", true, &c);
  if (st != PACE_OK) return st;
  KvRope r{nullptr, 0, 0, 0};
  if (rope) {
    if ((st = check_rope(rope)) != PACE_OK) return st;
    if (rope->rot > kv->cfg.d) return fail(PACE_ERR_INVALID_ARG, "kv_append: rot %d > d %d", rope->rot, kv->cfg.d);
    if (!rope_table || !aligned(rope_table, 16))
      return fail(PACE_ERR_INVALID_ARG, "kv_append: rope table is NULL or not 16-byte aligned");
    r = KvRope{static_cast<const float2 *>(rope_table), rope->rot, rope->max_pos, rope->layout};
  } else if (q || q_out || positions) {
    return fail(PACE_ERR_INVALID_ARG, "kv_append: q, q_out and positions go with a rope config");
  }
  if ((q == nullptr) != (q_out == nullptr)) return fail(PACE_ERR_INVALID_ARG, "kv_append: q and q_out go together");
  if (empty(step)) return ok();
  if (!aligned(positions, 4)) return fail(PACE_ERR_INVALID_ARG, "kv_append: positions must be 4-byte aligned");
  KvTensor tq{nullptr, 0, 0, 0}, tk, tv, to{nullptr, 0, 0, 0};
  const int io = kv->cfg.io_dtype;
  if (q && (st = check_tensor(q, io, "kv_append", "q", &tq)) != PACE_OK) return st;
  if (q && (st = check_tensor(q_out, io, "kv_append", "q_out", &to)) != PACE_OK) return st;
  if ((st = check_tensor(k, io, "kv_append", "k", &tk)) != PACE_OK) return st;
  if ((st = check_tensor(v, io, "kv_append", "v", &tv)) != PACE_OK) return st;
  const cudaError_t e = pace_launch_kv_append(c, tq, tk, tv, to, r, positions, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ok() : cuda_fail(e, "kv_append launch");
}

pace_status pace_kv_read(const pace_kv *kv, const pace_kv_step *step, const int32_t *first, const int32_t *end,
                         const pace_tensor *k_out, const pace_tensor *v_out, void *stream) {
  KvDev c;
  pace_status st = check_step(kv, step, "kv_read", false, &c);
  if (st != PACE_OK) return st;
  if (empty(step)) return ok();
  if (!aligned(first, 4) || !aligned(end, 4)) return fail(PACE_ERR_INVALID_ARG, "kv_read: first and end must be 4-byte aligned");
  if ((int64_t)step->batch * kv->cfg.kv_heads * (step->n_tokens / PACE_KV_TILE + 2) > (int64_t)INT32_MAX)
    return fail(PACE_ERR_UNSUPPORTED, "kv_read: more than 2^31 tiles");
  KvTensor tk, tv;
  if ((st = check_tensor(k_out, kv->cfg.io_dtype, "kv_read", "k_out", &tk)) != PACE_OK) return st;
  if ((st = check_tensor(v_out, kv->cfg.io_dtype, "kv_read", "v_out", &tv)) != PACE_OK) return st;
  const cudaError_t e = pace_launch_kv_read(c, first, end, tk, tv, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ok() : cuda_fail(e, "kv_read launch");
}

pace_status pace_kv_attend(pace_kv *kv, const pace_kv_step *step, const pace_tensor *q, const uint32_t *mask, float scale,
                           const pace_tensor *o, void *stream) {
  KvDev c;
  pace_status st = check_step(kv, step, "kv_attend", true, &c);
  if (st != PACE_OK) return st;
  if (!isfinite(scale)) return fail(PACE_ERR_INVALID_ARG, "kv_attend: scale must be finite");
  if (empty(step)) return ok();
  if (!aligned(mask, 4)) return fail(PACE_ERR_INVALID_ARG, "kv_attend: mask must be 4-byte aligned");
  KvTensor tq, to;
  if ((st = check_tensor(q, kv->cfg.io_dtype, "kv_attend", "q", &tq)) != PACE_OK) return st;
  if ((st = check_tensor(o, kv->cfg.io_dtype, "kv_attend", "o", &to)) != PACE_OK) return st;
  const cudaError_t e = pace_launch_kv_attend(c, tq, mask, scale, to, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ok() : cuda_fail(e, "kv_attend launch");
}

pace_status pace_kv_keep(pace_kv *kv, const pace_kv_step *step, const int32_t *idx, const int32_t *n_keep, void *stream) {
  KvDev c;
  pace_status st = check_step(kv, step, "kv_keep", true, &c);
  if (st != PACE_OK) return st;
  if (empty(step)) return ok();
  if (!idx || !n_keep || !aligned(idx, 4) || !aligned(n_keep, 4))
    return fail(PACE_ERR_INVALID_ARG, "kv_keep: idx or n_keep is NULL or not 4-byte aligned");
  const cudaError_t e = pace_launch_kv_keep(c, kv->cfg.max_new, idx, n_keep, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ok() : cuda_fail(e, "kv_keep launch");
}

pace_status pace_kv_get_status(const pace_kv *kv, int clear, int *status_out, void *stream) {
  if (!kv) return fail(PACE_ERR_INVALID_ARG, "kv_get_status: cache is NULL");
  if (!status_out) return fail(PACE_ERR_INVALID_ARG, "status_out is NULL");
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  int32_t word = 0;
  cudaError_t e = cudaMemcpyAsync(&word, kv->dev.status, 4, cudaMemcpyDeviceToHost, cs);
  if (e == cudaSuccess) e = cudaStreamSynchronize(cs);
  if (e == cudaSuccess && clear && word) e = cudaMemsetAsync(kv->dev.status, 0, 4, cs);
  if (e != cudaSuccess) return cuda_fail(e, "reading the status word");
  *status_out = word;
  if (word & PACE_KV_TIMEOUT) return fail(PACE_ERR_TIMEOUT, "a bounded device wait gave up");
  if (word)
    return fail(PACE_ERR_STATE, "cache calls met%s%s%s", word & PACE_KV_BAD_PAGE ? " a slot outside the pages" : "",
                word & PACE_KV_BAD_POSITION ? " a position outside the rotary table" : "",
                word & PACE_KV_BAD_KEEP ? " a kept path that does not rise, or its count" : "");
  return ok();
}

}  // extern "C"
