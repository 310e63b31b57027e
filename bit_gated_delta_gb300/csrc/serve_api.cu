// Host side of pace_serve.h: argument checks, the handles' regions, dispatch. Every entry point checks on the host and returns before
// any launch on error.
#include <string.h>

#include <new>

#include "delta_common.cuh"
#include "serve_internal.h"

struct pace_delta {
  pace_delta_config cfg;
  DeltaArgs args;           // the per-call fields are filled per call
};

struct pace_pages {
  pace_pages_config cfg;
  PagesDev dev;
};

namespace {

using pace::fail;
using pace::ok;

pace_status launched(cudaError_t e, const char *what) {
  return e == cudaSuccess ? ok() : fail(PACE_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// ---- the gated delta rule -----------------------------------------------------------------------------------------------------
pace_status check_delta_config(const pace_delta_config *c) {
  if (!c) return fail(PACE_ERR_INVALID_ARG, "config is NULL");
  const int hk = c->key_heads ? c->key_heads : c->heads;
  if (c->heads < 1 || c->heads > PACE_MAX_HEADS || hk < 1 || hk > c->heads || c->heads % hk)
    return fail(PACE_ERR_INVALID_ARG, "heads %d, key_heads %d: need 1 <= key_heads <= heads <= %d, key_heads dividing heads", c->heads,
                c->key_heads, PACE_MAX_HEADS);
  if (c->d != 64 && c->d != 128) return fail(PACE_ERR_UNSUPPORTED, "d = %d: supported 64, 128", c->d);
  if (c->n_slots < 1) return fail(PACE_ERR_INVALID_ARG, "n_slots %d < 1", c->n_slots);
  if (c->io_dtype != PACE_IO_BF16 && c->io_dtype != PACE_IO_F32) return fail(PACE_ERR_INVALID_ARG, "bad io_dtype");
  return PACE_OK;
}
size_t states_bytes(const pace_delta_config *c) { return (size_t)c->n_slots * c->heads * c->d * c->d * sizeof(float); }

pace_status check_rows(const pace_tensor *t, int io, const char *call, const char *name, KvTensor *out) {
  if (!t || !t->data) return fail(PACE_ERR_INVALID_ARG, "%s: %s is NULL", call, name);
  const int64_t per = io == PACE_IO_F32 ? 4 : 8;     // elements of 16 bytes
  if (!aligned(t->data, 16) || t->stride_b % per || t->stride_t % per || t->stride_h % per)
    return fail(PACE_ERR_INVALID_ARG, "%s: %s must be 16-byte aligned with strides of 16-byte multiples", call, name);
  *out = KvTensor{static_cast<char *>(t->data), t->stride_b, t->stride_t, t->stride_h};
  return PACE_OK;
}
pace_status check_gate(const pace_tensor *t, const char *call, const char *name, KvTensor *out) {
  if (!t || !t->data || !aligned(t->data, 4)) return fail(PACE_ERR_INVALID_ARG, "%s: %s is NULL or not 4-byte aligned", call, name);
  *out = KvTensor{static_cast<char *>(t->data), t->stride_b, t->stride_t, t->stride_h};
  return PACE_OK;
}

// Checks what the calls on states have in common and fills the device view.
pace_status check_delta(const pace_delta *delta, const pace_delta_step *s, const pace_tensor *k, const pace_tensor *v,
                        const pace_tensor *a, const pace_tensor *beta, const char *call, DeltaArgs *p) {
  if (!delta) return fail(PACE_ERR_INVALID_ARG, "%s: handle is NULL", call);
  if (!s) return fail(PACE_ERR_INVALID_ARG, "%s: step is NULL", call);
  if (s->batch < 0 || s->batch > PACE_KV_MAX_BATCH)
    return fail(PACE_ERR_INVALID_ARG, "%s: batch %d outside 0..%d", call, s->batch, PACE_KV_MAX_BATCH);
  if (s->n_tokens < 0 || s->n_tokens > 1 << 30) return fail(PACE_ERR_INVALID_ARG, "%s: n_tokens %d outside 0..2^30", call, s->n_tokens);
  if (!s->slots && s->batch > delta->cfg.n_slots)
    return fail(PACE_ERR_INVALID_ARG, "%s: batch %d without slots, but %d states", call, s->batch, delta->cfg.n_slots);
  *p = delta->args;
  p->batch = s->batch;
  p->n_tokens = s->n_tokens;
  if (s->batch == 0 || s->n_tokens == 0) return PACE_OK;
  if (!aligned(s->slots, 4) || !aligned(s->lens, 4) || !aligned(s->n_new, 4))
    return fail(PACE_ERR_INVALID_ARG, "%s: slots, lens and n_new must be 4-byte aligned", call);
  p->slots = s->slots;
  p->lens = s->lens;
  p->n_new = s->n_new;
  pace_status st;
  if ((st = check_rows(k, p->io, call, "k", &p->k)) != PACE_OK) return st;
  if ((st = check_rows(v, p->io, call, "v", &p->v)) != PACE_OK) return st;
  if ((st = check_gate(a, call, "a", &p->a)) != PACE_OK) return st;
  return check_gate(beta, call, "beta", &p->beta);
}

// ---- pages ----------------------------------------------------------------------------------------------------------------------
pace_status check_pages_config(const pace_pages_config *c) {
  if (!c) return fail(PACE_ERR_INVALID_ARG, "config is NULL");
  if (c->n_pages < 1 || c->n_pages > 1 << 30) return fail(PACE_ERR_INVALID_ARG, "n_pages %d outside 1..2^30", c->n_pages);
  if (c->page_tokens < PACE_KV_TILE || c->page_tokens > 4096 || c->page_tokens % PACE_KV_TILE)
    return fail(PACE_ERR_INVALID_ARG, "page_tokens %d is not a multiple of %d in %d..4096", c->page_tokens, PACE_KV_TILE,
                PACE_KV_TILE);
  if (c->max_batch < 1 || c->max_batch > PACE_KV_MAX_BATCH)
    return fail(PACE_ERR_INVALID_ARG, "max_batch %d outside 1..%d", c->max_batch, PACE_KV_MAX_BATCH);
  return PACE_OK;
}
// status (256 bytes), refs, src, dst, scratch, number of moves
pace_pages_layout pages_layout(const pace_pages_config *c, size_t *scratch) {
  const size_t each = ((size_t)c->n_pages * 4 + 255) & ~size_t(255);
  pace_pages_layout l;
  l.refs = 256;
  l.src = l.refs + each;
  l.dst = l.src + each;
  *scratch = l.dst + each;
  l.n_moves = *scratch + each;
  l.total_bytes = l.n_moves + 256;
  return l;
}
pace_status check_table(const pace_pages *pages, int batch, const int32_t *table, int cols, const char *call) {
  if (!pages) return fail(PACE_ERR_INVALID_ARG, "%s: handle is NULL", call);
  if (batch < 0 || batch > pages->cfg.max_batch)
    return fail(PACE_ERR_INVALID_ARG, "%s: batch %d outside 0..max_batch (%d)", call, batch, pages->cfg.max_batch);
  if (cols < 1 || (int64_t)cols * pages->cfg.page_tokens > (int64_t)1 << 30)
    return fail(PACE_ERR_INVALID_ARG, "%s: table_cols %d outside 1..2^30 tokens' pages", call, cols);
  if (batch > 0 && (!table || !aligned(table, 4))) return fail(PACE_ERR_INVALID_ARG, "%s: table is NULL or not 4-byte aligned", call);
  return PACE_OK;
}

}  // namespace

extern "C" {

// ---- the gated delta rule over states in slots ----------------------------------------------------------------------------------
pace_status pace_delta_bytes(const pace_delta_config *cfg, size_t *bytes_out) {
  pace_status st = check_delta_config(cfg);
  if (st != PACE_OK) return st;
  if (!bytes_out) return fail(PACE_ERR_INVALID_ARG, "bytes_out is NULL");
  *bytes_out = states_bytes(cfg) + 256;
  return ok();
}

pace_status pace_delta_alloc(const pace_delta_config *cfg, void *device_mem, size_t bytes, void *stream, pace_delta **out) {
  pace_status st = check_delta_config(cfg);
  if (st != PACE_OK) return st;
  if (!out) return fail(PACE_ERR_INVALID_ARG, "out is NULL");
  *out = nullptr;
  if (!device_mem || !aligned(device_mem, 256)) return fail(PACE_ERR_INVALID_ARG, "device_mem is NULL or not 256-byte aligned");
  const size_t need = states_bytes(cfg) + 256;
  if (bytes < need) return fail(PACE_ERR_INVALID_ARG, "device region of %zu bytes is smaller than the %zu the states need", bytes, need);
  pace_delta *d = new (std::nothrow) pace_delta;
  if (!d) return fail(PACE_ERR_INVALID_ARG, "host allocation of the handle failed");
  d->cfg = *cfg;
  memset(&d->args, 0, sizeof d->args);
  DeltaArgs &p = d->args;
  p.S = static_cast<float *>(device_mem);
  p.status = reinterpret_cast<int32_t *>(static_cast<char *>(device_mem) + states_bytes(cfg));
  p.H = cfg->heads;
  p.Hk = cfg->key_heads ? cfg->key_heads : cfg->heads;
  p.group = p.H / p.Hk;
  p.d = cfg->d;
  p.n_slots = cfg->n_slots;
  p.io = cfg->io_dtype;
  st = launched(cudaMemsetAsync(device_mem, 0, need, static_cast<cudaStream_t>(stream)), "clearing the states");
  if (st != PACE_OK) {
    delete d;
    return st;
  }
  *out = d;
  return st;
}

void pace_delta_free(pace_delta *delta) { delete delta; }

pace_status pace_delta_chunk(pace_delta *delta, const pace_delta_step *step, const pace_tensor *q, const pace_tensor *k,
                             const pace_tensor *v, const pace_tensor *a, const pace_tensor *beta, const pace_tensor *o,
                             void *stream) {
  DeltaArgs p;
  pace_status st = check_delta(delta, step, k, v, a, beta, "delta_chunk", &p);
  if (st != PACE_OK) return st;
  if ((q == nullptr) != (o == nullptr)) return fail(PACE_ERR_INVALID_ARG, "delta_chunk: q and o go together");
  if (step->batch == 0 || step->n_tokens == 0) return ok();
  if (q && (st = check_rows(q, p.io, "delta_chunk", "q", &p.q)) != PACE_OK) return st;
  if (q && (st = check_rows(o, p.io, "delta_chunk", "o", &p.o)) != PACE_OK) return st;
  p.write = 1;
  return launched(pace_launch_delta(p, static_cast<cudaStream_t>(stream)), "delta_chunk launch");
}

pace_status pace_delta_draft(pace_delta *delta, const pace_delta_step *step, const pace_tensor *q, const pace_tensor *k,
                             const pace_tensor *v, const pace_tensor *a, const pace_tensor *beta, const uint32_t *mask,
                             const pace_tensor *o, void *stream) {
  DeltaArgs p;
  pace_status st = check_delta(delta, step, k, v, a, beta, "delta_draft", &p);
  if (st != PACE_OK) return st;
  if (step->n_tokens > PACE_DELTA_MAX_DRAFT)
    return fail(PACE_ERR_INVALID_ARG, "delta_draft: n_tokens %d > %d", step->n_tokens, PACE_DELTA_MAX_DRAFT);
  if (step->batch == 0 || step->n_tokens == 0) return ok();
  if (!aligned(mask, 4)) return fail(PACE_ERR_INVALID_ARG, "delta_draft: mask must be 4-byte aligned");
  if ((st = check_rows(q, p.io, "delta_draft", "q", &p.q)) != PACE_OK) return st;
  if ((st = check_rows(o, p.io, "delta_draft", "o", &p.o)) != PACE_OK) return st;
  p.mask = mask;
  return launched(pace_launch_delta(p, static_cast<cudaStream_t>(stream)), "delta_draft launch");
}

pace_status pace_delta_keep(pace_delta *delta, const pace_delta_step *step, const pace_tensor *k, const pace_tensor *v,
                            const pace_tensor *a, const pace_tensor *beta, const int32_t *idx, int n_idx,
                            const int32_t *n_keep, void *stream) {
  DeltaArgs p;
  pace_status st = check_delta(delta, step, k, v, a, beta, "delta_keep", &p);
  if (st != PACE_OK) return st;
  if (n_idx < 0 || n_idx > 1 << 30) return fail(PACE_ERR_INVALID_ARG, "delta_keep: n_idx %d outside 0..2^30", n_idx);
  if (step->batch == 0 || step->n_tokens == 0 || n_idx == 0) return ok();
  if (!idx || !n_keep || !aligned(idx, 4) || !aligned(n_keep, 4))
    return fail(PACE_ERR_INVALID_ARG, "delta_keep: idx or n_keep is NULL or not 4-byte aligned");
  p.idx = idx;
  p.n_idx = n_idx;
  p.n_keep = n_keep;
  p.write = 1;
  return launched(pace_launch_delta(p, static_cast<cudaStream_t>(stream)), "delta_keep launch");
}

pace_status pace_delta_get_status(const pace_delta *delta, int clear, int *status_out, void *stream) {
  if (!delta) return fail(PACE_ERR_INVALID_ARG, "delta_get_status: handle is NULL");
  if (!status_out) return fail(PACE_ERR_INVALID_ARG, "status_out is NULL");
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  int32_t word = 0;
  cudaError_t e = cudaMemcpyAsync(&word, delta->args.status, 4, cudaMemcpyDeviceToHost, cs);
  if (e == cudaSuccess) e = cudaStreamSynchronize(cs);
  if (e == cudaSuccess && clear && word) e = cudaMemsetAsync(delta->args.status, 0, 4, cs);
  const pace_status st = launched(e, "reading the status word");
  if (st != PACE_OK) return st;
  *status_out = word;
  if (word & PACE_DELTA_TIMEOUT) return fail(PACE_ERR_TIMEOUT, "a bounded device wait gave up");
  if (word)
    return fail(PACE_ERR_STATE, "calls met%s%s", word & PACE_DELTA_BAD_SLOT ? " a slot outside the states, or one of two sequences" : "",
                word & PACE_DELTA_BAD_KEEP ? " a kept path that does not rise, or its count" : "");
  return ok();
}

pace_status pace_test_delta_wait_probe(pace_delta *delta, uint32_t ns) {
  if (!delta) return fail(PACE_ERR_INVALID_ARG, "test_delta_wait_probe: handle is NULL");
  delta->args.probe_ns = ns;
  return ok();
}

// ---- verification -----------------------------------------------------------------------------------------------------------------
pace_status pace_verify(int batch, int n_nodes, int vocab, int io_dtype, const int32_t *tokens, const pace_tensor *p,
                        const pace_tensor *q, const float *u, const uint32_t *mask, const int32_t *n_new, int32_t *idx,
                        int32_t *n_keep, int32_t *next, void *stream) {
  if (batch < 0 || batch > PACE_KV_MAX_BATCH) return fail(PACE_ERR_INVALID_ARG, "verify: batch %d outside 0..%d", batch, PACE_KV_MAX_BATCH);
  if (n_nodes < 1 || n_nodes > PACE_VERIFY_MAX_NODES)
    return fail(PACE_ERR_INVALID_ARG, "verify: n_nodes %d outside 1..%d", n_nodes, PACE_VERIFY_MAX_NODES);
  if (vocab < 1 || vocab > PACE_VERIFY_MAX_VOCAB)
    return fail(PACE_ERR_INVALID_ARG, "verify: vocab %d outside 1..%d", vocab, PACE_VERIFY_MAX_VOCAB);
  if (io_dtype != PACE_IO_BF16 && io_dtype != PACE_IO_F32) return fail(PACE_ERR_INVALID_ARG, "verify: bad io_dtype");
  if (batch == 0) return ok();
  const int es = io_dtype == PACE_IO_F32 ? 4 : 2;
  if (!p || !p->data || !aligned(p->data, es)) return fail(PACE_ERR_INVALID_ARG, "verify: p is NULL or not aligned to its elements");
  if (q && (!q->data || !aligned(q->data, es))) return fail(PACE_ERR_INVALID_ARG, "verify: q is not aligned to its elements");
  if (!tokens || !u || !idx || !n_keep || !next) return fail(PACE_ERR_INVALID_ARG, "verify: tokens, u, idx, n_keep or next is NULL");
  if (!aligned(tokens, 4) || !aligned(u, 4) || !aligned(mask, 4) || !aligned(n_new, 4) || !aligned(idx, 4) || !aligned(n_keep, 4) ||
      !aligned(next, 4))
    return fail(PACE_ERR_INVALID_ARG, "verify: tokens, u, mask, n_new, idx, n_keep and next must be 4-byte aligned");
  VerifyArgs a{batch, n_nodes, vocab, io_dtype, tokens, KvTensor{static_cast<char *>(p->data), p->stride_b, p->stride_t, 0},
               KvTensor{nullptr, 0, 0, 0}, u, mask, n_new, idx, n_keep, next};
  if (q) a.q = KvTensor{static_cast<char *>(q->data), q->stride_b, q->stride_t, 0};
  return launched(pace_launch_verify(a, static_cast<cudaStream_t>(stream)), "verify launch");
}

// ---- pages ------------------------------------------------------------------------------------------------------------------------
pace_status pace_pages_get_layout(const pace_pages_config *cfg, pace_pages_layout *out) {
  pace_status st = check_pages_config(cfg);
  if (st != PACE_OK) return st;
  if (!out) return fail(PACE_ERR_INVALID_ARG, "out is NULL");
  size_t scratch;
  *out = pages_layout(cfg, &scratch);
  return ok();
}

pace_status pace_pages_alloc(const pace_pages_config *cfg, void *device_mem, size_t bytes, void *stream, pace_pages **out) {
  pace_status st = check_pages_config(cfg);
  if (st != PACE_OK) return st;
  if (!out) return fail(PACE_ERR_INVALID_ARG, "out is NULL");
  *out = nullptr;
  if (!device_mem || !aligned(device_mem, 256)) return fail(PACE_ERR_INVALID_ARG, "device_mem is NULL or not 256-byte aligned");
  size_t scratch;
  const pace_pages_layout l = pages_layout(cfg, &scratch);
  if (bytes < l.total_bytes)
    return fail(PACE_ERR_INVALID_ARG, "device region of %zu bytes is smaller than the %zu the pages need", bytes, l.total_bytes);
  pace_pages *p = new (std::nothrow) pace_pages;
  if (!p) return fail(PACE_ERR_INVALID_ARG, "host allocation of the handle failed");
  char *base = static_cast<char *>(device_mem);
  auto at = [&](size_t off) { return reinterpret_cast<int32_t *>(base + off); };
  p->cfg = *cfg;
  p->dev = PagesDev{at(0), at(l.refs), at(l.src), at(l.dst), at(l.n_moves), at(scratch), cfg->n_pages, cfg->page_tokens};
  st = launched(cudaMemsetAsync(device_mem, 0, l.total_bytes, static_cast<cudaStream_t>(stream)), "clearing the pages");
  if (st != PACE_OK) {
    delete p;
    return st;
  }
  *out = p;
  return st;
}

void pace_pages_free(pace_pages *pages) { delete pages; }

pace_status pace_pages_select(pace_pages *pages, int batch, int32_t *table, int table_cols, int32_t *lens, const int32_t *src,
                              void *stream) {
  pace_status st = check_table(pages, batch, table, table_cols, "pages_select");
  if (st != PACE_OK) return st;
  if (batch == 0) return ok();
  if (!lens || !aligned(lens, 4) || !aligned(src, 4))
    return fail(PACE_ERR_INVALID_ARG, "pages_select: lens is NULL, or lens or src not 4-byte aligned");
  return launched(pace_launch_pages_select(pages->dev, batch, table, table_cols, lens, src, static_cast<cudaStream_t>(stream)),
                  "pages_select launch");
}

pace_status pace_pages_take(pace_pages *pages, int batch, int32_t *table, int table_cols, const int32_t *lens,
                            const int32_t *n_new, int32_t *fits, void *stream) {
  pace_status st = check_table(pages, batch, table, table_cols, "pages_take");
  if (st != PACE_OK) return st;
  if ((int64_t)batch * table_cols > INT32_MAX)             // (what the rows want is summed in 32 bits)
    return fail(PACE_ERR_UNSUPPORTED, "pages_take: a table of %lld cells, supported 2^31 - 1", (long long)batch * table_cols);
  if (batch > 0 && (!lens || !n_new || !fits || !aligned(lens, 4) || !aligned(n_new, 4) || !aligned(fits, 4)))
    return fail(PACE_ERR_INVALID_ARG, "pages_take: lens, n_new or fits is NULL or not 4-byte aligned");
  return launched(pace_launch_pages_take(pages->dev, batch, table, table_cols, lens, n_new, fits, static_cast<cudaStream_t>(stream)),
                  "pages_take launch");
}

pace_status pace_pages_compact(pace_pages *pages, int batch, int32_t *table, int table_cols, void *stream) {
  pace_status st = check_table(pages, batch, table, table_cols, "pages_compact");
  if (st != PACE_OK) return st;
  return launched(pace_launch_pages_compact(pages->dev, batch, table, table_cols, static_cast<cudaStream_t>(stream)),
                  "pages_compact launch");
}

pace_status pace_pages_get_status(const pace_pages *pages, int clear, int *status_out, void *stream) {
  if (!pages) return fail(PACE_ERR_INVALID_ARG, "pages_get_status: handle is NULL");
  if (!status_out) return fail(PACE_ERR_INVALID_ARG, "status_out is NULL");
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  int32_t word = 0;
  cudaError_t e = cudaMemcpyAsync(&word, pages->dev.status, 4, cudaMemcpyDeviceToHost, cs);
  if (e == cudaSuccess) e = cudaStreamSynchronize(cs);
  if (e == cudaSuccess && clear && word) e = cudaMemsetAsync(pages->dev.status, 0, 4, cs);
  const pace_status st = launched(e, "reading the status word");
  if (st != PACE_OK) return st;
  *status_out = word;
  if (word)
    return fail(PACE_ERR_STATE, "calls met%s%s", word & PACE_PAGES_BAD_CELL ? " a cell outside the pool, or a row without its last page or room" : "",
                word & PACE_PAGES_BAD_ROW ? " a source row outside the table" : "");
  return ok();
}

pace_status pace_kv_copy_pages(pace_kv *kv, const int32_t *src, const int32_t *dst, const int32_t *n, int max_n, void *stream) {
  if (!kv) return fail(PACE_ERR_INVALID_ARG, "kv_copy_pages: cache is NULL");
  if (max_n < 0) return fail(PACE_ERR_INVALID_ARG, "kv_copy_pages: max_n %d < 0", max_n);
  if (max_n == 0) return ok();
  if (!src || !dst || !aligned(src, 4) || !aligned(dst, 4) || !aligned(n, 4))
    return fail(PACE_ERR_INVALID_ARG, "kv_copy_pages: src or dst is NULL, or src, dst or n not 4-byte aligned");
  const KvDev &c = pace_kv_view(kv);
  return launched(pace_launch_kv_copy_pages(c.pool, pace_kv_page_bytes(kv), c.n_pages, c.status, src, dst, n, max_n,
                                            static_cast<cudaStream_t>(stream)),
                  "kv_copy_pages launch");
}

pace_status pace_kv_pool(const pace_kv *kv, void **pool, size_t *page_bytes) {
  if (!kv || !pool || !page_bytes) return fail(PACE_ERR_INVALID_ARG, "kv_pool: cache, pool or page_bytes is NULL");
  *pool = pace_kv_view(kv).pool;
  *page_bytes = pace_kv_page_bytes(kv);
  return ok();
}

}  // extern "C"
