// Launchers of the calls of pace_serve.h that work on sets of sequences: verification of drafts, pages.
#pragma once

#include "kv_common.cuh"
#include "pace_serve.h"

struct VerifyArgs {
  int batch, nodes, vocab, io;
  const int32_t *tokens;
  KvTensor p, q;            // q.p null: drafts named without probabilities
  const float *u;
  const uint32_t *mask;
  const int32_t *n_new;
  int32_t *idx, *n_keep, *next;
};
cudaError_t pace_launch_verify(const VerifyArgs &p, cudaStream_t s);

// Device view of a page count.
struct PagesDev {
  int32_t *status;          // word 0: status, 1: blocks done (zero between calls), 2: pages in use (pace_pages_compact)
  int32_t *refs, *src, *dst, *n_moves, *scratch;   // scratch [n_pages]
  int n_pages, page;
};
cudaError_t pace_launch_pages_select(const PagesDev &p, int batch, int32_t *table, int cols, int32_t *lens, const int32_t *src,
                                     cudaStream_t s);
cudaError_t pace_launch_pages_take(const PagesDev &p, int batch, int32_t *table, int cols, const int32_t *lens,
                                   const int32_t *n_new, int32_t *fits, cudaStream_t s);
cudaError_t pace_launch_pages_compact(const PagesDev &p, int batch, int32_t *table, int cols, cudaStream_t s);
cudaError_t pace_launch_kv_copy_pages(char *pool, size_t page_bytes, int n_pages, int32_t *status, const int32_t *src,
                                      const int32_t *dst, const int32_t *n, int max_n, cudaStream_t s);

// Failure-detection hook for tests (no fault, no hang): with ns > 0 every later call by chunks of this handle waits in each block on an mbarrier that
// nothing signals, for ns nanoseconds, and all its waits have that limit: no products are issued, the blocks run to their end, no state changes,
// PACE_DELTA_TIMEOUT is set; what the call writes to o is undefined. ns = 0 turns it off. Host-only; PACE_ERR_INVALID_ARG for a NULL handle.
extern "C" pace_status pace_test_delta_wait_probe(pace_delta *delta, uint32_t ns);

// The device view and page size of a cache (kv_api.cu).
const KvDev &pace_kv_view(const pace_kv *kv);
size_t pace_kv_page_bytes(const pace_kv *kv);
