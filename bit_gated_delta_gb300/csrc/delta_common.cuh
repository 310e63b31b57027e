// Shared by the kernels of the gated delta rule over states in slots (pace_serve.h): the device view of a call.
#pragma once

#include "kv_common.cuh"
#include "pace_serve.h"

struct DeltaArgs {
  float *S;                 // [n_slots][H][d][d]
  int32_t *status;
  int H, Hk, group, d, n_slots, io;
  int batch, n_tokens;      // rows of k, v, a and beta
  const int32_t *slots, *lens, *n_new;
  KvTensor q, k, v, o;      // q.p, o.p null: states only
  KvTensor a, beta;
  const uint32_t *mask;     // ancestors (trees of drafts)
  const int32_t *idx, *n_keep;   // kept paths
  int n_idx;
  int write;                // the states advance
  int sms;                  // multiprocessors of the device
  uint32_t probe_ns;        // failure-detection test: > 0 makes each block of the chunk kernels wait this long for what nothing signals (serve_internal.h)
};

namespace pace {
namespace delta {

// What one sequence of a call is, found by a whole warp (every lane gets it).
struct Seq {
  int n;                    // tokens, 0 where the sequence is left out
  int slot;
  bool fresh;               // begins with a zero state
};

// Tokens of sequence i as far as its counts say.
__device__ __forceinline__ int count_of(const DeltaArgs &p, int i) {
  const int rows = p.n_new ? min(max(p.n_new[i], 0), p.n_tokens) : p.n_tokens;
  return p.n_keep ? min(max(p.n_keep[i], 0), min(p.n_idx, rows)) : rows;
}

// The sequence by its own entries; bits of the status word that are wrong with it are added to `bad`.
__device__ __forceinline__ Seq sequence(const DeltaArgs &p, int b, int &bad) {
  const int lane = threadIdx.x & 31;
  Seq s;
  s.slot = p.slots ? p.slots[b] : b;
  s.fresh = p.lens && p.lens[b] == 0;
  s.n = count_of(p, b);
  if (p.n_keep) {           // the path ends before an index that does not rise inside the drafts
    const int rows = p.n_new ? min(max(p.n_new[b], 0), p.n_tokens) : p.n_tokens;
    if (p.n_keep[b] != s.n) bad |= PACE_DELTA_BAD_KEEP;
    const int32_t *row = p.idx + (long)b * p.n_idx;
    for (int i0 = 0; i0 < s.n; i0 += 32) {
      const int i = i0 + lane;
      const int x = i < s.n ? row[i] : 0, before = i > 0 && i < s.n ? row[i - 1] : -1;
      const unsigned off = __ballot_sync(0xffffffffu, i < s.n && (x <= before || x >= rows || x < 0));
      if (off) {
        s.n = i0 + __ffs(off) - 1;
        bad |= PACE_DELTA_BAD_KEEP;
      }
    }
  }
  if (s.n > 0 && (s.slot < 0 || s.slot >= p.n_slots)) {
    bad |= PACE_DELTA_BAD_SLOT;
    s.n = 0;
  }
  return s;
}
// Whether an earlier sequence of the call writes the same slot (the first of several does).
__device__ __forceinline__ bool taken(const DeltaArgs &p, int b, int slot) {
  if (!p.slots || !p.write) return false;
  bool found = false;
  for (int i = threadIdx.x & 31; i < b; i += 32) found |= p.slots[i] == slot && count_of(p, i) > 0;
  return __any_sync(0xffffffffu, found);
}

// Row of the call's tensors that holds token t of sequence b.
__device__ __forceinline__ int row_of(const DeltaArgs &p, int b, int t) { return p.idx ? p.idx[(long)b * p.n_idx + t] : t; }

}  // namespace delta
}  // namespace pace

// One call's launch (delta_step.cu chooses the kernel); the chunk kernels.
cudaError_t pace_launch_delta(const DeltaArgs &p, cudaStream_t s);
cudaError_t pace_launch_delta_chunk_bf16(const DeltaArgs &p, cudaStream_t s);
cudaError_t pace_launch_delta_chunk_f32(const DeltaArgs &p, cudaStream_t s);
