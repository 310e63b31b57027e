// Shared by the attention-layer kernels: device views, the tile layout of the quantized KV cache, and the page lookup.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <float.h>
#include <stdint.h>

#include "pace_common.cuh"
#include "pace_kv.h"

// Device view of one cache, passed by value.
struct KvDev {
  char *pool;               // [n_pages][kv_heads][page_tokens / 32] tiles
  int32_t *status;
  int32_t *count;           // arrivals of the split items of an attention call; zero between calls
  float *part;              // partial results of the split items
  int Hq, Hkv, group;       // group = query heads per KV head
  int d, bits, page, n_pages, io;
  int table_cols, batch, n_tokens;
  const int32_t *lens, *n_new, *table;
};

struct KvTensor {
  char *p;
  int64_t sb, st, sh;       // strides in elements
};

struct KvRope {
  const float2 *table;
  int rot, max_pos, interleaved;
};

namespace pace {
namespace kv {

constexpr int TILE = PACE_KV_TILE;
constexpr int GROUP = PACE_KV_GROUP;

// One 32-token tile of one head. Rows of D*BITS/8 bytes per token for K, then for V; scales bf16 [NG][32] and zero points
// u8 [NG][32] in row order (`pos`, `vpos`). The orders inside a row are those of the attention kernel's fragments: every
// shared-memory read of a warp then covers all 32 banks once, straight from the bytes a bulk copy brought.
//  * mma row r of a 16-token block holds token tau(r): tau(2m) = m, tau(2m+1) = 4 + (m^3) in each half of 8, so that the
//    two rows of a value pair and neighbouring key rows differ in the token bits that pick the banks;
//  * key dims 64g + 16c + .. belong to lane c of a quad: one 16-byte chunk (8 bits: of group g; 4 bits: of groups g, g+1);
//  * value dims 64g + 8j + .. belong to lane row j: one 8-byte unit (4 bits at D = 64: 4 bytes);
//  * chunks and units are XORed with low token bits where a row spans all banks.
template <int D, int BITS>
struct Tile {
  static constexpr int NG = D / GROUP;
  static constexpr int ROW = D * BITS / 8;
  static constexpr int K = 0, V = TILE * ROW, KS = 2 * TILE * ROW, VS = KS + NG * TILE * 2, KZ = VS + NG * TILE * 2,
                       VZ = KZ + (BITS == 4 ? NG * TILE : 0), BYTES = VZ + (BITS == 4 ? NG * TILE : 0);
  static_assert(BYTES % 16 == 0, "bulk copies move 16-byte pieces");

  // byte offset of key chunk ch (16 bytes; D = 64 at 4 bits: 8 bytes) of token t
  __host__ __device__ static constexpr int kchunk(int t, int ch) {
    if (BITS == 4 && D == 64) return K + t * ROW + ch * 8;
    return K + t * ROW + (ROW >= 128 ? (ch ^ ((t & 1) << 2)) : ch) * 16;
  }
  // byte offset of value unit u (8 bytes; D = 64 at 4 bits: 4 bytes) of token t
  __host__ __device__ static constexpr int vunit(int t, int u) {
    if (BITS == 4 && D == 64) return V + t * ROW + u * 4;
    return V + t * ROW + (ROW >= 128 ? (u ^ ((t & 3) << 2)) : (u ^ (((t >> 1) & 1) << 2))) * 8;
  }
  // byte offset of the codes of dims 8a .. 8a+7 (one word at 4 bits, two at 8)
  __host__ __device__ static constexpr int k8(int t, int a) {
    const int g = a >> 3, w = a & 7;
    if (BITS == 8) return kchunk(t, g * 4 + (w >> 1)) + (w & 1) * 8;
    if (D == 64) return kchunk(t, w >> 1) + (w & 1) * 4;
    return kchunk(t, (g >> 1) * 4 + (w >> 1)) + (g & 1) * 8 + (w & 1) * 4;
  }
  __host__ __device__ static constexpr int v8(int t, int a) {
    const int g = a >> 3, j = a & 7;
    if (BITS == 8) return vunit(t, g * 8 + j);
    if (D == 64) return vunit(t, j);
    return vunit(t, (g >> 1) * 8 + j) + (g & 1) * 4;
  }
  __host__ __device__ static constexpr int pos(int t) {
    const int u = t & 7, r = u < 4 ? 2 * u : 2 * ((u - 4) ^ 3) + 1;
    return r * 4 + (t >> 4) * 2 + ((t >> 3) & 1);
  }
  // place of a value's zero point: rows 2c and 2c+1, which share a register, side by side
  __host__ __device__ static constexpr int vpos(int t) { return (pos(t) >> 3) * 8 + (pos(t) & 3) * 2 + ((pos(t) >> 2) & 1); }
};

// mma row r (0..7) of each half of a 16-token block -> token in that half
__host__ __device__ constexpr int tau(int r) { return (r & 1) ? 4 + ((r >> 1) ^ 3) : (r >> 1); }

// Codes of eight consecutive elements: 4 bits: element 2p+e at nibble p + 4e of one word, so that (w >> 4p) & 0x000F000F is
// the pair (2p, 2p+1) in two halves; 8 bits: elements 0, 2, 1, 3 of each word from its lowest byte, for the same reason.
template <int BITS>
__device__ __forceinline__ uint2 pack8(const uint32_t (&u)[8]) {
  uint2 w = make_uint2(0, 0);
  if (BITS == 4) {
#pragma unroll
    for (int p = 0; p < 4; ++p) w.x |= (u[2 * p] << (4 * p)) | (u[2 * p + 1] << (16 + 4 * p));
  } else {
    w.x = u[0] | (u[2] << 8) | (u[1] << 16) | (u[3] << 24);
    w.y = u[4] | (u[6] << 8) | (u[5] << 16) | (u[7] << 24);
  }
  return w;
}
template <int BITS>
__device__ __forceinline__ void unpack8(uint2 w, int (&u)[8]) {
  if (BITS == 4) {
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      u[2 * p] = (w.x >> (4 * p)) & 15;
      u[2 * p + 1] = (w.x >> (16 + 4 * p)) & 15;
    }
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t x = h ? w.y : w.x;
      u[4 * h] = x & 255;
      u[4 * h + 2] = (x >> 8) & 255;
      u[4 * h + 1] = (x >> 16) & 255;
      u[4 * h + 3] = x >> 24;
    }
  }
}

// Page of slot `slot` of sequence b, or -1 when the slot is outside the table or the page outside the pool. (A table holds 2^30 tokens
// at most, so that slots inside it divide in 32 bits.)
__device__ __forceinline__ int page_of(const KvDev &c, int b, long slot) {
  if (slot < 0 || slot >= (long)c.table_cols * c.page) return -1;
  const unsigned col = (unsigned)slot / (unsigned)c.page;
  const int pg = c.table[(long)b * c.table_cols + col];
  return pg >= 0 && pg < c.n_pages ? pg : -1;
}
// Tile holding `slot` (page already checked): pages and heads are 64-bit offsets.
template <int TB>
__device__ __forceinline__ char *tile_at(const KvDev &c, int page, int head, long slot) {
  const unsigned tiles = (unsigned)c.page / TILE;
  return c.pool + (((long)page * c.Hkv + head) * tiles + ((unsigned)slot / TILE) % tiles) * (long)TB;
}
// Index in the pool of tile t (tokens 32t ..) of sequence b and KV head h, or -1; tpp = tiles a page.
__device__ __forceinline__ int tile_index(const KvDev &c, int b, int h, int t, int tpp) {
  const int col = t / tpp;
  if (col >= c.table_cols) return -1;
  const int pg = c.table[(long)b * c.table_cols + col];
  return pg >= 0 && pg < c.n_pages ? (pg * c.Hkv + h) * tpp + (t - col * tpp) : -1;
}
__device__ __forceinline__ int new_tokens(const KvDev &c, int b) {
  return c.n_new ? min(max(c.n_new[b], 0), c.n_tokens) : c.n_tokens;
}

}  // namespace kv
}  // namespace pace

// Kernel launchers (nothing synchronises).
cudaError_t pace_launch_rope_table(const pace_rope_config &r, float2 *table, cudaStream_t s);
cudaError_t pace_launch_rope(const KvRope &r, int n, int heads, int d, int io, const KvTensor &x, const int32_t *pos,
                             const KvTensor &out, int inverse, cudaStream_t s);
cudaError_t pace_launch_kv_append(const KvDev &c, const KvTensor &q, const KvTensor &k, const KvTensor &v,
                                  const KvTensor &qo, const KvRope &r, const int32_t *pos, cudaStream_t s);
cudaError_t pace_launch_kv_read(const KvDev &c, const int32_t *first, const int32_t *end, const KvTensor &k,
                                const KvTensor &v, cudaStream_t s);
cudaError_t pace_launch_kv_keep(const KvDev &c, int max_new, const int32_t *idx, const int32_t *n_keep, cudaStream_t s);
cudaError_t pace_launch_kv_attend(const KvDev &c, const KvTensor &q, const uint32_t *mask, float scale, const KvTensor &o,
                                  cudaStream_t s);
// Sizes of the attention call's work area (counters and partial results) for a configuration.
void pace_kv_attend_work(const pace_kv_config &cfg, size_t *count_bytes, size_t *part_bytes);
