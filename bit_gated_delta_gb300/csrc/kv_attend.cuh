// Attention of a few query rows over the quantized KV cache: o = sum_j p_j v_j, p = softmax(scale q.k_j).
//
// The rows of one KV head are its group's query heads for every new token, packed (row r = token r/G, head r%G), 8*NT of them a
// work item. A warp walks 32-token tiles with the running maximum and sum of the softmax; everything stays in registers:
//   S^T = K Q^T     A = 16 tokens of key codes (built in registers), B = the rows' queries
//   O^T = V^T P^T   A = 16 dims of value codes for 16 tokens, B = the weights, transposed inside the warp by movmatrix
// With tokens (then dims) on the 16-row side of the MMA, eight rows cost one m16n8k16 per 256 cached elements, half of what
// rows on that side would take, and the softmax handles no empty rows.
//
// The cache is bound by bytes only if its codes reach the tensor cores in about three instructions each (46 4-bit elements a
// clock and SM at the measured 6.8 TB/s against 128 lanes, half of that for bit operations), so codes become fp16 under the
// exponent of 1024 by one bit operation a pair and one exact subtraction on the other pipe (the conversion is described by Kim et al.,
// "Who Says Elephants Can't Run", 2022), and enter the products as integers.
// The scales of a key group multiply the fp32 accumulators, those of a value group enter the exponent of the weights. Queries and
// weights are fp16 relative to a power of two (11 bits); with fp32 I/O both are three bf16 parts, so nothing is rounded below 2^-24.
//
// Work: the tiles of all (sequence, KV head, row block) items form one line, cut into equal shares, one a block; a block's warps
// take its tiles in turn, each through its own ring of tiles filled by bulk copies (one copy a tile). Items cut by a share
// boundary leave partial results; the last block to finish an item joins them, in block order, so results do not depend on timing.
// Measured, one token, cold: 16 sequences of 30,000 to 32,767 tokens, 48 and 8 heads of 128, 8 bits 159 us (6.7 TB/s; 180 us after
// other writes have filled the L2); 64 sequences of 512 to 4096 tokens, 32 and 8 heads of 128, 4 bits 51 us (bytes 24; its instructions,
// three an element, would issue in 24 too: the rest are waits, of which the counters name fixed latency and barriers first. Most items
// are cut in two, each cut has its block-wide barriers and a join by one warp, and every call a chain of about 8 us); one sequence of
// 300 tokens 8 us. fp32 I/O: 16 sequences of 30,000 to 32,000 tokens, 32 and 8 heads of 64, 8 bits 162 us (bytes 77), of 128, 4 bits 219
// (82); trees of 25 tokens, 8 sequences of 2000 to 4000, heads of 128 152 us; chunks of 256, 2 sequences, 378 us: three products a tile, and
// eight rows an item, so that each pass over a head's tiles serves eight rows.
#pragma once

#include <cuda_fp16.h>

#include <algorithm>

#include "kv_common.cuh"
#include "umma.cuh"

namespace pace {
namespace kv {

// Wait for a barrier's phase, suspended by the hardware for up to a millisecond at a time so that waiting warps leave the issue slots
// to the others; gives up after about a second.
__device__ __forceinline__ bool bar_wait(uint64_t *bar, uint32_t parity) {
  for (int i = 0; i < 1000; ++i) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(umma::smem_u32(bar)), "r"(parity), "r"(1000000u)
        : "memory");
    if (ok) return true;
  }
  return false;
}
constexpr int MAX_BLOCKS = 1024;       // blocks of a launch (sizes the work area)
constexpr int MAX_ROWS_FLOATS = 8 * 258;   // floats of one partial result: 8*NT rows of D + 2 with NT * D <= 256 (rounded up)

__host__ __device__ constexpr int part_floats(int D, int NT) { return 8 * NT * (D + 2); }

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                              uint32_t b1) {   // d = A B
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}
__device__ __forceinline__ uint32_t movmatrix(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t sub_bf16x2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 r = __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&a), *reinterpret_cast<const __nv_bfloat162 *>(&b));
  return *reinterpret_cast<const uint32_t *>(&r);
}
__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// pair p of a word of 4-bit codes as bf16 128 + u
__device__ __forceinline__ uint32_t pair4(uint32_t w, int p) { return ((w >> (4 * p)) & 0x000F000Fu) | 0x43004300u; }
// bytes 0 and 2 of w (codes c + 128) as the exact bf16 pair of c
__device__ __forceinline__ uint32_t pair8(uint32_t w) {
  return sub_bf16x2((w & 0x007F007Fu) | 0x43004300u, (~w & 0x00800080u) | 0x43004300u);
}

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float log2_approx(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float exp2i(int e) { return __int_as_float((e + 127) << 23); }   // -126 <= e <= 127
__device__ __forceinline__ uint32_t h2mul(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2 *>(&a), *reinterpret_cast<const __half2 *>(&b));
  return *reinterpret_cast<const uint32_t *>(&r);
}
__device__ __forceinline__ uint32_t h2add(uint32_t a, uint32_t b) {
  const __half2 r = __hadd2(*reinterpret_cast<const __half2 *>(&a), *reinterpret_cast<const __half2 *>(&b));
  return *reinterpret_cast<const uint32_t *>(&r);
}
__device__ __forceinline__ uint32_t h2sub(uint32_t a, uint32_t b) {
  const __half2 r = __hsub2(*reinterpret_cast<const __half2 *>(&a), *reinterpret_cast<const __half2 *>(&b));
  return *reinterpret_cast<const uint32_t *>(&r);
}
__device__ __forceinline__ uint32_t h2fma(uint32_t a, uint32_t b, uint32_t c) {
  const __half2 r = __hfma2(*reinterpret_cast<const __half2 *>(&a), *reinterpret_cast<const __half2 *>(&b),
                            *reinterpret_cast<const __half2 *>(&c));
  return *reinterpret_cast<const uint32_t *>(&r);
}
__device__ __forceinline__ uint32_t h2fms(uint32_t a, uint32_t b, uint32_t c) {   // a b - c
  const __half2 r = __hfma2(*reinterpret_cast<const __half2 *>(&a), *reinterpret_cast<const __half2 *>(&b),
                            __hneg2(*reinterpret_cast<const __half2 *>(&c)));
  return *reinterpret_cast<const uint32_t *>(&r);
}
__device__ __forceinline__ uint32_t h2pack(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&v);
}
// The four pairs of a word of 4-bit codes as fp16 u - z, exactly: the nibble at bit 0 of a half under the exponent of 1024 reads
// 1024 + u, the one at bit 4 reads 1024 + 16 u = 16 (64 + u). z1024 and z64 are the pairs 1024 + z and 64 + z.
// `magic` is 0x64006400, kept in a register (opaque) so that mask and exponent are one three-input operation.
__device__ __forceinline__ uint32_t opaque(uint32_t x) {
  uint32_t y;
  asm volatile("mov.b32 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t mask_or(uint32_t w, uint32_t mask, uint32_t magic) {
  uint32_t y;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(y) : "r"(w), "r"(mask), "r"(magic));
  return y;
}
__device__ __forceinline__ void codes4(uint32_t w, uint32_t z1024, uint32_t z64, uint32_t magic, uint32_t (&r)[4]) {
  constexpr uint32_t SIXTEENTH = 0x2C002C00u;
  const uint32_t x = w >> 8;
  r[0] = h2sub(mask_or(w, 0x000F000Fu, magic), z1024);
  r[1] = h2fms(mask_or(w, 0x00F000F0u, magic), SIXTEENTH, z64);
  r[2] = h2sub(mask_or(x, 0x000F000Fu, magic), z1024);
  r[3] = h2fms(mask_or(x, 0x00F000F0u, magic), SIXTEENTH, z64);
}
// Bytes (0, 2) and (1, 3) of a word of 8-bit codes c + 128 as fp16 c.
__device__ __forceinline__ void codes8(uint32_t w, uint32_t &even, uint32_t &odd) {
  constexpr uint32_t M1152 = 0xE480E480u;
  even = h2add(__byte_perm(w, 0x64646464u, 0x4240), M1152);
  odd = h2add(__byte_perm(w, 0x64646464u, 0x4341), M1152);
}

// x ~= sum of PARTS bf16 parts, for a pair.
template <int PARTS>
__device__ __forceinline__ void split_pair(float x0, float x1, uint32_t (&p)[PARTS]) {
#pragma unroll
  for (int i = 0; i < PARTS; ++i) {
    p[i] = pack_bf16x2(x0, x1);
    x0 -= __uint_as_float(p[i] << 16);
    x1 -= __uint_as_float(p[i] & 0xFFFF0000u);
  }
}

struct AttendArgs {
  KvDev c;
  KvTensor q, o;
  const uint32_t *mask;
  float scale_log2;     // softmax scale * log2(e)
  int row_blocks;       // items of one (sequence, KV head)
  unsigned item0, items;   // the items of each sequence in this launch (numbered by head, then row block): all, or a range of one's
  uint32_t group_inv;   // ceil(2^31 / group)
};
// Token of a row, row / group: exact for rows below 2^31 / group. The kernel of many rows uses it (a division before every
// address took trees from 64 to 68 us); in the kernel of few rows, where a division is rare, it only moved the compiler's choices: 64
// sequences of 8192 tokens 136 us, not 129.
__device__ __forceinline__ int row_token(const AttendArgs &p, int row) { return (int)(((uint64_t)(uint32_t)row * p.group_inv) >> 31); }

// One stretch of an item on the line of tiles.
struct Segment {
  int b, h, rb;         // item
  int tile, end;        // tiles [tile, end) of it
  int tiles;            // of the whole item
};
// One sequence of the call: cached tokens, new tokens, both together (no more than the page table holds).
struct Seq {
  int len, fresh, tokens;
};

__device__ __forceinline__ Seq sequence(const KvDev &c, int b, bool report) {
  const int cap = c.table_cols * c.page, len = c.lens[b];
  const int fresh = new_tokens(c, b);
  Seq q{max(len, 0), fresh, 0};
  const long n = (long)q.len + fresh;
  q.tokens = (int)min(n, (long)cap);
  if (report && (n > cap || len < 0)) atomicOr(c.status, PACE_KV_BAD_PAGE);
  return q;
}
// The sequences, and the exclusive prefix sums of their items' tiles of TOK tokens (at least one each), in shared memory:
// seq[0..batch), cum[0..batch]; returns the most tiles of an item. `warp_sums` holds 64 values. (32 bits: the host keeps the line of one
// launch below 2^31 tiles.)
template <int TOK>
__device__ __forceinline__ unsigned tile_line(const KvDev &c, unsigned per_seq, Seq *seq, unsigned *cum, unsigned *warp_sums) {
  const int n = c.batch, nt = blockDim.x, per = (n + nt - 1) / nt, b0 = threadIdx.x * per;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  unsigned s = 0, most = 0;
  for (int i = 0; i < per && b0 + i < n; ++i) {
    const Seq q = sequence(c, b0 + i, blockIdx.x == 0);
    seq[b0 + i] = q;
    const unsigned tiles = max((q.tokens + TOK - 1) / TOK, 1);
    most = max(most, tiles);
    s += tiles * per_seq;
    cum[b0 + i + 1] = s;
  }
  if (threadIdx.x == 0) cum[0] = 0;
  if (n <= 32) {                                       // one warp holds them all
    if (w == 0) {
      most = __reduce_max_sync(0xffffffffu, most);
      if (lane == 0) warp_sums[32] = most;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned y = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += y;
      }
      if (lane < n) cum[lane + 1] = s;
    }
    __syncthreads();
    return warp_sums[32];
  }
  most = __reduce_max_sync(0xffffffffu, most);
  if (lane == 0) warp_sums[32 + w] = most;
  unsigned x = s;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_sums[w] = x;
  __syncthreads();
  unsigned base = x - s;
  for (int i = 0; i < w; ++i) base += warp_sums[i];
  for (int i = 0; i < per && b0 + i < n; ++i) cum[b0 + i + 1] += base;
  most = 0;
  for (int i = 0; i < nt >> 5; ++i) most = max(most, warp_sums[32 + i]);
  __syncthreads();
  return most;
}

// The item that holds line position p, and its stretch from there up to hi.
template <int TOK>
__device__ __forceinline__ Segment segment_at(const Seq *seq, const unsigned *cum, const AttendArgs &a, unsigned p, unsigned hi) {
  int lo = 0, up = a.c.batch;                  // last b with cum[b] <= p
  while (up - lo > 1) {
    const int mid = (lo + up) >> 1;
    if (cum[mid] <= p) lo = mid;
    else up = mid;
  }
  Segment s;
  s.b = lo;
  s.tiles = max((seq[lo].tokens + TOK - 1) / TOK, 1);
  const unsigned r = p - cum[lo], k = r / (unsigned)s.tiles, item = a.item0 + k;
  s.tile = (int)(r - k * s.tiles);
  s.h = item / a.row_blocks;
  s.rb = item - s.h * a.row_blocks;
  s.end = (int)min((unsigned)s.tiles, s.tile + (hi - p));
  return s;
}
// Where the line is cut: an item a block, where there are no more items than blocks and the longest is within `extra` tiles of an equal
// share; else at every `share` tiles, since an item that blocks share costs each of them the writing of a part and one of them the
// joining.
struct Cuts {
  unsigned share, total, per_seq;
  bool each;
};
template <int TOK>
__device__ __forceinline__ unsigned cut_at(const Seq *seq, const unsigned *cum, int batch, const Cuts &c, unsigned i) {
  if (!c.each) return i > c.total / c.share ? c.total : min(i * c.share, c.total);
  const unsigned b = i / c.per_seq;
  return b >= (unsigned)batch ? c.total : cum[b] + (i - b * c.per_seq) * max((seq[b].tokens + TOK - 1) / TOK, 1);
}
// This block's stretch [lo, hi). No share is less than `least` tiles, and items of up to `whole` tiles on average are not cut finer.
template <int TOK>
__device__ __forceinline__ Cuts make_cuts(const Seq *seq, const unsigned *cum, int batch, unsigned per_seq, unsigned most, unsigned least,
                                          unsigned whole, unsigned extra, unsigned &lo, unsigned &hi) {
  Cuts c;
  c.total = cum[batch];
  c.per_seq = per_seq;
  const unsigned items = per_seq * batch, mean = c.total / items, even = (c.total + gridDim.x - 1) / gridDim.x;
  c.each = items <= gridDim.x && most <= even + extra;
  c.share = max(even, mean <= whole ? mean : least);
  lo = cut_at<TOK>(seq, cum, batch, c, blockIdx.x);
  hi = cut_at<TOK>(seq, cum, batch, c, blockIdx.x + 1);
  return c;
}

// The stretches of a block from line position lo on, SEGS at most, into shared memory by one warp (a lane each): the one at lo, then
// whole items until hi. Returns how many; segs[n].tile of the one after them is the line position where they end.
constexpr int SEGS = 32;
template <int TOK>
__device__ __forceinline__ int list_segments(const Seq *seq, const unsigned *cum, const AttendArgs &p, unsigned lo, unsigned hi,
                                             Segment *segs) {
  const int lane = threadIdx.x & 31, row_blocks = p.row_blocks;
  const Segment a = segment_at<TOK>(seq, cum, p, lo, hi);
  const unsigned item = (unsigned)a.h * row_blocks + a.rb - p.item0 + lane, db = item / p.items;
  Segment s = a;
  unsigned at = lo;
  bool in = lane == 0;
  if (lane > 0 && a.b + (int)db < p.c.batch) {
    s.b = a.b + db;
    s.tiles = max((seq[s.b].tokens + TOK - 1) / TOK, 1);
    const unsigned k = item - db * p.items, own = p.item0 + k;
    s.h = own / row_blocks;
    s.rb = own - s.h * row_blocks;
    s.tile = 0;
    at = cum[s.b] + k * s.tiles;
    in = at < hi;
    s.end = in ? (int)min((unsigned)s.tiles, hi - at) : 0;
  }
  const int n = __popc(__ballot_sync(0xffffffffu, in));
  if (in) segs[lane] = s;
  if (lane == n - 1) segs[SEGS].tile = (int)(at + (s.end - s.tile));
  return n;
}

// Eight outputs of a row, bf16 or fp32.
template <bool F32>
__device__ __forceinline__ void store_out(char *dst, const float (&y)[8], float f) {
  if (F32) {
    reinterpret_cast<float4 *>(dst)[0] = make_float4(y[0] * f, y[1] * f, y[2] * f, y[3] * f);
    reinterpret_cast<float4 *>(dst)[1] = make_float4(y[4] * f, y[5] * f, y[6] * f, y[7] * f);
  } else {
    *reinterpret_cast<uint4 *>(dst) = make_uint4(pack_bf16x2(y[0] * f, y[1] * f), pack_bf16x2(y[2] * f, y[3] * f),
                                                 pack_bf16x2(y[4] * f, y[5] * f), pack_bf16x2(y[6] * f, y[7] * f));
  }
}

// One more block has left its part of an item: whether it was the last of n. The caller's barrier before and after make the parts of
// all blocks visible to the block that joins them.
__device__ __forceinline__ bool last_part(int32_t *count, int n) {
  int before;
  asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;" : "=r"(before) : "l"(count) : "memory");
  if (before != n - 1) return false;
  *count = 0;
  return true;
}

// Join the partial results of one item (rows of D values, then maximum and sum of each row) that blocks first..last left, and write
// its outputs. All THREADS threads of the block take part. A thread takes pieces of eight values, two at a time and four parts of
// each, so that their loads go out together; where there are fewer pieces than threads, groups of threads share the parts and
// meet in `area` (JoinShape::AREA bytes).
template <int D, int ROWS, int THREADS>
struct JoinShape {
  static constexpr int PIECES = ROWS * D / 8;
  static constexpr int GROUPS = THREADS > PIECES ? THREADS / PIECES : 1;
  static constexpr size_t AREA = (size_t)(GROUPS - 1) * PIECES * 10 * 4;
};
struct JoinSum {
  float M, L, y[8];
  __device__ __forceinline__ void clear() {
    M = -INFINITY, L = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) y[k] = 0.0f;
  }
  __device__ __forceinline__ void raise(float top) {
    const float keep = M == -INFINITY ? 0.0f : exp2_approx(M - top);
    M = top;
    L *= keep;
#pragma unroll
    for (int k = 0; k < 8; ++k) y[k] *= keep;
  }
  __device__ __forceinline__ void add(float m, float l, const float4 &u, const float4 &v) {
    const float f = m == -INFINITY ? 0.0f : exp2_approx(m - M);
    L += f * l;
    y[0] += f * u.x, y[1] += f * u.y, y[2] += f * u.z, y[3] += f * u.w;
    y[4] += f * v.x, y[5] += f * v.y, y[6] += f * v.z, y[7] += f * v.w;
  }
};
template <int D, int ROWS, int THREADS, bool F32>
__device__ void join_parts(const AttendArgs &p, const float *parts, long stride, int first, int last, int b, int h, int row0, int fresh,
                           float *area) {
  using J = JoinShape<D, ROWS, THREADS>;
  constexpr int CH = D / 8, U = J::GROUPS > 1 ? 1 : 2, P = 4;
  const int G = p.c.group, rows = p.c.n_tokens * G, grp = J::GROUPS > 1 ? threadIdx.x / J::PIECES : 0;
  JoinSum sum[U];
  auto gather = [&](int x0, int step) {               // pieces x0, x0 + step: this group's parts
    bool live[U];
#pragma unroll
    for (int q = 0; q < U; ++q) {
      sum[q].clear();
      live[q] = x0 + q * step < J::PIECES && row0 + (x0 + q * step) / CH < rows;
    }
    for (int i0 = first + grp; i0 <= last; i0 += P * J::GROUPS) {
      float2 e[U][P];
      float4 u[U][P], v[U][P];
#pragma unroll
      for (int q = 0; q < U; ++q)
#pragma unroll
        for (int k = 0; k < P; ++k) {
          const int i = i0 + k * J::GROUPS, x = x0 + q * step, row = x / CH;
          const float *src = parts + (2 * i + (i == first)) * stride;
          e[q][k] = make_float2(-INFINITY, 0.0f);
          u[q][k] = v[q][k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          if (i <= last && live[q]) {
            e[q][k] = __ldcg(reinterpret_cast<const float2 *>(src + ROWS * D + 2 * row));
            u[q][k] = __ldcg(reinterpret_cast<const float4 *>(src + x * 8));
            v[q][k] = __ldcg(reinterpret_cast<const float4 *>(src + x * 8 + 4));
          }
        }
#pragma unroll
      for (int q = 0; q < U; ++q) {
        float top = sum[q].M;
#pragma unroll
        for (int k = 0; k < P; ++k) top = fmaxf(top, e[q][k].x);
        sum[q].raise(top);
#pragma unroll
        for (int k = 0; k < P; ++k) sum[q].add(e[q][k].x, e[q][k].y, u[q][k], v[q][k]);
      }
    }
  };
  auto write = [&](int x, JoinSum &s) {
    const int rr = row0 + x / CH, t = rr / G;
    if (x >= J::PIECES || rr >= rows) return;
    char *dst = p.o.p + (b * p.o.sb + (long)t * p.o.st + (long)(h * G + rr - t * G) * p.o.sh + (x % CH) * 8) * (F32 ? 4 : 2);
    store_out<F32>(dst, s.y, t < fresh && s.L > 0.0f ? 1.0f / s.L : 0.0f);
  };
  if (J::GROUPS == 1) {
    for (int x = threadIdx.x; x < J::PIECES; x += U * THREADS) {
      gather(x, THREADS);
#pragma unroll
      for (int q = 0; q < U; ++q) write(x + q * THREADS, sum[q]);
    }
  } else {
    const int x = threadIdx.x % J::PIECES;
    float2 *ml = reinterpret_cast<float2 *>(area);
    float4 *ys = reinterpret_cast<float4 *>(area + (J::GROUPS - 1) * J::PIECES * 2);
    if (grp < J::GROUPS) gather(x, 0);
    if (grp > 0 && grp < J::GROUPS) {
      const int at = (grp - 1) * J::PIECES + x;
      ml[at] = make_float2(sum[0].M, sum[0].L);
      ys[2 * at] = make_float4(sum[0].y[0], sum[0].y[1], sum[0].y[2], sum[0].y[3]);
      ys[2 * at + 1] = make_float4(sum[0].y[4], sum[0].y[5], sum[0].y[6], sum[0].y[7]);
    }
    __syncthreads();
    if (grp == 0) {
      for (int q = 0; q < J::GROUPS - 1; ++q) {
        const int at = q * J::PIECES + x;
        const float2 e = ml[at];
        sum[0].raise(fmaxf(sum[0].M, e.x));
        sum[0].add(e.x, e.y, ys[2 * at], ys[2 * at + 1]);
      }
      write(x, sum[0]);
    }
    __syncthreads();
  }
}

template <int D, int BITS, int NT, int PARTS, int NW, int STAGES>
struct AttendShape {
  using L = Tile<D, BITS>;
  static constexpr int ROWS = 8 * NT, THREADS = NW * 32;
  static constexpr int QROW = D * (PARTS > 1 ? 4 : 2);                  // bytes of a query row
  static constexpr size_t RING = (size_t)NW * STAGES * L::BYTES;
  static constexpr size_t QRAW = (size_t)ROWS * QROW;                   // queries of the next segment
  static constexpr size_t QF = (size_t)NT * L::NG * PARTS * 1024;       // queries as fragments
  static constexpr size_t SCRATCH = (size_t)(NW - 1) * ROWS * D * 4;    // the warps' results, but the first one's
  static_assert(JoinShape<D, ROWS, THREADS>::AREA <= SCRATCH, "the groups of a join meet in the warps' areas");
  static constexpr size_t ML = (size_t)NW * ROWS * 2 * 4;
  static constexpr size_t OQRAW = RING, OQF = OQRAW + QRAW, OSCR = OQF + QF, OML = OSCR + SCRATCH, OROWS = OML + ML,
                          OBAR = OROWS + ROWS * 4, OSEG = OBAR + (NW * STAGES * 8 + 15) / 16 * 16,
                          OSUM = OSEG + (SEGS + 1) * sizeof(Segment), OCUM = OSUM + 64 * 4 + 16;
  // prefix sums of up to this many sequences: few capacities, so that the occupancy of each is asked for once
  __host__ __device__ static constexpr int capacity(int batch) { return batch <= 64 ? 64 : batch <= 256 ? 256 : PACE_KV_MAX_BATCH; }
  static constexpr size_t smem(int batch) { return OCUM + (size_t)(capacity(batch) + 1) * 4 + (size_t)capacity(batch) * sizeof(Seq); }
};

__device__ __forceinline__ void cp_async16(void *dst, const void *src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(umma::smem_u32(dst)), "l"(src), "r"(in ? 16 : 0) : "memory");
}

template <int D, int BITS, int NT, int PARTS, int NW, int STAGES, int MINB>
__global__ void __launch_bounds__(NW * 32, MINB) attend_kernel(AttendArgs p) {
  using S = AttendShape<D, BITS, NT, PARTS, NW, STAGES>;
  using L = Tile<D, BITS>;
  constexpr int NG = L::NG, ROWS = S::ROWS, ES = PARTS > 1 ? 4 : 2;
  constexpr bool F32 = PARTS > 1;
  extern __shared__ __align__(128) char smem[];
  char *qraw = smem + S::OQRAW;
  uint32_t *qf = reinterpret_cast<uint32_t *>(smem + S::OQF);
  float *scratch = reinterpret_cast<float *>(smem + S::OSCR);
  float *ml = reinterpret_cast<float *>(smem + S::OML);
  float *rowmul = reinterpret_cast<float *>(smem + S::OROWS);     // what a row's scores are multiplied by
  Segment *segs = reinterpret_cast<Segment *>(smem + S::OSEG);
  unsigned *wsum = reinterpret_cast<unsigned *>(smem + S::OSUM);
  int *flag = reinterpret_cast<int *>(wsum + 64);
  unsigned *cum = reinterpret_cast<unsigned *>(smem + S::OCUM);
  Seq *seq = reinterpret_cast<Seq *>(cum + S::capacity(p.c.batch) + 1);

  const KvDev &c = p.c;
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5, j = lane >> 2, cc = lane & 3;
  const int G = c.group, T = c.n_tokens, words = (T + 31) >> 5;
  char *ring = smem + (size_t)w * STAGES * L::BYTES;
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + S::OBAR) + w * STAGES;
  if (lane < STAGES) umma::mbar_init(&bars[lane], 1);
  umma::mbar_fence_init();
  pdl_enter();
  const unsigned most = tile_line<TILE>(c, p.items, seq, cum, wsum);

  // no share is less than a tile for every warp, or a whole average item of up to three: joining one costs about as much as three
  // rounds of tiles
  unsigned lo, hi;
  const Cuts cuts = make_cuts<TILE>(seq, cum, c.batch, p.items, most, NW, 3 * NW, 4 * NW, lo, hi);
  if (lo >= hi) return;
  auto segment = [&](unsigned at) { return segment_at<TILE>(seq, cum, p, at, hi); };

  // ---- queries of a segment, copied one segment ahead; rows past the new tokens are not read (they may hold anything) but zeros
  auto copy_queries = [&](const Segment &s) {
    constexpr int CH = S::QROW / 16;
    const int fresh = seq[s.b].fresh;                 // (T at most)
    for (int x = tid; x < ROWS * CH; x += S::THREADS) {
      const int row = x / CH, ch = x % CH, rr = s.rb * ROWS + row, t = rr / G;
      const bool in = t < fresh;
      const char *src = in ? p.q.p + (s.b * p.q.sb + (long)t * p.q.st + (long)(s.h * G + rr - t * G) * p.q.sh) * ES + ch * 16 : p.q.p;
      cp_async16(qraw + row * S::QROW + ch * 16, src, in);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };

  // ---- the warp's fetch side: its tiles of all segments of the round, STAGES ahead; the pages of its next 32 tiles (one a lane) are
  // looked up one batch ahead
  const int tpp = c.page / TILE;                      // tiles a page
  int nseg = 0;
  int fleft = 0, fnext = 0, fstage = 0, mytile = -1;               // batch in use: tiles left, next one's lane
  int nxseg = 0, nxtile = 0, nxpage = -1;                          // batch ahead: segment, first tile, the lane's page
  uint32_t bad = 0;                                   // stages whose page was bad (their tile is masked)
  bool dead = false;
  uint32_t phase = 0;                                 // parity per stage
  int issued = 0, used = 0;
  auto look_ahead = [&](int k, int t) {               // the batch at or after tile t of segment k
    while (k < nseg && t >= segs[k].end) {
      if (++k < nseg) t = segs[k].tile + w;
    }
    nxseg = k;
    nxtile = t;
    if (k < nseg) {
      const int mine = t + NW * lane, col = mine / tpp, b = segs[k].b;
      nxpage = mine < segs[k].end && mine * TILE < seq[b].tokens ? c.table[(long)b * c.table_cols + col] : -2;   // -2: no tokens
    }
  };
  auto fetch = [&]() {
    if (dead) return;
    if (fleft == 0) {
      if (nxseg >= nseg) return;
      const int fseg = nxseg, ftile = nxtile, t = ftile + NW * lane;
      fnext = 0;
      fleft = min(32, (segs[fseg].end - ftile + NW - 1) / NW);
      const bool ok = nxpage >= 0 && nxpage < c.n_pages;
      if (!ok && nxpage != -2) atomicOr(c.status, PACE_KV_BAD_PAGE);
      mytile = ok ? (nxpage * c.Hkv + segs[fseg].h) * tpp + t % tpp : -1;
      look_ahead(fseg, ftile + 32 * NW);
    }
    const int at = __shfl_sync(0xffffffffu, mytile, fnext);
    bad = at < 0 ? bad | (1u << fstage) : bad & ~(1u << fstage);
    if (lane == 0) {
      if (at < 0) {
        umma::mbar_arrive(&bars[fstage]);
      } else {
        umma::mbar_arrive_expect_tx(&bars[fstage], L::BYTES);
        umma::bulk_g2s(ring + fstage * L::BYTES, c.pool + (long)at * L::BYTES, L::BYTES, &bars[fstage]);
      }
    }
    ++issued;
    ++fnext;
    --fleft;
    fstage = fstage + 1 == STAGES ? 0 : fstage + 1;
  };
  const uint32_t magic = opaque(0x64006400u);
  int stage = 0;
  int pseg = 0;                                       // items shared with other blocks: 1 the one it began with, 2 the one it ends with
#pragma unroll 1
  for (unsigned round = lo; round < hi;) {            // SEGS segments a round
   if (w == 0) {
     const int n = list_segments<TILE>(seq, cum, p, round, hi, segs);
     if (lane == 0) segs[SEGS].end = n;
   }
   __syncthreads();
   nseg = segs[SEGS].end;
   round = (unsigned)segs[SEGS].tile;
   look_ahead(0, segs[0].tile + w);
   copy_queries(segs[0]);
#pragma unroll 1
   for (int i = 0; i < STAGES - 1; ++i) fetch();
#pragma unroll 1
   for (int k = 0; k < nseg; ++k) {
    const Segment sg = segs[k];
    const Seq sq = seq[sg.b];
    const int len = sq.len, nn = sq.fresh, tokens = sq.tokens;
    const int row0 = sg.rb * ROWS;
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();                                  // this segment's queries are here; the last one's areas are free
    // ---- queries as B fragments: lane (j, cc) takes dims 64g + 16cc .. + 15 of row j of each block of eight. bf16: as fp16 over a
    // power of two that puts the row's largest element in [1, 2), exact but below 2^-14 of it. fp32: as three bf16 parts.
    {
      constexpr int TPR = S::THREADS / ROWS < 32 ? S::THREADS / ROWS : 32, PAIRS = D / TPR / 2;      // threads a row
      const int row = tid / TPR, e0 = (tid % TPR) * 2 * PAIRS;
      const char *src = qraw + row * S::QROW + e0 * ES;
      const bool neg = p.scale_log2 < 0.0f;
      float mul = fabsf(p.scale_log2);
      auto put = [&](int i, int part, uint32_t v) {
        const int e = e0 + 2 * i, g = e >> 6, k = (e & 15) >> 1, ln = (row & 7) * 4 + ((e & 63) >> 4);
        qf[((((row >> 3) * NG + g) * PARTS + part) * 2 + (k >> 2)) * 128 + ln * 4 + (k & 3)] = v;
      };
      if (row >= ROWS) {
      } else if (!F32) {
        uint32_t x[PAIRS], top = 0;
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) {
          x[i] = reinterpret_cast<const uint32_t *>(src)[i];
          top = max(top, max((x[i] << 16) & 0x7FFF0000u, x[i] & 0x7FFF0000u));
        }
#pragma unroll
        for (int o = 1; o < TPR; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
        const int e = max(min((int)(top >> 23) - 127, 126), -126);
        const float down = neg ? -exp2i(-e) : exp2i(-e);
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) put(i, 0, h2pack(__uint_as_float(x[i] << 16) * down, __uint_as_float(x[i] & 0xFFFF0000u) * down));
        mul *= exp2i(e);
      } else {
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) {
          const float2 x = reinterpret_cast<const float2 *>(src)[i];
          uint32_t a[PARTS];
          split_pair<PARTS>(neg ? -x.x : x.x, neg ? -x.y : x.y, a);
#pragma unroll
          for (int e = 0; e < PARTS; ++e) put(i, e, a[e]);
        }
      }
      if (tid % TPR == 0 && row < ROWS) rowmul[row] = fmaxf(mul, FLT_MIN);          // (not 0: a masked score is -inf)
    }
    __syncthreads();
    if (k + 1 < nseg) copy_queries(segs[k + 1]);
    float crow[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) crow[n][0] = rowmul[8 * n + 2 * cc], crow[n][1] = rowmul[8 * n + 2 * cc + 1];

    float acc[NG][4][NT][4];
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[g][i][n][e] = 0.0f;
    float m[NT][2], l[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) m[n][0] = m[n][1] = -INFINITY, l[n][0] = l[n][1] = 0.0f;

#pragma unroll 1
    for (int tile = sg.tile + w; tile < sg.end; tile += NW) {
      fetch();
      if (!dead && !bar_wait(&bars[stage], (phase >> stage) & 1u)) {
        dead = true;
        if (lane == 0) atomicOr(c.status, PACE_KV_TIMEOUT);
      }
      dead = __any_sync(0xffffffffu, dead);
      if (!dead) phase ^= 1u << stage, ++used;
      const char *st = ring + stage * L::BYTES;
      const bool lost = dead || ((bad >> stage) & 1u);

      // ---- scores, without the rows' factors
      constexpr int GP = BITS == 4 && D > 64 ? 2 : 1;   // groups whose words share a chunk
      constexpr int KW = BITS == 4 ? 2 : 4;             // words of a token's 16 dims
      float s[2][NT][4];
#pragma unroll
      for (int g0 = 0; g0 < NG; g0 += GP) {
        uint32_t kw[2][2][GP * KW];
#pragma unroll
        for (int blk = 0; blk < 2; ++blk)
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const char *at = st + L::kchunk(16 * blk + 8 * half + tau(j), (g0 / GP) * 4 + cc);
            if (GP * KW == 2) {
              const uint2 x = *reinterpret_cast<const uint2 *>(at);
              kw[blk][half][0] = x.x, kw[blk][half][1] = x.y;
            } else {
              const uint4 x = *reinterpret_cast<const uint4 *>(at);
              kw[blk][half][0] = x.x, kw[blk][half][1] = x.y, kw[blk][half][2 % (GP * KW)] = x.z, kw[blk][half][3 % (GP * KW)] = x.w;
            }
          }
#pragma unroll
        for (int gi = 0; gi < GP; ++gi) {
          const int g = g0 + gi;
          uint32_t q[NT][PARTS][8];
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < PARTS; ++e) {
              const uint4 *src = reinterpret_cast<const uint4 *>(qf + ((n * NG + g) * PARTS + e) * 256) + lane;
              const uint4 x = src[0], y = src[32];
              q[n][e][0] = x.x, q[n][e][1] = x.y, q[n][e][2] = x.z, q[n][e][3] = x.w;
              q[n][e][4] = y.x, q[n][e][5] = y.y, q[n][e][6] = y.z, q[n][e][7] = y.w;
            }
          const uint2 ksw = *reinterpret_cast<const uint2 *>(st + L::KS + g * 64 + j * 8);
          uint32_t kz = 0;
          if (BITS == 4) kz = *reinterpret_cast<const uint32_t *>(st + L::KZ + g * 32 + j * 4);
#pragma unroll
          for (int blk = 0; blk < 2; ++blk) {
            uint32_t fr[2][8];                           // the group's pairs of the two tokens
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              const uint32_t *x = kw[blk][half] + gi * KW;
              uint32_t z = 0;                            // the pair 1024 + z or 128 + z
              if (BITS == 4) z = __byte_perm(kz, F32 ? 0x43434343u : 0x64646464u, 0x4040 | (2 * blk + half) * 0x0101);
              if (!F32) {
                if (BITS == 4) {
                  const uint32_t z64 = h2add(z, 0xE380E380u /* -960 */);
                  uint32_t r[4];
#pragma unroll
                  for (int h = 0; h < KW; ++h) {
                    codes4(x[h], z, z64, magic, r);
                    fr[half][4 * (h % 2)] = r[0], fr[half][4 * (h % 2) + 1] = r[1], fr[half][4 * (h % 2) + 2] = r[2], fr[half][4 * (h % 2) + 3] = r[3];
                  }
                } else {
#pragma unroll
                  for (int h = 0; h < KW; ++h) codes8(x[h], fr[half][2 * h], fr[half][2 * h + 1]);
                }
              } else {
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                  if (BITS == 4) fr[half][k] = sub_bf16x2(pair4(x[(k >> 2) % KW], k & 3), z);
                  else fr[half][k] = pair8((k & 1) ? x[(k >> 1) % KW] >> 8 : x[(k >> 1) % KW]);
                }
              }
            }
            // (fp32: the tensor cores cut off where they add, so that the small parts have a sum of their own)
            float d[NT][4], small[NT][4];
            if (F32) {
#pragma unroll
              for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) d[n][e] = small[n][e] = 0.0f;
            }
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
              for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < PARTS; ++e) {
                  if (!F32 && k == 0) mma_f16_first(d[n], fr[0][0], fr[1][0], fr[0][1], fr[1][1], q[n][e][0], q[n][e][1]);
                  else if (!F32) mma_f16(d[n], fr[0][2 * k], fr[1][2 * k], fr[0][2 * k + 1], fr[1][2 * k + 1], q[n][e][2 * k], q[n][e][2 * k + 1]);
                  else mma_bf16(e ? small[n] : d[n], fr[0][2 * k], fr[1][2 * k], fr[0][2 * k + 1], fr[1][2 * k + 1], q[n][e][2 * k], q[n][e][2 * k + 1]);
                }
            if (F32) {
#pragma unroll
              for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) d[n][e] += small[n][e];
            }
            const uint32_t sw = blk ? ksw.y : ksw.x;
            const float s0 = __uint_as_float(sw << 16), s1 = __uint_as_float(sw & 0xFFFF0000u);
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float sk = e < 2 ? s0 : s1;
                s[blk][n][e] = g == 0 ? sk * d[n][e] : fmaf(sk, d[n][e], s[blk][n][e]);
              }
          }
        }
      }
      // ---- masks: only tiles that reach past the context (or were lost)
      const int tok0 = tile * TILE;
      const bool edge = tok0 + TILE > len || lost;
      if (edge) {
#pragma unroll
        for (int blk = 0; blk < 2; ++blk)
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const int tk = tok0 + 16 * blk + 8 * half + tau(j), jd = tk - len;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int r = 0; r < 2; ++r) {
                bool see = jd < 0;
                if (!see && jd < nn && tk < tokens) {
                  const int t = (row0 + 8 * n + 2 * cc + r) / G;
                  if (t < T) see = p.mask ? (p.mask[((long)sg.b * T + t) * words + (jd >> 5)] >> (jd & 31)) & 1u : jd <= t;
                }
                if (!see || lost) s[blk][n][2 * half + r] = -INFINITY;
              }
          }
      }
      // ---- weights. bf16 I/O: the scale of a value group enters the exponent, w = 2^(s + log2 s_v - m + 6) with m the running
      // maximum of s + log2 s_v, so that fp16 weights keep 11 bits down to 2^-20 of a row's largest; the sum takes 2^(s - m + 6). fp32 I/O: the
      // scale multiplies the weight, and m is raised to 64 above the scores of tokens whose scale reaches 2^65, so that no sum of weighted
      // values leaves fp32 (held values reach 2^120). m is raised only when a score passes it by 2^8 (fp16 weights up to 2^14, sums in fp32).
      constexpr uint32_t BIG = 0x60000000u;              // 2^65
      uint32_t top = 0;
      float lv[NG][2][2], lm[2][2];                      // log2 of the value scales of the lane's tokens, their largest
#pragma unroll
      for (int blk = 0; blk < 2; ++blk)
#pragma unroll
        for (int half = 0; half < 2; ++half) lm[blk][half] = !F32 ? -60.0f : 0.0f;
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        const uint2 vsw = *reinterpret_cast<const uint2 *>(st + L::VS + g * 64 + j * 8);
#pragma unroll
        for (int blk = 0; blk < 2; ++blk) {
          const uint32_t sw = blk ? vsw.y : vsw.x;
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            float x = __uint_as_float(half ? sw & 0xFFFF0000u : sw << 16);
            if (edge && (tok0 + 16 * blk + 8 * half + tau(j) >= tokens || lost)) x = 0.0f;   // never written: may hold anything
            lv[g][blk][half] = !F32 ? log2_approx(x) : x;
            if (!F32) lm[blk][half] = fmaxf(lm[blk][half], lv[g][blk][half]);
            else top = max(top, __float_as_uint(x));     // (scales are not negative: their bits order as integers)
          }
        }
      }
      float mx[NT][2];
      bool grow = F32 && top >= BIG;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          mx[n][r] = fmaxf(fmaxf(fmaf(s[0][n][r], crow[n][r], lm[0][0]), fmaf(s[0][n][2 + r], crow[n][r], lm[0][1])),
                           fmaxf(fmaf(s[1][n][r], crow[n][r], lm[1][0]), fmaf(s[1][n][2 + r], crow[n][r], lm[1][1])));
          grow |= mx[n][r] > m[n][r] + 8.0f;
        }
      if (__any_sync(0xffffffffu, grow)) {
        if (F32 && top >= BIG) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float most = 0.0f;
#pragma unroll
            for (int g = 0; g < NG; ++g) most = fmaxf(most, lv[g][i >> 1][i & 1]);
            if (most >= __uint_as_float(BIG)) {
#pragma unroll
              for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int r = 0; r < 2; ++r) mx[n][r] = fmaxf(mx[n][r], fmaf(s[i >> 1][n][2 * (i & 1) + r], crow[n][r], 64.0f));
            }
          }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            float x = mx[n][r];
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
            const float mn = fmaxf(m[n][r], x);
            const float al = m[n][r] == -INFINITY ? 0.0f : exp2_approx(m[n][r] - mn);
            m[n][r] = mn;
            l[n][r] *= al;
#pragma unroll
            for (int g = 0; g < NG; ++g)
#pragma unroll
              for (int i = 0; i < 4; ++i) acc[g][i][n][r] *= al, acc[g][i][n][2 + r] *= al;
          }
      }
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float add = m[n][r] == -INFINITY ? 0.0f : 6.0f - m[n][r];
#pragma unroll
          for (int blk = 0; blk < 2; ++blk)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              float &x = s[blk][n][2 * half + r];
              x = fmaf(x, crow[n][r], add);
              const float pr = exp2_approx(x);
              l[n][r] += pr;
              if (F32) x = pr;
            }
        }
      // ---- output
#pragma unroll
      for (int g0 = 0; g0 < NG; g0 += GP) {
#pragma unroll
        for (int blk = 0; blk < 2; ++blk) {
          // value words of the lane's tokens: rows 2cc, 2cc+1 of each half
          const int t0 = 16 * blk + cc, t1 = 16 * blk + 4 + (cc ^ 3);
          uint2 v0, v1, v2, v3;
          if (BITS == 4 && D == 64) {
            v0 = make_uint2(*reinterpret_cast<const uint32_t *>(st + L::vunit(t0, j)), 0);
            v1 = make_uint2(*reinterpret_cast<const uint32_t *>(st + L::vunit(t1, j)), 0);
            v2 = make_uint2(*reinterpret_cast<const uint32_t *>(st + L::vunit(t0 + 8, j)), 0);
            v3 = make_uint2(*reinterpret_cast<const uint32_t *>(st + L::vunit(t1 + 8, j)), 0);
          } else {
            const int u = (g0 / GP) * 8 + j;
            v0 = *reinterpret_cast<const uint2 *>(st + L::vunit(t0, u));
            v1 = *reinterpret_cast<const uint2 *>(st + L::vunit(t1, u));
            v2 = *reinterpret_cast<const uint2 *>(st + L::vunit(t0 + 8, u));
            v3 = *reinterpret_cast<const uint2 *>(st + L::vunit(t1 + 8, u));
          }
#pragma unroll
          for (int gi = 0; gi < GP; ++gi) {
            const int g = g0 + gi;
            uint32_t bf[NT][PARTS][2];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              uint32_t x[PARTS], y[PARTS];
              const float v0s = lv[g][blk][0], v1s = lv[g][blk][1];
              if (!F32) {
                x[0] = h2pack(exp2_approx(s[blk][n][0] + v0s), exp2_approx(s[blk][n][1] + v0s));
                y[0] = h2pack(exp2_approx(s[blk][n][2] + v1s), exp2_approx(s[blk][n][3] + v1s));
              } else {
                split_pair<PARTS>(s[blk][n][0] * v0s, s[blk][n][1] * v0s, x);
                split_pair<PARTS>(s[blk][n][2] * v1s, s[blk][n][3] * v1s, y);
              }
#pragma unroll
              for (int e = 0; e < PARTS; ++e) bf[n][e][0] = movmatrix(x[e]), bf[n][e][1] = movmatrix(y[e]);
            }
            uint32_t a01[8], a23[8];                     // dims 8j + 0..7 (even: A row j, odd: row j + 8) of the two token pairs
            if (BITS == 4) {
              const uint32_t x0 = gi ? v0.y : v0.x, x1 = gi ? v1.y : v1.x, x2 = gi ? v2.y : v2.x, x3 = gi ? v3.y : v3.x;
              const uint32_t w[4] = {__byte_perm(x0, x1, 0x5410), __byte_perm(x0, x1, 0x7632), __byte_perm(x2, x3, 0x5410),
                                     __byte_perm(x2, x3, 0x7632)};
              const uint32_t vz = *reinterpret_cast<const uint32_t *>(st + L::VZ + g * 32 + cc * 8 + blk * 4);
              const uint32_t hi = F32 ? 0x43434343u : 0x64646464u;                              // 1024 + z or 128 + z
              const uint32_t z01 = __byte_perm(vz, hi, 0x4140), z23 = __byte_perm(vz, hi, 0x4342);
              if (!F32) {
                const uint32_t y01 = h2add(z01, 0xE380E380u), y23 = h2add(z23, 0xE380E380u);    // 64 + z
                uint32_t r[4];
#pragma unroll
                for (int o = 0; o < 2; ++o) {
                  codes4(w[o], z01, y01, magic, r);
                  a01[o] = r[0], a01[2 + o] = r[1], a01[4 + o] = r[2], a01[6 + o] = r[3];
                  codes4(w[2 + o], z23, y23, magic, r);
                  a23[o] = r[0], a23[2 + o] = r[1], a23[4 + o] = r[2], a23[6 + o] = r[3];
                }
              } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                  for (int o = 0; o < 2; ++o) a01[2 * i + o] = sub_bf16x2(pair4(w[o], i), z01), a23[2 * i + o] = sub_bf16x2(pair4(w[2 + o], i), z23);
              }
            } else {
#pragma unroll
              for (int h2 = 0; h2 < 2; ++h2) {
                const uint32_t x0 = h2 ? v0.y : v0.x, x1 = h2 ? v1.y : v1.x, x2 = h2 ? v2.y : v2.x, x3 = h2 ? v3.y : v3.x;
                const uint32_t w[4] = {__byte_perm(x0, x1, 0x5410), __byte_perm(x0, x1, 0x7632), __byte_perm(x2, x3, 0x5410),
                                       __byte_perm(x2, x3, 0x7632)};
#pragma unroll
                for (int o = 0; o < 2; ++o) {
                  if (!F32) {
                    codes8(w[o], a01[4 * h2 + o], a01[4 * h2 + 2 + o]);
                    codes8(w[2 + o], a23[4 * h2 + o], a23[4 * h2 + 2 + o]);
                  } else {
                    a01[4 * h2 + o] = pair8(w[o]), a01[4 * h2 + 2 + o] = pair8(w[o] >> 8);
                    a23[4 * h2 + o] = pair8(w[2 + o]), a23[4 * h2 + 2 + o] = pair8(w[2 + o] >> 8);
                  }
                }
              }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
              for (int n = 0; n < NT; ++n)
              {
                if (!F32) {
                  mma_f16(acc[g][i][n], a01[2 * i], a01[2 * i + 1], a23[2 * i], a23[2 * i + 1], bf[n][0][0], bf[n][0][1]);
                  continue;
                }
                // the smallest parts first, and added to the output outside the tensor cores: over thousands of tiles what they cut off
                // would always lean the same way
                float y[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int e = PARTS; e-- > 0;) mma_bf16(y, a01[2 * i], a01[2 * i + 1], a23[2 * i], a23[2 * i + 1], bf[n][e][0], bf[n][e][1]);
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[g][i][n][e] += y[e];
              }
          }
        }
      }
      if (!dead) stage = stage + 1 == STAGES ? 0 : stage + 1;
      __syncwarp();                                   // every lane is done with the stage before it is filled again
    }

    // ---- join the warps: the others leave their accumulators, as they lie in the fragments, for the first one
    const bool whole = sg.tile == 0 && sg.end == sg.tiles;
    constexpr int FR = NG * 4 * NT * 32;               // float4s a warp
    float4 *left = reinterpret_cast<float4 *>(scratch);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) l[n][r] += __shfl_xor_sync(0xffffffffu, l[n][r], o);
        if (w > 0 && j == 0) *reinterpret_cast<float2 *>(ml + (w * ROWS + 8 * n + 2 * cc + r) * 2) = make_float2(m[n][r], l[n][r]);
      }
    if (w > 0) {
#pragma unroll
      for (int g = 0; g < NG; ++g)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int n = 0; n < NT; ++n)
            left[(w - 1) * FR + ((g * 4 + i) * NT + n) * 32 + lane] = make_float4(acc[g][i][n][0], acc[g][i][n][1], acc[g][i][n][2], acc[g][i][n][3]);
    }
    __syncthreads();
    if (w == 0) {
      float M[NT][2], f0[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          M[n][r] = m[n][r];
          for (int i = 1; i < NW; ++i) M[n][r] = fmaxf(M[n][r], ml[(i * ROWS + 8 * n + 2 * cc + r) * 2]);
          f0[n][r] = m[n][r] == -INFINITY ? 0.0f : exp2_approx(m[n][r] - M[n][r]);
          l[n][r] *= f0[n][r];
        }
#pragma unroll
      for (int g = 0; g < NG; ++g)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[g][i][n][e] *= f0[n][e & 1];
#pragma unroll 2
      for (int i = 1; i < NW; ++i) {
        float f[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float2 e = *reinterpret_cast<const float2 *>(ml + (i * ROWS + 8 * n + 2 * cc + r) * 2);
            f[n][r] = e.x == -INFINITY ? 0.0f : exp2_approx(e.x - M[n][r]);
            l[n][r] = fmaf(f[n][r], e.y, l[n][r]);
          }
#pragma unroll
        for (int g = 0; g < NG; ++g)
#pragma unroll
          for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              const float4 x = left[(i - 1) * FR + ((g * 4 + t) * NT + n) * 32 + lane];
              acc[g][t][n][0] = fmaf(f[n][0], x.x, acc[g][t][n][0]), acc[g][t][n][1] = fmaf(f[n][1], x.y, acc[g][t][n][1]);
              acc[g][t][n][2] = fmaf(f[n][0], x.z, acc[g][t][n][2]), acc[g][t][n][3] = fmaf(f[n][1], x.w, acc[g][t][n][3]);
            }
      }
      // (an item that is shared and starts in this block is the block's last)
      float *mine = c.part + (long)(2 * blockIdx.x + (sg.tile == 0 ? 1 : 0)) * part_floats(D, NT);
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int row = 8 * n + 2 * cc + r, rr = row0 + row, t = rr / G;
          if (rr >= T * G) continue;
          const float inv = !whole ? 1.0f : t < nn && l[n][r] > 0.0f ? 1.0f / l[n][r] : 0.0f;
#pragma unroll
          for (int g = 0; g < NG; ++g) {
            const float y[8] = {acc[g][0][n][r], acc[g][0][n][2 + r], acc[g][1][n][r], acc[g][1][n][2 + r],
                                acc[g][2][n][r], acc[g][2][n][2 + r], acc[g][3][n][r], acc[g][3][n][2 + r]};
            const int e8 = 64 * g + 8 * j;
            if (whole) store_out<F32>(p.o.p + (sg.b * p.o.sb + (long)t * p.o.st + (long)(sg.h * G + rr - t * G) * p.o.sh + e8) * ES, y, inv);
            else store_out<true>(reinterpret_cast<char *>(mine + row * D + e8), y, 1.0f);
          }
          if (!whole && j == 0) *reinterpret_cast<float2 *>(mine + ROWS * D + 2 * row) = make_float2(M[n][r], l[n][r]);
        }
    }
    if (!whole) pseg |= sg.tile ? 1 : 2;
   }
   __syncthreads();                                   // the list of segments and the areas are free
  }
  // ---- items that several blocks share: the last to arrive joins the parts in block order
  if (pseg) {
    // (the first holds the block's first tile, the second its last)
    auto shared = [&](int k, Segment &it, int &first, int &last) {
      const unsigned at = k ? hi - 1 : lo;
      it = segment(at);
      first = (int)((at - it.tile) / cuts.share);
      last = (int)((at - it.tile + it.tiles - 1) / cuts.share);
    };
    if (tid < 2) {
      bool joins = false;
      if ((pseg >> tid) & 1) {
        Segment it;
        int first, last;
        shared(tid, it, first, last);
        joins = last_part(&c.count[first], last - first + 1);
      }
      flag[tid] = joins;
    }
    __syncthreads();
#pragma unroll 1
    for (int k = 0; k < 2; ++k)
      if (flag[k]) {
        Segment it;
        int first, last;
        shared(k, it, first, last);
        join_parts<D, ROWS, S::THREADS, F32>(p, c.part, part_floats(D, NT), first, last, it.b, it.h, it.rb * ROWS, seq[it.b].fresh, scratch);
      }
  }
  if (dead) {                                         // a wait gave up: let the copies in flight land (bounded) before leaving
    for (; used < issued; ++used) {
      bar_wait(&bars[stage], (phase >> stage) & 1u);
      phase ^= 1u << stage;
      stage = stage + 1 == STAGES ? 0 : stage + 1;
    }
  }
}

// Calls launch(args, tiles) for as many sequences at a time as keep the line of tiles of `tok` tokens, which is counted in 32 bits,
// below 2^31 whatever their lengths (all of them, but for the largest products of batch, heads, new tokens and table); where one sequence
// passes that, for ranges of its items (a table holds 2^25 tiles at most).
template <typename F>
cudaError_t by_batches(const AttendArgs &a, int tok, F launch) {
  const long tiles = ((long)a.c.table_cols * a.c.page + tok - 1) / tok, all = (long)a.c.Hkv * a.row_blocks;
  const long most = ((1L << 31) - 1) / tiles, step = std::min(all, most), seqs = std::max(1L, most / all);
  const int words = (a.c.n_tokens + 31) / 32, es = a.c.io == PACE_IO_F32 ? 4 : 2;
  for (long b = 0; b < a.c.batch; b += seqs)
    for (long item = 0; item < all; item += step) {
      AttendArgs part = a;
      part.item0 = (unsigned)item;
      part.items = (unsigned)std::min(step, all - item);
      part.c.batch = (int)std::min(seqs, a.c.batch - b);
      part.c.lens += b;
      if (part.c.n_new) part.c.n_new += b;
      part.c.table += b * a.c.table_cols;
      if (part.mask) part.mask += b * a.c.n_tokens * words;
      part.q.p += b * a.q.sb * es;
      part.o.p += b * a.o.sb * es;
      const cudaError_t e = launch(part, tiles * part.items * part.c.batch);
      if (e != cudaSuccess) return e;
    }
  return cudaSuccess;
}

// resident_blocks with a cache entry for each capacity: their shared memory differs, and the grid, and with it the cuts of the line and the
// bits of the results, must not depend on which batch was called first.
template <auto K, int CAPACITY>
int resident_blocks_of(int threads, size_t smem) {
  static std::atomic<int> cache[PACE_MAX_DEVICES];
  const int dev = current_device();
  int v = cache[dev].load(std::memory_order_relaxed);
  if (v <= 0) {
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&v, K, threads, smem) != cudaSuccess || v <= 0) v = 1;
    cache[dev].store(v, std::memory_order_relaxed);
  }
  return v;
}

template <int D, int BITS, int NT, int PARTS, int NW, int STAGES, int MINB>
cudaError_t launch_attend(AttendArgs a, cudaStream_t s) {
  using S = AttendShape<D, BITS, NT, PARTS, NW, STAGES>;
  constexpr auto K = attend_kernel<D, BITS, NT, PARTS, NW, STAGES, MINB>;
  static_assert(part_floats(D, NT) <= MAX_ROWS_FLOATS + 64, "the work area holds every shape's partial results");
  const size_t smem = S::smem(a.c.batch);
  cudaError_t e = smem_opt_in<K>(227 * 1024);
  if (e != cudaSuccess) return e;
  a.row_blocks = (a.c.n_tokens * a.c.group + S::ROWS - 1) / S::ROWS;
  const int capacity = S::capacity(a.c.batch);
  const int per_sm = capacity == 64    ? resident_blocks_of<K, 64>(S::THREADS, smem)
                     : capacity == 256 ? resident_blocks_of<K, 256>(S::THREADS, smem)
                                       : resident_blocks_of<K, PACE_KV_MAX_BATCH>(S::THREADS, smem);
  return by_batches(a, TILE, [&](const AttendArgs &part, long line) {
    // no more blocks than the longest possible line of tiles
    long grid = (long)per_sm * device_sm_count();
    if (grid > MAX_BLOCKS) grid = MAX_BLOCKS;
    if (grid > line) grid = line;
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg = pdl_config(dim3((unsigned)grid), dim3(S::THREADS), smem, s, attr);
    return cudaLaunchKernelEx(&cfg, K, part);
  });
}

}  // namespace kv
}  // namespace pace
