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
// exponent of 1024 by one bit operation a pair and one exact subtraction on the other pipe, and enter the products as integers.
// The scales of a key group multiply the fp32 accumulators, those of a value group enter the exponent of the weights. Queries and
// weights are fp16 relative to a power of two (11 bits); with fp32 I/O both are three bf16 parts, so nothing is rounded below 2^-24.
//
// Work: the tiles of all (sequence, KV head, row block) items form one line, cut into equal shares, one a block; a block's warps
// take its tiles in turn, each through its own ring of tiles filled by bulk copies (one copy a tile). Items cut by a share
// boundary leave partial results; the last block to finish an item joins them, in block order, so results do not depend on timing.
#pragma once

#include <cuda_fp16.h>

#include "kv_common.cuh"
#include "umma.cuh"

namespace pace {
namespace kv {

constexpr uint64_t WAIT_LIMIT_NS = 1000000000ull;
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
__device__ __forceinline__ uint32_t h2pack(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&v);
}
// The four pairs of a word of 4-bit codes as fp16 u - z, exactly: the nibble at bit 0 of a half under the exponent of 1024 reads
// 1024 + u, the one at bit 4 reads 1024 + 16 u = 16 (64 + u). z1024 and z64 are the pairs 1024 + z and 64 + z.
__device__ __forceinline__ void codes4(uint32_t w, uint32_t z1024, uint32_t z64, uint32_t (&r)[4]) {
  constexpr uint32_t SIXTEENTH = 0x2C002C00u;
  const uint32_t x = w >> 8, nz = z64 ^ 0x80008000u;
  r[0] = h2sub((w & 0x000F000Fu) | 0x64006400u, z1024);
  r[1] = h2fma((w & 0x00F000F0u) | 0x64006400u, SIXTEENTH, nz);
  r[2] = h2sub((x & 0x000F000Fu) | 0x64006400u, z1024);
  r[3] = h2fma((x & 0x00F000F0u) | 0x64006400u, SIXTEENTH, nz);
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
  int min_share;        // fewest tiles a block takes
};

// One position on the line of tiles.
struct Segment {
  int b, h, rb;         // item
  int tile, end;        // tiles [tile, end) of it
  int tiles;            // of the whole item
};

// Exclusive prefix sums over the sequences of their items' tiles, in shared memory: cum[0..batch].
__device__ __forceinline__ int seq_tokens(const KvDev &c, int b, bool &over) {
  const long cap = (long)c.table_cols * c.page;
  const long n = (long)max(c.lens[b], 0) + new_tokens(c, b);
  over = n > cap || c.lens[b] < 0;
  return (int)(n < cap ? n : cap);
}
__device__ __forceinline__ int seq_tiles(int tokens) { return max((tokens + TILE - 1) / TILE, 1); }

__device__ __forceinline__ void tile_line(const KvDev &c, long per_seq, long *cum, long *warp_sums) {
  const int n = c.batch, nt = blockDim.x, per = (n + nt - 1) / nt, b0 = threadIdx.x * per;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, nw = nt >> 5;
  long s = 0;
  for (int i = 0; i < per; ++i) {
    if (b0 + i >= n) break;
    bool over;
    const int tok = seq_tokens(c, b0 + i, over);
    if (over) atomicOr(c.status, PACE_KV_BAD_PAGE);
    s += seq_tiles(tok) * per_seq;
    cum[b0 + i + 1] = s;
  }
  long x = s;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_sums[w] = x;
  __syncthreads();
  long base = x - s;
  for (int i = 0; i < w && i < nw; ++i) base += warp_sums[i];
  for (int i = 0; i < per; ++i)
    if (b0 + i < n) cum[b0 + i + 1] += base;
  if (threadIdx.x == 0) cum[0] = 0;
  __syncthreads();
}

__device__ __forceinline__ Segment segment_at(const long *cum, int batch, int row_blocks, int kv_heads, long p, long hi) {
  int lo = 0, up = batch;                  // last b with cum[b] <= p
  while (up - lo > 1) {
    const int mid = (lo + up) >> 1;
    if (cum[mid] <= p) lo = mid;
    else up = mid;
  }
  Segment s;
  s.b = lo;
  s.tiles = (int)((cum[lo + 1] - cum[lo]) / ((long)row_blocks * kv_heads));
  const long r = p - cum[lo];
  const int item = (int)(r / s.tiles);
  s.tile = (int)(r - (long)item * s.tiles);
  s.h = item / row_blocks;
  s.rb = item - s.h * row_blocks;
  s.end = (int)min((long)s.tiles, s.tile + (hi - p));
  return s;
}

template <int D, int BITS, int NT, int PARTS, int NW, int STAGES>
struct AttendShape {
  using L = Tile<D, BITS>;
  static constexpr int ROWS = 8 * NT, THREADS = NW * 32;
  static constexpr int OROW = D + 4;                                    // padded scratch row
  static constexpr size_t RING = (size_t)NW * STAGES * L::BYTES;
  static constexpr size_t BARS = NW * STAGES * 8;
  static constexpr size_t SCRATCH = (size_t)NW * ROWS * OROW * 4;
  static constexpr size_t ML = (size_t)NW * ROWS * 2 * 4;
  static constexpr size_t FIXED = RING + BARS + SCRATCH + ML + 64 * 8 + 16;
  // prefix sums of up to this many sequences: few capacities, so that the occupancy of each is asked for once
  static constexpr int capacity(int batch) { return batch <= 128 ? 128 : PACE_KV_MAX_BATCH; }
  static constexpr size_t smem(int batch) { return FIXED + (size_t)(capacity(batch) + 1) * 8; }
};

template <int D, int BITS, int NT, int PARTS, int NW, int STAGES, int MINB>
__global__ void __launch_bounds__(NW * 32, MINB) attend_kernel(AttendArgs p) {
  using S = AttendShape<D, BITS, NT, PARTS, NW, STAGES>;
  using L = Tile<D, BITS>;
  constexpr int NG = L::NG, ROWS = S::ROWS;
  extern __shared__ __align__(128) char smem[];
  char *ring_all = smem;
  uint64_t *bars_all = reinterpret_cast<uint64_t *>(smem + S::RING);
  float *scratch = reinterpret_cast<float *>(smem + S::RING + S::BARS);
  float *ml = scratch + S::SCRATCH / 4;
  long *wsum = reinterpret_cast<long *>(reinterpret_cast<char *>(ml) + S::ML);
  long *cum = wsum + 64;
  int *flag = reinterpret_cast<int *>(cum + p.c.batch + 1);

  const KvDev &c = p.c;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, j = lane >> 2, cc = lane & 3;
  const int G = c.group, T = c.n_tokens, words = (T + 31) >> 5;
  char *ring = ring_all + (size_t)w * STAGES * L::BYTES;
  uint64_t *bars = bars_all + w * STAGES;
  if (lane < STAGES) umma::mbar_init(&bars[lane], 1);
  umma::mbar_fence_init();
  pdl_enter();
  tile_line(c, (long)p.row_blocks * c.Hkv, cum, wsum);

  const long total = cum[c.batch];
  const long even = (total + gridDim.x - 1) / gridDim.x;
  const long share = even > p.min_share ? even : p.min_share;
  const long lo = (long)blockIdx.x * share, hi = min(total, lo + share);
  if (lo >= total) return;

  // ---- the warp's fetch side: its tiles of all segments of the block, STAGES ahead
  long fpos = lo;                                     // line position of the fetch segment's end
  Segment f{0, 0, 0, 0, 0, 0};
  const int tpp = c.page / TILE;                      // tiles a page
  int ftile = 0, fbatch = 0, fstage = 0, mytile = -1;
  uint32_t bad = 0;                                   // stages whose page was bad (their tile is masked)
  bool dead = false;
  uint32_t phase = 0;                                 // parity per stage
  bool fdone = false;
  auto fetch = [&]() {
    while (!fdone && ftile >= f.end) {
      if (fpos >= hi) {
        fdone = true;
        break;
      }
      f = segment_at(cum, c.batch, p.row_blocks, c.Hkv, fpos, hi);
      fpos += f.end - f.tile;
      ftile = f.tile + w;
      fbatch = 32;
    }
    if (fdone || dead) return;
    if (fbatch == 32) {                               // the warp's next 32 tiles of this segment, one a lane
      const int t = ftile + NW * lane;
      mytile = t < f.end ? tile_index(c, f.b, f.h, t, tpp) : 0;
      if (mytile < 0) atomicOr(c.status, PACE_KV_BAD_PAGE);
      fbatch = 0;
    }
    const int at = __shfl_sync(0xffffffffu, mytile, fbatch);
    if (at < 0) {
      bad |= 1u << fstage;
      if (lane == 0) umma::mbar_arrive(&bars[fstage]);
    } else {
      bad &= ~(1u << fstage);
      if (lane == 0) {
        umma::mbar_arrive_expect_tx(&bars[fstage], L::BYTES);
        umma::bulk_g2s(ring + fstage * L::BYTES, c.pool + (long)at * L::BYTES, L::BYTES, &bars[fstage]);
      }
    }
    ftile += NW;
    ++fbatch;
    fstage = fstage + 1 == STAGES ? 0 : fstage + 1;
  };
  int issued = 0, used = 0;
  auto fetch_one = [&]() {
    fetch();
    if (!fdone && !dead) ++issued;
  };
  __syncwarp();
#pragma unroll 1
  for (int i = 0; i < STAGES - 1; ++i) fetch_one();

  int stage = 0;
#pragma unroll 1
  for (long pos = lo; pos < hi;) {
    const Segment sg = segment_at(cum, c.batch, p.row_blocks, c.Hkv, pos, hi);
    pos += sg.end - sg.tile;
    const int len = max(c.lens[sg.b], 0), nn = new_tokens(c, sg.b);
    bool over_;
    const int tokens = seq_tokens(c, sg.b, over_);
    const int row0 = sg.rb * ROWS;

    // ---- queries as B fragments: lane (j, cc) holds dims 64g + 16cc .. + 15 of row j of each block of eight
    uint32_t qf[NT][NG][PARTS][8];
    float crow[NT][2];                                // what a score of rows 2cc, 2cc+1 is multiplied by
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int row = row0 + 8 * n + j, t = row / G, hh = sg.h * G + row - t * G;
      const bool in = row < T * G;
      const long at = sg.b * p.q.sb + (long)t * p.q.st + (long)hh * p.q.sh + 16 * cc;
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        if (PARTS == 1) {
          uint4 x = make_uint4(0, 0, 0, 0), y = x;
          if (in) {
            const uint4 *src = reinterpret_cast<const uint4 *>(p.q.p + (at + 64 * g) * 2);
            x = src[0];
            y = src[1];
          }
          const uint32_t v[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
          for (int i = 0; i < 8; ++i) qf[n][g][0][i] = v[i];
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float4 x = make_float4(0, 0, 0, 0);
            if (in) x = reinterpret_cast<const float4 *>(p.q.p + (at + 64 * g) * 4)[i];
            uint32_t a[PARTS], b[PARTS];
            split_pair<PARTS>(x.x, x.y, a);
            split_pair<PARTS>(x.z, x.w, b);
#pragma unroll
            for (int e = 0; e < PARTS; ++e) qf[n][g][e][2 * i] = a[e], qf[n][g][e][2 * i + 1] = b[e];
          }
        }
      }
      crow[n][0] = crow[n][1] = p.scale_log2;
      if (PARTS == 1) {
        // bf16 -> fp16 over a power of two that puts the row's largest element in [1, 2): exact but below 2^-14 of it
        uint32_t top = 0;
#pragma unroll
        for (int g = 0; g < NG; ++g)
#pragma unroll
          for (int i = 0; i < 8; ++i) top = max(top, max((qf[n][g][0][i] << 16) & 0x7FFF0000u, qf[n][g][0][i] & 0x7FFF0000u));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int e = max(min((int)(top >> 23) - 127, 126), -126);
        const float down = exp2i(-e);
#pragma unroll
        for (int g = 0; g < NG; ++g)
#pragma unroll
          for (int i = 0; i < 8; ++i)
            qf[n][g][0][i] = h2pack(__uint_as_float(qf[n][g][0][i] << 16) * down, __uint_as_float(qf[n][g][0][i] & 0xFFFF0000u) * down);
        crow[n][0] = p.scale_log2 * exp2i(__shfl_sync(0xffffffffu, e, 8 * cc));
        crow[n][1] = p.scale_log2 * exp2i(__shfl_sync(0xffffffffu, e, 8 * cc + 4));
      }
    }

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
      fetch_one();
      if (!dead && !umma::mbar_wait(&bars[stage], (phase >> stage) & 1u, WAIT_LIMIT_NS)) {
        dead = true;
        if (lane == 0) atomicOr(c.status, PACE_KV_TIMEOUT);
      }
      dead = __any_sync(0xffffffffu, dead);
      if (!dead) phase ^= 1u << stage, ++used;
      const char *st = ring + stage * L::BYTES;
      const bool lost = dead || ((bad >> stage) & 1u);

      // ---- scores
      float s[2][NT][4];
      {
        uint2 ksw[NG];
        uint32_t kzw[NG];
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          ksw[g] = *reinterpret_cast<const uint2 *>(st + L::KS + g * 64 + j * 8);
          if (BITS == 4) kzw[g] = *reinterpret_cast<const uint32_t *>(st + L::KZ + g * 32 + j * 4);
        }
#pragma unroll
        for (int blk = 0; blk < 2; ++blk) {
          const int ta = 16 * blk + tau(j), tb = ta + 8;
          uint32_t wa[NG][BITS == 4 ? 2 : 4], wb[NG][BITS == 4 ? 2 : 4];
          if (BITS == 8) {
#pragma unroll
            for (int g = 0; g < NG; ++g) {
              const uint4 x = *reinterpret_cast<const uint4 *>(st + L::kchunk(ta, g * 4 + cc));
              const uint4 y = *reinterpret_cast<const uint4 *>(st + L::kchunk(tb, g * 4 + cc));
              wa[g][0] = x.x, wa[g][1] = x.y, wa[g][2 % (BITS == 4 ? 2 : 4)] = x.z, wa[g][3 % (BITS == 4 ? 2 : 4)] = x.w;
              wb[g][0] = y.x, wb[g][1] = y.y, wb[g][2 % (BITS == 4 ? 2 : 4)] = y.z, wb[g][3 % (BITS == 4 ? 2 : 4)] = y.w;
            }
          } else if (D == 64) {
            const uint2 x = *reinterpret_cast<const uint2 *>(st + L::kchunk(ta, cc));
            const uint2 y = *reinterpret_cast<const uint2 *>(st + L::kchunk(tb, cc));
            wa[0][0] = x.x, wa[0][1] = x.y, wb[0][0] = y.x, wb[0][1] = y.y;
          } else {
#pragma unroll
            for (int g = 0; g < NG; g += 2) {
              const uint4 x = *reinterpret_cast<const uint4 *>(st + L::kchunk(ta, (g >> 1) * 4 + cc));
              const uint4 y = *reinterpret_cast<const uint4 *>(st + L::kchunk(tb, (g >> 1) * 4 + cc));
              constexpr int g1 = NG > 1 ? 1 : 0;
              wa[g][0] = x.x, wa[g][1] = x.y, wa[g + g1][0] = x.z, wa[g + g1][1] = x.w;
              wb[g][0] = y.x, wb[g][1] = y.y, wb[g + g1][0] = y.z, wb[g + g1][1] = y.w;
            }
          }
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[blk][n][e] = 0.0f;
#pragma unroll
          for (int g = 0; g < NG; ++g) {
            float d[NT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int e = 0; e < 4; ++e) d[n][e] = 0.0f;
            uint32_t zka = 0, zkb = 0, z64a = 0, z64b = 0;
            if (BITS == 4) {
              const uint32_t hi = PARTS == 1 ? 0x64646464u : 0x43434343u;                     // 1024 + z or 128 + z
              zka = __byte_perm(kzw[g], hi, 0x4040 | (2 * blk) | ((2 * blk) << 8));
              zkb = __byte_perm(kzw[g], hi, 0x4040 | (2 * blk + 1) | ((2 * blk + 1) << 8));
              if (PARTS == 1) z64a = h2add(zka, 0xE380E380u /* -960 */), z64b = h2add(zkb, 0xE380E380u);
            }
            uint32_t fa[8], fb[8];                      // the group's pairs of the two tokens
            if (PARTS == 1) {
              if (BITS == 4) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  uint32_t r[4];
                  codes4(wa[g][h], zka, z64a, r);
                  fa[4 * h] = r[0], fa[4 * h + 1] = r[1], fa[4 * h + 2] = r[2], fa[4 * h + 3] = r[3];
                  codes4(wb[g][h], zkb, z64b, r);
                  fb[4 * h] = r[0], fb[4 * h + 1] = r[1], fb[4 * h + 2] = r[2], fb[4 * h + 3] = r[3];
                }
              } else {
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                  codes8(wa[g][h % (BITS == 4 ? 2 : 4)], fa[2 * h], fa[2 * h + 1]);
                  codes8(wb[g][h % (BITS == 4 ? 2 : 4)], fb[2 * h], fb[2 * h + 1]);
                }
              }
            } else {
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                if (BITS == 4) {
                  const uint32_t x = wa[g][k >> 1], y = wb[g][k >> 1];
                  fa[2 * k] = sub_bf16x2(pair4(x, 2 * (k & 1)), zka), fb[2 * k] = sub_bf16x2(pair4(y, 2 * (k & 1)), zkb);
                  fa[2 * k + 1] = sub_bf16x2(pair4(x, 2 * (k & 1) + 1), zka), fb[2 * k + 1] = sub_bf16x2(pair4(y, 2 * (k & 1) + 1), zkb);
                } else {
                  const uint32_t x = wa[g][k % (BITS == 4 ? 2 : 4)], y = wb[g][k % (BITS == 4 ? 2 : 4)];
                  fa[2 * k] = pair8(x), fb[2 * k] = pair8(y), fa[2 * k + 1] = pair8(x >> 8), fb[2 * k + 1] = pair8(y >> 8);
                }
              }
            }
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
              for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < PARTS; ++e) {
                  if (PARTS == 1) mma_f16(d[n], fa[2 * k], fb[2 * k], fa[2 * k + 1], fb[2 * k + 1], qf[n][g][e][2 * k], qf[n][g][e][2 * k + 1]);
                  else mma_bf16(d[n], fa[2 * k], fb[2 * k], fa[2 * k + 1], fb[2 * k + 1], qf[n][g][e][2 * k], qf[n][g][e][2 * k + 1]);
                }
            const uint32_t sw = blk ? ksw[g].y : ksw[g].x;
            const float s0 = __uint_as_float(sw << 16), s1 = __uint_as_float(sw & 0xFFFF0000u);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              s[blk][n][0] = fmaf(s0, d[n][0], s[blk][n][0]);
              s[blk][n][1] = fmaf(s0, d[n][1], s[blk][n][1]);
              s[blk][n][2] = fmaf(s1, d[n][2], s[blk][n][2]);
              s[blk][n][3] = fmaf(s1, d[n][3], s[blk][n][3]);
            }
          }
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[blk][n][e] *= crow[n][e & 1];
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
      // maximum of s + log2 s_v, so that fp16 weights keep 11 bits whatever the scales; the sum takes 2^(s - m). fp32 I/O: the
      // scale multiplies the weight. m is raised only when a score passes it by 2^8 (fp16 weights up to 2^14, sums in fp32).
      float lv[NG][2][2], lm[2][2];                      // log2 of the value scales of the lane's tokens, their largest
#pragma unroll
      for (int blk = 0; blk < 2; ++blk)
#pragma unroll
        for (int half = 0; half < 2; ++half) lm[blk][half] = PARTS == 1 ? -60.0f : 0.0f;
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
            lv[g][blk][half] = PARTS == 1 ? log2_approx(x) : x;
            if (PARTS == 1) lm[blk][half] = fmaxf(lm[blk][half], lv[g][blk][half]);
          }
        }
      }
      float mx[NT][2];
      bool grow = false;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          mx[n][r] = fmaxf(fmaxf(s[0][n][r] + lm[0][0], s[0][n][2 + r] + lm[0][1]), fmaxf(s[1][n][r] + lm[1][0], s[1][n][2 + r] + lm[1][1]));
          grow |= mx[n][r] > m[n][r] + 8.0f;
        }
      if (__any_sync(0xffffffffu, grow)) {
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
          const float mu = m[n][r] == -INFINITY ? 0.0f : m[n][r];
#pragma unroll
          for (int blk = 0; blk < 2; ++blk)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              float &x = s[blk][n][2 * half + r];
              x -= mu;
              const float pr = exp2_approx(x);
              l[n][r] += pr;
              x = PARTS == 1 ? x + 6.0f : pr;
            }
        }
      // ---- output
      constexpr int GP = BITS == 4 && D > 64 ? 2 : 1;   // groups whose words share a unit
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
              if (PARTS == 1) {
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
              const uint2 vzw = *reinterpret_cast<const uint2 *>(st + L::VZ + g * 32 + cc * 8);
              const int q0 = 2 * blk, q1 = 2 * blk + 1;
              const uint32_t hi = PARTS == 1 ? 0x64006400u : 0x43004300u;                       // 1024 + z or 128 + z
              const uint32_t z01 = (__byte_perm(vzw.x, vzw.y, q0 * 0x0011 + (4 + q0) * 0x1100) & 0x00FF00FFu) | hi;
              const uint32_t z23 = (__byte_perm(vzw.x, vzw.y, q1 * 0x0011 + (4 + q1) * 0x1100) & 0x00FF00FFu) | hi;
              if (PARTS == 1) {
                const uint32_t y01 = h2add(z01, 0xE380E380u), y23 = h2add(z23, 0xE380E380u);    // 64 + z
                uint32_t r[4];
#pragma unroll
                for (int o = 0; o < 2; ++o) {
                  codes4(w[o], z01, y01, r);
                  a01[o] = r[0], a01[2 + o] = r[1], a01[4 + o] = r[2], a01[6 + o] = r[3];
                  codes4(w[2 + o], z23, y23, r);
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
                  if (PARTS == 1) {
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
#pragma unroll
                for (int e = 0; e < PARTS; ++e) {
                  if (PARTS == 1) mma_f16(acc[g][i][n], a01[2 * i], a01[2 * i + 1], a23[2 * i], a23[2 * i + 1], bf[n][e][0], bf[n][e][1]);
                  else mma_bf16(acc[g][i][n], a01[2 * i], a01[2 * i + 1], a23[2 * i], a23[2 * i + 1], bf[n][e][0], bf[n][e][1]);
                }
          }
        }
      }
      if (!dead) stage = stage + 1 == STAGES ? 0 : stage + 1;
      __syncwarp();                                   // every lane is done with the stage before it is filled again
    }

    // ---- join the warps
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) l[n][r] += __shfl_xor_sync(0xffffffffu, l[n][r], o);
        const int row = 8 * n + 2 * cc + r;
        if (j == 0) {
          ml[(w * ROWS + row) * 2] = m[n][r];
          ml[(w * ROWS + row) * 2 + 1] = l[n][r];
        }
        float *dst = scratch + (w * ROWS + row) * S::OROW + 8 * j;
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          *reinterpret_cast<float4 *>(dst + 64 * g) = make_float4(acc[g][0][n][r], acc[g][0][n][2 + r], acc[g][1][n][r], acc[g][1][n][2 + r]);
          *reinterpret_cast<float4 *>(dst + 64 * g + 4) = make_float4(acc[g][2][n][r], acc[g][2][n][2 + r], acc[g][3][n][r], acc[g][3][n][2 + r]);
        }
      }
    __syncthreads();
    const bool whole = sg.tile == 0 && sg.end == sg.tiles;
    const long item_lo = pos - (sg.end - sg.tile) - sg.tile;          // line position of the item's first tile
    const int first = (int)(item_lo / share), last = (int)((item_lo + sg.tiles - 1) / share);
    const int PF = part_floats(D, NT);
    float *mine = c.part + (long)(2 * blockIdx.x + (blockIdx.x == first ? 1 : 0)) * PF;
    constexpr int CH = D / 8;                                          // 8-element pieces of a row
    for (int x = threadIdx.x; x < ROWS * CH; x += S::THREADS) {
      const int row = x / CH, e8 = (x % CH) * 8;
      const int rr = row0 + row, t = rr / G;
      float M = -INFINITY;
#pragma unroll
      for (int i = 0; i < NW; ++i) M = fmaxf(M, ml[(i * ROWS + row) * 2]);
      float y[8] = {0, 0, 0, 0, 0, 0, 0, 0}, Ls = 0.0f;
#pragma unroll
      for (int i = 0; i < NW; ++i) {
        const float mi = ml[(i * ROWS + row) * 2];
        float f2 = mi == -INFINITY ? 0.0f : exp2_approx(mi - M);
        Ls += f2 * ml[(i * ROWS + row) * 2 + 1];
        if (PARTS == 1) f2 *= 0x1p-6f;
        const float4 u = *reinterpret_cast<const float4 *>(scratch + (i * ROWS + row) * S::OROW + e8);
        const float4 v = *reinterpret_cast<const float4 *>(scratch + (i * ROWS + row) * S::OROW + e8 + 4);
        y[0] += f2 * u.x, y[1] += f2 * u.y, y[2] += f2 * u.z, y[3] += f2 * u.w;
        y[4] += f2 * v.x, y[5] += f2 * v.y, y[6] += f2 * v.z, y[7] += f2 * v.w;
      }
      if (whole) {
        if (rr >= T * G) continue;
        const float inv = t < nn && Ls > 0.0f ? 1.0f / Ls : 0.0f;
        char *dst = p.o.p + (sg.b * p.o.sb + (long)t * p.o.st + (long)(sg.h * G + rr - t * G) * p.o.sh + e8) * (PARTS > 1 ? 4 : 2);
        if (PARTS > 1) {
          reinterpret_cast<float4 *>(dst)[0] = make_float4(y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv);
          reinterpret_cast<float4 *>(dst)[1] = make_float4(y[4] * inv, y[5] * inv, y[6] * inv, y[7] * inv);
        } else {
          *reinterpret_cast<uint4 *>(dst) = make_uint4(pack_bf16x2(y[0] * inv, y[1] * inv), pack_bf16x2(y[2] * inv, y[3] * inv),
                                                       pack_bf16x2(y[4] * inv, y[5] * inv), pack_bf16x2(y[6] * inv, y[7] * inv));
        }
      } else {
        float *dst = mine + row * D + e8;
        *reinterpret_cast<float4 *>(dst) = make_float4(y[0], y[1], y[2], y[3]);
        *reinterpret_cast<float4 *>(dst + 4) = make_float4(y[4], y[5], y[6], y[7]);
        if (e8 == 0) {
          mine[ROWS * D + 2 * row] = M;
          mine[ROWS * D + 2 * row + 1] = Ls;
        }
      }
    }
    // ---- an item that several blocks share: the last to arrive joins the parts in block order
    if (!whole) {
      __threadfence();
      __syncthreads();
      if (threadIdx.x == 0) {
        const int before = atomicAdd(&c.count[first], 1);
        *flag = before == last - first;
        if (*flag) c.count[first] = 0;
      }
      __syncthreads();
      if (*flag) {
        __threadfence();
        for (int x = threadIdx.x; x < ROWS * CH; x += S::THREADS) {
          const int row = x / CH, e8 = (x % CH) * 8;
          const int rr = row0 + row, t = rr / G;
          if (rr >= T * G) continue;
          float M = -INFINITY;
          for (int i = first; i <= last; ++i) {
            const float *src = c.part + (long)(2 * i + (i == first ? 1 : 0)) * PF;
            M = fmaxf(M, __ldcg(src + ROWS * D + 2 * row));
          }
          float y[8] = {0, 0, 0, 0, 0, 0, 0, 0}, Ls = 0.0f;
#pragma unroll 4
          for (int i = first; i <= last; ++i) {
            const float *src = c.part + (long)(2 * i + (i == first ? 1 : 0)) * PF;
            const float2 e = __ldcg(reinterpret_cast<const float2 *>(src + ROWS * D + 2 * row));
            const float f2 = e.x == -INFINITY ? 0.0f : exp2_approx(e.x - M);
            Ls += f2 * e.y;
            const float4 u = __ldcg(reinterpret_cast<const float4 *>(src + row * D + e8));
            const float4 v = __ldcg(reinterpret_cast<const float4 *>(src + row * D + e8 + 4));
            y[0] += f2 * u.x, y[1] += f2 * u.y, y[2] += f2 * u.z, y[3] += f2 * u.w;
            y[4] += f2 * v.x, y[5] += f2 * v.y, y[6] += f2 * v.z, y[7] += f2 * v.w;
          }
          const float inv = t < nn && Ls > 0.0f ? 1.0f / Ls : 0.0f;
          char *dst = p.o.p + (sg.b * p.o.sb + (long)t * p.o.st + (long)(sg.h * G + rr - t * G) * p.o.sh + e8) * (PARTS > 1 ? 4 : 2);
          if (PARTS > 1) {
            reinterpret_cast<float4 *>(dst)[0] = make_float4(y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv);
            reinterpret_cast<float4 *>(dst)[1] = make_float4(y[4] * inv, y[5] * inv, y[6] * inv, y[7] * inv);
          } else {
            *reinterpret_cast<uint4 *>(dst) = make_uint4(pack_bf16x2(y[0] * inv, y[1] * inv), pack_bf16x2(y[2] * inv, y[3] * inv),
                                                         pack_bf16x2(y[4] * inv, y[5] * inv), pack_bf16x2(y[6] * inv, y[7] * inv));
          }
        }
      }
    }
    __syncthreads();                                  // scratch is free for the next segment
  }
  if (dead) {                                         // a wait gave up: let the copies in flight land (bounded) before leaving
    for (; used < issued; ++used) {
      umma::mbar_wait(&bars[stage], (phase >> stage) & 1u, WAIT_LIMIT_NS);
      phase ^= 1u << stage;
      stage = stage + 1 == STAGES ? 0 : stage + 1;
    }
  }
}

// resident_blocks of the capacity for large batches (its own cache entry)
template <auto K>
int resident_blocks_large(int threads, size_t smem) {
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
  a.min_share = NW;
  static int (*const resident[2])(int, size_t) = {resident_blocks<K>, resident_blocks_large<K>};
  const int per_sm = resident[S::capacity(a.c.batch) > 128](S::THREADS, smem);
  // no more blocks than the longest possible line of tiles has shares
  const long line = (long)a.c.batch * a.c.Hkv * a.row_blocks * (((long)a.c.table_cols * a.c.page + TILE - 1) / TILE);
  long grid = (long)per_sm * device_sm_count();
  if (grid > MAX_BLOCKS) grid = MAX_BLOCKS;
  const long shares = (line + a.min_share - 1) / a.min_share;
  if (grid > shares) grid = shares;
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg = pdl_config(dim3((unsigned)grid), dim3(S::THREADS), smem, s, attr);
  return cudaLaunchKernelEx(&cfg, K, a);
}

}  // namespace kv
}  // namespace pace
