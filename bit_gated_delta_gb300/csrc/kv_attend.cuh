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
// clock and SM at the measured 6.8 TB/s against 128 lanes), so codes become bf16 by bit operations and enter the products as
// exact integers: 4 bits: (w & 0x000F000F) | 0x43004300 is the pair 128 + u; values subtract 128 + z exactly, keys leave it to
// the scores (acc - (128 + z) * sum(q), per group). 8 bits: 128 + (u & 127) minus 128 or 256 by the top bit. The scales of
// a key group multiply the fp32 accumulators, those of a value group the weights before they are rounded to bf16 (fp32 I/O: three
// bf16 parts of queries and weights, and keys subtracted too, so nothing is rounded below 2^-24).
//
// Work: the tiles of all (sequence, KV head, row block) items form one line, cut into equal shares, one a block; a block's warps
// take its tiles in turn, each through its own ring of tiles filled by bulk copies (one copy a tile). Items cut by a share
// boundary leave partial results; the last block to finish an item joins them, in block order, so results do not depend on timing.
#pragma once

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
  constexpr bool SUBK = BITS == 4 && PARTS > 1;       // keys subtracted exactly; else the scores take it
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
  int ftile = 0, fbatch = 0, fstage = 0, mypage = -1;
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
    if (fbatch == 32) {                               // pages of the warp's next 32 tiles of this segment, one a lane
      const int t = ftile + NW * lane;
      mypage = t < f.end ? page_of(c, f.b, (long)t * TILE) : 0;
      if (mypage < 0) atomicOr(c.status, PACE_KV_BAD_PAGE);
      fbatch = 0;
    }
    const int page = __shfl_sync(0xffffffffu, mypage, fbatch);
    if (page < 0) {
      bad |= 1u << fstage;
      if (lane == 0) umma::mbar_arrive(&bars[fstage]);
    } else {
      bad &= ~(1u << fstage);
      if (lane == 0) {
        umma::mbar_arrive_expect_tx(&bars[fstage], L::BYTES);
        umma::bulk_g2s(ring + fstage * L::BYTES, tile_at<L::BYTES>(c, page, f.h, (long)ftile * TILE), L::BYTES, &bars[fstage]);
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
    float qs[NT][NG][2];                              // sum of the group's queries of rows 2cc, 2cc+1 (4-bit keys)
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
        if (BITS == 4 && !SUBK) {
          float s = 0.0f;
#pragma unroll
          for (int i = 0; i < 8; ++i) s += __uint_as_float(qf[n][g][0][i] << 16) + __uint_as_float(qf[n][g][0][i] & 0xFFFF0000u);
          s += __shfl_xor_sync(0xffffffffu, s, 1);
          s += __shfl_xor_sync(0xffffffffu, s, 2);
          qs[n][g][0] = __shfl_sync(0xffffffffu, s, 8 * cc);
          qs[n][g][1] = __shfl_sync(0xffffffffu, s, 8 * cc + 4);
        }
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
            uint32_t zka = 0, zkb = 0;
            if (SUBK) {
              zka = __byte_perm(kzw[g], 0, 0x4040 | (2 * blk) | ((2 * blk) << 8)) | 0x43004300u;
              zkb = __byte_perm(kzw[g], 0, 0x4040 | (2 * blk + 1) | ((2 * blk + 1) << 8)) | 0x43004300u;
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint32_t a0, a1, a2, a3;
              if (BITS == 4) {
                const uint32_t x = wa[g][k >> 1], y = wb[g][k >> 1];
                a0 = pair4(x, 2 * (k & 1)), a1 = pair4(y, 2 * (k & 1));
                a2 = pair4(x, 2 * (k & 1) + 1), a3 = pair4(y, 2 * (k & 1) + 1);
                if (SUBK) a0 = sub_bf16x2(a0, zka), a1 = sub_bf16x2(a1, zkb), a2 = sub_bf16x2(a2, zka), a3 = sub_bf16x2(a3, zkb);
              } else {
                const uint32_t x = wa[g][k % (BITS == 4 ? 2 : 4)], y = wb[g][k % (BITS == 4 ? 2 : 4)];
                a0 = pair8(x), a1 = pair8(y), a2 = pair8(x >> 8), a3 = pair8(y >> 8);
              }
#pragma unroll
              for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < PARTS; ++e)
                  mma_bf16(d[n], a0, a1, a2, a3, qf[n][g][e][2 * k], qf[n][g][e][2 * k + 1]);
            }
            const uint32_t sw = blk ? ksw[g].y : ksw[g].x;
            const float s0 = __uint_as_float(sw << 16) * p.scale_log2, s1 = __uint_as_float(sw & 0xFFFF0000u) * p.scale_log2;
            if (BITS == 4 && !SUBK) {
              // 2^23 + z from the byte, then 128 + z
              const float z0 = __uint_as_float(__byte_perm(kzw[g], 0x4B000000u, 0x7440 | (2 * blk))) - (8388608.0f - 128.0f);
              const float z1 = __uint_as_float(__byte_perm(kzw[g], 0x4B000000u, 0x7440 | (2 * blk + 1))) - (8388608.0f - 128.0f);
#pragma unroll
              for (int n = 0; n < NT; ++n) {
                d[n][0] = fmaf(-z0, qs[n][g][0], d[n][0]);
                d[n][1] = fmaf(-z0, qs[n][g][1], d[n][1]);
                d[n][2] = fmaf(-z1, qs[n][g][0], d[n][2]);
                d[n][3] = fmaf(-z1, qs[n][g][1], d[n][3]);
              }
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              s[blk][n][0] = fmaf(s0, d[n][0], s[blk][n][0]);
              s[blk][n][1] = fmaf(s0, d[n][1], s[blk][n][1]);
              s[blk][n][2] = fmaf(s1, d[n][2], s[blk][n][2]);
              s[blk][n][3] = fmaf(s1, d[n][3], s[blk][n][3]);
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
      // ---- running maximum: raised only when a score passes it by 2^8 (weights up to 256, the sum is fp32)
      float mx[NT][2];
      bool grow = false;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          mx[n][r] = fmaxf(fmaxf(s[0][n][r], s[0][n][2 + r]), fmaxf(s[1][n][r], s[1][n][2 + r]));
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
              const float pr = exp2_approx(s[blk][n][2 * half + r] - mu);
              s[blk][n][2 * half + r] = pr;
              l[n][r] += pr;
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
            const uint32_t sw = *reinterpret_cast<const uint32_t *>(st + L::VS + g * 64 + j * 8 + blk * 4);
            float s0 = __uint_as_float(sw << 16), s1 = __uint_as_float(sw & 0xFFFF0000u);
            if (edge) {                                 // slots never written may hold anything
              const int tk = tok0 + 16 * blk + tau(j);
              if (tk >= tokens || lost) s0 = 0.0f;
              if (tk + 8 >= tokens || lost) s1 = 0.0f;
            }
            uint32_t bf[NT][PARTS][2];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              uint32_t x[PARTS], y[PARTS];
              split_pair<PARTS>(s[blk][n][0] * s0, s[blk][n][1] * s0, x);
              split_pair<PARTS>(s[blk][n][2] * s1, s[blk][n][3] * s1, y);
#pragma unroll
              for (int e = 0; e < PARTS; ++e) bf[n][e][0] = movmatrix(x[e]), bf[n][e][1] = movmatrix(y[e]);
            }
            if (BITS == 4) {
              const uint32_t x0 = gi ? v0.y : v0.x, x1 = gi ? v1.y : v1.x, x2 = gi ? v2.y : v2.x, x3 = gi ? v3.y : v3.x;
              const uint32_t lo01 = __byte_perm(x0, x1, 0x5410), hi01 = __byte_perm(x0, x1, 0x7632);
              const uint32_t lo23 = __byte_perm(x2, x3, 0x5410), hi23 = __byte_perm(x2, x3, 0x7632);
              const uint2 vzw = *reinterpret_cast<const uint2 *>(st + L::VZ + g * 32 + cc * 8);
              const int q0 = 2 * blk, q1 = 2 * blk + 1;
              const uint32_t z01 = (__byte_perm(vzw.x, vzw.y, q0 * 0x0011 + (4 + q0) * 0x1100) & 0x00FF00FFu) | 0x43004300u;
              const uint32_t z23 = (__byte_perm(vzw.x, vzw.y, q1 * 0x0011 + (4 + q1) * 0x1100) & 0x00FF00FFu) | 0x43004300u;
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const uint32_t a0 = sub_bf16x2(pair4(lo01, i), z01), a1 = sub_bf16x2(pair4(hi01, i), z01);
                const uint32_t a2 = sub_bf16x2(pair4(lo23, i), z23), a3 = sub_bf16x2(pair4(hi23, i), z23);
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                  for (int e = 0; e < PARTS; ++e) mma_bf16(acc[g][i][n], a0, a1, a2, a3, bf[n][e][0], bf[n][e][1]);
              }
            } else {
#pragma unroll
              for (int h2 = 0; h2 < 2; ++h2) {
                const uint32_t x0 = h2 ? v0.y : v0.x, x1 = h2 ? v1.y : v1.x, x2 = h2 ? v2.y : v2.x, x3 = h2 ? v3.y : v3.x;
                const uint32_t lo01 = __byte_perm(x0, x1, 0x5410), hi01 = __byte_perm(x0, x1, 0x7632);
                const uint32_t lo23 = __byte_perm(x2, x3, 0x5410), hi23 = __byte_perm(x2, x3, 0x7632);
#pragma unroll
                for (int ii = 0; ii < 2; ++ii) {
                  const uint32_t a0 = pair8(lo01 >> (8 * ii)), a1 = pair8(hi01 >> (8 * ii));
                  const uint32_t a2 = pair8(lo23 >> (8 * ii)), a3 = pair8(hi23 >> (8 * ii));
#pragma unroll
                  for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < PARTS; ++e) mma_bf16(acc[g][2 * h2 + ii][n], a0, a1, a2, a3, bf[n][e][0], bf[n][e][1]);
                }
              }
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
        const float f2 = mi == -INFINITY ? 0.0f : exp2_approx(mi - M);
        Ls += f2 * ml[(i * ROWS + row) * 2 + 1];
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
