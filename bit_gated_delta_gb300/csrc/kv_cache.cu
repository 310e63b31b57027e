// Rotary positions and the quantized KV cache outside attention: the cos/sin table, rotation, append (rotation and
// quantization fused), read-back and the move of an accepted path.
//
// All of these move bytes: a lane owns eight consecutive elements (one 16-byte bf16 vector, two fp32 ones), D/8 lanes a head
// vector, 256/D vectors a warp; the floor of every call is its bytes at the copy bandwidth (6.8 TB/s; what only writes, 4.0).
// Measured, with cold caches:
//   rotation of 16,384 tokens, 32 heads of 128, bf16 (268 MB)                   40 us, 6.7 TB/s
//   append of 16 x 256 tokens, 48 and 8 heads of 128, 8 bits, 32 of 128 rotated  30 us (126 MB: 19 us); 20.0 M warp instructions would
//                                                                               issue in 16 us (slots 63% busy, DRAM 35%): the longest
//                                                                               stall is on the loads that each warp begins with
//   read-back of 4 x 20,000 to 32,768 tokens, 8 heads of 128, 4 bits            113 us; writing as many zeros takes 108
//   append of 64 single tokens 4 us, keep of 8 paths 4 us: a chain of three dependent loads
#include "kv_common.cuh"

namespace pace {
namespace kv {

constexpr int THREADS = 128;

template <int IO32>
__device__ __forceinline__ void load8(const char *p, float (&x)[8]) {
  if (IO32) {
    const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  } else {
    const uint4 a = *reinterpret_cast<const uint4 *>(p);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
}
template <int IO32>
__device__ __forceinline__ void store8(char *p, const float (&x)[8]) {
  if (IO32) {
    reinterpret_cast<float4 *>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t *>(&v);
    }
    *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// A rotated vector is cut into rot/8 pieces of four pairs and (d - rot)/8 pieces of eight elements that pass through, one a lane,
// so that no lane needs another's elements and each angle is read once: the two 4-element parts of piece a start at `lo` and `hi`.
struct Piece {
  int lo, hi;
  bool turn;
};
__device__ __forceinline__ Piece piece_of(const KvRope &r, int a) {
  const bool turn = 8 * a < r.rot, split = turn && !r.interleaved;
  return Piece{split ? 4 * a : 8 * a, split ? (r.rot >> 1) + 4 * a : 8 * a + 4, turn};
}
template <int IO32>
struct Four {
  using type = uint2;
};
template <>
struct Four<1> {
  using type = float4;
};
__device__ __forceinline__ float4 widen(const uint2 &w) {
  return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u), __uint_as_float(w.y << 16),
                     __uint_as_float(w.y & 0xFFFF0000u));
}
__device__ __forceinline__ float4 widen(const float4 &w) { return w; }
__device__ __forceinline__ void narrow(const float4 &x, uint2 &w) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(x.x, x.y), b = __floats2bfloat162_rn(x.z, x.w);
  w = make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
}
__device__ __forceinline__ void narrow(const float4 &x, float4 &w) { w = x; }

// (a, b) -> (a c - b s, b c + a s). Products and sums are rounded apart (no contraction), so that a rotated value is the same
// wherever it is formed.
__device__ __forceinline__ void turn(float &a, float &b, float c, float s) {
  const float u = a, v = b;
  a = __fsub_rn(__fmul_rn(u, c), __fmul_rn(v, s));
  b = __fadd_rn(__fmul_rn(v, c), __fmul_rn(u, s));
}

// HC heads of one token, from head h0: the angles of the lane's four pairs are read once for all of them.
template <int IO32, int HC>
__device__ __forceinline__ void rotate_heads(const KvRope &r, const char *src, int64_t src_h, char *dst, int64_t dst_h, int n, int a,
                                             int pos, float sign) {
  using V = typename Four<IO32>::type;
  constexpr int ES = IO32 ? 4 : 2;
  const Piece pc = piece_of(r, a);
  V lo[HC], hi[HC];
#pragma unroll
  for (int i = 0; i < HC; ++i)
    if (i < n) {
      lo[i] = *reinterpret_cast<const V *>(src + (i * src_h + pc.lo) * ES);
      hi[i] = *reinterpret_cast<const V *>(src + (i * src_h + pc.hi) * ES);
    }
  float4 t0 = make_float4(1, 0, 1, 0), t1 = t0;
  if (pc.turn) {
    const float4 *row = reinterpret_cast<const float4 *>(r.table + (long)pos * (r.rot >> 1) + 4 * a);
    t0 = row[0];
    t1 = row[1];
  }
#pragma unroll
  for (int i = 0; i < HC; ++i)
    if (i < n) {
      if (pc.turn) {
        float4 x = widen(lo[i]), y = widen(hi[i]);
        if (r.interleaved) {
          turn(x.x, x.y, t0.x, sign * t0.y);
          turn(x.z, x.w, t0.z, sign * t0.w);
          turn(y.x, y.y, t1.x, sign * t1.y);
          turn(y.z, y.w, t1.z, sign * t1.w);
        } else {
          turn(x.x, y.x, t0.x, sign * t0.y);
          turn(x.y, y.y, t0.z, sign * t0.w);
          turn(x.z, y.z, t1.x, sign * t1.y);
          turn(x.w, y.w, t1.z, sign * t1.w);
        }
        narrow(x, lo[i]);
        narrow(y, hi[i]);
      }
      *reinterpret_cast<V *>(dst + (i * dst_h + pc.lo) * ES) = lo[i];
      *reinterpret_cast<V *>(dst + (i * dst_h + pc.hi) * ES) = hi[i];
    }
}

// The same for eight consecutive elements a lane, as the quantizer holds them: the partner half comes by shuffle, and every lane of
// the warp takes part.
struct Angles {
  float2 cs[8];
};
__device__ __forceinline__ void load_angles(const KvRope &r, int pos, int a, Angles &g) {
  const int half = r.rot >> 1, e0 = 8 * a;
  const float2 *row = r.table + (long)pos * half;
  if (e0 >= r.rot) return;
  const float4 *q = reinterpret_cast<const float4 *>(row + (r.interleaved ? e0 >> 1 : (e0 < half ? e0 : e0 - half)));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (r.interleaved && i >= 2) break;
    const float4 t = q[i];
    g.cs[2 * i] = make_float2(t.x, t.y);
    g.cs[2 * i + 1] = make_float2(t.z, t.w);
  }
}
__device__ __forceinline__ void rotate8(const KvRope &r, const Angles &g, int a, bool on, float (&x)[8]) {
  const int half = r.rot >> 1, e0 = 8 * a, lane = threadIdx.x & 31;
  const bool in = on && e0 < r.rot;
  if (r.interleaved) {
    if (!in) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) turn(x[2 * i], x[2 * i + 1], g.cs[i].x, g.cs[i].y);
    return;
  }
  const bool lo = e0 < half;
  const int src = e0 < r.rot ? (lo ? lane + (half >> 3) : lane - (half >> 3)) : lane;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float p = __shfl_sync(0xffffffffu, x[i], src & 31), y = x[i];
    if (in) {
      if (lo) turn(y, p, g.cs[i].x, g.cs[i].y);
      else turn(p, y, g.cs[i].x, g.cs[i].y);
      x[i] = y;
    }
  }
}

// cos and sin in 64 bits, once per table: theta is exact to fp64, the product and the functions too, one rounding to fp32. A block forms
// each pair's theta (64-bit powers) once and walks positions, a thread one pair of them. Bound by the rate of 64-bit arithmetic: 32,768
// positions of 128 pairs 251 us (with 4 blocks an SM 265, with powers for every entry 1970; the same in torch operations 354).
constexpr int TABLE_THREADS = 256, TABLE_BLOCKS = 2;     // blocks an SM at most
__global__ void __launch_bounds__(TABLE_THREADS) rope_table_kernel(pace_rope_config r, float2 *table) {
  __shared__ double thetas[128];
  const int half = r.rot >> 1, rows = TABLE_THREADS / half, row = threadIdx.x / half, i = threadIdx.x - row * half;
  double m = r.mscale > 0.0 ? r.mscale : 1.0;
  if (r.scaling == PACE_ROPE_PARTS && !(r.mscale > 0.0)) m = 0.1 * log(r.factor) + 1.0;
  if (row == 0) {
    double base = r.base;
    if (r.scaling == PACE_ROPE_NTK) base *= pow(r.factor, (double)r.rot / (r.rot - 2));
    double theta = pow(base, -2.0 * i / r.rot);
    if (r.scaling == PACE_ROPE_LINEAR) theta /= r.factor;
    if (r.scaling == PACE_ROPE_PARTS) {
      const double turns = r.orig_pos * theta / 6.283185307179586476925;
      const double g = fmin(fmax((turns - r.beta_slow) / (r.beta_fast - r.beta_slow), 0.0), 1.0);
      theta *= g + (1.0 - g) / r.factor;
    }
    thetas[i] = theta;
  }
  __syncthreads();
  if (row >= rows) return;
  const double theta = thetas[i];
  for (long pos = (long)blockIdx.x * rows + row; pos < r.max_pos; pos += (long)gridDim.x * rows) {
    double s, c;
    sincos((double)pos * theta, &s, &c);
    table[pos * half + i] = make_float2((float)(m * c), (float)(m * s));
  }
}

// x [n][heads][d] -> out, HC heads a lane.
template <int IO32, int HC>
__global__ void __launch_bounds__(THREADS) rope_kernel(KvRope r, int n, int heads, int d, KvTensor x,
                                                       const int32_t *__restrict__ positions, KvTensor out, float sign) {
  constexpr int ES = IO32 ? 4 : 2;
  pdl_enter();
  // vectors are packed d/8 lanes each from lane 0 of a warp; lanes past the last whole vector idle
  const int lpv = d >> 3, vpw = 32 / lpv, lane = threadIdx.x & 31;
  const int sub = lane / lpv, a = lane - sub * lpv;
  const unsigned chunks = (heads + HC - 1) / HC;
  const unsigned item = (blockIdx.x * (THREADS / 32) + (threadIdx.x >> 5)) * vpw + sub;
  if (sub >= vpw || item >= n * chunks) return;
  const unsigned t = item / chunks, h0 = (item - t * chunks) * HC;
  const int pos = min(max(positions[t], 0), r.max_pos - 1);
  rotate_heads<IO32, HC>(r, x.p + ((long)t * x.st + (long)h0 * x.sh) * ES, x.sh, out.p + ((long)t * out.st + (long)h0 * out.sh) * ES,
                         out.sh, min(HC, (int)(heads - h0)), a, pos, sign);
}

// Quantize the lane's eight elements within their group of 64 (eight lanes): codes, scale, zero point. quant_group's
// arithmetic with the maxima taken by shuffle. Elements are cleaned (NaN to 0, sizes to 2^120) only where one of them needs it.
template <int BITS>
__device__ __forceinline__ void quant8(const float (&xin)[8], uint32_t (&u)[8], float &s, int &z) {
  float x[8], A = 0.0f, nan = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[i] = xin[i];
    A = fmaxf(A, fabsf(x[i]));
    nan = fmaf(x[i], 0.0f, nan);                         // NaN where an element is NaN or infinite
  }
  if (A > 0x1p120f || nan != 0.0f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = xin[i] != xin[i] ? 0.0f : fminf(fmaxf(xin[i], -0x1p120f), 0x1p120f);
    A = fminf(A, 0x1p120f);
  }
  constexpr int qmax = BITS == 8 ? 127 : 15;
  if (BITS == 8) {
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) A = fmaxf(A, __shfl_xor_sync(0xffffffffu, A, o));
    s = bf16_round(__fdiv_rn(A, (float)qmax));
    z = 128;
  } else {
    float lo = 0.0f, hi = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) lo = fminf(lo, x[i]), hi = fmaxf(hi, x[i]);
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) {
      lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
      hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
    s = bf16_round(__fdiv_rn(__fsub_rn(hi, lo), (float)qmax));
    z = s >= FLT_MIN ? min(max(__float2int_rn(__fmul_rn(-lo, __frcp_rn(s))), 0), qmax) : 0;
  }
  if (!(s >= FLT_MIN)) s = 0.0f;
  const float r = s > 0.0f ? __frcp_rn(s) : 0.0f;
  // Rounded to integers by adding 1.5 * 2^23: the sum's low bits hold the integer, plus `mid`. With 8 bits no code needs a limit: A / 127
  // exceeds s by 2^-8 of s at most, so that |x r| < 127.497.
  const float mid = 12582912.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int c = __float_as_int(__fadd_rn(__fmul_rn(x[i], r), mid)) - __float_as_int(mid);
    u[i] = (uint32_t)(BITS == 8 ? c + 128 : min(max(c + z, 0), qmax));
  }
}

// n / d as n m >> s, exact for n < 2^31 (m = ceil(2^s / d), s = 31 + ceil(log2 d): m d - 2^s < 2^(s - 31)).
struct Div {
  uint32_t m;
  int s;
};
inline Div make_div(uint32_t d) {
  int l = 0;
  while ((1ull << l) < d) ++l;
  return Div{(uint32_t)(((1ull << (31 + l)) + d - 1) / d), 31 + l};
}
__device__ __forceinline__ unsigned divide(unsigned n, const Div &d) { return (unsigned)(((uint64_t)n * d.m) >> d.s); }
struct AppendDivs {
  Div q_chunks, kv_chunks, n_tokens, page;
};

// The new tokens of a call. Some blocks rotate queries (HC heads a lane), which is bound by bytes; the others take key and value
// vectors, 256/D a warp and KC steps of them: keys are rotated, both quantized and written to their tile, which is bound by the
// arithmetic and its latency. The two kinds are spread evenly over the launch, kv_rate / 2^32 of the blocks being of the second.
template <int D, int BITS, int IO32, int HC, int KC>
__global__ void __launch_bounds__(THREADS) append_kernel(KvDev c, KvTensor q, KvTensor k, KvTensor v, KvTensor qo, KvRope r,
                                                         const int32_t *__restrict__ positions, uint64_t kv_rate, AppendDivs by) {
  using L = Tile<D, BITS>;
  constexpr int LPV = D / 8, VPW = 32 / LPV, ES = IO32 ? 4 : 2;
  const int lane = threadIdx.x & 31, sub = lane / LPV, a = lane % LPV;
  pdl_enter();
  const unsigned tokens = (unsigned)c.batch * c.n_tokens;
  auto position = [&](unsigned tok, int b, int t, bool report) {
    const long pos = positions ? positions[tok] : (long)c.lens[b] + t;
    if (pos >= 0 && pos < r.max_pos) return (int)pos;
    if (report && t < new_tokens(c, b)) atomicOr(c.status, PACE_KV_BAD_POSITION);
    return pos < 0 ? 0 : r.max_pos - 1;
  };
  const unsigned kv_block = (unsigned)((blockIdx.x * kv_rate) >> 32);  // blocks of the second kind before this one
  if ((unsigned)(((blockIdx.x + 1) * kv_rate) >> 32) == kv_block) {
    const unsigned chunks = (c.Hq + HC - 1) / HC;
    const unsigned item = ((blockIdx.x - kv_block) * (THREADS / 32) + (threadIdx.x >> 5)) * VPW + sub;
    if (item >= tokens * chunks) return;
    const unsigned tok = divide(item, by.q_chunks), h0 = (item - tok * chunks) * HC;
    const int b = divide(tok, by.n_tokens), t = tok - b * c.n_tokens;
    rotate_heads<IO32, HC>(r, q.p + (b * q.sb + t * q.st + h0 * q.sh) * ES, q.sh, qo.p + (b * qo.sb + t * qo.st + h0 * qo.sh) * ES,
                           qo.sh, min(HC, (int)(c.Hq - h0)), a, position(tok, b, t, a == 0), 1.0f);
    return;
  }
  const unsigned nvec = 2 * c.Hkv, chunks = (nvec + KC * VPW - 1) / (KC * VPW);
  const unsigned item = kv_block * (THREADS / 32) + (threadIdx.x >> 5);
  if (item >= tokens * chunks) return;                 // whole warps
  const unsigned tok = divide(item, by.kv_chunks);
  const int v0 = (item - tok * chunks) * KC * VPW;
  const int b = divide(tok, by.n_tokens), t = tok - b * c.n_tokens;
  float x[KC][8];
#pragma unroll
  for (int i = 0; i < KC; ++i) {
    const int vec = v0 + i * VPW + sub;
    const KvTensor &s = vec < c.Hkv ? k : v;
    if (vec < (int)nvec) load8<IO32>(s.p + (b * s.sb + t * s.st + (vec < c.Hkv ? vec : vec - c.Hkv) * s.sh + 8 * a) * ES, x[i]);
    else {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[i][e] = 0.0f;
    }
  }
  const int len = c.lens[b];
  const long slot = (long)len + t;
  const bool fresh = t < new_tokens(c, b);
  int page = -1;
  char *tiles = nullptr;                               // the slot's tile of head 0; heads are `head_bytes` apart
  const int head_bytes = c.page / TILE * L::BYTES;
  if (fresh && len >= 0 && slot < (long)c.table_cols * c.page) {         // (at most 2^30)
    const unsigned col = divide((unsigned)slot, by.page);
    page = c.table[(long)b * c.table_cols + col];
    if (page >= c.n_pages) page = -1;
    tiles = c.pool + ((long)page * c.Hkv * (c.page / TILE) + ((unsigned)slot - col * c.page) / TILE) * (long)L::BYTES;
  }
  if (fresh && page < 0 && lane == 0) atomicOr(c.status, PACE_KV_BAD_PAGE);
  Angles g;
  if (r.table && v0 < c.Hkv) load_angles(r, position(tok, b, t, lane == 0), a, g);
#pragma unroll
  for (int i = 0; i < KC; ++i) {
    const int vec = v0 + i * VPW + sub;
    const bool key = vec < c.Hkv;
    if (r.table && v0 < c.Hkv) rotate8(r, g, a, key, x[i]);
    uint32_t u[8];
    float s;
    int z;
    quant8<BITS>(x[i], u, s, z);
    if (vec >= (int)nvec || page < 0) continue;
    char *tile = tiles + (long)(key ? vec : vec - c.Hkv) * head_bytes;
    const int tt = (int)(slot % TILE);
    const uint2 w = pack8<BITS>(u);
    char *at = tile + (key ? L::k8(tt, a) : L::v8(tt, a));
    if (BITS == 4) *reinterpret_cast<uint32_t *>(at) = w.x;
    else *reinterpret_cast<uint2 *>(at) = w;
    if ((a & 7) == 0) {
      const int o = (a >> 3) * TILE + L::pos(tt);
      reinterpret_cast<__nv_bfloat16 *>(tile + (key ? L::KS : L::VS))[o] = __float2bfloat16_rn(s);
      if (BITS == 4) tile[key ? L::KZ + o : L::VZ + (a >> 3) * TILE + L::vpos(tt)] = (char)z;
    }
  }
}

// Held values of a range of slots. A block takes one 32-token tile of one head: it reads the tile's bytes once, each lane the
// codes of eight elements, and writes rows of the outputs. Bound by writing; blocks of neighbouring heads run together, so that whole
// rows are under way (tiles first instead of heads: 115 us, not 113).
template <int D, int BITS, int IO32>
__global__ void __launch_bounds__(THREADS) read_kernel(KvDev c, const int32_t *__restrict__ first,
                                                       const int32_t *__restrict__ end, KvTensor k, KvTensor v, int tiles) {
  using L = Tile<D, BITS>;
  constexpr int LPV = D / 8, ROWS = THREADS / LPV, ES = IO32 ? 4 : 2;
  const int a = threadIdx.x % LPV, row = threadIdx.x / LPV;
  pdl_enter();
  const unsigned hi = blockIdx.x / (unsigned)c.Hkv;
  const int head = blockIdx.x - hi * c.Hkv, b = hi / (unsigned)tiles, ti = hi - b * tiles;
  const long f = first ? first[b] : 0;
  const long e = end ? end[b] : (1L << 62);
  const long base = (f >= 0 ? f / TILE : -((-f + TILE - 1) / TILE)) * TILE + (long)ti * TILE;
  if (base >= f + c.n_tokens) return;
  const long live_end = e < f + c.n_tokens ? e : f + c.n_tokens;
  const bool any = base < live_end && base + TILE > f;
  const int page = any ? page_of(c, b, base) : -1;
  if (any && page < 0 && threadIdx.x == 0) atomicOr(c.status, PACE_KV_BAD_PAGE);
  const char *tile = page >= 0 ? tile_at<L::BYTES>(c, page, head, base) : nullptr;
  // all of the lane's codes and parameters are loaded before the first store: the stores could alias them
  constexpr int N = TILE / ROWS;
  uint2 w[2][N];
  __nv_bfloat16 sc[2][N];
  uint8_t z[2][N];
#pragma unroll
  for (int i = 0; i < 2 * N; ++i) {
    const int part = i / N, t = (i % N) * ROWS + row;
    const long slot = base + t;
    if (!tile || slot < f || slot >= live_end) continue;
    const char *at = tile + (part ? L::v8(t, a) : L::k8(t, a));
    if (BITS == 4) w[part][i % N] = make_uint2(*reinterpret_cast<const uint32_t *>(at), 0);
    else w[part][i % N] = *reinterpret_cast<const uint2 *>(at);
    const int p = (a >> 3) * TILE + L::pos(t);
    sc[part][i % N] = reinterpret_cast<const __nv_bfloat16 *>(tile + (part ? L::VS : L::KS))[p];
    if (BITS == 4) z[part][i % N] = (uint8_t)tile[part ? L::VZ + (a >> 3) * TILE + L::vpos(t) : L::KZ + p];
  }
#pragma unroll
  for (int i = 0; i < 2 * N; ++i) {
    const int part = i / N, t = (i % N) * ROWS + row;
    const long slot = base + t;
    if (slot < f || slot >= f + c.n_tokens) continue;
    const KvTensor &o = part ? v : k;
    float y[8];
    if (tile && slot < e) {
      int u[8];
      unpack8<BITS>(w[part][i % N], u);
      const float s = __bfloat162float(sc[part][i % N]);
      const int zero = BITS == 4 ? z[part][i % N] : 128;
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = s * (float)(u[j] - zero);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = 0.0f;
    }
    store8<IO32>(o.p + (b * o.sb + (slot - f) * o.st + head * o.sh + 8 * a) * ES, y);
  }
}

// Accepted drafts move to the front, codes and parameters as they are. One block per (sequence, head); rows go through shared
// memory 32 at a time: since idx rises strictly, idx[i] >= i, and a later batch never reads a row an earlier one wrote.
template <int D, int BITS>
__global__ void __launch_bounds__(THREADS) keep_kernel(KvDev c, int max_new, const int32_t *__restrict__ idx,
                                                       const int32_t *__restrict__ n_keep) {
  using L = Tile<D, BITS>;
  constexpr int WB = BITS == 4 ? 4 : 8;                 // bytes of eight elements
  constexpr int PER = D / 8;
  __shared__ __align__(16) char codes[TILE][2][PER * WB];
  __shared__ uint16_t scale[TILE][2][L::NG];
  __shared__ uint8_t zero[TILE][2][L::NG];
  const int b = blockIdx.x / c.Hkv, head = blockIdx.x % c.Hkv;
  pdl_enter();
  const int asked = n_keep[b], n = min(max(asked, 0), c.n_tokens);
  const long len = c.lens[b];
  const int32_t *row = idx + (long)b * c.n_tokens;
  int good = n;                                        // the first index that does not rise ends the path
  for (int i = threadIdx.x; i < n; i += THREADS)
    if (row[i] < 0 || row[i] >= max_new || (i > 0 && row[i] <= row[i - 1])) good = min(good, i);
  __shared__ int sgood;
  if (threadIdx.x == 0) sgood = n;
  __syncthreads();
  atomicMin(&sgood, good);
  __syncthreads();
  good = sgood;
  if ((good < n || asked != n) && threadIdx.x == 0) atomicOr(c.status, PACE_KV_BAD_KEEP);
  for (int i0 = 0; i0 < good; i0 += TILE) {
    const int m = min(TILE, good - i0);
    for (int w = threadIdx.x; w < m * 2 * PER; w += THREADS) {
      const int i = w / (2 * PER), part = (w / PER) & 1, a = w % PER;
      const long slot = len + row[i0 + i];
      const int page = page_of(c, b, len < 0 ? -1 : slot);
      if (page < 0) {
        atomicOr(c.status, PACE_KV_BAD_PAGE);
        continue;
      }
      const char *tile = tile_at<L::BYTES>(c, page, head, slot);
      const int t = (int)(slot % TILE);
      const char *at = tile + (part ? L::v8(t, a) : L::k8(t, a));
      if (BITS == 4) *reinterpret_cast<uint32_t *>(&codes[i][part][a * WB]) = *reinterpret_cast<const uint32_t *>(at);
      else *reinterpret_cast<uint2 *>(&codes[i][part][a * WB]) = *reinterpret_cast<const uint2 *>(at);
      if ((a & 7) == 0) {
        const int o = (a >> 3) * TILE + L::pos(t);
        scale[i][part][a >> 3] = reinterpret_cast<const uint16_t *>(tile + (part ? L::VS : L::KS))[o];
        if (BITS == 4) zero[i][part][a >> 3] = (uint8_t)tile[part ? L::VZ + (a >> 3) * TILE + L::vpos(t) : L::KZ + o];
      }
    }
    __syncthreads();
    for (int w = threadIdx.x; w < m * 2 * PER; w += THREADS) {
      const int i = w / (2 * PER), part = (w / PER) & 1, a = w % PER;
      const long from = len + row[i0 + i], slot = len + i0 + i;
      const int page = page_of(c, b, len < 0 ? -1 : slot);
      if (page < 0 || from == slot || page_of(c, b, from) < 0) continue;
      char *tile = tile_at<L::BYTES>(c, page, head, slot);
      const int t = (int)(slot % TILE);
      char *at = tile + (part ? L::v8(t, a) : L::k8(t, a));
      if (BITS == 4) *reinterpret_cast<uint32_t *>(at) = *reinterpret_cast<const uint32_t *>(&codes[i][part][a * WB]);
      else *reinterpret_cast<uint2 *>(at) = *reinterpret_cast<const uint2 *>(&codes[i][part][a * WB]);
      if ((a & 7) == 0) {
        const int o = (a >> 3) * TILE + L::pos(t);
        reinterpret_cast<uint16_t *>(tile + (part ? L::VS : L::KS))[o] = scale[i][part][a >> 3];
        if (BITS == 4) tile[part ? L::VZ + (a >> 3) * TILE + L::vpos(t) : L::KZ + o] = (char)zero[i][part][a >> 3];
      }
    }
    __syncthreads();
  }
}

// Launch with the programmatic-serialization attribute: the kernels wait for the one before at their first instruction.
template <typename... P, typename... A>
cudaError_t pdl_launch(void (*kernel)(P...), long blocks, cudaStream_t s, A... args) {
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg = pdl_config(dim3((unsigned)blocks), dim3(THREADS), 0, s, attr);
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <int D, int BITS, int IO32, int HC, int KC>
cudaError_t launch_append(const KvDev &c, const KvTensor &q, const KvTensor &k, const KvTensor &v, const KvTensor &qo,
                          const KvRope &r, const int32_t *pos, cudaStream_t s) {
  constexpr int VPW = 32 / (D / 8), W = THREADS / 32;
  const long tokens = (long)c.batch * c.n_tokens;
  const long q_items = q.p ? tokens * ((c.Hq + HC - 1) / HC) : 0, q_blocks = (q_items + W * VPW - 1) / (W * VPW);
  const long kv_warps = tokens * ((2 * c.Hkv + KC * VPW - 1) / (KC * VPW));
  const long kv_blocks = (kv_warps + W - 1) / W, blocks = q_blocks + kv_blocks;
  // (rounded up: the last block's count comes to kv_blocks, and no count to more)
  const uint64_t kv_rate = (((uint64_t)kv_blocks << 32) + blocks - 1) / blocks;
  const AppendDivs by{make_div((c.Hq + HC - 1) / HC), make_div((2 * c.Hkv + KC * VPW - 1) / (KC * VPW)), make_div(c.n_tokens), make_div(c.page)};
  return pdl_launch(append_kernel<D, BITS, IO32, HC, KC>, blocks, s, c, q, k, v, qo, r, pos, kv_rate, by);
}

}  // namespace kv
}  // namespace pace

using namespace pace;
using namespace pace::kv;

// Calls F<D, BITS, IO32> for the cache's head size, bits and I/O type.
#define KV_DISPATCH(c, F, ...)                                                                             \
  do {                                                                                                     \
    const int io32 = (c).io == PACE_IO_F32;                                                                \
    if ((c).bits == 4) {                                                                                   \
      if ((c).d == 64) return io32 ? F<64, 4, 1>(__VA_ARGS__) : F<64, 4, 0>(__VA_ARGS__);                  \
      if ((c).d == 128) return io32 ? F<128, 4, 1>(__VA_ARGS__) : F<128, 4, 0>(__VA_ARGS__);               \
      return io32 ? F<256, 4, 1>(__VA_ARGS__) : F<256, 4, 0>(__VA_ARGS__);                                 \
    }                                                                                                      \
    if ((c).d == 64) return io32 ? F<64, 8, 1>(__VA_ARGS__) : F<64, 8, 0>(__VA_ARGS__);                    \
    if ((c).d == 128) return io32 ? F<128, 8, 1>(__VA_ARGS__) : F<128, 8, 0>(__VA_ARGS__);                 \
    return io32 ? F<256, 8, 1>(__VA_ARGS__) : F<256, 8, 0>(__VA_ARGS__);                                   \
  } while (0)

cudaError_t pace_launch_rope_table(const pace_rope_config &r, float2 *table, cudaStream_t s) {
  const int rows = TABLE_THREADS / (r.rot / 2), most = TABLE_BLOCKS * device_sm_count();
  const long blocks = ((long)r.max_pos + rows - 1) / rows;
  rope_table_kernel<<<(unsigned)(blocks < most ? blocks : most), TABLE_THREADS, 0, s>>>(r, table);
  return cudaGetLastError();
}

namespace {
template <int IO32, int HC>
cudaError_t rope_go(const KvRope &r, int n, int heads, int d, const KvTensor &x, const int32_t *pos, const KvTensor &out,
                    int inverse, cudaStream_t s) {
  const int per_block = (THREADS / 32) * (32 / (d / 8));
  const long items = (long)n * ((heads + HC - 1) / HC);
  return pdl_launch(rope_kernel<IO32, HC>, (items + per_block - 1) / per_block, s, r, n, heads, d, x, pos, out, inverse ? -1.0f : 1.0f);
}
template <int D, int BITS, int IO32>
cudaError_t append_go(const KvDev &c, const KvTensor &q, const KvTensor &k, const KvTensor &v, const KvTensor &qo,
                      const KvRope &r, const int32_t *pos, cudaStream_t s) {
  const long vecs = (long)c.batch * c.n_tokens * ((q.p ? c.Hq : 0) + 2 * c.Hkv);
  // Two key or value vectors a lane, and four query heads, once there are lanes for a few waves: the angles, lengths and pages are read
  // once for them. 32 and 8 heads of 128, 4 bits, rotated: 2,600 lanes an SM 7.1 us either way, 10,000 17.5 and 15.5, 41,000 59 and 49;
  // with 320 (64 single tokens) one a lane takes 3.9 us and two 5.0.
  if (vecs * (D / 8) > 4096L * device_sm_count())
    return launch_append<D, BITS, IO32, 4, 2>(c, q, k, v, qo, r, pos, s);
  return launch_append<D, BITS, IO32, 1, 1>(c, q, k, v, qo, r, pos, s);
}
template <int D, int BITS, int IO32>
cudaError_t read_go(const KvDev &c, const int32_t *first, const int32_t *end, const KvTensor &k, const KvTensor &v,
                    cudaStream_t s) {
  const int tiles = (c.n_tokens + TILE - 1) / TILE + (first ? 1 : 0);
  const long blocks = (long)c.batch * c.Hkv * tiles;
  return pdl_launch(read_kernel<D, BITS, IO32>, blocks, s, c, first, end, k, v, tiles);
}
template <int D, int BITS, int IO32>
cudaError_t keep_go(const KvDev &c, int max_new, const int32_t *idx, const int32_t *n_keep, cudaStream_t s) {
  return pdl_launch(keep_kernel<D, BITS>, (long)c.batch * c.Hkv, s, c, max_new, idx, n_keep);
}
}  // namespace

cudaError_t pace_launch_rope(const KvRope &r, int n, int heads, int d, int io, const KvTensor &x, const int32_t *pos,
                             const KvTensor &out, int inverse, cudaStream_t s) {
  // Four heads a lane share its angles: 32 heads of 128, 860 lanes an SM 3.4 us with one and 3.2 with four, 28,000 35 and 23 us (134 MB,
  // 5.9 TB/s); with 215 lanes 2.7 and 2.8 us.
  const bool many = (long)n * heads * (d / 8) > 512L * device_sm_count();
  if (io == PACE_IO_F32)
    return many ? rope_go<1, 4>(r, n, heads, d, x, pos, out, inverse, s) : rope_go<1, 1>(r, n, heads, d, x, pos, out, inverse, s);
  return many ? rope_go<0, 4>(r, n, heads, d, x, pos, out, inverse, s) : rope_go<0, 1>(r, n, heads, d, x, pos, out, inverse, s);
}

cudaError_t pace_launch_kv_append(const KvDev &c, const KvTensor &q, const KvTensor &k, const KvTensor &v,
                                  const KvTensor &qo, const KvRope &r, const int32_t *pos, cudaStream_t s) {
  KV_DISPATCH(c, append_go, c, q, k, v, qo, r, pos, s);
}
cudaError_t pace_launch_kv_read(const KvDev &c, const int32_t *first, const int32_t *end, const KvTensor &k,
                                const KvTensor &v, cudaStream_t s) {
  KV_DISPATCH(c, read_go, c, first, end, k, v, s);
}
cudaError_t pace_launch_kv_keep(const KvDev &c, int max_new, const int32_t *idx, const int32_t *n_keep, cudaStream_t s) {
  KV_DISPATCH(c, keep_go, c, max_new, idx, n_keep, s);
}
