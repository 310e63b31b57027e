// Rotary positions and the quantized KV cache outside attention: the cos/sin table, rotation, append (rotation and
// quantization fused), read-back and the move of an accepted path.
//
// All of these move bytes: a lane owns eight consecutive elements (one 16-byte bf16 vector, two fp32 ones), D/8 lanes a head
// vector, 256/D vectors a warp. The arithmetic per element (a rotation, a group maximum over eight lanes, one rounding) is
// small beside the memory time, so the floor of every call is its bytes at the copy bandwidth.
#include "kv_common.cuh"

namespace pace {
namespace kv {

constexpr int THREADS = 128;

template <int IO32>
struct Vec8 {
  float x[8];
};

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

// cos and sin of the lane's eight elements (interleaved: of its four pairs) at one position.
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
// Rotate the lane's eight elements in place; every lane of the warp takes part (the partner half comes by shuffle). Products
// and sums are rounded apart (no contraction), so that the rotated value is the same wherever it is formed.
__device__ __forceinline__ void rotate8(const KvRope &r, const Angles &g, int a, bool on, float sign, float (&x)[8]) {
  const int half = r.rot >> 1, e0 = 8 * a, lane = threadIdx.x & 31;
  const bool in = on && e0 < r.rot;
  if (r.interleaved) {
    if (!in) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float c = g.cs[i].x, s = sign * g.cs[i].y, u = x[2 * i], v = x[2 * i + 1];
      x[2 * i] = __fsub_rn(__fmul_rn(u, c), __fmul_rn(v, s));
      x[2 * i + 1] = __fadd_rn(__fmul_rn(v, c), __fmul_rn(u, s));
    }
    return;
  }
  const bool lo = e0 < half;
  const int src = e0 < r.rot ? (lo ? lane + (half >> 3) : lane - (half >> 3)) : lane;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float p = __shfl_sync(0xffffffffu, x[i], src & 31);
    if (in) {
      const float c = g.cs[i].x, s = sign * g.cs[i].y;
      x[i] = lo ? __fsub_rn(__fmul_rn(x[i], c), __fmul_rn(p, s)) : __fadd_rn(__fmul_rn(x[i], c), __fmul_rn(p, s));
    }
  }
}

// cos and sin in 64 bits, once per table: theta is exact to fp64, the product and the functions too, one rounding to fp32.
__global__ void rope_table_kernel(pace_rope_config r, float2 *table) {
  const int half = r.rot >> 1;
  const long total = (long)r.max_pos * half;
  for (long idx = (long)blockIdx.x * blockDim.x + threadIdx.x; idx < total; idx += (long)gridDim.x * blockDim.x) {
    const int i = (int)(idx % half);
    const double pos = (double)(idx / half), e = -2.0 * i / r.rot;
    double base = r.base, m = r.mscale > 0.0 ? r.mscale : 1.0;
    if (r.scaling == PACE_ROPE_NTK) base *= pow(r.factor, (double)r.rot / (r.rot - 2));
    double theta = pow(base, e);
    if (r.scaling == PACE_ROPE_LINEAR) theta /= r.factor;
    if (r.scaling == PACE_ROPE_PARTS) {
      const double turns = r.orig_pos * theta / 6.283185307179586476925;
      const double g = fmin(fmax((turns - r.beta_slow) / (r.beta_fast - r.beta_slow), 0.0), 1.0);
      theta *= g + (1.0 - g) / r.factor;
      if (!(r.mscale > 0.0)) m = 0.1 * log(r.factor) + 1.0;
    }
    double s, c;
    sincos(pos * theta, &s, &c);
    table[idx] = make_float2((float)(m * c), (float)(m * s));
  }
}

// x [n][heads][d] -> out. A lane keeps its position's angles for HC heads, so the table is read once per HC vectors.
template <int IO32, int HC>
__global__ void __launch_bounds__(THREADS) rope_kernel(KvRope r, int n, int heads, int d, KvTensor x,
                                                       const int32_t *__restrict__ positions, KvTensor out, float sign) {
  constexpr int ES = IO32 ? 4 : 2;
  // vectors are packed d/8 lanes each from lane 0 of a warp; lanes past the last whole vector idle
  const int lpv = d >> 3, vpw = 32 / lpv, lane = threadIdx.x & 31;
  const int sub = lane / lpv, a = lane - sub * lpv;
  const int chunks = (heads + HC - 1) / HC;
  const long item = ((long)blockIdx.x * (THREADS / 32) + (threadIdx.x >> 5)) * vpw + sub;
  const bool live = sub < vpw && item < (long)n * chunks;
  const int t = live ? (int)(item / chunks) : 0, h0 = live ? (int)(item - (long)t * chunks) * HC : 0;
  float v[HC][8];
#pragma unroll
  for (int i = 0; i < HC; ++i)
    if (live && h0 + i < heads) load8<IO32>(x.p + ((long)t * x.st + (long)(h0 + i) * x.sh + 8 * a) * ES, v[i]);
  Angles g;
  if (live) load_angles(r, min(max(positions[t], 0), r.max_pos - 1), a, g);
#pragma unroll
  for (int i = 0; i < HC; ++i) {
    rotate8(r, g, a, live, sign, v[i]);
    if (live && h0 + i < heads) store8<IO32>(out.p + ((long)t * out.st + (long)(h0 + i) * out.sh + 8 * a) * ES, v[i]);
  }
}

// Quantize the lane's eight elements within their group of 64 (eight lanes): codes, scale, zero point. quant_group's
// arithmetic with the maxima taken by shuffle.
template <int BITS>
__device__ __forceinline__ void quant8(const float (&xin)[8], uint32_t (&u)[8], float &s, int &z) {
  float x[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[i] = fminf(fmaxf(xin[i], -0x1p120f), 0x1p120f);   // fmaxf drops a NaN
    if (xin[i] != xin[i]) x[i] = 0.0f;
  }
  constexpr int qmax = BITS == 8 ? 127 : 15;
  if (BITS == 8) {
    float A = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) A = fmaxf(A, fabsf(x[i]));
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
    z = s >= FLT_MIN ? min(max(__float2int_rn(__fmul_rn(-lo, __fdiv_rn(1.0f, s))), 0), qmax) : 0;
  }
  if (!(s >= FLT_MIN)) s = 0.0f;
  const float r = s > 0.0f ? __fdiv_rn(1.0f, s) : 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int c = __float2int_rn(__fmul_rn(x[i], r));
    u[i] = (uint32_t)(BITS == 8 ? min(max(c, -qmax), qmax) + 128 : min(max(c + z, 0), qmax));
  }
}

// The new tokens of a call: query vectors rotated, key vectors rotated and quantized, value vectors quantized. A warp holds
// 256/D vectors of one token (HC steps of them over the vectors q.., k.., v.. of that token).
template <int D, int BITS, int IO32, int HC>
__global__ void __launch_bounds__(THREADS) append_kernel(KvDev c, KvTensor q, KvTensor k, KvTensor v, KvTensor qo, KvRope r,
                                                         const int32_t *__restrict__ positions) {
  using L = Tile<D, BITS>;
  constexpr int LPV = D / 8, VPW = 32 / LPV, ES = IO32 ? 4 : 2;
  const int lane = threadIdx.x & 31, sub = lane / LPV, a = lane % LPV;
  const int nq = q.p ? c.Hq : 0, nvec = nq + 2 * c.Hkv;
  const int chunks = (nvec + HC * VPW - 1) / (HC * VPW);
  const long item = (long)blockIdx.x * (THREADS / 32) + (threadIdx.x >> 5);
  if (item >= (long)c.batch * c.n_tokens * chunks) return;   // whole warps
  const int tok = (int)(item / chunks), v0 = (int)(item - (long)tok * chunks) * HC * VPW;
  const int b = tok / c.n_tokens, t = tok - b * c.n_tokens;
  float x[HC][8];
  int kind[HC], head[HC];       // 0 query, 1 key, 2 value, -1 none
#pragma unroll
  for (int i = 0; i < HC; ++i) {
    const int vec = v0 + i * VPW + sub;
    kind[i] = vec < nq ? 0 : vec < nq + c.Hkv ? 1 : vec < nvec ? 2 : -1;
    head[i] = kind[i] == 0 ? vec : kind[i] == 1 ? vec - nq : vec - nq - c.Hkv;
    const KvTensor &s = kind[i] == 0 ? q : kind[i] == 1 ? k : v;
    if (kind[i] >= 0) load8<IO32>(s.p + (b * s.sb + t * s.st + head[i] * s.sh + 8 * a) * ES, x[i]);
    else {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[i][e] = 0.0f;
    }
  }
  const int len = c.lens[b];
  const long slot = (long)len + t;
  const bool fresh = t < new_tokens(c, b);
  const int page = fresh ? page_of(c, b, len < 0 ? -1 : slot) : -1;
  Angles g;
  if (r.table) {
    const long pos = positions ? positions[tok] : slot;
    const bool bad = pos < 0 || pos >= r.max_pos;
    if (bad && fresh && lane == 0 && v0 < nq + c.Hkv) atomicOr(c.status, PACE_KV_BAD_POSITION);
    load_angles(r, bad ? (pos < 0 ? 0 : r.max_pos - 1) : (int)pos, a, g);
  }
  if (fresh && page < 0 && lane == 0) atomicOr(c.status, PACE_KV_BAD_PAGE);
#pragma unroll
  for (int i = 0; i < HC; ++i) {
    if (r.table) rotate8(r, g, a, kind[i] == 0 || kind[i] == 1, 1.0f, x[i]);
    if (kind[i] == 0) store8<IO32>(qo.p + (b * qo.sb + t * qo.st + head[i] * qo.sh + 8 * a) * ES, x[i]);
    if (__all_sync(0xffffffffu, kind[i] <= 0)) continue;
    uint32_t u[8];
    float s;
    int z;
    quant8<BITS>(x[i], u, s, z);
    if (kind[i] <= 0 || page < 0) continue;
    char *tile = tile_at<L::BYTES>(c, page, head[i], slot);
    const int tt = (int)(slot % TILE);
    const bool key = kind[i] == 1;
    const uint2 w = pack8<BITS>(u);
    char *at = tile + (key ? L::k8(tt, a) : L::v8(tt, a));
    if (BITS == 4) *reinterpret_cast<uint32_t *>(at) = w.x;
    else *reinterpret_cast<uint2 *>(at) = w;
    if ((a & 7) == 0) {
      const int o = (a >> 3) * TILE + L::pos(tt);
      reinterpret_cast<__nv_bfloat16 *>(tile + (key ? L::KS : L::VS))[o] = __float2bfloat16_rn(s);
      if (BITS == 4) reinterpret_cast<uint8_t *>(tile + (key ? L::KZ : L::VZ))[o] = (uint8_t)z;
    }
  }
}

// Held values of a range of slots. A block takes one 32-token tile of one head: it reads the tile's bytes once, each lane the
// codes of eight elements, and writes rows of the outputs.
template <int D, int BITS, int IO32>
__global__ void __launch_bounds__(THREADS) read_kernel(KvDev c, const int32_t *__restrict__ first,
                                                       const int32_t *__restrict__ end, KvTensor k, KvTensor v, int tiles) {
  using L = Tile<D, BITS>;
  constexpr int LPV = D / 8, ROWS = THREADS / LPV, ES = IO32 ? 4 : 2;
  const int a = threadIdx.x % LPV, row = threadIdx.x / LPV;
  const long item = blockIdx.x;
  const int head = (int)(item % c.Hkv), ti = (int)((item / c.Hkv) % tiles), b = (int)(item / ((long)c.Hkv * tiles));
  const long f = first ? first[b] : 0;
  const long e = end ? end[b] : (1L << 62);
  const long base = (f >= 0 ? f / TILE : -((-f + TILE - 1) / TILE)) * TILE + (long)ti * TILE;
  if (base >= f + c.n_tokens) return;
  const long live_end = e < f + c.n_tokens ? e : f + c.n_tokens;
  const bool any = base < live_end && base + TILE > f;
  const int page = any ? page_of(c, b, base) : -1;
  if (any && page < 0 && threadIdx.x == 0) atomicOr(c.status, PACE_KV_BAD_PAGE);
  const char *tile = page >= 0 ? tile_at<L::BYTES>(c, page, head, base) : nullptr;
#pragma unroll
  for (int part = 0; part < 2; ++part) {
    const KvTensor &o = part ? v : k;
#pragma unroll
    for (int t0 = 0; t0 < TILE; t0 += ROWS) {
      const int t = t0 + row;
      const long slot = base + t;
      if (slot < f || slot >= f + c.n_tokens) continue;
      float y[8];
      if (slot < e && tile) {
        const char *at = tile + (part ? L::v8(t, a) : L::k8(t, a));
        uint2 w;
        if (BITS == 4) w = make_uint2(*reinterpret_cast<const uint32_t *>(at), 0);
        else w = *reinterpret_cast<const uint2 *>(at);
        const int p = (a >> 3) * TILE + L::pos(t);
        const float s = __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(tile + (part ? L::VS : L::KS))[p]);
        const int z = BITS == 4 ? reinterpret_cast<const uint8_t *>(tile + (part ? L::VZ : L::KZ))[p] : 128;
        int u[8];
        unpack8<BITS>(w, u);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = s * (float)(u[i] - z);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = 0.0f;
      }
      store8<IO32>(o.p + (b * o.sb + (slot - f) * o.st + head * o.sh + 8 * a) * ES, y);
    }
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
  const int n = min(max(n_keep[b], 0), c.n_tokens);
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
  if (good < n && threadIdx.x == 0) atomicOr(c.status, PACE_KV_BAD_KEEP);
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
        if (BITS == 4) zero[i][part][a >> 3] = reinterpret_cast<const uint8_t *>(tile + (part ? L::VZ : L::KZ))[o];
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
        if (BITS == 4) reinterpret_cast<uint8_t *>(tile + (part ? L::VZ : L::KZ))[o] = zero[i][part][a >> 3];
      }
    }
    __syncthreads();
  }
}

template <int D, int BITS, int IO32, int HC>
cudaError_t launch_append(const KvDev &c, const KvTensor &q, const KvTensor &k, const KvTensor &v, const KvTensor &qo,
                          const KvRope &r, const int32_t *pos, cudaStream_t s) {
  constexpr int VPW = 32 / (D / 8);
  const int nvec = (q.p ? c.Hq : 0) + 2 * c.Hkv, chunks = (nvec + HC * VPW - 1) / (HC * VPW);
  const long warps = (long)c.batch * c.n_tokens * chunks;
  append_kernel<D, BITS, IO32, HC><<<(unsigned)((warps + THREADS / 32 - 1) / (THREADS / 32)), THREADS, 0, s>>>(c, q, k, v, qo, r, pos);
  return cudaGetLastError();
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
  const long total = (long)r.max_pos * (r.rot / 2);
  const long blocks = (total + 255) / 256;
  rope_table_kernel<<<(unsigned)(blocks < 16384 ? blocks : 16384), 256, 0, s>>>(r, table);
  return cudaGetLastError();
}

namespace {
template <int IO32, int HC>
cudaError_t rope_go(const KvRope &r, int n, int heads, int d, const KvTensor &x, const int32_t *pos, const KvTensor &out,
                    int inverse, cudaStream_t s) {
  const int per_block = (THREADS / 32) * (32 / (d / 8));
  const long items = (long)n * ((heads + HC - 1) / HC);
  rope_kernel<IO32, HC><<<(unsigned)((items + per_block - 1) / per_block), THREADS, 0, s>>>(r, n, heads, d, x, pos, out,
                                                                                          inverse ? -1.0f : 1.0f);
  return cudaGetLastError();
}
template <int D, int BITS, int IO32>
cudaError_t append_go(const KvDev &c, const KvTensor &q, const KvTensor &k, const KvTensor &v, const KvTensor &qo,
                      const KvRope &r, const int32_t *pos, cudaStream_t s) {
  const long vecs = (long)c.batch * c.n_tokens * ((q.p ? c.Hq : 0) + 2 * c.Hkv);
  if (vecs * (D / 8) > 4L * 2048 * device_sm_count())
    return launch_append<D, BITS, IO32, 4>(c, q, k, v, qo, r, pos, s);
  return launch_append<D, BITS, IO32, 1>(c, q, k, v, qo, r, pos, s);
}
template <int D, int BITS, int IO32>
cudaError_t read_go(const KvDev &c, const int32_t *first, const int32_t *end, const KvTensor &k, const KvTensor &v,
                    cudaStream_t s) {
  const int tiles = (c.n_tokens + TILE - 1) / TILE + (first ? 1 : 0);
  const long blocks = (long)c.batch * c.Hkv * tiles;
  read_kernel<D, BITS, IO32><<<(unsigned)blocks, THREADS, 0, s>>>(c, first, end, k, v, tiles);
  return cudaGetLastError();
}
template <int D, int BITS, int IO32>
cudaError_t keep_go(const KvDev &c, int max_new, const int32_t *idx, const int32_t *n_keep, cudaStream_t s) {
  keep_kernel<D, BITS><<<(unsigned)(c.batch * c.Hkv), THREADS, 0, s>>>(c, max_new, idx, n_keep);
  return cudaGetLastError();
}
}  // namespace

cudaError_t pace_launch_rope(const KvRope &r, int n, int heads, int d, int io, const KvTensor &x, const int32_t *pos,
                             const KvTensor &out, int inverse, cudaStream_t s) {
  const bool many = (long)n * heads * (d / 8) > 4L * 2048 * device_sm_count();
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
