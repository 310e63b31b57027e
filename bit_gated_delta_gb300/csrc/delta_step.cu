// The gated delta rule token by token, the state in registers (pace_serve.h): S <- a S + k u^T, u = beta (v - a S^T k), o = S^T q.
//
// A block takes COLS columns of one state (columns of a state do not meet); a thread holds four columns of D*COLS/1024 rows. Per token
// both dots are taken of the old state in one pass, w = S^T k and p = S^T q, and joined over the row groups (shuffles, then one
// exchange through shared memory); u = beta (v - a w), o = a p + (q.k) u, so that the update needs no second exchange. fp32
// throughout, two operations an instruction. Bound by the states' bytes, read and written once: 64 tokens of 32 heads of 128 take 49 us (5.4 TB/s);
// a call of one token of 16 heads of 64 takes 3.2 us.
#include "delta_common.cuh"

namespace pace {
namespace delta {

constexpr int STEP_THREADS = 256, STEP_WARPS = STEP_THREADS / 32;
constexpr int STEP_STAGE = 8;            // tokens staged at a time
// The most tokens of a call that go one by one; longer ones, and trees, go by chunks (delta_chunk.cuh). Measured, us, one by one (by chunks), states not
// in L2. fp32: 1024 sequences and heads of 128, 10 tokens 89 (94), 12 100 (94), 14 112 (94); 64 of 10 tokens 16 (17), 14 21 (17); 1024 of 64, 12
// tokens 52 (57). bf16, heads of 128: 1024 of 6 tokens 61 (62), 8 74 (61); 256 of 8 tokens 20 (23), 10 24 (23); heads of 64: 1024 of 8 35 (43), 10 41 (44),
// 64 of 8 12 (12).
constexpr int step_most(int io, int d, bool many) { return io == PACE_IO_F32 ? 11 : d == 128 && many ? 6 : 8; }

__device__ __forceinline__ uint64_t pk(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 upk(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
template <bool F32>
__device__ __forceinline__ float4 load4(const KvTensor &x, long at) {
  if (F32) return *reinterpret_cast<const float4 *>(x.p + at * 4);
  const uint2 r = *reinterpret_cast<const uint2 *>(x.p + at * 2);
  return make_float4(__uint_as_float(r.x << 16), __uint_as_float(r.x & 0xFFFF0000u), __uint_as_float(r.y << 16),
                     __uint_as_float(r.y & 0xFFFF0000u));
}
template <bool F32>
__device__ __forceinline__ void store4(const KvTensor &x, long at, float4 y) {
  if (F32) {
    *reinterpret_cast<float4 *>(x.p + at * 4) = y;
  } else {
    const __nv_bfloat162 lo = __floats2bfloat162_rn(y.x, y.y), hi = __floats2bfloat162_rn(y.z, y.w);
    *reinterpret_cast<uint2 *>(x.p + at * 2) =
        make_uint2(*reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
  }
}

template <int D, int COLS, bool F32>
__global__ void __launch_bounds__(STEP_THREADS, D * COLS == 128 * 128 ? 2 : 4) delta_step_kernel(const DeltaArgs p) {
  constexpr int CG = COLS / 4, RG = STEP_THREADS / CG, R = D / RG, WG = 32 / CG;   // column quads, row groups, rows a thread, row groups a warp
  constexpr int PARTS = D / COLS;
  static_assert(R >= 1 && R % 2 == 0 && WG >= 1, "rows come in pairs");
  struct Shared {
    float2 k[STEP_STAGE][D], q[STEP_STAGE][D];           // each value twice, as the packed products take it
    float4 v[STEP_STAGE][CG];
    float a[STEP_STAGE], beta[STEP_STAGE];
    float4 w[2][STEP_WARPS][CG], p[2][STEP_WARPS][CG];   // partial dots of the warps, of tokens in turn
    float kq[2][STEP_WARPS];
  };
  __shared__ __align__(16) Shared sh;
  pdl_enter();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int part = blockIdx.x % PARTS, unit = blockIdx.x / PARTS, b = unit / p.H, h = unit - b * p.H;
  int bad = 0;
  Seq s = sequence(p, b, bad);
  const int c = tid % CG, row0 = tid / CG * R, col = part * COLS + 4 * c;
  const bool out = p.o.p != nullptr;
  const int hk = h / p.group;

  uint64_t S[R][2];
  float *state = p.S + ((long)s.slot * p.H + h) * D * D + (long)row0 * D + col;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (s.n > 0 && !s.fresh) x = *reinterpret_cast<const float4 *>(state + r * D);
    S[r][0] = pk(x.x, x.y);
    S[r][1] = pk(x.z, x.w);
  }

  if (s.n > 0 && taken(p, b, s.slot)) {                  // (looked at while the state is on its way)
    bad |= PACE_DELTA_BAD_SLOT;
    s.n = 0;
  }
  if (bad && part == 0 && h == 0 && tid == 0) atomicOr(p.status, bad);

  int turn = 0;
  // one token of the staged ones; `emit`: row of o that its output goes to (-1: none)
  auto token = [&](int i, int emit) {
    uint64_t w0 = 0, w1 = 0, p0 = 0, p1 = 0, kq = 0;
#pragma unroll
    for (int r = 0; r < R; r += 2) {
      const float4 k2 = *reinterpret_cast<const float4 *>(&sh.k[i][row0 + r]), q2 = *reinterpret_cast<const float4 *>(&sh.q[i][row0 + r]);
      const uint64_t ka = pk(k2.x, k2.y), kb = pk(k2.z, k2.w), qa = pk(q2.x, q2.y), qb = pk(q2.z, q2.w);
      w0 = fma2(ka, S[r][0], w0), w1 = fma2(ka, S[r][1], w1);
      w0 = fma2(kb, S[r + 1][0], w0), w1 = fma2(kb, S[r + 1][1], w1);
      p0 = fma2(qa, S[r][0], p0), p1 = fma2(qa, S[r][1], p1);
      p0 = fma2(qb, S[r + 1][0], p0), p1 = fma2(qb, S[r + 1][1], p1);
      kq = fma2(ka, qa, kq), kq = fma2(kb, qb, kq);
    }
    float2 x0 = upk(w0), x1 = upk(w1), y0 = upk(p0), y1 = upk(p1);
    float g = upk(kq).x;
#pragma unroll
    for (int m = CG; m < 32; m <<= 1) {
      x0.x += __shfl_xor_sync(0xffffffffu, x0.x, m), x0.y += __shfl_xor_sync(0xffffffffu, x0.y, m);
      x1.x += __shfl_xor_sync(0xffffffffu, x1.x, m), x1.y += __shfl_xor_sync(0xffffffffu, x1.y, m);
      y0.x += __shfl_xor_sync(0xffffffffu, y0.x, m), y0.y += __shfl_xor_sync(0xffffffffu, y0.y, m);
      y1.x += __shfl_xor_sync(0xffffffffu, y1.x, m), y1.y += __shfl_xor_sync(0xffffffffu, y1.y, m);
      g += __shfl_xor_sync(0xffffffffu, g, m);
    }
    if (lane < CG) {
      sh.w[turn][warp][lane] = make_float4(x0.x, x0.y, x1.x, x1.y);
      sh.p[turn][warp][lane] = make_float4(y0.x, y0.y, y1.x, y1.y);
      if (lane == 0) sh.kq[turn][warp] = g;
    }
    __syncthreads();
    float4 w = make_float4(0.0f, 0.0f, 0.0f, 0.0f), pq = w;
    g = 0.0f;
#pragma unroll
    for (int i2 = 0; i2 < STEP_WARPS; ++i2) {
      const float4 x = sh.w[turn][i2][c], y = sh.p[turn][i2][c];
      w.x += x.x, w.y += x.y, w.z += x.z, w.w += x.w;
      pq.x += y.x, pq.y += y.y, pq.z += y.z, pq.w += y.w;
      g += sh.kq[turn][i2];
    }
    turn ^= 1;
    const float a = sh.a[i], be = sh.beta[i];
    const float4 v = sh.v[i][c];
    const float4 u = make_float4(be * fmaf(-a, w.x, v.x), be * fmaf(-a, w.y, v.y), be * fmaf(-a, w.z, v.z), be * fmaf(-a, w.w, v.w));
    const uint64_t a2 = pk(a, a), u0 = pk(u.x, u.y), u1 = pk(u.z, u.w);
#pragma unroll
    for (int r = 0; r < R; r += 2) {
      const float4 k2 = *reinterpret_cast<const float4 *>(&sh.k[i][row0 + r]);
      const uint64_t ka = pk(k2.x, k2.y), kb = pk(k2.z, k2.w);
      S[r][0] = fma2(ka, u0, mul2(a2, S[r][0])), S[r][1] = fma2(ka, u1, mul2(a2, S[r][1]));
      S[r + 1][0] = fma2(kb, u0, mul2(a2, S[r + 1][0])), S[r + 1][1] = fma2(kb, u1, mul2(a2, S[r + 1][1]));
    }
    if (emit >= 0 && tid < CG)
      store4<F32>(p.o, b * p.o.sb + (long)emit * p.o.st + h * p.o.sh + col,
                  make_float4(fmaf(a, pq.x, g * u.x), fmaf(a, pq.y, g * u.y), fmaf(a, pq.z, g * u.z), fmaf(a, pq.w, g * u.w)));
  };
  // the i-th staged token is `t`
  auto stage = [&](int i, int t) {
    const int row = row_of(p, b, t);
    for (int x = tid; x < D / 4; x += STEP_THREADS) {
      const float4 k = load4<F32>(p.k, b * p.k.sb + (long)row * p.k.st + hk * p.k.sh + 4 * x);
      float4 q = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (p.q.p) q = load4<F32>(p.q, b * p.q.sb + (long)row * p.q.st + hk * p.q.sh + 4 * x);
      float4 *kd = reinterpret_cast<float4 *>(&sh.k[i][4 * x]), *qd = reinterpret_cast<float4 *>(&sh.q[i][4 * x]);
      kd[0] = make_float4(k.x, k.x, k.y, k.y), kd[1] = make_float4(k.z, k.z, k.w, k.w);
      qd[0] = make_float4(q.x, q.x, q.y, q.y), qd[1] = make_float4(q.z, q.z, q.w, q.w);
    }
    if (tid >= 64 && tid < 64 + CG)
      sh.v[i][tid - 64] = load4<F32>(p.v, b * p.v.sb + (long)row * p.v.st + h * p.v.sh + part * COLS + 4 * (tid - 64));
    if (tid == 128) sh.a[i] = reinterpret_cast<const float *>(p.a.p)[b * p.a.sb + (long)row * p.a.st + h * p.a.sh];
    if (tid == 160) sh.beta[i] = reinterpret_cast<const float *>(p.beta.p)[b * p.beta.sb + (long)row * p.beta.st + h * p.beta.sh];
  };

  for (int t0 = 0; t0 < s.n; t0 += STEP_STAGE) {
    const int m = min(STEP_STAGE, s.n - t0);
    __syncthreads();
    for (int i = 0; i < m; ++i) stage(i, t0 + i);
    __syncthreads();
    for (int i = 0; i < m; ++i) token(i, out ? t0 + i : -1);
  }
  if (p.write && s.n > 0) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float2 x = upk(S[r][0]), y = upk(S[r][1]);
      *reinterpret_cast<float4 *>(state + r * D) = make_float4(x.x, x.y, y.x, y.y);
    }
  }
  if (out)                                               // rows past the sequence's tokens
    for (int i = tid; i < (p.n_tokens - s.n) * CG; i += STEP_THREADS)
      store4<F32>(p.o, b * p.o.sb + (long)(s.n + i / CG) * p.o.st + h * p.o.sh + part * COLS + 4 * (i % CG), make_float4(0.0f, 0.0f, 0.0f, 0.0f));
}

template <int D, int COLS, bool F32>
cudaError_t launch_step(const DeltaArgs &p, cudaStream_t s) {
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg = pdl_config(dim3((unsigned)(p.batch * p.H * (D / COLS))), dim3(STEP_THREADS), 0, s, attr);
  return cudaLaunchKernelEx(&cfg, delta_step_kernel<D, COLS, F32>, p);
}

template <bool F32>
cudaError_t launch_step_t(const DeltaArgs &p, cudaStream_t s) {
  if (p.d == 64) return launch_step<64, 64, F32>(p, s);
  // (a quarter of the columns a block while all of them fit the multiprocessors: 16 heads of one sequence 3.3 us, whole states 4.3; 128 heads 5.8 and 5.7)
  if (p.batch * p.H * 4 <= device_sm_count()) return launch_step<128, 32, F32>(p, s);
  return launch_step<128, 128, F32>(p, s);
}

}  // namespace delta
}  // namespace pace

cudaError_t pace_launch_delta(const DeltaArgs &p, cudaStream_t s) {
  using namespace pace::delta;
  const int most = p.idx && p.n_idx < p.n_tokens ? p.n_idx : p.n_tokens;
  if ((p.mask && p.n_tokens > 1) || most > step_most(p.io, p.d, (long)p.batch * p.H > 4 * pace::device_sm_count()))
    return p.io == PACE_IO_F32 ? pace_launch_delta_chunk_f32(p, s) : pace_launch_delta_chunk_bf16(p, s);
  return p.io == PACE_IO_F32 ? launch_step_t<true>(p, s) : launch_step_t<false>(p, s);
}
