// The gated delta rule over states in slots by chunks of 64 tokens on the 5th-generation tensor cores (pace_serve.h).
//
// With G_t the product of the decays of t and its ancestors, R_ts that of the ancestors of t after s (t included; 0 where s is neither t nor
// an ancestor), and S the state at a chunk's start:
//   (I + M) u = beta (v - G S^T k),  M_ts = beta_t R_ts k_t.k_s (s < t)         T = (I + M)^-1, lower triangular
//   o_t = G_t S^T q_t + sum_s P_ts u_s,  P_ts = R_ts q_t.k_s (s <= t)
//   S' = G_C S + sum_t R_Ct k_t u_t^T
// which is the rule token by token, expanded. A tree of drafts is one chunk whose R has zeros, a prompt a chain of chunks.
//
// One block takes a sequence and head. Lane j of TMEM is column j of the state, of u and of o (as their transposes), so that each
// product's first operand comes from TMEM, where the thread that owns the column wrote it, and no value crosses lanes:
//   D1 = S^T [k | q]      A = S in registers, split in parts          B = rows k, q in shared memory
//   D2 = rhs T^T          A = rhs = beta (v - G w)                    B = T
//   D3 = (R_C u) k^T      A = R_C u                                   B = the rows k again, read along the other dimension
//   D4 = u P^T            A = u                                       B = P
// fp32 operands are split into bf16 parts (x = hi + mid + lo, 24 bits), of whose products those above 2^-24 are formed, smallest first; q and k
// of bf16 I/O enter as they are. bf16 I/O forms outputs from two parts (16 bits; o is rounded to 8). The state itself stays in fp32 registers
// and takes D3 by an ordinary addition: the tensor cores' additions cut off, which would add up over a long prompt.
//
// Roles: eight warps own the columns (two a quarter of TMEM's lanes: token blocks of 16 in turn, halves of the state's rows), four form R, M, P
// and T one chunk ahead, three copy rows in, one issues the products.
// Every wait is bounded; one that gives up sets the status word, after which the block goes on without waiting or products and leaves the state.
#pragma once

#include "delta_common.cuh"
#include "umma.cuh"

#include <type_traits>

namespace pace {
namespace delta {
using namespace umma;

constexpr int C = 64;                                    // tokens a chunk

template <int D, bool F32>
struct Shape {
  static constexpr int MAIN = 8, AUX = 4, W_MMA = MAIN + AUX, W_LOAD = W_MMA + 1, LOAD = 3, THREADS = (W_LOAD + LOAD) * 32;
  static constexpr int NX = F32 ? 3 : 1;                 // parts of q and k
  static constexpr int NO = F32 ? 3 : 2;                 // parts of u and P in the outputs
  static constexpr int NB = F32 ? 1 : 3;                 // chunks of rows in shared memory
  static constexpr int ROWS = C * D * 2;                 // one part of 64 rows
  static constexpr int XPART = 2 * ROWS, XBUF = NX * XPART;
  static constexpr int VBUF = C * D * (F32 ? 4 : 2);
  static constexpr int TPART = C * C * 2;
  static constexpr int LD = C + 4, LY = 36;              // rows of the fp32 tables
  static constexpr int OX = 0, OV = OX + NB * XBUF, OT = OV + NB * VBUF, OP = OT + 3 * TPART, OM = OP + NO * TPART,
                       OTF = OM + C * LD * 4, OY = OTF + C * LD * 4, OG = OY + 32 * LY * 4, OBAR = OG + 3 * 4 * C * 4,
                       NBAR = 2 * NB + 3 + 14, OMISC = OBAR + NBAR * 8, SMEM = OMISC + 16;
  static_assert(SMEM <= 227 * 1024 && OBAR % 8 == 0, "shared memory");
  // TMEM columns: parts of S, later of R_C u; rhs and u beside and over the parts whose products are done; w | p, later the state's
  // increment; u, later P u; dot products of the next chunk
  static constexpr uint32_t A1 = 0, A2 = 128, A3 = 0, A4 = F32 ? 96 : 192, D1 = 256, D3 = 256, D2 = 384, D4 = 384, D0 = 448;
};

// Byte offset of element (row, k) of an operand with `kdim` columns along which it is contiguous: cores of 8 rows x 16 bytes, those along
// the columns 128 bytes apart. The same bytes serve products over the rows.
__host__ __device__ constexpr uint32_t core_at(int row, int k, int kdim) {
  return (uint32_t)((row >> 3) * (kdim >> 3) * 128 + (k >> 3) * 128 + (row & 7) * 16 + (k & 7) * 2);
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ void less(float &x, float &y, uint32_t part) {        // (both differences in one instruction)
  uint64_t d;
  asm("{\n\t.reg .b64 a, b, m;\n\tmov.b64 a, {%1, %2};\n\tmov.b64 b, {%3, %4};\n\tmov.b64 m, {%5, %5};\n\tfma.rn.f32x2 %0, b, m, a;\n\t}"
      : "=l"(d)
      : "f"(x), "f"(y), "r"(part << 16), "r"(part & 0xFFFF0000u), "f"(-1.0f));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(d));
}
// NP bf16 parts of two values.
template <int NP>
__device__ __forceinline__ void split(float x, float y, uint32_t *part, int stride) {
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    part[i * stride] = pack2(x, y);
    if (i + 1 < NP) less(x, y, part[i * stride]);
  }
}
__device__ __forceinline__ void cp16(uint32_t dst, const void *src, uint32_t bytes) {      // (0: writes zeros)
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void aux_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
__host__ __device__ constexpr uint32_t idesc(int N, int mn_major) {   // M = 128, bf16, fp32 sums
  return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)mn_major << 16) | ((uint32_t)(N >> 3) << 17) | (8u << 24);
}
__device__ __forceinline__ uint32_t idesc_n(int N) { return idesc(0, 0) | ((uint32_t)(N >> 3) << 17); }

constexpr uint64_t WAIT_NS = 1000000000ull;

// y += m x for a pair of rows.
__device__ __forceinline__ void fma_pair(uint64_t &y, uint64_t m, float x) {
  asm("{\n\t.reg .b64 v;\n\tmov.b64 v, {%2, %2};\n\tfma.rn.f32x2 %0, %1, v, %0;\n\t}" : "+l"(y) : "l"(m), "f"(x));
}
__device__ __forceinline__ float2 pair(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}

template <int D, bool F32>
__global__ void __launch_bounds__(Shape<D, F32>::THREADS, 1) delta_chunk_kernel(const DeltaArgs p) {
  using Z = Shape<D, F32>;
  constexpr int NX = Z::NX, NO = Z::NO, NB = Z::NB, LD = Z::LD, LY = Z::LY, ES = F32 ? 4 : 2;
  extern __shared__ __align__(128) char smem[];
  uint64_t *bar = reinterpret_cast<uint64_t *>(smem + Z::OBAR);
  uint64_t *x_full = bar, *x_free = x_full + NB, *gates = x_free + NB, *a1 = gates + 3, *a2 = a1 + 1, *a3 = a2 + 1, *a4 = a3 + 1, *w_done = a4 + 1,
           *p_done = w_done + 1, *u_done = p_done + 1, *s_done = u_done + 1, *o_done = s_done + 1, *g_done = o_done + 1, *t_ready = g_done + 1,
           *p_ready = t_ready + 1, *drain = p_ready + 1;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + Z::OMISC);
  Seq *seq_slot = reinterpret_cast<Seq *>(tmem_slot + 1);
  static_assert(sizeof(Seq) <= 12, "kept beside the TMEM address");
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const int b = blockIdx.x / p.H, h = blockIdx.x - b * p.H, hk = h / p.group;
  const bool out = p.o.p != nullptr;

  if (warp == Z::W_MMA) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  if (tid == 0) {
    for (int i = 0; i < NB; ++i) mbar_init(&x_full[i], Z::LOAD), mbar_init(&x_free[i], 1);
    for (int i = 0; i < 3; ++i) mbar_init(&gates[i], Z::AUX);
    for (uint64_t *x : {a1, a2, a3, a4}) mbar_init(x, Z::MAIN);
    for (uint64_t *x : {w_done, p_done, u_done, s_done, o_done, g_done, drain}) mbar_init(x, 1);
    mbar_init(t_ready, Z::AUX), mbar_init(p_ready, Z::AUX);
    mbar_fence_init();
  }
  pdl_enter();
  if (warp == 0) {
    const Seq s = sequence(p, b, h == 0);
    if (lane == 0) *seq_slot = s;
  }
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const Seq s = *seq_slot;
  const int n = s.n, chunks = (n + C - 1) / C;
  constexpr uint32_t tmem = 0;          // the whole of TMEM is this block's: its first column (a constant keeps addresses uniform)
  float *state = p.S + ((long)s.slot * p.H + h) * D * D;
  // tokens of a chunk, and as the products count them
  auto tokens = [&](int c) { return min(C, n - c * C); };
  auto padded = [&](int c) { return (tokens(c) + 15) & ~15; };

  bool good = true;
  auto wait = [&](uint64_t *x, int phase) {              // (the whole warp)
    if (!good) return;
    if (__all_sync(0xffffffffu, mbar_try_wait(x, phase & 1))) return;
    good = __all_sync(0xffffffffu, mbar_wait(x, phase & 1, WAIT_NS));
  };
  auto arrive = [&](uint64_t *x) {
    __syncwarp();
    if (lane == 0) mbar_arrive(x);
  };

  if (warp < Z::MAIN) {
    // ---------------------------------------------------------------- columns
    const int grp = warp >> 2, j = (warp & 3) * 32 + lane;
    const uint32_t tl = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const bool on = (warp & 3) * 32 < D;                 // (heads of 64 leave half of the lanes alone)
    constexpr int HALF = D / 2;                          // rows of the state that the thread holds: HALF grp ..
    float S[HALF];
#pragma unroll
    for (int i = 0; i < HALF; ++i) S[i] = on && n > 0 && !s.fresh ? state[(long)(grp * HALF + i) * D + j] : 0.0f;
    auto publish = [&]() {                               // the state's parts, as the first operand of D1
      if (on) {
#pragma unroll
        for (int i = 0; i < HALF; i += 16) {
          uint32_t x[3][8];
#pragma unroll
          for (int e = 0; e < 8; ++e) split<3>(S[i + 2 * e], S[i + 2 * e + 1], &x[0][e], 8);
#pragma unroll
          for (int k = 0; k < 3; ++k) tmem_st8(tl + Z::A1 + k * (D / 2) + grp * (HALF / 2) + i / 2, x[k]);
        }
        tmem_wait_st();
      }
      fence_before_sync();
      arrive(a1);
    };
    if (chunks) publish();
    for (int c = 0; c < chunks; ++c) {
      const int nt = tokens(c), np = padded(c), buf = c % NB;
      const float *ga = reinterpret_cast<const float *>(smem + Z::OG) + (c % 3) * 4 * C;
      const float4 *beta = reinterpret_cast<const float4 *>(ga + C), *G = reinterpret_cast<const float4 *>(ga + 2 * C),
                   *rho = reinterpret_cast<const float4 *>(ga + 3 * C);
      const char *vrow = smem + Z::OV + buf * Z::VBUF + j * ES;
      // ---- rhs = beta (v - G w)
      wait(&gates[c % 3], c / 3);
      wait(&x_full[buf], c / NB);
      wait(w_done, c);
      if (F32 && out) wait(p_done, c);                   // (rhs lies over a part of S that q's products read)
      fence_after_sync();
      if (on) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int t0 = 16 * (grp + 2 * r);
          if (t0 < np) {
            uint32_t w[16], x[3][8];
            tmem_ld16(tl + Z::D1 + t0, w);
            float v[16];
            const char *at = vrow + t0 * D * ES;
#pragma unroll
            for (int e = 0; e < 16; ++e)
              v[e] = F32 ? *reinterpret_cast<const float *>(at + e * D * ES)
                         : __uint_as_float((uint32_t)*reinterpret_cast<const uint16_t *>(at + e * D * ES) << 16);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; e += 4) {
              const float4 g = G[(t0 + e) / 4], be = beta[(t0 + e) / 4];
              const float y0 = be.x * fmaf(-g.x, __uint_as_float(w[e]), v[e]), y1 = be.y * fmaf(-g.y, __uint_as_float(w[e + 1]), v[e + 1]);
              const float y2 = be.z * fmaf(-g.z, __uint_as_float(w[e + 2]), v[e + 2]), y3 = be.w * fmaf(-g.w, __uint_as_float(w[e + 3]), v[e + 3]);
              split<3>(y0, y1, &x[0][e / 2], 8);
              split<3>(y2, y3, &x[0][e / 2 + 1], 8);
            }
#pragma unroll
            for (int k = 0; k < 3; ++k) tmem_st8(tl + Z::A2 + k * (C / 2) + t0 / 2, x[k]);
          }
        }
        tmem_wait_st();
      }
      fence_before_sync();
      arrive(a2);
      // ---- G p, kept for the outputs
      float y[2][16];
      if (out) {
        wait(p_done, c);
        fence_after_sync();
        if (on) {
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const int t0 = 16 * (grp + 2 * r);
            if (t0 < np) {
              uint32_t x[16];
              tmem_ld16(tl + Z::D1 + C + t0, x);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; e += 4) {
                const float4 g = G[(t0 + e) / 4];
                y[r][e] = g.x * __uint_as_float(x[e]), y[r][e + 1] = g.y * __uint_as_float(x[e + 1]);
                y[r][e + 2] = g.z * __uint_as_float(x[e + 2]), y[r][e + 3] = g.w * __uint_as_float(x[e + 3]);
              }
            }
          }
        }
      }
      const float gC = G[C / 4 - 1].w;
      // ---- u, decayed to the chunk's end, and as it is
      wait(u_done, c);
      fence_after_sync();
      if (p.write) {
        if (on) {
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const int t0 = 16 * (grp + 2 * r);
            if (t0 < np) {
              uint32_t u[16], x[3][8];
              tmem_ld16(tl + Z::D2 + t0, u);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; e += 4) {
                const float4 g = rho[(t0 + e) / 4];
                split<3>(g.x * __uint_as_float(u[e]), g.y * __uint_as_float(u[e + 1]), &x[0][e / 2], 8);
                split<3>(g.z * __uint_as_float(u[e + 2]), g.w * __uint_as_float(u[e + 3]), &x[0][e / 2 + 1], 8);
              }
#pragma unroll
              for (int k = 0; k < 3; ++k) tmem_st8(tl + Z::A3 + k * (C / 2) + t0 / 2, x[k]);
            }
          }
          tmem_wait_st();
        }
        fence_before_sync();
        arrive(a3);
      }
      if (out) {
        if (on) {
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const int t0 = 16 * (grp + 2 * r);
            if (t0 < np) {
              uint32_t u[16], x[NO][8];
              tmem_ld16(tl + Z::D2 + t0, u);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 8; ++e) split<NO>(__uint_as_float(u[2 * e]), __uint_as_float(u[2 * e + 1]), &x[0][e], 8);
#pragma unroll
              for (int k = 0; k < NO; ++k) tmem_st8(tl + Z::A4 + k * (C / 2) + t0 / 2, x[k]);
            }
          }
          tmem_wait_st();
        }
        fence_before_sync();
        arrive(a4);
      }
      // ---- the state at the chunk's end
      if (p.write) {
        wait(s_done, c);
        fence_after_sync();
        if (on) {
#pragma unroll
          for (int i = 0; i < HALF; i += 16) {
            uint32_t x[16];
            tmem_ld16(tl + Z::D3 + grp * HALF + i, x);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) S[i + e] = fmaf(gC, S[i + e], __uint_as_float(x[e]));
          }
        }
        if (c + 1 < chunks) {
          if (F32 && out) wait(o_done, c);               // (u lies over parts of S)
          publish();
        }
      }
      // ---- outputs
      if (out) {
        wait(o_done, c);
        fence_after_sync();
        if (on) {
          const long st = p.o.st * ES;
          char *row = p.o.p + (b * p.o.sb + (long)(c * C) * p.o.st + h * p.o.sh + j) * ES;
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const int t0 = 16 * (grp + 2 * r);
            if (t0 < np) {
              uint32_t x[16];
              tmem_ld16(tl + Z::D4 + t0, x);
              tmem_wait_ld();
              char *at = row + t0 * st;
              auto put = [&](int e) {
                const float o = y[r][e] + __uint_as_float(x[e]);
                if (F32) *reinterpret_cast<float *>(at) = o;
                else *reinterpret_cast<__nv_bfloat16 *>(at) = __float2bfloat16_rn(o);
                at += st;
              };
              if (t0 + 16 <= nt) {
#pragma unroll
                for (int e = 0; e < 16; ++e) put(e);
              } else {
#pragma unroll
                for (int e = 0; e < 16; ++e)
                  if (t0 + e < nt) put(e);
              }
            }
          }
        }
        fence_before_sync();
      }
    }
    if (p.write && n > 0 && on && good) {
#pragma unroll
      for (int i = 0; i < HALF; ++i) state[(long)(grp * HALF + i) * D + j] = S[i];
    }
    if (out) {                                           // rows past the sequence's tokens
      constexpr int PIECES = D * ES / 16;
      for (long i = tid; i < (long)(p.n_tokens - n) * PIECES; i += Z::MAIN * 32)
        *reinterpret_cast<uint4 *>(p.o.p + (b * p.o.sb + (n + i / PIECES) * p.o.st + h * p.o.sh) * ES + i % PIECES * 16) = make_uint4(0, 0, 0, 0);
    }
  } else if (warp < Z::W_MMA) {
    // ---------------------------------------------------------------- tables of the chunks
    const int at = tid - Z::MAIN * 32, aw = warp - Z::MAIN, t = at & 63;
    const bool isq = at >= 64;                           // rows of k (M, T), then of q (P)
    float *M = reinterpret_cast<float *>(smem + Z::OM), *Tf = reinterpret_cast<float *>(smem + Z::OTF), *Y = reinterpret_cast<float *>(smem + Z::OY);
    const int words = (p.n_tokens + 31) >> 5;
    float a_next = 1.0f, b_next = 0.0f;                  // gates of the next chunk (threads 0..63)
    auto fetch = [&](int c) {
      a_next = 1.0f, b_next = 0.0f;
      if (!isq && c < chunks && t < tokens(c)) {
        const long row = row_of(p, b, c * C + t);
        a_next = reinterpret_cast<const float *>(p.a.p)[b * p.a.sb + row * p.a.st + h * p.a.sh];
        b_next = reinterpret_cast<const float *>(p.beta.p)[b * p.beta.sb + row * p.beta.st + h * p.beta.sh];
      }
    };
    for (int i = at; i < C * LD; i += 128) Tf[i] = 0.0f; // (the upper triangle stays so)
    fetch(0);
    for (int c = 0; c < chunks; ++c) {
      const int nt = tokens(c), np = padded(c);
      // ---- decays: a row of R, from its end
      float *ga = reinterpret_cast<float *>(smem + Z::OG) + (c % 3) * 4 * C, *beta = ga + C, *G = ga + 2 * C, *rho = ga + 3 * C;
      if (!isq) ga[t] = a_next, beta[t] = b_next;
      fetch(c + 1);
      uint32_t see[2] = {~0u, ~0u};                      // the token and its ancestors
      if (p.mask) {
        see[0] = see[1] = 0;
        if (t < nt) {
          const uint32_t *row = p.mask + ((long)b * p.n_tokens + t) * words;
          see[0] = row[0];
          if (words > 1) see[1] = row[1];
        }
      }
      if (t < 32) see[0] = (see[0] | 1u << t) & (2u << t) - 1, see[1] = 0;
      else see[1] = (see[1] | 1u << (t - 32)) & (2u << (t - 32)) - 1;
      aux_sync();
      float R[C];
      float r = isq ? 1.0f : beta[t];                    // (rows of M carry beta)
#pragma unroll
      for (int i = C - 4; i >= 0; i -= 4) {
        const float4 a = *reinterpret_cast<const float4 *>(ga + i);
        const float as[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int e = 3; e >= 0; --e) {
          const bool anc = see[(i + e) >> 5] & (1u << ((i + e) & 31));
          R[i + e] = anc ? r : 0.0f;
          r *= anc ? as[e] : 1.0f;
        }
      }
      if (isq) G[t] = r;
      if (at == 2 * C - 1) {
#pragma unroll
        for (int i = 0; i < C; i += 4) *reinterpret_cast<float4 *>(rho + i) = make_float4(R[i], R[i + 1], R[i + 2], R[i + 3]);
      }
      arrive(&gates[c % 3]);
      // ---- M, a column's entries in a row (entries on and above the diagonal are not read, or are zeros), and P
      wait(g_done, c);
      fence_after_sync();
      const uint32_t tl = tmem + ((uint32_t)(aw * 32) << 16) + Z::D0;
#pragma unroll
      for (int i0 = 0; i0 < C; i0 += 16) {
        uint32_t x[16];
        if (i0 < np) {
          tmem_ld16(tl + i0, x);
          tmem_wait_ld();
        } else {
#pragma unroll
          for (int e = 0; e < 16; ++e) x[e] = 0;
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) R[i0 + e] *= __uint_as_float(x[e]);
        if (!isq) {
#pragma unroll
          for (int e = 0; e < 16; ++e) M[(i0 + e) * LD + t] = R[i0 + e];
        }
      }
      fence_before_sync();
      aux_sync();
      // ---- T = (I + M)^-1: blocks of 16 on the diagonal (a lane a column, the column's later entries brought up to date as each is known);
      // then twice the block below two inverses, -T_b M_ba T_a. T_b is read by columns: it takes M's place.
      {
        const int o16 = 16 * aw, col = lane & 15;
        const float *m = M + o16 * LD + o16;
        float x[16];
        float4 row[4], next[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) next[k] = *reinterpret_cast<const float4 *>(m + 4 * k);
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = i == col ? 1.0f : 0.0f;
#pragma unroll
        for (int i = 0; i < 15; ++i) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            row[k] = next[k];
            if (i < 14 && 4 * k + 3 > i + 1) next[k] = *reinterpret_cast<const float4 *>(m + (i + 1) * LD + 4 * k);
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (4 * k > i) x[4 * k] = fmaf(-row[k].x, x[i], x[4 * k]);
            if (4 * k + 1 > i) x[4 * k + 1] = fmaf(-row[k].y, x[i], x[4 * k + 1]);
            if (4 * k + 2 > i) x[4 * k + 2] = fmaf(-row[k].z, x[i], x[4 * k + 2]);
            if (4 * k + 3 > i) x[4 * k + 3] = fmaf(-row[k].w, x[i], x[4 * k + 3]);
          }
        }
        __syncwarp();
        if (lane < 16) {
#pragma unroll
          for (int i = 0; i < 16; ++i) Tf[(o16 + i) * LD + o16 + col] = x[i];
#pragma unroll
          for (int i = 0; i < 16; i += 4)
            *reinterpret_cast<float4 *>(M + (o16 + col) * LD + o16 + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
        }
      }
      aux_sync();
      // rows 4 q .. of a 16 x 16 or 8 q .. of a 32 x 32 block: sum_s first(s, rows) second(s), over pairs of rows
      if (np > 16) {
        const int oa = (aw >> 1) * 32, ob = oa + 16, col = lane & 15, q = 4 * ((aw & 1) * 2 + (lane >> 4));
        float *y = Y + (aw >> 1) * 16 * LY;
        uint64_t s0 = 0, s1 = 0;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const ulonglong2 m = *reinterpret_cast<const ulonglong2 *>(M + (oa + i) * LD + ob + q);
          const float x = Tf[(oa + i) * LD + oa + col];
          fma_pair(s0, m.x, x), fma_pair(s1, m.y, x);
        }
        float2 v0 = pair(s0), v1 = pair(s1);
        y[q * LY + col] = -v0.x, y[(q + 1) * LY + col] = -v0.y, y[(q + 2) * LY + col] = -v1.x, y[(q + 3) * LY + col] = -v1.y;
        aux_sync();
        s0 = s1 = 0;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const ulonglong2 m = *reinterpret_cast<const ulonglong2 *>(M + (ob + i) * LD + ob + q);
          const float x = y[i * LY + col];
          fma_pair(s0, m.x, x), fma_pair(s1, m.y, x);
        }
        v0 = pair(s0), v1 = pair(s1);
        float *to = Tf + (ob + q) * LD + oa + col;
        to[0] = v0.x, to[LD] = v0.y, to[2 * LD] = v1.x, to[3 * LD] = v1.y;
        *reinterpret_cast<float4 *>(M + (oa + col) * LD + ob + q) = make_float4(v0.x, v0.y, v1.x, v1.y);
        aux_sync();
      }
      if (np > 32) {
        const int q = 8 * aw;
        uint64_t s[4] = {0, 0, 0, 0};
        auto add = [&](const float *m, float x) {
          const ulonglong2 m0 = *reinterpret_cast<const ulonglong2 *>(m), m1 = *reinterpret_cast<const ulonglong2 *>(m + 4);
          fma_pair(s[0], m0.x, x), fma_pair(s[1], m0.y, x), fma_pair(s[2], m1.x, x), fma_pair(s[3], m1.y, x);
        };
#pragma unroll 16
        for (int i = 0; i < 32; ++i) add(M + i * LD + 32 + q, Tf[i * LD + lane]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 v = pair(s[i]);
          Y[(q + 2 * i) * LY + lane] = -v.x, Y[(q + 2 * i + 1) * LY + lane] = -v.y;
          s[i] = 0;
        }
        aux_sync();
#pragma unroll 16
        for (int i = 0; i < 32; ++i) add(M + (32 + i) * LD + 32 + q, Y[i * LY + lane]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 v = pair(s[i]);
          Tf[(32 + q + 2 * i) * LD + lane] = v.x, Tf[(33 + q + 2 * i) * LD + lane] = v.y;
        }
        aux_sync();
      }
      if (c) wait(u_done, c - 1);
#pragma unroll
      for (int k = 0; k < 32; k += 8) {
        const int i = (at >> 6) * 32 + k;
        const float4 x = *reinterpret_cast<const float4 *>(Tf + t * LD + i), y = *reinterpret_cast<const float4 *>(Tf + t * LD + i + 4);
        uint32_t w[3][4];
        split<3>(x.x, x.y, &w[0][0], 4), split<3>(x.z, x.w, &w[0][1], 4), split<3>(y.x, y.y, &w[0][2], 4), split<3>(y.z, y.w, &w[0][3], 4);
#pragma unroll
        for (int e = 0; e < 3; ++e)
          *reinterpret_cast<uint4 *>(smem + Z::OT + e * Z::TPART + core_at(t, i, C)) = make_uint4(w[e][0], w[e][1], w[e][2], w[e][3]);
      }
      fence_smem_to_async();
      arrive(t_ready);
      if (out) {
        if (c) wait(o_done, c - 1);
        if (isq) {
#pragma unroll
          for (int i = 0; i < C; i += 8) {
            uint32_t w[NO][4];
#pragma unroll
            for (int e = 0; e < 4; ++e) split<NO>(R[i + 2 * e], R[i + 2 * e + 1], &w[0][e], 4);
#pragma unroll
            for (int e = 0; e < NO; ++e)
              *reinterpret_cast<uint4 *>(smem + Z::OP + e * Z::TPART + core_at(t, i, C)) = make_uint4(w[e][0], w[e][1], w[e][2], w[e][3]);
          }
        }
        fence_smem_to_async();
        arrive(p_ready);
      }
    }
  } else if (warp >= Z::W_LOAD) {
    // ---------------------------------------------------------------- rows of the chunks: one warp k, one q, one v
    const int what = warp - Z::W_LOAD;
    const KvTensor &src = what == 0 ? p.k : what == 1 ? p.q : p.v;
    const char *base = src.p + (b * src.sb + (what == 2 ? h : hk) * src.sh) * ES;
    const long st = src.st * ES;
    constexpr int PIECES = D * ES / 16, PER = 32 / PIECES > 0 ? 32 / PIECES : 1;   // of a row of v; rows a warp copies at once
    auto load = [&](int c) {
      const int nt = tokens(c);
      if (what < 2) {
        // eight lanes write one core of 8 rows
        const int k = (lane >> 3) * 8;
        const uint32_t to = smem_u32(smem) + Z::OX + (c % NB) * Z::XBUF + what * Z::ROWS + core_at(lane & 7, k, D);
        const char *from = base + (long)(c * C + (lane & 7)) * st + k * ES;
#pragma unroll
        for (int r0 = 0; r0 < C; r0 += 8, from += 8 * st) {
          const int r = r0 + (lane & 7);
          const bool live = r < nt;
          const char *at = from;
          if (p.idx) at = base + (live ? row_of(p, b, c * C + r) : 0) * st + k * ES;
          if (!live) at = src.p;
#pragma unroll
          for (int g = 0; g < D / 32; ++g) {
            const uint32_t dst = to + core_at(r0, g * 32, D);
            if (!F32) {
              cp16(dst, at + (live ? g * 32 * ES : 0), live ? 16 : 0);
            } else {
              float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f), y = x;
              if (live) x = reinterpret_cast<const float4 *>(at + g * 32 * ES)[0], y = reinterpret_cast<const float4 *>(at + g * 32 * ES)[1];
              uint32_t w[3][4];
              split<3>(x.x, x.y, &w[0][0], 4), split<3>(x.z, x.w, &w[0][1], 4), split<3>(y.x, y.y, &w[0][2], 4), split<3>(y.z, y.w, &w[0][3], 4);
#pragma unroll
              for (int i = 0; i < NX; ++i)
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst + i * Z::XPART), "r"(w[i][0]), "r"(w[i][1]), "r"(w[i][2]), "r"(w[i][3])
                             : "memory");
            }
          }
        }
      } else {
        const int piece = lane % PIECES, first = lane / PIECES;
        const uint32_t to = smem_u32(smem) + Z::OV + (c % NB) * Z::VBUF + first * D * ES + piece * 16;
        const char *from = base + (long)(c * C + first) * st + piece * 16;
#pragma unroll 8
        for (int r0 = 0; r0 < C; r0 += PER, from += PER * st) {
          const int r = r0 + first;
          const bool live = r < nt;
          const char *at = from;
          if (p.idx) at = base + (live ? row_of(p, b, c * C + r) : 0) * st + piece * 16;
          cp16(to + r0 * D * ES, live ? at : src.p, live ? 16 : 0);
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    static_assert(PIECES <= 32 && C % PER == 0, "v rows");
    const bool any = what != 1 || out;
    // a chunk's rows are announced behind the next one's copies
    for (int c = 0; c < chunks + (NB > 1); ++c) {
      if (c < chunks) {
        if (c >= NB) wait(&x_free[c % NB], c / NB - 1);  // (also without rows to copy: an early arrival would count for the chunk before)
        if (any) load(c);
      }
      if (NB > 1 && c < chunks) asm volatile("cp.async.wait_group 1;" ::: "memory");
      else asm volatile("cp.async.wait_group 0;" ::: "memory");
      fence_smem_to_async();
      if (NB == 1) arrive(&x_full[0]);
      else if (c > 0) arrive(&x_full[(c - 1) % NB]);
    }
  } else {
    // ---------------------------------------------------------------- products. The warp runs as one, so that descriptors stay in uniform
    // registers; one lane issues.
    uint32_t leader;
    asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(leader));
    const uint32_t base = smem_u32(smem);
    constexpr uint32_t SBO = (D / 8) * 128;
    // D (+)= A B^T summed over part pairs i + j <= MOST, smallest first; `one` issues a pair (the first of all clears D)
    auto pairs = [&](auto na, auto nb, auto most, auto one) {
#pragma unroll
      for (int sum = decltype(most)::value; sum >= 0; --sum)
#pragma unroll
        for (int i = 0; i < decltype(na)::value; ++i) {
          const int k = sum - i;
          if (k < 0 || k >= decltype(nb)::value) continue;
          const int top = decltype(most)::value, last = decltype(nb)::value - 1;
          one(i, k, sum == (top < last + decltype(na)::value - 1 ? top : last + decltype(na)::value - 1) && (i == 0 || k == last));
        }
    };
    using I2 = std::integral_constant<int, 2>;
    using I3 = std::integral_constant<int, 3>;
    using INX = std::integral_constant<int, NX>;
    using INO = std::integral_constant<int, NO>;
    using IMX = std::integral_constant<int, F32 ? 2 : 0>;
    using IMO = std::integral_constant<int, NO - 1>;
    const uint64_t x_row = smem_desc(base + Z::OX, 128, SBO), x_col = smem_desc(base + Z::OX, SBO, 128);   // rows, and along their other dimension
    const uint64_t t_row = smem_desc(base + Z::OT, 128, 1024), p_row = smem_desc(base + Z::OP, 128, 1024);
    constexpr uint32_t XB = Z::XBUF >> 4, XP = Z::XPART >> 4, TP = Z::TPART >> 4;
    auto dots = [&](int c) {                             // [k | q] k^T
      wait(&x_full[c % NB], c / NB);
      fence_after_sync();
      if (leader && good) {
        const uint32_t id = idesc_n(padded(c));
        const uint64_t x = x_row + (c % NB) * XB;
        pairs(INX{}, INX{}, IMX{}, [&](int i, int k, bool first) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) mma_ss(tmem + Z::D0, x + i * XP + kk * 16, x + k * XP + kk * 16, id, first && kk == 0 ? 0u : 1u);
        });
        commit(g_done);
      }
    };
    if (chunks) dots(0);
    for (int c = 0; c < chunks; ++c) {
      const int np = padded(c), steps = np / 16;
      const uint32_t id = idesc_n(np);
      const uint64_t x = x_row + (c % NB) * XB;
      wait(a1, c);
      fence_after_sync();
      if (leader && good) {
        pairs(I3{}, INX{}, I2{}, [&](int i, int k, bool first) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) mma_ts(tmem + Z::D1, tmem + Z::A1 + i * (D / 2) + 8 * kk, x + k * XP + kk * 16, id, first && kk == 0 ? 0u : 1u);
        });
        commit(w_done);
        if (out) {
          pairs(I3{}, INX{}, IMO{}, [&](int i, int k, bool first) {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              mma_ts(tmem + Z::D1 + C, tmem + Z::A1 + i * (D / 2) + 8 * kk, x + k * XP + (Z::ROWS >> 4) + kk * 16, id, first && kk == 0 ? 0u : 1u);
          });
          commit(p_done);
        }
      }
      wait(t_ready, c);
      wait(a2, c);
      fence_after_sync();
      // (columns t of step kk's tokens s >= 16 kk begin at t = 16 kk)
      if (leader && good) {
        pairs(I3{}, I3{}, I2{}, [&](int i, int k, bool first) {
#pragma unroll
          for (int kk = 0; kk < C / 16; ++kk)
            if (kk < steps)
              mma_ts(tmem + Z::D2 + 16 * kk, tmem + Z::A2 + i * (C / 2) + 8 * kk, t_row + k * TP + kk * ((2 * 1024 + 256) >> 4), id - kk * (2u << 17),
                     first && kk == 0 ? 0u : 1u);
        });
        commit(u_done);
      }
      if (NB > 1 && c + 1 < chunks) dots(c + 1);
      if (p.write) {
        wait(a3, c);
        fence_after_sync();
        if (leader && good) {
          const uint64_t xc = x_col + (c % NB) * XB;
          pairs(I3{}, INX{}, I2{}, [&](int i, int k, bool first) {
#pragma unroll
            for (int kk = 0; kk < C / 16; ++kk)
              if (kk < steps)
                mma_ts(tmem + Z::D3, tmem + Z::A3 + i * (C / 2) + 8 * kk, xc + k * XP + kk * (2 * SBO >> 4), idesc(D, 1), first && kk == 0 ? 0u : 1u);
          });
          commit(s_done);
          commit(&x_free[c % NB]);
        }
      }
      if (out) {
        wait(a4, c);
        wait(p_ready, c);
        fence_after_sync();
        if (leader && good) {
          pairs(INO{}, INO{}, IMO{}, [&](int i, int k, bool first) {
#pragma unroll
            for (int kk = 0; kk < C / 16; ++kk)
              if (kk < steps)
                mma_ts(tmem + Z::D4 + 16 * kk, tmem + Z::A4 + i * (C / 2) + 8 * kk, p_row + k * TP + kk * ((2 * 1024 + 256) >> 4), id - kk * (2u << 17),
                       first && kk == 0 ? 0u : 1u);
          });
          commit(o_done);
        }
      }
      if (NB == 1 && c + 1 < chunks) dots(c + 1);
    }
    if (leader) commit(drain);                           // every product has ended before the block frees its TMEM
    mbar_wait(drain, 0, WAIT_NS);
    __syncwarp();
  }
  if (!good && lane == 0) atomicOr(p.status, PACE_DELTA_TIMEOUT);
  fence_before_sync();
  __syncthreads();
  if (warp == Z::W_MMA) tmem_dealloc(*tmem_slot, 512);
}

template <int D, bool F32>
cudaError_t launch_chunk(const DeltaArgs &p, cudaStream_t s) {
  using Z = Shape<D, F32>;
  const cudaError_t e = smem_opt_in<delta_chunk_kernel<D, F32>>(Z::SMEM);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg = pdl_config(dim3((unsigned)(p.batch * p.H)), dim3(Z::THREADS), Z::SMEM, s, attr);
  return cudaLaunchKernelEx(&cfg, delta_chunk_kernel<D, F32>, p);
}

}  // namespace delta
}  // namespace pace
