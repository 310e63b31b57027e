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
// Roles: eight warps own the columns (two a quarter of TMEM's lanes: token blocks of 16 in turn, halves of the state's rows), four copy a
// chunk's rows in, form R, M, P and T one chunk ahead, one issues the products. T by halves: two 32 x 32 inverses (a thread a
// column, right-looking, so that a token's chain is one multiply-add), then -T22 M21 T11.
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
  static constexpr int MAIN = 8, AUX = 4, W_MMA = MAIN + AUX, THREADS = (W_MMA + 1) * 32;
  static constexpr int NX = F32 ? 3 : 1;                 // parts of q and k
  static constexpr int NO = F32 ? 3 : 2;                 // parts of u and P in the outputs
  static constexpr int NB = F32 ? 1 : 3;                 // chunks of rows in shared memory
  static constexpr int ROWS = C * D * 2;                 // one part of 64 rows
  static constexpr int XPART = 2 * ROWS, XBUF = NX * XPART;
  static constexpr int VBUF = C * D * (F32 ? 4 : 2);
  static constexpr int TPART = C * C * 2;
  static constexpr int LD = C + 4;                       // row of the fp32 tables
  static constexpr int OX = 0, OV = OX + NB * XBUF, OT = OV + NB * VBUF, OP = OT + 3 * TPART, OM = OP + NO * TPART,
                       OTF = OM + C * LD * 4, OY = OTF + C * LD * 4, OG = OY + 32 * 36 * 4, OBAR = OG + 3 * 4 * C * 4,
                       NBAR = 3 * NB + 3 + 14, OMISC = OBAR + NBAR * 8, SMEM = OMISC + 16;
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
// Three bf16 parts of two values.
__device__ __forceinline__ void split3(float x, float y, uint32_t &hi, uint32_t &mid, uint32_t &lo) {
  hi = pack2(x, y);
  x -= __uint_as_float(hi << 16), y -= __uint_as_float(hi & 0xFFFF0000u);
  mid = pack2(x, y);
  x -= __uint_as_float(mid << 16), y -= __uint_as_float(mid & 0xFFFF0000u);
  lo = pack2(x, y);
}
__device__ __forceinline__ void cp16(void *dst, const void *src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ void aux_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
__host__ __device__ constexpr uint32_t idesc(int N, int mn_major) {   // M = 128, bf16, fp32 sums
  return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)mn_major << 16) | ((uint32_t)(N >> 3) << 17) | (8u << 24);
}
__device__ __forceinline__ uint32_t idesc_n(int N) { return idesc(0, 0) | ((uint32_t)(N >> 3) << 17); }

constexpr uint64_t WAIT_NS = 1000000000ull;

template <int D, bool F32>
__global__ void __launch_bounds__(Shape<D, F32>::THREADS, 1) delta_chunk_kernel(const DeltaArgs p) {
  using Z = Shape<D, F32>;
  constexpr int NX = Z::NX, NO = Z::NO, NB = Z::NB, LD = Z::LD, ES = F32 ? 4 : 2;
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
    for (int i = 0; i < NB; ++i) mbar_init(&x_full[i], Z::AUX), mbar_init(&x_free[i], 1);
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
  const uint32_t tmem = *tmem_slot;
  float *state = p.S + ((long)s.slot * p.H + h) * D * D;
  // tokens of a chunk, and as the products count them
  auto tokens = [&](int c) { return min(C, n - c * C); };
  auto padded = [&](int c) { return (tokens(c) + 15) & ~15; };

  bool good = true;
  auto wait = [&](uint64_t *x, int phase) {              // (the whole warp)
    if (good && !mbar_wait(x, phase & 1, WAIT_NS)) good = false;
    good = __all_sync(0xffffffffu, good);
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
          for (int e = 0; e < 8; ++e) split3(S[i + 2 * e], S[i + 2 * e + 1], x[0][e], x[1][e], x[2][e]);
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
      const float *ga = reinterpret_cast<const float *>(smem + Z::OG) + (c % 3) * 4 * C, *beta = ga + C, *G = ga + 2 * C, *rho = ga + 3 * C;
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
            tmem_wait_ld();
            float y[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const char *at = vrow + (t0 + e) * D * ES;
              const float v = F32 ? *reinterpret_cast<const float *>(at) : __uint_as_float((uint32_t)*reinterpret_cast<const uint16_t *>(at) << 16);
              y[e] = beta[t0 + e] * fmaf(-G[t0 + e], __uint_as_float(w[e]), v);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) split3(y[2 * e], y[2 * e + 1], x[0][e], x[1][e], x[2][e]);
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
              for (int e = 0; e < 16; ++e) y[r][e] = G[t0 + e] * __uint_as_float(x[e]);
            }
          }
        }
      }
      // ---- u, decayed to the chunk's end, and as it is
      wait(u_done, c);
      fence_after_sync();
      const float gC = G[C - 1];
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
              for (int e = 0; e < 8; ++e)
                split3(rho[t0 + 2 * e] * __uint_as_float(u[2 * e]), rho[t0 + 2 * e + 1] * __uint_as_float(u[2 * e + 1]), x[0][e], x[1][e], x[2][e]);
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
              uint32_t u[16], x[3][8];
              tmem_ld16(tl + Z::D2 + t0, u);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 8; ++e) split3(__uint_as_float(u[2 * e]), __uint_as_float(u[2 * e + 1]), x[0][e], x[1][e], x[2][e]);
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
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const int t0 = 16 * (grp + 2 * r);
            if (t0 < np) {
              uint32_t x[16];
              tmem_ld16(tl + Z::D4 + t0, x);
              tmem_wait_ld();
              char *at = p.o.p + (b * p.o.sb + (long)(c * C + t0) * p.o.st + h * p.o.sh + j) * ES;
#pragma unroll
              for (int e = 0; e < 16; ++e, at += p.o.st * ES) {
                const float o = y[r][e] + __uint_as_float(x[e]);
                if (t0 + e < nt) {
                  if (F32) *reinterpret_cast<float *>(at) = o;
                  else *reinterpret_cast<__nv_bfloat16 *>(at) = __float2bfloat16_rn(o);
                }
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
    // ---------------------------------------------------------------- rows and tables of the chunks
    const int at = tid - Z::MAIN * 32, aw = warp - Z::MAIN, t = at & 63;
    const bool isq = at >= 64;
    float *M = reinterpret_cast<float *>(smem + Z::OM), *Tf = reinterpret_cast<float *>(smem + Z::OTF), *Y = reinterpret_cast<float *>(smem + Z::OY);
    const int words = (p.n_tokens + 31) >> 5;
    float a_next = 1.0f, b_next = 0.0f;                  // gates of the chunk being loaded (threads 0..63)
    auto row_at = [&](const KvTensor &x, int row, int head) { return x.p + (b * x.sb + (long)row * x.st + head * x.sh) * ES; };
    auto load = [&](int c) {
      const int nt = tokens(c);
      char *X = smem + Z::OX + (c % NB) * Z::XBUF, *V = smem + Z::OV + (c % NB) * Z::VBUF;
      // q and k: eight lanes write one core of 8 rows
#pragma unroll
      for (int it = 0; it < 2 * (D / 32) * 2; ++it) {
        const int unit = it * 4 + aw, block = unit / (D / 32), k = (unit % (D / 32)) * 32 + (lane >> 3) * 8;    // blocks 0..7: k, 8..15: q
        const int r = (block & 7) * 8 + (lane & 7);
        const bool q = block >= 8, live = r < nt;
        if (q && !out) continue;
        const KvTensor &src = q ? p.q : p.k;
        const char *from = live ? row_at(src, row_of(p, b, c * C + r), hk) + k * ES : src.p;
        char *to = X + (q ? Z::ROWS : 0) + core_at(r, k, D);
        if (!F32) {
          cp16(to, from, live);
        } else {
          float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f), y = x;
          if (live) x = reinterpret_cast<const float4 *>(from)[0], y = reinterpret_cast<const float4 *>(from)[1];
          uint32_t w[3][4];
          split3(x.x, x.y, w[0][0], w[1][0], w[2][0]);
          split3(x.z, x.w, w[0][1], w[1][1], w[2][1]);
          split3(y.x, y.y, w[0][2], w[1][2], w[2][2]);
          split3(y.z, y.w, w[0][3], w[1][3], w[2][3]);
#pragma unroll
          for (int i = 0; i < NX; ++i) *reinterpret_cast<uint4 *>(to + i * Z::XPART) = make_uint4(w[i][0], w[i][1], w[i][2], w[i][3]);
        }
      }
      constexpr int PIECES = D * ES / 16;
#pragma unroll
      for (int it = 0; it < C * PIECES / 128; ++it) {
        const int i = it * 128 + at, r = i / PIECES, piece = i % PIECES;
        const bool live = r < nt;
        cp16(V + r * D * ES + piece * 16, live ? row_at(p.v, row_of(p, b, c * C + r), h) + piece * 16 : p.v.p, live);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
      a_next = 1.0f, b_next = 0.0f;
      if (!isq && t < nt) {
        const long row = row_of(p, b, c * C + t);
        a_next = reinterpret_cast<const float *>(p.a.p)[b * p.a.sb + row * p.a.st + h * p.a.sh];
        b_next = reinterpret_cast<const float *>(p.beta.p)[b * p.beta.sb + row * p.beta.st + h * p.beta.sh];
      }
    };
    for (int i = at; i < C * LD; i += 128) Tf[i] = 0.0f;
    if (chunks && NB > 1) load(0);
    for (int c = 0; c < chunks; ++c) {
      const int nt = tokens(c), np = padded(c), buf = c % NB;
      if (NB == 1) {
        if (c) wait(&x_free[0], c - 1);
        load(c);
      }
      const float a = a_next, be = b_next;
      if (NB > 1 && c + 1 < chunks) {
        if (c + 1 >= NB) wait(&x_free[(c + 1) % NB], (c + 1) / NB - 1);
        load(c + 1);
        asm volatile("cp.async.wait_group 1;" ::: "memory");
      } else {
        asm volatile("cp.async.wait_group 0;" ::: "memory");
      }
      fence_smem_to_async();
      arrive(&x_full[buf]);
      // ---- decays
      float *ga = reinterpret_cast<float *>(smem + Z::OG) + (c % 3) * 4 * C, *beta = ga + C, *G = ga + 2 * C, *rho = ga + 3 * C;
      if (!isq) ga[t] = a, beta[t] = be;
      uint64_t see = ~0ull;                              // ancestors
      if (p.mask) {
        see = 0;
        if (t < nt) {
          const uint32_t *row = p.mask + ((long)b * p.n_tokens + t) * words;
          see = row[0] | (words > 1 ? (uint64_t)row[1] << 32 : 0);
        }
      }
      aux_sync();
      float R[C];
      float r = 1.0f;
#pragma unroll
      for (int i = C - 1; i >= 0; --i) {
        const bool anc = i == t || (i < t && ((see >> i) & 1));
        R[i] = anc ? r : 0.0f;
        if (anc) r *= ga[i];
      }
      if (!isq) G[t] = r;
      if (at == C - 1) {
#pragma unroll
        for (int i = 0; i < C; ++i) rho[i] = R[i];
      }
      arrive(&gates[c % 3]);
      // ---- M (kept by columns) and P
      wait(g_done, c);
      fence_after_sync();
      const uint32_t tl = tmem + ((uint32_t)(aw * 32) << 16) + Z::D0;
      const float scale = isq ? 1.0f : beta[t];
#pragma unroll
      for (int i0 = 0; i0 < C; i0 += 16) {
        if (i0 < np) {
          uint32_t x[16];
          tmem_ld16(tl + i0, x);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const int i = i0 + e;
            R[i] *= scale * __uint_as_float(x[e]);
            if (!isq) M[i * LD + t] = i < t ? R[i] : 0.0f;
          }
        }
      }
      fence_before_sync();
      aux_sync();
      // ---- T = (I + M)^-1
      if (aw < 2 && aw * 32 < np) {
        const float *m = M + aw * 32 * LD + aw * 32;
        float x[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) x[i] = i == lane ? 1.0f : 0.0f;
#pragma unroll
        for (int i = 0; i < 31; ++i)
#pragma unroll
          for (int k = (i + 1) & ~3; k < 32; k += 4) {
            const float4 y = *reinterpret_cast<const float4 *>(m + i * LD + k);
            if (k > i) x[k] = fmaf(-y.x, x[i], x[k]);
            if (k + 1 > i) x[k + 1] = fmaf(-y.y, x[i], x[k + 1]);
            if (k + 2 > i) x[k + 2] = fmaf(-y.z, x[i], x[k + 2]);
            if (k + 3 > i) x[k + 3] = fmaf(-y.w, x[i], x[k + 3]);
          }
#pragma unroll
        for (int i = 0; i < 32; ++i) Tf[(aw * 32 + i) * LD + aw * 32 + lane] = x[i];
      }
      aux_sync();
      if (np > 32) {
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = 0.0f;
#pragma unroll 8
        for (int i = 0; i < 32; ++i) {
          const float x = Tf[i * LD + lane];
          const float4 m0 = *reinterpret_cast<const float4 *>(M + i * LD + 32 + 8 * aw), m1 = *reinterpret_cast<const float4 *>(M + i * LD + 36 + 8 * aw);
          y[0] = fmaf(m0.x, x, y[0]), y[1] = fmaf(m0.y, x, y[1]), y[2] = fmaf(m0.z, x, y[2]), y[3] = fmaf(m0.w, x, y[3]);
          y[4] = fmaf(m1.x, x, y[4]), y[5] = fmaf(m1.y, x, y[5]), y[6] = fmaf(m1.z, x, y[6]), y[7] = fmaf(m1.w, x, y[7]);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) Y[(8 * aw + i) * 36 + lane] = y[i];
        aux_sync();
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = 0.0f;
#pragma unroll 2
        for (int k = 0; k < 32; k += 4) {
          float x[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) x[e] = Y[(k + e) * 36 + lane];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float4 m = *reinterpret_cast<const float4 *>(Tf + (32 + 8 * aw + i) * LD + 32 + k);
            y[i] = fmaf(-m.x, x[0], y[i]), y[i] = fmaf(-m.y, x[1], y[i]), y[i] = fmaf(-m.z, x[2], y[i]), y[i] = fmaf(-m.w, x[3], y[i]);
          }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) Tf[(32 + 8 * aw + i) * LD + lane] = y[i];
        aux_sync();
      }
      if (c) wait(u_done, c - 1);
#pragma unroll
      for (int k = 0; k < 32; k += 8) {
        const int i = (at >> 6) * 32 + k;
        const float4 x = *reinterpret_cast<const float4 *>(Tf + t * LD + i), y = *reinterpret_cast<const float4 *>(Tf + t * LD + i + 4);
        uint32_t w[3][4];
        split3(x.x, x.y, w[0][0], w[1][0], w[2][0]);
        split3(x.z, x.w, w[0][1], w[1][1], w[2][1]);
        split3(y.x, y.y, w[0][2], w[1][2], w[2][2]);
        split3(y.z, y.w, w[0][3], w[1][3], w[2][3]);
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
            uint32_t w[3][4];
#pragma unroll
            for (int e = 0; e < 4; ++e) split3(R[i + 2 * e], R[i + 2 * e + 1], w[0][e], w[1][e], w[2][e]);
#pragma unroll
            for (int e = 0; e < NO; ++e)
              *reinterpret_cast<uint4 *>(smem + Z::OP + e * Z::TPART + core_at(t, i, C)) = make_uint4(w[e][0], w[e][1], w[e][2], w[e][3]);
          }
        }
        fence_smem_to_async();
        arrive(p_ready);
      }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
  } else {
    // ---------------------------------------------------------------- products
    uint32_t leader;
    asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(leader));
    const uint32_t base = smem_u32(smem);
    constexpr uint32_t SBO = (D / 8) * 128;
    auto x_desc = [&](int c, int part, int q) { return smem_desc(base + Z::OX + (c % NB) * Z::XBUF + part * Z::XPART + q * Z::ROWS, 128, SBO); };
    // D (+)= A B^T summed over part pairs i + j <= MOST, smallest first; `one` issues a pair (the first of all clears D)
    auto pairs = [&](auto na, auto nb, auto most, auto one) {
      bool first = true;
#pragma unroll
      for (int sum = decltype(most)::value; sum >= 0; --sum)
#pragma unroll
        for (int i = 0; i < decltype(na)::value; ++i) {
          const int k = sum - i;
          if (k < 0 || k >= decltype(nb)::value) continue;
          one(i, k, first);
          first = false;
        }
    };
    using I1 = std::integral_constant<int, 1>;
    using I2 = std::integral_constant<int, 2>;
    using I3 = std::integral_constant<int, 3>;
    using INX = std::integral_constant<int, NX>;
    using INO = std::integral_constant<int, NO>;
    using IMO = std::integral_constant<int, NO - 1>;
    auto dots = [&](int c) {                             // [k | q] k^T
      wait(&x_full[c % NB], c / NB);
      fence_after_sync();
      if (leader && good) {
        const uint32_t id = idesc_n(padded(c));
        pairs(INX{}, INX{}, I2{}, [&](int i, int k, bool first) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            mma_ss(tmem + Z::D0, x_desc(c, i, 0) + kk * 16, x_desc(c, k, 0) + kk * 16, id, first && kk == 0 ? 0u : 1u);
        });
        commit(g_done);
      }
    };
    if (chunks) dots(0);
    for (int c = 0; c < chunks; ++c) {
      const int np = padded(c), steps = np / 16;
      const uint32_t id = idesc_n(np);
      wait(a1, c);
      fence_after_sync();
      if (leader && good) {
        pairs(I3{}, INX{}, I2{}, [&](int i, int k, bool first) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            mma_ts(tmem + Z::D1, tmem + Z::A1 + i * (D / 2) + 8 * kk, x_desc(c, k, 0) + kk * 16, id, first && kk == 0 ? 0u : 1u);
        });
        commit(w_done);
        if (out) {
          pairs(I3{}, INX{}, IMO{}, [&](int i, int k, bool first) {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              mma_ts(tmem + Z::D1 + C, tmem + Z::A1 + i * (D / 2) + 8 * kk, x_desc(c, k, 1) + kk * 16, id, first && kk == 0 ? 0u : 1u);
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
          for (int kk = 0; kk < steps; ++kk)
            mma_ts(tmem + Z::D2 + 16 * kk, tmem + Z::A2 + i * (C / 2) + 8 * kk,
                   smem_desc(base + Z::OT + k * Z::TPART + kk * (2 * 1024 + 256), 128, 1024), idesc_n(np - 16 * kk), first && kk == 0 ? 0u : 1u);
        });
        commit(u_done);
      }
      if (NB > 1 && c + 1 < chunks) dots(c + 1);
      if (p.write) {
        wait(a3, c);
        fence_after_sync();
        if (leader && good) {
          pairs(I3{}, INX{}, I2{}, [&](int i, int k, bool first) {
            for (int kk = 0; kk < steps; ++kk)
              mma_ts(tmem + Z::D3, tmem + Z::A3 + i * (C / 2) + 8 * kk,
                     smem_desc(base + Z::OX + (c % NB) * Z::XBUF + k * Z::XPART + kk * 2 * SBO, SBO, 128), idesc(D, 1), first && kk == 0 ? 0u : 1u);
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
            for (int kk = 0; kk < steps; ++kk)
              mma_ts(tmem + Z::D4 + 16 * kk, tmem + Z::A4 + i * (C / 2) + 8 * kk,
                     smem_desc(base + Z::OP + k * Z::TPART + kk * (2 * 1024 + 256), 128, 1024), idesc_n(np - 16 * kk), first && kk == 0 ? 0u : 1u);
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
  if (warp == Z::W_MMA) tmem_dealloc(tmem, 512);
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
