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
// of bf16 I/O enter as they are. bf16 I/O forms S^T q from two parts of the state and outputs from two of u and P (o is rounded to 8 bits); S^T k,
// which comes back into the state, from three (two left up to 2.4e-6 of the states' norm where decays are slow; the third costs 6% of a long
// prompt). Outputs from three parts as well are as far from those in 64 bits (1.66e-3, the rounding of o) and differ from these in one last bit of
// some hundreds, for 4 to 7 (u and P) or 15 to 19% (S too) more time. The state itself stays in fp32 registers and takes D3 by an ordinary
// addition: the tensor cores' additions cut off, which would add up over a long prompt.
//
// Roles: sixteen warps own the columns (four a quarter of TMEM's lanes: a block of 16 tokens and a quarter of the state's rows each), four form
// R, M and P (fp32 I/O: and split the rows of k and q), four T, one chunk ahead, three (two) copy rows, one issues the products.
// A sequence and head is a chain of chunks, each 4.7 us (9,700 cycles: parts of the state and w 2,500, rhs 1,600, u 1,100, its parts 900, the
// increment 1,200, waits), which bounds this form of the rule (u is formed by two dependent products); a block fills TMEM and shared memory, so that
// nothing overlaps another chain. Heads of 128, bf16: 96 chains of up to 16,384 tokens 1,200 us (1.07 TB/s), 512 of 695 to 2048 tokens 438 us (1.35 TB/s,
// 161 TFLOP/s by the rule's own count); fp32 512 chains of 512 tokens 382 us (bf16 185). Two warps that issue products, or outputs read later in columns
// of their own, took longer.
// Every wait is bounded; one that gives up sets the status word, after which the block goes on without waiting or products; the warps of the columns
// agree before they store a state, so that it is whole or as it was.
#pragma once

#include "delta_common.cuh"
#include "umma.cuh"

#include <type_traits>

namespace pace {
namespace delta {
using namespace umma;

constexpr int C = 64;                                    // tokens a chunk

// A sequence and head of the call, as a block keeps it: b, h; tokens (0: none, or left out); slot; whether it begins with a zero state.
struct Unit {
  uint32_t bh;
  int n;
  uint32_t slot;
};
constexpr int UNITS = 64;                                // most of a block
// Most chunks of a call whose blocks go from one sequence and head to the next. 512 of equal length, heads of 128, bf16: of 64 tokens 49 us, a block for
// each 57; of 128 71 and 76; of 256 117 and 114; of 512 205 and 187; 2048 of 64 tokens 151 and 184. fp32: 2048 of 64 tokens 217 and 258, of 256 697 and 715, of 512 1343
// and 1330; heads of 64 396 and 436 of 256, 739 and 772 of 512, 1420 and 1443 of 1024.
constexpr int CHUNKS_LASTING = 4;

template <int D, bool F32>
struct Shape {
  static constexpr int MAIN = 16, AUX = 4, W_TAB = MAIN, W_INV = W_TAB + AUX, W_MMA = W_INV + AUX, W_LOAD = W_MMA + 1, LOAD = F32 ? 2 : 3, THREADS = (W_LOAD + LOAD) * 32;
  static constexpr int NX = F32 ? 3 : 1;                 // parts of q and k
  static constexpr int NO = F32 ? 3 : 2;                 // parts of u and P in the outputs
  static constexpr int NB = !F32 ? 3 : D == 64 ? 2 : 1, NV = F32 && D == 128 ? 1 : 2;   // chunks of rows of q and k, and of v, in shared memory
  static constexpr int NM = F32 ? 1 : 2;                 // chunks of M
  static constexpr int NS = 3, NQ = F32 ? 3 : 2;         // parts of the state in w, and in p
  static constexpr int HELD = D / 4;                     // rows of the state that a thread holds
  static constexpr int ROWS = C * D * 2;                 // one part of 64 rows
  static constexpr int XPART = 2 * ROWS, XBUF = NX * XPART;
  static constexpr int VBUF = C * D * (F32 ? 4 : 2);     // rows of v, later those of o
  static constexpr int TPART = C * C * 2;
  static constexpr int LD = C + 4, LY = 36;              // rows of the fp32 tables
  static constexpr int OX = 0, OV = OX + NB * XBUF, OT = OV + NV * VBUF, OP = OT + 3 * TPART, OM = OP + 2 * NO * TPART, OY = OM + NM * C * LD * 4,
                       OG = OY + 32 * LY * 4, OBAR = OG + 3 * 4 * C * 4, NBAR = 2 * NB + 2 * NV + 2 * NM + 3 + 17, OMISC = OBAR + NBAR * 8,
                       OUNIT = OMISC + 16, SMEM = OUNIT + UNITS * (int)sizeof(Unit);
  static_assert(SMEM <= 227 * 1024 && OBAR % 8 == 0, "shared memory");
  // TMEM columns. What lies over something else is written when the products that read that have ended, or by products issued when the warps
  // that read it have said so (u over the outputs: o_read; tests/test_delta_order_host.py goes through all of them): R_C u over rhs (whose halves are done as
  // those of u are), the state's increment over its parts, u over w; with fp32 I/O rhs over the state's third part, and so q's products before rhs.
  static constexpr uint32_t W = 256, P = 320, D2 = 384, D4 = 384, D0 = 448, D3 = F32 ? 64 : 0;
  __host__ __device__ static constexpr uint32_t a1(int part) { return 64 * part; }
  __host__ __device__ static constexpr uint32_t a2(int part) { return 128 + 32 * part; }
  __host__ __device__ static constexpr uint32_t a3(int part) { return F32 && part < 2 ? 32 * part : 128 + 32 * part; }
  __host__ __device__ static constexpr uint32_t a4(int part) { return part < 2 ? W + 32 * part : 224; }
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
template <int ID>
__device__ __forceinline__ void sync4() { asm volatile("bar.sync %0, 128;" ::"n"(ID) : "memory"); }      // four warps (1: tables, 2..5: columns, 6: inverses)
__host__ __device__ constexpr uint32_t idesc(int N, int mn_major) {   // M = 128, bf16, fp32 sums
  return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)mn_major << 16) | ((uint32_t)(N >> 3) << 17) | (8u << 24);
}
__device__ __forceinline__ uint32_t idesc_n(int N) { return idesc(0, 0) | ((uint32_t)(N >> 3) << 17); }

// (A wait that is not over at the first look, out of line: the roles' loops together should stay in the instruction cache. Unrolled and
// in line, with eight column warps, 3.9 of the 10.5 warps a scheduler counts an issued instruction waited for theirs; so 0.3 do.)
static __device__ __noinline__ bool wait_long(uint64_t *bar, uint32_t parity, uint32_t *failed, uint32_t limit_ns) {
  if (mbar_wait(bar, parity, limit_ns)) return true;
  *reinterpret_cast<volatile uint32_t *>(failed) = 1;
  return false;
}
constexpr uint32_t WAIT_NS = 1000000000;

// y += m x for a pair of rows.
__device__ __forceinline__ void fma_pair(uint64_t &y, uint64_t m, float x) {
  asm("{\n\t.reg .b64 v;\n\tmov.b64 v, {%2, %2};\n\tfma.rn.f32x2 %0, %1, v, %0;\n\t}" : "+l"(y) : "l"(m), "f"(x));
}
__device__ __forceinline__ float2 pair(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}

// ONE: a block for each sequence and head; else blocks go on from one to the next, whose rows and tables are then under way.
template <int D, bool F32, bool ONE>
__global__ void __launch_bounds__(Shape<D, F32>::THREADS, 1) delta_chunk_kernel(const DeltaArgs p) {
  using Z = Shape<D, F32>;
  constexpr int NX = Z::NX, NO = Z::NO, NB = Z::NB, NV = Z::NV, NM = Z::NM, NS = Z::NS, NQ = Z::NQ, LD = Z::LD, LY = Z::LY, ES = F32 ? 4 : 2;
  extern __shared__ __align__(128) char smem[];
  uint64_t *bar = reinterpret_cast<uint64_t *>(smem + Z::OBAR);
  // (those of two: for the halves of a chunk's tokens)
  uint64_t *x_full = bar, *x_free = x_full + NB, *o_free = x_free + NB, *o_ready = o_free + NV, *m_ready = o_ready + NV, *m_free = m_ready + NM, *ready = m_free + NM,
           *a1 = ready + 3, *a2 = a1 + 1, *a3 = a2 + 2, *a4 = a3 + 2, *u_done = a4 + 1, *w_done = u_done + 2, *p_done = w_done + 1,
           *s_done = p_done + 1, *o_done = s_done + 1, *o_read = o_done + 1, *g_done = o_read + 1, *t_ready = g_done + 1, *drain = t_ready + 1;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + Z::OMISC), *failed = tmem_slot + 1;      // failed: a wait of the block gave up
  const uint32_t limit = p.probe_ns ? p.probe_ns : WAIT_NS;
  Unit *unit = reinterpret_cast<Unit *>(smem + Z::OUNIT);
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const bool out = p.o.p != nullptr;

  if (warp == Z::W_MMA) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  if (tid == 0) {
    for (int i = 0; i < NB; ++i) mbar_init(&x_full[i], F32 ? Z::AUX : 1), mbar_init(&x_free[i], 1);
    for (int i = 0; i < NV; ++i) mbar_init(&o_free[i], 1), mbar_init(&o_ready[i], Z::MAIN);
    for (int i = 0; i < NM; ++i) mbar_init(&m_ready[i], Z::AUX), mbar_init(&m_free[i], Z::AUX);
    for (int i = 0; i < 3; ++i) mbar_init(&ready[i], Z::AUX + 1);
    for (uint64_t *x : {a1, a4, o_read}) mbar_init(x, Z::MAIN);
    for (uint64_t *x : {a2, a2 + 1, a3, a3 + 1}) mbar_init(x, Z::MAIN / 2);
    for (uint64_t *x : {w_done, p_done, u_done, u_done + 1, s_done, o_done, g_done, drain}) mbar_init(x, 1);
    mbar_init(t_ready, Z::AUX);
    *failed = 0;
    mbar_fence_init();
  }
  pdl_enter();
  // ---- this block's sequences and heads. The longest sequences go out first; to lasting blocks in turn there and back
  const int total = p.batch * p.H, turns = ONE ? 1 : (total + gridDim.x - 1) / gridDim.x;
  uint16_t *order = reinterpret_cast<uint16_t *>(smem + Z::OX);
  const bool sorted = total > p.sms && (p.n_new || p.n_keep) && p.batch <= 256;
  if (sorted) {
    int *count = reinterpret_cast<int *>(smem + Z::OM);
    if (tid < p.batch) count[tid] = count_of(p, tid);
    __syncthreads();
    if (tid < p.batch) {
      int rank = 0;
      for (int i = 0; i < p.batch; ++i) rank += count[i] > count[tid] || (count[i] == count[tid] && i < tid);
      order[rank] = (uint16_t)tid;
    }
    __syncthreads();
  }
  auto zeros = [&](int b, int h, int n, int i, int step) {   // outputs past the sequence's tokens, by `step` threads
    constexpr int PIECES = D * ES / 16;
    char *o = p.o.p + (b * p.o.sb + h * p.o.sh) * ES;
    for (long x = (long)n * PIECES + i; x < (long)p.n_tokens * PIECES; x += step)
      *reinterpret_cast<uint4 *>(o + x / PIECES * p.o.st * ES + x % PIECES * 16) = make_uint4(0, 0, 0, 0);
  };
  for (int k = warp; k < turns; k += Z::THREADS / 32) {
    const int u = ONE ? blockIdx.x : k * gridDim.x + (k & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
    if (u >= total) {
      if (lane == 0) unit[k].n = 0;
      continue;
    }
    const int h = u % p.H, b = sorted ? order[u / p.H] : u / p.H;
    int bad = 0;
    Seq s = sequence(p, b, bad);
    if (s.n > 0 && taken(p, b, s.slot)) {
      bad |= PACE_DELTA_BAD_SLOT;
      s.n = 0;
    }
    if (bad && h == 0 && lane == 0) atomicOr(p.status, bad);
    if (lane == 0) unit[k] = Unit{(uint32_t)(b * PACE_MAX_HEADS + h), s.n, (uint32_t)s.slot | (uint32_t)s.fresh << 31};
    if (out && !ONE) zeros(b, h, s.n, lane, 32);
  }
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  constexpr uint32_t tmem = 0;          // the whole of TMEM is this block's: its first column (a constant keeps addresses uniform)
  // The unit that a role works on, and the place of the chunk among all chunks of the block (buffers and barriers go by that): its number g, and
  // what is left of it and how often it went around in a ring of three.
  int b = 0, h = 0, hk = 0, n = 0, chunks = 0, g = 0, ring = 0, rounds = 0;
  auto step = [&]() {
    ++g;
    if (!ONE && ++ring == 3) ring = 0, ++rounds;
  };
  auto g3 = [&]() { return ONE ? g % 3 : ring; };        // (counted where there are many short ones, divided where registers are dearer)
  auto r3 = [&]() { return ONE ? g / 3 : rounds; };
  auto take = [&](int k) {
    const Unit u = unit[k];
    b = u.bh / PACE_MAX_HEADS, h = u.bh % PACE_MAX_HEADS, hk = h / p.group, n = u.n;
    chunks = (n + C - 1) / C;
    return n > 0;
  };
  // tokens of a chunk, and as the products count them
  auto tokens = [&](int c) { return min(C, n - c * C); };
  auto padded = [&](int c) { return (tokens(c) + 15) & ~15; };
  auto at_x = [&]() { return NB == 3 ? g3() : g % NB; };
  auto round_x = [&]() { return NB == 3 ? r3() : g / NB; };

  bool good = true;
  auto wait = [&](uint64_t *x, int phase) {              // (by the whole warp)
    if (good && !mbar_try_wait(x, phase & 1)) good = wait_long(x, phase & 1, failed, limit);
    __syncwarp();
  };
  auto arrive = [&](uint64_t *x) {
    __syncwarp();
    if (lane == 0) mbar_arrive(x);
  };

  // Copies `per` rows at a time: lane's row `first` and piece of it; `one` gets its address and whether the row exists.
  auto rows = [&](const KvTensor &x, int head, int c, int first, int per, int piece, auto one) {
    const int nt = tokens(c);
    const long step = x.st * ES;
    const char *base = x.p + (b * x.sb + head * x.sh) * ES + piece, *at = base + (c * C + first) * step;
    const long next = per * step;
    if (nt == C && !p.idx) {
#pragma unroll 8
      for (int r = 0; r < C; r += per, at += next) one(r, at, true);
    } else {
#pragma unroll 1
      for (int r = 0; r < C; r += per, at += next) {
        const bool live = r + first < nt;
        const char *from = live ? at : x.p;
        if (p.idx && live) from = base + row_of(p, b, c * C + r + first) * step;
        one(r, from, live);
      }
    }
  };
  // k and q of a chunk into their buffer, by warp `part` of `PARTS`: eight lanes write one core of 8 rows
  auto load_x = [&](int c, auto parts, int part) {
    constexpr int PARTS = decltype(parts)::value;
    const int k = (lane >> 3) * 8, first = part * 8;
#pragma unroll 1
    for (int q = 0; q < (out ? 2 : 1); ++q) {
      const uint32_t to = smem_u32(smem) + Z::OX + at_x() * Z::XBUF + q * Z::ROWS + core_at(first + (lane & 7), k, D);
      rows(q ? p.q : p.k, hk, c, first + (lane & 7), 8 * PARTS, k * ES, [&](int r, const char *from, bool live) {
#pragma unroll
        for (int g = 0; g < D / 32; ++g) {
          const uint32_t dst = to + core_at(r, g * 32, D);
          if (!F32) {
            cp16(dst, from + g * 32 * ES, live ? 16 : 0);          // (a row that does not exist is not read)
          } else {
            float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f), y = x;
            if (live) x = reinterpret_cast<const float4 *>(from + g * 32 * ES)[0], y = reinterpret_cast<const float4 *>(from + g * 32 * ES)[1];
            uint32_t w[3][4];
            split<3>(x.x, x.y, &w[0][0], 4), split<3>(x.z, x.w, &w[0][1], 4), split<3>(y.x, y.y, &w[0][2], 4), split<3>(y.z, y.w, &w[0][3], 4);
#pragma unroll
            for (int i = 0; i < NX; ++i)
              asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst + i * Z::XPART), "r"(w[i][0]), "r"(w[i][1]), "r"(w[i][2]), "r"(w[i][3])
                           : "memory");
          }
        }
      });
    }
  };

  if (warp < Z::MAIN) {
    // ---------------------------------------------------------------- columns: four warps a quarter of the lanes, each with 16 of a chunk's
    // tokens and a quarter of the state's rows
    const int grp = warp >> 2, j = (warp & 3) * 32 + lane, t0 = 16 * grp, half = grp >> 1;
    const uint32_t tl = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const bool on = (warp & 3) * 32 < D;                 // (heads of 64 leave half of the lanes alone)
    constexpr int HELD = Z::HELD;
    float S[HELD];                                       // rows HELD grp .. of the state's column j
    // outputs of a chunk: read when they are done, stored through its rows of v when u's products have been given their rhs
    uint32_t held[F32 ? 16 : 8];
    auto read_outputs = [&](int c) {                     // (the chunk before g)
      const float4 *Gb = reinterpret_cast<const float4 *>(smem + Z::OG) + (g3() ? g3() - 1 : 2) * C + 2 * (C / 4);
      wait(o_done, g - 1);
      fence_after_sync();
      if (on && t0 < padded(c)) {
#pragma unroll
        for (int e0 = 0; e0 < 16; e0 += 8) {
          uint32_t x[8], y[8];
          tmem_ld8(tl + Z::D4 + t0 + e0, x);
          tmem_ld8(tl + Z::P + t0 + e0, y);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 8; e += 4) {
            const float4 g = Gb[(t0 + e0 + e) / 4];
            const float o0 = fmaf(g.x, __uint_as_float(y[e]), __uint_as_float(x[e])), o1 = fmaf(g.y, __uint_as_float(y[e + 1]), __uint_as_float(x[e + 1]));
            const float o2 = fmaf(g.z, __uint_as_float(y[e + 2]), __uint_as_float(x[e + 2])), o3 = fmaf(g.w, __uint_as_float(y[e + 3]), __uint_as_float(x[e + 3]));
            if (F32) {
              held[(e0 + e) % (F32 ? 16 : 8)] = __float_as_uint(o0), held[(e0 + e + 1) % (F32 ? 16 : 8)] = __float_as_uint(o1);
              held[(e0 + e + 2) % (F32 ? 16 : 8)] = __float_as_uint(o2), held[(e0 + e + 3) % (F32 ? 16 : 8)] = __float_as_uint(o3);
            } else {
              held[(e0 + e) / 2] = pack2(o0, o1), held[(e0 + e) / 2 + 1] = pack2(o2, o3);
            }
          }
        }
      }
      fence_before_sync();
      arrive(o_read);
    };
    auto store_outputs = [&](int c) {
      if (on && t0 < padded(c)) {
        char *to = smem + Z::OV + ((g - 1) % NV) * Z::VBUF + j * ES + t0 * D * ES;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          if (F32) *reinterpret_cast<uint32_t *>(to + e * D * ES) = held[e % (F32 ? 16 : 8)];
          else *reinterpret_cast<uint16_t *>(to + e * D * ES) = (uint16_t)(held[e / 2] >> (e & 1) * 16);
        }
      }
      arrive(&o_ready[(g - 1) % NV]);                    // (of this buffer: the next one's outputs may be there before these are looked for)
    };
    float gC = 1.0f;
#pragma unroll 1
    for (int k = 0; k < turns; ++k) {
      if (!take(k)) continue;
      auto state = [&]() {
        const Unit u = unit[k];
        return p.S + ((long)(u.slot & 0x7FFFFFFFu) * p.H + u.bh % PACE_MAX_HEADS) * D * D + (long)(grp * HELD) * D + j;
      };
      {
        const float *from = state();
        const bool held_before = on && !(unit[k].slot >> 31);
#pragma unroll
        for (int i = 0; i < HELD; ++i) S[i] = held_before ? from[i * D] : 0.0f;
      }
      // (the end of a chunk is worked off in the next one's turn, between what that chunk's products wait for)
#pragma unroll 1
      for (int c = 0; c <= chunks; ++c) {
        const float4 *ga = reinterpret_cast<const float4 *>(smem + Z::OG) + g3() * C, *beta = ga + C / 4, *G = ga + 2 * (C / 4), *rho = ga + 3 * (C / 4);
        // ---- the state at the end of the chunk before (its increment lies over parts: all four warps read theirs before any writes)
        if (c > 0 && p.write) {
          wait(s_done, g - 1);
          fence_after_sync();
          if (on) {
#pragma unroll
            for (int i = 0; i < HELD; i += 16) {
              uint32_t x[16];
              tmem_ld16(tl + Z::D3 + grp * HELD + i, x);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) S[i + e] = fmaf(gC, S[i + e], __uint_as_float(x[e]));
            }
            asm volatile("bar.sync %0, 128;" ::"r"(2 + (warp & 3)) : "memory");
          }
        }
        if (c < chunks) {
          // ---- its parts, as the first operand of w and p
          if (on) {
#pragma unroll
            for (int i = 0; i < HELD; i += 16) {
              uint32_t x[NS][8];
#pragma unroll
              for (int e = 0; e < 8; ++e) split<NS>(S[i + 2 * e], S[i + 2 * e + 1], &x[0][e], 8);
#pragma unroll
              for (int k = 0; k < NS; ++k) tmem_st8(tl + Z::a1(k) + (grp * HELD + i) / 2, x[k]);
            }
            tmem_wait_st();
          }
          fence_before_sync();
          arrive(a1);
        }
        if (out && c > 0) {
          read_outputs(c - 1);
          if (NV == 1) store_outputs(c - 1);                 // (this chunk's rows of v come where they leave)
        }
        const bool mine = on && t0 < padded(c);            // (the products read no tokens past these)
        if (c < chunks) {
          // ---- rhs = beta (v - G w)
          wait(&ready[g3()], r3());
          wait(w_done, g);
          if (F32 && out) wait(p_done, g);                   // (q's products read the part of S that rhs lies over)
          fence_after_sync();
          if (mine) {
            const char *at = smem + Z::OV + (g % NV) * Z::VBUF + j * ES + t0 * D * ES;
#pragma unroll (ONE ? 2 : 1)
            for (int e0 = 0; e0 < 16; e0 += 8, at += 8 * D * ES) {
              uint32_t w[8], x[3][4];
              tmem_ld8(tl + Z::W + t0 + e0, w);
              float v[8];
#pragma unroll
              for (int e = 0; e < 8; ++e)
                v[e] = F32 ? *reinterpret_cast<const float *>(at + e * D * ES)
                           : __uint_as_float((uint32_t)*reinterpret_cast<const uint16_t *>(at + e * D * ES) << 16);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 8; e += 4) {
                const float4 g = G[(t0 + e0 + e) / 4], be = beta[(t0 + e0 + e) / 4];
                const float y0 = be.x * fmaf(-g.x, __uint_as_float(w[e]), v[e]), y1 = be.y * fmaf(-g.y, __uint_as_float(w[e + 1]), v[e + 1]);
                const float y2 = be.z * fmaf(-g.z, __uint_as_float(w[e + 2]), v[e + 2]), y3 = be.w * fmaf(-g.w, __uint_as_float(w[e + 3]), v[e + 3]);
                split<3>(y0, y1, &x[0][e / 2], 4);
                split<3>(y2, y3, &x[0][e / 2 + 1], 4);
              }
#pragma unroll
              for (int k = 0; k < 3; ++k) tmem_st4(tl + Z::a2(k) + (t0 + e0) / 2, x[k]);
            }
            tmem_wait_st();
          }
          fence_before_sync();
          arrive(a2 + half);
        }
        if (NV > 1 && out && c > 0) store_outputs(c - 1);
        if (c == chunks) break;                            // (its place is the next unit's first chunk's)
        gC = G[C / 4 - 1].w;
        // ---- u, decayed to the chunk's end
        wait(u_done + half, g);
        fence_after_sync();
        if (p.write) {
          if (mine) {
#pragma unroll (ONE ? 2 : 1)
            for (int e0 = 0; e0 < 16; e0 += 8) {
              uint32_t u[8], x[3][4];
              tmem_ld8(tl + Z::D2 + t0 + e0, u);
              const float4 g = rho[(t0 + e0) / 4], f = rho[(t0 + e0) / 4 + 1];
              tmem_wait_ld();
              split<3>(g.x * __uint_as_float(u[0]), g.y * __uint_as_float(u[1]), &x[0][0], 4);
              split<3>(g.z * __uint_as_float(u[2]), g.w * __uint_as_float(u[3]), &x[0][1], 4);
              split<3>(f.x * __uint_as_float(u[4]), f.y * __uint_as_float(u[5]), &x[0][2], 4);
              split<3>(f.z * __uint_as_float(u[6]), f.w * __uint_as_float(u[7]), &x[0][3], 4);
#pragma unroll
              for (int k = 0; k < 3; ++k) tmem_st4(tl + Z::a3(k) + (t0 + e0) / 2, x[k]);
            }
            tmem_wait_st();
          }
          fence_before_sync();
          arrive(a3 + half);
        }
        // ---- u as it is (over w, which the other half's warps have read when their u is done)
        if (out) {
          if (half == 0) {
            wait(u_done + 1, g);
            fence_after_sync();
          }
          if (mine) {
#pragma unroll 1
            for (int e0 = 0; e0 < 16; e0 += 8) {
              uint32_t u[8], x[NO][4];
              tmem_ld8(tl + Z::D2 + t0 + e0, u);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 4; ++e) split<NO>(__uint_as_float(u[2 * e]), __uint_as_float(u[2 * e + 1]), &x[0][e], 4);
#pragma unroll
              for (int k = 0; k < NO; ++k) tmem_st4(tl + Z::a4(k) + (t0 + e0) / 2, x[k]);
            }
            tmem_wait_st();
          }
          fence_before_sync();
          arrive(a4);
        }
        step();
      }
      uint32_t bad = 1;
      if (p.write) {                                       // (all of them store or none)
        bad = *reinterpret_cast<volatile uint32_t *>(failed);
        asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %0, 0;\n\tbar.red.or.pred q, 7, %1, q;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "+r"(bad) : "n"(Z::MAIN * 32) : "memory");
      }
      if (on && !bad) {
        float *to = state();
#pragma unroll
        for (int i = 0; i < HELD; ++i) to[i * D] = S[i];
      }
    }
    if (ONE && out) zeros(unit[0].bh / PACE_MAX_HEADS, unit[0].bh % PACE_MAX_HEADS, unit[0].n, tid, Z::MAIN * 32);
  } else if (warp < Z::W_INV) {
    // ---------------------------------------------------------------- tables of the chunks
    const int at = tid - Z::W_TAB * 32, aw = warp - Z::W_TAB, t = at & 63;
    const bool isq = at >= 64;                           // rows of k (M, T), then of q (P)
    const int words = (p.n_tokens + 31) >> 5;
    float a_next, b_next;                                // gates of the next chunk (threads 0..63; others and rows past the end: of a row that exists)
    auto fetch = [&](int c) {
      const int i = min(c * C + t, n - 1);
      const long row = row_of(p, b, i);
      a_next = reinterpret_cast<const float *>(p.a.p)[b * p.a.sb + row * p.a.st + h * p.a.sh];
      b_next = reinterpret_cast<const float *>(p.beta.p)[b * p.beta.sb + row * p.beta.st + h * p.beta.sh];
    };
#pragma unroll 1
    for (int k = 0; k < turns; ++k) {
      if (!take(k)) continue;
      fetch(0);
#pragma unroll 1
      for (int c = 0; c < chunks; ++c) {
        if (F32) {
          // (rows of k and q in parts; 512 chains of 512 tokens, heads of 128: 383 us, with one warp for that 672)
          if (g >= NB) wait(&x_free[at_x()], round_x() - 1);
          load_x(c, std::integral_constant<int, Z::AUX>{}, aw);
          fence_smem_to_async();
          arrive(&x_full[at_x()]);
          if (c + 1 < chunks && !p.idx && (c + 1) * C + t < n) {     // the next chunk's, on their way
            const KvTensor &x = isq && out ? p.q : p.k;
            const char *next = x.p + (b * x.sb + ((c + 1) * C + t) * x.st + hk * x.sh) * ES;
            for (int i = 0; i < D * ES; i += 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(next + i));
          }
        }
        const int nt = tokens(c), np = padded(c);
        float *ga = reinterpret_cast<float *>(smem + Z::OG) + g3() * 4 * C, *beta = ga + C, *G = ga + 2 * C, *rho = ga + 3 * C;
        if (!isq) ga[t] = t < nt ? a_next : 1.0f, beta[t] = t < nt ? b_next : 0.0f;
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
        if (t < 32) see[0] = (see[0] | 1u << t) & ((2u << t) - 1), see[1] = 0;
        else see[1] = (see[1] | 1u << (t - 32)) & ((2u << (t - 32)) - 1);
        float *M = reinterpret_cast<float *>(smem + Z::OM) + (g % NM) * C * LD;
        sync4<1>();
        if (g >= NM) wait(&m_free[g % NM], g / NM - 1);
        wait(g_done, g);                                   // (with it the output products of the chunk before the last are done)
        fence_after_sync();
        // ---- a row of R from its end, times the dot products: M (a row's entries in a column; rows of M carry beta) and P
        float r = isq ? 1.0f : beta[t];
#pragma unroll 1
        for (int i0 = C - 16; i0 >= 0; i0 -= 16) {
          uint32_t x[16];
          if (i0 < np) {
            tmem_ld16(tmem + ((uint32_t)(aw * 32) << 16) + Z::D0 + i0, x);
          } else {
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] = 0;
          }
          const uint32_t bits = (i0 < 32 ? see[0] : see[1]) >> (i0 & 31);
          float R[16];
#pragma unroll
          for (int e0 = 12; e0 >= 0; e0 -= 4) {
            const float4 a = *reinterpret_cast<const float4 *>(ga + i0 + e0);
            const float as[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int e = 3; e >= 0; --e) {
              const bool anc = bits & (1u << (e0 + e));
              R[e0 + e] = anc ? r : 0.0f;
              r *= anc ? as[e] : 1.0f;
            }
          }
          if (at == 2 * C - 1) {
#pragma unroll
            for (int e = 0; e < 16; e += 4) *reinterpret_cast<float4 *>(rho + i0 + e) = make_float4(R[e], R[e + 1], R[e + 2], R[e + 3]);
          }
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 16; ++e) R[e] *= __uint_as_float(x[e]);
          if (!isq) {
#pragma unroll
            for (int e = 0; e < 16; ++e) M[(i0 + e) * LD + t] = R[e];
          } else if (out) {
            char *to = smem + Z::OP + (g & 1) * NO * Z::TPART + core_at(t, 0, C) + i0 * 16;
#pragma unroll
            for (int e0 = 0; e0 < 16; e0 += 8) {
              uint32_t w[NO][4];
#pragma unroll
              for (int e = 0; e < 4; ++e) split<NO>(R[e0 + 2 * e], R[e0 + 2 * e + 1], &w[0][e], 4);
#pragma unroll
              for (int k = 0; k < NO; ++k) *reinterpret_cast<uint4 *>(to + k * Z::TPART + e0 * 16) = make_uint4(w[k][0], w[k][1], w[k][2], w[k][3]);
            }
          }
        }
        if (isq) G[t] = r;
        fence_smem_to_async();
        fence_before_sync();
        arrive(&ready[g3()]);
        arrive(&m_ready[g % NM]);
        step();
      }
    }
  } else if (warp < Z::W_MMA) {
    // ---------------------------------------------------------------- inverses
    const int at = tid - Z::W_INV * 32, aw = warp - Z::W_INV, t = at & 63;
    float *Y = reinterpret_cast<float *>(smem + Z::OY);
#pragma unroll 1
    for (int k = 0; k < turns; ++k) {
      if (!take(k)) continue;
#pragma unroll 1
      for (int c = 0; c < chunks; ++c) {
        const int np = padded(c);
        float *M = reinterpret_cast<float *>(smem + Z::OM) + (g % NM) * C * LD;
        wait(&m_ready[g % NM], g / NM);
        // ---- T = (I + M)^-1 in M's place, by columns as M: blocks of 16 on the diagonal (a lane a column, whose later entries are brought up to
        // date as each is known); then twice the block below two inverses, -T_b M_ba T_a
        {
          const int o16 = 16 * aw, col = lane & 15;
          float *m = M + o16 * LD + o16;
          float x[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) x[i] = i == col ? 1.0f : 0.0f;
#pragma unroll
          for (int i = 0; i < 15; ++i) {
#pragma unroll
            for (int k = (i + 1) & ~3; k < 16; k += 4) {
              const float4 y = *reinterpret_cast<const float4 *>(m + i * LD + k);
              if (k > i) x[k] = fmaf(-y.x, x[i], x[k]);
              if (k + 1 > i) x[k + 1] = fmaf(-y.y, x[i], x[k + 1]);
              if (k + 2 > i) x[k + 2] = fmaf(-y.z, x[i], x[k + 2]);
              x[k + 3] = fmaf(-y.w, x[i], x[k + 3]);
            }
          }
          __syncwarp();
          if (lane < 16) {
#pragma unroll
            for (int i = 0; i < 16; i += 4) *reinterpret_cast<float4 *>(m + col * LD + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
          }
        }
        sync4<6>();
        // sums over i of row pairs m(i, rows) x(i)
        if (np > 16) {
          const int oa = (aw >> 1) * 32, ob = oa + 16, col = lane & 15, q = 4 * ((aw & 1) * 2 + (lane >> 4));
          float *y = Y + (aw >> 1) * 16 * LY;
          uint64_t s0 = 0, s1 = 0;
#pragma unroll 8
          for (int i = 0; i < 16; ++i) {
            const ulonglong2 m = *reinterpret_cast<const ulonglong2 *>(M + (oa + i) * LD + ob + q);
            const float x = M[(oa + col) * LD + oa + i];
            fma_pair(s0, m.x, x), fma_pair(s1, m.y, x);
          }
          float2 v0 = pair(s0), v1 = pair(s1);
          y[q * LY + col] = -v0.x, y[(q + 1) * LY + col] = -v0.y, y[(q + 2) * LY + col] = -v1.x, y[(q + 3) * LY + col] = -v1.y;
          sync4<6>();
          s0 = s1 = 0;
#pragma unroll 8
          for (int i = 0; i < 16; ++i) {
            const ulonglong2 m = *reinterpret_cast<const ulonglong2 *>(M + (ob + i) * LD + ob + q);
            const float x = y[i * LY + col];
            fma_pair(s0, m.x, x), fma_pair(s1, m.y, x);
          }
          v0 = pair(s0), v1 = pair(s1);
          *reinterpret_cast<float4 *>(M + (oa + col) * LD + ob + q) = make_float4(v0.x, v0.y, v1.x, v1.y);
          sync4<6>();
        }
        if (np > 32) {
          const int q = 8 * aw;
          uint64_t s[4] = {0, 0, 0, 0};
          auto add = [&](const float *m, float x) {
            const ulonglong2 m0 = *reinterpret_cast<const ulonglong2 *>(m), m1 = *reinterpret_cast<const ulonglong2 *>(m + 4);
            fma_pair(s[0], m0.x, x), fma_pair(s[1], m0.y, x), fma_pair(s[2], m1.x, x), fma_pair(s[3], m1.y, x);
          };
#pragma unroll 1
          for (int i0 = 0; i0 < 32; i0 += 8) {
            const float4 x0 = *reinterpret_cast<const float4 *>(M + lane * LD + i0), x1 = *reinterpret_cast<const float4 *>(M + lane * LD + i0 + 4);
            const float x[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
#pragma unroll
            for (int i = 0; i < 8; ++i) add(M + (i0 + i) * LD + 32 + q, x[i]);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 v = pair(s[i]);
            Y[(q + 2 * i) * LY + lane] = -v.x, Y[(q + 2 * i + 1) * LY + lane] = -v.y;
            s[i] = 0;
          }
          sync4<6>();
#pragma unroll 8
          for (int i = 0; i < 32; ++i) add(M + (32 + i) * LD + 32 + q, Y[i * LY + lane]);
          const float2 v0 = pair(s[0]), v1 = pair(s[1]), v2 = pair(s[2]), v3 = pair(s[3]);
          *reinterpret_cast<float4 *>(M + lane * LD + 32 + q) = make_float4(v0.x, v0.y, v1.x, v1.y);
          *reinterpret_cast<float4 *>(M + lane * LD + 36 + q) = make_float4(v2.x, v2.y, v3.x, v3.y);
          sync4<6>();
        }
        if (g) wait(u_done + 1, g - 1);
#pragma unroll 1
        for (int k = 0; k < 32; k += 8) {
          const int i = (at >> 6) * 32 + k;
          float x[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = M[(i + e) * LD + t];
          uint32_t w[3][4];
#pragma unroll
          for (int e = 0; e < 4; ++e) split<3>(x[2 * e], x[2 * e + 1], &w[0][e], 4);
          char *to = smem + Z::OT + core_at(t, 0, C) + i * 16;
#pragma unroll
          for (int e = 0; e < 3; ++e) *reinterpret_cast<uint4 *>(to + e * Z::TPART) = make_uint4(w[e][0], w[e][1], w[e][2], w[e][3]);
        }
        fence_smem_to_async();
        arrive(t_ready);
        arrive(&m_free[g % NM]);
        step();
      }
    }
  } else if (warp >= Z::W_LOAD) {
    // ---------------------------------------------------------------- rows of the chunks: one warp copies k and q (fp32: the tables' warps do), one v, one o
    const int what = warp - Z::W_LOAD + 3 - Z::LOAD;
    const uint32_t base = smem_u32(smem);
    auto load = [&](int c) {
      if (what == 0) {
        load_x(c, std::integral_constant<int, 1>{}, 0);
      } else {
        constexpr int PIECES = D * ES / 16, PER = 32 / PIECES;             // of a row; rows at once
        static_assert(PIECES <= 32 && C % PER == 0, "rows of v");
        const uint32_t to = base + Z::OV + (g % NV) * Z::VBUF + lane * 16;
        rows(p.v, h, c, lane / PIECES, PER, lane % PIECES * 16, [&](int r, const char *from, bool live) { cp16(to + r * D * ES, from, live ? 16 : 0); });
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
    };
#pragma unroll 1
    for (int k = 0; k < turns; ++k) {
      if (!take(k)) continue;
      if (what == 1 && !(unit[k].slot >> 31)) {            // the state, for the warps that will hold it
        const char *from = reinterpret_cast<const char *>(p.S + ((long)unit[k].slot * p.H + h) * D * D);
        for (int i = lane * 128; i < D * D * 4; i += 32 * 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(from + i));
      }
#pragma unroll 1
      for (int c = 0; c < chunks; ++c) {
        if (what < 2) {
          // v's buffer is free when the outputs written over it have left
          if (what == 0) {
            if (g >= NB) wait(&x_free[at_x()], round_x() - 1);
          } else if (g >= NV) {
            if (out) wait(&o_free[g % NV], g / NV - 1);
            else wait(&x_free[(g - NV) % NB], (g - NV) / NB);   // (v has been read before u is formed)
          }
          load(c);
          fence_smem_to_async();
          arrive(what == 0 ? &x_full[at_x()] : &ready[g3()]);
        } else if (out) {
          // (as many row copies by the bulk-copy unit, 256 bytes each, took 5300 cycles a chunk)
          constexpr int PIECES = D * ES / 16, PER = 32 / PIECES;
          wait(&o_ready[g % NV], g / NV);
          const int nt = tokens(c), first = lane / PIECES, piece = lane % PIECES;
          const char *from = smem + Z::OV + (g % NV) * Z::VBUF + first * D * ES + piece * 16;
          char *to = p.o.p + (b * p.o.sb + (long)(c * C + first) * p.o.st + h * p.o.sh) * ES + piece * 16;
          const long next = PER * p.o.st * ES;
          if (nt == C) {
#pragma unroll 8
            for (int r = 0; r < C; r += PER, to += next) *reinterpret_cast<uint4 *>(to) = *reinterpret_cast<const uint4 *>(from + r * D * ES);
          } else {
#pragma unroll 1
            for (int r = 0; r < C; r += PER, to += next)
              if (r + first < nt) *reinterpret_cast<uint4 *>(to) = *reinterpret_cast<const uint4 *>(from + r * D * ES);
          }
          arrive(&o_free[g % NV]);
        }
        step();
      }
    }
  } else {
    // ---------------------------------------------------------------- products. The warp runs as one, so that descriptors stay in uniform
    // registers; one lane issues.
    uint32_t leader;
    asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(leader));
    const uint32_t base = smem_u32(smem);
    auto all_good = [&]() { return good = __all_sync(0xffffffffu, good); };
    constexpr uint32_t SBO = (D / 8) * 128;
    // Part pairs i < NA, k < NK with i + k <= MOST, smallest first; `one` gets `add` for the first of all (0: its product clears D).
    auto pairs = [&](auto na, auto nk, auto most, uint32_t add, auto one) {
      constexpr int NA = decltype(na)::value, NK = decltype(nk)::value, TOP = decltype(most)::value < NA + NK - 2 ? decltype(most)::value : NA + NK - 2;
#pragma unroll
      for (int sum = TOP; sum >= 0; --sum)
#pragma unroll
        for (int i = 0; i < NA; ++i)
          if (sum - i >= 0 && sum - i < NK) one(i, sum - i, sum == TOP && (i == 0 || sum - i == NK - 1) ? add : 1u);
    };
    using I2 = std::integral_constant<int, 2>;
    using I3 = std::integral_constant<int, 3>;
    using INX = std::integral_constant<int, NX>;
    using INO = std::integral_constant<int, NO>;
    using IMO = std::integral_constant<int, NO - 1>;
    using INS = std::integral_constant<int, NS>;
    using IMS = std::integral_constant<int, NS - 1>;
    using INQ = std::integral_constant<int, NQ>;
    using IMQ = std::integral_constant<int, NQ - 1>;
    const uint64_t x_row = smem_desc(base + Z::OX, 128, SBO), x_col = smem_desc(base + Z::OX, SBO, 128);   // rows, and along their other dimension
    const uint64_t t_row = smem_desc(base + Z::OT, 128, 1024), p_row = smem_desc(base + Z::OP, 128, 1024);
    constexpr uint32_t XB = Z::XBUF >> 4, XP = Z::XPART >> 4, TP = Z::TPART >> 4;
    auto dots = [&](int np) {                            // [k | q] k^T of the chunk at this place
      wait(&x_full[at_x()], round_x());
      if (!all_good()) return;
      fence_after_sync();
      if (leader) {
        const uint32_t id = idesc_n(np);
        const uint64_t x = x_row + at_x() * XB;
        pairs(INX{}, INX{}, I2{}, 0, [&](int i, int k, uint32_t add) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) mma_ss(tmem + Z::D0, x + i * XP + kk * 16, x + k * XP + kk * 16, id, kk ? 1u : add);
        });
        commit(g_done);
      }
    };
    // tokens, padded, of the chunk after chunk c of unit k (c = chunks - 1: of the next unit that has any); 0: none
    auto after = [&](int k, int c) {
      if (c + 1 < chunks) return padded(c + 1);
      for (++k; k < turns; ++k)
        if (unit[k].n > 0) return (min(C, unit[k].n) + 15) & ~15;
      return 0;
    };
    if (p.probe_ns) wait(drain, 0);                      // (not signalled before the block's last commit)
    int np_next = after(-1, 0);
    if (np_next) dots(np_next);
#pragma unroll 1
    for (int k = 0; k < turns && all_good(); ++k) {      // (without products from a wait on that gave up)
      if (!take(k)) continue;
#pragma unroll 1
      for (int c = 0; c < chunks && good; ++c) {
        const int now = g, np = np_next, steps = np / 16;
        np_next = after(k, c);
        const uint32_t id = idesc_n(np);
        const uint32_t buf = at_x();
        const uint64_t x = x_row + buf * XB;
        wait(a1, now);
        if (!all_good()) break;
        fence_after_sync();
        if (leader)
          pairs(INS{}, INX{}, IMS{}, 0, [&](int i, int k, uint32_t add) {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) mma_ts(tmem + Z::W, tmem + Z::a1(i) + 8 * kk, x + k * XP + kk * 16, id, kk ? 1u : add);
          });
        if (leader) commit(w_done);
        auto of_q = [&]() {                                // p (the last one has been read)
          if (now) wait(o_read, now - 1);
          if (!all_good()) return;
          fence_after_sync();
          if (leader) {
            pairs(INQ{}, INX{}, IMQ{}, 0, [&](int i, int k, uint32_t add) {
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk)
                mma_ts(tmem + Z::P, tmem + Z::a1(i) + 8 * kk, x + k * XP + (Z::ROWS >> 4) + kk * 16, id, kk ? 1u : add);
            });
            if (F32) commit(p_done);
          }
        };
        if (F32 && out) of_q();
        if (NB > 1 && np_next) {
          wait(&ready[g3()], r3());                      // (the last dot products have been read)
          step();
          dots(np_next);
        }
        wait(t_ready, now);
        if (!F32 && out && now) wait(o_read, now - 1);     // (u lies where the last outputs did; fp32: q's products have waited for that)
        // (columns t of step kk's tokens s >= 16 kk begin at t = 16 kk; the first two blocks of u need the first two of rhs)
#pragma unroll 1
        for (int r = 0; r < 2; ++r) {
          wait(a2 + r, now);
          if (!all_good()) break;
          fence_after_sync();
          if (leader) {
            pairs(I3{}, I3{}, I2{}, r, [&](int i, int k, uint32_t add) {
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int kk = 2 * r + e;
                if (kk < steps)
                  mma_ts(tmem + Z::D2 + 16 * kk, tmem + Z::a2(i) + 8 * kk, t_row + k * TP + kk * ((2 * 1024 + 256) >> 4), id - kk * (2u << 17), e ? 1u : add);
              }
            });
            commit(u_done + r);
          }
        }
        if (!F32 && out) of_q();
        if (p.write) {
          const uint64_t xc = x_col + buf * XB;
#pragma unroll 1
          for (int r = 0; r < 2; ++r) {
            wait(a3 + r, now);
            if (!all_good()) break;
            fence_after_sync();
            if (leader)
              pairs(I3{}, INX{}, I2{}, r, [&](int i, int k, uint32_t add) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const int kk = 2 * r + e;
                  if (kk < steps) mma_ts(tmem + Z::D3, tmem + Z::a3(i) + 8 * kk, xc + k * XP + kk * (2 * SBO >> 4), idesc(D, 1), e ? 1u : add);
                }
              });
          }
          if (leader) commit(s_done);
        }
        if (leader) commit(&x_free[buf]);
        if (out) {
          wait(a4, now);
          if (!all_good()) break;
          fence_after_sync();
          if (leader) {
            pairs(INO{}, INO{}, IMO{}, 0, [&](int i, int k, uint32_t add) {
#pragma unroll
              for (int kk = 0; kk < C / 16; ++kk)
                if (kk < steps)
                  mma_ts(tmem + Z::D4 + 16 * kk, tmem + Z::a4(i) + 8 * kk, p_row + (now & 1) * NO * TP + k * TP + kk * ((2 * 1024 + 256) >> 4),
                         id - kk * (2u << 17), kk ? 1u : add);
            });
            commit(o_done);
          }
        }
        if (NB == 1 || !np_next) step();
        if (NB == 1 && np_next) dots(np_next);
      }
    }
    if (leader) commit(drain);                           // every product has ended before the block frees its TMEM
    wait_long(drain, 0, failed, WAIT_NS);
    __syncwarp();
  }
  if (!good) atomicOr(p.status, PACE_DELTA_TIMEOUT);
  fence_before_sync();
  __syncthreads();
  if (warp == Z::W_MMA) tmem_dealloc(*tmem_slot, 512);
}

template <int D, bool F32, bool ONE>
cudaError_t launch_chunk(const DeltaArgs &p, long blocks, cudaStream_t s) {
  using Z = Shape<D, F32>;
  const cudaError_t e = smem_opt_in<delta_chunk_kernel<D, F32, ONE>>(Z::SMEM);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg = pdl_config(dim3((unsigned)blocks), dim3(Z::THREADS), Z::SMEM, s, attr);
  return cudaLaunchKernelEx(&cfg, delta_chunk_kernel<D, F32, ONE>, p);
}

template <int D, bool F32>
cudaError_t launch_chunk(DeltaArgs p, cudaStream_t s) {
  const long units = (long)p.batch * p.H, most = p.n_keep && p.n_idx < p.n_tokens ? p.n_idx : p.n_tokens;
  p.sms = device_sm_count();
  if (units <= p.sms || most > CHUNKS_LASTING * C) return launch_chunk<D, F32, true>(p, units, s);
  return launch_chunk<D, F32, false>(p, units > (long)p.sms * UNITS ? (units + UNITS - 1) / UNITS : p.sms, s);
}

}  // namespace delta
}  // namespace pace
