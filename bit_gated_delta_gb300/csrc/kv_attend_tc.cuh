// Attention of many query rows over the quantized KV cache on the 5th-generation tensor cores (bf16 I/O).
//
// A work item is 128 query rows of one KV head (row r = token r/G, head r%G), or two such blocks that share the keys and values.
// Per 64 cached tokens:  S = Q K^T  and  O += P V,  both tcgen05: keys and values dequantized to fp16 in shared memory, Q there too
// (D = 128) or in TMEM, P in TMEM (over the scores it came from); S and O accumulate in TMEM in fp32.
//
// fp16 carries 11 bits, against 8 of bf16, so that held values, queries and weights are rounded to 11 bits; its range is
// kept by exact powers of two: a row of Q is scaled by its largest element, K and V of a tile by its largest group scale (E_k, E_v; in
// tiles with tokens of very different size, of which rows may see or weigh different ones, each token by its own; a group far below the
// largest of its token keeps fewer bits: 11 down to 2^-14 of it, one less for each power of two further). The powers return with the
// scores, and in O as a running exponent per row: the maximum and this exponent together follow the largest of score and value exponent,
// so that large values of no weight take no bits from the others. Scores, maxima, sums and outputs are held in fp32. A tile's weights are
// taken relative to the references so far, without a pass for new ones, while their sum stays below 60,000 (so each fits fp16); else
// the references are found and O rescaled.
//
// Roles (warps): softmax (four a group; thread = row = TMEM lane), four or eight that dequantize, two that copy tiles in (in turn) and
// prepare their scales (one the keys', one the values'), and one a softmax group that issues its products (issued by the softmax warps
// themselves, a prompt chunk took 206 us, not 172). Two softmax groups take turns, so that the tensor cores work on one group's products while the other forms its
// weights: the groups are two row blocks (SHARE, above 128 rows), or even and odd tiles of one block (ALT, joined through TMEM). With
// heads of 256 one group's O fills half of TMEM, and there is one group (ONE). Scores are formed two tiles ahead of the weights.
//
// Bound: at D = 128 a tile of 64 tokens takes 650 cycles of tensor work a block of 128 rows (measured: 49 cycles a product of N = 64
// with both operands in shared memory, 65 one of N = 128), 8192 exponentials (260 cycles a scheduler and group) and 16,384 codes to
// dequantize. SHARE runs at 2150 cycles (1.05 us) a tile for two row blocks, of which the tensor cores work 1300; the dequantizing
// warps, four of which serve both blocks, are what it waits for (eight cost the softmax warps more issue slots and registers than they
// gain). ALT runs at 1800: the chain of scale preparation, dequantization and products through shared memory. Fixed per call about 10 us
// (first look-ups, queries, first tile, outputs), per further item of a block about 8 us.
// Measured (4-bit cache, cold): prompt chunks of 256 tokens, 4 sequences, 32 and 8 heads of 128, over 6000 to 8000 tokens 136 us, 860 TFLOP/s
// of the measured 1880; trees of 25 drafts, 16 sequences, over 2049 to 4096 tokens 63 us (62 before lost halves and the size of context
// tokens were looked at), 64 rows over 8000 tokens 120 us; 7 drafts, 32 sequences of 1000 to 6000 tokens, 16 and 2 heads of 256, 66 us.
// Every wait is bounded; one that gives up sets the status word, and the block leaves after its copies and products have ended.
#pragma once

#include <type_traits>

#include "kv_attend.cuh"

namespace pace {
namespace kv {

enum { TC_SHARE = 0, TC_ALT = 1, TC_ONE = 2 };
constexpr int KVT = 64;               // cached tokens a tile
constexpr int TC_BLOCKS = 160;        // most blocks of a launch (one an SM)
// The fewest tiles a block takes (heads of 128, one sequence of 2000 tokens under a tree: 22 us with 4, 23 with 2, 24 with 8).
constexpr int TC_LEAST = 4;
// An item a block while the longest is so many tiles above an equal share: sharing costs a block the queries, the first tile and the
// outputs of another item, about as many tiles' time as this (eight sequences of up to 2048 tokens under trees, heads of 64: 22 us
// shared, 28 an item a block; sixteen with heads of 128: 71 and 66 us). Heads of 256, with 24 and with 8: 16 sequences of 2000 to 4000
// tokens, 8 KV heads, 40 rows 83 and 93 us; 64 of 300 to 1200, 2 heads 38 and 58; 8 of 500 to 2000, 8 heads, 100 rows 52 and 44.
__host__ __device__ constexpr unsigned tc_extra(int D) { return D == 64 ? 10 : 24; }

template <int D, int BITS, int MODE>
struct TcShape {
  using L = Tile<D, BITS>;
  static constexpr int NWG = MODE == TC_ONE ? 1 : 2;
  static constexpr int NRB = MODE == TC_SHARE ? 2 : 1;                  // row blocks an item
  static constexpr int ROWS = 128 * NRB;
  // dequantized stages (ALT: score tiles are formed four tiles ahead, two a group) and raw ones
  static constexpr int KS = MODE == TC_ALT ? 4 : 2, VS = KS;
  static constexpr int RS = BITS == 4 ? (D == 256 ? 3 : 4) : (D == 256 || (MODE == TC_ALT && D == 128) ? 2 : 4);
  static constexpr int NDEQ = MODE == TC_SHARE ? 4 : 8;                 // dequantizing warps (SHARE: a tile serves two row blocks)
  static constexpr int W_DEQ = 4 * NWG, W_PAR = W_DEQ + NDEQ, W_MMA = W_PAR + 2;
  static constexpr int WARPS = W_MMA + NWG, THREADS = WARPS * 32;
  // TMEM columns: O, two score tiles a group (each later its weights), and Q where it fits beside them; else Q is in shared memory
  static constexpr bool QSMEM = D == 128;
  static constexpr int CO = 0, CS = NWG * D, CQ = CS + NWG * 2 * KVT;
  static_assert(CQ + (QSMEM ? 0 : NRB * D / 2) <= 512, "TMEM");
  // shared memory
  static constexpr int KB = KVT * D * 2;                                // one dequantized tile
  static constexpr int QB = QSMEM ? 128 * D * 2 : 0;                    // one block of queries
  static constexpr int RAW = 2 * L::BYTES;
  static constexpr int OK = 0, OV = OK + KS * KB, OQ = OV + VS * KB, ORAW = OQ + NRB * QB, OPAR = ORAW + RS * RAW;
  static constexpr int PB = BITS == 4 ? 16 : 4;                         // scale (and zero points) of one token and group
  static constexpr int PAR = 2 * L::NG * KVT * PB;                      // of a tile
  static constexpr int OEXP = OPAR + 2 * PAR;                           // exponents [8 tiles][k, v][64] int8
  static constexpr int OHOW = OEXP + 8 * 2 * KVT;                       // bit 0: a tile's tokens have their own; 1, 2: lost halves [8][k, v]
  static constexpr int OML = OHOW + 16;                                 // m, l, exponent of each group's rows (ALT)
  // where each softmax warp turns its rows' outputs, ROWB bytes of a row at a time: the queries' area where there is one
  static constexpr int ROWB = QSMEM ? 128 : 64;
  static constexpr int OOUT = QSMEM ? OQ : OML + (MODE == TC_ALT ? 128 * 24 : 0);
  static constexpr int OUT_GROUP = QSMEM ? NRB * QB / NWG : 4 * 32 * ROWB;   // (ALT: both groups are done when either writes)
  static constexpr int OBAR = QSMEM ? OML + (MODE == TC_ALT ? 128 * 24 : 0) : OOUT + NWG * OUT_GROUP;
  static_assert(OUT_GROUP >= 4 * 32 * ROWB, "outputs");
  static constexpr int NBAR = 2 * RS + 2 * KS + 2 * VS + 7 * NWG + 5;
  static constexpr int OMISC = OBAR + NBAR * 8;                         // raw flags [RS], tmem base
  static constexpr int OCUM = (OMISC + 32 + 15) / 16 * 16;
  static constexpr size_t smem(int batch) { return OCUM + 64 * 4 + (size_t)(batch + 1) * 4 + (size_t)batch * sizeof(Seq); }
  static_assert(OCUM + 256 + 4 + 1024 * 16 <= 227 * 1024, "shared memory");
};
constexpr int JOIN_THREADS = 256;
constexpr int TC_PART_FLOATS = 256 * 130;   // one partial result: 256 rows of 128 + 2 (128 of 256 + 2 are fewer)

__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, int b_mn_major) {
  return (1u << 4) | ((uint32_t)b_mn_major << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
// two fp32 operations at once
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float &a, float &b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ void bar_sync(int id, int count) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(count) : "memory"); }

// Eight 4-bit codes (one word) times their scale: p.x = scale pair, p.y = -(1024 + z), p.z = -(64 + z). The nibble at bit 0 of a half
// under the exponent of 1024 reads 1024 + u, the one at bit 4 reads 1024 + 16 u = 16 (64 + u): both give u - z exactly.
__device__ __forceinline__ uint4 dequant4(uint32_t w, const uint4 &p, uint32_t magic) {
  const uint32_t x = w >> 8;
  return make_uint4(h2mul(h2add(mask_or(w, 0x000F000Fu, magic), p.y), p.x), h2mul(h2fma(mask_or(w, 0x00F000F0u, magic), 0x2C002C00u /* 1/16 */, p.z), p.x),
                    h2mul(h2add(mask_or(x, 0x000F000Fu, magic), p.y), p.x), h2mul(h2fma(mask_or(x, 0x00F000F0u, magic), 0x2C002C00u, p.z), p.x));
}
// Eight 8-bit codes (two words): a byte under the exponent of 1024 reads 1024 + u, u = c + 128.
__device__ __forceinline__ uint4 dequant8(uint32_t w0, uint32_t w1, uint32_t s) {
  const uint32_t off = 0xE480E480u;   // -1152
  return make_uint4(h2mul(h2add(__byte_perm(w0, 0x64646464u, 0x4240), off), s), h2mul(h2add(__byte_perm(w0, 0x64646464u, 0x4341), off), s),
                    h2mul(h2add(__byte_perm(w1, 0x64646464u, 0x4240), off), s), h2mul(h2add(__byte_perm(w1, 0x64646464u, 0x4341), off), s));
}

// 64 visibility bits of the columns of a tile for row t < nn: columns jd0 + c of the new tokens (negative: context).
__device__ __forceinline__ uint64_t visible(const AttendArgs &p, int b, int t, int jd0, int nn) {
  const int T = p.c.n_tokens;
  const int c0 = jd0 < 0 ? min(-jd0, 64) : 0;
  const uint64_t ctx = c0 >= 64 ? ~0ull : (1ull << c0) - 1;
  if (c0 >= 64) return ctx;
  const int j0 = jd0 + c0;                             // first new token of the tile
  const int n = min(64 - c0, nn - j0);                 // columns that hold one
  if (n <= 0) return ctx;
  uint64_t bits;
  if (!p.mask) {
    const int k = t - j0 + 1;
    bits = k <= 0 ? 0 : k >= 64 ? ~0ull : (1ull << k) - 1;
  } else {
    const int words = (T + 31) >> 5, w0 = j0 >> 5, sh = j0 & 31;
    const uint32_t *row = p.mask + ((long)b * T + t) * words;
    const uint32_t a = row[w0], m = w0 + 1 < words ? row[w0 + 1] : 0, z = w0 + 2 < words ? row[w0 + 2] : 0;
    bits = (uint64_t)__funnelshift_r(a, m, sh) | ((uint64_t)__funnelshift_r(m, z, sh) << 32);
  }
  if (n < 64) bits &= (1ull << n) - 1;
  return ctx | (bits << c0);
}

// The item that begins in a block and goes on in later ones, as that block leaves it for the join: sequence (-1: none), head and row
// block, last block, new tokens.
__device__ __forceinline__ int4 *tc_shared(const KvDev &c) { return reinterpret_cast<int4 *>(c.part + (size_t)2 * TC_BLOCKS * TC_PART_FLOATS); }

// Joins the parts of shared items in block order, in a launch of its own behind the attention's: one SM draws about 100 GB/s from
// L2, and parts of 64 to 128 KB that the last of an item's blocks joined by itself took it up to 100 us. A block takes four to
// sixteen rows of an item at a time, a thread one 16-byte piece of a row, eight parts under way.
template <int D, int ROWS>
__global__ void __launch_bounds__(JOIN_THREADS, 4) tc_join_kernel(AttendArgs p, int blocks) {
  const KvDev &c = p.c;
  const int G = c.group, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  static_assert(TC_BLOCKS <= JOIN_THREADS, "a thread looks at a block");
  constexpr int CH = D / 4, SLICE = JOIN_THREADS / CH, SLICES = ROWS / SLICE, U = 8;
  __shared__ int list[TC_BLOCKS], count[JOIN_THREADS / 32];
  pdl_enter();
  const bool mine = tid < blocks && __ldcg(&tc_shared(c)[tid]).x >= 0;
  const unsigned vote = __ballot_sync(0xffffffffu, mine);
  if (lane == 0) count[warp] = __popc(vote);
  __syncthreads();
  int n = 0, before = 0;
  for (int i = 0; i < JOIN_THREADS / 32; ++i) {
    before += i < warp ? count[i] : 0;
    n += count[i];
  }
  if (mine) list[before + __popc(vote & ((1u << lane) - 1))] = tid;
  __syncthreads();
  for (int unit = blockIdx.x; unit < n * SLICES; unit += gridDim.x) {
    const int first = list[unit / SLICES], r = (unit % SLICES) * SLICE + tid / CH, ch = tid % CH;
    const int4 it = __ldcg(&tc_shared(c)[first]);
    const int h = it.y / p.row_blocks, row = (it.y - h * p.row_blocks) * ROWS + r, t = row_token(p, row);
    if (row >= c.n_tokens * G) continue;
    float M = -INFINITY, L = 0.0f;
    float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int i0 = first; i0 <= it.z; i0 += U) {
      float2 e[U];                                         // maximum and sum of the row
      float4 v[U];
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const int i = i0 + k;
        const float *part = c.part + (long)(2 * i + (i == first)) * TC_PART_FLOATS;
        e[k] = make_float2(-INFINITY, 0.0f);
        v[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (i <= it.z) {
          e[k] = __ldcg(reinterpret_cast<const float2 *>(part + ROWS * D + 2 * r));
          v[k] = __ldcg(reinterpret_cast<const float4 *>(part + r * D) + ch);
        }
      }
      float m = M;
#pragma unroll
      for (int k = 0; k < U; ++k) m = fmaxf(m, e[k].x);
      const float f = M == -INFINITY ? 0.0f : exp2_approx(M - m);
      y.x *= f, y.y *= f, y.z *= f, y.w *= f;
      L *= f;
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const float w = e[k].x == -INFINITY ? 0.0f : exp2_approx(e[k].x - m);
        L = fmaf(w, e[k].y, L);
        y.x = fmaf(w, v[k].x, y.x), y.y = fmaf(w, v[k].y, y.y), y.z = fmaf(w, v[k].z, y.z), y.w = fmaf(w, v[k].w, y.w);
      }
      M = m;
    }
    const float inv = t < it.w && L > 0.0f ? 1.0f / L : 0.0f;
    *reinterpret_cast<uint2 *>(p.o.p + (it.x * p.o.sb + (long)t * p.o.st + (long)(h * G + row - t * G) * p.o.sh + ch * 4) * 2) =
        make_uint2(pack_bf16x2(y.x * inv, y.y * inv), pack_bf16x2(y.z * inv, y.w * inv));
  }
}

template <int D, int BITS, int MODE>
__global__ void __launch_bounds__(TcShape<D, BITS, MODE>::THREADS, 1) attend_tc_kernel(AttendArgs p) {
  using S = TcShape<D, BITS, MODE>;
  using L = Tile<D, BITS>;
  using namespace umma;
  constexpr int NG = L::NG, NWG = S::NWG, KS = S::KS, VS = S::VS, RS = S::RS;
  // A row's weights are 2^(score - m + value exponent - E + OFFSET), its sum l counts 2^(score - m + OFFSET): m is the largest score when
  // it was last looked for, m + E - ROOM the largest of score + value exponent. So the token that adds most to the output has a weight of
  // 2^(OFFSET - ROOM), above which fp16 has room for 2^8 more and below which it keeps 11 bits down to 2^-21, whatever the values of tokens
  // that weigh nothing.
  constexpr float ROOM = 3.0f, OFFSET = 10.0f;
  extern __shared__ __align__(128) char smem[];
  const KvDev &c = p.c;
  uint64_t *bar = reinterpret_cast<uint64_t *>(smem + S::OBAR);
  // (s_full, p_ready and pv_done: two a group, taken in turn by its tiles)
  uint64_t *raw_full = bar, *raw_free = raw_full + RS, *k_full = raw_free + RS, *k_free = k_full + KS, *v_full = k_free + KS,
           *v_free = v_full + VS, *s_full = v_free + VS, *p_ready = s_full + 2 * NWG, *pv_done = p_ready + 2 * NWG,
           *q_ready = pv_done + 2 * NWG, *par_full = q_ready + NWG, *par_free = par_full + 2, *drain = par_free + 2;
  int *raw_flags = reinterpret_cast<int *>(smem + S::OMISC);            // [RS]
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(raw_flags + 4);
  unsigned *wsum = reinterpret_cast<unsigned *>(smem + S::OCUM);
  unsigned *cum = wsum + 64;
  Seq *seq = reinterpret_cast<Seq *>(cum + c.batch + 1);
  int8_t *exps = reinterpret_cast<int8_t *>(smem + S::OEXP);
  volatile uint8_t *how = reinterpret_cast<uint8_t *>(smem + S::OHOW);
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);   // (known to be uniform)
  const int G = c.group, T = c.n_tokens;

  if (tid == 0) {
    for (int i = 0; i < RS; ++i) mbar_init(&raw_full[i], 1), mbar_init(&raw_free[i], S::NDEQ);
    for (int i = 0; i < KS; ++i) mbar_init(&k_full[i], S::NDEQ), mbar_init(&k_free[i], S::NRB);
    for (int i = 0; i < VS; ++i) mbar_init(&v_full[i], S::NDEQ), mbar_init(&v_free[i], S::NRB);
    for (int i = 0; i < 2 * NWG; ++i) mbar_init(&s_full[i], 1), mbar_init(&p_ready[i], 4), mbar_init(&pv_done[i], 1);
    for (int i = 0; i < NWG; ++i) mbar_init(&q_ready[i], 4);
    for (int i = 0; i < 2; ++i) mbar_init(&par_full[i], 2), mbar_init(&par_free[i], S::NDEQ);
    mbar_init(drain, NWG);
    mbar_fence_init();
  }
  if (warp == S::W_MMA) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  pdl_enter();
  fence_before_sync();
  const unsigned most = tile_line<KVT>(c, p.items, seq, cum, wsum);      // (its barriers also publish the set-up above)
  fence_after_sync();
  constexpr uint32_t tmem = 0;          // the whole of TMEM is this block's: its first column (a constant keeps addresses uniform)

  unsigned lo, hi;
  const Cuts cuts = make_cuts<KVT>(seq, cum, c.batch, p.items, most, TC_LEAST, 0, tc_extra(D), lo, hi);
  auto at = [&](unsigned pos) { return segment_at<KVT>(seq, cum, p, pos, hi); };
  if (tid == 0) {
    const Segment end = lo < hi ? at(hi - 1) : Segment{};
    const bool on = lo < hi && hi - 1 - end.tile >= lo && end.end < end.tiles;
    tc_shared(c)[blockIdx.x] = on ? make_int4(end.b, end.h * p.row_blocks + end.rb, (int)((hi - 1 - end.tile + end.tiles - 1) / cuts.share), seq[end.b].fresh)
                                  : make_int4(-1, 0, 0, 0);
  }
  // A role whose wait gives up goes on without waiting or touching the tensor cores, but keeps the barriers it shares, so that no
  // other warp is left at one; the others' waits then run out too.
  auto gave_up = [&]() { atomicOr(c.status, PACE_KV_TIMEOUT); };

  if (warp >= S::W_DEQ && warp < S::W_PAR) {
    // ---------------------------------------------------------------- dequantize
    const int dw = warp - S::W_DEQ;
    const uint32_t magic = opaque(0x64006400u);
    int n = 0;
    bool good = true;
    for (unsigned pos = lo; pos < hi;) {
      const Segment sg = at(pos);
      pos += sg.end - sg.tile;
      for (int tile = sg.tile; tile < sg.end; ++tile, ++n) {
        const int rs = n % RS;
        const char *raw = smem + S::ORAW + rs * S::RAW;
        char *par = smem + S::OPAR + (n & 1) * S::PAR;
        good = good && bar_wait(&par_full[n & 1], (n >> 1) & 1);          // (the warps that prepare scales have waited for the tile)
        good = __all_sync(0xffffffffu, good);
        if (!good) continue;
        // codes: warp = 8 or 16 tokens; eight lanes write eight tokens' pieces of one 128-byte core
        constexpr int OCT = 8 / S::NDEQ;
        auto param = [&](int part, int g, int t) {
          const char *at = par + ((part * NG + g) * KVT + t) * S::PB;
          return BITS == 4 ? *reinterpret_cast<const uint4 *>(at) : make_uint4(*reinterpret_cast<const uint32_t *>(at), 0, 0, 0);
        };
        auto put = [&](char *dst, int t, int a, const uint4 &v) {
          *reinterpret_cast<uint4 *>(dst + ((t >> 3) * (D / 8) + a) * 128 + (t & 7) * 16) = v;
        };
        {
          const int ks = n % KS;
          char *dst = smem + S::OK + ks * S::KB;
          constexpr int CHUNKS = BITS == 8 ? D / 16 : D == 64 ? 4 : D / 32;
          uint4 word[OCT][CHUNKS / 4];                        // (read before the wait)
#pragma unroll
          for (int o = 0; o < OCT; ++o)
#pragma unroll
            for (int q = 0; q < CHUNKS; q += 4) {
              const int t = (dw * OCT + o) * 8 + (lane & 7), ch = q + (lane >> 3);
              const char *src = raw + (t >> 5) * L::BYTES + L::kchunk(t & 31, ch);
              if (BITS == 4 && D == 64) {
                const uint2 x = *reinterpret_cast<const uint2 *>(src);
                word[o][q / 4] = make_uint4(x.x, x.y, 0, 0);
              } else {
                word[o][q / 4] = *reinterpret_cast<const uint4 *>(src);
              }
            }
          if (n >= KS) good = good && bar_wait(&k_free[ks], (n / KS - 1) & 1);
          good = __all_sync(0xffffffffu, good);
          if (!good) continue;
#pragma unroll
          for (int o = 0; o < OCT; ++o)
#pragma unroll
            for (int q = 0; q < CHUNKS; q += 4) {
              const int t = (dw * OCT + o) * 8 + (lane & 7), ch = q + (lane >> 3);
              const uint4 w = word[o][q / 4];
              if (BITS == 8) {
                const int g = ch >> 2, a = 8 * g + 2 * (ch & 3);
                const uint32_t s = param(0, g, t).x;
                put(dst, t, a, dequant8(w.x, w.y, s));
                put(dst, t, a + 1, dequant8(w.z, w.w, s));
              } else if (D == 64) {
                const uint4 pr = param(0, 0, t);
                put(dst, t, 2 * ch, dequant4(w.x, pr, magic));
                put(dst, t, 2 * ch + 1, dequant4(w.y, pr, magic));
              } else {
                const int g = 2 * (ch >> 2), a = 8 * g + 2 * (ch & 3);
                const uint4 p0 = param(0, g, t), p1 = param(0, NG > 1 ? g + 1 : g, t);
                put(dst, t, a, dequant4(w.x, p0, magic));
                put(dst, t, a + 1, dequant4(w.y, p0, magic));
                put(dst, t, a + 8, dequant4(w.z, p1, magic));
                put(dst, t, a + 9, dequant4(w.w, p1, magic));
              }
            }
          fence_smem_to_async();
          __syncwarp();
          if (lane == 0) mbar_arrive(&k_full[ks]);
        }
        {
          const int vs = n % VS;
          char *dst = smem + S::OV + vs * S::KB;
          constexpr int UNITS = BITS == 8 ? D / 8 : D == 64 ? 8 : D / 16;
          uint2 word[OCT][UNITS / 4];
#pragma unroll
          for (int o = 0; o < OCT; ++o)
#pragma unroll
            for (int q = 0; q < UNITS; q += 4) {
              const int t = (dw * OCT + o) * 8 + (lane & 7), u = q + (lane >> 3);
              const char *src = raw + (t >> 5) * L::BYTES + L::vunit(t & 31, u);
              if (BITS == 4 && D == 64) word[o][q / 4] = make_uint2(*reinterpret_cast<const uint32_t *>(src), 0);
              else word[o][q / 4] = *reinterpret_cast<const uint2 *>(src);
            }
          if (n >= VS) good = good && bar_wait(&v_free[vs], (n / VS - 1) & 1);
          good = __all_sync(0xffffffffu, good);
          if (!good) continue;
#pragma unroll
          for (int o = 0; o < OCT; ++o)
#pragma unroll
            for (int q = 0; q < UNITS; q += 4) {
              const int t = (dw * OCT + o) * 8 + (lane & 7), u = q + (lane >> 3);
              const uint2 w = word[o][q / 4];
              if (BITS == 8) {
                put(dst, t, u, dequant8(w.x, w.y, param(1, u >> 3, t).x));
              } else if (D == 64) {
                put(dst, t, u, dequant4(w.x, param(1, 0, t), magic));
              } else {
                const int g = 2 * (u >> 3), a = 8 * g + (u & 7);
                put(dst, t, a, dequant4(w.x, param(1, g, t), magic));
                put(dst, t, a + 8, dequant4(w.y, param(1, NG > 1 ? g + 1 : g, t), magic));
              }
            }
          fence_smem_to_async();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&v_full[vs]);
            mbar_arrive(&raw_free[rs]);
            mbar_arrive(&par_free[n & 1]);
          }
        }
      }
    }
    if (!good && lane == 0) gave_up();
  } else if (warp >= S::W_PAR && warp < S::W_MMA) {
    // ---------------------------------------------------------------- copies of tiles; their scales and exponents: lane = token
    // (one warp the keys', one the values')
    const int pw = warp - S::W_PAR, ps = L::pos(lane), vp = L::vpos(lane);
    int n = 0;
    bool good = true;
    // the copying side, RS - 1 tiles ahead, the two warps in turn: segment, storage tiles [at, end) of it, and pool indexes, one a lane:
    // of the 32 from `base` on, and of the 32 after those (their look-up is under way meanwhile)
    const int tpp = c.page / TILE;
    unsigned lpos = lo;
    Segment ls{0, 0, 0, 0, 0, 0};
    int lat = 0, lend = 0, lbase = 0, mytile = -2, later = -2, copied = 0;
    auto look_up = [&](int t) { return t < lend && t * TILE < seq[ls.b].tokens ? tile_index(c, ls.b, ls.h, t, tpp) : -2; };
    auto copy_next = [&]() {
      if (lat >= lend) {
        if (lpos >= hi) return;
        ls = at(lpos);
        lpos += ls.end - ls.tile;
        lat = lbase = 2 * ls.tile;
        lend = 2 * ls.end;
        mytile = look_up(lat + lane);
        later = look_up(lat + 32 + lane);
        if (mytile == -1) atomicOr(c.status, PACE_KV_BAD_PAGE);
      }
      if (lat - lbase >= 32) {
        lbase = lat;
        mytile = later;
        later = look_up(lat + 32 + lane);
        if (mytile == -1) atomicOr(c.status, PACE_KV_BAD_PAGE);
      }
      if ((copied & 1) == pw) {
        const int pa = __shfl_sync(0xffffffffu, mytile, lat - lbase), pb = __shfl_sync(0xffffffffu, mytile, lat - lbase + 1);
        const int stage = copied % RS;
        if (copied >= RS) good = __all_sync(0xffffffffu, good && bar_wait(&raw_free[stage], (copied / RS - 1) & 1));
        if (!good) return;
        if (lane == 0) {
          raw_flags[stage] = (pa >= 0 ? 1 : 0) | (pb >= 0 ? 2 : 0);
          const uint32_t bytes = ((pa >= 0) + (pb >= 0)) * L::BYTES;
          if (bytes) mbar_arrive_expect_tx(&raw_full[stage], bytes);
          else mbar_arrive(&raw_full[stage]);
          char *dst = smem + S::ORAW + stage * S::RAW;
          if (pa >= 0) bulk_g2s(dst, c.pool + (long)pa * L::BYTES, L::BYTES, &raw_full[stage]);
          if (pb >= 0) bulk_g2s(dst + L::BYTES, c.pool + (long)pb * L::BYTES, L::BYTES, &raw_full[stage]);
        }
      }
      ++copied;
      lat += 2;
    };
    for (int i = 0; i < RS - 1; ++i) copy_next();
    for (unsigned pos = lo; pos < hi;) {
      const Segment sg = at(pos);
      pos += sg.end - sg.tile;
      const int tokens = seq[sg.b].tokens;
      for (int tile = sg.tile; tile < sg.end; ++tile, ++n) {
        const int rs = n % RS;
        good = good && bar_wait(&raw_full[rs], (n / RS) & 1);
        if (n >= 2) good = good && bar_wait(&par_free[n & 1], ((n >> 1) - 1) & 1);
        good = __all_sync(0xffffffffu, good);
        const char *raw = smem + S::ORAW + rs * S::RAW;
        char *par = smem + S::OPAR + (n & 1) * S::PAR + pw * NG * KVT * S::PB;
        float s[2][NG], top[2];                           // the lane's tokens: one of each storage tile
        uint32_t z[2][NG];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const char *st = raw + half * L::BYTES;
          const bool live = tile * KVT + half * TILE + lane < tokens && ((raw_flags[rs] >> half) & 1);
          top[half] = 0.0f;
#pragma unroll
          for (int g = 0; g < NG; ++g) {
            const __nv_bfloat16 x = reinterpret_cast<const __nv_bfloat16 *>(st + (pw ? L::VS : L::KS))[g * TILE + ps];
            s[half][g] = live ? __bfloat162float(x) : 0.0f;
            if (BITS == 4) z[half][g] = reinterpret_cast<const uint8_t *>(st + (pw ? L::VZ : L::KZ))[g * TILE + (pw ? vp : ps)];
            top[half] = fmaxf(top[half], s[half][g]);
          }
        }
        // (scales are not negative: their bits order as integers)
        const uint32_t b0 = __float_as_uint(top[0]), b1 = __float_as_uint(top[1]);
        const float all = __uint_as_float(__reduce_max_sync(0xffffffffu, max(b0, b1)));
        // one exponent for the tile keeps eleven bits of every group whose scale is within 2^14 of the largest; where tokens spread by more
        // than 2^12 (the largest may weigh nothing, or be hidden from some rows), each token gets its own
        const uint32_t least = __reduce_min_sync(0xffffffffu, min(b0 ? b0 : 0x7F7FFFFFu, b1 ? b1 : 0x7F7FFFFFu));
        const bool own = all > 4096.0f * __uint_as_float(least);
        // (with the storage tiles that were not brought: those without a page, and past the table's end)
        if (lane == 0) how[(n & 7) * 2 + pw] = (uint8_t)(own | (~raw_flags[rs] & 3) << 1);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int t = half * TILE + lane;
          const float ref = own ? top[half] : all;
          // (zero values have the lowest exponent: they ask for no room beside others)
          const int e = ref > 0.0f ? (int)(__float_as_uint(ref) >> 23) - 127 : pw ? -126 : 0;
          exps[((n & 7) * 2 + pw) * KVT + t] = (int8_t)e;
          const float down = exp2i(-e);                   // (e >= -126: scales are normal numbers or zero)
#pragma unroll
          for (int g = 0; g < NG; ++g) {
            const float sc = s[half][g] * down;
            char *dst = par + (g * KVT + t) * S::PB;
            if (BITS == 4)                                // with -(1024 + z) and -(64 + z) as fp16 pairs
              *reinterpret_cast<uint4 *>(dst) = make_uint4(h2pack(sc, sc), (0xE400u | z[half][g]) * 0x10001u, (0xD400u | (z[half][g] << 4)) * 0x10001u, 0);
            else
              *reinterpret_cast<uint32_t *>(dst) = h2pack(sc, sc);
          }
        }
        __syncwarp();
        if (lane == 0 && good) mbar_arrive(&par_full[n & 1]);
        copy_next();
      }
    }
    if (!good && lane == 0) gave_up();
    for (int i = max(0, copied - RS); i < copied; ++i)    // the warp's copies still in flight land before the block leaves
      if ((i & 1) == pw) bar_wait(&raw_full[i % RS], (i / RS) & 1);
  } else if (warp >= S::W_MMA && warp < S::W_MMA + NWG) {
    // ---------------------------------------------------------------- a group's products. The warp runs as one, so that descriptors and
    // addresses stay in uniform registers; one lane issues. Products run in the order of issue: a score tile may overwrite weights
    // whose product was issued before.
    const int w = warp - S::W_MMA;
    constexpr int STEP = MODE == TC_ALT ? 2 : 1;
    const int i0 = MODE == TC_ALT ? w : 0;
    bool good = true;
    const bool leader = elect_one();
    int ntile = 0, nq = 0, np = 0;                        // tiles of the segments before; segments and tiles of this group
    constexpr uint32_t ID_S = idesc_f16(128, KVT, 0), ID_O = idesc_f16(128, D, 1);
    const uint64_t kdesc = smem_desc(smem_u32(smem) + S::OK, 128, (D / 8) * 128);
    const uint64_t vdesc = smem_desc(smem_u32(smem) + S::OV, (D / 8) * 128, 128);
    const int blk = MODE == TC_SHARE ? w : 0;             // its block of queries
    const uint64_t qdesc = smem_desc(smem_u32(smem) + S::OQ + blk * S::QB, 128, (D / 8) * 128);
    const uint32_t cS = tmem + S::CS + w * 2 * KVT, cO = tmem + S::CO + w * D, cQ = tmem + S::CQ + blk * (D / 2);
    auto ready = [&](uint64_t *b, int phase) {            // (all lanes together: one left behind could miss the phase it waits for)
      good = __all_sync(0xffffffffu, good && bar_wait(b, phase & 1));
      return good;
    };
    auto scores = [&](int tl, int task) {                 // two tiles ahead of the weights
      const int ks = tl % KS;
      if (!ready(&k_full[ks], tl / KS)) return;
      fence_after_sync();
      if (leader) {
        const uint64_t kd = kdesc + (uint64_t)(ks * (S::KB >> 4));
        const uint32_t to = cS + (task & 1) * KVT;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          if (S::QSMEM) mma_ss(to, qdesc + i * (256 >> 4), kd + i * (256 >> 4), ID_S, i ? 1u : 0u);
          else mma_ts(to, cQ + 8 * i, kd + i * (256 >> 4), ID_S, i ? 1u : 0u);
        }
        commit(&s_full[2 * w + (task & 1)]);
        commit(&k_free[ks]);
      }
    };
    for (unsigned pos = lo; pos < hi && good;) {
      const Segment sg = at(pos);
      pos += sg.end - sg.tile;
      const int tiles = sg.end - sg.tile;
      if (i0 < tiles) {
        ready(&q_ready[w], nq++);
        if (good) scores(ntile + i0, np);
        if (good && i0 + STEP < tiles) scores(ntile + i0 + STEP, np + 1);
        for (int i = i0; i < tiles && good; i += STEP, ++np) {
          const int tl = ntile + i, vs = tl % VS;
          ready(&v_full[vs], tl / VS);
          if (!ready(&p_ready[2 * w + (np & 1)], np >> 1)) break;
          fence_after_sync();
          if (leader) {
            const uint64_t vd = vdesc + (uint64_t)(vs * (S::KB >> 4));
            const uint32_t from = cS + (np & 1) * KVT;
#pragma unroll
            for (int k = 0; k < KVT / 16; ++k) mma_ts(cO, from + 8 * k, vd + k * ((2 * (D / 8) * 128) >> 4), ID_O, i == i0 && k == 0 ? 0u : 1u);
            commit(&v_free[vs]);
            commit(&pv_done[2 * w + (np & 1)]);
          }
          if (i + 2 * STEP < tiles) scores(tl + 2 * STEP, np + 2);
        }
      }
      ntile += tiles;
    }
    if (!good && lane == 0) gave_up();
    if (leader) commit(drain);                            // every product has ended before the block frees its TMEM
    bar_wait(drain, 0);
    __syncwarp();
  } else if (warp < S::W_DEQ) {
    // ---------------------------------------------------------------- softmax: thread = row
    const int w = warp >> 2, row_lane = tid & 127;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tO = tmem + lanes + S::CO + w * D;
    const float sl2 = fabsf(p.scale_log2);
    const uint32_t flip = p.scale_log2 < 0.0f ? 0x80008000u : 0u;
    int ntile = 0, task = 0;                              // tiles of the segments before; tiles of this group
    bool good = true;
    for (unsigned pos = lo; pos < hi;) {
      const Segment sg = at(pos);
      pos += sg.end - sg.tile;
      const int tiles = sg.end - sg.tile;
      const int len = seq[sg.b].len, nn = seq[sg.b].fresh;
      const int row = sg.rb * S::ROWS + (MODE == TC_SHARE ? w * 128 : 0) + row_lane;
      const int t = row_token(p, row), hh = sg.h * G + row - t * G;
      const bool in = t < nn;                             // (rows past the new tokens are not read, as they may hold anything, but zeros)
      // ---- the row's query as fp16 over a power of two, for the products (ALT: both groups read the row, each converts half of it)
      float crow = 0.0f;
      if (good) {
        const int blk = MODE == TC_SHARE ? w : 0;
        uint32_t top = 0;
        auto widen = [&](const uint4 &x) {
          const uint32_t v[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) top = max(top, max((v[e] << 16) & 0x7FFF0000u, v[e] & 0x7FFF0000u));
        };
        float down = 0.0f;
        auto power = [&]() {
          const int e = max(min((int)(top >> 23) - 127, 126), -126);
          crow = sl2 * exp2i(e);
          down = exp2i(-e);
        };
        auto conv = [&](uint32_t v) { return h2pack(__uint_as_float(v << 16) * down, __uint_as_float(v & 0xFFFF0000u) * down); };
        if (S::QSMEM) {
          // the block's rows by coalesced asynchronous copies to where the converted ones will lie; then each thread its row in place
          char *block = smem + S::OQ + blk * S::QB;
          constexpr int CH = D / 8, STRIDE = MODE == TC_ALT ? 256 : 128;
          const int r0 = sg.rb * S::ROWS + blk * 128;
#pragma unroll 4
          for (int x = MODE == TC_ALT ? tid : row_lane; x < 128 * CH; x += STRIDE) {
            // (four pieces of eight rows a warp: its writes to shared memory meet no bank twice)
            const int r = (x >> 5) / (CH / 4) * 8 + (x & 7), ch = (x >> 5) % (CH / 4) * 4 + ((x >> 3) & 3), rr = r0 + r, tt = row_token(p, rr);
            const bool ok = tt < nn;
            const char *src = ok ? p.q.p + (sg.b * p.q.sb + (long)tt * p.q.st + (long)(sg.h * G + rr - tt * G) * p.q.sh + ch * 8) * 2 : p.q.p;
            cp_async16(block + (r >> 3) * CH * 128 + ch * 128 + (r & 7) * 16, src, ok);
          }
          asm volatile("cp.async.wait_all;" ::: "memory");
          if (MODE == TC_ALT) bar_sync(2, 256);
          else bar_sync(3 + w, 128);
          char *mine = block + (row_lane >> 3) * CH * 128 + (row_lane & 7) * 16;
          uint4 x[CH];
#pragma unroll
          for (int i = 0; i < CH; ++i) {
            x[i] = *reinterpret_cast<const uint4 *>(mine + i * 128);
            widen(x[i]);
          }
          power();
          if (MODE == TC_ALT) bar_sync(2, 256);           // (both groups have read)
          auto put = [&](auto from, auto to) {
#pragma unroll
            for (int i = decltype(from)::value; i < decltype(to)::value; ++i)
              *reinterpret_cast<uint4 *>(mine + i * 128) = make_uint4(conv(x[i].x ^ flip), conv(x[i].y ^ flip), conv(x[i].z ^ flip), conv(x[i].w ^ flip));
          };
          using std::integral_constant;
          if (MODE != TC_ALT) put(integral_constant<int, 0>{}, integral_constant<int, CH>{});
          else if (w == 0) put(integral_constant<int, 0>{}, integral_constant<int, CH / 2>{});         // (each group half of the row)
          else put(integral_constant<int, CH / 2>{}, integral_constant<int, CH>{});
          fence_smem_to_async();
        } else {
          const char *src = p.q.p + (sg.b * p.q.sb + (long)t * p.q.st + (long)hh * p.q.sh) * 2;
          constexpr int HALF = D > 128 ? 2 : 1;           // (at D = 256 the row waits in TMEM where the converted one will be: registers)
          uint4 x[D / 8 / HALF];
          auto load = [&](int h) {
#pragma unroll
            for (int i = 0; i < D / 8 / HALF; ++i)
              x[i] = in ? reinterpret_cast<const uint4 *>(src)[h * (D / 8 / HALF) + i] : make_uint4(0, 0, 0, 0);
          };
          const uint32_t tQ = tmem + lanes + S::CQ + blk * (D / 2);
          for (int h = 0; h < HALF; ++h) {
            load(h);
#pragma unroll
            for (int i = 0; i < D / 8 / HALF; ++i) widen(x[i]);
            if (HALF > 1) {
#pragma unroll
              for (int i = 0; i < D / 32 / HALF; ++i) {
                uint32_t r[16];
#pragma unroll
                for (int k = 0; k < 16; ++k) r[k] = (&x[4 * i + (k >> 2)].x)[k & 3];
                tmem_st16(tQ + 16 * (h * (D / 32 / HALF) + i), r);
              }
            }
          }
          if (HALF > 1) tmem_wait_st();
          power();
#pragma unroll
          for (int i = 0; i < D / 32; ++i) {
            if (MODE == TC_ALT && (i & 1) != w) continue;                 // (each group half of the row)
            uint32_t r[16];
            if (HALF > 1) {
              tmem_ld16(tQ + 16 * i, r);
              tmem_wait_ld();
            }
#pragma unroll
            for (int k = 0; k < 16; ++k) r[k] = conv((HALF > 1 ? r[k] : (&x[4 * (HALF > 1 ? 0 : i) + (k >> 2)].x)[k & 3]) ^ flip);
            tmem_st16(tQ + 16 * i, r);
          }
          tmem_wait_st();
        }
      } else if (S::QSMEM) {                              // (the barriers of the other side)
        if (MODE == TC_ALT) bar_sync(2, 256), bar_sync(2, 256);
        else bar_sync(3 + w, 128);
      }
      constexpr int STEP = MODE == TC_ALT ? 2 : 1;
      const int i0 = MODE == TC_ALT ? w : 0;
      fence_before_sync();
      if (MODE == TC_ALT) bar_sync(2, 256);               // (each group uses what both wrote)
      __syncwarp();
      if (lane == 0 && good && i0 < tiles) mbar_arrive(&q_ready[w]);
      float m = -INFINITY, l = 0.0f, E = -126.0f;
      bool first = true;
      for (int i = i0; i < tiles; i += STEP, ++task) {
        const int tl = ntile + i, tok0 = (sg.tile + i) * KVT, buf = 2 * w + (task & 1);
        const uint32_t tS = tmem + lanes + S::CS + buf * KVT;
        bool edge = tok0 + KVT > len;                     // new tokens or the end in the tile
        uint64_t vis = edge && in ? visible(p, sg.b, t, tok0 - len, nn) : 0ull;
        good = __all_sync(0xffffffffu, good && bar_wait(&s_full[buf], (task >> 1) & 1));
        fence_after_sync();
        const int8_t *ek = exps + ((tl & 7) * 2) * KVT, *ev = ek + KVT;
        const uint32_t kind = *reinterpret_cast<const volatile uint16_t *>(how + (tl & 7) * 2);
        const bool apart = kind & 0x0101u;                // each token by its own exponents
        if (kind & 6u) {                                  // no row sees a lost half
          vis = (edge ? vis : in ? ~0ull : 0ull) & ((kind & 2u ? 0ull : 0xFFFFFFFFull) | (kind & 4u ? 0ull : ~0ull << 32));
          edge = true;
        }
        bool done = !good;
        // ---- weights by the references at hand: if their sum fits fp16 each of them does, and no maximum is needed
        const bool sees = in && (!edge || vis), unset = sees && m == -INFINITY;   // unset: the long way finds its first references
        if (good && !__any_sync(0xffffffffu, first || apart || unset)) {
          // (values 2^60 below the row's, zeros among them: formed 2^-60 lower for the sum's sake, and here only if all of them are 0 in fp16)
          const float dE = sees ? fmaxf((float)ev[0] - E, -60.0f) : 0.0f, most = dE == -60.0f ? 0x1p-25f : 60000.0f;
          const float cs = crow * exp2i(ek[0]), add = in ? OFFSET + dE - (m == -INFINITY ? 0.0f : m) : -126.0f;
          uint32_t h[2][16];
          const uint64_t cs2 = pack2(cs, cs), ad2 = pack2(add, add);
          uint64_t sum2[2] = {0ull, 0ull};
          auto form = [&](auto masked) {                  // (two copies, so that whole tiles pay nothing for masks)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              uint32_t r[2][16];
              tmem_ld16(tS + 32 * half, r[0]);
              tmem_ld16(tS + 32 * half + 16, r[1]);
              tmem_wait_ld();
              const uint32_t v = (uint32_t)(vis >> (32 * half));
#pragma unroll
              for (int k = 0; k < 16; ++k) {
                float x, y;
                unpack2(fma2(pack2(__uint_as_float(r[k >> 3][(2 * k) & 15]), __uint_as_float(r[k >> 3][(2 * k + 1) & 15])), cs2, ad2), x, y);
                x = exp2_approx(x);
                y = exp2_approx(y);
                if (decltype(masked)::value) {
                  x = v & (1u << (2 * k)) ? x : 0.0f;
                  y = v & (1u << (2 * k + 1)) ? y : 0.0f;
                }
                h[half][k] = h2pack(x, y);
                sum2[k & 1] = add2(sum2[k & 1], pack2(x, y));
              }
            }
          };
          if (edge) form(std::true_type{});
          else form(std::false_type{});
          float sum, odd;
          unpack2(add2(sum2[0], sum2[1]), sum, odd);
          sum += odd;
          if (__all_sync(0xffffffffu, sum <= most)) {
            l = fmaf(sum, exp2_approx(-dE), l);
            tmem_st16(tS, h[0]);
            tmem_st16(tS + 16, h[1]);
            tmem_wait_st();
            done = true;
          }
        }
        // ---- the long way, sixteen columns at a time. own: each token by its own exponents
        auto long_way = [&](auto own) {
          constexpr bool OWN = decltype(own)::value;
          const float cs = fmaxf(crow * exp2i(ek[0]), FLT_MIN);           // (not 0: a masked score is -inf)
          // the largest visible score, and score with its value exponent
          float mx = -INFINITY, rx = -INFINITY;
#pragma unroll 1
          for (int k = 0; k < 4; ++k) {
            uint32_t r[16];
            tmem_ld16(tS + 16 * k, r);
            tmem_wait_ld();
            const uint32_t v = edge ? (uint32_t)(vis >> (16 * k)) : 0xFFFFu;
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const bool see = (v >> e) & 1;
              const float x = __uint_as_float(r[e]) * (OWN ? crow * exp2i(ek[16 * k + e]) : cs);
              mx = fmaxf(mx, see ? x : -INFINITY);
              if (OWN) rx = fmaxf(rx, see ? x + (float)ev[16 * k + e] : -INFINITY);
            }
          }
          if (!OWN) rx = mx + (float)ev[0];
          // set the row's references, and with them what is in O (once the product before has ended)
          const float m2 = fmaxf(m, mx), before_top = m + E - ROOM;
          const float E2 = m2 == m && !(rx > before_top) ? E : fminf(fmaxf(fmaxf(before_top, rx) - m2 + ROOM, -126.0f), 127.0f);
          l *= m == -INFINITY ? 0.0f : exp2_approx(m - m2);
          if (!first) {
            const float f = m == -INFINITY ? 0.0f : exp2_approx((m - m2) + (E - E2));
            const int before = task - 1;
            good = __all_sync(0xffffffffu, bar_wait(&pv_done[2 * w + (before & 1)], (before >> 1) & 1));
            fence_after_sync();
            if (__any_sync(0xffffffffu, f != 1.0f)) {
#pragma unroll 1
              for (int k = 0; k < D / 32; ++k) {
                uint32_t r[2][16];
                tmem_ld16(tO + 32 * k, r[0]);
                tmem_ld16(tO + 32 * k + 16, r[1]);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 32; ++e) r[e >> 4][e & 15] = __float_as_uint(__uint_as_float(r[e >> 4][e & 15]) * f);
                tmem_st16(tO + 32 * k, r[0]);
                tmem_st16(tO + 32 * k + 16, r[1]);
              }
            }
          }
          m = m2;
          E = E2;
          first = false;
          const float dE = OWN ? 0.0f : fmaxf((float)ev[0] - E, -60.0f);
          const float off = OFFSET - (m == -INFINITY ? 0.0f : m), add = off + dE;
          float sum = 0.0f;
#pragma unroll 1
          for (int k = 0; k < 4; ++k) {
            uint32_t r[16], h[8];
            tmem_ld16(tS + 16 * k, r);
            tmem_wait_ld();
            const uint32_t v = edge ? (uint32_t)(vis >> (16 * k)) : 0xFFFFu;
            float x[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const bool see = (v >> e) & 1;
              const float c = OWN ? crow * exp2i(ek[16 * k + e]) : cs;
              x[e] = see ? exp2_approx(fmaf(__uint_as_float(r[e]), c, add)) : 0.0f;
              sum += x[e];
              if (OWN) x[e] = see ? exp2_approx(fmaf(__uint_as_float(r[e]), c, add + ((float)ev[16 * k + e] - E))) : 0.0f;
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) h[e] = h2pack(x[2 * e], x[2 * e + 1]);
            tmem_st8(tS + 8 * k, h);                      // (columns that were read)
          }
          l = fmaf(sum, exp2_approx(-dE), l);
          tmem_wait_st();
        };
        if (!done) {
          if (apart) long_way(std::true_type{});
          else long_way(std::false_type{});
        }
        fence_before_sync();
        __syncwarp();
        if (lane == 0 && good) mbar_arrive(&p_ready[buf]);
      }
      // ---- the segment's result
      if (i0 < tiles) {
        const int before = task - 1;
        good = __all_sync(0xffffffffu, good && bar_wait(&pv_done[2 * w + (before & 1)], (before >> 1) & 1));
        fence_after_sync();
      }
      const bool whole = sg.tile == 0 && sg.end == sg.tiles;
      float *part = c.part + (long)(2 * blockIdx.x + (sg.tile == 0 ? 1 : 0)) * TC_PART_FLOATS;   // (a shared item that starts here is the last)
      const int prow = (MODE == TC_SHARE ? w * 128 : 0) + row_lane;
      float f0 = 1.0f, f1 = 0.0f, M = m, Ls = l, E0 = E, E1 = 0.0f;
      bool two = false;
      if (MODE == TC_ALT) {
        float *mlp = reinterpret_cast<float *>(smem + S::OML) + row_lane * 6;
        mlp[3 * w] = m, mlp[3 * w + 1] = l, mlp[3 * w + 2] = E;
        fence_before_sync();
        bar_sync(2, 256);
        fence_after_sync();
        two = tiles > 1;
        M = fmaxf(mlp[0], mlp[3]);
        f0 = mlp[0] == -INFINITY ? 0.0f : exp2_approx(mlp[0] - M);
        f1 = mlp[3] == -INFINITY ? 0.0f : exp2_approx(mlp[3] - M);
        Ls = f0 * mlp[1] + f1 * mlp[4];
        E0 = mlp[2];
        E1 = mlp[5];
      }
      {                                                    // (outputs of a call whose wait gave up are not to be used)
        const int K0 = MODE == TC_ALT ? w * (D / 32) : 0, K1 = MODE == TC_ALT ? K0 + D / 32 : D / 16;     // (ALT: each group half of the columns)
        const uint32_t tO0 = tmem + lanes + S::CO + (MODE == TC_ALT ? 0 : w * D);
        // (held values reach 2^120: beyond 2^40 their weighted sums are formed 2^64 smaller, and a part is left so, under a reference 64 higher)
        const float high = fmaxf(E0, E1) > 40.0f ? 64.0f : 0.0f;
        const float inv = t < nn && Ls > 0.0f ? exp2_approx(high) / Ls : 0.0f;
        const float g0 = f0 * exp2_approx(E0 - high), g1 = f1 * exp2_approx(E1 - high);
        auto columns = [&](int k, float (&y)[16]) {       // columns 16k .. of the row
          uint32_t r[16], r1[16];
          tmem_ld16(tO0 + 16 * k, r);
          if (MODE == TC_ALT && two) tmem_ld16(tO0 + D + 16 * k, r1);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            y[e] = __uint_as_float(r[e]) * g0;
            if (MODE == TC_ALT && two) y[e] = fmaf(__uint_as_float(r1[e]), g1, y[e]);
          }
        };
        // through shared memory, so that rows leave in whole lines (or half lines): 16-byte piece i of a row lies at i ^ swizzle
        constexpr int PC = S::ROWB / 16;
        // (where queries lie, each group within its own: the other's products may still read theirs)
        char *area = smem + S::OOUT + w * S::OUT_GROUP + (warp & 3) * 32 * S::ROWB;
        auto slot = [&](int r, int i) { return area + r * S::ROWB + (i ^ (PC == 8 ? r & 7 : (r >> 1) & 3)) * 16; };
        const int r0 = (MODE == TC_SHARE ? w * 128 : 0) + (warp & 3) * 32;
        auto exchange = [&](const uint4 *z, auto &&store) {
          __syncwarp();                                   // the columns before have left
#pragma unroll
          for (int i = 0; i < PC; ++i) *reinterpret_cast<uint4 *>(slot(lane, i)) = z[i];
          __syncwarp();
#pragma unroll 4
          for (int x = lane; x < 32 * PC; x += 32) store(r0 + x / PC, x % PC, *reinterpret_cast<const uint4 *>(slot(x / PC, x % PC)));
        };
        if (whole) {
#pragma unroll 1
          for (int k = K0; k < K1; k += PC / 2) {
            uint4 z[PC];
#pragma unroll
            for (int j = 0; j < PC / 2; ++j) {
              float y[16];
              columns(k + j, y);
#pragma unroll
              for (int h = 0; h < 2; ++h)
                z[2 * j + h] = make_uint4(pack_bf16x2(y[8 * h] * inv, y[8 * h + 1] * inv), pack_bf16x2(y[8 * h + 2] * inv, y[8 * h + 3] * inv),
                                          pack_bf16x2(y[8 * h + 4] * inv, y[8 * h + 5] * inv), pack_bf16x2(y[8 * h + 6] * inv, y[8 * h + 7] * inv));
            }
            exchange(z, [&](int r, int i, const uint4 &v) {
              const int rr = sg.rb * S::ROWS + r, tt = row_token(p, rr);
              if (rr < T * G)
                *reinterpret_cast<uint4 *>(p.o.p + (sg.b * p.o.sb + (long)tt * p.o.st + (long)(sg.h * G + rr - tt * G) * p.o.sh + 16 * k + 8 * i) * 2) = v;
            });
          }
        } else {
#pragma unroll 1
          for (int k = K0; k < K1; k += PC / 4) {
            uint4 z[PC];
#pragma unroll
            for (int j = 0; j < PC / 4; ++j) {
              float y[16];
              columns(k + j, y);
#pragma unroll
              for (int h = 0; h < 4; ++h)
                z[4 * j + h] = make_uint4(__float_as_uint(y[4 * h]), __float_as_uint(y[4 * h + 1]), __float_as_uint(y[4 * h + 2]), __float_as_uint(y[4 * h + 3]));
            }
            exchange(z, [&](int r, int i, const uint4 &v) { *reinterpret_cast<uint4 *>(part + r * D + 16 * k + 4 * i) = v; });
          }
        }
        if (!whole && (MODE != TC_ALT || w == 0)) {
          part[S::ROWS * D + 2 * prow] = M + high;
          part[S::ROWS * D + 2 * prow + 1] = Ls * exp2_approx(-high);
        }
      }
      fence_before_sync();
      if (NWG == 2) bar_sync(2, 256);                     // both groups have read what the next segment overwrites
      ntile += tiles;
    }
    if (!good && lane == 0) gave_up();
  }
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  if (warp == S::W_MMA) tmem_dealloc(*tmem_slot, 512);
}

template <int D, int BITS, int MODE>
cudaError_t launch_attend_tc(AttendArgs a, cudaStream_t s) {
  using S = TcShape<D, BITS, MODE>;
  constexpr auto K = attend_tc_kernel<D, BITS, MODE>;
  static_assert(S::ROWS * (D + 2) <= TC_PART_FLOATS, "the work area holds every shape's partial results");
  const size_t smem = S::smem(a.c.batch);
  cudaError_t e = smem_opt_in<K>(227 * 1024);
  if (e != cudaSuccess) return e;
  a.row_blocks = (a.c.n_tokens * a.c.group + S::ROWS - 1) / S::ROWS;
  return by_batches(a, KVT, [&](const AttendArgs &part, long line) {
    long grid = std::min((long)device_sm_count(), (long)TC_BLOCKS);
    grid = std::min(grid, line);
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg = pdl_config(dim3((unsigned)grid), dim3(S::THREADS), smem, s, attr);
    cudaError_t e = cudaLaunchKernelEx(&cfg, K, part);
    if (e != cudaSuccess) return e;
    const cudaLaunchConfig_t join = pdl_config(dim3((unsigned)device_sm_count() * 4), dim3(JOIN_THREADS), 0, s, attr);
    return cudaLaunchKernelEx(&join, tc_join_kernel<D, S::ROWS>, part, (int)grid);
  });
}

}  // namespace kv
}  // namespace pace
