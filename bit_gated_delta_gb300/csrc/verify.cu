// Verification of drafted tokens against the target's probabilities (pace_serve.h).
//
// A cluster of blocks takes a sequence, each block a stretch of the vocabulary, each warp a stretch of that. The walk over the nodes needs p and q
// at the drafts only, which are fetched for all nodes at once; every block walks by itself. The rows are read where the walk needs a sum:
// after a refused draft (R = max(R - q Z, 0), whose sum is the next Z) and for the next token. So a chain reads one row of p and q
// a sequence, whatever its length. The next token is found by the prefix of the blocks' sums, of the warps', and in one warp of the tokens.
//
// Sums in fixed point. A value r in 0..1 enters as two integers: the upper from the bits of r + 1 (units of 2^-23, exact), the rest
// from the bits of rest + 1.5 * 2^-23 (units of 2^-46; from 2^17 tokens on as much larger that a row of ones stays below 2^63: 2^-45 up
// to 2^18 - 1 tokens). Differences p - q carry their rounding error along (it is exact in fp32), so that sums have the accuracy of
// 64-bit floating point at the fp32 rate (the fp64 pipe is a 64th of it), and no order changes them.
//
// Bound by the latency of the rows' loads (16 a thread under way): 64 chains of 7 drafts over 131,072 fp32 tokens, 67 MB, 36 us, 1.9 TB/s (rows in L2 28);
// one over 8,192 tokens 8 us, dependent loads and a cluster barrier. Each refused sibling with others behind it is a pass over the rows: trees of 25 nodes
// against draft probabilities, 16 over 50,001 tokens 26 us, 64 over 131,072 tokens 73.
#include <cooperative_groups.h>

#include "serve_internal.h"

namespace cg = cooperative_groups;

namespace pace {
namespace verify {

constexpr int NODES = PACE_VERIFY_MAX_NODES;
constexpr int THREADS = 512, WARPS = THREADS / 32;
constexpr int MAX_BLOCKS = 8;                            // of a cluster
constexpr int UNROLL = 8;                                // tokens a lane has under way
constexpr int SPAN = 32 * UNROLL, MARKS = 32;            // tokens of a step of a warp; prefixes that a warp keeps

template <bool F32>
__device__ __forceinline__ float prob(const char *row, long v) {
  // clamped to 0..1, NaN is 0
  return __saturatef(F32 ? __ldg(reinterpret_cast<const float *>(row) + v)
                         : __bfloat162float(__ldg(reinterpret_cast<const __nv_bfloat16 *>(row) + v)));
}

// What refused drafts left of one token: R = p, then R = max(R - q Z_i, 0) for the Z of each refusal, as a sum of two floats.
struct Rest {
  float r, e;
};
struct Factor {
  float hi, lo;                                          // Z of a refusal
};
__device__ __forceinline__ Rest first_rest(float p, float q) {       // Z = 1
  const float r = p - q;
  if (!(r > 0.0f)) return Rest{0.0f, 0.0f};
  return Rest{r, (p - r) - q};                           // (p >= q: the error of the difference)
}
__device__ __forceinline__ Rest next_rest(Rest x, float q, Factor z) {
  const float m = __fmul_rn(q, z.hi), em = fmaf(q, z.lo, fmaf(q, z.hi, -m));
  const float s = __fadd_rn(x.r, -m), b = __fadd_rn(s, -x.r);
  const float err = __fadd_rn(__fadd_rn(x.r, -__fadd_rn(s, -b)), -__fadd_rn(m, b));
  const float e = __fadd_rn(err, __fadd_rn(x.e, -em)), r = __fadd_rn(s, e);
  if (!(r > 0.0f)) return Rest{0.0f, 0.0f};
  return Rest{r, __fadd_rn(e, -__fadd_rn(r, -s))};
}

// Units of sums over a vocabulary: 2^-(23 + shift).
struct Units {
  int shift;
  float m;                                               // 1.5 * 2^-shift: neighbours are a unit apart
  double one;                                            // a unit
  __device__ __forceinline__ explicit Units(int vocab) {
    shift = 23 - max(0, 32 - __clz(vocab) - 17);
    m = __uint_as_float((127 - shift) << 23 | 0x400000);
    one = __hiloint2double((1023 - 23 - shift) << 20, 0);
  }
};
// The value as upper (2^-23) and lower part (units).
__device__ __forceinline__ void units(Rest x, const Units &z, uint32_t &hi, int &lo) {
  const float t = __fadd_rn(x.r, 1.0f);
  hi = __float_as_uint(t) - 0x3F800000u;
  const float rest = __fadd_rn(__fadd_rn(x.r, -__fadd_rn(t, -1.0f)), x.e);
  lo = (int)(__float_as_uint(__fadd_rn(rest, z.m)) - __float_as_uint(z.m));
}
__device__ __forceinline__ int64_t to_units(Rest x, const Units &z) {
  uint32_t hi;
  int lo;
  units(x, z, hi, lo);
  return ((int64_t)hi << z.shift) + lo;
}

struct Walk {               // shared by the block
  int tok[NODES], par[NODES], path[NODES];
  float p[NODES], q[NODES], u[NODES];                    // at each draft, in its parent's rows
  Factor z[NODES];                                       // of the refusals at the node so far
  int refused[NODES];                                    // those drafts
  int64_t warp_sum[WARPS];
  int64_t mark[WARPS][MARKS];                            // sums of a warp's groups of steps
  int64_t block_sum[2][MAX_BLOCKS];
  int node, kept, refusals, more;                        // where the walk is; whether it goes on after the sum
  double Z;
};

// R of the tokens v, v + 32, .. below hi at the walk's node, in units.
template <bool F32, bool Q>
__device__ __forceinline__ void step(const Walk &w, const Units &z, const char *prow, const char *qrow, int v, int hi, int refusals, uint32_t (&up)[UNROLL],
                                     int (&down)[UNROLL]) {
  float p[UNROLL], q[UNROLL];
#pragma unroll
  for (int k = 0; k < UNROLL; ++k) {
    p[k] = v + 32 * k < hi ? prob<F32>(prow, v + 32 * k) : 0.0f;
    q[k] = Q && refusals > 0 && v + 32 * k < hi ? prob<F32>(qrow, v + 32 * k) : 0.0f;
  }
#pragma unroll
  for (int k = 0; k < UNROLL; ++k) {
    Rest x{p[k], 0.0f};
    if (Q && refusals > 0) {
      x = first_rest(p[k], q[k]);
      for (int i = 1; i < refusals; ++i) x = next_rest(x, q[k], w.z[i]);
    }
    units(x, z, up[k], down[k]);
  }
}

template <bool F32, bool Q>
__global__ void __launch_bounds__(THREADS) verify_kernel(const VerifyArgs a, int blocks) {
  __shared__ Walk w;
  const Units z(a.vocab);
  cg::cluster_group cluster = cg::this_cluster();
  if (blocks > 1) cluster.barrier_arrive();              // (a block has begun: others may write to its shared memory)
  pdl_enter();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.x / blocks, part = blockIdx.x - b * blocks;
  const int n = a.n_new ? min(max(a.n_new[b], 0), a.nodes) : a.nodes;
  const int es = F32 ? 4 : 2;
  const char *pb = a.p.p + b * a.p.sb * es, *qb = Q ? a.q.p + b * a.q.sb * es : nullptr;
  auto prow = [&](int i) { return pb + i * a.p.st * es; };
  auto qrow = [&](int i) { return qb + i * a.q.st * es; };

  // the drafts
  const int words = (a.nodes + 31) >> 5;
  for (int i = tid; i < n; i += THREADS) {
    const int y = a.tokens[(long)b * a.nodes + i];
    const bool known = y >= 0 && y < a.vocab;
    int par = i - 1;
    if (a.mask && i > 0) {
      const uint32_t *row = a.mask + ((long)b * a.nodes + i) * words;
      par = -1;
      for (int k = i >> 5; k >= 0 && par < 0; --k) {
        uint32_t m = row[k];
        if (k == i >> 5) m &= (1u << (i & 31)) - 1;
        if (m) par = k * 32 + 31 - __clz(m);
      }
    }
    w.tok[i] = known ? y : -1;
    w.par[i] = par;
    w.u[i] = a.u[(long)b * a.nodes + i];
    w.p[i] = i > 0 && par >= 0 && known ? prob<F32>(prow(par), y) : 0.0f;
    w.q[i] = !Q ? 1.0f : i > 0 && par >= 0 && known ? prob<F32>(qrow(par), y) : 0.0f;
  }
  if (tid == 0) w.node = 0, w.kept = 1, w.refusals = 0, w.Z = 1.0, w.path[0] = 0;
  __syncthreads();

  // this block's and warp's tokens
  const int per_block = (a.vocab + blocks - 1) / blocks, v0 = min(part * per_block, a.vocab), v1 = min(v0 + per_block, a.vocab);
  const int per_warp = ((v1 - v0 + WARPS - 1) / WARPS + 31) / 32 * 32, lo = min(v0 + warp * per_warp, v1), hi = min(lo + per_warp, v1);
  const int group = max(1, (per_warp + MARKS * SPAN - 1) / (MARKS * SPAN));       // steps a mark covers
  int turn = 0;
  int64_t total = 0;
  if (blocks > 1) cluster.barrier_wait();
  bool whole = false;                                    // nothing was left: the node's own row counts
  int tried = 0;                                         // drafts up to this one are settled (warp 0)
  while (n > 0) {
    // ---- walk until a sum is wanted: that of a refused draft with others behind it (more), or the next token's
    if (warp == 0 && !whole) {
      int node = w.node, refusals = w.refusals, kept = w.kept;
      double Z = w.Z;
      auto next_draft = [&]() {                          // of the node; n where there is none
        for (int k = tried / 32 * 32; k < n; k += 32) {
          const int j = k + lane;
          const unsigned m = __ballot_sync(0xffffffffu, j > tried && j < n && w.par[j] == node);
          if (m) return k + __ffs(m) - 1;
        }
        return n;
      };
      int i = next_draft();
      bool more = false;
      while (i < n && !more) {
        tried = i;
        const int y = w.tok[i];
        double R = w.p[i];                               // what the refusals before left of y
        bool less;
        if (Q && refusals == 0) {                        // (64 bits only where 32 leave it open: that pipe is slow)
          const float x = w.u[i] * w.q[i], y32 = w.p[i];
          less = x < y32;
          if (!(fabsf(x - y32) > 1e-6f * y32)) less = (double)w.u[i] * (double)w.q[i] < R;
        } else {
          const double q = w.q[i];
          if (Q) {
            for (int k = 0; k < refusals; ++k) R = fmax(R - q * ((double)w.z[k].hi + (double)w.z[k].lo), 0.0);
          } else {
            for (int k = 0; k < refusals; ++k)
              if (w.refused[k] == y) R = 0.0;
          }
          less = (double)w.u[i] * q * Z < R;
        }
        const bool keep = y >= 0 && less, refuse = y >= 0 && !keep;
        __syncwarp();
        if (lane == 0) {
          if (keep) w.path[kept] = i;
          if (refuse) {
            w.refused[refusals] = y;
            w.z[refusals] = Factor{(float)Z, (float)(Z - (double)(float)Z)};
          }
        }
        __syncwarp();
        if (keep) node = i, refusals = 0, Z = 1.0, ++kept;
        i = next_draft();
        if (refuse) {
          ++refusals;
          if (Q) more = i < n;
          else Z = fmax(Z - R, 0.0);
        }
      }
      if (lane == 0) w.node = node, w.refusals = refusals, w.kept = kept, w.Z = Z, w.more = more;
    }
    __syncthreads();
    // ---- the sum of R over the vocabulary
    const int node = w.node, refusals = whole ? 0 : w.refusals;
    const bool more = !whole && w.more;
    const char *pr = prow(node), *qr = Q ? qrow(node) : nullptr;
    // values of a step of SPAN tokens from v0 on, lane by lane within rows of 32
    int64_t sum = 0;
    for (int g = 0; g < MARKS; ++g) {
      const int g0 = lo + g * group * SPAN, g1 = min(g0 + group * SPAN, hi);
      if (g0 >= hi) break;
      int64_t part_sum = 0;
      for (int v = g0; v < g1; v += SPAN) {
        uint32_t h[UNROLL];
        int l[UNROLL];
        step<F32, Q>(w, z, pr, qr, v + lane, hi, refusals, h, l);
        uint32_t up = 0;
        int down = 0;
#pragma unroll
        for (int k = 0; k < UNROLL; ++k) up += h[k], down += l[k];
        part_sum += ((int64_t)up << z.shift) + down;
      }
#pragma unroll
      for (int m = 16; m > 0; m >>= 1) part_sum += __shfl_xor_sync(0xffffffffu, part_sum, m);
      sum += part_sum;
      if (lane == 0) w.mark[warp][g] = part_sum;
    }
    if (!Q && lane == 0)                                 // refused tokens count as zero (once each)
      for (int i = 0; i < refusals; ++i) {
        const int y = w.refused[i];
        bool again = y < lo || y >= hi;
        for (int k = 0; k < i && !again; ++k) again = w.refused[k] == y;
        if (!again) {
          const int64_t x = to_units(Rest{prob<F32>(pr, y), 0.0f}, z);
          sum -= x;
          w.mark[warp][(y - lo) / (group * SPAN)] -= x;
        }
      }
    if (lane == 0) w.warp_sum[warp] = sum;
    __syncthreads();
    if (tid < blocks) {
      int64_t s = 0;
      for (int i = 0; i < WARPS; ++i) s += w.warp_sum[i];
      *cluster.map_shared_rank(&w.block_sum[turn][part], tid) = s;
    }
    if (blocks > 1) cluster.sync();
    else __syncthreads();
    total = 0;
    for (int i = 0; i < blocks; ++i) total += w.block_sum[turn][i];
    turn ^= 1;
    if (!more) {
      if (total > 0 || refusals == 0) break;
      whole = true;
    } else if (tid == 0) {
      w.Z = (double)total * z.one;
    }
    __syncthreads();
  }

  // ---- the token that the prefix passes u_0 of the sum at
  if (n > 0 && total > 0) {
    const int node = w.node, refusals = whole ? 0 : w.refusals;
    const char *pr = prow(node), *qr = Q ? qrow(node) : nullptr;
    int64_t at = min((int64_t)(fmax((double)w.u[0], 0.0) * (double)total), total - 1);   // the first prefix above it
    const int64_t *sums = w.block_sum[turn ^ 1];
    for (int i = 0; i < part; ++i) at -= sums[i];
    if (at >= 0 && at < sums[part]) {
      int64_t s = 0;
      for (int i = 0; i < warp; ++i) s += w.warp_sum[i];
      at -= s;
      if (at >= 0 && at < w.warp_sum[warp]) {
        // the group of steps, the step, the row of 32, the lane
        // (bounded for rows that change under the call, whose sums do not agree)
        int g = 0;
        while (g < MARKS - 1 && at >= w.mark[warp][g]) at -= w.mark[warp][g++];
        int v = -1;
        for (int v0 = lo + g * group * SPAN; v < 0 && v0 < hi; v0 += SPAN) {
          uint32_t h[UNROLL];
          int l[UNROLL];
          step<F32, Q>(w, z, pr, qr, v0 + lane, hi, refusals, h, l);
#pragma unroll
          for (int k = 0; k < UNROLL; ++k) {
            int64_t mine = ((int64_t)h[k] << z.shift) + l[k];
            if (!Q)
              for (int i = 0; i < refusals; ++i)
                if (w.refused[i] == v0 + 32 * k + lane) mine = 0;
            int64_t upto = mine;
#pragma unroll
            for (int m = 1; m < 32; m <<= 1) {
              const int64_t y = __shfl_up_sync(0xffffffffu, upto, m);
              if (lane >= m) upto += y;
            }
            const unsigned past = __ballot_sync(0xffffffffu, upto > at);
            if (v < 0) {
              if (past) v = v0 + 32 * k + __ffs(past) - 1;
              else at -= __shfl_sync(0xffffffffu, upto, 31);
            }
          }
        }
        if (lane == 0) a.next[b] = v < 0 ? hi - 1 : v;
      }
    }
  }
  if (part == 0) {
    for (int i = tid; i < a.nodes; i += THREADS) a.idx[(long)b * a.nodes + i] = n > 0 ? w.path[min(i, w.kept - 1)] : 0;
    if (tid == 0) {
      a.n_keep[b] = n > 0 ? w.kept : 0;
      if (n == 0 || total <= 0) a.next[b] = -1;
    }
  }
}

template <bool F32, bool Q>
cudaError_t launch(const VerifyArgs &a, int blocks, cudaStream_t s) {
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = pdl_config(dim3((unsigned)(a.batch * blocks)), dim3(THREADS), 0, s, attr);
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)blocks;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, verify_kernel<F32, Q>, a, blocks);
}

}  // namespace verify
}  // namespace pace

cudaError_t pace_launch_verify(const VerifyArgs &a, cudaStream_t s) {
  using namespace pace::verify;
  // blocks a sequence: as many as two a multiprocessor hold, but no shorter stretches than 2048 tokens
  int blocks = 1;
  while (blocks < MAX_BLOCKS && a.batch * blocks * 2 <= 2 * pace::device_sm_count() && a.vocab / (blocks * 2) >= 2048) blocks *= 2;
  if (a.io == PACE_IO_F32) return a.q.p ? launch<true, true>(a, blocks, s) : launch<true, false>(a, blocks, s);
  return a.q.p ? launch<false, true>(a, blocks, s) : launch<false, false>(a, blocks, s);
}
