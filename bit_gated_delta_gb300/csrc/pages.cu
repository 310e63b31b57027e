// Pages of the caches (pace_serve.h): rows that share, take and give back pages, renumbering, and the copying of pages.
//
// The bookkeeping calls move a few integers a row; what they cost is their chain of dependent loads and barriers, so each is one
// launch (compaction two), with the loads that do not depend on one another issued together: for 256 rows of 128 columns select takes 4.4 us,
// take (eight tokens a row) and select 10; compaction of 8,192 pages 10. take is made for steps of drafts: a row's cells are read and filled one after
// the other (84 ns each in a row alone), so that the pages of 64 prompts of 8,192 tokens (pages of 64) take 43 us, those of one of 131,072 (of 32) 343. Copies are bound by bytes: 1,658 pages of 135 kB in 71 us, 6.3 TB/s.
#include <limits.h>

#include "serve_internal.h"

namespace pace {
namespace pages {

__device__ __forceinline__ int covering(int tokens, int page) { return tokens <= 0 ? 0 : (int)(((unsigned)tokens + page - 1) / (unsigned)page); }

// ---- select ---------------------------------------------------------------------------------------------------------------
// A block takes eight columns of the table (one 32-byte sector of each row): it reads them whole, then writes them whole, so that rows
// may trade places. The lengths are written by the last block to have read them.
constexpr int SEL_THREADS = 256, SEL_COLS = 8;

__global__ void __launch_bounds__(SEL_THREADS) select_kernel(const PagesDev p, int batch, int32_t *table, int cols, int32_t *lens,
                                                             const int32_t *src) {
  __shared__ int32_t cell[PACE_KV_MAX_BATCH * SEL_COLS];
  __shared__ int32_t from[PACE_KV_MAX_BATCH], len[PACE_KV_MAX_BATCH];
  __shared__ bool last;
  pdl_enter();
  const int tid = threadIdx.x, c0 = blockIdx.x * SEL_COLS;
  int bad = 0;
  for (int b = tid; b < batch; b += SEL_THREADS) {
    int f = src ? src[b] : b;
    if (f < -1 || f >= batch) {
      bad |= PACE_PAGES_BAD_ROW;
      f = b;
    }
    from[b] = f;
    len[b] = f < 0 ? 0 : lens[f];
  }
  for (int i = tid; i < batch * SEL_COLS; i += SEL_THREADS) {
    const int b = i / SEL_COLS, c = c0 + i % SEL_COLS;
    int x = c < cols ? table[(long)b * cols + c] : -1;
    if (x < -1 || x >= p.n_pages) {
      bad |= PACE_PAGES_BAD_CELL;
      x = -2;                                            // holds no page, and has to be written
    }
    cell[i] = x;
  }
  __syncthreads();
  if (tid == 0) {
    __threadfence();
    last = atomicAdd(p.status + 1, 1) == (int)gridDim.x - 1;
  }
  for (int i = tid; i < batch * SEL_COLS; i += SEL_THREADS) {
    const int b = i / SEL_COLS, c = c0 + i % SEL_COLS, f = from[b], old = cell[i];
    if (c >= cols) continue;
    int x = f >= 0 && c < covering(len[b], p.page) ? cell[f * SEL_COLS + i % SEL_COLS] : -1;
    if (x < 0) x = -1;
    if (x == old) continue;
    table[(long)b * cols + c] = x;
    if (x >= 0) atomicAdd(p.refs + x, 1);
    if (old >= 0) atomicAdd(p.refs + old, -1);
  }
  if (bad && blockIdx.x == 0) atomicOr(p.status, bad);
  else if (bad & PACE_PAGES_BAD_CELL) atomicOr(p.status, PACE_PAGES_BAD_CELL);
  __syncthreads();
  if (last) {                                            // every block has read the lengths
    if (src)
      for (int b = tid; b < batch; b += SEL_THREADS) lens[b] = len[b];
    if (tid == 0) p.status[1] = 0;
  }
}

// ---- take, compact: one block ------------------------------------------------------------------------------------------------
constexpr int ONE = 1024;
constexpr int PER = 16;                                  // pages a thread looks at in one go (four loads of four)

// Exclusive prefix of x over the block, and the sum.
__device__ __forceinline__ int block_prefix(int x, int *warp_sum, int &total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int y = x;
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const int z = __shfl_up_sync(0xffffffffu, y, m);
    if (lane >= m) y += z;
  }
  __syncthreads();                                       // (the sums of the call before have been read)
  if (lane == 31) warp_sum[warp] = y;
  __syncthreads();
  int s = lane < ONE / 32 ? warp_sum[lane] : 0;
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const int z = __shfl_up_sync(0xffffffffu, s, m);
    if (lane >= m) s += z;
  }
  total = __shfl_sync(0xffffffffu, s, 31);
  const int before = __shfl_sync(0xffffffffu, s, max(warp - 1, 0));
  return y - x + (warp ? before : 0);
}

// The counts of the pages first + PER tid .. of a tile; pages past the pool read as used.
__device__ __forceinline__ void load_refs(const PagesDev &p, int first, int (&r)[PER]) {
  const int at = first + PER * threadIdx.x;
#pragma unroll
  for (int i = 0; i < PER; i += 4) {
    if (at + i + 4 <= p.n_pages) {
      const int4 v = *reinterpret_cast<const int4 *>(p.refs + at + i);
      r[i] = v.x, r[i + 1] = v.y, r[i + 2] = v.z, r[i + 3] = v.w;
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) r[i + j] = at + i + j < p.n_pages ? p.refs[at + i + j] : 1;
    }
  }
}

// Thread b is row b. Shared last pages are counted in a hash table of pages: how many rows of the call write in it, and the one with the most
// tokens in it (of several the first). That one may keep it, whichever of the others the pool has no page for: it writes behind their tokens.
constexpr int HASH = 2048, PAGE_TOKENS_MAX = 4096;
__global__ void __launch_bounds__(ONE) take_kernel(const PagesDev p, int batch, int32_t *table, int cols, const int32_t *lens,
                                                   const int32_t *n_new, int32_t *fits) {
  __shared__ int key[HASH], writers[HASH], keeper[HASH], warp_sum[32];
  pdl_enter();
  const int b = threadIdx.x;
  for (int i = b; i < HASH; i += ONE) key[i] = -1, writers[i] = 0, keeper[i] = INT_MAX;
  int len = 0, n = 0;
  if (b < batch) {
    n = max(n_new[b], 0);
    len = lens[b];
  }
  int r[PER];
  load_refs(p, 0, r);                                    // (needed later, does not depend on the rows)
  bool bad = false, on = n > 0;
  const int32_t *row = table + (long)b * cols;
  const int c0 = covering(len, p.page);                  // first column past the tokens so far
  const bool inside = on && len > 0 && len % p.page != 0;
  int end = 0;
  if (on) {
    bad = len < 0 || (long)len + n > (long)cols * p.page;
    if (!bad) end = covering(len + n, p.page);
  }
  int last = -1, held = 0;
  if (inside && !bad) {
    last = row[c0 - 1];
    bad = last < 0 || last >= p.n_pages;
    if (!bad) {
      held = p.refs[last];
      bad = held < 1;
    }
  }
  int need = 0;
  if (on && !bad)
    for (int c = c0; c < end; ++c) {
      const int x = row[c];
      bad |= x < -1 || x >= p.n_pages;
      need += x < 0;
    }
  if (bad) on = false, need = 0;
  __syncthreads();
  // who writes in a shared page
  const bool shared = on && inside && held > 1;
  const int place = (PAGE_TOKENS_MAX - (inside ? len % p.page : 0)) * PACE_KV_MAX_BATCH + b;      // the keeper's is the lowest
  int at = 0;
  if (shared) {
    at = (int)(((unsigned)last * 2654435761u) >> 21);
    while (true) {                                       // (twice as many places as rows)
      const int k = atomicCAS(&key[at], -1, last);
      if (k == -1 || k == last) break;
      at = (at + 1) & (HASH - 1);
    }
    atomicAdd(&writers[at], 1);
    atomicMin(&keeper[at], place);
  }
  __syncthreads();
  const bool copy = shared && !(writers[at] == held && keeper[at] == place);
  need += copy;
  int wanted;
  const int rank = block_prefix(need, warp_sum, wanted);
  // the lowest free pages, as many as there are up to those wanted
  int have = 0;
  for (int first = 0; first < p.n_pages && have < wanted; first += ONE * PER) {
    if (first) load_refs(p, first, r);
    int mine = 0, found;
#pragma unroll
    for (int i = 0; i < PER; ++i) mine += r[i] == 0;
    int to = have + block_prefix(mine, warp_sum, found);
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (r[i] == 0) {
        if (to < wanted) p.scratch[to] = first + PER * b + i;
        ++to;
      }
    have += found;
  }
  __syncthreads();
  const bool ok = !bad && rank + need <= have;
  const bool moves = ok && copy;
  int n_moves;
  const int m = block_prefix(moves, warp_sum, n_moves);
  if (b < batch) fits[b] = (ok || need == 0) && !bad;
  if (b == 0) *p.n_moves = n_moves;
  if (ok && need > 0) {
    int32_t *cells = table + (long)b * cols;
    int next = rank;
    if (copy) {
      const int page = p.scratch[next++];
      cells[c0 - 1] = page;
      p.refs[page] = 1;
      atomicAdd(p.refs + last, -1);
      p.src[m] = last;
      p.dst[m] = page;
    }
    for (int c = c0; c < end; ++c)
      if (cells[c] < 0) {
        const int page = p.scratch[next++];
        cells[c] = page;
        p.refs[page] = 1;
      }
  }
  if (bad) atomicOr(p.status, PACE_PAGES_BAD_CELL);
}

// Finds the moves; scratch[x] = where a used page x above the count of used pages goes (-1: it is free).
__global__ void __launch_bounds__(ONE) compact_kernel(const PagesDev p) {
  __shared__ int warp_sum[32];
  pdl_enter();
  const int tid = threadIdx.x;
  int r[PER], used = 0;
  for (int first = 0; first < p.n_pages; first += ONE * PER) {
    load_refs(p, first, r);
    const int at = first + PER * tid;
    int mine = 0, sum;
#pragma unroll
    for (int i = 0; i < PER; ++i) mine += at + i < p.n_pages && r[i] != 0;
    block_prefix(mine, warp_sum, sum);
    used += sum;
  }
  int holes = 0, movers = 0;
  for (int first = 0; first < p.n_pages; first += ONE * PER) {
    if (p.n_pages > ONE * PER) load_refs(p, first, r);
    const int at = first + PER * tid;
    int hole = 0, mover = 0, sum;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      hole += at + i < used && r[i] == 0;
      mover += at + i >= used && at + i < p.n_pages && r[i] != 0;
    }
    int h = holes + block_prefix(hole, warp_sum, sum);
    holes += sum;
    int m = movers + block_prefix(mover, warp_sum, sum);
    movers += sum;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      if (at + i < used) {
        if (r[i] == 0) p.dst[h++] = at + i;
      } else if (at + i < p.n_pages) {
        if (r[i] != 0) p.src[m++] = at + i;
        else p.scratch[at + i] = -1;
      }
    }
  }
  __syncthreads();
  for (int i = tid; i < movers; i += ONE) {              // (as many movers as holes)
    const int s = p.src[i], d = p.dst[i];
    p.scratch[s] = d;
    p.refs[d] = p.refs[s];
    p.refs[s] = 0;
  }
  if (tid == 0) {
    *p.n_moves = movers;
    p.status[2] = used;
  }
}

__global__ void __launch_bounds__(256) renumber_kernel(const PagesDev p, int32_t *table, long cells) {
  pdl_enter();
  const int used = p.status[2];
  int bad = 0;
  for (long i = (long)blockIdx.x * 256 + threadIdx.x; i < cells; i += (long)gridDim.x * 256) {
    const int x = table[i];
    if (x < -1 || x >= p.n_pages) {
      bad = PACE_PAGES_BAD_CELL;
    } else if (x >= used) {
      const int to = p.scratch[x];
      if (to >= 0) table[i] = to;
      else bad = PACE_PAGES_BAD_CELL;
    }
  }
  if (bad) atomicOr(p.status, bad);
}

// ---- copying ------------------------------------------------------------------------------------------------------------------
// A block copies a piece of a page a turn, eight 16-byte loads a thread under way, with the next piece's page numbers on their way
// beside them. Pieces are equal parts of a page.
constexpr int COPY_THREADS = 256, COPY_DEPTH = 8, COPY_ROW = COPY_THREADS * 16;

__host__ __device__ inline int copy_pieces(long page_bytes) { return (int)((page_bytes + COPY_ROW * COPY_DEPTH - 1) / (COPY_ROW * COPY_DEPTH)); }

__global__ void __launch_bounds__(COPY_THREADS) copy_kernel(char *pool, long page_bytes, int n_pages, int32_t *status,
                                                            const int32_t *src, const int32_t *dst, const int32_t *count, int max_n) {
  pdl_enter();
  const int pieces = copy_pieces(page_bytes);
  const long piece = (page_bytes + (long)pieces * COPY_ROW - 1) / ((long)pieces * COPY_ROW) * COPY_ROW;
  const int n = count ? min(max(*count, 0), max_n) : max_n;
  const long end = (long)n * pieces;
  int s = 0, d = 0;
  if (blockIdx.x < end) s = src[blockIdx.x / pieces], d = dst[blockIdx.x / pieces];
  for (long w = blockIdx.x; w < end; w += gridDim.x) {
    const long next = w + gridDim.x, first = (w % pieces) * piece;
    int s1 = 0, d1 = 0;
    if (next < end) s1 = src[next / pieces], d1 = dst[next / pieces];
    if (s < 0 || s >= n_pages || d < 0 || d >= n_pages) {
      if (first == 0 && threadIdx.x == 0) atomicOr(status, PACE_KV_BAD_PAGE);
    } else {
      const long last = min(first + piece, page_bytes);
      const char *from = pool + s * page_bytes;
      char *to = pool + d * page_bytes;
      uint4 v[COPY_DEPTH];
#pragma unroll
      for (int k = 0; k < COPY_DEPTH; ++k) {
        const long x = first + k * COPY_ROW + threadIdx.x * 16;
        if (x < last) v[k] = __ldcs(reinterpret_cast<const uint4 *>(from + x));
      }
#pragma unroll
      for (int k = 0; k < COPY_DEPTH; ++k) {
        const long x = first + k * COPY_ROW + threadIdx.x * 16;
        if (x < last) __stcs(reinterpret_cast<uint4 *>(to + x), v[k]);
      }
    }
    s = s1, d = d1;
  }
}

template <typename... P, typename... A>
cudaError_t launch(void (*kernel)(P...), long blocks, int threads, cudaStream_t s, A... args) {
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg = pdl_config(dim3((unsigned)blocks), dim3(threads), 0, s, attr);
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace pages
}  // namespace pace

cudaError_t pace_launch_pages_select(const PagesDev &p, int batch, int32_t *table, int cols, int32_t *lens, const int32_t *src,
                                     cudaStream_t s) {
  using namespace pace::pages;
  return launch(select_kernel, (cols + SEL_COLS - 1) / SEL_COLS, SEL_THREADS, s, p, batch, table, cols, lens, src);
}
cudaError_t pace_launch_pages_take(const PagesDev &p, int batch, int32_t *table, int cols, const int32_t *lens,
                                   const int32_t *n_new, int32_t *fits, cudaStream_t s) {
  using namespace pace::pages;
  return launch(take_kernel, 1, ONE, s, p, batch, table, cols, lens, n_new, fits);
}
cudaError_t pace_launch_pages_compact(const PagesDev &p, int batch, int32_t *table, int cols, cudaStream_t s) {
  using namespace pace::pages;
  cudaError_t e = launch(compact_kernel, 1, ONE, s, p);
  const long cells = (long)batch * cols;
  if (e == cudaSuccess && cells > 0)
    e = launch(renumber_kernel, cells < 256L * 2048 ? (cells + 255) / 256 : 2048, 256, s, p, table, cells);
  return e;
}
cudaError_t pace_launch_kv_copy_pages(char *pool, size_t page_bytes, int n_pages, int32_t *status, const int32_t *src,
                                      const int32_t *dst, const int32_t *n, int max_n, cudaStream_t s) {
  using namespace pace::pages;
  const long pieces = (long)max_n * copy_pieces((long)page_bytes);
  const long most = 6L * pace::device_sm_count();
  return launch(copy_kernel, pieces < most ? pieces : most, COPY_THREADS, s, pool, (long)page_bytes, n_pages, status, src, dst, n, max_n);
}
