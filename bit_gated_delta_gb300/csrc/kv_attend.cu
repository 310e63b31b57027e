// Choice of the attention kernel, and its work area.
#include <algorithm>

#include "kv_attend_tc.cuh"

namespace pace {
namespace kv {
cudaError_t attend_4(const AttendArgs &a, int rows, bool few, cudaStream_t s);
cudaError_t attend_8(const AttendArgs &a, int rows, bool few, cudaStream_t s);
cudaError_t attend_tc_4(const AttendArgs &a, int rows, cudaStream_t s);
cudaError_t attend_tc_8(const AttendArgs &a, int rows, cudaStream_t s);
}  // namespace kv
}  // namespace pace

using namespace pace::kv;

namespace {
// Rows of one KV head from which the tensor-memory kernel takes over (bf16 I/O). It works on 128 rows whatever their number, and the
// other on 8 (heads of 256), 16 (128) or 32 (64) at a time. One bound for all head sizes, since up to it codes enter the products exactly.
// 16 sequences of 8000 tokens, 8 KV heads, 4 bits, this kernel's and the other's us at 16, 32, 40 and 64 rows: heads of 64 93 and 44, 95 and
// 62, 95 and 93, 95 and 93; of 128 118 and 60, 120 and 97, 120 and 140, 120 and 179; of 256 148 and 126, 148 and 226, 149 and 279, 150 and
// 434 (for speed alone this kernel would take heads of 256 from 17 rows on). One sequence of 2000 tokens, heads of 128: 21 and 21, 21 and 15,
// 21 and 21, 29 and 21.
constexpr int TC_ROWS = 33;
// Rows of an item of the other kernel (fp32 I/O takes three products a tile, and eight rows).
int block_rows(const KvDev &c) { return c.io == PACE_IO_F32 ? 8 : 2048 / c.d; }
bool use_tc(int io, int rows) { return io == PACE_IO_BF16 && rows >= TC_ROWS; }
}  // namespace

void pace_kv_attend_work(const pace_kv_config &cfg, size_t *count_bytes, size_t *part_bytes) {
  *count_bytes = MAX_BLOCKS * sizeof(int32_t);
  size_t n = (size_t)2 * MAX_BLOCKS * (MAX_ROWS_FLOATS + 64);
  if (use_tc(cfg.io_dtype, cfg.max_new * (cfg.q_heads / cfg.kv_heads))) n = std::max(n, (size_t)2 * TC_BLOCKS * TC_PART_FLOATS + TC_BLOCKS * 4);
  *part_bytes = n * sizeof(float);
}

cudaError_t pace_launch_kv_attend(const KvDev &c, const KvTensor &q, const uint32_t *mask, float scale, const KvTensor &o,
                                  cudaStream_t s) {
  AttendArgs a{c, q, o, mask, scale * 1.44269504088896340736f, 0, 0, 0, (0x80000000u + c.group - 1) / c.group};
  const int rows = c.n_tokens * c.group;
  if (use_tc(c.io, rows)) return c.bits == 4 ? attend_tc_4(a, rows, s) : attend_tc_8(a, rows, s);
  // Blocks of 8 or 16 warps, one an SM, while there are no more items than SMs: an item then stays with one block, or few blocks join its
  // results. Heads of 128, 4-bit, one token: 144 items of 700 tokens 12 us (smaller blocks 13), of 3000 tokens 22 (28); 160 items 20 (14)
  // and 34 (29). Under 32 rows, two items a head: 64 heads of 3000 tokens 25 (29), 96 heads 40 (35).
  const long items = (long)c.batch * c.Hkv * ((rows + block_rows(c) - 1) / block_rows(c));
  const bool few = items <= pace::device_sm_count();
  return c.bits == 4 ? attend_4(a, rows, few, s) : attend_8(a, rows, few, s);
}
