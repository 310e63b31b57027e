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
// Rows of one KV head from which the tensor-memory kernel takes over (bf16 I/O).
constexpr int TC_ROWS = 33;
constexpr int FEW_ITEMS = 64;
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
  AttendArgs a{c, q, o, mask, scale * 1.44269504088896340736f, 0, (0x80000000u + c.group - 1) / c.group};
  const int rows = c.n_tokens * c.group;
  if (use_tc(c.io, rows)) return c.bits == 4 ? attend_tc_4(a, rows, s) : attend_tc_8(a, rows, s);
  const bool few = (long)c.batch * c.Hkv <= FEW_ITEMS;
  return c.bits == 4 ? attend_4(a, rows, few, s) : attend_8(a, rows, few, s);
}
