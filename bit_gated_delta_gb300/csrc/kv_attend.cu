// Choice of the attention kernel, and its work area.
#include <math.h>

#include "kv_attend.cuh"

namespace pace {
namespace kv {
cudaError_t attend_4(const AttendArgs &a, int rows, cudaStream_t s);
cudaError_t attend_8(const AttendArgs &a, int rows, cudaStream_t s);
}  // namespace kv
}  // namespace pace

using namespace pace::kv;

void pace_kv_attend_work(const pace_kv_config &, size_t *count_bytes, size_t *part_bytes) {
  *count_bytes = MAX_BLOCKS * sizeof(int32_t);
  *part_bytes = (size_t)2 * MAX_BLOCKS * (MAX_ROWS_FLOATS + 64) * sizeof(float);
}

cudaError_t pace_launch_kv_attend(const KvDev &c, const KvTensor &q, const uint32_t *mask, float scale, const KvTensor &o,
                                  cudaStream_t s) {
  AttendArgs a{c, q, o, mask, scale * 1.44269504088896340736f, 0, 0};
  const int rows = c.n_tokens * c.group;
  return c.bits == 4 ? attend_4(a, rows, s) : attend_8(a, rows, s);
}
