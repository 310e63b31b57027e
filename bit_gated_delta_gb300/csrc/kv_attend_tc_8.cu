// Attention of many rows over a 8-bit cache: instantiations of kv_attend_tc.cuh.
#include "kv_attend_tc.cuh"

namespace pace {
namespace kv {
cudaError_t attend_tc_8(const AttendArgs &a, int rows, cudaStream_t s) {
  if (a.c.d == 256) return launch_attend_tc<256, 8, TC_ONE>(a, s);
  if (rows <= 128) return a.c.d == 64 ? launch_attend_tc<64, 8, TC_ALT>(a, s) : launch_attend_tc<128, 8, TC_ALT>(a, s);
  return a.c.d == 64 ? launch_attend_tc<64, 8, TC_SHARE>(a, s) : launch_attend_tc<128, 8, TC_SHARE>(a, s);
}
}  // namespace kv
}  // namespace pace
