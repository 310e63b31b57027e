// Attention of many rows over a 4-bit cache: instantiations of kv_attend_tc.cuh.
#include "kv_attend_tc.cuh"

namespace pace {
namespace kv {
cudaError_t attend_tc_4(const AttendArgs &a, int rows, cudaStream_t s) {
  if (a.c.d == 256) return launch_attend_tc<256, 4, TC_ONE>(a, s);
  if (rows <= 128) return a.c.d == 64 ? launch_attend_tc<64, 4, TC_ALT>(a, s) : launch_attend_tc<128, 4, TC_ALT>(a, s);
  return a.c.d == 64 ? launch_attend_tc<64, 4, TC_SHARE>(a, s) : launch_attend_tc<128, 4, TC_SHARE>(a, s);
}
}  // namespace kv
}  // namespace pace
