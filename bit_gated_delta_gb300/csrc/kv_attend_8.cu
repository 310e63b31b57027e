// Attention over a 8-bit cache: instantiations of kv_attend.cuh.
#include "kv_attend.cuh"

namespace pace {
namespace kv {
// `few`: no more items than SMs (see pace_launch_kv_attend).
cudaError_t attend_8(const AttendArgs &a, int rows, bool few, cudaStream_t s) {
  const bool f32 = a.c.io == PACE_IO_F32;
  if (a.c.d == 64) {
    if (f32) return few ? launch_attend<64, 8, 1, 3, 8, 2, 1>(a, s) : launch_attend<64, 8, 1, 3, 4, 3, 3>(a, s);
    if (rows <= 8) return few ? launch_attend<64, 8, 1, 1, 16, 2, 1>(a, s) : launch_attend<64, 8, 1, 1, 4, 3, 3>(a, s);
    if (rows <= 16) return few ? launch_attend<64, 8, 2, 1, 8, 2, 1>(a, s) : launch_attend<64, 8, 2, 1, 4, 3, 3>(a, s);
    return few ? launch_attend<64, 8, 4, 1, 8, 2, 1>(a, s) : launch_attend<64, 8, 4, 1, 4, 3, 2>(a, s);
  }
  if (a.c.d == 128) {
    if (f32) return few ? launch_attend<128, 8, 1, 3, 8, 2, 1>(a, s) : launch_attend<128, 8, 1, 3, 4, 2, 2>(a, s);
    if (rows <= 8) return few ? launch_attend<128, 8, 1, 1, 8, 2, 1>(a, s) : launch_attend<128, 8, 1, 1, 4, 2, 2>(a, s);
    return few ? launch_attend<128, 8, 2, 1, 8, 2, 1>(a, s) : launch_attend<128, 8, 2, 1, 4, 2, 2>(a, s);
  }
  if (f32) return launch_attend<256, 8, 1, 3, 4, 2, 1>(a, s);
  return launch_attend<256, 8, 1, 1, 4, 2, 1>(a, s);
}
}  // namespace kv
}  // namespace pace
