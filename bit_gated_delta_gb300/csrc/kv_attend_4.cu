// Attention over a 4-bit cache: instantiations of kv_attend.cuh.
#include "kv_attend.cuh"

namespace pace {
namespace kv {
// `few`: no more items than SMs (see pace_launch_kv_attend).
cudaError_t attend_4(const AttendArgs &a, int rows, bool few, cudaStream_t s) {
  const bool f32 = a.c.io == PACE_IO_F32;
  if (a.c.d == 64) {
    if (f32) return few ? launch_attend<64, 4, 1, 3, 8, 2, 1>(a, s) : launch_attend<64, 4, 1, 3, 4, 4, 3>(a, s);
    if (rows <= 8) return few ? launch_attend<64, 4, 1, 1, 16, 2, 1>(a, s) : launch_attend<64, 4, 1, 1, 4, 4, 4>(a, s);
    if (rows <= 16) return few ? launch_attend<64, 4, 2, 1, 8, 2, 1>(a, s) : launch_attend<64, 4, 2, 1, 4, 4, 3>(a, s);
    return few ? launch_attend<64, 4, 4, 1, 8, 2, 1>(a, s) : launch_attend<64, 4, 4, 1, 4, 4, 2>(a, s);
  }
  if (a.c.d == 128) {
    if (f32) return few ? launch_attend<128, 4, 1, 3, 8, 2, 1>(a, s) : launch_attend<128, 4, 1, 3, 4, 3, 2>(a, s);
    if (rows <= 8) return few ? launch_attend<128, 4, 1, 1, 16, 2, 1>(a, s) : launch_attend<128, 4, 1, 1, 4, 2, 4>(a, s);
    return few ? launch_attend<128, 4, 2, 1, 8, 2, 1>(a, s) : launch_attend<128, 4, 2, 1, 4, 3, 2>(a, s);
  }
  if (f32) return few ? launch_attend<256, 4, 1, 3, 8, 2, 1>(a, s) : launch_attend<256, 4, 1, 3, 4, 2, 1>(a, s);
  return few ? launch_attend<256, 4, 1, 1, 8, 2, 1>(a, s) : launch_attend<256, 4, 1, 1, 4, 2, 2>(a, s);
}
}  // namespace kv
}  // namespace pace
