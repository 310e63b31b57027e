#include "delta_chunk.cuh"

cudaError_t pace_launch_delta_chunk_f32(const DeltaArgs &p, cudaStream_t s) {
  using namespace pace::delta;
  return p.d == 128 ? launch_chunk<128, true>(p, s) : launch_chunk<64, true>(p, s);
}
