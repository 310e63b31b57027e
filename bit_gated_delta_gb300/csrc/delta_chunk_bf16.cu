#include "delta_chunk.cuh"

cudaError_t pace_launch_delta_chunk_bf16(const DeltaArgs &p, cudaStream_t s) {
  using namespace pace::delta;
  return p.d == 128 ? launch_chunk<128, false>(p, s) : launch_chunk<64, false>(p, s);
}
