// The paged decode kernel (decode_kernel.cuh) over a bf16 cache with changed
// scores: capped, biased by distance, limited to a window.

#include "decode_kernel.cuh"

namespace pa {

cudaError_t launch_decode_biased(const DecodeParams& p, int head_dim, int group, bool split,
                                 cudaStream_t stream) {
  if (head_dim == 128) return launch_decode_d<128, 0, true>(p, group, split, stream);
  if (head_dim == 64) return launch_decode_d<64, 0, true>(p, group, split, stream);
  return cudaErrorInvalidValue;
}

}  // namespace pa
